"""The expert layer on the GPU against the 64-bit reference of moe_ref."""
import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_amd as bsg
import moe_ref
import seeded_inputs as si

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def weights_of(fmt, E, H, I, seed):
    rng = np.random.default_rng(seed)
    w = {"w13": [], "s13": [], "w2": [], "s2": []}
    for _ in range(E):
        for name, s, shape in (("w13", "s13", (2 * I, H)), ("w2", "s2", (H, I))):
            x = (rng.standard_normal(shape) * shape[1] ** -0.5).astype(np.float32)
            q = si.quantize_mxfp8(x) if fmt == "mxfp8" else si.quantize_nvfp4(x)
            w[name].append(q[0])
            w[s].append(q[1])
    return {k: np.stack(v) for k, v in w.items()}


def run_case(fmt, T, E, K, H, I, dtype, seed=0, alphas=True, gain=1.0, renormalize=True, x=None, router=None, max_tokens=None, w=None, graph=False):
    rng = np.random.default_rng(seed + 1)
    w = w or weights_of(fmt, E, H, I, seed)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(DT[dtype]) if x is None else x
    router = torch.from_numpy(rng.standard_normal((E, H)) * 2 * H ** -0.5).to(DT[dtype]) if router is None else router
    a13 = rng.uniform(0.5, 2.0, E).astype(np.float32) * (0.01 if fmt == "nvfp4" else 1.0) if alphas else None
    a2 = rng.uniform(0.5, 2.0, E).astype(np.float32) * np.float32(gain) if alphas else None
    want, ids, weights = moe_ref.moe(fmt, x.double().numpy(), router.double().numpy(), w["w13"], w["s13"], w["w2"], w["s2"], K, a13, a2, renormalize)
    label = f"{fmt} T={T} E={E} K={K} H={H} I={I} {dtype} renorm={renormalize}"
    print("[moe]", label, flush=True)
    wide = torch.zeros(T, H + 24, dtype=DT[dtype], device="cuda")
    wide[:, 8:H + 8] = x.cuda()
    room = torch.full((T, H + 16), 3.0, dtype=DT[dtype], device="cuda")
    out = room[:, :H]
    got_ids, got_w = torch.full((T, K), -1, dtype=torch.int32, device="cuda"), torch.zeros(T, K, device="cuda")
    args = (wide[:, 8:H + 8], router.cuda(), dev(w["w13"]), dev(w["s13"]), dev(w["w2"]), dev(w["s2"]), out)
    kw = dict(alpha13=None if a13 is None else dev(a13), alpha2=None if a2 is None else dev(a2), ids=got_ids, weights=got_w)
    with bsg.MoEPlan(fmt, E, K, H, I, max_tokens or T, dtype=dtype, renormalize=renormalize) as plan:
        plan.run(*args, **kw)
        torch.cuda.synchronize()
        first = out.clone()
        plan.run(*args, **kw)
        torch.cuda.synchronize()
        assert torch.equal(first, out), "not deterministic"
        if graph:
            side = torch.cuda.Stream()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                plan.run(*args, **kw)
            for i in range(4):
                wide[:, 8:H + 8] = torch.roll(x.cuda(), i, 1)
                plan.run(*args, **kw)
                torch.cuda.synchronize()
                eager = out.clone()
                room.zero_()
                g.replay()
                torch.cuda.synchronize()
                assert torch.equal(out, eager), i
            return
    assert (room[:, H:] == 3.0).all()
    assert np.array_equal(got_ids.cpu().numpy(), ids), label
    assert np.abs(got_w.double().cpu().numpy() - weights).max() <= 2e-6, label
    # decoded weights and 16-bit x are exact, SiLU(gate) up keeps 16 bits, sums are fp32: relative to the norm of a
    # row the result is off by 2^-17 times a small factor, then rounded once
    got = out.double().cpu().numpy()
    scale = np.sqrt((want ** 2).mean(1, keepdims=True))
    lim = UNIT[dtype] * np.abs(want) + 2.0 ** -13 * scale + (2.0 ** -24 if dtype == "f16" else 0)
    if dtype == "f16":  # beyond the type's range the rounded result is an infinity; at its edge either is right
        over, edge = np.abs(want) > 65520.0 + lim, np.abs(np.abs(want) - 65520.0) <= lim
        assert np.array_equal(got[over], np.copysign(np.inf, want[over])), label
        got, want, lim = got[~over & ~edge], want[~over & ~edge], lim[~over & ~edge]
    err = np.abs(got - want)
    assert bool((err <= lim).all()), (label, float((err / lim).max()))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T", [1, 2, 16, 17, 33, 64])
def test_tokens(fmt, dtype, T):
    run_case(fmt, T, 8, 2, 256, 128, dtype, seed=T)


@pytest.mark.parametrize("T", [1, 2, 16, 17, 33, 64])
def test_tokens_with_outputs_of_order_one(T):
    # NVFP4 codes of a Gaussian reach 2688 before the global scale
    run_case("nvfp4", T, 8, 2, 256, 128, "f16", seed=T, gain=1e-6)
    run_case("nvfp4", T, 6, 3, 128, 64, "f16", seed=T, gain=1e-5, renormalize=False)


@pytest.mark.parametrize("H,I", [(32, 32), (32, 96), (96, 32), (160, 64), (544, 224), (1056, 352), (64, 1056)])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp8"])
def test_odd_sizes(fmt, H, I):
    run_case(fmt, 3, 5, 2, H, I, "bf16", seed=H + I)


@pytest.mark.parametrize("E,K", [(1, 1), (2, 2), (3, 1), (17, 5), (64, 8), (100, 16), (16, 16), (257, 4), (512, 2)])
def test_experts(E, K):
    run_case("nvfp4", 5, E, K, 64, 32, "bf16", seed=E * 20 + K, max_tokens=64)


def test_without_alphas_and_without_renormalisation():
    run_case("mxfp8", 4, 6, 3, 128, 64, "bf16", seed=1, alphas=False, renormalize=False)
    run_case("nvfp4", 20, 6, 3, 128, 64, "f16", seed=2, renormalize=False)


def test_ties_go_to_the_lowest_expert():
    x = torch.ones(2, 64, dtype=torch.bfloat16)
    router = torch.zeros(9, 64, dtype=torch.bfloat16)
    run_case("nvfp4", 2, 9, 4, 64, 32, "bf16", seed=3, x=x, router=router)
    router[5] = 0.5
    router[7] = 0.5
    router[8] = -0.25
    run_case("nvfp4", 2, 9, 4, 64, 32, "bf16", seed=3, x=x, router=router)


def test_all_tokens_on_one_expert():
    router = torch.zeros(8, 64, dtype=torch.float16)
    router[3] = 1.0
    run_case("mxfp8", 64, 8, 1, 64, 64, "f16", seed=4, x=torch.rand(64, 64, generator=torch.Generator().manual_seed(1)).half() + 0.5, router=router)


def test_large_and_small_magnitudes():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(3, 128, generator=g)
    run_case("mxfp8", 3, 4, 2, 128, 64, "bf16", seed=5, x=(x * 1e15).bfloat16(), router=torch.randn(4, 128, generator=g).bfloat16() * 1e-15)
    run_case("nvfp4", 3, 4, 2, 128, 64, "bf16", seed=6, x=(x * 1e-15).bfloat16())
    run_case("nvfp4", 3, 4, 2, 128, 64, "f16", seed=7, x=(x * 1e-3).half())


def test_extreme_block_scales():
    # E8M0 from far below fp16's range to far above it, decoded exactly
    w = weights_of("mxfp8", 2, 64, 64, 8)
    w["s13"][:, :64] -= 100   # gate, and up, rows
    w["s2"] += 100
    run_case("mxfp8", 3, 2, 2, 64, 64, "bf16", seed=8, w=w, alphas=False)


def test_a_nan_token_stays_alone():
    w = weights_of("nvfp4", 4, 64, 32, 9)
    g = torch.Generator().manual_seed(3)
    x, router = torch.randn(3, 64, generator=g).bfloat16(), torch.randn(4, 64, generator=g).bfloat16()
    outs = []
    for bad in (False, True):
        y = x.clone()
        if bad:
            y[1, 5] = float("nan")
        out = torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda")
        ids = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
        with bsg.MoEPlan("nvfp4", 4, 2, 64, 32, 3) as plan:
            plan.run(y.cuda(), router.cuda(), dev(w["w13"]), dev(w["s13"]), dev(w["w2"]), dev(w["s2"]), out, ids=ids)
            torch.cuda.synchronize()
        assert ((ids >= 0) & (ids < 4)).all()
        outs.append(out.float().cpu())
    assert torch.isnan(outs[1][1]).all()
    assert torch.equal(outs[0][[0, 2]], outs[1][[0, 2]])


def test_in_a_graph():
    run_case("nvfp4", 5, 16, 4, 256, 128, "bf16", seed=10, graph=True)
    run_case("mxfp8", 33, 16, 2, 256, 128, "f16", seed=11, graph=True)


@pytest.mark.parametrize("change,status", [
    (dict(top_k=9), "BSG_ERR_SHAPE"), (dict(hidden=48), "BSG_ERR_SHAPE"), (dict(inter=0), "BSG_ERR_SHAPE"), (dict(experts=0), "BSG_ERR_SHAPE"),
    (dict(max_tokens=65), "BSG_ERR_UNSUPPORTED"), (dict(max_tokens=0), "BSG_ERR_SHAPE"), (dict(experts=513), "BSG_ERR_UNSUPPORTED"),
    (dict(experts=32, top_k=17), "BSG_ERR_UNSUPPORTED"), (dict(hidden=65568), "BSG_ERR_UNSUPPORTED"),
])
def test_plan_refusals(change, status):
    with pytest.raises(bsg.BsgError) as e:
        bsg.MoEPlan(**(dict(fmt="nvfp4", experts=8, top_k=2, hidden=64, inter=64, max_tokens=4) | change))
    assert e.value.status_name == status


def test_call_refusals():
    w = {k: dev(v) for k, v in weights_of("nvfp4", 2, 64, 32, 0).items()}
    x, router = torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    with bsg.MoEPlan("nvfp4", 2, 1, 64, 32, 2) as plan:
        a = (router, w["w13"], w["s13"], w["w2"], w["s2"])
        with pytest.raises(bsg.BsgError) as e:
            plan.run(x, *a, x.clone())
        assert e.value.status_name == "BSG_ERR_SHAPE"
        wide = torch.zeros(2, 68, dtype=torch.bfloat16, device="cuda")
        with pytest.raises(bsg.BsgError) as e:
            plan.run(wide[:, :64], *a, x[:2].clone())
        assert e.value.status_name == "BSG_ERR_ALIGN"
        with pytest.raises(bsg.BsgError) as e:
            plan.run(torch.zeros(2, 72, dtype=torch.bfloat16, device="cuda")[:, 4:68], *a, x[:2].clone())
        assert e.value.status_name == "BSG_ERR_ALIGN"
        for bad in (lambda: plan.run(x[:2, :32], *a, x[:2]), lambda: plan.run(x[:2], router[:1], *a[1:], x[:2]),
                    lambda: plan.run(x[:2], router, w["w13"][:1], *a[2:], x[:2])):
            with pytest.raises(ValueError):
                bad()
        plan.run(x[:0], *a, x[:0])
        plan.run(x[:2], *a, x[:2].clone())
        torch.cuda.synchronize()
