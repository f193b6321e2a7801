"""Every kernel of the E4M3 products on calls that reach all parts of its loops (f8_cases), on numbers of which no sum is
rounded: codes of +-1 .. 1.875, and products of scales that are powers of two from 2^-2 to 2^2.  All sums then have steps of 2^-8,
and random signs keep them below 2^15: 23 bits.  So outputs of products are the exact sums rounded once, whatever the kernel,
the order and the parts."""
import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_amd as bsg
import f8_cases
import f8_ref as ref
from test_gpu_f8 import DT, activations, check, dev, ffn_weights, operands

pytestmark = pytest.mark.gpu

ONE = 7 << 3


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def narrow(shape, g):
    """Codes of +-1 .. 1.875."""
    r = torch.randint(0, 16, shape, dtype=torch.uint8, device="cuda", generator=g)
    return (r & 8) << 4 | ONE | r & 7


def powers(shape, g, middle=0):
    return torch.ldexp(torch.ones(shape, device="cuda"), torch.randint(middle - 1, middle + 2, shape, device="cuda", generator=g))


def exact(x, sx, w, sw):
    """The sums in 64 bits: x codes [t][k], sx [blocks][t or more], w codes [n][k], sw [blocks of n][blocks of k]."""
    table = torch.from_numpy(ref.values(np.arange(256))).cuda()
    out = torch.zeros(len(x), len(w), dtype=torch.float64, device="cuda")
    for a in range(0, x.shape[1], 8192):
        b = slice(a // 128, a // 128 + 64)
        xs = sx[b, :len(x)].t().double().repeat_interleave(128, 1)[:, :x[:, a:a + 8192].shape[1]]
        ws = sw[:, b].double().repeat_interleave(128, 0)[:len(w)].repeat_interleave(128, 1)[:, :xs.shape[1]]
        out += (table[x[:, a:a + 8192].int()] * xs) @ (table[w[:, a:a + 8192].int()] * ws).t()
    assert out.abs().max() < 2.0 ** 15  # with steps of 2^-8: 23 bits
    return out


def devices_cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("case", f8_cases.PRODUCTS + f8_cases.FEW_PRODUCTS, ids=str)
def test_products_are_exact_sums(case):
    check_product(case, False)


@pytest.mark.parametrize("case", f8_cases.EXACT_PRODUCTS + f8_cases.FEW_PRODUCTS, ids=str)
def test_exact_products_are_exact_sums(case):
    check_product(case, True)


def check_product(case, of_exact_plan):
    t, n, k = case[:3]
    dtype = "f16" if t % 2 == 0 else "bf16"
    print("[f8] exact product", *case, dtype, flush=True)
    assert devices_cus() == f8_cases.CUS, "the cases are for such a device"
    g = generator(t + n + k)
    x, sx, w, sw = narrow((t, k), g), powers((ref.blocks(k), (t + 3) // 4 * 4), g), narrow((n, k), g), powers((ref.blocks(n), ref.blocks(k)), g)
    sx[:, t:] = float("nan")
    want = exact(x, sx, w, sw).float().to(DT[dtype])
    out = torch.full((t + 2, n), 7.0, dtype=DT[dtype], device="cuda")
    with bsg.F8Plan(n, k, t, dtype=dtype, exact=of_exact_plan) as plan:
        for _ in range(2):
            out[:t] = -7.0
            plan.run(x, sx, w, sw, out[:t])
            torch.cuda.synchronize()
            wrong = (out[:t] != want).nonzero()
            assert len(wrong) == 0, (len(wrong), wrong[:5].tolist())
    assert (out[t:] == 7).all()


@pytest.mark.parametrize("case", f8_cases.GATED + f8_cases.FEW_GATED, ids=str)
def test_gate_and_up_are_exact_sums(case):
    check_gated(case, False)


@pytest.mark.parametrize("case", f8_cases.EXACT_GATED, ids=str)
def test_exact_gate_and_up_are_exact_sums(case):
    check_gated(case, True)


def check_gated(case, of_exact_plan):
    """The second product picks inner values, one for each output: out[j] is the quantised value at pick[j]."""
    t, inter, hidden = case[:3]
    dtype = "f16" if t % 2 == 0 else "bf16"
    print("[f8] exact gate and up", *case, dtype, flush=True)
    assert devices_cus() == f8_cases.CUS, "the cases are for such a device"
    g = generator(t + inter + hidden)
    bi, bh = ref.blocks(inter), ref.blocks(hidden)
    x, w13 = narrow((t, hidden), g), narrow((2 * inter, hidden), g)
    s13 = powers((2, bi, bh), g, -1 - round(np.log2(hidden) / 2))  # sums of about 1
    pick = torch.randperm(inter, device="cuda", generator=g).repeat(-(-hidden // inter))[:hidden]
    pick[:2] = torch.tensor([0, inter - 1], device="cuda")
    w2 = torch.zeros((hidden, inter), dtype=torch.uint8, device="cuda")
    w2[torch.arange(hidden, device="cuda"), pick] = ONE
    s2 = torch.ones((bh, bi), device="cuda")
    values = torch.from_numpy(ref.values(np.arange(256))).cuda()[x.int()]
    out = torch.full((t + 1, hidden), 7.0, dtype=DT[dtype], device="cuda")
    with bsg.F8FFNPlan(hidden, inter, t, dtype=dtype, exact=of_exact_plan) as plan:
        plan.run(values.to(DT[dtype]), w13, s13, w2, s2, out[:t])
        torch.cuda.synchronize()
        first = out.clone()
        plan.run(values.to(DT[dtype]), w13, s13, w2, s2, out[:t])
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), first.view(torch.int16)), "not deterministic"
    assert (out[t:] == 7).all()
    # tokens at the tiles' edges and every 13th (the reference's bounds take a while)
    rows = np.arange(t) if t <= 128 else np.unique(np.concatenate([np.arange(0, t, 13), np.arange(255, t, 256), np.arange(256, t, 256), [t - 1]]))
    ones = torch.ones((bh, len(rows)), device="cuda")  # (x itself: its scales are powers of two, its codes narrow)
    gate, up = (exact(x[torch.from_numpy(rows).cuda()], ones, w, s).cpu().numpy() for w, s in zip(w13.view(2, inter, hidden), s13))
    h = ref.silu(gate) * up
    # the exponential, the sum and the reciprocal of SiLU cost 8 roundings and the exponent's own, |gate| of them, the products two
    d = np.abs(h) * (10 + np.abs(gate)) * ref.U32 + 1e-38
    held, off = ref.row_values(*ref.quantize(h)), ref._changes(h, d)
    at = pick.cpu().numpy()
    check(out[:t].double().cpu().numpy()[rows], held[:, at], off[:, at], dtype, case)
    assert np.median(off) == 0  # nearly every inner value has one possible code


@pytest.mark.parametrize("dtype,bias", [("bf16", False), ("f16", True)])
@pytest.mark.parametrize("t,n,k", [(9, 144, 400), (17, 144, 1040), (32, 272, 16), (33, 144, 2064), (65, 400, 1040), (130, 528, 2064),
                                   (700, 272, 400), (1003, 2064, 528)])
def test_exact_products_of_any_codes(t, n, k, dtype, bias):
    """No more than fp32's roundings off, for codes of which the other kernels drop bits."""
    print("[f8] exact plan", t, n, k, dtype, flush=True)
    x, sx, w, sw, b = operands(t, n, k, t + n)
    want, s = ref.product(ref.row_values(x, sx.astype(np.float64)), ref.weight_values(w, sw), b if bias else None)
    with bsg.F8Plan(n, k, t, dtype=dtype, bias=bias, exact=True) as plan:
        out = torch.full((t + 1, n), 7.0, dtype=DT[dtype], device="cuda")
        plan.run(dev(x), dev(sx), dev(w), dev(sw), out[:t], bias=dev(b) if bias else None)
        torch.cuda.synchronize()
    assert (out[t:] == 7).all()
    check(out[:t].double().cpu().numpy(), want, ref.sum_bound(k, True) * s, dtype, (t, n, k))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("t,hidden,inter", [(5, 144, 272), (33, 272, 400), (65, 400, 528), (300, 528, 272), (1100, 272, 1040)])
def test_exact_feed_forward_of_any_numbers(monkeypatch, t, hidden, inter, dtype):
    monkeypatch.setattr(ref, "FEW", 1 << 30)  # (the reference's bounds for exact products)
    monkeypatch.setattr(ref, "WIDE", 1 << 30)
    print("[f8] exact feed-forward", t, hidden, inter, dtype, flush=True)
    held, doubles = ffn_weights(hidden, inter, t)
    x = activations(t, hidden, dtype, t + hidden)
    out = torch.full((t + 1, hidden), 7.0, dtype=DT[dtype], device="cuda")
    with bsg.F8FFNPlan(hidden, inter, t, dtype=dtype, exact=True) as plan:
        plan.run(x.cuda(), *(dev(a) for a in held), out[:t])
        torch.cuda.synchronize()
    assert (out[t:] == 7).all()
    check(out[:t].double().cpu().numpy(), *ref.ffn(x.double().numpy(), *doubles), dtype, (t, hidden, inter))


def test_exact_plans_refuse_and_replay_as_others():
    t, n, k = 100, 144, 272
    x, sx, w, sw, _ = (dev(a) for a in operands(t, n, k, 1))
    out, side = torch.empty(t, n, dtype=torch.bfloat16, device="cuda"), torch.cuda.Stream()
    with bsg.F8Plan(n, k, t, exact=True) as plan:
        with pytest.raises(ValueError):
            plan.run(x[:, :128], sx, w, sw, out)
        plan.run(x, sx, w, sw, out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            plan.run(x, sx, w, sw, out)
        for i in range(3):
            x.copy_(dev(operands(t, n, k, 10 + i)[0]))
            graph.replay()
            torch.cuda.synchronize()
            got = out.clone()
            plan.run(x, sx, w, sw, out)
            torch.cuda.synchronize()
            assert torch.equal(got.view(torch.int16), out.view(torch.int16))


def test_exact_products_of_more_tiles_than_a_grid_has():
    """Outputs of 137 GB: 4098 x 1024 tiles of 512 threads.  Tokens around the end of a range, and every 4099th, against the exact
    sums."""
    t, n, k, g = (1 << 19) + 200, 1 << 17, 16, generator(1)
    torch.cuda.empty_cache()
    print("[f8] exact product of", t, n, k, flush=True)
    x, sx, w, sw = narrow((t, k), g), powers((1, t), g), narrow((n, k), g), powers((ref.blocks(n), 1), g)
    out = torch.empty(t, n, dtype=torch.bfloat16, device="cuda")
    rows = torch.cat([torch.arange(0, t, 4099), torch.arange((1 << 19) - 130, t)]).unique().cuda()
    out[rows] = -7.0
    with bsg.F8Plan(n, k, t, exact=True) as plan:
        plan.run(x, sx, w, sw, out)
        torch.cuda.synchronize()
    for some in rows.split(128):
        assert torch.equal(out[some], exact(x[some], sx[:, some], w, sw).bfloat16())
    del out
    torch.cuda.empty_cache()


def test_exact_gate_and_up_of_more_tiles_than_a_grid_has():
    """Inner codes of 69 GB: 16384 x 512 tiles of 512 threads, two ranges of tokens, against calls with some of the tokens."""
    t, hidden, inter, g = 1 << 20, 16, 1 << 16, generator(2)
    torch.cuda.empty_cache()
    print("[f8] exact feed-forward of", t, hidden, inter, flush=True)
    x = torch.randn(t, hidden, device="cuda", generator=g).bfloat16()
    w13, s13 = narrow((2 * inter, hidden), g), powers((2, inter // 128, 1), g, -2)
    w2 = torch.zeros((hidden, inter), dtype=torch.uint8, device="cuda")
    w2[torch.arange(hidden, device="cuda"), torch.randperm(inter, device="cuda", generator=g)[:hidden]] = ONE  # (picks inner values)
    held = w13, s13, w2, torch.ones((1, inter // 128), device="cuda")
    out = torch.full((t, hidden), 7.0, dtype=torch.bfloat16, device="cuda")
    with bsg.F8FFNPlan(hidden, inter, t, exact=True) as plan:
        plan.run(x, *held, out)
        torch.cuda.synchronize()
    with bsg.F8FFNPlan(hidden, inter, 4096, exact=True) as plan:
        for a in [*range(0, t, 1 << 17), (t >> 1) - 2048, t - 4096]:
            some = torch.empty(4096, hidden, dtype=torch.bfloat16, device="cuda")
            plan.run(x[a:a + 4096], *held, some)
            torch.cuda.synchronize()
            assert torch.equal(out[a:a + 4096].view(torch.int16), some.view(torch.int16)), a
    torch.cuda.empty_cache()


def test_workspaces_are_those_of_the_plans_sizes():
    def bytes_of(plan):
        with plan:
            return plan.workspace_bytes()

    assert bytes_of(bsg.F8Plan(4096, 896, 8192)) == 0             # seven blocks of K are not split
    assert bytes_of(bsg.F8Plan(262144, 8192, 8192)) == 0          # nor is K where tiles alone fill the device
    assert 0 < bytes_of(bsg.F8Plan(16, 1024, 64)) <= 2 * 128 * 128 * 4 + 64
    assert bytes_of(bsg.F8Plan(8192, 8192, 8192)) <= f8_cases.CUS * (256 * 128 * 4 + 12)
    small = bytes_of(bsg.F8FFNPlan(128, 128, 64))                 # codes, scales, inner values of 16 tokens
    assert small <= 64 * (128 + 128) + 2 * 4 * 64 + 16 * 128 * 4 + 7 * 256
