"""The expert layer at the ends of its arguments' ranges, against the 64-bit reference of moe_ref."""
import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_amd as bsg
import moe_ref
from test_gpu_moe import UNIT, dev, run_case, weights_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 5])
def test_tokens_up_to_the_largest_bf16(T):
    # weights of 2^-9 times E2M1 and alphas near 2^-120 keep every result of the definition inside fp32
    E, K, H, I = 4, 2, 128, 64
    rng = np.random.default_rng(T)
    w13, w2 = rng.integers(0, 256, (E, 2 * I, H // 2), np.uint8), rng.integers(0, 256, (E, H, I // 2), np.uint8)
    s13, s2 = np.full((E, 2 * I, H // 16), 1, np.uint8), np.full((E, H, I // 16), 40, np.uint8)
    x = torch.from_numpy(rng.standard_normal((T, H)) * 1e38).clamp(-3.38e38, 3.38e38).bfloat16()
    x[0, 7] = torch.finfo(torch.bfloat16).max
    router = torch.from_numpy(rng.integers(1, 4, (E, H)) * rng.choice([-1.0, 1.0], (E, H)) * 2.0 ** -126).bfloat16()
    a13 = (rng.uniform(0.5, 2.0, E) * 2.0 ** -122).astype(np.float32)
    want, ids, _ = moe_ref.moe("nvfp4", x.double().numpy(), router.double().numpy(), w13, s13, w2, s2, K, a13)
    assert np.isfinite(want).all()
    out, got_ids = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, K, dtype=torch.int32, device="cuda")
    print(f"[moe] largest bf16 T={T}", flush=True)
    with bsg.MoEPlan("nvfp4", E, K, H, I, T) as plan:
        plan.run(x.cuda(), router.cuda(), dev(w13), dev(s13), dev(w2), dev(s2), out, alpha13=dev(a13), ids=got_ids)
        torch.cuda.synchronize()
    assert np.array_equal(got_ids.cpu().numpy(), ids)
    got = out.double().cpu().numpy()
    lim = UNIT["bf16"] * np.abs(want) + 2.0 ** -13 * np.sqrt((want ** 2).mean(1, keepdims=True))
    assert (np.abs(got - want) <= lim).all()


@pytest.mark.parametrize("fmt,dtype", [("nvfp4", "bf16"), ("nvfp4", "f16"), ("mxfp8", "bf16"), ("mxfp8", "f16")])
@pytest.mark.parametrize("H,I", [(4128, 64), (64, 4128), (8224, 32), (96, 8224), (4096, 4224)])
@pytest.mark.parametrize("T", [1, 17])
def test_rows_longer_than_a_chunk(fmt, dtype, H, I, T):
    # scales are staged 4096 at a time, tokens prepared 8192 at a time; the rest of the last chunk is no whole slab
    run_case(fmt, T, 3, 2, H, I, dtype, seed=H + I)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp8"])
def test_a_row_of_65536(fmt):
    run_case(fmt, 3, 2, 1, 65536, 32, "bf16", seed=5)
    run_case(fmt, 3, 2, 1, 32, 65536, "bf16", seed=6)


@pytest.mark.parametrize("T", [1, 4])
def test_nan_and_extreme_scale_codes_of_weights(T):
    # E8M0 0 is 2^-127 and 255 NaN; E4M3 0x7F is NaN, as a weight and as an NVFP4 scale
    for fmt, top, least in (("mxfp8", 255, 0), ("nvfp4", 0x7F, 1)):
        E, H, I = 2, 64, 64
        w = {k: v.copy() for k, v in weights_of(fmt, E, H, I, 60).items()}
        w["s2"][1, 5, 1] = top             # output dim 5 of expert 1
        w["s13"][0, 3, 0] = least          # one gate row of expert 0: zero beside the others, or nearly
        if fmt == "mxfp8":
            w["w2"][1, 9, 40] = 0x7F
        x = torch.randn(T, H, generator=torch.Generator().manual_seed(61)).bfloat16()
        router = torch.zeros(E, H, dtype=torch.bfloat16)
        for e in range(E):  # each expert alone, by the sign of its logits
            r = router.clone()
            ones = x.clone()
            ones[:, 0] = 1.0
            r[e, 0] = 8.0
            want, ids, _ = moe_ref.moe(fmt, ones.double().numpy(), r.double().numpy(), w["w13"], w["s13"], w["w2"], w["s2"], 1)
            assert (ids == e).all()
            out = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
            with bsg.MoEPlan(fmt, E, 1, H, I, T) as plan:
                plan.run(ones.cuda(), r.cuda(), dev(w["w13"]), dev(w["s13"]), dev(w["w2"]), dev(w["s2"]), out)
                torch.cuda.synchronize()
            got = out.double().cpu().numpy()
            bad = np.isnan(want)
            assert np.array_equal(np.isnan(got), bad), (fmt, e)
            assert bad[:, 5].all() == (e == 1) and bad.any() == (e == 1)
            scale = np.sqrt(np.nanmean(want ** 2, 1, keepdims=True))
            assert (np.abs(got - want)[~bad] <= (UNIT["bf16"] * np.abs(want) + 2.0 ** -13 * scale)[~bad]).all(), (fmt, e)
