"""E4M3 products with a scale for each block of 128 on the GPU against the 64-bit reference of f8_ref: quantising, products
and the gated feed-forward block over token counts, odd sizes, strides, streams, graphs and special values."""
import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_amd as bsg
import f8_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def activations(rows, cols, dtype, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp(0.7 * rng.standard_normal(cols))
    return torch.from_numpy(x).to(DT[dtype])


def codes_of(rng, shape):
    """Codes of Gaussians of which the largest of many is about 448."""
    x = rng.standard_normal(shape) * 100
    return ref.nearest(np.minimum(np.abs(x), 448.0), ref.E4M3).astype(np.uint8) | np.where(x < 0, 128, 0).astype(np.uint8)


def narrow_codes(rng, shape):
    """Codes of +-1 .. 1.875: products of which no matrix instruction drops a bit."""
    return (rng.integers(0, 2, shape) << 7 | 7 << 3 | rng.integers(0, 8, shape)).astype(np.uint8)


def weights(n, k, seed, gain=1.0, make=codes_of):
    rng = np.random.default_rng(seed)
    s = np.exp(0.5 * rng.standard_normal((ref.blocks(n), ref.blocks(k)))) * gain / 100
    return make(rng, (n, k)), s.astype(np.float32)


def check(got, want, off, dtype, label):
    """got: the rounding of a value that is at most `off` from want."""
    bad = np.isnan(want)
    assert np.array_equal(np.isnan(got), bad), label
    lim = off + ref.HALF[dtype] * (np.abs(want) + off) + ref.TINY[dtype]
    err = np.abs(got - want) - lim
    assert (err[~bad] <= 0).all(), (label, float(err[~bad].max()), float((np.abs(got - want) / lim)[~bad].max()))


# ------------------------------------------------------------------------------------------------ quantize
def run_quantize(x):
    rows, cols = x.shape
    codes = torch.full((rows, cols), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full(bsg.f8_scales_shape(rows, cols), 7.0, device="cuda")
    bsg.f8_quantize(x.cuda(), codes, scales)
    torch.cuda.synchronize()
    return codes.cpu().numpy(), scales.cpu().numpy()


def check_quantize(x):
    codes, scales = run_quantize(x)
    want, ws = ref.quantize(x.double().numpy())
    rows = len(x)
    fine = (want & 127) != 127
    assert np.array_equal((codes & 127) == 127, ~fine)
    assert np.array_equal(codes[fine], want[fine])
    ok = np.isfinite(ws) & np.repeat(fine[:, ::128].T, 1, 0)
    assert np.array_equal(scales[:, :rows][ok], ws[ok])
    assert (scales[:, rows:] == 7.0).all()  # entries past the rows stay


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 112), (16, 128), (17, 144), (65, 1040), (5, 4096), (130, 1024), (1, 16 * 129)])
def test_quantize(rows, cols, dtype):
    check_quantize(activations(rows, cols, dtype, rows + cols))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quantize_every_value(dtype):
    # every finite value beside every largest magnitude of its binade and the next ones: all roundings and ties
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    v = bits.view(DT[dtype])
    v = v[torch.isfinite(v)]
    v = v[: len(v) // 128 * 128].view(-1, 128)
    check_quantize(v)
    order = v.float().abs().flatten().argsort()
    check_quantize(v.flatten()[order].view(-1, 128))
    check_quantize(v.flatten()[order].view(128, -1).t().contiguous())  # far apart in one block


def test_quantize_special_blocks():
    x = torch.zeros(6, 384, dtype=torch.bfloat16)
    x[1, 5], x[1, 200] = float("inf"), 3.0
    x[2, 130], x[2, 0] = float("nan"), -1.0
    x[3] = -0.0
    x[4, :128] = 448.0
    x[4, 128:256] = 450.0          # just beyond: the next scale
    x[5, 0], x[5, 1] = 2.0 ** -133, 3e38
    codes, scales = run_quantize(x)
    assert (codes[1, :128] & 127 == 127).all() and (codes[2, 128:256] & 127 == 127).all()
    assert scales[1, 1] == 2.0 ** -7 and codes[1, 200] == 0x7C and (codes[1, 256:] == 0).all()  # 3 = 384 2^-7
    assert (codes[3] == 0x80).all() and (scales[:, 3] == 2.0 ** -126).all()
    assert scales[0, 4] == 1 and (codes[4, :128] == 0x7E).all() and scales[1, 4] == 2
    check_quantize(x)


def test_quantize_strides_and_stream():
    wide = activations(20, 400, "f16", 1).cuda()
    x = wide[1:18:2, 8:280]
    room = torch.full((9, 320), 0x33, dtype=torch.uint8, device="cuda")
    scales = torch.full((4, 16), 7.0, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    bsg.f8_quantize(x, room[:, 16:288].view(torch.float8_e4m3fn), scales[:3, :12], stream=side)
    torch.cuda.synchronize()
    want, ws = ref.quantize(x.double().cpu().numpy())
    got = room.cpu().numpy()
    assert np.array_equal(got[:, 16:288], want) and (got[:, :16] == 0x33).all() and (got[:, 288:] == 0x33).all()
    s = scales.cpu().numpy()
    assert np.array_equal(s[:3, :9], ws) and (s[:, 9:] == 7).all() and (s[3] == 7).all()


def test_quantize_nothing():
    z = torch.zeros(0, 32, dtype=torch.bfloat16, device="cuda")
    bsg.f8_quantize(z, torch.zeros(0, 32, dtype=torch.uint8, device="cuda"), torch.zeros(1, 0, device="cuda"))


# ------------------------------------------------------------------------------------------------ product
def operands(t, n, k, seed, make=codes_of, w_make=None):
    rng = np.random.default_rng(seed)
    x = make(rng, (t, k))
    sx = np.full((ref.blocks(k), (t + 3) // 4 * 4), np.nan, np.float32)  # entries past the tokens are never used
    sx[:, :t] = np.exp(rng.standard_normal((ref.blocks(k), t))) / 100
    w, sw = weights(n, k, seed + 1, make=w_make or make)
    return x, sx, w, sw, rng.standard_normal(n).astype(np.float32)


def run_product(x, sx, w, sw, bias, dtype, stream=None):
    t, n = len(x), len(w)
    with bsg.F8Plan(n, x.shape[1], t, dtype=dtype, bias=bias is not None) as plan:
        out = torch.full((t + 2, n), 7.0, dtype=DT[dtype], device="cuda")
        args = dev(x), dev(sx), dev(w), dev(sw), out[:t]
        plan.run(*args, bias=None if bias is None else dev(bias), stream=stream)
        torch.cuda.synchronize()
        assert (out[t:] == 7).all()  # rows behind the last token stay
        first = out.clone()
        plan.run(*args, bias=None if bias is None else dev(bias), stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), first.view(torch.int16)), "not deterministic"
    return out[:t].double().cpu().numpy()


def product_case(t, n, k, dtype, with_bias, seed, make=codes_of, exact_range=False):
    label = f"t={t} n={n} k={k} {dtype} bias={with_bias}"
    print("[f8]", label, flush=True)
    x, sx, w, sw, bias = operands(t, n, k, seed, make)
    bias = bias if with_bias else None
    want, s = ref.product(ref.row_values(x, sx.astype(np.float64)), ref.weight_values(w, sw), bias)
    got = run_product(x, sx, w, sw, bias, dtype)
    check(got, want, ref.sum_bound(k, t <= ref.FEW, exact_range) * s, dtype, label)


@pytest.mark.parametrize("dtype,bias", [("bf16", False), ("f16", True)])
@pytest.mark.parametrize("n,k", [(16, 16), (48, 128), (144, 144), (272, 1040), (128, 2048), (400, 4112)])
@pytest.mark.parametrize("t", [1, 2, 15, 16, 17, 32, 33, 48, 49, 64, 65])
def test_products_of_few_tokens(t, n, k, dtype, bias):
    product_case(t, n, k, dtype, bias, t + n + k)


@pytest.mark.parametrize("dtype,bias", [("bf16", True), ("f16", False)])
@pytest.mark.parametrize("t,n,k", [(127, 128, 128), (128, 16, 272), (129, 144, 400), (257, 528, 1040), (700, 272, 144), (100, 1040, 2064)])
def test_products_of_many_tokens(t, n, k, dtype, bias):
    product_case(t, n, k, dtype, bias, t + n + k)
    product_case(t, n, k, dtype, bias, t, narrow_codes, True)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("t,n,k", [(4100, 4112, 272), (4096, 4096, 1168), (2049, 8208, 16)])
def test_products_of_many_large_tiles(t, n, k, dtype):
    product_case(t, n, k, dtype, dtype == "f16", t + k, narrow_codes, True)


def test_every_code_is_multiplied_by_its_value():
    # row i of the weights picks element i: every code of x beside 1, and every code of w beside 1
    one = 7 << 3
    for t in (2, 70):
        eye = np.where(np.eye(256, dtype=bool), one, 0).astype(np.uint8)
        x = np.tile(np.arange(256, dtype=np.uint8), (t, 1))
        x[:, [0x7F, 0xFF]] = 0
        ones = np.ones((2, (t + 3) // 4 * 4), np.float32)
        got = run_product(x, ones, eye, np.ones((2, 2), np.float32), None, "f16")
        assert np.array_equal(got, ref.values(x))
        w = np.zeros((256, 256), np.uint8)
        w[np.arange(256), np.arange(256)] = x[0]
        got = run_product(np.full((t, 256), one, np.uint8), ones, w, np.ones((2, 2), np.float32), None, "f16")
        assert np.array_equal(got, ref.values(x))


@pytest.mark.parametrize("t", [5, 40, 90])
def test_nan_codes_and_scales_stay_in_their_rows(t):
    x, sx, w, sw, _ = operands(t, 272, 272, t)
    x[1, 40] = 0x7F
    sx[1, 3] = np.nan
    w[200, 3] = 0xFF
    got = run_product(x, sx, w, sw, None, "bf16")
    want, s = ref.product(ref.row_values(x, sx.astype(np.float64)), ref.weight_values(w, sw))
    assert np.isnan(want[1]).all() and np.isnan(want[3]).all() and np.isnan(want[:, 200]).all()
    rest = np.ones(want.shape, bool)
    rest[[1, 3]] = False
    rest[:, 200] = False
    assert np.array_equal(np.isnan(got), ~rest)
    check(got[rest], want[rest], (ref.sum_bound(272, t <= ref.FEW) * s)[rest], "bf16", "rest")


@pytest.mark.parametrize("t", [7, 60, 150])
def test_strided_rows_and_another_stream(t):
    n, k = 144, 272
    x, sx, w, sw, bias = operands(t, n, k, t)
    wide = torch.full((t + 1, 336), 0x7F, dtype=torch.uint8, device="cuda")  # NaN between and behind the rows
    wide[:t, 32:32 + k] = dev(x)
    scales = torch.full((4, t + 40), float("nan"), device="cuda")[:, : (t + 40) // 4 * 4].contiguous()
    scales[:3, :t] = dev(sx)[:, :t]
    room = torch.full((t, 168), 7.0, dtype=torch.float16, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with bsg.F8Plan(n, k, t + 5, dtype="f16", bias=True) as plan:
        plan.run(wide[:t, 32:32 + k], scales[:3], dev(w), dev(sw), room[:, 8:152], bias=dev(bias), stream=side)
        torch.cuda.synchronize()
    assert (room[:, :8] == 7).all() and (room[:, 152:] == 7).all()
    want, s = ref.product(ref.row_values(x, sx.astype(np.float64)), ref.weight_values(w, sw), bias)
    check(room[:, 8:152].double().cpu().numpy(), want, ref.sum_bound(k, t <= ref.FEW) * s, "f16", "strided")


@pytest.mark.parametrize("t,n,k", [(7, 144, 272), (20, 144, 272), (61, 144, 272), (510, 6160, 144), (1003, 6160, 400), (2042, 6160, 400)])
def test_scales_in_the_last_columns_of_their_storage(t, n, k):
    """A view of the scales that ends where its storage does, whose rows are shorter than a tile: nothing behind it is read,
    and the result has the bits of a copy's."""
    print("[f8] view of scales", t, n, k, flush=True)
    x, sx, w, sw, _ = operands(t, n, k, t)
    held = torch.full((ref.blocks(k), 16 + sx.shape[1]), float("nan"), device="cuda")
    held[:, 16:16 + t] = dev(sx)[:, :t]
    x, w, sw = dev(x), dev(w), dev(sw)
    outs = [torch.full((t, n), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    with bsg.F8Plan(n, k, t) as plan:
        for scales, out in zip((held[:, 16:], held[:, 16:].contiguous()), outs):
            plan.run(x, scales, w, sw, out)
    torch.cuda.synchronize()
    assert torch.isfinite(outs[0]).all() and torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))


def test_scales_near_the_ends_of_fp32():
    x, sx, w, sw, _ = operands(3, 16, 272, 1, narrow_codes)
    for a, b in ((1e30, 1e-30), (1e-37, 1e35)):
        want, s = ref.product(ref.row_values(x, np.float32(sx * a).astype(np.float64)), ref.weight_values(w, np.float32(sw * b)))
        got = run_product(x, np.float32(sx * a), w, np.float32(sw * b), None, "bf16")
        check(got, want, ref.sum_bound(272, True) * s + 1e-40, "bf16", (a, b))


def scales_at_the_limits(t, n, k, seed):
    """Operands of which block 0 of k has scales of rows from 2^-120 to 2^66 and of weights from 2^-118 to 2^61, whose
    products lie below 2^127 and may be subnormal; every other token's codes are zero there, the others' everywhere else."""
    x, sx, w, sw, _ = operands(t, n, k, seed, narrow_codes)
    rng = np.random.default_rng(seed)
    sx[0, :t] = np.ldexp(1 + rng.random(t), rng.choice([-120, -100, -60, -20, 0, 40, 65], t))
    sw[:, 0] = np.ldexp(1 + rng.random(len(sw)), rng.choice([-118, -50, 0, 40, 60], len(sw)))
    sx[0, :4], sw[:2, 0] = [1.5 * 2.0 ** 65, 1.75 * 2.0 ** 65, 1.5, 1.25 * 2.0 ** -100], [1.25 * 2.0 ** 60, 1.75 * 2.0 ** -40]
    x[::2, :128] = 0
    x[1::2, 128:] = 0
    return x, sx, w, sw


@pytest.mark.parametrize("t,n,k", [(5, 272, 272), (16, 784, 400), (20, 784, 272), (40, 784, 400), (70, 784, 272), (510, 6160, 144),
                                   (1003, 6160, 400), (2042, 6160, 400)])
def test_scales_whose_products_reach_the_ends_of_fp32(t, n, k):
    print("[f8] scales at the limits", t, n, k, flush=True)
    x, sx, w, sw = scales_at_the_limits(t, n, k, t)
    want, s = ref.product(ref.row_values(x, sx.astype(np.float64)), ref.weight_values(w, sw))
    factors = sx[0, :t, None].astype(np.float64) * np.repeat(sw[:, 0].astype(np.float64), 128)[None, :n]
    # the inputs are what they are meant to be: products of scales near both ends, with sums of zero and with others
    assert (factors[::2] > 2.0 ** 125).any() and (factors[1::2] > 2.0 ** 125).any() and (factors[1::2] < 2.0 ** -126).any()
    got = run_product(x, sx, w, sw, None, "bf16")
    # beside the roundings of fp32 sums, 2^-24 or 2^-150 of subnormal ones: half a step of a subnormal product of scales, times a
    # block's sum of at most 128 * 1.875^2 < 2^9 for these codes
    off = ref.sum_bound(k, t <= ref.FEW, True) * s + (2.0 ** 9 + k + 4) * 2.0 ** -150
    most = (2 - 2.0 ** -8) * 2.0 ** 127  # from here on bf16 is infinite
    infinite = np.isinf(got)
    assert not np.isnan(got).any() and infinite.any()
    assert (np.abs(want) + off >= most)[infinite].all() and (np.abs(want) - off < most)[~infinite].all()
    assert np.array_equal(np.sign(got)[infinite], np.sign(want)[infinite])
    check(got[~infinite], want[~infinite], off[~infinite], "bf16", (t, n, k))


# ------------------------------------------------------------------------------------------------ feed-forward block
def ffn_weights(hidden, inter, seed, make=codes_of):
    (w1, s1), (w3, s3) = weights(inter, hidden, seed, hidden ** -0.5, make), weights(inter, hidden, seed + 1, hidden ** -0.5, make)
    w2, s2 = weights(hidden, inter, seed + 2, inter ** -0.5, make)
    return (np.concatenate((w1, w3)), np.stack((s1, s3)), w2, s2), (ref.weight_values(w1, s1), ref.weight_values(w3, s3), ref.weight_values(w2, s2))


def run_ffn(x, held, hidden, inter, dtype):
    t = len(x)
    with bsg.F8FFNPlan(hidden, inter, t, dtype=dtype) as plan:
        out = torch.full((t + 1, hidden), 7.0, dtype=DT[dtype], device="cuda")
        ws = [dev(a) for a in held]
        plan.run(x.cuda(), *ws, out[:t])
        torch.cuda.synchronize()
        first = out.clone()
        plan.run(x.cuda(), *ws, out[:t])
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), first.view(torch.int16)), "not deterministic"
        assert (out[t:] == 7).all()
    return out[:t].double().cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hidden,inter", [(16, 16), (144, 272), (400, 128), (1040, 656)])
@pytest.mark.parametrize("t", [1, 2, 16, 17, 33, 64, 65, 130, 300])
def test_feed_forward(t, hidden, inter, dtype):
    label = f"ffn t={t} hidden={hidden} inter={inter} {dtype}"
    print("[f8]", label, flush=True)
    held, doubles = ffn_weights(hidden, inter, t)
    x = activations(t, hidden, dtype, t + hidden)
    want, off = ref.ffn(x.double().numpy(), *doubles)
    check(run_ffn(x, held, hidden, inter, dtype), want, off, dtype, label)


@pytest.mark.parametrize("t,hidden,inter", [(65, 144, 272), (200, 528, 400), (300, 272, 1040), (2100, 144, 4112)])
def test_feed_forward_of_numbers_that_the_matrix_units_keep(t, hidden, inter):
    # x of +-1 .. 1.875 in 16 bits and such weights: gate and up lose nothing but roundings to fp32, so nearly every inner
    # value has one possible code
    held, doubles = ffn_weights(hidden, inter, t, narrow_codes)
    x = torch.from_numpy(ref.values(narrow_codes(np.random.default_rng(t), (t, hidden)))).bfloat16()
    want, off = ref.ffn(x.double().numpy(), *doubles, exact_range=True)
    check(run_ffn(x, held, hidden, inter, "bf16"), want, off, "bf16", (t, hidden, inter))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_feed_forward_of_more_large_tiles_than_run_at_once(dtype):
    """8 x 64 tiles of 256 tokens and 128 inner values, the last of both shorter: every workgroup does two, and the second
    one's copies go where the first kept its tokens' largest magnitudes.  The reference has the tokens at the tiles' edges
    and every 13th; tokens do not depend on each other."""
    t, hidden, inter = 2040, 528, 8176
    print("[f8] ffn", t, hidden, inter, dtype, flush=True)
    held, doubles = ffn_weights(hidden, inter, 5, narrow_codes)
    x = torch.from_numpy(ref.values(narrow_codes(np.random.default_rng(6), (t, hidden)))).to(DT[dtype])
    got = run_ffn(x, held, hidden, inter, dtype)
    rows = np.unique(np.concatenate([np.arange(0, t, 13), np.arange(255, t, 256), np.arange(256, t, 256), [t - 1]]))
    want, off = ref.ffn(x[rows].double().numpy(), *doubles, exact_range=True)
    check(got[rows], want, off, dtype, (t, hidden, inter))


@pytest.mark.parametrize("t", [3, 40, 100])
def test_feed_forward_infinite_and_nan_tokens_stay_in_their_rows(t):
    held, doubles = ffn_weights(144, 144, t)
    x = activations(t, 144, "bf16", t)
    clean = run_ffn(x, held, 144, 144, "bf16")
    x[0, 3], x[2, 140] = float("inf"), float("nan")
    got = run_ffn(x, held, 144, 144, "bf16")
    assert np.isnan(got[[0, 2]]).all()
    rest = np.ones(t, bool)
    rest[[0, 2]] = False
    assert np.array_equal(got[rest], clean[rest])


def test_feed_forward_strides_stream_and_smaller_calls():
    held, doubles = ffn_weights(144, 272, 5)
    wide = activations(100, 176, "f16", 6).cuda()
    room = torch.full((100, 160), 7.0, dtype=torch.float16, device="cuda")
    side = torch.cuda.Stream()
    ws = [dev(a) for a in held]
    torch.cuda.synchronize()
    with bsg.F8FFNPlan(144, 272, 100, dtype="f16") as plan:
        assert plan.workspace_bytes() > 0
        for t in (100, 7, 33, 1, 70):
            room.fill_(7.0)
            torch.cuda.synchronize()
            plan.run(wide[:t, 16:160], *ws, room[:t, 8:152], stream=side)
            torch.cuda.synchronize()
            want, off = ref.ffn(wide[:t, 16:160].double().cpu().numpy(), *doubles)
            check(room[:t, 8:152].double().cpu().numpy(), want, off, "f16", t)
            assert (room[:, :8] == 7).all() and (room[:, 152:] == 7).all() and (room[t:] == 7).all()
        plan.run(wide[:0, 16:160], *ws, room[:0, 8:152])


# ------------------------------------------------------------------------------------------------ graphs
@pytest.mark.parametrize("t", [1, 20, 100])
def test_captured_calls_replay(t):
    n, k = 272, 400
    held, _ = ffn_weights(n, n, 3)
    ws = [dev(a) for a in held]
    w, sw = (dev(a) for a in weights(n, k, 9))
    x = activations(t, k, "bf16", 1).cuda()
    codes = torch.empty(t, k, dtype=torch.uint8, device="cuda")
    scales = torch.empty(bsg.f8_scales_shape(t, k), device="cuda")
    mid, out = (torch.empty(t, n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    with bsg.F8Plan(n, k, t) as plan, bsg.F8FFNPlan(n, n, t) as ffn:
        def chain():
            bsg.f8_quantize(x, codes, scales)
            plan.run(codes, scales, w, sw, mid)
            ffn.run(mid, *ws, out)

        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            chain()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            chain()
        for i in range(4):
            x.copy_(activations(t, k, "bf16", 20 + i))
            graph.replay()
            torch.cuda.synchronize()
            got = out.clone()
            out.zero_()
            chain()
            torch.cuda.synchronize()
            assert torch.equal(got.view(torch.int16), out.view(torch.int16)), i


# ------------------------------------------------------------------------------------------------ refusals
def test_what_the_binding_and_the_plans_refuse():
    t, n, k = 6, 32, 144
    x, w = torch.zeros(t, k, dtype=torch.uint8, device="cuda"), torch.zeros(n, k, dtype=torch.uint8, device="cuda")
    sx, sw = torch.ones(bsg.f8_scales_shape(t, k), device="cuda"), torch.ones(1, 2, device="cuda")
    out = torch.zeros(t, n, dtype=torch.bfloat16, device="cuda")
    wide = torch.zeros(t, k + 24, dtype=torch.uint8, device="cuda")
    with bsg.F8Plan(n, k, 8) as plan, bsg.F8Plan(n, k, 8, bias=True) as biased:
        good = dict(x=x, x_scales=sx, w=w, w_scales=sw, out=out)
        plan.run(**good)
        for change, status in [
            (dict(x=x[:, :128]), None), (dict(x=x.short()), None), (dict(x=x.t()), None), (dict(x_scales=sx[:1]), None),
            (dict(x_scales=sx[:, :4]), None), (dict(x_scales=sx.double()), None), (dict(x_scales=sx[:, :6].contiguous()), 4),
            (dict(w=w[:16]), None), (dict(w=w.int()), None), (dict(w_scales=sw[:, :1]), None), (dict(w_scales=sw.half()), None),
            (dict(out=out.half()), None), (dict(out=out[:5]), None), (dict(out=out[:, :16]), None),
            (dict(x=wide[:, 8:8 + k]), 4), (dict(x=wide[:, :k]), 4),
            (dict(x=x.repeat(2, 1)[:9], x_scales=torch.ones(2, 12, device="cuda"), out=out.repeat(2, 1)[:9]), 2),
        ]:
            with pytest.raises((ValueError, bsg.BsgError)) as e:
                plan.run(**(good | change))
            assert status is None and isinstance(e.value, ValueError) or getattr(e.value, "status", None) == status, (change, e.value)
        for bias in (None, torch.zeros(n, device="cuda").half(), torch.zeros(n - 1, device="cuda")):
            with pytest.raises(ValueError):
                biased.run(**good, bias=bias)
    h = torch.zeros(t, k, dtype=torch.bfloat16, device="cuda")
    w13, s13 = torch.zeros(64, k, dtype=torch.uint8, device="cuda"), torch.ones(2, 1, 2, device="cuda")
    w2, s2 = torch.zeros(k, 32, dtype=torch.uint8, device="cuda"), torch.ones(2, 1, device="cuda")
    with bsg.F8FFNPlan(k, 32, 8) as ffn:
        ffn.run(h, w13, s13, w2, s2, h.clone())
        for args in ((h.half(), w13, s13, w2, s2, h), (h, w13[:32], s13, w2, s2, h), (h, w13, s13[:1], w2, s2, h),
                     (h, w13, s13, w2.t(), s2, h), (h, w13, s13, w2, s2.double(), h), (h, w13, s13, w2, s2, h[:3])):
            with pytest.raises(ValueError):
                ffn.run(*args)
        with pytest.raises(bsg.BsgError):
            ffn.run(h.repeat(2, 1), w13, s13, w2, s2, h.repeat(2, 1))
    with pytest.raises(ValueError):
        bsg.f8_quantize(h.float(), x, sx)
    with pytest.raises(ValueError):
        bsg.f8_quantize(h, x[:, :128], sx)
    torch.cuda.synchronize()


def test_weights_laid_out_the_other_way_are_refused():
    t, n, k = 6, 272, 144
    x, sx = torch.zeros(t, k, dtype=torch.uint8, device="cuda"), torch.ones(bsg.f8_scales_shape(t, k), device="cuda")
    w, sw = torch.zeros(n, k, dtype=torch.uint8, device="cuda"), torch.ones(3, 2, device="cuda")
    out = torch.zeros(t, n, dtype=torch.bfloat16, device="cuda")
    with bsg.F8Plan(n, k, t) as plan:
        for good in ((w, sw), (w.view(2, n // 2, k), sw), (w.flatten(), sw.flatten())):
            plan.run(x, sx, *good, out)
        for bad in ((w.view(k, n), sw), (w.t().contiguous(), sw), (w, sw.t().contiguous()), (w, sw.view(6, 1))):
            with pytest.raises(ValueError):
                plan.run(x, sx, *bad, out)
    h = torch.zeros(t, k, dtype=torch.bfloat16, device="cuda")
    w13, s13 = torch.zeros(2 * n, k, dtype=torch.uint8, device="cuda"), torch.ones(2, 3, 2, device="cuda")
    w2, s2 = torch.zeros(k, n, dtype=torch.uint8, device="cuda"), torch.ones(2, 3, device="cuda")
    with bsg.F8FFNPlan(k, n, t) as ffn:
        ffn.run(h, w13, s13, w2, s2, h.clone())
        ffn.run(h, w13.view(2, n, k), s13.view(6, 2), w2, s2, h.clone())
        for bad in ((w13.view(k, 2 * n), s13, w2, s2), (w13, s13.transpose(1, 2).contiguous(), w2, s2),
                    (w13, s13, w2.view(n, k), s2), (w13, s13, w2, s2.view(3, 2))):
            with pytest.raises(ValueError):
                ffn.run(h, *bad, h.clone())
    torch.cuda.synchronize()


@pytest.mark.parametrize("other", [torch.float8_e5m2, torch.bool])
def test_one_byte_types_that_are_no_codes_are_refused(other):
    x, w = torch.zeros(4, 32, dtype=torch.uint8, device="cuda"), torch.zeros(16, 32, dtype=torch.uint8, device="cuda")
    sx, sw, out = torch.ones(1, 4, device="cuda"), torch.ones(1, 1, device="cuda"), torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
    with bsg.F8Plan(16, 32, 4) as plan:
        for kind in (torch.uint8, torch.int8, torch.float8_e4m3fn):
            plan.run(x.view(kind), sx, w.view(kind), sw, out)
        for args in ((x.view(other), sx, w, sw, out), (x, sx, w.view(other), sw, out)):
            with pytest.raises(ValueError):
                plan.run(*args)
    torch.cuda.synchronize()


@pytest.mark.parametrize("n", [272, 2064])
def test_rows_whose_offsets_pass_32_bits(n):
    """Rows 2^21 and more apart, so that the last lie beyond 2^32 bytes: the same bits as from neighbouring rows."""
    t, k, far = 2100, 144, (1 << 21) + 16
    x = activations(t, k, "bf16", 7).cuda()
    w, sw = (dev(a) for a in weights(n, k, 8))

    def spread(cols, dtype):
        held = torch.empty(t * far, dtype=dtype, device="cuda").view(t, far)
        return held[:, :cols]

    results = []
    for make in (lambda cols, dtype: torch.empty(t, cols, dtype=dtype, device="cuda"), spread):
        a, codes, out = make(k, torch.bfloat16), make(k, torch.uint8), make(n, torch.bfloat16)
        a.copy_(x)
        scales = torch.ones(bsg.f8_scales_shape(t, k), device="cuda")
        bsg.f8_quantize(a, codes, scales)
        with bsg.F8Plan(n, k, t) as plan:
            plan.run(codes, scales, w, sw, out)
        torch.cuda.synchronize()
        results.append((codes.cpu(), scales.cpu(), out.cpu()))
    for near, distant in zip(*results):
        assert torch.equal(near.contiguous().view(torch.uint8), distant.contiguous().view(torch.uint8))
    torch.cuda.empty_cache()  # (13 GB)
