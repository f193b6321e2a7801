"""Paged attention at the ends of its arguments' ranges: very long contexts, weights far below the largest, soft caps far
above the scores, unbounded windows, the largest magnitudes, uneven batches.  References are 64-bit (kv_ref), or closed
forms where a cache's pages repeat."""
import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_amd as bsg
import kv_ref
from test_gpu_kv import DT, append_case, attend, check, dev, filled, layout, run_case

pytestmark = pytest.mark.gpu


def repeated(c, table, q, scale, dtype, **kw):
    """One query over positions whose pages are table's: (out, lse) of the library and of the closed form.  H = 1."""
    P, D, n = c.p, c.dim, len(table) * c.p
    with bsg.KVPlan(q.shape[0], 1, D, P, len(c.bytes), 1, dtype=dtype, scale=scale, **kw) as plan:
        b = bsg.KVBatch(dev(np.array([0, 1], np.int32)), dev(np.array([n], np.int32)), dev(table[None].astype(np.int32)), 1, 1, n)
        qd = torch.from_numpy(q[None]).to(DT[dtype]).cuda()
        out, lse = torch.full_like(qd, 7.0), torch.full((1, q.shape[0]), 7.0, device="cuda")
        plan.attend(b, qd, dev(c.bytes), out, lse=lse)
        torch.cuda.synchronize()
    times = np.bincount(table, minlength=len(c.bytes))
    k, v = (np.array([[c.load(p, s, 0, is_v) for s in range(P)] for p in range(len(times))]) for is_v in (False, True))
    s = np.einsum("psd,hd->hps", k, qd.double().cpu().numpy()[0]) * scale
    top = s.max((1, 2))
    w = np.exp(s - top[:, None, None]) * times[:, None]
    total = w.sum((1, 2))
    return (out.double().cpu().numpy()[0], lse.double().cpu().numpy()[0], np.einsum("hps,psd->hd", w, v) / total[:, None],
            top + np.log(total))


def test_half_a_billion_positions():
    # one sequence and one head cut into as many pieces as the card takes: their bounds pass 2^31 on the way.  A piece that
    # is left out changes the log-sum-exp by 1/511 or more; sums of 2^16 terms a lane in 32 bits are off by about 2^-24 2^8.
    rng = np.random.default_rng(0)
    c = kv_ref.Cache(2, 1, 64, 256)
    for page in range(2):
        for is_v in (False, True):
            code, s = kv_ref.quantize(rng.standard_normal((256, 64)))
            for p in range(256):
                c.store(page, p, 0, is_v, code[p], s[p])
    table = (np.arange(1 << 21) % 3 == 2).astype(np.int32)
    print("[kv] 2^29 positions", flush=True)
    got, lse, want, want_lse = repeated(c, table, rng.standard_normal((1, 64)), 0.125, "f16")
    assert np.abs(lse - want_lse).max() < 2.0 ** -10
    assert np.abs(got - want).max() < 2.0 ** -10


def test_more_units_than_a_call_can_count_are_refused():
    n = 1 << 24
    lens, pages = torch.ones(n, dtype=torch.int32, device="cuda"), torch.zeros(n, 1, dtype=torch.int32, device="cuda")
    x = torch.zeros(1, 16, 64, dtype=torch.bfloat16, device="cuda").expand(n, 16, 64)
    with bsg.KVPlan(16, 16, 64, 16, 1, n) as plan:
        batch = bsg.KVBatch(torch.arange(n + 1, dtype=torch.int32, device="cuda"), lens, pages, n, 1, 1)
        with pytest.raises(bsg.BsgError) as e:
            plan.attend(batch, x, torch.zeros(plan.page_bytes, dtype=torch.uint8, device="cuda"), x)
        assert e.value.status_name == "BSG_ERR_UNSUPPORTED"
        torch.cuda.synchronize()


@pytest.mark.parametrize("new,lens,G", [
    ([300] + [1] * 20, [400] + [5 + 9 * i for i in range(20)], 4),               # one prompt, single tokens
    ([0, 2, 330, 0, 9, 1, 1, 8, 7, 30, 1, 0], [9, 2, 330, 0, 40, 700, 1, 8, 3, 30, 64, 5], 4),
    ([1] * 70 + [280] + [3] * 70, [9 + i for i in range(70)] + [500] + [40 + i for i in range(70)], 4),  # past 64 sequences
    ([40] + [1] * 9 + [5, 0], [900] + [30 + i for i in range(9)] + [5, 3], 40),   # groups that are too wide for the other kernel
])
@pytest.mark.parametrize("H,D,dtype,kw", [(1, 64, "f16", {}), (8, 64, "bf16", {"window": 50}), (3, 128, "bf16", {"causal": False})], ids=str)
def test_uneven_batches_list_their_row_blocks(new, lens, G, H, D, dtype, kw):
    run_case(new, lens, H=H, G=G, D=D, dtype=dtype, seed=len(new) + H, **kw)


def test_a_long_prompt_beside_many_single_tokens():
    # 64 heads on 8: 32768 new tokens of one sequence and one of 1023 others, in one call and apart
    n, others, hq, hk, D, P = 32768, 1023, 64, 8, 64, 64
    g = torch.Generator(device="cuda").manual_seed(0)
    q = torch.randn(n + others, hq, D, generator=g, device="cuda").bfloat16()
    lens = torch.randint(1, 200, (others,), generator=g, device="cuda", dtype=torch.int32)
    pages = torch.randint(0, 600, (others + 1, n // P), generator=g, device="cuda", dtype=torch.int32)
    with bsg.KVPlan(hq, hk, D, P, 600, n + others) as plan:
        cache = torch.randint(0, 56, (600 * plan.page_bytes,), generator=g, device="cuda", dtype=torch.uint8)
        print("[kv] 32768 tokens beside 1023 single ones", flush=True)

        def attend(a, z, starts, lens, pages, max_q, max_kv):
            out, lse = torch.zeros_like(q[a:z]), torch.zeros(z - a, hq, device="cuda")
            plan.attend(bsg.KVBatch(dev(np.array(starts, np.int32)), lens, pages, z - a, max_q, max_kv), q[a:z], cache, out, lse=lse)
            torch.cuda.synchronize()
            return out, lse
        one = torch.tensor([n], dtype=torch.int32, device="cuda")
        whole = attend(0, n + others, np.r_[0, n:n + others + 1], torch.cat((one, lens)), pages, n, n)
        apart = [attend(0, n, [0, n], one, pages[:1], n, n), attend(n, n + others, np.arange(others + 1), lens, pages[1:], 1, n)]
    for got, want in zip(whole, zip(*apart)):
        want = torch.cat(want)
        assert torch.isfinite(got).all()
        # values reach 6 x 0.94 (E4M3 code 55): the two calls differ by their roundings only
        assert ((got.float() - want.float()).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -10 * 5.7).all()


@pytest.mark.parametrize("window", [(1 << 30) - 1, 1 << 30, (1 << 31) - 1])
def test_windows_without_an_end(window):
    # more new tokens than positions: the first queries see nothing, the others all up to their own
    run_case([7, 2, 1], [3, 1, 90], seed=23, window=window)
    run_case([70, 40], [20, 500], seed=24, window=window)
    args = dict(new=[40], lens=[900], H=1, G=4, D=64, P=32, dtype="f16", seed=25)
    for a, b in zip(run_case(**args, window=window), run_case(**args)):
        assert np.array_equal(a, b)  # cut into the same parts as without a window


def test_queries_up_to_the_largest_bf16():
    def case(new, lens, seed):
        q_start, pages, n_pages = layout(new, lens, 16, seed)
        c = filled(lens, 2, 64, 16, pages, n_pages, seed + 1)
        q = torch.randn(sum(new), 8, 64, generator=torch.Generator().manual_seed(seed)) * 1e38
        q = q.clamp(-3.38e38, 3.38e38).bfloat16()
        q[0, 0, 5] = torch.finfo(torch.bfloat16).max
        scale = 3e-38
        want, wl = kv_ref.attend(q.double().numpy(), c, q_start, lens, pages, 2, scale=float(np.float32(scale)))
        got, lse = attend(c, q.cuda(), q_start, lens, pages, 2, 16, 64, "bf16", scale=scale)
        assert np.isfinite(want).all()
        check(got, lse, want, wl, "bf16", 4.5, f"largest {new}")
    case([3, 1], [90, 40], 26)
    case([50], [120], 27)


@pytest.mark.parametrize("softcap", [0.5, 8.0, 50.0, 65.0, 2500.0, 1e5, 1e30, 3e38])
@pytest.mark.parametrize("new,lens", [([3, 1], [90, 300]), ([40, 70], [300, 200])], ids=["few", "many"])
def test_soft_caps(softcap, new, lens):
    # a capped score is within 2^-19 of itself, or 2^-16, so a cap far above the scores changes nothing
    run_case(new, lens, D=64, dtype="f16", seed=21, softcap=softcap, q_gain=2.0)
    run_case(new, lens, D=128, dtype="bf16", seed=22, softcap=softcap)


def test_weights_far_below_the_largest_are_kept():
    # in each run of 32 positions (a wave's) one of weight 1 and value 0 beside 31 of weight 2^-36 and value 6: beside 2^14
    # those are 2^-22 in fp16, exactly, and what is left is the output's rounding
    c = kv_ref.Cache(1, 1, 64, 128)
    code, s = kv_ref.quantize(np.full(64, 6.0))
    one, s1 = kv_ref.quantize(np.r_[6.0, np.zeros(63)])
    for p in range(128):
        c.store(0, p, 0, True, code, s)
    for p in (5, 37, 69, 101):
        c.store(0, p, 0, False, one, s1)
        c.store(0, p, 0, True, np.zeros(64, np.uint8), np.zeros(4, np.uint8))
    q = np.zeros((1, 64))
    q[0, 0] = 1.0
    got, lse, want, want_lse = repeated(c, np.zeros(1, np.int32), q, float(np.float32(36 * np.log(2.0) / 6)), "bf16")
    assert 2.6e-9 < want.min() and want.max() < 2.8e-9
    assert (np.abs(got - want) <= 2.0 ** -8 * want).all(), (got, want)
    assert np.abs(lse - want_lse).max() < 1e-4


@pytest.mark.parametrize("D,new", [(64, [4000, 0, 99, 1]), (128, [1, 2050, 49])])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rope,interleaved", [(0, False), (64, False), (64, True), (32, True)])
def test_append_of_many_tokens(D, new, dtype, rope, interleaved):
    # enough rows for workgroups of four heads each; 18 heads leave two of them in the last
    append_case(new, [n + 7 * i for i, n in enumerate(new)], 3, 4, D, 64, dtype, rope, interleaved, seed=len(new) + rope)


def test_append_keeps_the_sign_of_zeros():
    # -0 rounds to E2M1's -0 (code 8), beside other elements and in a block of zeros
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 0, 1:32:2] = -0.0
    x[0, 0, 0] = 3.0
    with bsg.KVPlan(1, 1, 64, 16, 1, 1) as plan:
        cache = torch.full((plan.page_bytes,), 0x55, dtype=torch.uint8, device="cuda")
        batch = bsg.KVBatch(dev(np.array([0, 1], np.int32)), dev(np.array([1], np.int32)), dev(np.zeros((1, 1), np.int32)), 1, 1, 1)
        plan.append(batch, x, x, cache)
        k, v = torch.ones_like(x), torch.ones_like(x)
        plan.read(batch, cache, k, v)
        torch.cuda.synchronize()
    for part in (cache[:32], cache[16 * 32:16 * 32 + 32]):
        assert part.tolist() == [0x87] + [0x80] * 15 + [0] * 16
    assert torch.equal(k.view(torch.int16), x.view(torch.int16)) and torch.equal(v.view(torch.int16), x.view(torch.int16))


@pytest.mark.parametrize("new,lens", [([9, 1], [130, 300]), ([40, 33], [90, 700])], ids=["4 waves", "8 waves"])
def test_scales_and_large_scores_of_many_rows(new, lens):
    run_case(new, lens, seed=31, scale=0.3, k_scale=0.25, v_scale=3.0)
    run_case(new, lens, D=64, dtype="f16", seed=32, scale=-0.2, k_scale=4.0, v_scale=0.125)
    run_case(new, lens, seed=33, q_gain=300.0)
    run_case(new, lens, seed=34, q_gain=1e-30)
    run_case(new, lens, D=64, seed=35, q_gain=1e30, scale=1e-30)


def ramp(n, D, rise):
    """Keys along one direction whose scores against it (at scale 1 / sqrt(D)) rise by `rise` (base 2) each 64 positions."""
    d = np.where(np.arange(D) % 3 == 1, -1.0, 1.0)
    return np.arange(n)[:, None] * d * (rise * np.log(2.0) / 64 / np.sqrt(D)), d


@pytest.mark.parametrize("rise", [0.3, 1.0, 2.4, 4.9, 7.0, -3.0])
@pytest.mark.parametrize("new,D,dtype", [(9, 64, "f16"), (9, 128, "bf16"), (40, 128, "f16"), (40, 64, "bf16")])
def test_scores_that_rise_slowly(rise, new, D, dtype):
    # the reference of a row's weights is only replaced when a score lies 5 above it: between, weights reach 2^15.  Rows'
    # own slopes differ, some fall.  Split positions (kv_ref), and one workgroup per row block (512 heads).
    n, G = 1200, 4
    q_start, pages, n_pages = layout([new], [n], 32, 40)
    c = filled([n], 1, D, 32, pages, n_pages, 41)
    k, d = ramp(n, D, rise)
    code, s = kv_ref.quantize(k)
    for p in range(n):
        c.store(pages[0][p // 32], p % 32, 0, False, code[p], s[p])
    rng = np.random.default_rng(42)
    slopes = rng.uniform(-1, 1, (new, G, 1))
    slopes[0, 0] = slopes[-1, -1] = 1.0
    q = torch.from_numpy(slopes * d + 0.05 * rng.standard_normal((new, G, D))).to(DT[dtype])
    want, wl = kv_ref.attend(q.double().numpy(), c, q_start, [n], pages, 1)
    print(f"[kv] rise {rise} {new} {D} {dtype}", flush=True)
    got, lse = attend(c, q.cuda(), q_start, [n], pages, 1, 32, D, dtype)
    check(got, lse, want, wl, dtype, 5.0, f"rise {rise} {new} {D} {dtype}")
    H, n = 512, 450
    q_start, pages, n_pages = layout([n], [n], 32, 43)
    lens, pg = dev(np.array([n], np.int32)), dev(pages)
    g = torch.Generator().manual_seed(44)
    rows = 40 if new == 9 else 150
    with bsg.KVPlan(H, H, D, 32, n_pages, n, dtype=dtype) as plan:
        kv = [torch.from_numpy(ramp(n, D, rise)[0])[:, None].expand(n, H, D).to(DT[dtype]).contiguous().cuda(),
              torch.randn(n, H, D, generator=g).to(DT[dtype]).cuda()]
        cache = torch.full((n_pages * plan.page_bytes,), 0x7F, dtype=torch.uint8, device="cuda")
        whole = bsg.KVBatch(dev(q_start), lens, pg, n, n, n)
        plan.append(whole, *kv, cache)
        plan.read(whole, cache, *kv)
        q = (torch.rand(rows, H, 1, generator=g) * 2 - 1) * torch.from_numpy(d) + 0.05 * torch.randn(rows, H, D, generator=g)
        q = q.to(DT[dtype]).cuda()
        out, lse = torch.zeros_like(q), torch.zeros(rows, H, device="cuda")
        plan.attend(bsg.KVBatch(dev(np.array([0, rows], np.int32)), lens, pg, rows, rows, n), q, cache, out, lse=lse)
        torch.cuda.synchronize()
    qd, k, v = (x.double().transpose(0, 1).contiguous() for x in (q, *kv))
    s = torch.matmul(qd, k.transpose(1, 2).contiguous()) * D ** -0.5
    hidden = torch.arange(n, device="cuda")[None] > torch.arange(n - rows, n, device="cuda")[:, None]
    s = s.masked_fill(hidden, float("-inf"))
    want = torch.matmul(s.softmax(-1), v).transpose(0, 1)
    check(out.double().cpu().numpy(), lse.double().cpu().numpy(), want.cpu().numpy(), s.logsumexp(-1).T.cpu().numpy(), dtype,
          float(v.abs().max()), f"rise {rise} {rows} rows of {H} heads")


@pytest.mark.parametrize("v_scale", [3e36, 2e-38])
def test_value_scales_at_the_ends_of_their_range(v_scale):
    # the results are v_scale times ordinary numbers and fit bf16; the largest stored value is below 6 x 448 of them
    for new, lens in (([1, 3], [90, 300]), ([40], [200]), ([12], [900])):
        run_case(new, lens, D=64, seed=50, v_scale=v_scale)
