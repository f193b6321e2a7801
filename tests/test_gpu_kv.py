"""Paged NVFP4 cache on the GPU against the 64-bit reference of kv_ref: append (rotation, quantisation,
placement), read, and attention over masks, lengths, layouts and strides where kernels go wrong."""
import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_amd as bsg
import kv_ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
# unit roundoff of the output type; 2^-8 and 2^-11 (bf16, fp16)
UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def layout(new, lens, P, seed, spare=2):
    """q_start, pages (a random order, page 0 never used) and the number of pages."""
    rng = np.random.default_rng(seed)
    per = [-(-n // P) for n in lens]
    order = rng.permutation(np.arange(1, sum(per) + 1 + spare)).astype(np.int32)
    pages = np.zeros((len(lens), max(max(per), 1)), np.int32)
    at = 0
    for b, n in enumerate(per):
        pages[b, :n] = order[at:at + n]
        at += n
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32), pages, sum(per) + 1 + spare


def filled(lens, H, D, P, pages, n_pages, seed, fill=0x7F, page_stride=0, k_gain=1.0):
    """A cache whose used slots hold quantised Gaussians and whose other bytes are `fill` (0x7F: NaN scales)."""
    rng = np.random.default_rng(seed)
    c = kv_ref.Cache(n_pages, H, D, P, fill, page_stride)
    for b, n in enumerate(lens):
        for h in range(H if n else 0):
            for is_v in (False, True):
                code, s = kv_ref.quantize(rng.standard_normal((n, D)) * (1.0 if is_v else k_gain))
                for p in range(n):
                    c.store(pages[b][p // P], p % P, h, is_v, code[p], s[p])
    return c


def attend(c, q, q_start, lens, pages, H, P, D, dtype, max_q=None, stream=None, out=None, **kw):
    T, hq = q.shape[:2]
    new = np.diff(q_start)
    with bsg.KVPlan(hq, H, D, P, len(c.bytes), max(T, len(lens)), dtype=dtype, page_stride=c.stride if
                    c.stride != H * P * D * 9 // 8 else 0, **kw) as plan:
        batch = bsg.KVBatch(dev(q_start), dev(np.asarray(lens, np.int32)), dev(pages), T, max_q or int(new.max()), int(max(lens)) or 1)
        out = torch.full((T, hq, D), 7.0, dtype=DT[dtype], device="cuda") if out is None else out
        lse = torch.full((T, hq), 7.0, dtype=torch.float32, device="cuda")
        plan.attend(batch, q, dev(c.bytes), out, lse=lse, stream=stream)
        torch.cuda.synchronize()
        first = out.clone()
        plan.attend(batch, q, dev(c.bytes), out, lse=lse, stream=stream)  # the counters are back at zero
        torch.cuda.synchronize()
        assert torch.equal(torch.nan_to_num(out.float(), 9e9), torch.nan_to_num(first.float(), 9e9)), "not deterministic"
        return out.double().cpu().numpy(), lse.double().cpu().numpy()


def check(got, lse, want, want_lse, dtype, v_max, label):
    """P is held to 2^-12 of itself (fp16), sums in fp32, one rounding of the output: |error| <= 2 u |o| +
    2^-11 max|v| (a weighted mean of values, each weight off by at most 2^-12 and their sum by as much)."""
    bad = np.isnan(want)
    assert np.array_equal(np.isnan(got), bad), label
    err = np.abs(got - want)[~bad]
    lim = (2 * UNIT[dtype] * np.abs(want) + 2.0 ** -11 * v_max + 1e-7)[~bad]
    assert (err <= lim).all(), (label, float((err - lim).max()))
    fin = np.isfinite(want_lse)
    assert np.array_equal(np.isneginf(want_lse), np.isneginf(lse)) and np.array_equal(np.isnan(want_lse), np.isnan(lse)), label
    assert (np.abs(lse - want_lse)[fin] <= 2e-5 + 2e-6 * np.abs(want_lse[fin])).all(), label


def run_case(new, lens, H=2, G=4, D=128, P=16, dtype="bf16", seed=0, fill=0x7F, page_stride=0, q_gain=1.0, edit=None, **kw):
    q_start, pages, n_pages = layout(new, lens, P, seed)
    c = filled(lens, H, D, P, pages, n_pages, seed + 1, fill, page_stride)
    if edit:
        edit(c, pages)
    rng = np.random.default_rng(seed + 2)
    q = torch.from_numpy(rng.standard_normal((int(q_start[-1]), H * G, D)) * q_gain).to(DT[dtype])
    want, want_lse = kv_ref.attend(q.double().numpy(), c, q_start, lens, pages, H, **kw)
    v_max = max([np.nanmax(np.abs(np.array([c.load(pages[b][p // P], p % P, h, True, kw.get("v_scale", 1.0)) for p in range(n)])), initial=0)
                 for b, n in enumerate(lens) for h in range(H)] + [0])
    label = f"new={new} lens={lens} H={H} G={G} D={D} P={P} {dtype} {kw}"
    print("[kv]", label, flush=True)
    got, lse = attend(c, q.cuda(), q_start, lens, pages, H, P, D, dtype, **kw)
    check(got, lse, want, want_lse, dtype, v_max, label)
    return got, lse


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("P", [16, 64, 256])
def test_one_token_lengths(D, dtype, P):
    # around the 16-position groups, the 64-position tiles and the pages; longer ones split over workgroups
    run_case([1] * 9, [1, 15, 16, 17, 63, 64, 65, 257, 1030], D=D, dtype=dtype, P=P, seed=P + D)


@pytest.mark.parametrize("H,G", [(1, 1), (3, 1), (1, 5), (2, 8), (1, 16), (1, 17), (1, 32), (1, 40), (1, 71)])
def test_head_groups(H, G):
    run_case([1, 1], [130, 77], H=H, G=G, D=64, seed=H * 100 + G)


@pytest.mark.parametrize("new,lens", [
    ([3], [3]), ([2, 5, 1], [40, 5, 129]), ([7, 7], [300, 71]), ([33], [33]), ([70, 1, 17], [200, 90, 17]), ([129], [400]),
])
@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "f16")])
@pytest.mark.parametrize("kw", [{}, {"window": 20}, {"window": 1}, {"causal": False}, {"softcap": 3.0}], ids=str)
def test_several_tokens(new, lens, D, dtype, kw):
    run_case(new, lens, D=D, dtype=dtype, seed=len(lens), **kw)


@pytest.mark.parametrize("window", [1, 5, 64, 100, 1000])
def test_window_of_one_token(window):
    run_case([1, 1, 1], [400, 3, 130], window=window, seed=window)


def test_long_context_joined_from_many_parts():
    run_case([1], [9001], H=1, G=4, D=64, P=64, seed=3)
    run_case([1, 1], [4100, 37], H=1, G=2, D=128, P=32, seed=4)


def test_more_than_256_sequences():
    lens = [1 + (37 * i) % 50 for i in range(301)]
    run_case([1] * 301, lens, H=1, G=2, D=64, seed=5)


def test_empty_sequences_and_empty_rows():
    # no context; no new token; fewer positions than new tokens (the first queries see nothing)
    got, lse = run_case([1, 0, 2, 4, 1], [0, 30, 1, 2, 0], seed=6)
    assert np.isneginf(lse[0]).all() and (got[0] == 0).all() and (got[1] == 0).all()
    run_case([0, 1, 0], [5, 40, 0], seed=7)


def test_nothing_to_do():
    with bsg.KVPlan(2, 1, 64, 16, 4, 8) as plan:
        z = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
        b = bsg.KVBatch(dev(np.zeros(1, np.int32)), dev(np.zeros(0, np.int32)), dev(np.zeros((0, 1), np.int32)), 0, 0, 0)
        plan.attend(b, z, torch.zeros(4 * plan.page_bytes, dtype=torch.uint8, device="cuda"), z)
        torch.cuda.synchronize()


def test_scales_and_large_scores():
    run_case([2, 1], [90, 33], seed=8, scale=0.3, k_scale=0.25, v_scale=3.0)
    run_case([1, 1], [200, 64], seed=9, q_gain=300.0)      # one position takes nearly all the weight
    run_case([1, 1], [200, 64], seed=10, q_gain=1e-30)     # bf16 magnitudes far below fp16's
    run_case([1, 1], [100, 64], seed=11, q_gain=1e30, scale=1e-30)


def test_page_stride_and_other_layers_bytes():
    run_case([2, 1], [90, 33], seed=12, page_stride=2 * 16 * 128 * 9 // 8 + 4096)


def test_nan_blocks_reach_exactly_the_queries_that_see_them():
    def poison(c, pages):
        c.part(pages[0][30 // 16], 0, 3)[2, 30 % 16] = 0x7F   # value block 2 of position 30
        c.part(pages[0][33 // 16], 1, 2)[33 % 16, 1] = 0x7F   # a key block of position 33
    got, _ = run_case([6, 1], [36, 20], seed=13, edit=poison)          # position 30 is the first query's own
    assert np.isnan(got[0, :4, 32:48]).all() and not np.isnan(got[0, :4, :32]).any()
    assert not np.isnan(got[2, 4:]).any() and np.isnan(got[3, 4:]).all()
    run_case([5, 1], [36, 20], seed=14, edit=poison)                   # every query sees it
    run_case([6, 1], [36, 20], seed=15, edit=poison, window=3)
    run_case([40, 1], [40, 20], seed=16, edit=poison)


def test_infinite_and_nan_queries_stay_in_their_rows():
    q_start, pages, n_pages = layout([1, 1], [40, 50], 16, 0)
    c = filled([40, 50], 1, 64, 16, pages, n_pages, 1)
    q = torch.randn(2, 2, 64, generator=torch.Generator().manual_seed(0)).bfloat16()
    q[0, 0, 3] = float("nan")
    q[1, 1, 3] = float("inf")
    want, _ = kv_ref.attend(q.double().numpy(), c, q_start, [40, 50], pages, 1)
    got, _ = attend(c, q.cuda(), q_start, [40, 50], pages, 1, 16, 64, "bf16")
    assert np.isnan(got[0, 0]).all()
    for t, j in ((0, 1), (1, 0)):
        assert np.abs(got[t, j] - want[t, j]).max() < 0.02


def test_strided_tensors_and_another_stream():
    q_start, pages, n_pages = layout([2, 3], [40, 50], 16, 0)
    c = filled([40, 50], 2, 64, 16, pages, n_pages, 1)
    wide = torch.randn(8, 5, 72, generator=torch.Generator().manual_seed(1)).half().cuda()
    q = wide[1:6, :4, 8:72]
    want, wl = kv_ref.attend(q.double().cpu().numpy(), c, q_start, [40, 50], pages, 2)
    room = torch.full((4, 5, 64), 5.0, dtype=torch.float16, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, lse = attend(c, q, q_start, [40, 50], pages, 2, 16, 64, "f16", stream=side, out=room.transpose(0, 1))
    check(got, lse, want, wl, "f16", 4.0, "strided")


def test_bound_larger_than_the_contexts():
    # max_q and max_kv are upper bounds: a captured call serves later, shorter batches
    q_start, pages, n_pages = layout([1, 3], [40, 50], 16, 0)
    pages = np.concatenate([pages, np.zeros((2, 60), np.int32)], 1)
    c = filled([40, 50], 2, 64, 16, pages, n_pages, 1)
    q = torch.randn(4, 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    want, wl = kv_ref.attend(q.double().numpy(), c, q_start, [40, 50], pages, 2)
    with bsg.KVPlan(4, 2, 64, 16, n_pages, 64) as plan:
        out, lse = torch.zeros(4, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 4, device="cuda")
        for max_q, max_kv in ((3, 50), (4, 1000), (4, 64)):
            plan.attend(bsg.KVBatch(dev(q_start), dev(np.array([40, 50], np.int32)), dev(pages), 4, max_q, max_kv), q.cuda(),
                        dev(c.bytes), out, lse=lse)
            torch.cuda.synchronize()
            check(out.double().cpu().numpy(), lse.double().cpu().numpy(), want, wl, "bf16", 4.0, f"bounds {max_q} {max_kv}")


def test_numbers_outside_the_cache_are_harmless():
    # lengths and page numbers beyond what the host was told: nothing is read or written out of bounds
    c = kv_ref.Cache(4, 1, 64, 16)
    room = torch.zeros(3 * c.stride + c.bytes.size, dtype=torch.uint8, device="cuda")
    cache = room[c.stride: c.stride + c.bytes.size]
    pages = dev(np.array([[2, -7, 1 << 30], [9, 4, 3]], np.int32))
    x = torch.ones(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    with bsg.KVPlan(2, 1, 64, 16, 4, 8) as plan:
        for lens in ([1, 1], [40, 48], [1 << 30, -5], [33, 18]):
            b = bsg.KVBatch(dev(np.array([0, 1, 2], np.int32)), dev(np.array(lens, np.int32)), pages, 2, 1, 48)
            plan.append(b, x[:, :1], x[:, :1], cache, q=x, q_out=x.clone())
            plan.attend(b, x, cache, x.clone())
            plan.read(b, cache, x[:, :1].clone(), x[:, :1].clone())
            torch.cuda.synchronize()
    outside = torch.cat((room[: c.stride], room[c.stride + c.bytes.size:]))
    assert not outside.any()


def test_attend_in_a_graph():
    q_start, pages, n_pages = layout([1, 1], [700, 50], 16, 0)
    c = filled([700, 50], 2, 64, 16, pages, n_pages, 1)
    cache, pg, qs = dev(c.bytes), dev(pages), dev(q_start)
    lens = dev(np.array([700, 50], np.int32))
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    out = torch.zeros_like(q)
    with bsg.KVPlan(4, 2, 64, 16, n_pages, 64) as plan:
        batch = bsg.KVBatch(qs, lens, pg, 2, 1, 700)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            plan.attend(batch, q, cache, out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            plan.attend(batch, q, cache, out)
        for n in (700, 333, 1, 64):
            lens.copy_(torch.tensor([n, 50 - n % 50]))
            eager = torch.zeros_like(q)
            plan.attend(batch, q, cache, eager)
            torch.cuda.synchronize()
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, eager), n


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "f16")])
@pytest.mark.parametrize("kw", [{}, {"window": 300}, {"causal": False}], ids=str)
@pytest.mark.parametrize("new,lens,G", [([9], [1500], 4), ([40, 3, 0, 21], [700, 64, 900, 129], 8), ([65, 10], [1100, 12], 2)])
def test_many_rows_in_parts(new, lens, G, D, dtype, kw):
    # few row blocks over long contexts: positions are split, some parts are empty for the shorter sequences
    run_case(new, lens, H=1, G=G, D=D, dtype=dtype, P=32, seed=len(lens) + G, **kw)


@pytest.mark.parametrize("D,dtype,G", [(128, "bf16", 4), (64, "f16", 20)])
@pytest.mark.parametrize("kw", [{}, {"window": 40}, {"causal": False}], ids=str)
@pytest.mark.parametrize("new,lens", [
    ([60, 1, 1], [150, 300, 17]),                                         # one prompt, single tokens
    ([1, 3, 0, 45, 8, 9, 1, 33, 2], [700, 3, 40, 45, 8, 200, 0, 90, 65]),  # either side of the kernels' limit, empty ones
    ([1] * 30 + [34] + [1] * 30, [5 + 7 * i for i in range(61)]),
])
def test_mixed_batches(new, lens, D, dtype, G, kw):
    run_case(new, lens, H=1, G=G, D=D, dtype=dtype, seed=len(lens) + G, **kw)


def test_nan_blocks_in_one_part():
    def poison(c, pages):
        c.part(pages[0][1000 // 16], 0, 3)[1, 1000 % 16] = 0x7F
        c.part(pages[0][1195 // 16], 1, 3)[3, 1195 % 16] = 0x7F
    got, _ = run_case([20, 1], [1200, 20], seed=17, edit=poison)
    assert np.isnan(got[:20, :4, 16:32]).all() and not np.isnan(got[0, 4:]).any() and np.isnan(got[15, 4:, 48:64]).all()
    got, _ = run_case([20, 1], [1200, 20], seed=18, edit=poison, window=190)
    assert np.isnan(got[9, :4, 16:32]).all() and not np.isnan(got[10, :4]).any()


@pytest.mark.parametrize("new,H,D,dtype", [(40, 512, 64, "f16"), (150, 256, 128, "bf16")])
@pytest.mark.parametrize("P,window", [(16, 0), (16, 1100), (128, 0)])
def test_many_rows_over_many_pages_in_one_part(new, H, D, dtype, P, window):
    # heads enough for every compute unit: one workgroup walks a whole context, past the pages it looks up at first.
    # The cache is filled by append and its values are taken from read (both checked above byte by byte).
    n = 1301
    g = torch.Generator().manual_seed(new)
    q_start, pages, n_pages = layout([n], [n], P, 7)
    lens, pg = dev(np.array([n], np.int32)), dev(pages)
    print(f"[kv] many pages {new} {H} {D} {dtype} {P} {window}", flush=True)
    with bsg.KVPlan(H, H, D, P, n_pages, n, dtype=dtype, window=window) as plan:
        kv = [torch.randn(n, H, D, generator=g).to(DT[dtype]).cuda() for _ in range(2)]
        cache = torch.full((n_pages * plan.page_bytes,), 0x7F, dtype=torch.uint8, device="cuda")
        whole = bsg.KVBatch(dev(q_start), lens, pg, n, n, n)
        plan.append(whole, *kv, cache)
        plan.read(whole, cache, *kv)
        q = torch.randn(new, H, D, generator=g).to(DT[dtype]).cuda()
        out, lse = torch.zeros_like(q), torch.zeros(new, H, device="cuda")
        plan.attend(bsg.KVBatch(dev(np.array([0, new], np.int32)), lens, pg, new, new, n), q, cache, out, lse=lse)
        torch.cuda.synchronize()
    qd, k, v = (x.double().transpose(0, 1).contiguous() for x in (q, *kv))
    s = torch.matmul(qd, k.transpose(1, 2).contiguous()) * D ** -0.5
    i, j = torch.arange(n - new, n, device="cuda")[:, None], torch.arange(n, device="cuda")[None]
    s = s.masked_fill((j > i) | (j <= i - window if window else j < 0), float("-inf"))
    want = torch.matmul(s.softmax(-1), v).transpose(0, 1)
    check(out.double().cpu().numpy(), lse.double().cpu().numpy(), want.cpu().numpy(), s.logsumexp(-1).T.cpu().numpy(), dtype,
          float(v.abs().max()), f"many pages {new} {H} {D} {P} {window}")


def test_many_rows_in_parts_in_a_graph():
    q_start, pages, n_pages = layout([30, 20], [900, 500], 16, 0)
    c = filled([900, 500], 2, 64, 16, pages, n_pages, 1)
    cache, pg, qs = dev(c.bytes), dev(pages), dev(q_start)
    lens = dev(np.array([900, 500], np.int32))
    q = torch.randn(50, 8, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    out = torch.zeros_like(q)
    with bsg.KVPlan(8, 2, 64, 16, n_pages, 64) as plan:
        batch = bsg.KVBatch(qs, lens, pg, 50, 30, 900)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            plan.attend(batch, q, cache, out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            plan.attend(batch, q, cache, out)
        for n in (900, 333, 30, 64):
            lens.copy_(torch.tensor([n, n // 2]))
            eager = torch.zeros_like(q)
            plan.attend(batch, q, cache, eager)
            torch.cuda.synchronize()
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, eager), n


# ------------------------------------------------------------------------------------------------ append
def append_case(new, lens, H, G, D, P, dtype, rope, interleaved, seed, k_scale=1.0, v_scale=1.0, special=None, scaling=None):
    q_start, pages, n_pages = layout(new, lens, P, seed)
    T = int(q_start[-1])
    rng = np.random.default_rng(seed)
    qkv = torch.from_numpy(rng.standard_normal((T, (G + 2) * H, D)) * np.exp2(rng.integers(-12, 6, (T, (G + 2) * H, 1)))).to(DT[dtype])
    if special is not None:
        special(qkv)
    qkv = qkv.cuda()
    q, k, v = qkv[:, : G * H], qkv[:, G * H: (G + 1) * H], qkv[:, (G + 1) * H:]
    table = bsg.rope_table(max(lens), rope, scaling=scaling) if rope else None
    c = kv_ref.Cache(n_pages, H, D, P, 0x55)
    cache = dev(c.bytes)
    q_out = torch.zeros(T, G * H, D, dtype=DT[dtype], device="cuda")
    back = torch.zeros(2, T, H, D, dtype=DT[dtype], device="cuda")
    print(f"[kv append] new={new} lens={lens} H={H} G={G} D={D} P={P} {dtype} rope={rope} {interleaved}", flush=True)
    with bsg.KVPlan(G * H, H, D, P, n_pages, max(T, len(lens)), dtype=dtype, rope_dim=rope, k_scale=k_scale, v_scale=v_scale,
                    rope_layout="interleaved" if interleaved else "half") as plan:
        batch = bsg.KVBatch(dev(q_start), dev(np.asarray(lens, np.int32)), dev(pages), T, max(new), max(lens))
        plan.append(batch, k, v, cache, q=q, q_out=q_out, rope=None if table is None else dev(table))
        plan.read(batch, cache, back[0], back[1])
        in_place = q.clone()
        plan.append(batch, k, v, cache, q=in_place, q_out=in_place, rope=None if table is None else dev(table))
        torch.cuda.synchronize()
    place = kv_ref.positions(q_start, lens)
    pos = np.array([p for _, p in place])
    rq = kv_ref.rotate(q.float().cpu().numpy(), pos, table, interleaved)
    rk = kv_ref.rotate(k.float().cpu().numpy(), pos, table, interleaved)
    assert torch.equal(torch.from_numpy(rq).to(DT[dtype]).view(torch.int16), q_out.cpu().view(torch.int16)) or special is not None
    assert torch.equal(in_place.view(torch.int16), q_out.view(torch.int16))
    for which, x, g in ((0, rk, k_scale), (1, v.float().cpu().numpy(), v_scale)):
        code, s = kv_ref.quantize(x, g)
        for t, (b, p) in enumerate(place):
            for h in range(H):
                c.store(pages[b][p // P], p % P, h, which == 1, code[t, h], s[t, h])
        held = torch.from_numpy(kv_ref.values(code, s, g).astype(np.float32)).to(DT[dtype])
        got = back[which].cpu()
        assert torch.equal(torch.nan_to_num(held.float(), 1e9), torch.nan_to_num(got.float(), 1e9))
    got = cache.cpu().numpy()
    nan = None
    if special is not None:  # codes of a NaN block mean nothing
        mine, theirs = kv_ref.Cache(n_pages, H, D, P), kv_ref.Cache(n_pages, H, D, P)
        mine.bytes[:], theirs.bytes[:] = got, c.bytes
        for b, p in place:
            for h in range(H):
                for is_v in (False, True):
                    a, e = (x.load(pages[b][p // P], p % P, h, is_v) for x in (mine, theirs))
                    assert np.array_equal(a, e, equal_nan=True)
                    nan = True if np.isnan(e).any() else nan
        assert nan
    else:
        assert np.array_equal(got, c.bytes), int((got != c.bytes).sum())


@pytest.mark.parametrize("D,rope", [(64, 0), (64, 64), (64, 32), (64, 16), (128, 128), (128, 64), (128, 48), (128, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_bytes(D, rope, dtype, interleaved):
    append_case([1, 5, 0, 40, 17], [9, 5, 3, 100, 33], 2, 2, D, 16, dtype, rope, interleaved, seed=D + rope)


@pytest.mark.parametrize("P", [16, 32, 128, 256])
@pytest.mark.parametrize("n", [1, 300])
def test_append_pages_and_many_sequences(P, n):
    append_case([1] * n, [1 + (i * 13) % 70 for i in range(n)], 1, 3, 64, P, "bf16", 64, False, seed=P + n)


def test_append_scales_and_long_context_tables():
    append_case([3, 2], [30, 2000], 2, 1, 128, 64, "bf16", 128, False, seed=1, k_scale=0.125, v_scale=4.0,
                scaling=("parts", 4.0, 512))
    append_case([3, 2], [30, 20], 2, 1, 128, 64, "f16", 128, True, seed=2, k_scale=0.3, v_scale=0.7, scaling=("linear", 2.0))


def test_append_zero_infinite_and_nan_blocks():
    def special(x):
        x[0, 2, :16] = 0
        x[0, 3, :16] = -0.0
        x[1, 2, 0], x[1, 3, 17] = float("inf"), float("-inf")
        x[2, 2, 5], x[2, 3, 40] = float("nan"), float("nan")
        x[3, 3, :] = 1e-30 if x.dtype == torch.bfloat16 else 0
        x[3, 2, :] = 3e38 if x.dtype == torch.bfloat16 else 6e4
    for dtype in ("bf16", "f16"):
        append_case([5], [20], 1, 2, 64, 16, dtype, 0, False, seed=3, special=special)


def test_every_scale_and_every_halfway_point():
    # value blocks whose largest element makes each E4M3 scale, with elements on and beside E2M1's halfway points
    scales = kv_ref.E4M3[1:]
    half = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    rows = []
    for s in scales:
        rows.append(np.concatenate([[6.0 * s], half * s, -half * s, [0.0]]))
    x = np.array(rows).astype(np.float32).reshape(-1, 16)
    x = np.concatenate([x, np.nextafter(x, np.float32(0)), np.nextafter(x, np.float32(np.inf))])
    x = x[: len(x) // 4 * 4].reshape(-1, 1, 64)
    x = torch.from_numpy(x).half().float().numpy()  # fp16 inputs: exact for the points themselves
    T = len(x)
    q_start, pages, n_pages = layout([T], [T], 64, 0)
    c = kv_ref.Cache(n_pages, 1, 64, 64)
    cache = dev(c.bytes)
    with bsg.KVPlan(1, 1, 64, 64, n_pages, T, dtype="f16") as plan:
        t = torch.from_numpy(x).half().cuda()
        plan.append(bsg.KVBatch(dev(q_start), dev(np.array([T], np.int32)), dev(pages), T, T, T), t, t, cache)
        torch.cuda.synchronize()
    code, s = kv_ref.quantize(x)
    for p in range(T):
        for is_v in (False, True):
            c.store(pages[0][p // 64], p % 64, 0, is_v, code[p, 0], s[p, 0])
    assert np.array_equal(cache.cpu().numpy(), c.bytes)


def test_append_then_attend_token_by_token_equals_the_prompt_at_once():
    # a prompt appended and attended in one call, in chunks, and token by token: the same cache, nearly the same outputs
    H, G, D, P, n = 2, 2, 64, 16, 75
    q_start, pages, n_pages = layout([n], [n], P, 0)
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn(n, (G + 2) * H, D, generator=g).bfloat16().cuda()
    table, pg = dev(bsg.rope_table(n, D)), dev(pages)
    got = []
    with bsg.KVPlan(G * H, H, D, P, n_pages, n, rope_dim=D) as plan:
        for chunk in (n, 20, 1):
            cache = torch.full((n_pages * plan.page_bytes,), 0x7F, dtype=torch.uint8, device="cuda")
            out = torch.zeros(n, G * H, D, dtype=torch.bfloat16, device="cuda")
            for a in range(0, n, chunk):
                z = min(n, a + chunk)
                b = bsg.KVBatch(dev(np.array([0, z - a], np.int32)), dev(np.array([z], np.int32)), pg, z - a, z - a, z)
                x = qkv[a:z]
                q = torch.empty(z - a, G * H, D, dtype=torch.bfloat16, device="cuda")
                plan.append(b, x[:, G * H:(G + 1) * H], x[:, (G + 1) * H:], cache, q=x[:, : G * H], q_out=q, rope=table)
                plan.attend(b, q, cache, out[a:z])
            torch.cuda.synchronize()
            got.append((cache.cpu(), out.float().cpu()))
    for cache, out in got[1:]:
        used = sorted(pages[0].tolist())
        size = len(cache) // n_pages
        full = [p for p in used if p != pages[0][n // P]]  # the last page is partly unused
        for p in full:
            assert torch.equal(cache[p * size:(p + 1) * size], got[0][0][p * size:(p + 1) * size])
        assert (out - got[0][1]).abs().max() <= 2.0 ** -6


# ------------------------------------------------------------------------------------------------ refusals
@pytest.mark.parametrize("change,status", [
    (dict(q_heads=3), "BSG_ERR_SHAPE"), (dict(kv_heads=0), "BSG_ERR_SHAPE"), (dict(head_dim=96), "BSG_ERR_UNSUPPORTED"),
    (dict(page_tokens=24), "BSG_ERR_UNSUPPORTED"), (dict(page_tokens=8), "BSG_ERR_UNSUPPORTED"), (dict(num_pages=0), "BSG_ERR_SHAPE"),
    (dict(max_tokens=0), "BSG_ERR_SHAPE"), (dict(rope_dim=24), "BSG_ERR_SHAPE"), (dict(rope_dim=256), "BSG_ERR_SHAPE"),
    (dict(window=-1), "BSG_ERR_SHAPE"), (dict(window=4, causal=False), "BSG_ERR_UNSUPPORTED"), (dict(page_stride=100), "BSG_ERR_SHAPE"),
    (dict(page_stride=(1 << 20) + 8), "BSG_ERR_ALIGN"), (dict(k_scale=-1.0), "BSG_ERR_SHAPE"), (dict(v_scale=float("nan")), "BSG_ERR_SHAPE"),
    (dict(softcap=float("inf")), "BSG_ERR_SHAPE"), (dict(scale=float("nan")), "BSG_ERR_SHAPE"),
])
def test_plan_refusals(change, status):
    kw = dict(q_heads=4, kv_heads=2, head_dim=64, page_tokens=16, num_pages=4, max_tokens=8) | change
    with pytest.raises(bsg.BsgError) as e:
        bsg.KVPlan(**kw)
    assert e.value.status_name == status


def test_call_refusals():
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    with bsg.KVPlan(4, 2, 64, 16, 4, 8, rope_dim=64) as plan:
        cache = torch.zeros(4 * plan.page_bytes + 16, dtype=torch.uint8, device="cuda")
        qs, ln, pg = dev(np.array([0, 1, 2], np.int32)), dev(np.array([3, 4], np.int32)), dev(np.zeros((2, 2), np.int32))
        good = bsg.KVBatch(qs, ln, pg, 2, 1, 32)
        rope = torch.zeros(32, 2, 32, device="cuda")

        def refused(status, f):
            with pytest.raises(bsg.BsgError) as e:
                f()
            assert e.value.status_name == status, e.value

        refused("BSG_ERR_SHAPE", lambda: plan.attend(bsg.KVBatch(qs, ln, pg, 2, 1, 33), x, cache, x))   # pages too few
        refused("BSG_ERR_SHAPE", lambda: plan.attend(bsg.KVBatch(qs, ln, pg, 2, 0, 32), x, cache, x))
        refused("BSG_ERR_SHAPE", lambda: plan.attend(bsg.KVBatch(qs, ln, pg, 2, 3, 32), x, cache, x))
        refused("BSG_ERR_SHAPE", lambda: plan.attend(bsg.KVBatch(qs, ln, pg, 9, 9, 32), x[:1].expand(9, 4, 64), cache, x[:1].expand(9, 4, 64)))
        refused("BSG_ERR_ALIGN", lambda: plan.attend(good, x, cache[1:], x))
        refused("BSG_ERR_NULL", lambda: plan.attend(good, x, None, x))
        refused("BSG_ERR_NULL", lambda: plan.append(good, k, k, cache))                                 # no table
        refused("BSG_ERR_SHAPE", lambda: plan.append(good, k, k, cache, rope=rope[:31]))
        refused("BSG_ERR_NULL", lambda: plan.append(good, k, k, cache, q=x, rope=rope))                 # q without q_out
        flat = torch.zeros(2 * 4 * 64 + 8, dtype=torch.bfloat16, device="cuda")
        refused("BSG_ERR_ALIGN", lambda: plan.attend(good, flat[4:4 + 512].view(2, 4, 64), cache, x))
        odd = torch.zeros(2, 4, 68, dtype=torch.bfloat16, device="cuda")[..., :64]
        refused("BSG_ERR_ALIGN", lambda: plan.attend(good, odd, cache, x))
        for f in (lambda: plan.attend(good, x[:1], cache, x), lambda: plan.attend(good, x.transpose(1, 2), cache, x),
                  lambda: plan.append(good, k, k, cache, rope=rope[..., :31]), lambda: bsg.KVBatch(qs[:2], ln, pg, 2, 1, 32)):
            with pytest.raises(ValueError):
                f()
        plan.attend(good, x, cache, x.clone())  # still usable
        torch.cuda.synchronize()
