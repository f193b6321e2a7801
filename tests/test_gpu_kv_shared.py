"""Attention for batches that share their first positions, on the GPU against the 64-bit reference of kv_ref: the sizes and
masks where the shared part's kernel, the few-row kernel behind it and their join can go wrong."""
import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_amd as bsg
import kv_ref
from test_gpu_kv import DT, check, dev, filled

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def small_cases_are_shared_too(monkeypatch):
    monkeypatch.setenv("BSG_FORCE_SHARED", "1")


def layout(new, lens, shared, P, seed):
    """q_start, pages (the first shared / P of every row the same) and the number of pages."""
    rng = np.random.default_rng(seed)
    common = shared // P
    own = [max(0, -(-n // P) - common) for n in lens]
    order = rng.permutation(np.arange(1, common + sum(own) + 3)).astype(np.int32)
    pages = np.zeros((len(lens), common + max(own + [1])), np.int32)
    pages[:, :common] = order[:common]
    at = common
    for b, n in enumerate(own):
        pages[b, common:common + n] = order[at:at + n]
        at += n
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32), pages, common + sum(own) + 3


def held(lens, shared, H, D, P, pages, n_pages, seed):
    """A cache whose used slots hold quantised Gaussians, the shared ones written once."""
    c = filled([max(list(lens) + [shared])], H, D, P, [list(pages[int(np.argmax(lens))])], n_pages, seed)
    rest = [n if b != int(np.argmax(lens)) else 0 for b, n in enumerate(lens)]
    rng = np.random.default_rng(seed + 7)
    for b, n in enumerate(rest):
        for h in range(H if n > shared else 0):
            for is_v in (False, True):
                code, s = kv_ref.quantize(rng.standard_normal((n - shared, D)))
                for p in range(shared, n):
                    c.store(pages[b][p // P], p % P, h, is_v, code[p - shared], s[p - shared])
    return c


def run(c, q, q_start, lens, pages, shared, H, P, D, dtype, max_q=None, stream=None, **kw):
    T, hq = q.shape[:2]
    with bsg.KVPlan(hq, H, D, P, len(c.bytes), max(T, len(lens)), dtype=dtype, **kw) as plan:
        batch = bsg.KVBatch(dev(q_start), dev(np.asarray(lens, np.int32)), dev(pages), T, max_q or int(np.diff(q_start).max()),
                            max(max(lens), shared))
        cache, out = dev(c.bytes), torch.full((T, hq, D), 7.0, dtype=DT[dtype], device="cuda")
        lse = torch.full((T, hq), 7.0, dtype=torch.float32, device="cuda")
        first = None
        for _ in range(3):  # the workspace's counters are back at zero, and sums have one order
            out.fill_(7.0)
            plan.attend(batch, q, cache, out, lse=lse, stream=stream, shared=shared)
            torch.cuda.synchronize()
            first = out.clone() if first is None else first
            assert torch.equal(torch.nan_to_num(out.float(), 9e9), torch.nan_to_num(first.float(), 9e9)), "not deterministic"
            plan.attend(batch, q, cache, out)  # an ordinary call in between uses the same workspace
        torch.cuda.synchronize()
        return first.double().cpu().numpy(), lse.double().cpu().numpy()


def case(new, lens, shared, H=2, G=4, D=128, P=16, dtype="bf16", seed=0, edit=None, q_gain=1.0, **kw):
    q_start, pages, n_pages = layout(new, lens, shared, P, seed)
    c = held(lens, shared, H, D, P, pages, n_pages, seed + 1)
    if edit:
        edit(c, pages)
    q = torch.from_numpy(np.random.default_rng(seed + 2).standard_normal((int(q_start[-1]), H * G, D)) * q_gain).to(DT[dtype])
    want, want_lse = kv_ref.attend(q.double().numpy(), c, q_start, lens, pages, H, **kw)
    v_max = max([np.nanmax(np.abs(np.array([c.load(pages[b][p // P], p % P, h, True, kw.get("v_scale", 1.0)) for p in range(n)])), initial=0)
                 for b, n in enumerate(lens) for h in range(H)] + [0])
    label = f"new={new} lens={lens} shared={shared} H={H} G={G} D={D} P={P} {dtype} {kw}"
    print("[kv]", label, flush=True)
    got, lse = run(c, q.cuda(), q_start, lens, pages, shared, H, P, D, dtype, **kw)
    check(got, lse, want, want_lse, dtype, v_max, label)
    return got, lse


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "f16"), (128, "bf16")])
@pytest.mark.parametrize("P,shared", [(16, 16), (16, 48), (16, 64), (16, 80), (16, 1008), (32, 640), (64, 64), (256, 768)])
def test_one_token_each(P, shared, D, dtype):
    # own positions from one to beyond a tile; more rows than one block of 128 holds where the heads are 8 x 12
    case([1] * 12, [shared + n for n in (1, 2, 15, 16, 17, 63, 64, 65, 1, 130, 3, 300)], shared, D=D, P=P, dtype=dtype, seed=P + shared)


@pytest.mark.parametrize("H,G,seqs", [(1, 1, 40), (3, 1, 33), (1, 5, 9), (2, 8, 20), (1, 16, 3), (1, 32, 2), (1, 8, 70), (8, 4, 40), (1, 17, 4)])
def test_head_groups(H, G, seqs):
    case([1] * seqs, [96 + 1 + (7 * i) % 40 for i in range(seqs)], 96, H=H, G=G, D=64, seed=H * 100 + G)


@pytest.mark.parametrize("new", [[3, 1, 2, 8, 5, 1], [2] * 20, [1, 0, 7, 0, 0, 4, 3, 8, 0], [4] * 30])
@pytest.mark.parametrize("kw", [{}, {"causal": False}, {"softcap": 3.0}, {"scale": 0.3, "k_scale": 0.25, "v_scale": 3.0}], ids=str)
def test_several_tokens(new, kw):
    case(new, [160 + t + (11 * i) % 50 for i, t in enumerate(new)], 160, D=64, dtype="f16", seed=len(new), **kw)


@pytest.mark.parametrize("causal", [True, False])
def test_sequences_that_end_in_the_shared_positions(causal):
    # contexts that end before, at and just behind them, one without any, one shorter than its new tokens
    got, lse = case([1, 1, 1, 2, 3, 1, 2, 8], [0, 5, 100, 112, 113, 130, 1, 120], 112, seed=4, causal=causal)
    assert np.isneginf(lse[0]).all() and (got[0] == 0).all()
    case([8, 2, 8, 4], [112, 50, 111, 115], 112, seed=5, D=64, causal=causal)


def test_more_than_64_sequences_with_empty_ones():
    new = [0 if i % 3 == 0 else 1 + i % 4 for i in range(150)] + [0] * 90 + [2]
    case(new, [48 + t + i % 5 for i, t in enumerate(new)], 48, H=1, G=3, D=64, seed=6)


def test_calls_that_are_answered_as_ordinary_ones():
    case([1, 1], [200, 190], 160, H=1, G=4, seed=7)           # few rows in all
    case([1], [200], 160, H=1, G=40, seed=8)                  # one sequence
    case([40, 3], [250, 190], 160, H=1, G=4, seed=9)          # many rows of one sequence
    case([1] * 12, [200 + i for i in range(12)], 160, seed=10, window=50)
    case([1] * 12, [200 + i for i in range(12)], 0, seed=11)


def test_nan_blocks_reach_exactly_the_queries_that_see_them():
    def poison(c, pages):
        c.part(pages[0][30 // 16], 0, 3)[2, 30 % 16] = 0x7F  # value block 2 of shared position 30
        c.part(pages[1][100 // 16], 1, 2)[100 % 16, 1] = 0x7F  # a key block of sequence 1's own position 100
    lens = [97, 101, 31, 30, 20, 98, 150, 99, 98]
    got, _ = case([1] * 9, lens, 96, seed=13, edit=poison)
    for b in range(9):
        assert np.isnan(got[b, :4, 32:48]).all() == (lens[b] > 30) and not np.isnan(got[b, :4, :32]).any()
        assert np.isnan(got[b, 4:]).all() == (b == 1)
    case([5] * 4 + [3], [97, 104, 33, 30, 99], 96, seed=14, edit=poison)


def test_infinite_and_nan_queries_stay_in_their_rows():
    q_start, pages, n_pages = layout([1] * 10, [100] * 10, 96, 16, 0)
    c = held([100] * 10, 96, 1, 64, 16, pages, n_pages, 1)
    q = torch.randn(10, 4, 64, generator=torch.Generator().manual_seed(0)).bfloat16()
    q[0, 0, 3], q[7, 1, 3] = float("nan"), float("inf")
    want, want_lse = kv_ref.attend(q.double().numpy(), c, q_start, [100] * 10, pages, 1)
    got, lse = run(c, q.cuda(), q_start, [100] * 10, pages, 96, 1, 16, 64, "bf16")
    assert np.isnan(got[0, 0]).all()
    rest = np.ones((10, 4), bool)
    rest[0, 0] = rest[7, 1] = False
    check(got[rest], lse[rest], want[rest], want_lse[rest], "bf16", 4.0, "rest")


def test_one_position_takes_nearly_all_the_weight():
    case([1] * 12, [130 + i for i in range(12)], 96, seed=15, q_gain=300.0)
    case([1] * 12, [130 + i for i in range(12)], 96, seed=16, q_gain=1e-30)


def test_longer_prefix_in_many_parts_and_another_stream():
    lens = [4096 + 1 + 9 * i for i in range(10)]
    q_start, pages, n_pages = layout([1] * 10, lens, 4096, 64, 17)
    c = held(lens, 4096, 1, 64, 64, pages, n_pages, 18)
    q = torch.randn(10, 4, 64, generator=torch.Generator().manual_seed(2)).bfloat16()
    want, want_lse = kv_ref.attend(q.double().numpy(), c, q_start, lens, pages, 1)
    side = torch.cuda.Stream()
    q = q.cuda()
    torch.cuda.synchronize()
    got, lse = run(c, q, q_start, lens, pages, 4096, 1, 64, 64, "bf16", stream=side)
    check(got, lse, want, want_lse, "bf16", 4.0, "long")


def test_bounds_larger_than_the_batch():
    # max_q and max_kv are upper bounds, the page table wider than the contexts
    new, lens = [1, 3, 2, 1, 1, 2, 1], [100, 99, 130, 97, 98, 99, 100]
    q_start, pages, n_pages = layout(new, lens, 96, 16, 3)
    pages = np.concatenate([pages, np.full((7, 30), 1 << 30, np.int32)], 1)
    c = held(lens, 96, 2, 64, 16, pages, n_pages, 4)
    q = torch.randn(11, 16, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    want, want_lse = kv_ref.attend(q.double().numpy(), c, q_start, lens, pages, 2)
    with bsg.KVPlan(16, 2, 64, 16, n_pages, 40) as plan:
        batch = bsg.KVBatch(dev(q_start), dev(np.asarray(lens, np.int32)), dev(pages), 11, 4, 500)
        out, lse = torch.zeros(11, 16, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(11, 16, device="cuda")
        plan.attend(batch, q.cuda(), dev(c.bytes), out, lse=lse, shared=96)
        torch.cuda.synchronize()
    check(out.double().cpu().numpy(), lse.double().cpu().numpy(), want, want_lse, "bf16", 4.0, "bounds")


def test_a_captured_call_replays_with_growing_contexts():
    P, shared, seqs = 16, 96, 12
    last = [shared + 60] * seqs
    q_start, pages, n_pages = layout([1] * seqs, last, shared, P, 5)
    c = held(last, shared, 2, 64, P, pages, n_pages, 6)
    cache, gen = dev(c.bytes), torch.Generator().manual_seed(3)
    q = torch.randn(seqs, 8, 64, generator=gen).bfloat16().cuda()
    lens = torch.full((seqs,), shared + 1, dtype=torch.int32, device="cuda")
    with bsg.KVPlan(8, 2, 64, P, n_pages, seqs) as plan:
        batch = bsg.KVBatch(dev(q_start), lens, dev(pages), seqs, 1, max(last))
        out, lse = torch.zeros_like(q), torch.zeros(seqs, 8, device="cuda")
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            plan.attend(batch, q, cache, out, lse=lse, shared=shared)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            plan.attend(batch, q, cache, out, lse=lse, shared=shared)
        for step in (1, 2, 33, 60):
            lens.fill_(shared + step)
            lens[3] = shared - step if step < 60 else 0
            q.copy_(torch.randn(seqs, 8, 64, generator=gen).bfloat16())
            graph.replay()
            torch.cuda.synchronize()
            got = out.double().cpu().numpy(), lse.double().cpu().numpy()
            want, want_lse = kv_ref.attend(q.double().cpu().numpy(), c, q_start, lens.tolist(), pages, 2)
            check(*got, want, want_lse, "bf16", 4.0, step)


@pytest.mark.parametrize("D,new,dtype", [(128, 1, "bf16"), (64, 4, "f16")])
def test_the_choice_by_cost(monkeypatch, D, new, dtype):
    # without the switch: a long common beginning (read once) and a short one (not), the same results but for rounding
    monkeypatch.delenv("BSG_FORCE_SHARED")
    gen = torch.Generator(device="cuda").manual_seed(D)
    P, H, G, seqs = 64, 8, 4, 48
    for shared in (8192, 128):
        common, own = shared // P, 3
        n_pages = common + own * seqs
        pages = torch.cat((torch.arange(common, device="cuda").expand(seqs, common),
                           common + torch.arange(own * seqs, device="cuda").view(seqs, own)), 1).int().contiguous()
        lens = (shared + new + torch.arange(seqs, device="cuda") * 3 % 150).int()
        with bsg.KVPlan(H * G, H, D, P, n_pages, seqs * new, dtype=dtype) as plan:
            starts = torch.arange(0, seqs * new + 1, new, dtype=torch.int32, device="cuda")
            batch = bsg.KVBatch(starts, lens, pages, seqs * new, new, int(lens.max()))
            cache = torch.randint(0, 256, (n_pages * plan.page_bytes,), dtype=torch.uint8, device="cuda", generator=gen)
            chunk = cache.view(n_pages, H, -1)[:, :, P * D:]
            chunk.copy_(torch.randint(0x28, 0x40, chunk.shape, dtype=torch.uint8, device="cuda", generator=gen))  # scales
            q = torch.randn(seqs * new, H * G, D, device="cuda", generator=gen).to(DT[dtype])
            outs = [torch.empty_like(q) for _ in range(2)]
            lses = [torch.empty(seqs * new, H * G, device="cuda") for _ in range(2)]
            plan.attend(batch, q, cache, outs[0], lse=lses[0], shared=shared)
            plan.attend(batch, q, cache, outs[1], lse=lses[1])
            torch.cuda.synchronize()
        # both are within check()'s bound of the exact result
        v_max = 6 * 1.875
        a, b = (x.double() for x in outs)
        assert ((a - b).abs() <= 4 * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -11) * b.abs() + 2.0 ** -10 * v_max + 2e-7).all(), shared
        assert ((lses[0] - lses[1]).abs() <= 2 * (2e-5 + 2e-6 * lses[1].abs())).all(), shared


@pytest.mark.parametrize("shared", [-16, 8, 24, 128])
def test_refused_counts(shared):
    z = torch.zeros(2, 32, 64, dtype=torch.bfloat16, device="cuda")
    with bsg.KVPlan(32, 1, 64, 16, 9, 2) as plan:
        batch = bsg.KVBatch(dev(np.array([0, 1, 2], np.int32)), dev(np.array([99, 97], np.int32)), dev(np.zeros((2, 7), np.int32)), 2, 1, 100)
        with pytest.raises(bsg.BsgError) as e:
            plan.attend(batch, z, torch.zeros(9 * plan.page_bytes, dtype=torch.uint8, device="cuda"), z.clone(), shared=shared)
        assert e.value.status_name == "BSG_ERR_SHAPE"


def test_plans_with_a_window_have_no_room_for_shared_parts():
    """Positions are never shared under a window: such plans hold what either kernel needs, others both.  A window that no
    context reaches is none."""
    def bytes_of(**kw):
        with bsg.KVPlan(32, 8, 128, 16, 64, 512, **kw) as plan:
            return plan.info()["workspace_bytes"]

    few, rows = 512 * 2 * 32 * (128 + 4) * 4, 2 * 256 * 256 * (128 + 2) * 4  # parts on 256 CUs
    both, windowed = bytes_of(), bytes_of(window=1000)
    assert both - windowed == few and rows <= windowed < both
    assert bytes_of(window=(1 << 31) - 1) == both
