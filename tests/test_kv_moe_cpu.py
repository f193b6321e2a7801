"""Paged cache, attention and expert layer without a GPU: refusals through the C ABI (all decided before a device is
touched), the rotation table, and pins of the 64-bit references that the GPU tests compare with."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_amd as bsg
import kv_ref
import moe_ref
import seeded_inputs as si

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = {name: code for code, name in bsg.STATUS.items()}


def create(cls, create_fn, values, change):
    prob = cls(**(dict(struct_size=ctypes.sizeof(cls)) | values | change))
    h = ctypes.c_void_p(1)
    st = getattr(bsg.load_library(), create_fn)(ctypes.byref(prob), ctypes.byref(h))
    assert not h.value
    return bsg.STATUS[st]


KV = dict(dtype=1, q_heads=8, kv_heads=2, head_dim=64, page_tokens=16, num_pages=4, page_stride=0, max_tokens=8, flags=0,
          rope_dim=0, window=0, scale=0.0, softcap=0.0, k_scale=1.0, v_scale=1.0, device=-1)
MOE = dict(format=1, dtype=1, flags=0, experts=8, top_k=2, hidden=64, inter=64, max_tokens=4, device=-1, reserved=0)


@pytest.mark.parametrize("change,status", [
    (dict(struct_size=8), "BSG_ERR_ABI"), (dict(dtype=0), "BSG_ERR_ABI"), (dict(flags=4), "BSG_ERR_ABI"),
    (dict(q_heads=7), "BSG_ERR_SHAPE"), (dict(kv_heads=0), "BSG_ERR_SHAPE"), (dict(kv_heads=2048, q_heads=2048), "BSG_ERR_SHAPE"),
    (dict(head_dim=80), "BSG_ERR_UNSUPPORTED"), (dict(head_dim=0), "BSG_ERR_SHAPE"), (dict(page_tokens=48), "BSG_ERR_UNSUPPORTED"),
    (dict(page_tokens=512), "BSG_ERR_UNSUPPORTED"), (dict(num_pages=0), "BSG_ERR_SHAPE"), (dict(num_pages=1 << 31), "BSG_ERR_SHAPE"),
    (dict(max_tokens=0), "BSG_ERR_SHAPE"), (dict(max_tokens=1 << 25), "BSG_ERR_SHAPE"), (dict(page_stride=-16), "BSG_ERR_SHAPE"),
    (dict(page_stride=4104), "BSG_ERR_ALIGN"),
    (dict(rope_dim=8), "BSG_ERR_SHAPE"), (dict(rope_dim=80), "BSG_ERR_SHAPE"), (dict(window=-2), "BSG_ERR_SHAPE"),
    (dict(window=3, flags=2), "BSG_ERR_UNSUPPORTED"), (dict(scale=float("inf")), "BSG_ERR_SHAPE"),
    (dict(softcap=-1.0), "BSG_ERR_SHAPE"), (dict(k_scale=1e-40), "BSG_ERR_SHAPE"), (dict(v_scale=float("nan")), "BSG_ERR_SHAPE"),
])
def test_kv_plan_refusals(change, status):
    assert create(bsg.KVProblem, "bsg_kv_plan_create", KV, change) == status


@pytest.mark.parametrize("change,status", [
    (dict(struct_size=8), "BSG_ERR_ABI"), (dict(format=3), "BSG_ERR_ABI"), (dict(dtype=0), "BSG_ERR_ABI"),
    (dict(flags=2), "BSG_ERR_ABI"), (dict(reserved=1), "BSG_ERR_ABI"), (dict(experts=0), "BSG_ERR_SHAPE"),
    (dict(top_k=0), "BSG_ERR_SHAPE"), (dict(top_k=9), "BSG_ERR_SHAPE"), (dict(hidden=48), "BSG_ERR_SHAPE"),
    (dict(inter=0), "BSG_ERR_SHAPE"), (dict(max_tokens=0), "BSG_ERR_SHAPE"), (dict(max_tokens=65), "BSG_ERR_UNSUPPORTED"),
    (dict(experts=513), "BSG_ERR_UNSUPPORTED"), (dict(top_k=17, experts=32), "BSG_ERR_UNSUPPORTED"),
    (dict(hidden=65568), "BSG_ERR_UNSUPPORTED"),
])
def test_moe_plan_refusals(change, status):
    assert create(bsg.MoEProblem, "bsg_moe_plan_create", MOE, change) == status


def test_null_and_foreign_handles():
    lib, block = bsg.load_library(), ctypes.create_string_buffer(8192)
    fake = ctypes.addressof(block)
    null = CODE["BSG_ERR_NULL"]
    assert lib.bsg_kv_plan_create(None, None) == null and lib.bsg_moe_plan_create(None, None) == null
    for h in (None, fake):
        assert lib.bsg_kv_append(h, *[None] * 6, 0, None, None) == null
        assert lib.bsg_kv_attend(h, *[None] * 6) == null
        assert lib.bsg_kv_read(h, *[None] * 5) == null
        assert lib.bsg_kv_plan_query(h, None) == null
        assert lib.bsg_moe_run(h, 1, None, 0, None, None, 0, None, None, None) == null
    assert lib.bsg_kv_plan_destroy(None) == 0 and lib.bsg_moe_plan_destroy(None) == 0
    assert lib.bsg_kv_plan_destroy(fake) == null and lib.bsg_moe_plan_destroy(fake) == null


def test_other_architectures_are_refused():
    code = ("import block_scaled_precision_gemm_amd as b\n"
            "for make in (lambda: b.KVPlan(8, 2, 64, 16, 4, 8), lambda: b.MoEPlan('nvfp4', 8, 2, 64, 64, 4)):\n"
            "    try: make()\n"
            "    except b.BsgError as e: assert e.status_name == 'BSG_ERR_DEVICE', e\n"
            "    else: raise SystemExit('made')\n")
    env = dict(os.environ, BSG_FORCE_ARCH="gfx942", PYTHONPATH=ROOT)
    subprocess.run([sys.executable, "-c", code], env=env, check=True, timeout=120)


def test_page_bytes():
    assert bsg.kv_page_bytes(8, 128, 64) == 8 * 64 * 128 * 9 // 8
    assert bsg.kv_page_bytes(1, 64, 16) == 16 * 64 * 9 // 8
    for bad in ((0, 64, 16), (1, 96, 16), (1, 64, 24), (1, 64, 512)):
        assert bsg.kv_page_bytes(*bad) == 0


# ------------------------------------------------------------------------------------------------ rotation table
def test_rope_table():
    t = bsg.rope_table(50, 16, base=100.0)
    assert t.shape == (50, 2, 8) and t.dtype == np.float32
    for p in (0, 1, 49):
        for i in range(8):
            a = p * 100.0 ** (-i / 8)
            assert t[p, 0, i] == np.float32(np.cos(a)) and t[p, 1, i] == np.float32(np.sin(a))
    assert np.abs(bsg.rope_table(100001, 32)[100000, 0, 0] - np.cos(100000.0)) < 1e-7  # 64-bit angles


def test_rope_table_scalings():
    plain = bsg.rope_table(200, 32)
    assert np.allclose(bsg.rope_table(200, 32, scaling=("linear", 4.0))[4::4], plain[1:50], atol=1e-6)
    angle = np.arctan2(*(bsg.rope_table(2, 32, scaling=("base", 8.0))[1, i] for i in (1, 0)))
    own = 10000.0 ** (-np.arange(16) / 16)
    assert np.isclose(angle[0], own[0]) and np.isclose(angle[-1], own[-1] / 8)  # the fastest as it was, the slowest by f
    t = bsg.rope_table(2, 64, scaling=("parts", 4.0, 4096))
    gain, own = 1 + 0.1 * np.log(4.0), 10000.0 ** (-np.arange(32) / 32)
    angle, turns = np.arctan2(t[1, 1], t[1, 0]), own * 4096 / (2 * np.pi)
    assert np.allclose(np.hypot(t[1, 0], t[1, 1]), gain)
    assert np.allclose(angle[turns >= 32], own[turns >= 32], rtol=1e-5)
    assert np.allclose(angle[turns <= 1], own[turns <= 1] / 4, rtol=1e-5)
    mid = (turns < 32) & (turns > 1)
    assert mid.any() and (angle[mid] <= own[mid] * (1 + 1e-5)).all() and (angle[mid] >= own[mid] / 4 * (1 - 1e-5)).all()
    for bad in (("cubic", 2.0),):
        with pytest.raises(ValueError):
            bsg.rope_table(8, 16, scaling=bad)
    for rows, dim in ((0, 16), (4, 15), (4, 0)):
        with pytest.raises(ValueError):
            bsg.rope_table(rows, dim)


# ------------------------------------------------------------------------------------------------ references
def test_reference_formats_against_torch():
    codes = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(codes.view(torch.float8_e4m3fn).double().numpy(), kv_ref.E4M3)
    x = torch.from_numpy(np.random.default_rng(0).uniform(0, 448, 4000))
    x = torch.cat((x, torch.from_numpy((kv_ref.E4M3[1:] + kv_ref.E4M3[:-1]) / 2)))  # the halfway points: ties to even
    want = x.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(kv_ref.nearest(x.float().double().numpy(), kv_ref.E4M3), want)
    mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    assert list(kv_ref.nearest(mid, kv_ref.E2M1)) == [0, 2, 2, 4, 4, 6, 6]


def test_reference_blocks_are_the_librarys_operands():
    from oracle.oracle import dequant_nvfp4
    x = np.random.default_rng(1).standard_normal((40, 64)).astype(np.float32) * 3
    code, s = kv_ref.quantize(x)
    held = kv_ref.values(code, s)
    assert np.array_equal(dequant_nvfp4(code[:, 0::2] | code[:, 1::2] << 4, s, 64), held)
    # the block's largest element becomes 6 scales, and a scale is off by at most 2^-4: half of E2M1's widest step
    # (of 2, between 4 and 6), or what is clipped above 6
    step = np.repeat(np.abs(x).reshape(40, 4, 16).max(-1) / 6, 16, 1)
    assert (np.abs(held - x) <= step * (1 + 2.0 ** -4)).all()


def test_reference_attention_against_torch():
    rng = np.random.default_rng(2)
    H, G, D, P, lens, new = 2, 3, 64, 16, [40, 17], [5, 17]
    pages = np.array([[3, 0, 2], [1, 4, 0]], np.int32)
    c = kv_ref.Cache(5, H, D, P)
    k, v = rng.standard_normal((2, 2, 40, H, D))
    for b in range(2):
        for h in range(H):
            for x, is_v in ((k, False), (v, True)):
                code, s = kv_ref.quantize(x[b, : lens[b], h])
                x[b, : lens[b], h] = kv_ref.values(code, s)
                for p in range(lens[b]):
                    c.store(pages[b][p // P], p % P, h, is_v, code[p], s[p])
    q = rng.standard_normal((22, H * G, D))
    got, lse = kv_ref.attend(q, c, np.array([0, 5, 22]), lens, pages, H, window=9)
    at = 0
    for b, n in enumerate(new):
        qb = torch.from_numpy(q[at:at + n]).transpose(0, 1)
        kb, vb = (torch.from_numpy(x[b, : lens[b]]).transpose(0, 1).repeat_interleave(G, 0) for x in (k, v))
        i, j = torch.arange(n)[:, None] + lens[b] - n, torch.arange(lens[b])[None]
        s = (qb @ kb.mT / 8).masked_fill((j > i) | (j <= i - 9), float("-inf"))
        assert np.allclose((s.softmax(-1) @ vb).transpose(0, 1).numpy(), got[at:at + n], atol=1e-12)
        assert np.allclose(s.logsumexp(-1).T.numpy(), lse[at:at + n], atol=1e-12)
        at += n


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp8"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_reference_experts_against_torch(fmt, renormalize):
    from oracle.oracle import dequant_mxfp8, dequant_nvfp4
    rng = np.random.default_rng(3)
    E, H, I, T, K = 4, 64, 32, 5, 2
    parts = {k: [] for k in ("w13", "s13", "w2", "s2", "d13", "d2")}
    for _ in range(E):
        for w, s, d, shape in (("w13", "s13", "d13", (2 * I, H)), ("w2", "s2", "d2", (H, I))):
            x = rng.standard_normal(shape).astype(np.float32)
            codes, scales = (si.quantize_nvfp4(x) if fmt == "nvfp4" else si.quantize_mxfp8(x))[:2]
            parts[w].append(codes)
            parts[s].append(scales)
            parts[d].append(dequant_nvfp4(codes, scales, shape[1]) if fmt == "nvfp4" else dequant_mxfp8(codes, scales))
    p = {k: np.stack(v) for k, v in parts.items()}
    x, router = rng.standard_normal((T, H)), rng.standard_normal((E, H))
    got, ids, weights = moe_ref.moe(fmt, x, router, p["w13"], p["s13"], p["w2"], p["s2"], K, renormalize=renormalize)
    xt = torch.from_numpy(x)
    prob = (xt @ torch.from_numpy(router).T).softmax(-1)
    top, at = prob.topk(K)
    top = top / top.sum(-1, keepdim=True) if renormalize else top
    assert np.array_equal(at.numpy(), ids) and np.allclose(top.numpy(), weights, atol=1e-12)
    dense = torch.zeros(T, E, dtype=torch.float64).scatter(1, at, top)
    h = torch.matmul(xt, torch.from_numpy(p["d13"]).mT)  # [E][T][2 I]
    h = torch.nn.functional.silu(h[..., :I]) * h[..., I:]
    want = (torch.matmul(h, torch.from_numpy(p["d2"]).mT) * dense.T[..., None]).sum(0)
    assert np.allclose(want.numpy(), got, rtol=1e-10, atol=1e-10)
