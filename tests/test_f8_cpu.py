"""E4M3 products with a scale for each block of 128 without a GPU: refusals through the C ABI, which are decided before a
device is touched, and pins of the 64-bit reference that the GPU tests compare with."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_amd as bsg
import f8_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = {name: code for code, name in bsg.STATUS.items()}
PLAN = dict(dtype=1, flags=0, device=-1, n=64, k=64, max_tokens=8)
FFN = dict(dtype=1, flags=0, device=-1, hidden=64, inter=64, max_tokens=8)


def create(cls, fn, values):
    h = ctypes.c_void_p(1)
    st = getattr(bsg.load_library(), fn)(ctypes.byref(cls(**(dict(struct_size=ctypes.sizeof(cls)) | values))), ctypes.byref(h))
    assert not h.value
    return bsg.STATUS[st]


@pytest.mark.parametrize("change,status", [
    (dict(struct_size=8), "BSG_ERR_ABI"), (dict(dtype=0), "BSG_ERR_ABI"), (dict(dtype=3), "BSG_ERR_ABI"), (dict(flags=2), "BSG_ERR_ABI"),
    (dict(n=0), "BSG_ERR_SHAPE"), (dict(n=24), "BSG_ERR_SHAPE"), (dict(n=-16), "BSG_ERR_SHAPE"), (dict(k=8), "BSG_ERR_SHAPE"),
    (dict(k=(1 << 18) + 16), "BSG_ERR_SHAPE"), (dict(n=1 << 40), "BSG_ERR_SHAPE"), (dict(max_tokens=0), "BSG_ERR_SHAPE"),
    (dict(max_tokens=(1 << 24) + 1), "BSG_ERR_SHAPE"),
])
def test_plan_refusals(change, status):
    assert create(bsg.F8Problem, "bsg_f8_plan_create", PLAN | change) == status
    ffn = {dict(n="hidden", k="inter").get(k, k): v for k, v in change.items()}
    assert create(bsg.F8FFNProblem, "bsg_f8_ffn_plan_create", FFN | ffn) == status


def test_a_feed_forward_plan_has_no_flags():
    assert create(bsg.F8FFNProblem, "bsg_f8_ffn_plan_create", FFN | dict(flags=1)) == "BSG_ERR_ABI"


@pytest.mark.parametrize("flags", [3, 5, 8, 12, 1 << 31])
def test_unknown_flags(flags):
    if flags != 5:  # (5: a bias and exact products)
        assert create(bsg.F8Problem, "bsg_f8_plan_create", PLAN | dict(flags=flags)) == "BSG_ERR_ABI"
    assert create(bsg.F8FFNProblem, "bsg_f8_ffn_plan_create", FFN | dict(flags=flags)) == "BSG_ERR_ABI"


GOOD = dict(dtype=1, rows=3, cols=144, x=4096, x_stride=144, codes=8192, codes_stride=144, scales=16384, scale_stride=4)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=0), "BSG_ERR_ABI"), (dict(rows=-1), "BSG_ERR_SHAPE"), (dict(rows=(1 << 24) + 1), "BSG_ERR_SHAPE"),
    (dict(cols=0), "BSG_ERR_SHAPE"), (dict(cols=140), "BSG_ERR_SHAPE"), (dict(x=None), "BSG_ERR_NULL"), (dict(codes=None), "BSG_ERR_NULL"),
    (dict(scales=None), "BSG_ERR_NULL"), (dict(x=4104), "BSG_ERR_ALIGN"), (dict(x_stride=148), "BSG_ERR_ALIGN"),
    (dict(x_stride=136), "BSG_ERR_SHAPE"), (dict(x_stride=-144), "BSG_ERR_SHAPE"), (dict(x_stride=1 << 22), "BSG_ERR_SHAPE"),
    (dict(codes=8200), "BSG_ERR_ALIGN"), (dict(codes_stride=152), "BSG_ERR_ALIGN"), (dict(codes_stride=128), "BSG_ERR_SHAPE"),
    (dict(scales=16386), "BSG_ERR_ALIGN"), (dict(scale_stride=6), "BSG_ERR_ALIGN"), (dict(scale_stride=0), "BSG_ERR_SHAPE"),
    (dict(scale_stride=1 << 25), "BSG_ERR_SHAPE"),
])
def test_quantize_refusals(change, status):
    assert bsg.STATUS[bsg.load_library().bsg_f8_quantize(*(GOOD | change).values(), None)] == status


def test_no_rows_are_nothing_to_do():
    assert bsg.load_library().bsg_f8_quantize(*(GOOD | dict(rows=0, x=None)).values(), None) == 0


def test_null_and_foreign_handles():
    lib, block = bsg.load_library(), ctypes.create_string_buffer(8192)
    fake, null = ctypes.addressof(block), CODE["BSG_ERR_NULL"]
    assert lib.bsg_f8_plan_create(None, None) == null and lib.bsg_f8_ffn_plan_create(None, None) == null
    n = ctypes.c_uint64()
    for h in (None, fake):
        assert lib.bsg_f8_run(h, 1, None, None, None, None, None, 0, None) == null
        assert lib.bsg_f8_ffn_run(h, 1, None, 0, None, None, 0, None) == null
        assert lib.bsg_f8_plan_workspace(h, ctypes.byref(n)) == null and lib.bsg_f8_ffn_plan_workspace(h, ctypes.byref(n)) == null
        assert lib.bsg_kv_attend_shared(h, None, 16, None, None, None, None, None) == null
    assert lib.bsg_f8_plan_destroy(None) == 0 and lib.bsg_f8_ffn_plan_destroy(None) == 0
    assert lib.bsg_f8_plan_destroy(fake) == null and lib.bsg_f8_ffn_plan_destroy(fake) == null


def test_other_architectures_are_refused():
    code = ("import block_scaled_precision_gemm_amd as b\n"
            "for make in (lambda: b.F8Plan(64, 64, 4), lambda: b.F8FFNPlan(64, 64, 4)):\n"
            "    try: make()\n"
            "    except b.BsgError as e: assert e.status_name == 'BSG_ERR_DEVICE', e\n"
            "    else: raise SystemExit('made')\n")
    env = dict(os.environ, BSG_FORCE_ARCH="gfx942", PYTHONPATH=ROOT)
    subprocess.run([sys.executable, "-c", code], env=env, check=True, timeout=120)


def test_scales_shape():
    assert bsg.f8_scales_shape(1, 16) == (1, 4) and bsg.f8_scales_shape(8, 129) == (2, 8) and bsg.f8_scales_shape(0, 128) == (1, 0)


N, K = 272, 144  # (blocks: 3 and 2)


@pytest.mark.parametrize("w,s", [((N, K), (3, 2)), ((2, N // 2, K), (3, 2)), ((N * K,), (6,)), ((N * K,), (3, 2)), ((N, K), (3, 1, 2))])
def test_weights_as_they_lie(w, s):
    bsg._f8_weights((("w", torch.zeros(w, dtype=torch.uint8), torch.ones(s), (N, K), (3, 2)),), torch.float32)


@pytest.mark.parametrize("w,s", [((K, N), (3, 2)), ((N, K), (2, 3)), ((N, K // 2, 2), (3, 2)), ((N, K), (6, 1)), ((1, N * K), (3, 2)),
                                 ((N, K), (1, 6)), ((N, K), (3, 3)), ((N, K + 16), (3, 2))])
def test_weights_of_another_layout_are_refused(w, s):
    # a contiguous [k][n] matrix has as many codes as [n][k], and would be multiplied as other weights
    with pytest.raises(ValueError, match="codes or bytes .272, 144."):
        bsg._f8_weights((("w", torch.zeros(w, dtype=torch.uint8), torch.ones(s), (N, K), (3, 2)),), torch.float32)


# ------------------------------------------------------------------------------------------------ reference
def test_reference_values_against_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.nan_to_num(ref.values(codes.numpy()), nan=9e9), np.nan_to_num(want, nan=9e9))


def test_reference_quantize_against_torch():
    x = torch.randn(50, 400, generator=torch.Generator().manual_seed(0)).bfloat16()
    codes, scales = ref.quantize(x.double().numpy())
    for b in range(4):
        part = x[:, 128 * b:128 * b + 128].float()
        s = torch.from_numpy(scales[b]).float()[:, None]
        assert (part.abs().amax(1, keepdim=True) <= 448 * s).all() and (part.abs().amax(1, keepdim=True) > 224 * s).all()
        assert np.array_equal((part / s).to(torch.float8_e4m3fn).view(torch.uint8).numpy(), codes[:, 128 * b:128 * b + 128])


def test_reference_block_against_torch():
    g = torch.Generator().manual_seed(1)
    x, w1, w3, w2 = (torch.randn(s, generator=g).double() / 8 for s in ((5, 144), (272, 144), (272, 144), (144, 272)))
    want, off = ref.ffn(x.numpy(), w1.numpy(), w3.numpy(), w2.numpy())

    def q(v):
        out = torch.empty_like(v)
        for a in range(0, v.shape[1], 128):
            b = v[:, a:a + 128]
            s = torch.exp2(torch.ceil(torch.log2(b.abs().amax(1, keepdim=True) / 448)))
            out[:, a:a + 128] = (b / s).float().to(torch.float8_e4m3fn).double() * s
        return out

    got = q(torch.nn.functional.silu(q(x) @ w1.T) * (q(x) @ w3.T)) @ w2.T
    assert (np.abs(got.numpy() - want) <= off + 1e-12).all()
    # The bound says something.  A sum of 144 may be off by 148 2^-24 of its magnitudes, some 12 times its value: 1e-4.  A step
    # of a code is 9% of a value, so 0.25% of the inner values have two possible codes; 272 of them, 9% of each added up
    # without signs, against a sum of random signs, are 272 * 0.0025 * 0.09 / 272^0.5 = 0.4% of it: bf16's half step.
    assert np.median(off / np.abs(want)) < 2.0 ** -8


@pytest.mark.parametrize("kind", [torch.float8_e5m2, torch.bool])
def test_codes_of_other_types_are_refused(kind):
    # E5M2 has the size of E4M3, and would be taken for other numbers
    x, codes = torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(4, 32, dtype=torch.uint8).view(kind)
    with pytest.raises(ValueError, match="E4M3"):
        bsg.f8_quantize(x, codes, torch.zeros(bsg.f8_scales_shape(4, 32)))
