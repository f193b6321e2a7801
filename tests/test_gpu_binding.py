"""What the Python binding refuses before the library is called: tensors that are too small, or of another type."""
import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_amd as bsg
from test_gpu_kv import dev
from test_gpu_moe import weights_of

pytestmark = pytest.mark.gpu


def kv_calls(plan, batch, x, k, cache):
    return (lambda: plan.append(batch, k, k, cache), lambda: plan.attend(batch, x, cache, x.clone()),
            lambda: plan.read(batch, cache, k.clone(), k.clone()))


@pytest.mark.parametrize("page_stride", [0, 4096])
def test_caches_that_are_too_small(page_stride):
    x, k = (torch.zeros(2, h, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    batch = bsg.KVBatch(dev(np.array([0, 1, 2], np.int32)), dev(np.array([3, 4], np.int32)), dev(np.zeros((2, 1), np.int32)), 2, 1, 16)
    with bsg.KVPlan(4, 2, 64, 16, 4, 8, page_stride=page_stride) as plan:
        assert plan.page_bytes == bsg.kv_page_bytes(2, 64, 16) and plan.page_stride == (page_stride or plan.page_bytes)
        need = 3 * plan.page_stride + plan.page_bytes
        whole = torch.zeros(2 * need, dtype=torch.uint8, device="cuda")
        for cache in (whole[:need - 16], whole[::2], whole[:need // 2 // 2 * 2].view(torch.int16)):
            for f in kv_calls(plan, batch, x, k, cache):
                with pytest.raises(ValueError):
                    f()
        for cache in (whole[:need], whole[:need].view(torch.int16), whole.data_ptr()):
            for f in kv_calls(plan, batch, x, k, cache):
                f()
        torch.cuda.synchronize()


def test_page_tables_that_end_before_max_kv():
    # a view of a wider table: its rows' stride would cover 64 positions, its columns hold 32
    x, k = (torch.zeros(2, h, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    pages = dev(np.zeros((2, 4), np.int32))
    starts, lens = dev(np.array([0, 1, 2], np.int32)), dev(np.array([3, 4], np.int32))
    with bsg.KVPlan(4, 2, 64, 16, 4, 8) as plan:
        cache = torch.zeros(4 * plan.page_bytes, dtype=torch.uint8, device="cuda")
        for f in kv_calls(plan, bsg.KVBatch(starts, lens, pages[:, :2], 2, 1, 33), x, k, cache):
            with pytest.raises(bsg.BsgError) as e:
                f()
            assert e.value.status_name == "BSG_ERR_SHAPE"
        for f in kv_calls(plan, bsg.KVBatch(starts, lens, pages[:, :2], 2, 1, 32), x, k, cache):
            f()
        torch.cuda.synchronize()


@pytest.mark.parametrize("dtype,other", [("bf16", torch.float16), ("f16", torch.bfloat16)])
def test_tensors_of_another_type(dtype, other):
    own = torch.bfloat16 if dtype == "bf16" else torch.float16
    batch = bsg.KVBatch(dev(np.array([0, 1, 2], np.int32)), dev(np.array([3, 4], np.int32)), dev(np.zeros((2, 1), np.int32)), 2, 1, 16)
    with bsg.KVPlan(4, 2, 64, 16, 4, 8, dtype=dtype) as plan:
        cache = torch.zeros(4 * plan.page_bytes, dtype=torch.uint8, device="cuda")
        for t in (other, torch.float32):
            for f in kv_calls(plan, batch, *(torch.zeros(2, h, 64, dtype=t, device="cuda") for h in (4, 2)), cache):
                with pytest.raises(ValueError):
                    f()
        for t in (own, torch.int16):
            for f in kv_calls(plan, batch, *(torch.zeros(2, h, 64, dtype=t, device="cuda") for h in (4, 2)), cache):
                f()
        torch.cuda.synchronize()
    w = {k: dev(v) for k, v in weights_of("nvfp4", 2, 64, 32, 0).items()}
    a = (w["w13"], w["s13"], w["w2"], w["s2"])
    x, router = torch.zeros(2, 64, dtype=own, device="cuda"), torch.zeros(2, 64, dtype=own, device="cuda")
    with bsg.MoEPlan("nvfp4", 2, 1, 64, 32, 2, dtype=dtype) as plan:
        for args in ((x.to(other), router, *a, x.clone()), (x, router.to(other), *a, x.clone()), (x, router, *a, x.to(other))):
            with pytest.raises(ValueError):
                plan.run(*args)
        plan.run(x, router, *a, x.clone())
        plan.run(x.view(torch.int16), router, *a, x.clone())
        torch.cuda.synchronize()


def test_other_32_bit_numbers():
    x, k = (torch.zeros(2, h, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    batch = bsg.KVBatch(dev(np.array([0, 1, 2], np.int32)), dev(np.array([3, 4], np.int32)), dev(np.zeros((2, 1), np.int32)), 2, 1, 16)
    ints, floats = torch.int32, torch.float32
    with bsg.KVPlan(4, 2, 64, 16, 4, 8, rope_dim=64) as plan:
        cache = torch.zeros(4 * plan.page_bytes, dtype=torch.uint8, device="cuda")
        for f in (lambda: plan.append(batch, k, k, cache, rope=torch.zeros(16, 2, 32, dtype=ints, device="cuda")),
                  lambda: plan.attend(batch, x, cache, x.clone(), lse=torch.zeros(2, 4, dtype=ints, device="cuda"))):
            with pytest.raises(ValueError):
                f()
    w = {k: dev(v) for k, v in weights_of("nvfp4", 2, 64, 32, 0).items()}
    x, router = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    with bsg.MoEPlan("nvfp4", 2, 1, 64, 32, 2) as plan:
        for name, n, t in (("alpha13", 2, ints), ("alpha2", 2, ints), ("ids", 2, floats), ("weights", 2, ints)):
            with pytest.raises(ValueError):
                plan.run(x, router, w["w13"], w["s13"], w["w2"], w["s2"], x.clone(), **{name: torch.zeros(n, dtype=t, device="cuda")})
