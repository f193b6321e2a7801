"""A layer of the E4M3 products around the paged cache, as a server would run it: a prompt that all sequences begin with,
their own first tokens, then single tokens, eagerly and from a captured graph.  Every stage is compared with its 64-bit
reference on the stage's own inputs."""
import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_amd as bsg
import f8_ref as ref
import kv_ref
import test_gpu_kv
from test_gpu_f8 import DT, check, dev, ffn_weights, weights

pytestmark = pytest.mark.gpu

HIDDEN, INTER, HQ, H, D, P, PREFIX, PAGES, MOST = 256, 272, 8, 2, 64, 16, 96, 64, 128
QKV = (HQ + 2 * H) * D


def np64(t):
    return t.double().cpu().numpy()


class Linear:
    """x [tokens][k] of 16 bits -> [tokens][n], by way of codes."""

    def __init__(self, n, k, seed, dtype):
        self.w, self.s = weights(n, k, seed, k ** -0.5)
        self.held, self.plan = (dev(self.w), dev(self.s)), bsg.F8Plan(n, k, MOST, dtype=dtype)
        self.codes = torch.empty(MOST, k, dtype=torch.uint8, device="cuda")
        self.scales = torch.empty(bsg.f8_scales_shape(MOST, k), device="cuda")

    def __call__(self, x, out):
        codes = self.codes[:len(x)]
        bsg.f8_quantize(x, codes, self.scales)
        self.plan.run(codes, self.scales, *self.held, out)
        return out

    def check(self, x, out, dtype, label):
        xv = ref.row_values(*ref.quantize(np64(x)))
        want, size = ref.product(xv, ref.weight_values(self.w, self.s))
        check(np64(out), want, ref.sum_bound(xv.shape[1], len(x) <= ref.FEW) * size, dtype, label)


class Layer:
    def __init__(self, dtype):
        self.dtype, kind = dtype, DT[dtype]
        self.qkv, self.o = Linear(QKV, HIDDEN, 1, dtype), Linear(HIDDEN, HQ * D, 2, dtype)
        self.kv = bsg.KVPlan(HQ, H, D, P, PAGES, MOST, dtype=dtype, rope_dim=D)
        self.rope = dev(bsg.rope_table(512, D))
        self.cache = torch.zeros(PAGES, self.kv.page_bytes, dtype=torch.uint8, device="cuda")
        self.ffn = bsg.F8FFNPlan(HIDDEN, INTER, MOST, dtype=dtype)
        held, self.ffn_values = ffn_weights(HIDDEN, INTER, 3)
        self.ffn_held = [dev(a) for a in held]
        self.buf = {n: torch.zeros(MOST, w, dtype=kind, device="cuda")
                    for n, w in (("qkv", QKV), ("a", HQ * D), ("o", HIDDEN), ("f", HIDDEN))}

    def __call__(self, x, batch, shared, seen=None):
        t = len(x)
        b = {n: v[:t] for n, v in self.buf.items()}
        heads = self.qkv(x, b["qkv"]).view(t, HQ + 2 * H, D)
        q, k, v = heads[:, :HQ], heads[:, HQ:HQ + H], heads[:, HQ + H:]
        if seen:
            seen("qkv", x, b["qkv"])
        self.kv.append(batch, k, v, self.cache, q=q, q_out=q, rope=self.rope)
        self.kv.attend(batch, q, self.cache, b["a"].view(t, HQ, D), shared=shared)
        if seen:
            seen("attention", q, b["a"].view(t, HQ, D))
        y = x + self.o(b["a"], b["o"])
        if seen:
            seen("o", b["a"], b["o"])
        self.ffn.run(y, *self.ffn_held, b["f"])
        if seen:
            seen("ffn", y, b["f"])
        return y + b["f"]


@pytest.mark.parametrize("dtype,seqs,force", [("bf16", 5, "1"), ("f16", 20, "1"), ("bf16", 20, "")])
def test_a_shared_prompt_then_single_tokens(monkeypatch, dtype, seqs, force):
    monkeypatch.setenv("BSG_FORCE_SHARED", force) if force else monkeypatch.delenv("BSG_FORCE_SHARED", raising=False)
    layer = Layer(dtype)
    g = torch.Generator().manual_seed(seqs)
    order = np.random.default_rng(seqs).permutation(np.arange(1, PAGES)).astype(np.int32)
    common = PREFIX // P
    pages = np.stack([np.concatenate((order[:common], order[common + 2 * b:common + 2 * b + 2])) for b in range(seqs)])

    def tokens(n):
        return torch.randn(n, HIDDEN, generator=g).to(DT[dtype]).cuda()

    def batch(q_start, lens, rows, max_kv):
        return bsg.KVBatch(dev(np.asarray(q_start, np.int32)), dev(np.asarray(lens, np.int32)), dev(rows), int(q_start[-1]),
                           int(np.diff(q_start).max()), max_kv)

    def step(x, q_start, lens, rows, shared):
        def seen(name, got_x, got):
            torch.cuda.synchronize()
            label = f"{name} {dtype} tokens={len(x)} shared={shared}"
            print("[layer]", label, flush=True)
            if name in ("qkv", "o"):
                getattr(layer, name).check(got_x, got, dtype, label)
            elif name == "ffn":
                check(np64(got), *ref.ffn(np64(got_x), *layer.ffn_values), dtype, label)
            else:
                c = kv_ref.Cache(PAGES, H, D, P)
                c.bytes[:] = layer.cache.cpu().numpy()
                want, lse = kv_ref.attend(np64(got_x), c, q_start, lens, rows, H)
                v_max = max(np.abs(c.load(rows[b][p // P], p % P, h, True)).max() for b, n in enumerate(lens) for p in range(n)
                            for h in range(H))
                test_gpu_kv.check(np64(got), lse, want, lse, dtype, v_max, label)
        out = layer(x, batch(q_start, lens, rows, max(lens)), shared, seen)
        torch.cuda.synchronize()
        assert out.isfinite().all(), "a layer of ordinary numbers stays finite"
        return out

    step(tokens(PREFIX), [0, PREFIX], [PREFIX], pages[:1, :common], 0)
    step(tokens(3 * seqs), np.arange(seqs + 1) * 3, [PREFIX + 3] * seqs, pages, PREFIX)
    lens = np.array([PREFIX + 3] * seqs)
    x = tokens(seqs)
    for _ in range(2):
        lens += 1
        x = step(x, np.arange(seqs + 1), lens.tolist(), pages, PREFIX)

    # The same step from a graph: every replay against the eager step on the same cache, which writes the same slots.
    starts = np.arange(seqs + 1)
    held = batch(starts, lens + 1, pages, PREFIX + 2 * P)
    kv_len, x_in = held._held[1], x.clone()
    layer(x_in, held, PREFIX)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        x_out = layer(x_in, held, PREFIX)
    for i in range(4):
        lens += 1
        kv_len.copy_(torch.from_numpy(lens.astype(np.int32)))
        x_in.copy_(tokens(seqs))
        graph.replay()
        torch.cuda.synchronize()
        got, cache = x_out.clone(), layer.cache.clone()
        want = layer(x_in, held, PREFIX)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(cache, layer.cache), f"replay {i}"
