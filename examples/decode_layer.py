"""One decoder layer served with the library: prompts of uneven lengths enter together, then every sequence
decodes token by token.

    python examples/decode_layer.py [--seqs 3] [--prompt 130] [--steps 32]

A step of the layer, on whatever new tokens its sequences have:
  1. query, key and value projection            Plan (MXFP8 GEMM)
  2. rotary positions, keys and values stored   KVPlan.append (paged NVFP4 cache)
  3. attention over everything stored           KVPlan.attend
  4. output projection                          Plan (MXFP8 GEMM)
  5. expert layer                               MoEPlan.run (NVFP4 experts)
Norms, residuals and the activations' quantisation are plain torch.  Weights are random.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import block_scaled_precision_gemm_amd as bsg  # noqa: E402


def to_mxfp8(x):
    """[rows][K] -> E4M3 codes [rows][K] and E8M0 scale codes [rows][K / 32] (uint8)."""
    blocks = x.float().unflatten(-1, (-1, 32))
    exponent = torch.frexp(blocks.abs().amax(-1)).exponent - 9  # largest magnitude to [256, 512)
    exponent = exponent.clamp(-127, 127)
    codes = torch.ldexp(blocks, -exponent[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).flatten(-2), (exponent + 127).to(torch.uint8)


def to_nvfp4(x):
    """[..., K] -> packed E2M1 codes [..., K / 2] and E4M3 scale codes [..., K / 16] (uint8)."""
    blocks = x.float().unflatten(-1, (-1, 16))
    scale = (blocks.abs().amax(-1) / 6).clamp(2.0 ** -9, 448).to(torch.float8_e4m3fn)
    size = blocks.abs() / scale.float()[..., None]
    halfway = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    codes = (torch.bucketize(size, halfway) + 8 * (blocks < 0)).to(torch.uint8).flatten(-2)
    return codes[..., ::2] | codes[..., 1::2] << 4, scale.view(torch.uint8)


def norm(x):
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class Linear:
    """x W^T with W in MXFP8; a plan for each number of rows."""

    def __init__(self, w):
        self.n, self.k = w.shape
        self.w, self.s = to_mxfp8(w)
        self.plans = {}

    def __call__(self, x):
        m = x.shape[0]
        if m not in self.plans:
            self.plans[m] = bsg.Plan("mxfp8", m, self.n, self.k)
        a, sa = to_mxfp8(x)
        y = torch.empty(m, self.n, dtype=torch.bfloat16, device=x.device)
        self.plans[m].run(a, self.w, sa, self.s, y)
        return y


class Pages:
    """Which pages each sequence owns; a page is taken when a sequence grows into it."""

    def __init__(self, seqs, page_tokens, num_pages, max_kv):
        self.page_tokens, self.max_kv = page_tokens, max_kv
        self.free = list(range(num_pages))[::-1]
        self.owned = [[] for _ in range(seqs)]
        self.lens = [0] * seqs

    def grow(self, new):
        """The KVBatch of new[b] more tokens for each sequence."""
        for b, n in enumerate(new):
            self.lens[b] += n
            while len(self.owned[b]) * self.page_tokens < self.lens[b]:
                self.owned[b].append(self.free.pop())
        width = max(map(len, self.owned))
        table = torch.tensor([p + [0] * (width - len(p)) for p in self.owned], dtype=torch.int32)
        starts = torch.tensor([0] + new).cumsum(0).int()
        return bsg.KVBatch(starts.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda(), table.cuda(), sum(new), max(new),
                           max(self.lens))


class Layer:
    def __init__(self, hidden, q_heads, kv_heads, head_dim, experts, top_k, inter, page_tokens, num_pages, max_tokens, max_kv,
                 seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weights(*shape):
            return torch.randn(*shape, generator=g, device="cuda") * shape[-1] ** -0.5

        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.qkv = Linear(weights((q_heads + 2 * kv_heads) * head_dim, hidden))
        self.o = Linear(weights(hidden, q_heads * head_dim))
        self.router = weights(experts, hidden).bfloat16()
        self.w13, self.s13 = to_nvfp4(weights(experts, 2 * inter, hidden))
        self.w2, self.s2 = to_nvfp4(weights(experts, hidden, inter))
        self.kv = bsg.KVPlan(q_heads, kv_heads, head_dim, page_tokens, num_pages, max_tokens, rope_dim=head_dim)
        self.moe = bsg.MoEPlan("nvfp4", experts, top_k, hidden, inter, 64)
        self.cache = torch.zeros(num_pages * self.kv.page_bytes, dtype=torch.uint8, device="cuda")
        self.rope = torch.from_numpy(bsg.rope_table(max_kv, head_dim)).cuda()

    def attention(self, qkv, batch):
        qkv = qkv.view(-1, self.q_heads + 2 * self.kv_heads, self.head_dim)
        q, k, v = qkv.split((self.q_heads, self.kv_heads, self.kv_heads), 1)
        self.kv.append(batch, k, v, self.cache, q=q, q_out=q, rope=self.rope)
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        self.kv.attend(batch, q, self.cache, out)
        return out.flatten(1)

    def experts(self, x):
        out = torch.empty_like(x)
        for t in range(0, x.shape[0], 64):  # a prompt passes in groups of tokens
            self.moe.run(x[t:t + 64], self.router, self.w13, self.s13, self.w2, self.s2, out[t:t + 64])
        return out

    def __call__(self, x, batch):
        x = x + self.o(self.attention(self.qkv(norm(x)), batch))
        return x + self.experts(norm(x))


def serve(layer, pages, prompts, steps, x):
    """Prompts (their lengths) in one call, then `steps` single tokens per sequence.  Synthetic: a sequence's next
    input is the norm of its last output.  Returns the outputs of every call."""
    batch = pages.grow(prompts)
    outs = [layer(x, batch)]
    last = torch.tensor(prompts).cumsum(0).cuda() - 1
    for _ in range(steps):
        x = norm(outs[-1][last])
        outs.append(layer(x, pages.grow([1] * len(prompts))))
        last = torch.arange(len(prompts), device=x.device)
    return outs


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--seqs", type=int, default=3)
    ap.add_argument("--prompt", type=int, default=130, help="tokens of the longest prompt")
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    prompts = [max(1, a.prompt * (i + 1) // a.seqs) for i in range(a.seqs)]
    max_kv, page = a.prompt + 2 * a.steps + 1, 16
    num_pages = 2 * a.seqs * -(-max_kv // page)
    layer = Layer(2048, 32, 8, 64, 32, 4, 1024, page, num_pages, max(sum(prompts), a.seqs), max_kv)
    x = torch.randn(sum(prompts), 2048, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    serve(layer, Pages(a.seqs, page, num_pages, max_kv), prompts, 2, x)  # plans made, kernels loaded
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    outs = serve(layer, Pages(a.seqs, page, num_pages, max_kv), prompts, a.steps, x)
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t0) * 1e3
    print(f"{a.seqs} prompts of up to {a.prompt} tokens and {a.steps} steps: {ms:.2f} ms; "
          f"mean magnitude of the last output {outs[-1].float().abs().mean().item():.3f}")


if __name__ == "__main__":
    main()
