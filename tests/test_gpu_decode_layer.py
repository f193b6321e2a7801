"""The example layer end to end on the GPU: every stage against its 64-bit reference on the stage's own inputs."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import kv_ref
import moe_ref
from oracle.oracle import dequant_mxfp8

pytestmark = pytest.mark.gpu

ROOT = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..")


def example():
    spec = importlib.util.spec_from_file_location("decode_layer", os.path.join(ROOT, "examples", "decode_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def np64(x):
    return x.double().cpu().numpy()


def test_prompts_then_single_tokens():
    ex = example()
    prompts, steps, page, H, D, hidden = [70, 5, 33], 3, 16, 2, 64, 256
    layer = ex.Layer(hidden, 8, H, D, 8, 3, 64, page, 40, sum(prompts), 128)
    seen = []

    def watch(name, call):
        def wrapped(*a):
            held = [t.clone() if torch.is_tensor(t) else t for t in a]
            out = call(*a)
            seen.append((name, held, out.clone()))
            return out
        return wrapped

    layer.qkv, layer.o = watch("qkv", layer.qkv), watch("o", layer.o)
    layer.attention, layer.experts = watch("attention", layer.attention), watch("experts", layer.experts)
    pages = ex.Pages(3, page, 40, 128)
    linear = {"qkv": layer.qkv.__closure__, "o": layer.o.__closure__}
    linear = {k: next(c.cell_contents for c in v if isinstance(c.cell_contents, ex.Linear)) for k, v in linear.items()}
    x = torch.randn(sum(prompts), hidden, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    outs = ex.serve(layer, pages, prompts, steps, x)
    torch.cuda.synchronize()
    assert len(outs) == 1 + steps and len(seen) == 4 * len(outs) and all(o.isfinite().all() for o in outs)

    held, lens, starts = kv_ref.Cache(40, H, D, page, 0), [0, 0, 0], None
    table = layer.rope.cpu().numpy()
    for i, (name, args, out) in enumerate(seen):
        print("[layer]", i, name, flush=True)
        got = np64(out)
        if name in linear:
            a, sa = (t.cpu().numpy() for t in ex.to_mxfp8(args[0]))
            w, sw = (t.cpu().numpy() for t in (linear[name].w, linear[name].s))
            # exact operands, fp32 sums of at most 512 products, one rounding to bf16
            am, wm = dequant_mxfp8(a, sa), dequant_mxfp8(w, sw)
            want, mass = am @ wm.T, np.abs(am) @ np.abs(wm).T
            assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -14 * mass).all()
            # the activations' own quantisation: half a step of E4M3 (2^-4), or clipped to 448 of up to 512
            assert (np.abs(am - np64(args[0])).max() <= 2.0 ** -3 * np.abs(np64(args[0])).max())
        elif name == "attention":
            new = prompts if i < 4 else [1, 1, 1]
            lens = [n + m for n, m in zip(lens, new)]
            starts = np.concatenate([[0], np.cumsum(new)])
            place = kv_ref.positions(starts, lens)
            qkv = args[0].float().cpu().numpy().reshape(-1, 8 + 2 * H, D)
            pos = np.array([p for _, p in place])
            q = kv_ref.rotate(qkv[:, :8], pos, table, False)
            q = np64(torch.from_numpy(q).bfloat16())
            for which, rows in ((False, kv_ref.rotate(qkv[:, 8:8 + H], pos, table, False)), (True, qkv[:, 8 + H:])):
                code, s = kv_ref.quantize(rows)
                for t, (b, p) in enumerate(place):
                    for h in range(H):
                        held.store(pages.owned[b][p // page], p % page, h, which, code[t, h], s[t, h])
            owned = [o + [0] * 40 for o in pages.owned]
            want, _ = kv_ref.attend(q, held, starts, lens, owned, H)
            v_max = np.abs(qkv[:, 8 + H:]).max() * 1.25  # a value is at most half an E2M1 step above its own
            want = want.reshape(got.shape)  # weights held to 2^-12 and their sum to as much, one rounding to bf16
            assert (np.abs(got - want) <= 2.0 ** -7 * np.abs(want) + 2.0 ** -11 * v_max).all()
        else:
            w13, s13, w2, s2 = (t.cpu().numpy() for t in (layer.w13, layer.s13, layer.w2, layer.s2))
            want, _, _ = moe_ref.moe("nvfp4", np64(args[0]), np64(layer.router), w13, s13, w2, s2, 3)
            size = np.sqrt((want ** 2).mean(1, keepdims=True))  # SiLU(gate) up keeps 16 bits, sums are fp32
            assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -13 * size).all()
    for b, n in enumerate(pages.lens):
        assert n == prompts[b] + steps
    mine = kv_ref.Cache(40, H, D, page)
    mine.bytes[:] = layer.cache.cpu().numpy().reshape(mine.bytes.shape)
    assert np.array_equal(mine.bytes, held.bytes)
