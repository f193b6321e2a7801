"""Operators beside the block-scaled GEMM and the paged cache: cases, inputs, plain forms and their 64-bit values.

Eight-bit products for a decoder layer's projections and its feed-forward block, and attention for sequences that begin alike:

* quantize: 16-bit rows as E4M3 codes with one scale for each 128 columns of a row, the least power of two that fits;
* product: rows of codes and fp32 scales like these times weights in E4M3 with one fp32 scale for each 128 x 128 block, outputs in 16 bits;
* ffn: the gated feed-forward block over such weights, 16 bits in and out: gate and up, SiLU(gate) up in E4M3 again, down;
* attend: attention over a paged NVFP4 cache for a batch whose sequences share their first positions.

`own` False: plain torch in 32 bits, rounded once at the end.  `own` True: the library's operators.
"""
import math
import random

import torch

own = False

BLOCK = 128
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------------------------- cases
def _quantize(name, tokens, cols, dtype):
    return dict(name=name, op="quantize", tokens=tokens, cols=cols, dtype=dtype)


def _product(name, tokens, n, k, dtype, bias):
    return dict(name=name, op="product", tokens=tokens, n=n, k=k, dtype=dtype, bias=bias)


def _ffn(name, tokens, hidden, inter, dtype):
    return dict(name=name, op="ffn", tokens=tokens, hidden=hidden, inter=inter, dtype=dtype)


def _attend(name, seqs, tokens, shared, context, q_heads, kv_heads, dim, page, dtype):
    return dict(name=name, op="attend", seqs=seqs, tokens=tokens, shared=shared, context=context, q_heads=q_heads,
                kv_heads=kv_heads, dim=dim, page=page, dtype=dtype)


def listed():
    return [
        # one token before a projection: nothing but latency
        _quantize("quantize_one", 1, 4096, "bf16"),
        # a long prompt before a projection, an odd number of tokens
        _quantize("quantize_prompt", 8191, 8192, "bf16"),
        # one token through an attention projection
        _product("product_one", 1, 4096, 4096, "bf16", False),
        # a decode batch through a large projection: the weights' bytes count
        _product("product_batch", 61, 8192, 8192, "bf16", False),
        # some prompts' tokens, sizes that fill no tile, a bias
        _product("product_ragged", 1003, 2064, 4112, "f16", True),
        # a long prompt: arithmetic counts
        _product("product_prompt", 8192, 8192, 8192, "bf16", False),
        # one token through a small block: latency
        _ffn("ffn_one", 1, 2048, 4096, "bf16"),
        # a decode batch: the weights' bytes count
        _ffn("ffn_batch", 33, 4096, 8192, "bf16"),
        # a prompt, an odd number of tokens
        _ffn("ffn_prompt", 4095, 4096, 8192, "f16"),
        # a few chats after a short instruction, small pages
        _attend("shared_few", 7, 1, 1008, 300, 32, 8, 128, 16, "bf16"),
        # a serving batch that answers questions about one long document
        _attend("shared_batch", 64, 1, 16384, 2000, 64, 8, 128, 64, "bf16"),
        # the same with drafted tokens to check, small heads
        _attend("shared_verify", 24, 5, 4096, 1000, 32, 8, 64, 32, "f16"),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op, dtype = rng.choice(("quantize", "product", "product", "ffn", "ffn", "attend")), rng.choice(("bf16", "f16"))
    if op == "quantize":
        case = _quantize("", _log_int(rng, 1, 8191), 16 * _log_int(rng, 8, 512), dtype)
    elif op == "product":
        n, k = 16 * _log_int(rng, 16, 512), 16 * _log_int(rng, 16, 512)
        case = _product("", _log_int(rng, 1, 8192), n, k, dtype, rng.random() < 0.3)
    elif op == "ffn":
        case = _ffn("", _log_int(rng, 1, 4095), 16 * _log_int(rng, 32, 256), 16 * _log_int(rng, 32, 512), dtype)
    else:
        kv_heads, group, dim, page = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 8)), rng.choice((64, 128)), rng.choice((16, 32, 64))
        seqs, tokens = _log_int(rng, 2, 64), 1 if rng.random() < 0.6 else rng.randint(2, 8)
        case = _attend("", seqs, tokens, page * _log_int(rng, max(1, 128 // page), 16384 // page),
                       _log_int(rng, 16, 2000), kv_heads * group, kv_heads, dim, page, dtype)
    del case["name"]
    return case


def _contexts(case):
    """Positions of each sequence, the shared ones and its new tokens among them: a property of the case alone.  What
    lies behind the shared ones spreads over its logarithm up to `context`, which the first sequence has."""
    rng = random.Random("%d %d %d %d" % (case["seqs"], case["tokens"], case["shared"], case["context"]))
    t, most = case["tokens"], max(case["tokens"], case["context"])
    return [case["shared"] + (most if i == 0 else max(t, _log_int(rng, max(1, most // 16), most))) for i in range(case["seqs"])]


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    t = case.get("tokens")
    if case["op"] == "quantize":
        return {"bytes": t * (3 * case["cols"] + 4 * _blocks(case["cols"])), "flops": 4.0 * t * case["cols"]}
    if case["op"] == "product":
        n, k = case["n"], case["k"]
        return {"bytes": t * (k + 4 * _blocks(k)) + n * k + 4 * _blocks(n) * _blocks(k) + 2 * t * n + (4 * n if case["bias"] else 0),
                "flops": 2.0 * t * n * k}
    if case["op"] == "ffn":
        h, i = case["hidden"], case["inter"]
        return {"bytes": 4 * t * h + 3 * h * i + 12 * _blocks(h) * _blocks(i), "flops": 6.0 * t * h * i}
    lens, tokens, hq, hk, d = _contexts(case), case["seqs"] * t, case["q_heads"], case["kv_heads"], case["dim"]
    held = case["shared"] + sum(n - case["shared"] for n in lens)
    pairs = sum(n * t - t * (t - 1) // 2 for n in lens)
    return {"bytes": held * 2 * hk * d * 9 / 16 + tokens * hq * (4 * d + 4), "flops": 4.0 * hq * d * pairs}


# ---------------------------------------------------------------------------------------------- formats
def _wide(scales, n):
    """Scales of blocks as scales of elements along the last dimension, `n` of them."""
    return scales.repeat_interleave(BLOCK, -1)[..., :n]


def _row_blocks(x):
    """float32 rows [rows][cols] as E4M3 codes [rows][cols] with scales [blocks][rows] (plain)."""
    cols = x.shape[1]
    padded = torch.nn.functional.pad(x, (0, _blocks(cols) * BLOCK - cols)).unflatten(1, (-1, BLOCK))
    m, e = torch.frexp(padded.abs().amax(-1))
    e = (e - 9 + (m > 0.875).int()).clamp(min=-126)  # 448 = 0.875 * 2^9
    e = torch.where(m > 0, e, torch.full_like(e, -126))
    q = torch.ldexp(padded, -e[..., None])
    return q.flatten(1)[:, :cols].to(torch.float8_e4m3fn), torch.ldexp(torch.ones_like(m), e).t()


def _row_values(codes, scales):
    """float32 values of such rows (plain)."""
    return codes.float() * _wide(scales.t(), codes.shape[1])


def _tile_values(codes, scales):
    """float32 values of weights [n][k] with scales [n blocks][k blocks] (plain)."""
    return codes.float() * _wide(_wide(scales, codes.shape[1]).t(), codes.shape[0]).t()


def _tiles(x):
    """Weights [n][k] as E4M3 codes with a scale for each 128 x 128 block."""
    n, k = x.shape
    b = torch.nn.functional.pad(x, (0, _blocks(k) * BLOCK - k, 0, _blocks(n) * BLOCK - n))
    b = b.unflatten(0, (-1, BLOCK)).unflatten(2, (-1, BLOCK))
    s = (b.abs().amax((1, 3)) / 448.0).clamp(min=2.0 ** -100)
    q = (b / s[:, None, :, None]).clamp(-448.0, 448.0).flatten(2, 3).flatten(0, 1)[:n, :k]
    return q.to(torch.float8_e4m3fn), s


def _nvfp4(x):
    """NVFP4 blocks of the last dimension: packed codes and E4M3 scales."""
    b = x.float().unflatten(-1, (-1, 16))
    s = (b.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = s.float().unsqueeze(-1)
    z = torch.where(f > 0, b / f, torch.zeros_like(b)).abs()
    code = ((z > 0.25).to(torch.uint8) + (z >= 0.75) + (z > 1.25) + (z >= 1.75) + (z > 2.5) + (z >= 3.5) + (z > 5.0))
    code = (code + 8 * (b < 0)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.view(torch.uint8)


def _nvfp4_values(packed, scales):
    """float32 values of packed codes [..., n/2] with scales [..., n/16] (plain)."""
    one = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=packed.device)
    byte = torch.arange(256, device=packed.device)
    v = torch.stack((one[byte & 15], one[byte >> 4]), -1)[packed.long()].flatten(-2)
    return (v.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _parts(cache, case):
    """Views of pages [...][kv heads][bytes]: key codes, value codes, key scales [token][block], value scales [block][token]."""
    p, d = case["page"], case["dim"]
    a, b, c = p * d // 2, p * d, p * d + p * d // 16
    return (cache[..., :a].unflatten(-1, (p, d // 2)), cache[..., a:b].unflatten(-1, (p, d // 2)),
            cache[..., b:c].unflatten(-1, (p, d // 16)), cache[..., c:].unflatten(-1, (d // 16, p)))


# ---------------------------------------------------------------------------------------------- inputs
def _activations(shape, g):
    """Activations as a layer meets them: a few channels larger than the rest, tokens of different size."""
    x = torch.randn(shape, device="cuda", generator=g)
    channel = torch.exp(0.7 * torch.randn(shape[1:], device="cuda", generator=g))
    token = torch.exp(0.3 * torch.randn((shape[0], 1), device="cuda", generator=g))
    return 0.5 * x * channel * token


def _weights(n, k, g):
    return _tiles(torch.randn((n, k), device="cuda", generator=g) * k ** -0.5)


def _paged(case, g):
    """A filled cache with its pages in no order, and a page table whose rows begin with the same pages."""
    lens, p, d, hk = _contexts(case), case["page"], case["dim"], case["kv_heads"]
    common = case["shared"] // p
    each = [-(-n // p) - common for n in lens]
    pages = common + sum(each) + 3
    order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    table = torch.zeros((len(lens), common + max(each)), dtype=torch.int32, device="cuda")
    table[:, :common] = order[:common]
    at = common
    for i, n in enumerate(each):
        table[i, common:common + n] = order[at:at + n]
        at += n
    cache = torch.empty((pages, hk, p * d * 9 // 8), dtype=torch.uint8, device="cuda")
    kc, vc, ks, vs = _parts(cache, case)
    gain = torch.exp(0.5 * torch.randn((hk, 1, d), device="cuda", generator=g))
    step = max(1, (1 << 27) // (hk * p * d))
    for a in range(0, pages, step):
        m = min(step, pages - a)
        kc[a:a + m], ks[a:a + m] = _nvfp4(torch.randn((m, hk, p, d), device="cuda", generator=g) * gain)
        vc[a:a + m], s = _nvfp4(torch.randn((m, hk, p, d), device="cuda", generator=g))
        vs[a:a + m] = s.transpose(-1, -2)
    t = case["tokens"]
    starts = torch.arange(0, t * len(lens) + 1, t, dtype=torch.int32, device="cuda")
    return dict(cache=cache, table=table, starts=starts, kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def _inputs(case, seed):
    """What both sides are given, on the GPU, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype, t = DTYPES[case["dtype"]], case["tokens"]
    st = dict(case=case)
    if case["op"] == "quantize":
        st["x"] = _activations((t, case["cols"]), g).to(dtype)
    elif case["op"] == "product":
        n, k = case["n"], case["k"]
        st["w"], st["sw"] = _weights(n, k, g)
        st["x"], s = _row_blocks(_activations((t, k), g).to(dtype).float())
        st["sx"] = torch.zeros((_blocks(k), -(-t // 4) * 4), device="cuda")  # rows of scales as the quantiser is given them
        st["sx"][:, :t] = s
        st["bias"] = torch.randn((n,), device="cuda", generator=g) if case["bias"] else None
    elif case["op"] == "ffn":
        h, i = case["hidden"], case["inter"]
        gate, up, down = _weights(i, h, g), _weights(i, h, g), _weights(h, i, g)
        st["w13"], st["s13"] = torch.cat((gate[0].view(torch.uint8), up[0].view(torch.uint8))).view(torch.float8_e4m3fn), torch.stack((gate[1], up[1]))
        st["w2"], st["s2"] = down
        st["x"] = _activations((t, h), g).to(dtype)
    else:
        st |= _paged(case, g)
        st["q"] = torch.randn((case["seqs"] * t, case["q_heads"], case["dim"]), device="cuda", generator=g).to(dtype)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if not own:
        return st
    import block_scaled_precision_gemm_amd as bsg
    dtype, t = DTYPES[case["dtype"]], case["tokens"]
    if case["op"] == "quantize":
        st["codes"] = torch.empty((t, case["cols"]), dtype=torch.float8_e4m3fn, device="cuda")
        st["scales"] = torch.empty(bsg.f8_scales_shape(t, case["cols"]), dtype=torch.float32, device="cuda")
    elif case["op"] == "product":
        st["plan"] = bsg.F8Plan(case["n"], case["k"], t, dtype=case["dtype"], bias=case["bias"])
        st["out"] = torch.empty((t, case["n"]), dtype=dtype, device="cuda")
    elif case["op"] == "ffn":
        st["plan"] = bsg.F8FFNPlan(case["hidden"], case["inter"], t, dtype=case["dtype"])
        st["out"] = torch.empty((t, case["hidden"]), dtype=dtype, device="cuda")
    else:
        tokens, hq = st["q"].shape[:2]
        lens = _contexts(case)
        st["plan"] = bsg.KVPlan(hq, case["kv_heads"], case["dim"], case["page"], st["cache"].shape[0], tokens, dtype=case["dtype"])
        st["batch"] = bsg.KVBatch(st["starts"], st["kv_len"], st["table"], tokens, t, max(lens))
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty((tokens, hq), dtype=torch.float32, device="cuda")
    return st


# ---------------------------------------------------------------------------------------------- one pass
def run(st):
    return {"quantize": _run_quantize, "product": _run_product, "ffn": _run_ffn, "attend": _run_attend}[st["case"]["op"]](st)


def _run_quantize(st):
    if own:
        import block_scaled_precision_gemm_amd as bsg
        bsg.f8_quantize(st["x"], st["codes"], st["scales"])
        return {"codes": st["codes"], "scales": st["scales"][:, :st["x"].shape[0]]}
    codes, scales = _row_blocks(st["x"].float())
    return {"codes": codes, "scales": scales}


def _run_product(st):
    if own:
        st["plan"].run(st["x"], st["sx"], st["w"], st["sw"], st["out"], bias=st["bias"])
        return {"out": st["out"]}
    x = _row_values(st["x"], st["sx"][:, :st["x"].shape[0]])
    y = x @ _tile_values(st["w"], st["sw"]).t()
    return {"out": (y if st["bias"] is None else y + st["bias"]).to(DTYPES[st["case"]["dtype"]])}


def _run_ffn(st):
    if own:
        st["plan"].run(st["x"], st["w13"], st["s13"], st["w2"], st["s2"], st["out"])
        return {"out": st["out"]}
    x, inter = _row_values(*_row_blocks(st["x"].float())), st["case"]["inter"]
    gate = x @ _tile_values(st["w13"][:inter], st["s13"][0]).t()
    up = x @ _tile_values(st["w13"][inter:], st["s13"][1]).t()
    h = _row_values(*_row_blocks(gate / (1.0 + torch.exp(-gate)) * up))
    return {"out": (h @ _tile_values(st["w2"], st["s2"]).t()).to(DTYPES[st["case"]["dtype"]])}


def _run_attend(st):
    case = st["case"]
    if own:
        st["plan"].attend(st["batch"], st["q"], st["cache"], st["out"], lse=st["lse"], shared=case["shared"])
        return {"out": st["out"], "lse": st["lse"]}
    hk, d, t, b = case["kv_heads"], case["dim"], case["tokens"], case["seqs"]
    g, common = case["q_heads"] // hk, case["shared"] // case["page"]

    def values(pages):  # [...][heads][positions][dim] of page numbers [...][pages]
        kc, vc, ks, vs = _parts(st["cache"][pages.long()], case)
        k = _nvfp4_values(kc, ks.contiguous()).transpose(-4, -3).flatten(-3, -2)
        v = _nvfp4_values(vc, vs.transpose(-1, -2).contiguous()).transpose(-4, -3).flatten(-3, -2)
        return k, v

    k0, v0 = values(st["table"][0, :common])
    k1, v1 = values(st["table"][:, common:])
    q = st["q"].float().unflatten(0, (b, t)).unflatten(2, (hk, g)).permute(2, 0, 1, 3, 4).flatten(2, 3)  # [heads][seqs][tokens x group][dim]
    first = torch.matmul(q.flatten(1, 2), k0.transpose(-1, -2)).unflatten(1, (b, t * g)) * d ** -0.5
    rest = torch.matmul(q.transpose(0, 1), k1.transpose(-1, -2)).transpose(0, 1) * d ** -0.5
    last = st["kv_len"][:, None] - t + torch.arange(t, device="cuda") - case["shared"]  # of each new token, behind the shared ones
    seen = torch.arange(k1.shape[2], device="cuda") <= last[..., None]
    rest = rest.masked_fill(~seen.repeat_interleave(g, 1), -math.inf)
    top = torch.maximum(first.amax(-1, keepdim=True), rest.amax(-1, keepdim=True))
    first, rest = torch.exp(first - top), torch.exp(rest - top)
    total = first.sum(-1, keepdim=True) + rest.sum(-1, keepdim=True)
    o = torch.matmul(first.flatten(1, 2), v0).unflatten(1, (b, t * g)) + torch.matmul(rest.transpose(0, 1), v1).transpose(0, 1)
    lse = (top + torch.log(total)).squeeze(-1)
    o = (o / total).unflatten(2, (t, g)).permute(1, 2, 0, 3, 4).reshape(st["q"].shape)
    return {"out": o.to(DTYPES[case["dtype"]]), "lse": lse.unflatten(2, (t, g)).permute(1, 2, 0, 3).reshape(b * t, -1)}


# ---------------------------------------------------------------------------------------------- 64 bits
def _e4m3_64(code):
    """Value of E4M3 codes from their fields: exponent 0 is m 2^-9, else (1 + m/8) 2^(e-7)."""
    code = code.to(torch.int64)
    e, m = (code >> 3) & 15, (code & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (1.0 + m / 8.0) * torch.exp2((e - 7).double()))
    return torch.where((code & 128) != 0, -v, v)


def _e2m1_64(code):
    """Value of E2M1 codes from their fields: exponent 0 is m/2, else (1 + m/2) 2^(e-1)."""
    code = code.to(torch.int64)
    e, m = (code >> 1) & 3, (code & 1).double()
    v = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.exp2((e - 1).double()))
    return torch.where((code & 8) != 0, -v, v)


def _codes_64(codes):
    return _e4m3_64(torch.arange(256, device=codes.device))[codes.view(torch.uint8).long()]


def _nearest_e4m3_64(x):
    """The nearest E4M3 value of each double up to 448, halfway cases to the even code."""
    values = _e4m3_64(torch.arange(127, device=x.device))
    a = x.abs().contiguous()
    hi = torch.searchsorted(values, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    down, up = a - values[lo], values[hi] - a
    return torch.copysign(torch.where((down < up) | ((down == up) & (lo % 2 == 0)), values[lo], values[hi]), x)


def _blocks_64(x):
    """Codes' values and scales [blocks][rows] of doubles, block by block."""
    q, s = torch.zeros_like(x), []
    for a in range(0, x.shape[1], BLOCK):
        b = x[:, a:a + BLOCK]
        most = b.abs().amax(1)
        p = torch.ceil(torch.log2(most.clamp(min=448.0 * 2.0 ** -126) / 448.0))
        p = torch.where(448.0 * torch.exp2(p - 1.0) >= most, p - 1.0, p)  # (the logarithm is rounded)
        p = torch.where(448.0 * torch.exp2(p) < most, p + 1.0, p).clamp(min=-126.0)
        s.append(torch.exp2(p))
        q[:, a:a + BLOCK] = _nearest_e4m3_64(b / s[-1][:, None])
    return q, torch.stack(s)


def _times_64(q, s, w, sw):
    """Rows with codes' values q and scales s times weights: every block's product by itself, scaled, and added up."""
    out = torch.zeros((q.shape[0], w.shape[0]), dtype=torch.float64, device=q.device)
    v = _codes_64(w)
    row = torch.arange(w.shape[0], device=q.device) // BLOCK
    for b, a in enumerate(range(0, q.shape[1], BLOCK)):
        out += (q[:, a:a + BLOCK] * s[b].double()[:, None]) @ (v[:, a:a + BLOCK] * sw[row, b].double()[:, None]).t()
    return out


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "quantize":
        q, s = _blocks_64(st["x"].double())
        return {"codes": q, "scales": s}
    if case["op"] == "product":
        y = _times_64(_codes_64(st["x"]), st["sx"][:, :case["tokens"]], st["w"], st["sw"])
        return {"out": y if st["bias"] is None else y + st["bias"].double()}
    if case["op"] == "ffn":
        q, s = _blocks_64(st["x"].double())
        gate = _times_64(q, s, st["w13"][:case["inter"]], st["s13"][0])
        up = _times_64(q, s, st["w13"][case["inter"]:], st["s13"][1])
        return {"out": _times_64(*_blocks_64(gate * torch.sigmoid(gate) * up), st["w2"], st["s2"])}
    return _exact_attend(st)


def _exact_attend(st):
    case = st["case"]
    d, g, t = case["dim"], case["q_heads"] // case["kv_heads"], case["tokens"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["q"].shape[:2], dtype=torch.float64, device="cuda")

    def rows(codes, scales):
        v = torch.empty(codes.shape[:-1] + (codes.shape[-1] * 2,), dtype=torch.float64, device=codes.device)
        v[..., 0::2], v[..., 1::2] = _e2m1_64(codes & 15), _e2m1_64(codes >> 4)
        return v * _e4m3_64(scales).repeat_interleave(16, -1)

    for i, n in enumerate(_contexts(case)):
        kc, vc, ks, vs = _parts(st["cache"][st["table"][i, :-(-n // case["page"])].long()], case)
        hidden = torch.arange(n, device="cuda") > torch.arange(n - t, n, device="cuda")[:, None]
        for h in range(case["kv_heads"]):
            k = rows(kc[:, h].flatten(0, 1), ks[:, h].flatten(0, 1))[:n]
            v = rows(vc[:, h].flatten(0, 1), vs[:, h].transpose(-1, -2).flatten(0, 1))[:n]
            q = st["q"][i * t:(i + 1) * t, h * g:(h + 1) * g].double()
            s = torch.einsum("tgd,kd->tgk", q, k) / math.sqrt(d)
            s = s.masked_fill(hidden[:, None], -math.inf)
            z = torch.logsumexp(s, -1)
            out[i * t:(i + 1) * t, h * g:(h + 1) * g] = torch.exp(s - z[..., None]) @ v
            lse[i * t:(i + 1) * t, h * g:(h + 1) * g] = z
    return {"out": out, "lse": lse}
