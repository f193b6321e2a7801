"""The decode-layer operators around the block-scaled GEMM: cases, inputs, plain forms and their 64-bit values.

Three operators of a transformer layer whose projections are block-scaled products:

* append: rotate new keys and queries by their positions, store keys and values as NVFP4 blocks in a paged cache,
  and read the stored positions back as the values that the cache holds;
* attend: attention of one, several or many new tokens of each sequence over that cache;
* moe: a mixture-of-experts layer (router, gate/up, SiLU, down, weighted sum) for few tokens, its weights NVFP4 or MXFP8.

`own` False: plain torch in 32 bits, rounded once at the end.  `own` True: the library's operators.
"""
import math
import random

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------------------------- cases
def _append(name, seqs, tokens, context, q_heads, kv_heads, dim, page, dtype, rope, layout):
    return dict(name=name, op="append", seqs=seqs, tokens=tokens, context=context, q_heads=q_heads, kv_heads=kv_heads,
                dim=dim, page=page, dtype=dtype, rope=rope, layout=layout)


def _attend(name, seqs, tokens, context, q_heads, kv_heads, dim, page, dtype, window):
    return dict(name=name, op="attend", seqs=seqs, tokens=tokens, context=context, q_heads=q_heads, kv_heads=kv_heads,
                dim=dim, page=page, dtype=dtype, window=window)


def _moe(name, fmt, tokens, experts, top_k, hidden, inter, dtype):
    return dict(name=name, op="moe", fmt=fmt, tokens=tokens, experts=experts, top_k=top_k, hidden=hidden, inter=inter,
                dtype=dtype)


def listed():
    return [
        # one chat decoding its next token: nothing but latency
        _append("append_one", 1, 1, 777, 32, 8, 128, 16, "bf16", 128, "half"),
        # a decode batch; small heads, half of each rotated, neighbouring pairs
        _append("append_batch", 61, 1, 2000, 16, 4, 64, 32, "f16", 32, "interleaved"),
        # prompts of uneven lengths entering the cache in one call
        _append("append_prompts", 7, 4096, 4096, 32, 8, 128, 64, "bf16", 128, "half"),
        # one chat over an ordinary context: a small call, few pages
        _attend("attend_one", 1, 1, 1001, 32, 8, 128, 16, "bf16", 0),
        # one very long document: the cache's length is all the parallelism there is
        _attend("attend_long", 1, 1, 131072, 32, 4, 128, 64, "bf16", 0),
        # a serving batch whose contexts differ widely, the largest read of the cache here
        _attend("attend_batch", 64, 1, 16384, 64, 8, 128, 64, "bf16", 0),
        # checking drafted tokens: five new tokens a sequence, small heads, a sliding window
        _attend("attend_verify", 24, 5, 4097, 32, 8, 64, 32, "f16", 1024),
        # a chunk of a long prompt against what is already there: arithmetic counts
        _attend("attend_chunk", 2, 2048, 8192, 32, 8, 128, 64, "bf16", 0),
        # one token through a small expert layer: latency
        _moe("moe_small", "nvfp4", 1, 32, 4, 1024, 512, "bf16"),
        # one token of an ordinary expert layer
        _moe("moe_one", "nvfp4", 1, 64, 8, 4096, 2048, "bf16"),
        # some tokens, eight-bit experts, odd count
        _moe("moe_mx", "mxfp8", 7, 16, 2, 2048, 4096, "f16"),
        # a decode batch that reaches nearly every expert: the largest read of weights here
        _moe("moe_batch", "nvfp4", 33, 64, 8, 4096, 2048, "bf16"),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op, dtype = rng.choice(("append", "attend", "moe")), rng.choice(("bf16", "f16"))
    if op == "moe":
        fmt = rng.choice(("nvfp4", "mxfp8"))
        experts = rng.choice((8, 16, 32, 64) if fmt == "nvfp4" else (8, 16, 32))
        case = _moe("", fmt, _log_int(rng, 1, 33), experts, rng.randint(1, 8), 32 * rng.choice((16, 25, 32, 47, 64, 90, 128)),
                    32 * rng.choice((8, 13, 16, 31, 45, 64)), dtype)
    else:
        kv_heads, group, dim, page = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 8)), rng.choice((64, 128)), rng.choice((16, 32, 64))
        if op == "append":
            seqs = _log_int(rng, 1, 64)
            tokens = 1 if rng.random() < 0.4 else _log_int(rng, seqs + 1, 4096)
            case = _append("", seqs, tokens, _log_int(rng, 64, 4096), kv_heads * min(group, 4), kv_heads, dim, page, dtype,
                           rng.choice((0, dim // 2, dim)), rng.choice(("half", "interleaved")))
        else:
            kind = rng.choice(("one", "few", "chunk"))
            if kind == "chunk":
                seqs, tokens, context = rng.randint(1, 2), _log_int(rng, 33, 2048), _log_int(rng, 2048, 8192)
                group = min(group, 4)
            else:
                seqs, tokens = _log_int(rng, 1, 64), 1 if kind == "one" else rng.randint(2, 8)
                context = _log_int(rng, 64, min(131072, 64 * 16384 // seqs))
            case = _attend("", seqs, tokens, context, kv_heads * group, kv_heads, dim, page, dtype,
                           rng.choice((0, 0, max(1, context // 3))))
    del case["name"]
    return case


def _lengths(case):
    """(new tokens, context with them) of each sequence: a property of the case alone.

    append: `tokens` 1 gives every sequence one token; more are split unevenly over the sequences.  attend: every
    sequence has `tokens` new ones.  Contexts spread over their logarithm up to `context`, which the first one has."""
    rng = random.Random("%s %d %d %d" % (case["op"], case["seqs"], case["tokens"], case["context"]))
    n = case["seqs"]
    if case["op"] == "append" and case["tokens"] > 1:
        cuts = sorted(rng.sample(range(1, case["tokens"]), n - 1)) if n > 1 else []
        new = [b - a for a, b in zip([0] + cuts, cuts + [case["tokens"]])]
        return new, [t + rng.randint(0, case["context"]) for t in new]
    new = [case["tokens"]] * n
    return new, [max(t, case["context"] if i == 0 else _log_int(rng, max(1, case["context"] // 16), case["context"]))
                 for i, t in enumerate(new)]


def _spans(case):
    """For each sequence the number of (new token, visible position) pairs and of positions that any of them sees."""
    window = case.get("window", 0)
    pairs, seen = [], []
    for t, n in zip(*_lengths(case)):
        ends = range(n - t + 1, n + 1)
        pairs.append(sum(min(e, window) if window else e for e in ends))
        seen.append(min(n, window + t - 1) if window else n)
    return pairs, seen


def work(case):
    if case["op"] == "moe":
        t, e, k, h, i = (case[x] for x in ("tokens", "experts", "top_k", "hidden", "inter"))
        k = min(k, e)
        reached = e * (1.0 - (1.0 - k / e) ** t)  # experts that t tokens reach, each choosing k of them evenly
        per = 9 / 16 if case["fmt"] == "nvfp4" else 33 / 32
        return {"bytes": 3 * h * i * per * reached + e * h * 2 + 4 * t * h + 8 * t * k, "flops": 6.0 * h * i * t * k + 2.0 * t * h * e}
    new, _ = _lengths(case)
    tokens, hq, hk, d = sum(new), case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        per = (hq + 2 * hk) * d * 2 + hq * d * 2 + 2 * (2 * hk * d * 9 / 16) + 2 * hk * d * 2 + 4 * case["rope"]
        return {"bytes": tokens * per, "flops": tokens * (3 * case["rope"] * (hq + hk) + 8 * 2 * hk * d)}
    pairs, seen = _spans(case)
    return {"bytes": sum(seen) * 2 * hk * d * 9 / 16 + tokens * hq * (4 * d + 4), "flops": 4.0 * hq * d * sum(pairs)}


# ---------------------------------------------------------------------------------------------- formats
def _scale_and_codes(x):
    """NVFP4 blocks of the last dimension (plain): E4M3 scales, and E2M1 codes (sign in bit 3)."""
    b = x.float().unflatten(-1, (-1, 16))
    s = (b.abs().amax(-1) * (1.0 / 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = s.float().unsqueeze(-1)
    z = torch.where(f > 0, b / f, torch.zeros_like(b)).abs()
    code = ((z > 0.25).to(torch.uint8) + (z >= 0.75) + (z > 1.25) + (z >= 1.75) + (z > 2.5) + (z >= 3.5) + (z > 5.0))
    return s.view(torch.uint8), (code + 8 * (b < 0)).to(torch.uint8).flatten(-2)


def _packed(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _byte_values(device):
    """float32 [256][2]: the two E2M1 values of a packed byte."""
    one = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=device)
    byte = torch.arange(256, device=device)
    return torch.stack((one[byte & 15], one[byte >> 4]), -1)


def _nvfp4_values(packed, scales):
    """float32 values of packed codes [..., n/2] with scales [..., n/16] (plain)."""
    v = _byte_values(packed.device)[packed.long()].flatten(-2)
    return (v.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _mxfp8(x):
    """MXFP8 blocks of the last dimension: E4M3 codes, E8M0 scale codes."""
    b = x.float().unflatten(-1, (-1, 32))
    e = torch.ceil(torch.log2(b.abs().amax(-1).clamp(min=2.0 ** -100) / 448.0))
    q = (b * torch.exp2(-e).unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).flatten(-2), (e + 127).to(torch.uint8)


def _mxfp8_values(codes, scales):
    v = codes.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32))
    return (v * torch.exp2(scales.float() - 127.0).unsqueeze(-1)).flatten(-2)


def _parts(cache, case):
    """Views of a cache [pages][kv heads][bytes]: key codes, value codes, key scales [token][block], value scales [block][token]."""
    p, d = case["page"], case["dim"]
    a, b, c = p * d // 2, p * d, p * d + p * d // 16
    return (cache[..., :a].unflatten(-1, (p, d // 2)), cache[..., a:b].unflatten(-1, (p, d // 2)),
            cache[..., b:c].unflatten(-1, (p, d // 16)), cache[..., c:].unflatten(-1, (d // 16, p)))


# ---------------------------------------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _keys(shape, g):
    """Keys as projections give them: a few channels of each head much larger than the rest."""
    x = torch.randn(shape, device="cuda", generator=g)
    gain = torch.exp(0.5 * torch.randn(shape[-2:], device="cuda", generator=g))
    return x * gain


def _paged(case, g):
    """A filled cache with its pages in no order, the page table, and the tokens' bookkeeping."""
    new, lens = _lengths(case)
    p, d, hk = case["page"], case["dim"], case["kv_heads"]
    per_seq = [-(-n // p) for n in lens]
    pages = sum(per_seq) + 3
    order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    table = torch.zeros((len(lens), max(per_seq)), dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(per_seq):
        table[i, :n] = order[at:at + n]
        at += n
    cache = torch.empty((pages, hk, p * d * 9 // 8), dtype=torch.uint8, device="cuda")
    kc, vc, ks, vs = _parts(cache, case)
    step = max(1, (1 << 27) // (hk * p * d))
    for a in range(0, pages, step):
        m = min(step, pages - a)
        s, c = _scale_and_codes(_keys((m, p, hk, d), g).transpose(1, 2))
        kc[a:a + m], ks[a:a + m] = _packed(c), s
        s, c = _scale_and_codes(torch.randn((m, hk, p, d), device="cuda", generator=g))
        vc[a:a + m], vs[a:a + m] = _packed(c), s.transpose(-1, -2)
    starts = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32, device="cuda")
    return dict(cache=cache, table=table, starts=starts, kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def _inputs(case, seed):
    """What both sides are given, on the GPU, from the seed alone."""
    g = _generator(seed)
    dtype = DTYPES[case["dtype"]]
    st = dict(case=case)
    if case["op"] == "moe":
        t, e, h, i = (case[x] for x in ("tokens", "experts", "hidden", "inter"))
        made = {"w13": [], "s13": [], "w2": [], "s2": [], "a13": [], "a2": []}
        for _ in range(e):
            for w, s, a, rows, cols in (("w13", "s13", "a13", 2 * i, h), ("w2", "s2", "a2", h, i)):
                x = torch.randn((rows, cols), device="cuda", generator=g) * cols ** -0.5
                if case["fmt"] == "nvfp4":
                    scale = x.abs().max() / (448.0 * 6.0)
                    sc, codes = _scale_and_codes(x / scale)
                    made[w].append(_packed(codes))
                else:
                    scale = torch.ones((), device="cuda")
                    codes, sc = _mxfp8(x)
                    made[w].append(codes)
                made[s].append(sc)
                made[a].append(scale)
        st |= {k: torch.stack(v).contiguous() for k, v in made.items()}
        st["router"] = (torch.randn((e, h), device="cuda", generator=g) * 2.0 * h ** -0.5).to(dtype)
        st["x"] = torch.randn((t, h), device="cuda", generator=g).to(dtype)
        return st
    new, lens = _lengths(case)
    tokens, hq, hk, d = sum(new), case["q_heads"], case["kv_heads"], case["dim"]
    st |= _paged(case, g)
    st["max_q"], st["max_kv"] = max(new), max(lens)
    if case["op"] == "append":
        # the projection's output: queries, keys and values of a token side by side
        qkv = torch.cat((torch.randn((tokens, hq, d), device="cuda", generator=g), _keys((tokens, hk, d), g),
                         torch.randn((tokens, hk, d), device="cuda", generator=g)), 1).to(dtype)
        st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        st["turns"] = None
        if case["rope"]:
            half = case["rope"] // 2
            freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
            angle = torch.arange(max(lens), dtype=torch.float64, device="cuda")[:, None] * freq
            st["turns"] = torch.stack((angle.cos(), angle.sin()), 1).float().contiguous()  # [position][cos, sin][pair]
    else:
        st["q"] = torch.randn((tokens, hq, d), device="cuda", generator=g).to(dtype)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if not own:
        return st
    import block_scaled_precision_gemm_amd as bsg
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "moe":
        k = min(case["top_k"], case["experts"])
        st["plan"] = bsg.MoEPlan(case["fmt"], case["experts"], k, case["hidden"], case["inter"], case["tokens"], dtype=case["dtype"])
        st["out"] = torch.empty_like(st["x"])
        st["ids"] = torch.empty((case["tokens"], k), dtype=torch.int32, device="cuda")
        st["weights"] = torch.empty((case["tokens"], k), dtype=torch.float32, device="cuda")
        return st
    tokens, hq, hk, d = st["q"].shape[0], case["q_heads"], case["kv_heads"], case["dim"]
    st["plan"] = bsg.KVPlan(hq, hk, d, case["page"], st["cache"].shape[0], tokens, dtype=case["dtype"], window=case.get("window", 0),
                            rope_dim=case.get("rope", 0), rope_layout=case.get("layout", "half"))
    st["batch"] = bsg.KVBatch(st["starts"], st["kv_len"], st["table"], tokens, st["max_q"], st["max_kv"])
    st["out"] = torch.empty((tokens, hq, d), dtype=dtype, device="cuda")
    if case["op"] == "append":
        st["k_back"], st["v_back"] = (torch.empty((tokens, hk, d), dtype=dtype, device="cuda") for _ in range(2))
    else:
        st["lse"] = torch.empty((tokens, hq), dtype=torch.float32, device="cuda")
    return st


# ---------------------------------------------------------------------------------------------- one pass
def run(st):
    return {"append": _run_append, "attend": _run_attend, "moe": _run_moe}[st["case"]["op"]](st)


def _token_places(st):
    """For each new token its sequence and its position (plain)."""
    starts, lens = st["starts"].long(), st["kv_len"].long()
    t = torch.arange(st["q"].shape[0], device="cuda")
    seq = torch.searchsorted(starts[1:].contiguous(), t, right=True)
    return seq, lens[seq] - (starts[seq + 1] - starts[seq]) + t - starts[seq]


def _rotated(x, cos, sin, layout):
    """float32 of x with its first dims rotated (plain): two products and a sum for each, rounded one by one."""
    x = x.float()
    if cos is None:
        return x
    r = 2 * cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    if layout == "half":
        a, b = x[..., : r // 2], x[..., r // 2: r]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., r:]), -1)
    a, b = x[..., 0:r:2], x[..., 1:r:2]
    return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), x[..., r:]), -1)


def _run_append(st):
    case = st["case"]
    if own:
        st["plan"].append(st["batch"], st["k"], st["v"], st["cache"], q=st["q"], q_out=st["out"], rope=st["turns"])
        st["plan"].read(st["batch"], st["cache"], st["k_back"], st["v_back"])
        return {"q": st["out"], "k": st["k_back"], "v": st["v_back"]}
    dtype = DTYPES[case["dtype"]]
    seq, pos = _token_places(st)
    cos, sin = (st["turns"][pos, 0], st["turns"][pos, 1]) if case["rope"] else (None, None)
    page, slot = st["table"][seq, pos // case["page"]].long(), pos % case["page"]
    kc, vc, ks, vs = _parts(st["cache"], case)
    s, c = _scale_and_codes(_rotated(st["k"], cos, sin, case["layout"]))
    kc[page, :, slot], ks[page, :, slot] = _packed(c), s
    s, c = _scale_and_codes(st["v"])
    vc[page, :, slot], vs[page, :, :, slot] = _packed(c), s
    return {"q": _rotated(st["q"], cos, sin, case["layout"]).to(dtype),
            "k": _nvfp4_values(kc[page, :, slot], ks[page, :, slot].contiguous()).to(dtype),
            "v": _nvfp4_values(vc[page, :, slot], vs[page, :, :, slot].contiguous()).to(dtype)}


def _run_attend(st):
    case = st["case"]
    if own:
        st["plan"].attend(st["batch"], st["q"], st["cache"], st["out"], lse=st["lse"])
        return {"out": st["out"], "lse": st["lse"]}
    dtype, hk, d, g = DTYPES[case["dtype"]], case["kv_heads"], case["dim"], case["q_heads"] // case["kv_heads"]
    n, most = st["kv_len"].shape[0], st["max_q"]
    gathered = st["cache"][st["table"].long()]  # [seqs][pages][heads][bytes]
    kc, vc, ks, vs = _parts(gathered, case)
    k = _nvfp4_values(kc, ks.contiguous()).transpose(1, 2).flatten(2, 3)  # [seqs][heads][positions][dim]
    v = _nvfp4_values(vc, vs.transpose(-1, -2).contiguous()).transpose(1, 2).flatten(2, 3)
    starts, lens = st["starts"].long(), st["kv_len"].long()
    i = torch.arange(most, device="cuda")
    token = (starts[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    last = lens[:, None] - (starts[1:] - starts[:-1])[:, None] + i  # position of each query
    q = st["q"].float()[token].unflatten(2, (hk, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [seqs][heads][queries x group][dim]
    at = torch.arange(k.shape[2], device="cuda")
    seen = (at <= last[..., None]) & (last[..., None] < lens[:, None, None])
    if case["window"]:
        seen &= at > last[..., None] - case["window"]
    s = torch.matmul(q, k.transpose(-1, -2)) * d ** -0.5
    s = s.unflatten(2, (most, g)).masked_fill(~seen[:, None, :, None, :], -math.inf).flatten(2, 3)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = top + torch.log(total)
    seq = torch.searchsorted(starts[1:].contiguous(), torch.arange(st["q"].shape[0], device="cuda"), right=True)
    row = torch.arange(st["q"].shape[0], device="cuda") - starts[seq]
    o = o.unflatten(2, (most, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    lse = lse.squeeze(-1).unflatten(2, (most, g)).permute(0, 2, 1, 3).flatten(2, 3)
    return {"out": o[seq, row].to(dtype), "lse": lse[seq, row]}


def _run_moe(st):
    case = st["case"]
    if own:
        st["plan"].run(st["x"], st["router"], st["w13"], st["s13"], st["w2"], st["s2"], st["out"], alpha13=st["a13"],
                       alpha2=st["a2"], ids=st["ids"], weights=st["weights"])
        return {"out": st["out"], "ids": st["ids"], "weights": st["weights"]}
    values = _nvfp4_values if case["fmt"] == "nvfp4" else _mxfp8_values
    x, inter, experts = st["x"].float(), case["inter"], case["experts"]
    k = min(case["top_k"], experts)
    logits = x @ st["router"].float().t()
    p = torch.exp(logits - logits.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    best, ids = torch.sort(p, dim=-1, descending=True, stable=True)
    best, ids = best[:, :k], ids[:, :k]
    weights = best / best.sum(-1, keepdim=True)
    if ids.numel() <= experts:  # the chosen experts' weights, once for each choice
        e = ids.flatten()
        xs, w13, s13, w2, s2 = x.repeat_interleave(k, 0)[:, None], st["w13"][e], st["s13"][e], st["w2"][e], st["s2"][e]
        a13, a2 = st["a13"][e][:, None, None], st["a2"][e][:, None, None]
    else:  # every expert's, with every token
        xs, w13, s13, w2, s2 = x.expand(experts, -1, -1), st["w13"], st["s13"], st["w2"], st["s2"]
        a13, a2 = st["a13"][:, None, None], st["a2"][:, None, None]
    gu = torch.matmul(xs, values(w13, s13).transpose(-1, -2)) * a13
    gate, up = gu[..., :inter], gu[..., inter:]
    y = torch.matmul(gate / (1.0 + torch.exp(-gate)) * up, values(w2, s2).transpose(-1, -2)) * a2
    if ids.numel() <= experts:
        y = y.unflatten(0, ids.shape).squeeze(2)
    else:
        y = y[ids, torch.arange(x.shape[0], device="cuda")[:, None]]
    out = (y * weights[..., None]).sum(1)
    return {"out": out.to(DTYPES[case["dtype"]]), "ids": ids.to(torch.int32), "weights": weights}


# ---------------------------------------------------------------------------------------------- 64 bits
def _e2m1_64(code):
    """Value of E2M1 codes from their fields: exponent 0 is m/2, else (1 + m/2) 2^(e-1)."""
    code = code.to(torch.int64)
    e, m = (code >> 1) & 3, (code & 1).double()
    v = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.exp2((e - 1).double()))
    return torch.where((code & 8) != 0, -v, v)


def _e4m3_64(code):
    code = code.to(torch.int64)
    e, m = (code >> 3) & 15, (code & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (1.0 + m / 8.0) * torch.exp2((e - 7).double()))
    return torch.where((code & 128) != 0, -v, v)


def _rows_64(fmt, codes, scales):
    """Doubles of block-scaled rows."""
    if fmt == "nvfp4":
        v = torch.empty(codes.shape[:-1] + (codes.shape[-1] * 2,), dtype=torch.float64, device=codes.device)
        v[..., 0::2], v[..., 1::2] = _e2m1_64(codes & 15), _e2m1_64(codes >> 4)
        return v * _e4m3_64(scales).repeat_interleave(16, -1)
    return _e4m3_64(codes) * torch.exp2(scales.double() - 127.0).repeat_interleave(32, -1)


def _nearest_64(x, values):
    """The nearest of the sorted `values` to each x >= 0, halfway cases to the even index, beyond the last to it."""
    hi = torch.searchsorted(values, x.contiguous()).clamp(max=values.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    down, up = x - values[lo], values[hi] - x
    return torch.where((down < up) | ((down == up) & (lo % 2 == 0)), values[lo], values[hi])


def _stored_64(x):
    """What an NVFP4 block of 16 holds of doubles x."""
    scales = _e4m3_64(torch.arange(127, device=x.device))
    steps = _e2m1_64(torch.arange(8, device=x.device))
    b = x.reshape(x.shape[:-1] + (-1, 16))
    s = _nearest_64((b.abs().amax(-1) / 6.0).clamp(max=448.0), scales)[..., None]
    q = _nearest_64((b / torch.where(s > 0, s, torch.ones_like(s))).abs(), steps) * s
    return torch.where(b < 0, -q, q).reshape(x.shape)


def exact(case, seed):
    return {"append": _exact_append, "attend": _exact_attend, "moe": _exact_moe}[case["op"]](_inputs(case, seed))


def _exact_append(st):
    case = st["case"]
    new, lens = _lengths(case)
    out = {"q": [], "k": [], "v": []}
    at = 0
    for t, n in zip(new, lens):
        for name in out:
            x = st[name][at:at + t].double().clone()
            if name != "v" and case["rope"]:
                r = case["rope"]
                tab = st["turns"][n - t:n].double()
                turn = torch.complex(tab[:, 0], tab[:, 1])[:, None]
                i = torch.arange(r // 2, device="cuda")
                first, second = (i, i + r // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1)
                z = torch.complex(x[..., first], x[..., second]) * turn
                x[..., first], x[..., second] = z.real, z.imag
            out[name].append(x if name == "q" else _stored_64(x))
        at += t
    return {k: torch.cat(v) for k, v in out.items()}


def _exact_attend(st):
    case = st["case"]
    d, g, window = case["dim"], case["q_heads"] // case["kv_heads"], case["window"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b, (t, n) in enumerate(zip(*_lengths(case))):
        low = max(0, n - t - window + 1) // case["page"] if window else 0
        kc, vc, ks, vs = _parts(st["cache"][st["table"][b, low:-(-n // case["page"])].long()], case)
        first = low * case["page"]
        pos = torch.arange(n - t, n, device="cuda")
        for h in range(case["kv_heads"]):
            k = _rows_64("nvfp4", kc[:, h].flatten(0, 1), ks[:, h].flatten(0, 1))[: n - first]
            v = _rows_64("nvfp4", vc[:, h].flatten(0, 1), vs[:, h].transpose(-1, -2).flatten(0, 1))[: n - first]
            key = torch.arange(first, n, device="cuda")
            for a in range(0, t, 512):
                q = st["q"][at + a:at + min(t, a + 512), h * g:(h + 1) * g].double()
                s = torch.einsum("tgd,kd->tgk", q, k) / math.sqrt(d)
                here = pos[a:a + 512, None]
                hidden = (key > here) | ((key <= here - window) if window else torch.zeros_like(key > here))
                s = s.masked_fill(hidden[:, None], -math.inf)
                z = torch.logsumexp(s, -1)
                out[at + a:at + a + q.shape[0], h * g:(h + 1) * g] = torch.exp(s - z[..., None]) @ v
                lse[at + a:at + a + q.shape[0], h * g:(h + 1) * g] = z
        at += t
    return {"out": out, "lse": lse}


def _exact_moe(st):
    case = st["case"]
    inter, experts = case["inter"], case["experts"]
    k = min(case["top_k"], experts)
    x = st["x"].double()
    p = torch.softmax(torch.einsum("th,eh->te", x, st["router"].double()), -1)
    ids = torch.argsort(-p, dim=-1, stable=True)[:, :k]
    weights = p.gather(1, ids)
    weights = weights / weights.sum(1, keepdim=True)
    out = torch.zeros_like(x)
    for e in range(experts):
        t, place = torch.nonzero(ids == e, as_tuple=True)
        if not t.numel():
            continue
        w13 = _rows_64(case["fmt"], st["w13"][e], st["s13"][e]) * st["a13"][e].double()
        w2 = _rows_64(case["fmt"], st["w2"][e], st["s2"][e]) * st["a2"][e].double()
        gate, up = x[t] @ w13[:inter].t(), x[t] @ w13[inter:].t()
        out.index_add_(0, t, weights[t, place, None] * ((gate * torch.sigmoid(gate) * up) @ w2.t()))
    return {"out": out, "ids": ids.to(torch.int32), "weights": weights}
