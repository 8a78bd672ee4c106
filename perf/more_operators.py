"""Rotary positions and the cache in 8 bits, as measured: queries and keys rotated by their
positions (and the gradients rotated back), new rows appended to a paged cache of 8-bit
values with a scale for each block of tokens and head, rows read back from it, and the
attention of new tokens over it.

`own` says which side `run` computes: the operators' plain form in elementary torch
operations (False), or the framework's calls (True).  Both take what `prepare` returns.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn
E4M3_MOST = 448.0
LEAST_EXPONENT = -64  # of a block's scale


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # the next token of one conversation, far into it: latency
        {"name": "rotary_one", "op": "rotary", "lens": "1", "start": 77777, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "scaling": "parts", "dtype": "bf16"},
        # a batch of prompts of ordinary lengths, neighbouring features paired, half of the head
        {"name": "rotary_prompt", "op": "rotary", "lens": "1500,311,2047,129,1,777,1024,303", "start": 0, "hq": 32,
         "hkv": 8, "d": 128, "rot": 64, "interleaved": True, "scaling": "none", "dtype": "fp16"},
        # a small fine-tuning batch of short samples, heads of an odd size
        {"name": "rotary_train_short", "op": "rotary_train", "lens": "200,31,257,8", "start": 0, "hq": 4, "hkv": 4,
         "d": 72, "rot": 72, "interleaved": False, "scaling": "linear", "dtype": "fp16"},
        # training on one long document, positions stretched
        {"name": "rotary_train_long", "op": "rotary_train", "lens": "16384", "start": 0, "hq": 32, "hkv": 8, "d": 128,
         "rot": 128, "interleaved": False, "scaling": "base", "dtype": "bf16"},
        # the next token of a full batch goes into the cache: latency
        {"name": "append8_step", "op": "append8", "chunks": ",".join(["1"] * 64),
         "ctx": ",".join(str(200 + (i * 977) % 710) for i in range(64)), "hkv": 8, "d": 128, "page": 64, "block": 16,
         "dtype": "bf16"},
        # a batch of prompts goes into an empty cache
        {"name": "append8_fill", "op": "append8", "chunks": "4096,1500,311,2047,129,1,777,1024,303",
         "ctx": "4096,1500,311,2047,129,1,777,1024,303", "hkv": 8, "d": 128, "page": 64, "block": 64, "dtype": "bf16"},
        # chunks of prompts that go on where their last block is begun
        {"name": "append8_chunk", "op": "append8", "chunks": "512,300,1,77", "ctx": "2560,1001,4099,177", "hkv": 4,
         "d": 80, "page": 16, "block": 16, "dtype": "fp16"},
        # the next token of one short conversation: latency
        {"name": "paged8_one", "op": "paged8", "chunks": "1", "ctx": "777", "hq": 32, "hkv": 8, "d": 128, "page": 16,
         "block": 16, "dtype": "bf16"},
        # the next token of a few very long contexts: bytes of the cache
        {"name": "paged8_long", "op": "paged8", "chunks": "1,1,1,1", "ctx": "65537,40000,131071,9001", "hq": 32,
         "hkv": 8, "d": 128, "page": 64, "block": 64, "dtype": "bf16"},
        # the next token of a full batch
        {"name": "paged8_batch", "op": "paged8", "chunks": ",".join(["1"] * 64),
         "ctx": ",".join(str(1000 + (i * 977) % 7100) for i in range(64)), "hq": 32, "hkv": 8, "d": 128, "page": 64,
         "block": 16, "dtype": "fp16"},
        # a long prompt taken in chunks, beside requests that are already answering
        {"name": "paged8_chunk", "op": "paged8", "chunks": "512,512,1,300", "ctx": "16000,2048,5000,300", "hq": 32,
         "hkv": 8, "d": 128, "page": 32, "block": 32, "dtype": "bf16"},
        # a chunk of a prompt, smaller heads
        {"name": "paged8_chunk_small", "op": "paged8", "chunks": "256,199", "ctx": "8192,4099", "hq": 16, "hkv": 4,
         "d": 64, "page": 16, "block": 16, "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _text(xs):
    return ",".join(str(x) for x in xs)


def draw(rng):
    op = rng.choice(["rotary", "rotary_train", "append8", "paged8", "paged8", "paged8"])
    c = {"op": op, "dtype": rng.choice(["bf16", "fp16"])}
    hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8])
    if op in ("rotary", "rotary_train"):
        d = rng.choice([64, 72, 80, 96, 128, 128])
        c.update(lens=_text(_log(rng, 1, 2000) for _ in range(rng.randint(1, 8))), start=rng.choice([0, _log(rng, 1, 10 ** 6)]),
                 hkv=hkv, hq=hkv * min(g, 4), d=d, rot=rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)]),
                 interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "base", "parts"]))
        return c
    page = rng.choice([16, 32, 64, 128])
    c.update(d=rng.choice([64, 80, 96, 128, 128]), hkv=hkv, page=page,
             block=rng.choice([x for x in (16, 32, 64, 128) if x <= page]))
    if op == "append8":
        n = _log(rng, 1, 64)
        chunks = [_log(rng, 1, rng.choice([1, max(2, 6000 // n)])) for _ in range(n)]
        c.update(chunks=_text(chunks), ctx=_text(m + rng.choice([0, _log(rng, 1, 20000 // n)]) for m in chunks))
    else:
        n = _log(rng, 1, 64)
        hi = min(400, max(4, 1600 // n)) if rng.random() < 0.5 else 1
        chunks = [_log(rng, 1, hi) for _ in range(n)]
        c.update(chunks=_text(chunks), ctx=_text(m + _log(rng, 1, 60000 // n + 2000) for m in chunks), hq=hkv * g)
    return c


def _ints(text):
    return [int(x) for x in text.split(",")]


# ------------------------------------------------------------------------------ inputs
def _offsets(lens, dev):
    return torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32).to(dev)


def frequencies(rot, scaling):
    """Angles a position, in 64 bits, of a rotary embedding over `rot` features, and the factor of
    its values: as trained; positions divided by 8; the base raised for contexts 8 times as long; or each
    frequency divided by up to 8 according to how often it turns within the 8192 tokens trained on."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    base = 10000.0
    if scaling == "base" and rot > 2:
        base *= 8.0 ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / 8.0, 1.0
    if scaling != "parts":
        return f, 1.0
    turns = 8192 * f / (2 * math.pi)
    keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
    return f * keep + f / 8.0 * (1.0 - keep), 0.1 * math.log(8.0) + 1.0


def _scale_for(most):
    """The least power of two s with most <= 448 s."""
    m, e = torch.frexp(most)
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=LEAST_EXPONENT)
    return torch.ldexp(torch.ones_like(most), torch.where(most > 0, e, torch.full_like(e, LEAST_EXPONENT)))


def _quantised(x, block):
    """A cache's pages [P, page, H, D] in 8 bits, and the scales [P, H, page / block]."""
    p, page, h, d = x.shape
    y = x.float().view(p, page // block, block, h, d)
    s = _scale_for(y.abs().amax((2, 4)))
    return (y / s[:, :, None, :, None]).to(E4M3).view(p, page, h, d), s.permute(0, 2, 1).contiguous()


def prepare(case, seed):
    """What a user's program holds before the call: the parts of a fused projection in the model's
    type, positions and frequencies, the offsets of packed sequences, the cache's pages, scales, table
    and lengths."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt, d, hkv = DT[case["dtype"]], case["d"], case["hkv"]

    def normal(*shape, sigma=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * sigma).to(dt)

    s = {"case": dict(case)}
    if case["op"] in ("rotary", "rotary_train"):
        lens, hq = _ints(case["lens"]), case["hq"]
        t = sum(lens)
        inv_freq, s["factor"] = frequencies(case["rot"], case["scaling"])
        qkv = normal(t, (hq + 2 * hkv) * d)
        s.update(q=qkv[:, :hq * d].view(t, hq, d), k=qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d),
                 positions=torch.cat([torch.arange(case["start"], case["start"] + n) for n in lens]).to(torch.int32).to(dev),
                 inv_freq=inv_freq.to(dev))
        if case["op"] == "rotary_train":
            s.update(dq=normal(t, hq, d), dk=normal(t, hkv, d))
        return s
    ctx, chunks, page, block = _ints(case["ctx"]), _ints(case["chunks"]), case["page"], case["block"]
    n, t, cols = len(ctx), sum(chunks), max(-(-x // page) for x in ctx)
    pages = n * cols + 3
    order = torch.randperm(pages, generator=gen, device=dev)[:n * cols].to(torch.int32)
    for name in ("k", "v"):
        s[name + "_pages"], s[name + "_scales"] = _quantised(normal(pages, page, hkv, d), block)
    s.update(cu=_offsets(chunks, dev), table=order.view(n, cols), seq_lens=torch.tensor(ctx, dtype=torch.int32, device=dev))
    if case["op"] == "paged8":
        # queries with a little more spread than unit: some keys stand out
        s["q"] = normal(t, case["hq"], d, sigma=1.3)
        return s
    # one token in ten stands out: a block it enters needs a larger scale than it had
    kv = normal(t, 2 * hkv * d)
    kv *= torch.where(torch.rand(t, 1, generator=gen, device=dev) < 0.1, 4.0, 1.0).to(dt)
    s.update(k=kv[:, :hkv * d].view(t, hkv, d), v=kv[:, hkv * d:].view(t, hkv, d))
    # what is read back: the new tokens, and as many earlier ones as their first block may hold
    back = [min(x, m + block) for x, m in zip(ctx, chunks)]
    s.update(cu_back=_offsets(back, dev), back=sum(back))
    return s


# ------------------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    if op in ("rotary", "rotary_train"):
        return _plain_rotary(s)
    return _plain_append(s) if op == "append8" else _plain_paged(s)


def _own(s, op):
    from memory_efficient_biased_gb300 import evo_seq as Q
    if op in ("rotary", "rotary_train"):
        how = {"interleaved": s["case"]["interleaved"], "factor": s["factor"]}
        q, k = Q.evo_rotary(s["q"], s["k"], s["positions"], s["inv_freq"], **how)
        if op == "rotary":
            return {"q": q, "k": k}
        dq, dk = Q.evo_rotary(s["dq"], s["dk"], s["positions"], s["inv_freq"], inverse=True, **how)
        return {"q": q, "k": k, "dq": dq, "dk": dk}
    cache = s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]
    if op == "append8":
        Q.evo_cache8_append(s["k"], s["v"], s["cu"], s["seq_lens"], *cache, s["table"])
        k, v = Q.evo_cache8_read(*cache, s["cu_back"], s["seq_lens"], s["table"], s["back"], s["k"].dtype)
        return {"k": k, "v": v, "k_scales": s["k_scales"], "v_scales": s["v_scales"]}
    out, lse = Q.evo_paged8_fwd(s["q"], *cache, s["cu"], s["seq_lens"], s["table"])
    return {"out": out, "lse": lse}


def _turned(x, cos, sin, interleaved):
    rot, y = 2 * cos.shape[-1], x.float()
    cos, sin = cos[:, None], sin[:, None]
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    a, b = a * cos - b * sin, b * cos + a * sin
    z = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((z, y[..., rot:]), -1).to(x.dtype)


def _plain_rotary(s):
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]  # far positions: 32 bits would lose the angle
    cos, sin = (angle.cos() * s["factor"]).float(), (angle.sin() * s["factor"]).float()
    out = {x: _turned(s[x], cos, sin, c["interleaved"]) for x in ("q", "k")}
    if c["op"] == "rotary_train":
        out.update({x: _turned(s[x], cos, -sin, c["interleaved"]) for x in ("dq", "dk")})
    return out


def _places(cu, t):
    """Sequence of each packed token, and its place there."""
    at = torch.arange(t, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), at.to(torch.int32), right=True)
    return b, at - cu.long()[b]


def _first(cu, seq_lens):
    """Place of each sequence's first row, where its rows are the last of its tokens."""
    return seq_lens.long() - (cu.long()[1:] - cu.long()[:-1])


def _plain_append(s):
    c, cu, table = s["case"], s["cu"], s["table"].long()
    page, block, hkv, d = c["page"], c["block"], c["hkv"], c["d"]
    out = {}
    b, at = _places(cu, s["k"].shape[0])
    first = _first(cu, s["seq_lens"])
    to = first[b] + at
    p, blk = table[b, to // page], to % page // block
    older = to // block * block < first[b]  # the block holds tokens from before
    rb, rat = _places(s["cu_back"], s["back"])
    rto = _first(s["cu_back"], s["seq_lens"])[rb] + rat
    rp, rblk = table[rb, rto // page], rto % page // block
    for name in ("k", "v"):
        pages, scales, x = s[name + "_pages"], s[name + "_scales"], s[name].float()
        flat = scales.permute(0, 2, 1).reshape(-1, hkv)          # [pages * blocks, H]
        i = p * (page // block) + blk
        most = torch.zeros_like(flat).index_reduce_(0, i, x.abs().amax(-1), "amax")
        touched = torch.zeros(flat.shape[0], dtype=torch.bool, device=x.device).index_fill_(0, i, True)
        kept = torch.zeros(flat.shape[0], device=x.device).index_reduce_(0, i, older.float(), "amax") > 0
        new = torch.where(kept[:, None], torch.maximum(flat, _scale_for(most)), _scale_for(most))
        new = torch.where(touched[:, None], new, flat)
        shrink = (flat / new).view(-1, page // block, 1, hkv, 1)
        codes = pages.float().view(-1, page // block, block, hkv, d) * torch.where(
            (touched & kept).view(-1, page // block, 1, 1, 1), shrink, torch.ones_like(shrink))
        codes = codes.view(-1, page, hkv, d)
        codes[p, to % page] = x / new[i][:, :, None]
        pages.copy_(codes.to(E4M3))
        scales.copy_(new.view(-1, page // block, hkv).permute(0, 2, 1))
        out[name] = (pages.float()[rp, rto % page] * scales[rp, :, rblk][:, :, None]).to(s[name].dtype)
    return {**out, "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def _padded(x, cu, length):
    """[T, ...] -> [B, length, ...] in 32 bits, zeros behind each sequence."""
    at = torch.arange(length, device=cu.device)
    c = cu.long()
    live = at < (c[1:] - c[:-1])[:, None]
    y = x[(c[:-1, None] + at).clamp(max=max(x.shape[0] - 1, 0))].float()
    return y * live.view(live.shape + (1,) * (x.dim() - 1))


def _plain_paged(s):
    c, cu, dt, table = s["case"], s["cu"], s["q"].dtype, s["table"].long()
    block, hkv, d, g = c["block"], c["hkv"], c["d"], c["hq"] // c["hkv"]
    t, n, length = s["q"].shape[0], table.shape[0], max(_ints(c["chunks"]))
    b, at = _places(cu, t)
    kk, vv = ((s[x + "_pages"].view(torch.uint8)[table].view(E4M3).float().view(n, -1, block, hkv, d)
               * s[x + "_scales"][table].permute(0, 1, 3, 2).reshape(n, -1, 1, hkv, 1)).view(n, -1, hkv, d).permute(0, 2, 1, 3)
              for x in ("k", "v"))
    q = _padded(s["q"], cu, length).view(n, length, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, g * length, d)
    key, row = torch.arange(kk.shape[2], device=cu.device), torch.arange(length, device=cu.device)
    seen = key <= _first(cu, s["seq_lens"])[:, None, None] + row[:, None]
    x = (torch.matmul(q, kk.transpose(-1, -2)) * d ** -0.5).view(n, hkv, g, length, -1)
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    o = torch.matmul((e / total).view(n, hkv, g * length, -1), vv).view(n, hkv, g, length, d)
    lse = (m + torch.log(total)).squeeze(-1)
    return {"out": o[b, :, :, at].reshape(t, c["hq"], d).to(dt), "lse": lse[b, :, :, at].reshape(t, c["hq"]).t().contiguous()}


# ------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    d, hkv = case["d"], case["hkv"]
    if case["op"] in ("rotary", "rotary_train"):
        t, heads, passes = sum(_ints(case["lens"])), case["hq"] + hkv, 2 if case["op"] == "rotary_train" else 1
        return {"bytes": passes * 4 * t * heads * d + 4 * t + 4 * case["rot"], "flops": passes * 3 * t * heads * case["rot"]}
    ctx, chunks = _ints(case["ctx"]), _ints(case["chunks"])
    t, blocks = sum(chunks), 8 * hkv / case["block"]  # bytes of scales a token, keys and values
    if case["op"] == "append8":
        back = sum(min(x, m + case["block"]) for x, m in zip(ctx, chunks))
        # rows in, codes and scales out; codes and scales in, rows out
        return {"bytes": t * (6 * hkv * d + blocks) + back * (6 * hkv * d + blocks), "flops": (2 * t + back) * 2 * hkv * d}
    pairs = sum(m * x - m * (m - 1) // 2 for m, x in zip(chunks, ctx))
    return {"bytes": sum(ctx) * (2 * hkv * d + blocks) + 4 * t * case["hq"] * d + 4 * t * case["hq"],
            "flops": 4 * d * case["hq"] * pairs}


# ------------------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rotary", "rotary_train"):
        return _exact_rotary(case, s)
    return _exact_append(case, s) if case["op"] == "append8" else _exact_paged(case, s)


def _exact_rotary(case, s):
    # a pair of features is a complex number, times factor · exp(i angle)
    half, turn = case["rot"] // 2, s["positions"].double()[:, None] * s["inv_freq"]
    turn = torch.polar(torch.full_like(turn, s["factor"]), turn)[:, None]
    one, two = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["interleaved"] else (slice(0, half), slice(half, 2 * half))
    out = {}
    for name in ("q", "k", "dq", "dk"):
        if name in s:
            out[name] = s[name].double()
            z = torch.complex(out[name][..., one], out[name][..., two]) * (turn.conj() if name[0] == "d" else turn)
            out[name][..., one], out[name][..., two] = z.real, z.imag
    return out


def _rounded8(x):
    """x rounded to three bits behind the leading one, steps of 2^-9 at the least (ties to even)."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30))).clamp(min=-6.0) - 3.0)
    return torch.round(x / step) * step


def _exact_append(case, s):
    page, block, hkv = case["page"], case["block"], case["hkv"]
    out = {"k": [], "v": [], "k_scales": None, "v_scales": None}
    for name in ("k", "v"):
        codes, scales = s[name + "_pages"].double(), s[name + "_scales"].double()
        begin = 0
        for b, (size, total) in enumerate(zip(_ints(case["chunks"]), _ints(case["ctx"]))):
            rows = s[name][begin:begin + size].double()
            begin, first = begin + size, total - size
            for at in range(first // block * block, total, block):
                p, i = int(s["table"][b, at // page]), at % page
                lo, hi = max(at, first), min(at + block, total)
                new = rows[lo - first:hi - first]
                scale = torch.full((hkv,), 2.0 ** LEAST_EXPONENT, dtype=torch.float64, device=new.device)
                most = new.abs().amax((0, 2))
                fit = torch.exp2(torch.ceil(torch.log2(most.clamp(min=2.0 ** -300) / E4M3_MOST)))
                scale = torch.maximum(scale, fit)
                if lo > at:
                    scale = torch.maximum(scale, scales[p, :, i // block])
                    codes[p, i:i + block] = _rounded8(codes[p, i:i + block] * (scales[p, :, i // block] / scale)[:, None])
                codes[p, lo % page:lo % page + hi - lo] = _rounded8(new / scale[:, None])
                scales[p, :, i // block] = scale
            back = torch.arange(total - min(total, size + block), total, device=rows.device)
            p = s["table"][b].long()[back // page]
            out[name].append(codes[p, back % page] * scales[p, :, back % page // block][:, :, None])
        out[name] = torch.cat(out[name])
        out[name + "_scales"] = scales
    return out


def _exact_paged(case, s):
    g, scale, dev = case["hq"] // case["hkv"], 1.0 / math.sqrt(case["d"]), s["q"].device
    page, block, begin = case["page"], case["block"], 0
    t, hq, d = s["q"].shape
    out = torch.zeros(t, hq, d, dtype=torch.float64, device=dev)
    lse = torch.zeros(hq, t, dtype=torch.float64, device=dev)
    for b, (size, total) in enumerate(zip(_ints(case["chunks"]), _ints(case["ctx"]))):
        rows = slice(begin, begin + size)
        begin += size
        j = torch.arange(total, device=dev)
        p = s["table"][b].long()[j // page]
        k, v = (s[x + "_pages"].view(torch.uint8)[p, j % page].view(E4M3).double() * s[x + "_scales"].double()[p, :, j % page // block][:, :, None]
                for x in ("k", "v"))
        hidden = torch.ones(size, total, dtype=torch.bool, device=dev).triu(total - size + 1)
        for h in range(hq):
            x = (s["q"][rows, h].double() @ k[:, h // g].T) * scale
            x[hidden] = -math.inf
            lse[h, rows] = torch.logsumexp(x, 1)
            out[rows, h] = torch.exp(x - lse[h, rows][:, None]) @ v[:, h // g]
    return {"out": out, "lse": lse}
