"""The attention operators over causal sequences, as measured: attention over packed
prompts (forward, and forward with backward), attention of a chunk of new tokens over a
paged cache (with and without the sums of the attention weights), and eviction from that
cache by those sums.

`own` says which side `run` computes: the operators' plain form in elementary torch
operations (False), or the framework's calls (True).  Both take what `prepare` returns.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # a handful of short requests answered at once: latency
        {"name": "prompt_short", "op": "prompt", "lens": "1,17,64,5", "hq": 8, "hkv": 2, "d": 64, "dtype": "fp16"},
        # a batch of prompts of ordinary lengths, packed without padding
        {"name": "prompt_packed", "op": "prompt", "lens": "1500,311,2047,129,1,777,1024,303", "hq": 32, "hkv": 8,
         "d": 128, "dtype": "bf16"},
        # one long document
        {"name": "prompt_long", "op": "prompt", "lens": "16384", "hq": 16, "hkv": 4, "d": 128, "dtype": "bf16"},
        # a small fine-tuning batch of short samples, as many key heads as query heads
        {"name": "train_short", "op": "train", "lens": "200,31,257,8", "hq": 4, "hkv": 4, "d": 64, "dtype": "fp16"},
        # a training batch: samples of different lengths packed into one row
        {"name": "train_packed", "op": "train", "lens": "4096,1031,2500,565", "hq": 16, "hkv": 4, "d": 128,
         "dtype": "bf16"},
        # the next token of one short conversation: latency
        {"name": "decode_one", "op": "paged", "chunks": "1", "ctx": "777", "hq": 32, "hkv": 8, "d": 128, "page": 16,
         "dtype": "bf16", "weights": False},
        # the next token of a few very long contexts: bytes of the cache
        {"name": "decode_long", "op": "paged", "chunks": "1,1,1,1", "ctx": "65537,40000,131071,9001", "hq": 32, "hkv": 8,
         "d": 128, "page": 64, "dtype": "bf16", "weights": False},
        # a long prompt taken in chunks, beside requests that are already answering
        {"name": "chunk", "op": "paged", "chunks": "512,512,1,300", "ctx": "16000,2048,5000,300", "hq": 32, "hkv": 8,
         "d": 128, "page": 32, "dtype": "bf16", "weights": False},
        # the next token of a full batch, with the weights that eviction needs
        {"name": "decode_weights", "op": "paged", "chunks": ",".join(["1"] * 64),
         "ctx": ",".join(str(1000 + (i * 977) % 7100) for i in range(64)), "hq": 32, "hkv": 8, "d": 128, "page": 64,
         "dtype": "bf16", "weights": True},
        # a chunk of a prompt, with the weights that eviction needs
        {"name": "chunk_weights", "op": "paged", "chunks": "256,199", "ctx": "8192,4099", "hq": 16, "hkv": 4, "d": 64,
         "page": 16, "dtype": "fp16", "weights": True},
        # one conversation's cache cut back by a little
        {"name": "evict_one", "op": "evict", "ctx": "1100", "budget": 1024, "recent": 64, "hkv": 8, "d": 128, "page": 16,
         "dtype": "bf16"},
        # a batch's caches halved
        {"name": "evict_batch", "op": "evict", "ctx": ",".join(str(4000 + (i * 1237) % 4500) for i in range(16)),
         "budget": 4096, "recent": 256, "hkv": 8, "d": 128, "page": 64, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _text(xs):
    return ",".join(str(x) for x in xs)


def draw(rng):
    op = rng.choice(["prompt", "train", "paged", "paged", "evict"])
    c = {"op": op, "dtype": rng.choice(["bf16", "fp16"]), "d": rng.choice([64, 72, 80, 96, 128, 128])}
    hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8])
    if op in ("prompt", "train"):
        n = rng.randint(1, 8)
        lens = [_log(rng, 1, 4000) for _ in range(n)]
        hkv = min(hkv, 4)
        c.update(lens=_text(lens), hkv=hkv, hq=hkv * min(g, 4))
    elif op == "paged":
        n = _log(rng, 1, 64)
        many = rng.random() < 0.5
        hi = min(400, max(4, 1600 // n)) if many else 1
        chunks = [_log(rng, 1, hi) for _ in range(n)]
        ctx = [m + _log(rng, 1, 60000 // n + 2000) for m in chunks]
        c.update(chunks=_text(chunks), ctx=_text(ctx), hkv=hkv, hq=hkv * g, page=rng.choice([16, 32, 64, 128]),
                 weights=rng.random() < 0.5)
    else:
        n = _log(rng, 1, 16)
        budget = _log(rng, 64, 4000)
        ctx = [_log(rng, max(1, budget // 2), budget * 2 + 100) for _ in range(n)]
        c.update(ctx=_text(ctx), budget=budget, recent=rng.randint(0, budget // 2), hkv=hkv,
                 page=rng.choice([16, 32, 64, 128]))
    return c


def _ints(text):
    return [int(x) for x in text.split(",")]


# ------------------------------------------------------------------------------ inputs
def _offsets(lens, dev):
    return torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32).to(dev)


def prepare(case, seed):
    """What a user's program holds before the call: projections in the model's type, the
    offsets of packed sequences, the cache's pages, its table and lengths, the sums."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt, d, hkv = DT[case["dtype"]], case["d"], case["hkv"]

    def normal(*shape, sigma=1.0):
        # queries and keys with a little more spread than unit: some keys stand out
        return (torch.randn(*shape, generator=gen, device=dev) * sigma).to(dt)

    s = {"case": dict(case)}
    if case["op"] in ("prompt", "train"):
        lens, hq = _ints(case["lens"]), case["hq"]
        t = sum(lens)
        s.update(cu=_offsets(lens, dev), q=normal(t, hq, d, sigma=1.3), k=normal(t, hkv, d), v=normal(t, hkv, d))
        if case["op"] == "train":
            s["do"] = normal(t, hq, d)
        return s
    ctx, page = _ints(case["ctx"]), case["page"]
    n, cols = len(ctx), max(-(-x // page) for x in ctx)
    need = n * cols
    pages = need + 3
    order = torch.randperm(pages, generator=gen, device=dev)[:need].to(torch.int32)
    s.update(k_pages=normal(pages, page, hkv, d), v_pages=normal(pages, page, hkv, d), table=order.view(n, cols),
             seq_lens=torch.tensor(ctx, dtype=torch.int32, device=dev))
    if case["op"] == "paged":
        chunks, hq = _ints(case["chunks"]), case["hq"]
        t = sum(chunks)
        s.update(cu=_offsets(chunks, dev), q=normal(t, hq, d, sigma=1.3), k=normal(t, hkv, d), v=normal(t, hkv, d))
        s["weights"] = torch.rand(n, hkv, cols * page, generator=gen, device=dev) if case["weights"] else None
    else:
        # sums of attention weights: a few keys hold most of it, many hold the same small value
        w = torch.rand(n, hkv, cols * page, generator=gen, device=dev)
        s["weights0"] = torch.where(w < 0.25, (w * 64).floor() / 64, w ** 6 * 8)
        s.update(seq_lens0=s["seq_lens"].clone(), weights=s["weights0"].clone())
    return s


# ------------------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    if op == "prompt":
        return _plain_prompt(s)
    if op == "train":
        return _plain_train(s)
    return _plain_paged(s) if op == "paged" else _plain_evict(s)


def _own(s, op):
    from memory_efficient_biased_gb300 import evo_seq as Q
    if op == "prompt":
        out, lse = Q.evo_prompt_fwd(s["q"], s["k"], s["v"], s["cu"])
        return {"out": out, "lse": lse}
    if op == "train":
        out, lse = Q.evo_prompt_fwd(s["q"], s["k"], s["v"], s["cu"])
        dq, dk, dv = Q.evo_prompt_bwd(s["q"], s["k"], s["v"], s["cu"], out, lse, s["do"])
        return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    if op == "paged":
        Q.evo_cache_append(s["k"], s["v"], s["cu"], s["seq_lens"], s["k_pages"], s["v_pages"], s["table"])
        out, lse = Q.evo_paged_fwd(s["q"], s["k_pages"], s["v_pages"], s["cu"], s["seq_lens"], s["table"],
                                   weights=s["weights"])
        return {"out": out, "lse": lse, "k_pages": s["k_pages"], "v_pages": s["v_pages"], "weights": s["weights"]}
    # the pass puts lengths and sums back first, so that a repeated pass evicts again
    s["seq_lens"].copy_(s["seq_lens0"])
    s["weights"].copy_(s["weights0"])
    kept = Q.evo_cache_evict(s["k_pages"], s["v_pages"], s["table"], s["seq_lens"], s["weights"], s["case"]["budget"],
                             s["case"]["recent"])
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "seq_lens": s["seq_lens"], "weights": s["weights"],
            "kept": kept}


def _places(cu, t):
    """Sequence of each packed token, and its place there."""
    at = torch.arange(t, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), at.to(torch.int32), right=True)
    return b, at - cu.long()[b]


def _padded(x, cu, length):
    """[T, ...] -> [B, length, ...] in 32 bits, zeros behind each sequence."""
    at = torch.arange(length, device=cu.device)
    c = cu.long()
    live = at < (c[1:] - c[:-1])[:, None]
    y = x[(c[:-1, None] + at).clamp(max=max(x.shape[0] - 1, 0))].float()
    return y * live.view(live.shape + (1,) * (x.dim() - 1))


def _softmax(x):
    """softmax over the last axis and its log-sum-exp; a row of -inf gives zeros and -inf."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1)
    return e / torch.where(total == 0, torch.ones_like(total), total), lse


def _prompt_scores(s):
    c, cu = s["case"], s["cu"]
    length, g, d = max(_ints(c["lens"])), c["hq"] // c["hkv"], c["d"]
    q, k, v = (_padded(s[n], cu, length) for n in ("q", "k", "v"))
    q = q.view(q.shape[0], length, c["hkv"], g, d).permute(0, 2, 3, 1, 4)  # [B, Hkv, G, L, D]
    k, v = (x.permute(0, 2, 1, 3)[:, :, None] for x in (k, v))             # [B, Hkv, 1, L, D]
    at = torch.arange(length, device=cu.device)
    x = torch.matmul(q, k.transpose(-1, -2)) * d ** -0.5
    x = x.masked_fill_(at[None, :] > at[:, None], -math.inf)
    p, lse = _softmax(x)
    return q, k, v, p, lse


def _packed(x, b, at, heads):
    """[B, Hkv, G, L, D] -> [T, heads, D]."""
    return x[b, :, :, at].reshape(b.shape[0], heads, x.shape[-1])


def _plain_prompt(s):
    c, dt = s["case"], s["q"].dtype
    _, _, v, p, lse = _prompt_scores(s)
    b, at = _places(s["cu"], s["q"].shape[0])
    out = _packed(torch.matmul(p, v), b, at, c["hq"]).to(dt)
    return {"out": out, "lse": lse[b, :, :, at].reshape(b.shape[0], c["hq"]).t().contiguous()}


def _plain_train(s):
    c, cu, dt = s["case"], s["cu"], s["q"].dtype
    q, k, v, p, lse = _prompt_scores(s)
    length, g, d = q.shape[3], q.shape[2], c["d"]
    b, at = _places(cu, s["q"].shape[0])
    o = torch.matmul(p, v)
    do = _padded(s["do"], cu, length).view(-1, length, c["hkv"], g, d).permute(0, 2, 3, 1, 4)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2, keepdim=True)
    ds = p * (torch.matmul(do, v.transpose(-1, -2)) - (do * o).sum(-1, keepdim=True))
    dq = torch.matmul(ds, k) * d ** -0.5
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2, keepdim=True) * d ** -0.5
    return {"out": _packed(o, b, at, c["hq"]).to(dt),
            "lse": lse[b, :, :, at].reshape(b.shape[0], c["hq"]).t().contiguous(),
            "dq": _packed(dq, b, at, c["hq"]).to(dt), "dk": _packed(dk, b, at, c["hkv"]).to(dt),
            "dv": _packed(dv, b, at, c["hkv"]).to(dt)}


def _plain_paged(s):
    c, cu, dt, table = s["case"], s["cu"], s["q"].dtype, s["table"].long()
    page, hkv, d, g = c["page"], c["hkv"], c["d"], c["hq"] // c["hkv"]
    t, n, length = s["q"].shape[0], table.shape[0], max(_ints(c["chunks"]))
    b, at = _places(cu, t)
    first = s["seq_lens"].long() - (cu.long()[1:] - cu.long()[:-1])  # place of each sequence's first new token
    to = first[b] + at
    s["k_pages"][table[b, to // page], to % page] = s["k"]
    s["v_pages"][table[b, to // page], to % page] = s["v"]
    kk, vv = (s[x][table].view(n, -1, hkv, d).permute(0, 2, 1, 3).float() for x in ("k_pages", "v_pages"))
    q = _padded(s["q"], cu, length).view(n, length, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, g * length, d)
    key, row = torch.arange(kk.shape[2], device=cu.device), torch.arange(length, device=cu.device)
    seen = key <= first[:, None, None] + row[:, None]                  # [B, L, keys]
    live = (row < (cu.long()[1:] - cu.long()[:-1])[:, None])           # [B, L]
    x = (torch.matmul(q, kk.transpose(-1, -2)) * d ** -0.5).view(n, hkv, g, length, -1)
    x = x.masked_fill_(~(seen & live[:, :, None])[:, None, None], -math.inf)
    p, lse = _softmax(x)
    o = torch.matmul(p.view(n, hkv, g * length, -1), vv).view(n, hkv, g, length, d)
    w = s["weights"]
    if w is not None:
        w += p.sum((2, 3))
    return {"out": _packed(o, b, at, c["hq"]).to(dt),
            "lse": lse[b, :, :, at].reshape(t, c["hq"]).t().contiguous(),
            "k_pages": s["k_pages"], "v_pages": s["v_pages"], "weights": w}


def _plain_evict(s):
    c, table = s["case"], s["table"].long()
    budget, recent, page, hkv = c["budget"], c["recent"], c["page"], c["hkv"]
    lens, w = s["seq_lens"], s["weights"]
    lens.copy_(s["seq_lens0"])
    w.copy_(s["weights0"])
    n, cap = table.shape[0], w.shape[2]
    key = torch.arange(cap, device=w.device)
    size = lens.long()[:, None, None]
    over = size > budget
    old = key < size - recent
    order = torch.sort(torch.where(old, w, torch.full_like(w, -math.inf)), dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, key.expand_as(order).contiguous())
    keep = torch.where(over, (old & (rank < budget - recent)) | (~old & (key < size)), key < size)
    kept = torch.sort(torch.where(keep, key, torch.full_like(key, cap)), dim=-1).values[..., :budget]
    if kept.shape[-1] < budget:
        kept = torch.nn.functional.pad(kept, (0, budget - kept.shape[-1]), value=cap)
    live = kept < cap
    at = kept.clamp(max=cap - 1)
    to = torch.arange(budget, device=w.device).clamp(max=cap - 1)
    src = table[torch.arange(n, device=w.device)[:, None, None], at // page] * page + at % page    # [B, Hkv, budget]
    dst = (table[:, to // page] * page + to % page)[:, None].expand_as(src)
    head = torch.arange(hkv, device=w.device)[None, :, None]
    # where nothing is kept (a short sequence) the row is written back onto itself
    dst = torch.where(live & over, dst, src)
    head = head.expand_as(src)
    for name in ("k_pages", "v_pages"):
        flat = s[name].view(-1, hkv, c["d"])
        flat[dst, head] = flat[src, head]
    new = torch.where(live, torch.gather(w, -1, at), torch.zeros_like(at, dtype=w.dtype))
    new = torch.nn.functional.pad(new, (0, max(0, cap - budget)))[..., :cap]
    w.copy_(torch.where(over & (key < size), new, w))
    lens.clamp_(max=budget)
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "seq_lens": lens, "weights": w,
            "kept": torch.where(live, kept, torch.full_like(kept, -1)).to(torch.int32)}


# ------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    d, hkv = case["d"], case["hkv"]
    if case["op"] in ("prompt", "train"):
        lens, hq = _ints(case["lens"]), case["hq"]
        t, pairs = sum(lens), sum(x * (x + 1) // 2 for x in lens)
        rows, keys = t * hq * d * 2, t * hkv * d * 2
        if case["op"] == "prompt":
            return {"bytes": 2 * rows + 2 * keys + t * hq * 4, "flops": 4 * d * hq * pairs}
        # q, do, k, v in; out, dq, dk, dv, lse out
        return {"bytes": 4 * rows + 4 * keys + t * hq * 4, "flops": 14 * d * hq * pairs}
    ctx = _ints(case["ctx"])
    if case["op"] == "paged":
        chunks, hq = _ints(case["chunks"]), case["hq"]
        t = sum(chunks)
        pairs = sum(m * x - m * (m - 1) // 2 if x >= m else x * (x + 1) // 2 for m, x in zip(chunks, ctx))
        size = 2 * sum(ctx) * hkv * d * 2 + 2 * t * hkv * d * 2 + 2 * t * hq * d * 2 + t * hq * 4
        return {"bytes": size + (8 * sum(ctx) * hkv if case["weights"] else 0), "flops": 4 * d * hq * pairs}
    cut = [x for x in ctx if x > case["budget"]]
    rows = len(cut) * (case["budget"] - case["recent"]) + len(cut) * case["recent"]
    size = rows * hkv * d * 2 * 2 * 2 + sum(cut) * hkv * 8 + len(ctx) * hkv * case["budget"] * 4
    return {"bytes": max(size, 64), "flops": sum(cut) * hkv}


# ------------------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(case, s)
    g, scale, dev = case["hq"] // case["hkv"], 1.0 / math.sqrt(case["d"]), s["q"].device
    paged, train = case["op"] == "paged", case["op"] == "train"
    sizes = _ints(case["chunks"] if paged else case["lens"])
    t, hq, d = s["q"].shape
    out = torch.zeros(t, hq, d, dtype=torch.float64, device=dev)
    lse = torch.zeros(hq, t, dtype=torch.float64, device=dev)
    grads = {x: torch.zeros(s[x[1:]].shape, dtype=torch.float64, device=dev) for x in ("dq", "dk", "dv")} if train else {}
    w = s["weights"].double() if paged and s["weights"] is not None else None
    begin = 0
    for b, size in enumerate(sizes):
        rows = slice(begin, begin + size)
        begin += size
        k, v = s["k"][rows].double(), s["v"][rows].double()
        if paged:
            total, page = _ints(case["ctx"])[b], case["page"]
            pages = s["table"][b].tolist()
            for name, new in (("k_pages", s["k"]), ("v_pages", s["v"])):
                spot = torch.arange(total - size, total, device=dev)
                s[name][torch.tensor(pages, device=dev)[spot // page], spot % page] = new[rows]
            k, v = (torch.cat([s[name][p] for p in pages])[:total].double() for name in ("k_pages", "v_pages"))
        total = k.shape[0]
        hidden = torch.ones(size, total, dtype=torch.bool, device=dev).triu(total - size + 1)
        for h in range(hq):
            e = h // g
            x = (s["q"][rows, h].double() @ k[:, e].T) * scale
            x[hidden] = -math.inf
            z = torch.logsumexp(x, 1)
            p = torch.exp(x - z[:, None])
            lse[h, rows] = z
            out[rows, h] = p @ v[:, e]
            if w is not None:
                w[b, e, :total] += p.sum(0)
            if train:
                do = s["do"][rows, h].double()
                ds = p * (do @ v[:, e].T - (do * out[rows, h]).sum(1, keepdim=True)) * scale
                grads["dq"][rows, h] = ds @ k[:, e]
                grads["dk"][rows, e] += ds.T @ s["q"][rows, h].double()
                grads["dv"][rows, e] += p.T @ do
    if paged:
        return {"out": out, "lse": lse, "k_pages": s["k_pages"].double(), "v_pages": s["v_pages"].double(), "weights": w}
    return {"out": out, "lse": lse, **grads}


def _exact_evict(case, s):
    budget, recent, page = case["budget"], case["recent"], case["page"]
    w = s["weights0"].cpu().double().numpy()
    new = w.copy()
    pages = {name: s[name].double() for name in ("k_pages", "v_pages")}
    lens = _ints(case["ctx"])
    for b, size in enumerate(lens):
        if size <= budget:
            continue
        slot = torch.tensor([p * page + i for p in s["table"][b].tolist() for i in range(page)][:size],
                            device=s["table"].device)
        for h in range(case["hkv"]):
            old = sorted(range(size - recent), key=lambda j: (-w[b, h, j], j))[:budget - recent]
            kept = sorted(old) + list(range(size - recent, size))
            new[b, h, :size] = 0
            new[b, h, :budget] = w[b, h, kept]
            at = slot[torch.tensor(kept, device=slot.device)]
            for x in pages.values():
                flat = x.view(-1, case["hkv"], case["d"])
                flat[slot[:budget], h] = flat[at, h]
    return {"k_pages": pages["k_pages"], "v_pages": pages["v_pages"], "seq_lens": None,
            "weights": torch.from_numpy(new), "kept": None}
