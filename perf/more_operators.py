"""Bounded contexts as workloads: their cases, inputs, plain forms and definitions.

Four operators, one list of cases:
  prefill   causal attention over packed prompts through a sliding window, with a few first
            tokens (sinks) that stay visible
  decode    the same for new (or drafted) tokens over a paged cache
  weights   the attention weight that cached tokens get from the last queries, added up
  evict     the cached tokens of the least weight leave, the others move to other pages
`run` computes a case in its plain form (elementary torch operations in 32
bits), or, with `own`, through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

D = 128
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- the cases -----------------------------------------------------------------
def listed():
    return [
        # a few chat turns that arrive together, a small window: launch latency counts
        dict(name="prefill_short", op="prefill", io="bf16", n=4, q=331, k=331, mix=1, hq=32, hkv=8, window=64, sinks=4),
        # a ragged batch of prompts packed together, few kv heads, a window shorter than most of them
        dict(name="prefill_ragged", op="prefill", io="bf16", n=24, q=11003, k=11003, mix=2, hq=16, hkv=2, window=256, sinks=16),
        # one long document through a long window, behind a cached prefix
        dict(name="prefill_long", op="prefill", io="bf16", n=1, q=15001, k=16384, mix=0, hq=32, hkv=8, window=4096, sinks=4),
        # a parity run in 32 bits, odd lengths, three heads per kv head
        dict(name="prefill_f32", op="prefill", io="f32", n=3, q=2011, k=2011, mix=3, hq=12, hkv=4, window=300, sinks=5),
        # one user, one token, a window over the end of a long context
        dict(name="decode_one", op="decode", io="bf16", b=1, t=1, hq=32, hkv=8, page=64, total=65531, mix=0, window=8192, sinks=64, tree=False),
        # a serving batch, one token each, contexts from a few to thousands of tokens
        dict(name="decode_batch", op="decode", io="bf16", b=128, t=1, hq=32, hkv=8, page=16, total=400003, mix=4, window=1024, sinks=4, tree=False),
        # a large draft tree of few users, verified in one call
        dict(name="decode_tree", op="decode", io="bf16", b=8, t=64, hq=32, hkv=4, page=32, total=40009, mix=5, window=2048, sinks=4, tree=True),
        # the weights that one user's long context gets from a new token
        dict(name="weights_one", op="weights", io="bf16", b=1, t=1, hq=32, hkv=8, page=64, total=65531, mix=0, accept=False),
        # a serving batch's weights after a step, some of four drafts accepted
        dict(name="weights_batch", op="weights", io="bf16", b=128, t=4, hq=32, hkv=8, page=16, total=400003, mix=4, accept=True),
        # prompts judged by their last 64 tokens before they are cut down
        dict(name="weights_prompt", op="weights", io="bf16", b=8, t=64, hq=32, hkv=4, page=32, total=40009, mix=5, accept=False),
        # a small batch in 32 bits cut down
        dict(name="evict_small", op="evict", io="f32", n=3, total=1501, mix=6, hkv=2, page=16, keep=200, sinks=4, recent=60),
        # a batch whose contexts have outgrown their budget
        dict(name="evict_batch", op="evict", io="bf16", n=32, total=250007, mix=7, hkv=8, page=64, keep=4096, sinks=4, recent=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "decode", "weights", "evict"])
    mix = rng.randrange(1, 1 << 20)
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8])
    io = "f32" if rng.random() < 0.15 else "bf16"
    page = rng.choice([16, 32, 64, 128])
    window, sinks = _log(rng, 64, 8192), rng.choice([0, 1, 4, 16, 64, 129])
    if op == "prefill":
        n = _log(rng, 1, 40)
        q = max(n, _log(rng, 40, 2500 if io == "f32" else int(min(15000, 12000 * math.sqrt(32 / (hkv * group))))))
        k = q if rng.random() < 0.7 else q + _log(rng, 1, 2000)
        return dict(op=op, io=io, n=n, q=q, k=k, mix=mix, hq=hkv * group, hkv=hkv, window=window, sinks=sinks)
    if op in ("decode", "weights"):
        b = _log(rng, 1, 130)
        t = 1 if rng.random() < 0.4 else rng.randrange(2, 65)
        rows = b * t * hkv * group
        top = min(390000 * 8 // hkv, 64 * 40009 * 32 * 8 // max(rows, 2048)) // (4 if io == "f32" else 1)
        total = max(b * (t if op == "weights" else 1), _log(rng, 64, max(100, top)))
        case = dict(op=op, io=io, b=b, t=t, hq=hkv * group, hkv=hkv, page=page, total=total, mix=mix)
        if op == "decode":
            return dict(case, window=window, sinks=sinks, tree=t > 1 and rng.random() < 0.7)
        return dict(case, accept=t > 1 and rng.random() < 0.5)
    n = _log(rng, 1, 100)
    total = max(n, _log(rng, 200, 250000 // (2 if io == "f32" else 1)))
    keep = max(1, int(total / n * rng.uniform(0.1, 1.2)))
    return dict(op=op, io=io, n=n, total=total, mix=mix, hkv=hkv, page=page, keep=keep, sinks=sinks, recent=rng.choice([0, keep // 4, keep // 2]))


# ---- sizes ----------------------------------------------------------------------
def _split(n, total, mix, least=1):
    """n lengths of at least `least` that add up to total; a different mix, other lengths (log-normal)."""
    r = np.random.RandomState(mix)
    w = np.exp(0.8 * r.standard_normal(n))
    cut = np.floor(np.cumsum(w) / w.sum() * (total - least * n) + 0.5).astype(np.int64)
    return np.diff(np.concatenate([[0], cut])) + least


def _lens(case):
    """Lengths (and prefix lengths before them) of a prefill case."""
    lq = _split(case["n"], case["q"], case["mix"])
    extra = case["k"] - case["q"]
    r = np.random.RandomState(case["mix"] + 1)
    pre = r.multinomial(extra, np.full(case["n"], 1.0 / case["n"])) if extra else np.zeros(case["n"], np.int64)
    return lq, lq + pre


def _cached(case):
    """Cached tokens of the sequences of a decode or weights case (those of weights: the new ones among them)."""
    return _split(case["b"], case["total"], case["mix"], case["t"] if case["op"] == "weights" else 1)


def _masks(case):
    """int64 [b, t] of visible drafts: a random tree (each draft's parent an earlier draft or none), or the chain."""
    b, t = case["b"], case["t"]
    r = np.random.RandomState(case["mix"] + 2)
    m = np.zeros((b, t), np.uint64)
    for i in range(t):
        parent = np.maximum(i - 1 - r.randint(0, 3, b), -1) if case["tree"] else np.full(b, i - 1)
        up = np.where(parent >= 0, m[np.arange(b), np.maximum(parent, 0)], 0).astype(np.uint64)
        m[:, i] = up | np.uint64(1 << i)
    return m.view(np.int64)


def _accepted(case):
    """Per sequence, the accepted drafts (a rising subset of its t drafts, the first among them), or all of its tokens."""
    b, t = case["b"], case["t"]
    if not case["accept"]:
        return np.tile(np.arange(t), (b, 1)), np.full(b, t)
    r = np.random.RandomState(case["mix"] + 4)
    picks = [np.concatenate([[0], 1 + np.sort(r.permutation(t - 1)[: r.randint(0, t)])]) for _ in range(b)]
    index = np.zeros((b, t), np.int64)
    for i, p in enumerate(picks):
        index[i, : len(p)] = p
    return index, np.array([len(p) for p in picks])


def _kept(case):
    lens = _split(case["n"], case["total"], case["mix"])
    return lens, np.minimum(lens, case["keep"])


def _through(seen, window, sinks):
    """Of the first `seen` keys those that a window and the sinks leave."""
    return np.where(seen <= window, seen, window + np.minimum(sinks, seen - window))


def work(case):
    es = 2 if case["io"] == "bf16" else 4
    row = D * es
    if case["op"] == "prefill":
        lq, lk = _lens(case)
        seen = sum(int(_through(np.arange(k - q + 1, k + 1), case["window"], case["sinks"]).sum()) for q, k in zip(lq, lk))
        keys = sum(min(int(k), int(case["window"] + q - 1) + case["sinks"]) for q, k in zip(lq, lk))  # that some row sees
        return {"bytes": float(row * (2 * case["q"] * case["hq"] + 2 * keys * case["hkv"]) + 4 * case["q"] * case["hq"]), "flops": 4.0 * D * seen * case["hq"]}
    if case["op"] == "decode":
        lens, rows = _cached(case), case["b"] * case["t"]
        drafts = np.array([[bin(int(x) & (1 << 64) - 1).count("1") for x in r] for r in _masks(case)])
        seen = _through(lens[:, None] + drafts, case["window"], case["sinks"]).sum() * case["hq"]
        keys = int(_through(lens + 1, case["window"], case["sinks"]).sum()) - case["b"]
        return {"bytes": float(2 * row * case["hkv"] * (keys + rows) + 2 * row * rows * case["hq"] + 4 * rows * case["hq"] + 4 * keys // case["page"]), "flops": 4.0 * D * float(seen)}
    if case["op"] == "weights":
        rows = int(_accepted(case)[1].sum()) * case["hq"]
        return {"bytes": float((row + 8) * case["hkv"] * case["total"] + (row + 4) * rows + 4 * case["total"] // case["page"]), "flops": 2.0 * D * float((_accepted(case)[1] * _cached(case)).sum()) * case["hq"]}
    lens, kept = _kept(case)
    return {"bytes": float(case["hkv"] * ((4 * row + 4) * int(kept.sum()) + 8 * int(lens.sum()))), "flops": 0.0}


# ---- inputs ----------------------------------------------------------------------
def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _ints(a):
    return torch.as_tensor(np.ascontiguousarray(a)).to(torch.int32).cuda()


def _table(lens, page, order):
    """int32 [n, width] of page numbers, taken from `order` as they come; -1 past the end."""
    used = (lens + page - 1) // page
    t = np.full((len(lens), max(int(used.max()), 1)), -1, np.int32)
    at = 0
    for i, u in enumerate(used):
        t[i, :u] = order[at : at + u]
        at += int(u)
    return t, at


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    r = np.random.RandomState(seed % (1 << 31))
    dt = DTYPES[case["io"]]
    s = {"op": case["op"], "case": case, "scale": D**-0.5}
    if own:
        import kimi_delta_attention_rule_gb300 as kda

        s["kda"] = kda
    if case["op"] == "prefill":
        lq, lk = _lens(case)
        cu = lambda a: np.concatenate([[0], np.cumsum(a)])  # noqa: E731
        # queries twice as long as normal ones: rows that look at a few keys more than at the rest
        s.update(q=_normal(g, (case["q"], case["hq"], D), dt, 2.0), k=_normal(g, (case["k"], case["hkv"], D), dt), v=_normal(g, (case["k"], case["hkv"], D), dt), cu_q=_ints(cu(lq)), cu_k=_ints(cu(lk)))
        if own:
            s["workspace"] = s["kda"].attn_prefill_workspace(s["q"], s["k"], s["cu_q"])
    elif case["op"] in ("decode", "weights"):
        b, t, page = case["b"], case["t"], case["page"]
        lens = _cached(case)
        pages = int(((lens + page - 1) // page).sum()) + 3
        table, _ = _table(lens, page, r.permutation(pages))
        s.update(q=_normal(g, (b, t, case["hq"], D), dt, 2.0), k_pages=_normal(g, (pages, case["hkv"], page, D), dt), table=_ints(table), lens=_ints(lens))
        if case["op"] == "decode":
            s.update(v_pages=_normal(g, (pages, case["hkv"], page, D), dt), k_new=_normal(g, (b, t, case["hkv"], D), dt), v_new=_normal(g, (b, t, case["hkv"], D), dt),
                     mask=torch.from_numpy(_masks(case)).cuda() if case["tree"] else None)
            if own:
                s["workspace"] = s["kda"].attn_decode_workspace(s["q"], s["k_pages"], s["table"])
        else:
            index, count = _accepted(case)
            s.update(index=_ints(index) if case["accept"] else None, count=_ints(count) if case["accept"] else None)
            # what the steps before have given each token, few of them much
            s["weights"] = torch.exp(2.0 * torch.randn((b, case["hkv"], table.shape[1] * page), generator=g, device="cuda") - 4.0)
            s["lse"] = _row_lse(s)
    else:
        n, page = case["n"], case["page"]
        lens, kept = _kept(case)
        old, new = int(((lens + page - 1) // page).sum()), int(((kept + page - 1) // page).sum())
        order = r.permutation(old + new)
        table, at = _table(lens, page, order)
        dst, _ = _table(kept, page, order[at:])
        shape = (old + new, case["hkv"], page, D)
        w = torch.exp(2.0 * torch.randn((n, case["hkv"], table.shape[1] * page), generator=g, device="cuda") - 4.0)
        w *= torch.rand(w.shape, generator=g, device="cuda") > 0.1  # some tokens have got nothing: equal ones
        s.update(k_pages=_normal(g, shape, dt), v_pages=_normal(g, shape, dt), table=_ints(table), dst=_ints(dst), lens=_ints(lens), keep=_ints(np.full(n, case["keep"])), weights=w,
                 weights_out=torch.zeros_like(w), kept=torch.full(w.shape, -1, dtype=torch.int32, device="cuda"))
        if own:
            s["workspace"] = s["kda"].evict_workspace(s["weights"])
    return s


# ---- one pass ---------------------------------------------------------------------
def run(s):
    if s["op"] == "prefill":
        return _own_prefill(s) if own else _plain_prefill(s)
    if s["op"] == "decode":
        return _own_decode(s) if own else _plain_decode(s)
    if s["op"] == "weights":
        return _own_weights(s) if own else _plain_weights(s)
    return _own_evict(s) if own else _plain_evict(s)


def _own_prefill(s):
    out, lse = s["kda"].kda_attn_prefill_window(s["q"], s["k"], s["v"], s["scale"], s["case"]["window"], s["case"]["sinks"], cu_seqlens=s["cu_q"], cu_seqlens_k=s["cu_k"], output_lse=True, workspace=s["workspace"])
    return {"out": out, "lse": lse}


def _own_decode(s):
    out, lse = s["kda"].kda_attn_decode_window(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["scale"], s["case"]["window"], s["case"]["sinks"], k_new=s["k_new"], v_new=s["v_new"], tree_mask=s["mask"], output_lse=True, workspace=s["workspace"])
    return {"out": out, "lse": lse}


def _own_weights(s):
    weights = s["weights"].clone()  # those before this step again, for each pass
    s["kda"].kda_attn_weights(s["q"], s["k_pages"], s["table"], s["lens"], s["lse"], s["scale"], weights, index=s["index"], count=s["count"])
    return weights


def _own_evict(s):
    c = s["case"]
    s["kda"].kda_cache_evict(s["k_pages"], s["v_pages"], s["weights"], s["table"], s["lens"], s["keep"], sinks=c["sinks"], recent=c["recent"], dst_table=s["dst"], weights_out=s["weights_out"], kept=s["kept"], workspace=s["workspace"])
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "weights": s["weights_out"], "kept": s["kept"]}


# ---- plain forms --------------------------------------------------------------------
def _softmax_product(logits, v):
    """(softmax(logits) v, logsumexp) over the last axis; rows of -inf alone: 0 and -inf. Uses logits up."""
    top = logits.amax(-1, keepdim=True)
    p = logits.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total == 0, 1.0, total)
    return out, (top + torch.log(total)).squeeze(-1)


def _plain_prefill(s):
    q, k, v, case = s["q"], s["k"], s["v"], s["case"]
    (tq, hq, d), (tk, hkv, _) = q.shape, k.shape
    g = hq // hkv
    at_q, at_k = torch.arange(tq, device=q.device), torch.arange(tk, device=q.device)
    seq_q, seq_k = torch.bucketize(at_q, s["cu_q"][1:], right=True), torch.bucketize(at_k, s["cu_k"][1:], right=True)
    last = s["cu_k"][1:][seq_q] - s["cu_q"][1:][seq_q] + at_q  # the last key that a row sees
    behind = (at_k[None, :] <= last[:, None] - case["window"]) & (at_k - s["cu_k"][seq_k] >= case["sinks"])
    hidden = (seq_q[:, None] != seq_k[None, :]) | (at_k[None, :] > last[:, None]) | behind
    rows = q.float().view(tq, hkv, g, d).permute(1, 2, 0, 3).reshape(hkv, g * tq, d) * s["scale"]
    logits = rows @ k.float().permute(1, 2, 0)
    logits.view(hkv, g, tq, tk).masked_fill_(hidden, -math.inf)
    out, lse = _softmax_product(logits, v.float().transpose(0, 1))
    return {"out": out.view(hq, tq, d).transpose(0, 1).to(q.dtype).contiguous(), "lse": lse.view(hq, tq).t().contiguous()}


def _flat(pages, table):
    """The rows of each sequence's pages in order, in 32 bits: [b, hkv, width, d]."""
    rows = pages[table.clamp(min=0).long()].permute(0, 2, 1, 3, 4)
    return rows.reshape(rows.shape[0], rows.shape[1], -1, D).float()


def _plain_decode(s):
    q, lens, case = s["q"], s["lens"], s["case"]
    b, t, hq, d = q.shape
    keys, vals = (torch.cat([_flat(pages, s["table"]), new.transpose(1, 2).float()], 2) for pages, new in ((s["k_pages"], s["k_new"]), (s["v_pages"], s["v_new"])))
    hkv, width = keys.shape[1], keys.shape[2] - t
    drafts, at = torch.arange(t, device=q.device), torch.arange(width, device=q.device)
    if s["mask"] is None:
        seen = (drafts[None, :] <= drafts[:, None]).expand(b, t, t)
    else:
        seen = (s["mask"][:, :, None] >> drafts) & 1 == 1
    first = lens[:, None] - case["window"] + seen.sum(-1)  # the window counts the drafts that a token sees
    inside = (at < lens[:, None])[:, None, :] & ((at >= first[:, :, None]) | (at < case["sinks"]))
    hidden = ~torch.cat([inside, seen], 2)
    rows = q.float().view(b, t, hkv, -1, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d) * s["scale"]
    logits = rows @ keys.transpose(2, 3)
    logits.view(b, hkv, -1, t, width + t).masked_fill_(hidden[:, None, None], -math.inf)
    out, lse = _softmax_product(logits, vals)
    return {"out": out.view(b, hq, t, d).transpose(1, 2).to(q.dtype).contiguous(), "lse": lse.view(b, hq, t).transpose(1, 2).contiguous()}


def _row_logits(s):
    """Logits [b, hkv, g, t, width] of a weights case, -inf where a token does not see the key; token i of the
    accepted ones is at position lens - count + i."""
    q, lens = s["q"], s["lens"]
    b, t, hq, d = q.shape
    keys = _flat(s["k_pages"], s["table"])
    hkv, width = keys.shape[1], keys.shape[2]
    place = torch.arange(t, device=q.device).expand(b, t)
    count = torch.full((b,), t, device=q.device) if s["count"] is None else s["count"].long()
    if s["index"] is not None:  # the place of each token among the accepted ones, past all of them for the others
        chosen = torch.where(place < count[:, None], s["index"].long(), t)
        place = torch.full((b, t + 1), t, device=q.device).scatter_(1, chosen, place)[:, :t]
    seen = torch.where(place < count[:, None], lens[:, None] - count[:, None] + place + 1, 0)
    hidden = torch.arange(width, device=q.device) >= seen[:, :, None]
    rows = q.float().view(b, t, hkv, -1, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d) * s["scale"]
    logits = (rows @ keys.transpose(2, 3)).view(b, hkv, -1, t, width)
    return logits.masked_fill_(hidden[:, None, None], -math.inf)


def _row_lse(s):
    """The logarithms that attention gives with those rows: [b, t, hq] (-inf for a token that is not accepted)."""
    lse = torch.logsumexp(_row_logits(s), -1)
    return lse.permute(0, 3, 1, 2).reshape(s["q"].shape[:3]).contiguous()


def _plain_weights(s):
    logits = _row_logits(s)
    lse = s["lse"].view(*logits.shape[:1], logits.shape[3], *logits.shape[1:3]).permute(0, 2, 3, 1)
    p = logits.sub_(torch.where(lse == -math.inf, math.inf, lse)[..., None]).exp_()
    return s["weights"] + p.sum((2, 3))


def _plain_evict(s):
    case, lens, w = s["case"], s["lens"].long(), s["weights"]
    n, hkv, cap = w.shape
    page = s["k_pages"].shape[2]
    at = torch.arange(cap, device=w.device)
    keep = torch.minimum(lens, s["keep"].long())
    sinks = keep.clamp(max=case["sinks"])
    recent = (keep - sinks).clamp(max=case["recent"])
    safe = (at < sinks[:, None]) | (at >= (lens - recent)[:, None])
    key = torch.where(safe[:, None], math.inf, w).masked_fill((at >= lens[:, None])[:, None], -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True)[1]
    inside = (at < keep[:, None])[:, None].expand(n, hkv, cap)
    slots = torch.sort(torch.where(inside, order, cap), dim=-1)[0]  # those that stay, in their order
    seq, head, to = inside.nonzero(as_tuple=True)
    slot = slots[seq, head, to]
    s["kept"][seq, head, to] = slot.int()
    s["weights_out"].masked_fill_((at < lens[:, None])[:, None], 0.0)
    s["weights_out"][seq, head, to] = w[seq, head, slot]
    old, new = s["table"].long()[seq, slot // page], s["dst"].long()[seq, to // page]
    s["k_pages"][new, head, to % page] = s["k_pages"][old, head, slot % page]
    s["v_pages"][new, head, to % page] = s["v_pages"][old, head, slot % page]
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "weights": s["weights_out"], "kept": s["kept"]}


# ---- the definitions, in 64 bits -------------------------------------------------------
def _rows_exact(q, k, v, seen, scale):
    """One head: q [r, D], k and v [c, D] in 64 bits, seen bool [r, c]."""
    w = torch.where(seen, scale * (q @ k.T), -math.inf)
    lse = torch.logsumexp(w, 1)
    p = torch.exp(w - torch.where(lse == -math.inf, 0.0, lse)[:, None])
    return p @ v, lse


def _pick(first, last, window, sinks):
    """The keys that tokens see of which the first sees `first` keys and the last `last`: a few first ones, then a stretch."""
    lo = max(first - window, 0)
    return list(range(min(sinks, lo))) + list(range(lo, last))


def exact(case, seed):
    s = prepare(case, seed)
    scale = s["scale"]
    if case["op"] == "prefill":
        lq, lk = _lens(case)
        g, block = case["hq"] // case["hkv"], 1024
        if 4.0 * D * case["hq"] * float((lq * np.minimum(lk, case["window"] + case["sinks"] + block)).sum()) > 3e12:
            return None
        out, lse = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
        a = c = 0
        for m, n in zip(lq.tolist(), lk.tolist()):
            for i in range(0, m, block):
                j = min(m, i + block)
                keys = torch.tensor(_pick(n - m + i + 1, n - m + j, case["window"], case["sinks"]), device="cuda")
                pos = torch.arange(n - m + i, n - m + j, device="cuda")[:, None]
                seen = (keys <= pos) & ((keys > pos - case["window"]) | (keys < case["sinks"]))
                for h in range(case["hq"]):
                    k, v = s["k"][c + keys, h // g].double(), s["v"][c + keys, h // g].double()
                    out[a + i : a + j, h], lse[a + i : a + j, h] = _rows_exact(s["q"][a + i : a + j, h].double(), k, v, seen, scale)
            a, c = a + m, c + n
        return {"out": out, "lse": lse}
    if case["op"] in ("decode", "weights"):
        b, t, hkv, page = case["b"], case["t"], case["hkv"], case["page"]
        g = case["hq"] // hkv
        q = s["q"].double()
        lens = s["lens"].tolist()
        cached = lambda pages, i: pages[s["table"][i, : (lens[i] + page - 1) // page].long()].transpose(1, 2).reshape(-1, hkv, D)[: lens[i]].transpose(0, 1).double()  # noqa: E731
        if case["op"] == "decode":
            out, lse = torch.empty_like(q), torch.empty(q.shape[:3], dtype=torch.float64, device="cuda")
            masks = _masks(case).view(np.uint64)
            for i in range(b):
                tree = np.array([[bool(int(masks[i, x]) >> y & 1) for y in range(t)] for x in range(t)])
                inside = np.zeros((t, lens[i]), bool)
                for x in range(t):
                    inside[x, max(0, lens[i] + int(tree[x].sum()) - case["window"]) :] = True
                    inside[x, : case["sinks"]] = True
                use = np.flatnonzero(inside.any(0))
                seen = torch.from_numpy(np.concatenate([inside[:, use], tree], 1)).cuda().repeat(g, 1)
                use = torch.from_numpy(use).cuda()
                k, v = (torch.cat([cached(pages, i)[:, use], new[i].transpose(0, 1).double()], 1) for pages, new in ((s["k_pages"], s["k_new"]), (s["v_pages"], s["v_new"])))
                for h in range(hkv):
                    o, x = _rows_exact(q[i, :, h * g : (h + 1) * g].transpose(0, 1).reshape(g * t, D), k[h], v[h], seen, scale)
                    out[i, :, h * g : (h + 1) * g] = o.view(g, t, D).transpose(0, 1)
                    lse[i, :, h * g : (h + 1) * g] = x.view(g, t).T
            return {"out": out, "lse": lse}
        if 2.0 * D * case["hq"] * case["t"] * case["total"] > 3e12:
            return None
        index, count = _accepted(case)
        weights = s["weights"].double()
        for i in range(b):
            k, n = cached(s["k_pages"], i), int(count[i])
            rows = torch.from_numpy(index[i, :n]).cuda()
            seen = torch.ones(n, lens[i], dtype=torch.bool, device="cuda").tril(lens[i] - n)
            for h in range(case["hq"]):
                p = torch.exp(scale * (q[i, rows, h] @ k[h // g].T) - s["lse"][i, rows, h].double()[:, None])
                weights[i, h // g, : lens[i]] += torch.where(seen, p, 0.0).sum(0)
        return weights
    kp, vp, page = s["k_pages"].clone(), s["v_pages"].clone(), case["page"]
    w, w_out, kept = s["weights"].cpu().numpy(), np.zeros(s["weights"].shape, np.float32), np.full(s["kept"].shape, -1, np.int64)
    table, dst = s["table"].cpu().numpy(), s["dst"].cpu().numpy()
    moves = []
    for i, n in enumerate(s["lens"].tolist()):
        keep = min(n, case["keep"])
        sinks = min(case["sinks"], keep)
        recent = min(case["recent"], keep - sinks)
        for h in range(case["hkv"]):
            rest = np.arange(sinks, n - recent)
            heavy = rest[np.lexsort((rest, -w[i, h, rest].astype(np.float64)))][: keep - sinks - recent]
            stay = np.sort(np.concatenate([np.arange(sinks), heavy, np.arange(n - recent, n)]))
            kept[i, h, :keep] = stay
            w_out[i, h, :keep] = w[i, h, stay]
            to = np.arange(keep)
            moves.append(np.stack([table[i, stay // page], stay % page, dst[i, to // page], to % page, np.full(keep, h)]))
    m = torch.from_numpy(np.concatenate(moves, 1).astype(np.int64)).cuda()
    kp[m[2], m[4], m[3]], vp[m[2], m[4], m[3]] = s["k_pages"][m[0], m[4], m[1]], s["v_pages"][m[0], m[4], m[1]]
    return {"k_pages": kp, "v_pages": vp, "weights": torch.from_numpy(w_out), "kept": torch.from_numpy(kept)}
