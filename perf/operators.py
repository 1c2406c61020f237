"""The attention and page-cache operators as workloads: their cases, inputs,
plain forms and definitions.

Three operators, one list of cases:
  prefill   causal attention over packed prompts with grouped heads
  decode    attention of new (or drafted) tokens over a paged cache
  pages     append / fork / compact of that cache's pages
`run` computes a case in its plain form (elementary torch operations in 32
bits), or, with `own`, through the package's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

D = 128
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- the cases -----------------------------------------------------------------
def listed():
    return [
        # four short prompts that arrive together: launch latency counts
        dict(name="prefill_short", op="prefill", io="bf16", n=4, q=331, k=331, mix=1, hq=32, hkv=8),
        # one prompt of the benchmark's length and heads
        dict(name="prefill_8192", op="prefill", io="bf16", n=1, q=8192, k=8192, mix=0, hq=32, hkv=8),
        # a ragged batch of prompts packed together, few kv heads
        dict(name="prefill_ragged", op="prefill", io="bf16", n=24, q=11003, k=11003, mix=2, hq=16, hkv=2),
        # a long tool result appended to a long context (keys of the prefix gathered before it)
        dict(name="prefill_append", op="prefill", io="bf16", n=1, q=1500, k=30011, mix=0, hq=32, hkv=4),
        # a parity run in 32 bits, odd lengths, three heads per kv head
        dict(name="prefill_f32", op="prefill", io="f32", n=3, q=2011, k=2011, mix=3, hq=12, hkv=4),
        # one user, one token, a long context: the latency of a single stream
        dict(name="decode_one_long", op="decode", io="bf16", b=1, t=1, hq=32, hkv=8, page=64, total=65531, mix=0, tree=False),
        # a serving batch, one token each, contexts from a few to thousands of tokens
        dict(name="decode_batch", op="decode", io="bf16", b=128, t=1, hq=32, hkv=8, page=16, total=400003, mix=4, tree=False),
        # a large draft tree of few users, verified in one call
        dict(name="decode_tree64", op="decode", io="bf16", b=8, t=64, hq=32, hkv=4, page=32, total=40009, mix=5, tree=True),
        # a small draft tree in 32 bits
        dict(name="decode_tree_f32", op="decode", io="f32", b=6, t=11, hq=8, hkv=4, page=16, total=9001, mix=6, tree=True),
        # the prompts of a batch written into the pages of the cache
        dict(name="pages_append", op="append", io="bf16", n=8, total=16385, mix=7, hkv=8, page=64, accept=0),
        # parallel samples: each of the parents' sequences forked, after the last step's forks are freed
        dict(name="pages_fork", op="fork", io="bf16", n=61, total=120011, mix=8, hkv=8, page=64, pages=8192),
        # a long-running cache made dense again
        dict(name="pages_compact", op="compact", io="bf16", n=300, total=350000, mix=9, hkv=8, page=64, pages=16384),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "decode", "decode", "decode", "append", "fork", "compact"])
    mix = rng.randrange(1, 1 << 20)
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8])
    io = "f32" if rng.random() < 0.15 else "bf16"
    page = rng.choice([16, 32, 64, 128])
    if op == "prefill":
        n = _log(rng, 1, 40)
        cap = 2500 if io == "f32" else int(min(9000, 8192 * math.sqrt(32 / (hkv * group))))
        q = max(n, _log(rng, 40, cap))
        k = q if rng.random() < 0.7 else q + _log(rng, 1, 2000)
        return dict(op=op, io=io, n=n, q=q, k=k, mix=mix, hq=hkv * group, hkv=hkv)
    if op == "decode":
        b = _log(rng, 1, 130)
        t = 1 if rng.random() < 0.4 else rng.randrange(2, 65)
        rows = b * t * hkv * group
        top = min(390000 * 8 // hkv, 64 * 40009 * 32 * 8 // max(rows, 2048)) // (4 if io == "f32" else 1)
        total = max(b, _log(rng, 64, max(100, top)))
        return dict(op=op, io=io, b=b, t=t, hq=hkv * group, hkv=hkv, page=page, total=total, mix=mix, tree=t > 1 and rng.random() < 0.7)
    if op == "append":
        n = _log(rng, 1, 200)
        return dict(op=op, io=io, n=n, total=max(n, _log(rng, 1, 16000)), mix=mix, hkv=hkv, page=page, accept=0 if rng.random() < 0.5 else rng.randrange(2, 65))
    n = _log(rng, 1, 60 if op == "fork" else 300)
    pages = _log(rng, 1024, 8192 if op == "fork" else 16000)
    total = max(n, _log(rng, 200, max(300, (pages // 2 - 2 * n) * page)))
    if pages // 2 <= 2 * n:
        n = pages // 8
    return dict(op=op, io=io, n=n, total=max(n, min(total, (pages // 2 - n) * page)), mix=mix, hkv=min(hkv, 4) if io == "f32" else hkv, page=page if op == "fork" else min(page, 64), pages=pages)


# ---- sizes ----------------------------------------------------------------------
def _split(n, total, mix):
    """n lengths of at least one that add up to total; a different mix, other lengths (log-normal)."""
    r = np.random.RandomState(mix)
    w = np.exp(0.8 * r.standard_normal(n))
    cut = np.floor(np.cumsum(w) / w.sum() * (total - n) + 0.5).astype(np.int64)
    return np.diff(np.concatenate([[0], cut])) + 1


def _lens(case):
    """Lengths (and prefix lengths before them) of a prefill case."""
    lq = _split(case["n"], case["q"], case["mix"])
    extra = case["k"] - case["q"]
    r = np.random.RandomState(case["mix"] + 1)
    pre = r.multinomial(extra, np.full(case["n"], 1.0 / case["n"])) if extra else np.zeros(case["n"], np.int64)
    return lq, lq + pre


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


def _fork_rows(case):
    """Lengths of the parents, and which parent each of the n children forks."""
    parents = max(1, case["n"] // 4)
    lens = _split(parents, max(parents, case["total"]), case["mix"])
    return lens, np.random.RandomState(case["mix"] + 3).randint(0, parents, case["n"])


def _accepted(case):
    """Per sequence, the accepted drafts (a rising subset of its `accept` drafts)."""
    r = np.random.RandomState(case["mix"] + 4)
    t = case["accept"]
    picks = [np.sort(r.permutation(t)[: r.randint(0, t + 1)]) for _ in range(case["n"])]
    index = np.zeros((case["n"], t), np.int64)
    for i, p in enumerate(picks):
        index[i, : len(p)] = p
    return index, np.array([len(p) for p in picks])


def work(case):
    es = 2 if case["io"] == "bf16" else 4
    row = D * es
    if case["op"] == "prefill":
        lq, lk = _lens(case)
        seen = sum(int(a) * int(b) - int(a) * (int(a) - 1) // 2 for a, b in zip(lq, lk))
        return {"bytes": float(row * (2 * case["q"] * case["hq"] + 2 * case["k"] * case["hkv"]) + 4 * case["q"] * case["hq"]), "flops": 4.0 * D * seen * case["hq"]}
    if case["op"] == "decode":
        drafts = int(np.unpackbits(_masks(case).view(np.uint8)).sum())
        rows = case["b"] * case["t"]
        seen = case["total"] * case["t"] * case["hq"] + drafts * case["hq"]
        return {"bytes": float(2 * row * case["hkv"] * (case["total"] + rows) + 2 * row * rows * case["hq"] + 4 * rows * case["hq"] + 4 * case["total"] // case["page"]), "flops": 4.0 * D * seen}
    entry = row * case["hkv"]
    if case["op"] == "append":
        rows = int(_accepted(case)[1].sum()) if case["accept"] else case["total"]
        return {"bytes": float(max(rows, 1) * entry * 4), "flops": 0.0}
    if case["op"] == "fork":
        lens, src = _fork_rows(case)
        copies = int((lens[src] % case["page"] != 0).sum())
        shared = int(((lens[src] + case["page"] - 1) // case["page"]).sum())
        return {"bytes": float(4 * copies * entry * case["page"] + 4 * case["pages"] + 16 * shared), "flops": 0.0}
    lens = _split(case["n"], case["total"], case["mix"])
    used = (lens + case["page"] - 1) // case["page"]
    moved = _movers(case, used)
    return {"bytes": float(4 * moved * entry * case["page"] + 8 * case["pages"] + 8 * int(used.sum())), "flops": 0.0}


def _movers(case, used):
    live = np.random.RandomState(case["mix"] + 5).permutation(case["pages"])[: int(used.sum())]
    return int((live >= len(live)).sum())


# ---- inputs ----------------------------------------------------------------------
def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _ints(a):
    return torch.as_tensor(np.ascontiguousarray(a)).to(torch.int32).cuda()


def _table(lens, page, pages, order, width=0):
    """int32 [n, width] of page numbers, taken from `order` as they come; -1 past the end."""
    used = (lens + page - 1) // page
    t = np.full((len(lens), max(int(used.max()), width, 1)), -1, np.int32)
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
    elif case["op"] == "decode":
        b, t = case["b"], case["t"]
        lens = _split(b, case["total"], case["mix"])
        pages = int(((lens + case["page"] - 1) // case["page"]).sum()) + 3
        table, _ = _table(lens, case["page"], pages, r.permutation(pages))
        s.update(q=_normal(g, (b, t, case["hq"], D), dt, 2.0), k_new=_normal(g, (b, t, case["hkv"], D), dt), v_new=_normal(g, (b, t, case["hkv"], D), dt),
                 k_pages=_normal(g, (pages, case["hkv"], case["page"], D), dt), v_pages=_normal(g, (pages, case["hkv"], case["page"], D), dt),
                 table=_ints(table), lens=_ints(lens), mask=torch.from_numpy(_masks(case)).cuda() if case["tree"] else None)
        if own:
            s["workspace"] = s["kda"].attn_decode_workspace(s["q"], s["k_pages"], s["table"])
    elif case["op"] == "append":
        n, page = case["n"], case["page"]
        before = r.randint(0, 3 * page, n)
        if case["accept"]:
            index, count = _accepted(case)
            s.update(index=_ints(index), count=_ints(count), cu=None)
            rows, most = (n, case["accept"]), np.full(n, case["accept"])
        else:
            take = _split(n, case["total"], case["mix"])
            s.update(index=None, count=None, cu=_ints(np.concatenate([[0], np.cumsum(take)])))
            rows, most = (case["total"],), take
        pages = int((3 + (most + page - 1) // page).sum()) + 2
        table, _ = _table(before + most, page, pages, r.permutation(pages))
        shape = (pages, case["hkv"], page, D)
        s.update(k=_normal(g, rows + (case["hkv"], D), dt), v=_normal(g, rows + (case["hkv"], D), dt), k_pages=_normal(g, shape, dt), v_pages=_normal(g, shape, dt), table=_ints(table), start=_ints(before))
    else:
        page, pages, n = case["page"], case["pages"], case["n"]
        order = r.permutation(pages)
        if case["op"] == "fork":
            lens, src = _fork_rows(case)
            p = len(lens)
            table, at = _table(lens, page, pages, order)
            table = np.concatenate([table, np.full((n, table.shape[1]), -1, np.int32)])
            lens = np.concatenate([lens, np.zeros(n, np.int64)])
            s.update(src=_ints(src), dst=_ints(p + np.arange(n)))
        else:
            lens = _split(n, case["total"], case["mix"])
            order = np.random.RandomState(case["mix"] + 5).permutation(pages)
            table, at = _table(lens, page, pages, r.permutation(order[: int(((lens + page - 1) // page).sum())]))
        refs = np.zeros(pages, np.int64)
        refs[table[table >= 0]] = 1
        shape = (pages, case["hkv"], page, D)
        s.update(k_pages=_normal(g, shape, dt), v_pages=_normal(g, shape, dt), table=_ints(table), lens=_ints(lens), refs=_ints(refs))
        if own:
            s["workspace"] = s["kda"].cache_workspace(s["refs"])
    return s


# ---- one pass ---------------------------------------------------------------------
def run(s):
    if s["op"] == "prefill":
        return _own_prefill(s) if own else _plain_prefill(s)
    if s["op"] == "decode":
        return _own_decode(s) if own else _plain_decode(s)
    if s["op"] == "append":
        return _own_append(s) if own else _plain_append(s)
    if s["op"] == "fork":
        return _own_fork(s) if own else _plain_fork(s)
    return _own_compact(s) if own else _plain_compact(s)


def _own_prefill(s):
    out, lse = s["kda"].kda_attn_prefill(s["q"], s["k"], s["v"], s["scale"], cu_seqlens=s["cu_q"], cu_seqlens_k=s["cu_k"], output_lse=True, workspace=s["workspace"])
    return {"out": out, "lse": lse}


def _own_decode(s):
    out, lse = s["kda"].kda_attn_decode(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["scale"], k_new=s["k_new"], v_new=s["v_new"], tree_mask=s["mask"], output_lse=True, workspace=s["workspace"])
    return {"out": out, "lse": lse}


def _own_append(s):
    s["kda"].kda_cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["start"], cu_seqlens=s["cu"], index=s["index"], count=s["count"])
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _own_fork(s):
    kda, page = s["kda"], s["case"]["page"]
    kda.kda_cache_free(s["table"], s["lens"], s["refs"], s["dst"], workspace=s["workspace"])
    copies = kda.kda_cache_fork(s["table"], s["lens"], s["refs"], s["src"], s["dst"], page, workspace=s["workspace"])
    kda.kda_cache_copy([s["k_pages"], s["v_pages"]], copies)
    return {"table": s["table"], "lens": s["lens"], "refs": s["refs"], "copies": copies, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _own_compact(s):
    kda, table, refs = s["kda"], s["table"].clone(), s["refs"].clone()  # the fragmented cache again, for each pass
    copies, count = kda.kda_cache_compact(table, refs, workspace=s["workspace"])
    kda.kda_cache_copy([s["k_pages"], s["v_pages"]], copies, count)
    return {"table": table, "refs": refs, "copies": copies, "count": count, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


# ---- plain forms --------------------------------------------------------------------
def _softmax_product(logits, v):
    """(softmax(logits) v, logsumexp) over the last axis; rows of -inf alone: 0 and -inf. Uses logits up."""
    top = logits.amax(-1, keepdim=True)
    p = logits.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total == 0, 1.0, total)
    return out, (top + torch.log(total)).squeeze(-1)


def _plain_prefill(s):
    q, k, v = s["q"], s["k"], s["v"]
    (tq, hq, d), (tk, hkv, _) = q.shape, k.shape
    g = hq // hkv
    at_q, at_k = torch.arange(tq, device=q.device), torch.arange(tk, device=q.device)
    seq_q, seq_k = torch.bucketize(at_q, s["cu_q"][1:], right=True), torch.bucketize(at_k, s["cu_k"][1:], right=True)
    last = s["cu_k"][1:][seq_q] - s["cu_q"][1:][seq_q] + at_q  # the last key that a row sees
    hidden = (seq_q[:, None] != seq_k[None, :]) | (at_k[None, :] > last[:, None])
    rows = q.float().view(tq, hkv, g, d).permute(1, 2, 0, 3).reshape(hkv, g * tq, d) * s["scale"]
    logits = rows @ k.float().permute(1, 2, 0)
    logits.view(hkv, g, tq, tk).masked_fill_(hidden, -math.inf)
    out, lse = _softmax_product(logits, v.float().transpose(0, 1))
    return {"out": out.view(hq, tq, d).transpose(0, 1).to(q.dtype).contiguous(), "lse": lse.view(hq, tq).t().contiguous()}


def _plain_decode(s):
    q, table, lens = s["q"], s["table"], s["lens"]
    b, t, hq, d = q.shape
    hkv, page = s["k_pages"].shape[1], s["k_pages"].shape[2]
    g, width = hq // hkv, table.shape[1] * page
    at = table.clamp(min=0).long()
    # [b, m, hkv, page, d] -> [b, hkv, m * page + t, d]: the cache's rows and then the drafts'
    keys, vals = (torch.cat([pages[at].permute(0, 2, 1, 3, 4).reshape(b, hkv, width, d), new.transpose(1, 2)], 2).float() for pages, new in ((s["k_pages"], s["k_new"]), (s["v_pages"], s["v_new"])))
    drafts = torch.arange(t, device=q.device)
    if s["mask"] is None:
        seen = (drafts[None, :] <= drafts[:, None]).expand(b, t, t)
    else:
        seen = (s["mask"][:, :, None] >> drafts) & 1 == 1
    inside = (torch.arange(width, device=q.device) < lens[:, None])[:, None, :].expand(b, t, width)
    hidden = ~torch.cat([inside, seen], 2)
    rows = q.float().view(b, t, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * t, d) * s["scale"]
    logits = rows @ keys.transpose(2, 3)
    logits.view(b, hkv, g, t, width + t).masked_fill_(hidden[:, None, None], -math.inf)
    out, lse = _softmax_product(logits, vals)
    return {"out": out.view(b, hq, t, d).transpose(1, 2).to(q.dtype).contiguous(), "lse": lse.view(b, hq, t).transpose(1, 2).contiguous()}


def _plain_append(s):
    page, dev = s["k_pages"].shape[2], s["table"].device
    if s["cu"] is not None:
        cu = s["cu"].long()
        row = torch.arange(s["k"].shape[0], device=dev)
        seq = torch.bucketize(row, cu[1:], right=True)
        pos = s["start"].long()[seq] + row - cu[seq]
        k, v = s["k"], s["v"]
    else:
        n, t = s["index"].shape
        i = torch.arange(t, device=dev).expand(n, t)
        keep = i < s["count"][:, None]
        seq = torch.arange(n, device=dev)[:, None].expand(n, t)[keep]
        pos = s["start"].long()[seq] + i[keep]
        pick = s["index"].long()[keep]
        k, v = s["k"][seq, pick], s["v"][seq, pick]
    at = s["table"].long()[seq, pos // page]
    s["k_pages"][at, :, pos % page] = k
    s["v_pages"][at, :, pos % page] = v
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_fork(s):
    table, lens, refs, src, dst, page = s["table"], s["lens"], s["refs"], s["src"].long(), s["dst"].long(), s["case"]["page"]
    old = table[dst]  # free the last forks
    refs.scatter_add_(0, old.clamp(min=0).long().view(-1), -(old >= 0).int().view(-1))
    n, width = old.shape
    have = lens[src]
    full, part = have // page, have % page != 0
    at = torch.arange(width, device=table.device)
    entries = table[src]
    entries = torch.where(at < (full + part)[:, None], entries, -1)
    fresh = torch.sort((refs != 0).int(), stable=True)[1][:n].int()  # the free pages, lowest first
    mine = fresh[(torch.cumsum(part, 0) - 1).clamp(min=0)]
    tail = (at == full[:, None]) & part[:, None]
    last = entries.gather(1, full[:, None].long().clamp(max=width - 1)).squeeze(1)
    copies = torch.stack([torch.where(part, last, -1), torch.where(part, mine, -1)], 1)
    entries = torch.where(tail, mine[:, None], entries)
    refs.scatter_add_(0, entries.clamp(min=0).long().view(-1), (entries >= 0).int().view(-1))
    table[dst] = entries
    lens[dst] = have
    a, z = last[part].long(), mine[part].long()
    s["k_pages"][z] = s["k_pages"][a]
    s["v_pages"][z] = s["v_pages"][a]
    return {"table": table, "lens": lens, "refs": refs, "copies": copies, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_compact(s):
    table, refs = s["table"].clone(), s["refs"].clone()
    live = refs > 0
    at = torch.arange(refs.numel(), device=refs.device)
    n = live.sum()
    a, z = at[live & (at >= n)], at[~live & (at < n)]  # pages that move, and where to
    name = at.int().scatter(0, a, z.int())
    table = torch.where(table >= 0, name[table.clamp(min=0).long()], table)
    refs[z] = refs[a]
    refs[a] = 0
    copies = torch.full((refs.numel(), 2), -1, dtype=torch.int32, device=refs.device)
    copies[: a.numel()] = torch.stack([a, z], 1).int()
    s["k_pages"][z] = s["k_pages"][a]
    s["v_pages"][z] = s["v_pages"][a]
    count = torch.full((1,), a.numel(), dtype=torch.int32, device=refs.device)
    return {"table": table, "refs": refs, "copies": copies, "count": count, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


# ---- the definitions, in 64 bits -------------------------------------------------------
def _rows_exact(q, k, v, seen, scale):
    """One head: q [r, D], k and v [c, D] in 64 bits, seen bool [r, c]."""
    w = torch.where(seen, scale * (q @ k.T), -math.inf)
    lse = torch.logsumexp(w, 1)
    p = torch.exp(w - torch.where(lse == -math.inf, 0.0, lse)[:, None])
    return p @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "prefill":
        lq, lk = _lens(case)
        if 4.0 * D * case["hq"] * float((lq * lk).sum()) > 3e12:
            return None
        q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
        a = c = 0
        for m, n in zip(lq.tolist(), lk.tolist()):
            seen = torch.ones(m, n, dtype=torch.bool, device="cuda").tril(n - m)
            for h in range(case["hq"]):
                kv = h // (case["hq"] // case["hkv"])
                out[a : a + m, h], lse[a : a + m, h] = _rows_exact(q[a : a + m, h], k[c : c + n, kv], v[c : c + n, kv], seen, s["scale"])
            a, c = a + m, c + n
        return {"out": out, "lse": lse}
    if case["op"] == "decode":
        b, t, page = case["b"], case["t"], case["page"]
        g = case["hq"] // case["hkv"]
        masks = _masks(case).view(np.uint64)
        q = s["q"].double()
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], dtype=torch.float64, device="cuda")
        for i in range(b):
            n = int(s["lens"][i])
            at = s["table"][i, : (n + page - 1) // page].long()
            flat = lambda pages, new: torch.cat([pages[at].transpose(1, 2).reshape(-1, case["hkv"], D)[:n], new[i]]).double().transpose(0, 1)  # noqa: E731
            k, v = flat(s["k_pages"], s["k_new"]), flat(s["v_pages"], s["v_new"])
            tree = np.array([[bool(int(masks[i, x]) >> y & 1) for y in range(t)] for x in range(t)])
            seen = torch.cat([torch.ones(t, n, dtype=torch.bool), torch.from_numpy(tree)], 1).cuda().repeat(g, 1)
            for h in range(case["hkv"]):
                o, x = _rows_exact(q[i, :, h * g : (h + 1) * g].transpose(0, 1).reshape(g * t, D), k[h], v[h], seen, s["scale"])
                out[i, :, h * g : (h + 1) * g] = o.view(g, t, D).transpose(0, 1)
                lse[i, :, h * g : (h + 1) * g] = x.view(g, t).T
        return {"out": out, "lse": lse}
    kp, vp = s["k_pages"].clone(), s["v_pages"].clone()
    table = s["table"].cpu().numpy().copy()
    page = case["page"]
    if case["op"] == "append":
        start = s["start"].tolist()
        for i in range(case["n"]):
            if case["accept"]:
                rows = s["index"][i, : int(s["count"][i])].long()
                k, v = s["k"][i, rows], s["v"][i, rows]
            else:
                k, v = (x[int(s["cu"][i]) : int(s["cu"][i + 1])] for x in (s["k"], s["v"]))
            done = 0
            while done < k.shape[0]:
                off = (start[i] + done) % page
                step = min(page - off, k.shape[0] - done)
                p = int(table[i, (start[i] + done) // page])
                kp[p, :, off : off + step] = k[done : done + step].transpose(0, 1)
                vp[p, :, off : off + step] = v[done : done + step].transpose(0, 1)
                done += step
        return {"k_pages": kp, "v_pages": vp}
    refs = s["refs"].cpu().numpy().copy()
    pairs = []
    if case["op"] == "fork":
        lens = s["lens"].cpu().numpy().copy()
        free = iter(np.flatnonzero(refs == 0).tolist())
        for a, z in zip(s["src"].tolist(), s["dst"].tolist()):
            n = int(lens[a])
            pair = (-1, -1)
            for j in range((n + page - 1) // page):
                p = int(table[a, j])
                if (j + 1) * page > n:
                    pair = (p, next(free))
                    p = pair[1]
                table[z, j] = p
                refs[p] += 1
            lens[z] = n
            pairs.append(pair)
        more = {"lens": torch.from_numpy(lens)}
    else:
        count = int((refs > 0).sum())
        a, z = [p for p in range(count, case["pages"]) if refs[p]], [p for p in range(count) if not refs[p]]
        pairs = list(zip(a, z))
        name = dict(pairs)
        table = np.array([[name.get(p, p) for p in row] for row in table.tolist()], np.int32)
        for p, to in pairs:
            refs[to], refs[p] = refs[p], 0
        more = {"count": torch.tensor([len(pairs)])}
    moved = torch.tensor([p for p in pairs if p[0] >= 0], dtype=torch.int64).view(-1, 2).cuda()
    kp[moved[:, 1]], vp[moved[:, 1]] = s["k_pages"][moved[:, 0]], s["v_pages"][moved[:, 0]]
    pairs += [(-1, -1)] * (case["pages"] - len(pairs) if case["op"] == "compact" else 0)
    return {"table": torch.from_numpy(table), "refs": torch.from_numpy(refs), "copies": torch.tensor(pairs), "k_pages": kp, "v_pages": vp, **more}
