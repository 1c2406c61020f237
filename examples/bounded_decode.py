"""Attention with a bounded context (random weights): one layer that reads a sliding window
and gives back the pages behind it, and one that keeps the tokens which get the most attention.

  windowed   kda_attn_prefill_window, then kda_attn_decode_window token by token; a page that has left
             the window is given back (KDA_PAGE_GONE in the block table keeps its place)
  evicting   kda_attn_prefill, its weights from the prompt's last tokens (kda_attn_weights), the cut to a
             budget (kda_cache_evict, kda_cache_trim); then per token kda_attn_decode,
             kda_cache_append, kda_attn_weights, and a cut whenever a sequence has grown past it

`python examples/bounded_decode.py` prints, for each layer, the pages in use at the end and how
far its outputs are from those over the whole context.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kimi_delta_attention_rule_gb300 as kda  # noqa: E402

D, PAGE, BF = 128, 16, torch.bfloat16
SCALE = D**-0.5


class Cache:
    """The pages of `rows` sequences of at most `cols` pages each, filled with prompts."""

    def __init__(self, k, v, lens, cu, cols):
        dev, n = k.device, len(lens)
        self.table = torch.full((n, cols), -1, dtype=torch.int32, device=dev)
        self.refs = torch.zeros(n * cols, dtype=torch.int32, device=dev)
        self.k, self.v = (torch.zeros(n * cols, k.shape[1], PAGE, D, dtype=BF, device=dev) for _ in range(2))
        self.lens = torch.tensor(lens, dtype=torch.int32, device=dev)
        self.ws = kda.cache_workspace(self.refs, n)
        kda.kda_cache_alloc(self.table, self.lens, self.refs, PAGE, workspace=self.ws)
        kda.kda_cache_append(k, v, self.k, self.v, self.table, torch.zeros_like(self.lens), cu_seqlens=cu, workspace=self.ws)

    def append(self, k, v):
        kda.kda_cache_alloc(self.table, self.lens + 1, self.refs, PAGE, workspace=self.ws)
        kda.kda_cache_append(k, v, self.k, self.v, self.table, self.lens, workspace=self.ws)
        self.lens += 1

    def give_back(self, out):
        """Pages out (bool, as the table) leave their rows; those behind them keep their places."""
        out = out & (self.table >= 0)
        self.refs.index_add_(0, self.table.clamp(min=0).flatten().long(), -out.flatten().int())
        self.table.masked_fill_(out, kda.KDA_PAGE_GONE)

    def free(self):
        kda.kda_cache_free(self.table, self.lens, self.refs, torch.arange(len(self.lens), dtype=torch.int32, device=self.lens.device),
                           workspace=self.ws)

    def check(self):
        status = kda.kda_workspace_status(self.ws)
        assert status == kda.KDA_OK, kda.status_string(status)


def windowed(prompt, steps, window=64, sinks=4):
    """Outputs [steps, n, Hq, D] of the tokens after the prompts, and the cache."""
    (q, k, v), lens, cu = prompt
    kda.kda_attn_prefill_window(q, k, v, SCALE, window, sinks, cu_seqlens=cu)
    c = Cache(k, v, lens, cu, (max(lens) + len(steps)) // PAGE + 1)
    cols, kept_sinks = torch.arange(c.table.shape[1], device=k.device), (sinks + PAGE - 1) // PAGE
    outs = []
    for q, k, v in steps:
        outs.append(kda.kda_attn_decode_window(q, c.k, c.v, c.table, c.lens, SCALE, window, sinks, k_new=k, v_new=v)[0][:, 0])
        c.append(k, v)
        # the next token's window starts at lens + 1 - window: pages that end before it go back
        c.give_back((cols >= kept_sinks) & ((cols + 1) * PAGE <= (c.lens + 1 - window)[:, None]))
    c.check()
    return torch.stack(outs), c


def evicting(prompt, steps, budget=64, slack=16, sinks=4, recent=16, observed=16):
    (q, k, v), lens, cu = prompt
    _, lse = kda.kda_attn_prefill(q, k, v, SCALE, cu_seqlens=cu, output_lse=True)
    c = Cache(k, v, lens, cu, max(max(lens), budget + slack + 1) // PAGE + 2)
    weights = torch.zeros(len(lens), k.shape[1], c.table.shape[1] * PAGE, device=k.device)
    space = kda.evict_workspace(weights)
    last = cu[1:, None].long() - observed + torch.arange(observed, device=k.device)
    kda.kda_attn_weights(q[last], c.k, c.table, c.lens, lse[last].contiguous(), SCALE, weights)

    def cut(limit):
        keep = torch.where(c.lens > limit, budget, -1).int()
        kda.kda_cache_evict(c.k, c.v, weights, c.table, c.lens, keep, sinks, recent, refs=c.refs, workspace=space)
        kda.kda_cache_trim(c.table, c.lens, c.refs, keep, PAGE, workspace=c.ws)

    cut(budget)
    outs = []
    for q, k, v in steps:
        out, lse = kda.kda_attn_decode(q, c.k, c.v, c.table, c.lens, SCALE, k_new=k, v_new=v, output_lse=True)
        outs.append(out[:, 0])
        c.append(k, v)
        kda.kda_attn_weights(q, c.k, c.table, c.lens, lse, SCALE, weights)
        cut(budget + slack)
    c.check()
    assert kda.kda_workspace_status(space) == kda.KDA_OK
    return torch.stack(outs), c


def whole(prompt, steps):
    (_, k, v), lens, cu = prompt
    c = Cache(k, v, lens, cu, (max(lens) + len(steps)) // PAGE + 1)
    outs = []
    for q, k, v in steps:
        outs.append(kda.kda_attn_decode(q, c.k, c.v, c.table, c.lens, SCALE, k_new=k, v_new=v)[0][:, 0])
        c.append(k, v)
    return torch.stack(outs), c


def main(seed=0, lens=(150, 40, 333), tokens=40, hq=8, hkv=2, dev="cuda:0"):
    g = torch.Generator().manual_seed(seed)
    rows = lambda *shape: torch.randn(*shape, D, generator=g).to(dev).to(BF)  # noqa: E731
    heads = lambda *shape: (rows(*shape, hq), rows(*shape, hkv), rows(*shape, hkv))  # noqa: E731
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=dev)
    prompt = (heads(sum(lens)), list(lens), cu)
    steps = [heads(len(lens), 1) for _ in range(tokens)]
    ref, full = whole(prompt, steps)
    results = {"whole": (0.0, int((full.refs > 0).sum()), full)}
    for name, layer in (("windowed", windowed), ("evicting", evicting)):
        out, cache = layer(prompt, steps)
        error = float((out.float() - ref.float()).norm() / ref.float().norm())
        results[name] = (error, int((cache.refs > 0).sum()), cache)
    return results


if __name__ == "__main__":
    for name, (error, pages, _) in main().items():
        print("%-9s %3d pages in use, outputs %.3f from those over the whole context" % (name, pages, error))
