"""A serving loop with bounded contexts: prompts, their weights, eviction to other pages, forks, drafts with
accepted tokens, eviction in place and trimming, against a mirror that holds every kv head's rows itself
and computes attention and weights in 64 bits. What stays is checked by the definition on the
kernel's own weights; those, and all attention outputs, are held to the bounds of attn_ref and
test_attn_weights."""
import math

import pytest
import torch

import kimi_delta_attention_rule_gb300 as kda
from tests import attn_ref
from tests.test_attn_decode import BF, DEV, F32, SCALE, normal, tree_masks
from tests.test_cache_evict import staying

pytestmark = pytest.mark.gpu
HQ, HKV, PAGE, ROWS, COLS, PAGES = 6, 2, 16, 6, 24, 120
G = HQ // HKV
SINKS, RECENT = 4, 12


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Mirror:
    """Per row and kv head: k, v [n, 128] and weights [n] in 64 bits with their bound."""

    def __init__(self):
        self.k, self.v, self.w, self.e = ({} for _ in range(4))

    def add(self, b, h, k, v):
        z = torch.zeros(k.shape[0], dtype=torch.float64, device=DEV)
        for store, x in ((self.k, k), (self.v, v), (self.w, z), (self.e, z)):
            store[b, h] = torch.cat([store[b, h], x]) if (b, h) in store else x.clone()

    def weigh(self, b, h, q, lse):
        """q [c, G, 128], lse [c, G]: of the last c tokens."""
        k = self.k[b, h].double()
        n, c = k.shape[0], q.shape[0]
        seen = torch.arange(n, device=DEV)[None] <= n - c + torch.arange(c, device=DEV)[:, None]
        for g in range(G):
            s = SCALE * (q[:, g].double() @ k.T)
            p = torch.where(seen, torch.exp(s - lse[:, g].double()[:, None]), 0.0)
            e0 = 136 * 2 * 2.0**-24 * SCALE * (q[:, g].double().abs() @ k.abs().T)
            e = e0 + 4 * 2.0**-24 * (s.abs() + lse[:, g].double().abs()[:, None]) + 2.0**-21 + c * G * 2.0**-24
            self.w[b, h] = self.w[b, h] + p.sum(0)
            self.e[b, h] = self.e[b, h] + (1.1 * e * p).sum(0) + 2.0**-24 * self.w[b, h]


def check_weights(m, w, rows):
    for b in rows:
        for h in range(HKV):
            n = m.w[b, h].shape[0]
            assert ((w[b, h, :n].double() - m.w[b, h]).abs() <= m.e[b, h] + 2.0**-24 * m.w[b, h]).all()
            assert (w[b, h, n:] == 0).all()


def check_kept(m, w, kept, keep):
    """The choice by the definition on the kernel's weights w; the mirror follows."""
    for b, budget in enumerate(keep):
        for h in range(HKV if budget >= 0 and (b, 0) in m.k else 0):
            n = m.k[b, h].shape[0]
            want = staying(w[b, h, :n].tolist(), n, budget, SINKS, RECENT)
            if n > budget or kept is not None:
                assert kept[b, h, :len(want)].tolist() == want
            at = torch.tensor(want, dtype=torch.long, device=DEV)
            for store in (m.k, m.v, m.w, m.e):
                store[b, h] = store[b, h][at]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("window", [None, 40])
def test_serving_loop(dt, window):
    lens = [150, 37, 90]
    n = len(lens)
    table = torch.full((ROWS, COLS), -1, dtype=torch.int32, device=DEV)
    length, refs = torch.zeros(ROWS, dtype=torch.int32, device=DEV), torch.zeros(PAGES, dtype=torch.int32, device=DEV)
    kp, vp = (torch.full((PAGES, HKV, PAGE, 128), math.nan, device=DEV, dtype=dt) for _ in range(2))
    w = torch.zeros(ROWS, HKV, COLS * PAGE, device=DEV)
    ws, ews = kda.cache_workspace(refs, ROWS), kda.evict_workspace(w)
    m = Mirror()

    def fine():
        assert kda.kda_workspace_status(ws) == kda.KDA_OK and kda.kda_workspace_status(ews) == kda.KDA_OK

    # prompts
    T = sum(lens)
    q, k, v = normal(1, (T, HQ, 128), dt, 2.0), normal(2, (T, HKV, 128), dt), normal(3, (T, HKV, 128), dt)
    cu = ints([sum(lens[:i]) for i in range(n + 1)])
    _, lse = kda.kda_attn_prefill(q, k, v, SCALE, cu_seqlens=cu, output_lse=True)
    length[:n] = ints(lens)
    kda.kda_cache_alloc(table, length, refs, PAGE, workspace=ws)
    kda.kda_cache_append(k, v, kp, vp, table[:n], ints([0] * n), cu_seqlens=cu, workspace=ws)
    # what their last 32 tokens look at
    last = torch.stack([torch.arange(int(cu[i + 1]) - 32, int(cu[i + 1]), device=DEV) for i in range(n)])
    kda.kda_attn_weights(q[last], kp, table[:n], length[:n].clone(), lse[last].contiguous(), SCALE, w[:n])
    for b in range(n):
        for h in range(HKV):
            rows = slice(int(cu[b]), int(cu[b + 1]))
            m.add(b, h, k[rows, h], v[rows, h])
            m.weigh(b, h, q[last[b], h * G:(h + 1) * G], lse[last[b], h * G:(h + 1) * G])
    check_weights(m, w, range(n))

    # row 2 is forked to row 4; then all are cut to 60 tokens on other pages
    copies = kda.kda_cache_fork(table, length, refs, ints([2]), ints([4]), PAGE, workspace=ws)
    kda.kda_cache_copy([kp, vp], copies)
    kda.kda_cache_copy([w], ints([[2, 4]]))
    for h in range(HKV):
        for store in (m.k, m.v, m.w, m.e):
            store[4, h] = store[2, h].clone()
    keep = [60] * ROWS
    dst = torch.full((ROWS, 4), -1, dtype=torch.int32, device=DEV)
    kda.kda_cache_alloc(dst, length.clamp(max=60), refs, PAGE, workspace=ws)
    before = w.clone()
    kept = kda.kda_cache_evict(kp, vp, w, table, length, ints(keep), SINKS, RECENT, dst_table=dst, refs=refs, workspace=ews)
    check_kept(m, before, kept, keep)
    kda.kda_cache_free(table, length, refs, ints([0, 1, 2, 4]), workspace=ws)
    table[:, :4] = dst
    length.copy_(ints([min(60, x) for x in (150, 37, 90, 0, 90, 0)]))
    fine()
    assert int(refs.sum()) == int((table >= 0).sum()) and int(refs.max()) == 1
    check_weights(m, w, [0, 1, 2, 4])

    # steps of four drafts, of which some are accepted; a row past 70 tokens is cut to 50 in place
    live, tokens = ints([0, 1, 2, 4]).long(), 4
    for step in range(8):
        B = len(live)
        qs, ks, vs = (normal(100 * step + i, (B, tokens, heads, 128), dt, s) for i, heads, s in ((1, HQ, 2.0), (2, HKV, 1.0), (3, HKV, 1.0)))
        mask = tree_masks(B, tokens, 7 + step)
        t_b, l_b = table[live].contiguous(), length[live].contiguous()
        if window is None:
            out, lse = kda.kda_attn_decode(qs, kp, vp, t_b, l_b, SCALE, k_new=ks, v_new=vs, tree_mask=mask, output_lse=True)
        else:
            out, lse = kda.kda_attn_decode_window(qs, kp, vp, t_b, l_b, SCALE, window, SINKS, k_new=ks, v_new=vs, tree_mask=mask,
                                                  output_lse=True)
        for i, b in enumerate(live.tolist()):
            tree = torch.tensor([[bool(int(x) >> s & 1) for s in range(tokens)] for x in mask[i].tolist()], device=DEV)
            for h in range(HKV):
                c = m.k[b, h].shape[0]
                j = torch.arange(c, device=DEV)[None]
                seen = torch.ones(tokens, c, dtype=torch.bool, device=DEV)
                if window is not None:
                    seen = (j >= (c - window + tree.sum(1))[:, None]) | (j < SINKS)
                seen = torch.cat([seen, tree], 1)
                kk, vv = torch.cat([m.k[b, h], ks[i, :, h]]), torch.cat([m.v[b, h], vs[i, :, h]])
                for g in range(h * G, (h + 1) * G):
                    attn_ref.check(out[i, :, g], lse[i, :, g], attn_ref.attend(qs[i, :, g], kk, vv, seen, SCALE))
        # the path from the root to the last draft is accepted
        paths = [[s for s in range(tokens) if int(x[-1]) >> s & 1] for x in mask.tolist()]
        index = ints([p + [0] * (tokens - len(p)) for p in paths])
        count = ints([len(p) for p in paths])
        want = length.clone()
        want[live] += count
        kda.kda_cache_alloc(table, want, refs, PAGE, workspace=ws)
        kda.kda_cache_append(ks, vs, kp, vp, table[live].contiguous(), l_b, index=index, count=count, workspace=ws)
        length.copy_(want)
        part = w[live].contiguous()
        kda.kda_attn_weights(qs, kp, table[live].contiguous(), length[live].contiguous(), lse, SCALE, part, index=index, count=count)
        w[live] = part
        for i, b in enumerate(live.tolist()):
            for h in range(HKV):
                m.add(b, h, ks[i, paths[i], h], vs[i, paths[i], h])
                m.weigh(b, h, qs[i, paths[i], h * G:(h + 1) * G], lse[i, paths[i], h * G:(h + 1) * G])
        check_weights(m, w, live.tolist())
        keep = [50 if x > 70 else -1 for x in length.tolist()]
        before = w.clone()
        kept = kda.kda_cache_evict(kp, vp, w, table, length, ints(keep), SINKS, RECENT, refs=refs, workspace=ews)
        check_kept(m, before, kept, keep)
        kda.kda_cache_trim(table, length, refs, ints(keep), PAGE, workspace=ws)
        fine()
        assert length.tolist() == [m.k[b, 0].shape[0] if (b, 0) in m.k else 0 for b in range(ROWS)]
        assert ((table >= 0).sum(1) == (length + PAGE - 1) // PAGE).all() and int(refs.sum()) == int((table >= 0).sum())
        check_weights(m, w, live.tolist())
    assert max(length.tolist()) <= 74
    for b in live.tolist():
        for h in range(HKV):
            c = m.k[b, h].shape[0]
            at = torch.arange(c, device=DEV)
            pages = table[b].long()[at // PAGE]
            assert torch.equal(kp[pages, h, at % PAGE], m.k[b, h]) and torch.equal(vp[pages, h, at % PAGE], m.v[b, h])
