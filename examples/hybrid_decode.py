"""A two-layer hybrid model on the library's kernels: one KDA layer and one
full-attention layer (random weights), through what a server does with them.

  prompts      kda_layer_prologue, kda_prefill, kda_layer_epilogue; kda_attn_prefill;
               the keys and values go to pages (kda_cache_alloc, kda_cache_append)
  fork         every prompt becomes two samples: pages are shared (kda_cache_fork), the
               last, partly filled ones copied, as are the KDA state and the
               convolution window (kda_cache_copy)
  drafts       a few drafted tokens per sample are checked in one call
               (kda_layer_prologue_decode, kda_decode, kda_attn_decode); the accepted
               ones are kept: their keys and values are appended, and the KDA layer
               takes them again from the state before the drafts
  housekeeping finished samples are freed, the pool made dense (kda_cache_free,
               kda_cache_compact, kda_cache_copy)

`python examples/hybrid_decode.py` prints, for each sample, how far its last hidden
state is from that of one prefill over all of its tokens.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kimi_delta_attention_rule_gb300 as kda  # noqa: E402

D, W = 128, 4  # head dimension, width of the short convolutions
BF = torch.bfloat16


def ints(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


class Model:
    """Weights of the two layers; heads of the KDA layer H, of the attention Hq over Hkv."""

    def __init__(self, H=4, Hq=8, Hkv=2, width=512, vocab=97, seed=0, dev="cuda:0"):
        g = torch.Generator().manual_seed(seed)
        rand = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(dev)  # noqa: E731
        self.H, self.Hq, self.Hkv, self.dev, self.vocab = H, Hq, Hkv, dev, vocab
        w = width**-0.5
        self.embed = rand(vocab, width).to(BF)
        self.kda_in = rand(width, 5 * H * D, scale=w).to(BF)  # q, k, v, decay, output gate
        self.kda_beta = rand(width, H, scale=w).to(BF)
        self.conv = [rand(H, D, W, scale=0.5).contiguous() for _ in range(3)]
        self.norm = torch.ones(D, device=dev)
        self.kda_out = rand(H * D, width, scale=(H * D) ** -0.5).to(BF)
        self.qkv = rand(width, (Hq + 2 * Hkv) * D, scale=w).to(BF)
        self.attn_out = rand(Hq * D, width, scale=(Hq * D) ** -0.5).to(BF)
        self.scale = D**-0.5

    def kda_rows(self, x):
        """The KDA layer's projections of x [T, width]: raw rows and beta."""
        rows = (x @ self.kda_in).view(-1, 5, self.H, D)
        return [rows[:, i].contiguous() for i in range(5)], (x @ self.kda_beta).contiguous()

    def qkv_rows(self, x):
        rows = (x @ self.qkv).view(-1, self.Hq + 2 * self.Hkv, D)  # views: the kernels take the stride
        return rows[:, : self.Hq], rows[:, self.Hq : self.Hq + self.Hkv], rows[:, self.Hq + self.Hkv :]


class Server:
    """`rows` sequences at most, on `pages` pages of `page` tokens."""

    def __init__(self, model, rows=8, pages=64, page=16, cols=16):
        m, dev = model, model.dev
        self.m, self.page = m, page
        self.table = torch.full((rows, cols), -1, dtype=torch.int32, device=dev)
        self.lens = torch.zeros(rows, dtype=torch.int32, device=dev)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=dev)
        self.k, self.v = (torch.empty(pages, m.Hkv, page, D, dtype=BF, device=dev) for _ in range(2))
        # entry `row`: a sequence's KDA state and convolution window; entry rows + row: spare
        self.state = torch.zeros(2 * rows, m.H, D, D, device=dev)
        self.window = torch.zeros(2 * rows, 3, W - 1, m.H, D, dtype=BF, device=dev)
        self.rows, self.ws = rows, kda.cache_workspace(self.refs, rows)
        self.tokens = [[] for _ in range(rows)]

    def check(self):
        status = kda.kda_workspace_status(self.ws)
        assert status == kda.KDA_OK, kda.status_string(status)

    def reserve(self, rows, more):
        """Pages for `more` further tokens of each of these rows."""
        want = self.lens.clone()
        want[rows] += more
        kda.kda_cache_alloc(self.table, want, self.refs, self.page, workspace=self.ws)

    def prefill(self, prompts):
        """Prompts (lists of tokens) into rows 0, 1, ..; their last hidden states."""
        m, n = self.m, len(prompts)
        lens = [len(p) for p in prompts]
        cu = ints([sum(lens[:i]) for i in range(n + 1)], m.dev)
        x = m.embed[torch.tensor(sum(prompts, []), device=m.dev)]
        (qr, kr, vr, ar, gate), beta = m.kda_rows(x)
        q, k, v, g, b = kda.kda_layer_prologue(qr, kr, vr, ar, beta, *m.conv, cu_seqlens=cu)
        o, final = kda.kda_prefill(q, k, v, g, b, m.scale, cu_seqlens=cu)
        x = x + kda.kda_layer_epilogue(o, gate, m.norm).view(-1, m.H * D) @ m.kda_out
        self.state[:n] = final
        for i in range(n):  # the last W - 1 raw rows, zeros before the first
            for j, raw in enumerate((qr, kr, vr)):
                last = raw[int(cu[i]) : int(cu[i + 1])][-(W - 1) :]
                self.window[i, j, W - 1 - last.shape[0] :] = last
        q, k, v = m.qkv_rows(x)
        o, _ = kda.kda_attn_prefill(q, k, v, m.scale, cu_seqlens=cu)
        self.reserve(list(range(n)), ints(lens, m.dev))
        kda.kda_cache_append(k, v, self.k, self.v, self.table[:n], self.lens[:n].clone(), cu_seqlens=cu, workspace=self.ws)
        self.lens[:n] = ints(lens, m.dev)
        for i, p in enumerate(prompts):
            self.tokens[i] = list(p)
        x = x + o.reshape(-1, m.Hq * D) @ m.attn_out
        return x[(cu[1:] - 1).long()]

    def fork(self, src, dst):
        dev = self.m.dev
        copies = kda.kda_cache_fork(self.table, self.lens, self.refs, ints(src, dev), ints(dst, dev), self.page,
                                    workspace=self.ws)
        kda.kda_cache_copy([self.k, self.v], copies)
        pairs = ints(list(zip(src, dst)), dev)
        kda.kda_cache_copy([self.state], pairs)
        kda.kda_cache_copy([self.window], pairs)
        for a, z in zip(src, dst):
            self.tokens[z] = list(self.tokens[a])

    def kda_layer(self, rows, tokens):
        """The KDA layer over T tokens [B, T] of these rows, from their states (which move on)."""
        m, (B, T) = self.m, tokens.shape
        x = m.embed[tokens]
        (qr, kr, vr, ar, gate), beta = m.kda_rows(x.view(B * T, -1))
        shape = lambda t: t.view(B, T, m.H, D)  # noqa: E731
        idx = ints(rows, m.dev)
        q, k, v, g, b = kda.kda_layer_prologue_decode(shape(qr), shape(kr), shape(vr), shape(ar), beta.view(B, T, m.H), *m.conv,
                                                      self.window, state_indices=idx)
        o = kda.kda_decode(q, k, v, g, b, m.scale, self.state, state_indices=idx)
        y = kda.kda_layer_epilogue(o.view(B * T, m.H, D), gate, m.norm).view(B, T, m.H * D)
        return x + y @ m.kda_out

    def verify(self, rows, drafts, accepted):
        """Drafts [B, T] of these rows checked in one call, the first accepted[b] of
        them kept. Returns the hidden states [B, T, width]."""
        m, dev = self.m, self.m.dev
        B, T = len(rows), len(drafts[0])
        tokens = torch.tensor(drafts, device=dev)
        keep = ints([(r, self.rows + r) for r in rows], dev)  # the states before the drafts
        for pool in (self.state, self.window):
            kda.kda_cache_copy([pool], keep)
        x = self.kda_layer(rows, tokens)
        q, k, v = (t.view(B, T, -1, D) for t in m.qkv_rows(x.view(B * T, -1)))
        table, lens = self.table[rows].contiguous(), self.lens[rows].contiguous()
        o, _ = kda.kda_attn_decode(q, self.k, self.v, table, lens, m.scale, k_new=k, v_new=v)
        out = x + o.reshape(B, T, m.Hq * D) @ m.attn_out
        # the accepted drafts' keys and values into the pages
        count = ints(accepted, dev)
        self.reserve(rows, count)
        kda.kda_cache_append(k, v, self.k, self.v, self.table[rows].contiguous(), lens, count=count, workspace=self.ws)
        self.lens[rows] += count
        # and into the KDA states, again from those before the drafts
        for pool in (self.state, self.window):
            kda.kda_cache_copy([pool], keep.flip(1).contiguous())
        for a in sorted(set(accepted) - {0}):
            which = [i for i in range(B) if accepted[i] == a]
            self.kda_layer([rows[i] for i in which], tokens[which][:, :a])
        for r, d, a in zip(rows, drafts, accepted):
            self.tokens[r] += d[:a]
        return out

    def finish(self, rows):
        kda.kda_cache_free(self.table, self.lens, self.refs, ints(rows, self.m.dev), workspace=self.ws)
        copies, count = kda.kda_cache_compact(self.table, self.refs, workspace=self.ws)
        kda.kda_cache_copy([self.k, self.v], copies, count)
        for r in rows:
            self.tokens[r] = []


def main(seed=0):
    g = torch.Generator().manual_seed(seed)
    model = Model(seed=seed)
    draw = lambda n: torch.randint(0, model.vocab, (n,), generator=g).tolist()  # noqa: E731
    server = Server(model)
    prompts = [draw(37), draw(16), draw(50)]
    server.prefill(prompts)
    server.fork([0, 1, 2], [3, 4, 5])
    last = {}
    rows = [0, 1, 2, 3, 4, 5]
    for step in range(4):
        T = 4
        accepted = [1 + (r + step) % T for r in rows]
        out = server.verify(rows, [draw(T) for _ in rows], accepted)
        for i, r in enumerate(rows):
            last[r] = out[i, accepted[i] - 1]
        if step == 1:
            server.finish([1, 4])
            rows = [0, 2, 3, 5]
            del last[1], last[4]
    server.check()
    errors = {}
    for r in rows:  # one prefill over all of the sample's tokens, on a server of its own
        ref = Server(model, rows=1).prefill([server.tokens[r]])[0].float()
        errors[r] = float((last[r].float() - ref).norm() / ref.norm())
    return server, errors


if __name__ == "__main__":
    server, errors = main()
    for r, e in errors.items():
        print("sample %d: %d tokens, last hidden state %.4f from one prefill over them" % (r, len(server.tokens[r]), e))
