"""kda_cache_evict and kda_cache_trim against plain definitions: which tokens stay (ties, NaN, infinities,
signed zeros, budgets and protected ends of any size), where they go (in place and to other pages),
what is left alone, shared pages, malformed rows, and their refusals. All results are exact."""
import ctypes
import math

import pytest
import torch

import kimi_delta_attention_rule_gb300 as kda
from kimi_delta_attention_rule_gb300 import build as kbuild

OK, INVALID, UNSUPPORTED = kda.KDA_OK, kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
FAKE, ODD = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100008)


def test_refusals():
    kbuild.build()
    lib = kda.load()
    need = kda.kda_cache_evict_workspace_size(4)
    assert need >= 256 and kda.kda_cache_evict_workspace_size(-1) == 0

    def f(**kw):
        a = dict(kp=FAKE, vp=FAKE, P=9, page=16, t=FAKE, ld=5, rows=4, cols=5, dst=None, dld=0, dcols=0, refs=None, lens=FAKE,
                 keep=FAKE, sinks=1, recent=2, Hkv=2, D=128, io=0, w=FAKE, wo=FAKE, kept=FAKE, cap=80, ws=FAKE, nbytes=need)
        a.update(kw)
        return lib.kda_cache_evict(*a.values(), None)
    for kw in (dict(D=64), dict(io=5), dict(page=8), dict(page=40)):
        assert f(**kw) == UNSUPPORTED, kw
    for kw in (dict(Hkv=0), dict(P=-1), dict(rows=-1), dict(cols=-1), dict(ld=4), dict(sinks=-1), dict(recent=-1), dict(cap=-1),
               dict(dst=ctypes.c_void_p(0x200000), dcols=3, dld=2), dict(dst=ctypes.c_void_p(0x200000), dcols=-1),
               dict(dst=FAKE, dcols=3, dld=5), dict(dst=FAKE, dcols=5, dld=6), dict(kp=None), dict(vp=None), dict(t=None), dict(lens=None),
               dict(keep=None), dict(w=None), dict(wo=None), dict(kept=None), dict(ws=None), dict(kp=ODD), dict(vp=ODD), dict(ws=ODD),
               dict(nbytes=need - 1), dict(w=ctypes.c_void_p(0x100002)), dict(P=1 << 27), dict(rows=1 << 25), dict(cols=1 << 24, ld=1 << 24, page=256)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(rows=0), dict(cap=0), dict(P=0), dict(cols=0)):
        assert f(**{**kw, "kp": None}) == OK, kw

    def g(**kw):
        a = dict(t=FAKE, ld=5, rows=4, cols=5, lens=FAKE, refs=FAKE, P=9, page=16, want=FAKE, ws=FAKE, nbytes=1 << 20)
        a.update(kw)
        return lib.kda_cache_trim(*a.values(), None)
    for kw in (dict(rows=-1), dict(cols=-1), dict(ld=4), dict(P=-1), dict(page=0), dict(t=None), dict(refs=None), dict(lens=None),
               dict(want=None), dict(ws=None), dict(ws=ODD), dict(nbytes=16), dict(refs=ODD)):
        assert g(**kw) == INVALID, kw
    assert g(rows=0) == OK and g(cols=0) == OK


# ---- the definition ------------------------------------------------------------------
def staying(w, n, keep, sinks, recent):
    """Slots of one head that stay: w a list of n weights."""
    if n <= keep:
        return list(range(n))
    a = min(sinks, keep)
    z = min(recent, keep - a)
    order = sorted(range(a, n - z), key=lambda i: (not math.isnan(w[i]), -(0.0 if math.isnan(w[i]) else w[i]), i))
    return sorted(list(range(a)) + order[:keep - a - z] + list(range(n - z, n)))


class Cache:
    """Sequences of these lengths on shuffled pages, every row and weight its own value; `spare` further pages."""

    def __init__(self, lens, page=16, hkv=2, dt=BF, seed=0, spare=0, cols=None, cap=None, weights=None):
        g = torch.Generator().manual_seed(seed)
        used = [(n + page - 1) // page for n in lens]
        P = sum(used) + spare
        order = torch.randperm(P, generator=g).int()
        cols = cols or max(used + [1])
        self.table = torch.full((len(lens), cols), -1, dtype=torch.int32)
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = order[at:at + u]
            at += u
        self.table = self.table.to(DEV)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.refs = torch.zeros(P, dtype=torch.int32, device=DEV)
        self.refs[order[:at].long().to(DEV)] = 1
        self.page, self.hkv = page, hkv
        gd = torch.Generator(device=DEV).manual_seed(seed + 1)
        self.kp, self.vp = (torch.randn(P, hkv, page, 128, generator=gd, device=DEV).to(dt) for _ in range(2))
        cap = cap or max(cols * page, 1)
        self.w = torch.exp(2 * torch.randn(len(lens), hkv, cap, generator=gd, device=DEV))
        if weights is not None:
            weights(self.w)
        self.ws = kda.evict_workspace(self.w)

    def row(self, pool, table, b, i):
        return pool[int(table[b, i // self.page]), :, i % self.page]

    def expect(self, keep, sinks, recent, table=None, rows=None):
        """What the call leaves: pools, weights, kept."""
        table = self.table if table is None else table
        kp, vp, w = self.kp.clone(), self.vp.clone(), self.w.clone()
        kept = torch.full(w.shape, -1, dtype=torch.int32, device=DEV)
        lens, ws = self.lens.tolist(), self.w.tolist()
        old, new = self.table.long(), table.long()
        for b in range(len(lens)) if rows is None else rows:
            if keep[b] < 0:
                continue
            for h in range(self.hkv):
                stay = torch.tensor(staying(ws[b][h][:lens[b]], lens[b], keep[b], sinks, recent), dtype=torch.long, device=DEV)
                n = len(stay)
                to = torch.arange(n, device=DEV)
                kept[b, h, :n] = stay.int()
                w[b, h, :lens[b]] = 0
                w[b, h, :n] = self.w[b, h, stay]
                for pool, was in ((kp, self.kp), (vp, self.vp)):
                    pool[new[b, to // self.page], h, to % self.page] = was[old[b, stay // self.page], h, stay % self.page]
        return kp, vp, w, kept

    def evict(self, keep, sinks, recent, **kw):
        kept = kda.kda_cache_evict(self.kp, self.vp, self.w, self.table, self.lens,
                                   torch.tensor(keep, dtype=torch.int32, device=DEV), sinks, recent, workspace=self.ws, **kw)
        return kept, kda.kda_workspace_status(self.ws)


def same(a, b):  # bit for bit (NaN too)
    whole = {BF: torch.int16, F32: torch.int32}.get(a.dtype, a.dtype)
    return torch.equal(a.view(whole), b.view(whole))


def in_place(c, keep, sinks, recent, **kw):
    want = c.expect(keep, sinks, recent)
    kept, st = c.evict(keep, sinks, recent, **kw)
    assert st == OK
    for x, y in zip((c.kp, c.vp, c.w, kept), want):
        assert same(x, y)


def elsewhere(c, keep, sinks, recent, cols=None, **kw):
    lens = c.lens.tolist()
    n = [min(a, max(k, 0)) for a, k in zip(lens, keep)]
    dst = torch.full((len(lens), cols or max([(x + c.page - 1) // c.page for x in n] + [1])), -1, dtype=torch.int32, device=DEV)
    kda.kda_cache_alloc(dst, torch.tensor(n, dtype=torch.int32, device=DEV), c.refs, c.page)
    want = c.expect(keep, sinks, recent, dst)
    out = c.w.clone()
    before = c.w.clone()
    kept, st = c.evict(keep, sinks, recent, dst_table=dst, weights_out=out, refs=c.refs, **kw)
    assert st == OK and same(c.w, before)
    for x, y in zip((c.kp, c.vp, out, kept), want):
        assert same(x, y)


LENS = [0, 1, 15, 16, 17, 100, 128, 300, 777]


@pytest.mark.gpu
@pytest.mark.parametrize("how", [in_place, elsewhere])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_budgets(page, dt, how):
    for keep, sinks, recent in ((64, 4, 16), (1, 0, 0), (0, 4, 4), (777, 1, 1), (130, 0, 130), (99, 99, 0), (50, 30, 40), (2**31 - 1, 2, 2)):
        how(Cache(LENS, page, 2, dt, seed=keep & 255, spare=100), [keep] * len(LENS), sinks, recent)


@pytest.mark.gpu
@pytest.mark.parametrize("how", [in_place, elsewhere])
@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_a_budget_for_each_row(hkv, how):
    how(Cache(LENS, 16, hkv, BF, seed=3, spare=120), [0, 1, 15, -1, 3, 100, 40, -7, 512], 2, 3)


def ties(w):
    w.copy_(torch.floor(w * 0.7).clamp(max=3.0))


def odd_values(w):
    flat = w.view(-1)
    for i, v in enumerate((math.nan, math.inf, -math.inf, -0.0, 0.0, -1.0, 1e-45, -1e-45, 3e38)):
        flat[i::11] = v


@pytest.mark.gpu
@pytest.mark.parametrize("how", [in_place, elsewhere])
@pytest.mark.parametrize("fill", [ties, odd_values, lambda w: w.zero_(), lambda w: w.fill_(math.nan), lambda w: w.fill_(7.0)])
def test_equal_and_odd_weights(fill, how):
    for keep in (1, 37, 120, 299):
        how(Cache([300, 55, 128], 16, 2, BF, seed=4, spare=60, weights=fill), [keep] * 3, 5, 11)


@pytest.mark.gpu
@pytest.mark.parametrize("how", [in_place, elsewhere])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("lens,keep", [([9000], 5000), ([4096, 4097, 8191], 4095), ([20000], 19999), ([13000], 17)])
def test_long_rows(lens, keep, dt, how):
    """Several rounds of the choice, many chunks of moves; in place, CTAs that share a row's bytes."""
    how(Cache(lens, 64, 1, dt, seed=5, spare=sum(lens) // 64 + 4), [keep] * len(lens), 4, min(64, keep // 2))


@pytest.mark.gpu
@pytest.mark.parametrize("how", [in_place, elsewhere])
@pytest.mark.parametrize("fill", [lambda w: None, ties, odd_values])
@pytest.mark.parametrize("length,keep", [(30001, 9001), (49149, 40001), (49152, 127), (49153, 49100), (60001, 20011)])
def test_rows_about_what_a_block_holds(length, keep, fill, how):
    """49,152 weights lie in shared memory, the rest is read again; equal ones across all of it."""
    how(Cache([length, 4099], 256, 1, BF, seed=length % 91, spare=260, weights=fill), [keep, keep], 5, 33)


@pytest.mark.gpu
@pytest.mark.parametrize("how", [in_place, elsewhere])
@pytest.mark.parametrize("rows,most", [(90, 120), (90, 400), (25, 2600)])
def test_many_rows(rows, most, how):
    g = torch.Generator().manual_seed(6)
    lens = torch.randint(0, most, (rows,), generator=g).tolist()
    keep = torch.randint(-1, most * 3 // 4, (rows,), generator=g).tolist()
    how(Cache(lens, 16, 8, BF, seed=6, spare=3000), keep, 4, 10)


@pytest.mark.gpu
def test_weights_past_the_length_are_left_alone():
    c = Cache([100], 16, 1, BF, seed=7, cap=133)
    tail = c.w[..., 100:].clone()
    in_place(c, [40], 1, 1)
    assert torch.equal(c.w[..., 100:], tail) and (c.w[..., 40:100] == 0).all()


@pytest.mark.gpu
def test_the_same_table_is_in_place():
    for lens in ([500, 60], [9000]):
        c = Cache(lens, 16, 2, BF, seed=15)
        in_place(c, [40] * len(lens), 3, 20, dst_table=c.table)


@pytest.mark.gpu
def test_twice_in_a_row_and_captured():
    c = Cache([500, 333], 16, 2, BF, seed=8)
    in_place(c, [200, 300], 3, 20)
    c.lens.copy_(torch.tensor([200, 300], dtype=torch.int32))
    in_place(c, [150, 10], 3, 5)
    c.lens.copy_(torch.tensor([150, 10], dtype=torch.int32))
    want = c.expect([60, 10], 3, 5)
    keep = torch.tensor([60, 10], dtype=torch.int32, device=DEV)
    kept = torch.full(c.w.shape, -1, dtype=torch.int32, device=DEV)
    state = [t.clone() for t in (c.kp, c.vp, c.w)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_cache_evict(c.kp, c.vp, c.w, c.table, c.lens, keep, 3, 5, kept=kept, workspace=c.ws)
    for t, s in zip((c.kp, c.vp, c.w), state):
        t.copy_(s)
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip((c.kp, c.vp, c.w, kept), want):
        assert same(x, y)


@pytest.mark.gpu
def test_shared_pages_are_refused_in_place_and_read_elsewhere():
    c = Cache([100, 60, 0], 16, 2, BF, seed=9, spare=30)
    copies = kda.kda_cache_fork(c.table, c.lens, c.refs, torch.tensor([0], dtype=torch.int32, device=DEV),
                                torch.tensor([2], dtype=torch.int32, device=DEV), c.page)
    kda.kda_cache_copy([c.kp, c.vp], copies)
    c.w[2] = c.w[0].flip(-1)
    keep = [30, 30, 50]
    want = c.expect(keep, 2, 4, rows=[1])
    kept, st = c.evict(keep, 2, 4, refs=c.refs)
    assert st == kda.KDA_ERR_DEVICE
    for x, y in zip((c.kp, c.vp, c.w, kept), want):
        assert same(x, y)
    c.lens[1] = 30
    elsewhere(c, keep, 2, 4)


@pytest.mark.gpu
def test_malformed_rows_are_skipped_and_flagged():
    for spoil in (lambda c: c.lens.__setitem__(1, -1), lambda c: c.lens.__setitem__(1, 16 * c.table.shape[1] + 1),
                  lambda c: c.table.__setitem__((1, 4), -1), lambda c: c.table.__setitem__((1, 0), c.kp.shape[0]),
                  lambda c: c.table.__setitem__((1, 5), 2**31 - 1)):
        c = Cache([100, 90, 70], 16, 2, BF, seed=10)
        spoil(c)
        want = c.expect([40] * 3, 2, 4, rows=[0, 2])
        kept, st = c.evict([40] * 3, 2, 4)
        assert st == kda.KDA_ERR_DEVICE
        for x, y in zip((c.kp, c.vp, c.w, kept), want):
            assert same(x, y)
    c = Cache([100, 90, 70], 16, 2, BF, seed=11, cap=99)  # the first row has no room for its weights
    want = c.expect([40] * 3, 2, 4, rows=[1, 2])
    kept, st = c.evict([40] * 3, 2, 4)
    assert st == kda.KDA_ERR_DEVICE
    for x, y in zip((c.kp, c.vp, c.w, kept), want):
        assert same(x, y)
    c = Cache([100, 90, 70], 16, 2, BF, seed=12, spare=9)
    dst = torch.full((3, 3), -1, dtype=torch.int32, device=DEV)
    kda.kda_cache_alloc(dst, torch.tensor([40, 20, 40], dtype=torch.int32, device=DEV), c.refs, 16)  # row 1: a page too few
    want = c.expect([40] * 3, 2, 4, dst, rows=[0, 2])
    kept, st = c.evict([40] * 3, 2, 4, dst_table=dst)
    assert st == kda.KDA_ERR_DEVICE
    for x, y in zip((c.kp, c.vp, c.w, kept), want):
        assert same(x, y)


@pytest.mark.gpu
def test_trim():
    c = Cache([100, 60, 0, 64, 33], 16, 1, BF, seed=13, spare=30, cols=9)
    kda.kda_cache_fork(c.table, c.lens, c.refs, torch.tensor([0], dtype=torch.int32, device=DEV),
                       torch.tensor([2], dtype=torch.int32, device=DEV), 16)
    kda.kda_cache_alloc(c.table, torch.tensor([0, 0, 0, 100, 0], dtype=torch.int32, device=DEV), c.refs, 16)  # ahead of its length
    want = [33, 200, 0, 64, -1]
    table, refs, lens = c.table.clone(), c.refs.clone(), c.lens.clone()
    for r, n in enumerate(want):
        if n < 0:
            continue
        lens[r] = min(int(lens[r]), n)
        for j in range((n + 15) // 16, 9):
            if table[r, j] >= 0:
                refs[table[r, j].long()] -= 1
                table[r, j] = -1
    ws = kda.cache_workspace(c.refs)
    kda.kda_cache_trim(c.table, c.lens, c.refs, torch.tensor(want, dtype=torch.int32, device=DEV), 16, workspace=ws)
    assert kda.kda_workspace_status(ws) == OK
    assert torch.equal(c.table, table) and torch.equal(c.refs, refs) and torch.equal(c.lens, lens)
    c.table[1, 2] = c.kp.shape[0] + 5
    kda.kda_cache_trim(c.table, c.lens, c.refs, torch.tensor([-1, 16, -1, -1, -1], dtype=torch.int32, device=DEV), 16, workspace=ws)
    assert kda.kda_workspace_status(ws) == kda.KDA_ERR_DEVICE and c.table[1].tolist()[1:] == [-1] * 8 and c.lens[1] == 16


@pytest.mark.gpu
def test_python_refusals():
    c = Cache([40, 50], 16, 2, BF, seed=14)
    keep = torch.tensor([9, 9], dtype=torch.int32, device=DEV)
    call = lambda **kw: kda.kda_cache_evict(**{**dict(k_pages=c.kp, v_pages=c.vp, weights=c.w, block_table=c.table, seq_lens=c.lens,  # noqa: E731
                                                      keep=keep), **kw})
    for kw in (dict(v_pages=c.vp.float()), dict(weights=c.w[:1]), dict(weights=c.w.double()), dict(weights=c.w[..., ::2]), dict(keep=keep[:1]),
               dict(keep=keep.long()), dict(seq_lens=c.lens[:1]), dict(dst_table=c.table[:1]), dict(refs=c.refs[:-1]), dict(kept=c.w),
               dict(weights_out=c.w[..., :-1].contiguous()), dict(dst_table=torch.zeros(2, 0, dtype=torch.int32, device=DEV))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(sinks=-1), dict(recent=-1), dict(k_pages=c.kp.half(), v_pages=c.vp.half())):
        with pytest.raises(kda.KDAError):
            call(**kw)
