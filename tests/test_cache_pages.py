"""The kda_cache_* calls against plain loops: every result is a whole number or
a copy, so all are compared for equality."""
import random

import pytest
import torch

import kimi_delta_attention_rule_gb300 as kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Model:
    """The cache's bookkeeping in plain Python."""

    def __init__(self, pages, rows, cols, page):
        self.page, self.cols = page, cols
        self.refs, self.table, self.lens = [0] * pages, [[-1] * cols for _ in range(rows)], [0] * rows

    def free_pages(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def alloc(self, want):
        need = []
        for r, w in zip(self.table, want):
            used = sum(e >= 0 for e in r)
            need.append(max(0, -(-w // self.page) - used))
        free = self.free_pages()
        if sum(need) > len(free):
            return False
        for r, n in zip(self.table, need):
            used = sum(e >= 0 for e in r)
            for e in range(n):
                r[used + e] = free.pop(0)
                self.refs[r[used + e]] = 1
        return True

    def fork(self, src, dst):
        free, pairs = self.free_pages(), []
        if sum(1 for a, z in zip(src, dst) if a >= 0 and z >= 0 and self.lens[a] % self.page) > len(free):
            return None
        for a, z in zip(src, dst):
            pairs.append([-1, -1])
            if a < 0 or z < 0:
                continue
            full, part = divmod(self.lens[a], self.page)
            for j in range(full):
                self.table[z][j] = self.table[a][j]
                self.refs[self.table[a][j]] += 1
            if part:
                pairs[-1] = [self.table[a][full], free.pop(0)]
                self.table[z][full] = pairs[-1][1]
                self.refs[pairs[-1][1]] = 1
            self.lens[z] = self.lens[a]
        return pairs

    def free(self, rows):
        for r in rows:
            if r < 0:
                continue
            for j, e in enumerate(self.table[r]):
                if e >= 0:
                    self.refs[e] -= 1
                    self.table[r][j] = -1
            self.lens[r] = 0

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        a = [p for p in range(live, len(self.refs)) if self.refs[p]]
        z = [p for p in range(live) if not self.refs[p]]
        for x, y in zip(a, z):
            self.refs[y], self.refs[x] = self.refs[x], 0
        name = dict(zip(a, z))
        self.table = [[name.get(e, e) for e in r] for r in self.table]
        return [list(p) for p in zip(a, z)]

    def device(self):
        return ints(self.table), ints(self.lens), ints(self.refs)

    def agrees(self, table, lens, refs):
        assert table.tolist() == self.table
        assert lens.tolist() == self.lens
        assert refs.tolist() == self.refs


@pytest.mark.parametrize("pages,rows,cols,page,seed", [(7, 5, 3, 16, 0), (40, 12, 9, 16, 1), (1000, 60, 40, 32, 2),
                                                       (9001, 300, 37, 64, 3), (70000, 130, 600, 16, 4)])
def test_a_life_of_a_cache(pages, rows, cols, page, seed):
    """Random allocations, forks, frees and compactions, one after the other."""
    rnd = random.Random(seed)
    m = Model(pages, rows, cols, page)
    table, lens, refs = m.device()
    ws = kda.cache_workspace(refs, rows)
    for step in range(12):
        want = [min(cols * page, n + rnd.randrange(0, 3 * page)) if rnd.random() < 0.5 else 0 for n in m.lens]
        ok = m.alloc(want)
        kda.kda_cache_alloc(table, ints(want), refs, page, workspace=ws)
        assert kda.kda_workspace_status(ws) == (kda.KDA_OK if ok else kda.KDA_ERR_NO_SPACE)
        m.agrees(table, lens, refs)
        if ok:
            for r, w in enumerate(want):
                if w > m.lens[r]:
                    m.lens[r] = w - rnd.randrange(0, 2)
            lens.copy_(ints(m.lens))
        drop = rnd.sample(range(rows), rnd.randrange(0, rows // 3 + 1)) + [-1]
        m.free(drop)
        kda.kda_cache_free(table, lens, refs, ints(drop), workspace=ws)
        m.agrees(table, lens, refs)
        # fork rows that hold something into empty ones (a source more than once)
        full = [r for r in range(rows) if m.lens[r]]
        empty = [r for r in range(rows) if m.table[r][0] < 0 and not m.lens[r]]
        dst = rnd.sample(empty, len(empty) // 2)
        src = [rnd.choice(full) if full and rnd.random() < 0.9 else -1 for _ in dst]
        pairs = m.fork(src, dst)
        if dst:
            got = kda.kda_cache_fork(table, lens, refs, ints(src), ints(dst), page, workspace=ws)
            assert kda.kda_workspace_status(ws) == (kda.KDA_OK if pairs is not None else kda.KDA_ERR_NO_SPACE)
            assert got.tolist() == (pairs if pairs is not None else [[-1, -1]] * len(dst))
            m.agrees(table, lens, refs)
        if step % 3 == 2:
            pairs = m.compact()
            got, count = kda.kda_cache_compact(table, refs, workspace=ws)
            assert count.tolist() == [len(pairs)]
            assert got.tolist() == pairs + [[-1, -1]] * (pages - len(pairs))
            m.agrees(table, lens, refs)
    assert kda.kda_workspace_status(ws) == kda.KDA_OK


def test_fork_flags_rows_that_do_not_fit():
    m = Model(20, 6, 4, 16)
    m.alloc([40, 20, 0, 0, 0, 16])
    m.lens = [40, 20, 0, 0, 0, 16]
    table, lens, refs = m.device()
    ws = kda.cache_workspace(refs, 6)
    # a row past the table, a destination in use, itself; the good one is done all the same
    got = kda.kda_cache_fork(table, lens, refs, ints([0, 1, 0, 9]), ints([2, 5, 0, 3]), 16, workspace=ws)
    assert kda.kda_workspace_status(ws) == kda.KDA_ERR_DEVICE
    pairs = m.fork([0], [2])
    assert got.tolist() == pairs + [[-1, -1]] * 3
    m.agrees(table, lens, refs)
    kda.kda_cache_free(table, lens, refs, ints([99, 2]), workspace=ws)
    assert kda.kda_workspace_status(ws) == kda.KDA_ERR_DEVICE
    m.free([2])
    m.agrees(table, lens, refs)


def test_alloc_flags_bad_wishes():
    m = Model(20, 3, 4, 16)
    table, lens, refs = m.device()
    ws = kda.cache_workspace(refs, 3)
    kda.kda_cache_alloc(table, ints([65, -1, 64]), refs, 16, workspace=ws)
    assert kda.kda_workspace_status(ws) == kda.KDA_ERR_DEVICE
    m.alloc([0, 0, 64])
    m.agrees(table, lens, refs)


def test_tables_with_a_row_stride():
    m = Model(30, 4, 5, 16)
    wide = torch.full((4, 11), -7, dtype=torch.int32, device=DEV)
    table = wide[:, 2:7]
    table.copy_(ints(m.table))
    _, lens, refs = m.device()
    want = [80, 3, 0, 33]
    m.alloc(want)
    kda.kda_cache_alloc(table, ints(want), refs, 16)
    m.lens = [77, 3, 0, 32]
    lens.copy_(ints(m.lens))
    pairs = m.fork([0], [2])
    assert kda.kda_cache_fork(table, lens, refs, ints([0]), ints([2]), 16).tolist() == pairs
    m.free([0])
    kda.kda_cache_free(table, lens, refs, ints([0]))
    m.compact()
    kda.kda_cache_compact(table, refs)
    m.agrees(table, lens, refs)
    assert (wide[:, :2] == -7).all() and (wide[:, 7:] == -7).all()


def test_compact_of_a_dense_and_of_an_empty_pool():
    for m in (Model(9, 2, 3, 16), Model(9, 2, 3, 16)):
        if m is not None:
            m.alloc([40, 20])
        table, lens, refs = m.device()
        got, count = kda.kda_cache_compact(table, refs)
        assert count.tolist() == [0] and (got == -1).all()
        m.agrees(table, lens, refs)
    refs = torch.zeros(5, dtype=torch.int32, device=DEV)
    got, count = kda.kda_cache_compact(ints([[-1, -1]]), refs)
    assert count.tolist() == [0] and (got == -1).all()


@pytest.mark.parametrize("shape,dt", [((11, 2, 16, 128), BF), ((7, 3, 5, 8), F32), ((300, 16), torch.uint8),
                                      ((5, 4, 128, 128), F32), ((9, 40000), torch.int64)])
def test_copy(shape, dt):
    g = torch.Generator(device=DEV).manual_seed(1)
    pools = [torch.randint(0, 100, shape, generator=g, device=DEV).to(dt) for _ in range(19)]
    n = shape[0]
    pairs = [[0, 1], [-1, 2], [2, -1], [n, 3], [3, n], [n - 2, n - 1], [4, 4]]
    ref = [p.clone() for p in pools]
    for p in ref:
        p[1] = p[0]
        p[n - 1] = p[n - 2]
    kda.kda_cache_copy(pools, ints(pairs))
    for a, b in zip(pools, ref):
        assert torch.equal(a, b)
    kda.kda_cache_copy(pools, ints([[1, 3], [0, 2]]), count=ints([1]))
    for a, b in zip(pools, ref):
        b[3] = b[1]
        assert torch.equal(a, b)
    kda.kda_cache_copy(pools, ints([[1, 3], [0, 2]]), count=ints([0]))
    for a, b in zip(pools, ref):
        assert torch.equal(a, b)


def append_ref(k, v, kp, vp, table, start, pick, page):
    kp, vp = kp.clone(), vp.clone()
    for b, rows in enumerate(pick):
        for i, r in enumerate(rows):
            pos = start[b] + i
            if pos < 0 or pos // page >= len(table[b]) or not 0 <= table[b][pos // page] < kp.shape[0]:
                continue
            kp[table[b][pos // page], :, pos % page] = k[r]
            vp[table[b][pos // page], :, pos % page] = v[r]
    return kp, vp


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("hkv,page", [(1, 16), (3, 32), (8, 256)])
def test_append_packed(hkv, page, dt):
    rnd = random.Random(hkv)
    take = [1, 0, 37, 300, 0, 5]
    start = [rnd.randrange(0, 2 * page) for _ in take]
    cols = 40
    order = rnd.sample(range(260), 6 * cols)
    table = [order[b * cols:(b + 1) * cols] for b in range(6)]
    fused = torch.randn(sum(take), 2 * hkv + 3, 128, device=DEV).to(dt)
    k, v = fused[:, 1:1 + hkv], fused[:, 1 + hkv:1 + 2 * hkv]
    kp, vp = torch.randn(260, hkv, page, 128, device=DEV).to(dt), torch.randn(260, hkv, page, 128, device=DEV).to(dt)
    cu = [sum(take[:b]) for b in range(7)]
    ref = append_ref(k, v, kp, vp, table, start, [range(cu[b], cu[b + 1]) for b in range(6)], page)
    kda.kda_cache_append(k, v, kp, vp, ints(table), ints(start), cu_seqlens=ints(cu))
    assert torch.equal(kp, ref[0]) and torch.equal(vp, ref[1])


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T", [1, 6, 64])
def test_append_accepted_drafts(T, dt):
    rnd = random.Random(T)
    N, hkv, page = 9, 2, 16
    picks = [sorted(rnd.sample(range(T), rnd.randrange(0, T + 1))) for _ in range(N)]
    index = [p + [10**6] * (T - len(p)) for p in picks]  # past the count: anything
    table = [[20 * b + j for j in range(20)] for b in range(N)]
    start = [rnd.randrange(0, 200) for _ in range(N)]
    k, v = torch.randn(N, T, hkv, 128, device=DEV).to(dt), torch.randn(N, T, hkv, 128, device=DEV).to(dt)
    kp, vp = torch.zeros(180, hkv, page, 128, device=DEV, dtype=dt), torch.zeros(180, hkv, page, 128, device=DEV, dtype=dt)
    flat = lambda x: x.reshape(N * T, hkv, 128)  # noqa: E731
    ref = append_ref(flat(k), flat(v), kp, vp, table, start, [[b * T + r for r in p] for b, p in enumerate(picks)], page)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    kda.kda_cache_append(k, v, kp, vp, ints(table), ints(start), index=ints(index), count=ints([len(p) for p in picks]),
                         workspace=ws)
    assert kda.kda_workspace_status(ws) == kda.KDA_OK
    assert torch.equal(kp, ref[0]) and torch.equal(vp, ref[1])
    kda.kda_cache_append(k, v, kp, vp, ints(table), ints(start))  # all, in order
    ref = append_ref(flat(k), flat(v), kp, vp, table, start, [range(b * T, b * T + T) for b in range(N)], page)
    assert torch.equal(kp, ref[0]) and torch.equal(vp, ref[1])


def test_append_skips_and_flags_rows_without_a_page():
    hkv, page = 1, 16
    k, v = torch.randn(3, 2, hkv, 128, device=DEV), torch.randn(3, 2, hkv, 128, device=DEV)
    kp, vp = torch.zeros(4, hkv, page, 128, device=DEV), torch.zeros(4, hkv, page, 128, device=DEV)
    table, start = [[0, 1], [2, 4], [3, -1]], [31, 15, -1]  # past the table, past the pool, before the start
    ref = append_ref(k.view(6, 1, 128), v.view(6, 1, 128), kp, vp, table, start, [[0, 1], [2, 3], [4, 5]], page)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    kda.kda_cache_append(k, v, kp, vp, ints(table), ints(start), workspace=ws)
    assert kda.kda_workspace_status(ws) == kda.KDA_ERR_DEVICE
    assert torch.equal(kp, ref[0]) and torch.equal(vp, ref[1])
    for kw in (dict(index=ints([[0, 2], [0, 1], [0, 1]])), dict(count=ints([3, 0, 0]))):
        kda.kda_cache_append(k, v, kp.clone(), vp.clone(), ints(table), ints([0, 0, 0]), workspace=ws, **kw)
        assert kda.kda_workspace_status(ws) == kda.KDA_ERR_DEVICE


def test_captured_calls():
    m = Model(50, 8, 6, 16)
    m.alloc([90, 20, 33])
    m.lens = [90, 20, 33, 0, 0, 0, 0, 0]
    table, lens, refs = m.device()
    ws, copies = kda.cache_workspace(refs, 8), torch.empty(2, 2, dtype=torch.int32, device=DEV)
    pool = torch.randn(50, 2, 16, 128, device=DEV)
    src, dst = ints([0, 2]), ints([4, 5])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.kda_cache_free(table, lens, refs, dst, workspace=ws)
        kda.kda_cache_fork(table, lens, refs, src, dst, 16, copies=copies, workspace=ws)
        kda.kda_cache_copy([pool], copies)
    pairs = m.fork([0, 2], [4, 5])
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        m.agrees(table, lens, refs)
        assert copies.tolist() == pairs
        assert all(torch.equal(pool[a], pool[z]) for a, z in pairs)


def test_binding_refuses():
    m = Model(20, 3, 4, 16)
    table, lens, refs = m.device()
    one = ints([0])
    for bad in (lambda: kda.kda_cache_free(table.long(), lens, refs, one), lambda: kda.kda_cache_free(table, lens[:2], refs, one),
                lambda: kda.kda_cache_fork(table, lens, refs, one, ints([1, 2]), 16),
                lambda: kda.kda_cache_alloc(table, lens[:2], refs, 16), lambda: kda.kda_cache_free(table, lens, refs.long(), one),
                lambda: kda.kda_cache_copy([torch.zeros(4, 8, device=DEV), torch.zeros(4, 9, device=DEV)], ints([[0, 1]])),
                lambda: kda.kda_cache_copy([torch.zeros(4, 8, device=DEV)], ints([0, 1])),
                lambda: kda.kda_cache_free(table.t(), lens, refs, one)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: kda.kda_cache_copy([torch.zeros(4, 3, device=DEV)], ints([[0, 1]])),  # 12-byte entries
                lambda: kda.kda_cache_fork(table, lens, refs, ints([0] * 4), ints([1] * 4), 16),  # more forks than rows
                lambda: kda.kda_cache_alloc(table, lens, refs, 0),
                lambda: kda.kda_cache_free(table, lens, refs, one, workspace=torch.zeros(256, dtype=torch.uint8, device=DEV))):
        with pytest.raises(kda.KDAError):
            bad()
