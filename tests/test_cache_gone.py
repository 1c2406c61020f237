"""Pages that a row has given back while those behind them keep their places (KDA_PAGE_GONE), through every
call on the cache, and the example's window that lets pages go."""
import os
import sys

import pytest
import torch

import kimi_delta_attention_rule_gb300 as kda
from kimi_delta_attention_rule_gb300 import build as kbuild
from tests.test_attn_decode import BF, DEV, F32, SCALE, normal

OK, BAD, GONE = kda.KDA_OK, kda.KDA_ERR_DEVICE, -2
PAGE = 16


def test_the_entry_is_the_headers():
    assert kda.KDA_PAGE_GONE == GONE
    assert "#define KDA_PAGE_GONE (-2)" in open(os.path.join(kbuild.INCLUDE, "kda.h")).read()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Cache:
    def __init__(self, want, cols, pages):
        self.table = torch.full((len(want), cols), -1, dtype=torch.int32, device=DEV)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
        self.lens = ints(want)
        self.ws = kda.cache_workspace(self.refs, len(want))
        self.alloc(want)

    def alloc(self, want):
        kda.kda_cache_alloc(self.table, ints(want), self.refs, PAGE, workspace=self.ws)

    def give_back(self, row, cols):
        for j in cols:
            self.refs[self.table[row, j].long()] -= 1
            self.table[row, j] = GONE

    def status(self):
        return kda.kda_workspace_status(self.ws)

    def consistent(self):
        used = self.table[self.table >= 0].long()
        assert torch.equal(torch.bincount(used, minlength=len(self.refs)).int(), self.refs)


@pytest.mark.gpu
@pytest.mark.parametrize("gone", [[0], [1], [2, 3, 4], [0, 1, 2, 3, 4, 5], list(range(1, 39)), list(range(39)), list(range(0, 39, 2))])
def test_alloc_goes_on_behind_them(gone):
    c = Cache([39 * PAGE + 3, 20], 70, 200)
    before = c.table.clone()
    c.give_back(0, gone)
    want = c.table.clone()
    c.alloc([45 * PAGE, 20])
    free = sorted(set(range(200)) - set(before[0, [j for j in range(40) if j not in gone]].tolist()) - set(before[1, :2].tolist()))
    want[0, 40:45] = ints(free[:5])  # the lowest free pages, the given-back ones among them
    assert c.status() == OK and torch.equal(c.table, want)
    c.consistent()
    c.alloc([3, 20])  # a row never loses pages
    assert c.status() == OK and torch.equal(c.table, want)


@pytest.mark.gpu
@pytest.mark.parametrize("gone", [[0], [0, 1, 2], [3, 4], list(range(30))])
def test_a_reused_page_survives_its_first_row(gone):
    """What a row gave back belongs to whoever has taken it: freeing or trimming the row leaves it alone."""
    for way in ("free", "trim", "trim all"):
        c = Cache([31 * PAGE, 0], 31, 31)  # every page
        c.give_back(0, gone)
        c.alloc([31 * PAGE, len(gone) * PAGE])
        assert c.status() == OK and sorted(c.table[1, :len(gone)].tolist()) == sorted(gone)
        other, keep = c.table[1].clone(), 31
        if way == "free":
            kda.kda_cache_free(c.table, c.lens, c.refs, ints([0]), workspace=c.ws)
            assert int(c.lens[0]) == 0 and (c.table[0] == -1).all()
        else:
            keep = 2 if way == "trim" else 0
            row = c.table[0].clone()
            kda.kda_cache_trim(c.table, c.lens, c.refs, ints([keep * PAGE, -1]), PAGE, workspace=c.ws)
            assert int(c.lens[0]) == keep * PAGE and torch.equal(c.table[0, :keep], row[:keep]) and (c.table[0, keep:] == -1).all()
        assert c.status() == OK and torch.equal(c.table[1], other) and (c.refs[other[:len(gone)].long()] == 1).all()
        c.consistent()


@pytest.mark.gpu
def test_fork_passes_them_on():
    c = Cache([40 * PAGE + 5, 0, 3 * PAGE, 0], 50, 200)
    c.give_back(0, [0, 1, 7, 35])
    c.give_back(2, [0, 1, 2])
    row = c.table[0].clone()
    copies = kda.kda_cache_fork(c.table, c.lens, c.refs, ints([0, 2]), ints([1, 3]), PAGE, workspace=c.ws)
    assert c.status() == OK and torch.equal(c.table[1, :40], row[:40]) and torch.equal(c.table[3], c.table[2])
    assert copies.tolist()[0][0] == int(row[40]) and copies.tolist()[1] == [-1, -1] and c.lens.tolist() == [645, 645, 48, 48]
    c.consistent()
    # a row whose first page is gone is no empty row
    table, refs = c.table.clone(), c.refs.clone()
    kda.kda_cache_fork(c.table, c.lens, c.refs, ints([0]), ints([3]), PAGE, workspace=c.ws)
    assert c.status() == BAD and torch.equal(c.table, table) and torch.equal(c.refs, refs)
    kda.kda_cache_free(c.table, c.lens, c.refs, ints([0, 1, 2, 3]), workspace=c.ws)
    assert c.status() == OK and (c.table == -1).all() and not c.refs.any()


@pytest.mark.gpu
def test_a_fork_that_ends_in_one_is_flagged():
    c = Cache([2 * PAGE + 5, 0], 9, 40)
    c.give_back(0, [2])
    table, refs = c.table.clone(), c.refs.clone()
    kda.kda_cache_fork(c.table, c.lens, c.refs, ints([0]), ints([1]), PAGE, workspace=c.ws)
    assert c.status() == BAD and torch.equal(c.table, table) and torch.equal(c.refs, refs)


@pytest.mark.gpu
def test_compact_leaves_them():
    c = Cache([20 * PAGE, 9 * PAGE, 5 * PAGE], 20, 60)
    c.give_back(0, range(3, 12))
    c.give_back(1, [0])
    table, refs = c.table.clone(), c.refs.clone()
    copies, count = kda.kda_cache_compact(c.table, c.refs, workspace=c.ws)
    live = int((refs > 0).sum())
    name = {a: b for a, b in copies[:int(count)].tolist()}
    assert c.status() == OK and c.table.tolist() == [[name.get(p, p) for p in r] for r in table.tolist()]
    assert (c.refs[:live] == 1).all() and not c.refs[live:].any()
    c.consistent()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
def test_calls_on_their_tokens_are_flagged(dt):
    c = Cache([8 * PAGE, 8 * PAGE], 8, 20)
    kp, vp = normal(1, (20, 1, PAGE, 128), dt), normal(2, (20, 1, PAGE, 128), dt)
    c.give_back(0, [3])
    old = kp.clone(), vp.clone()
    rows = normal(3, (2, 1, 1, 128), dt)
    kda.kda_cache_append(rows, rows, kp, vp, c.table, ints([3 * PAGE + 1, 5]), workspace=c.ws)
    assert c.status() == BAD
    at = int(c.table[1, 0])
    old[0][at, :, 5], old[1][at, :, 5] = rows[1, 0], rows[1, 0]
    assert torch.equal(kp, old[0]) and torch.equal(vp, old[1])
    w = torch.rand(2, 1, 8 * PAGE, device=DEV)
    first, ws = w[0].clone(), kda.evict_workspace(w)
    kda.kda_cache_evict(kp, vp, w, c.table, c.lens, ints([40, 40]), 2, 4, workspace=ws)
    assert kda.kda_workspace_status(ws) == BAD and torch.equal(w[0], first) and not w[1, :, 40:].any()
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    kda.kda_attn_weights(rows, kp, c.table, c.lens, torch.zeros(2, 1, 1, device=DEV), SCALE, w, workspace=ws)
    assert kda.kda_workspace_status(ws) == BAD
    ws = kda.attn_decode_workspace(rows, kp, c.table)
    kda.kda_attn_decode(rows, kp, vp, c.table, c.lens, SCALE, workspace=ws)
    assert kda.kda_workspace_status(ws) == BAD


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
def test_a_windowed_layer_whose_pages_go_round(dt):
    """Two rows in a pool that holds neither's whole context: what one gives back the other takes; each token's output is,
    bit for bit, that of a cache that keeps everything."""
    window, sinks, steps, hkv = 40, 4, 150, 2
    cols = steps // PAGE + 1
    kp, vp = (torch.full((10, hkv, PAGE, 128), float("nan"), device=DEV, dtype=dt) for _ in range(2))
    kall, vall = (torch.zeros(2 * cols, hkv, PAGE, 128, device=DEV, dtype=dt) for _ in range(2))
    c = Cache([0, 0], cols, 10)
    whole = torch.arange(2 * cols, dtype=torch.int32, device=DEV).view(2, cols)
    for t in range(steps):
        q, k, v = normal(3 * t, (2, 1, 4, 128), dt, 2.0), normal(3 * t + 1, (2, 1, hkv, 128), dt), normal(3 * t + 2, (2, 1, hkv, 128), dt)
        ws, ws2 = kda.attn_decode_workspace(q, kp, c.table), kda.attn_decode_workspace(q, kall, whole)
        a, _ = kda.kda_attn_decode_window(q, kp, vp, c.table, c.lens, SCALE, window, sinks, k_new=k, v_new=v, workspace=ws)
        b, _ = kda.kda_attn_decode_window(q, kall, vall, whole, c.lens, SCALE, window, sinks, k_new=k, v_new=v, workspace=ws2)
        assert torch.equal(a, b) and kda.kda_workspace_status(ws) == OK
        c.alloc([t + 1] * 2)
        kda.kda_cache_append(k, v, kp, vp, c.table, c.lens, workspace=c.ws)
        kda.kda_cache_append(k, v, kall, vall, whole, c.lens)
        c.lens += 1
        for row in range(2):
            c.give_back(row, [j for j in range(1, cols) if (j + 1) * PAGE <= t + 2 - window and int(c.table[row, j]) >= 0])
        assert c.status() == OK
    c.consistent()
    assert int((c.table == GONE).sum()) == 2 * ((steps + 1 - window) // PAGE - 1)
    kda.kda_cache_free(c.table, c.lens, c.refs, ints([0, 1]), workspace=c.ws)
    assert c.status() == OK and not c.refs.any() and (c.table == -1).all()


@pytest.mark.gpu
def test_the_example_gives_every_page_back_once():
    sys.path.insert(0, os.path.join(kbuild.ROOT, "examples"))
    import bounded_decode as ex
    for name, (_, pages, cache) in ex.main(seed=3).items():
        used = cache.table[cache.table >= 0].long()
        assert torch.equal(torch.bincount(used, minlength=len(cache.refs)).int(), cache.refs), name
        assert int((cache.refs > 0).sum()) == pages
        cache.free()
        cache.check()
        assert not cache.refs.any() and (cache.table == -1).all()
