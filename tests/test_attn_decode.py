"""kda_attn_decode against plain 64-bit attention: one token and trees of drafts
over a paged cache, page ends inside tiles, short and empty caches, masks that
leave a row empty, what lies in unused places, malformed tables and lengths."""
import math

import pytest
import torch

import kimi_delta_attention_rule_gb300 as kda
from tests import attn_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SCALE = 128**-0.5
BF, F32 = torch.bfloat16, torch.float32


def normal(seed, shape, dt, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dt)


def make(lens, T, hq, hkv, page, dt, seed=0, spare=2, fill=math.nan):
    """A cache of these lengths on shuffled pages; everything unused is `fill`."""
    g = torch.Generator().manual_seed(seed)
    used = [(n + page - 1) // page for n in lens]
    P = sum(used) + spare
    order = torch.randperm(P, generator=g).tolist()
    cols = max(used + [1])
    table = torch.full((len(lens), cols), -1, dtype=torch.int32)
    kp, vp = torch.full((P, hkv, page, 128), fill, device=DEV, dtype=dt), torch.full((P, hkv, page, 128), fill, device=DEV, dtype=dt)
    ks, vs = [], []
    for b, n in enumerate(lens):
        k, v = normal(seed + 10 * b + 1, (n, hkv, 128), dt), normal(seed + 10 * b + 2, (n, hkv, 128), dt)
        ks.append(k)
        vs.append(v)
        for j in range(used[b]):
            p = order.pop()
            table[b, j] = p
            m = min(page, n - j * page)
            kp[p, :, :m] = k[j * page:j * page + m].transpose(0, 1)
            vp[p, :, :m] = v[j * page:j * page + m].transpose(0, 1)
    B = len(lens)
    return dict(q=normal(seed + 3, (B, T, hq, 128), dt, 2.0), kn=normal(seed + 4, (B, T, hkv, 128), dt),
                vn=normal(seed + 5, (B, T, hkv, 128), dt), kp=kp, vp=vp, table=table.to(DEV),
                lens=torch.tensor(lens, dtype=torch.int32, device=DEV), ks=ks, vs=vs)


def call(x, mask=None, new=True, **kw):
    ws = kda.attn_decode_workspace(x["q"], x["kp"], x["table"])
    out, lse = kda.kda_attn_decode(x["q"], x["kp"], x["vp"], x["table"], x["lens"], SCALE, k_new=x["kn"] if new else None,
                                   v_new=x["vn"] if new else None, tree_mask=mask, output_lse=True, workspace=ws, **kw)
    torch.cuda.synchronize()
    return out, lse, kda.kda_workspace_status(ws)


def check(x, out, lse, mask=None, new=True, rows=None):
    B, T, hq, _ = x["q"].shape
    hkv = x["kn"].shape[2]
    G = hq // hkv
    for b in range(B) if rows is None else rows:
        n = x["ks"][b].shape[0]
        if mask is None:
            tree = torch.ones(T, T, dtype=torch.bool).tril()
        else:
            bits = [int(m) & (2**64 - 1) for m in mask[b].tolist()]
            tree = torch.tensor([[bool(m >> s & 1) for s in range(T)] for m in bits])
        seen = torch.ones(T, n, dtype=torch.bool)
        k, v = x["ks"][b], x["vs"][b]
        if new:
            seen = torch.cat([seen, tree], 1)
            k, v = torch.cat([k, x["kn"][b]]), torch.cat([v, x["vn"][b]])
        for h in range(hq):
            ref = attn_ref.attend(x["q"][b, :, h], k[:, h // G], v[:, h // G], seen.to(DEV), SCALE)
            attn_ref.check(out[b, :, h], lse[b, :, h], ref)


def tree_masks(B, T, seed, own=True):
    g = torch.Generator().manual_seed(seed)
    m = [[0] * T for _ in range(B)]
    for b in range(B):
        for t in range(T):
            parent = int(torch.randint(-1, t, (1,), generator=g)) if t else -1
            m[b][t] = (m[b][parent] if parent >= 0 else 0) | (1 << t if own else 0)
    return torch.tensor([[v - 2**64 if v >= 2**63 else v for v in r] for r in m], dtype=torch.int64, device=DEV)


EDGE = [1, 15, 16, 17, 127, 128, 129, 300]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_one_token(page, dt):
    x = make(EDGE, 1, 8, 2, page, dt, seed=1)
    out, lse, st = call(x)
    assert st == kda.KDA_OK
    check(x, out, lse)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (3, 1), (5, 1), (16, 2), (64, 1), (7, 7)])
@pytest.mark.parametrize("T", [1, 5])
def test_head_groups(hq, hkv, T, dt):
    x = make([70, 200], T, hq, hkv, 32, dt, seed=2)
    out, lse, _ = call(x)
    check(x, out, lse)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,hq,hkv", [(2, 4, 2), (11, 8, 4), (16, 8, 1), (33, 6, 2), (63, 4, 2), (64, 8, 1), (64, 2, 1), (64, 1, 1)])
def test_trees(T, hq, hkv, dt):
    x = make([0, 1, 31, 64, 290], T, hq, hkv, 16, dt, seed=3)
    mask = tree_masks(5, T, T)
    out, lse, st = call(x, mask)
    assert st == kda.KDA_OK
    check(x, out, lse, mask)


@pytest.mark.parametrize("dt", [BF, F32])
def test_chain_is_the_default(dt):
    x = make([40, 130], 6, 4, 2, 16, dt, seed=4)
    chain = torch.tensor([[(2 << t) - 1 for t in range(6)]] * 2, dtype=torch.int64, device=DEV)
    out, lse, _ = call(x)
    check(x, out, lse)
    out2, lse2, _ = call(x, chain)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T", [1, 4, 64])
def test_masks_that_leave_rows_empty(T, dt):
    """No cached token and no draft seen: zeros and -inf; bits past T do not count."""
    x = make([0, 20, 0], T, 4, 1, 16, dt, seed=5)
    mask = torch.zeros(3, T, dtype=torch.int64, device=DEV)
    if T < 64:
        mask[2] = -1 << T  # bits from T on
    if T > 1:
        mask[0, 1] = 1
    out, lse, st = call(x, mask)
    assert st == kda.KDA_OK
    check(x, out, lse, mask)
    assert (out[0, 0] == 0).all() and (lse[0, 0] == -math.inf).all()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T", [1, 3, 40])
def test_cache_alone(T, dt):
    x = make([0, 5, 257], T, 8, 2, 64, dt, seed=6)
    out, lse, _ = call(x, new=False)
    check(x, out, lse, new=False)


@pytest.mark.parametrize("dt,T,hq,hkv", [(BF, 1, 8, 2), (BF, 20, 8, 1), (BF, 64, 8, 2), (F32, 3, 4, 2)])
def test_long_caches(dt, T, hq, hkv):
    """One sequence over all CTAs, next to short ones."""
    x = make([9001, 3, 700, 2500], T, hq, hkv, 64, dt, seed=7)
    mask = tree_masks(4, T, 5) if T > 1 else None
    out, lse, _ = call(x, mask)
    check(x, out, lse, mask)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T", [1, 7])
def test_large_batch_of_ragged_lengths(T, dt):
    lens = [(37 * i) % 411 for i in range(70)]
    x = make(lens, T, 4, 2, 16, dt, seed=8)
    out, lse, _ = call(x)
    check(x, out, lse)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("fill", [math.nan, math.inf, -math.inf])
def test_unused_places_are_not_used(dt, fill):
    """Page tails, spare pages and the next sequence's drafts hold NaN or infinity."""
    x = make([5, 16, 140], 3, 4, 2, 16, dt, seed=9, fill=fill)
    x["kn"][1:] = fill
    x["vn"][1:] = fill
    x["q"][1:] = fill
    out, lse, _ = call(x)
    check(x, out, lse, rows=[0])


@pytest.mark.parametrize("dt", [BF, F32])
def test_nan_draft_that_a_row_does_not_see(dt):
    x = make([30], 4, 2, 1, 16, dt, seed=10)
    x["kn"][0, 3] = math.nan
    out, _, _ = call(x)
    assert torch.isfinite(out[0, :3]).all() and torch.isnan(out[0, 3]).all()


@pytest.mark.parametrize("dt", [BF, F32])
def test_views_and_wide_tables(dt):
    """q, k_new, v_new as views of one projection; a block table with spare columns
    (holding anything) and a row stride of its own."""
    x = make([50, 190], 3, 8, 2, 32, dt, seed=11)
    fused = torch.cat([x["q"], x["kn"], x["vn"]], 2)
    wide = torch.full((2, 40), 10**9, dtype=torch.int32, device=DEV)
    wide[:, 3:3 + x["table"].shape[1]] = x["table"]
    ref, ref_lse, _ = call(x)
    y = dict(x, q=fused[:, :, :8], kn=fused[:, :, 8:10], vn=fused[:, :, 10:], table=wide[:, 3:30])
    out, lse, st = call(y)
    assert st == kda.KDA_OK
    check(x, out, lse)
    one = dict(x, q=x["q"][:, 1:2], kn=x["kn"][:, 1:2], vn=x["vn"][:, 1:2])  # one token of each, strided
    out, lse, _ = call(one)
    check(one, out, lse)


@pytest.mark.parametrize("dt", [BF, F32])
def test_shared_pages(dt):
    """Two sequences on the same pages (a shared prefix)."""
    x = make([100, 100], 2, 4, 2, 16, dt, seed=12)
    x["table"][1] = x["table"][0]
    x["ks"][1], x["vs"][1] = x["ks"][0], x["vs"][0]
    out, lse, _ = call(x)
    check(x, out, lse)


@pytest.mark.parametrize("dt", [BF, F32])
def test_bad_pages_and_lengths_are_reported(dt):
    x = make([100, 40, 60, 30], 2, 4, 2, 16, dt, seed=13, fill=0.0)
    x["table"][0, 2] = -1
    x["table"][1, 1] = x["kp"].shape[0]
    x["lens"][2] = 16 * x["table"].shape[1] + 1
    ws = kda.attn_decode_workspace(x["q"], x["kp"], x["table"])
    out = torch.full_like(x["q"], 7.0)
    kda.kda_attn_decode(x["q"], x["kp"], x["vp"], x["table"], x["lens"], SCALE, k_new=x["kn"], v_new=x["vn"], out=out,
                        workspace=ws)
    assert kda.kda_workspace_status(ws) == kda.KDA_ERR_DEVICE
    assert (out[2] == 7.0).all()  # a bad length: nothing written
    x["lens"][2] = -5
    out, lse, st = call(x)
    assert st == kda.KDA_ERR_DEVICE
    check(x, out, lse, rows=[3])  # a sequence of its own is not touched by the others' faults
    assert torch.isfinite(out[:2]).all()


def test_repeatable_and_captured():
    x = make([5000, 17, 900], 4, 8, 2, 64, BF, seed=14)
    ref, ref_lse, _ = call(x)
    ws, out = kda.attn_decode_workspace(x["q"], x["kp"], x["table"]), torch.empty_like(x["q"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.kda_attn_decode(x["q"], x["kp"], x["vp"], x["table"], x["lens"], SCALE, k_new=x["kn"], v_new=x["vn"], out=out,
                            workspace=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    x["lens"][0] = 333  # a captured call reads the lengths when it runs
    x["ks"][0], x["vs"][0] = x["ks"][0][:333], x["vs"][0][:333]
    g.replay()
    torch.cuda.synchronize()
    check(x, out, call(x)[1])


def test_empty_calls():
    x = make([4], 2, 4, 2, 16, BF, seed=15)
    out, _ = kda.kda_attn_decode(x["q"][:0], x["kp"], x["vp"], x["table"][:0], x["lens"][:0], SCALE)
    assert out.shape == (0, 2, 4, 128)
    none = torch.empty(0, 2, 16, 128, dtype=BF, device=DEV)  # a pool without pages
    x["lens"][0] = 0
    x["ks"][0], x["vs"][0] = x["ks"][0][:0], x["vs"][0][:0]
    out, lse = kda.kda_attn_decode(x["q"], none, none, x["table"], x["lens"], SCALE, k_new=x["kn"], v_new=x["vn"],
                                   output_lse=True)
    check(x, out, lse)


def test_binding_refuses():
    x = make([40], 2, 4, 2, 16, BF, seed=16)
    args = lambda **kw: dict(dict(q=x["q"], k_pages=x["kp"], v_pages=x["vp"], block_table=x["table"], seq_lens=x["lens"],  # noqa: E731
                                  scale=SCALE, k_new=x["kn"], v_new=x["vn"]), **kw)
    for kw in (dict(v_pages=x["vp"].float()), dict(k_new=x["kn"][:, :1]), dict(block_table=x["table"].long()),
               dict(seq_lens=x["lens"].long()), dict(tree_mask=torch.zeros(1, 2, dtype=torch.int32, device=DEV)),
               dict(tree_mask=torch.zeros(1, 3, dtype=torch.int64, device=DEV)), dict(seq_lens=x["lens"].cpu()),
               dict(q=x["q"].transpose(1, 2))):
        with pytest.raises(ValueError):
            kda.kda_attn_decode(**args(**kw))
    for kw in (dict(scale=0.0), dict(k_new=None), dict(workspace=torch.zeros(256, dtype=torch.uint8, device=DEV)),
               dict(scale=math.nan)):
        with pytest.raises(kda.KDAError):
            kda.kda_attn_decode(**args(**kw))
