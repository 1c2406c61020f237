"""kda_attn_prefill_window and kda_attn_decode_window against plain 64-bit attention:
windows and sinks at and around tile and page edges, keys of the two stretches that meet,
rows that see nothing, draft trees, pages that were given back, and their refusals."""
import ctypes
import math

import pytest
import torch

import kimi_delta_attention_rule_gb300 as kda
from kimi_delta_attention_rule_gb300 import build as kbuild
from tests import attn_ref
from tests.test_attn_decode import BF, DEV, F32, SCALE, make, normal, tree_masks

INVALID, UNSUPPORTED, OK = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_OK
FAKE, BIG = ctypes.c_void_p(0x100000), 1 << 40


# ---- refusals, on the host ---------------------------------------------------------
def test_refusals():
    kbuild.build()
    lib = kda.load()

    def prefill(window=8, sinks=2, D=128, scale=0.1, nbytes=BIG, n=2, q=FAKE):
        return lib.kda_attn_prefill_window(q, FAKE, FAKE, 1024, 256, 256, scale, window, sinks, FAKE, FAKE, n, 10, 10, 8, 2, D, 0,
                                           FAKE, None, FAKE, nbytes, None)

    def decode(window=8, sinks=2, T=3, kn=FAKE, page=16, nbytes=BIG, B=2):
        return lib.kda_attn_decode_window(FAKE, 1024, kn, kn, 256, 256, FAKE, FAKE, 9, page, FAKE, 4, 4, FAKE, None, 0.1, window,
                                          sinks, B, T, 8, 2, 128, 0, FAKE, None, FAKE, nbytes, None)
    for f in (prefill, decode):
        for kw in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(window=-2**31), dict(nbytes=16)):
            assert f(**kw) == INVALID, kw
    assert decode(window=2) == INVALID and decode(window=2, kn=None, nbytes=16) == INVALID  # (the latter: its workspace)
    assert prefill(D=64) == UNSUPPORTED and prefill(scale=math.nan) == INVALID and prefill(q=None) == INVALID
    assert decode(T=65, window=65) == UNSUPPORTED and decode(page=24) == UNSUPPORTED
    assert prefill(n=0) == OK and decode(B=0) == OK and decode(T=0) == OK


@pytest.mark.gpu
def test_python_refusals():
    q = torch.zeros(4, 2, 128, device=DEV, dtype=BF)
    for bad in (0, -3):
        with pytest.raises(kda.KDAError):
            kda.kda_attn_prefill_window(q, q, q, SCALE, bad)
    with pytest.raises(ValueError):
        kda.kda_attn_prefill_window(q, q, q, SCALE, 2**31)
    with pytest.raises(kda.KDAError):
        kda.kda_attn_prefill_window(q, q, q, SCALE, 2, sinks=-1)


# ---- prefill -----------------------------------------------------------------------
def offsets(x):
    return torch.tensor([0] + torch.tensor(x).cumsum(0).tolist(), dtype=torch.int32, device=DEV)


def seen_rows(lq, lk, window, sinks):
    p = torch.arange(lk - lq, lk, device=DEV)[:, None]
    j = torch.arange(lk, device=DEV)[None]
    return (j <= p) & ((j > p - window) | (j < sinks))


def run_prefill(lq, lk, hq, hkv, dt, window, sinks, seed=0):
    q, k, v = normal(seed + 1, (sum(lq), hq, 128), dt, 2.0), normal(seed + 2, (sum(lk), hkv, 128), dt), normal(seed + 3, (sum(lk), hkv, 128), dt)
    ws = kda.attn_prefill_workspace(q, k, offsets(lq))
    out, lse = kda.kda_attn_prefill_window(q, k, v, SCALE, window, sinks, cu_seqlens=offsets(lq), cu_seqlens_k=offsets(lk),
                                           output_lse=True, workspace=ws)
    assert kda.kda_workspace_status(ws) == kda.KDA_OK
    a = c = 0
    for m, n in zip(lq, lk):
        seen = seen_rows(m, n, window, sinks)
        for h in range(hq):
            kv = h * hkv // hq
            attn_ref.check(out[a:a + m, h], lse[a:a + m, h],
                           attn_ref.attend(q[a:a + m, h], k[c:c + n, kv], v[c:c + n, kv], seen, SCALE))
        a, c = a + m, c + n
    return q, k, v, out, lse


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (63, 0), (64, 4), (65, 64), (127, 1), (128, 0), (128, 128), (129, 129),
                                          (200, 5), (300, 257), (1000, 7), (2**31 - 1, 2**31 - 1)])
def test_prompts(window, sinks, dt):
    lens = [1, 17, 128, 129, 300, 777]
    run_prefill(lens, lens, 4, 2, dt, window, sinks, seed=5)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (5, 1), (16, 2), (64, 1)])
def test_head_groups(hq, hkv, dt):
    run_prefill([70, 260], [70, 260], hq, hkv, dt, 50, 3, seed=6)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 4), (300, 0), (700, 130)])
def test_prefix_and_rows_without_keys(window, sinks, dt):
    run_prefill([5, 60, 9, 300, 1, 40], [500, 1201, 9, 1300, 0, 10], 4, 1, dt, window, sinks, seed=7)


@pytest.mark.gpu
@pytest.mark.parametrize("window", [500, 1024])
def test_long_prompt_on_many_sms(window):
    run_prefill([5003], [6000], 8, 1, BF, window, 4, seed=8)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("window", [30, 64, 150])
def test_many_short_prompts(window, dt):
    """More items than SMs have room for at a time, of a few tiles each."""
    g = torch.Generator().manual_seed(window)
    lens = torch.randint(0, 90, (60,), generator=g).tolist()
    run_prefill(lens, lens, 12, 4, dt, window, 3, seed=window)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
def test_window_past_the_end_is_the_plain_call(dt):
    lens = [3, 700, 129]
    q, k, v, out, lse = run_prefill(lens, lens, 4, 2, dt, 700, 0, seed=9)
    o, x = kda.kda_attn_prefill(q, k, v, SCALE, cu_seqlens=offsets(lens), output_lse=True)
    assert torch.equal(o, out) and torch.equal(x, lse)


@pytest.mark.gpu
def test_nothing_behind_the_window_is_used():
    """Tiles that no row of an item looks at may hold anything; inside a shared tile a NaN in k is masked."""
    q, k, v = normal(1, (64, 4, 128), BF), normal(2, (1024, 2, 128), BF), normal(3, (1024, 2, 128), BF)
    ref = kda.kda_attn_prefill_window(q, k, v, SCALE, 200, 4)[0]
    k2, v2 = k.clone(), v.clone()
    k2[128:640] = v2[128:640] = math.nan
    k2[4:128] = math.inf
    k2[640:1024 - 64 - 199] = math.nan
    assert torch.equal(kda.kda_attn_prefill_window(q, k2, v2, SCALE, 200, 4)[0], ref)


# ---- decode ------------------------------------------------------------------------
def decode(x, window, sinks, mask=None, new=True, **kw):
    ws = kda.attn_decode_workspace(x["q"], x["kp"], x["table"])
    out, lse = kda.kda_attn_decode_window(x["q"], x["kp"], x["vp"], x["table"], x["lens"], SCALE, window, sinks,
                                          k_new=x["kn"] if new else None, v_new=x["vn"] if new else None, tree_mask=mask,
                                          output_lse=True, workspace=ws, **kw)
    assert kda.kda_workspace_status(ws) == kda.KDA_OK
    return out, lse


def check_decode(x, out, lse, window, sinks, mask=None, new=True):
    B, T, hq, _ = x["q"].shape
    G = hq // x["kn"].shape[2]
    for b in range(B):
        n = x["ks"][b].shape[0]
        if mask is None:
            tree = torch.ones(T, T, dtype=torch.bool).tril()
        else:
            tree = torch.tensor([[bool((int(m) & (2**64 - 1)) >> s & 1) for s in range(T)] for m in mask[b].tolist()])
        taken = tree.sum(1).clamp(min=1) if new else torch.zeros(T, dtype=torch.long)
        j = torch.arange(n)[None]
        seen = (j >= (n - window + taken)[:, None]) | (j < sinks)
        k, v = x["ks"][b], x["vs"][b]
        if new:
            seen = torch.cat([seen, tree], 1)
            k, v = torch.cat([k, x["kn"][b]]), torch.cat([v, x["vn"][b]])
        for h in range(hq):
            attn_ref.check(out[b, :, h], lse[b, :, h],
                           attn_ref.attend(x["q"][b, :, h], k[:, h // G], v[:, h // G], seen.to(DEV), SCALE))


EDGE = [0, 1, 16, 127, 128, 129, 300, 1500]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("page,window,sinks", [(16, 1, 0), (16, 100, 4), (32, 128, 0), (64, 129, 128), (128, 257, 300), (256, 64, 1),
                                               (16, 2**31 - 1, 0), (32, 1, 2**31 - 1)])
@pytest.mark.parametrize("new", [True, False])
def test_one_token(page, window, sinks, new, dt):
    x = make(EDGE, 1, 8, 2, page, dt, seed=21)
    out, lse = decode(x, window, sinks, new=new)
    check_decode(x, out, lse, window, sinks, new=new)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,hq,hkv,window", [(2, 4, 2, 2), (11, 8, 4, 30), (33, 6, 2, 33), (64, 8, 1, 64), (64, 4, 2, 700), (64, 1, 1, 129)])
def test_trees(T, hq, hkv, window, dt):
    x = make([0, 1, 31, 64, 290, 1100], T, hq, hkv, 16, dt, seed=22)
    for mask in (None, tree_masks(6, T, T)):
        out, lse = decode(x, window, 5, mask)
        check_decode(x, out, lse, window, 5, mask)


@pytest.mark.gpu
@pytest.mark.parametrize("B,window", [(1, 64), (38, 64), (39, 400), (60, 64), (60, 900), (80, 64), (80, 300)])
def test_many_trees(B, window):
    """Row tiles that are items of their own, pairs of them on a CTA each, and items that CTAs share."""
    g = torch.Generator().manual_seed(B)
    x = make(torch.randint(0, 1200, (B,), generator=g).tolist(), 64, 8, 1, 32, BF, seed=29)
    mask = tree_masks(B, 64, B)
    out, lse = decode(x, window, 3, mask)
    check_decode(x, out, lse, window, 3, mask)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
def test_masks_without_the_token_itself(dt):
    x = make([7, 200, 500], 6, 4, 2, 32, dt, seed=23)
    mask = tree_masks(3, 6, 1, own=False)  # some rows see no draft, some others' only
    out, lse = decode(x, 70, 2, mask)
    check_decode(x, out, lse, 70, 2, mask)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("T", [1, 5])
def test_pages_behind_the_window_can_be_gone(page, T, dt):
    lens, window, sinks = [3, 400, 1500, 2000], 333, 20
    x = make(lens, T, 8, 2, page, dt, seed=24)
    out, lse = decode(x, window, sinks)
    check_decode(x, out, lse, window, sinks)
    for b, n in enumerate(lens):
        for j in range((n + page - 1) // page):
            if j * page >= sinks and (j + 1) * page <= n + 1 - window:
                p = int(x["table"][b, j])
                x["kp"][p] = x["vp"][p] = math.nan
                x["table"][b, j] = (-1, 2**31 - 1, -2**31)[j % 3]
    again, lse2 = decode(x, window, sinks)
    assert torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
def test_a_missing_page_inside_the_window_is_flagged(dt):
    x = make([500], 1, 4, 2, 16, dt, seed=25)
    x["table"][0, 30] = -1
    ws = kda.attn_decode_workspace(x["q"], x["kp"], x["table"])
    kda.kda_attn_decode_window(x["q"], x["kp"], x["vp"], x["table"], x["lens"], SCALE, 100, 4, workspace=ws)
    assert kda.kda_workspace_status(ws) == kda.KDA_ERR_DEVICE


@pytest.mark.gpu
def test_a_batch_over_many_sms():
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(1, 3000, (80,), generator=g).tolist()
    x = make(lens, 1, 8, 2, 16, BF, seed=26)
    out, lse = decode(x, 700, 4)
    check_decode(x, out, lse, 700, 4)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("B,T,hq,window", [(90, 5, 8, 40), (90, 18, 16, 64), (100, 1, 4, 150), (50, 40, 12, 200)])
def test_many_short_items(B, T, hq, window, dt):
    g = torch.Generator().manual_seed(B + T)
    x = make(torch.randint(0, 400, (B,), generator=g).tolist(), T, hq, 4, 32, dt, seed=31)
    mask = tree_masks(B, T, B)
    out, lse = decode(x, window, 3, mask)
    check_decode(x, out, lse, window, 3, mask)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
def test_decode_window_past_the_end_is_the_plain_call(dt):
    x = make([0, 5, 300, 900], 4, 8, 2, 32, dt, seed=27)
    out, lse = decode(x, 2000, 0)
    o, y = kda.kda_attn_decode(x["q"], x["kp"], x["vp"], x["table"], x["lens"], SCALE, k_new=x["kn"], v_new=x["vn"], output_lse=True)
    assert torch.equal(o, out) and torch.equal(y, lse)


@pytest.mark.gpu
def test_decode_goes_on_where_prefill_ended():
    """The last token of a prompt through either call: the same window."""
    n, window, sinks = 1000, 300, 9
    q, k, v = normal(1, (n, 8, 128), BF), normal(2, (n, 2, 128), BF), normal(3, (n, 2, 128), BF)
    o = kda.kda_attn_prefill_window(q, k, v, SCALE, window, sinks)[0]
    kp, vp = torch.zeros(63, 2, 16, 128, device=DEV, dtype=BF), torch.zeros(63, 2, 16, 128, device=DEV, dtype=BF)
    table = torch.arange(63, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([n - 1], dtype=torch.int32, device=DEV)
    kda.kda_cache_append(k[None, :-1], v[None, :-1], kp, vp, table, torch.zeros_like(lens))
    one = kda.kda_attn_decode_window(q[None, -1:], kp, vp, table, lens, SCALE, window, sinks, k_new=k[None, -1:], v_new=v[None, -1:])[0]
    # both are a bf16 rounding (2^-8) and twice the bound of p's rounding from one value; |o| <= max |v|
    tol = 2.0**-8 * (one[0, 0].float().abs() + o[-1].float().abs()) + 2 * 2.0**-8 * v.float().abs().amax()
    assert ((one[0, 0].float() - o[-1].float()).abs() <= tol).all()


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    x = make([40, 900, 2500], 3, 8, 2, 32, BF, seed=28)
    ref = decode(x, 256, 4)
    ws = kda.attn_decode_workspace(x["q"], x["kp"], x["table"])
    out, lse = torch.empty_like(ref[0]), torch.empty_like(ref[1])

    def step():
        kda.kda_attn_decode_window(x["q"], x["kp"], x["vp"], x["table"], x["lens"], SCALE, 256, 4, k_new=x["kn"], v_new=x["vn"],
                                   out=out, lse=lse, workspace=ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert torch.equal(out, ref[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x["lens"].copy_(torch.tensor([10, 300, 2400], dtype=torch.int32))
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        now = decode(x, 256, 4)
        assert torch.equal(out, now[0]) and torch.equal(lse, now[1])
