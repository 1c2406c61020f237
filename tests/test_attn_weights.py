"""kda_attn_weights against plain 64-bit sums: lengths at tile and page edges, accepted drafts,
rows that see nothing, what lies in unused places, malformed inputs, and its refusals.

Bound (u = 2^-24), per cached token, with p = sum of its exact terms: a term exp(s - lse) is off,
relative to itself, by the logit's error e0 = 136 * 2 u scale sum_d |q_d k_d| (attn_ref), by
the rounding of s - lse and of its product with log2 e (4 u (|s| + |lse|)) and by 2^-21 from the
exponential; n terms add up with n u; exp(e) - 1 <= 1.1 e for e < 0.1. The sum is added to w: u |w|."""
import ctypes
import math

import pytest
import torch

import kimi_delta_attention_rule_gb300 as kda
from kimi_delta_attention_rule_gb300 import build as kbuild
from tests.test_attn_decode import BF, DEV, F32, SCALE, make, normal

OK, INVALID, UNSUPPORTED = kda.KDA_OK, kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED
FAKE, ODD = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100008)


def test_refusals():
    kbuild.build()
    lib = kda.load()

    def f(**kw):
        a = dict(q=FAKE, ldq=1024, kp=FAKE, P=9, page=16, table=FAKE, ld=4, cols=4, lens=FAKE, lse=FAKE, index=None, count=None,
                 scale=0.1, B=2, T=3, Hq=8, Hkv=2, D=128, io=0, w=FAKE, cap=64, ws=None)
        a.update(kw)
        return lib.kda_attn_weights(*a.values(), None)
    for kw in (dict(D=64), dict(io=2), dict(T=65), dict(page=8), dict(page=48), dict(Hq=130, ldq=130 * 128)):
        assert f(**kw) == UNSUPPORTED, kw
    for kw in (dict(Hq=9), dict(B=-1), dict(T=-1), dict(P=-1), dict(ld=3), dict(cap=-1), dict(scale=0.0), dict(scale=1e-31), dict(scale=math.nan),
               dict(q=None), dict(kp=None), dict(table=None), dict(lens=None), dict(lse=None), dict(w=None), dict(q=ODD), dict(kp=ODD),
               dict(ws=ODD), dict(ldq=1000), dict(ldq=1028), dict(P=1 << 27), dict(cols=1 << 24, ld=1 << 24, page=256),
               dict(w=ctypes.c_void_p(0x100002)), dict(B=1 << 20, T=64, Hq=8, Hkv=2, ldq=1 << 40)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(B=0), dict(T=0), dict(cap=0), dict(cols=0), dict(P=0)):
        assert f(**{**kw, "q": None, "w": None}) == OK, kw


def rows_of(x, b, index, count):
    T = x["q"].shape[1]
    n = T if count is None else int(count[b])
    return list(range(T))[:n] if index is None else index[b, :n].tolist()


def reference(x, index=None, count=None):
    """lse fp32 [B, T, Hq] of the rows (what attention gives, rounded), and per (b, kv head) the
    exact sums from that lse and their bound."""
    B, T, hq, _ = x["q"].shape
    hkv = x["kp"].shape[1]
    G = hq // hkv
    lse = torch.full((B, T, hq), math.nan, device=DEV)
    sums, bounds = [], []
    for b in range(B):
        k = x["ks"][b].double()
        n, toks = k.shape[0], rows_of(x, b, index, count)
        c = len(toks)
        s_b, t_b = torch.zeros(hkv, n, dtype=torch.float64, device=DEV), torch.zeros(hkv, n, dtype=torch.float64, device=DEV)
        seen = torch.arange(n, device=DEV)[None] <= n - c + torch.arange(c, device=DEV)[:, None]
        for h in range(hq if c else 0):
            q = x["q"][b, toks, h].double()
            s = torch.where(seen, SCALE * (q @ k[:, h // G].T), -math.inf)
            l = torch.logsumexp(s, 1).float()
            lse[b, toks, h] = l
            p = torch.where(seen & (l > -math.inf)[:, None], torch.exp(s - l.double()[:, None]), 0.0)
            e0 = 136 * 2 * 2.0**-24 * SCALE * (q.abs() @ k[:, h // G].abs().T)
            e = e0 + 4 * 2.0**-24 * (torch.where(seen, s, 0.0).abs() + torch.where(l > -math.inf, l, 0.0).abs()[:, None]) + 2.0**-21
            e = e + c * G * 2.0**-24
            assert (e < 0.1).all()
            s_b[h // G] += p.sum(0)
            t_b[h // G] += (1.1 * e * p).sum(0)
        sums.append(s_b)
        bounds.append(t_b)
    return lse, sums, bounds


def run(x, index=None, count=None, ref=None, cap=None, before=None, **kw):
    lse, sums, bounds = ref or reference(x, index, count)
    B, hkv = x["q"].shape[0], x["kp"].shape[1]
    cap = cap or x["table"].shape[1] * x["kp"].shape[2]
    w = normal(77, (B, hkv, cap), F32).abs() if before is None else before.clone()
    start = w.clone()
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    got = kda.kda_attn_weights(x["q"], x["kp"], x["table"], x["lens"], lse, SCALE, w, index=index, count=count, workspace=ws, **kw)
    assert got is w
    return w, start, sums, bounds, kda.kda_workspace_status(ws)


def check(x, w, start, sums, bounds, rows=None):
    for b in range(w.shape[0]) if rows is None else rows:
        n = x["ks"][b].shape[0]
        exact = start[b, :, :n].double() + sums[b]
        d = (w[b, :, :n].double() - exact).abs() - (bounds[b] + 2.0**-24 * exact.abs())
        assert n == 0 or (d <= 0).all(), (b, float(d.max()))
        assert torch.equal(w[b, :, n:], start[b, :, n:])  # behind the end: as it was


LENS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 700]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_one_token(page, dt):
    x = make(LENS, 1, 8, 2, page, dt, seed=40)
    *r, st = run(x)
    assert st == OK
    check(x, *r)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,hq,hkv", [(1, 1, 1), (2, 3, 1), (5, 5, 1), (4, 16, 2), (3, 64, 1), (17, 8, 4), (33, 6, 2), (64, 4, 2), (64, 8, 1),
                                      (64, 64, 1), (40, 13, 1)])
def test_tokens_and_heads(T, hq, hkv, dt):
    """The last T tokens; with fewer cached ones than that, the first of them see nothing."""
    x = make([0, 1, T, 128, 290], T, hq, hkv, 16, dt, seed=41)
    *r, st = run(x)
    assert st == OK
    check(x, *r)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T", [4, 64])
def test_accepted_drafts(T, dt):
    x = make([200, 131, 64, 500, 77], T, 8, 2, 32, dt, seed=42)
    g = torch.Generator().manual_seed(T)
    count = torch.tensor([T, 0, 1, T - 1, T // 2], dtype=torch.int32, device=DEV)
    index = torch.stack([torch.randperm(T, generator=g) for _ in range(5)]).int().to(DEV)  # any order: as it is given
    ref = reference(x, index, count)
    assert torch.isnan(ref[0]).any()  # rows that are not accepted are not read
    *r, st = run(x, index, count, ref)
    assert st == OK
    check(x, *r)
    *r, st = run(x, None, count)
    check(x, *r)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
def test_rows_without_a_logarithm(dt):
    x = make([100, 300], 6, 4, 2, 16, dt, seed=43)
    lse, _, _ = reference(x)
    lse[0, 2] = -math.inf
    lse[1, :, 1] = -math.inf
    x0 = dict(x, q=x["q"].clone())
    w, start, _, _, st = run(x, ref=(lse, None, None))
    assert st == OK and torch.isfinite(w).all()
    # the same as from the rows that are left
    q, l = x0["q"], lse.clone()
    q[0, 2] = 0
    l[0, 2] = math.inf  # exp(0 - inf) = 0
    q[1, :, 1] = 0
    l[1, :, 1] = math.inf
    w2, *_ = run(x0, ref=(l, None, None), before=start)
    assert torch.equal(w, w2)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
def test_infinities_and_nan_stay_with_their_token(dt):
    x = make([300], 3, 8, 2, 16, dt, seed=44)
    clean, start, _, _, _ = run(x)
    ref = reference(x)
    for at, value in ((5, math.nan), (130, math.inf), (299, -math.inf)):
        x["kp"][int(x["table"][0, at // 16]), :, at % 16] = value
    w, *_ = run(x, ref=ref, before=start)
    keep = torch.ones(w.shape[2], dtype=torch.bool, device=DEV)
    keep[[5, 130, 299]] = False
    assert torch.equal(w[..., keep], clean[..., keep])
    assert torch.isnan(w[0, :, 5]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
def test_malformed_rows_are_skipped_and_flagged(dt):
    x = make([100, 200, 300, 150], 4, 4, 2, 16, dt, seed=45)
    count = torch.full((4,), 4, dtype=torch.int32, device=DEV)
    index = torch.arange(4, dtype=torch.int32, device=DEV).repeat(4, 1)
    ref = reference(x, index, count)
    for n in (-1, 16 * x["table"].shape[1] + 1, 2**31 - 1):
        y = dict(x, lens=x["lens"].clone())
        y["lens"][1] = n
        w, start, sums, bounds, st = run(y, index, count, ref)
        assert st == kda.KDA_ERR_DEVICE and torch.equal(w[1], start[1])
        check(x, w, start, sums, bounds, rows=[0, 2, 3])
    for n in (-1, 5):
        c = count.clone()
        c[2] = n
        w, start, sums, bounds, st = run(x, index, c, ref)
        assert st == kda.KDA_ERR_DEVICE and torch.equal(w[2], start[2])
        check(x, w, start, sums, bounds, rows=[0, 1, 3])
    w, start, sums, bounds, st = run(x, index, count, ref, cap=299)  # the third sequence has no room
    assert st == kda.KDA_ERR_DEVICE and torch.equal(w[2], start[2])
    check(x, w, start, sums, bounds, rows=[0, 1, 3])
    bad = index.clone()
    bad[0, 1], bad[3, 3] = -1, 4
    w, start, sums, bounds, st = run(x, bad, count, ref)
    assert st == kda.KDA_ERR_DEVICE
    check(x, w, start, sums, bounds, rows=[1, 2])
    for page in (-1, x["kp"].shape[0], 2**31 - 1):
        y = dict(x, table=x["table"].clone())
        y["table"][2, 3] = page
        w, start, sums, bounds, st = run(y, index, count, ref)
        assert st == kda.KDA_ERR_DEVICE
        check(x, w, start, sums, bounds, rows=[0, 1, 3])


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
def test_strided_rows_and_new_weights(dt):
    x = make([70, 333], 5, 8, 2, 32, dt, seed=46)
    wide = normal(1, (2, 5, 12, 128), dt)
    wide[:, :, :8] = x["q"]
    ref = reference(x)
    w = kda.kda_attn_weights(wide[:, :, :8], x["kp"], x["table"], x["lens"], ref[0], SCALE)
    assert w.shape == (2, 2, x["table"].shape[1] * 32)
    check(x, w, torch.zeros_like(w), ref[1], ref[2])


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
def test_many_sequences(dt):
    g = torch.Generator().manual_seed(4)
    lens = (torch.randint(1, 900, (70,), generator=g) * (torch.rand(70, generator=g) > 0.2)).tolist()
    x = make(lens, 2, 4, 2, 16, dt, seed=47)
    *r, st = run(x)
    assert st == OK
    check(x, *r)


@pytest.mark.gpu
def test_one_long_sequence():
    x = make([20011], 3, 8, 1, 64, BF, seed=48)
    *r, st = run(x)
    assert st == OK
    check(x, *r)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,hq,hkv", [(64, 32, 4), (40, 32, 4), (64, 24, 4), (43, 32, 4), (32, 32, 4), (60, 4, 4)])
def test_many_rows_of_long_sequences(T, hq, hkv, dt):
    """A CTA goes from one sequence's rows to the next one's."""
    x = make([5000, 129, 1, 4001, 63, 6100, 2500, 3333], T, hq, hkv, 32, dt, seed=51)
    *r, st = run(x)
    assert st == OK
    check(x, *r)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
def test_same_bits_captured_and_on_another_stream(dt):
    x = make([1000, 40, 333], 12, 8, 2, 16, dt, seed=49)
    ref = reference(x)
    w, start, *_ = run(x, ref=ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    w2, *_ = run(x, ref=ref, before=start, stream=side)
    side.synchronize()
    assert torch.equal(w, w2)
    buf = start.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_attn_weights(x["q"], x["kp"], x["table"], x["lens"], ref[0], SCALE, buf)
    buf.copy_(start)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(buf, w)
    graph.replay()  # adds again
    torch.cuda.synchronize()
    w3, *_ = run(x, ref=ref, before=w)
    assert torch.equal(buf, w3)


@pytest.mark.gpu
def test_python_refusals():
    x = make([40], 2, 4, 2, 16, BF, seed=50)
    lse = torch.zeros(1, 2, 4, device=DEV)
    w = torch.zeros(1, 2, 48, device=DEV)
    call = lambda **kw: kda.kda_attn_weights(**{**dict(q=x["q"], k_pages=x["kp"], block_table=x["table"], seq_lens=x["lens"], lse=lse,  # noqa: E731
                                                       scale=SCALE, weights=w), **kw})
    call()
    for kw in (dict(lse=lse[:, :1]), dict(lse=lse.double()), dict(weights=w[:, :1]), dict(weights=w.half()), dict(weights=w[..., ::2]),
               dict(index=torch.zeros(1, 2, device=DEV)), dict(count=torch.zeros(2, dtype=torch.int32, device=DEV)),
               dict(seq_lens=x["lens"].cpu()), dict(q=x["q"].float())):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(TypeError):
        call(lse=None)
    with pytest.raises(kda.KDAError):
        call(scale=-1.0)
    with pytest.raises(kda.KDAError):
        call(q=x["q"].half(), k_pages=x["kp"].half())
