"""kda_attn_prefill against plain 64-bit attention: lengths from one token up,
odd sizes, every kind of head group, appended prompts, rows that see nothing,
strided rows, values past a sequence's end."""
import math

import pytest
import torch

import kimi_delta_attention_rule_gb300 as kda
from tests import attn_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SCALE = 128**-0.5


def rows(seed, n, h, dt, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(n, h, 128, generator=g, device=DEV) * scale).to(dt)


def offsets(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=DEV)


def check(q, k, v, lq, lk, out, lse, scale=SCALE):
    G = q.shape[1] // k.shape[1]
    a = c = 0
    for m, n in zip(lq, lk):
        seen = torch.ones(m, n, dtype=torch.bool, device=DEV).tril(n - m)
        for h in range(q.shape[1]):
            ref = attn_ref.attend(q[a:a + m, h], k[c:c + n, h // G], v[c:c + n, h // G], seen, scale)
            attn_ref.check(out[a:a + m, h], lse[a:a + m, h], ref)
        a, c = a + m, c + n


def run(lq, lk, hq, hkv, dt, seed=0, qscale=2.0):
    q, k, v = rows(seed, sum(lq), hq, dt, qscale), rows(seed + 1, sum(lk), hkv, dt), rows(seed + 2, sum(lk), hkv, dt)
    ws = kda.attn_prefill_workspace(q, k, offsets(lq))
    out, lse = kda.kda_attn_prefill(q, k, v, SCALE, cu_seqlens=offsets(lq), cu_seqlens_k=offsets(lk), output_lse=True,
                                    workspace=ws)
    torch.cuda.synchronize()
    assert kda.kda_workspace_status(ws) == kda.KDA_OK
    check(q, k, v, lq, lk, out, lse)


BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("lens", [[1], [64], [128], [129], [1, 1, 2], [127, 128, 129], [0, 33, 0, 70, 0], [300, 5]])
def test_lengths(lens, dt):
    run(lens, lens, 4, 2, dt)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (8, 8), (5, 1), (12, 4), (8, 1), (13, 1), (32, 2), (64, 1)])
def test_head_groups(hq, hkv, dt):
    run([37, 150], [37, 150], hq, hkv, dt, seed=3)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("lq,lk", [([1], [700]), ([5, 3], [300, 129]), ([40], [3000]), ([130, 17], [131, 400])])
def test_appended_tokens(lq, lk, dt):
    run(lq, lk, 8, 2, dt, seed=5)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("lq,lk", [([300], [5]), ([70, 40], [0, 40]), ([130], [1]), ([200, 3], [0, 0]), ([520], [260])])
def test_rows_that_see_nothing(lq, lk, dt):
    run(lq, lk, 4, 2, dt, seed=7)


@pytest.mark.parametrize("dt,lens,hq,hkv", [(BF, [2500], 8, 2), (BF, [1900, 3, 700, 1], 2, 2), (BF, [4100], 2, 1), (F32, [1300, 90], 4, 1)])
def test_long(lens, hq, hkv, dt):
    """Items that several CTAs share, several items per CTA."""
    run(lens, lens, hq, hkv, dt, seed=9)


@pytest.mark.parametrize("dt", [BF, F32])
def test_one_row_over_a_very_long_prefix(dt):
    run([2], [40001], 2, 1, dt, seed=11)


@pytest.mark.parametrize("dt", [BF, F32])
def test_many_sequences(dt):
    lens = [(7 * i) % 23 for i in range(300)]
    run(lens, lens, 4, 2, dt, seed=13)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("N,hkv", [(3000, 2), (70000, 4)])
def test_very_many_single_tokens(N, hkv, dt):
    """A sequence of one token is its own v: lengths that add up to far less than the
    bound that the work search counts in."""
    G = 2
    q, k, v = rows(15, N, G * hkv, dt), rows(16, N, hkv, dt), rows(17, N, hkv, dt)
    cu = torch.arange(N + 1, dtype=torch.int32, device=DEV)
    out, lse = kda.kda_attn_prefill(q, k, v, SCALE, cu_seqlens=cu, output_lse=True)
    assert torch.equal(out, v.repeat_interleave(G, 1))
    kk = k.repeat_interleave(G, 1).double()
    x = SCALE * (q.double() * kk).sum(2)
    tol = 136 * 2.0**-24 * 2 * SCALE * (q.double() * kk).abs().sum(2) + 2.0**-21 + 2.0**-22 * x.abs()
    assert ((lse.double() - x).abs() <= tol).all()


@pytest.mark.parametrize("dt", [BF, F32])
def test_one_long_among_very_many_short(dt):
    """40,000 sequences of nothing or one token around one of 5,000."""
    lens = [i % 2 for i in range(20000)] + [5000] + [(i + 1) % 2 for i in range(20000)]
    n = sum(lens)
    q, k, v = rows(18, n, 2, dt), rows(19, n, 1, dt), rows(20, n, 1, dt)
    cu = offsets(lens)
    out, lse = kda.kda_attn_prefill(q, k, v, SCALE, cu_seqlens=cu, output_lse=True)
    a = int(cu[20000])
    check(q[a:a + 5000], k[a:a + 5000], v[a:a + 5000], [5000], [5000], out[a:a + 5000], lse[a:a + 5000])
    short = torch.ones(n, dtype=torch.bool, device=DEV)
    short[a:a + 5000] = False
    assert torch.equal(out[short], v.repeat_interleave(2, 1)[short])


@pytest.mark.parametrize("dt", [BF, F32])
def test_growing_maxima(dt):
    """Keys that grow along the sequence: the running maximum moves at every tile
    (by far more than 2^8 once), and logits reach several hundred."""
    n = 700
    q, k, v = rows(21, n, 2, dt), rows(22, n, 1, dt), rows(23, n, 1, dt)
    k = (k.float() * torch.linspace(0.05, 40, n, device=DEV)[:, None, None]).to(dt)
    out, lse = kda.kda_attn_prefill(q, k, v, SCALE, output_lse=True)
    check(q, k, v, [n], [n], out, lse)


def test_equal_lengths_without_offsets():
    q, k, v = rows(1, 3 * 90, 4, BF), rows(2, 3 * 90, 2, BF), rows(3, 3 * 90, 2, BF)
    out, lse = kda.kda_attn_prefill(q, k, v, SCALE, N=3, output_lse=True)
    check(q, k, v, [90] * 3, [90] * 3, out, lse)
    cu = offsets([90] * 3)
    assert torch.equal(out, kda.kda_attn_prefill(q, k, v, SCALE, cu_seqlens=cu)[0])
    short = kda.kda_attn_prefill(q[:3], k, v, SCALE, N=3, output_lse=True)  # one token over 90 keys, three times
    check(q[:3], k, v, [1] * 3, [90] * 3, *short)


@pytest.mark.parametrize("dt", [BF, F32])
def test_views_of_one_projection(dt):
    qkv = rows(31, 200, 8 + 2 + 2, dt)
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    out, lse = kda.kda_attn_prefill(q, k, v, SCALE, output_lse=True)
    check(q, k, v, [200], [200], out, lse)
    assert torch.equal(out, kda.kda_attn_prefill(q.contiguous(), k.contiguous(), v.contiguous(), SCALE)[0])


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_other_sequences_do_not_leak(dt, bad):
    """Sequence 1 holds NaN or infinity: 0 and 2 are as without it."""
    lens = [150, 61, 200]
    q, k, v = rows(41, 411, 4, dt), rows(42, 411, 2, dt), rows(43, 411, 2, dt)
    for x in (q, k, v):
        x[150:211] = bad
    out, lse = kda.kda_attn_prefill(q, k, v, SCALE, cu_seqlens=offsets(lens), output_lse=True)
    for a, n in ((0, 150), (211, 200)):
        check(q[a:a + n], k[a:a + n], v[a:a + n], [n], [n], out[a:a + n], lse[a:a + n])


@pytest.mark.parametrize("dt", [BF, F32])
def test_nan_in_a_hidden_key(dt):
    """A NaN key reaches the rows that see it, not those before it."""
    q, k, v = rows(51, 100, 2, dt), rows(52, 100, 1, dt), rows(53, 100, 1, dt)
    k[60] = math.nan
    out, _ = kda.kda_attn_prefill(q, k, v, SCALE)
    assert torch.isfinite(out[:60]).all() and torch.isnan(out[60:]).all()


def test_repeatable_and_on_another_stream():
    q, k, v = rows(61, 3000, 8, BF), rows(62, 3000, 2, BF), rows(63, 3000, 2, BF)
    out, lse = kda.kda_attn_prefill(q, k, v, SCALE, output_lse=True)
    ws = kda.attn_prefill_workspace(q, k)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        again, lse2 = kda.kda_attn_prefill(q, k, v, SCALE, output_lse=True, workspace=ws, stream=st)
    st.synchronize()
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_graph_capture():
    q, k, v = rows(71, 1000, 8, BF), rows(72, 1000, 2, BF), rows(73, 1000, 2, BF)
    ws, out = kda.attn_prefill_workspace(q, k), torch.empty_like(q)
    ref = kda.kda_attn_prefill(q, k, v, SCALE)[0]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.kda_attn_prefill(q, k, v, SCALE, out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("cu", [[0, 50, 40, 100], [3, 50, 60, 100], [0, 50, 60, 101]])
def test_malformed_offsets_are_reported(cu, dt):
    q, k, v = rows(81, 100, 4, dt), rows(82, 100, 2, dt), rows(83, 100, 2, dt)
    bad = torch.tensor(cu, dtype=torch.int32, device=DEV)
    ws, out = kda.attn_prefill_workspace(q, k, bad), torch.full_like(q, 7.0)
    kda.kda_attn_prefill(q, k, v, SCALE, cu_seqlens=bad, out=out, workspace=ws)
    assert kda.kda_workspace_status(ws) == kda.KDA_ERR_DEVICE
    assert kda.kda_workspace_status(ws) == kda.KDA_OK
    assert (out == 7.0).all()
    out2, lse = kda.kda_attn_prefill(q, k, v, SCALE, cu_seqlens=offsets([30, 70]), output_lse=True, workspace=ws)
    check(q, k, v, [30, 70], [30, 70], out2, lse)
    assert kda.kda_workspace_status(ws) == kda.KDA_OK


def test_empty_calls():
    q, k = torch.empty(0, 4, 128, dtype=BF, device=DEV), torch.empty(0, 2, 128, dtype=BF, device=DEV)
    out, lse = kda.kda_attn_prefill(q, k, k, SCALE, output_lse=True)
    assert out.shape == (0, 4, 128) and lse.shape == (0, 4)
    q = rows(1, 5, 4, BF)  # no keys at all
    out, lse = kda.kda_attn_prefill(q, k, k, SCALE, output_lse=True)
    torch.cuda.synchronize()
    assert (out == 0).all() and (lse == -math.inf).all()


def test_binding_refuses():
    q, k = rows(1, 10, 4, BF), rows(2, 10, 2, BF)
    for bad in (lambda: kda.kda_attn_prefill(q, k, k.float(), SCALE), lambda: kda.kda_attn_prefill(q, k, k[:9], SCALE),
                lambda: kda.kda_attn_prefill(q.transpose(0, 1), k, k, SCALE),
                lambda: kda.kda_attn_prefill(q.cpu(), k, k, SCALE),
                lambda: kda.kda_attn_prefill(q, k, k, SCALE, cu_seqlens=torch.zeros(2, dtype=torch.int64, device=DEV)),
                lambda: kda.kda_attn_prefill(q, k, k, SCALE, out=torch.empty_like(k)),
                lambda: kda.kda_attn_prefill(q, k, k, SCALE, N=3)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(kda.KDAError):
        kda.kda_attn_prefill(q, k, k, -1.0)
    with pytest.raises(kda.KDAError):
        kda.kda_attn_prefill(q, k, k, SCALE, workspace=torch.zeros(256, dtype=torch.uint8, device=DEV))
