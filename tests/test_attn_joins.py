"""Rows that several SMs share, and calls that follow one another without a wait: the
bits of a result do not depend on which part was done first, a workspace is left as
it has to be found, and a call sees what the work before it in the stream wrote."""
import pytest
import torch

import kimi_delta_attention_rule_gb300 as kda
from tests import attn_ref
from tests.test_attn_decode import SCALE, make, tree_masks

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def rows(seed, n, h, dt):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(n, h, 128, generator=g, device=DEV).to(dt)


def offsets(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=DEV)


def prefill(lq, lk, hq, hkv, dt, seed):
    q, k, v = rows(seed, sum(lq), hq, dt), rows(seed + 1, sum(lk), hkv, dt), rows(seed + 2, sum(lk), hkv, dt)
    cq, ck, ws = offsets(lq), offsets(lk), kda.attn_prefill_workspace(q, k, offsets(lq))

    def call(q=q):
        return kda.kda_attn_prefill(q, k, v, SCALE, cu_seqlens=cq, cu_seqlens_k=ck, output_lse=True, workspace=ws)

    return call, ws, (q, k, v)


def decode(lens, T, hq, hkv, page, dt, seed):
    x = make(lens, T, hq, hkv, page, dt, seed=seed)
    mask, ws = tree_masks(len(lens), T, seed), kda.attn_decode_workspace(x["q"], x["kp"], x["table"])

    def call(q=x["q"]):
        return kda.kda_attn_decode(q, x["kp"], x["vp"], x["table"], x["lens"], SCALE, k_new=x["kn"], v_new=x["vn"],
                                   tree_mask=mask, output_lse=True, workspace=ws)

    return call, ws, (x["q"],)


# parts of an item: two, three and more, one row of many, with and without the neighbour's early part
CASES = [
    ("prompt", lambda dt: prefill([3000], [3000], 8, 2, dt, 1)),
    ("ragged", lambda dt: prefill([700, 3, 1300, 90, 1, 512], [700, 3, 1300, 90, 1, 512], 8, 1, dt, 2)),
    ("appended", lambda dt: prefill([300, 40], [9000, 2000], 8, 2, dt, 3)),
    ("few rows, long prefix", lambda dt: prefill([3], [40000], 8, 1, dt, 4)),
    ("large trees", lambda dt: decode([9000, 1500, 4000], 64, 16, 2, 32, dt, 5)),
    ("one token", lambda dt: decode([20000, 300], 1, 8, 2, 64, dt, 6)),
]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("name,build", CASES, ids=[c[0] for c in CASES])
def test_bits_and_workspace(name, build, dt):
    call, ws, _ = build(dt)
    other, _, _ = prefill([900, 20], [900, 20], 4, 2, BF, 9)  # on another stream: takes SMs away
    side = torch.cuda.Stream()
    ref, ref_lse = call()
    torch.cuda.synchronize()
    for i in range(12):
        if i % 2:
            with torch.cuda.stream(side):
                for _ in range(i):
                    other()
        out, lse = call()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
        assert kda.kda_workspace_status(ws) == kda.KDA_OK
        assert not ws[:256].any()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("name,build", CASES, ids=[c[0] for c in CASES])
def test_calls_in_a_row(name, build, dt):
    """The queries change between calls, on the stream alone."""
    call, _, (q, *_) = build(dt)
    qs = [q * (0.25 + 0.25 * i) for i in range(6)]
    refs = []
    for x in qs:
        refs.append(call(q=x))
        torch.cuda.synchronize()
    y, got = torch.empty_like(q), []
    for x in qs:
        y.copy_(x)
        got.append(call(q=y))
    torch.cuda.synchronize()
    for (out, lse), (ref, ref_lse) in zip(got, refs):
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


@pytest.mark.parametrize("io", [BF, F32])
def test_append_then_read(io):
    """A step of a server, over and over: append, attend, fork, copy, free, all on the stream."""
    B, hq, hkv, page, cols = 6, 8, 2, 32, 16
    P = 3 * B * cols
    kp, vp = torch.zeros(P, hkv, page, 128, dtype=io, device=DEV), torch.zeros(P, hkv, page, 128, dtype=io, device=DEV)
    table = torch.full((2 * B, cols), -1, dtype=torch.int32, device=DEV)
    lens, refs = torch.zeros(2 * B, dtype=torch.int32, device=DEV), torch.zeros(P, dtype=torch.int32, device=DEV)
    ws = kda.cache_workspace(refs, 2 * B)
    want = torch.tensor([cols * page] * B + [0] * B, dtype=torch.int32, device=DEV)
    kda.kda_cache_alloc(table, want, refs, page, workspace=ws)
    src = torch.arange(B, dtype=torch.int32, device=DEV)
    dst = src + B
    wa = kda.attn_decode_workspace(torch.empty(B, 1, hq, 128, dtype=io, device=DEV), kp, table[:B])
    k, v = rows(31, B * 40, hkv, io).view(B, 40, hkv, 128), rows(32, B * 40, hkv, io).view(B, 40, hkv, 128)
    q = rows(33, B * 40, hq, io).view(40, B, 1, hq, 128)
    outs, forks = [], []
    for t in range(40):
        kda.kda_cache_append(k[:, t:t + 1], v[:, t:t + 1], kp, vp, table[:B], lens[:B], workspace=ws)
        lens[:B] += 1
        outs.append(kda.kda_attn_decode(q[t], kp, vp, table[:B], lens[:B], SCALE, output_lse=True, workspace=wa))
        copies = kda.kda_cache_fork(table, lens, refs, src, dst, page, workspace=ws)
        kda.kda_cache_copy([kp, vp], copies)
        forks.append(kda.kda_attn_decode(q[t], kp, vp, table[B:], lens[B:], SCALE, output_lse=True, workspace=wa))
        kda.kda_cache_free(table, lens, refs, dst, workspace=ws)
    torch.cuda.synchronize()
    assert kda.kda_workspace_status(ws) == kda.KDA_OK and kda.kda_workspace_status(wa) == kda.KDA_OK
    for t in range(40):
        assert torch.equal(outs[t][0], forks[t][0]) and torch.equal(outs[t][1], forks[t][1])
        for b in range(B):
            for h in range(hq):
                seen = torch.ones(1, t + 1, dtype=torch.bool, device=DEV)
                ref = attn_ref.attend(q[t, b, :, h], k[b, :t + 1, h // 4], v[b, :t + 1, h // 4], seen, SCALE)
                attn_ref.check(outs[t][0][b, :, h], outs[t][1][b, :, h], ref)


@pytest.mark.parametrize("name,build", CASES, ids=[c[0] for c in CASES])
def test_captured_behind_copies_and_other_streams(name, build):
    """A graph whose calls follow a copy, a kernel and two streams that join."""
    call, ws, (q, *_) = build(BF)
    ref, ref_lse = call()
    torch.cuda.synchronize()
    x, y, z = q.clone(), torch.empty_like(q), torch.empty_like(q)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    outs = []
    with torch.cuda.graph(g):
        y.copy_(x)  # a copy node
        outs.append(call(q=y))
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            z.copy_(x)
            z.mul_(1.0)
        y.mul_(1.0)
        here.wait_stream(side)  # two nodes before the next call
        outs.append(call(q=z))
        outs.append(call(q=y))
    for _ in range(3):
        y.zero_()
        z.zero_()
        g.replay()
        torch.cuda.synchronize()
        for out, lse in outs:
            assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    assert kda.kda_workspace_status(ws) == kda.KDA_OK and not ws[:256].any()


@pytest.mark.parametrize("dt", [BF, F32])
def test_what_a_call_allocates_belongs_to_its_stream(dt):
    """On another stream than the current one, without a workspace or outputs of the
    caller's: nothing of the call waits for, or shares memory with, the current stream."""
    q, k, v = rows(41, 1200, 8, dt), rows(42, 1200, 2, dt), rows(43, 1200, 2, dt)
    x = make([900, 40], 2, 8, 2, 32, dt, seed=44)
    ref = kda.kda_attn_prefill(q, k, v, SCALE, output_lse=True)
    ref2 = kda.kda_attn_decode(x["q"], x["kp"], x["vp"], x["table"], x["lens"], SCALE, k_new=x["kn"], v_new=x["vn"],
                               output_lse=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        torch.cuda._sleep(20_000_000)  # the current stream is busy for some ten milliseconds
        done = torch.cuda.Event()
        done.record()
        junk = torch.full((1 << 22,), 0xFF, dtype=torch.uint8, device=DEV)  # freed at once, written late
        del junk
        got = kda.kda_attn_prefill(q, k, v, SCALE, output_lse=True, stream=side)
        got2 = kda.kda_attn_decode(x["q"], x["kp"], x["vp"], x["table"], x["lens"], SCALE, k_new=x["kn"], v_new=x["vn"],
                                   output_lse=True, stream=side)
        side.synchronize()
        assert not done.query()  # the side stream did not wait
        with torch.cuda.stream(side):
            for a, b in zip(got + got2, ref + ref2):
                assert torch.equal(a, b)
        torch.cuda.synchronize()
