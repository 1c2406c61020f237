"""Attention calls of which many rows in a row see no key: sequences without keys, tokens ahead of a sequence's first key,
empty caches without new keys. They come out as zeros and -inf, those among them right, in any number."""
import math

import pytest
import torch

import kimi_delta_attention_rule_gb300 as kda
from tests import attn_ref
from tests.test_attn_decode import BF, DEV, F32, SCALE, make, normal
from tests.test_attn_window import offsets

pytestmark = pytest.mark.gpu


def prefill(lq, lk, hq, hkv, dt, window):
    q, k, v = normal(1, (sum(lq), hq, 128), dt, 2.0), normal(2, (sum(lk), hkv, 128), dt), normal(3, (sum(lk), hkv, 128), dt)
    ws = kda.attn_prefill_workspace(q, k, offsets(lq))
    kw = dict(cu_seqlens=offsets(lq), cu_seqlens_k=offsets(lk), output_lse=True, workspace=ws, out=torch.full_like(q, math.nan),
              lse=torch.full((sum(lq), hq), math.nan, device=DEV))
    out, lse = kda.kda_attn_prefill(q, k, v, SCALE, **kw) if window is None else kda.kda_attn_prefill_window(q, k, v, SCALE, window, 3, **kw)
    assert kda.kda_workspace_status(ws) == kda.KDA_OK
    a = c = 0
    for m, n in zip(lq, lk):
        p, j = torch.arange(n - m, n, device=DEV)[:, None], torch.arange(n, device=DEV)[None]
        seen = (j <= p) & ((j > p - (window or 2**31)) | (j < 3))
        for h in range(0, hq, 3):
            attn_ref.check(out[a:a + m, h], lse[a:a + m, h], attn_ref.attend(q[a:a + m, h], k[c:c + n, h * hkv // hq], v[c:c + n, h * hkv // hq], seen, SCALE))
        none = p[:, 0] < 0
        assert (out[a:a + m][none] == 0).all() and (lse[a:a + m][none] == -math.inf).all()
        a, c = a + m, c + n


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("window", [None, 50, 2**31 - 1])
@pytest.mark.parametrize("lq,lk", [([300, 1, 1, 200], [300, 0, 1, 200]), ([2000, 9, 9, 9, 9, 500], [2000, 0, 0, 0, 0, 700]), ([1500], [20]),
                                   ([700, 900, 40], [700, 5, 38]), ([1] * 60 + [900], [0] * 59 + [3, 900]), ([5, 700], [0, 700]),
                                   ([40, 3], [0, 9]), ([1000, 800], [1000, 1])])
@pytest.mark.parametrize("hq,hkv", [(8, 8), (56, 8)])
def test_prompts(lq, lk, hq, hkv, window, dt):
    prefill(lq, lk, hq, hkv, dt, window)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("window", [None, 70, 2**31 - 1])
@pytest.mark.parametrize("T,hq,hkv", [(1, 8, 8), (3, 16, 8), (64, 24, 8)])
@pytest.mark.parametrize("lens", [[3000] + [0] * 30 + [2000, 900], [0, 0, 5000, 0, 0, 0, 0, 0, 1, 0], [0] * 40, [100, 0, 0, 0, 17], [2500] * 20 + [0] * 44])
def test_padded_batches_without_new_keys(lens, T, hq, hkv, window, dt):
    """Sequences of a batch that hold nothing (yet, or any more): a serving batch's free places."""
    if T == 64:
        lens = lens[:12]
    x = make(lens, T, hq, hkv, 32, dt, seed=99)
    ws = kda.attn_decode_workspace(x["q"], x["kp"], x["table"])
    kw = dict(output_lse=True, workspace=ws, out=torch.full_like(x["q"], math.nan), lse=torch.full(x["q"].shape[:3], math.nan, device=DEV))
    if window is None:
        out, lse = kda.kda_attn_decode(x["q"], x["kp"], x["vp"], x["table"], x["lens"], SCALE, **kw)
    else:
        out, lse = kda.kda_attn_decode_window(x["q"], x["kp"], x["vp"], x["table"], x["lens"], SCALE, window, 3, **kw)
    assert kda.kda_workspace_status(ws) == kda.KDA_OK
    for b, n in enumerate(lens):
        if n == 0:
            assert (out[b] == 0).all() and (lse[b] == -math.inf).all()
            continue
        j = torch.arange(n, device=DEV)
        seen = ((j >= n - (window or 2**31)) | (j < 3)).expand(T, n)
        for h in range(0, hq, 5):
            attn_ref.check(out[b, :, h], lse[b, :, h], attn_ref.attend(x["q"][b, :, h], x["ks"][b][:, h * hkv // hq], x["vs"][b][:, h * hkv // hq], seen, SCALE))
