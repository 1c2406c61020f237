"""How far an infinity or a NaN in v reaches through a window: the rows that look at it, at most those of blocks that read
its key tile, and never another channel or sequence."""
import math

import pytest
import torch

import kimi_delta_attention_rule_gb300 as kda
from tests import attn_ref
from tests.test_attn_decode import BF, DEV, F32, SCALE, make, normal
from tests.test_attn_window import offsets, seen_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,tile,rows", [(BF, 128, 256), (F32, 64, 64)])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("at,window,sinks,prefix", [(700, 100, 4, 0), (700, 300, 0, 77), (333, 1, 20, 500), (900, 64, 140, 100)])
def test_prompts(at, window, sinks, prefix, bad, dt, tile, rows):
    lq, hq, hkv = [90, 1200, 50], 4, 2
    lk, block = [lq[0], lq[1] + prefix, lq[2]], rows // (hq // hkv)
    q, k, v = normal(1, (sum(lq), hq, 128), dt, 2.0), normal(2, (sum(lk), hkv, 128), dt), normal(3, (sum(lk), hkv, 128), dt)
    v[lk[0] + at, :, 5] = 0
    ref_v = v.clone()
    v[lk[0] + at, :, 5] = bad
    out, lse = kda.kda_attn_prefill_window(q, k, v, SCALE, window, sinks, cu_seqlens=offsets(lq), cu_seqlens_k=offsets(lk), output_lse=True)
    a = c = 0
    for b, (m, n) in enumerate(zip(lq, lk)):
        seen = seen_rows(m, n, window, sinks)
        for h in range(hq):
            ref = attn_ref.attend(q[a:a + m, h], k[c:c + n, h // 2], ref_v[c:c + n, h // 2], seen, SCALE)
            o = out[a:a + m, h].clone()
            if b == 1:
                looks = seen[:, at]
                assert not torch.isfinite(o[looks, 5]).any()  # (none in the case whose windows all start behind it)
                near = seen[:, max(0, at - tile + 1):at + tile].any(1)  # a key that may share its tile
                reached = torch.tensor([bool(near[i // block * block:(i // block + 1) * block].any()) for i in range(m)], device=DEV)
                assert not reached.all()
                o[reached, 5] = ref[0][reached, 5].to(dt)
            attn_ref.check(o, lse[a:a + m, h], ref)
        a, c = a + m, c + n


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T", [1, 20])
def test_decode(T, dt):
    """In a page that no call reads: nothing. In one that is read: its channel, in its sequence's rows."""
    x = make([900, 1000], T, 8, 2, 32, dt, seed=97)
    window, sinks = 100, 4
    call = lambda vp: kda.kda_attn_decode_window(x["q"], x["kp"], vp, x["table"], x["lens"], SCALE, window, sinks, k_new=x["kn"],  # noqa: E731
                                                 v_new=x["vn"], output_lse=True)
    out, lse = call(x["vp"])
    for slot, read in ((40, False), (799, False), (850, True), (899, True)):  # the first window starts at 801, in the page from 800 on
        v = x["vp"].clone()
        v[int(x["table"][0, slot // 32]), :, slot % 32, 5] = math.nan
        o, y = call(v)
        assert torch.equal(y, lse) and torch.equal(o[1], out[1])
        channel = torch.arange(128, device=DEV) == 5
        assert torch.equal(o[0][..., ~channel], out[0][..., ~channel])
        assert torch.equal(o[0], out[0]) if not read else torch.isnan(o[0][..., 5]).any()
