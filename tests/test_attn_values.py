"""What attention does with values that a bound on rounding does not tell apart: every key
counts once, an infinity in v stays in its channel and its key tile, other types have no
kernel."""
import math

import pytest
import torch

import kimi_delta_attention_rule_gb300 as kda
from tests import attn_ref
from tests.test_attn_decode import call, make, tree_masks
from tests.test_attn_prefill import DEV, SCALE, offsets, rows

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
WIDTH = 127  # key j of a sequence has a one in channel j % WIDTH


def one_hot(n, h, dt, first=0):
    v = torch.zeros(n, h, 128, device=DEV)
    at = torch.arange(first, first + n, device=DEV)
    v[at - first, :, at % WIDTH] = 1
    return v.to(dt)


def check_counts(out, lse, counts):
    """Rows of [r, 128] counts of the keys seen per channel. With q = 0 every p is 1: l and O are whole
    numbers below 2^24, so out is off by the roundings of 1 / l, the product and the
    result, lse by the logarithm's last place and its own. One key more or less is 1/71 of its channel's."""
    assert counts.max() <= 71
    n = counts.sum(1, keepdim=True)
    want = counts / n.clamp(min=1)
    u = attn_ref.U[out.dtype] + 2.0**-22
    assert ((out.double() - want).abs() <= u * want).all()
    some = n[:, 0] > 0
    assert torch.equal(lse == -math.inf, ~some)
    x = torch.log(n[some, 0])
    assert ((lse[some].double() - x).abs() <= 2.0**-22 * x).all()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("lq,lk,hq,hkv", [([5000], [5000], 4, 1), ([300], [9000], 8, 2), ([129, 1, 700], [129, 2000, 700], 2, 2),
                                          ([1], [8999], 8, 1), ([200], [150], 3, 1)])
def test_every_key_of_a_prompt_counts_once(lq, lk, hq, hkv, dt):
    q, k = torch.zeros(sum(lq), hq, 128, dtype=dt, device=DEV), rows(1, sum(lk), hkv, dt)
    v = torch.cat([one_hot(n, hkv, dt) for n in lk])
    out, lse = kda.kda_attn_prefill(q, k, v, SCALE, cu_seqlens=offsets(lq), cu_seqlens_k=offsets(lk), output_lse=True)
    a = 0
    for m, n in zip(lq, lk):
        sums = torch.cat([torch.zeros(1, 128, dtype=torch.float64, device=DEV), one_hot(n, 1, F32)[:, 0].double().cumsum(0)])
        seen = (torch.arange(m, device=DEV) + n - m + 1).clamp(min=0)
        for h in range(hq):
            check_counts(out[a:a + m, h], lse[a:a + m, h], sums[seen])
        a += m


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,hq,hkv,page", [(1, 8, 2, 16), (7, 4, 1, 32), (20, 8, 2, 64), (64, 8, 1, 128)])
def test_every_key_of_a_cache_counts_once(T, hq, hkv, page, dt):
    lens = [8900, 130, 1, 0, 128]
    x = make(lens, T, hq, hkv, page, dt, seed=21)
    x["q"].zero_()
    for b, n in enumerate(lens):
        v = one_hot(n, hkv, dt)
        for j in range(0, n, page):
            x["vp"][x["table"][b, j // page], :, :min(page, n - j)] = v[j:j + page].transpose(0, 1)
        x["vn"][b] = one_hot(T, hkv, dt, first=n)
    mask = tree_masks(len(lens), T, 22)
    out, lse, st = call(x, mask)
    assert st == kda.KDA_OK
    for b, n in enumerate(lens):
        tree = (mask[b][:, None] >> torch.arange(T, device=DEV) & 1).double()
        counts = one_hot(n, 1, F32)[:, 0].double().sum(0) + tree @ one_hot(T, 1, F32, first=n)[:, 0].double()
        for h in range(hq):
            check_counts(out[b, :, h], lse[b, :, h], counts)


@pytest.mark.parametrize("dt,tile", [(BF, 128), (F32, 64)])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_an_infinity_in_v(dt, tile, bad):
    """Channel 5 of v's row 200 of sequence 1: the rows that see it have no finite channel 5, those
    whose keys end before its tile do; nothing else changes."""
    lens = [90, 400, 50]
    q, k, v = rows(61, 540, 4, dt, 2.0), rows(62, 540, 2, dt), rows(63, 540, 2, dt)
    v[90 + 200, :, 5] = 0
    ref_v = v.clone()
    v[90 + 200, :, 5] = bad
    out, lse = kda.kda_attn_prefill(q, k, v, SCALE, cu_seqlens=offsets(lens), output_lse=True)
    a = 0
    for b, n in enumerate(lens):
        seen = torch.ones(n, n, dtype=torch.bool, device=DEV).tril()
        for h in range(4):
            ref = attn_ref.attend(q[a:a + n, h], k[a:a + n, h // 2], ref_v[a:a + n, h // 2], seen, SCALE)
            o = out[a:a + n, h].clone()
            if b == 1:
                assert not torch.isfinite(o[200:, 5]).any()
                o[200 // tile * tile:, 5] = ref[0][200 // tile * tile:, 5].to(dt)
            attn_ref.check(o, lse[a:a + n, h], ref)
        a += n


def test_other_types_have_no_kernel():
    q, k = torch.zeros(4, 2, 128, dtype=torch.float16, device=DEV), torch.zeros(4, 1, 128, dtype=torch.float16, device=DEV)
    pages, table = torch.zeros(2, 1, 16, 128, dtype=torch.float16, device=DEV), torch.zeros(2, 1, dtype=torch.int32, device=DEV)
    i32 = torch.zeros(2, dtype=torch.int32, device=DEV)
    for f in (lambda t: t, lambda t: t.double(), lambda t: t.to(torch.float8_e4m3fn)):
        for fn in (lambda: kda.kda_attn_prefill(f(q), f(k), f(k), 1.0),
                   lambda: kda.kda_attn_decode(f(q)[:2, None], f(pages), f(pages), table, i32, 1.0),
                   lambda: kda.kda_cache_append(f(k), f(k), f(pages), f(pages), table, i32[:1], cu_seqlens=i32)):
            with pytest.raises(kda.KDAError) as e:
                fn()
            assert e.value.code == kda.KDA_ERR_UNSUPPORTED


def test_compact_of_a_pool_without_a_live_page():
    table, refs = torch.full((2, 3), -1, dtype=torch.int32, device=DEV), torch.zeros(9, dtype=torch.int32, device=DEV)
    got, count = kda.kda_cache_compact(table, refs)
    assert count.tolist() == [0] and (got == -1).all() and (table == -1).all() and not refs.any()
