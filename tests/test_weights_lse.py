"""What kda_attn_weights adds up with the lse of each attention call: probabilities, one in all for each row, with
those over the whole context; through a window its formula still, which is then no probability, as the header says."""
import os

import pytest
import torch

import kimi_delta_attention_rule_gb300 as kda
from kimi_delta_attention_rule_gb300 import build as kbuild
from tests.test_attn_decode import BF, DEV, F32, SCALE, make, normal, tree_masks


def test_the_header_tells_them_apart():
    text = " ".join(open(os.path.join(kbuild.INCLUDE, "kda.h")).read().replace(" *", " ").split())
    assert "from the attention call of these rows" not in text
    assert "The sum has no window: with the lse of kda_attn_prefill_window or kda_attn_decode_window" in text
    for source in ("csrc/kda_attn_weights.cuh", "__init__.py"):
        text = open(os.path.join(kbuild.PKG, source)).read()
        assert "no probabilities" in text or "through a window" in text


def filled(lens, T, hq, hkv, dt, seed):
    """A cache that the T new tokens of each sequence can be appended to."""
    x = make(lens, T, hq, hkv, 16, dt, seed=seed, spare=0, fill=0.0)
    pages, cols = 200, 40
    table = torch.full((len(lens), cols), -1, dtype=torch.int32, device=DEV)
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    kp, vp = (torch.zeros(pages, hkv, 16, 128, device=DEV, dtype=dt) for _ in range(2))
    kda.kda_cache_alloc(table, x["lens"] + T, refs, 16)
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    kda.kda_cache_append(torch.cat(x["ks"]), torch.cat(x["vs"]), kp, vp, table, torch.zeros_like(x["lens"]), cu_seqlens=cu)
    return dict(x, kp=kp, vp=vp, table=table, cu=cu)


def check_sums(w, rows, G, dt):
    """w [.., cap] adds up to `rows` rows' probabilities per query head. A logit of two kernels' fp32 dot products
    differs by at most 2 * 136 * 2 * 2^-24 scale |q||k|, here below 2^-14 (|q| < 2 * 16, |k| < 16, scale |q||k| < 46); lse
    and the exponentials by less than 2^-19; sums of up to 700 terms by 700 * 2^-24."""
    total = w.double().sum(-1)
    tol = (272 * 2 * 2.0**-24 * 46 + 2.0**-18 + 700 * 2.0**-24) * G * rows
    assert ((total - G * rows).abs() <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,hq,hkv", [(1, 8, 2), (6, 8, 2), (40, 8, 2)])
def test_a_chain_and_an_accepted_path(T, hq, hkv, dt):
    lens, G = [600, 3, 77], hq // hkv
    x = filled(lens, T, hq, hkv, dt, 90)
    for tree in (False, True):
        mask = tree_masks(3, T, T + 1) if tree else None
        _, lse = kda.kda_attn_decode(x["q"], x["kp"], x["vp"], x["table"], x["lens"], SCALE, k_new=x["kn"], v_new=x["vn"], tree_mask=mask,
                                     output_lse=True)
        paths = [[s for s in range(T) if not tree or int(r[-1]) >> s & 1] for r in (mask.tolist() if tree else [[0]] * 3)]
        index = torch.tensor([p + [0] * (T - len(p)) for p in paths], dtype=torch.int32, device=DEV)
        count = torch.tensor([len(p) for p in paths], dtype=torch.int32, device=DEV)
        kda.kda_cache_append(x["kn"], x["vn"], x["kp"], x["vp"], x["table"], x["lens"], index=index, count=count)
        w = kda.kda_attn_weights(x["q"], x["kp"], x["table"], x["lens"] + count, lse, SCALE, index=index, count=count)
        check_sums(w, count[:, None], G, dt)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
def test_a_whole_prompt_by_stretches_of_64(dt):
    n, hq, hkv = 300, 4, 2
    x = filled([n], 1, hq, hkv, dt, 91)
    q = normal(7, (n, hq, 128), dt, 2.0)
    _, lse = kda.kda_attn_prefill(q, x["ks"][0], x["vs"][0], SCALE, output_lse=True)
    w = torch.zeros(1, hkv, 640, device=DEV)
    for a in range(0, n, 64):
        z = min(n, a + 64)
        kda.kda_attn_weights(q[None, a:z], x["kp"], x["table"], torch.tensor([z], dtype=torch.int32, device=DEV), lse[None, a:z].contiguous(), SCALE, w)
    check_sums(w, torch.tensor([[n]], device=DEV), hq // hkv, dt)
    assert not w[..., n:].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
def test_with_a_windows_lse_they_are_no_probabilities(dt):
    x = filled([600, 300], 1, 8, 2, dt, 92)
    _, lse = kda.kda_attn_decode_window(x["q"], x["kp"], x["vp"], x["table"], x["lens"], SCALE, 30, 2, k_new=x["kn"], v_new=x["vn"], output_lse=True)
    kda.kda_cache_append(x["kn"], x["vn"], x["kp"], x["vp"], x["table"], x["lens"])
    w = kda.kda_attn_weights(x["q"], x["kp"], x["table"], x["lens"] + 1, lse, SCALE)
    assert (w.double().sum(-1) > 2 * 4).all()  # one for each of four heads would be 4
