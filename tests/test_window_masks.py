"""kda_attn_decode_window under draft masks that are no plain chain or tree of their own bits: tokens whose
masks lack their own bit, and drafts that all see one another."""
import os

import pytest
import torch

import kimi_delta_attention_rule_gb300 as kda
from kimi_delta_attention_rule_gb300 import build as kbuild
from tests import attn_ref
from tests.test_attn_decode import BF, DEV, F32, SCALE, make, tree_masks


def without_own_bits(mask):
    own = torch.tensor([(1 << t) - (2**64 if t == 63 else 0) for t in range(mask.shape[1])], dtype=torch.int64, device=mask.device)
    return mask & ~own


def reference(x, b, mask, window, sinks):
    """Keys that the tokens of sequence b look at, [T, cached + T]: of the new ones those of the mask, of the cache the
    positions from seq_len - (window - n) on and the sinks; n new tokens are seen, the token itself counted."""
    T, L = x["q"].shape[1], x["ks"][b].shape[0]
    seen = torch.zeros(T, L + T, dtype=torch.bool)
    for t in range(T):
        visible = {s for s in range(T) if (int(mask[b, t]) & (2**64 - 1)) >> s & 1}
        n = len(visible | {t})
        for j in range(L):
            seen[t, j] = j >= L - (window - n) or j < sinks
        for s in visible:
            seen[t, L + s] = True
    return seen.to(DEV)


def check(x, mask, window, sinks):
    ws = kda.attn_decode_workspace(x["q"], x["kp"], x["table"])
    out, lse = kda.kda_attn_decode_window(x["q"], x["kp"], x["vp"], x["table"], x["lens"], SCALE, window, sinks, k_new=x["kn"],
                                          v_new=x["vn"], tree_mask=mask, output_lse=True, workspace=ws)
    assert kda.kda_workspace_status(ws) == kda.KDA_OK
    G = x["q"].shape[2] // x["kn"].shape[2]
    for b in range(x["q"].shape[0]):
        seen = reference(x, b, mask, window, sinks)
        k, v = torch.cat([x["ks"][b], x["kn"][b]]), torch.cat([x["vs"][b], x["vn"][b]])
        for h in range(x["q"].shape[2]):
            attn_ref.check(out[b, :, h], lse[b, :, h], attn_ref.attend(x["q"][b, :, h], k[:, h // G], v[:, h // G], seen, SCALE))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,hq,hkv,window", [(2, 4, 2, 2), (6, 4, 2, 9), (24, 8, 2, 30), (64, 4, 2, 64), (64, 8, 1, 90)])
def test_ancestors_without_the_token_itself(T, hq, hkv, window, dt):
    x = make([0, 7, 100, 230], T, hq, hkv, 32, dt, seed=70)
    mask = tree_masks(4, T, T)
    mask[1] = torch.tensor([(2 << t) - 1 - (2**64 if t == 63 else 0) for t in range(T)], device=DEV)  # a chain: T - 1 ancestors
    mask = without_own_bits(mask)
    seen = torch.tensor([[bin(int(m) & (2**64 - 1)).count("1") for m in r] for r in mask.tolist()])
    assert (seen[:, 0] == 0).all() and int(seen.max()) == T - 1
    check(x, mask, window, 2)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("T,hq,hkv,window", [(2, 4, 2, 40), (20, 8, 2, 20), (64, 4, 2, 300), (64, 8, 1, 64)])
def test_drafts_that_all_see_one_another(T, hq, hkv, window, page, dt):
    """Every window starts T before the end. Pages that end at or before the length + 1 - window can be gone; those
    behind them, which no token looks at either, are there."""
    x = make([0, 30, 200, 700, 1100], T, hq, hkv, page, dt, seed=71)
    mask = torch.full((5, T), (1 << T) - 1 if T < 63 else -1, dtype=torch.int64, device=DEV)
    sinks = 3
    for b, n in enumerate(x["lens"].tolist()):
        for j in range((n + page - 1) // page):
            if j * page >= sinks and (j + 1) * page <= n + 1 - window:
                p = int(x["table"][b, j])
                x["kp"][p] = x["vp"][p] = float("nan")
                x["table"][b, j] = (kda.KDA_PAGE_GONE, -1, 2**31 - 1)[j % 3]
    check(x, mask, window, sinks)


def test_the_contract_names_the_pages():
    """A page may go by its place and the length alone, not by what a step's mask lets its tokens see."""
    text = " ".join(open(os.path.join(kbuild.INCLUDE, "kda.h")).read().replace(" *", " ").split())
    assert "Pages of which no token of the call sees a key" not in text
    assert "Pages without a sink that end at or before position seq_lens[b] + 1 - window (without k_new: seq_lens[b] - window) are not read" in text


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("B,T,hq,hkv,window", [(4, 64, 6, 2, 70), (3, 64, 5, 1, 64), (3, 40, 13, 1, 50), (2, 64, 64, 1, 100), (3, 9, 33, 1, 20),
                                               (4, 43, 12, 2, 600), (2, 50, 27, 1, 3000)])
def test_row_tiles_that_heads_do_not_divide(B, T, hq, hkv, window, dt):
    """More than 128 rows per kv head, in row tiles of whole tokens: each with a CTA of its own, or shared."""
    x = make([0, 37, 400, 1000][:B], T, hq, hkv, 16, dt, seed=72)
    check(x, tree_masks(B, T, T + hq), window, 3)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T", [3, 64])
def test_several_tokens_over_the_cache_alone(T, dt):
    """Without keys of their own all look at the last `window` cached ones, which may be fewer than the tokens."""
    x = make([0, 1, 17, 300, 999], T, 8, 2, 32, dt, seed=73)
    for window, sinks in ((2, 0), (40, 5), (500, 129)):
        ws = kda.attn_decode_workspace(x["q"], x["kp"], x["table"])
        out, lse = kda.kda_attn_decode_window(x["q"], x["kp"], x["vp"], x["table"], x["lens"], SCALE, window, sinks, output_lse=True, workspace=ws)
        assert kda.kda_workspace_status(ws) == kda.KDA_OK
        for b, n in enumerate(x["lens"].tolist()):
            j = torch.arange(n, device=DEV)
            seen = ((j >= n - window) | (j < sinks)).expand(T, n)
            for h in range(8):
                attn_ref.check(out[b, :, h], lse[b, :, h], attn_ref.attend(x["q"][b, :, h], x["ks"][b][:, h // 4], x["vs"][b][:, h // 4], seen, SCALE))
