"""The waits of the bf16 attention kernel's windowed instances are limited like the plain ones': whichever
role stops, wherever, the call ends with KDA_ERR_TIMEOUT in its workspace and the next one is right."""
import ctypes

import pytest
import torch

import kimi_delta_attention_rule_gb300 as kda
from kimi_delta_attention_rule_gb300 import build as kbuild
from tests.test_attn_decode import BF, DEV, SCALE, make, tree_masks
from tests.test_attn_waits import rows

FAKE = ctypes.c_void_p(0x100000)


def test_testing_entry_points_reject_bad_arguments():
    kbuild.build()
    lib = kda.load()
    pre = lambda io, warp, at, w=9, s=2: lib.kda_testing_attn_prefill_window_timeout(  # noqa: E731
        FAKE, FAKE, FAKE, 1024, 256, 256, 0.1, w, s, None, None, 1, 4, 4, 8, 2, 128, io, FAKE, None, FAKE, 16, warp, at, None)
    dec = lambda io, warp, at, w=9, s=2: lib.kda_testing_attn_decode_window_timeout(  # noqa: E731
        FAKE, 1024, FAKE, FAKE, 256, 256, FAKE, FAKE, 9, 16, FAKE, 4, 4, FAKE, None, 0.1, w, s, 2, 3, 8, 2, 128, io, FAKE, None, FAKE, 16,
        warp, at, None)
    for f in (pre, dec):
        for args in ((kda.KDA_F32, 0, 0), (kda.KDA_BF16, -1, 0), (kda.KDA_BF16, 12, 0), (kda.KDA_BF16, 0, -1),
                     (kda.KDA_BF16, 0, 0, 0), (kda.KDA_BF16, 0, 0, 9, -1), (kda.KDA_BF16, 0, 0)):  # the last: a workspace of 16 bytes
            assert f(*args) == kda.KDA_ERR_INVALID_ARG, args
    assert dec(kda.KDA_BF16, 0, 0, 2) == kda.KDA_ERR_INVALID_ARG  # a window shorter than the drafts


def prefill(lens, hq, hkv, window, sinks):
    n = sum(lens)
    q, k, v = rows(1, n, hq), rows(2, n, hkv), rows(3, n, hkv)
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    ws = kda.attn_prefill_workspace(q, k, cu)

    def lose(warp, at):
        out = torch.empty_like(q)
        return kda.load().kda_testing_attn_prefill_window_timeout(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), hq * 128, hkv * 128, hkv * 128, SCALE, window, sinks, cu.data_ptr(), None,
            len(lens), n, n, hq, hkv, 128, kda.KDA_BF16, out.data_ptr(), None, ws.data_ptr(), ws.numel(), warp, at,
            kda._stream_ptr(None)), out

    return lose, lambda: kda.kda_attn_prefill_window(q, k, v, SCALE, window, sinks, cu_seqlens=cu, workspace=ws)[0], ws


def decode(lens, T, hq, hkv, page, window, sinks):
    x = make(lens, T, hq, hkv, page, BF, seed=95)
    mask, ws = tree_masks(len(lens), T, 96), kda.attn_decode_workspace(x["q"], x["kp"], x["table"])

    def lose(warp, at):
        out, t = torch.empty_like(x["q"]), x["table"]
        return kda.load().kda_testing_attn_decode_window_timeout(
            x["q"].data_ptr(), hq * 128, x["kn"].data_ptr(), x["vn"].data_ptr(), hkv * 128, hkv * 128, x["kp"].data_ptr(),
            x["vp"].data_ptr(), x["kp"].shape[0], page, t.data_ptr(), t.stride(0), t.shape[1], x["lens"].data_ptr(),
            mask.data_ptr(), SCALE, window, sinks, len(lens), T, hq, hkv, 128, kda.KDA_BF16, out.data_ptr(), None, ws.data_ptr(),
            ws.numel(), warp, at, kda._stream_ptr(None)), out

    return lose, lambda: kda.kda_attn_decode_window(x["q"], x["kp"], x["vp"], x["table"], x["lens"], SCALE, window, sinks, k_new=x["kn"],
                                                    v_new=x["vn"], tree_mask=mask, workspace=ws)[0], ws


FORMS = {
    "short prompts": lambda: prefill([300, 31, 7], 8, 2, 60, 4),
    "prompts that CTAs share": lambda: prefill([2500, 200, 3000, 900], 8, 2, 700, 20),
    "trees, a CTA for each row tile": lambda: decode([3000, 500, 1500], 64, 16, 2, 32, 200, 5),
    "trees of two row tiles that CTAs share": lambda: decode([9000, 500, 7000], 64, 16, 2, 32, 6000, 5),
    "trees of one row tile": lambda: decode([9000, 17, 8000], 20, 8, 2, 64, 5000, 130),
    "one token": lambda: decode([9000, 300, 40], 1, 8, 2, 16, 5000, 4),
    "one token, a CTA each": lambda: decode([900, 30, 0], 1, 8, 2, 16, 300, 4),
}


@pytest.mark.gpu
@pytest.mark.parametrize("warp", [0, 3, 4, 7, 8, 9, 10, 11])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: f)
def test_a_role_that_stops_ends_the_call(form, warp):
    """(Test-only entry points: one warp of every CTA gives up at a wait of its own, the others'
    waits of 20 ms run out; nothing faults or hangs.)"""
    lose, call, ws = FORMS[form]()
    ref = call()
    torch.cuda.synchronize()
    assert kda.kda_workspace_status(ws) == kda.KDA_OK
    ended = 0
    for at in (0, 1, 2, 3, 5, 8, 13, 40):
        rc, out = lose(warp, at)
        assert rc == kda.KDA_OK, kda.status_string(rc)
        status = kda.kda_workspace_status(ws)
        if status == kda.KDA_OK:  # it has no such wait
            assert torch.equal(out, ref)
        else:
            assert status == kda.KDA_ERR_TIMEOUT
            ended += 1
        again = call()
        torch.cuda.synchronize()
        assert torch.equal(again, ref)
        assert kda.kda_workspace_status(ws) == kda.KDA_OK and not ws[:256].any()
    # (the scheduler waits only for descriptors that come back: calls of few parts have none)
    assert ended > 0 or warp == 10
