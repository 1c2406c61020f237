"""The bf16 attention kernel's waits are limited: whichever of its roles stops, wherever,
the call ends with KDA_ERR_TIMEOUT in its workspace and the next one is right."""
import ctypes
import os
import re

import pytest
import torch

import kimi_delta_attention_rule_gb300 as kda
from kimi_delta_attention_rule_gb300 import build as kbuild
from tests.test_attn_decode import BF, DEV, SCALE, make, tree_masks

SOURCE = os.path.join(kbuild.CSRC, "kda_attn_tc.cu")


def test_no_role_waits_without_a_limit():
    """Roles meet at mbarriers, through the one bounded wait; a named barrier would wait
    forever for a warp that has given up. The one that there is, between the two warps of a join's
    rows, has an arrival for a warp that leaves, and after a part's first meeting its partner looks
    whether it has. The whole CTA meets where every path arrives: after the set-up and at the end."""
    code = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    named = re.findall(r"\bbar(?:rier)?\.(?:cta\.)?(?:sync|red|arrive)\b[^;]*", code)
    assert named == ["barrier.sync %0, 64", "barrier.arrive %0, 64"]
    assert len(re.findall(r"try_wait", code)) == 1
    body = code[code.index("attn_tc_kernel(const"):]
    assert len(re.findall(r"__syncthreads\(\)", body)) == 2 and "cooperative_groups" not in code
    part = body[body.index("hand_over(quad);"):]
    meetings = [m.end() for m in re.finditer(r"hand_over\(quad\);", part)]
    assert len(meetings) == 4  # either warp: twice a half of the row
    for first in (meetings[0], meetings[2]):
        assert re.match(r"\s*if \(p == 0 && gone\[quad\] != 0\) \{\s*alive = false;\s*break;", part[first:])
    left = part.index("if (DUAL && !alive && __all_sync(0xffffffffu, gone[quad] == 0))")
    assert meetings[3] < left < part.index("hand_over_gone(quad);")
    # nothing that can give up stands between a part's first and last meeting
    assert "warp_wait" not in part[:meetings[1]] and "warp_wait" not in part[meetings[1]:meetings[3]]


FAKE = ctypes.c_void_p(0x100000)


def test_testing_entry_points_reject_bad_arguments():
    kbuild.build()
    lib = kda.load()
    pre = lambda io, warp, at: lib.kda_testing_attn_prefill_timeout(  # noqa: E731
        FAKE, FAKE, FAKE, 1024, 256, 256, 0.1, None, None, 1, 4, 4, 8, 2, 128, io, FAKE, None, FAKE, 16, warp, at, None)
    dec = lambda io, warp, at: lib.kda_testing_attn_decode_timeout(  # noqa: E731
        FAKE, 1024, None, None, 0, 0, FAKE, FAKE, 9, 16, FAKE, 4, 4, FAKE, None, 0.1, 2, 3, 8, 2, 128, io, FAKE, None, FAKE, 16,
        warp, at, None)
    for f in (pre, dec):
        for args in ((kda.KDA_F32, 0, 0), (kda.KDA_BF16, -1, 0), (kda.KDA_BF16, 12, 0), (kda.KDA_BF16, 0, -1),
                     (kda.KDA_BF16, 0, 0)):  # the last: a workspace of 16 bytes
            assert f(*args) == kda.KDA_ERR_INVALID_ARG, args


def rows(seed, n, h):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(n, h, 128, generator=g, device=DEV).to(BF)


def prefill(lq, lk, hq, hkv):
    q, k, v = rows(1, sum(lq), hq), rows(2, sum(lk), hkv), rows(3, sum(lk), hkv)
    cq, ck = (torch.tensor([0] + torch.tensor(x).cumsum(0).tolist(), dtype=torch.int32, device=DEV) for x in (lq, lk))
    ws = kda.attn_prefill_workspace(q, k, cq)

    def lose(warp, at):
        out = torch.empty_like(q)
        return kda.load().kda_testing_attn_prefill_timeout(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), hq * 128, hkv * 128, hkv * 128, SCALE, cq.data_ptr(), ck.data_ptr(),
            len(lq), q.shape[0], k.shape[0], hq, hkv, 128, kda.KDA_BF16, out.data_ptr(), None, ws.data_ptr(), ws.numel(), warp,
            at, kda._stream_ptr(None)), out

    def call():
        return kda.kda_attn_prefill(q, k, v, SCALE, cu_seqlens=cq, cu_seqlens_k=ck, workspace=ws)[0]

    return lose, call, ws


def decode(lens, T, hq, hkv, page):
    x = make(lens, T, hq, hkv, page, BF, seed=30)
    mask, ws = tree_masks(len(lens), T, 31), kda.attn_decode_workspace(x["q"], x["kp"], x["table"])

    def lose(warp, at):
        out, t = torch.empty_like(x["q"]), x["table"]
        return kda.load().kda_testing_attn_decode_timeout(
            x["q"].data_ptr(), hq * 128, x["kn"].data_ptr(), x["vn"].data_ptr(), hkv * 128, hkv * 128, x["kp"].data_ptr(),
            x["vp"].data_ptr(), x["kp"].shape[0], page, t.data_ptr(), t.stride(0), t.shape[1], x["lens"].data_ptr(),
            mask.data_ptr(), SCALE, len(lens), T, hq, hkv, 128, kda.KDA_BF16, out.data_ptr(), None, ws.data_ptr(), ws.numel(),
            warp, at, kda._stream_ptr(None)), out

    def call():
        return kda.kda_attn_decode(x["q"], x["kp"], x["vp"], x["table"], x["lens"], SCALE, k_new=x["kn"], v_new=x["vn"],
                                   tree_mask=mask, workspace=ws)[0]

    return lose, call, ws


FORMS = {
    "short prompts": lambda: prefill([100, 31, 7], [100, 31, 7], 8, 2),
    "prompts that CTAs share": lambda: prefill([1500, 200, 700], [1500, 200, 3000], 8, 1),
    "trees of two row tiles": lambda: decode([3000, 500, 1500], 64, 16, 2, 32),
    "trees of one row tile": lambda: decode([3000, 17, 1500], 20, 8, 2, 64),
    "one token": lambda: decode([9000, 300, 40], 1, 8, 2, 16),
    "short caches": lambda: decode([200, 30, 0], 2, 8, 2, 16),
}


@pytest.mark.gpu
@pytest.mark.parametrize("warp", [0, 1, 3, 4, 6, 7, 8, 9, 10, 11])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: f)
def test_a_role_that_stops_ends_the_call(form, warp):
    """(Test-only entry points: one warp of every CTA gives up at a wait of its own, the others'
    waits of 20 ms run out; nothing faults or hangs.)"""
    lose, call, ws = FORMS[form]()
    ref = call()
    torch.cuda.synchronize()
    assert kda.kda_workspace_status(ws) == kda.KDA_OK
    ended = 0
    for at in (0, 1, 2, 3, 4, 5, 6, 8, 11, 40):
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
    # (the scheduler waits only for descriptors that come back: short calls have four at the most)
    assert ended > 0 or warp == 10
