"""The bf16 kernel of kda_attn_weights waits with limits: whichever of its roles stops, wherever, the
call ends with KDA_ERR_TIMEOUT in its workspace and the next one is right."""
import ctypes
import os
import re

import pytest
import torch

import kimi_delta_attention_rule_gb300 as kda
from kimi_delta_attention_rule_gb300 import build as kbuild
from tests.test_attn_decode import BF, DEV, SCALE, make


def test_no_role_waits_without_a_limit():
    """One bounded wait; the whole CTA meets after the set-up and at the end, where every path arrives."""
    code = re.sub(r"//[^\n]*", "", open(os.path.join(kbuild.CSRC, "kda_attn_weights_tc.cu")).read())
    assert len(re.findall(r"try_wait", code)) == 1 and not re.findall(r"\bbar(?:rier)?\.", code) and "cooperative_groups" not in code
    body = code[code.index("weights_tc_kernel(const"):code.index("launch_kernel(const")]
    assert len(re.findall(r"__syncthreads\(\)", body)) == 2
    assert len(re.findall(r"\breturn;", body)) == 1  # before anything is set up


FAKE = ctypes.c_void_p(0x100000)


def test_testing_entry_point_rejects_bad_arguments():
    kbuild.build()
    f = lambda io, warp, at: kda.load().kda_testing_attn_weights_timeout(  # noqa: E731
        FAKE, 1024, FAKE, 9, 16, FAKE, 4, 4, FAKE, FAKE, None, None, 0.1, 2, 3, 8, 3, 128, io, FAKE, 64, None, warp, at, None)
    for args in ((kda.KDA_F32, 0, 0), (kda.KDA_BF16, -1, 0), (kda.KDA_BF16, 22, 0), (kda.KDA_BF16, 0, -1),
                 (kda.KDA_BF16, 0, 0)):  # the last: heads that do not divide
        assert f(*args) == kda.KDA_ERR_INVALID_ARG, args


# (lengths, T, query heads, kv heads, with an index): 4, 40, 200 and 512 rows
FORMS = {"4 rows": ([9000, 300, 40], 1, 8, 2, False), "40 rows": ([3000, 17, 1500], 10, 8, 2, False), "200 rows": ([3000, 500], 50, 8, 2, False),
         "512 rows": ([2500, 1500, 100], 64, 16, 2, False), "512 rows by index": ([2500, 1500, 100], 64, 16, 2, True)}


@pytest.mark.gpu
@pytest.mark.parametrize("warp", [0, 3, 5, 10, 15, 16, 17, 18, 19, 21])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: f)
def test_a_role_that_stops_ends_the_call(form, warp):
    """(Test-only entry point: one warp of every CTA gives up at a wait of its own, the others' waits of
    20 ms run out; nothing faults or hangs.)"""
    lens, T, hq, hkv, by_index = FORMS[form]
    x = make(lens, T, hq, hkv, 32, BF, seed=60)
    B, t = len(lens), x["table"]
    lse = torch.full((B, T, hq), 4.0, device=DEV)
    index = torch.arange(T, dtype=torch.int32, device=DEV).flip(0).repeat(B, 1) if by_index else None
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    cap = t.shape[1] * 32

    def call():
        w = torch.zeros(B, hkv, cap, device=DEV)
        return kda.kda_attn_weights(x["q"], x["kp"], t, x["lens"], lse, SCALE, w, index=index, workspace=ws)

    def lose(at):
        w = torch.zeros(B, hkv, cap, device=DEV)
        return kda.load().kda_testing_attn_weights_timeout(
            x["q"].data_ptr(), hq * 128, x["kp"].data_ptr(), x["kp"].shape[0], 32, t.data_ptr(), t.stride(0), t.shape[1],
            x["lens"].data_ptr(), lse.data_ptr(), index.data_ptr() if by_index else None, None, SCALE, B, T, hq, hkv, 128,
            kda.KDA_BF16, w.data_ptr(), cap, ws.data_ptr(), warp, at, kda._stream_ptr(None)), w

    ref = call()
    assert kda.kda_workspace_status(ws) == kda.KDA_OK
    ended = 0
    for at in (0, 1, 2, 3, 5, 9, 30):
        rc, w = lose(at)
        assert rc == kda.KDA_OK, kda.status_string(rc)
        status = kda.kda_workspace_status(ws)
        if status == kda.KDA_OK:  # it has no such wait
            assert torch.equal(w, ref)
        else:
            assert status == kda.KDA_ERR_TIMEOUT
            ended += 1
        assert torch.equal(call(), ref)
        assert kda.kda_workspace_status(ws) == kda.KDA_OK
    assert ended > 0
