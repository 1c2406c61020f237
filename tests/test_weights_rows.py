"""The rows' tensor copies in the bf16 kernel of kda_attn_weights are waited for before a CTA ends, also
where a warp has given up: read from the source, and in calls of every way in which rows come."""
import os
import re

import pytest
import torch

import kimi_delta_attention_rule_gb300 as kda
from kimi_delta_attention_rule_gb300 import build as kbuild
from tests.test_attn_decode import BF, make
from tests.test_attn_weights import check, reference, run

SOURCE = os.path.join(kbuild.CSRC, "kda_attn_weights_tc.cu")


def test_copies_of_rows_complete_without_any_warp():
    """Each copy's barrier has one arrival, that of the copying warp itself ahead of the copies, so its phase
    ends with them; that warp counts them and waits for the last one wherever it leaves its loop."""
    code = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    rows = code[code.index("} else if (warp >= kWarpRows) {"):code.index("} else if (warp == kWarpTma) {")]
    bar = re.search(r"full = bar\(sh\.(\w+)\[half\]\)", rows).group(1)
    assert len(re.findall(r"attn::tma_3d\(lead, [^;]*, full\);", rows)) == len(re.findall(r"attn::tma_3d", rows)) == 2
    assert re.search(r"mbar_init\(bar\(sh\.%s\[i\]\), 1\)" % bar, code)
    assert not re.search(r"mbar_arrive\(bar\(sh\.%s\b" % bar, code)
    # nothing that can give up stands between the copies and their count
    copying = rows[rows.index("attn::expect_tx"):rows.index("sent[1] +=")]
    assert "wait" not in copying and "break" not in copying and "return" not in copying
    end = rows[rows.rindex("++nd;"):]
    assert re.search(r"for \(int i = 0; i < 2; \+\+i\) alive = wait_warp<kLimit>\(bar\(sh\.%s\[i\]\), \(sent\[i\] - 1\) & 1\)" % bar, end)
    assert "return" not in rows.replace("return i <", "")


@pytest.mark.gpu
@pytest.mark.parametrize("T,hq,hkv", [(1, 8, 2), (12, 8, 2), (50, 8, 2), (64, 16, 2), (33, 24, 2), (43, 32, 4), (64, 64, 1)])
@pytest.mark.parametrize("by_index", [False, True])
def test_parts_of_many_sequences(T, hq, hkv, by_index):
    """Many changes of rows per CTA: every tile and half of them is used over and over."""
    lens = [T + 90 * i for i in range(40)]
    x = make(lens, T, hq, hkv, 16, BF, seed=80)
    index = torch.arange(T, dtype=torch.int32, device="cuda:0").repeat(len(lens), 1) if by_index else None
    ref = reference(x, index)
    *r, st = run(x, index, None, ref)
    assert st == kda.KDA_OK
    check(x, *r)
