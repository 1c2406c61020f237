"""kda_attn_decode over page numbers that are not in the pool: a pool without any page.
Their keys and values read as zeros, and the call is flagged."""
import pytest
import torch

import kimi_delta_attention_rule_gb300 as kda
from tests.test_attn_decode import BF, DEV, F32, call, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,hq,hkv", [(1, 8, 2), (3, 4, 2), (40, 8, 1), (64, 4, 1)])
@pytest.mark.parametrize("lens", [[1, 40, 16], [300, 0, 129]])
def test_a_pool_without_pages(lens, T, hq, hkv, dt):
    x = make(lens, T, hq, hkv, 16, dt, seed=20)
    x["kp"], x["vp"] = (torch.empty(0, hkv, 16, 128, dtype=dt, device=DEV) for _ in range(2))
    x["ks"], x["vs"] = ([torch.zeros(n, hkv, 128, dtype=dt, device=DEV) for n in lens] for _ in range(2))
    out, lse, st = call(x)
    assert st == kda.KDA_ERR_DEVICE
    check(x, out, lse)
