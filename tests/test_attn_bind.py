"""What the attention and cache calls refuse before they look at a device: on the CPU."""
import pytest
import torch

import kimi_delta_attention_rule_gb300 as kda
from kimi_delta_attention_rule_gb300 import build as kbuild


@pytest.fixture(scope="module", autouse=True)
def built():
    kbuild.build()


def test_host_tensors_are_refused():
    q, k = torch.zeros(4, 2, 128, dtype=torch.bfloat16), torch.zeros(4, 1, 128, dtype=torch.bfloat16)
    pages, table = torch.zeros(2, 1, 16, 128, dtype=torch.bfloat16), torch.zeros(2, 1, dtype=torch.int32)
    i32 = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: kda.kda_attn_prefill(q, k, k, 1.0),
                 lambda: kda.kda_attn_decode(q[:2, None], pages, pages, table, i32, 1.0),
                 lambda: kda.kda_cache_alloc(table, i32, i32, 16),
                 lambda: kda.kda_cache_fork(table, i32, i32, i32, i32, 16),
                 lambda: kda.kda_cache_free(table, i32, i32, i32),
                 lambda: kda.kda_cache_compact(table, i32),
                 lambda: kda.kda_cache_copy([pages], table),
                 lambda: kda.kda_cache_append(k, k, pages, pages, table, i32[:1], cu_seqlens=i32)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_other_objects_are_refused():
    q = torch.zeros(4, 2, 128)
    for call in (lambda: kda.kda_attn_prefill(None, q, q, 1.0), lambda: kda.kda_attn_prefill(q, q, [1], 1.0),
                 lambda: kda.kda_cache_alloc(3, q, q, 16), lambda: kda.kda_cache_copy(7, q),
                 lambda: kda.kda_cache_copy([None], q)):
        with pytest.raises(TypeError):
            call()
    kda.kda_cache_copy([], q)  # nothing to do


def test_other_dtypes_have_no_kernel():
    """Every entry that takes rows names the types that it has; the check needs no device of its own."""
    q = torch.zeros(4, 2, 128, dtype=torch.float16)
    with pytest.raises((ValueError, kda.KDAError)):
        kda.kda_attn_prefill(q, q, q, 1.0)
