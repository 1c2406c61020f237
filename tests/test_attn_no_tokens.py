"""Calls without a token: T = 0 is nothing to do, and the workspace it asks for is
one that a call of some tokens could start with (the status word's)."""
import subprocess
import sys

import pytest
import torch

import kimi_delta_attention_rule_gb300 as kda
from kimi_delta_attention_rule_gb300 import build as kbuild


@pytest.fixture(scope="module", autouse=True)
def built():
    kbuild.build()


@pytest.mark.parametrize("io", [kda.KDA_BF16, kda.KDA_F32])
@pytest.mark.parametrize("B", [0, 1, 2])
def test_workspace_queries(B, io):
    """(In a process of its own: a division by zero would end this one.)"""
    code = ("import kimi_delta_attention_rule_gb300 as kda\n"
            "print(kda.kda_attn_decode_workspace_size(%d, 0, 8, 2, 128, 16, 4, %d),"
            " kda.kda_attn_prefill_workspace_size(%d, 0, 0, 8, 2, 128, %d))" % (B, io, B, io))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=kbuild.ROOT)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    assert all(int(n) >= 256 for n in r.stdout.split()), r.stdout


def test_workspace_of_a_batch_without_tokens():
    q = torch.empty(3, 0, 8, 128, dtype=torch.bfloat16)
    pages, table = torch.empty(4, 2, 16, 128, dtype=torch.bfloat16), torch.zeros(3, 5, dtype=torch.int32)
    assert kda.attn_decode_workspace(q, pages, table).numel() >= 256


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B", [0, 1, 3])
def test_calls_are_no_ops(B, dt):
    """Empty q, k_new, v_new (and slices of a wider projection), with and without a workspace."""
    dev = "cuda:0"
    pages = torch.zeros(4, 2, 16, 128, dtype=dt, device=dev)
    table, lens = torch.zeros(B, 5, dtype=torch.int32, device=dev), torch.ones(B, dtype=torch.int32, device=dev)
    fused = torch.empty(B, 2, 12, 128, dtype=dt, device=dev)[:, :0]
    for q, k, v in ((torch.empty(B, 0, 8, 128, dtype=dt, device=dev),) + (torch.empty(B, 0, 2, 128, dtype=dt, device=dev),) * 2,
                    (fused[:, :, :8], fused[:, :, 8:10], fused[:, :, 10:])):
        for ws in (None, kda.attn_decode_workspace(q, pages, table)):
            for new in (dict(k_new=k, v_new=v), {}):
                out, lse = kda.kda_attn_decode(q, pages, pages, table, lens, 0.1, output_lse=True, workspace=ws, **new)
                assert out.shape == (B, 0, 8, 128) and lse.shape == (B, 0, 8)
        kda.kda_cache_append(k, v, pages, pages, table, lens)
        kda.kda_cache_append(k, v, pages, pages, table, lens, index=table[:, :0].contiguous(), count=torch.zeros_like(lens))
    torch.cuda.synchronize()
    assert not pages.any()
