"""A windowed call over a batch with one long context among short ones, as many items as SMs or nearly: the long
context's work is shared, so the call takes no longer than the plain one over the whole contexts."""
import pytest
import torch

import kimi_delta_attention_rule_gb300 as kda
from tests.test_attn_decode import BF, DEV, SCALE, normal

pytestmark = pytest.mark.gpu


def times(*calls):
    """The least time of each call in a graph of ten, in us, in turn."""
    graphs = []
    for f in calls:
        f()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(10):
                f()
        g.replay()
        graphs.append(g)
    best = [1e9] * len(calls)
    for _ in range(5):
        for i, g in enumerate(graphs):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            g.replay()
            b.record()
            b.synchronize()
            best[i] = min(best[i], a.elapsed_time(b) * 100)
    return best


# Direct items took 8 to 12 times as long as the plain call here, shared ones about as long; half of that is the limit.
@pytest.mark.parametrize("window", [65536, 40000])
@pytest.mark.parametrize("T,G,hkv", [(1, 4, 8), (4, 4, 4), (64, 16, 1)])
def test_one_long_context(T, G, hkv, window):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    B = sms // (hkv * max(1, T * G // 128))
    lens = [65000] + [100] * (B - 1)
    page, used = 64, [(n + 63) // 64 for n in lens]
    table = torch.full((B, max(used)), -1, dtype=torch.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = torch.arange(at, at + u, dtype=torch.int32)
        at += u
    table, n = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    kp, vp = normal(1, (at, hkv, page, 128), BF), normal(2, (at, hkv, page, 128), BF)
    q, kn, vn = normal(3, (B, T, G * hkv, 128), BF), normal(4, (B, T, hkv, 128), BF), normal(5, (B, T, hkv, 128), BF)
    ws = kda.attn_decode_workspace(q, kp, table)
    plain, win = times(lambda: kda.kda_attn_decode(q, kp, vp, table, n, SCALE, k_new=kn, v_new=vn, workspace=ws),
                       lambda: kda.kda_attn_decode_window(q, kp, vp, table, n, SCALE, window, 4, k_new=kn, v_new=vn, workspace=ws))
    assert win <= 4 * plain, (win, plain)


def test_one_long_prefix():
    """The same of one new token each behind prefixes, through the prompts' call."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    hkv, G = 8, 4
    B = sms // hkv
    lk = [65000] + [100] * (B - 1)
    cu = lambda x: torch.tensor([0] + torch.tensor(x).cumsum(0).tolist(), dtype=torch.int32, device=DEV)  # noqa: E731
    q, k, v = normal(1, (B, G * hkv, 128), BF), normal(2, (sum(lk), hkv, 128), BF), normal(3, (sum(lk), hkv, 128), BF)
    ws, cq, ck = kda.attn_prefill_workspace(q, k, cu([1] * B)), cu([1] * B), cu(lk)
    plain, win = times(lambda: kda.kda_attn_prefill(q, k, v, SCALE, cu_seqlens=cq, cu_seqlens_k=ck, workspace=ws),
                       lambda: kda.kda_attn_prefill_window(q, k, v, SCALE, 65536, 4, cu_seqlens=cq, cu_seqlens_k=ck, workspace=ws))
    assert win <= 4 * plain, (win, plain)
