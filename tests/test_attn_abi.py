"""Refusals of the attention and cache entry points, on the host: every call here
returns before any launch (no device memory is touched)."""
import ctypes
import math

import pytest

import kimi_delta_attention_rule_gb300 as kda
from kimi_delta_attention_rule_gb300 import build as kbuild

FAKE = ctypes.c_void_p(0x100000)  # never dereferenced
ODD = ctypes.c_void_p(0x100008)   # 8-byte aligned
BIG = 1 << 40
OK, INVALID, UNSUPPORTED = kda.KDA_OK, kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load()


def prefill(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, ldq=1024, ldk=256, ldv=256, scale=0.1, cu_q=FAKE, cu_k=FAKE, N=2, Tq=10, Tk=10, Hq=8, Hkv=2,
             D=128, io=0, out=FAKE, lse=None, ws=FAKE, nbytes=16)
    a.update(kw)
    return lib.kda_attn_prefill(a["q"], a["k"], a["v"], a["ldq"], a["ldk"], a["ldv"], a["scale"], a["cu_q"], a["cu_k"], a["N"],
                                a["Tq"], a["Tk"], a["Hq"], a["Hkv"], a["D"], a["io"], a["out"], a["lse"], a["ws"], a["nbytes"], None)


def test_new_status(lib):
    assert kda.status_string(kda.KDA_ERR_NO_SPACE) == "KDA_ERR_NO_SPACE"


def test_prefill_refusals(lib):
    for kw in (dict(D=64), dict(io=3), dict(Hq=130, Hkv=2, ldq=130 * 128)):
        assert prefill(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(Hq=7), dict(Hkv=0), dict(N=-1), dict(Tq=-1), dict(Tk=-2), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=math.nan), dict(scale=math.inf), dict(cu_q=None), dict(cu_k=None, Tk=11), dict(q=None), dict(k=None),
               dict(v=None), dict(out=None), dict(ws=None), dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(out=ODD), dict(ws=ODD),
               dict(ldq=1023), dict(ldq=1016), dict(ldk=260), dict(ldv=252), dict(nbytes=16), dict(lse=ctypes.c_void_p(0x100002)),
               dict(N=1 << 20, Tq=1 << 20, cu_q=None, cu_k=None)):
        assert prefill(lib, **{**dict(nbytes=BIG), **kw}) == INVALID, kw
    assert prefill(lib, io=1, ldk=258, nbytes=BIG) == INVALID  # fp32 rows: 16 bytes too
    # nothing to do: nothing is looked at
    assert prefill(lib, N=0, q=None, ws=None) == OK and prefill(lib, Tq=0, Tk=0, q=None, ws=None) == OK
    assert kda.kda_attn_prefill_workspace_size(2, 10, 10, 8, 3, 128, 0) == 0
    assert kda.kda_attn_prefill_workspace_size(2, 10, 10, 8, 2, 128, 0) > 256


def decode(lib, **kw):
    a = dict(q=FAKE, ldq=1024, kn=FAKE, vn=FAKE, ldk=256, ldv=256, kp=FAKE, vp=FAKE, P=9, page=16, table=FAKE, ld=4, cols=4,
             lens=FAKE, mask=None, scale=0.1, B=2, T=3, Hq=8, Hkv=2, D=128, io=0, out=FAKE, lse=None, ws=FAKE, nbytes=16)
    a.update(kw)
    return lib.kda_attn_decode(a["q"], a["ldq"], a["kn"], a["vn"], a["ldk"], a["ldv"], a["kp"], a["vp"], a["P"], a["page"],
                               a["table"], a["ld"], a["cols"], a["lens"], a["mask"], a["scale"], a["B"], a["T"], a["Hq"], a["Hkv"],
                               a["D"], a["io"], a["out"], a["lse"], a["ws"], a["nbytes"], None)


def test_decode_refusals(lib):
    for kw in (dict(D=96), dict(io=2), dict(T=65), dict(page=8), dict(page=48), dict(page=512), dict(Hq=130, ldq=130 * 128)):
        assert decode(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(Hq=9), dict(B=-1), dict(T=-1), dict(P=-1), dict(ld=3), dict(scale=-0.5), dict(kn=None), dict(vn=None),
               dict(kn=None, vn=None, mask=FAKE), dict(q=None), dict(out=None), dict(lens=None), dict(table=None), dict(kp=None),
               dict(vp=None), dict(ws=None), dict(q=ODD), dict(kn=ODD), dict(kp=ODD), dict(vp=ODD), dict(out=ODD),
               dict(mask=ctypes.c_void_p(0x100004)), dict(ldq=1000), dict(ldk=128), dict(ldv=255), dict(nbytes=16),
               dict(P=1 << 27, page=16), dict(cols=1 << 24, ld=1 << 24, page=256)):
        assert decode(lib, **{**dict(nbytes=BIG), **kw}) == INVALID, kw
    assert decode(lib, B=0, q=None, ws=None) == OK and decode(lib, T=0, q=None, ws=None) == OK
    assert kda.kda_attn_decode_workspace_size(2, 65, 8, 2, 128, 16, 4, 0) == 0
    assert kda.kda_attn_decode_workspace_size(2, 3, 8, 2, 128, 17, 4, 0) == 0


def test_cache_refusals(lib):
    need = kda.kda_cache_workspace_size(9, 4)
    assert need >= 256 and kda.kda_cache_workspace_size(-1, 4) == 0
    base = dict(t=FAKE, ld=5, rows=4, cols=5, refs=FAKE, P=9, ws=FAKE, nbytes=need)
    calls = {
        "alloc": lambda a: lib.kda_cache_alloc(a["t"], a["ld"], a["rows"], a["cols"], a.get("x", FAKE), a["refs"], a["P"],
                                               a.get("page", 16), a["ws"], a["nbytes"], None),
        "fork": lambda a: lib.kda_cache_fork(a["t"], a["ld"], a["rows"], a["cols"], a.get("x", FAKE), a["refs"], a["P"],
                                             a.get("page", 16), FAKE, a.get("dst", FAKE), a.get("n", 2), a.get("copies", FAKE),
                                             a["ws"], a["nbytes"], None),
        "free": lambda a: lib.kda_cache_free(a["t"], a["ld"], a["rows"], a["cols"], a.get("x", FAKE), a["refs"], a["P"], FAKE,
                                             a.get("n", 2), a["ws"], a["nbytes"], None),
        "compact": lambda a: lib.kda_cache_compact(a["t"], a["ld"], a["rows"], a["cols"], a["refs"], a["P"],
                                                   a.get("copies", FAKE), a.get("x", FAKE), a["ws"], a["nbytes"], None),
    }
    for name, f in calls.items():
        for kw in (dict(rows=-1), dict(cols=-1), dict(ld=4), dict(P=-1), dict(t=None), dict(refs=None), dict(ws=None), dict(ws=ODD),
                   dict(nbytes=need - 1), dict(refs=ODD), dict(x=None)):
            assert f({**base, **kw}) == INVALID, (name, kw)
    assert calls["alloc"]({**base, "page": 0}) == INVALID and calls["alloc"]({**base, "rows": 0}) == OK
    for kw in (dict(page=0), dict(n=-1), dict(n=5), dict(dst=None), dict(copies=None), dict(copies=ctypes.c_void_p(0x100004))):
        assert calls["fork"]({**base, **kw}) == INVALID, kw
    assert calls["fork"]({**base, "n": 0}) == OK
    assert calls["free"]({**base, "n": -1}) == INVALID and calls["free"]({**base, "n": 0}) == OK
    assert calls["compact"]({**base, "copies": None}) == INVALID


def test_copy_refusals(lib):
    two = (ctypes.c_void_p * 2)(0x100000, 0x200000)
    f = lambda pools=two, n=2, entry=64, entries=9, pairs=FAKE, m=3: lib.kda_cache_copy(pools, n, entry, entries, pairs, m, None, None)  # noqa: E731
    for kw in (dict(n=-1), dict(entry=-16), dict(entry=24), dict(entries=-1), dict(m=-1), dict(pools=None), dict(pairs=None),
               dict(pairs=ctypes.c_void_p(0x100004)), dict(pools=(ctypes.c_void_p * 2)(0x100000, 0x200008)),
               dict(pools=(ctypes.c_void_p * 2)(0x100000, None)), dict(entry=1 << 40)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(n=0), dict(m=0), dict(entries=0), dict(entry=0)):
        assert f(**kw) == OK, kw


def test_append_refusals(lib):
    def f(**kw):
        a = dict(k=FAKE, v=FAKE, ldk=256, ldv=256, cu=None, N=2, T=3, index=None, count=None, start=FAKE, t=FAKE, ld=4, cols=4, P=9,
                 page=16, Hkv=2, D=128, io=0, kp=FAKE, vp=FAKE, ws=None)
        a.update(kw)
        return lib.kda_cache_append(a["k"], a["v"], a["ldk"], a["ldv"], a["cu"], a["N"], a["T"], a["index"], a["count"], a["start"],
                                    a["t"], a["ld"], a["cols"], a["P"], a["page"], a["Hkv"], a["D"], a["io"], a["kp"], a["vp"],
                                    a["ws"], None)
    for kw in (dict(D=64), dict(io=9), dict(page=20)):
        assert f(**kw) == UNSUPPORTED, kw
    for kw in (dict(Hkv=0), dict(N=-1), dict(T=-1), dict(P=-1), dict(ld=3), dict(cu=FAKE, index=FAKE), dict(cu=FAKE, count=FAKE),
               dict(k=None), dict(v=None), dict(start=None), dict(t=None), dict(kp=None), dict(vp=None), dict(cols=0), dict(k=ODD),
               dict(v=ODD), dict(kp=ODD), dict(vp=ODD), dict(ldk=255), dict(ldv=252), dict(ws=ODD), dict(N=1 << 20, T=1 << 20)):
        assert f(**kw) == INVALID, kw
    assert f(N=0, k=None) == OK and f(T=0, k=None) == OK
