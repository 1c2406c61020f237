"""The page calls count pages, rows and table entries in 32 bits, some tens of thousands past
the last one: sizes that would wrap are refused before any launch."""
import ctypes

import pytest

import kimi_delta_attention_rule_gb300 as kda
from kimi_delta_attention_rule_gb300 import build as kbuild

FAKE = ctypes.c_void_p(0x100000)  # never dereferenced
MOST = (1 << 31) - (1 << 16)      # pages, and entries of a table
TOP = (1 << 31) - 1


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load()


def calls(lib, rows, cols, pages):
    t = (FAKE, cols, rows, cols)
    ws = (FAKE, 1 << 40, None)
    return {"alloc": lambda: lib.kda_cache_alloc(*t, FAKE, FAKE, pages, 16, *ws),
            "fork": lambda: lib.kda_cache_fork(*t, FAKE, FAKE, pages, 16, FAKE, FAKE, 1, FAKE, *ws),
            "free": lambda: lib.kda_cache_free(*t, FAKE, FAKE, pages, FAKE, 1, *ws),
            "compact": lambda: lib.kda_cache_compact(*t, FAKE, pages, FAKE, FAKE, *ws)}


@pytest.mark.parametrize("rows,cols,pages", [(1, 1, TOP), (1, 1, MOST + 1), (1, TOP, 9), (TOP, 1, 9), (1 << 16, 1 << 16, 9),
                                             (1, MOST + 1, 9), (3, 1 << 30, 9)])
@pytest.mark.parametrize("name", ["alloc", "fork", "free", "compact"])
def test_sizes_that_would_wrap_are_refused(lib, name, rows, cols, pages):
    assert calls(lib, rows, cols, pages)[name]() == kda.KDA_ERR_INVALID_ARG
