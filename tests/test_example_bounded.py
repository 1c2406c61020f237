"""The example of bounded contexts runs, and its caches hold no more than they should."""
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.gpu
def test_bounded_decode():
    import bounded_decode as ex
    results = ex.main()
    _, pages, full = results["whole"]
    assert pages == sum((n + 40 + 15) // 16 for n in (150, 40, 333))
    _, window_pages, _ = results["windowed"]
    # per sequence: a page of sinks, and those that the last 64 tokens touch
    assert window_pages <= 3 * (1 + 64 // 16 + 1)
    _, pages, cache = results["evicting"]
    assert max(cache.lens.tolist()) <= 64 + 16 and pages <= 3 * 5 and pages == int((cache.table >= 0).sum())
    assert all(error == error for error, _, _ in results.values())
