"""examples/hybrid_decode.py: prefill, fork, drafts, freeing and compaction of a KDA
layer and an attention layer together give what one prefill gives."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("seed", [0, 1])
def test_decoded_samples_match_one_prefill(seed):
    spec = importlib.util.spec_from_file_location("hybrid_decode", os.path.join(ROOT, "examples", "hybrid_decode.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    server, errors = example.main(seed)
    # two layers of bf16 rows, each rounded half a dozen times on both ways (2^-8 each)
    assert len(errors) == 4 and max(errors.values()) < 12 * 2.0**-8
    # pages are taken lowest first, so a pool once made dense stays dense
    live = int((server.refs > 0).sum())
    assert (server.refs[:live] > 0).all() and (server.refs[live:] == 0).all()
