"""The example's two loops, whole: drafted trees and beam search over the paged cache, checked by
running the finished sequences through fresh pages in one pass."""
import importlib.util
import os

import pytest

from tests.gpu_util import ROOT, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def result():
    require_gpu()
    spec = importlib.util.spec_from_file_location("cached_decode", os.path.join(ROOT, "examples", "cached_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m.main()


def test_drafted_trees(result):
    """Every round accepts at least one token per lane, and the drafter is right often enough to
    take fewer rounds than tokens.  The bounds are bf16's: two roundings of activations of 2^-9
    each in two layers of four products, against logits' and keys' own spread."""
    assert result["rounds"] < 20 and result["tokens"] >= 40
    assert result["worst"] < 0.1 and result["moved"] < 0.02


def test_beam_search(result):
    assert result["scores"] == sorted(result["scores"], reverse=True)
    assert len({tuple(s) for s in result["seqs"]}) == len(result["seqs"])
    assert result["off"] < 0.3  # twelve log-probabilities
