"""Refusals of a layer's calls beyond what their kernels count and hold: on the host, before any launch (no GPU needed)."""
import pytest

from block_wise_kv_gb300 import build, dllm
from test_layer_host import A, FAR, _rope, _rows, _scores

MOST = (1 << 31) - 1  # rows of an int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    dllm.load()


@pytest.mark.parametrize("rows", [MOST, MOST - 1, MOST - 6, MOST - 255])
def test_more_rows_than_are_counted(rows):
    assert _scores(rows=rows, vocab=1, stride=1, tokens=None, logp=None, lse=A + 64 * FAR, top=0) == dllm.DLLM_ERR_UNSUPPORTED
    q = _rows(p=A, rs=128, hs=64, out=A, ors=128, ohs=64, heads=2)
    k = _rows(p=A + 256 * FAR, rs=64, hs=64, out=A + 256 * FAR, ors=64, ohs=64, heads=1)
    desc = dllm.layer_desc(128, 2, 64, 1e4)
    assert _rope(desc, rows, A + 600 * FAR, q, k, A + 700 * FAR, rotary=64) == dllm.DLLM_ERR_UNSUPPORTED


def _apart(**kw):
    """A call whose buffers lie apart but for the given ones."""
    return _scores(**{**dict(rows=4, vocab=1000, stride=1100, lse=A + 5 * FAR, entropy=A + 6 * FAR, err=A + 7 * FAR), **kw})


@pytest.mark.parametrize("kw", [
    # an output over another, over the tokens, the error word over an output
    dict(lse=A + 2 * FAR), dict(entropy=A + 5 * FAR + 12), dict(ids=A + 4 * FAR), dict(best=A + 3 * FAR + 28), dict(best=A + 2 * FAR + 12),
    dict(logp=A + FAR), dict(ids=A + FAR + 12), dict(lse=A + FAR - 12), dict(err=A + 6 * FAR + 8), dict(err=A + FAR),
    # over the logits: their first and last elements, the columns of a row, out of the columns between rows
    dict(lse=A), dict(entropy=A - 12), dict(lse=A + 2 * (3 * 1100 + 998)), dict(ids=A + 2 * 1100), dict(best=A + 2 * 500), dict(err=A + 4),
    dict(lse=A + 2 * 998), dict(ids=A + 2 * 1090)])
def test_scores_are_not_written_over_what_is_read_or_over_each_other(kw):
    assert _apart(**kw) == dllm.DLLM_ERR_INVALID_ARGUMENT
