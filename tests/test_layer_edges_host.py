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
    """(One value a row, and one head: 4 GB and 256 GB, which fit the memory.)"""
    assert _scores(rows=rows, vocab=1, stride=1, tokens=None, logp=None, lse=A + 64 * FAR, top=0) == dllm.DLLM_ERR_UNSUPPORTED
    q = _rows(p=A, rs=64, hs=64, out=A, ors=64, ohs=64, heads=1)
    k = _rows(p=A + 256 * FAR, rs=64, hs=64, out=A + 256 * FAR, ors=64, ohs=64, heads=1)
    desc = dllm.layer_desc(64, 1, 64, 1e4)
    assert _rope(desc, rows, A + 600 * FAR, q, k, A + 700 * FAR, rotary=64) == dllm.DLLM_ERR_UNSUPPORTED
