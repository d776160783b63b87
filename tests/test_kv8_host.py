"""Refusals of the 8-bit paged cache's entry points: on the host, before any launch (no GPU needed)."""
import ctypes

import pytest
import torch

from block_wise_kv_gb300 import build, dllm

A = 0x10000  # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    dllm.load()


def _desc(**kw):
    return dllm.layer_desc(**{**dict(d_model=4096, n_heads=32, head_dim=128, rope_theta=1e4), **kw})


def _batch(batch=2, max_pages=12, M=64, R=1536, max_block=32, max_seq=768, ptr=A):
    return dllm.BatchC(batch, max_pages, M, R, max_block, max_seq, ptr, ptr, ptr, ptr, ptr, ptr, None)


def _kv8(k=A, v=A, ks=A, vs=A, pages=24, heads=8):
    return dllm.Kv8CacheC(k, v, ks, vs, pages, heads)


def _status(fn, *a):
    return getattr(dllm.load(), fn)(*[ctypes.byref(x) if isinstance(x, ctypes.Structure) else x for x in a])


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), 1), (dict(v=A + 8), 1), (dict(ks=A + 4), 1), (dict(vs=None), 1), (dict(pages=0), 1),
    (dict(heads=0), 1), (dict(heads=5), 1), (dict(heads=64), 1), (dict(pages=1 << 22), 2)])
def test_cache_is_checked(kw, status):
    kv = _kv8(**kw)
    size = ctypes.c_size_t()
    assert _status("dllm_kv8_write", _desc(), _batch(), A, 1024, 128, A, 1024, 128, kv, None) == status
    assert dllm.load().dllm_kv8_attention_workspace_size(ctypes.byref(_desc()), ctypes.byref(_batch()), ctypes.byref(kv),
                                                         ctypes.byref(size)) == status
    assert _status("dllm_kv8_attention", _desc(), _batch(), A, 4096, kv, A, 0, None, A, 1 << 40, None) == status


@pytest.mark.parametrize("args", [
    (None, 1024, 128, A, 1024, 128), (A, 1024, 128, A + 8, 1024, 128), (A, 1020, 128, A, 1024, 128),
    (A, 1024, 4, A, 1024, 128), (A, 1024, 128, A, -1024, 128), (A, 1024, 128, A, 1024, -128)])
def test_write_rows_are_checked(args):
    assert _status("dllm_kv8_write", _desc(), _batch(), *args, _kv8(), None) == dllm.DLLM_ERR_INVALID_ARGUMENT


def test_write_pool_wants_the_cache_heads():
    cache = dllm.CacheC(A, A, None, None, None, None, 24)
    assert _status("dllm_kv8_write_pool", _desc(), _batch(), cache, _kv8(heads=8), None) == dllm.DLLM_ERR_INVALID_ARGUMENT
    cache = dllm.CacheC(A, None, None, None, None, None, 24)
    assert _status("dllm_kv8_write_pool", _desc(), _batch(), cache, _kv8(heads=32), None) == dllm.DLLM_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("change,status", [
    (dict(q=None), 1), (dict(q=A + 8), 1), (dict(stride=4088), 1), (dict(stride=4100), 1), (dict(o=A + 2), 1),
    (dict(o=None), 1), (dict(rows=2), 1), (dict(lse=A + 2), 1), (dict(ws=A + 128), 1), (dict(ws=None), 1), (dict(ws_bytes=64), 3)])
def test_attention_arguments_are_checked(change, status):
    a = {**dict(q=A, stride=4096, o=A, rows=0, lse=A, ws=A, ws_bytes=1 << 40), **change}
    assert _status("dllm_kv8_attention", _desc(), _batch(), a["q"], a["stride"], _kv8(), a["o"], a["rows"], a["lse"], a["ws"],
                   a["ws_bytes"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 1), (dict(batch=65536), 2), (dict(max_pages=2), 1), (dict(max_pages=0), 1), (dict(M=-1), 1),
    (dict(R=-1), 1), (dict(max_seq=0), 1), (dict(ptr=A + 2), 1), (dict(ptr=None), 1)])
def test_plan_batch_is_checked(kw, status):
    ring = dllm.PageRingC(A, A, A + 64, 24)
    assert _status("dllm_batch_plan", _batch(**kw), A, A + 256, A, A, A, ring, None, None, None, None) == status


@pytest.mark.parametrize("ring", [(None, A, A + 64, 24), (A, None, A + 64, 24), (A, A, None, 24), (A, A, A, 24),
                                  (A, A, A + 4, 24), (A, A, A + 64, 0)])
def test_plan_ring_is_checked(ring):
    assert _status("dllm_batch_plan", _batch(), A, A + 256, A, A, A, dllm.PageRingC(*ring), None, None, None,
                   None) == dllm.DLLM_ERR_INVALID_ARGUMENT


def test_plan_buffers_are_checked():
    ring = dllm.PageRingC(A, A, A + 64, 24)
    for held, out, table, cub, cus, slot in ((None, A, A, A, A, None), (A, None, A, A, A, None), (A, A, A, A, A, None),
                                             (A, A + 4, A, A, A, None), (A, A + 64, None, A, A, None),
                                             (A, A + 64, A, None, A, None), (A, A + 64, A, A, A + 2, None),
                                             (A, A + 64, A, A, A, A + 4)):
        assert _status("dllm_batch_plan", _batch(), held, out, table, cub, cus, ring, slot, None, None,
                       None) == dllm.DLLM_ERR_INVALID_ARGUMENT
    assert _status("dllm_batch_plan", _batch(), A, A + 64, A, A, A, dllm.PageRingC(A, A, A + 64, 1 << 26), None, None, None,
                   None) == dllm.DLLM_ERR_UNSUPPORTED


def test_attention_refuses_more_rows_to_a_head_than_it_counts():
    wide = _desc(n_heads=40000, head_dim=64, d_model=64)
    b = _batch(batch=1, max_pages=1024, M=65536, R=65536, max_block=65536, max_seq=65536)
    assert _status("dllm_kv8_attention", wide, b, A, 1 << 22, _kv8(heads=1), A, 0, None, A, 1 << 40, None) == dllm.DLLM_ERR_UNSUPPORTED


def test_an_empty_batch_launches_nothing():
    b = _batch(batch=0, M=0, R=0)
    assert _status("dllm_kv8_write", _desc(), b, None, 0, 0, None, 0, 0, _kv8(), None) == 0
    assert _status("dllm_kv8_attention", _desc(), b, None, 0, _kv8(), None, 0, None, None, 0, None) == 0
    assert dllm.dllm_kv8_attention_workspace_size(_desc(), b, _kv8()) == 0


def test_binding_checks_layouts():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(dllm.DllmError):
        dllm.dllm_kv8_write(_desc(), _batch(), x.transpose(1, 2), x, _kv8())
    with pytest.raises(dllm.DllmError):
        dllm.dllm_kv8_attention(_desc(), _batch(), x[:, :, ::2], _kv8(), x, None, None)
    with pytest.raises(dllm.DllmError):
        dllm.dllm_kv8_attention(_desc(), _batch(), x[:, ::2], _kv8(), x, None, None)
    k = torch.zeros(3, 2, 64, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.ones(3, 2, 4)
    dllm.Kv8Cache.of(k, k.clone(), s, s.clone())
    with pytest.raises(ValueError):
        dllm.Kv8Cache.of(k, k[:2], s, s)
    with pytest.raises(ValueError):
        dllm.Kv8Cache.of(k, k, s, torch.ones(3, 2, 8))
    with pytest.raises(ValueError):
        dllm.Kv8Cache.of(k.view(torch.uint8), k, s, s)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        dllm.BatchView(i.view(2, 2), i.long(), i, i, i, i, 1, 1, 1, 1)
    with pytest.raises(ValueError):
        dllm.PageRing(i, i[::2], i)
    r = dllm.PageRing(i, i[:2], torch.ones(2, dtype=torch.int32))
    assert r.swapped().state is r.state_out and r.swapped().state_out is r.state and r.c.num_pages == 4


def _refused():
    return pytest.raises(dllm.DllmError, match="invalid argument")


@pytest.mark.parametrize("k,v", [((64, 8, 64), (64, 8, 64)), ((64, 4, 128), (64, 4, 128)), ((64, 8, 128), (64, 4, 128)),
                                 ((8, 64, 128), (8, 64, 128)), ((64, 1024), (64, 1024))])
def test_binding_checks_the_rows_shapes(k, v):
    with _refused():
        dllm.dllm_kv8_write(_desc(), _batch(), torch.zeros(k, dtype=torch.bfloat16), torch.zeros(v, dtype=torch.bfloat16),
                            _kv8())
    q = torch.zeros(k, dtype=torch.bfloat16)
    with _refused():
        dllm.dllm_kv8_attention(_desc(), _batch(), q, _kv8(), q, None, torch.zeros(4096, dtype=torch.uint8))


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32, torch.float8_e4m3fn])
def test_binding_checks_the_rows_types(dtype):
    good, bad = torch.zeros(64, 8, 128, dtype=torch.bfloat16), torch.zeros(64, 8, 128).to(dtype)
    for k, v in ((good, bad), (bad, good)):
        with _refused():
            dllm.dllm_kv8_write(_desc(), _batch(), k, v, _kv8())
    good, bad = torch.zeros(64, 32, 128, dtype=torch.bfloat16), torch.zeros(64, 32, 128).to(dtype)
    for q, o in ((good, bad), (bad, good)):
        with _refused():
            dllm.dllm_kv8_attention(_desc(), _batch(), q, _kv8(), o, None, torch.zeros(4096, dtype=torch.uint8))


@pytest.mark.parametrize("which", range(8))
def test_binding_checks_the_plans_types(which):
    t = [torch.zeros(8, dtype=torch.int32) for _ in range(8)]
    t[which] = t[which].long()
    ring = dllm.PageRing(torch.zeros(4, dtype=torch.int32), *torch.zeros(2, 2, dtype=torch.int32))
    with _refused():
        dllm.dllm_batch_plan(_batch(), *t[:5], ring.c, *t[5:])
