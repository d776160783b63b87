"""What the Python binding of the 8-bit cache's calls takes and refuses, tensor by tensor.  The library is replaced by
one that counts its calls, so that a good call is seen to arrive and a bad one is seen not to; no GPU is needed."""
import pytest
import torch

from block_wise_kv_gb300 import dllm

H, KV, D, M, R, BATCH, PAGES = 4, 2, 64, 20, 150, 3, 5


class Elsewhere(torch.Tensor):
    """A tensor that says it lies on another device."""

    def get_device(self):
        return 1


def _elsewhere(t):
    return t.as_subclass(Elsewhere)


class Counting:
    def __init__(self):
        self.calls = 0

    def dllm_status_string(self, status):
        return b"invalid argument" if status == dllm.DLLM_ERR_INVALID_ARGUMENT else b""

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return dllm.DLLM_OK

        return call


@pytest.fixture
def lib(monkeypatch):
    fake = Counting()
    monkeypatch.setattr(dllm, "_lib", fake)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1)  # the tensors' own: the host's
    return fake


def _desc():
    return dllm.layer_desc(H * D, H, D, 1e4)


def _batch():
    return dllm.BatchC(BATCH, PAGES, M, R, 10, 100, 0, 0, 0, 0, 0, 0, None)


def _kv8():
    return dllm.Kv8CacheC(0, 0, 0, 0, 9, KV)


def _ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _refused(lib, fn, **args):
    lib.calls = 0
    with pytest.raises(dllm.DllmError, match="invalid argument"):
        fn(**args)
    assert lib.calls == 0


# ------------------------------------------------------------------ the plan
def _plan_args(**change):
    ring = dllm.PageRing(_ints(9), _ints(2), _ints(2))
    return {**dict(batch=_batch(), pages_held=_ints(BATCH), pages_held_out=_ints(BATCH), block_table=_ints(BATCH, PAGES),
                   cu_block=_ints(BATCH + 1), cu_seq=_ints(BATCH + 1), ring=ring.c, row_slot=_ints(M), row_seq=_ints(M),
                   row_pos=_ints(M), stream=0), **change}


@pytest.mark.parametrize("change", [
    {}, dict(row_slot=None, row_pos=None), dict(row_slot=_ints(M + 7)), dict(block_table=_ints(BATCH * PAGES)),
    dict(cu_block=_ints(40)[:BATCH + 1])])
def test_a_plan_that_fits_arrives(lib, change):
    dllm.dllm_batch_plan(**_plan_args(**change))
    assert lib.calls == 1


def test_the_batchs_own_buffers_arrive(lib):
    table, cub, cus = _ints(BATCH, PAGES), _ints(BATCH + 1), _ints(BATCH + 1)
    view = dllm.BatchView(table, _ints(BATCH), _ints(BATCH), _ints(BATCH), cub, cus, M, R, 10, 100)
    dllm.dllm_batch_plan(**_plan_args(batch=view.c, block_table=table, cu_block=cub, cu_seq=cus))
    assert lib.calls == 1


SIZES = dict(pages_held=BATCH, pages_held_out=BATCH, block_table=BATCH * PAGES, cu_block=BATCH + 1, cu_seq=BATCH + 1,
             row_slot=M, row_seq=M, row_pos=M)


@pytest.mark.parametrize("name", SIZES)
def test_a_plans_tensor_that_is_short_strided_of_another_type_or_elsewhere_is_refused(lib, name):
    n = SIZES[name]
    for bad in (_ints(n - 1), _ints(2 * n)[::2], torch.zeros(n), torch.zeros(n, dtype=torch.int64),
                torch.zeros(2 * n, dtype=torch.int16)):
        _refused(lib, dllm.dllm_batch_plan, **_plan_args(**{name: bad}))
    _refused(lib, dllm.dllm_batch_plan, **_plan_args(**{name: _elsewhere(_ints(n))}))


def test_tensors_of_another_device_than_the_current_one_are_refused(lib, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    _refused(lib, dllm.dllm_batch_plan, **_plan_args())
    _refused(lib, dllm.dllm_kv8_write, **_write_args())
    _refused(lib, dllm.dllm_kv8_attention, **_attention_args())


# ------------------------------------------------------------------ the write
def _rows(m=M, heads=KV, d=D, dtype=torch.bfloat16):
    return torch.zeros(m, heads, d, dtype=dtype)


def _write_args(**change):
    return {**dict(desc=_desc(), batch=_batch(), k_rows=_rows(), v_rows=_rows(), kv8=_kv8(), stream=0), **change}


@pytest.mark.parametrize("change", [
    {}, dict(k_rows=_rows(M + 3), v_rows=_rows(M + 3)), dict(k_rows=_rows(M, 8)[:, 2:4]),
    dict(v_rows=_rows(1).expand(M, -1, -1)), dict(k_rows=torch.zeros(M, 12 * D, dtype=torch.bfloat16)[:, D:3 * D].view(M, KV, D))])
def test_rows_that_fit_arrive(lib, change):
    dllm.dllm_kv8_write(**_write_args(**change))
    assert lib.calls == 1


def test_rows_that_do_not_fit_are_refused(lib):
    short = _rows(M - 1)
    for change in (dict(k_rows=short, v_rows=short), dict(v_rows=short), dict(k_rows=_rows(M, KV, 2 * D)[:, :, ::2]),
                   dict(k_rows=_rows(dtype=torch.float16)), dict(v_rows=_rows(M, KV + 1)),
                   dict(k_rows=_elsewhere(_rows())), dict(v_rows=_elsewhere(_rows()))):
        _refused(lib, dllm.dllm_kv8_write, **_write_args(**change))


# ------------------------------------------------------------------ the attention
def _attention_args(**change):
    return {**dict(desc=_desc(), batch=_batch(), q=_rows(M, H), kv8=_kv8(), o=_rows(M, H), lse=torch.zeros(M, H),
                   ws=torch.zeros(4096, dtype=torch.uint8), o_rows=dllm.DLLM_ROWS_BLOCK, stream=0), **change}


def _full(**change):
    return _attention_args(**{**dict(o=_rows(R, H), lse=torch.zeros(R, H), o_rows=dllm.DLLM_ROWS_FULL), **change})


@pytest.mark.parametrize("args", [
    _attention_args(), _attention_args(lse=None), _attention_args(q=_rows(M + 1, 3 * H)[:, H:2 * H]),
    _attention_args(o=torch.zeros(M, H * D, dtype=torch.bfloat16), lse=torch.zeros(M * H)), _attention_args(o=_rows(M + 5, H)),
    _full(), _full(lse=None), _full(q=_rows(M, H))])
def test_queries_that_fit_arrive(lib, args):
    dllm.dllm_kv8_attention(**args)
    assert lib.calls == 1


def test_a_single_head_has_any_head_stride(lib):
    desc = dllm.layer_desc(128, 1, 128, 1e4)
    q = torch.zeros(M, 128, 3, dtype=torch.bfloat16).transpose(1, 2)[:, :1].contiguous().as_strided((M, 1, 128), (128, 7, 1))
    dllm.dllm_kv8_attention(desc, _batch(), q, dllm.Kv8CacheC(0, 0, 0, 0, 9, 1), _rows(M, 1, 128), None,
                            torch.zeros(4096, dtype=torch.uint8), stream=0)
    assert lib.calls == 1


@pytest.mark.parametrize("make,rows", [(_attention_args, M), (_full, R)])
def test_outputs_that_do_not_fit_are_refused(lib, make, rows):
    for change in (dict(o=_rows(rows - 1, H)), dict(o=_rows(rows, 2 * H)[:, ::2]), dict(o=_rows(rows, H).transpose(0, 1)),
                   dict(o=_rows(rows, H, 2 * D)[:, :, :D]), dict(o=torch.zeros(rows, H, D)),
                   dict(lse=torch.zeros(rows - 1, H)), dict(lse=torch.zeros(rows, H, dtype=torch.bfloat16)),
                   dict(lse=torch.zeros(rows, H, dtype=torch.float64)), dict(lse=torch.zeros(rows, 2 * H)[:, :H]),
                   dict(q=_rows(M - 1, H)), dict(q=_rows(M, H, 2 * D)[:, :, :D]), dict(ws=torch.zeros(8192, dtype=torch.uint8)[::2]),
                   dict(q=_elsewhere(_rows(M, H))), dict(o=_elsewhere(_rows(rows, H))), dict(lse=_elsewhere(torch.zeros(rows, H))),
                   dict(ws=_elsewhere(torch.zeros(4096, dtype=torch.uint8)))):
        _refused(lib, dllm.dllm_kv8_attention, **make(**change))


# ------------------------------------------------------------------ the structs
def _view(**change):
    t = {**dict(block_table=_ints(BATCH, PAGES), seq_len=_ints(BATCH), block_start=_ints(BATCH), block_len=_ints(BATCH),
                cu_block=_ints(BATCH + 1), cu_seq=_ints(BATCH + 1), error=_ints(1)), **change}
    error = t.pop("error")
    return dllm.BatchView(*t.values(), M, R, 10, 100, error)


def test_a_views_tensors_hold_the_batch():
    v = _view(cu_block=_ints(BATCH + 9), block_table=_ints(BATCH + 1, PAGES), error=None)
    assert (v.c.batch, v.c.max_pages_per_seq) == (BATCH, PAGES)
    _view(block_table=_ints(0, 4), seq_len=_ints(0), block_start=_ints(0), block_len=_ints(0), cu_block=_ints(1), cu_seq=_ints(1))
    for change in (dict(block_table=_ints(BATCH - 1, PAGES)), dict(block_table=_ints(BATCH * PAGES)), dict(seq_len=_ints(BATCH, 1)),
                   dict(block_start=_ints(BATCH - 1)), dict(block_len=_ints(BATCH - 1)), dict(cu_block=_ints(BATCH)),
                   dict(cu_seq=_ints(BATCH)), dict(error=_ints(0)), dict(cu_seq=_ints(BATCH + 1).to("meta")),
                   dict(error=_ints(1).to("meta"))):
        with pytest.raises(ValueError):
            _view(**change)


def test_a_rings_and_a_caches_tensors_are_of_one_device_and_long_enough():
    dllm.PageRing(_ints(7), _ints(2), _ints(2))
    for bad in ((_ints(7), _ints(1), _ints(2)), (_ints(7), _ints(2), _ints(1)), (_ints(7, 1), _ints(2), _ints(2)),
                (_ints(7).to("meta"), _ints(2), _ints(2)), (_ints(7), _ints(2), _ints(2).to("meta"))):
        with pytest.raises(ValueError):
            dllm.PageRing(*bad)
    k = torch.zeros(3, 2, 64, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.ones(3, 2, 4)
    dllm.Kv8Cache.of(k, k.clone(), s, s.clone())
    with pytest.raises(ValueError):
        dllm.Kv8Cache.of(k, k, s, s.to("meta"))
