"""Refusals of a layer's products, head norms and token scores: on the host, before any launch (no GPU needed), and what
their Python binding takes."""
import ctypes

import pytest
import torch

from block_wise_kv_gb300 import build, dllm

A = 0x10000000  # never dereferenced
FAR = 0x100000000


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    dllm.load()


def _status(fn, *a):
    return getattr(dllm.load(), fn)(*[ctypes.byref(x) if isinstance(x, ctypes.Structure) else x for x in a])


# ------------------------------------------------------------------ dllm_linear
def _layer(**kw):
    return dllm.linear_desc(**{**dict(in_features=256, out_features=512), **kw})


def _linear(layer=None, rows=4, **kw):
    a = {**dict(x=A, xs=256, gain=None, w=A + FAR, bias=None, r=None, rs=512, y=A + 2 * FAR, ys=512, err=None, ws=None,
                wsb=0), **kw}
    return _status("dllm_linear", layer or _layer(), rows, a["x"], a["xs"], a["gain"], a["w"], a["bias"], a["r"], a["rs"],
                   a["y"], a["ys"], a["err"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(in_features=0), 1), (dict(in_features=-8), 1), (dict(in_features=12), 2), (dict(out_features=0), 1),
    (dict(act=4), 1), (dict(act=-1), 1), (dict(gated=2), 1), (dict(rms_eps=-1.0), 1), (dict(rms_eps=float("nan")), 1),
    (dict(rms_eps=float("inf")), 1), (dict(out_features=1 << 30), 2), (dict(in_features=(1 << 31) - 8), 2)])
def test_linear_layer_is_checked(kw, status):
    layer = _layer(**kw)
    if "gated" in kw:
        layer.gated = 2
    assert _linear(layer) == status
    size = ctypes.c_size_t()
    assert dllm.load().dllm_linear_workspace_size(ctypes.byref(layer), 4, 1, ctypes.byref(size)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(x=A + 8), 1), (dict(xs=248), 1), (dict(xs=260), 1), (dict(w=None), 1), (dict(w=A + FAR + 2), 1),
    (dict(gain=A + 2), 1), (dict(bias=A + 1), 1), (dict(r=A + 3 * FAR + 1), 1), (dict(r=A + 3 * FAR, rs=511), 1),
    (dict(y=None), 1), (dict(y=A + 2 * FAR + 1), 1), (dict(ys=511), 1), (dict(err=A + 2), 1), (dict(xs=1 << 39), 2),
    (dict(gain=A + FAR), 3), (dict(gain=A + FAR, wsb=1 << 20), 1), (dict(gain=A + FAR, ws=A + 128, wsb=1 << 20), 1),
    # y over what the call reads
    (dict(y=A), 1), (dict(y=A + 16), 1), (dict(y=A + FAR), 1), (dict(bias=A + 2 * FAR), 1),
    (dict(r=A + 2 * FAR + 2), 1), (dict(r=A + 2 * FAR, rs=520), 1), (dict(gain=A + FAR, ws=A + 2 * FAR, wsb=1 << 20), 1),
    (dict(gain=A + FAR, ws=A, wsb=1 << 20), 1), (dict(gain=A + FAR, ws=A + FAR, wsb=1 << 20), 1),
    (dict(gain=A + 5 * FAR, ws=A + 5 * FAR, wsb=1 << 20), 1), (dict(gain=A + 5 * FAR, bias=A + 6 * FAR, ws=A + 6 * FAR, wsb=1 << 20), 1),
    (dict(gain=A + 5 * FAR, r=A + 6 * FAR, ws=A + 6 * FAR, wsb=1 << 20), 1)])
def test_linear_arguments_are_checked(kw, status):
    assert _linear(**kw) == status


def test_linear_rows_are_checked():
    assert _linear(rows=-1) == 1 and _linear(rows=0, x=None, w=None, y=None) == 0
    size = ctypes.c_size_t(5)
    lib = dllm.load()
    assert lib.dllm_linear_workspace_size(ctypes.byref(_layer()), -1, 1, ctypes.byref(size)) == 1
    assert lib.dllm_linear_workspace_size(ctypes.byref(_layer()), 3, 1, None) == 1
    assert dllm.dllm_linear_workspace_size(_layer(), 3, False) == 0
    assert dllm.dllm_linear_workspace_size(_layer(), 3, True) == 1536
    assert dllm.dllm_linear_workspace_size(_layer(), 0, True) == 0


# ------------------------------------------------------------------ dllm_head_norm_rope
def _rows(p=A, rs=1024, hs=128, out=A + FAR, ors=1024, ohs=128, gain=None, heads=8):
    return dllm.HeadRowsC(p, rs, hs, out, ors, ohs, gain, heads)


def _rope(desc=None, rows=4, pos=A + 8 * FAR, q=None, k=None, table=A + 9 * FAR, max_pos=100, rotary=128, pairs=0, err=None):
    desc = desc or dllm.layer_desc(1024, 8, 128, 1e4)
    q = q or _rows()
    k = k or _rows(A + 2 * FAR, 256, 128, A + 3 * FAR, 256, 128, None, 2)
    return _status("dllm_head_norm_rope", desc, rows, pos, q, k, table, max_pos, rotary, pairs, err, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(pos=None), 1), (dict(pos=A + 8 * FAR + 2), 1), (dict(table=None), 1),
    (dict(table=A + 9 * FAR + 8), 1), (dict(max_pos=0), 1), (dict(rotary=32), 2), (dict(rotary=256), 2), (dict(pairs=2), 1),
    (dict(pairs=-1), 1), (dict(err=A + 1), 1), (dict(desc=dllm.layer_desc(512, 8, 64, 1e4)), 2),
    (dict(desc=dllm.layer_desc(512, 4, 128, 1e4)), 1), (dict(desc=dllm.layer_desc(960, 10, 96, 1e4)), 2)])
def test_rope_arguments_are_checked(kw, status):
    assert _rope(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(p=None), 1), (dict(p=A + 8), 1), (dict(rs=1020), 1), (dict(hs=-128), 1), (dict(out=None), 1), (dict(out=A + FAR + 2), 1),
    (dict(ors=1028), 1), (dict(gain=A + 4 * FAR + 8), 1), (dict(heads=0), 1), (dict(heads=7), 1), (dict(ors=512), 1),
    (dict(ohs=64), 1), (dict(ohs=0), 1), (dict(rs=1 << 32), 2),
    # the output over what is read: itself at other strides, a little behind, the positions, the table, the gain, the keys
    (dict(out=A, ors=2048), 1), (dict(out=A + 16), 1), (dict(out=A + 8 * FAR), 1), (dict(out=A + 9 * FAR), 1),
    (dict(out=A + 4 * FAR, gain=A + 4 * FAR), 1), (dict(out=A + 2 * FAR), 1), (dict(out=A + 3 * FAR), 1)])
def test_rope_rows_are_checked(kw, status):
    assert _rope(q=_rows(**kw)) == status


def test_rope_keys_are_checked():
    assert _rope(k=_rows(A + 2 * FAR, 256, 128, A, 256, 128, None, 2)) == 1      # over the queries' input
    assert _rope(k=_rows(A + 2 * FAR, 256, 128, A + 3 * FAR, 128, 128, None, 2)) == 1
    many = 1 << 17
    assert _rope(k=_rows(A + 2 * FAR, many * 128, 128, A + 40 * FAR, many * 128, 128, None, many)) == 2
    assert _rope(rows=0, pos=None) == 0


# ------------------------------------------------------------------ dllm_token_scores
def _scores(rows=4, vocab=1000, logits=A, kind=0, stride=1000, scale=1.0, tokens=A + FAR, logp=A + 2 * FAR, lse=None,
            entropy=None, top=2, ids=A + 3 * FAR, best=A + 4 * FAR, err=None):
    return dllm.load().dllm_token_scores(rows, vocab, logits, kind, stride, scale, tokens, logp, lse, entropy, top, ids, best,
                                         err, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(vocab=0), 1), (dict(logits=None), 1), (dict(logits=A + 1), 1), (dict(logits=A + 2, kind=1), 1),
    (dict(kind=2), 1), (dict(stride=999), 1), (dict(stride=1 << 32), 2), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(tokens=None), 1), (dict(logp=None), 1),
    (dict(tokens=A + 2), 1), (dict(logp=A + 2), 1), (dict(lse=A + 2), 1), (dict(entropy=A + 2), 1), (dict(top=-1), 1),
    (dict(top=33), 2), (dict(ids=None), 1), (dict(best=None), 1), (dict(best=A + 2), 1), (dict(err=A + 2), 1),
    (dict(vocab=(1 << 30) + 1, stride=1 << 31), 2)])
def test_score_arguments_are_checked(kw, status):
    assert _scores(**kw) == status


def test_no_rows_launch_nothing():
    assert _scores(rows=0, logits=None) == 0
    assert dllm.load().dllm_token_scores(0, 5, None, 0, 0, 1.0, None, None, None, None, 0, None, None, None, None) == 0


# ------------------------------------------------------------------ the binding
class Elsewhere(torch.Tensor):
    def get_device(self):
        return 1


class Counting:
    def __init__(self):
        self.calls = 0

    def dllm_status_string(self, status):
        return b"invalid argument"

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return dllm.DLLM_OK

        return call


@pytest.fixture
def fake(monkeypatch):
    lib = Counting()
    monkeypatch.setattr(dllm, "_lib", lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1)  # the tensors' own: the host's
    return lib


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _arrives(fake, fn, args):
    fake.calls = 0
    fn(**args, stream=0)
    assert fake.calls == 1


def _refused(fake, fn, args):
    fake.calls = 0
    with pytest.raises(dllm.DllmError, match="invalid argument"):
        fn(**args, stream=0)
    assert fake.calls == 0


def _linear_args(**kw):
    return {**dict(layer=dllm.linear_desc(64, 40), x=_bf(5, 64), w=_bf(40, 64), y=_bf(5, 40)), **kw}


def test_linear_tensors(fake):
    for kw in ({}, dict(x=_bf(5, 80)[:, 8:72]), dict(y=_bf(5, 50)[:, 3:43]), dict(residual=_bf(5, 44)[:, :40], bias=_bf(40)),
               dict(rms_gain=_bf(64), ws=torch.zeros(1024, dtype=torch.uint8)), dict(error=torch.zeros(1, dtype=torch.int32)),
               dict(layer=dllm.linear_desc(64, 20, gated=True), y=_bf(5, 20), bias=_bf(40), residual=_bf(5, 20)),
               dict(x=_bf(1, 64), y=_bf(1, 40)), dict(x=_bf(0, 64), y=_bf(0, 40))):
        _arrives(fake, dllm.dllm_linear, _linear_args(**kw))
    for kw in (dict(x=_bf(5, 72)), dict(x=_bf(5, 128)[:, ::2]), dict(x=torch.zeros(5, 64)), dict(w=_bf(41, 64)),
               dict(w=_bf(40, 80)[:, :64]), dict(w=_bf(64, 40).t()), dict(w=torch.zeros(40, 64, dtype=torch.float16)),
               dict(y=_bf(4, 40)), dict(y=_bf(5, 80)[:, ::2]), dict(y=torch.zeros(5, 40)), dict(residual=_bf(4, 40)),
               dict(residual=torch.zeros(5, 40)), dict(residual=_bf(40, 5).t()), dict(bias=_bf(39)), dict(bias=_bf(80)[::2]),
               dict(bias=torch.zeros(40)), dict(rms_gain=_bf(63)), dict(rms_gain=torch.zeros(64)),
               dict(error=torch.zeros(1, dtype=torch.int64)), dict(ws=torch.zeros(2048, dtype=torch.uint8)[::2]),
               dict(layer=dllm.linear_desc(64, 40, gated=True))):
        _refused(fake, dllm.dllm_linear, _linear_args(**kw))
    for name, t in dict(x=_bf(5, 64), w=_bf(40, 64), y=_bf(5, 40), residual=_bf(5, 40), bias=_bf(40), rms_gain=_bf(64),
                        ws=torch.zeros(1024, dtype=torch.uint8), error=torch.zeros(1, dtype=torch.int32)).items():
        _refused(fake, dllm.dllm_linear, _linear_args(**{name: t.as_subclass(Elsewhere)}))


def _rope_args(**kw):
    return {**dict(desc=dllm.layer_desc(512, 4, 128, 1e4), q=_bf(5, 4, 128), q_out=_bf(5, 4, 128), k=_bf(5, 2, 128),
                   k_out=_bf(5, 2, 128), row_pos=torch.zeros(5, dtype=torch.int32), rope_table=torch.zeros(9, 64, 2)), **kw}


def test_rope_tensors(fake):
    for kw in ({}, dict(k=None, k_out=None), dict(q=_bf(5, 9, 128)[:, 2:6]), dict(q_gain=_bf(128), k_gain=_bf(128)),
               dict(rope_table=torch.zeros(9, 32, 2)), dict(row_pos=torch.zeros(8, dtype=torch.int32)),
               dict(k=_bf(2, 5, 128).transpose(0, 1)), dict(error=torch.zeros(1, dtype=torch.int32))):
        _arrives(fake, dllm.dllm_head_norm_rope, _rope_args(**kw))
    for kw in (dict(q=_bf(5, 4, 64)), dict(q_out=_bf(5, 3, 128)), dict(q=_bf(5, 4, 256)[:, :, ::2]), dict(k=_bf(4, 2, 128), k_out=_bf(4, 2, 128)),
               dict(k_out=_bf(5, 2, 256)[:, :, ::2]), dict(q=torch.zeros(5, 4, 128)), dict(k_out=torch.zeros(5, 2, 128)),
               dict(row_pos=torch.zeros(4, dtype=torch.int32)), dict(row_pos=torch.zeros(5, dtype=torch.int64)), dict(row_pos=None),
               dict(rope_table=torch.zeros(9, 64)), dict(rope_table=torch.zeros(9, 64, 2, dtype=torch.float64)),
               dict(rope_table=torch.zeros(9, 2, 64).transpose(1, 2)), dict(q_gain=_bf(64)), dict(k_gain=torch.zeros(128)),
               dict(error=torch.zeros(1))):
        _refused(fake, dllm.dllm_head_norm_rope, _rope_args(**kw))
    for name, t in _rope_args(q_gain=_bf(128), k_gain=_bf(128), error=torch.zeros(1, dtype=torch.int32)).items():
        if name != "desc":
            _refused(fake, dllm.dllm_head_norm_rope, _rope_args(**{name: t.as_subclass(Elsewhere)}))


def _score_args(**kw):
    return {**dict(logits=_bf(5, 100), tokens=torch.zeros(5, dtype=torch.int32), logp=torch.zeros(5), lse=torch.zeros(5),
                   entropy=torch.zeros(5), top_ids=torch.zeros(5, 3, dtype=torch.int32), top_logp=torch.zeros(5, 3)), **kw}


def test_score_tensors(fake):
    for kw in ({}, dict(logits=torch.zeros(5, 120)[:, 7:100]), dict(tokens=None, logp=None), dict(top_ids=None, top_logp=None),
               dict(lse=None, entropy=None), dict(top_ids=torch.zeros(5, 0, dtype=torch.int32), top_logp=torch.zeros(5, 0))):
        _arrives(fake, dllm.dllm_token_scores, _score_args(**kw))
    for kw in (dict(logits=_bf(5, 100, 1)), dict(logits=_bf(100, 5).t()), dict(logits=torch.zeros(5, 100, dtype=torch.float16)),
               dict(tokens=None), dict(logp=None), dict(tokens=torch.zeros(5, dtype=torch.int64)), dict(tokens=torch.zeros(4, dtype=torch.int32)),
               dict(logp=_bf(5)), dict(logp=torch.zeros(4)), dict(lse=torch.zeros(10)[::2]), dict(entropy=torch.zeros(4)),
               dict(top_ids=None), dict(top_logp=None), dict(top_logp=torch.zeros(5, 4)), dict(top_ids=torch.zeros(5, 3, dtype=torch.int64)),
               dict(top_ids=torch.zeros(3, 5, dtype=torch.int32).t()), dict(error=torch.zeros(1))):
        _refused(fake, dllm.dllm_token_scores, _score_args(**kw))
    for name, t in _score_args(error=torch.zeros(1, dtype=torch.int32)).items():
        _refused(fake, dllm.dllm_token_scores, _score_args(**{name: t.as_subclass(Elsewhere)}))
