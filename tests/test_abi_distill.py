"""Distillation and adapters without a GPU: bad arguments are rejected before any HIP
call, scratch sizes, and the binding's own refusals."""

import ctypes

import pytest

from test_abi import A8, A16, ODD, WS, WSN, lib  # noqa: F401
from top_sampling_vocabs_amd import _lib


def loss(lib, **kw):  # noqa: F811
    a = dict(logits=A16, dtype=0, B=4, V=64, stride=64, T=None, bm=None, bms=0, ids=A16,
             values=A16, K=2, rest=0, loss=A16, state=A16, status=A16, ws=WS, wsn=WSN)
    a.update(kw)
    return lib.qs_distill_loss(a["logits"], a["dtype"], a["B"], a["V"], a["stride"], a["T"],
                               a["bm"], a["bms"], a["ids"], a["values"], a["K"], a["rest"],
                               a["loss"], a["state"], a["status"], a["ws"], a["wsn"], None)


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(dtype=2), dict(B=-1), dict(B=1 << 22), dict(V=0),
    dict(V=(1 << 30) + 1, stride=1 << 31), dict(stride=60), dict(stride=65), dict(logits=ODD),
    dict(T=ODD), dict(bm=A16, bms=1), dict(bm=ODD, bms=2), dict(ids=None), dict(ids=ODD),
    dict(values=None), dict(values=ODD), dict(K=0), dict(K=-1), dict(K=1025), dict(rest=2),
    dict(rest=-1), dict(loss=None), dict(loss=ODD), dict(state=None), dict(state=ODD),
    dict(state=ctypes.c_void_p(0x100008)), dict(status=None), dict(status=ODD),
])
def test_distill_loss_rejects_bad_arguments(lib, kw):  # noqa: F811
    assert loss(lib, **kw) == _lib.QS_ERR_INVALID_ARG


def test_distill_loss_workspace(lib):  # noqa: F811
    assert loss(lib, B=0, logits=None) == _lib.QS_OK
    f = lib.qs_distill_loss_workspace_bytes
    for bad in ((0, 64, 0), (-1, 64, 0), (1 << 22, 64, 0), (4, 0, 0), (4, (1 << 30) + 1, 0),
                (4, 64, 2)):
        assert f(*bad) == 0
    for shape in ((1, 32000, 0), (256, 151936, 1), (2048, 151936, 1), (1, 1 << 30, 0),
                  ((1 << 22) - 1, 64, 1), (1, 1, 0)):
        need = f(*shape)
        assert need <= 1 << 32
        if need:
            kw = dict(B=shape[0], V=shape[1], dtype=shape[2], stride=-(-shape[1] // 8) * 8)
            assert loss(lib, **kw, wsn=need - 1) == _lib.QS_ERR_WORKSPACE
            assert loss(lib, **kw, ws=None) == _lib.QS_ERR_WORKSPACE
            assert loss(lib, **kw, ws=ctypes.c_void_p(0x400080)) == _lib.QS_ERR_WORKSPACE


@pytest.mark.parametrize("V,dtype", [(151936, 1), (65537, 1), (131073, 1), (32769, 0), (128256, 0),
                                     (1 << 20, 0), (1 << 24, 1), (1000, 1)])
def test_distill_loss_workspace_serves_smaller_batches(lib, V, dtype):  # noqa: F811
    f = lib.qs_distill_loss_workspace_bytes
    sizes = [f(B, V, dtype) for B in list(range(1, 2600)) + [4096, 1 << 16, (1 << 22) - 1]]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(dtype=3), dict(B=-1), dict(V=0), dict(stride=65), dict(ids=None),
    dict(ids=ODD), dict(values=None), dict(K=0), dict(K=1025), dict(rest=2), dict(state=None),
    dict(state=ODD), dict(state=ctypes.c_void_p(0x100008)), dict(status=None), dict(g=None), dict(g=ODD), dict(grad=None),
    dict(grad=ODD), dict(gs=60), dict(gs=65), dict(T=ODD), dict(bm=A16, bms=1),
    dict(grad=A16, gs=128),
])
def test_distill_loss_backward_rejects_bad_arguments(lib, kw):  # noqa: F811
    a = dict(logits=A16, dtype=0, B=4, V=64, stride=64, T=None, bm=None, bms=0, ids=A16,
             values=A16, K=2, rest=0, state=A16, status=A16, g=A16, grad=A8, gs=64)
    a.update(kw)
    assert lib.qs_distill_loss_backward(
        a["logits"], a["dtype"], a["B"], a["V"], a["stride"], a["T"], a["bm"], a["bms"], a["ids"],
        a["values"], a["K"], a["rest"], a["state"], a["status"], a["g"], a["grad"], a["gs"],
        None) == _lib.QS_ERR_INVALID_ARG


def adapt(lib, **kw):  # noqa: F811
    a = dict(logits=A16, dtype=0, B=4, V=64, stride=64, x=A16, K=32, xs=32, down=A16, ds=256,
             drs=32, up=A16, us=512, urs=8, count=3, rank=8, index=A16, scale=None, out=A8, os=64,
             status=A16, ws=WS, wsn=WSN)
    a.update(kw)
    return lib.qs_apply_adapters(a["logits"], a["dtype"], a["B"], a["V"], a["stride"], a["x"],
                                 a["K"], a["xs"], a["down"], a["ds"], a["drs"], a["up"], a["us"],
                                 a["urs"], a["count"], a["rank"], a["index"], a["scale"], a["out"],
                                 a["os"], a["status"], a["ws"], a["wsn"], None)


HALF = ctypes.c_void_p(0x100008)


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(logits=ODD), dict(dtype=2), dict(B=-1), dict(B=(1 << 18) + 1),
    dict(V=0), dict(V=(1 << 24) + 1, stride=1 << 25, os=1 << 25), dict(stride=60), dict(stride=65),
    dict(x=None), dict(x=HALF), dict(K=0), dict(K=36), dict(K=65544, xs=65544, drs=65544),
    dict(xs=24), dict(xs=36), dict(down=None), dict(down=HALF), dict(ds=252), dict(ds=-256),
    dict(drs=24), dict(drs=36), dict(up=None), dict(up=HALF), dict(us=4), dict(us=-512),
    dict(urs=0), dict(urs=12), dict(count=-1), dict(count=1 << 31), dict(rank=0), dict(rank=4),
    dict(rank=12, urs=16), dict(rank=136, urs=136), dict(index=None), dict(index=ODD),
    dict(scale=ODD), dict(out=None), dict(out=HALF), dict(os=60), dict(os=65),
    dict(out=A16, os=128), dict(status=None), dict(status=ODD),
])
def test_apply_adapters_rejects_bad_arguments(lib, kw):  # noqa: F811
    assert adapt(lib, **kw) == _lib.QS_ERR_INVALID_ARG


def test_adapters_workspace(lib):  # noqa: F811
    assert adapt(lib, B=0, logits=None) == _lib.QS_OK
    f = lib.qs_adapters_workspace_bytes
    for bad in ((0, 8), (-1, 8), ((1 << 18) + 1, 8), (4, 0), (4, 12), (4, 136), (4, -8)):
        assert f(*bad) == 0
    need = f(4, 8)
    assert need > 0
    assert adapt(lib, wsn=need - 1) == _lib.QS_ERR_WORKSPACE
    assert adapt(lib, ws=None) == _lib.QS_ERR_WORKSPACE
    assert adapt(lib, ws=ctypes.c_void_p(0x400080)) == _lib.QS_ERR_WORKSPACE
    for rank in range(8, 129, 8):
        sizes = [f(B, rank) for B in list(range(1, 300)) + [1 << 18]]
        assert all(a <= b for a, b in zip(sizes, sizes[1:]))


def test_names_are_loaded_on_first_use():
    import top_sampling_vocabs_amd as qs
    for name in ("distill_loss", "distill_loss_backward", "distill_loss_workspace_for",
                 "apply_adapters", "adapters_workspace_for", "token_logprobs", "sample_hidden"):
        assert callable(getattr(qs, name)), name
    with pytest.raises(AttributeError):
        qs.no_such_call


def test_host_tensors_are_refused(lib):  # noqa: F811
    torch = pytest.importorskip("torch")
    import top_sampling_vocabs_amd as qs
    lg, ids = torch.zeros(2, 64), torch.zeros(2, 4, dtype=torch.int32)
    val, g = torch.zeros(2, 4), torch.zeros(2)
    with pytest.raises(ValueError):
        qs.distill_loss(lg, ids, val)
    with pytest.raises(ValueError):
        qs.distill_loss_backward(lg, ids, val, torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32),
                                 g)
    h = torch.zeros(2, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        qs.apply_adapters(lg, h, torch.zeros(1, 8, 32, dtype=torch.bfloat16),
                          torch.zeros(1, 64, 8, dtype=torch.bfloat16),
                          torch.zeros(2, dtype=torch.int32))
