"""Router and adapter entry points: sizes, and the argument checks the host
makes before it touches a device (they need no GPU: every call here is refused
before the first CUDA call)."""
import ctypes

import pytest

import __graft_entry__

__graft_entry__.build()
import trellis_quantized_moe_gb300 as X  # noqa: E402
from trellis_quantized_moe_gb300 import binding as B  # noqa: E402

P = 1 << 20          # an aligned address that nothing dereferences
NULL, DTYPE, SHAPE, ALIGN, WORKSPACE, ROUTING = -1, -3, -4, -5, -6, -7


def test_router_sizes():
    assert X.exl3_router_workspace_bytes(1, 1) > 0
    assert X.exl3_router_workspace_bytes(1, 1025) == 0
    assert X.exl3_router_workspace_bytes(-1, 8) == 0
    assert X.exl3_router_workspace_bytes(1 << 16, 192) % 256 == 0


def test_adapter_sizes():
    assert [X.exl3_lora_h_cols(r) for r in (0, 1, 16, 17, 128, 129)] == [0, 32, 32, 64, 256, 0]
    assert X.exl3_lora_plan_bytes(0, 1) > 0
    assert X.exl3_lora_plan_bytes(5, 0) == 0 and X.exl3_lora_plan_bytes(5, 1025) == 0
    assert X.exl3_lora_workspace_bytes(7, 2, 128, 256, 8) > 0
    assert X.exl3_lora_workspace_bytes(7, 2, 130, 256, 8) == 0
    assert X.exl3_lora_workspace_bytes(7, 2, 128, 256, 129) == 0


def _rf(**kw):
    d = dict(logits=P, dt=2, M=4, E=8, k=2, renorm=0, ids=P, rw=P, rwdt=2, stats=P, valid=None,
             counts=None, loss=None, ws=None, wsb=0)
    d.update(kw)
    return B.lib().exl3_router_forward(*d.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), NULL), (dict(ids=None), NULL), (dict(rw=None), NULL),
    (dict(counts=P), NULL), (dict(loss=P), NULL), (dict(counts=P, loss=P), NULL),
    (dict(dt=3), DTYPE), (dict(rwdt=-1), DTYPE),
    (dict(M=-1), SHAPE), (dict(M=1 << 29), SHAPE),
    (dict(E=0), ROUTING), (dict(E=1025), ROUTING), (dict(k=0), ROUTING), (dict(k=9), ROUTING),
    (dict(E=64, k=33), ROUTING),
    (dict(logits=P + 8), ALIGN), (dict(ids=P + 2), ALIGN), (dict(rw=P + 2), ALIGN),
    (dict(counts=P, loss=P, ws=P + 16, wsb=1 << 20), ALIGN),
])
def test_router_forward_refuses(kw, code):
    assert _rf(**kw) == code


def _rb(**kw):
    d = dict(logits=P, dt=2, M=4, E=8, k=2, renorm=0, ids=P, stats=P, d_rw=P, rwdt=2, valid=None,
             counts=None, d_loss=None, d_logits=P)
    d.update(kw)
    return B.lib().exl3_router_backward(*d.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), NULL), (dict(ids=None), NULL), (dict(stats=None), NULL),
    (dict(d_logits=None), NULL), (dict(d_rw=None), NULL), (dict(counts=P), NULL),
    (dict(d_loss=P), NULL), (dict(dt=4), DTYPE), (dict(M=-2), SHAPE), (dict(k=9), ROUTING),
    (dict(d_logits=P + 4), ALIGN), (dict(d_rw=P + 1), ALIGN), (dict(stats=P + 4), ALIGN),
])
def test_router_backward_refuses(kw, code):
    assert _rb(**kw) == code


def test_plan_refuses():
    f = B.lib().exl3_lora_plan
    size = X.exl3_lora_plan_bytes(4, 2)
    assert f(None, 3, 4, 2, P, size, None) == NULL
    assert f(P, 3, 4, 2, None, size, None) == NULL
    assert f(P, 2, 4, 2, P, size, None) == DTYPE
    assert f(P, 3, -4, 2, P, size, None) == SHAPE
    assert f(P, 3, 4, 0, P, size, None) == SHAPE
    assert f(P, 3, 4, 2, P + 16, size, None) == ALIGN
    assert f(P, 3, 4, 2, P, size - 1, None) == WORKSPACE


def _ad(**kw):
    d = dict(A=P, B=P, rank=P, scale=P, N=2, max_rank=8, in_features=256, out_features=128)
    d.update(kw)
    return B.exl3_adapters(*d.values())


_WSB = 1 << 40


def _lf(ad=None, **kw):
    d = dict(x=P, dt=1, M=4, ad=ctypes.byref(_ad(**(ad or {}))), plan=P, pb=_WSB, base=P, y=P, h=P, ws=P, wsb=_WSB)
    d.update(kw)
    return B.lib().exl3_lora_forward(*d.values(), None)


def _lb(ad=None, grads=None, **kw):
    d = dict(dy=P, x=P, h=P, dt=1, M=4, ad=ctypes.byref(_ad(**(ad or {}))), plan=P, pb=_WSB, dxb=P, dx=P,
             g=ctypes.byref(_ad(**(grads or {}))), ws=P, wsb=_WSB)
    d.update(kw)
    return B.lib().exl3_lora_backward(*d.values(), None)


@pytest.mark.parametrize("call", [_lf, _lb])
@pytest.mark.parametrize("kw,code", [
    (dict(ad=dict(A=None)), NULL), (dict(ad=dict(B=None)), NULL), (dict(ad=dict(rank=None)), NULL),
    (dict(ad=dict(scale=None)), NULL), (dict(plan=None), NULL), (dict(ws=None), NULL),
    (dict(x=None), NULL), (dict(dt=2), DTYPE), (dict(M=-1), SHAPE), (dict(ad=dict(N=0)), SHAPE),
    (dict(ad=dict(N=1025)), SHAPE), (dict(ad=dict(max_rank=0)), SHAPE),
    (dict(ad=dict(max_rank=129)), SHAPE), (dict(ad=dict(in_features=200)), SHAPE),
    (dict(ad=dict(out_features=0)), SHAPE), (dict(M=1 << 29, ad=dict(in_features=1 << 20)), SHAPE), (dict(ad=dict(A=P + 4)), ALIGN),
    (dict(ad=dict(rank=P + 2)), ALIGN), (dict(plan=P + 16), ALIGN), (dict(ws=P + 128), ALIGN),
    (dict(x=P + 8), ALIGN), (dict(h=P + 2), ALIGN), (dict(wsb=64), WORKSPACE), (dict(pb=64), WORKSPACE),
])
def test_adapter_calls_refuse(call, kw, code):
    assert call(**kw) == code


def test_forward_and_backward_refuse_their_own():
    assert _lf(y=None) == NULL and _lf(base=P + 8) == ALIGN
    args = (P, 1, 4, None, P, _WSB, P, P, P, P, _WSB, None)
    assert B.lib().exl3_lora_forward(*args) == NULL
    assert _lb(dy=None) == NULL and _lb(h=None) == NULL and _lb(dx=None, g=None) == NULL
    assert _lb(dx=P + 2) == ALIGN
    assert _lb(grads=dict(N=3)) == SHAPE and _lb(grads=dict(in_features=128)) == SHAPE
    assert _lb(grads=dict(A=None)) == NULL


def test_binding_checks_shapes():
    torch = pytest.importorskip("torch")
    a, b = torch.zeros(4, 128), torch.zeros(4, 256)
    with pytest.raises(ValueError):
        X.DeviceAdapters([a], [b, b], [1.0])
    with pytest.raises(ValueError):
        X.DeviceAdapters([a], [b[:3]], [1.0])
    with pytest.raises(ValueError):
        X.DeviceAdapters([a], [b.half()], [1.0])
    with pytest.raises(ValueError):
        X.DeviceAdapters([], [], [])
    lg = torch.zeros(3, 8)
    with pytest.raises(ValueError):
        X.exl3_router_forward(lg, torch.zeros(3, 2, dtype=torch.int64), torch.zeros(3, 2))
    with pytest.raises(ValueError):
        X.exl3_router_forward(lg.t(), torch.zeros(8, 2, dtype=torch.int32), torch.zeros(8, 2))
    with pytest.raises(ValueError):
        X.exl3_router_forward(lg, torch.zeros(3, 2, dtype=torch.int32), torch.zeros(2, 2))
