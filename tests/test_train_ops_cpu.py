"""Argument checks of the training operators (layer norm, gradient norm and clipping, AdamW) that
the library makes on the host before any HIP call, and the binding's own."""
import ctypes
import math
import os
import re

import pytest
import torch

from fno_spectral_convolution_amd import binding as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

BAD = L.FNO_ERR_INVALID_ARGUMENT
P = 1 << 20  # an aligned address that no call gets as far as reading


def _desc(**kw):
    base = dict(dtype=0, reserved=0, batch=4, channels=8, npts=3, x_stride=24, y_stride=24,
                grad_x_stride=24, eps=1e-5)
    base.update(kw)
    d = L.fno_layer_norm_desc()
    for k, v in base.items():
        setattr(d, k, v)
    return d


def _fwd(d, x=P, gamma=P, beta=P, y=P, stats=P):
    return L._lib.fno_layer_norm_fwd(d, x, gamma, beta, y, stats, None)


def _bwd(d, x=P, gamma=P, stats=P, gy=P, gx=P, gg=P, gb=P, ws=P, ws_bytes=1 << 30):
    return L._lib.fno_layer_norm_bwd(d, x, gamma, stats, gy, gx, gg, gb, ws, ws_bytes, None)


def test_header_binding_and_library_agree():
    src = open(os.path.join(ROOT, "include", "fno_train.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(fno_[a-z0-9_]+)\s*\(", src)))
    assert names == sorted(L.TRAIN_EXPORTS)
    lib = ctypes.CDLL(L.LIB_PATH)
    for name in names:
        assert hasattr(lib, name) and hasattr(L, name), name


def test_struct_layouts():
    assert ctypes.sizeof(L.fno_layer_norm_desc) == 8 + 3 * 8 + 3 * 8 + 8
    assert ctypes.sizeof(L.fno_tensor) == 24
    assert ctypes.sizeof(L.fno_adamw_desc) == 48


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), BAD), (dict(reserved=1), BAD), (dict(batch=-1), BAD), (dict(npts=-1), BAD),
    (dict(channels=0), BAD), (dict(x_stride=-1), BAD), (dict(eps=-1e-9), BAD),
    (dict(eps=math.nan), BAD), (dict(eps=math.inf), BAD), (dict(npts=1 << 62), BAD),
    (dict(batch=1 << 50, x_stride=1 << 40), BAD),
    (dict(channels=1 << 31), L.FNO_ERR_UNSUPPORTED),
])
def test_layer_norm_descriptor_refused(kw, status):
    d = _desc(**kw)
    assert _fwd(d) == status and L.last_error_message()
    assert _bwd(d) == status
    n = ctypes.c_size_t()
    assert L._lib.fno_layer_norm_workspace_bytes(d, ctypes.byref(n)) == status


def test_layer_norm_pointers_refused():
    d = _desc()
    assert L._lib.fno_layer_norm_fwd(None, P, P, P, P, P, None) == BAD
    for kw in (dict(x=None), dict(y=None), dict(x=P + 2), dict(y=P + 1), dict(gamma=P + 2),
               dict(beta=P + 2), dict(stats=P + 1)):
        assert _fwd(d, **kw) == BAD, kw
    assert _fwd(_desc(dtype=1), x=P + 1) == BAD
    assert _fwd(_desc(y_stride=23)) == BAD            # outputs would overlap
    assert _fwd(_desc(x_stride=30)) == BAD            # in place with another stride
    for kw in (dict(x=None), dict(gy=None), dict(stats=None), dict(gx=P + 2), dict(gg=P + 2),
               dict(gb=P + 1)):
        assert _bwd(d, **kw) == BAD, kw
    big = _desc(npts=1 << 20, x_stride=8 << 20, y_stride=8 << 20, grad_x_stride=8 << 20)
    for kw in (dict(ws=None), dict(ws=P + 8), dict(ws_bytes=0)):
        assert _bwd(big, **kw) == BAD, kw
    n = ctypes.c_size_t()
    assert L._lib.fno_layer_norm_workspace_bytes(d, ctypes.byref(n)) == L.FNO_OK and n.value == 0
    assert L._lib.fno_layer_norm_workspace_bytes(big, ctypes.byref(n)) == L.FNO_OK and n.value > 0
    assert _bwd(_desc(grad_x_stride=23)) == BAD
    assert _bwd(_desc(y_stride=30)) == BAD            # grad_x is grad_y with another stride
    assert L._lib.fno_layer_norm_workspace_bytes(d, None) == BAD


def test_layer_norm_without_rows_needs_no_pointers():
    for kw in (dict(batch=0), dict(npts=0)):
        assert _fwd(_desc(**kw), None, None, None, None, None) == L.FNO_OK
        assert _bwd(_desc(**kw), None, None, None, None, None, None, None, None, 0) == L.FNO_OK


def _list(*entries):
    a = (L.fno_tensor * max(len(entries), 1))()
    for e, (data, n, dt) in zip(a, entries):
        e.data, e.elems, e.dtype, e.reserved = data, n, dt, 0
    return a


def _create(n, tensors, table=P, table_bytes=1 << 30, out=True):
    h = ctypes.c_void_p()
    return L._lib.fno_tensor_list_create(n, tensors, table, table_bytes, None,
                                         ctypes.byref(h) if out else None)


def test_tensor_lists_refused():
    odd = _list((P, 4, 0))
    odd[0].reserved = 1
    n = ctypes.c_size_t()
    for count, ts in ((-1, _list((P, 4, 0))), (1 << 40, _list((P, 4, 0))), (1, None),
                      (1, _list((None, 4, 0))), (1, _list((P + 2, 4, 0))),
                      (1, _list((P + 1, 4, 1))), (1, _list((P, -1, 0))), (1, _list((P, 4, 9))),
                      (1, _list((P, 1 << 37, 0))), (1, odd)):
        assert _create(count, ts) == BAD
        assert L._lib.fno_tensor_list_bytes(count, ts, ctypes.byref(n)) == BAD
    huge = _list(*[(P, 1 << 36, 1)] * 64)
    assert _create(64, huge) == L.FNO_ERR_UNSUPPORTED
    ok = _list((P, 4, 0), (None, 0, 2), (P + 2, 5000, 1))
    assert L._lib.fno_tensor_list_bytes(3, ok, None) == BAD
    assert L._lib.fno_tensor_list_bytes(3, ok, ctypes.byref(n)) == L.FNO_OK and n.value >= 72 + 16
    assert _create(3, ok, table=None) == BAD and _create(3, ok, table=P + 4) == BAD
    assert _create(3, ok, table_bytes=n.value - 1) == BAD
    assert _create(3, ok, out=False) == BAD
    assert L._lib.fno_tensor_list_destroy(None) == L.FNO_OK


def test_tensor_list_host_logic():
    """The whole host side of a list (checks, chunks, table) runs before its first HIP call."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the made-up addresses must not reach it")
    ok = _list((P, 4, 0), (None, 0, 2), (P + 2, 5000, 1), (P, 1 << 22, 0))
    assert _create(4, ok) == L.FNO_ERR_HIP


def test_calls_without_lists_refused():
    d = L.fno_adamw_desc(1e-3, 0.9, 0.99, 1e-8, 0.0, 1)
    assert L._lib.fno_grad_norm(None, 1.0, 1.0, P, P, 1 << 30, None) == BAD
    assert L._lib.fno_clip_grad_norm(None, None, 1.0, 1.0, P, P, 1 << 30, None) == BAD
    assert L._lib.fno_adamw(None, None, None, None, d, None, None) == BAD
    assert L._lib.fno_adamw(None, None, None, None, None, None, None) == BAD
    assert L._lib.fno_grad_norm_workspace_bytes(None, None) == BAD


@pytest.mark.parametrize("kw", [
    dict(lr=math.nan), dict(lr=math.inf), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0),
    dict(beta2=math.nan), dict(eps=-1.0), dict(eps=math.inf), dict(weight_decay=math.nan),
    dict(step=0),
])
def test_adamw_descriptor_refused(kw):
    base = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, step=1)
    base.update(kw)
    assert L._lib.fno_adamw(None, None, None, None, L.fno_adamw_desc(**base), None, None) == BAD
    assert "AdamW" in L.last_error_message()


def test_binding_refuses():
    x = torch.zeros(4, 8, 6)
    with pytest.raises(ValueError, match="GPU"):
        L.layer_norm_fwd(x)
    with pytest.raises(ValueError, match="float32"):
        L.layer_norm_fwd(x.double())
    with pytest.raises(ValueError, match="batch, channels"):
        L.layer_norm_fwd(x[0, 0])
    with pytest.raises(ValueError, match="packed"):
        L.layer_norm_fwd(x.transpose(1, 2))
    with pytest.raises(ValueError, match="float32"):
        L.layer_norm_fwd(x.to(torch.complex64))
    with pytest.raises(ValueError, match="packed"):
        L.TensorList([x.transpose(0, 1)])
    with pytest.raises(ValueError, match="GPU"):
        L.TensorList([x])
    with pytest.raises(ValueError, match="GPU"):
        L.grad_norm([x])


@pytest.mark.parametrize("ws", [
    torch.zeros(1, dtype=torch.uint8).expand(1 << 20),  # more elements than it has memory
    torch.zeros(2 << 20, dtype=torch.uint8)[::2],
], ids=["expanded", "strided"])
def test_norm_workspace_is_packed_memory_of_the_device(ws, monkeypatch):
    """The library sees an address and a size alone: whether they are memory of the device is the
    binding's to ask.  CPU tensors stand for the GPU's, and no call goes out."""
    calls = []
    monkeypatch.setattr(L, "_on_gpu", lambda x: x.get_device())
    monkeypatch.setattr(L, "_on_stream", lambda index, fn, *args: calls.append(args) or L.FNO_OK)
    x, stats = torch.zeros(2, 8, 1 << 16), torch.zeros(2, 2, 1 << 16)
    good = torch.zeros(1 << 20, dtype=torch.uint8)
    L.layer_norm_bwd(x, None, stats, x, ws=good)
    assert len(calls) == 1
    with pytest.raises(ValueError, match="ws"):
        L.layer_norm_bwd(x, None, stats, x, ws=ws)
    assert len(calls) == 1


def test_norm_workspace_on_another_device(monkeypatch):
    calls = []
    monkeypatch.setattr(L, "_on_gpu", lambda x: 0)
    monkeypatch.setattr(L, "_on_stream", lambda index, fn, *args: calls.append(args) or L.FNO_OK)
    x = torch.zeros(2, 8, 1 << 16)
    with pytest.raises(ValueError, match="ws"):
        L.layer_norm_bwd(x, None, None, x, want=("x",), ws=torch.zeros(1 << 20, dtype=torch.uint8))
    assert not calls


@pytest.mark.parametrize("kw", [
    dict(batch=1 << 40, channels=1 << 20, npts=1 << 20),
    dict(batch=1 << 31, channels=(1 << 31) - 1, npts=1),
    dict(batch=1 << 58, channels=8, npts=1),
])
def test_layer_norm_of_too_many_elements_refused(kw):
    """Strides of 0 keep every offset small: the number of elements has its own limit, 2^60."""
    d = _desc(x_stride=0, y_stride=0, grad_x_stride=0, **kw)
    n = ctypes.c_size_t()
    assert L._lib.fno_layer_norm_workspace_bytes(d, ctypes.byref(n)) == BAD
    assert _fwd(d) == BAD and _bwd(d, gx=None) == BAD
    assert "overflow" in L.last_error_message()


def test_optimiser_step_refused_during_capture(monkeypatch):
    """The step's number and learning rate go into its launches as values: a replay would repeat one
    update.  No GPU here: the calls are recorded, and the stream's answer is made up."""
    from fno_spectral_convolution_amd.optim import AdamW
    calls, capturing = [], [True]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    monkeypatch.setattr(L, "_on_stream", lambda index, fn, *args: fn(*args, 0))
    monkeypatch.setattr(L, "grad_norm", lambda *a, **k: calls.append("grad_norm"))
    monkeypatch.setattr(L, "adamw", lambda *a, **k: calls.append("adamw"))
    opt = AdamW.__new__(AdamW)
    opt.lr, opt.betas, opt.eps, opt.weight_decay, opt.max_norm = 1e-3, (0.9, 0.99), 1e-8, 0.0, 1.0
    opt._params = opt._grads = opt._m = opt._v = type("List", (), {"index": 0})()
    opt.record, opt.steps = None, 4
    with pytest.raises(RuntimeError, match="captur"):
        opt.step()
    assert not calls and opt.steps == 4
    capturing[0] = False
    opt.step()
    assert calls == ["grad_norm", "adamw"] and opt.steps == 5
