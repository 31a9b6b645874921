"""Argument checks of the operators between blocks (group norm, dropout) that the library makes on the
host before any HIP call, and the binding's own; the mask's generator against its published answers."""
import ctypes
import math

import pytest
import torch

from fno_spectral_convolution_amd import binding as L
from tests.test_gpu_between_ops import _factor, _philox

BAD = L.FNO_ERR_INVALID_ARGUMENT
P = 1 << 20  # an aligned address that no call gets as far as reading
Q = 1 << 21


def _fill(d, base, kw):
    base.update(kw)
    for k, v in base.items():
        setattr(d, k, v)
    return d


def _desc(**kw):
    return _fill(L.fno_group_norm_desc(), dict(
        dtype=0, channels_last=0, activation=1, reserved=0, batch=4, channels=8, groups=2, npts=3,
        x_stride=24, y_stride=24, grad_x_stride=24, eps=1e-5), kw)


def _ddesc(**kw):
    return _fill(L.fno_dropout_desc(), dict(dtype=0, reserved=0, batch=4, elems=24, x_stride=24,
                                            residual_stride=24, y_stride=24), kw)


def _drop(**kw):
    return _fill(L.fno_dropout(), dict(p=0.5, seed=1, draw=2, counter=None), kw)


def _fwd(d, drop=None, x=P, gamma=P, beta=P, y=Q, stats=P, ws=P, ws_bytes=1 << 40):
    return L._lib.fno_group_norm_fwd(d, drop, x, gamma, beta, y, stats, ws, ws_bytes, None)


def _bwd(d, drop=None, x=P, gamma=P, beta=P, stats=P, gy=P, gx=Q, gg=P, gb=P, ws=P,
         ws_bytes=1 << 40):
    return L._lib.fno_group_norm_bwd(d, drop, x, gamma, beta, stats, gy, gx, gg, gb, ws, ws_bytes, None)


def test_struct_layouts():
    assert ctypes.sizeof(L.fno_group_norm_desc) == 16 + 7 * 8 + 8
    assert ctypes.sizeof(L.fno_dropout) == 32
    assert ctypes.sizeof(L.fno_dropout_desc) == 8 + 5 * 8


@pytest.mark.parametrize("ctr,key,want", [
    ((0, 0), 0, (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    (((1 << 64) - 1, (1 << 64) - 1), (1 << 64) - 1, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x85a308d3243f6a88, 0x0370734413198a2e), 0x299f31d0a4093822,
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_philox_known_answers(ctr, key, want):
    """The tests' own generator gives the published answers of Philox4x32-10."""
    block, draw = ctr
    signed = block - (1 << 64) if block >> 63 else block
    # _philox takes block as int64: its high word by an arithmetic shift, masked here as there
    t = torch.tensor([signed], dtype=torch.int64)
    a = _philox_words(t, draw, key)
    assert a == list(want)


def _philox_words(t, draw, key):
    lo, hi = t & 0xffffffff, (t >> 32) & 0xffffffff
    if int(hi) < 1 << 31:
        return _philox(t, draw, key)[0].tolist()
    # beyond what an int64 index reaches: the same rounds on split words
    a, b, c, d = int(lo), int(hi), draw & 0xffffffff, draw >> 32
    k0, k1 = key & 0xffffffff, key >> 32
    for _ in range(10):
        p, q = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = (q >> 32) ^ b ^ k0, q & 0xffffffff, (p >> 32) ^ d ^ k1, p & 0xffffffff
        k0, k1 = (k0 + 0x9E3779B9) & 0xffffffff, (k1 + 0xBB67AE85) & 0xffffffff
    return [a, b, c, d]


def test_mask_positions():
    """Element i's bits do not depend on where a range of elements starts."""
    f = _factor((100,), 0.5, 3, 1, device="cpu")
    for first in (1, 7, 8, 33):
        assert torch.equal(_factor((50,), 0.5, 3, 1, first, "cpu"), f[first:first + 50])


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), BAD), (dict(reserved=1), BAD), (dict(channels_last=2), BAD),
    (dict(activation=3), BAD), (dict(activation=-1), BAD), (dict(batch=-1), BAD), (dict(npts=-1), BAD),
    (dict(channels=0), BAD), (dict(groups=0), BAD), (dict(groups=3), BAD), (dict(groups=16), BAD),
    (dict(x_stride=-1), BAD), (dict(eps=-1e-9), BAD), (dict(eps=math.nan), BAD),
    (dict(eps=math.inf), BAD), (dict(npts=1 << 62), BAD), (dict(batch=1 << 30, x_stride=1 << 40), BAD),
    (dict(batch=1 << 30, channels=1 << 20, npts=1 << 20, x_stride=0, y_stride=0), BAD),
    (dict(batch=1 << 29, channels=1 << 28, npts=1, x_stride=0, y_stride=0, grad_x_stride=0), BAD),
    (dict(channels=1 << 30), L.FNO_ERR_UNSUPPORTED), (dict(batch=1 << 31), L.FNO_ERR_UNSUPPORTED),
])
def test_group_norm_descriptor_refused(kw, status):
    d = _desc(**kw)
    assert _fwd(d) == status and L.last_error_message()
    assert _bwd(d) == status
    n = ctypes.c_size_t()
    assert L._lib.fno_group_norm_workspace_bytes(d, ctypes.byref(n), None) == status


@pytest.mark.parametrize("last", [0, 1])
def test_group_norm_pointers_refused(last):
    d = _desc(channels_last=last)
    assert L._lib.fno_group_norm_fwd(None, None, P, P, P, Q, P, P, 1 << 40, None) == BAD
    for kw in (dict(x=None), dict(y=None), dict(x=P + 2), dict(y=P + 1), dict(gamma=P + 2),
               dict(beta=P + 2), dict(stats=P + 1)):
        assert _fwd(d, **kw) == BAD, kw
    assert _fwd(_desc(dtype=1, channels_last=last), x=P + 1) == BAD
    assert _fwd(_desc(y_stride=23, channels_last=last)) == BAD    # outputs would overlap
    assert _fwd(_desc(x_stride=30, channels_last=last), y=P) == BAD  # in place, another stride
    for kw in (dict(x=None), dict(gy=None), dict(stats=None), dict(gx=P + 2), dict(gg=P + 2),
               dict(gb=P + 1)):
        assert _bwd(d, **kw) == BAD, kw
    big = _desc(npts=1 << 20, x_stride=8 << 20, y_stride=8 << 20, grad_x_stride=8 << 20,
                channels_last=last)
    for kw in (dict(ws=None), dict(ws=P + 8), dict(ws_bytes=0)):
        assert _fwd(big, **kw) == BAD and _bwd(big, **kw) == BAD, kw
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert L._lib.fno_group_norm_workspace_bytes(big, ctypes.byref(f), ctypes.byref(b)) == L.FNO_OK
    assert f.value > 0 and b.value > 0
    assert L._lib.fno_group_norm_workspace_bytes(big, None, None) == L.FNO_OK
    assert _bwd(_desc(grad_x_stride=23, channels_last=last)) == BAD
    assert _bwd(_desc(y_stride=30, channels_last=last), gx=P, gy=P, x=Q) == BAD


@pytest.mark.parametrize("kw", [dict(p=-0.1), dict(p=1.0), dict(p=1 - 2.0 ** -18), dict(p=math.nan),
                                dict(p=2.0), dict(counter=P + 4)])
def test_dropout_refused(kw):
    drop = _drop(**kw)
    assert _fwd(_desc(), drop) == BAD and "dropout" in L.last_error_message()
    assert _bwd(_desc(), drop) == BAD
    assert L._lib.fno_dropout_fwd(_ddesc(), drop, P, P, Q, None) == BAD
    assert L._lib.fno_dropout_bwd(_ddesc(), drop, P, Q, None) == BAD


@pytest.mark.parametrize("kw", [dict(dtype=5), dict(reserved=1), dict(batch=-1), dict(elems=-1),
                                dict(x_stride=-1), dict(residual_stride=-1), dict(y_stride=-1),
                                dict(y_stride=23), dict(elems=1 << 62), dict(batch=1 << 40, x_stride=1 << 40)])
def test_dropout_descriptor_refused(kw):
    assert L._lib.fno_dropout_fwd(_ddesc(**kw), _drop(), P, P, Q, None) == BAD
    assert L._lib.fno_dropout_bwd(_ddesc(**kw), _drop(), P, Q, None) == BAD


def test_dropout_pointers_refused():
    d, drop = _ddesc(), _drop()
    assert L._lib.fno_dropout_fwd(None, drop, P, P, Q, None) == BAD
    assert L._lib.fno_dropout_fwd(d, None, P, P, Q, None) == BAD
    for x, r, y in ((None, P, Q), (P, P, None), (P + 2, P, Q), (P, P + 1, Q), (P, P, Q + 3)):
        assert L._lib.fno_dropout_fwd(d, drop, x, r, y, None) == BAD
    assert L._lib.fno_dropout_fwd(_ddesc(x_stride=30), drop, P, Q, P, None) == BAD
    assert L._lib.fno_dropout_fwd(_ddesc(residual_stride=30), drop, Q, P, P, None) == BAD
    assert L._lib.fno_dropout_bwd(_ddesc(x_stride=30), drop, P, P, None) == BAD


@pytest.mark.parametrize("last", [0, 1])
@pytest.mark.parametrize("kw", [
    dict(batch=1 << 26, channels=(1 << 30) - 1, npts=1), dict(batch=1, channels=(1 << 30) - 2, npts=1),
    dict(batch=(1 << 31) - 1, channels=16, npts=1 << 21), dict(batch=1, channels=1, npts=1 << 56),
    dict(batch=3, channels=(1 << 30) - 4, npts=1 << 24), dict(batch=1, channels=1 << 26, npts=1 << 30),
    dict(batch=(1 << 31) - 1, channels=1, npts=2),
], ids=str)
@pytest.mark.parametrize("groups", [1, "all"])
def test_workspaces_of_the_largest_descriptors(kw, last, groups):
    """Sizes at the limits: the workspaces' layout stays within 64 bits (the sanitizers look on)."""
    for dtype in (0, 1):
        d = _desc(dtype=dtype, channels_last=last, groups=kw["channels"] if groups == "all" else 1,
                  x_stride=0, y_stride=0, grad_x_stride=0, **kw)
        f, b = ctypes.c_size_t(), ctypes.c_size_t()
        assert L._lib.fno_group_norm_workspace_bytes(d, ctypes.byref(f), ctypes.byref(b)) == L.FNO_OK
        assert f.value < 1 << 62 and b.value < 1 << 62


def test_without_elements_no_pointers_are_needed():
    drop = _drop()
    for kw in (dict(batch=0), dict(npts=0)):
        d = _desc(**kw)
        assert L._lib.fno_group_norm_fwd(d, None, None, None, None, None, None, None, 0, None) == L.FNO_OK
        assert _bwd(d, None, None, None, None, None, None, None, None, None, None, 0) == L.FNO_OK
    for kw in (dict(batch=0), dict(elems=0)):
        assert L._lib.fno_dropout_fwd(_ddesc(**kw), drop, None, None, None, None) == L.FNO_OK


def test_binding_refuses():
    x = torch.zeros(4, 8, 6)
    drop = L.Dropout(0.5, 1)
    with pytest.raises(ValueError, match="GPU"):
        L.group_norm_fwd(x, 2)
    with pytest.raises(ValueError, match="float32"):
        L.group_norm_fwd(x.double(), 2)
    with pytest.raises(ValueError, match="batch, channels"):
        L.group_norm_fwd(x[0, 0], 2)
    with pytest.raises(ValueError, match="packed"):
        L.group_norm_fwd(x.transpose(1, 2), 2)
    with pytest.raises(ValueError, match="act"):
        L.group_norm_fwd(x, 2, act="tanh")
    with pytest.raises(L.FnoError, match="groups"):
        L.group_norm_fwd(x, 5)
    with pytest.raises(ValueError, match="GPU"):
        L.dropout_fwd(x, drop)
    with pytest.raises(ValueError, match="packed"):
        L.dropout_bwd(x.transpose(1, 2), drop)
    with pytest.raises(ValueError, match="float32"):
        L.dropout_fwd(x.double(), drop)
    with pytest.raises(ValueError, match="batch"):
        L.dropout_fwd(x[0, 0, 0], drop)
    for p in (-0.1, 1.0, math.nan, 1 - 2.0 ** -18):
        with pytest.raises(ValueError, match="p must"):
            L.Dropout(p, 1)
    for kw in (dict(seed=-1), dict(seed=1 << 64), dict(seed=1, draw=-1), dict(seed=1, draw=1 << 64)):
        with pytest.raises(ValueError, match="2\\^64"):
            L.Dropout(0.5, **kw)
    with pytest.raises(ValueError, match="GPU"):
        L.Dropout(0.5, 1, counter=torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="int64"):
        L.Dropout(0.5, 1, counter=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="int64"):
        L.Dropout(0.5, 1, counter=torch.zeros(1))


@pytest.mark.parametrize("p", [math.inf, -math.inf, math.nan, -0.1, 1.0, 1 - 2.0 ** -18, 2.0])
def test_probabilities_that_are_none(p):
    with pytest.raises(ValueError, match="p must be in"):
        L.Dropout(p, 1)
