"""The strides that a norm's calls look at: a forward, and a query of both directions' workspaces, not
at grad_x's."""
import ctypes

import pytest

from fno_spectral_convolution_amd import binding as L
from tests import test_between_ops_cpu as between
from tests import test_train_ops_cpu as train

BAD = L.FNO_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("stride", [-1, 1 << 62, -(1 << 63)])
def test_forward_does_not_look_at_grad_x_stride(stride):
    # without points nothing is launched and only the descriptor is looked at
    none = dict(x=None, gamma=None, beta=None, y=None, stats=None)
    for desc, fwd, bwd in ((train._desc, train._fwd, train._bwd),
                           (between._desc, between._fwd, between._bwd)):
        assert fwd(desc(npts=0, grad_x_stride=stride), **none) == L.FNO_OK
        assert bwd(desc(grad_x_stride=stride)) == BAD
        assert "stride" in L.last_error_message() or "overflow" in L.last_error_message()
        for kw in (dict(x_stride=stride), dict(y_stride=stride)):
            assert fwd(desc(**kw)) == BAD
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    sizes = []
    for kw in (dict(grad_x_stride=stride), {}):
        d = between._desc(npts=1 << 20, x_stride=8 << 20, y_stride=8 << 20, **kw)
        assert L._lib.fno_group_norm_workspace_bytes(d, ctypes.byref(f), ctypes.byref(b)) == L.FNO_OK
        sizes.append((f.value, b.value))
    assert sizes[0] == sizes[1] and min(sizes[0]) > 0
    assert L._lib.fno_layer_norm_workspace_bytes(train._desc(grad_x_stride=stride), ctypes.byref(b)) == BAD


@pytest.mark.parametrize("last", [0, 1])
@pytest.mark.parametrize("channels", [1, 3, 64, 320])
def test_workspaces_grow_with_the_points(channels, last):
    """Up to the largest descriptor: no count in a workspace's layout wraps."""
    sizes = [(0, 0)]
    for k in range(31, 57):
        if channels << k > 1 << 56:
            break
        d = between._desc(channels=channels, groups=1, npts=1 << k, batch=1, channels_last=last,
                          x_stride=0, y_stride=0, grad_x_stride=0)
        f, b = ctypes.c_size_t(), ctypes.c_size_t()
        assert L._lib.fno_group_norm_workspace_bytes(d, ctypes.byref(f), ctypes.byref(b)) == L.FNO_OK
        assert f.value >= sizes[-1][0] and b.value >= sizes[-1][1], k
        sizes.append((f.value, b.value))
    assert len(sizes) > 15
