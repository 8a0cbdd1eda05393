"""Host-side checks of outputs that are other tensors of the same call.  One
output may stand in place of one input; every other output at the same address
comes back as a refusal, also where that pair is given.  The allowed pairs are
called with a workspace that is refused after them, or with no rows, so that
nothing is launched."""
import pytest

from mamba_ssd_chunked_02_amd import block_ops as ops
from test_abi_block import STEP, at, call, gated_shape, norm_shape
from test_abi_host import E_SHAPE, E_WS

NORM = ["x", "residual", "weight", "scale", "y", "out", "rstd"]
NORMB = ["dy", "dout", "out", "weight", "rstd", "x", "scale", "dx", "dresidual", "dweight", "dscale"]


@pytest.fixture(scope="module")
def lib():
    return ops._lib()


@pytest.mark.parametrize("other", ["y", "rstd"])
@pytest.mark.parametrize("dtype2", [0, 1])
def test_residual_norm_in_place(lib, other, dtype2):
    """out in place of the residual, and a second output there too."""
    sh = norm_shape(dtype2=dtype2)
    assert call(lib.ssd_add_rms_norm, NORM, sh, ws=False, out=at(1), **{other: at(1)}) == E_SHAPE
    for name in ("weight", "scale"):
        assert call(lib.ssd_add_rms_norm, NORM, sh, ws=False, out=at(1), **{name: at(1)}) == E_SHAPE, name
    if dtype2 == 0:  # x and the residual of two types are not one tensor
        assert call(lib.ssd_add_rms_norm, NORM, sh, ws=False, out=at(1), x=at(1)) == E_SHAPE


@pytest.mark.parametrize("pair", ["dx", "dresidual"])
def test_residual_norm_backward_in_place(lib, pair):
    """dx or dresidual in place of dout, and a second output there too."""
    for name in ("dx", "dresidual", "dweight", "dscale"):
        if name != pair:
            assert call(lib.ssd_add_rms_norm_backward, NORMB, norm_shape(), **{pair: at(1), name: at(1)}) == E_SHAPE, name
    for name in ("weight", "rstd", "scale"):
        assert call(lib.ssd_add_rms_norm_backward, NORMB, norm_shape(), **{pair: at(1), name: at(1)}) == E_SHAPE, name
    # nothing in place of anything: NULLs are no pair
    assert call(lib.ssd_add_rms_norm_backward, NORMB, norm_shape(), dout=None, dresidual=None, dweight=at(0)) == E_SHAPE


@pytest.mark.parametrize("ydtype", [0, 1])
def test_step_in_place(lib, ydtype):
    """state_out in place of the state, and y there too."""
    sh = gated_shape(ydtype=ydtype)
    assert call(lib.ssd_gated_scan_step, STEP, sh, ws=False, state_out=at(0), y=at(0)) == E_SHAPE
    for name in ("x", "r", "i", "lam"):
        assert call(lib.ssd_gated_scan_step, STEP, sh, ws=False, state_out=at(0), **{name: at(0)}) == E_SHAPE, name


def test_allowed_pairs_pass(lib):
    """They get as far as the workspace's size, or have no rows to work on."""
    for kw in (dict(dx=at(1)), dict(dresidual=at(1)), dict(dx=at(1), dy=at(1)), dict(dresidual=at(1), dy=at(1)),
               dict(dx=at(1), x=at(1)), dict(dresidual=at(1), out=at(1))):
        assert call(lib.ssd_add_rms_norm_backward, NORMB, norm_shape(), size=8, **kw) == E_WS, kw
    assert call(lib.ssd_add_rms_norm_backward, NORMB, norm_shape(dtype2=0), size=8, dresidual=at(1)) == E_WS
    none = norm_shape(rows=0)
    assert call(lib.ssd_add_rms_norm, NORM, none, ws=False, out=at(1)) == 0
    assert call(lib.ssd_add_rms_norm, NORM, none, ws=False, out=at(1), x=at(1)) == 0
    assert call(lib.ssd_gated_scan_step, STEP, gated_shape(batch=0), ws=False, state_out=at(0)) == 0
