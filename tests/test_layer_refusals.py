"""What the layer calls refuse before anything is launched."""
import pytest

import multiresolution_hash_grid_b200 as hg

A = hg.HASHGRID_ERR_ARG
P = 0x1000


def forward(layer, x=P, ldx=8, N=2, w=P, b=None, r=None, ldr=4, y=P, ldy=4, yt=hg.HASHGRID_BF16, z=None, work=None, size=0):
    return hg.lib.hashgrid_linear_forward(layer.handle, x, ldx, N, w, b, r, ldr, y, ldy, yt, z, work, size, None, None)


def backward(layer, dy=P, lddy=4, x=P, ldx=8, N=2, w=P, z=P, dx=P, lddx=8, xt=hg.HASHGRID_F32, dw=P, wt=hg.HASHGRID_F32, db=P, work=P,
             size=1 << 20):
    return hg.lib.hashgrid_linear_backward(layer.handle, dy, lddy, x, ldx, N, w, z, dx, lddx, xt, dw, wt, db, work, size, None, None)


@pytest.mark.parametrize("N,ld", [((1 << 30) + 1, 1 << 33), ((1 << 31) - 300, (1 << 37) - 1), ((1 << 29) + 1, 1 << 34), (1 << 20, 1 << 36)])
def test_extents_beyond_64_bits(N, ld):
    """(N - 1) ld elements whose bytes pass 64 bits come out as a small extent, which any buffer would hold."""
    layer = hg.Linear(8, 4)
    assert forward(layer, N=N, ldx=ld) == A and "any memory" in hg.hashgrid_last_error()
    assert backward(layer, dw=None, db=None, N=N, lddy=ld) == A and "any memory" in hg.hashgrid_last_error()

