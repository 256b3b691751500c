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



def bytes_of(t):
    """The addresses that a tensor's elements take."""
    import numpy as np
    rows, cols = t.shape if t.dim() == 2 else (1, t.numel())
    at = t.data_ptr() + np.arange(rows)[:, None] * ((t.stride(0) if t.dim() == 2 else 0) * t.element_size())
    return set((at + np.arange(cols * t.element_size())[None]).ravel().tolist())


@pytest.mark.gpu
def test_outputs_that_overlap_are_refused_and_columns_of_one_buffer_are_not():
    """Arrays anywhere in one buffer, of equal or of other strides: a call is refused if and only if a byte of an output is
    one of another array too."""
    import random

    import torch
    rng = random.Random(5)
    seen = {True: 0, False: 0}
    buf = torch.zeros(1 << 14, device="cuda").bfloat16()
    for trial in range(600):
        N, K, M = rng.randrange(1, 12), rng.choice([1, 8, 24]), rng.choice([1, 8, 16])
        layer = hg.Linear(K, M)
        unit = rng.choice([32, 64, 128])

        def place(rows, cols, ld=None):
            ld = rng.choice([unit, 2 * unit, rng.randrange(cols, 80)]) if ld is None else ld
            at = 8 * rng.randrange(0, rng.choice([6, 40, 600]))
            return torch.as_strided(buf, (rows, cols), (ld, 1), at)
        x, y, w = place(N, K), place(N, M), place(M, K, K)
        r = y if rng.random() < 0.3 else place(N, M)
        z = place(N, M, M)
        in_place = r.data_ptr() == y.data_ptr() and (r.stride(0) == y.stride(0) or N == 1)
        out, ins = [y, z], [x, w] + ([] if in_place else [r])
        sets = [bytes_of(t) for t in out + ins]
        want = any(sets[i] & sets[j] for i in range(2) for j in range(i + 1, len(sets)))
        work = torch.empty(max(16, hg.hashgrid_linear_forward_workspace(layer.handle, N, x.stride(0))), dtype=torch.uint8, device="cuda")
        try:
            hg.hashgrid_linear_forward(layer.handle, x, x.stride(0), N, w, None, r, r.stride(0), y, y.stride(0), hg.HASHGRID_BF16, z, work,
                                       work.numel())
            got = False
        except hg.HashGridError as e:
            assert e.code == A and "overlap" in str(e)
            got = True
        assert got == want, (trial, N, K, M, [(t.storage_offset(), t.stride()) for t in out + ins])
        seen[want] += 1
    torch.cuda.synchronize()
    assert min(seen.values()) > 60, seen
    layer = hg.Linear(16, 16)
    x, w = torch.zeros(40, 16, device="cuda").bfloat16(), torch.zeros(16, 16, device="cuda").bfloat16()
    dy, f = torch.zeros(40, 16, device="cuda").bfloat16(), torch.zeros(2048, device="cuda")
    work = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    for bad in (dict(dL_dx=dy), dict(dL_dx=x), dict(dL_dw=f[:256].view(16, 16), dL_db=f[240:256]), dict(dL_dw=w), dict(workspace=None)):
        with pytest.raises(hg.HashGridError, match="overlap"):
            if "workspace" in bad:
                layer.backward(dy, x, w, dL_dw=work[:1024].view(torch.float32).view(16, 16), workspace=work)
            else:
                layer.backward(dy, x, w, workspace=work, **bad)
    assert layer.backward(dy, x, w, dL_dx=None, dL_dw=f[:256].view(16, 16), dL_db=f[256:272], workspace=work)[0] is None
    layer.backward(dy, dy, w, workspace=work)                    # inputs may be one another


@pytest.mark.parametrize("seed", [1 << 32, -(1 << 32), 5 << 33])
def test_seeds_that_32_bits_make_zero(seed):
    """Zero means rounding to nearest, which a caller who gave another seed did not ask for."""
    with pytest.raises(hg.HashGridError, match="seed") as e:
        hg.hashgrid_adamw_step(None, 1, 1e-3, seed=seed, stream=0)
    assert e.value.code == A
