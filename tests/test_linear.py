"""Linear layers (hashgrid_linear_*) against a plain computation in 64 bits, and their refusals.

Tolerances, per element, u = 2^-24 and e = eps / 2 of the 16-bit type (the largest relative error
of one rounding; its subnormals are absolute, 2^-25 for fp16):
  a sum of K exact products in fp32, in any order and with additions that may truncate (2u each):
      S = 2u (K + 2) sum |products|;
  z: S + 2u |z| (the bias), then one rounding to 16 bits, e |z|;
  y: an activation's slope is at most 1.13, its own evaluation is off by at most 16u (|z| + 1),
      the residual's addition by 2u |y|, the rounding by e |y|;
  dz: the slope is off by at most 32u (1 + |z|), the rounding by e |dz|; what that makes of dx and dw
      is the same sum over these errors, to which the sum's own S and the output's rounding come;
  db: sums unrounded dz.
"""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import multiresolution_hash_grid_b200 as hg

U = 2.0 ** -24
TYPES = {hg.HASHGRID_F16: torch.float16, hg.HASHGRID_BF16: torch.bfloat16}
ACTS = [hg.HASHGRID_ACT_NONE, hg.HASHGRID_ACT_RELU, hg.HASHGRID_ACT_GELU, hg.HASHGRID_ACT_SILU]


def act64(z, act):
    if act == hg.HASHGRID_ACT_RELU:
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == hg.HASHGRID_ACT_GELU:
        return 0.5 * z * torch.special.erfc(-z / 2 ** 0.5)
    return z * torch.sigmoid(z) if act == hg.HASHGRID_ACT_SILU else z


def slope64(z, act):
    if act == hg.HASHGRID_ACT_RELU:
        return (z > 0).double()
    if act == hg.HASHGRID_ACT_GELU:
        return 0.5 * torch.special.erfc(-z / 2 ** 0.5) + z * torch.exp(-z * z / 2) / (2 * np.pi) ** 0.5
    if act == hg.HASHGRID_ACT_SILU:
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def half_step(dtype):
    """(relative, absolute) error of one rounding."""
    return {torch.float16: (2.0 ** -11, 2.0 ** -25), torch.bfloat16: (2.0 ** -8, 0.0), torch.float32: (U, 0.0)}[dtype]


def rows_of(n, width, pad, dtype, gen, scale=1.0, fill=float("nan")):
    """[n, width] values, rows width + pad apart, with `fill` between them."""
    full = torch.full((n, width + pad), fill, device="cuda", dtype=dtype)
    full[:, :width] = (torch.randn(n, width, device="cuda", generator=gen) * scale).to(dtype)
    return full[:, :width]


def close(got, want, tol, what):
    bad = ((got.double() - want).abs() > tol) | ~torch.isfinite(got.double())
    if bool(bad.any()):
        i = int(bad.flatten().nonzero()[0])
        d = (got.double() - want).abs()
        raise AssertionError(f"{what}: {int(bad.sum())} of {got.numel()} values off, first at {i}: {got.flatten()[i].item()} "
                             f"against {want.flatten()[i].item()}, tolerance {tol.flatten()[i].item()}; largest {d.max().item()}")


def check_forward(N, K, M, dtype, act, bias=True, residual=True, keep=True, y32=False, pad=0, seed=0):
    t = TYPES[dtype]
    gen = torch.Generator(device="cuda").manual_seed(1000 + seed)
    yt = torch.float32 if y32 else t
    x = rows_of(N, K, pad, t, gen)
    w = (torch.randn(M, K, device="cuda", generator=gen) / K ** 0.5).to(t)
    b = torch.randn(M, device="cuda", generator=gen) if bias else None
    r = rows_of(N, M, pad, yt, gen) if residual else None
    ybuf = torch.full((N + 40, M + pad), 7.0, device="cuda", dtype=yt)      # rows behind the last one stay too
    zbuf = torch.full((N * M + 64,), 7.0, device="cuda", dtype=t)
    z = zbuf[:N * M].view(N, M) if keep else None
    layer = hg.Linear(K, M, dtype, act)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    need = hg.hashgrid_linear_forward_workspace(layer.handle, N, K + pad if N > 1 else K)
    work = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN, whatever is read from it
    layer.forward(x, w, b, residual=r, y=ybuf[:N, :M], z=z, workspace=work[:max(16, need)], device_status=status)
    torch.cuda.synchronize()
    assert int(status[0]) == 0
    assert bool((work[need:] == 0xFF).all())
    assert bool((ybuf[:, M:] == 7.0).all()) and bool((ybuf[N:] == 7.0).all()) and bool((zbuf[N * M:] == 7.0).all())
    X, W = x.double(), w.double()
    z64 = X @ W.t() + (b.double() if bias else 0)
    S = 2 * U * (K + 2) * (X.abs() @ W.abs().t()) + 2 * U * z64.abs()
    a64 = act64(z64, act)
    y64 = a64 + (r.double() if residual else 0)
    e, absolute = half_step(yt)
    close(ybuf[:N, :M], y64, 1.13 * S + 16 * U * (z64.abs() + 1) + 2 * U * y64.abs() + e * y64.abs() * 1.01 + absolute, "y")
    if keep:
        e, absolute = half_step(t)
        close(z, z64, S + e * (z64.abs() + S) + absolute, "z")


def check_backward(N, K, M, dtype, act, dx32=False, dw32=True, pad=0, seed=0, want=(True, True, True)):
    t = TYPES[dtype]
    gen = torch.Generator(device="cuda").manual_seed(2000 + seed)
    x = rows_of(N, K, pad, t, gen)
    w = (torch.randn(M, K, device="cuda", generator=gen) / M ** 0.5).to(t)
    dy = rows_of(N, M, pad, t, gen)
    z = torch.randn(N, M, device="cuda", generator=gen).to(t)
    z[::3, ::2] = 0.0                        # the kink itself: relu's slope there is 0
    xt, wt = torch.float32 if dx32 else t, torch.float32 if dw32 else t
    dxbuf = torch.full((N + 40, K + pad), 7.0, device="cuda", dtype=xt)
    dw = torch.full((M, K), 7.0, device="cuda", dtype=wt)
    db = torch.full((M,), 7.0, device="cuda")
    layer = hg.Linear(K, M, dtype, act)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    need = hg.hashgrid_linear_backward_workspace(layer.handle, N, M + pad if N > 1 else M, K + pad if N > 1 else K)
    work = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN, whatever is read from it
    layer.backward(dy, x, w, z=None if act == hg.HASHGRID_ACT_NONE else z, dL_dx=dxbuf[:N, :K] if want[0] else None,
                   dL_dw=dw if want[1] else None, dL_db=db if want[2] else None, workspace=work[:max(16, need)],
                   device_status=status)
    torch.cuda.synchronize()
    assert int(status[0]) == 0
    assert bool((work[need:] == 0xFF).all()) and bool((dxbuf[:, K:] == 7.0).all()) and bool((dxbuf[N:] == 7.0).all())
    X, W, DY, Z = x.double(), w.double(), dy.double(), z.double()
    dz = DY * slope64(Z, act)
    e, absolute = half_step(t)
    smooth = act in (hg.HASHGRID_ACT_GELU, hg.HASHGRID_ACT_SILU)
    raw = (32 * U * (1 + Z.abs()) * DY.abs()) if smooth else torch.zeros_like(dz)
    err = raw + (e * dz.abs() * 1.01 + absolute) if smooth else raw
    for on, got, ref, mag, carried, terms, name in (
            (want[0], dxbuf[:N, :K], dz @ W, dz.abs() @ W.abs(), err @ W.abs(), M, "dx"),
            (want[1], dw, dz.t() @ X, dz.abs().t() @ X.abs(), err.t() @ X.abs(), N, "dw"),
            (want[2], db, dz.sum(0), dz.abs().sum(0), raw.sum(0), N, "db")):
        if not on:
            assert bool((got == 7.0).all()), name
            continue
        eo, ao = half_step(got.dtype)
        close(got, ref, 2 * U * (terms + 2) * mag + carried * 1.01 + eo * ref.abs() * 1.01 + ao, name)
        # a typical error is far below the worst case: a sum of independent errors grows by its root
        rel = float((got.double() - ref).norm() / ref.norm().clamp(min=1e-300))
        assert rel <= 2 * (eo + (e if smooth and name != "db" else 0)) + 2e-5, (name, rel)


SHAPES = [(1, 1, 1), (1, 64, 64), (2, 5, 3), (7, 33, 9), (16, 256, 200), (127, 64, 64), (128, 16, 16), (129, 64, 128),
          (130, 65, 129), (300, 1, 257), (257, 300, 1), (33, 520, 264), (1000, 32, 64), (513, 136, 72), (64, 1024, 512)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [hg.HASHGRID_F16, hg.HASHGRID_BF16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_shapes(shape, dtype):
    N, K, M = shape
    for i, act in enumerate(ACTS):
        check_forward(N, K, M, dtype, act, bias=i != 1, residual=i != 2, keep=i != 3, y32=i == 3, pad=(0, 8, 3, 1)[i], seed=i)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [hg.HASHGRID_F16, hg.HASHGRID_BF16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward_shapes(shape, dtype):
    N, K, M = shape
    for i, act in enumerate(ACTS):
        check_backward(N, K, M, dtype, act, dx32=i == 1, dw32=i != 2, pad=(0, 8, 3, 1)[i], seed=i)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
def test_aligned_sizes_with_every_output_type(act):
    for y32 in (False, True):
        check_forward(640, 192, 320, hg.HASHGRID_BF16, act, y32=y32, pad=0)
        check_backward(640, 192, 320, hg.HASHGRID_BF16, act, dx32=y32, dw32=not y32, pad=16)


@pytest.mark.gpu
@pytest.mark.parametrize("want", [(True, False, False), (False, True, False), (False, False, True), (True, False, True)])
@pytest.mark.parametrize("act", [hg.HASHGRID_ACT_NONE, hg.HASHGRID_ACT_SILU])
def test_gradients_that_are_left_out(want, act):
    check_backward(200, 48, 72, hg.HASHGRID_BF16, act, want=want)


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,M", [(70001, 32, 64), (50000, 64, 4), (40003, 27, 31), (3000, 1024, 768)])
def test_many_rows(N, K, M):
    check_forward(N, K, M, hg.HASHGRID_BF16, hg.HASHGRID_ACT_RELU, residual=False)
    check_backward(N, K, M, hg.HASHGRID_BF16, hg.HASHGRID_ACT_RELU)


@pytest.mark.gpu
@pytest.mark.parametrize("K,M", [(64, 64), (32, 64), (64, 8), (8, 128), (128, 64), (128, 128), (24, 40), (104, 72), (27, 31), (1, 2), (61, 128),
                                 (128, 5), (65, 66)])
def test_narrow_layers_over_many_rows(K, M):
    """Layers whose backward pass is one kernel; 128 tiles a block and a ragged last one, and three to five a block."""
    for i, (N, act) in enumerate([(4 * 148 * 128 + 77, hg.HASHGRID_ACT_RELU), (600 * 148 + 1, hg.HASHGRID_ACT_NONE),
                                  (1300 * 148 + 128, hg.HASHGRID_ACT_SILU), (90001, hg.HASHGRID_ACT_GELU)]):
        check_backward(N, K, M, hg.HASHGRID_BF16 if i else hg.HASHGRID_F16, act, dx32=i == 1, dw32=i != 2, pad=(0, 8, 24, 3)[i],
                       want=(i != 3, True, i != 2))


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,M", [(19100, 512, 160), (9700, 520, 300), (9601, 1000, 417), (19001, 777, 224), (5000, 1600, 1030)])
def test_wide_products(N, K, M):
    """256-row tiles of every width, even and odd, with 16- and 32-bit results."""
    check_forward(N, K, M, hg.HASHGRID_BF16, hg.HASHGRID_ACT_SILU, pad=8)
    check_forward(N, K, M, hg.HASHGRID_F16, hg.HASHGRID_ACT_NONE, residual=False, y32=True)
    check_backward(N, M, K, hg.HASHGRID_BF16, hg.HASHGRID_ACT_NONE, dx32=True)
    check_backward(N, K, M, hg.HASHGRID_BF16, hg.HASHGRID_ACT_GELU, dw32=False, pad=8)


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,M", [(2865, 12, 1), (3000, 588, 1), (3000, 20, 1), (1, 12, 1), (2900, 588, 2)])
def test_one_output_over_many_rows(N, K, M):
    """A weight gradient of one row, summed in parts that follow one another without a gap."""
    check_backward(N, K, M, hg.HASHGRID_F16, hg.HASHGRID_ACT_RELU)
    check_backward(N, K, M, hg.HASHGRID_BF16, hg.HASHGRID_ACT_NONE, dw32=False, want=(False, True, False))


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,M", [(40000, 128, 128), (40000, 64, 64), (40000, 200, 40)])
def test_many_rows_with_fp32_results_and_kept_z(N, K, M):
    """The second staging area leaves less shared memory to weights that stay there."""
    check_forward(N, K, M, hg.HASHGRID_BF16, hg.HASHGRID_ACT_SILU, y32=True)
    check_forward(N, K, M, hg.HASHGRID_F16, hg.HASHGRID_ACT_RELU, y32=True, residual=False)


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,M", [(4096, 4096, 2048), (300, 8200, 264), (64, 30000, 72), (40, 5000, 37)])
def test_long_sums_in_fp32(N, K, M):
    """fp32 results of sums over thousands of terms: the tensor cores' truncating additions alone would be off by 1e-9 a
    term. With sums of 1024 terms added in fp32, an addition rounding by at most 2^-24, the bias is that of 1024 terms,
    1.1e-6, and the additions add less than 2^-24 times their number's root."""
    gen = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn(N, K, device="cuda", generator=gen).bfloat16()
    w = torch.randn(M, K, device="cuda", generator=gen).bfloat16()
    ref = x.double() @ w.double().t()
    y = hg.Linear(K, M).forward(x, w, y=torch.empty(N, M, device="cuda"))
    bound = 1.1e-6 * 1.2 + U * (K / 1024) ** 0.5
    assert float((y.double() - ref).norm() / ref.norm()) < bound
    # the same product as a weight gradient (rows K) and as an input gradient
    _, dw, _ = hg.Linear(M, N).backward(x.t().contiguous(), w.t().contiguous(), torch.zeros(N, M, device="cuda").bfloat16(), dL_dx=None)
    assert float((dw.double() - ref).norm() / ref.norm()) < bound
    dx, _, _ = hg.Linear(M, K).backward(x, torch.zeros(N, M, device="cuda").bfloat16(), w.t().contiguous(), dL_dw=None, dL_db=None,
                                        dL_dx=torch.empty(N, M, device="cuda"))
    assert float((dx.double() - ref).norm() / ref.norm()) < bound


@pytest.mark.gpu
def test_no_rows():
    layer = hg.Linear(32, 48, hg.HASHGRID_F16, hg.HASHGRID_ACT_GELU)
    x = torch.empty(0, 32, device="cuda", dtype=torch.float16)
    w = torch.randn(48, 32, device="cuda").half()
    assert layer.forward(x, w).shape == (0, 48)
    dx, dw, db = layer.backward(torch.empty(0, 48, device="cuda", dtype=torch.float16), x, w,
                                dL_dw=torch.full((48, 32), 3.0, device="cuda"), dL_db=torch.full((48,), 3.0, device="cuda"))
    assert dx.shape == (0, 32) and int(dw.count_nonzero()) == 0 and int(db.count_nonzero()) == 0


@pytest.mark.gpu
def test_values_that_are_not_finite_stay_in_their_rows():
    """An infinity or a NaN in one row of x reaches that row of y (and, in the backward pass, the columns of dw that
    it belongs to) and nothing else."""
    layer = hg.Linear(40, 24, hg.HASHGRID_BF16)
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(200, 40, device="cuda", generator=gen).bfloat16()
    w = torch.randn(24, 40, device="cuda", generator=gen).bfloat16()
    clean = layer.forward(x, w)
    x2 = x.clone()
    x2[3, 7], x2[150, 0] = float("inf"), float("nan")
    y = layer.forward(x2, w)
    keep = torch.ones(200, dtype=torch.bool, device="cuda")
    keep[[3, 150]] = False
    assert torch.equal(y[keep], clean[keep]) and not bool(torch.isfinite(y[~keep].float()).any())
    dy = torch.randn(200, 24, device="cuda", generator=gen).bfloat16()
    _, dw0, _ = layer.backward(dy, x, w)
    _, dw1, _ = layer.backward(dy, x2, w)
    cols = torch.ones(40, dtype=torch.bool, device="cuda")
    cols[[0, 7]] = False
    assert torch.equal(dw0[:, cols], dw1[:, cols]) and not bool(torch.isfinite(dw1[:, ~cols]).any())


@pytest.mark.gpu
@pytest.mark.parametrize("act", [hg.HASHGRID_ACT_RELU, hg.HASHGRID_ACT_GELU, hg.HASHGRID_ACT_SILU])
@pytest.mark.parametrize("N", [40, 9000])
def test_gradients_at_the_ends_of_the_range(act, N):
    """z at and beyond what 16 bits hold: the slope is 1 above, 0 below; a NaN stays in its row (relu's slope there is 0)."""
    z = torch.zeros(N, 16, device="cuda", dtype=torch.float16)
    z[:, 0], z[:, 1], z[:, 2], z[:, 3] = 65504.0, -65504.0, float("inf"), float("-inf")
    z[3, 4] = float("nan")
    dy = torch.ones_like(z)
    x, w = torch.ones(N, 8, device="cuda").half(), torch.eye(16, 8, device="cuda").half()
    dx, dw, db = hg.Linear(8, 16, hg.HASHGRID_F16, act).backward(dy, x, w, z=z)
    want = torch.tensor([1.0, 0.0, 1.0, 0.0], device="cuda")
    # z enters the slope as at most 80 in size, where silu's is 80 exp(-80) = 1.4e-33 off at most
    assert torch.equal(dx[0, :4].float(), want) and float((db[:4] - want * N).abs().max()) <= 1.5e-33 * N
    assert torch.equal(dw[:4], (want * N)[:, None].expand(4, 8))      # of the rounded dz
    nan = act != hg.HASHGRID_ACT_RELU
    assert bool(torch.isnan(dx[3, 4])) == nan and bool(torch.isnan(db[4])) == nan and not bool(torch.isnan(db[5:]).any())
    assert not bool(torch.isnan(dx[:3]).any()) and not bool(torch.isnan(dx[4:]).any())


@pytest.mark.gpu
def test_one_row_with_any_stride():
    """A single row's stride means nothing: a large or an odd one is taken all the same."""
    layer = hg.Linear(24, 40)
    gen = torch.Generator(device="cuda").manual_seed(12)
    x, w = torch.randn(1, 24, device="cuda", generator=gen).bfloat16(), torch.randn(40, 24, device="cuda", generator=gen).bfloat16()
    want = layer.forward(x, w)
    for ld in (24, 41, 1 << 20, (1 << 36) + 1, 1 << 45):
        y = torch.zeros(1, 40, device="cuda", dtype=torch.bfloat16)
        work = torch.zeros(1 << 16, device="cuda", dtype=torch.uint8)
        hg.hashgrid_linear_forward(layer.handle, x, ld, 1, w, None, None, 0, y, max(ld, 40), hg.HASHGRID_BF16, None, work, 1 << 16)
        assert torch.equal(y, want), ld


@pytest.mark.gpu
def test_residual_in_place_and_slices_of_one_buffer():
    """y = act(x w^T) + y, and x and y side by side in one buffer (a concatenation)."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    buf = torch.randn(333, 96, device="cuda", generator=gen).bfloat16()
    w = torch.randn(64, 32, device="cuda", generator=gen).bfloat16()
    layer = hg.Linear(32, 64, hg.HASHGRID_BF16, hg.HASHGRID_ACT_RELU)
    want = layer.forward(buf[:, :32].contiguous(), w, residual=buf[:, 32:].contiguous())
    got = layer.forward(buf[:, :32], w, residual=buf[:, 32:], y=buf[:, 32:])
    assert torch.equal(got, want)


@pytest.mark.gpu
def test_equal_calls_give_equal_bits():
    gen = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(30000, 72, device="cuda", generator=gen).bfloat16()
    w = torch.randn(80, 72, device="cuda", generator=gen).bfloat16()
    dy = torch.randn(30000, 80, device="cuda", generator=gen).bfloat16()
    layer = hg.Linear(72, 80)
    one = [layer.forward(x, w), *layer.backward(dy, x, w)]
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(one, [layer.forward(x, w), *layer.backward(dy, x, w)]))


@pytest.mark.gpu
def test_gradients_against_differences():
    """dx, dw and db against central differences of sum(dy * y) in 64 bits, at the rounded operands."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    for act in ACTS:
        x = torch.randn(5, 6, device="cuda", generator=gen).half()
        w = torch.randn(4, 6, device="cuda", generator=gen).half()
        b = torch.randn(4, device="cuda", generator=gen)
        dy = torch.randn(5, 4, device="cuda", generator=gen).half()
        layer = hg.Linear(6, 4, hg.HASHGRID_F16, act)
        z = torch.empty(5, 4, device="cuda", dtype=torch.float16)
        layer.forward(x, w, b, z=z)
        dx, dw, db = layer.backward(dy, x, w, z=z, dL_dx=torch.empty(5, 6, device="cuda"))
        at = [x.double(), w.double(), b.double()]

        def loss(v):
            return float((act64(v[0] @ v[1].t() + v[2], act) * dy.double()).sum())
        h = 1e-5
        for k, got in enumerate((dx, dw, db)):
            for i in range(got.numel()):
                up, down = [t.clone() for t in at], [t.clone() for t in at]
                up[k].view(-1)[i] += h
                down[k].view(-1)[i] -= h
                d = (loss(up) - loss(down)) / (2 * h)
                # z is rounded to fp16 before its slope is taken (2^-11 |z| times a curvature of at most 1), and dz too:
                # at most 2 * 2^-11 * 6 of each of up to 6 terms of size 4
                assert abs(float(got.view(-1)[i]) - d) < 2 * 2.0 ** -11 * 6 * 4, (act, k, i)


@pytest.mark.gpu
def test_streams_and_graphs():
    """On a stream of its own; captured, replayed on new inputs; two graphs with a workspace each."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    layer = hg.Linear(64, 96, hg.HASHGRID_BF16, hg.HASHGRID_ACT_SILU)
    x = torch.randn(5000, 64, device="cuda", generator=gen).bfloat16()
    w = torch.randn(96, 64, device="cuda", generator=gen).bfloat16()
    dy = torch.randn(5000, 96, device="cuda", generator=gen).bfloat16()
    z = torch.empty(5000, 96, device="cuda", dtype=torch.bfloat16)
    y = layer.forward(x, w, z=z)
    want = [y, *layer.backward(dy, x, w, z=z)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [layer.forward(x, w, z=z, stream=s), *layer.backward(dy, x, w, z=z, stream=s)]
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    if hg.CHECKED:
        return
    xs, dys = x.clone(), dy.clone()
    graphs = []
    for _ in range(2):
        zz, work = torch.empty_like(z), layer.workspace(5000, "cuda")
        out = [torch.empty_like(t) for t in want]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.forward(xs, w, y=out[0], z=zz)
            layer.backward(dys, xs, w, z=zz, dL_dx=out[1], dL_dw=out[2], dL_db=out[3], workspace=work)
        graphs.append((g, out, zz, work))           # a graph's buffers live as long as it does
    xs.copy_(x.flip(0))
    dys.copy_(dy.flip(0))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for (g, *_), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    yr = layer.forward(xs, w, z=z)
    again = [yr, *layer.backward(dys, xs, w, z=z)]
    for _, out, *_ in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out, again))


@pytest.mark.gpu
@pytest.mark.skipif(hg.CHECKED, reason="the checked build is for one stream at a time")
def test_calls_on_several_streams_at_once():
    """Wide products, products split over clusters, narrow layers' backward passes, optimiser steps and the fixed head on
    streams of their own, all at once and many times over, give what they give alone: they share SMs, their shared
    memory and their tensor memory."""
    gen = torch.Generator(device="cuda").manual_seed(14)

    def rand(*shape):
        return torch.randn(*shape, device="cuda", generator=gen).bfloat16()
    jobs = []
    for N, K, M, act in ((6000, 1024, 1536, hg.HASHGRID_ACT_GELU), (16, 2048, 1024, hg.HASHGRID_ACT_NONE), (20000, 64, 64, hg.HASHGRID_ACT_RELU),
                         (333, 77, 130, hg.HASHGRID_ACT_SILU), (40, 4096, 264, hg.HASHGRID_ACT_NONE)):
        layer, x, w, dy = hg.Linear(K, M, activation=act), rand(N, K), rand(M, K), rand(N, M)
        z, work = rand(N, M), layer.workspace(N, "cuda")
        out = [torch.empty(N, M, device="cuda", dtype=torch.bfloat16), torch.empty(N, K, device="cuda"), torch.empty(M, K, device="cuda"),
               torch.empty(M, device="cuda")]

        def job(layer=layer, x=x, w=w, dy=dy, z=z, work=work, out=out, act=act):
            layer.forward(x, w, y=out[0], workspace=work)
            layer.backward(dy, x, w, z=None if act == hg.HASHGRID_ACT_NONE else z, dL_dx=out[1], dL_dw=out[2], dL_db=out[3], workspace=work)
        jobs.append((job, out))
    grid = hg.HashGrid(16, 2, 14, 16, 512)
    table, pts = torch.rand(16, 1 << 14, 2, device="cuda", generator=gen), torch.rand(50000, 3, device="cuda", generator=gen)
    ws, bs, y = [rand(o, i) for o, i in ((64, 32), (64, 64), (4, 64))], [torch.zeros(64, device="cuda")] * 3, torch.empty(50000, 4, device="cuda")
    jobs.append((lambda: hg.hashgrid_mlp_forward(grid.handle, pts, 50000, table, ws[0], bs[0], ws[1], bs[1], ws[2], bs[2], y), [y]))
    alone = []
    for job, out in jobs:
        job()
        torch.cuda.synchronize()
        alone.append([t.clone() for t in out])
    streams = [torch.cuda.Stream() for _ in jobs]
    for _, out in jobs:
        for t in out:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(30):
        for (job, _), s in zip(jobs, streams):
            with torch.cuda.stream(s):
                job()
    torch.cuda.synchronize()
    for (_, out), want in zip(jobs, alone):
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.gpu
def test_training_step_of_an_encoder_with_its_head():
    """Encode, two layers, their gradients, the tables' gradient and one optimiser step over the head, each held
    against 64 bits on the values that it was given."""
    gen = torch.Generator(device="cuda").manual_seed(10)
    grid = hg.HashGrid(L=4, F=2, log2T=10, N_min=2, N_max=16)
    table = torch.rand(4, 1024, 2, device="cuda", generator=gen) * 2 - 1
    pts = torch.rand(777, 3, device="cuda", generator=gen)
    l1, l2 = hg.Linear(8, 64, activation=hg.HASHGRID_ACT_RELU), hg.Linear(64, 4)
    master = [torch.randn(64, 8, device="cuda", generator=gen) * 0.3, torch.zeros(64, device="cuda"),
              torch.randn(4, 64, device="cuda", generator=gen) * 0.1, torch.zeros(4, device="cuda")]
    w1, w2 = master[0].bfloat16(), master[2].bfloat16()
    enc = grid.forward(pts, table).bfloat16()
    z = torch.empty(777, 64, device="cuda", dtype=torch.bfloat16)
    h = l1.forward(enc, w1, master[1], z=z)
    y = l2.forward(h, w2, master[3], y=torch.empty(777, 4, device="cuda"))
    dy = (2 * (y - 0.5) / y.numel()).bfloat16()
    dh, dw2, db2 = l2.backward(dy, h, w2)
    denc, dw1, db1 = l1.backward(dh, enc, w1, z=z, dL_dx=torch.empty(777, 8, device="cuda"))
    dtable = grid.backward(pts, denc)
    grads = [dw1, db1, dw2, db2]
    before = [p.clone() for p in master]
    opt = hg.AdamW(master, grads, copies=[w1, None, w2, None], weight_decay=[0.1, 0.0, 0.1, 0.0])
    opt.step(1, lr=1e-2, eps=1e-8, zero_grad=True)
    torch.cuda.synchronize()
    d = torch.double
    W1, W2 = before[0].bfloat16().to(d), before[2].bfloat16().to(d)
    h64 = act64(enc.to(d) @ W1.t(), hg.HASHGRID_ACT_RELU)
    close(h, h64, 2.0 ** -8 * h64.abs() * 1.01 + 2 * U * 10 * (enc.to(d).abs() @ W1.abs().t()), "h")
    dz = dh.to(d) * (z.to(d) > 0)
    close(denc, dz @ W1, 2 * U * 66 * (dz.abs() @ W1.abs()), "denc")
    want = {0: dz.t() @ enc.to(d), 1: dz.sum(0), 2: dy.to(d).t() @ h.to(d), 3: dy.to(d).sum(0)}
    for k, g64 in want.items():
        # first step: m / c1 = g, sqrt(v / c2) = |g|; the gradient is off by at most 1e-5 of its column's size
        upd = 1e-2 * g64 / (g64.abs() + 1e-8)
        decay = 1e-2 * (0.1 if k in (0, 2) else 0.0)
        sure = g64.abs() > 1e-4 * g64.abs().max()
        err = (master[k].to(d) - (before[k].to(d) * (1 - decay) - upd)).abs()
        assert float(err[sure].max()) < 1e-5, k
    assert torch.equal(w1, master[0].bfloat16()) and torch.equal(w2, master[2].bfloat16())
    assert all(int(g.count_nonzero()) == 0 for g in grads)
    assert bool(torch.isfinite(dtable).all()) and int(dtable.count_nonzero()) > 0


@pytest.mark.gpu
@pytest.mark.timeout(900)
def test_layers_and_optimiser_under_the_checked_build():
    """These tests and those of the optimiser once more with every plain access range-checked (TMA copies are held to
    their arrays by their tensor maps)."""
    if hg.CHECKED:
        pytest.skip("this is the checked build")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_linear.py", "tests/test_adamw.py", "-m", "gpu", "-q", "-x",
                        "-p", "no:cacheprovider"], cwd=root, env=dict(os.environ, HASHGRID_CHECKED="1"), capture_output=True,
                       text=True, timeout=800)
    assert r.returncode == 0 and " passed" in r.stdout, r.stdout[-3000:] + r.stderr[-2000:]


def test_refusals():
    lib, vp = hg.lib, ctypes.c_void_p
    for args in [(0, 4, 2, 0), (4, 0, 2, 0), (65537, 4, 2, 0), (4, 65537, 2, 0), (4, 4, 0, 0), (4, 4, 3, 0), (4, 4, 2, 4),
                 (4, 4, 2, -1)]:
        h = vp(7)
        assert lib.hashgrid_linear_create(*args, ctypes.byref(h)) == hg.HASHGRID_ERR_ARG and h.value is None
    assert lib.hashgrid_linear_create(4, 4, 2, 0, None) == hg.HASHGRID_ERR_ARG
    layer = hg.Linear(8, 4, hg.HASHGRID_F16, hg.HASHGRID_ACT_RELU)
    assert hg.hashgrid_linear_params(layer.handle) == {"in": 8, "out": 4, "dtype": 1, "activation": 1}
    h, p = layer.handle, 0x1000

    def forward(x=p, ldx=8, N=2, w=p, b=p, r=None, ldr=4, y=p, ldy=4, yt=1, z=None):
        return lib.hashgrid_linear_forward(h, x, ldx, N, w, b, r, ldr, y, ldy, yt, z, None, 0, None, None)
    A, L = hg.HASHGRID_ERR_ARG, hg.HASHGRID_ERR_ALIGN
    assert lib.hashgrid_linear_forward(None, p, 8, 2, p, p, None, 4, p, 4, 1, None, None, 0, None, None) == A
    assert forward(N=0, x=None, w=None, y=None) == hg.HASHGRID_OK
    assert forward(N=-1) == A and forward(N=2 ** 31) == A
    assert forward(yt=2) == A and forward(yt=3) == A            # fp16 layer: y is fp16 or fp32
    assert forward(ldx=7) == A and forward(x=None) == A and forward(x=p + 2) == L
    host = np.zeros(4096, np.uint8)
    at = host.ctypes.data + (-host.ctypes.data) % 16
    assert forward(x=at) == A

    def backward(dy=p, lddy=4, x=p, ldx=8, N=2, w=p, z=p, dx=p, lddx=8, xt=0, dw=None, wt=0, db=None, work=p, size=1 << 20):
        return lib.hashgrid_linear_backward(h, dy, lddy, x, ldx, N, w, z, dx, lddx, xt, dw, wt, db, work, size, None, None)
    assert backward(dx=None) == hg.HASHGRID_OK                   # nothing is asked for
    assert backward(N=-1) == A and backward(xt=2) == A and backward(wt=2) == A and backward(lddy=3) == A
    assert backward(dy=p + 4) == L and backward(dy=None) == A
    size = hg.hashgrid_linear_backward_workspace
    assert size(None, 5, 4, 8) == 0 and size(h, -1, 4, 8) == 0 and 0 < size(h, 100, 8, 8) < size(h, 100, 8, 9)
    assert hg.hashgrid_linear_forward_workspace(h, 100, 8) == 0 < hg.hashgrid_linear_forward_workspace(h, 100, 9)
    for f in (lambda n: size(h, n, 5, 9), lambda n: hg.hashgrid_linear_forward_workspace(h, n, 9)):
        sizes = [f(n) for n in list(range(1, 200)) + [10 ** k for k in range(3, 9)] + [16383, 16384, 16385]]
        assert [f(n) for n in range(1, 200)] == sorted(f(n) for n in range(1, 200)) and f(16384) <= f(16385) and min(sizes) >= 0


def test_binding_refuses_wrong_tensors():
    layer = hg.Linear(8, 4, hg.HASHGRID_BF16)
    x, w = torch.zeros(3, 8, dtype=torch.bfloat16), torch.zeros(4, 8, dtype=torch.bfloat16)
    for bad in (dict(x=x.float()), dict(x=torch.zeros(3, 9, dtype=torch.bfloat16)), dict(w=w.half()), dict(w=w.t()),
                dict(x=torch.zeros(8, 3, dtype=torch.bfloat16).t()), dict(b=torch.zeros(5)), dict(b=torch.zeros(4).double()),
                dict(z=torch.zeros(3, 5, dtype=torch.bfloat16)), dict(residual=torch.zeros(2, 4, dtype=torch.bfloat16)),
                dict(y=torch.zeros(3, 4, dtype=torch.float16)),
                dict(y=torch.zeros(3, 4), residual=torch.zeros(3, 4, dtype=torch.bfloat16))):
        with pytest.raises(hg.HashGridError) as e:
            layer.forward(**{"x": x, "w": w, **bad})
        assert e.value.code == hg.HASHGRID_ERR_ARG


@pytest.mark.gpu
def test_gpu_refusals():
    """What needs device pointers to be refused: extents, missing arrays, the workspace's size."""
    layer = hg.Linear(8, 4, hg.HASHGRID_BF16, hg.HASHGRID_ACT_GELU)
    big = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    p = big.data_ptr()
    lib, h = hg.lib, layer.handle
    assert lib.hashgrid_linear_forward(h, p, 1 << 30, 100, p, None, None, 4, p, 4, 2, None, None, 0, None, None) == hg.HASHGRID_ERR_ARG
    assert "allocation ends" in hg.hashgrid_last_error()
    args = [h, p, 4, p, 8, 100, p, None, p, 8, 0, None, 0, None, p, 1 << 20, None, None]
    assert lib.hashgrid_linear_backward(*args) == hg.HASHGRID_ERR_ARG and "z is NULL" in hg.hashgrid_last_error()
    args[7], args[15] = p, hg.hashgrid_linear_backward_workspace(h, 100, 4, 8) - 1
    assert lib.hashgrid_linear_backward(*args) == hg.HASHGRID_ERR_ARG and "workspace" in hg.hashgrid_last_error()
    args = [h, p, 9, 100, p, None, None, 4, p, 4, 2, None, None, 0, None, None]
    assert lib.hashgrid_linear_forward(*args) == hg.HASHGRID_ERR_ARG and "workspace" in hg.hashgrid_last_error()
    with pytest.raises(hg.HashGridError):
        layer.forward(torch.zeros(5, 8, dtype=torch.bfloat16), torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda"),
                      y=torch.zeros(5, 4, dtype=torch.bfloat16, device="cuda"))
