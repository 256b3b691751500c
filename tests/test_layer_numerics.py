"""Values of the layers that other tests do not reach: long sums, NaN, many groups of tiles, the way on to the tables."""
import numpy as np
import pytest
import torch

import multiresolution_hash_grid_b200 as hg
from tests.test_linear import ACTS, U, check_backward, check_forward, close, half_step, rows_of, slope64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("N,K,M", [(1 << 19, 1024, 1280), (300001, 1100, 1030), (1 << 17, 1500, 1700), (50000, 2048, 2048)])
def test_long_sums_with_16_bit_results(N, K, M, dtype):
    """A weight gradient in 16 bits whose rows are not cut into parts. The tensor cores' additions cut off, 1.1e-9 of the
    result a term, 5.8e-4 for 2^19 terms, more than the rounding of fp16 at the end. An accumulator takes at most 49152
    terms of such a sum, which lose 5.41e-5; or 768, which lose 8.4e-7, and the at most 683 additions of those round by
    2^-24 each, together 4.1e-5 at the very worst. Rounding the result to nearest moves no sum of values of either
    sign: it adds half a step, 2^-11 or 2^-8, times 1 / sqrt(values), a thousandth."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    dy = torch.randn(N, M, device="cuda", generator=gen).to(dtype)
    x = torch.randn(N, K, device="cuda", generator=gen).to(dtype)
    w = torch.zeros(M, K, device="cuda", dtype=dtype)
    code = hg.HASHGRID_F16 if dtype == torch.float16 else hg.HASHGRID_BF16
    _, dw, _ = hg.Linear(K, M, code).backward(dy, x, w, dL_dx=None, dL_db=None, dL_dw=torch.empty_like(w))
    ref = torch.zeros(M, K, device="cuda", dtype=torch.float64)
    for at in range(0, N, 1 << 16):
        ref += dy[at:at + (1 << 16)].double().t() @ x[at:at + (1 << 16)].double()
    d = dw.double() - ref
    bias = float((d * ref.sign()).sum() / ref.abs().sum())
    assert abs(bias) < 5.41e-5 + {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[dtype] * 4 / (K * M) ** 0.5, bias


@pytest.mark.parametrize("N,K,M", [(9600, 65536, 512), (1280, 65536, 1024)])
def test_widest_layers_with_16_bit_results(N, K, M):
    """The longest sums of the forward pass: gathered by pairs of blocks, and split into shares."""
    check_forward(N, K, M, hg.HASHGRID_BF16, hg.HASHGRID_ACT_SILU)
    check_forward(N, K, M, hg.HASHGRID_F16, hg.HASHGRID_ACT_NONE, residual=False, keep=False)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("N,K,M", [(64, 40, 24), (70, 33, 35), (16, 2048, 1024), (9000, 64, 64), (19100, 512, 160)])
def test_relu_passes_a_nan_on(N, K, M, dtype):
    """A NaN in a row of x is one in that row of y, as the formula's maximum has it, and no other row has any. Where the loss
    then gives NaN gradients they go on: z = NaN stops no gradient."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    code = hg.HASHGRID_F16 if dtype == torch.float16 else hg.HASHGRID_BF16
    layer = hg.Linear(K, M, code, hg.HASHGRID_ACT_RELU)
    x = torch.randn(N, K, device="cuda", generator=gen).to(dtype)
    w = torch.randn(M, K, device="cuda", generator=gen).to(dtype)
    x[3, 1] = float("nan")
    for y in (torch.empty(N, M, device="cuda", dtype=dtype), torch.empty(N, M, device="cuda")):
        z = torch.empty(N, M, device="cuda", dtype=dtype)
        layer.forward(x, w, y=y, z=z)
        assert bool(torch.isnan(y[3]).all()) and int(torch.isnan(y).sum()) == M
    dy = torch.randn(N, M, device="cuda", generator=gen).to(dtype)
    dy[3] = float("nan")
    dx, dw, db = layer.backward(dy, x, w, z=z)
    assert bool(torch.isnan(dx[3]).all()) and int(torch.isnan(dx).sum()) == K
    assert bool(torch.isnan(dw).all()) and bool(torch.isnan(db).all())
    assert not bool(torch.isnan(layer.forward(x, torch.zeros_like(w), torch.full((M,), -1.0, device="cuda"))[:3]).any())


@pytest.mark.parametrize("act", [hg.HASHGRID_ACT_GELU, hg.HASHGRID_ACT_SILU])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("N,K,M,pad", [(1, 64, 64, 0), (16, 2048, 1024, 0), (200, 48, 72, 8), (4099, 173, 257, 3), (33, 9, 7, 1), (90001, 64, 64, 0),
                                       (90001, 64, 24, 8), (90001, 27, 31, 3), (20000, 128, 128, 0), (40000, 200, 40, 0), (9700, 1000, 300, 0),
                                       (19100, 160, 512, 0), (30000, 16, 816, 8), (50000, 64, 4, 0), (40000, 40, 200, 0),
                                       (50000, 64, 256, 8), (700, 1100, 1900, 0)])
def test_fp32_gradients_behind_smooth_activations(N, K, M, pad, dtype, act):
    """dz enters the products as two numbers of the layer's type: off by the square of its half step, 2^-16 for bf16 and 2^-22
    for fp16 (at least half of fp16's smallest number, 2^-25), not by the half step. The slope is off by 32 * 2^-24 (1 + |z|),
    and the sums run over twice as many terms, the low half of them 2^-8 as large."""
    gen = torch.Generator(device="cuda").manual_seed(N + M)
    x, dy = rows_of(N, K, pad, dtype, gen), rows_of(N, M, pad, dtype, gen)
    w = (torch.randn(M, K, device="cuda", generator=gen) / M ** 0.5).to(dtype)
    z = torch.randn(N, M, device="cuda", generator=gen).to(dtype)
    layer = hg.Linear(K, M, hg.HASHGRID_F16 if dtype == torch.float16 else hg.HASHGRID_BF16, act)
    dx, dw, db = layer.backward(dy, x, w, z=z, dL_dx=torch.empty(N, K, device="cuda"))
    X, W, DY, Z = x.double(), w.double(), dy.double(), z.double()
    dz = DY * slope64(Z, act)
    slope = 32 * U * (1 + Z.abs()) * DY.abs()
    err = slope + dz.abs() * half_step(dtype)[0] ** 2 * 1.01 + half_step(dtype)[1]
    for got, ref, mag, carried, terms, name in ((dx, dz @ W, dz.abs() @ W.abs(), err @ W.abs(), M, "dx"),
                                                (dw, dz.t() @ X, dz.abs().t() @ X.abs(), err.t() @ X.abs(), N, "dw"),
                                                (db, dz.sum(0), dz.abs().sum(0), slope.sum(0), N, "db")):
        close(got, ref, 2 * U * (2 * terms + 4) * mag + carried + 2 * U * ref.abs(), name)
        assert float((got.double() - ref).norm() / ref.norm()) < 2.0 ** -16 + 2e-5, name


@pytest.mark.parametrize("N", [40, 9000])
def test_gradients_beyond_the_range_of_fp16(N):
    """A slope above 1 takes dz beyond fp16's largest number: its two parts still hold it, and infinities and NaN stay."""
    z = torch.full((N, 16), 1.5, device="cuda").half()
    dy = torch.full((N, 16), 60000.0, device="cuda").half()
    dy[1, 0], dy[2, 1], dy[3, 2] = float("inf"), float("-inf"), float("nan")
    w = (torch.eye(16, device="cuda") / 64).half()
    x = torch.full((N, 16), 2.0 ** -10, device="cuda").half()
    dx, dw, db = hg.Linear(16, 16, hg.HASHGRID_F16, hg.HASHGRID_ACT_GELU).backward(dy, x, w, z=z, dL_dx=torch.empty(N, 16, device="cuda"))
    want = float(60000 * slope64(torch.tensor(1.5, dtype=torch.float64), hg.HASHGRID_ACT_GELU))
    assert want > 65504 and float((dx[4:] * 64 - want).abs().max()) < want * (2.0 ** -22 + 64 * U)
    assert float((dw[3:] * 1024 - want * N).abs().max()) < want * N * (2.0 ** -22 + 2 * U * (2 * N + 4) + 64 * U)
    assert float(dw[0, 0]) == float("inf") and float(dw[1, 0]) == float("-inf") and bool(torch.isnan(dw[2]).all())
    assert bool(torch.isnan(dx[3]).all()) and not bool(torch.isfinite(dx[1:3, :2].diagonal()).any())
    assert float(db[0]) == float("inf") and float(db[1]) == float("-inf") and bool(torch.isnan(db[2]))


@pytest.mark.parametrize("tiles", [6, 7, 12, 13, 18, 25])
@pytest.mark.parametrize("K,M", [(64, 64), (32, 64), (128, 24), (128, 128), (24, 104)])
def test_one_pass_backward_over_many_groups_of_tiles(K, M, tiles):
    """So many tiles of 128 rows for each of 148 blocks, with one more for some and a ragged last one: dW's sums leave tensor
    memory every six tiles, by two accumulators in turn, each several times over, and in groups of one tile too."""
    for rows in ((148 * tiles) * 128, (148 * tiles) * 128 + 1, (148 * tiles + 100) * 128 - 51):
        act = ACTS[(tiles + rows) % 4]
        check_backward(rows, K, M, hg.HASHGRID_BF16, act, dx32=tiles % 2 == 0, dw32=True, seed=tiles, want=(tiles % 5 != 0, True, True))


@pytest.mark.skipif(hg.CHECKED, reason="the checked build is for one stream at a time")
def test_optimiser_steps_beside_layers():
    """Steps of three lists on streams of their own, while layers run on others, do what they do alone."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    base = [torch.randn(n, device="cuda", generator=gen) for n in (1, 255, 4097, 1 << 20, 300000)]
    grad = [torch.randn(p.numel(), device="cuda", generator=gen).bfloat16() for p in base]

    def lists():
        made = []
        for bits in (32, 8, 8):
            p = [t.clone() for t in base]
            made.append((p, hg.AdamW(p, [g.clone() for g in grad], bits=bits, weight_decay=0.01)))
        return made
    layer, work = hg.Linear(64, 64, activation=hg.HASHGRID_ACT_RELU), hg.Linear(64, 64).workspace(60000, "cuda")
    wide = hg.Linear(1024, 512)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen).bfloat16()  # noqa: E731
    x, w, dy, z, xw, ww = rnd(60000, 64), rnd(64, 64), rnd(60000, 64), rnd(60000, 64), rnd(5000, 1024), rnd(512, 1024)
    out = [torch.empty(60000, 64, device="cuda"), torch.empty(64, 64, device="cuda"), torch.empty(64, device="cuda")]
    yw = torch.empty(5000, 512, device="cuda").bfloat16()

    def layers():
        layer.backward(dy, x, w, z=z, dL_dx=out[0], dL_dw=out[1], dL_db=out[2], workspace=work)
        wide.forward(xw, ww, y=yw)
    layers()
    alone = lists()
    for k in range(1, 31):
        for i, (_, opt) in enumerate(alone):
            opt.step(k, lr=1e-3, seed=i)
    torch.cuda.synchronize()
    want = [t.clone() for t in out + [yw]]
    beside = lists()
    for t in out + [yw]:
        t.zero_()
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for k in range(1, 31):
        with torch.cuda.stream(streams[3]):
            layers()
        for i, (_, opt) in enumerate(beside):
            with torch.cuda.stream(streams[i]):
                opt.step(k, lr=1e-3, seed=i)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out + [yw], want))
    for (p, a), (q, b) in zip(alone, beside):
        assert all(torch.equal(s, t) for s, t in zip(p, q))
        assert all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(a.m + a.v, b.m + b.v))


def test_gradient_of_the_tables_through_the_layers():
    """What two layers hand down as dL/d(encoding), in fp32, becomes the tables' gradient that the oracle has for it."""
    import oracle
    from tests.test_parity import check_gradient
    gen = torch.Generator(device="cuda").manual_seed(11)
    grid, og = hg.HashGrid(L=4, F=2, log2T=10, N_min=2, N_max=16), oracle.Grid(4, 2, 10, 2, 16)
    table = torch.rand(4, 1024, 2, device="cuda", generator=gen) * 2 - 1
    pts = torch.rand(1777, 3, device="cuda", generator=gen)
    l1, l2 = hg.Linear(8, 64, activation=hg.HASHGRID_ACT_SILU), hg.Linear(64, 4)
    w1, w2 = (torch.randn(*s, device="cuda", generator=gen).bfloat16() for s in ((64, 8), (4, 64)))
    enc = grid.forward(pts, table).bfloat16()
    z = torch.empty(1777, 64, device="cuda", dtype=torch.bfloat16)
    h = l1.forward(enc, w1, z=z)
    dy = torch.randn(1777, 4, device="cuda", generator=gen).bfloat16()
    dh, _, _ = l2.backward(dy, h, w2)
    denc, _, _ = l1.backward(dh, enc, w1, z=z, dL_dx=torch.empty(1777, 8, device="cuda"))
    dtable = grid.backward(pts, denc)
    torch.cuda.synchronize()
    ref = og.backward(pts.cpu().numpy(), denc.cpu().numpy())
    check_gradient(dtable.cpu().numpy(), ref)
    assert np.abs(ref).max() > 0.1
