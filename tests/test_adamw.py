"""AdamW over many tensors (hashgrid_adamw_*), against the documented formula: the states bit for bit (every
operation on them is one rounded fp32 operation, which numpy computes too), the parameters in 64 bits."""
import ctypes

import numpy as np
import pytest
import torch

import multiresolution_hash_grid_b200 as hg

f32 = np.float32
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def mix(h):
    h = np.asarray(h, np.uint32)
    for s, f in ((16, 0x7FEB352D), (15, 0x846CA68B)):
        h = h ^ (h >> np.uint32(s))
        h = (h.astype(np.uint64) * f).astype(np.uint32)
    return h ^ (h >> np.uint32(16))


def bits_of(n, seed, step, k):
    key = (seed * 0x9E3779B1 + step * 0x85EBCA77 + k * 0xC2B2AE3D) & 0xFFFFFFFF
    return mix(np.arange(n, dtype=np.uint32) ^ mix(key))


def e4m3_values():
    """The values of codes 0..126, by the format's definition (4 exponent bits with bias 7, 3 mantissa bits)."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))


VALUES = e4m3_values()


def nearest_code(y):
    """Codes of 0 <= y <= 448 (fp64 of fp32 values), ties to the even code."""
    hi = np.clip(np.searchsorted(VALUES, y, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = VALUES[hi] - y, y - VALUES[lo]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def encode(x, r16, root):
    """Codes (as signed values) and scales of one tensor, x fp32."""
    n = x.size
    blocks = -(-n // 256)
    full = np.zeros(blocks * 256, f32)
    full[:n] = x
    full = full.reshape(blocks, 256)
    mag = np.abs(full)
    top = np.where(np.isfinite(mag), mag, 0).max(1).astype(f32)
    scale = (top / f32(448)).astype(f32)
    with np.errstate(all="ignore"):
        inv = np.where(top > f32(2.0 ** -100), f32(448) / top, f32(0)).astype(f32)
        y = (mag * inv[:, None]).astype(f32)
    y = np.where(np.isfinite(y), y, 0).astype(f32).reshape(-1)[:n]
    if r16 is None:
        v = VALUES[nearest_code(y.astype(np.float64))]
    else:  # in 64 bits: one spacing of the code grid, a part of it added, cut down
        y64 = y.astype(np.float64)
        spacing = 2.0 ** (np.floor(np.log2(np.maximum(y64, 2.0 ** -6))) - 3)
        part = (r16.astype(np.float64) * 16 + 8) / 2 ** 20
        low = np.where(y < f32(2.0 ** -6), f32(2.0 ** -6), f32(0))
        y64 = np.where(low > 0, (y + low).astype(f32).astype(np.float64) - 2.0 ** -6, y64)
        v = np.minimum(np.floor(y64 / spacing + part) * spacing, 448.0)
    if root:
        v = np.where(x > 0, np.maximum(v, 2.0 ** -9), v)
    v = np.where(x < 0, -v, v)
    return np.where(np.isfinite(x), v, np.nan), scale


def reference(g, m, v, b1, b2):
    """m and v in fp32, one rounding an operation."""
    b1, b2 = f32(b1), f32(b2)
    m = m * b1 + g * f32(1 - float(b1))
    v = v * b2 + (g * g) * f32(1 - float(b2))
    assert m.dtype == v.dtype == f32
    return m, v


def make(sizes, param, grad, state, seed, copy=None, zeros=0.2):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    p = [(torch.randn(n, device="cuda", generator=gen) * 0.1).to(TORCH[param]) for n in sizes]
    g = [(torch.randn(n, device="cuda", generator=gen) * 10.0 ** (-k % 5 - 3) *
          (torch.rand(n, device="cuda", generator=gen) > zeros)).to(TORCH[grad]) for k, n in enumerate(sizes)]
    c = None if copy is None else [torch.full((n,), 9.0, device="cuda", dtype=TORCH[copy]) for n in sizes]
    return p, g, c


def host(t):
    return t.float().cpu().numpy()


def run_steps(sizes, param="f32", grad="f32", bits=32, copy=None, seed=0, steps=3, decay=0.05, lr_scale=1.0, data=1):
    p, g, c = make(sizes, param, grad, bits, data, copy)
    opt = hg.AdamW(p, g, bits=bits, copies=c, weight_decay=decay, lr_scale=lr_scale)
    for t in range(1, steps + 1):
        p0, g0 = [host(x) for x in p], [host(x) for x in g]
        m0, v0 = [host(x) for x in opt.m], [host(x) for x in opt.v]
        if bits == 8:
            rep = lambda s, n: np.repeat(host(s), 256)[:n]  # noqa: E731
            m0 = [(x * rep(s, x.size)).astype(f32) for x, s in zip(m0, opt.m_scales)]
            v0 = [(x * rep(s, x.size)).astype(f32) for x, s in zip(v0, opt.v_scales)]
            v0 = [(x * x).astype(f32) for x in v0]
        opt.step(t, lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8, seed=seed)
        torch.cuda.synchronize()
        for k, n in enumerate(sizes):
            rm, rv = reference(g0[k], m0[k], v0[k], 0.9, 0.99)
            # the step in 64 bits: m, v, its root, the corrections, the products and the quotient (2 ulp) are some sixteen
            # half steps of fp32 of a step of lr |m| c1 / root, the product and difference of p four; then p's own rounding
            b1, b2, lr = float(f32(0.9)), float(f32(0.99)), lr_scale * float(f32(1e-2))
            m = m0[k] * b1 + g0[k].astype(np.float64) * (1 - b1)
            root = np.sqrt((v0[k] * b2 + g0[k].astype(np.float64) ** 2 * (1 - b2)) / (1 - b2 ** t)) + 1e-8
            size = lr * (np.abs(m0[k] * b1) + np.abs(g0[k].astype(np.float64) * (1 - b1))) / (1 - b1 ** t) / root
            p64 = p0[k].astype(np.float64) * (1 - lr * float(f32(decay))) - lr * m / (1 - b1 ** t) / root
            half, least = {"f32": (2.0 ** -24, 0), "bf16": (2.0 ** -8, 0), "f16": (2.0 ** -11, 2.0 ** -25)}[param]
            tol = 2.0 ** -24 * (16 * size + 4 * np.abs(p0[k])) + half * np.abs(p64) * 1.01 + least + 1e-30
            assert np.all(np.abs(host(p[k]) - p64) <= tol), (t, k, n)
            if copy is not None:
                assert torch.equal(c[k], p[k].to(TORCH[copy])), (t, k, n)
            if bits == 32:
                assert np.array_equal(host(opt.m[k]), rm) and np.array_equal(host(opt.v[k]), rv), (t, k, n)
            else:
                r = None if seed == 0 else bits_of(n, seed, t, k)
                for name, x, code, scale, root in (("m", rm, opt.m[k], opt.m_scales[k], False),
                                                   ("v", np.sqrt(rv), opt.v[k], opt.v_scales[k], True)):
                    r16 = None if r is None else (r >> np.uint32(16) if root else r & np.uint32(0xFFFF))
                    cw, sw = encode(x, r16, root)
                    assert np.array_equal(host(scale), sw), (name, t, k, n)
                    assert np.array_equal(host(code), cw.astype(f32)), (name, t, k, n)


SIZES = [1, 3, 4, 5, 127, 128, 131, 255, 256, 257, 1000, 2048, 70001]


@pytest.mark.gpu
@pytest.mark.parametrize("grad", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("param", ["f32", "bf16", "f16"])
def test_32_bit_states(param, grad):
    run_steps(SIZES, param, grad, copy="bf16" if param == "f32" else None)


@pytest.mark.gpu
@pytest.mark.parametrize("seed", [0, 1, 0xFFFFFFFF])
@pytest.mark.parametrize("param,grad", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
def test_8_bit_states(param, grad, seed):
    run_steps(SIZES, param, grad, bits=8, seed=seed, copy="f16" if param == "f32" else None)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_more_tensors_than_one_launch_takes(bits):
    run_steps([(37 * k) % 700 for k in range(901)], bits=bits, seed=77, steps=2)


@pytest.mark.gpu
def test_mixed_list_with_rates_of_its_own():
    """fp32 and 8-bit states, every type, per-tensor rates and decays in one list equal lists of one."""
    kinds = [("f32", "f32", 32), ("bf16", "f32", 8), ("f16", "f16", 32), ("f32", "bf16", 8), ("bf16", "bf16", 32)]
    lists = [make([300 + 111 * k], a, b, bits, 50 + k) for k, (a, b, bits) in enumerate(kinds)]
    lone = [make([300 + 111 * k], a, b, bits, 50 + k) for k, (a, b, bits) in enumerate(kinds)]
    rate, decay = [1.0, 5.0, 0.5, 2.0, 0.0], [0.0, 0.1, 0.2, 0.3, 0.4]
    zeros = lambda n, bits: (torch.zeros(n, device="cuda") if bits == 32 else  # noqa: E731
                             torch.zeros(n, device="cuda", dtype=torch.uint8))
    m = [zeros(l[0][0].numel(), k[2]) for l, k in zip(lists, kinds)]
    v = [zeros(l[0][0].numel(), k[2]) for l, k in zip(lists, kinds)]
    opt = hg.AdamW([l[0][0] for l in lists], [l[1][0] for l in lists], m=m, v=v, lr_scale=rate, weight_decay=decay)
    ones = [hg.AdamW(l[0], l[1], bits=k[2], lr_scale=r, weight_decay=d) for l, k, r, d in zip(lone, kinds, rate, decay)]
    for t in (1, 2, 3):
        opt.step(t, lr=1e-2)
        for o in ones:
            o.step(t, lr=1e-2)
    for k, (a, b) in enumerate(zip(lists, lone)):
        assert torch.equal(a[0][0], b[0][0]), k
        assert torch.equal(opt.m[k].view(torch.uint8), ones[k].m[0].view(torch.uint8)), k


@pytest.mark.gpu
def test_zero_grad_and_untouched_neighbours():
    """The gradient is cleared when asked, also at ragged ends; what lies behind a tensor's end stays."""
    for n in (5, 257, 4099):
        for gt in (torch.float32, torch.bfloat16):
            bufs = {k: torch.full((n + 64,), 3.0, device="cuda", dtype=gt if k == "g" else torch.float32) for k in "pgmv"}
            opt = hg.AdamW([bufs["p"][:n]], [bufs["g"][:n]], m=[bufs["m"][:n]], v=[bufs["v"][:n]])
            opt.step(1, lr=1e-3, zero_grad=False)
            assert bool((bufs["g"] == 3.0).all())
            opt.step(2, lr=1e-3, zero_grad=True)
            assert int(bufs["g"][:n].count_nonzero()) == 0
            assert all(bool((b[n:] == 3.0).all()) for b in bufs.values())
    codes = torch.full((300,), 0x11, device="cuda", dtype=torch.uint8)
    scales = torch.full((4,), 0.5, device="cuda")
    p, g = torch.ones(258, device="cuda"), torch.ones(258, device="cuda")
    opt = hg.AdamW([p], [g], m=[codes[:258]], v=[torch.zeros(258, device="cuda", dtype=torch.uint8)],
                   block_scales=([scales[:2]], [torch.zeros(2, device="cuda")]))
    opt.step(1, lr=1e-3)
    assert bool((codes[258:] == 0x11).all()) and bool((scales[2:] == 0.5).all()) and int(codes[257]) != 0x11


@pytest.mark.gpu
def test_8_bit_extremes():
    """A block of zeros, one of a single tiny value beside a large one, an infinity, a NaN: the scale comes from what is
    finite, a positive v keeps a code, a value that is not finite is NaN and its neighbours are as without it."""
    n = 1024
    g = torch.zeros(n, device="cuda")
    g[256] = 1.0
    g[300] = 1e-12
    g[600], g[601], g[602] = float("inf"), float("nan"), 2.0
    p = torch.zeros(n, device="cuda")
    opt = hg.AdamW([p], [g], bits=8)
    opt.step(1, lr=1e-3)
    m, v = host(opt.m[0]), host(opt.v[0])
    ms, vs = host(opt.m_scales[0]), host(opt.v_scales[0])
    assert ms[0] == 0 and vs[0] == 0 and not m[:256].any() and not v[:256].any() and ms[3] == 0
    assert m[256] == 448 and v[256] == 448 and m[300] == 0 and v[300] == f32(2.0 ** -9)
    assert np.isnan(m[[600, 601]]).all() and np.isnan(v[[600, 601]]).all() and m[602] == 448 and v[602] == 448
    assert ms[2] == f32(f32(2) * f32(1 - float(f32(0.9)))) / f32(448)
    g.zero_()
    for t in range(2, 60):
        opt.step(t, lr=1e-3, seed=t)
    assert np.isfinite(host(p)[300]) and abs(host(p)[300]) < 0.1     # no step grew beyond its size
    assert host(opt.v[0])[300] > 0


@pytest.mark.gpu
def test_stochastic_rounding_follows_an_average_that_nearest_rounding_cannot():
    """sqrt(v) of half the elements should grow from 1 towards 1.25 with b2 = 0.999 in steps that are far below half a
    code; the mean over 16384 elements (a standard error of at most 0.0625 / 128) is held to it."""
    n = 1 << 15
    root = torch.ones(n, device="cuda")
    root[::2] = 2.0
    g = root.clone()
    g[1::2] = 1.25
    out = {}
    for seed in (0, 1):
        p = torch.zeros(n, device="cuda")
        v8 = (root * 224).to(torch.float8_e4m3fn)
        opt = hg.AdamW([p], [g], m=[torch.zeros(n, device="cuda", dtype=torch.uint8)], v=[v8],
                       block_scales=([torch.zeros(n // 256, device="cuda")], [torch.full((n // 256,), 1 / 224, device="cuda")]))
        for t in range(1, 501):
            opt.step(1000 + t, lr=0.0, beta2=0.999, seed=seed and t)
        out[seed] = float((host(opt.v[0]) * np.repeat(host(opt.v_scales[0]), 256))[1::2].mean())
    exact = np.sqrt(1.25 ** 2 + (1 - 1.25 ** 2) * 0.999 ** 500)
    assert abs(out[0] - 1.0) < 1e-3                      # nearest: it never moves
    # stochastic: unbiased in sqrt(v), and v = E[root]^2 + var, var <= (spacing / 2)^2 = 0.0625^2 / 4 a step, of which a
    # thousandth decays: the average of the root is off by less than half its variance
    assert abs(out[1] - exact) < 0.01, (out[1], exact)


@pytest.mark.gpu
def test_device_step_stream_and_graph():
    sizes = [1000, 7, 4096]
    a, ga, _ = make(sizes, "f32", "f32", 8, 3)
    b, gb, _ = make(sizes, "f32", "f32", 8, 3)
    want, opt = hg.AdamW(a, ga, bits=8), hg.AdamW(b, gb, bits=8)
    t = torch.zeros(1, dtype=torch.int64, device="cuda")
    opt.step(0, lr=1e-2, seed=5, device_step=t)                    # t = 0: nothing happens
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and int(opt.m[0].view(torch.uint8).count_nonzero()) == 0
    if hg.CHECKED:
        return
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        t.add_(1)
        opt.step(0, lr=1e-2, seed=5, device_step=t)
    for k in range(1, 6):
        want.step(k, lr=1e-2, seed=5)
        graph.replay()
    torch.cuda.synchronize()
    for k in range(3):
        assert torch.equal(a[k], b[k]) and torch.equal(want.v[k].view(torch.uint8), opt.v[k].view(torch.uint8))


def test_refusals():
    lib, A, L = hg.lib, hg.HASHGRID_ERR_ARG, hg.HASHGRID_ERR_ALIGN
    P = 0x1000
    good = dict(param=P, grad=P, m=P, v=P, m_scale=None, v_scale=None, copy=None, n=0, param_dtype=0, grad_dtype=0,
                state_dtype=0, copy_dtype=2, lr_scale=1.0, weight_decay=0.0)

    def create(*tensors, count=None):
        arr = (hg.AdamwTensor * max(1, len(tensors)))(*[hg.AdamwTensor(**{**good, **t}) for t in tensors])
        h = ctypes.c_void_p(3)
        rc = lib.hashgrid_adamw_create(arr, len(tensors) if count is None else count, ctypes.byref(h))
        if rc == 0:
            lib.hashgrid_adamw_destroy(h)
        else:
            assert h.value is None
        return rc
    assert create(count=0) == A and create({}, count=65537) == A
    assert lib.hashgrid_adamw_create(None, 1, ctypes.byref(ctypes.c_void_p())) == A
    assert lib.hashgrid_adamw_create((hg.AdamwTensor * 1)(), 1, None) == A
    for bad in (dict(n=-1), dict(n=2 ** 38), dict(param_dtype=3), dict(grad_dtype=3), dict(state_dtype=1), dict(copy=P, copy_dtype=0),
                dict(weight_decay=-0.1), dict(weight_decay=float("nan")), dict(lr_scale=float("inf")), dict(m_scale=P),
                dict(n=4, param=None), dict(n=4, state_dtype=3)):
        assert create(bad) == A, bad
    assert create(dict(n=4, param=P + 4)) == L
    assert lib.hashgrid_adamw_destroy(None) == hg.HASHGRID_OK
    f = ctypes.c_float
    assert lib.hashgrid_adamw_step(None, 1, None, f(1e-3), f(0.9), f(0.99), f(1e-8), 0, 0, None) == A
    with pytest.raises(hg.HashGridError):
        hg.AdamW([torch.zeros(4)], [torch.zeros(5)])
    with pytest.raises(hg.HashGridError):
        hg.AdamW([torch.zeros(4, 4).t()[:, :2]], [torch.zeros(8)])
    with pytest.raises(hg.HashGridError):
        hg.AdamW([torch.zeros(4)], [torch.zeros(4)], weight_decay=[0.0, 0.0])
    with pytest.raises(hg.HashGridError):
        hg.AdamW([torch.zeros(4)], [torch.zeros(4)], bits=16)


@pytest.mark.gpu
def test_gpu_refusals():
    p, g = torch.zeros(512, device="cuda"), torch.zeros(512, device="cuda")
    with pytest.raises(hg.HashGridError, match="overlap"):
        hg.AdamW([p, p], [g, torch.zeros_like(g)])
    with pytest.raises(hg.HashGridError, match="overlap"):
        hg.AdamW([p], [p])
    with pytest.raises(hg.HashGridError, match="aligned"):
        hg.AdamW([p[1:]], [g[:511]])
    opt = hg.AdamW([p], [g])
    for bad in (dict(step=0), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=0.0), dict(lr=float("nan"))):
        with pytest.raises(hg.HashGridError):
            opt.step(**{"step": 1, "lr": 1e-3, **bad})
    with pytest.raises(hg.HashGridError):
        opt.step(1, lr=1e-3, device_step=torch.ones(1, dtype=torch.int64))
    hg.AdamW([p[:0]], [g[:0]]).step(1, lr=1e-3)                     # a list without elements: nothing to do
