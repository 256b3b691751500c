"""The trainable head behind the hash-grid encoding, as operators: a linear layer with bias, activation and
residual in its epilogue (``Linear.forward``), its gradients (``Linear.backward``), and one AdamW step over all of
a model's tensors with states in 32 or 8 bits (``AdamW.step``).

``listed()`` and ``draw()`` give cases, ``prepare()`` their inputs, ``run()`` one pass in plain torch operations or,
with ``own``, through the package, ``work()`` the bytes and operations of a pass, ``exact()`` the results in 64 bits.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BLOCK = 256          # elements that share a scale in an 8-bit state
TOP = 448.0          # largest e4m3 value
MASK = 0xFFFFFFFF
LR, BETA1, BETA2, EPS, DECAY, STEP = 1e-3, 0.9, 0.99, 1e-8, 1e-2, 100


def listed():
    def forward(name, rows, into, out, dtype, act, residual, keep, pad=0, y="same"):
        return dict(name=name, op="forward", rows=rows, into=into, out=out, dtype=dtype, act=act, residual=residual,
                    keep=keep, pad=pad, y=y)

    def backward(name, rows, into, out, dtype, act, dw, pad=0):
        return dict(name=name, op="backward", rows=rows, into=into, out=out, dtype=dtype, act=act, dw=dw, pad=pad)

    def adamw(name, sizes, count, low, high, param, grad, state, copy, seed):
        return dict(name=name, op="adamw", sizes=sizes, count=count, low=low, high=high, param=param, grad=grad,
                    state=state, copy=copy, seed=seed)

    return [
        # one query point (or token) through a wide hidden layer: the latency of a call
        forward("forward_one_row", 1, 1024, 1024, "bf16", "silu", True, False),
        # a handful of rows through a large layer: the weights' bytes count
        forward("forward_rows16", 16, 4096, 4096, "bf16", "none", True, False),
        # the first layer of the head on 2^14 rays x 64 samples of the 16-level, 2-feature grid, kept for training
        forward("forward_encoding", 1 << 20, 32, 64, "bf16", "relu", False, True),
        # odd widths and padded rows
        forward("forward_odd", 10007, 333, 515, "f16", "gelu", True, False, pad=8),
        # a wide hidden layer with a residual on a large batch: the matrix product counts
        forward("forward_wide", 8192, 4096, 4096, "bf16", "gelu", True, False),
        # the 64-wide hidden layer's gradients on the same ray samples
        backward("backward_hidden", 1 << 20, 64, 64, "bf16", "relu", "f32"),
        # odd widths, padded rows, gradients in 16 bits
        backward("backward_odd", 4099, 173, 257, "f16", "silu", "same", pad=3),
        # a wide layer's gradients on a large batch
        backward("backward_wide", 8192, 2048, 4096, "bf16", "none", "f32"),
        # the 32 -> 64 -> 64 -> 4 head's six tensors, with the 16-bit copies its kernels read
        adamw("adamw_head", "head", 6, 4, 4096, "f32", "f32", "f32", "bf16", 0),
        # the 16 x 2^19 x 2 table with its head, trained densely
        adamw("adamw_table", "table", 7, 4, 1 << 24, "f32", "f32", "f32", "none", 0),
        # many tensors of uneven sizes, 16-bit parameters and gradients, 8-bit states, stochastic rounding
        adamw("adamw_many_8bit", "drawn 7", 160, 1, 1 << 20, "bf16", "bf16", "8bit", "none", 1234567),
        # a few large tensors, 32-bit parameters, 8-bit states rounded to nearest
        adamw("adamw_large_8bit", "drawn 8", 6, 1 << 22, 1 << 25, "f32", "f32", "8bit", "bf16", 0),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["forward", "backward", "adamw"])
    if op == "adamw":
        count = _log_int(rng, 1, 300)
        high = _log_int(rng, 1, max(1, (1 << 27) // (4 * count)) if count > 1 else 1 << 25)
        param = rng.choice(["f32", "bf16", "f16"])
        return dict(op=op, sizes="drawn %d" % rng.randrange(1 << 20), count=count, low=1, high=high, param=param,
                    grad=rng.choice(["f32", param]), state=rng.choice(["f32", "8bit"]),
                    copy=rng.choice(["none", "bf16", "f16"]) if param == "f32" else "none",
                    seed=rng.choice([0, rng.randrange(1, 1 << 32)]))
    while True:
        rows, into, out = _log_int(rng, 1, 1 << 20), _log_int(rng, 1, 4096), _log_int(rng, 1, 4096)
        if rng.random() < 0.5:  # widths that the tensor cores' tiles like
            into, out = -(-into // 16) * 16, -(-out // 16) * 16
        if rows * (into + out) <= 1 << 27 and rows * into * out <= (1 << 37 if op == "forward" else 1 << 36):
            break
    case = dict(op=op, rows=rows, into=into, out=out, dtype=rng.choice(["bf16", "f16"]),
                act=rng.choice(["none", "relu", "gelu", "silu"]), pad=rng.choice([0, 0, 8, rng.randrange(1, 40)]))
    if op == "forward":
        case.update(residual=rng.random() < 0.5, keep=rng.random() < 0.5, y=rng.choice(["same", "same", "f32"]))
    else:  # the derivative of a smooth activation is rounded to 16 bits, and so is what comes of it
        case.update(dw=rng.choice(["f32", "same"]) if case["act"] in ("none", "relu") else "same")
    return case


def _sizes(case):
    head = [64 * 32, 64, 64 * 64, 64, 4 * 64, 4]
    if case["sizes"] == "head":
        return head
    if case["sizes"] == "table":
        return [16 * (1 << 19) * 2] + head
    rng = random.Random(case["sizes"])
    return [_log_int(rng, case["low"], case["high"]) for _ in range(case["count"])]


def _rows(n, width, pad, dtype, gen, scale=1.0):
    """[n, width] values whose rows lie width + pad elements apart."""
    full = torch.randn(n, width + pad, device="cuda", generator=gen).mul_(scale).to(dtype)
    return full[:, :width]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    if case["op"] == "adamw":
        return _prepare_adamw(case, gen)
    t, rows, into, out = TYPES[case["dtype"]], case["rows"], case["into"], case["out"]
    s = dict(case=case, x=_rows(rows, into, case["pad"], t, gen),
             w=(torch.randn(out, into, device="cuda", generator=gen) / math.sqrt(into)).to(t))
    if case["op"] == "forward":
        y = t if case["y"] == "same" else torch.float32
        s["b"] = torch.randn(out, device="cuda", generator=gen) * 0.1
        s["r"] = _rows(rows, out, case["pad"], y, gen) if case["residual"] else None
        s["y"] = torch.empty(rows, out, device="cuda", dtype=y)
        s["z"] = torch.empty(rows, out, device="cuda", dtype=t) if case["keep"] else None
    else:
        s["z"] = None if case["act"] == "none" else torch.randn(rows, out, device="cuda", generator=gen).to(t)
        s["dy"] = _rows(rows, out, case["pad"], t, gen, 0.05)
        s["dx"] = torch.empty(rows, into, device="cuda", dtype=t)
        s["dw"] = torch.empty(out, into, device="cuda", dtype=t if case["dw"] == "same" else torch.float32)
        s["db"] = torch.empty(out, device="cuda")
    if own:
        import multiresolution_hash_grid_b200 as hg
        s["layer"] = hg.Linear(into, out, dtype={"bf16": hg.HASHGRID_BF16, "f16": hg.HASHGRID_F16}[case["dtype"]],
                               activation={"none": hg.HASHGRID_ACT_NONE, "relu": hg.HASHGRID_ACT_RELU,
                                           "gelu": hg.HASHGRID_ACT_GELU, "silu": hg.HASHGRID_ACT_SILU}[case["act"]])
        if case["op"] == "backward":
            s["work"] = s["layer"].workspace(rows, "cuda")
    return s


def _prepare_adamw(case, gen):
    """The tensors lie one behind the other in flat buffers, each from a multiple of 256 elements on (what lies
    between them is zero and stays zero); the lists hold the tensors themselves."""
    sizes = _sizes(case)
    blocks = [-(-n // BLOCK) for n in sizes]
    total = sum(blocks)
    start = [0]
    for k in blocks:
        start.append(start[-1] + k)
    sz = torch.tensor(sizes, device="cuda")
    reps = torch.tensor(blocks, device="cuda")
    index = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), reps, output_size=total)
    first = torch.tensor(start[:-1], device="cuda")
    at = (torch.arange(total, device="cuda") - first[index]) * BLOCK        # a block's first element in its tensor
    inside = (at[:, None] + torch.arange(BLOCK, device="cuda")) < sz[index][:, None]

    def normal():
        return torch.randn(total, BLOCK, device="cuda", generator=gen).mul_(inside)

    # gradients of tensors differ by orders of magnitude, a quarter of the elements were not reached
    size = (10.0 ** (torch.rand(len(sizes), device="cuda", generator=gen) * 3 - 4))[index][:, None]
    g = normal() * size * (torch.rand(total, BLOCK, device="cuda", generator=gen) > 0.25)
    p = (normal() * 0.05).to(TYPES[case["param"]])
    m, root = normal() * size * 0.3, normal().abs_() * size
    s = dict(case=case, index=index, at=at, p=p, g=g.to(TYPES[case["grad"]]),
             lr=torch.full((len(sizes),), 1.0, device="cuda"), decay=torch.full((len(sizes),), DECAY, device="cuda"))
    s["lr"][0] = 5.0        # the first tensor learns faster and does not decay, as a table does
    s["decay"][0] = 0.0
    if case["state"] == "f32":
        s["m"], s["v"] = m, root * root
    else:
        s["m"], s["ms"] = _nearest8(m)
        s["v"], s["vs"] = _nearest8(root)
    if case["copy"] != "none":
        s["copy"] = p.to(TYPES[case["copy"]])
    if own:
        import multiresolution_hash_grid_b200 as hg

        def parts(t):
            t = t.view(-1)
            return [t[o * BLOCK: o * BLOCK + n] for o, n in zip(start, sizes)]

        def scales(t):
            return [t[o:o + k] for o, k in zip(start, blocks)]

        s["opt"] = hg.AdamW(parts(s["p"]), parts(s["g"]), parts(s["m"]), parts(s["v"]),
                            block_scales=None if case["state"] == "f32" else
                            (scales(s["ms"]), scales(s["vs"])),
                            copies=parts(s["copy"]) if "copy" in s else None,
                            lr_scale=s["lr"].tolist(), weight_decay=s["decay"].tolist())
    return s


def _nearest8(x):
    """[blocks, 256] values as e4m3 and one scale a block."""
    top = x.abs().amax(1, keepdim=True)
    scale = top / torch.full_like(top, TOP)
    inverse = torch.where(top > 0, torch.full_like(top, TOP) / top, torch.zeros_like(top))
    return (x * inverse).to(torch.float8_e4m3fn), scale.view(-1)


def run(s):
    op = s["case"]["op"]
    if op == "adamw":
        return _run_adamw(s)
    if op == "forward":
        if own:
            s["layer"].forward(s["x"], s["w"], s["b"], residual=s["r"], y=s["y"], z=s["z"])
            return {"y": s["y"]} if s["z"] is None else {"y": s["y"], "z": s["z"]}
        z = s["x"].float() @ s["w"].float().t() + s["b"]
        y = _act(z, s["case"]["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        y = y.to(s["y"].dtype)
        return {"y": y} if s["z"] is None else {"y": y, "z": z.to(s["z"].dtype)}
    if own:
        s["layer"].backward(s["dy"], s["x"], s["w"], z=s["z"], dL_dx=s["dx"], dL_dw=s["dw"], dL_db=s["db"],
                            workspace=s["work"])
        return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}
    # sums over many rows lose digits in 32 bits
    wide = torch.float64 if s["case"]["rows"] > 16384 else torch.float32
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _slope(s["z"].float(), s["case"]["act"])
    dx = (dz @ s["w"].float()).to(s["dx"].dtype)
    dz = dz.to(wide)
    return {"dx": dx, "dw": (dz.t() @ s["x"].to(wide)).to(s["dw"].dtype), "db": dz.sum(0, dtype=torch.float64).float()}


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def _f32(x):
    """A number as the nearest 32-bit float."""
    return float(torch.tensor(x, dtype=torch.float32))


def _run_adamw(s):
    c = s["case"]
    if own:
        s["opt"].step(STEP, lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, seed=c["seed"])
    else:
        _plain_adamw(s, c)
    got = {k: s[k] for k in ("p", "m", "v", "ms", "vs", "copy") if k in s}
    return got


def _plain_adamw(s, c):
    b1, b2, lr = _f32(BETA1), _f32(BETA2), _f32(LR)
    c1, c2 = _f32(1 / (1 - b1 ** STEP)), _f32(1 / (1 - b2 ** STEP))
    g, p = s["g"].float(), s["p"].float()
    if c["state"] == "f32":
        m, v = s["m"], s["v"]
    else:
        m = s["m"].float() * s["ms"][:, None]
        root = s["v"].float() * s["vs"][:, None]
        v = root * root
    m = m * b1 + g * _f32(1 - b1)
    v = v * b2 + (g * g) * _f32(1 - b2)
    rate = (s["lr"] * lr)[s["index"]][:, None]
    keep = (1 - s["lr"].double() * lr * s["decay"].double()).float()[s["index"]][:, None]
    p = p * keep - rate * ((m * c1) / (torch.sqrt(v * c2) + _f32(EPS)))
    s["p"].copy_(p)
    if "copy" in s:
        s["copy"].copy_(p)
    if c["state"] == "f32":
        s["m"].copy_(m)
        s["v"].copy_(v)
        return
    root = torch.sqrt(v)
    if c["seed"] == 0:
        (m8, ms), (v8, vs) = _nearest8(m), _nearest8(root)
    else:
        h = _mixed(s, c["seed"])
        (m8, ms), (v8, vs) = _stochastic8(m, h & 0xFFFF), _stochastic8(root, h >> 16)
    least = torch.full_like(m, 2.0 ** -9)
    v8 = torch.where(root > 0, torch.maximum(v8.float(), least), torch.zeros_like(root)).to(torch.float8_e4m3fn)
    s["m"].copy_(m8)
    s["v"].copy_(v8)
    s["ms"].copy_(ms)
    s["vs"].copy_(vs)


def _mix(h):
    """A 32-bit integer mix on 64-bit tensors: xor of the high bits, two odd factors."""
    h = h ^ (h >> 16)
    h = (h * 0x7FEB352D) & MASK
    h = h ^ (h >> 15)
    h = (h * 0x846CA68B) & MASK
    return h ^ (h >> 16)


def _mixed(s, seed):
    """32 random bits for each element, from the seed, the step, the tensor's place in the list and the element's."""
    key = (s["index"] * 0xC2B2AE3D + (seed * 0x9E3779B1 + STEP * 0x85EBCA77 & MASK)) & MASK
    return _mix((s["at"][:, None] + torch.arange(BLOCK, device="cuda")) ^ _mix(key)[:, None])


def _stochastic8(x, r):
    """[blocks, 256] values as e4m3 and a scale a block, rounded up with the probability of the part cut off."""
    top = x.abs().amax(1, keepdim=True)
    scale = top / torch.full_like(top, TOP)
    y = x.abs() * torch.where(top > 0, torch.full_like(top, TOP) / top, torch.zeros_like(top))
    low = torch.where(y < 2.0 ** -6, torch.full_like(y, 2.0 ** -6), torch.zeros_like(y))
    bits = ((y + low).view(torch.int32) + (r * 16 + 8).to(torch.int32)) & ~0xFFFFF
    y = torch.minimum(bits.view(torch.float32) - low, torch.full_like(y, TOP))
    return torch.where(x < 0, -y, y).to(torch.float8_e4m3fn), scale.view(-1)


def work(case):
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        of = {"f32": 4, "bf16": 2, "f16": 2, "none": 0}
        state = 16 if case["state"] == "f32" else 4 + 16 / BLOCK
        return {"bytes": n * (2 * of[case["param"]] + of[case["grad"]] + state + of[case["copy"]]), "flops": 15 * n}
    rows, into, out = case["rows"], case["into"], case["out"]
    if case["op"] == "forward":
        y = 4 if case["y"] == "f32" else 2
        moved = 2 * rows * into + 2 * into * out + 4 * out + rows * out * (y * (2 if case["residual"] else 1) + (2 if case["keep"] else 0))
        return {"bytes": moved, "flops": 2 * rows * into * out}
    moved = 2 * rows * out * (1 if case["act"] == "none" else 2) + 4 * rows * into + 2 * into * out + (2 if case["dw"] == "same" else 4) * into * out + 4 * out
    return {"bytes": moved, "flops": 4 * rows * into * out}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(s, case)
    x, w = s["x"].double(), s["w"].double()
    normal = lambda t: 0.5 * torch.special.erfc(-t * 2 ** -0.5)  # noqa: E731
    if case["op"] == "forward":
        z = torch.nn.functional.linear(x, w, s["b"].double())
        y = {"none": lambda: z, "relu": lambda: z.clamp(min=0), "gelu": lambda: z * normal(z),
             "silu": lambda: z * torch.sigmoid(z)}[case["act"]]()
        y = y if s["r"] is None else y + s["r"].double()
        return {"y": y} if s["z"] is None else {"y": y, "z": z}
    dz = s["dy"].double()
    if case["act"] != "none":
        z = s["z"].double()
        dz = dz * {"relu": lambda: torch.heaviside(z, torch.zeros_like(z)),
                   "gelu": lambda: normal(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi),
                   "silu": lambda: torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)}[case["act"]]()
    return {"dx": torch.einsum("no,oi->ni", dz, w), "dw": torch.einsum("no,ni->oi", dz, x), "db": torch.einsum("no->o", dz)}


def _exact_adamw(s, case):
    b1, b2, lr, eps = (float(torch.tensor(v, dtype=torch.float32)) for v in (BETA1, BETA2, LR, EPS))
    g, p = s["g"].double(), s["p"].double()
    eight = case["state"] == "8bit"
    m0 = s["m"].double() * s["ms"].double().unsqueeze(1) if eight else s["m"].double()
    v0 = (s["v"].double() * s["vs"].double().unsqueeze(1)).square() if eight else s["v"].double()
    m = torch.lerp(g, m0, b1)
    v = torch.lerp(g.square(), v0, b2)
    rate = (lr * s["lr"].double())[s["index"]].unsqueeze(1)
    step = (m / (1 - b1 ** STEP)) / ((v / (1 - b2 ** STEP)).sqrt() + eps)
    new = p - rate * (step + s["decay"].double()[s["index"]].unsqueeze(1) * p)
    got = {"p": new, "m": m, "v": v}
    if "copy" in s:
        got["copy"] = new
    if not eight:
        return got
    if case["seed"] == 0:
        up_m = up_v = None
    else:
        h = torch.arange(BLOCK, device="cuda") + s["at"].unsqueeze(1)
        key = (case["seed"] * 0x9E3779B1 + STEP * 0x85EBCA77 + s["index"] * 0xC2B2AE3D) % (1 << 32)
        for a, f in ((16, 0x7FEB352D), (15, 0x846CA68B)):
            key = (key ^ (key >> a)) * f % (1 << 32)
        h = h ^ (key ^ (key >> 16)).unsqueeze(1)
        for a, f in ((16, 0x7FEB352D), (15, 0x846CA68B)):
            h = (h ^ (h >> a)) * f % (1 << 32)
        h = h ^ (h >> 16)
        up_m, up_v = ((h % 65536) * 16 + 8) / 2.0 ** 20, ((h // 65536) * 16 + 8) / 2.0 ** 20
    for name, t, up in (("m", m, up_m), ("v", v.sqrt(), up_v)):
        top = t.abs().amax(1, keepdim=True)
        y = t.abs() / torch.where(top > 0, top, 1.0) * TOP
        quantum = torch.exp2(torch.log2(y.clamp(min=2.0 ** -6)).floor() - 3)
        y = ((torch.round(y / quantum) if up is None else torch.floor(y / quantum + up)) * quantum).clamp(max=TOP)
        if name == "v":
            y = torch.where(t > 0, y.clamp(min=2.0 ** -9), 0.0)
        got[name], got[name + "s"] = torch.sign(t) * y, (top / TOP).squeeze(1)
    return got
