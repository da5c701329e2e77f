"""Operators around a block of layers that runs in 8 bits, as they are measured:
products of 8-bit integers with a scale per token and channel and the
quantisation that makes them, the norms after and before a block fused with its
gate and residual scale (forward and backward), and the use of activations that
are kept in 8 bits between the two passes.

``run`` computes them in their plain form (elementary torch operations in 32
bits, rounded once at the end; 64 bits decide the rounding to integers), or,
where ``own`` is true, through ``fp32_gemm_08_amd``.  ``exact`` computes them
from their definitions in 64 bits.

Definitions.
  i8_gemm      C[m][n] = sA[m] * sB[n] * sum_k qA[m][k] * qB[n][k], the sum in integers.
  i8_quantize  a = max(max|x|, 2^-90) over a row, s = a / 127, q = 127 x / a to the
               nearest integer, ties to even.
  block_norm   z = o * rstd_post * w_post,  rstd_post = 1/sqrt(mean(o^2) + eps)
               h = alpha * x + gate * z,  y = h * rstd * w,  rstd = 1/sqrt(mean(h^2) + eps)
               gate has a row for every rows/G consecutive rows of x.  y in 8 bits (e4m3)
               for the next product, h and o in 8 bits for the backward pass: blocks of 128
               values of a row, a = max(max|x|, 2^-90), s = a / 448, q = x * (448 / a)
               rounded, scales in an array (ceil(cols/128), rows).
  block_norm_bwd  n = h * rstd,  g = dy * w,  d = rstd * (g - n * mean(g * n)) + dh
               dx = alpha * d,  dw = sum of dy * n,  dgate = sum over a gate's rows of d * z
               m = o * rstd_post,  dw_post = sum of gate * d * m,  p = gate * d * w_post
               do = rstd_post * (p - m * mean(p * m))
               with h and o in 16 or 32 bits or as kept in 8 bits.
  requantize   X = q * s, kept with blocks along its rows, to 8 bits with blocks along its
               columns, transposed: the operand of a product that sums over the rows.
"""
import torch

own = False

BLOCK = 128
FLOOR = 2.0 ** -90
EPS = 1e-6
E4M3 = torch.float8_e4m3fn
LARGEST = 448.0
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
WORKSPACE = 64 << 20   # bytes a program lends to the calls that take a workspace


def _gemm(name, m, n, k, out="bf16", pad=True):
    c = {"op": "i8_gemm", "m": m, "n": n, "k": k, "out": out, "pad": pad}
    return dict(c, name=name) if name else c


def _quantize(name, rows, cols, type):
    c = {"op": "i8_quantize", "rows": rows, "cols": cols, "type": type}
    return dict(c, name=name) if name else c


def _norm(name, rows, cols, type, groups=1, alpha=1.0, post=True, keep=True):
    c = {"op": "block_norm", "rows": rows, "cols": cols, "type": type, "groups": groups, "alpha": alpha, "post": post, "keep": keep}
    return dict(c, name=name) if name else c


def _norm_bwd(name, rows, cols, type, groups=1, alpha=1.0, post=True, kept=True):
    c = {"op": "block_norm_bwd", "rows": rows, "cols": cols, "type": type, "groups": groups, "alpha": alpha, "post": post, "kept": kept}
    return dict(c, name=name) if name else c


def _requantize(name, rows, cols, pad=True):
    c = {"op": "requantize", "rows": rows, "cols": cols, "pad": pad}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token through a square layer: latency and the weights' bytes count
        _gemm("i8 gemm 1 token", 1, 4096, 4096),
        # a batch of 64 single tokens through a layer that widens: the weights' bytes count
        _gemm("i8 gemm 64 tokens", 64, 16384, 4096),
        # a long prompt: the matrix cores count
        _gemm("i8 gemm 8192 tokens", 8192, 8192, 8192),
        # odd sizes, rows packed without padding, so that they start at every byte
        _gemm("i8 gemm odd packed", 1000, 1017, 999, out="f32", pad=False),
        # one token's activations before a product
        _quantize("i8 quantize 1 token", 1, 4096, "bf16"),
        # those of a long prompt
        _quantize("i8 quantize 16384 tokens", 16384, 4096, "bf16"),
        # one token between two blocks, nothing kept
        _norm("block norm 1 token", 1, 4096, "bf16", keep=False),
        # a training batch of 8 sequences with a gate each, h and o kept in 8 bits
        _norm("block norm 16384 tokens", 16384, 4096, "bf16", groups=8),
        # its backward pass from what was kept
        _norm_bwd("block norm backward 16384", 16384, 4096, "bf16", groups=8),
        # odd sizes in 32 bits, a gate per channel, a scaled residual, nothing kept in 8 bits
        _norm_bwd("block norm backward odd", 1000, 1017, "f32", alpha=0.75, kept=False),
        # a training batch's kept activations for the weight's gradient
        _requantize("requantize 16384 tokens", 16384, 4096),
        # odd sizes, packed
        _requantize("requantize odd packed", 1000, 1017, pad=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def _size(rng, lo, hi, step):
    """Over the logarithm of lo..hi; half the time a multiple of `step`."""
    v = _log(rng, lo, hi)
    return max(step, v // step * step) if rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["i8_gemm", "i8_gemm", "i8_quantize", "block_norm", "block_norm_bwd", "requantize"])
    if op == "i8_gemm":
        n, k = _size(rng, 64, 16384, 128), _size(rng, 32, 16384, 128)
        m = min(_size(rng, 1, 16384, 1), (1 << 39) // (n * k))
        return _gemm(None, m, n, k, out=rng.choice(["bf16", "bf16", "f16", "f32"]), pad=rng.random() < 0.75)
    cols = _size(rng, 64, 16384, 128)
    rows = min(_size(rng, 1, 65536, 1), (1 << 26) // cols)
    type = rng.choice(["bf16", "bf16", "f32", "f16"])
    if op == "i8_quantize":
        return _quantize(None, rows, cols, type)
    if op == "requantize":
        return _requantize(None, rows, cols, pad=rng.random() < 0.75)
    groups = rng.choice([1, 1, _log(rng, 1, 64), rows])
    groups = max(g for g in range(1, min(groups, rows) + 1) if rows % g == 0) if groups < rows else rows
    make = _norm if op == "block_norm" else _norm_bwd
    return make(None, rows, cols, type, groups, rng.choice([1.0, 1.0, 0.75, 2.5]), rng.random() < 0.75, rng.random() < 0.6)


# ---------------------------------------------------------------- the plain forms

def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _quantize_rows(x):
    """x in 32 bits -> e4m3 values in blocks along the rows, and their scales."""
    r, k = x.shape
    kb = _blocks(k)
    p = x.new_zeros(r, kb * BLOCK)
    p[:, :k] = x
    a = p.view(r, kb, BLOCK).abs().amax(2).clamp_min(FLOOR)
    q = (x * (LARGEST / a).repeat_interleave(BLOCK, 1)[:, :k]).to(E4M3)
    return q, (a / LARGEST).t().contiguous()


def _values(q, s):
    """What e4m3 values and their scales stand for, in 32 bits."""
    return q.float() * s.t().repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _gate_rows(st, x):
    """The gate's row for each row of x, in x's type."""
    return st["gate"].to(x.dtype).repeat_interleave(x.shape[0] // st["case"]["groups"], 0)


def _run_plain(st):
    c = st["case"]
    if c["op"] == "i8_gemm":
        p = st["A"].float() @ st["B"].float().t()
        return {"C": (p * st["SA"][:, None] * st["SB"]).to(TYPES[c["out"]])}
    if c["op"] == "i8_quantize":
        x = st["X"].double()
        a = x.abs().amax(1, keepdim=True).clamp_min(FLOOR)
        return {"Q": (127.0 * x / a).round().to(torch.int8), "S": a[:, 0].float() / 127.0}
    if c["op"] == "requantize":
        q, s = _quantize_rows(_values(st["Q"], st["S"]).t().contiguous())
        return {"QT": q, "ST": s}
    if c["op"] == "block_norm":
        t, o = TYPES[c["type"]], st["O"].float()
        out, z = {}, o
        if c["post"]:
            out["rstd_post"] = torch.rsqrt((o * o).mean(1) + EPS)
            z = o * out["rstd_post"][:, None] * st["w_post"].float()
        h = c["alpha"] * st["X"].float() + _gate_rows(st, o) * z
        out["rstd"] = torch.rsqrt((h * h).mean(1) + EPS)
        out["H"] = h.to(t)
        out["Q"], out["S"] = _quantize_rows(h * out["rstd"][:, None] * st["W"].float())
        if c["keep"]:
            out["H8"], out["SH"] = _quantize_rows(h)
            out["O8"], out["SO"] = _quantize_rows(o)
        return out
    t, dy, gate = TYPES[c["type"]], st["DY"].float(), _gate_rows(st, st["DY"].float())
    h, o = (_values(st["H"], st["SH"]), _values(st["O"], st["SO"])) if c["kept"] else (st["H"].float(), st["O"].float())
    rstd = st["rstd"][:, None]
    n, g = h * rstd, dy * st["W"].float()
    d = rstd * (g - n * (g * n).mean(1, keepdim=True)) + st["DH"].float()
    out = {"DX": (c["alpha"] * d).to(t), "DW": (dy * n).sum(0)}
    z, do = o, gate * d
    if c["post"]:
        rstd, w = st["rstd_post"][:, None], st["w_post"].float()
        m, p = o * rstd, do * w
        z = m * w
        out["DW_post"] = (do * m).sum(0)
        do = rstd * (p - m * (p * m).mean(1, keepdim=True))
    out["DO"] = do.to(t)
    out["DGate"] = (d * z).view(c["groups"], -1, d.shape[1]).sum(1)
    return out


# ---------------------------------------------------------------- the framework's calls

def _run_own(st):
    import fp32_gemm_08_amd as lib

    c, o = st["case"], st["out"]
    if c["op"] == "i8_gemm":
        lib.i8_gemm(st["A"], st["SA"], st["B"], st["SB"], o["C"], workspace=st["workspace"])
    elif c["op"] == "i8_quantize":
        lib.i8_quantize(st["X"], o["Q"], o["S"])
    elif c["op"] == "requantize":
        lib.f8_requantize(st["Q"], st["S"], o["QT"], o["ST"])
    elif c["op"] == "block_norm":
        lib.block_norm(st["X"], st["O"], st["W"], EPS, w_post=st.get("w_post"), gate=st["gate"], alpha=c["alpha"], H=o["H"],
                       Q=o["Q"], S=o["S"], H8=o.get("H8"), SH=o.get("SH"), O8=o.get("O8"), SO=o.get("SO"), rstd=o["rstd"],
                       rstd_post=o.get("rstd_post"))
    else:
        lib.block_norm_backward(st["DY"], st["H"], st["O"], st["W"], st["rstd"], o["DX"], o["DO"], SH=st.get("SH"),
                                SO=st.get("SO"), w_post=st.get("w_post"), rstd_post=st.get("rstd_post"), gate=st["gate"],
                                alpha=c["alpha"], dH=st["DH"], dW=o["DW"], dW_post=o.get("DW_post"), dGate=o["DGate"],
                                workspace=st["workspace"])
    return o


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- inputs

def _activations(g, rows, cols, type):
    """Normal values whose columns differ in size, a few of them far larger than the rest."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    size = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    size = torch.where(torch.rand(cols, generator=g, device="cuda") < 0.002, size * 30, size)
    return (x * size).to(type)


def _gradients(g, rows, cols, type):
    """Small values whose rows differ in size."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    return (x * (1e-1 * torch.exp(torch.randn(rows, 1, generator=g, device="cuda")))).to(type)


def _empty(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _bytes_empty(rows, cols, dtype, pad=True):
    """Rows that start on 16-byte boundaries, or packed ones."""
    ld = (cols + 15) // 16 * 16 if pad else cols
    return torch.zeros(rows, ld, dtype=torch.uint8, device="cuda").view(dtype)[:, :cols]


def _held(q, pad=True):
    out = _bytes_empty(q.shape[0], q.shape[1], q.dtype, pad)
    out.view(torch.uint8).copy_(q.view(torch.uint8))
    return out


def _i8_operand(x, pad):
    a = x.abs().amax(1, keepdim=True).clamp_min(FLOOR)
    return _held((x * (127.0 / a)).round().to(torch.int8), pad), (a / 127.0)[:, 0].contiguous()


def _weights(g, n, type):
    return (1.0 + 0.1 * torch.randn(n, generator=g, device="cuda")).to(type)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": case}
    if case["op"] == "i8_gemm":
        m, n, k = case["m"], case["n"], case["k"]
        st["A"], st["SA"] = _i8_operand(_activations(g, m, k, torch.float32), case["pad"])
        st["B"], st["SB"] = _i8_operand(0.02 * torch.randn(n, k, generator=g, device="cuda"), case["pad"])
        st["out"] = {"C": _empty(m, n, dtype=TYPES[case["out"]])}
        st["workspace"] = _empty(WORKSPACE, dtype=torch.uint8)
        return st
    r, k = case["rows"], case["cols"]
    kb = _blocks(k)
    if case["op"] == "i8_quantize":
        st["X"] = _activations(g, r, k, TYPES[case["type"]])
        st["out"] = {"Q": _bytes_empty(r, k, torch.int8), "S": _empty(r)}
        return st
    if case["op"] == "requantize":
        q, st["S"] = _quantize_rows(_activations(g, r, k, torch.float32))
        st["Q"] = _held(q, case["pad"])
        st["out"] = {"QT": _bytes_empty(k, r, E4M3, case["pad"]), "ST": _empty(_blocks(r), k)}
        return st
    t = TYPES[case["type"]]
    st["W"] = _weights(g, k, t)
    if case["post"]:
        st["w_post"] = _weights(g, k, t)
    st["gate"] = (0.5 * torch.randn(case["groups"], k, generator=g, device="cuda")).to(t)
    o = _activations(g, r, k, torch.float32)
    if case["op"] == "block_norm":
        st["X"], st["O"] = _activations(g, r, k, t), o.to(t)
        out = {"H": _empty(r, k, dtype=t), "Q": _bytes_empty(r, k, E4M3), "S": _empty(kb, r), "rstd": _empty(r)}
        if case["post"]:
            out["rstd_post"] = _empty(r)
        if case["keep"]:
            out["H8"], out["SH"] = _bytes_empty(r, k, E4M3), _empty(kb, r)
            out["O8"], out["SO"] = _bytes_empty(r, k, E4M3), _empty(kb, r)
        st["out"] = out
        return st
    h = _activations(g, r, k, torch.float32)
    st["rstd"] = torch.rsqrt(h.square().mean(1) + EPS)
    if case["post"]:
        st["rstd_post"] = torch.rsqrt(o.square().mean(1) + EPS)
    if case["kept"]:
        q, st["SH"] = _quantize_rows(h)
        st["H"] = _held(q)
        q, st["SO"] = _quantize_rows(o)
        st["O"] = _held(q)
    else:
        st["H"], st["O"] = h.to(t), o.to(t)
    st["DY"], st["DH"] = _gradients(g, r, k, t), _gradients(g, r, k, t)
    st["out"] = {"DX": _empty(r, k, dtype=t), "DO": _empty(r, k, dtype=t), "DW": _empty(k), "DGate": _empty(case["groups"], k)}
    if case["post"]:
        st["out"]["DW_post"] = _empty(k)
    st["workspace"] = _empty(WORKSPACE, dtype=torch.uint8)
    return st


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "i8_gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + m * n * BYTES[case["out"]] + 4 * (m + n), "flops": 2 * m * n * k}
    r, k = case["rows"], case["cols"]
    held = r * k + 4 * r * _blocks(k)   # in 8 bits with row blocks
    if case["op"] == "i8_quantize":
        return {"bytes": r * k * (BYTES[case["type"]] + 1) + 4 * r, "flops": 3 * r * k}
    if case["op"] == "requantize":
        return {"bytes": held + r * k + 4 * k * _blocks(r), "flops": 3 * r * k}
    t, vectors = BYTES[case["type"]], 1 + case["post"]
    if case["op"] == "block_norm":
        return {"bytes": 3 * t * r * k + held * (1 + 2 * case["keep"]) + t * k * (vectors + case["groups"]) + 4 * r * vectors,
                "flops": (9 + 4 * case["post"] + 4 * case["keep"]) * r * k}
    return {"bytes": 4 * t * r * k + 2 * (held if case["kept"] else t * r * k) + t * k * (vectors + case["groups"]) +
            4 * k * (vectors + case["groups"]) + 4 * r * vectors, "flops": (13 + 10 * case["post"]) * r * k}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_rows(x):
    """e4m3 values in row blocks before they are rounded, and scales; x in 64 bits."""
    big = torch.empty_like(x)
    r, k = x.shape
    scales = torch.empty(_blocks(k), r, dtype=torch.float64, device=x.device)
    for j in range(_blocks(k)):
        cols = slice(j * BLOCK, min(k, (j + 1) * BLOCK))
        top = torch.maximum(x[:, cols].max(1).values, -x[:, cols].min(1).values)
        scales[j] = torch.clamp(top, min=FLOOR) / LARGEST
        big[:, cols] = x[:, cols] / scales[j][:, None]
    return big, scales


def _exact_values(q, s):
    v = q.to(torch.float64)
    for j in range(s.shape[0]):
        v[:, j * BLOCK:(j + 1) * BLOCK] *= s[j].double()[:, None]
    return v


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "i8_gemm":
        c = torch.mm(st["A"].double(), st["B"].double().t().contiguous())
        return {"C": c.mul_(st["SA"].double()[:, None]).mul_(st["SB"].double()[None, :])}
    if case["op"] == "i8_quantize":
        x = st["X"].double()
        return {"Q": None, "S": torch.maximum(x.max(1).values, -x.min(1).values).clamp(min=FLOOR) / 127}
    if case["op"] == "requantize":
        q, s = _exact_rows(_exact_values(st["Q"], st["S"]).t().contiguous())
        return {"QT": q, "ST": s}
    per_gate = case["rows"] // case["groups"]
    gate = st["gate"].double()[torch.arange(case["rows"], device="cuda") // per_gate]
    w, alpha = st["W"].double(), case["alpha"]
    if case["op"] == "block_norm":
        o = st["O"].double()
        out, h = {}, alpha * st["X"].double()
        if case["post"]:
            out["rstd_post"] = (o.pow(2).sum(1) / o.shape[1] + EPS).pow(-0.5)
            h += gate * (st["w_post"].double() * o * out["rstd_post"][:, None])
        else:
            h += gate * o
        out["H"], out["rstd"] = h, (h.pow(2).sum(1) / h.shape[1] + EPS).pow(-0.5)
        out["Q"], out["S"] = _exact_rows(out["rstd"][:, None] * h * w)
        if case["keep"]:
            out["H8"], out["SH"] = _exact_rows(h)
            out["O8"], out["SO"] = _exact_rows(o)
        return out
    h, o = ((_exact_values(st["H"], st["SH"]), _exact_values(st["O"], st["SO"])) if case["kept"]
            else (st["H"].double(), st["O"].double()))
    dy, rstd, cols = st["DY"].double(), st["rstd"].double()[:, None], case["cols"]
    # d_j = rstd w_j dy_j - rstd^3 h_j / cols * sum_i dy_i w_i h_i + dh_j
    d = rstd * w * dy - rstd.pow(3) * h * (dy * w * h).sum(1, keepdim=True) / cols + st["DH"].double()
    out = {"DX": alpha * d, "DW": (dy * h * rstd).sum(0)}
    back = gate * d
    if case["post"]:
        rp, wp = st["rstd_post"].double()[:, None], st["w_post"].double()
        out["DW_post"] = (back * o * rp).sum(0)
        out["DO"] = rp * wp * back - rp.pow(3) * o * (back * wp * o).sum(1, keepdim=True) / cols
        z = o * rp * wp
    else:
        out["DO"], z = back, o
    at = torch.arange(case["rows"], device="cuda") // per_gate
    out["DGate"] = torch.zeros(case["groups"], cols, dtype=torch.float64, device="cuda").index_add_(0, at, d * z)
    return out
