"""Timing cases for the operators on weights held in four bits.

Five operators that serve and fine-tune the sparse FFN layer, and the dense
projections beside it, from weights in 4 bits with group scales:

* fp4_quant: a weight matrix in 4 bits (e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and
  their negatives) with one bfloat16 scale for each group of 32, 64 or 128
  columns of a row.
* fp4_dequant: the bfloat16 or float32 matrix that such a matrix stands for.
* fp4_matmul: out = X W^T for any number of tokens, one upwards.
* fp4_matmul_dx: its gradient dX = dY W (the weights are frozen).
* fp4_decode_fwd: the whole sparse layer y = (ReLU(X Wg^T) * (X Wu^T)) Wd for
  at most 64 tokens, each matrix in 4 bits.

A 4-bit matrix [rows][cols] is q [rows][cols rounded up to 128, / 2] bytes
(column 2b in the low half of byte b; zeros in the columns past `cols`) and
scale [columns rounded up to 128, / group][rows]. A scale is amax / 6, amax held
within [2^-64, 2^127], rounded to six significant bits, so that value times
scale is a bfloat16 number.

`run` computes an operator in plain torch operations in 32 bits, or, where
`own` is true, by the library's call.
"""
import math

import torch

own = False

DEV = "cuda:0"
AMAX_MIN, AMAX_MAX = 2.0 ** -64, 2.0 ** 127
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SZ = {"f32": 4, "bf16": 2}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# the layers of synth.py: 2048 -> 5632 (8192 tokens), 1024 -> 2816 (4096
# tokens), 2304 -> 6144 (decoding, 1 to 64 tokens), 256 -> 1024 (64 tokens, float32)
MOST_FLOPS = 2.0 * 8192 * 5632 * 2048  # the largest listed products
MOST_ELEMS = 32768 * 4096              # the largest listed weights
MOST_QUANT = 5632 * 2048               # the largest listed quantised matrix


def listed():
    return [
        # a float32 master after an optimizer step, and what the forward then sees
        {"name": "quant-master", "op": "fp4_quant", "R": 5632, "C": 2048, "x": "f32",
         "group": 128, "out": "bf16"},
        # a checkpoint's matrix with a width that is no multiple of anything
        {"name": "quant-odd", "op": "fp4_quant", "R": 2811, "C": 999, "x": "bf16", "group": 32,
         "out": "f32"},
        # the bfloat16 copy of the gate's weights that a long prefill multiplies by
        {"name": "dequant-prefill", "op": "fp4_dequant", "R": 6144, "C": 2304, "group": 64,
         "out": "bf16"},
        # the small layer's float32 copy
        {"name": "dequant-tiny", "op": "fp4_dequant", "R": 1024, "C": 256, "group": 32,
         "out": "f32"},
        # one decoded token
        {"name": "mm4-decode-1", "op": "fp4_matmul", "T": 1, "N": 6144, "K": 2304, "group": 128,
         "x": "bf16", "out": "bf16"},
        # a few sequences, the largest weights the layer takes, float32 results
        {"name": "mm4-wide-8", "op": "fp4_matmul", "T": 8, "N": 32768, "K": 4096, "group": 32,
         "x": "bf16", "out": "f32"},
        # ragged everywhere, float32 activations
        {"name": "mm4-ragged", "op": "fp4_matmul", "T": 333, "N": 2811, "K": 1090, "group": 64,
         "x": "f32", "out": "f32"},
        # a prompt batch
        {"name": "mm4-prefill", "op": "fp4_matmul", "T": 8192, "N": 5632, "K": 2048, "group": 128,
         "x": "bf16", "out": "bf16"},
        # the gradient of a training batch through frozen weights
        {"name": "dx4-train", "op": "fp4_matmul_dx", "T": 8192, "N": 5632, "K": 2048,
         "group": 128, "x": "bf16", "out": "bf16"},
        # the gradient of a few tokens (a prompt vector being tuned)
        {"name": "dx4-few", "op": "fp4_matmul_dx", "T": 17, "N": 6144, "K": 2304, "group": 64,
         "x": "f32", "out": "f32"},
        # one decoded token through the sparse layer, 1% of its gates open
        {"name": "layer4-1", "op": "fp4_decode_fwd", "T": 1, "d": 2304, "f": 6144, "group": 128,
         "x": "bf16", "density": 0.01},
        # a full decoding batch
        {"name": "layer4-64", "op": "fp4_decode_fwd", "T": 64, "d": 2304, "f": 6144, "group": 32,
         "x": "bf16", "density": 0.01},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width over [lo, hi]: a multiple of 64, of 8, or any number."""
    v = _log(rng, lo, hi)
    m = rng.choice((64, 64, 8, 1))
    return min(hi, max(lo, v // m * m))


def draw(rng):
    op = rng.choice(("fp4_quant", "fp4_dequant", "fp4_matmul", "fp4_matmul", "fp4_matmul_dx",
                     "fp4_decode_fwd"))
    group, two = rng.choice((32, 64, 128)), ("f32", "bf16")
    if op in ("fp4_quant", "fp4_dequant"):
        C = _width(rng, 64, 8192)
        c = {"op": op, "R": min(_log(rng, 1, 32768), MOST_QUANT // C), "C": C, "group": group,
             "out": rng.choice(two)}
        return c if op == "fp4_dequant" else {**c, "x": rng.choice(two)}
    if op == "fp4_decode_fwd":
        d, f = 64 * _log(rng, 1, 64), 128 * _log(rng, 1, 64)
        return {"op": op, "T": _log(rng, 1, 64), "d": d, "f": f, "group": group,
                "x": rng.choice(two), "density": rng.choice((0.005, 0.01, 0.02, 0.05, 0.2))}
    K = _width(rng, 64, 8192)
    N = min(_width(rng, 64, 32768), MOST_ELEMS // K)
    T = max(1, min(_log(rng, 1, 8192), int(MOST_FLOPS / (2.0 * N * K))))
    return {"op": op, "T": T, "N": N, "K": K, "group": group, "x": rng.choice(two),
            "out": rng.choice(two)}


# ---------------------------------------------------------------- inputs
def _normal(shape, g, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale


def _pad128(n):
    return -(-n // 128) * 128


def _weights(rows, cols, g, scale):
    """Weights: normal, rows of different sizes, a few large ones."""
    w = _normal((rows, cols), g, scale) * torch.exp(0.3 * _normal((rows, 1), g))
    return torch.where(torch.rand((rows, cols), generator=g, device=DEV) < 1e-3, w * 8.0, w)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    op, group = case["op"], case["group"]
    if op in ("fp4_quant", "fp4_dequant"):
        R, C = case["R"], case["C"]
        w = _weights(R, C, g, 0.02)
        if R > 300:
            w[5::97] = 0  # pruned rows
        if op == "fp4_quant":
            s["w_"] = w.to(DT[case["x"]])
        else:
            s["w4_"] = _quant_plain(w, group)
    elif op == "fp4_decode_fwd":
        T, d, f = case["T"], case["d"], case["f"]
        x = _normal((T, d), g)
        x[:, 0] = 1.0  # the constant that the gates' offset multiplies
        s["x_"] = x.to(DT[case["x"]])
        wg, wu = (_normal((f, d), g, d ** -0.5) for _ in range(2))
        wg[:, 0] = math.sqrt(2.0) * float(torch.erfinv(torch.tensor(2.0 * case["density"] - 1.0)))
        wd = _normal((f, d), g, f ** -0.5)
        s["wg4_"], s["wu4_"], s["wd4_"] = (_quant_plain(w, group) for w in (wg, wu, wd))
    else:
        T, N, K = case["T"], case["N"], case["K"]
        s["w4_"] = _quant_plain(_weights(N, K, g, K ** -0.5), group)
        if op == "fp4_matmul":
            s["x_"] = _normal((T, K), g).to(DT[case["x"]])
        else:
            s["dy_"] = _normal((T, N), g, 1e-2).to(DT[case["x"]])
    return s


# ---------------------------------------------------------------- plain forms
def _quant_plain(w, group):
    """float32 [rows][cols] -> (q [rows][cols up to 128, / 2], scale [groups][rows])."""
    rows, cols = w.shape
    cp = _pad128(cols)
    p = torch.zeros((rows, cp), dtype=torch.float32, device=w.device)
    p[:, :cols] = w
    p = p.view(rows, cp // group, group)
    m, e = torch.frexp(p.abs().amax(2).double().clamp(AMAX_MIN, AMAX_MAX) / 6.0)
    s = torch.ldexp(torch.round(m * 64.0) / 64.0, e).to(torch.bfloat16)
    y = p.double() / s.double()[:, :, None]  # 64 bits: the quotient next to a tie
    a = y.abs()
    # codes 0 to 7: steps of 0.5 below 2, of 1 below 4, of 2 above
    c = torch.where(a < 2, torch.round(2 * a),
                    torch.where(a < 4, torch.round(a) + 2, torch.round(a / 2) + 4)).clamp(max=7)
    c = (c.to(torch.uint8) + 8 * (y < 0).to(torch.uint8)).view(rows, cp)
    return c[:, ::2] + 16 * c[:, 1::2], s.t().contiguous()


def _dequant_plain(w4, cols, group):
    """The float32 values that a 4-bit matrix stands for."""
    q, s = w4
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=q.device)
    c = torch.stack((q & 15, q >> 4), 2).view(q.shape[0], -1)
    v = table[c.int()].view(q.shape[0], -1, group) * s.t().float()[:, :, None]
    return v.view(q.shape[0], -1)[:, :cols]


def _plain(s):
    op, group = s["op"], s["group"]
    if op == "fp4_quant":
        q, scale = _quant_plain(s["w_"].float(), group)
        return {"values": _dequant_plain((q, scale), s["C"], group).to(DT[s["out"]]),
                "scale": scale}
    if op == "fp4_dequant":
        return _dequant_plain(s["w4_"], s["C"], group).to(DT[s["out"]])
    if op == "fp4_decode_fwd":
        x = s["x_"].float()
        wg, wu, wd = (_dequant_plain(s[k], s["d"], group) for k in ("wg4_", "wu4_", "wd4_"))
        return (torch.relu(x @ wg.t()) * (x @ wu.t())) @ wd
    w = _dequant_plain(s["w4_"], s["K"], group)
    if op == "fp4_matmul":
        return (s["x_"].float() @ w.t()).to(DT[s["out"]])
    return (s["dy_"].float() @ w).to(DT[s["out"]])


# ---------------------------------------------------------------- one pass
def run(s):
    if not own:
        return _plain(s)
    from activation_sparse_ffn_gemm_amd import _lib as tw
    op, group = s["op"], s["group"]
    if op == "fp4_quant":
        w4 = tw.fp4_quant(s["w_"], group=group)
        return {"values": tw.fp4_dequant(w4, out_dtype=DT[s["out"]]), "scale": w4.scale}
    if op == "fp4_dequant":
        return tw.fp4_dequant(tw.Fp4(*s["w4_"], cols=s["C"], group=group),
                              out_dtype=DT[s["out"]])
    if op == "fp4_decode_fwd":
        return tw.fp4_decode_fwd(s["x_"], *(tw.Fp4(*s[k], cols=s["d"], group=group)
                                            for k in ("wg4_", "wu4_", "wd4_")))
    w4 = tw.Fp4(*s["w4_"], cols=s["K"], group=group)
    if op == "fp4_matmul":
        return tw.fp4_matmul(s["x_"], w4, out_dtype=DT[s["out"]])
    return tw.fp4_matmul_dx(s["dy_"], w4, out_dtype=DT[s["out"]])


# ---------------------------------------------------------------- work
def _fp4_bytes(rows, cols, group):
    return rows * _pad128(cols) // 2 + 2 * rows * _pad128(cols) // group


def work(case):
    op, group = case["op"], case["group"]
    if op in ("fp4_quant", "fp4_dequant"):
        R, C = case["R"], case["C"]
        by = _fp4_bytes(R, C, group) + R * C * SZ[case["out"]]
        if op == "fp4_quant":  # the codes are written and read back
            by += _fp4_bytes(R, C, group) + R * C * SZ[case["x"]]
        return {"bytes": by, "flops": (8 if op == "fp4_quant" else 2) * R * C}
    if op == "fp4_decode_fwd":
        T, d, f = case["T"], case["d"], case["f"]
        # every row of Wg, and the rows of Wu and Wd that some token's gate opens
        touched = f * (1.0 - (1.0 - case["density"]) ** T)
        by = _fp4_bytes(1, d, group) * (f + 2 * touched) + T * d * (SZ[case["x"]] + 4)
        return {"bytes": int(by), "flops": 2.0 * T * f * d * (1 + 2 * case["density"])}
    T, N, K = case["T"], case["N"], case["K"]
    i, o = (K, N) if op == "fp4_matmul" else (N, K)
    by = _fp4_bytes(N, K, group) + T * i * SZ[case["x"]] + T * o * SZ[case["out"]]
    return {"bytes": by, "flops": 2.0 * T * N * K}


# ---------------------------------------------------------------- 64 bits
def _scale_exact(amax):
    """amax / 6 to six significant bits, in float64: nearest, ties to even, on
    the number's own bits (52 of them after the first, five are kept)."""
    u = (amax.clamp(min=AMAX_MIN, max=AMAX_MAX) / 6.0).view(torch.int64)
    u = u + (1 << 46) - 1 + ((u >> 47) & 1)
    return ((u >> 47) << 47).view(torch.float64)


def _quant_exact(w, group):
    """Scales and values of float64 w: |w| against each border between two
    neighbouring values, a border's own place going to the even one."""
    rows, cols = w.shape
    n = _pad128(cols) // group
    scale = torch.empty((n, rows), dtype=torch.float64, device=w.device)
    values = torch.zeros_like(w)
    zero = w.new_zeros(rows)
    for k in range(n):
        part = w[:, group * k:group * k + group]
        scale[k] = s = _scale_exact(part.abs().max(1).values if part.shape[1] else zero)
        a, v = part.abs(), torch.zeros_like(part)
        for lo, hi, up in ((0, .5, False), (.5, 1, True), (1, 1.5, False), (1.5, 2, True),
                           (2, 3, False), (3, 4, True), (4, 6, False)):
            border = (lo + hi) / 2 * s[:, None]
            past = a >= border if up else a > border
            v += torch.where(past, (hi - lo) * s[:, None], torch.zeros_like(v))
        values[:, group * k:group * k + group] = torch.copysign(v, part)
    return values, scale


def _value_exact(w4, cols, group):
    """float64 values from the bits: sign, two exponent bits, one mantissa bit."""
    q, s = w4
    out = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.float64, device=q.device)
    for half in range(2):
        c = ((q >> (4 * half)) & 15).double()
        sign = 1 - 2 * torch.floor(c / 8)
        e, m = torch.floor(c.remainder(8) / 2), c.remainder(2)
        power = torch.where(e == 3, 4.0, torch.where(e == 2, 2.0, 1.0))
        v = torch.where(e > 0, (1 + m / 2) * power, m / 2)
        out[:, half::2] = sign * v
    rep = torch.arange(out.shape[1], device=q.device) // group
    return (out * s.double().t()[:, rep])[:, :cols].contiguous()


def exact(case, seed):
    s = prepare(case, seed)
    op, group = case["op"], case["group"]
    if op == "fp4_quant":
        values, scale = _quant_exact(s["w_"].double(), group)
        return {"values": values, "scale": scale}
    if op == "fp4_dequant":
        return _value_exact(s["w4_"], case["C"], group)
    if op == "fp4_decode_fwd":
        x, d = s["x_"].double(), case["d"]
        g = x @ _value_exact(s["wg4_"], d, group).t().contiguous()
        u = x @ _value_exact(s["wu4_"], d, group).t().contiguous()
        return torch.where(g > 0, g * u, torch.zeros_like(g)) @ _value_exact(s["wd4_"], d, group)
    w = _value_exact(s["w4_"], case["K"], group)
    if op == "fp4_matmul":
        return s["x_"].double() @ w.t().contiguous()
    return s["dy_"].double() @ w
