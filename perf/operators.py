"""Timing cases for the pre-norm and 8-bit product operators of a sparse FFN block.

Four operators that stand around the activation-sparse FFN layer in a
pre-norm Transformer block:

* rmsnorm_fwd: the residual stream's update h = residual + x and its
  root-mean-square norm n = h / sqrt(mean(h^2) + eps) * gain, written in
  bfloat16 or float32 (the FFN's input) or in 8 bits with scales.
* rmsnorm_bwd: its gradients dh (the gradient that comes down the skip
  connection included) and dgain.
* fp8_quant: a matrix in 8 bits (e4m3) with one float32 scale for each block
  of 128 columns of a row, or of 128 rows by 128 columns, and the same of its
  transpose (the operands of a product's two gradients).
* fp8_matmul: out = A B^T of two such matrices.

An 8-bit matrix [rows][cols] is q [rows][cols rounded up to 128] (zeros in
the columns past `cols`) and scale [ceil(cols / 128)][ceil(rows / block_rows)];
it stands for q * scale. The scale of a block is max(amax, 2^-64) / 448.

`run` computes an operator in plain torch operations in 32 bits, or, where
`own` is true, by the library's call.
"""
import math

import torch

own = False

DEV = "cuda:0"
EPS = 1e-6
E4M3_MAX = 448.0
AMAX_MIN = 2.0 ** -64
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SZ = {"f32": 4, "bf16": 2, "e4m3": 1}
# the layers of synth.py: 2048 -> 5632 (8192 tokens), 1024 -> 2816 (4096
# tokens), 2304 -> 6144 (decoding, 1 to 64 tokens), 256 -> 1024 (64 tokens, float32)
MOST_FLOPS = 2.0 * 8192 * 5632 * 2048  # the largest listed product
MOST_ELEMS = 8192 * 2048               # the largest listed norm and quantised matrix


def listed():
    return [
        # one decoded token of the 2304-wide layer: launch latency
        {"name": "norm-decode", "op": "rmsnorm_fwd", "T": 1, "d": 2304, "x": "f32",
         "res": "bf16", "gain": "bf16", "out": "bf16"},
        # the FFN's float32 output joins the residual stream, next product in 8 bits
        {"name": "norm-prefill-fp8", "op": "rmsnorm_fwd", "T": 8192, "d": 2048, "x": "f32",
         "res": "bf16", "gain": "bf16", "out": "e4m3"},
        # a width that is no multiple of anything, float32 stream
        {"name": "norm-odd", "op": "rmsnorm_fwd", "T": 1029, "d": 999, "x": "bf16",
         "res": "f32", "gain": "f32", "out": "bf16"},
        # the FFN's float32 dx and the skip connection's gradient, training batch
        {"name": "norm-bwd-train", "op": "rmsnorm_bwd", "T": 8192, "d": 2048, "dn": "f32",
         "h": "bf16", "gain": "bf16", "dres": "f32", "dh": "f32"},
        # the small float32 layer's step
        {"name": "norm-bwd-tiny", "op": "rmsnorm_bwd", "T": 64, "d": 256, "dn": "f32",
         "h": "f32", "gain": "f32", "dres": "f32", "dh": "f32"},
        # a gradient for both products of the backward: along its rows and along its columns
        {"name": "quant-grad-both", "op": "fp8_quant", "R": 8192, "C": 2048, "x": "bf16",
         "block_rows": 1, "layout": "both"},
        # the weights after an optimizer step: 128 x 128 blocks, and the transpose's
        {"name": "quant-weight-both", "op": "fp8_quant", "R": 2816, "C": 1024, "x": "f32",
         "block_rows": 128, "layout": "both"},
        # one decoded token
        {"name": "mm-decode-1", "op": "fp8_matmul", "M": 1, "N": 6144, "K": 2304,
         "a_rows": 1, "b_rows": 128, "out": "bf16"},
        # a ragged decoding batch, the down direction
        {"name": "mm-decode-50", "op": "fp8_matmul", "M": 50, "N": 2304, "K": 6144,
         "a_rows": 1, "b_rows": 128, "out": "bf16"},
        # ragged everywhere: tokens, a contraction that ends inside a block, an odd width
        {"name": "mm-ragged", "op": "fp8_matmul", "M": 1029, "N": 2811, "K": 1088,
         "a_rows": 1, "b_rows": 128, "out": "bf16"},
        # the dense up projection over a prompt batch
        {"name": "mm-prefill", "op": "fp8_matmul", "M": 8192, "N": 5632, "K": 2048,
         "a_rows": 1, "b_rows": 128, "out": "bf16"},
        # a weight's gradient: both operands scaled along the tokens, float32 out
        {"name": "mm-wgrad", "op": "fp8_matmul", "M": 5632, "N": 2048, "K": 8192,
         "a_rows": 1, "b_rows": 1, "out": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width over [lo, hi]: a multiple of 64, of 8, or any number."""
    v = _log(rng, lo, hi)
    m = rng.choice((64, 64, 8, 1))
    return min(hi, max(lo, v // m * m))


def draw(rng):
    op = rng.choice(("rmsnorm_fwd", "rmsnorm_bwd", "fp8_quant", "fp8_matmul"))
    two = ("f32", "bf16")
    if op in ("rmsnorm_fwd", "rmsnorm_bwd"):
        d = _width(rng, 64, 8192)
        T = min(_log(rng, 1, 8192), MOST_ELEMS // d)
        if op == "rmsnorm_fwd":
            return {"op": op, "T": T, "d": d, "x": rng.choice(two),
                    "res": rng.choice(("none", "f32", "bf16")), "gain": rng.choice(two),
                    "out": rng.choice(("f32", "bf16", "e4m3", "e4m3"))}
        return {"op": op, "T": T, "d": d, "dn": rng.choice(two), "h": rng.choice(two),
                "gain": rng.choice(two), "dres": rng.choice(("none", "f32", "bf16")),
                "dh": rng.choice(two)}
    if op == "fp8_quant":
        C = _width(rng, 64, 8192)
        R = min(_log(rng, 1, 8192), MOST_ELEMS // C)
        return {"op": op, "R": R, "C": C, "x": rng.choice(two),
                "block_rows": rng.choice((1, 1, 128)),
                "layout": rng.choice(("rows", "cols", "both"))}
    N, K = _width(rng, 64, 8192), _width(rng, 64, 8192)
    M = max(1, min(_log(rng, 1, 8192), int(MOST_FLOPS / (2.0 * N * K))))
    a_rows, b_rows = rng.choice(((1, 128), (1, 128), (1, 1)))
    return {"op": op, "M": M, "N": N, "K": K, "a_rows": a_rows, "b_rows": b_rows,
            "out": rng.choice(two)}


# ---------------------------------------------------------------- inputs
def _normal(shape, g, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale


def _stream(T, d, g, dtype):
    """A residual stream: channels of different sizes, a few of them large."""
    chan = torch.exp(0.5 * _normal((d,), g))
    chan = torch.where(torch.rand((d,), generator=g, device=DEV) < 0.002, chan * 30.0, chan)
    return (_normal((T, d), g) * chan).to(dtype)


def _pad128(n):
    return -(-n // 128) * 128


def _quantised(rows, cols, block_rows, g, scale):
    """A quantised matrix of normal values, rows of different sizes."""
    x = _normal((rows, cols), g, scale) * torch.exp(0.5 * _normal((rows, 1), g))
    q, s = _quant_plain(x, block_rows)
    return q, s.contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "rmsnorm_fwd":
        T, d = case["T"], case["d"]
        s["x_"] = _normal((T, d), g, 0.3).to(DT[case["x"]])
        s["res_"] = None if case["res"] == "none" else _stream(T, d, g, DT[case["res"]])
        s["gain_"] = (1.0 + _normal((d,), g, 0.2)).to(DT[case["gain"]])
        if T > 8:  # padding tokens: rows of zeros
            s["x_"][5::97] = 0
            if s["res_"] is not None:
                s["res_"][5::97] = 0
    elif op == "rmsnorm_bwd":
        T, d = case["T"], case["d"]
        s["dn_"] = _normal((T, d), g, 1e-2).to(DT[case["dn"]])
        s["h_"] = _stream(T, d, g, DT[case["h"]])
        s["gain_"] = (1.0 + _normal((d,), g, 0.2)).to(DT[case["gain"]])
        s["dres_"] = None if case["dres"] == "none" else \
            _normal((T, d), g, 1e-2).to(DT[case["dres"]])
    elif op == "fp8_quant":
        R, C = case["R"], case["C"]
        s["x_"] = (_normal((R, C), g, 0.02)
                   * torch.exp(_normal((R, 1), g))).to(DT[case["x"]])
        if R > 300 and case["block_rows"] == 1:
            s["x_"][5::97] = 0
    else:
        M, N, K = case["M"], case["N"], case["K"]
        s["a_"] = _quantised(M, K, case["a_rows"], g, 1.0)
        s["b_"] = _quantised(N, K, case["b_rows"], g, 1.0 / math.sqrt(K))
    return s


# ---------------------------------------------------------------- plain forms
def _quant_plain(x, block_rows):
    """float32 [rows][cols] -> (q [rows][cols up to 128], scale [col blocks][row blocks])."""
    rows, cols = x.shape
    rp, cp = -(-rows // block_rows) * block_rows, _pad128(cols)
    p = torch.zeros((rp, cp), dtype=torch.float32, device=x.device)
    p[:rows, :cols] = x
    b = p.view(rp // block_rows, block_rows, cp // 128, 128)
    s = b.abs().amax(dim=(1, 3)).clamp(min=AMAX_MIN) / E4M3_MAX
    q = (b / s[:, None, :, None]).to(torch.float8_e4m3fn)
    return q.view(rp, cp)[:rows], s.t()


def _dequant_plain(q, scale, block_rows):
    """The float32 values that a quantised matrix stands for."""
    s = scale.t().repeat_interleave(block_rows, 0)[:q.shape[0]].repeat_interleave(128, 1)
    return q.float() * s


def _rmsnorm_fwd_plain(s):
    h = s["x_"].float()
    if s["res_"] is not None:
        h = h + s["res_"].float()
    r = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
    n = h * r * s["gain_"].float()
    out = {}
    if s["res_"] is not None:
        out["h"] = h.to(s["res_"].dtype)
    if s["out"] == "e4m3":
        out["q"], out["scale"] = _quant_plain(n, 1)
    else:
        out["n"] = n.to(DT[s["out"]])
    return out


def _rmsnorm_bwd_plain(s):
    dn, h, gain = s["dn_"].float(), s["h_"].float(), s["gain_"].float()
    r = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
    xh = h * r
    dg = dn * gain
    dh = r * (dg - xh * (dg * xh).mean(1, keepdim=True))
    if s["dres_"] is not None:
        dh = dh + s["dres_"].float()
    return {"dh": dh.to(DT[s["dh"]]), "dgain": (dn * xh).sum(0)}


def _fp8_quant_plain(s):
    x, out = s["x_"].float(), {}
    if s["layout"] != "cols":
        out["q"], out["scale"] = _quant_plain(x, s["block_rows"])
    if s["layout"] != "rows":
        out["q_t"], out["scale_t"] = _quant_plain(x.t(), s["block_rows"])
    return out


def _fp8_matmul_plain(s):
    a = _dequant_plain(*s["a_"], s["a_rows"])
    b = _dequant_plain(*s["b_"], s["b_rows"])
    return (a @ b.t()).to(DT[s["out"]])


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["op"]
    if not own:
        if op == "rmsnorm_fwd":
            return _rmsnorm_fwd_plain(s)
        if op == "rmsnorm_bwd":
            return _rmsnorm_bwd_plain(s)
        if op == "fp8_quant":
            return _fp8_quant_plain(s)
        return _fp8_matmul_plain(s)
    from activation_sparse_ffn_gemm_amd import _lib as tw
    if op == "rmsnorm_fwd":
        n, h = tw.rmsnorm_fwd(s["x_"], s["gain_"], residual=s["res_"], eps=EPS,
                              out_dtype=DT[s["out"]])
        out = {} if s["res_"] is None else {"h": h}
        if s["out"] == "e4m3":
            out["q"], out["scale"] = n.q, n.scale
        else:
            out["n"] = n
        return out
    if op == "rmsnorm_bwd":
        dh, dgain = tw.rmsnorm_bwd(s["dn_"], s["h_"], s["gain_"], dres=s["dres_"], eps=EPS,
                                   dh_dtype=DT[s["dh"]])
        return {"dh": dh, "dgain": dgain}
    if op == "fp8_quant":
        rows, cols = tw.fp8_quant(s["x_"], block_rows=s["block_rows"], layout=s["layout"])
        out = {}
        if rows is not None:
            out["q"], out["scale"] = rows.q, rows.scale
        if cols is not None:
            out["q_t"], out["scale_t"] = cols.q, cols.scale
        return out
    a = tw.Fp8(*s["a_"], cols=s["K"], block_rows=s["a_rows"])
    b = tw.Fp8(*s["b_"], cols=s["K"], block_rows=s["b_rows"])
    # a bfloat16 result takes the 8-bit instruction's own short sums (their error
    # is far below its rounding), a float32 result, a weight's gradient, full ones
    return tw.fp8_matmul(a, b, out_dtype=DT[s["out"]], fast_sums=s["out"] == "bf16")


# ---------------------------------------------------------------- work
def _fp8_bytes(rows, cols, block_rows):
    return rows * _pad128(cols) + 4 * -(-rows // block_rows) * -(-cols // 128)


def work(case):
    op = case["op"]
    if op == "rmsnorm_fwd":
        T, d = case["T"], case["d"]
        n = T * d
        by = n * SZ[case["x"]] + d * SZ[case["gain"]]
        if case["res"] != "none":
            by += 2 * n * SZ[case["res"]]
        by += _fp8_bytes(T, d, 1) if case["out"] == "e4m3" else n * SZ[case["out"]]
        return {"bytes": by, "flops": (8 if case["out"] == "e4m3" else 5) * n}
    if op == "rmsnorm_bwd":
        n, d = case["T"] * case["d"], case["d"]
        by = n * (SZ[case["dn"]] + SZ[case["h"]] + SZ[case["dh"]]) + d * (SZ[case["gain"]] + 4)
        by += 0 if case["dres"] == "none" else n * SZ[case["dres"]]
        return {"bytes": by, "flops": 12 * n}
    if op == "fp8_quant":
        R, C, br = case["R"], case["C"], case["block_rows"]
        by = R * C * SZ[case["x"]]
        by += 0 if case["layout"] == "cols" else _fp8_bytes(R, C, br)
        by += 0 if case["layout"] == "rows" else _fp8_bytes(C, R, br)
        return {"bytes": by, "flops": 4 * R * C * (2 if case["layout"] == "both" else 1)}
    M, N, K = case["M"], case["N"], case["K"]
    by = _fp8_bytes(M, K, case["a_rows"]) + _fp8_bytes(N, K, case["b_rows"])
    return {"bytes": by + M * N * SZ[case["out"]], "flops": 2.0 * M * N * K}


# ---------------------------------------------------------------- 64 bits
def _round_e4m3(v):
    """float64 values rounded to the e4m3 grid, ties to even: 4 significant
    bits down to 2^-6, then steps of 2^-9."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), e.clamp(min=-5) - 4)
    return torch.round(v / step) * step


def _quant_exact(v, block_rows):
    """The quantised matrix of float64 v: its float32 scales (a scale is held
    in 32 bits) and, on them, the nearest values of the grid."""
    rows, cols = v.shape
    rb, cb = -(-rows // block_rows), -(-cols // 128)
    scale = torch.empty((cb, rb), dtype=torch.float64, device=v.device)
    q = torch.zeros((rows, cb * 128), dtype=torch.float64, device=v.device)
    for k in range(cb):
        part = v[:, 128 * k:128 * k + 128]
        top = part.abs().max(1).values
        top = torch.cat([top, top.new_zeros(rb * block_rows - rows)])
        scale[k] = torch.maximum(top.view(rb, block_rows).max(1).values,
                                 top.new_tensor(AMAX_MIN)) / E4M3_MAX
        held = scale[k].float().double()
        per_row = held[torch.arange(rows, device=v.device) // block_rows]
        q[:, 128 * k:128 * k + part.shape[1]] = _round_e4m3(part / per_row[:, None])
    return q, scale


def exact(case, seed):
    s = prepare(case, seed)
    op, out = case["op"], {}
    if op == "rmsnorm_fwd":
        h = s["x_"].double() if s["res_"] is None else s["x_"].double() + s["res_"].double()
        n = h / torch.sqrt(h.square().sum(1, keepdim=True) / case["d"] + EPS)
        n = n * s["gain_"].double()
        if s["res_"] is not None:
            out["h"] = h
        if case["out"] == "e4m3":
            out["q"], out["scale"] = _quant_exact(n, 1)
        else:
            out["n"] = n
        return out
    if op == "rmsnorm_bwd":
        # by the quotient rule on n = gain h / m, m = sqrt(mean(h^2) + eps):
        # dh = gain dn / m - h sum(gain dn h) / (d m^3)
        dn, h, gain = s["dn_"].double(), s["h_"].double(), s["gain_"].double()
        m = torch.sqrt(h.square().sum(1, keepdim=True) / case["d"] + EPS)
        dot = (gain * dn * h).sum(1, keepdim=True)
        dh = gain * dn / m - h * dot / (case["d"] * m ** 3)
        if s["dres_"] is not None:
            dh = dh + s["dres_"].double()
        return {"dh": dh, "dgain": (dn * h / m).sum(0)}
    if op == "fp8_quant":
        x = s["x_"].double()
        if case["layout"] != "cols":
            out["q"], out["scale"] = _quant_exact(x, case["block_rows"])
        if case["layout"] != "rows":
            out["q_t"], out["scale_t"] = _quant_exact(x.t().contiguous(), case["block_rows"])
        return out
    (qa, sa), (qb, sb) = s["a_"], s["b_"]
    M, N = case["M"], case["N"]
    ia = torch.arange(M, device=DEV) // case["a_rows"]
    ib = torch.arange(N, device=DEV) // case["b_rows"]
    acc = torch.zeros((M, N), dtype=torch.float64, device=DEV)
    for k in range(qa.shape[1] // 128):
        pa = qa[:, 128 * k:128 * k + 128].double() * sa[k].double()[ia][:, None]
        pb = qb[:, 128 * k:128 * k + 128].double() * sb[k].double()[ib][:, None]
        acc += pa @ pb.t().contiguous()
    return acc
