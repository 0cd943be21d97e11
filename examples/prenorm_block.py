"""The sparse layer as the feed-forward half of a pre-norm block, followed by
a dense projection in 8 bits: a few training steps, then the same block
serving a prefill and single tokens.

    h1, n1 = norm(a, residual=h0)      a: the other branch's output (given)
    y      = sparse layer(n1)
    h2, n2 = norm(y, residual=h1)
    out    = n2 W^T                    W [d_out][d_model], in 8 bits

Training keeps float32 masters of every weight; the sparse layer runs on
bfloat16 copies, the projection on 8-bit copies (both orientations, one scale
a 128 x 128 block), made once a step. The projection's two gradients are 8-bit
products as well: of d_out quantised along both of its axes with W^T and with
n2^T. Serving norms straight into 8 bits, so that the normed stream crosses
HBM in one byte an element.

    python examples/prenorm_block.py [--tokens 4096] [--d-model 1024] [--d-ff 2816] [--steps 5]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from activation_sparse_ffn_gemm_amd import _lib as tw  # noqa: E402
from activation_sparse_ffn_gemm_amd import synth  # noqa: E402

BF = torch.bfloat16
E4 = torch.float8_e4m3fn


class PrenormBlock:
    """Weights of one block on one GPU. ``master`` holds what is trained."""

    def __init__(self, wg_t, wu_t, wd, proj, max_ovf, K=128, eps=1e-6):
        d = wg_t.shape[1]
        ones = torch.ones(d, dtype=torch.float32, device=wg_t.device)
        self.master = {"g1": ones, "g2": ones.clone(), "wg": wg_t.float(), "wu": wu_t.float(),
                       "wd": wd.float(), "proj": proj.float()}
        self.K, self.max_ovf, self.eps = K, max_ovf, eps
        self.status = torch.zeros(1, dtype=torch.int32, device=wg_t.device)
        self.refresh()

    def refresh(self):
        """The copies that the kernels read, of the masters as they are now."""
        m = self.master
        self.wg, self.wu, self.wd = (m[k].to(BF) for k in ("wg", "wu", "wd"))
        self.proj, self.proj_t = tw.fp8_quant(m["proj"], block_rows=128, layout="both")

    def train_forward(self, a, h0):
        """(out, what the backward needs)."""
        m = self.master
        n1, h1 = tw.rmsnorm_fwd(a, m["g1"], residual=h0, eps=self.eps)
        packed = tw.gate_pack(n1, self.wg, status=self.status)
        hy = tw.to_hybrid(packed, self.K, self.max_ovf, status=self.status)
        y = tw.hybrid_fwd(n1, hy, self.wu, self.wd, status=self.status)
        n2, h2 = tw.rmsnorm_fwd(y, m["g2"], residual=h1, eps=self.eps)
        n2_q, n2_qt = tw.fp8_quant(n2, layout="both")
        out = tw.fp8_matmul(n2_q, self.proj, fast_sums=True)
        return out, (n1, h1, hy, h2, n2_qt)

    def backward(self, saved, dout):
        """Gradients of the masters (a dict) and of the stream h0 (and of a)."""
        n1, h1, hy, h2, n2_qt = saved
        m, g = self.master, {}
        dq, dqt = tw.fp8_quant(dout, layout="both")
        g["proj"] = tw.fp8_matmul(dqt, n2_qt, out_dtype=torch.float32)
        dn2 = tw.fp8_matmul(dq, self.proj_t, fast_sums=True)
        dh2, g["g2"] = tw.rmsnorm_bwd(dn2, h2, m["g2"], eps=self.eps)
        dn1, g["wg"], g["wu"], g["wd"] = tw.ffn_bwd(n1, dh2.to(BF), hy, self.wg, self.wu, self.wd,
                                                    status=self.status)
        dh0, g["g1"] = tw.rmsnorm_bwd(dn1, h1, m["g1"], dres=dh2, eps=self.eps)
        return g, dh0

    def step(self, a, h0, target, lr):
        """One step of gradient descent on sum((out - target)^2) / (2 T)."""
        out, saved = self.train_forward(a, h0)
        diff = out.float() - target
        grads, _ = self.backward(saved, (diff / out.shape[0]).to(BF))
        for k, v in grads.items():
            self.master[k] -= lr * v
        self.refresh()
        return 0.5 * diff.square().sum() / out.shape[0]

    def serve(self, a, h0):
        """(out, h2): the forward alone, for any number of tokens."""
        m = self.master
        n1, h1 = tw.rmsnorm_fwd(a, m["g1"], residual=h0, eps=self.eps)
        if n1.shape[0] <= tw.DECODE_T:
            _, y = tw.decode_fwd(n1, self.wg, self.wu, self.wd, status=self.status)
        else:
            y = tw.ffn_fwd(n1, tw.gate_pack(n1, self.wg, status=self.status), self.wu, self.wd,
                           status=self.status)
        n2, h2 = tw.rmsnorm_fwd(y, m["g2"], residual=h1, eps=self.eps, out_dtype=E4)
        return tw.fp8_matmul(n2, self.proj, fast_sums=True), h2

    def check(self):
        code = int(self.status.item())
        if code:
            raise RuntimeError(f"device status {code}: more nonzeros than the sparse layouts hold")


def make_case(tokens, d_model, d_ff, d_out, density=0.01, skew=0.0, seed=0, device="cuda:0"):
    """(block, a, h0): synthetic weights and streams; column 0 of the stream
    carries the constant that keeps the gate at about ``density``."""
    w = synth.Workload("prenorm-block", tokens, d_model, d_ff, "bf16", density, skew_frac=skew,
                       skew_density=0.3)
    d = synth.make_inputs(w, seed=seed)
    gen = torch.Generator().manual_seed(seed)
    a = 0.1 * torch.randn((tokens, d_model), generator=gen)
    a[:, 0] = 0
    proj = torch.randn((d_out, d_model), generator=gen) / d_model ** 0.5
    block = PrenormBlock(d["wg_t"].to(device), d["wu_t"].to(device), d["wd"].to(device),
                         proj.to(device), max_ovf=max(16, tokens // 4))
    return block, a.to(BF).to(device), d["x"].float().to(device)


def _time(fn, n=20):
    for _ in range(3):
        fn()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(n):
        fn()
    torch.cuda.synchronize()
    return (time.perf_counter() - t0) / n


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--tokens", type=int, default=4096)
    p.add_argument("--d-model", type=int, default=1024)
    p.add_argument("--d-ff", type=int, default=2816)
    p.add_argument("--d-out", type=int, default=1024)
    p.add_argument("--density", type=float, default=0.01)
    p.add_argument("--steps", type=int, default=5)
    p.add_argument("--lr", type=float, default=0.02)
    o = p.parse_args(argv)
    block, a, h0 = make_case(o.tokens, o.d_model, o.d_ff, o.d_out, o.density, skew=0.02)
    target = torch.randn((o.tokens, o.d_out), device=a.device,
                         generator=torch.Generator(a.device).manual_seed(1))
    losses = []
    for i in range(o.steps):
        losses.append(float(block.step(a, h0, target, o.lr)))
        block.check()
        print(f"step {i}: loss {losses[-1]:.4f}", flush=True)
    out, _ = block.serve(a, h0)
    few, _ = block.serve(a[:1], h0[:1])
    block.check()
    gap = float((few.float() - out[:1].float()).norm() / out[:1].float().norm())
    print(f"one token alone against the same token in the prefill: {gap:.1e} of its norm")
    t = _time(lambda: block.serve(a, h0))
    print(f"prefill of {o.tokens} tokens: {t * 1e3:.3f} ms, {o.tokens / t / 1e6:.2f} M tokens/s")
    t = _time(lambda: block.serve(a[:1], h0[:1]))
    print(f"one token: {t * 1e6:.0f} us")
    return losses


if __name__ == "__main__":
    main()
