"""A gated MLP trained with 8-bit products and 8-bit activations, its weight
gradients sent through the gradient codec.

    y = (silu(x Wg^T) * (x Wu^T)) Wd^T

Forward and input-gradient products run on INT8 codes (a scale per token and
per channel), what the backward pass needs of the activations is kept as
8-bit checkpoints, weight gradients are taken from those, and each gradient
travels as an INT8 payload with error feedback, as it would between workers
(one worker here), before a plain SGD step on the fp32 master weights.

    python examples/gated_mlp_8bit.py [--tokens T] [--width D] [--hidden H] [--steps N]

needs one GPU and the built library (python -m embedding_communication_codecs_amd.build).
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import embedding_communication_codecs_amd as qc  # noqa: E402

BF16 = torch.bfloat16
BUCKET = 4096


def up(v: int, unit: int) -> int:
    return -(-v // unit) * unit


class Int8Rows:
    """Codes and scales of a matrix, a scale per row."""

    def __init__(self, rows, dim, dev):
        self.rows, self.dim, self.ld = rows, dim, up(dim, 16)
        self.codes = torch.empty((rows, self.ld), dtype=torch.int8, device=dev)
        self.scale = torch.empty(rows, dtype=torch.float32, device=dev)

    def set(self, x):
        t = qc.QC_BF16 if x.dtype == BF16 else qc.QC_F32
        qc.qc_encode_int8_rowwise(x, t, self.rows, self.dim, x.stride(0), self.codes, self.ld, self.scale)
        return self

    def times(self, w: "Int8Rows", out):
        """out[i][j] = row i of this matrix times row j of w."""
        qc.qc_matmul_int8(self.codes, self.scale, self.ld, w.codes, w.scale, w.ld, self.rows, w.rows, self.dim, out,
                          qc.QC_BF16, out.stride(0))
        return out


class Kept:
    """An activation matrix held in 8 bits until the backward pass."""

    def __init__(self, rows, dim, dev):
        self.rows, self.dim = rows, dim
        cb, eb = qc.ckpt8_bytes(rows, dim)
        self.codes = torch.empty(cb, dtype=torch.int8, device=dev)
        self.exps = torch.empty(eb, dtype=torch.uint8, device=dev)

    def set(self, x):
        qc.qc_encode_ckpt8(x, qc.QC_BF16, self.rows, self.dim, x.stride(0), self.codes, self.exps)
        return self

    def nbytes(self):
        return self.codes.numel() + self.exps.numel()


class Sender:
    """A weight gradient's way through the codec: INT8 payload with error
    feedback out, fp32 back."""

    def __init__(self, n, dev):
        self.n = n
        nb = qc.nbuckets(n, BUCKET)
        self.ef = torch.zeros(n, dtype=torch.float32, device=dev)
        self.codes = torch.empty(qc.payload_bytes(qc.QC_UNIFORM, n, BUCKET, 8), dtype=torch.uint8, device=dev)
        self.scale, self.zero = (torch.empty(nb, dtype=torch.float32, device=dev) for _ in range(2))

    def send(self, grad):
        qc.qc_encode_uniform(grad, self.ef, self.n, BUCKET, 8, self.codes, self.scale, self.zero)
        qc.qc_dequant_accumulate(qc.QC_UNIFORM, self.codes, self.scale, self.zero, 1, self.n, BUCKET, 8, grad, False)
        return grad


class GatedMlp8:
    def __init__(self, tokens, width, hidden, dev, seed=0):
        g = torch.Generator(device=dev).manual_seed(seed)
        self.t, self.d, self.h = tokens, width, hidden
        new = lambda *s, dtype=BF16: torch.empty(s, dtype=dtype, device=dev)  # noqa: E731
        self.w_in = torch.randn((2 * hidden, width), generator=g, device=dev) * width ** -0.5  # gate rows, then up
        self.w_out = torch.randn((width, hidden), generator=g, device=dev) * hidden ** -0.5
        # weights as codes, by output channel and (for the gradients of the inputs) by input channel
        self.q_in, self.q_in_t = Int8Rows(2 * hidden, width, dev), Int8Rows(width, 2 * hidden, dev)
        self.q_out, self.q_out_t = Int8Rows(width, hidden, dev), Int8Rows(hidden, width, dev)
        # activations as codes, and what is kept of them
        self.q_x, self.q_h = Int8Rows(tokens, width, dev), Int8Rows(tokens, hidden, dev)
        self.q_dy, self.q_dgu = Int8Rows(tokens, width, dev), Int8Rows(tokens, 2 * hidden, dev)
        self.k_x, self.k_h = Kept(tokens, width, dev), Kept(tokens, hidden, dev)
        self.k_gate, self.k_up = Kept(tokens, hidden, dev), Kept(tokens, hidden, dev)
        self.gu, self.act, self.y = new(tokens, 2 * hidden), new(tokens, hidden), new(tokens, width)
        self.dact, self.dgu, self.dx = new(tokens, hidden), new(tokens, 2 * hidden), new(tokens, width)
        self.dw_in, self.dw_out = torch.empty_like(self.w_in), torch.empty_like(self.w_out)
        need = max(qc.qc_ckpt8_wgrad_workspace(tokens, 2 * hidden, width, qc.QC_BF16),
                   qc.qc_ckpt8_wgrad_workspace(tokens, width, hidden, qc.QC_BF16), 16)
        self.work = torch.empty(need, dtype=torch.uint8, device=dev)
        self.load()

    def load(self):
        """The weights' codes, once per optimizer step."""
        self.q_in.set(self.w_in)
        self.q_in_t.set(self.w_in.t().contiguous())
        self.q_out.set(self.w_out)
        self.q_out_t.set(self.w_out.t().contiguous())

    def forward(self, x):
        h, ld = self.h, 2 * self.h
        self.k_x.set(x)
        self.q_x.set(x).times(self.q_in, self.gu)
        qc.qc_swiglu_ckpt8(self.gu[:, :h], self.gu[:, h:], qc.QC_BF16, ld, self.t, h, self.act, h, self.k_gate.codes,
                           self.k_gate.exps, self.k_up.codes, self.k_up.exps)
        self.k_h.set(self.act)
        return self.q_h.set(self.act).times(self.q_out, self.y)

    def _wgrad(self, dy, kept, dw):
        qc.qc_ckpt8_wgrad(dy, qc.QC_BF16, dy.stride(0), kept.codes, kept.exps, self.t, dy.shape[1], kept.dim, dw,
                          qc.QC_F32, kept.dim, False, self.work)

    def backward(self, dy):
        h, ld = self.h, 2 * self.h
        self._wgrad(dy, self.k_h, self.dw_out)
        self.q_dy.set(dy).times(self.q_out_t, self.dact)
        qc.qc_swiglu_ckpt8_backward(self.dact, qc.QC_BF16, h, self.k_gate.codes, self.k_gate.exps, self.k_up.codes,
                                    self.k_up.exps, self.t, h, self.dgu[:, :h], self.dgu[:, h:], ld)
        self._wgrad(self.dgu, self.k_x, self.dw_in)
        return self.q_dgu.set(self.dgu).times(self.q_in_t, self.dx)

    def kept_bytes(self):
        return sum(k.nbytes() for k in (self.k_x, self.k_h, self.k_gate, self.k_up))


def train(tokens=2048, width=1024, hidden=2048, steps=30, lr=0.5, seed=0, log=print):
    """Fits the MLP to another of the same shape; returns the losses."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed + 1)
    model = GatedMlp8(tokens, width, hidden, dev, seed)
    teacher = GatedMlp8(tokens, width, hidden, dev, seed + 2)
    send_in, send_out = Sender(model.w_in.numel(), dev), Sender(model.w_out.numel(), dev)
    losses = []
    for step in range(steps):
        x = torch.randn((tokens, width), generator=gen, device=dev).to(BF16)
        want = teacher.forward(x).float()
        diff = model.forward(x).float() - want
        losses.append(diff.square().mean().item())
        model.backward((diff * (2.0 / tokens)).to(BF16))
        model.w_in -= lr * send_in.send(model.dw_in)
        model.w_out -= lr * send_out.send(model.dw_out)
        model.load()
        if step % 10 == 0 or step == steps - 1:
            log(f"step {step:4d}  loss {losses[-1]:.4f}")
    in_bf16 = 2 * tokens * (width + 3 * hidden)
    log(f"activations kept: {model.kept_bytes() / 1e6:.1f} MB (bf16: {in_bf16 / 1e6:.1f} MB)")
    return losses


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("tokens", 2048), ("width", 1024), ("hidden", 2048), ("steps", 30)):
        p.add_argument(f"--{name}", type=int, default=value)
    p.add_argument("--lr", type=float, default=0.5)
    train(**vars(p.parse_args()))
