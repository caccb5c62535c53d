"""Train the projected n-gram layer in 8 bits on one GPU, then decode with it.

The layer: hash and gather-sum of the n-gram table, gated with the 1-gram
embedding and added to the residual stream; root-mean-square norm with an 8-bit output; projection
in 8 bits.  A training step runs, all in this library's kernels,

  forward   ngram_hash, ngram_embed_bag, ngram_gate_add    h = e1[w] + W_g * sum of 16 rows
            ngram_add_norm                                 s = stream + h, y = norm(s), q = 8-bit y
            ngram_project_fp8                              out = P q
  backward  ngram_quant_fp8 of dL/dout (rows and transposed) and of y (transposed)
            ngram_project_fp8 twice                        dy = P^T dout, dP = dout^T y
            ngram_add_norm_grad                            dh, dgamma
            ngram_grad_table, ngram_grad_e1, ngram_grad_gate
  update    ngram_adamw                                    P, gamma, W_g
            ngram_adamw_rows                               touched rows of the table and of e1
            ngram_quant_fp8                                P in 8 bits again, both layouts

The table, e1 and their moments are kept as they would be at full size: bf16
rows and 8-bit moments, 4 bytes an element and 2 bytes of scales for 128
elements, so that a 20M x 2560 table with its moments is 206 GB and fits one
card.  Synthetic task: the outputs of a fixed random layer of the same form.

    python examples/train_projected_fp8.py [--steps 60]
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402

EPS = 1e-6


class Rows:
    """A bf16 table with 8-bit moments."""

    def __init__(self, values):
        self.p = values.to(torch.bfloat16).contiguous()
        R, d = self.p.shape
        blocks = -(-d // ng.FP8_BLOCK)
        zeros = lambda *s: torch.zeros(s, dtype=torch.uint8, device=values.device)  # noqa: E731
        self.m, self.v = zeros(R, d), zeros(R, d)
        self.m_scale, self.v_scale = zeros(R, blocks).fill_(127), zeros(R, blocks).fill_(127)

    def update(self, rows, grad, count, **step):
        ng.ngram_adamw_rows(self.p, self.m, self.v, rows, grad, count, self.m_scale, self.v_scale, **step)


class Layer:
    """The projected n-gram layer with its optimiser state."""

    def __init__(self, R=20_000, V=2_000, d=256, d_out=384, device="cuda:0", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        normal = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
        self.d, self.d_out, self.V = d, d_out, V
        self.table, self.e1 = Rows(0.02 * normal(R, d)), Rows(0.1 * normal(V, d))
        self.W_g = torch.rand(d, generator=g, device=device)
        self.gamma = torch.ones(d, device=device)
        self.P = normal(d_out, d) * d ** -0.5
        self.grads = {k: torch.zeros_like(getattr(self, k)) for k in ("P", "gamma", "W_g")}
        params = [getattr(self, k) for k in self.grads]
        self.dense = ng.AdamWTensors(params, list(self.grads.values()), [torch.zeros_like(p) for p in params],
                                     [torch.zeros_like(p) for p in params])
        self.rows = ng.Table(self.table.p, R, d)
        self.lay_out()

    def lay_out(self):
        """P in 8 bits: as the forward reads it and transposed, for dL/dy."""
        self.Pq, self.Pt = ng.ngram_quant_fp8(self.P, transposed=True, block_rows=ng.FP8_BLOCK)

    def forward(self, tokens, offsets, stream, history=None, keep=True):
        """Outputs [n][d_out] bf16; ``stream`` [n][d] bf16 is updated in place.  ``keep``: for a backward to come."""
        n = tokens.numel()
        if not keep:                                    # serving: lookup, gate and residual in one launch
            ng.ngram_forward(tokens, offsets, self.rows, self.W_g, stream, e1=self.e1.p, residual=stream, history=history)
            return ng.ngram_project_fp8(ng.ngram_add_norm(stream, self.gamma, EPS).q, self.Pq)
        ids = ng.ngram_hash(tokens, offsets, self.rows.R, history=history)
        sums = ng.ngram_embed_bag(self.rows, ids)
        h = torch.empty((n, self.d), dtype=torch.bfloat16, device=tokens.device)
        ng.ngram_gate_add(sums, tokens, self.W_g, h, e1=self.e1.p)
        norm = ng.ngram_add_norm(h, self.gamma, EPS, residual=stream, sum_out=stream, keep_y=True, keep_r=True)
        self.kept = (tokens, ids, sums, norm)
        return ng.ngram_project_fp8(norm.q, self.Pq)

    def backward(self, dout):
        """Gradients from dL/dout [n][d_out] bf16; returns dL/dstream [n][d] bf16."""
        tokens, ids, sums, norm = self.kept
        gq, gt = ng.ngram_quant_fp8(dout, transposed=True)
        _, yt = ng.ngram_quant_fp8(norm.y, rows=False, transposed=True)
        dy = ng.ngram_project_fp8(gq, self.Pt)
        ng.ngram_project_fp8(gt, yt, out=self.grads["P"])
        dh, _ = ng.ngram_add_norm_grad(dy, norm.sum, norm.r, self.gamma, dgamma_out=self.grads["gamma"])
        ng.ngram_grad_gate(ids, dh, sums, grad_Wg_out=self.grads["W_g"])
        self.sparse = (ng.ngram_grad_table(ids, self.W_g, dh, self.rows.R), ng.ngram_grad_e1(tokens, ids, dh, self.V))
        return dh

    def update(self, step, lr=3e-3, seed=0):
        h = {"lr": lr, "step": step, "eps": 1e-10}
        # equal places of two tables round alike under one seed
        ng.ngram_adamw(self.dense, seed=3 * seed, **h)
        for i, (rows, grad) in enumerate(zip((self.table, self.e1), self.sparse), start=1):
            rows.update(*grad, seed=3 * seed + i, **h)
        self.lay_out()


def batch(V, n, seqs, seed, device="cuda:0"):
    g = torch.Generator(device=device).manual_seed(seed)
    tokens = (torch.rand(n, generator=g, device=device) ** 3 * V).to(torch.int32)
    return tokens, torch.arange(0, n + 1, n // seqs, dtype=torch.int32, device=device)


def train(steps=60, n=2048, seqs=8, seed=1, say=print):
    """The loss of each step."""
    teacher, layer = Layer(seed=100), Layer(seed=seed)
    losses = []
    for step in range(1, steps + 1):
        tokens, offsets = batch(layer.V, n, seqs, seed * 1000 + step % 8)
        empty = lambda: torch.zeros((n, layer.d), dtype=torch.bfloat16, device=tokens.device)  # noqa: E731
        want = teacher.forward(tokens, offsets, empty(), keep=False).float()
        miss = layer.forward(tokens, offsets, empty()).float() - want
        losses.append(float((miss * miss).mean()))
        layer.backward((miss * (2.0 / miss.numel())).to(torch.bfloat16))
        layer.update(step, seed=seed)
        if say and (step == 1 or step % 10 == 0):
            say(f"step {step:3d}  loss {losses[-1]:.4f}", flush=True)
    return layer, losses


def decode(layer, tokens):
    """The outputs of one sequence token by token, each with the two tokens before it as history."""
    pad, out = ng.PAD_ID, []
    offsets = torch.tensor([0, 1], dtype=torch.int32, device=tokens.device)
    before = [pad, pad]
    for t in range(tokens.numel()):
        stream = torch.zeros((1, layer.d), dtype=torch.bfloat16, device=tokens.device)
        history = torch.tensor([before], dtype=torch.int32, device=tokens.device)
        out.append(layer.forward(tokens[t:t + 1], offsets, stream, history=history, keep=False))
        before = [before[1], int(tokens[t])]
    return torch.cat(out)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    args = ap.parse_args()
    layer, losses = train(args.steps)
    tokens, _ = batch(layer.V, 16, 1, 7)
    stream = torch.zeros((16, layer.d), dtype=torch.bfloat16, device=tokens.device)
    whole = layer.forward(tokens, torch.tensor([0, 16], dtype=torch.int32, device=tokens.device), stream, keep=False)
    gap = (decode(layer, tokens).float() - whole.float()).abs().max().item()
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}; 16 tokens one by one against one batch: largest difference {gap:.3g}")


if __name__ == "__main__":
    main()
