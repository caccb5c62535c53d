"""Distil the projected n-gram layer from a teacher's top logits on one GPU, then search with it in 4 bits.

The layer of train_projected_fp8.py with the vocabulary as its outputs.  A training step runs

  forward   the layer in 8 bits, to logits [n][V]
  loss      ngram_distill            against the teacher's 32 likeliest tokens and its log sum over all of them,
                                     the gradient in the logits' place
  backward  the layer's, and AdamW

and a step of the search, for `beams` beams of every sequence,

  ngram_forward, ngram_add_norm      tokens and two-token histories to hidden states
  ngram_project_int4                 logits from the projection's weights in 4 bits
  ngram_beam_step                    the next tokens, histories, scores and parents, in place
  ngram_beam_reorder                 what the beams have written so far follows them

captured in a HIP graph: nothing of it comes back to the host.

    python examples/distill_and_search.py [--steps 40]
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
for path in (ROOT, os.path.join(ROOT, "examples")):
    if path not in sys.path:
        sys.path.insert(0, path)

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from train_projected_fp8 import EPS, Layer, batch  # noqa: E402

END = 0


def teacher_lists(teacher, tokens, offsets, k=32, temperature=2.0):
    """What a stored teacher would hold for each token: its k largest logits, their tokens, and log sum exp at the temperature."""
    stream = torch.zeros((tokens.numel(), teacher.d), dtype=torch.bfloat16, device=tokens.device)
    logits = 4.0 * teacher.forward(tokens, offsets, stream, keep=False).float()
    top = logits.topk(k, dim=1)
    return top.values.contiguous(), top.indices.to(torch.int32).contiguous(), torch.logsumexp(logits / temperature, dim=1)


def train(steps=40, n=1024, seqs=8, V=1000, seed=1, temperature=2.0, say=print):
    """The student and the loss of each step."""
    teacher, layer = (Layer(V=V, d_out=V, seed=s) for s in (100, seed))
    losses = []
    for step in range(1, steps + 1):
        tokens, offsets = batch(V, n, seqs, seed * 1000 + step % 8)
        values, ids, lse = teacher_lists(teacher, tokens, offsets, temperature=temperature)
        stream = torch.zeros((n, layer.d), dtype=torch.bfloat16, device=tokens.device)
        logits = layer.forward(tokens, offsets, stream)
        loss, _, dlogits = ng.ngram_distill(logits, values, ids, temperature, lse, scale=1.0 / n, dlogits_out=logits)
        losses.append(float(loss.mean()))
        layer.backward(dlogits)
        layer.update(step, seed=seed)
        if say and (step == 1 or step % 10 == 0):
            say(f"step {step:3d}  loss {losses[-1]:.4f}", flush=True)
    return layer, losses


class Search:
    """Beam search over the layer's outputs for ``batch`` sequences that start with ``first`` [batch] int32."""

    def __init__(self, layer, first, beams=4, most=32, end=END):
        self.layer, self.beams, self.end = layer, beams, end
        dev, rows = first.device, first.numel() * beams
        self.head = ng.ngram_quant_int4(layer.P, group=64)
        self.tokens = first.repeat_interleave(beams).to(torch.int32)
        self.history = torch.full((rows, 2), ng.PAD_ID, dtype=torch.int32, device=dev)
        # the first beam alone is alive at the start
        self.scores = torch.where(torch.arange(rows, device=dev) % beams == 0, 0.0, float("-inf"))
        self.parents = torch.zeros(rows, dtype=torch.int32, device=dev)
        self.finished = torch.zeros(rows, dtype=torch.bool, device=dev)
        self.written = torch.zeros((rows, most), dtype=torch.int32, device=dev)
        self.written[:, 0] = self.tokens
        self.length = 1
        self.offsets = torch.arange(rows + 1, dtype=torch.int32, device=dev)
        self.stream = torch.empty((rows, layer.d), dtype=torch.bfloat16, device=dev)
        self.out = ng.BeamOut(self.scores, self.tokens, self.parents, self.history, self.finished)
        self.workspace = ng.beam_step_workspace(first.numel(), beams, layer.d_out, torch.float32, dev)
        self.states = ng.BeamStates([self.written])
        self.graph = None

    def logits(self, tokens, history):
        """[rows][V] fp32 of tokens that come after their histories."""
        self.stream.zero_()
        ng.ngram_forward(tokens, self.offsets, self.layer.rows, self.layer.W_g, self.stream, e1=self.layer.e1.p, residual=self.stream,
                         history=history)
        y = ng.ngram_add_norm(self.stream, self.layer.gamma, EPS, keep_y=True, quantise=False).y
        return ng.ngram_project_int4(y, self.head, dtype=torch.float32)

    def step(self):
        ng.ngram_beam_step(self.logits(self.tokens, self.history), self.scores, self.beams, self.tokens, self.history, self.finished, self.end,
                           out=self.out, workspace=self.workspace)
        ng.ngram_beam_reorder(self.states, self.parents, self.beams)

    def capture(self):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        keep = [t.clone() for t in (*self.out, self.written)]
        with torch.cuda.stream(side):
            self.step()
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph, stream=side):
                self.step()
        torch.cuda.current_stream().wait_stream(side)
        for t, k in zip((*self.out, self.written), keep):
            t.copy_(k)

    def run(self, steps):
        """(tokens [rows][1 + steps], scores [rows]), each sequence's beams the best first."""
        for _ in range(steps):
            self.step() if self.graph is None else self.graph.replay()
            self.written[:, self.length] = self.tokens
            self.length += 1
        return self.written[:, :self.length], self.scores


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=40)
    args = ap.parse_args()
    layer, losses = train(args.steps)
    first = torch.tensor([5, 17], dtype=torch.int32, device="cuda:0")
    search = Search(layer, first)
    search.capture()
    written, scores = search.run(12)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}; best of {search.beams} beams after 12 steps:")
    for row in range(0, written.shape[0], search.beams):
        print(f"  {scores[row].item():.3f}  {written[row].tolist()}")


if __name__ == "__main__":
    main()
