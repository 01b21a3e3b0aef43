"""A data-parallel training loop over K emulated ranks, with the optimizer sharded and the weight
gathered in 4 bits.

    python examples/sharded_update.py [steps]

A linear layer y = x w^T learns a given one. Every step, on every rank: forward through the gathered
4-bit weight, gradient of the rank's own batch, ReduceScatter of the gradients (average); then on each
rank's shard: the gradient's norm and clip factor, AdamW with 8-bit states, quantisation of the updated
rows, and the AllGather of their codes and scales.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gradient_sync_amd as dps  # noqa: E402


class Trainer:
    def __init__(self, ranks=8, n=1024, k=512, batch=256, lr=2e-3, max_norm=50.0, seed=0, device="cuda"):
        if n % (16 * ranks):
            raise ValueError("a shard is a multiple of 16 rows")
        self.ranks, self.n, self.k, self.batch, self.max_norm, self.device = ranks, n, k, batch, max_norm, device
        self.gen = torch.Generator(device=device).manual_seed(seed)
        self.target = self._randn(n, k) * k ** -0.5
        rows = n // ranks
        # flat per-rank gradients, and the shards: rows [r * rows, (r + 1) * rows) of the weight
        self.grads = [torch.empty(n * k, device=device) for _ in range(ranks)]
        self.grad_shards = [torch.empty(rows * k, device=device) for _ in range(ranks)]
        self.params = [(self._randn(rows, k) * 0.02).view(-1) for _ in range(ranks)]
        self.copies = [p.bfloat16() for p in self.params]
        m, v, scales = dps.AdamW.new_state(self.params, bits=8)
        self.ctrl = dps.StepCtrl(device=device)
        self.norm = dps.GradNorm(self.grad_shards, self.ctrl)
        self.update = dps.AdamW(self.params, self.grad_shards, m, v, copies=self.copies, scales=scales, lr=lr,
                                betas=(0.9, 0.99), weight_decay=0.0, seed=seed)
        self.quantized = [dps.Mxfp4(rows, k, device=device) for _ in range(ranks)]
        self.weights = [dps.Mxfp4(n, k, device=device) for _ in range(ranks)]     # one gathered copy per rank
        self.gather()

    def _randn(self, *shape):
        return torch.randn(shape, generator=self.gen, device=self.device)

    def gather(self):
        """Each rank quantises its rows; the codes and the scales are gathered on every rank."""
        for copy, q in zip(self.copies, self.quantized):
            dps.dp_mxfp4_quantize(copy.view(q.rows, q.cols), out=q)
        words = lambda t: t.view(-1).view(torch.int32)
        dps.dp_all_gather([words(q.codes) for q in self.quantized], [words(w.codes) for w in self.weights])
        dps.dp_all_gather([words(q.scales) for q in self.quantized], [words(w.scales) for w in self.weights])

    def step(self):
        """One update; the mean loss over the ranks' batches before it, on the GPU."""
        losses = []
        for r in range(self.ranks):
            x = self._randn(self.batch, self.k).bfloat16()
            y = dps.dp_mxfp4_linear(x, self.weights[r], dtype=torch.float32)
            off = y - x.float() @ self.target.t()
            losses.append(off.square().mean())
            dy = dps.dp_mxfp4_quantize(off * (2.0 / self.batch), transposed="only")
            xt = dps.dp_mxfp4_quantize(x, transposed="only")
            dps.dp_gemm_mxfp4(dy, xt, out=self.grads[r].view(self.n, self.k))
        dps.dp_reduce_scatter(self.grads, self.grad_shards, op="avg")
        self.norm.run(self.max_norm)
        self.update.step(ctrl=self.ctrl)
        self.gather()
        return torch.stack(losses).mean()


def main(steps=200):
    t = Trainer()
    for i in range(steps):
        loss = t.step()
        if i % 20 == 0 or i == steps - 1:
            print(f"step {int(t.ctrl.step):4d}  loss {float(loss):.5f}  gradient norm {float(t.ctrl.norm):.4f}  "
                  f"clip factor {float(t.ctrl.scale):.4f}", flush=True)


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 200)
