"""One optimizer shard trained through the library's operators.

A small language model of residual blocks, written by hand: token embedding,
blocks of norm -> two-layer perceptron -> post-norm, gate, residual add, and
the loss over the vocabulary.  What a training step needs besides plain matrix
products comes from the library:

  block_norm, block_norm_backward    the norms around every block, forward and
                                     backward, keeping f and h_out in 8 bits
  checkpoint8                        the perceptron's two inputs, kept in 8 bits
  checkpoint8_weight_grad            its weight gradients from those
  linear_cross_entropy               the loss, and the gradients of the last
                                     hidden rows and of the vocabulary's weight
  FusedAdamShard                     the update: the matrices' gradients were
                                     written (or added) where the shard reads
                                     them, the norms' vectors are copied there

    python examples/train_step.py --steps 30
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import adamw_optimizer_step_persistent_gb300 as fadam  # noqa: E402

DEVICE, DTYPE = "cuda", torch.bfloat16


class Model:
    """fp32 masters and gradients in one flat buffer each (the optimizer's
    shard), bf16 weights that the step writes out."""

    def __init__(self, vocab=1000, width=256, hidden=688, blocks=2, lr=3e-3, seed=0):
        gen = torch.Generator().manual_seed(seed)
        shapes = {"embed": (vocab, width), "head": (vocab, width), "norm0": (width,)}
        for b in range(blocks):
            shapes |= {f"up{b}": (hidden, width), f"down{b}": (width, hidden),
                       f"post{b}": (width,), f"pre{b}": (width,), f"gate{b}": (1, width)}
        starts, total = {}, 0
        for name, shape in shapes.items():
            starts[name] = total
            total += -(-torch.Size(shape).numel() // 64) * 64     # views start on 128 bytes

        def buffer(dtype):
            return torch.zeros(total, dtype=dtype, device=DEVICE)

        def views(flat):
            return {n: flat[s:s + torch.Size(shapes[n]).numel()].view(shapes[n])
                    for n, s in starts.items()}

        self.blocks, self.alpha = blocks, blocks ** -0.5
        master, self.grads = views(buffer(torch.float32)), views(buffer(torch.float32))
        m, v, self.w = views(buffer(torch.float32)), views(buffer(torch.float32)), views(buffer(DTYPE))
        for name, shape in shapes.items():
            vector = name.startswith(("post", "pre", "gate", "norm"))
            init = torch.ones(shape) if vector else torch.randn(shape, generator=gen) * shape[-1] ** -0.5
            master[name].copy_(init)
            self.w[name].copy_(init)
        names = list(shapes)
        self.optimizer = fadam.FusedAdamShard([{
            "params": [master[n] for n in names], "exp_avgs": [m[n] for n in names],
            "exp_avg_sqs": [v[n] for n in names], "grads": [self.grads[n] for n in names],
            "params_out": [self.w[n] for n in names], "lr": lr, "betas": (0.9, 0.95),
            "weight_decay": 0.01}], capturable=True)

    def step(self, tokens, targets, first=True):
        """Forward and backward of one micro-batch.  Gradients are added to
        those of the step's earlier micro-batches unless it is the first."""
        w, g = self.w, self.grads
        shut = torch.zeros_like(w["norm0"]).view(1, -1)
        # the first norm is a block norm whose block adds nothing (gate 0)
        h = w["embed"][tokens]
        start = fadam.block_norm(h, h, w["norm0"], gate=shut)
        h, x, kept = start.h_out, start.x_out, []
        for b in range(self.blocks):
            a = torch.relu(x @ w[f"up{b}"].t())
            n = fadam.block_norm(a @ w[f"down{b}"].t(), h, w[f"pre{b}"], post_weight=w[f"post{b}"],
                                 gate=w[f"gate{b}"], residual_scale=self.alpha, checkpoint=True)
            kept.append((fadam.checkpoint8(x), fadam.checkpoint8(a), n))
            h, x = n.h_out, n.x_out

        loss = fadam.linear_cross_entropy(x, w["head"], targets, ignore_index=-1,
                                          grad_weight=g["head"], accumulate=not first)
        dh, dx = None, loss.grad_x
        for b in reversed(range(self.blocks)):
            kept_x, kept_a, n = kept[b]
            d = fadam.block_norm_backward(dh, dx, n.f_checkpoint, n.h_checkpoint, n.rstd_post,
                                          n.rstd_pre, w[f"pre{b}"], post_weight=w[f"post{b}"],
                                          gate=w[f"gate{b}"], residual_scale=self.alpha)
            self._add(first, **{f"post{b}": d.post_weight, f"pre{b}": d.pre_weight, f"gate{b}": d.gate})
            fadam.checkpoint8_weight_grad(d.f, kept_a, out=g[f"down{b}"], accumulate=not first)
            da = (d.f @ w[f"down{b}"]) * (kept_a.codes > 0)
            fadam.checkpoint8_weight_grad(da, kept_x, out=g[f"up{b}"], accumulate=not first)
            dh, dx = d.h, da @ w[f"up{b}"]
        d = fadam.block_norm_backward(dh, dx, torch.zeros_like(h), start.h_out, None, start.rstd_pre,
                                      w["norm0"], gate=shut)
        self._add(first, norm0=d.pre_weight)
        if first:
            g["embed"].zero_()
        g["embed"].index_add_(0, tokens, d.h.float())
        return loss.loss

    def _add(self, first, **grads):
        for name, grad in grads.items():
            self.grads[name].copy_(grad) if first else self.grads[name].add_(grad)


def batches(vocab, rows, seed):
    """Sequences that count upwards by a step that the first two tokens give;
    the first target of each is masked (it cannot be known)."""
    gen = torch.Generator().manual_seed(seed)
    while True:
        begin = torch.randint(0, vocab, (rows // 32, 1), generator=gen)
        stride = torch.randint(1, 4, (rows // 32, 1), generator=gen)
        text = (begin + stride * torch.arange(33)) % vocab
        targets = text[:, 1:].clone()
        targets[:, 0] = -1
        yield text[:, :-1].reshape(-1).to(DEVICE), targets.reshape(-1).to(DEVICE)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--rows", type=int, default=2048)
    ap.add_argument("--micro-batches", type=int, default=2)
    a = ap.parse_args(argv)
    model, data, losses = Model(), batches(1000, a.rows, 1), []
    for step in range(a.steps):
        total = 0.0
        for i in range(a.micro_batches):
            total = total + model.step(*next(data), first=i == 0) / a.micro_batches
        model.optimizer.set_grad_scale(1.0 / a.micro_batches)
        model.optimizer.step()
        losses.append(float(total))
        if step % 10 == 0 or step == a.steps - 1:
            print(f"step {step}: loss {losses[-1]:.4f}")
    assert fadam.ops_status() == 0 and model.optimizer.device_status() == 0
    return losses


if __name__ == "__main__":
    main()
