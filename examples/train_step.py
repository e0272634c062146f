"""One optimizer shard trained through the library's operators.

A small language model of residual blocks, written by hand: token embedding,
blocks of norm -> attention within its document, or two-layer perceptron ->
post-norm, gate, residual add, and the loss over the vocabulary.  What a
training step needs besides plain matrix products comes from the library:

  embedding, embedding_weight_grad   the rows of the embedding, and its gradient
  attention, attention_backward      over packed documents, capped scores and a
                                     bias by distance in place of positions
  block_norm, block_norm_backward    the norms around every block, forward and
                                     backward, keeping f and h_out in 8 bits
  checkpoint8                        the inputs of the linear layers, kept in 8
                                     bits
  checkpoint8_weight_grad            their weight gradients from those
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

    def __init__(self, vocab=1000, width=256, hidden=688, blocks=2, heads=4, kv_heads=2, lr=3e-3, seed=0):
        gen = torch.Generator().manual_seed(seed)
        shapes = {"embed": (vocab, width), "head": (vocab, width), "norm0": (width,)}
        head = width // heads
        for b in range(blocks):
            shapes |= {f"qkv{b}": ((heads + 2 * kv_heads) * head, width), f"out{b}": (width, width),
                       f"up{b}": (hidden, width), f"down{b}": (width, hidden)}
            for part in "am":      # around attention, around the perceptron
                shapes |= {f"post{part}{b}": (width,), f"pre{part}{b}": (width,),
                           f"gate{part}{b}": (1, width)}
        starts, total = {}, 0
        for name, shape in shapes.items():
            starts[name] = total
            total += -(-torch.Size(shape).numel() // 64) * 64     # views start on 128 bytes

        def buffer(dtype):
            return torch.zeros(total, dtype=dtype, device=DEVICE)

        def views(flat):
            return {n: flat[s:s + torch.Size(shapes[n]).numel()].view(shapes[n])
                    for n, s in starts.items()}

        self.blocks, self.alpha = blocks, (2 * blocks) ** -0.5
        self.heads, self.kv_heads, self.head = heads, kv_heads, head
        self.slopes = 2.0 ** (-8.0 * torch.arange(1, heads + 1, device=DEVICE) / heads)
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

    def _norm(self, name, f, h):
        """A block's output into the residual stream, and the next block's input."""
        w = self.w
        return fadam.block_norm(f, h, w["pre" + name], post_weight=w["post" + name], gate=w["gate" + name],
                                residual_scale=self.alpha, checkpoint=True)

    def _norm_backward(self, name, n, dh, dx, first):
        w = self.w
        d = fadam.block_norm_backward(dh, dx, n.f_checkpoint, n.h_checkpoint, n.rstd_post, n.rstd_pre,
                                      w["pre" + name], post_weight=w["post" + name],
                                      gate=w["gate" + name], residual_scale=self.alpha)
        self._add(first, **{"post" + name: d.post_weight, "pre" + name: d.pre_weight, "gate" + name: d.gate})
        return d

    def step(self, tokens, targets, documents=None, first=True):
        """Forward and backward of one micro-batch of packed documents, which
        start at the offsets `documents` (none: the tokens are one).  Gradients are
        added to those of the step's earlier micro-batches unless it is the first."""
        w, g, add = self.w, self.grads, not first
        masks = dict(documents=documents, slopes=self.slopes, softcap=30.0)
        shut = torch.zeros_like(w["norm0"]).view(1, -1)
        # the first norm is a block norm whose block adds nothing (gate 0)
        h = fadam.embedding(tokens, w["embed"])
        start = fadam.block_norm(h, h, w["norm0"], gate=shut)
        h, x, kept = start.h_out, start.x_out, []
        for b in range(self.blocks):
            qkv = (x @ w[f"qkv{b}"].t()).view(x.shape[0], -1, self.head)
            q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
            o = fadam.attention(q, k, v, **masks)
            rows = o.out.view(x.shape)
            na = self._norm(f"a{b}", rows @ w[f"out{b}"].t(), h)
            kept_qkv, kept_out, y = fadam.checkpoint8(x), fadam.checkpoint8(rows), na.x_out
            a = torch.relu(y @ w[f"up{b}"].t())
            nm = self._norm(f"m{b}", a @ w[f"down{b}"].t(), na.h_out)
            kept.append((kept_qkv, (q, k, v), o, kept_out, na, fadam.checkpoint8(y), fadam.checkpoint8(a), nm))
            h, x = nm.h_out, nm.x_out

        loss = fadam.linear_cross_entropy(x, w["head"], targets, ignore_index=-1,
                                          grad_weight=g["head"], accumulate=add)
        dh, dx = None, loss.grad_x
        for b in reversed(range(self.blocks)):
            kept_qkv, qkv, o, kept_out, na, kept_y, kept_a, nm = kept[b]
            d = self._norm_backward(f"m{b}", nm, dh, dx, first)
            fadam.checkpoint8_weight_grad(d.f, kept_a, out=g[f"down{b}"], accumulate=add)
            da = (d.f @ w[f"down{b}"]) * (kept_a.codes > 0)
            fadam.checkpoint8_weight_grad(da, kept_y, out=g[f"up{b}"], accumulate=add)
            d = self._norm_backward(f"a{b}", na, d.h, da @ w[f"up{b}"], first)
            fadam.checkpoint8_weight_grad(d.f, kept_out, out=g[f"out{b}"], accumulate=add)
            do = (d.f @ w[f"out{b}"]).view(o.out.shape)
            dqkv = torch.cat(fadam.attention_backward(do, *qkv, o.out, o.lse, **masks), 1).flatten(1)
            fadam.checkpoint8_weight_grad(dqkv, kept_qkv, out=g[f"qkv{b}"], accumulate=add)
            dh, dx = d.h, dqkv @ w[f"qkv{b}"]
        d = fadam.block_norm_backward(dh, dx, torch.zeros_like(h), start.h_out, None, start.rstd_pre,
                                      w["norm0"], gate=shut)
        self._add(first, norm0=d.pre_weight)
        fadam.embedding_weight_grad(d.h, tokens, out=g["embed"], accumulate=add)
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
        yield (text[:, :-1].reshape(-1).to(DEVICE), targets.reshape(-1).to(DEVICE),
               torch.arange(0, rows // 32 * 32 + 1, 32, dtype=torch.int32, device=DEVICE))


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
