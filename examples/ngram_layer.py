"""The front of a model around the hashed n-gram lookup, trained and then served
token by token, every step in the library's kernels (torch: the gate's small
product, the vocabulary's, the weights' SGD, the loss of the first run).

    r    = sqrt(C) * E[tokens]                      engram_embed (a float stream)
    e    = table[hash(tokens)]                      engram_lookup
    x    = norm of e, head by head                  engram_residual_norm, 8-bit checkpoint of x
    y    = causal dilated convolution of x          engram_ple_conv
    out  = r + scale * sigmoid(gate) * norm(y)      engram_residual_norm, 8-bit checkpoint of y
    next = norm(out)

The backward reads the checkpoints, not x and y; it ends in both tables: the
embedding's gradient by sorted tokens and the hashed rows' fused SignSGD step.

    logits = next E^T, the embedding's rows again
    loss and its gradient from a teacher's top logits     engram_distill
    a beam search: the best continuations, then the       engram_beam_select
    beams' rings and histories in their order             engram_beam_fork

    python examples/ngram_layer.py [--steps 20]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gram_hashed_embedding_amd import engram as E  # noqa: E402
from gram_hashed_embedding_amd import layer as L  # noqa: E402
from gram_hashed_embedding_amd import vocab as V  # noqa: E402
from gram_hashed_embedding_amd import workloads  # noqa: E402

KERNEL = 4


class NgramLayer:
    """The layer's weights (bf16, with float masters where SGD updates them)."""

    def __init__(self, wl, vocab, seed=0, device="cuda"):
        self.wl, self.heads = wl, wl.heads
        self.channels, self.dilation = wl.heads * wl.dim, wl.ngram_size
        self.scale = math.sqrt(self.channels)
        self.hash = (wl.ngram_size, wl.heads_per_ngram, wl.eos_id, wl.multipliers(), wl.primes,
                     wl.offsets)
        self.table = workloads.make_table(wl.table_rows, wl.dim, seed, device)
        C = self.channels
        g = torch.Generator(device).manual_seed(seed)

        def draw(*shape, std=1.0, mean=0.0):
            return torch.empty(shape, device=device).normal_(mean, std, generator=g)

        self.master = dict(embed=draw(vocab, C, std=0.02), w_in=draw(C, std=0.02, mean=1.0),
                           conv=draw(C, KERNEL, std=0.5), bias=draw(C, std=0.02),
                           w_post=draw(C, std=0.02, mean=1.0), scale=draw(C, std=0.02, mean=0.5),
                           w_next=draw(C, std=0.02, mean=1.0), gate=draw(C, self.heads, std=0.05))
        self.cast()

    def cast(self):
        self.w = {k: v.to(torch.bfloat16) for k, v in self.master.items()}

    def combine(self, r, y, codes=False):
        """The branch y added to the stream r, and the next norm."""
        gate = r.to(torch.bfloat16) @ self.w["gate"]
        return gate, L.engram_residual_norm(
            r, y, gate=gate, w_post=self.w["w_post"], scale=self.w["scale"],
            w_next=self.w["w_next"], groups=self.heads, save_codes=codes)

    def forward(self, tokens, seq_ids=None):
        """(next, what the backward needs)."""
        shape = (*tokens.shape, self.channels)
        r = L.engram_embed(tokens, self.w["embed"], self.scale, out_dtype=torch.float32)
        e = E.engram_lookup(tokens, self.table, *self.hash, seq_ids=seq_ids).view(shape)
        n = L.engram_residual_norm(e, w_next=self.w["w_in"], groups=self.heads, next_codes=True)
        y = E.engram_ple_conv(n.next, self.w["conv"], self.dilation, bias=self.w["bias"],
                              seq_ids=seq_ids)
        gate, f = self.combine(r, y, codes=True)
        kept = dict(tokens=tokens, seq_ids=seq_ids, r=r, e=e, rstd_in=n.rstd_next,
                    x_codes=n.next_codes, x_scales=n.next_scales, gate=gate, out=f.out,
                    rstd_post=f.rstd_post, rstd_next=f.rstd_next, y_codes=f.y_codes,
                    y_scales=f.y_scales)
        return f.next, kept

    def backward(self, d_next, kept, lr, table_lr):
        """Every weight's gradient, applied."""
        k, w, wl = kept, self.w, self.wl
        tokens = k["tokens"]
        b = L.engram_residual_norm_backward(
            None, d_next, out=k["out"], rstd_post=k["rstd_post"], rstd_next=k["rstd_next"],
            y_codes=k["y_codes"], y_scales=k["y_scales"], gate=k["gate"], w_post=w["w_post"],
            scale=w["scale"], w_next=w["w_next"], groups=self.heads)
        c = L.engram_ple_conv_backward(b.y, w["conv"], self.dilation, x_codes=k["x_codes"],
                                       x_scales=k["x_scales"], code_width=wl.dim,
                                       seq_ids=k["seq_ids"])
        a = L.engram_residual_norm_backward(None, c.x, out=k["e"], rstd_next=k["rstd_in"],
                                            w_next=w["w_in"], groups=self.heads)
        # the gate's product: its weight, and its part of the stream's gradient
        r = k["r"].view(-1, self.channels).to(torch.bfloat16)
        d_gate = b.gate.view(-1, self.heads)
        grads = dict(w_in=a.w_next, conv=c.weight, bias=c.bias, w_post=b.w_post, scale=b.scale,
                     w_next=b.w_next, gate=(r.t().contiguous() @ d_gate).float())
        d_r = b.residual + (d_gate @ w["gate"].t().contiguous()).view_as(b.residual)
        grads["embed"] = L.engram_embed_grad(tokens, d_r, w["embed"].shape[0], self.scale)
        plan = E.engram_scatter_plan_tokens(tokens, wl.table_rows, wl.dim, *self.hash,
                                            seq_ids=k["seq_ids"])
        E.engram_scatter_apply_signsgd(a.residual.view(-1, wl.dim), plan, self.table, table_lr)
        for name, g in grads.items():
            self.master[name] -= lr * g
        self.cast()

    # ---------------------------------------------------------- vocabulary --
    def logits(self, hidden):
        return hidden @ self.w["embed"].t()

    def distill(self, tokens, ids, teacher, lr, table_lr, **kw):
        """One step towards a teacher's top logits (ids, teacher [batch, seq, top]; further
        arguments as engram_distill's): the mean loss."""
        hidden, kept = self.forward(tokens)
        weight = torch.full(tokens.shape, 1.0 / tokens.numel(), device=tokens.device)
        logits = self.logits(hidden)
        d = V.engram_distill(logits, ids, teacher, grad_loss=weight, grad=logits, **kw)
        flat = d.grad.view(-1, d.grad.shape[-1])
        # the product's two gradients: the layer's, and the rows' as the vocabulary's side
        d_hidden = (flat @ self.w["embed"]).view_as(hidden)
        d_rows = (flat.t().contiguous() @ hidden.view(-1, self.channels)).float()
        self.backward(d_hidden, kept, lr, table_lr)
        self.master["embed"] -= lr * d_rows
        self.cast()
        return d.loss.mean()

    # ------------------------------------------------------------- serving --
    def ring(self, sequences, device="cuda"):
        """An empty ring of the convolution's latest inputs for each sequence."""
        rows = (KERNEL - 1) * self.dilation
        return torch.empty((sequences, rows, self.channels), dtype=torch.bfloat16, device=device)

    def step(self, history, position, ring, slots=None):
        """next for one token a sequence: history int64 [batch, up to n] ends in it, position
        int64 [batch] counts it from its sequence's start; slots: each sequence's ring."""
        batch, have = history.shape
        r = L.engram_embed(history[:, -1].contiguous(), self.w["embed"], self.scale,
                           out_dtype=torch.float32)
        e = E.engram_lookup_slice(history, have - 1, have, self.table, *self.hash)
        n = L.engram_residual_norm(e.view(batch, self.channels), w_next=self.w["w_in"],
                                   groups=self.heads)
        y = L.engram_ple_conv_step(n.next, ring, self.w["conv"], self.dilation, position,
                                   slots=slots, bias=self.w["bias"])
        return self.combine(r, y)[1].next

    def search(self, first, beams, steps, eos=-1):
        """A beam search of `steps` tokens after each sequence's `first` (int64 [batch]): (tokens
        [batch, beams, 1 + steps], scores [batch, beams], finished), the best first.  A beam
        that nothing is left for has score -inf."""
        batch, n = first.shape[0], self.wl.ngram_size
        device = first.device
        chosen = first[:, None, None].expand(batch, beams, 1).contiguous()
        # the first step has one beam; the others' scores keep them out of the choice
        scores = torch.full((batch, beams), -math.inf, device=device)
        scores[:, 0] = 0.0
        finished = torch.zeros((batch, beams), dtype=torch.bool, device=device)
        ring, slots = self.ring(batch * beams, device), None
        for t in range(steps):
            have = min(n, t + 1)
            # (a beam without tokens of its own, -1, steps on from token 0 and is not chosen)
            recent = chosen[:, :, t + 1 - have:].clamp(min=0).view(batch * beams, have)
            position = torch.full((batch * beams,), t, dtype=torch.int64, device=device)
            hidden = self.step(recent.contiguous(), position, ring,
                               None if slots is None else slots.view(-1))
            b = V.engram_beam_select(self.logits(hidden), scores, finished=finished if eos >= 0
                                     else None, eos=eos)
            f = V.engram_beam_fork(b.parents, ring, slots=slots, tokens=b.tokens, history=chosen,
                                   new_len=t + 2)
            scores, finished, slots, chosen = b.scores, b.finished, f.slots, f.history
        return chosen, scores, finished


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=0.5)
    ap.add_argument("--table-lr", type=float, default=1e-3)
    args = ap.parse_args(argv)
    wl = workloads.tiny()
    net = NgramLayer(wl, vocab=1000)
    tokens = torch.from_numpy(wl.tokens(0)).cuda()
    target = workloads.make_bf16((*tokens.shape, net.channels), 7, "cuda")
    losses = []
    for step in range(args.steps):
        out, kept = net.forward(tokens)
        diff = out.float() - target.float()
        losses.append(float(0.5 * diff.square().mean()))
        # the mean over positions, a sum over channels
        net.backward((diff / tokens.numel()).to(torch.bfloat16), kept, args.lr, args.table_lr)
        print(f"step {step}: loss {losses[-1]:.4f}", flush=True)

    whole, _ = net.forward(tokens)
    ring, worst = net.ring(wl.batch), 0.0
    for t in range(wl.seq):
        history = tokens[:, max(0, t + 1 - wl.ngram_size):t + 1].contiguous()
        position = torch.full((wl.batch,), t, dtype=torch.int64, device="cuda")
        one = net.step(history, position, ring)
        worst = max(worst, float((one.float() - whole[:, t].float()).abs().max()))
    print(f"{wl.seq} tokens one at a time: largest difference from the whole sequence {worst}")

    # a teacher of the same shape, of which the best 16 logits at every position are known
    teacher = NgramLayer(wl, vocab=1000, seed=1)
    told = teacher.logits(teacher.forward(tokens)[0]).float()
    top = torch.topk(told, 16, dim=-1)
    for step in range(min(args.steps, 5)):
        loss = net.distill(tokens, top.indices.contiguous(), top.values.contiguous(), args.lr,
                           args.table_lr, teacher_lse=torch.logsumexp(told, -1), rest=True)
        print(f"distillation step {step}: loss {float(loss):.4f}", flush=True)
    found, scores, _ = net.search(tokens[:, 0].contiguous(), beams=4, steps=6)
    for row, score in zip(found[0].tolist(), scores[0].tolist()):
        print(f"beam {row}: {score:.3f}")
    return losses, worst


if __name__ == "__main__":
    main()
