"""A small recurrent language model trained data-parallel with compressed gradients.

The whole step runs through this library:

    layer norm -> gates and inputs (adacomp_linear) -> gated recurrence -> adacomp_linear onto the residual stream
    softmax cross entropy over the vocabulary, whose logits are not kept (adacomp_vocab_loss)
    every learner compresses its gradients (adacomp_compress_group)
    the learners' messages are summed (adacomp_decode_accumulate_group)
    the sum's norm clips it (adacomp_grad_norm), and AdamW takes the step (adacomp_adamw_step)

The learners run one after the other on one GPU, each on its own batch and with its own
residues. Tensors of less than 4096 elements (norms) are summed as they are. The text is a
random Markov chain, so the least loss is known: its entropy. `generate` continues a text
one token at a time, handing the recurrence's state on.

    python examples/recurrent_lm.py [--steps 200] [--learners 2] [--state-bits 8]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import residual_gradient_compression_gb300 as ac  # noqa: E402


class LayerNorm(torch.autograd.Function):
    """Rows of x normalised; h: adacomp_layer_norm_init."""

    @staticmethod
    def forward(ctx, x, w, b, h):
        rows = x.numel() // x.shape[-1]
        y = torch.empty_like(x)
        mean, rstd = torch.empty(rows, device=x.device), torch.empty(rows, device=x.device)
        ac.adacomp_layer_norm_forward(h, x, w, b, y, mean, rstd)
        ctx.save_for_backward(x, w, mean, rstd)
        ctx.h = h
        return y

    @staticmethod
    def backward(ctx, dy):
        x, w, mean, rstd = ctx.saved_tensors
        dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
        ws = torch.empty(ac.adacomp_layer_norm_backward_ws_bytes(ctx.h, mean.numel()), dtype=torch.uint8, device=x.device)
        ac.adacomp_layer_norm_backward(ctx.h, dy.contiguous(), x, w, mean, rstd, dx, dw, db, ws)
        return dx, dw, db, None


class Recurrence(torch.autograd.Function):
    """zx: the gates' and the inputs' halves of one buffer [batch, steps, 2 * channels]."""

    @staticmethod
    def forward(ctx, zx, h):
        batch, steps, c = zx.shape[0], zx.shape[1], zx.shape[2] // 2
        y = torch.empty(batch, steps, c, dtype=zx.dtype, device=zx.device)
        carry = torch.empty(ac.adacomp_recurrence_carry_bytes(h, batch, steps) // 4, device=zx.device)
        ac.adacomp_recurrence_forward(h, zx[..., :c], zx[..., c:], y, carry=carry)
        ctx.save_for_backward(zx, carry)
        ctx.h = h
        return y

    @staticmethod
    def backward(ctx, dy):
        zx, carry = ctx.saved_tensors
        c, dzx = zx.shape[2] // 2, torch.empty_like(zx)
        ac.adacomp_recurrence_backward(ctx.h, zx[..., :c], zx[..., c:], dy.contiguous(), carry, dzx[..., :c], dzx[..., c:])
        return dzx, None


class Linear(torch.autograd.Function):
    """x w^T, onto a residual if there is one; h: adacomp_linear_init."""

    @staticmethod
    def forward(ctx, x, w, residual, h):
        y = torch.empty(*x.shape[:-1], w.shape[0], dtype=x.dtype, device=x.device)
        ws = scratch(ac.adacomp_linear_forward_ws_bytes(h, x.numel() // x.shape[-1]), x)
        ac.adacomp_linear_forward(h, x, w, y, ws, residual=residual)
        ctx.save_for_backward(x, w)
        ctx.h, ctx.added = h, residual is not None
        return y

    @staticmethod
    def backward(ctx, dy):
        x, w = ctx.saved_tensors
        dy, dx, dw = dy.contiguous(), torch.empty_like(x), torch.empty_like(w)
        ws = scratch(ac.adacomp_linear_backward_ws_bytes(ctx.h, x.numel() // x.shape[-1]), x)
        ac.adacomp_linear_backward(ctx.h, dy, x, w, ws, dx=dx, dw=dw)
        return dx, dw, dy if ctx.added else None, None


class CrossEntropy(torch.autograd.Function):
    """Each row's loss against the rows of w; negative targets have none. h: adacomp_vocab_init."""

    @staticmethod
    def forward(ctx, x, w, target, h):
        rows = target.numel()
        loss, lse = torch.empty(rows, device=x.device), torch.empty(rows, device=x.device)
        ac.adacomp_vocab_loss_forward(h, x, w, target, loss, lse, scratch(ac.adacomp_vocab_loss_forward_ws_bytes(h, rows), x))
        ctx.save_for_backward(x, w, target, lse)
        ctx.h = h
        return loss

    @staticmethod
    def backward(ctx, dloss):
        x, w, target, lse = ctx.saved_tensors
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        ws = scratch(ac.adacomp_vocab_loss_backward_ws_bytes(ctx.h, target.numel()), x)
        ac.adacomp_vocab_loss_backward(ctx.h, x, w, target, lse, dloss.contiguous(), ws, dx=dx, dw=dw)
        return dx, dw, None, None


def scratch(nbytes, like):
    return torch.empty(nbytes, dtype=torch.uint8, device=like.device)


class Model:
    """Weights in one flat list: embedding, and per block (norm w, norm b, gates and inputs, output)."""

    def __init__(self, vocab=64, width=128, blocks=2, seed=0):
        g = torch.Generator().manual_seed(seed)
        init = lambda *s, scale: (torch.randn(*s, generator=g) * scale).cuda().requires_grad_()  # noqa: E731
        self.width, self.blocks = width, blocks
        self.weights = [init(vocab, width, scale=0.02)]
        for _ in range(blocks):
            gates = init(2 * width, width, scale=width ** -0.5)
            self.weights += [torch.ones(width, device="cuda", requires_grad=True),
                             torch.zeros(width, device="cuda", requires_grad=True), gates,
                             init(width, width, scale=width ** -0.5)]
        self.weights += [torch.ones(width, device="cuda", requires_grad=True),
                         torch.zeros(width, device="cuda", requires_grad=True)]
        self.norm = ac.adacomp_layer_norm_init(width, ac.F32, ac.F32, 1e-5)
        self.recurrence = ac.adacomp_recurrence_init(width, ac.F32)
        self.gates, self.proj = ac.adacomp_linear_init(width, 2 * width), ac.adacomp_linear_init(width, width)
        self.head, self.vocab = ac.adacomp_linear_init(width, vocab), ac.adacomp_vocab_init(width, vocab)

    def hidden(self, tokens):
        w = self.weights
        x = w[0][tokens]
        for i in range(self.blocks):
            nw, nb, gates, out = w[1 + 4 * i:5 + 4 * i]
            zx = Linear.apply(LayerNorm.apply(x, nw, nb, self.norm), gates, None, self.gates)
            x = Linear.apply(Recurrence.apply(zx, self.recurrence), out, x, self.proj)
        return LayerNorm.apply(x, w[-2], w[-1], self.norm)

    def logits(self, tokens):
        return Linear.apply(self.hidden(tokens), self.weights[0], None, self.head)

    def loss(self, tokens):
        x = self.hidden(tokens[:, :-1])
        return CrossEntropy.apply(x.reshape(-1, self.width), self.weights[0], tokens[:, 1:].reshape(-1), self.vocab).mean()

    @torch.no_grad()
    def generate(self, tokens, count):
        """The likeliest continuation, one token at a time; returns tokens and the last logits."""
        batch, w, c = tokens.shape[0], self.weights, self.width
        states = [torch.zeros(batch, c, device="cuda") for _ in range(self.blocks)]
        y, n = torch.empty(batch, 1, c, device="cuda"), torch.empty(batch, c, device="cuda")
        zx, logits = torch.empty(batch, 1, 2 * c, device="cuda"), torch.empty(batch, w[0].shape[0], device="cuda")
        ws = scratch(max(ac.adacomp_linear_forward_ws_bytes(h, batch) for h in (self.gates, self.proj, self.head)), n)
        out = tokens
        for t in range(tokens.shape[1] + count - 1):
            x = w[0][out[:, t]]
            for i, state in enumerate(states):
                nw, nb, gates, proj = w[1 + 4 * i:5 + 4 * i]
                ac.adacomp_layer_norm_forward(self.norm, x, nw, nb, n)
                ac.adacomp_linear_forward(self.gates, n, gates, zx, ws)
                ac.adacomp_recurrence_forward(self.recurrence, zx[..., :c], zx[..., c:], y, h0=state, h_last=state)
                ac.adacomp_linear_forward(self.proj, y, proj, x, ws, residual=x)
            ac.adacomp_layer_norm_forward(self.norm, x, w[-2], w[-1], n)
            ac.adacomp_linear_forward(self.head, n, w[0], logits, ws)
            if t + 1 >= tokens.shape[1]:
                out = torch.cat([out, logits.argmax(1, keepdim=True)], 1)
        return out, logits


class Exchange:
    """The learners' compressed gradients and their sum."""

    def __init__(self, weights, learners, bin_len=50):
        big = [i for i, w in enumerate(weights) if w.numel() >= 4096]
        self.big, self.small = big, [i for i in range(len(weights)) if i not in big]
        ns = [weights[i].numel() for i in big]
        self.learners, self.layers = learners, len(big)
        zeros = lambda n, t: torch.zeros(n, dtype=t, device="cuda")  # noqa: E731
        self.h = ac.adacomp_init_group(ns, [bin_len] * len(big), [ac.F32] * len(big))
        self.residues = [[zeros(n, torch.float32) for n in ns] for _ in range(learners)]
        self.messages = [[zeros(b, torch.uint8) for b in self.h.max_msg_bytes] for _ in range(learners)]
        self.ws = [zeros(self.h.compress_ws_bytes, torch.uint8) for _ in range(learners)]
        self.decode_ws = zeros(self.h.decode_ws_bytes(learners), torch.uint8)
        self.sum = [torch.zeros_like(w) for w in weights]

    def compress(self, learner, grads):
        ac.adacomp_compress_group(self.h, self.residues[learner], [grads[i] for i in self.big], self.messages[learner],
                                  self.ws[learner])
        for i in self.small:
            self.sum[i] += grads[i]

    def gather(self):
        """The sum over the learners, and the bytes of their messages."""
        lengths = [[ac.adacomp_query(self.h, ws, layer)[0] for layer in range(self.layers)] for ws in self.ws]
        ac.adacomp_decode_accumulate_group(
            self.h, [[self.messages[k][l] for k in range(self.learners)] for l in range(self.layers)],
            [[lengths[k][l] for k in range(self.learners)] for l in range(self.layers)],
            [self.sum[i] for i in self.big], self.decode_ws)
        if ac.adacomp_decode_status(self.h, self.decode_ws) != ac.OK:
            raise RuntimeError("a message was rejected")
        return self.sum, sum(map(sum, lengths))

    def clear(self):
        for t in self.sum:
            t.zero_()


class AdamW:
    """Moments in 32 or 8 bits; matrices decay, norms do not."""

    def __init__(self, weights, state_bits, decay=0.01):
        ns, types = [w.numel() for w in weights], [ac.F32] * len(weights)
        self.h = ac.adacomp_adamw_init(ns, types, types, [decay if w.dim() > 1 else 0.0 for w in weights], state_bits)
        kind = torch.float8_e4m3fn if state_bits == 8 else torch.float32
        zeros = lambda sizes, t=torch.float32: ac.adacomp_pointers(  # noqa: E731
            [torch.zeros(n, dtype=torch.float32, device="cuda").to(t) for n in sizes])
        self.weights = ac.adacomp_pointers([w.detach() for w in weights])
        self.m, self.v = zeros(ns, kind), zeros(ns, kind)
        blocks = [-(-n // ac.ADAMW_BLOCK) for n in ns]
        self.m_scale, self.v_scale = (zeros(blocks), zeros(blocks)) if state_bits == 8 else (None, None)
        self.ws = torch.zeros(self.h.norm_ws_bytes, dtype=torch.uint8, device="cuda")
        self.norm = torch.zeros(2, device="cuda")  # the norm, and the coefficient for the step
        self.steps = 0

    def step(self, grads, grad_scale, lr=3e-3, betas=(0.9, 0.99), eps=1e-8, max_norm=1.0):
        self.steps += 1
        ac.adacomp_grad_norm(self.h, grads, self.norm, self.ws, max_norm=max_norm, grad_scale=grad_scale)
        ac.adacomp_adamw_step(self.h, self.weights, grads, self.m, self.v, lr, *betas, eps, 1 - betas[0] ** self.steps,
                              1 - betas[1] ** self.steps, m_scale=self.m_scale, v_scale=self.v_scale,
                              coefficient=self.norm[1:])


class Text:
    """A random Markov chain over the vocabulary with a few likely successors for every token."""

    def __init__(self, vocab=64, successors=4, seed=1):
        g = torch.Generator().manual_seed(seed)
        p = torch.zeros(vocab, vocab)
        for t in range(vocab):
            p[t, torch.randperm(vocab, generator=g)[:successors]] = torch.rand(successors, generator=g) + 0.2
        self.p = (p / p.sum(1, keepdim=True)).cuda()
        self.g = torch.Generator(device="cuda").manual_seed(seed + 1)

    def entropy(self):
        p = self.p.double()
        state = torch.full((p.shape[0],), 1.0 / p.shape[0], dtype=torch.float64, device="cuda")
        for _ in range(200):
            state = state @ p
        return float(-(state[:, None] * p * torch.log(p.clamp(min=1e-300))).sum())

    def batch(self, rows, steps):
        t = [torch.randint(0, self.p.shape[0], (rows,), generator=self.g, device="cuda")]
        for _ in range(steps):
            t.append(torch.multinomial(self.p[t[-1]], 1, generator=self.g)[:, 0])
        return torch.stack(t, 1)


def train(steps=200, learners=2, state_bits=8, rows=16, length=64, report=None):
    """Returns the model and each step's mean loss over the learners."""
    text, model = Text(), Model()
    exchange, adamw = Exchange(model.weights, learners), AdamW(model.weights, state_bits)
    losses = []
    for step in range(steps):
        exchange.clear()
        total = 0.0
        for k in range(learners):
            loss = model.loss(text.batch(rows, length))
            exchange.compress(k, torch.autograd.grad(loss, model.weights))
            total += float(loss.detach()) / learners
        grads, sent = exchange.gather()
        adamw.step(grads, 1.0 / learners)
        losses.append(total)
        if report and (step % 20 == 0 or step == steps - 1):
            dense = 4 * learners * sum(model.weights[i].numel() for i in exchange.big)
            report(f"step {step:4d}  loss {total:.3f} (entropy {text.entropy():.3f}, chance {math.log(64):.3f})  "
                   f"gradient norm {float(adamw.norm[0]):.3f}  sent {sent} of {dense} bytes")
    return model, losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--learners", type=int, default=2)
    ap.add_argument("--state-bits", type=int, default=8, choices=(8, 32))
    a = ap.parse_args()
    model, _ = train(a.steps, a.learners, a.state_bits, report=print)
    text = Text(seed=1).batch(2, 4)
    print("continued:", model.generate(text, 12)[0].tolist())


if __name__ == "__main__":
    main()
