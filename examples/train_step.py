"""Training a small language model of RG-LRU or selective state space blocks with the package's operators.

    python examples/train_step.py [--steps N] [--bits 8|32] [--mixer rglru|ssm]

A model of `layers` residual blocks: each takes the normed stream through one
projection to a branch and a gate, mixes the branch over time by the RG-LRU
layer, norms it, gates it, scales it, adds it to the FP32 residual stream and norms the
sum for the next block (block_norm does all of the last five).  The head is
tied to the embedding; its loss never forms the logits (linear_ce).  One AdamW
step updates all weights, BF16 copies of FP32 ones (adamw_step).

With the state space mixer a block's branch goes through the short convolution and the selective
scan instead, gated by the other half of its projection, and the tokens through the embedding lookup; such a
model also generates (`generate`): a prompt at once, then token by token on the states that it leaves.

The data is synthetic: each token follows from the one before by a fixed
permutation most of the time, which the model learns in a few hundred steps.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from linear_recurrence_sequence_amd import autograd, lm, ssm  # noqa: E402

bf, f32 = torch.bfloat16, torch.float32


class Model:
    """Weights in BF16 with FP32 copies, or FP32 where an operator takes that; names map to tensors."""

    def __init__(self, vocab, d, layers, device="cuda", seed=0, mixer="rglru", states=16, taps=4):
        g = torch.Generator(device=device).manual_seed(seed)
        self.layers, self.vocab, self.d, self.mixer, self.states, self.rank = layers, vocab, d, mixer, states, d // 16

        def normal(*shape, std):
            return torch.randn(shape, generator=g, device=device) * std

        m = {"embed": normal(vocab, d, std=d ** -0.5)}
        v = {"norm_in": torch.ones(d, device=device)}
        for i in range(layers):
            m[f"in{i}"] = normal(2 * d, d, std=d ** -0.5)
            if mixer == "rglru":
                for k in ("x", "a"):
                    m[f"w_{k}{i}"] = normal(16, d // 16, d // 16, std=(d // 16) ** -0.5)
                    v[f"b_{k}{i}"] = torch.zeros(d, device=device)
                v[f"alpha{i}"] = torch.full((d,), 2.0, device=device)
            else:
                m[f"proj{i}"] = normal(self.rank + 2 * states, d, std=d ** -0.5)      # what dt is formed from, b and c
                m[f"dt{i}"] = normal(d, self.rank, std=self.rank ** -0.5)
                v[f"conv{i}"], v[f"conv_bias{i}"] = normal(d, taps, std=taps ** -0.5), torch.zeros(d, device=device)
                step = torch.exp(torch.rand(d, generator=g, device=device) * 4.6 - 6.9)   # 0.001 to 0.1
                v[f"dt_bias{i}"] = step + torch.log(-torch.expm1(-step))                  # softplus of it is the step
                v[f"log_rate{i}"] = torch.log(torch.arange(1.0, states + 1, device=device)).repeat(d, 1)
                v[f"skip{i}"] = torch.ones(d, device=device)
            for k in ("w_post", "w_pre"):
                v[f"{k}{i}"] = torch.ones(d, device=device)
            v[f"scale{i}"] = torch.full((d,), 0.5, device=device)
        self.matrices = {k: t.to(bf).requires_grad_() for k, t in m.items()}
        self.masters = m
        self.vectors = {k: t.requires_grad_() for k, t in v.items()}

    def loss(self, tokens, targets, z_weight=1e-4):
        """Mean cross entropy over the targets that are not negative, with a penalty on lse^2."""
        m, v = self.matrices, self.vectors
        if self.mixer == "ssm":
            x = autograd.embed(tokens, m["embed"], out_dtype=f32)
            x, n = autograd.block_norm(x, torch.zeros_like(x, dtype=bf), None, None, None, v["norm_in"])
        else:
            x = torch.nn.functional.embedding(tokens, m["embed"])
            x, n = autograd.block_norm(x.float(), torch.zeros_like(x), None, None, None, v["norm_in"])
        for i in range(self.layers):
            both = n @ m[f"in{i}"].t()
            if self.mixer == "ssm":
                u, _ = autograd.causal_conv(both[..., : self.d], v[f"conv{i}"], v[f"conv_bias{i}"])
                y, _ = autograd.ssm_scan(u, **self.scan_args(i, u, both))
                x, n = autograd.block_norm(x, y, None, v[f"w_post{i}"], v[f"scale{i}"], v[f"w_pre{i}"])
                continue
            y, _ = autograd.rglru_layer(both[..., : self.d].contiguous(), m[f"w_x{i}"], v[f"b_x{i}"], m[f"w_a{i}"], v[f"b_a{i}"],
                                        v[f"alpha{i}"])
            x, n = autograd.block_norm(x, y, both[..., self.d:], v[f"w_post{i}"], v[f"scale{i}"], v[f"w_pre{i}"], gate_act="silu")
        loss, lse = autograd.linear_ce(n, m["embed"], targets, softcap=30.0)
        counts = (targets >= 0).sum()
        return loss.sum() / counts + z_weight * (lse * lse).mean(), loss.sum().detach() / counts

    def scan_args(self, i, u, both):
        """What the scan of block i takes beside u, for one token or many: the projections of u, and the gate."""
        m, v = self.matrices, self.vectors
        p = u @ m[f"proj{i}"].t()
        b, c = (p[..., self.rank + k * self.states:self.rank + (k + 1) * self.states].unsqueeze(-2) for k in (0, 1))
        return dict(dt=p[..., : self.rank] @ m[f"dt{i}"].t(), a=-torch.exp(v[f"log_rate{i}"]), b=b, c=c, d=v[f"skip{i}"], z=both[..., self.d:],
                    dt_bias=v[f"dt_bias{i}"])

    @torch.no_grad()
    def run(self, tokens, states=None, lengths=None):
        """(last rows of the logits, states) of prompts [batch, length], or of one token each [batch] on the states that a prompt left,
        which move on in place.  lengths: of prompts that are padded."""
        m, v, one = self.matrices, self.vectors, tokens.dim() == 1
        states = [None] * self.layers if states is None else states
        x = lm.embed_fwd(tokens, m["embed"], out_dtype=f32)
        x, n, _ = lm.block_norm_fwd(x, torch.zeros_like(x, dtype=bf), None, None, None, v["norm_in"])
        for i in range(self.layers):
            both = n @ m[f"in{i}"].t()
            branch, w, bias = both[..., : self.d], v[f"conv{i}"], v[f"conv_bias{i}"]
            if one:
                taps, h = states[i]
                u = ssm.causal_conv_step(branch, w, bias, taps)
                y = ssm.ssm_scan_step(h, u, **self.scan_args(i, u, both))
            else:
                u, taps = ssm.causal_conv_fwd(branch, w, bias, lengths=lengths)
                y, h, _ = ssm.ssm_scan_fwd(u, **self.scan_args(i, u, both), lengths=lengths, want_saved=False)
                states[i] = taps, h
            x, n, _ = lm.block_norm_fwd(x, y, None, v[f"w_post{i}"], v[f"scale{i}"], v[f"w_pre{i}"])
        if not one:
            last = (tokens.shape[1] if lengths is None else lengths.long()) - 1
            n = n[torch.arange(n.shape[0], device=n.device), last]
        return n @ m["embed"].t(), states

    def generate(self, prompts, count, lengths=None):
        """The `count` likeliest tokens after each prompt [batch, length], one after the other."""
        logits, states = self.run(prompts, lengths=lengths)
        out = [logits.argmax(-1)]
        for _ in range(count - 1):
            logits, states = self.run(out[-1], states)
            out.append(logits.argmax(-1))
        return torch.stack(out, 1)


class AdamW:
    def __init__(self, model, lr=3e-3, weight_decay=0.01, bits=8):
        self.model, self.lr, self.decay, self.t = model, lr, weight_decay, 0
        self.state = {k: lm.adamw_state(p, bits) for k, p in {**model.matrices, **model.vectors}.items()}

    def step(self):
        self.t += 1
        for params, masters, decay in ((self.model.matrices, self.model.masters, self.decay), (self.model.vectors, None, 0.0)):
            s = [self.state[k] for k in params]
            eight = "m_scale" in s[0]
            lm.adamw_step([p.data for p in params.values()], [p.grad for p in params.values()], [a["m"] for a in s], [a["v"] for a in s],
                          step=self.t, lr=self.lr, betas=(0.9, 0.95), weight_decay=decay,
                          masters=None if masters is None else [masters[k] for k in params],
                          m_scales=[a["m_scale"] for a in s] if eight else None, v_scales=[a["v_scale"] for a in s] if eight else None)
            for p in params.values():
                p.grad = None


def batch(vocab, rows, length, gen, follow):
    """Tokens, and the next ones as targets; a tenth of the targets do not count."""
    t = torch.randint(0, vocab, (rows, length + 1), generator=gen, device="cuda")
    keep = torch.rand((rows, length + 1), generator=gen, device="cuda") < 0.9
    for i in range(1, length + 1):
        t[:, i] = torch.where(keep[:, i], follow[t[:, i - 1]], t[:, i])
    drop = torch.rand((rows, length), generator=gen, device="cuda") < 0.1
    return t[:, :-1].contiguous(), torch.where(drop, torch.full_like(t[:, 1:], -100), t[:, 1:]).contiguous()


def train(steps=200, vocab=512, d=256, layers=2, rows=4, length=128, bits=8, seed=0, report=20, mixer="rglru"):
    """Runs `steps` steps and returns the losses."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    follow = torch.randperm(vocab, generator=gen, device="cuda")
    model = Model(vocab, d, layers, seed=seed, mixer=mixer)
    opt = AdamW(model, bits=bits)
    losses = []
    for i in range(steps):
        tokens, targets = batch(vocab, rows, length, gen, follow)
        loss, ce = model.loss(tokens, targets)
        loss.backward()
        opt.step()
        losses.append(float(ce))
        if report and i % report == 0:
            print(f"step {i:4d}  cross entropy {losses[-1]:.4f}", flush=True)
    return losses


if __name__ == "__main__":
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--steps", type=int, default=200)
    a.add_argument("--bits", type=int, default=8, choices=(8, 32))
    a.add_argument("--mixer", default="rglru", choices=("rglru", "ssm"))
    a = a.parse_args()
    out = train(steps=a.steps, bits=a.bits, mixer=a.mixer)
    print(f"last cross entropy {out[-1]:.4f}")
