"""A stack of gated recurrent blocks: prompt, streaming and training.

    python examples/gated_recurrence.py

A block adds what the block before gave to the stream and norms the sum in one
call, projects it, runs a short convolution along the tokens and the gated
linear recurrence over what comes out, and multiplies with a second branch.  The
prompt runs as one call a block that leaves the convolution's last inputs and
the recurrence's state, generation goes on from them token by token, and a few
training steps fit a batch of packed documents to its own delayed copy.  The
projections are torch here; the rest is the library's calls.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from diagonal_state_space_gb300 import api  # noqa: E402

silu = torch.nn.functional.silu


class GatedStack:
    """x [B, L, H] -> [B, L, H] through `layers` blocks of C channels; dtype is the operators'."""

    def __init__(self, H, C, layers=2, taps=4, dtype=torch.float32, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        w = lambda n, m: torch.randn(n, m, generator=gen, device=device) * m ** -0.5  # noqa: E731
        self.dtype, self.taps = dtype, taps
        self.layers = [dict(norm=torch.ones(H, device=device), shift=torch.zeros(H, device=device), w_in=w(C, H), w_side=w(C, H),
                            conv=w(C, taps), bias=torch.zeros(C, device=device), w_a=w(C, C), w_x=w(C, C), w_out=w(H, C),
                            lam=torch.linspace(-5.0, 1.0, C, device=device)) for _ in range(layers)]

    def _project(self, p, n):
        n = n.float()
        return (n @ p["w_in"].t()).to(self.dtype), n @ p["w_side"].t()

    def _gates(self, p, c):
        c = c.float()
        return (c @ p["w_a"].t()).to(self.dtype), (c @ p["w_x"].t()).to(self.dtype)

    def forward(self, x, states=None, reset=None, keep=False):
        """The output and each block's (last inputs, state); with keep also what backward() takes."""
        total, delta, out, kept = None, x.to(self.dtype), [], []
        for i, p in enumerate(self.layers):
            past, h0 = (None, None) if states is None else states[i]
            saved = api.new_layernorm_saved(delta) if keep else None
            into, resid = delta, total
            n = api.s5_add_layernorm(delta, p["norm"], p["shift"], residual=resid, saved=saved)
            n, total = (n, delta) if resid is None else n
            u, side = self._project(p, n)
            c, past = api.s5_short_conv_forward(u, p["conv"], bias=p["bias"], activation="silu", past=past, past_out=True, reset=reset)
            a, g = self._gates(p, c)
            rate = torch.nn.functional.softplus(p["lam"])
            scan = api.new_gated_scan_saved(c) if keep else None
            h, last = api.s5_gated_scan_forward(c, a, g, rate, h0=h0, h_last=True, reset=reset, saved=scan)
            delta = ((h.float() * silu(side)) @ p["w_out"].t()).to(self.dtype)
            out.append((past, last))
            if keep:
                kept.append(dict(into=into, resid=resid, n=n, saved=saved, u=u, side=side, c=c, a=a, g=g, rate=rate, scan=scan, h=h))
        y = total.float() + delta.float()
        return (y, out, dict(layers=kept, reset=reset)) if keep else (y, out)

    def step(self, x, states):
        """One token x [B, H]; the states are updated in place."""
        total, delta = None, x.to(self.dtype)
        for p, (past, state) in zip(self.layers, states):
            n = api.s5_add_layernorm(delta, p["norm"], p["shift"], residual=total)
            n, total = (n, delta) if total is None else n
            u, side = self._project(p, n)
            c = api.s5_short_conv_step(u, p["conv"], past, bias=p["bias"], activation="silu")
            a, g = self._gates(p, c)
            h = api.s5_gated_scan_step(c, a, g, torch.nn.functional.softplus(p["lam"]), state)
            delta = ((h.float() * silu(side)) @ p["w_out"].t()).to(self.dtype)
        return total.float() + delta.float()

    def backward(self, kept, dy):
        """Gradients of sum(dy * y) by the parameters, a dict a block, and by x."""
        flat = lambda t: t.float().flatten(0, 1)  # noqa: E731
        reset, grads = kept["reset"], []
        dtotal = ddelta = dy.to(self.dtype)
        for p, k in zip(reversed(self.layers), reversed(kept["layers"])):
            prod, s = k["h"].float() * silu(k["side"]), torch.sigmoid(k["side"])
            d = ddelta.float() @ p["w_out"]
            out = dict(w_out=flat(ddelta).t() @ flat(prod))
            dside = d * k["h"].float() * s * (1 + k["side"] * (1 - s))
            g = api.s5_gated_scan_backward(k["c"], k["a"], k["g"], k["rate"], (d * silu(k["side"])).to(self.dtype), k["scan"], reset=reset)
            out.update(w_a=flat(g["dgate_a"]).t() @ flat(k["c"]), w_x=flat(g["dgate_x"]).t() @ flat(k["c"]),
                       lam=g["drate"] * torch.sigmoid(p["lam"]))
            dc = (g["dx"].float() + g["dgate_a"].float() @ p["w_a"] + g["dgate_x"].float() @ p["w_x"]).to(self.dtype)
            v = api.s5_short_conv_backward(k["u"], p["conv"], dc, bias=p["bias"], activation="silu", reset=reset)
            out.update(conv=v["dweight"], bias=v["dbias"], w_in=flat(v["dx"]).t() @ flat(k["n"]), w_side=flat(dside).t() @ flat(k["n"]))
            dn = (v["dx"].float() @ p["w_in"] + dside @ p["w_side"]).to(self.dtype)
            m = api.s5_add_layernorm_backward(k["into"], dn, k["saved"], p["norm"], p["shift"], residual=k["resid"], dtotal=dtotal)
            out.update(norm=m["dweight"], shift=m["dbias"])
            dtotal = ddelta = m["dx"]
            grads.append(out)
        return grads[::-1], ddelta


def finished():
    """Raises if a wait inside the recurrence's kernels ran out: their results are then not valid."""
    if api.s5_gated_scan_fault():
        raise RuntimeError("a wait inside a kernel ran out")


def prompt_and_stream(B=2, L=200, H=64, C=96, tokens=8, dtype=torch.float32, seed=1):
    """Largest difference of streamed outputs from those of one call over all tokens, over the outputs' size."""
    m = GatedStack(H, C, dtype=dtype, seed=seed)
    x = torch.randn(B, L + tokens, H, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")
    want, _ = m.forward(x)
    y, states = m.forward(x[:, :L].contiguous())
    got = torch.cat([y] + [m.step(x[:, L + i].contiguous(), states)[:, None] for i in range(tokens)], 1)
    finished()
    return float((got - want).norm() / want.norm())


def train(steps=60, B=2, L=256, H=64, C=96, lag=1, rate=3e-3, seed=2):
    """Losses while one batch of packed documents is fitted to its own delayed copy y_t = x_{t - lag} (Adam)."""
    m = GatedStack(H, C, seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(B, L, H, generator=gen, device="cuda")
    reset = torch.rand(B, L, generator=gen, device="cuda") < 1 / 64
    target = torch.nn.functional.pad(x, (0, 0, lag, 0))[:, :L].masked_fill(reset[..., None], 0.0)
    moments = [{n: (torch.zeros_like(p), torch.zeros_like(p)) for n, p in layer.items()} for layer in m.layers]
    losses = []
    for i in range(1, steps + 1):
        y, _, kept = m.forward(x, reset=reset, keep=True)
        losses.append(float((y - target).square().mean()))
        grads, _ = m.backward(kept, 2 * (y - target) / y.numel())
        for layer, mom, g in zip(m.layers, moments, grads):
            for name, p in layer.items():
                a, b = mom[name]
                a.lerp_(g[name], 0.1)
                b.lerp_(g[name].square(), 0.01)
                p -= rate * (a / (1 - 0.9 ** i)) / ((b / (1 - 0.99 ** i)).sqrt() + 1e-8)
    finished()
    return losses


if __name__ == "__main__":
    print("streaming against one call: relative difference %.2e" % prompt_and_stream())
    losses = train()
    print("loss %.4f -> %.4f in %d steps" % (losses[0], losses[-1], len(losses)))
