"""A gated delta rule mixer: prompt, streaming and training.

    python examples/delta_mixer.py

Tokens are projected to queries, keys, values and gates; queries and keys get
unit norm and their position's rotation in one call; the gated delta rule mixes
the sequence.  The prompt runs as one call that leaves the state, generation
goes on from it token by token, and a few training steps fit a batch to its own
delayed copy.  The projections and the gates' functions are torch
here; the mixer's operators are the library's calls.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from diagonal_state_space_gb300 import api, init  # noqa: E402


class DeltaMixer:
    """x [B, L, H] -> y [B, L, H] with Hk key heads and Hv value heads of D."""

    def __init__(self, H, Hk=2, Hv=4, D=128, rot=64, seed=0, device="cuda"):
        self.Hk, self.Hv, self.D = Hk, Hv, D
        gen = torch.Generator(device=device).manual_seed(seed)
        w = lambda n, m: torch.randn(n, m, generator=gen, device=device) * m ** -0.5  # noqa: E731
        # rows: q, k, v, decay, beta
        self.w_in = w(2 * Hk * D + Hv * D + 2 * Hv, H)
        self.w_out = w(H, Hv * D)
        self.log_a = torch.zeros(Hv, device=device)
        freq, self.amp = init.rotary_frequencies(rot)
        self.freq = torch.from_numpy(freq).to(device)

    def parameters(self):
        return dict(w_in=self.w_in, w_out=self.w_out, log_a=self.log_a)

    def _inputs(self, x, start):
        """The operators' inputs, and what their backward pass needs."""
        B, L, _ = x.shape
        Hk, Hv, D = self.Hk, self.Hv, self.D
        p = x @ self.w_in.t()
        n = 2 * Hk * D + Hv * D
        qkv = p[..., :n].to(torch.bfloat16)      # one array; q, k and v are views of it
        q, k = qkv[..., :Hk * D].unflatten(-1, (Hk, D)), qkv[..., Hk * D:2 * Hk * D].unflatten(-1, (Hk, D))
        v = qkv[..., 2 * Hk * D:].unflatten(-1, (Hv, D))
        a, b = p[..., n:n + Hv], p[..., n + Hv:]
        g = -torch.exp(self.log_a) * torch.nn.functional.softplus(a - 3.0)
        beta = torch.sigmoid(b)
        pos = (torch.arange(L, device=x.device) + start).expand(B, L).contiguous()
        qn, kn = api.s5_qk_norm_rotary(q, k, pos, self.freq, norm="l2", amplitude=self.amp)
        return dict(q=q, k=k, v=v, a=a, g=g, beta=beta, pos=pos, qn=qn, kn=kn)

    def forward(self, x, state=None, start=0, keep=False):
        """y and the state after x; with keep also what backward() takes."""
        t = self._inputs(x, start)
        saved = api.new_delta_saved(t["qn"], t["v"]) if keep else None
        o, last = api.s5_delta_forward(t["qn"], t["kn"], t["v"], t["g"], t["beta"], s0=state, s_last=True, saved=saved)
        y = o.float().flatten(-2) @ self.w_out.t()
        return (y, last, dict(t, x=x, o=o, saved=saved)) if keep else (y, last)

    def step(self, x, state, position):
        """One token x [B, H]; state is updated in place."""
        t = {n: u[:, 0] for n, u in self._inputs(x[:, None], position).items()}
        o = api.s5_delta_step(t["qn"], t["kn"], t["v"].contiguous(), t["g"], t["beta"], state)
        return o.float().flatten(-2) @ self.w_out.t()

    def backward(self, kept, dy):
        """Gradients of sum(dy * y) by the parameters."""
        x, o = kept["x"], kept["o"]
        dw_out = dy.flatten(0, 1).t() @ o.float().flatten(-2).flatten(0, 1)
        do = (dy @ self.w_out).unflatten(-1, (self.Hv, self.D)).to(torch.bfloat16)
        d = api.s5_delta_backward(kept["qn"], kept["kn"], kept["v"], kept["g"], kept["beta"], do, kept["saved"])
        n = api.s5_qk_norm_rotary_backward(kept["q"], kept["k"], d["dq"], d["dk"], kept["pos"], self.freq, norm="l2",
                                           amplitude=self.amp)
        db = d["dbeta"] * kept["beta"] * (1 - kept["beta"])
        da = -d["dg"] * torch.exp(self.log_a) * torch.sigmoid(kept["a"] - 3.0)
        dp = torch.cat([n["dq"].flatten(-2), n["dk"].flatten(-2), d["dv"].flatten(-2)], -1).float()
        dp = torch.cat([dp, da, db], -1)
        return dict(w_in=dp.flatten(0, 1).t() @ x.flatten(0, 1), w_out=dw_out, log_a=(d["dg"] * kept["g"]).sum((0, 1)))


def finished():
    """Raises if a wait inside the mixer's kernels ran out: their results are then not valid."""
    if api.s5_delta_fault() or api.s5_rotary_fault():
        raise RuntimeError("a wait inside a mixer kernel ran out")


def prompt_and_stream(B=2, L=200, H=256, tokens=8, seed=1):
    """Largest difference of streamed outputs from those of one call over all
    tokens, over the outputs' size."""
    m = DeltaMixer(H, seed=seed)
    x = torch.randn(B, L + tokens, H, device="cuda")
    want, _ = m.forward(x)
    y, state = m.forward(x[:, :L])
    got = [m.step(x[:, L + i], state, L + i) for i in range(tokens)]
    got = torch.cat([y] + [u[:, None] for u in got], 1)
    finished()
    return float((got - want).norm() / want.norm())


def train(steps=60, B=2, L=128, H=64, lag=1, rate=3e-3, seed=2):
    """Losses while one batch is fitted to its own delayed copy y_t = x_{t - lag} (Adam)."""
    m = DeltaMixer(H, seed=seed)
    x = torch.randn(B, L, H, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")
    target = torch.nn.functional.pad(x, (0, 0, lag, 0))[:, :L]
    moments = {n: (torch.zeros_like(p), torch.zeros_like(p)) for n, p in m.parameters().items()}
    losses = []
    for i in range(1, steps + 1):
        y, _, kept = m.forward(x, keep=True)
        losses.append(float((y - target).square().mean()))
        grads = m.backward(kept, 2 * (y - target) / y.numel())
        for name, p in m.parameters().items():
            a, b = moments[name]
            a.lerp_(grads[name], 0.1)
            b.lerp_(grads[name].square(), 0.01)
            p -= rate * (a / (1 - 0.9 ** i)) / ((b / (1 - 0.99 ** i)).sqrt() + 1e-8)
    finished()
    return losses


if __name__ == "__main__":
    print("streaming against one call: relative difference %.2e" % prompt_and_stream())
    losses = train()
    print("loss %.4f -> %.4f in %d steps" % (losses[0], losses[-1], len(losses)))
