"""What the GPU tests of the gated recurrence, the short convolution and layer norm share: inputs that are exact in
their type, and comparisons with the float64 forms value by value."""
import numpy as np
import torch

import _recurrent_ref as ref

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def host(t):
    return None if t is None else t.double().cpu().numpy()


def rnd(shape, kind, seed, scale=1.0):
    """A tensor and its values."""
    t = (torch.from_numpy(np.random.default_rng(seed).standard_normal(shape)) * scale).cuda().to(TYPES[kind])
    return t, host(t)


def close(got, want, name):
    """Each value within its bound and half a step of its type (a flushed denormal besides)."""
    value, bound = want
    kind = "bf16" if got.dtype == torch.bfloat16 else "f32"
    g = host(got)
    assert g.shape == value.shape, name
    room = bound + ref.HALF[kind] * (np.abs(value) + bound) + 1e-36
    off = np.abs(g - value)
    bad = ~(off <= room)
    assert not bad.any(), "%s: %d of %d off, worst %.3g where %.3g is allowed, at %s" % (
        name, bad.sum(), bad.size, off[bad].max(), room[bad][off[bad].argmax()], np.argwhere(bad)[off[bad].argmax()])


def same(a, b):
    """Equal bits, through tuples and dicts."""
    if isinstance(a, dict):
        return a.keys() == b.keys() and all(same(a[k], b[k]) for k in a)
    if isinstance(a, (tuple, list)):
        return len(a) == len(b) and all(same(x, y) for x, y in zip(a, b))
    if a is None or b is None:
        return a is b
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
