"""GPU test of the gated recurrence over a long row, every value against float64: what 16384 tokens leave of a rounding."""
import pytest
import torch

from _recurrent_gpu import TYPES, close
from test_gpu_gated_scan import make, run, want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("C", [72, 33])
def test_a_long_row(C, kind):
    """drate's sum takes 160 roundings at most: 128 tokens of a thread (512 tiles in clusters of 16, four tokens each), the
    warp's two groups, four warps and 16 blocks; single channels 256 tokens (eight each), so twice the room."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    t = make(1, 16384, C, kind, h0=True, marks=0.0005, seed=C)
    got, exp = run(t), want(t)
    for n, (value, bound) in exp.items():
        close(got[n], (value, 2 * bound if n == "drate" and C % 2 else bound), n)
