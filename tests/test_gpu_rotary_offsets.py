"""GPU test of offsets past 32 bits inside one token of the rotation."""
import numpy as np
import pytest
import torch

from diagonal_state_space_gb300 import api

import _mixer_ref as ref
from _parity import check

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_a_token_of_more_than_2_31_values(layout):
    H, D = (1 << 28) + 515, 8
    x = torch.empty(1, H, D, device="cuda", dtype=torch.bfloat16).normal_()
    pos, freq = torch.tensor([12345], device="cuda"), np.array([1.0, 0.1, 0.01, 0.001])
    y = api.s5_rotary(x, pos, torch.from_numpy(freq).cuda(), layout=layout)
    for rows in (slice(0, 600), slice((1 << 27) - 300, (1 << 27) + 300), slice((1 << 28) - 300, H)):
        want = ref.turn(x[:, rows].double().cpu().numpy(), np.array([12345]), freq, layout, 1.0)
        # 16 roundings of 2^-24 and the one to bf16, as in test_gpu_rotary.py
        check(y[:, rows].double().cpu().numpy(), want, 16 * 2.0 ** -24 + 2.0 ** -8, "y")
