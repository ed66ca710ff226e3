"""smoke() passes, and runs every kernel family that it is there to try."""
import pytest
import torch

import __graft_entry__ as entry

pytestmark = pytest.mark.gpu
KERNELS = ["fwd_simt", "fwd_tc", "gemm_tc", "delta_prep", "delta_scan", "delta_adjoint", "delta_local", "column_sweep",
           "row_sweep", "decay_grads", "delta_step", "rotary_fwd", "rotary_bwd"]


def test_smoke_runs_the_kernels():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from torch.profiler import ProfilerActivity, profile
    with profile(activities=[ProfilerActivity.CUDA]):     # the first one of a process may record nothing
        torch.zeros(1, device="cuda").add_(1)
        torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        entry.smoke()
        torch.cuda.synchronize()
    names = " ".join(e.key for e in p.key_averages())
    if "kernel" not in names:
        pytest.skip("the profiler records no kernels here")
    assert not [k for k in KERNELS if k not in names]
