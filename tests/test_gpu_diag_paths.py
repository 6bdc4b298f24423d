"""The diagonal scan's calls on paths that only some sizes take: dense batches
that are not cut, packed ones taken longest first, long gradient pieces; and
what NaN in one row reaches in the gradients."""
import pytest
import torch

import diag_ref as R
import ssd_selective_scan_b200 as ssd
import test_gpu_diag as fwd

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def test_dense_scan_that_is_not_cut_takes_no_workspace():
    """16384 sequences of one token, and 600 of 100: results, and what the call
    allocates beside them."""
    for b, L, E in ((16384, 1, 128), (600, 100, 64)):
        p = R.scan_inputs((b, L), E, 16, 1, F32, seed=b, device="cuda")
        init = 0.5 * torch.randn(b, E, 16, device="cuda")
        y, fs = torch.empty(b, L, E, device="cuda"), torch.empty_like(init)
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        held = torch.cuda.memory_allocated()
        ssd.diag_scan_fwd(**p, init_state=init, y=y, final_state=fs)
        assert torch.cuda.max_memory_allocated() == held
        some = [0, 1, b // 2, b - 1]
        ry, rf = fwd.dense_ref({k: (v[some] if v is not None and k in ("u", "dt_raw", "B", "C", "z") else v) for k, v in p.items()}, init[some])
        R.close(y[some], ry, "y")
        R.close(fs[some], rf, "final state")
