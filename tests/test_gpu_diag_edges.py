"""The diagonal scan's calls where they meet the rest of a program: memory that
another stream still uses, prompts among single tokens, states that forget at
once, slots of earlier states given back."""
import numpy as np
import pytest
import torch

import diag_ref as R
import ssd_selective_scan_b200 as ssd
import test_gpu_diag as fwd
import test_gpu_diag_bwd as bwd

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
DTYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])

def test_results_do_not_take_memory_in_use():
    """A result on another stream is not laid into a block that was freed on
    the current one while work there still reads it."""
    p = R.scan_inputs((2, 600), 64, 16, 1, F32, seed=3, device="cuda")
    want, _ = ssd.diag_scan_fwd(**p)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [torch.ones_like(want) for _ in range(8)]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)              # about 0.1 s
    copies = [h.clone() for h in held]          # waits behind it
    del held
    results = [ssd.diag_scan_fwd(**p, stream=side) for _ in range(4)]
    torch.cuda.synchronize()
    for c in copies:
        assert (c == 1).all()
    for y, _ in results:
        assert torch.equal(y, want)
