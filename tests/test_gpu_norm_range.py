"""fs_block_norm and fs_block_norm_bwd at the ends of their ranges, against a statement in 64 bits (GPU
only).  Tolerances as in test_gpu_norm.py: half a step of the result's type, and 2^-18 (bf16 x) or 2^-19
(fp32) of the terms' magnitudes, twice that in the backward pass."""
import pytest
import torch

from long_context_lm_gb300 import fs
import layer_ref as ref
from test_gpu_norm import BF, FP, TYPES, loss, make, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 33])
@pytest.mark.parametrize("D,groups", [(40, 5), (64, 1), (64, 8), (100, 1), (256, 4), (512, 1), (512, 16), (1024, 16)])
@pytest.mark.parametrize("dt,rdt", TYPES)
@pytest.mark.parametrize("next", [False, True])
def test_gradients_with_eps_0(M, D, groups, dt, rdt, next):
    # rows that are not zero have factors without eps, and a block's places without a row add nothing
    form, next_gain, dz, dy = make(M, D, dt, rdt, True, True, True, seed=D + M)
    form.update(groups=groups, scale=0.7, eps=0.0)
    dy, next_gain = (dy, next_gain) if next else (None, None)
    got = fs.fs_block_norm_bwd(dz=dz, dy=dy, next_gain=next_gain, **form)
    want = ref.norm_grads(dz=dz, dy=dy, next_gain=next_gain, **form)
    for n in ("x", "gate", "residual", "gain", "next_gain"):
        assert (got[n] is None) == (n == "next_gain" and not next)
        if got[n] is not None:
            near(got[n], *want[n], 2 * loss(dt))
