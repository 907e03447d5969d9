"""How near the layers around RMA attention come to FP32 arithmetic, against the FP64 oracle.

Beside the elementwise bounds, a share: how many BF16 outputs are not the rounding of the oracle's value.  A value
whose error before the rounding is e is rounded to a neighbour with probability 2 e / step, the step between BF16 values
being 2^-8 to 2^-7 of the value.  FP32 arithmetic, or factors carried in 22 bits (a pair of FP16 or TF32 values without
lo x lo, 2^-22), leaves errors of a few 2^-22 of the terms, taken together less than 2^-20 of the sum of the absolute
terms since they are of either sign.  That sum is about 2^4 of the value for sums of 128 and more terms of either sign:
2 * 2^-20 * 2^4 / 2^-8 = 2^-7 of the outputs, a hundredth at most.  One factor of 11 bits (2^-12 of each term, of either
sign: 2^-15 to 2^-16 of their sum) makes it a tenth and more.
"""
import numpy as np
import pytest
import torch

import oracle
from _gpu import lib  # noqa: F401
from test_gpu_layers import BF, _device, close, delta_case, f64  # noqa: F401

pytestmark = pytest.mark.gpu


def share_off(got, ref):
    """Share of the finite entries of `ref` whose BF16 rounding `got` is not."""
    live = ~np.isnan(ref)
    want = torch.from_numpy(np.where(live, ref, 0.0)).to(torch.float32).to(BF).double().numpy()
    return (f64(got).reshape(ref.shape) != want)[live].mean()


def delta_reference(x, hk, **more):
    return oracle.delta_rule(*[f64(x[k]) for k in ("qkv", "a", "b", "a_log", "dt_bias", "state")], hk, **more)


@pytest.mark.parametrize("batch,n,hk,hv,fresh", [(1, 100, 4, 8, True), (2, 64, 1, 4, False), (3, 130, 2, 2, False),
                                                 (40, 70, 1, 5, False), (1, 2050, 1, 2, True)])
def test_block_outputs_are_of_fp32_arithmetic(batch, n, hk, hv, fresh):
    rma, st, d, x = delta_case(batch, n, hk, hv, seed=300 + n, fresh=fresh)
    out = torch.empty(batch, n, hv, 128, dtype=BF, device="cuda")
    rma.gdn_prefill(st, 0, d["qkv"], d["a"], d["b"], d["a_log"], d["dt_bias"], out, st.workspace(n))
    ref, S, osize, _ = delta_reference(x, hk)
    # sums of 128 terms and more in accumulators of 23 bits: at most 2^-16 of their absolute sum, in the updates and again here
    close(out, ref, 2.0 ** -15 * osize, "out")
    assert share_off(out, ref) <= 0.01
