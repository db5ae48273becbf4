"""Corners of the expert-layer operators on the GPU: what the header promises where
inputs are not finite, sizes are extreme or contractions long."""
import numpy as np
import pytest
import torch

from tests import experts_ref as R
from tests.test_gpu_experts import TYPES, te

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------ router


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("e", [8, 70, 300])
def test_route_absent_choices_weigh_zero_beside_nan_and_inf(e, dtype):
    """A row with fewer than k live experts ends in ids -1 and weights 0, also where a
    live logit is NaN or +inf."""
    x = torch.full((4, e), -float("inf"))
    x[0, 2] = float("nan")
    x[1, 3], x[1, 4] = float("inf"), 1.0
    x[2, 5], x[2, 1] = float("nan"), 2.0
    x[3, 6] = 0.5
    for renorm in (False, True):
        ids, w = te().route(x.to(TYPES[dtype]).cuda(), 5, renormalize=renorm)
        want_ids, want_w = R.route(x.double().numpy(), 5, None, renorm)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        assert np.array_equal(R.f64(w), want_w, equal_nan=True)


# ------------------------------------------------------------------ 8-bit product


def test_product_of_a_segment_of_almost_2_to_31_rows():
    """Its row tiles are counted without passing 32 bits (without a contraction: the
    operands take no memory, the results are zeros)."""
    m = (1 << 31) - 2
    a, b = te().quantize_f8(torch.empty(m, 0).cuda()), te().quantize_f8(torch.empty(1, 0).cuda())
    offsets = torch.tensor([0, m], dtype=torch.int32).cuda()
    y = torch.full((m, 1), 7.0, dtype=torch.bfloat16, device="cuda")
    te().tbe_matmul_f8(a, b, offsets, y)
    assert not y.any()
