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


@pytest.mark.parametrize("square", [False, True])
def test_every_scale_byte_stands_for_the_same_in_checks_and_products(square):
    """F8Matrix.float() and the product agree on all 256 bytes: 2^(s - 127), NaN for 255."""
    rows = 256 * (128 if square else 1)
    values = torch.full((rows, 128), 448.0).to(torch.float8_e4m3fn).cuda()
    values[:, 1::2] = 0
    scales = torch.zeros(256, 4, dtype=torch.uint8)
    scales[:, 0] = torch.arange(256)
    a = te().F8Matrix(values, scales.cuda(), rows, 128, square)
    want = 448.0 * np.exp2(np.arange(256) - 127.0)
    got = R.f64(a.float())[::128 if square else 1]
    assert np.isnan(got[255]).all() and not np.isnan(got[:255]).any()
    # 448 * 2^(s - 127) passes float32 from s = 247 on
    assert np.array_equal(got[:247, 0], want[:247]) and np.isinf(got[247:255, 0]).all()
    assert not got[:255, 1].any()
    # against 64 elements of 2^-6 at the scale that brings the sum to 448 * 2^-3
    one = torch.full((1, 128), 2.0 ** -6).to(torch.float8_e4m3fn).cuda()
    for s in (0, 1, 2, 100, 127, 200, 247, 253, 254):
        by = torch.zeros(1, 4, dtype=torch.uint8)
        by[0, 0] = 254 - s - 3 if s < 252 else 0
        b = te().F8Matrix(one, by.cuda(), 1, 128)
        y = R.f64(te().matmul_f8(b, a))[0, ::128 if square else 1]
        assert y[s] == 448 * 2.0 ** (s - 127 + int(by[0, 0]) - 127)
        assert np.isnan(y[255])
