"""Corners of the expert-layer operators on the GPU: what the header promises where
inputs are not finite, sizes are extreme or contractions long."""
import numpy as np
import pytest
import torch

from tests import experts_ref as R
from tests.test_gpu_experts import (HALF_ULP, TINY, TYPES, check_form, close, hard_matrix, rnd,
                                    strided, te)

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


# The matrix cores cut every product of a group of eight toward zero at 2^-13 of the power
# of two of the group's largest, so that the other seven lose less than 7 * 2^-13 of it
# together; sixteen products at a time go into the float32 sum, which then is off by a unit
# of its last place at most (2^-23 of the terms before it).
def sum_bound(k):
    return 7 * 2.0 ** -13 + k * 2.0 ** -27


def check_sums(y, a, b, k, half_ulp):
    """y against the float64 sums over the represented values a [m, k], b [n, k]."""
    want = torch.zeros(a.shape[0], b.shape[0], dtype=torch.float64, device="cuda")
    terms = torch.zeros_like(want)
    for i in range(0, a.shape[1], 1 << 18):
        p, q = a[:, i:i + (1 << 18)].double(), b[:, i:i + (1 << 18)].double().t().contiguous()
        want += p @ q
        terms += p.abs() @ q.abs()
    off = (y.double() - want).abs() - half_ulp * want.abs()
    assert float((off / terms).max()) <= sum_bound(k)


def test_product_where_small_terms_stand_beside_large_ones():
    """Large terms that cancel leave what the small ones sum to, within the bound."""
    k = 256
    x = torch.full((64, k), 1.875 * 2.0 ** -6)
    x[:, ::8] = 256.0 * torch.tensor([1.0, -1.0]).repeat(k // 16)
    for i in range(64):  # every distance, and signs that do not cancel
        x[i] *= torch.where(torch.arange(k) % 8 == 0, 2.0 ** -(i % 16), 1.0)
        if i >= 32:
            x[i] = x[i].abs()
    a = te().quantize_f8(x.cuda())
    b = te().quantize_f8(torch.ones(5, k).cuda())
    assert torch.equal(a.float(), x.cuda())
    check_sums(te().matmul_f8(a, b, dtype=torch.float16), a.float(), b.float(), k, 2.0 ** -11)


@pytest.mark.parametrize("kind", ["positive", "constant", "wide"])
def test_segment_product_over_half_a_million_rows(kind):
    """The gradient of weights over long segments of terms of one sign, a short one beside."""
    ends, p, q = [0, 128, 128 + (1 << 19), 128 + (1 << 19) + 256], 40, 33
    rows = ends[-1]
    g = torch.Generator(device="cuda").manual_seed(3)

    def values(width, c):
        if kind == "constant":
            return torch.full((rows, width), c, device="cuda")
        v = torch.rand(rows, width, generator=g, device="cuda")
        return v + 0.5 if kind == "positive" else torch.exp2(-16 * v)
    x, y = values(p, 1.125).to(torch.bfloat16), values(q, 1.375).to(torch.bfloat16)
    a, b = te().quantize_f8(x, transpose=True), te().quantize_f8(y, transpose=True)
    out = te().matmul_f8_segments(a, b, torch.tensor(ends, dtype=torch.int32).cuda())
    av, bv = a.float(), b.float()
    for e in range(3):
        s = slice(ends[e], ends[e + 1])
        check_sums(out[e], av[:, s], bv[:, s], ends[e + 1] - ends[e], 2.0 ** -8)


@pytest.mark.parametrize("kind", ["positive", "constant"])
def test_product_over_four_million_columns(kind):
    k = 1 << 22
    g = torch.Generator(device="cuda").manual_seed(4)

    def values(rows, c):
        if kind == "constant":
            return torch.full((rows, k), c, dtype=torch.bfloat16, device="cuda")
        return (torch.rand(rows, k, generator=g, device="cuda") + 0.5).to(torch.bfloat16)
    a, b = te().quantize_f8(values(32, 1.125)), te().quantize_f8(values(24, 1.125))
    check_sums(te().matmul_f8(a, b), a.float(), b.float(), k, 2.0 ** -8)


def bad_places(x, spread):
    """x with infinities and NaN at even and odd columns and rows, at the ends of blocks,
    beside the largest finite value, and a block of nothing else."""
    inf, nan = float("inf"), float("nan")
    r, c = x.shape
    for i, (row, col, v) in enumerate([(0, 0, inf), (0, 3, -inf), (1, 126, nan), (1, 128, inf),
                                       (2, 127, -nan), (2, 200, inf), (r - 1, c - 1, nan),
                                       (r - 1, c - 2, -inf), (r // 2, 64, inf), (r // 2, 65, nan)]):
        if row < r and col < c and (spread or i % 2):
            x[row, col] = v
    if r > 5 and c > 128:
        x[4, :128] = inf
        x[5, :128:2], x[5, 1:128:2] = nan, -inf
        x[3, 130 % c] = torch.finfo(x.dtype).max
    return x


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("r,c,pad", [(9, 256, 0), (130, 259, 0), (257, 136, 1), (6, 130, 8)])
def test_quantize_not_finite(r, c, pad, spread, dtype):
    """Infinities and NaN become NaN in every form and type, and leave the scales to the
    finite elements beside them."""
    x = bad_places(hard_matrix(r, c, dtype, 3), spread)
    h = R.f64(x)
    x = strided(x, pad) if pad else x
    for square in (False, True):
        check_form(te().quantize_f8(x, square=square), h, square, "rows")
        check_form(te().quantize_f8(x, transpose=True, square=square), h.T, square, "columns")
        a, b = te().quantize_f8_pair(x, square=square)
        check_form(a, h, square, "pair rows")
        check_form(b, h.T, square, "pair columns")


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("n,width", [(9, 256), (130, 259), (6, 1030)])
def test_dispatch_f8_not_finite(n, width, dtype):
    g = np.random.default_rng([n, width])
    ids = g.integers(-1, 5, size=(n, 3))
    r = te().ExpertRows(torch.from_numpy(ids).int().cuda(), 5, align=16)
    x = bad_places(hard_matrix(n, width, dtype, 4), True)
    rows = R.f64(r.dispatch(x))
    check_form(r.dispatch_f8(x), rows, False, "dispatched")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("e", [7, 64, 65, 128, 129, 256, 300, 512, 513, 1024])
def test_route_gradient_of_every_layout_by_probability(e, dtype):
    """Each element of the gradient within its own softmax term's bound."""
    k = min(e, 9)
    g = np.random.default_rng([e, 2])
    x = torch.from_numpy(g.integers(-40, 41, size=(11, e)) / 8.0).to(TYPES[dtype]).cuda()
    x[3, ::3] = -float("inf")
    for renorm in (False, True):
        ids, _ = te().route(x, k, renormalize=renorm)
        dw = rnd(11, k, seed=e)
        h, pick = R.f64(x), ids.cpu().numpy().astype(np.int64)
        want = R.route_backward(h, pick, R.f64(dw), renorm)
        p = np.exp(h - h.max(axis=1, keepdims=True))
        chosen = np.zeros_like(p)
        np.put_along_axis(chosen, np.where(pick < 0, 0, pick), 1.0, 1)
        p = p * chosen if renorm else p
        p /= p.sum(axis=1, keepdims=True)
        # p and the dot product carry the softmax's (e + 8) roundings each, and the
        # difference of two terms of at most max|dw| its own
        scale = 2 * np.abs(R.f64(dw)).max(axis=1, keepdims=True)
        close(te().route_backward(x, ids, dw, renormalize=renorm), want,
              (2 * e + 16) * 2.0 ** -24 * scale * p + HALF_ULP[dtype] * np.abs(want)
              + TINY[dtype], "grad_logits")


def test_products_repeat_themselves():
    """The same bits from the same operands, whatever the tile."""
    for rows, n, k in ((300, 200, 1000), (2300, 2100, 520), (6500, 2304, 512)):
        a, b = te().quantize_f8(rnd(rows, k, dtype="bf16")), te().quantize_f8(rnd(n, k, seed=2))
        first = te().matmul_f8(a, b)
        assert all(torch.equal(te().matmul_f8(a, b), first) for _ in range(4)), (rows, n, k)
        ends = torch.tensor([0, 128, 512], dtype=torch.int32).cuda()
        at = te().quantize_f8(rnd(512, rows, dtype="bf16"), transpose=True)
        bt = te().quantize_f8(rnd(512, n, dtype="bf16", seed=3), transpose=True)
        one = te().matmul_f8_segments(at, bt, ends)
        assert all(torch.equal(te().matmul_f8_segments(at, bt, ends), one) for _ in range(4))
