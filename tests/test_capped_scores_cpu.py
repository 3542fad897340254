"""Without a GPU: the formulas of capped scores in the decode kernels, emulated step by step in float32 and compared with float64 over caps and scores of every size."""
import numpy as np
import pytest

F = np.float32
LOG2E = F(1.4426950408889634)


def capped_log2(z, cap, exp2_error=0.0, any_cap=True):
    """cap tanh(z / cap) log2 e; exp2_error: relative error given to the exponential."""
    z = z.astype(F)
    inn, out = F(2.0 * 1.4426950408889634 / cap), F(1.4426950408889634 * cap)
    w = (z * inn).astype(F)
    t = (w * w).astype(F)
    with np.errstate(over="ignore"):
        e = (np.exp2(w.astype(np.float64)) * (1 + exp2_error)).astype(F)
    r = (F(2) / (F(1) + e)).astype(F)
    far = (out.astype(np.float64) - out.astype(np.float64) * r).astype(F)  # one rounding, as a fused multiply-add
    if not any_cap:
        return far
    p = (t.astype(np.float64) * F(1.923608e-3) + F(-4.0037751e-2)).astype(F)
    p = (t.astype(np.float64) * p + 1.0).astype(F)
    near = ((z * LOG2E).astype(F) * p).astype(F)
    return np.where(np.abs(w) < F(0.36067376), near, far)


# ex2.approx is within 2^-22 of the value; the quotient within 2 units in the last place of a value below 2, the
# subtraction rounds once: (2^-23 + 2^-22 + 2^-24) / tanh(1/8) = 3.4e-6 at most, less above; the series 2.1e-7 and four
# roundings. Scores are fp32 numbers.
@pytest.mark.parametrize("cap", [1e-6, 0.05, 1.0, 30.0, 50.0, 147.0, 150.0, 1e3, 1e4, 1e5, 1e6])
@pytest.mark.parametrize("exp2_error", [0.0, 2.0 ** -22, -(2.0 ** -22)])
def test_relative_error(cap, exp2_error):
    u = np.concatenate([np.linspace(-3, 3, 200_001), np.geomspace(1e-9, 40, 100_000), -np.geomspace(1e-9, 40, 100_000)])
    z = (u * cap).astype(F)
    z = z[z != 0]
    want = cap * np.tanh(z.astype(np.float64) / cap) * 1.4426950408889634
    got = capped_log2(z, cap, exp2_error).astype(np.float64)
    assert np.abs(got / want - 1).max() <= 3.4e-6


@pytest.mark.parametrize("cap", [1e3, 1e4, 1e5, 1e6])
def test_scores_of_ordinary_size_under_a_large_cap(cap):
    # the error of a weight is that of its score times ln 2: 2^-8 is a bf16 rounding of the weight
    z = np.linspace(-60, 60, 400_001).astype(F)
    want = cap * np.tanh(z.astype(np.float64) / cap) * 1.4426950408889634
    assert np.abs(capped_log2(z, cap).astype(np.float64) - want).max() * np.log(2) <= 2.0 ** -12


@pytest.mark.parametrize("cap", [1e-6, 0.05, 1.0, 30.0, 147.0])
def test_the_plain_form_serves_small_caps(cap):
    # 1 - 2 / (1 + e^2u) for every u: the error of a score, times ln 2, is that of its weight
    u = np.concatenate([np.linspace(-12, 12, 400_001), np.geomspace(1e-9, 1, 50_000)])
    z = (u * cap).astype(F)
    want = cap * np.tanh(z.astype(np.float64) / cap) * 1.4426950408889634
    for err in (0.0, 2.0 ** -22, -(2.0 ** -22)):
        assert np.abs(capped_log2(z, cap, err, any_cap=False).astype(np.float64) - want).max() * np.log(2) <= 1e-4


def test_limits():
    z = np.array([np.inf, -np.inf, 0.0, 3e38, -3e38], F)
    with np.errstate(all="ignore"):
        got = capped_log2(z, 5.0)
    full = F(1.4426950408889634 * 5.0)
    assert got.tolist() == [full, -full, 0.0, full, -full]
