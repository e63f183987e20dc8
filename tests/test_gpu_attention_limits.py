"""The operators around the projections where numbers leave the ordinary range:
normalised rows past bf16's and fp32's ends, against their 64-bit forms; and where
the launch changes with the length."""

import numpy as np
import pytest
import torch

import segmented_rank_gemm_amd as srg
from tests import attention_reference as R
from tests.test_gpu_attention import Call, check_norm, nearest_e4m3, norm_case

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ norm
def nearest_bf16(v):
    """(v rounded to bf16, how far each v is from a border between two of them)."""
    a = np.abs(v)
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(a, 1e-300))), -126) - 7)
    n = a / step
    near = np.abs(n - np.floor(n) - 0.5) * step
    rounded = np.rint(n) * step
    return np.copysign(np.where(rounded >= 2.0 ** 128, np.inf, rounded), v), near


def check_rows(x, w, group):
    """The norm of x (no residual, eps 0), each output the nearest of its type."""
    T, hidden = x.shape
    y, y8 = torch.empty_like(x), torch.empty(T, hidden, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(T, hidden // group, device="cuda")
    srg.lora_rms_norm(x, w, 0.0, y=y, y8=y8, scales=scales)
    _, v, s = R.rms_norm(x, None, w, 0.0, group)
    want, near = nearest_bf16(v)
    got = R.f64(y)
    # of the values that are not next to a border (one rounding to fp32 in between)
    ok = near > 2.0 ** -23 * np.abs(v) + 2.0 ** -149
    assert not np.isnan(got).any()
    assert (got == want)[ok].all(), (got != want)[ok].sum()
    # at most half a step from it elsewhere; past the largest number, the infinity
    fine = np.abs(v) < 2.0 ** 128 * (1 - 2.0 ** -9)
    assert (np.abs(got - v)[fine] <= (R.HALF_BF16 + 2.0 ** -23) * np.abs(v[fine]) + 2.0 ** -134).all()
    assert (R.f64(scales) == s).all()
    codes, near = nearest_e4m3((v.reshape(T, -1, group) / R.f64(scales)[..., None]).reshape(T, hidden))
    wrong = (R.f64(y8) != codes) & (near > 2.0 ** -40)
    assert not wrong.any(), wrong.sum()
    return v, s


@pytest.mark.parametrize("hidden,group", [(256, 256), (256, 32), (2304, 2304), (8192, 256), (65536, 65536),
                                          (65536, 256)])
def test_rms_norm_past_the_largest_number(hidden, group):
    """Few elements and huge weights: h w is a finite fp32 number, v is not."""
    x = torch.zeros(4, hidden, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(hidden, dtype=torch.bfloat16, device="cuda")
    x[0, 5], x[1, 5], x[1, 7] = 0.125, 0.0625, -0.0703125
    x[2, hidden - 1], x[2, 3] = -0.125, 2.0 ** -20
    x[3, 5], x[3, 200] = 1.5, 1.0
    w[5], w[7], w[hidden - 1], w[200] = 2.0 ** 127, 1.25 * 2.0 ** 124, 1.9921875 * 2.0 ** 127, 3.0
    v, s = check_rows(x, w, group)
    assert (np.abs(v) > 2.0 ** 128).any() and np.isfinite(s).all()


@pytest.mark.parametrize("hidden,group", [(65536, 65536), (65536, 32), (16384, 128)])
def test_rms_norm_of_products_below_the_normal_numbers(hidden, group):
    """h w below 2^-126 keeps all of its bits, and so do v and its codes."""
    rng = np.random.default_rng(hidden + group)
    x = R.bf16(rng.standard_normal((3, hidden)) * 2.0 ** -70).cuda()
    w = R.bf16((1 + rng.random(hidden)) * 2.0 ** -65).cuda()
    # 1 / rms just below 2^10
    x[:, 77] = 1.01 * 2.0 ** -10 * hidden ** 0.5
    w[77] = 2.0 ** -120
    v, _ = check_rows(x, w, group)
    assert (np.abs(v) < 2.0 ** -118).mean() > 0.99 and (np.abs(v) > 2.0 ** -126).mean() > 0.3


@pytest.mark.parametrize("hidden", [504, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384, 16392, 32768,
                                    32776])
def test_rms_norm_where_the_threads_and_their_chunks_change(hidden):
    x, w, r = norm_case(np.random.default_rng(hidden), 3, hidden, True)
    sums, y = torch.empty_like(x), torch.empty_like(x)
    y8, scales = torch.empty(3, hidden, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(3, 1, device="cuda")
    srg.lora_rms_norm(x, w, 1e-5, residual=r, residual_out=sums, y=y, y8=y8, scales=scales)
    check_norm(x, w, r, 1e-5, hidden, sums, y, y8, scales)


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("scale", [3e38, -3.4e38, 2e38])
def test_attention_scales_near_the_largest_number(scale):
    """Scores of zero stay zero whatever the scale: every query takes the mean of the
    tokens that it sees."""
    c = Call(19, [90, 200], [3, 40], 4, 2, 64, 16, 50)
    c.qh = torch.zeros_like(c.qh)
    c.q.zero_()
    c.scale = scale
    c.run()
    c.check()
