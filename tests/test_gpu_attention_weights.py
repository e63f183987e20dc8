"""Attention over the 4-bit cache against a bound that follows the weights: they
are rounded to bf16 and divided by the sum of what was rounded, so that an error
of a weight moves the result by no more than that share of how far its value lies
from the result."""

import numpy as np
import pytest

import segmented_rank_gemm_amd as srg  # noqa: F401  (the library, loudly)
from tests import attention_reference as R
from tests.test_gpu_attention import Call, dev, sample

pytestmark = pytest.mark.gpu


def bounded(c, only=None):
    """(out, slack) of a Call in 64 bits.  slack, with p the weights of a row:
    * the result's rounding to bf16: 2^-8 of it;
    * every weight is off by a share of at most `share`: its rounding to bf16
      (2^-8), its score's error and its power's (2^-22).  A score's: sums of d
      products in fp32 (d * 2^-24 of scale * sum |q||k|), the scale, the exponent's
      argument and the differences of running maxima in fp32 (2^-22 of the largest
      score).  In the quotient a share moves the result by that share of p |v - result|;
    * sums over n weights in fp32, on both sides of the quotient: n * 2^-24 of the
      sum of p |v|, and of the result;
    * powers below 2^-126 are none in fp32 or as a bf16 operand, whether a weight's or
      those that join sums of different maxima, of weights up to 2^8: what is lost of
      each weight is at most 2^-118 of the largest, which the sum is no less than."""
    T, hq, kv, d, page, window, _ = c.shape
    q, scale = R.f64(c.qh), abs(c.scale)
    out, slack = np.zeros((T, hq, d)), np.zeros((T, hq, d))
    for s in range(len(c.lens)):
        queries = c.start[s + 1] - c.start[s]
        place = c.lens[s] - queries + np.arange(queries)
        tokens = np.arange(max(int(c.lens[s]), 0))
        ids = c.table[s, tokens // page]
        there = (ids >= 0) & (ids < c.pages)
        tokens, ids = tokens[there], ids[there]
        for h in range(hq):
            rows = np.arange(queries) if only is None else np.nonzero(only[c.start[s]:c.start[s + 1], h])[0]
            if not len(tokens) or not len(rows):
                continue
            k = c.values[ids, 0, h // (hq // kv), tokens % page]
            v = c.values[ids, 1, h // (hq // kv), tokens % page]
            for i in rows:
                r = c.start[s] + i
                seen = tokens <= place[i]
                if window:
                    seen &= tokens > place[i] - window
                n = int(seen.sum())
                if not n:
                    continue
                score = c.scale * (k[seen] @ q[r, h])
                size = scale * (np.abs(k[seen]) @ np.abs(q[r, h])).max()
                p = np.exp(score - score.max())
                p /= p.sum()
                o = p @ v[seen]
                share = R.HALF_BF16 + size * d * 2.0 ** -24 + (np.abs(score).max() + 1) * 2.0 ** -22
                out[r, h] = o
                slack[r, h] = (R.HALF_BF16 * np.abs(o) + 1.01 * share * (p @ np.abs(v[seen] - o)) +
                               1.01 * n * 2.0 ** -24 * (p @ np.abs(v[seen]) + np.abs(o)) +
                               n * 2.0 ** -118 * np.abs(v[seen]).max() + 1e-38)
    return out, slack


def check(c, only=None):
    c.run()
    out, slack = bounded(c, only)
    got = R.f64(c.out)
    assert np.isfinite(got).all()
    over = np.abs(got - out) - slack
    if only is not None:
        over = over[only]
    assert (over <= 0).all(), (over.max(), (over > 0).sum(), over.size)
    assert c.runs_alike()


# lens, queries, q_heads, kv_heads, head_dim, page, window
SHAPES = [
    ([700, 64, 5], [1, 1, 1], 16, 2, 128, 16, 0),
    ([3000, 900], [1, 1], 8, 2, 64, 64, 0),
    ([700, 300], [20, 7], 6, 2, 64, 16, 0),
    ([500, 900], [150, 40], 8, 2, 128, 32, 200),
    ([300, 431, 280, 290], [300, 250, 140, 290], 64, 8, 128, 64, 0),  # operands shared by a workgroup
    ([300, 431, 280, 290], [300, 250, 140, 290], 64, 8, 64, 16, 90),
]


@pytest.mark.parametrize("scale", [0.06, 1.0, -3.0])
@pytest.mark.parametrize("case", SHAPES, ids=[str(i) for i in range(len(SHAPES))])
def test_weights_divided_by_their_own_sum(case, scale):
    c = Call(60 + case[0][0], *case)
    c.scale = scale
    check(c, None if sum(case[1]) < 100 else sample(*c.shape[:2], 600))


@pytest.mark.parametrize("scale", [0.06, 1.0, 4.0])
@pytest.mark.parametrize("case", SHAPES, ids=[str(i) for i in range(len(SHAPES))])
def test_equal_values_come_back(case, scale):
    """All tokens' values alike: every mean of them is that value, exactly (what the
    sums lose, n * 2^-23 of it, is far less than half a step of bf16)."""
    c = Call(80 + case[0][0], *case)
    T, hq, kv, d, page, _, _ = c.shape
    c.scale = scale
    row = np.random.default_rng(1).integers(0, 256, d // 2).astype(np.uint8)
    data = c.data.copy()
    data[:, 1, :, :page * d // 2] = np.tile(row, page)
    scales = data[:, 1, :, page * d // 2:]
    scales[scales != 255] = 127
    c.cache = dev(data)
    c.run()
    codes = np.stack([row & 15, row >> 4], -1).reshape(d)
    want = np.concatenate([R.LEVELS, -R.LEVELS])[codes]
    got = R.f64(c.out)
    assert (got == want).all(), np.abs(got - want).max()
