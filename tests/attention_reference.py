"""The operators around the projections, written plainly in 64 bits on the CPU
for the tests: norms, the 4-bit cache format, rotation and attention."""

from __future__ import annotations

import math

import numpy as np
import torch

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
HALF_BF16 = 2.0 ** -8   # a rounding to bf16 is off by at most this share of the value
HALF_E4M3 = 2.0 ** -4


def f64(t) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def bf16(a: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.asarray(a, dtype=np.float64)).to(torch.bfloat16)


# ---------------------------------------------------------------- norm
def rms_norm(x, residual, weight, eps, group):
    """(h, v, scales): the rounded sum, the normalised row and its scales, in 64 bits."""
    h = f64(x)
    if residual is not None:
        h = f64((x.float().cpu() + residual.float().cpu()).bfloat16())
    with np.errstate(all="ignore"):
        r = 1.0 / np.sqrt((h * h).sum(-1, keepdims=True) / h.shape[1] + eps)
        v = h * r * f64(weight)
        groups = np.abs(v).reshape(len(v), -1, group).max(-1)
    s = np.maximum((groups / 448.0).astype(np.float32), np.float32(2.0 ** -126))
    return h, v, s


# ---------------------------------------------------------------- 4-bit blocks
def block_exponent(largest: float) -> int:
    """The smallest e in [-125, 125] with largest <= 7 * 2^e, by trying each."""
    for e in range(-125, 126):
        if largest <= 7.0 * 2.0 ** e:
            return e
    return 125


def held(v: np.ndarray) -> np.ndarray:
    """What the cache holds for rows of multiples of 32 elements: each element's
    nearest scaled level, ties to the even code, by comparing with all of them."""
    blocks = v.reshape(-1, 32)
    out = np.empty_like(blocks)
    for i, b in enumerate(blocks):
        if not np.isfinite(b).all():
            out[i] = np.nan
            continue
        p = 2.0 ** block_exponent(np.abs(b).max())
        far = np.abs(np.abs(b)[:, None] / p - LEVELS)
        near = far.min(1, keepdims=True)
        # of two levels equally near, the one with the even code
        code = np.where(far == near, np.where(np.arange(8) % 2 == 0, 2, 1), 0).argmax(1)
        out[i] = np.sign(b) * LEVELS[code] * p
    return out.reshape(v.shape)


def random_cache(rng, num_pages, kv_heads, d, page, low=120, high=129):
    """A cache of random codes and scales: (bytes, values [pages, 2, kv_heads, page, d])."""
    codes = rng.integers(0, 16, (num_pages, 2, kv_heads, page, d), dtype=np.uint8)
    scales = rng.integers(low, high, (num_pages, 2, kv_heads, page, d // 32), dtype=np.uint8)
    packed = codes[..., 0::2] | (codes[..., 1::2] << 4)
    data = np.concatenate([packed.reshape(num_pages, 2, kv_heads, -1),
                           scales.swapaxes(-1, -2).reshape(num_pages, 2, kv_heads, -1)], axis=-1)
    signed = np.concatenate([LEVELS, -LEVELS])[codes]
    values = signed * np.repeat(2.0 ** (scales.astype(np.float64) - 127), 32, axis=-1)
    return data, values


# ---------------------------------------------------------------- rotation
def rotate(x: np.ndarray, rope: np.ndarray, positions, interleaved: bool) -> np.ndarray:
    """x [tokens, heads, d] with its first rot_dim elements turned, element by element."""
    out = x.copy()
    half = rope.shape[1] // 2
    for t, p in enumerate(positions):
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            c, s = rope[p, i], rope[p, half + i]
            out[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            out[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
    return out


# ---------------------------------------------------------------- attention
def attention(q, values, query_start, seq_lens, page_table, page, scale, window=0,
              max_seq_len=None, max_query_len=1 << 30, only=None):
    """(out, slack), of the rows in `only` ([tokens, q_heads], all by default), for q [tokens, q_heads, d] and cache values [pages, 2, kv_heads,
    page, d].  slack bounds how far a kernel may be that keeps scores and sums in
    fp32 and rounds the weights and the result to bf16 (see attention_slack)."""
    T, hq, d = q.shape
    pages, kv = values.shape[0], values.shape[2]
    out = np.full((T, hq, d), np.nan)
    slack = np.zeros((T, hq, d))
    for s in range(len(seq_lens)):
        first, queries = query_start[s], query_start[s + 1] - query_start[s]
        length = max(0, seq_lens[s] if max_seq_len is None else min(seq_lens[s], max_seq_len))
        for i in range(min(queries, max_query_len)):
            if not 0 <= first + i < T or (only is not None and not only[first + i].any()):
                continue
            place = length - queries + i
            low = max(0, place - window + 1) if window else 0
            seen = [t for t in range(low, min(place + 1, length))
                    if 0 <= page_table[s][t // page] < pages]
            if not seen:
                out[first + i] = 0.0
                continue
            seen = np.array(seen)
            held_at = np.asarray(page_table[s])[seen // page]
            for h in range(hq):
                if only is not None and not only[first + i, h]:
                    continue
                k = values[held_at, 0, h // (hq // kv), seen % page]
                v = values[held_at, 1, h // (hq // kv), seen % page]
                score = scale * (k @ q[first + i, h])
                p = np.exp(score - score.max())
                p /= p.sum()
                out[first + i, h] = p @ v
                size = abs(scale) * np.abs(q[first + i, h]).max() * np.abs(k).sum(1).max()
                slack[first + i, h] = attention_slack(out[first + i, h], p @ np.abs(v), size, d,
                                                      len(seen), np.abs(score).max())
    return out, slack


def attention_slack(out, spread, size, d, n, top):
    """Bound on the error of one output row, element by element.

    * the result's rounding to bf16: 2^-8 of it;
    * each weight's rounding to bf16: 2^-8 of it, so 2^-8 of sum p|v| (`spread`);
    * a score's error turns into that share of its weight and of the total (twice
      in the quotient): the products of d terms summed in fp32 (d * 2^-24 of
      `size`, which bounds sum |q||k| * scale), q held in two 8-bit parts of a
      32-element block (2^-16 of the block's largest), the exponent's argument
      and the power itself in fp32 (2^-22 of the largest score, and 2^-22);
    * sums over n weights in fp32: n * 2^-24, on both sides of the quotient."""
    score = size * (d * 2.0 ** -24 + 2.0 ** -16) + (top + 1) * 2.0 ** -22
    return HALF_BF16 * np.abs(out) + (HALF_BF16 + 2 * score + 2 * n * 2.0 ** -24) * spread * 1.01 + 1e-38


def rope_reference(rows, rot_dim, base=10000.0):
    return np.array([[math.cos(p * base ** (-2 * i / rot_dim)) for i in range(rot_dim // 2)] +
                     [math.sin(p * base ** (-2 * i / rot_dim)) for i in range(rot_dim // 2)]
                     for p in range(rows)]).reshape(rows, rot_dim)
