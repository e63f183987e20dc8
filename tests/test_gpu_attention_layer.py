"""The example layer end to end: each stage of its last step against the 64-bit
form of that stage on the stage's own inputs."""

import numpy as np
import pytest
import torch

import segmented_rank_gemm_amd as srg
from examples import attention_layer as E
from tests import attention_reference as R

pytestmark = pytest.mark.gpu


def test_example_layer():
    cfg = E.Config(hidden=1024, q_heads=8, kv_heads=2, head_dim=128, rank=8, page=16, pages=64, positions=256)
    step, _, lens = E.run(cfg, prompts=(70, 1, 33), new_tokens=3, seed=4)
    layer, T = step.layer, step.tokens
    # norm
    h, v, scales = R.rms_norm(step.x, step.residual, layer.norm, cfg.eps, cfg.hidden)
    assert np.array_equal(R.f64(step.h), h)
    assert (np.abs(R.f64(step.y) - v) <= (R.HALF_BF16 + 2.0 ** -23) * np.abs(v)).all()
    assert (R.f64(step.scales) == scales).all()
    # products: bf16 of the base product, then of it plus the low-rank part
    base = (R.f64(step.y8) * R.f64(step.scales)) @ (R.f64(layer.base8) * R.f64(layer.base_scales).T).T
    low = np.zeros_like(base)
    at = 0
    for a, b, n in zip(layer.lora_a, layer.lora_b, cfg.slices):
        for t in range(T):
            l = int(step.adapter[t])
            if l >= 0:
                low[t, at:at + n] = (R.f64(step.y)[t] @ R.f64(a)[l].T) @ R.f64(b)[l].T
        at += n
    # two roundings to bf16, products and sums in fp32 of 1024 terms of magnitude
    # below 1 (8-bit products may be added up in fewer bits: 2^-13 of the terms' sum)
    terms = np.abs(R.f64(step.y8) * R.f64(step.scales)) @ np.abs(R.f64(layer.base8) * R.f64(layer.base_scales).T).T
    slack = 2.1 * R.HALF_BF16 * (np.abs(base) + np.abs(low)) + 2.0 ** -12 * (terms + 1)
    assert (np.abs(R.f64(step.qkv) - base - low) <= slack).all()
    # rotation and append, from the rounded q, k, v
    x = R.f64(step.qkv).reshape(T, -1, cfg.head_dim)
    hq, kv = cfg.q_heads, cfg.kv_heads
    turned = R.rotate(x[:, :hq + kv], R.f64(layer.rope), step.positions.tolist(), False)
    assert (np.abs(R.f64(step.q) - turned[:, :hq]) <= (R.HALF_BF16 + 2.0 ** -23) * np.abs(turned[:, :hq])).all()
    k, val = (torch.empty(T, kv, cfg.head_dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    srg.lora_kv_read(step.slots, layer.cache, k, val)
    assert np.array_equal(R.f64(k), R.held(turned[:, hq:].astype(np.float32).astype(np.float64)))
    assert np.array_equal(R.f64(val), R.held(x[:, hq + kv:]))
    # attention over what the cache holds
    every = torch.arange(cfg.pages * cfg.page, device="cuda")
    k, val = (torch.empty(len(every), kv, cfg.head_dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    srg.lora_kv_read(every, layer.cache, k, val)
    values = np.stack([R.f64(k), R.f64(val)], 1).reshape(cfg.pages, cfg.page, 2, kv, cfg.head_dim).transpose(0, 2, 3, 1, 4)
    assert step.seq_lens.tolist() == lens
    out, slack = R.attention(R.f64(step.q), values, step.query_start.tolist(), lens,
                             step.page_table.tolist(), cfg.page, cfg.head_dim ** -0.5)
    assert (np.abs(R.f64(step.out) - out) <= slack).all()
