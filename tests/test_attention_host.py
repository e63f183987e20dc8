"""Host-side checks of the operators around the projections (no GPU needed): the
header's entry points are exported, invalid arguments are refused before anything
is enqueued, calls over nothing return, and the tests' own 64-bit forms hold."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import segmented_rank_gemm_amd as srg
from tests import attention_reference as R

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
FAKE = 0x10000  # a 256-byte aligned non-null address that is never dereferenced
OK, INVALID, UNSUPPORTED = 0, 1, 2


def test_header_entry_points_are_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(INCLUDE, "lora_attention.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(lora_[a-z_]+)\s*\(", text)))
    assert names == ["lora_kv_append", "lora_kv_attention", "lora_kv_attention_workspace_bytes",
                     "lora_kv_read", "lora_rms_norm"]
    L = ctypes.CDLL(srg.LIB_PATH)
    for n in names:
        assert hasattr(L, n) and hasattr(srg, n) and n in srg.__all__, n


NORM = dict(x=FAKE, ldx=64, residual=FAKE, ldr=64, weight=FAKE, eps=1e-5, num_tokens=3, hidden=64,
            residual_out=FAKE, ldo=64, y=FAKE, ldy=64, y8=FAKE, ldy8=64, scales=FAKE, group=64,
            stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(x=FAKE + 8), INVALID), (dict(ldx=56), INVALID),
    (dict(ldx=68), INVALID), (dict(weight=None), INVALID), (dict(weight=FAKE + 2), INVALID),
    (dict(residual=None), INVALID), (dict(residual=FAKE + 2), INVALID), (dict(ldr=60), INVALID),
    (dict(ldo=8), INVALID), (dict(ldy=8), INVALID), (dict(y=FAKE + 8), INVALID),
    (dict(y8=FAKE + 4), INVALID), (dict(y8=None), INVALID), (dict(scales=None), INVALID),
    (dict(scales=FAKE + 2), INVALID), (dict(ldy8=63), INVALID), (dict(ldy8=60), INVALID),
    (dict(residual_out=None, y=None, y8=None, scales=None), INVALID),
    (dict(eps=-1e-9), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(num_tokens=-1), INVALID), (dict(num_tokens=(1 << 24) + 1), INVALID),
    (dict(num_tokens=(1 << 22) + 1), INVALID),
    (dict(hidden=0), INVALID), (dict(hidden=60), INVALID), (dict(hidden=65544, ldx=65544), INVALID),
    (dict(group=0), INVALID), (dict(group=48), INVALID), (dict(group=16), UNSUPPORTED),
    (dict(group=8), UNSUPPORTED),
])
def test_rms_norm_refuses(change, status):
    assert srg.lib().lora_rms_norm(*{**NORM, **change}.values()) == status


APPEND = dict(qkv=FAKE, ldqkv=1024, positions=FAKE, slots=FAKE, rope=FAKE, rope_rows=10, rot_dim=64,
              interleaved=0, num_tokens=2, q_heads=4, kv_heads=2, head_dim=128, q_out=FAKE, ldq=512,
              cache=FAKE, num_pages=3, page_size=16, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(qkv=None), INVALID), (dict(qkv=FAKE + 2), INVALID), (dict(ldqkv=1016), INVALID),
    (dict(ldqkv=1028), INVALID), (dict(positions=None), INVALID), (dict(slots=None), INVALID),
    (dict(rope=None), INVALID), (dict(rope=FAKE + 4), INVALID), (dict(rope_rows=0), INVALID),
    (dict(rot_dim=-16), INVALID), (dict(rot_dim=144), INVALID), (dict(rot_dim=24), INVALID),
    (dict(interleaved=2), INVALID), (dict(interleaved=-1), INVALID), (dict(num_tokens=-1), INVALID),
    (dict(q_heads=0), INVALID), (dict(q_heads=1025), INVALID), (dict(kv_heads=0), INVALID),
    (dict(kv_heads=1025), INVALID), (dict(q_out=None), INVALID), (dict(ldq=504), INVALID),
    (dict(cache=None), INVALID), (dict(cache=FAKE + 8), INVALID), (dict(num_pages=0), INVALID),
    (dict(page_size=0), INVALID), (dict(page_size=24), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=512), UNSUPPORTED), (dict(head_dim=96, rot_dim=64), UNSUPPORTED),
    (dict(head_dim=0), INVALID),
])
def test_kv_append_refuses(change, status):
    assert srg.lib().lora_kv_append(*{**APPEND, **change}.values()) == status


READ = dict(slots=FAKE, num_tokens=2, kv_heads=2, head_dim=64, cache=FAKE, num_pages=3, page_size=32,
            k_out=FAKE, ldk=128, v_out=FAKE, ldv=128, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(slots=None), INVALID), (dict(num_tokens=-1), INVALID), (dict(k_out=None, v_out=None), INVALID),
    (dict(ldk=120), INVALID), (dict(ldv=130), INVALID), (dict(k_out=FAKE + 8), INVALID),
    (dict(cache=None), INVALID), (dict(num_pages=-1), INVALID), (dict(head_dim=32), UNSUPPORTED),
    (dict(page_size=48), UNSUPPORTED),
])
def test_kv_read_refuses(change, status):
    assert srg.lib().lora_kv_read(*{**READ, **change}.values()) == status


ATTENTION = dict(q=FAKE, ldq=512, query_start=FAKE, seq_lens=FAKE, page_table=FAKE, ld_table=4,
                 cache=FAKE, num_pages=3, page_size=16, num_tokens=2, num_seqs=2, max_query_len=1,
                 max_seq_len=64, q_heads=4, kv_heads=2, head_dim=128, scale=1.0, window=0, out=FAKE,
                 ldo=512, workspace=FAKE, workspace_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(ldq=504), INVALID), (dict(ldq=513), INVALID),
    (dict(query_start=None), INVALID), (dict(seq_lens=None), INVALID), (dict(page_table=None), INVALID),
    (dict(ld_table=3), INVALID), (dict(max_seq_len=65), INVALID), (dict(max_seq_len=0), INVALID),
    (dict(max_seq_len=(1 << 30) + 1, ld_table=1 << 40), INVALID), (dict(max_query_len=0), INVALID),
    (dict(num_seqs=-1), INVALID), (dict(num_seqs=(1 << 16) + 1), INVALID),
    (dict(num_seqs=1 << 16), INVALID), (dict(max_query_len=(1 << 21) + 1), UNSUPPORTED),
    (dict(num_tokens=-1), INVALID), (dict(q_heads=5), INVALID), (dict(q_heads=1), INVALID),
    (dict(q_heads=1026), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(window=-1), INVALID), (dict(out=None), INVALID),
    (dict(ldo=8), INVALID), (dict(cache=FAKE + 4), INVALID), (dict(head_dim=256, ldq=1024, ldo=1024), UNSUPPORTED),
    (dict(page_size=40), UNSUPPORTED),
])
def test_kv_attention_refuses(change, status):
    assert srg.lib().lora_kv_attention(*{**ATTENTION, **change}.values()) == status


def test_kv_attention_refuses_a_missing_or_short_workspace():
    sizes = dict(num_seqs=2, max_query_len=1, max_seq_len=1 << 20, q_heads=4, kv_heads=2, head_dim=128)
    need = srg.lora_kv_attention_workspace_bytes(*sizes.values())
    if need == 0:
        pytest.skip("these sizes need no workspace")
    call = {**ATTENTION, **sizes, "ld_table": 1 << 16}
    f = srg.lib().lora_kv_attention
    assert f(*{**call, "workspace": None}.values()) == INVALID
    assert f(*{**call, "workspace_bytes": need - 1}.values()) == INVALID
    assert f(*{**call, "workspace": FAKE + 128}.values()) == INVALID


@pytest.mark.parametrize("sizes", [(-1, 1, 64, 4, 2, 128), (1, 0, 64, 4, 2, 128), (1, 1, 0, 4, 2, 128),
                                   (1, 1, 64, 5, 2, 128), (1, 1, 64, 4, 2, 80), (0, 1, 64, 4, 2, 128)])
def test_workspace_query_of_sizes_that_are_refused(sizes):
    assert srg.lora_kv_attention_workspace_bytes(*sizes) == 0


def test_calls_over_nothing_return():
    L = srg.lib()
    none = dict.fromkeys(["x", "residual", "weight", "residual_out", "y", "y8", "scales"])
    assert L.lora_rms_norm(*{**NORM, **none, "num_tokens": 0}.values()) == OK
    none = dict.fromkeys(["qkv", "positions", "slots", "q_out"])
    assert L.lora_kv_append(*{**APPEND, **none, "num_tokens": 0}.values()) == OK
    none = dict.fromkeys(["slots", "k_out", "v_out"])
    assert L.lora_kv_read(*{**READ, **none, "num_tokens": 0}.values()) == OK
    assert L.lora_kv_attention(*{**ATTENTION, "q": None, "out": None, "num_tokens": 0}.values()) == OK
    none = dict.fromkeys(["query_start", "seq_lens", "page_table"])
    assert L.lora_kv_attention(*{**ATTENTION, **none, "num_seqs": 0}.values()) == OK


def test_binding_takes_device_tensors_only():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        srg.lora_rms_norm(x, x[0], 1e-5, y=x)
    with pytest.raises(ValueError):
        srg.kv_cache_shape(4, 2, 96, 16)
    with pytest.raises(ValueError):
        srg.lora_kv_read(torch.zeros(1), torch.zeros(1), None, None)
    assert srg.kv_cache_shape(4, 2, 128, 16) == (4, 2, 2, 16 * 68)


@pytest.mark.parametrize("rot_dim", [16, 64, 128])
def test_rope_table(rot_dim):
    t = srg.rope_table(300, rot_dim, device="cpu")
    assert t.shape == (300, rot_dim) and t.dtype == torch.float32
    # one rounding to fp32 of a number of magnitude up to 1, and pow's own error on the angle
    assert np.abs(t.double().numpy() - R.rope_reference(300, rot_dim)).max() <= 2.0 ** -24


def test_the_reference_format():
    assert [R.block_exponent(x) for x in (0.0, 7.0, 7.1, 6.0, 3.5, 3.6, 1e39)] == [-125, 0, 1, 0, -1, 0, 125]
    v = np.zeros(32)
    v[:13] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -5, 0.26, 7, -6.99]
    assert list(R.held(v)[:13]) == [6, 0, 1, 1, 2, 2, 4, 4, 0, -4, 0.5, 6, -6]
    assert np.isnan(R.held(np.where(np.arange(32) == 3, np.inf, 1.0))).all()
    data, values = R.random_cache(np.random.default_rng(0), 2, 1, 64, 16)
    assert data.shape == (2, 2, 1, 16 * 34) and values.shape == (2, 2, 1, 16, 64)
    # element 37 of token 3: the odd half of byte 18 of its row; the second block's scale
    code, byte = int(data[1, 1, 0, 3 * 32 + 18] >> 4), int(data[1, 1, 0, 16 * 32 + 16 + 3])
    assert values[1, 1, 0, 3, 37] == (-1) ** (code >> 3) * R.LEVELS[code & 7] * 2.0 ** (byte - 127)
