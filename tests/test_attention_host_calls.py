"""Host-side checks of the operators around the projections beside their refusals
(no GPU needed): calls over nothing with no tensors at all, sizes past the library's
integers, and the norm's instances in the library."""

import re

import pytest

import segmented_rank_gemm_amd as srg
from tests.test_attention_host import APPEND, ATTENTION, INVALID, NORM, OK, READ, UNSUPPORTED

TENSORS = ("x", "residual", "weight", "residual_out", "y", "y8", "scales", "qkv", "positions", "slots", "rope",
           "q_out", "cache", "k_out", "v_out", "q", "query_start", "seq_lens", "page_table", "out", "workspace")


def over_nothing(call, **more):
    """The call with none of its tensors."""
    return {**{k: None if k in TENSORS else v for k, v in call.items()}, **more}.values()


def test_calls_over_nothing_need_no_tensors():
    L = srg.lib()
    assert L.lora_rms_norm(*over_nothing(NORM, num_tokens=0)) == OK
    assert L.lora_kv_append(*over_nothing(APPEND, num_tokens=0)) == OK
    assert L.lora_kv_append(*over_nothing(APPEND, num_tokens=0, num_pages=0)) == OK
    assert L.lora_kv_read(*over_nothing(READ, num_tokens=0)) == OK
    # long enough that the call would need a workspace
    long = dict(max_seq_len=1 << 20, ld_table=1 << 16, workspace_bytes=0)
    assert srg.lora_kv_attention_workspace_bytes(2, 1, 1 << 20, 4, 2, 128) > 0
    for none in (dict(num_tokens=0), dict(num_seqs=0), dict(num_tokens=0, num_seqs=0)):
        assert L.lora_kv_attention(*over_nothing(ATTENTION, **none)) == OK, none
        assert L.lora_kv_attention(*over_nothing(ATTENTION, **long, **none)) == OK, none


@pytest.mark.parametrize("change,status", [
    (dict(page_size=24), UNSUPPORTED), (dict(page_size=0), INVALID), (dict(head_dim=96), UNSUPPORTED),
    (dict(kv_heads=0), INVALID), (dict(num_pages=-1), INVALID)])
def test_calls_over_nothing_still_refuse_sizes(change, status):
    L = srg.lib()
    assert L.lora_kv_append(*over_nothing(APPEND, num_tokens=0, **change)) == status
    assert L.lora_kv_read(*over_nothing(READ, num_tokens=0, **change)) == status
    assert L.lora_kv_attention(*over_nothing(ATTENTION, num_seqs=0, **change)) == (
        INVALID if change == dict(kv_heads=0) else status)


def test_calls_over_something_need_them():
    L = srg.lib()
    assert L.lora_kv_append(*{**APPEND, "num_pages": 0}.values()) == INVALID
    assert L.lora_kv_read(*{**READ, "cache": None}.values()) == INVALID
    assert L.lora_kv_attention(*{**ATTENTION, "cache": None}.values()) == INVALID


@pytest.mark.parametrize("sizes", [((1 << 32) + 1, 1, 64, 4, 2, 128), (1, (1 << 32) + 1, 64, 4, 2, 128),
                                   (1, 1, (1 << 32) + 64, 4, 2, 128), (1, 1, 1 << 31, 4, 2, 128),
                                   (1, 1, -(1 << 32) + 64, 4, 2, 128), (1, 1, 64, (1 << 32) + 4, 2, 128)])
def test_sizes_past_the_librarys_integers_are_refused(sizes):
    """They would arrive as others: (1 << 32) + 64 tokens as 64."""
    with pytest.raises(ValueError, match="32 bits"):
        srg.lora_kv_attention_workspace_bytes(*sizes)
    with pytest.raises(ValueError, match="32 bits"):
        srg.kv_attention_workspace(*sizes)


def norm_instance(hidden):
    """(threads a row, chunks of 8 elements a thread) for rows of this length."""
    threads = next(t for most, t in ((1024, 64), (4096, 256), (32768, 512), (65536, 1024)) if hidden <= most)
    each = -(-(hidden // 8) // threads)
    return threads, 1 << (each - 1).bit_length()


def test_every_norm_kernel_in_the_library_serves_some_length():
    names = set(re.findall(rb"rms_norm_kernelILi(\d+)ELi(\d+)E", open(srg.LIB_PATH, "rb").read()))
    held = {(int(t), int(c)) for t, c in names}
    assert held == {norm_instance(h) for h in range(8, 65536 + 8, 8)}


def test_rms_norm_refuses_the_one_grid_that_cannot_be_launched():
    """2^22 rows of 1024 threads: 2^32, one more than a grid dimension holds."""
    wide = dict(hidden=32776, ldx=32776, ldr=32776, ldo=32776, ldy=32776, ldy8=32776, group=32776)
    assert srg.lib().lora_rms_norm(*{**NORM, **wide, "num_tokens": 1 << 22}.values()) == UNSUPPORTED
