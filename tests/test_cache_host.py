"""Host-side checks of drafted tokens and caches of bounded length (no GPU needed): the
header's entry points are exported, invalid arguments are refused before anything is
enqueued, calls over nothing return, and the tests' own 64-bit forms hold."""

import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import segmented_rank_gemm_amd as srg
from segmented_rank_gemm_amd import cache
from tests import cache_reference as C

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
FAKE = 0x10000  # a 256-byte aligned non-null address that is never dereferenced
OK, INVALID, UNSUPPORTED = 0, 1, 2


def test_header_entry_points_are_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(INCLUDE, "lora_cache.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(lora_[a-z_]+)\s*\(", text)))
    assert names == ["lora_draft_masks", "lora_kv_attention_mass", "lora_kv_compact", "lora_kv_select",
                     "lora_kv_select_workspace_bytes", "lora_kv_tree_attention", "lora_kv_tree_attention_workspace_bytes"]
    L = ctypes.CDLL(srg.LIB_PATH)
    for n in names:
        assert hasattr(L, n) and hasattr(srg, n) and n in srg.__all__, n
    assert int(re.search(r"LORA_MAX_MASK_WORDS (\d+)", open(os.path.join(INCLUDE, "lora_cache.h")).read())[1]) \
        == srg.LORA_MAX_MASK_WORDS


def test_masks_have_words():
    with pytest.raises(ValueError, match="no words"):
        cache._words(torch.zeros(5, 0, dtype=torch.int64), 5)


MASKS = dict(parents=FAKE, query_start=FAKE, num_tokens=5, num_seqs=2, masks=FAKE, mask_words=1, first=FAKE,
             positions=FAKE, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(parents=None), INVALID), (dict(query_start=None), INVALID), (dict(masks=None, positions=None), INVALID),
    (dict(masks=FAKE + 4), INVALID), (dict(mask_words=0), INVALID), (dict(mask_words=-1), INVALID),
    (dict(mask_words=9), UNSUPPORTED), (dict(num_tokens=-1), INVALID), (dict(num_tokens=(1 << 22) + 1), INVALID),
    (dict(num_seqs=-1), INVALID), (dict(num_seqs=65536), INVALID)])
def test_draft_masks_refuses(change, status):
    assert srg.lib().lora_draft_masks(*{**MASKS, **change}.values()) == status


STEP = dict(query_start=FAKE, seq_lens=FAKE, page_table=FAKE, ld_table=4, cache=FAKE, num_pages=3, page_size=16,
            num_tokens=5, num_seqs=2, max_query_len=4, max_seq_len=64, q_heads=4, kv_heads=2, head_dim=64, scale=0.125,
            window=0, masks=FAKE, mask_words=1)
TREE = dict(q=FAKE, ldq=256, **STEP, out=FAKE, ldo=256, lse=FAKE, ldl=4, workspace=None, workspace_bytes=0, stream=None)
MASS = dict(q=FAKE, ldq=256, lse=FAKE, ldl=4, **STEP, mass=FAKE, stream=None)
STEP_REFUSED = [
    (dict(q=None), INVALID), (dict(q=FAKE + 2), INVALID), (dict(ldq=248), INVALID), (dict(ldq=260), INVALID),
    (dict(query_start=None), INVALID), (dict(seq_lens=None), INVALID), (dict(page_table=None), INVALID),
    (dict(ld_table=3), INVALID), (dict(cache=None), INVALID), (dict(cache=FAKE + 8), INVALID),
    (dict(num_pages=0), INVALID), (dict(num_pages=-1), INVALID), (dict(page_size=0), INVALID),
    (dict(page_size=24), UNSUPPORTED), (dict(page_size=512), UNSUPPORTED), (dict(num_tokens=-1), INVALID),
    (dict(num_tokens=(1 << 22) + 1), INVALID), (dict(num_seqs=-1), INVALID), (dict(num_seqs=65536), INVALID),
    (dict(max_query_len=0), INVALID), (dict(max_query_len=65), INVALID),
    (dict(max_query_len=577, mask_words=9), UNSUPPORTED), (dict(max_seq_len=0), INVALID),
    (dict(max_seq_len=(1 << 30) + 1), INVALID), (dict(q_heads=5), INVALID), (dict(q_heads=0), INVALID),
    (dict(kv_heads=0), INVALID), (dict(head_dim=0), INVALID), (dict(head_dim=96, ldq=384, ldo=384), UNSUPPORTED),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID), (dict(window=-1), INVALID),
    (dict(masks=FAKE + 4), INVALID), (dict(mask_words=0), INVALID), (dict(mask_words=9), UNSUPPORTED),
    (dict(lse=FAKE + 2), INVALID), (dict(ldl=3), INVALID),
    (dict(masks=None, max_query_len=1 << 22), UNSUPPORTED)]


@pytest.mark.parametrize("change,status", STEP_REFUSED + [
    (dict(out=None), INVALID), (dict(out=FAKE + 8), INVALID), (dict(ldo=248), INVALID), (dict(ldo=260), INVALID)])
def test_tree_attention_refuses(change, status):
    assert srg.lib().lora_kv_tree_attention(*{**TREE, **change}.values()) == status


def test_tree_attention_refuses_small_workspaces():
    sizes = dict(num_seqs=1, max_query_len=4, max_seq_len=65536, q_heads=4, kv_heads=2, head_dim=64)
    need = srg.lora_kv_tree_attention_workspace_bytes(**sizes)
    assert need > 0 and need % 4 == 0
    for change in (dict(workspace=None, workspace_bytes=need), dict(workspace=FAKE, workspace_bytes=need - 1),
                   dict(workspace=FAKE + 64, workspace_bytes=need)):
        args = {**TREE, **sizes, "ld_table": 4096, **change}
        assert srg.lib().lora_kv_tree_attention(*args.values()) == INVALID
    for change in (dict(head_dim=96), dict(q_heads=3), dict(num_seqs=-1), dict(max_query_len=0)):
        assert srg.lora_kv_tree_attention_workspace_bytes(**{**sizes, **change}) == 0


@pytest.mark.parametrize("max_query_len", [1, 3, 13, 32, 33, 64, 512])
@pytest.mark.parametrize("heads", [(8, 8), (64, 8), (6, 2), (40, 1)])
@pytest.mark.parametrize("seqs", [1, 3, 64])
def test_workspaces_serve_shorter_calls(max_query_len, heads, seqs):
    """What is enough for max_seq_len is enough for any shorter one (and a window, which makes
    calls shorter)."""
    last = 0
    for n in [1, 64, 65, 500, 512, 513, 1000, 4096, 5000, 8192, 32768, 100000, 131072, 1 << 20]:
        need = srg.lora_kv_tree_attention_workspace_bytes(seqs, max_query_len, n, *heads, 128)
        assert need >= last
        last = need


@pytest.mark.parametrize("change,status", STEP_REFUSED + [
    (dict(lse=None), INVALID), (dict(mass=None), INVALID), (dict(mass=FAKE + 4), INVALID)])
def test_attention_mass_refuses(change, status):
    change = {k: v for k, v in change.items() if k != "ldo"}
    assert srg.lib().lora_kv_attention_mass(*{**MASS, **change}.values()) == status


SELECT = dict(mass=FAKE, num_pages=3, page_size=16, seq_lens=FAKE, page_table=FAKE, ld_table=4, num_seqs=2, kv_heads=2,
              max_seq_len=64, sinks=2, recent=3, kept=FAKE, budget=10, new_lens=FAKE + 64, workspace=None,
              workspace_bytes=0, stream=None)
LONG = dict(ld_table=2048, max_seq_len=32768)  # in pieces



@pytest.mark.parametrize("change,status", [
    (dict(mass=None), INVALID), (dict(mass=FAKE + 8), INVALID), (dict(num_pages=0), INVALID),
    (dict(num_pages=-1), INVALID), (dict(page_size=0), INVALID), (dict(page_size=8, ld_table=8), UNSUPPORTED),
    (dict(page_size=48), UNSUPPORTED), (dict(seq_lens=None), INVALID), (dict(page_table=None), INVALID),
    (dict(ld_table=3), INVALID), (dict(num_seqs=-1), INVALID), (dict(num_seqs=65536), INVALID),
    (dict(kv_heads=0), INVALID), (dict(kv_heads=1025), INVALID), (dict(max_seq_len=0), INVALID),
    (dict(max_seq_len=(1 << 30) + 1), INVALID), (dict(sinks=-1), INVALID), (dict(recent=-1), INVALID),
    (dict(sinks=8), INVALID), (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), INVALID), (dict(kept=None), INVALID),
    (dict(budget=0), INVALID), (dict(budget=(1 << 30) + 1), INVALID), (dict(new_lens=None), INVALID),
    (dict(new_lens=FAKE), INVALID), (dict(LONG), INVALID), (dict(LONG, workspace=FAKE, workspace_bytes=100), INVALID),
    (dict(LONG, workspace=FAKE + 16, workspace_bytes=1 << 30), INVALID), (dict(LONG, workspace_bytes=1 << 30), INVALID)])
def test_select_refuses(change, status):
    assert srg.lib().lora_kv_select(*{**SELECT, **change}.values()) == status


@pytest.mark.parametrize("off", [0, 4, 4 * 6, -4, -4 * 6])
def test_select_refuses_lengths_that_share_places(off):
    """A key head's workgroup would read a length that another one has already replaced."""
    args = {**SELECT, "num_seqs": 7, "new_lens": FAKE + off}
    assert srg.lib().lora_kv_select(*args.values()) == INVALID


def test_select_workspace():
    size = srg.lora_kv_select_workspace_bytes
    assert size(2, 2, 64) == size(64, 8, 131072) == size(0, 8, 131072) == size(1, 8, 1 << 30) == 0
    for seqs, heads, most in ((0, 0, 131072), (-1, 8, 131072), (1, 8, 0), (1, 8, -5), (1, 1025, 131072), (65536, 1, 131072)):
        assert size(seqs, heads, most) == 0
    # two histograms of 2048 counts of 16 bits a piece of 8192 tokens, and 32 bytes
    for seqs, heads, pieces in ((1, 8, 4), (4, 8, 16), (32, 1, 128)):
        for most in ((pieces - 1) * 8192 + 1, pieces * 8192):
            assert size(seqs, heads, most) == seqs * heads * pieces * (2 * 4096 + 32)
    assert srg.kv_select_workspace(64, 8, 8192, device="cpu") is None
    assert srg.kv_select_workspace(1, 8, 131072, device="cpu").numel() == size(1, 8, 131072)


COMPACT = dict(kept=FAKE, num_lists=2, max_kept=5, counts=FAKE, first=FAKE, page_table=FAKE, ld_table=4, table_pages=4,
               dst_table=FAKE, ld_dst=2, dst_pages=2, cache=FAKE, num_pages=9, page_size=16, num_seqs=2, kv_heads=2,
               head_dim=64, mass=FAKE, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(kept=None), INVALID), (dict(num_lists=3), INVALID), (dict(num_lists=0), INVALID),
    (dict(max_kept=-1), INVALID), (dict(max_kept=(1 << 30) + 1), INVALID), (dict(counts=None), INVALID),
    (dict(page_table=None), INVALID), (dict(ld_table=3), INVALID), (dict(table_pages=0), INVALID),
    (dict(ld_dst=1), INVALID), (dict(dst_pages=0), INVALID), (dict(cache=None), INVALID),
    (dict(cache=FAKE + 8), INVALID), (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID),
    (dict(page_size=24), UNSUPPORTED), (dict(num_seqs=-1), INVALID), (dict(num_seqs=65536), INVALID),
    (dict(kv_heads=0), INVALID), (dict(head_dim=32), UNSUPPORTED), (dict(mass=FAKE + 4), INVALID)])
def test_compact_refuses(change, status):
    assert srg.lib().lora_kv_compact(*{**COMPACT, **change}.values()) == status


@pytest.mark.parametrize("dst_pages", [4, 2])
def test_compact_refuses_its_own_table_as_the_other(dst_pages):
    """(in place is without another table)"""
    args = {**COMPACT, "page_table": FAKE, "dst_table": FAKE, "ld_dst": 4, "dst_pages": dst_pages}
    assert srg.lib().lora_kv_compact(*args.values()) == INVALID


def test_calls_over_nothing():
    L = srg.lib()
    nothing = lambda d, *names: [0 if k in names else (None if v in (FAKE, FAKE + 64) else v) for k, v in d.items()]  # noqa: E731
    for name in ("num_tokens", "num_seqs"):
        assert L.lora_draft_masks(*nothing(MASKS, name)) == OK
        assert L.lora_kv_tree_attention(*nothing(TREE, name)) == OK
        assert L.lora_kv_attention_mass(*nothing(MASS, name)) == OK
    assert L.lora_kv_select(*nothing(SELECT, "num_seqs")) == OK
    assert L.lora_kv_compact(*nothing(COMPACT, "num_seqs")) == OK
    assert L.lora_kv_compact(*nothing(COMPACT, "max_kept")) == OK


# ------------------------------------------------------------------ the tests' own forms
def test_ancestors_and_words():
    assert C.ancestors([-1, 0, 0, 2, 5, 3]) == [{0}, {0, 1}, {0, 2}, {0, 2, 3}, {4}, {0, 2, 3, 5}]
    words = C.words_of([{0, 63, 64}, set()], 2)
    assert words.tolist() == [[1 - 2 ** 63, 1], [0, 0]]


def test_visible():
    assert C.visible(5, 2, 0) == [0, 1, 2, 3] and C.visible(5, 2, 1) == [0, 1, 2, 3, 4]
    assert C.visible(5, 2, 1, window=2) == [3, 4] and C.visible(1, 3, 0) == [] and C.visible(1, 3, 2) == [0]
    assert C.visible(5, 3, 0, {0, 2}) == [0, 1, 2, 4] and C.visible(5, 3, 0, set()) == [0, 1]
    assert C.visible(5, 3, 0, {0, 2, 7}, window=3) == [1, 2, 4] and C.visible(5, 3, 0, {0, 1, 2}, window=2) == [3, 4]
    assert C.visible(2, 4, 0, {0, 1, 3}) == [1]
    # a chain's masks are what a query sees without masks, windows and short sequences among it
    for length in range(6):
        for queries in range(1, 5):
            for window in (0, 1, 3):
                for i in range(queries):
                    assert C.visible(length, queries, i, set(range(i + 1)), window) == \
                        C.visible(length, queries, i, None, window), (length, queries, i, window)


def test_select_and_compact_forms():
    assert C.select([1.0, 5.0, 5.0, math.nan, 0.0, 9.0], 6, 1, 1, 4) == [0, 1, 2, 5]
    assert C.select([1.0, 5.0], 2, 0, 0, 4) == [0, 1]
    assert C.select([math.nan, -math.inf, 0.0], 3, 0, 0, 2) == [0, 2]
    places = np.arange(2 * 2 * 1 * 2 * 3, dtype=np.uint8).reshape(2, 2, 1, 2, 3)
    mass = np.arange(4.0).reshape(2, 1, 2)
    table = np.array([[1, 0]])
    got, weights = C.compact(places, mass, np.array([[[1, 2, 3]]]), [3], None, table, None)
    assert np.array_equal(got[1, :, :, 0], places[1, :, :, 1]) and np.array_equal(got[1, :, :, 1], places[0, :, :, 0])
    assert np.array_equal(got[0, :, :, 0], places[0, :, :, 1]) and np.array_equal(got[0, :, :, 1], places[0, :, :, 1])
    assert weights.ravel().tolist() == [1.0, 1.0, 3.0, 0.0]
