"""Which kernels attention over the 4-bit cache launches, read from a captured
graph, and each of them where its rows are cut in the middle of a query, its tokens
into more parts than the join takes at once, or both."""

import ctypes

import numpy as np
import pytest
import torch

import segmented_rank_gemm_amd as srg
from tests import attention_reference as R
from tests.test_gpu_attention import Call, dev, nearest_e4m3, norm_case, sample
from tests.test_gpu_attention_weights import check

pytestmark = pytest.mark.gpu


class Dim3(ctypes.Structure):
    _fields_ = [("x", ctypes.c_uint32), ("y", ctypes.c_uint32), ("z", ctypes.c_uint32)]


class KernelNode(ctypes.Structure):
    _fields_ = [("block", Dim3), ("extra", ctypes.c_void_p), ("func", ctypes.c_void_p), ("grid", Dim3),
                ("args", ctypes.c_void_p), ("shared", ctypes.c_uint32)]


def launches(c):
    """(grid, threads) of the kernels that a call enqueues, in their order."""
    c.run()                                   # the library's code is loaded
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        c.run()
    hip = srg.lib()                           # its dependencies hold the HIP runtime in use
    handle, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert hip.hipGraphGetNodes(handle, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert hip.hipGraphGetNodes(handle, nodes, ctypes.byref(n)) == 0
    out = []
    for node in nodes:
        k = KernelNode()
        assert hip.hipGraphKernelNodeGetParams(ctypes.c_void_p(node), ctypes.byref(k)) == 0
        out.append(((k.grid.x, k.grid.y, k.grid.z), k.block.x))
    return out


def tiles(c, rows_a_tile):
    T, hq, kv, _, _, _, most = c.shape
    return -(-most * (hq // kv) // rows_a_tile)


# ------------------------------------------------------------------ operands shared by a workgroup
# lens, queries, q_heads, kv_heads, head_dim, page, window: groups that divide
# neither 128 rows nor 32, so that tiles and waves begin inside a query
SHARED = [
    ([500, 200, 640, 333, 200, 260, 210, 450], [180, 200, 1, 150, 199, 33, 77, 200], 48, 16, 64, 32, 0),
    ([500, 200, 640, 333, 200, 260, 210, 450], [180, 200, 1, 150, 199, 33, 77, 200], 48, 16, 128, 128, 37),
    ([300, 250, 120, 0, 400, 201, 210, 220], [200, 200, 130, 3, 160, 200, 180, 43], 40, 8, 128, 16, 0),
    ([300, 250, 120, 5, 400, 201, 210, 220], [200, 200, 130, 9, 160, 200, 180, 43], 40, 8, 64, 64, 90),
    ([300, 280, 350, 260, 90, 300, 240], [250, 101, 250, 240, 97, 170, 230], 44, 4, 128, 32, 0),
    ([300, 280, 350, 260, 90, 300, 240], [250, 101, 250, 240, 97, 170, 230], 44, 4, 64, 16, 133),
]


@pytest.mark.parametrize("case", SHARED, ids=[str(i) for i in range(len(SHARED))])
def test_shared_operands_of_rows_cut_inside_a_query(case):
    c = Call(100 + case[2], *case)
    assert launches(c) == [((case[3], tiles(c, 128), len(case[0])), 256)]
    check(c, sample(*c.shape[:2], 1200))


def test_shared_operands_of_rows_cut_inside_a_query_bad_pages():
    c = Call(120, *SHARED[0])
    for s in range(0, 8, 2):
        c.table[s, 2 + s // 4] = -3 if s % 4 else c.pages
    c.dev[2] = dev(c.table)
    assert len(launches(c)) == 1
    check(c, sample(*c.shape[:2], 1200))


# ------------------------------------------------------------------ parts
# several row tiles with several parts, the last tile partial; groups of 4, 6 and 12
SPLIT = [
    ([3000], [40], 4, 1, 64, 16, 0),
    ([3000], [41], 4, 1, 128, 64, 700),
    ([2000, 130, 900], [37, 1, 20], 12, 2, 128, 32, 0),
    ([2500, 700], [37, 37], 12, 1, 64, 64, 0),
    ([1500], [9], 12, 2, 64, 16, 0),
]


@pytest.mark.parametrize("case", SPLIT, ids=[str(i) for i in range(len(SPLIT))])
def test_parts_of_several_row_tiles(case):
    c = Call(140 + case[0][0], *case)
    first, join = launches(c)
    assert first[1] == 256 and first[0][1] >= 2 * tiles(c, 32) and join[1] == 256
    check(c, sample(*c.shape[:2], 400))


@pytest.mark.parametrize("case", [
    ([16500, 5000], [100, 70], 12, 2, 64, 64, 0),    # 6 heads a key head: 19 tiles, the last of 24 rows
    ([16500, 16400], [90, 100], 10, 2, 64, 16, 0),   # 5 heads a key head
], ids=["6", "5"])
def test_twice_the_parts_for_long_sequences(case):
    c = Call(160 + case[2], *case)
    (grid, threads), join = launches(c)
    units = tiles(c, 32) * case[3] * len(case[0])
    assert threads == 256 and grid[1] > tiles(c, 32) * -(-256 // units), "the doubled rule"
    check(c, sample(*c.shape[:2], 120))


@pytest.mark.parametrize("scale", [0.05, 2.0, -2.0])
@pytest.mark.parametrize("case", [
    ([20000], [1], 8, 1, 128, 64, 0),
    ([20000], [1], 2, 1, 64, 16, 0),
    ([30000, 9, 700], [1, 1, 1], 4, 1, 128, 16, 0),
    ([14000], [3], 8, 1, 64, 64, 0),                 # two tiles' rows, 24 of 32
    ([33000, 2500], [1, 1], 4, 1, 64, 32, 30000),
], ids=["128", "64", "ragged", "rows", "window"])
def test_more_parts_than_the_join_takes_at_once(case, scale):
    """A row's parts are taken by 8 (head_dim 128) or 16 (64) groups of threads: with
    more of them each takes several, its sums rescaled from one to the next."""
    c = Call(180 + case[2] + len(case[0]), *case)
    c.scale = scale
    (grid, _), (_, threads) = launches(c)
    assert threads == 256 and grid[1] > 256 // (case[4] // 4)
    check(c)


def test_parts_and_rising_scores():
    """Scores that grow along the sequence, and that fall: every part's maximum is
    another, and the last or the first outweighs the others."""
    for order in (1, -1):
        c = Call(200, [20000], [1], 4, 1, 128, 64)
        data, values = c.data.copy(), c.values.copy()
        # scale bytes of the keys by the token's place: 2^-9 .. 2^0
        for i in range(20000 // 64 + 1):
            p = c.table[0, i]
            byte = 118 + (i * 10) // 313 if order > 0 else 127 - (i * 10) // 313
            s = data[p, 0, 0, 64 * 64:]
            old = s.copy()
            s[old != 255] = byte
            shift = np.where(old.reshape(4, 64).T == 255, 1.0, 2.0 ** (byte - old.reshape(4, 64).T.astype(float)))
            values[p, 0, 0] *= np.repeat(shift, 32, axis=1)
        c.cache, c.values, c.scale = dev(data), values, 1.0
        check(c)


# ------------------------------------------------------------------ what must not be written, and codes
def test_sequences_that_start_out_of_range_write_nothing():
    c = Call(11, [48, 32, 16], [1, 2, 1], 4, 2, 64, 16)
    c.out.fill_(3.0)
    c.dev[0] = dev(np.array([-4, -3, 90, 2 ** 31 - 1], dtype=np.int32))
    c.run()
    torch.cuda.synchronize()
    assert (c.out == 3).all()


@pytest.mark.parametrize("hidden,group", [(512, 512), (4096, 4096), (11008, 128)])
def test_norm_codes_are_rounded_once(hidden, group):
    """No code on the wrong side of a border by more than 2^-40 of the quotient."""
    x, w, r = norm_case(np.random.default_rng(17), 256, hidden, True)
    y8 = torch.empty(256, hidden, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(256, hidden // group, device="cuda")
    srg.lora_rms_norm(x, w, 1e-5, residual=r, y8=y8, scales=scales)
    _, v, s = R.rms_norm(x, r, w, 1e-5, group)
    assert (R.f64(scales) == s).all()
    want, near = nearest_e4m3((v.reshape(256, -1, group) / s[..., None]).reshape(256, hidden))
    assert not ((R.f64(y8) != want) & (near > 2.0 ** -40)).any()


@pytest.mark.parametrize("more", [dict(window=(1 << 32) + 5), dict(window=1 << 32), dict(window=5 - (1 << 32)),
                                  dict(max_query_len=(1 << 32) + 1)])
def test_attention_refuses_sizes_past_32_bits(more):
    """A window of 2^32 + 5 would arrive as one of 5."""
    c = Call(220, [40], [1], 4, 2, 64, 16)
    call = dict(max_query_len=1, window=0)
    with pytest.raises(ValueError, match="32 bits"):
        srg.lora_kv_attention(c.q, *c.dev, c.cache, c.out, c.scale, c.workspace, **{**call, **more})
    assert (c.out == 3).all()


def test_page_size_tells_caches_of_one_shape_apart():
    """Heads of 128 in pages of 64 tokens, read as heads of 64 in pages of 128."""
    shape = srg.kv_cache_shape(6, 2, 128, 64)
    assert shape == srg.kv_cache_shape(6, 2, 64, 128)
    cache = torch.zeros(shape, dtype=torch.uint8, device="cuda")
    slots = torch.arange(3, device="cuda")
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    table, lens = torch.zeros(1, 3, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for d in (128, 64):
        q, k, v = torch.ones(3, 4, d, **bf16), torch.empty(3, 2, d, **bf16), torch.empty(3, 2, d, **bf16)
        out = torch.full((1, 4, d), 3.0, **bf16)
        calls = [lambda **more: srg.lora_kv_append(torch.ones(3, 8 * d, **bf16), None, slots, None, cache, q, **more),
                 lambda **more: srg.lora_kv_read(slots, cache, k, v, **more),
                 lambda **more: srg.lora_kv_attention(q[:1], start, lens, table, cache, out, 1.0, None, 1, **more)]
        for call in calls:
            if d == 128:
                call(page_size=64), call()
                for wrong in (128, 32, 0):
                    with pytest.raises(ValueError, match="page_size"):
                        call(page_size=wrong)
            else:
                with pytest.raises(ValueError, match="page_size 64"):
                    call(page_size=64)
        assert bool((out == (1 if d == 128 else 3)).all())
