"""The operators around the projections on the GPU against their 64-bit forms:
odd sizes, strides, empty rows, poisoned and bad places, other streams, graphs."""

import numpy as np
import pytest
import torch

import segmented_rank_gemm_amd as srg
from tests import attention_reference as R

pytestmark = pytest.mark.gpu

NAN_BITS = 0x7FC1


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return t.to(dtype).cuda() if dtype is not None else t.cuda()


def padded(rows, width, extra, dtype=torch.bfloat16, fill=float("nan")):
    """(view [rows, width], whole): a matrix whose rows lie `extra` elements apart."""
    whole = torch.full((rows, width + extra), fill, device="cuda").to(dtype)
    return whole[:, :width], whole


# ------------------------------------------------------------------ norm
def norm_case(rng, T, hidden, residual, spread=1.0):
    x = R.bf16(rng.standard_normal((T, hidden)) * spread).cuda()
    w = R.bf16(1 + 0.3 * rng.standard_normal(hidden)).cuda()
    r = R.bf16(3 * rng.standard_normal((T, hidden)) * spread).cuda() if residual else None
    return x, w, r


def check_norm(x, w, r, eps, group, sums, y, y8, scales):
    h, v, s = R.rms_norm(x, r, w, eps, group)
    if sums is not None:
        assert np.array_equal(R.f64(sums), h, equal_nan=True)
    if y is not None:
        fine = np.isfinite(v)
        err = np.abs(R.f64(y)[fine] - v[fine])
        # one rounding to bf16, after one to fp32
        assert (err <= (R.HALF_BF16 + 2.0 ** -23) * np.abs(v[fine]) + 2.0 ** -133).all(), err.max()
        assert np.isnan(R.f64(y)[~fine]).all()
    if y8 is not None:
        got = R.f64(scales)
        assert np.array_equal(np.isnan(got), np.isnan(s))
        ok = ~np.isnan(s)
        # v and the division by 448 in 64 bits, one rounding to fp32
        assert (np.abs(got - s)[ok] <= 2.0 ** -23 * s[ok]).all()
        codes = R.f64(y8).reshape(*s.shape, group)
        assert np.isnan(codes[~ok]).all()
        u = v.reshape(*s.shape, group)[ok] / got[ok][:, None]
        # one rounding to e4m3 (steps of 2^-9 below its normal numbers), after one to fp32
        slack = np.maximum(R.HALF_E4M3 * np.abs(u), 2.0 ** -10) * (1 + 2.0 ** -18)
        assert (np.abs(codes[ok] - u) <= slack).all()
        assert (np.abs(codes[ok]) <= 448).all()


@pytest.mark.parametrize("T,hidden,residual,group", [
    (1, 8, True, 8), (3, 64, False, 32), (2, 256, True, 256), (5, 264, True, 264),
    (7, 1024, False, 128), (16, 4096, True, 4096), (33, 4096, True, 64), (3, 4104, True, 4104),
    (9, 8192, True, 8192), (5, 11008, False, 128), (4, 11008, True, 11008), (2, 16640, True, 256),
    (2, 32768, False, 32768), (1, 65536, True, 65536), (2, 65536, True, 32), (300, 512, True, 512),
])
def test_rms_norm(T, hidden, residual, group):
    x, w, r = norm_case(np.random.default_rng(T * hidden), T, hidden, residual)
    sums = torch.empty_like(x) if residual else None
    y, y8 = torch.empty_like(x), torch.empty(T, hidden, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(T, hidden // group, device="cuda")
    srg.lora_rms_norm(x, w, 1e-5, residual=r, residual_out=sums, y=y, y8=y8, scales=scales)
    check_norm(x, w, r, 1e-5, group, sums, y, y8, scales)


def nearest_e4m3(u):
    """(values, how far each u is from a border between two, relative to u)."""
    levels = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    middles = (levels[1:] + levels[:-1]) / 2
    a = np.abs(u)
    code = np.searchsorted(middles, a)
    near = np.minimum(np.abs(a - middles[np.minimum(code, 125)]), np.abs(a - middles[np.maximum(code - 1, 0)]))
    return np.copysign(levels[code], u), near / np.maximum(a, 1e-300)


@pytest.mark.parametrize("hidden,group", [(512, 512), (4096, 4096), (11008, 128)])
def test_rms_norm_codes_are_those_of_the_formula(hidden, group):
    """v is kept to 2^-40 and more up to its rounding: away from a border by more
    than the 2^-24 of the fp32 number in between, each code is the nearest one."""
    x, w, r = norm_case(np.random.default_rng(7), 256, hidden, True)
    y = torch.empty_like(x)
    y8, scales = torch.empty(256, hidden, dtype=torch.float8_e4m3fn, device="cuda"), \
        torch.empty(256, hidden // group, device="cuda")
    srg.lora_rms_norm(x, w, 1e-5, residual=r, y=y, y8=y8, scales=scales)
    _, v, s = R.rms_norm(x, r, w, 1e-5, group)
    assert (R.f64(scales) == s).all()
    want, near = nearest_e4m3((v.reshape(256, -1, group) / s[..., None]).reshape(256, hidden))
    wrong = (R.f64(y8) != want) & (near > 2.0 ** -40)
    # an fp32 number in between may round to a border itself: a share of 2^-24 / 2^-4 of
    # them comes that near, and half of those then go to the wrong side
    assert wrong.sum() == (wrong & (near < 2.0 ** -24)).sum() and wrong.mean() <= 2.0 ** -20
    bits = torch.from_numpy(v).float().bfloat16()
    assert (bits == y.cpu()).double().mean() >= 1 - 2.0 ** -30


@pytest.mark.parametrize("which", ["y", "y8", "sum", "y+y8 without sum"])
def test_rms_norm_outputs_may_be_left_out(which):
    x, w, r = norm_case(np.random.default_rng(3), 5, 520, True)
    sums = torch.empty_like(x) if which == "sum" else None
    y = torch.empty_like(x) if which.startswith("y") and which != "y8" else None
    y8 = torch.empty(5, 520, dtype=torch.float8_e4m3fn, device="cuda") if "y8" in which else None
    scales = torch.empty(5, 1, device="cuda") if "y8" in which else None
    srg.lora_rms_norm(x, w, 1e-6, residual=r, residual_out=sums, y=y, y8=y8, scales=scales)
    check_norm(x, w, r, 1e-6, 520, sums, y, y8, scales)


def test_rms_norm_strides_leave_the_rest_alone():
    x, w, r = norm_case(np.random.default_rng(4), 6, 136, True)
    (xs, _), (rs, _), (os, ow), (ys, yw) = (padded(6, 136, e) for e in (8, 24, 16, 40))
    y8s, y8w = padded(6, 136, 8, torch.float8_e4m3fn, 2.0)
    scales = torch.empty(6, 1, device="cuda")
    xs.copy_(x), rs.copy_(r)
    srg.lora_rms_norm(xs, w, 1e-5, residual=rs, residual_out=os, y=ys, y8=y8s, scales=scales)
    check_norm(x, w, r, 1e-5, 136, os, ys, y8s, scales)
    assert ow[:, 136:].isnan().all() and yw[:, 136:].isnan().all()
    assert (y8w[:, 136:].float() == 2).all()


@pytest.mark.parametrize("hidden", [264, 4096, 20000])
def test_rms_norm_in_place(hidden):
    x, w, r = norm_case(np.random.default_rng(5), 4, hidden, True)
    x0, r0, y = x.clone(), r.clone(), torch.empty_like(x)
    srg.lora_rms_norm(x, w, 1e-5, residual=r, residual_out=r, y=x)
    check_norm(x0, w, r0, 1e-5, hidden, r, x, None, None)
    x, r = x0.clone(), r0.clone()
    srg.lora_rms_norm(x, w, 1e-5, residual=r, residual_out=x, y=y)
    check_norm(x0, w, r0, 1e-5, hidden, x, y, None, None)


@pytest.mark.parametrize("hidden,group", [(512, 512), (512, 32), (2304, 2304), (2304, 256), (12288, 12288),
                                          (12288, 64)])
def test_rms_norm_of_special_rows(hidden, group):
    x, w, _ = norm_case(np.random.default_rng(6), 8, hidden, False)
    x[0] = 0                      # nothing: scales of 2^-126, zeros
    x[1, 77] = float("inf")       # its own v NaN, the others 0
    x[2, 5] = float("nan")        # all NaN
    x[3] = 3e38                   # the squares pass fp32
    x[4] = 1e-38
    w[9] = 0
    x[5, 100] = -float("inf")
    x[6] *= 1e-30
    y, y8 = torch.empty_like(x), torch.empty(8, hidden, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(8, hidden // group, device="cuda")
    for eps in (1e-5, 0.0):
        y.fill_(1), y8.fill_(1), scales.fill_(1)
        srg.lora_rms_norm(x[0 if eps else 1:], w, eps, y=y[0 if eps else 1:], y8=y8[0 if eps else 1:],
                          scales=scales[0 if eps else 1:])
        a = 0 if eps else 1
        check_norm(x[a:], w, None, eps, group, None, y[a:], y8[a:], scales[a:])
    assert y[2].isnan().all() and int(y[1].isnan().sum()) == 1


# ------------------------------------------------------------------ append and read
def cache_of(pages, kv, d, page, fill=0xA5):
    return torch.full(srg.kv_cache_shape(pages, kv, d, page), fill, dtype=torch.uint8, device="cuda")


def append_case(seed, T, hq, kv, d, page, rot, pages=None, rows=500, ld_extra=0, spread=2.0):
    rng = np.random.default_rng(seed)
    pages = pages or T // page + 3
    x = R.bf16(rng.standard_normal((T, (hq + 2 * kv) * d)) * spread)
    qkv, _ = padded(T, (hq + 2 * kv) * d, ld_extra)
    qkv.copy_(x)
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    positions = rng.integers(0, rows, T).astype(np.int32)
    rope = srg.rope_table(rows, rot) if rot else None
    return x, qkv, slots, positions, rope, pages


def check_append(x, slots, positions, rope, hq, kv, d, pages, page, interleaved, q_out, cache, before):
    T = len(slots)
    v = R.f64(x).reshape(T, hq + 2 * kv, d)
    if rope is not None:
        turned = R.rotate(v[:, :hq + kv], R.f64(rope), positions, interleaved)
        v = np.concatenate([turned, v[:, hq + kv:]], axis=1)
    q, k = v[:, :hq], v[:, hq:hq + kv].astype(np.float32).astype(np.float64)
    # one rounding to bf16, after one to fp32
    assert (np.abs(R.f64(q_out) - q) <= (R.HALF_BF16 + 2.0 ** -23) * np.abs(q)).all()
    ok = (slots >= 0) & (slots < pages * page)
    k_out, v_out = (torch.full((T, kv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    srg.lora_kv_read(dev(slots), cache, k_out, v_out)
    for got, want in ((k_out, k), (v_out, v[:, hq + kv:])):
        got = R.f64(got)
        assert np.array_equal(got[ok], R.held(want[ok]), equal_nan=True)
        assert (got[~ok] == 0).all()
    # the places of no token are as they were
    codes = cache[..., :page * d // 2].unflatten(-1, (page, d // 2)).cpu().numpy()
    scales = cache[..., page * d // 2:].unflatten(-1, (d // 32, page)).cpu().numpy()
    free = np.ones(pages * page, dtype=bool)
    free[slots[ok]] = False
    at = np.nonzero(free)[0]
    assert (codes[at // page, :, :, at % page] == before).all()
    assert (scales[at // page, :, :, :, at % page] == before).all()


@pytest.mark.parametrize("T,hq,kv,d,page,rot,interleaved,ld_extra", [
    (1, 1, 1, 64, 16, 64, False, 0), (1, 32, 32, 128, 64, 128, False, 0), (7, 8, 1, 128, 16, 128, False, 8),
    (33, 16, 2, 128, 32, 64, False, 0), (65, 6, 3, 64, 16, 32, True, 24), (40, 4, 4, 128, 128, 128, True, 0),
    (19, 12, 4, 64, 256, 16, False, 0), (23, 5, 5, 128, 64, 0, False, 0), (300, 64, 8, 128, 64, 128, False, 0),
    (17, 3, 1, 64, 64, 48, False, 0), (17, 3, 1, 64, 64, 48, True, 0),
])
def test_kv_append(T, hq, kv, d, page, rot, interleaved, ld_extra):
    x, qkv, slots, positions, rope, pages = append_case(T + d, T, hq, kv, d, page, rot, ld_extra=ld_extra)
    cache = cache_of(pages, kv, d, page)
    q_out = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")
    srg.lora_kv_append(qkv, dev(positions), dev(slots), rope, cache, q_out, interleaved=interleaved)
    check_append(x, slots, positions, rope, hq, kv, d, pages, page, interleaved, q_out, cache, 0xA5)


def test_kv_append_special_blocks():
    T, hq, kv, d, page = 12, 1, 2, 64, 16
    x, qkv, slots, positions, _, pages = append_case(1, T, hq, kv, d, page, 0)
    v = x.view(T, hq + 2 * kv, d)
    v[0, 1:] = 0
    v[1, 1, 3] = float("inf")
    v[2, 2, 40] = float("nan")
    v[3, 3, 0] = -float("inf")
    v[4, 1:] = 3e38
    v[5, 1:] = 1e-38
    v[6, 1:] = torch.tensor([2.0 ** -133] * 64)   # below the smallest scale's half step
    v[7, 1, :8] = torch.tensor([7.0, 6.0, 5.0, 2.5, 1.75, 1.25, 0.25, -0.75])
    v[7, 1, 8:32] = 0
    v[8, 1, :32] = 7.0625                           # past 7 / 8 of the next power
    v[9, 2:] = -0.0
    v[10, 1:] = 2.0 ** 127
    v[11, 1:] = torch.linspace(-1, 1, 64) * 2.0 ** -126
    qkv.copy_(x)
    cache = cache_of(pages, kv, d, page)
    q_out = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")
    srg.lora_kv_append(qkv, None, dev(slots), None, cache, q_out)
    check_append(x, slots, positions, None, hq, kv, d, pages, page, False, q_out, cache, 0xA5)


def test_kv_append_places_and_positions_out_of_range():
    T, hq, kv, d, page = 16, 4, 2, 128, 16
    x, qkv, slots, positions, rope, pages = append_case(2, T, hq, kv, d, page, 128)
    slots[[0, 3, 5]] = [-1, pages * page, 1 << 60]
    slots[7] = -(1 << 60)
    cache = cache_of(pages, kv, d, page)
    q_out = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")
    srg.lora_kv_append(qkv, dev(positions), dev(slots), rope, cache, q_out)
    check_append(x, slots, positions, rope, hq, kv, d, pages, page, False, q_out, cache, 0xA5)
    # a position that the table does not have: the token is padding
    bad = positions.copy()
    bad[[1, 2, 4]] = [-1, 500, 2 ** 31 - 1]
    cache2, q2 = cache_of(pages, kv, d, page), torch.full_like(q_out, 3.0)
    srg.lora_kv_append(qkv, dev(bad), dev(slots), rope, cache2, q2)
    assert (q2[[1, 2, 4]] == 3).all()
    keep = [i for i in range(T) if i not in (1, 2, 4)]
    assert torch.equal(q2[keep], q_out[keep])
    check_append(x[keep], slots[keep], positions[keep], rope, hq, kv, d, pages, page, False, q2[keep], cache2, 0xA5)


def test_kv_append_far_positions():
    """Rows of the table at its far end, and a q_out with rows apart."""
    T, hq, kv, d, page = 8, 2, 2, 128, 64
    x, qkv, slots, _, _, pages = append_case(3, T, hq, kv, d, page, 0)
    rope = srg.rope_table(131072, 128)
    positions = (131071 - np.arange(T)).astype(np.int32)
    cache = cache_of(pages, kv, d, page)
    whole = torch.full((T, hq * d + 64), 3.0, dtype=torch.bfloat16, device="cuda")
    q_out = whole.as_strided((T, hq, d), (hq * d + 64, d, 1))
    srg.lora_kv_append(qkv, dev(positions), dev(slots), rope, cache, q_out)
    check_append(x, slots, positions, rope, hq, kv, d, pages, page, False, q_out, cache, 0xA5)
    assert (whole[:, hq * d:] == 3).all()


def test_kv_read_repeats_and_one_side():
    data, values = R.random_cache(np.random.default_rng(8), 3, 2, 128, 16)
    data[1, 0, 1, 16 * 64 + 2 * 16 + 5] = 255   # a block that held an infinity
    cache = dev(data)
    slots = np.array([5, 5, 47, -1, 21, 48, 0], dtype=np.int64)
    k, v = (torch.full((7, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    srg.lora_kv_read(dev(slots), cache, k, None)
    srg.lora_kv_read(dev(slots), cache, None, v)
    for i, s in enumerate(slots):
        for part, got in ((0, k), (1, v)):
            want = values[s // 16, part, :, s % 16] if 0 <= s < 48 else np.zeros((2, 128))
            if s == 21 and part == 0:
                want = want.copy()
                want[1, 64:96] = np.nan
            assert np.array_equal(R.f64(got[i]), want, equal_nan=True), (i, part)


# ------------------------------------------------------------------ attention
class Call:
    """One call's tensors: random cache, pages in random order, every place that no
    sequence holds poisoned with NaN scales."""

    def __init__(self, seed, lens, queries, hq, kv, d, page, window=0, spare=3, pages=None, extra=0,
                 row_order=True):
        rng = np.random.default_rng(seed)
        need = [-(-l // page) for l in lens]
        self.pages = pages or sum(need) + spare
        self.data, self.values = R.random_cache(rng, self.pages, kv, d, page)
        ids = rng.permutation(self.pages)
        self.table = np.full((len(lens), max(1, max(need)) + 1), -5, dtype=np.int32)
        poison = np.ones((self.pages, page), dtype=bool)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = ids[at:at + n]
            for i in range(n):
                poison[ids[at + i], :min(page, lens[s] - i * page)] = False
            at += n
        scales = self.data[..., page * d // 2:].reshape(self.pages, 2, kv, d // 32, page)
        scales[np.broadcast_to(poison[:, None, None, None], scales.shape)] = 255
        self.data[..., page * d // 2:] = scales.reshape(self.pages, 2, kv, -1)
        self.values[np.broadcast_to(poison[:, None, None, :, None], self.values.shape)] = np.nan
        self.start = np.concatenate([[0], np.cumsum(queries)]).astype(np.int32)
        self.lens = np.array(lens, dtype=np.int32)
        T = int(self.start[-1])
        self.shape = (T, hq, kv, d, page, window, max(queries))
        self.qh = R.bf16(rng.standard_normal((T, hq, d)))
        self.q = torch.full((T, hq * d + extra), float("nan"), dtype=torch.bfloat16, device="cuda") \
            .as_strided((T, hq, d), (hq * d + extra, d, 1))
        self.q.copy_(self.qh)
        self.whole = torch.full((T, hq * d + extra), 3.0, dtype=torch.bfloat16, device="cuda")
        self.out = self.whole.as_strided((T, hq, d), (hq * d + extra, d, 1))
        self.scale = 0.5 * d ** -0.5
        self.cache = dev(self.data)
        self.dev = [dev(a) for a in (self.start, self.lens, self.table)]
        self.workspace = srg.kv_attention_workspace(len(lens), max(queries), self.table.shape[1] * page, hq, kv, d)
        if self.workspace is not None:
            self.workspace.fill_(255)   # NaN in every float

    def run(self, stream=None, **more):
        srg.lora_kv_attention(self.q, *self.dev, self.cache, self.out, self.scale, self.workspace,
                              self.shape[6], window=self.shape[5], stream=stream, **more)

    def want(self, **more):
        T, hq, kv, d, page, window, _ = self.shape
        return R.attention(R.f64(self.qh), self.values, self.start, self.lens, self.table, page, self.scale,
                           window, **more)

    def check(self, want=None, rows=None):
        out, slack = want or self.want()
        got = R.f64(self.out)
        rows = slice(None) if rows is None else rows
        assert np.isfinite(got[rows]).all()
        over = np.abs(got[rows] - out[rows]) - slack[rows]
        assert (over <= 0).all(), (over.max(), np.unravel_index(over.argmax(), over.shape))
        assert self.runs_alike()
        return out, slack

    def runs_alike(self):
        # a second call, on the workspace as the first one left it, gives the same bits
        first = self.out.clone()
        self.run()
        torch.cuda.synchronize()
        return torch.equal(first.view(torch.int16), self.out.view(torch.int16))


CASES = [
    # lens, queries, q_heads, kv_heads, head_dim, page, window
    ([1], [1], 1, 1, 64, 16, 0),
    ([1, 2, 15, 16, 17], [1] * 5, 4, 2, 128, 16, 0),
    ([31, 32, 33, 63, 64, 65], [1] * 6, 8, 1, 128, 64, 0),
    ([0, 5, 0, 127, 128, 129], [1] * 6, 3, 3, 64, 32, 0),
    ([200], [1], 16, 1, 128, 128, 0),
    ([255, 257], [1, 1], 24, 1, 128, 256, 0),      # more rows than one tile of 16
    ([300, 77], [1, 1], 40, 2, 64, 16, 0),
    ([1000], [1], 32, 32, 128, 64, 0),
    ([3000, 1, 511], [1, 1, 1], 8, 2, 128, 16, 0),
    ([5000], [1], 2, 1, 64, 64, 0),
    ([9, 40, 3], [3, 5, 3], 6, 2, 128, 16, 0),     # a few drafted tokens
    ([2, 0, 4], [5, 2, 4], 4, 4, 64, 16, 0),       # more queries than tokens: empty rows
    ([100, 33], [17, 33], 4, 1, 128, 32, 0),
    ([130], [130], 8, 2, 64, 64, 0),               # a whole prompt
    ([257, 64, 5], [70, 64, 5], 2, 2, 128, 16, 0),
    ([400], [90], 12, 1, 64, 32, 0),
    ([600, 20], [1, 1], 4, 2, 128, 16, 33),        # windows
    ([70, 300], [40, 64], 4, 2, 64, 16, 7),
    ([90, 100], [3, 2], 8, 8, 128, 16, 1),
    ([500], [200], 4, 1, 128, 64, 150),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_kv_attention(case):
    c = Call(len(case[0]) + case[0][0], *case)
    c.run()
    c.check()


def spread(n, longest, seed):
    return np.random.default_rng(seed).integers(0, longest, n).tolist()


# More sequences than a wave ranks, and launches that just fill the device, in which
# the order of the sequences turns round half way.
BATCHES = [
    (spread(70, 41, 1), [1] * 70, 4, 2, 64, 16, 0),
    (spread(65, 90, 2), [1, 3] * 32 + [1], 6, 2, 128, 16, 20),
    (spread(40, 70, 3), [1] * 40, 16, 8, 64, 16, 0),
    (spread(64, 70, 4), [1] * 64, 8, 8, 64, 32, 0),
    (spread(33, 70, 5), [2] * 33, 32, 8, 128, 16, 0),
]


@pytest.mark.parametrize("case", BATCHES, ids=[str(i) for i in range(len(BATCHES))])
def test_kv_attention_batches(case):
    c = Call(40 + len(case[0]), *case)
    c.run()
    c.check()


# Many rows over enough (sequence, key head, 128 rows) that operands are shared by a
# workgroup: lens, queries, q_heads, kv_heads, head_dim, page, window
MANY = [
    ([128, 300, 1, 0, 64, 65, 190, 257] * 2, [128] * 16, 32, 32, 64, 16, 0),
    ([300, 900, 431, 77], [300, 129, 250, 77], 64, 8, 128, 64, 0),
    ([300, 900, 431, 77], [300, 129, 250, 90], 64, 8, 128, 16, 100),
    ([500, 200, 640], [180, 200, 1], 48, 16, 64, 32, 0),
    ([500, 200, 640], [180, 200, 1], 48, 16, 128, 128, 37),
]


def sample(T, hq, n, seed=0):
    rng = np.random.default_rng(seed)
    only = np.zeros((T, hq), dtype=bool)
    only[rng.integers(0, T, n), rng.integers(0, hq, n)] = True
    only[[0, -1]] = True
    return only


@pytest.mark.parametrize("case", MANY, ids=[str(i) for i in range(len(MANY))])
def test_kv_attention_many_rows(case):
    c = Call(30 + len(case[0]), *case)
    for s in range(0, len(case[0]), 2):             # and pages that do not exist
        if c.table.shape[1] > 3:
            c.table[s, 2] = c.pages + s
    c.dev[2] = dev(c.table)
    c.run()
    only = sample(*c.shape[:2], 1500)
    out, slack = c.want(only=only)
    got = R.f64(c.out)
    assert np.isfinite(got).all()
    assert (np.abs(got - out) <= slack)[only].all()
    assert c.runs_alike()


@pytest.mark.parametrize("window", [0, 60])
def test_kv_attention_many_rows_nan_values(window):
    c = Call(31, [400, 310, 350, 300], [300, 290, 280, 300], 64, 8, 64, 32, window)
    data, hit = c.data.copy(), np.zeros((*c.shape[:2], 64), dtype=bool)
    for s, t in ((0, 120), (0, 399), (1, 5), (2, 200), (3, 0)):
        page, at = c.table[s, t // 32], t % 32
        data[page, 1, 3, 32 * 32 + (t % 2) * 32 + at] = 255     # head 3, block t % 2
        queries, length = c.start[s + 1] - c.start[s], c.lens[s]
        for i in range(queries):
            place = length - queries + i
            if t <= place and (not window or t > place - window):
                hit[c.start[s] + i, 24:32, (t % 2) * 32:(t % 2) * 32 + 32] = True
    c.cache = dev(data)
    c.run()
    got = R.f64(c.out)
    assert np.array_equal(np.isnan(got), hit)
    only = sample(*c.shape[:2], 1000, 1)
    only[:, 24:32] |= sample(c.shape[0], 8, 400, 2)
    out, slack = c.want(only=only)
    assert (np.abs(got - out) <= slack)[only[..., None] & ~hit].all()


def test_kv_attention_strides_and_rows_of_no_sequence():
    c = Call(9, [40, 50], [3, 2], 4, 2, 64, 16, extra=24)
    # the second sequence starts one row later: row 3 is nobody's; row 5 would be past the end
    c.start = np.array([0, 3, 5], dtype=np.int32)
    c.run()
    c.check()
    assert (c.whole[:, 4 * 64:] == 3).all()
    q, out = c.q, c.out
    more = torch.full((7, 4 * 64), 3.0, dtype=torch.bfloat16, device="cuda").view(7, 4, 64)
    big = torch.zeros(7, 4, 64, dtype=torch.bfloat16, device="cuda")
    big[1:6] = q
    start = dev(np.array([1, 4, 6], dtype=np.int32))
    srg.lora_kv_attention(big, start, *c.dev[1:], c.cache, more, c.scale, c.workspace, 3)
    assert torch.equal(more[1:6], out) and (more[0] == 3).all() and (more[6] == 3).all()


def test_kv_attention_bad_pages_are_skipped():
    c = Call(10, [100, 64, 40], [1, 4, 1], 8, 2, 128, 16)
    c.table[0, 1], c.table[0, 6], c.table[1, 0] = -1, c.pages, 2 ** 31 - 1
    c.table[2, :3] = [-1, -2 ** 31, c.pages + 7]   # nothing left: zeros
    c.dev[2] = dev(c.table)
    c.run()
    out, _ = c.check()
    assert (out[-1] == 0).all() and (c.out[-1] == 0).all()


def test_kv_attention_bad_lengths_and_starts_stay_inside():
    """Lengths past the table, negative lengths, and starts out of range."""
    c = Call(11, [48, 32, 16], [1, 2, 1], 4, 2, 64, 16)
    c.lens = np.array([48, -7, 16], dtype=np.int32)
    c.dev[1] = dev(c.lens)
    c.run()
    c.check()
    assert (c.out[1:3] == 0).all()
    before = c.out.clone()
    c.out.fill_(3.0)
    c.dev[0] = dev(np.array([-4, -3, 90, 2 ** 31 - 1], dtype=np.int32))
    c.run()
    torch.cuda.synchronize()
    kept = (c.out == 3).flatten(1).all(1)
    assert kept.any() and torch.isfinite(before).all()
    # a length past max_seq_len counts as max_seq_len
    c = Call(12, [80], [1], 4, 1, 64, 16)
    c.dev[1] = dev(np.array([2 ** 31 - 1], dtype=np.int32))
    c.run(max_seq_len=64)
    c.lens = np.array([64], dtype=np.int32)
    out, slack = c.want()
    assert (np.abs(R.f64(c.out) - out) <= slack).all()


def test_kv_attention_queries_past_the_most_are_left():
    c = Call(13, [50], [6], 4, 2, 64, 16)
    srg.lora_kv_attention(c.q, *c.dev, c.cache, c.out, c.scale, c.workspace, 4)
    out, slack = c.want()
    assert (np.abs(R.f64(c.out) - out) <= slack)[:4].all() and (c.out[4:] == 3).all()


def test_kv_attention_special_queries_keep_to_their_rows():
    c = Call(14, [70, 70], [2, 1], 4, 2, 128, 16)
    c.q[1, 2, 5] = float("nan")
    c.q[2, 0, 9] = float("inf")
    c.run()
    got = R.f64(c.out)
    out, slack = c.want()
    assert np.isnan(got[1, 2]).all() and np.isnan(got[2, 0]).all()
    ok = np.ones((3, 4), dtype=bool)
    ok[1, 2] = ok[2, 0] = False
    assert (np.abs(got - out) <= slack)[ok].all()


def test_kv_attention_special_keys_and_values():
    """A seen NaN block: a key's reaches all of the row, a value's its own elements."""
    c = Call(15, [40, 40], [1, 1], 2, 2, 64, 16)
    data = c.data.copy()
    page0, page1 = c.table[0, 1], c.table[1, 1]
    data[page0, 0, 1, 16 * 32 + 4] = 255           # sequence 0, head 1, token 20, first block's key
    data[page1, 1, 0, 16 * 32 + 16 + 4] = 255      # sequence 1, head 0, token 20, second block's value
    c.cache = dev(data)
    c.run()
    got = R.f64(c.out)
    out, slack = c.want()
    assert np.isnan(got[0, 1]).all() and np.isnan(got[1, 0, 32:]).all()
    ok = np.ones(got.shape, dtype=bool)
    ok[0, 1] = False
    ok[1, 0, 32:] = False
    assert (np.abs(got - out) <= slack)[ok].all()


def test_kv_attention_far_scores():
    """Scores hundreds apart: the running maximum moves a long way, both ways."""
    for sign in (1, -1):
        c = Call(16, [700], [1], 4, 2, 128, 16)
        c.scale = sign * 3.0
        c.run()
        c.check()


def test_kv_attention_scale_of_zero_takes_the_mean():
    c = Call(19, [90, 200], [3, 40], 4, 2, 64, 16, 50)
    c.scale = 0.0
    c.run()
    c.check()


@pytest.mark.parametrize("queries,window", [(5, 0), (5, 3), (40, 0), (150, 0), (150, 20)])
def test_kv_attention_nan_value_that_some_queries_see(queries, window):
    """A NaN value block among the last tokens reaches the queries that see its
    token, and its own elements only."""
    c = Call(20, [170], [queries], 2, 1, 128, 32, window)
    t = 170 - queries + queries // 2               # seen from query queries // 2 on
    data, values = c.data.copy(), c.values.copy()
    page, at = c.table[0, t // 32], t % 32
    data[page, 1, 0, 32 * 64 + 2 * 32 + at] = 255   # elements 64..95
    c.cache = dev(data)
    c.run()
    got = R.f64(c.out)
    out, slack = c.want()
    hit = np.zeros(got.shape, dtype=bool)
    last = queries if not window else queries // 2 + window
    hit[queries // 2:last, :, 64:96] = True
    assert np.isnan(got[hit]).all() and np.isfinite(got[~hit]).all()
    assert (np.abs(got - out) <= slack)[~hit].all()


@pytest.mark.parametrize("window", [1, 64, 65, 500, 4999, 5000, 2 ** 31 - 1])
def test_kv_attention_windows_on_the_long_workspace(window):
    """The workspace is sized without the window; with one the parts are others."""
    c = Call(21, [5000, 300], [1, 1], 2, 1, 64, 16, window)
    c.run()
    c.check()


def test_kv_attention_past_four_gigabytes():
    kv, d, page = 8, 128, 64
    pages = 66000                                   # 4.6 GB
    shape = srg.kv_cache_shape(pages, kv, d, page)
    c = Call(17, [130, 64], [1, 1], 16, kv, d, page)
    cache = torch.full(shape, 255, dtype=torch.uint8, device="cuda")
    cache[pages - c.pages:] = c.cache
    table = np.where(c.table >= 0, c.table + pages - c.pages, c.table)
    srg.lora_kv_attention(c.q, *c.dev[:2], dev(table), cache, c.out, c.scale, c.workspace, 1)
    out, slack = c.want()
    assert (np.abs(R.f64(c.out) - out) <= slack).all()
    slots = np.array([pages * page - 1, (pages - 1) * page], dtype=np.int64)
    qkv = R.bf16(np.random.default_rng(1).standard_normal((2, 24 * d))).cuda()
    q_out = torch.empty(2, 8, d, dtype=torch.bfloat16, device="cuda")
    k_out, v_out = (torch.empty(2, kv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    srg.lora_kv_append(qkv, None, dev(slots), None, cache, q_out)
    srg.lora_kv_read(dev(slots), cache, k_out, v_out)
    x = R.f64(qkv).reshape(2, 24, d)
    assert np.array_equal(R.f64(k_out), R.held(x[:, 8:16])) and np.array_equal(R.f64(v_out), R.held(x[:, 16:]))


@pytest.mark.parametrize("case", [CASES[8], CASES[10], CASES[13]], ids=["long", "drafts", "prompt"])
def test_kv_attention_same_bits_each_time_and_on_another_stream(case):
    c = Call(18, *case)
    c.run()
    first = c.out.clone()
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, other, None):
        c.out.fill_(3.0)
        torch.cuda.synchronize()
        c.run(stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(first.view(torch.int16), c.out.view(torch.int16))


def test_layer_in_a_graph():
    """Norm, append and attention captured once and replayed on other tokens, places
    and lengths, each replay against the same calls made one by one."""
    T, hq, kv, d, page, hidden, pages = 4, 8, 2, 128, 16, 1536, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    x, res = (torch.empty(T, hidden, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w = torch.ones(hidden, dtype=torch.bfloat16, device="cuda")
    sums, y = torch.empty_like(x), torch.empty_like(x)
    y8 = torch.empty(T, hidden, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(T, 1, device="cuda")
    positions = torch.zeros(T, dtype=torch.int32, device="cuda")
    slots = torch.zeros(T, dtype=torch.int64, device="cuda")
    start = torch.arange(T + 1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(T, dtype=torch.int32, device="cuda")
    table = torch.randperm(pages, device="cuda", generator=g).int().view(T, pages // T).contiguous()
    cache = dev(R.random_cache(np.random.default_rng(2), pages, kv, d, page)[0])
    rope = srg.rope_table(512, d)
    q, out = (torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = srg.kv_attention_workspace(T, 1, table.shape[1] * page, hq, kv, d)

    def layer():
        srg.lora_rms_norm(x, w, 1e-5, residual=res, residual_out=sums, y=y, y8=y8, scales=scales)
        srg.lora_kv_append(y, positions, slots, rope, cache, q)
        srg.lora_kv_attention(q, start, lens, table, cache, out, d ** -0.5, ws, 1)

    def new(k):
        x.normal_(generator=g), res.normal_(generator=g)
        n = torch.randint(1, table.shape[1] * page, (T,), device="cuda", generator=g)
        lens.copy_(n), positions.copy_(n - 1)
        slots.copy_(table.gather(1, ((n - 1) // page)[:, None]).long()[:, 0] * page + (n - 1) % page)

    new(0)
    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for k in range(4):
        new(k)
        held = cache.clone()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (sums, y, scales, q, out, cache)]
        cache.copy_(held)
        layer()
        torch.cuda.synchronize()
        for a, b in zip(got, (sums, y, scales, q, out, cache)):
            assert torch.equal(a, b), k


def test_binding_refuses_what_does_not_fit():
    """Tensors of another type, shape or layout are refused before the library is
    called, by name."""
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    y8, s = torch.empty(4, 256, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(4, 2, device="cuda")
    norm = lambda **k: srg.lora_rms_norm(**{**dict(x=x, weight=w, eps=1e-5, y=torch.empty_like(x)), **k})  # noqa: E731
    for error, name, more in [
            (TypeError, "x", dict(x=x.float())), (TypeError, "x", dict(x=x.cpu())),
            (ValueError, "x", dict(x=x[0])), (ValueError, "x", dict(x=x.t().contiguous().t(), weight=w)),
            (TypeError, "weight", dict(weight=None)), (ValueError, "weight", dict(weight=w[:8])),
            (ValueError, "weight", dict(weight=torch.ones(512, dtype=torch.bfloat16, device="cuda")[::2])),
            (ValueError, "y", dict(y=x[:3])), (TypeError, "y8", dict(y8=x, scales=s)),
            (ValueError, "scales", dict(y8=y8, scales=s[:, 0])), (ValueError, "scales", dict(y8=y8, scales=torch.empty(4, 3, device="cuda"))),
            (ValueError, "scales", dict(y8=y8, scales=torch.empty(4, 4, device="cuda")[:, :2]))]:
        with pytest.raises(error, match=name):
            norm(**more)
    with pytest.raises(srg.LoraError):
        norm(y8=y8)                                  # no scales
    with pytest.raises(srg.LoraError):
        norm(eps=-1.0)
    cache = cache_of(4, 2, 128, 16)
    slots, q = torch.zeros(3, dtype=torch.int64, device="cuda"), torch.empty(3, 4, 128, dtype=torch.bfloat16, device="cuda")
    qkv = torch.zeros(3, 8 * 128, dtype=torch.bfloat16, device="cuda")
    append = lambda **k: srg.lora_kv_append(**{**dict(qkv=qkv, positions=None, slots=slots, rope=None, cache=cache,  # noqa: E731
                                                      q_out=q), **k})
    for error, name, more in [
            (ValueError, "qkv", dict(qkv=qkv[:, :-8])), (TypeError, "slots", dict(slots=slots.int())),
            (ValueError, "cache", dict(cache=cache[..., :-2].contiguous())), (ValueError, "cache", dict(cache=cache[:, :1])),
            (ValueError, "q_out", dict(q_out=q[0])), (ValueError, "q_out", dict(q_out=q.transpose(1, 2).contiguous().transpose(1, 2))),
            (TypeError, "positions", dict(rope=srg.rope_table(8, 128)))]:
        with pytest.raises(error, match=name):
            append(**more)
    with pytest.raises(ValueError, match="k_out"):
        srg.lora_kv_read(slots, cache, q, None)
    c = Call(50, [20], [1], 4, 2, 64, 16)
    for error, name, more in [
            (ValueError, "query_start", {0: c.dev[0][:1]}), (TypeError, "seq_lens", {1: c.dev[1].long()}),
            (ValueError, "page_table", {2: c.dev[2][0]})]:
        with pytest.raises(error, match=name):
            srg.lora_kv_attention(c.q, *[more.get(i, t) for i, t in enumerate(c.dev)], c.cache, c.out, 1.0, None, 1)
    with pytest.raises(ValueError, match="max_seq_len"):
        c.run(max_seq_len=1000)
