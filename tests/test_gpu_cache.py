"""Drafted tokens and caches of bounded length on the GPU against their 64-bit forms:
trees of every size, masks that leave rows empty, windows, padded batches, bad places,
ties, moves onto places that others still read."""

import numpy as np
import pytest
import torch

import segmented_rank_gemm_amd as srg
from tests import attention_reference as R
from tests import cache_reference as C

pytestmark = pytest.mark.gpu


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return t.to(dtype).cuda() if dtype is not None else t.cuda()


def ints(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ masks
@pytest.mark.parametrize("counts,words", [
    ([1], 1), ([5, 0, 64], 1), ([63, 65, 1], 2), ([200, 7], 4), ([512, 130], 8), ([3] * 70, 1)])
def test_draft_masks(counts, words):
    rng = np.random.default_rng(sum(counts))
    trees = [C.random_tree(rng, n, roots=1 + n // 20) for n in counts]
    start = [0] + list(np.cumsum(counts))
    parents = [p for tree in trees for p in tree]
    masks = torch.full((start[-1], words), -7, dtype=torch.int64, device="cuda")
    positions = torch.full((start[-1],), -9, dtype=torch.int32, device="cuda")
    first = [int(x) for x in rng.integers(0, 100000, len(counts))]
    srg.lora_draft_masks(ints(parents), ints(start), masks, positions, ints(first))
    paths = [p for tree in trees for p in C.ancestors(tree)]
    assert np.array_equal(masks.cpu().numpy(), C.words_of(paths, words))
    base = np.repeat(first, counts)
    assert positions.cpu().tolist() == [b + len(p) - 1 for b, p in zip(base, paths)]
    srg.lora_draft_masks(ints(parents), ints(start), positions=positions)
    assert positions.cpu().tolist() == [len(p) - 1 for p in paths]


def test_draft_masks_of_a_chain():
    n = 512
    masks = torch.zeros(n, 8, dtype=torch.int64, device="cuda")
    positions = torch.zeros(n, dtype=torch.int32, device="cuda")
    srg.lora_draft_masks(ints([i - 1 for i in range(n)]), ints([0, n]), masks, positions)
    assert np.array_equal(masks.cpu().numpy(), C.words_of([set(range(i + 1)) for i in range(n)], 8))
    assert positions.cpu().tolist() == list(range(n))


def test_draft_masks_bad_parents_are_roots_and_other_rows_are_left():
    # sequences: a start below 0, one whose rows go past the tokens, one of more drafts than bits
    parents = [3, 0, -5, 2, 4, 1, 2 ** 31 - 1, 0, 6] + list(range(-1, 69))
    T = len(parents)
    for start, done in (([0, 9, 79], range(0, 73)), ([-2, 3, 3, 9, 200], range(3, 67)), ([0, 0, 0, 0], []),
                        ([5, 2, T, 100], range(2, 66))):
        masks = torch.full((T, 1), -7, dtype=torch.int64, device="cuda")
        positions = torch.full((T,), -9, dtype=torch.int32, device="cuda")
        srg.lora_draft_masks(ints(parents), ints(start), masks, positions)
        want, depth = np.full((T, 1), -7), [-9] * T
        for s in range(len(start) - 1):
            if not 0 <= start[s] < T or start[s + 1] <= start[s]:
                continue
            mine = parents[start[s]:min(start[s + 1], T)][:64]
            for i, path in enumerate(C.ancestors(mine)):
                want[start[s] + i] = C.words_of([path], 1)[0]
                depth[start[s] + i] = len(path) - 1
        assert np.array_equal(masks.cpu().numpy(), want) and positions.cpu().tolist() == depth


# ------------------------------------------------------------------ attention and mass
class Step:
    """Sequences of random lengths and queries over a random cache, with masks or without."""

    def __init__(self, seed, lens, queries, hq, kv, d, page, bits="tree", words=None, window=0, spare=3,
                 extra_rows=0, low=120, high=128):
        rng = np.random.default_rng(seed)
        self.lens, self.queries, self.page, self.window, self.d = lens, queries, page, window, d
        self.start = [0] + [int(x) for x in np.cumsum(queries)]
        self.T = self.start[-1] + extra_rows
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages)
        self.table = np.full((len(lens), max(1, max(need))), -1, dtype=np.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.cache, self.values = R.random_cache(rng, self.pages, kv, d, page, low, high)
        self.q = R.bf16(rng.standard_normal((self.T, hq, d)))
        self.max_q = max(1, max(queries))
        self.words = words or -(-self.max_q // 64)
        if bits == "tree":
            self.bits = [p for n in queries for p in C.ancestors(C.random_tree(rng, n, 1 + n // 30))]
        elif bits == "any":  # not a tree's: bits of tokens behind, and of none, and rows without any
            self.bits = [set(int(x) for x in np.flatnonzero(rng.random(64 * self.words) < p))
                         for p in rng.choice([0.0, 0.02, 0.5, 1.0], self.T)]
        else:
            self.bits = None
        if self.bits is not None:
            self.bits += [set() for _ in range(self.T - len(self.bits))]
        self.scale = d ** -0.5
        self.hq, self.kv = hq, kv

    def masks(self):
        return None if self.bits is None else dev(C.words_of(self.bits, self.words))

    def want(self, **more):
        return C.tree_attention(R.f64(self.q), self.values, self.start, self.lens, self.table, self.page, self.scale,
                                self.bits, self.window, **more)

    def attend(self, lse=True, **more):
        B = len(self.lens)
        out = torch.full((self.T, self.hq, self.d), float("nan"), dtype=torch.bfloat16, device="cuda")
        sums = torch.full((self.T, self.hq), float("nan"), device="cuda") if lse else None
        ws = srg.kv_tree_attention_workspace(B, self.max_q, self.table.shape[1] * self.page, self.hq, self.kv, self.d)
        if ws is not None:
            ws.fill_(255)
        srg.lora_kv_tree_attention(self.q.cuda(), ints(self.start), ints(self.lens), dev(self.table), dev(self.cache),
                                   out, self.scale, self.masks(), ws, self.max_q, window=self.window, lse=sums,
                                   page_size=self.page, **more)
        return out, sums

    def draw(self, mass, lse, **more):
        srg.lora_kv_attention_mass(self.q.cuda(), lse, ints(self.start), ints(self.lens), dev(self.table),
                                   dev(self.cache), mass, self.scale, self.masks(), self.max_q, window=self.window,
                                   page_size=self.page, **more)


def check(got, want, slack, name):
    got, fine = R.f64(got), np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), name
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), name
    excess = np.abs(got - np.where(fine, want, 0))[fine] - slack[fine]
    assert excess.size == 0 or excess.max() <= 0, (name, excess.max())


CASES = {
    "one draft": dict(lens=[40], queries=[1], hq=4, kv=2, d=64, page=16),
    "one token": dict(lens=[1], queries=[1], hq=2, kv=1, d=128, page=16),
    "tree of 26": dict(lens=[500], queries=[26], hq=4, kv=4, d=128, page=64),
    "ragged": dict(lens=[77, 5, 300, 0, 64, 130], queries=[13, 5, 1, 2, 7, 0], hq=12, kv=2, d=64, page=16),
    "shorter than their queries": dict(lens=[3, 9, 1], queries=[9, 9, 30], hq=8, kv=2, d=64, page=16),
    "any masks": dict(lens=[77, 5, 300, 64, 129], queries=[13, 8, 1, 33, 60], hq=6, kv=2, d=64, page=32, bits="any"),
    "any masks, wide": dict(lens=[180, 260], queries=[150, 101], hq=2, kv=2, d=64, page=16, bits="any", words=5),
    "many rows": dict(lens=[150, 200, 90], queries=[40, 33, 64], hq=16, kv=2, d=128, page=64),
    "many rows, 64": dict(lens=[150, 200], queries=[70, 33], hq=16, kv=2, d=64, page=128),
    "512 drafts": dict(lens=[530], queries=[512], hq=2, kv=2, d=64, page=256),
    "window": dict(lens=[77, 5, 300, 64], queries=[13, 5, 6, 7], hq=6, kv=2, d=64, page=16, window=20),
    "window of one": dict(lens=[77, 5, 300, 64], queries=[13, 5, 6, 7], hq=6, kv=2, d=128, page=16, window=1),
    "window inside the drafts": dict(lens=[130, 90], queries=[100, 80], hq=4, kv=2, d=64, page=16, bits="any", window=9),
    "window, many rows": dict(lens=[250, 300], queries=[70, 33], hq=16, kv=2, d=128, page=64, bits="any", window=50),
    "no masks": dict(lens=[77, 5, 300, 0, 64], queries=[13, 5, 1, 2, 7], hq=6, kv=2, d=64, page=16, bits=None),
    "no masks, window": dict(lens=[77, 5, 300, 64], queries=[13, 9, 1, 64], hq=6, kv=2, d=128, page=16, bits=None, window=11),
    "no masks, many rows": dict(lens=[250, 200], queries=[70, 133], hq=16, kv=2, d=128, page=64, bits=None),
    "long, in parts": dict(lens=[2500, 1700], queries=[20, 9], hq=4, kv=2, d=64, page=64),
    "long, one row, in parts": dict(lens=[4000], queries=[1], hq=2, kv=1, d=128, page=64, bits=None),
    "group of 3": dict(lens=[100, 133], queries=[11, 21], hq=9, kv=3, d=64, page=16),
    "group of 40": dict(lens=[100, 133], queries=[2, 5], hq=40, kv=1, d=64, page=16),
}


@pytest.mark.parametrize("name", CASES)
def test_tree_attention(name):
    s = Step(len(name), **CASES[name])
    out, lse = s.attend()
    want = s.want()
    check(lse, want["lse"], want["lse_slack"], "lse")
    check(out, want["out"], want["out_slack"], "out")
    again, _ = s.attend(lse=False)  # without the sums: the same outputs
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("name", CASES)
def test_attention_mass(name):
    s = Step(len(name) + 1, **CASES[name])
    lse = torch.from_numpy(s.want()["lse"]).float().cuda()
    want = s.want(lse_in=R.f64(lse))
    old = np.random.default_rng(1).random((s.pages, s.kv, s.page)) * 10
    old = old.astype(np.float32).astype(np.float64)
    # whatever the step's own places held does not count
    with_nan = np.where(want["fresh"][:, None, :], np.nan, old)
    mass = dev(with_nan, torch.float32)
    s.draw(mass, lse)
    after, slack = C.mass_after(with_nan, want)
    check(mass, after, slack, "mass")
    # and once more on top of it
    s.draw(mass, lse)
    after, more = C.mass_after(after, want)
    check(mass, after, slack + more, "mass twice")


def test_mass_adds_up_to_the_rows():
    s = Step(5, **CASES["many rows"])
    _, lse = s.attend()
    mass = torch.zeros(s.pages, s.kv, s.page, device="cuda")
    s.draw(mass, lse)
    # every row's weights add up to one; each is off by at most its lse's and its own score's error
    want = s.want()
    slack = 2 * want["lse_slack"].max() * s.T * s.hq
    assert abs(float(mass.double().sum()) - s.T * s.hq) <= slack


@pytest.mark.parametrize("masked", [True, False])
def test_nan_blocks_reach_only_the_rows_that_see_them(masked):
    """A draft's NaN key or value is seen by its descendants alone (or by the tokens behind it)."""
    s = Step(3, [40, 90], [9, 7], 8, 2, 64, 16, bits="tree" if masked else None)
    rows = [s.start[0] + 3, s.start[1] + 2]
    for seq, (row, part) in enumerate(zip(rows, (0, 1))):
        t = s.lens[seq] - s.queries[seq] + (row - s.start[seq])
        page, inside = s.table[seq, t // 16], t % 16
        s.cache[page, part, 0, 16 * 32 + inside] = 255  # the first block of head 0
        s.values[page, part, 0, inside, :32] = np.nan
    out, lse = s.attend()
    want = s.want()
    assert np.isnan(want["out"]).any() and np.isfinite(want["out"]).any()
    check(out, want["out"], want["out_slack"], "out")
    check(lse, want["lse"], want["lse_slack"], "lse")
    mass = torch.zeros(s.pages, s.kv, s.page, device="cuda")
    s.draw(mass, lse)
    want = s.want(lse_in=R.f64(lse))
    after, slack = C.mass_after(np.zeros((s.pages, s.kv, s.page)), want)
    # the NaN key's row sums are NaN, and so is all that those rows see
    check(mass, after, slack, "mass")


def test_bad_pages_and_rows_of_no_sequence():
    s = Step(8, [100, 70, 33], [6, 5, 4], 8, 2, 64, 16, extra_rows=3)
    s.table[0, 2], s.table[0, 6], s.table[1, 0], s.table[2, 1] = -1, s.pages, 2 ** 31 - 1, -2 ** 31
    out, lse = s.attend()
    want = s.want()
    check(out[:15], want["out"][:15], want["out_slack"][:15], "out")
    check(lse[:15], want["lse"][:15], want["lse_slack"][:15], "lse")
    assert out[15:].isnan().all() and lse[15:].isnan().all()
    mass = torch.full((s.pages, s.kv, s.page), 3.0, device="cuda")
    s.draw(mass, torch.where(lse.isnan(), 0.0, lse))
    after, slack = C.mass_after(np.full((s.pages, s.kv, s.page), 3.0), s.want(lse_in=R.f64(lse)))
    check(mass, after, slack, "mass")
    assert (after == 3).any()


def test_padded_batch():
    """Sequences without queries, with a start below 0 or past the tokens, and lengths past the
    table's; more queries than the call takes."""
    s = Step(9, [60, 50, 70, 80], [5, 6, 7, 8], 4, 2, 64, 16)
    s.start = [-1, 5, 5, 18, 900]
    s.lens = [60, 50, 70, 2 ** 31 - 1]
    most = s.table.shape[1] * 16
    s.max_q = 6
    for bits in (s.bits, None):
        s.bits = bits
        out, lse = s.attend()
        want = s.want(max_seq_len=most, max_query_len=6)
        written = ~np.isnan(want["lse"])
        assert written.any() and not written.all()
        check(out, want["out"], want["out_slack"], "out")
        check(lse, want["lse"], want["lse_slack"], "lse")
        mass = torch.ones(s.pages, s.kv, s.page, device="cuda")
        s.draw(mass, torch.where(lse.isnan(), 0.0, lse))
        after, slack = C.mass_after(np.ones((s.pages, s.kv, s.page)),
                                    s.want(max_seq_len=most, max_query_len=6, lse_in=R.f64(lse)))
        check(mass, after, slack, "mass")


@pytest.mark.parametrize("end", [2 ** 31 - 1, 2 ** 31 - 20, 2 ** 30 + 60, 2 ** 30, 1000])
@pytest.mark.parametrize("bits", ["tree", None])
def test_more_queries_than_tokens(end, bits):
    """A sequence whose rows go on past all: of a length far below, they see nothing."""
    s = Step(12, [60, 300], [5, 40], 4, 2, 64, 16, bits=bits)
    s.start, s.max_q = [0, 5, end], 40
    out, lse = s.attend()
    assert (out[5:] == 0).all() and (lse[5:] == -torch.inf).all()
    mass = torch.ones(s.pages, s.kv, s.page, device="cuda")
    s.draw(mass, torch.where(lse == -torch.inf, 1.0, lse))
    for t in range(300):
        assert (mass[s.table[1][t // 16], :, t % 16] == 0).all(), t


@pytest.mark.parametrize("d,lens,queries,hq,kv,window", [
    (128, [1536], [26], 32, 32, 0),                                # one row tile a workgroup, in parts
    (128, [3000], [26], 32, 32, 1400),                             # with a window, and room for longer walks
    (64, [2000, 1537, 40], [20, 26, 3], 16, 16, 1300),
    (64, [700] * 20 + [1500, 3, 0, 1100], [13] * 22 + [1, 4], 24, 4, 0),     # single tiles of 288 pairs
    (64, [700] * 20 + [2500, 3, 0, 1100], [13] * 22 + [1, 4], 24, 4, 1024),
])
@pytest.mark.parametrize("bits", ["tree", None])
def test_one_row_tile_a_workgroup(d, lens, queries, hq, kv, window, bits):
    s = Step(13, lens, queries, hq, kv, d, 64, bits=bits, window=window)
    out, lse = s.attend()
    want = s.want()
    check(out, want["out"], want["out_slack"], "out")
    check(lse, want["lse"], want["lse_slack"], "lse")


@pytest.mark.parametrize("lens,queries,last,most,words,hq,kv,d,window", [
    ([2000], [16], 1000, 16, 1, 1, 1, 64, 64),                       # tiles of 16 rows, one part
    ([3000, 2500], [300, 1], 512, 1, 8, 2, 2, 128, 100),             # 512 drafts, of which some count
    ([3000, 2500], [300, 130], 700, 13, 2, 4, 4, 64, 1300),          # several parts
    ([4500, 5500], [200, 20], 190, 20, 3, 4, 2, 128, 2500),          # tiles of 32 rows, several parts
    ([4500, 5500], [200, 20], 2 ** 31 - 1, 20, 3, 4, 2, 64, 2500),
    ([6000], [64], 5000, 64, 2, 8, 1, 128, 400),
    ([2100 + 7 * b for b in range(24)], [1] * 20 + [70, 3, 200, 2], 900, 32, 1, 16, 16, 64, 90),   # of 32, one part
    ([1500 + 7 * b for b in range(8)], [1, 2, 3, 70, 0, 1, 2, 2], 600, 32, 1, 256, 32, 64, 90),    # of 128
])
def test_more_queries_than_the_call_takes_in_a_window(lens, queries, last, most, words, hq, kv, d, window):
    """Drafts from max_query_len on have no rows, and are seen where masks have bits for them."""
    s = Step(14, lens, queries, hq, kv, d, 64, bits="any", words=words, window=window)
    s.start[-1], s.max_q = s.start[-2] + last if last < 2 ** 31 - 1 else last, most
    out, lse = s.attend()
    want = s.want(max_query_len=most)
    assert (~np.isnan(want["lse"])).any()
    check(lse, want["lse"], want["lse_slack"], "lse")
    check(out, want["out"], want["out_slack"], "out")
    mass = torch.ones(s.pages, s.kv, s.page, device="cuda")
    s.draw(mass, torch.where(lse.isnan(), 0.0, lse))
    after, slack = C.mass_after(np.ones(mass.shape), s.want(max_query_len=most, lse_in=R.f64(lse)))
    check(mass, after, slack, "mass")


def test_strides_and_scales():
    s = Step(10, [70, 90], [9, 12], 8, 2, 64, 16)
    out, lse = s.attend()
    q = torch.zeros(s.T, 11, 64, dtype=torch.bfloat16, device="cuda")[:, :8]
    q.copy_(s.q)
    outs = torch.full((s.T, 10, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    sums = torch.full((s.T, 13), 5.0, device="cuda")
    table = torch.full((2, 17), -1, dtype=torch.int32, device="cuda")
    table[:, :s.table.shape[1]] = dev(s.table)
    ws = srg.kv_tree_attention_workspace(2, s.max_q, s.table.shape[1] * 16, 8, 2, 64)
    args = (ints(s.start), ints(s.lens), table[:, :s.table.shape[1]], dev(s.cache))
    srg.lora_kv_tree_attention(q, *args, outs[:, :8], s.scale, s.masks(), ws, s.max_q, lse=sums[:, :8])
    assert torch.equal(outs[:, :8].view(torch.int16), out.view(torch.int16)) and torch.equal(sums[:, :8], lse)
    assert (outs[:, 8:] == 5).all() and (sums[:, 8:] == 5).all()
    masses = []
    for l in (sums[:, :8], lse):
        masses.append(torch.zeros(s.pages, 2, 16, device="cuda"))
        srg.lora_kv_attention_mass(q, l, *args, masses[-1], s.scale, s.masks(), s.max_q)
    assert torch.equal(*masses)
    # negative and zero scales
    for scale in (-0.3, 0.0):
        s.scale = scale
        out, lse = s.attend()
        want = s.want()
        check(out, want["out"], want["out_slack"], "out")
        check(lse, want["lse"], want["lse_slack"], "lse")
        mass = torch.zeros(s.pages, 2, 16, device="cuda")
        s.draw(mass, lse)
        after, slack = C.mass_after(np.zeros(mass.shape), s.want(lse_in=R.f64(lse)))
        check(mass, after, slack, "mass")


def test_rows_without_a_sum_count_for_nothing():
    s = Step(11, [70], [4], 4, 2, 64, 16)
    _, lse = s.attend()
    lse[1] = -torch.inf
    mass = torch.zeros(s.pages, s.kv, s.page, device="cuda")
    s.draw(mass, lse)
    after, slack = C.mass_after(np.zeros(mass.shape), s.want(lse_in=R.f64(lse)))
    check(mass, after, slack, "mass")


@pytest.mark.parametrize("kw", [
    dict(lens=[77, 300, 64], queries=[3, 4, 1], hq=8, kv=2, d=64, page=16),                   # one tile of rows
    dict(lens=[90, 300, 40], queries=[13, 21, 9], hq=8, kv=2, d=128, page=64),                # several
    dict(lens=[90, 300], queries=[13, 21], hq=8, kv=2, d=64, page=16, window=30),
    dict(lens=[150, 330, 90], queries=[40, 33, 64], hq=16, kv=2, d=128, page=64),             # many
    dict(lens=[250, 300], queries=[70, 45], hq=15, kv=3, d=64, page=64, window=100)])
@pytest.mark.parametrize("bits", ["tree", None])
@pytest.mark.parametrize("silent", [0.0, 0.3])
def test_rows_without_a_sum_count_for_nothing_whatever_they_hold(kw, bits, silent):
    """Rejected drafts, whose sums a program sets to -infinity: NaN and infinities of their
    queries, and of keys that only they see, reach no weight."""
    s = Step(15, bits=bits, **kw)
    lse = s.want()["lse"].copy()
    rng = np.random.default_rng(4)
    out = rng.random((s.T, s.hq)) < silent
    out[:s.start[1]] = True  # all of the first sequence's
    out[np.array(s.start[1:]) - 1] = True  # and the last of each, which alone sees the last token
    lse[out] = -np.inf
    q = s.q.float().numpy()
    q[out] = rng.choice([np.nan, np.inf, -np.inf], (int(out.sum()), s.d))
    s.q = R.bf16(q)
    for b, length in enumerate(s.lens):
        page, inside = s.table[b, (length - 1) // s.page], (length - 1) % s.page
        s.cache[page, 0, :, s.page * (s.d // 2) + inside] = 255
        s.values[page, 0, :, inside, :32] = np.nan
    lse = torch.from_numpy(lse).float().cuda()
    mass = torch.ones(s.pages, s.kv, s.page, device="cuda")
    s.draw(mass, lse)
    after, slack = C.mass_after(np.ones(mass.shape), s.want(lse_in=R.f64(lse)))
    assert np.isfinite(after).all()
    check(mass, after, slack, "mass")


@pytest.mark.parametrize("hq,d", [(2, 64), (8, 128), (16, 128), (16, 64)])
@pytest.mark.parametrize("bits", ["tree", None])
def test_nan_sums_beside_rows_without_a_sum(hq, d, bits):
    """A NaN key reaches what the rows that see it, and count, see; not the others' tokens."""
    s = Step(16, [150, 330], [40, 33], hq, 2, d, 64, bits=bits)
    t = s.lens[0] - s.queries[0] + 20
    page, inside = s.table[0, t // 64], t % 64
    s.cache[page, 0, 0, 64 * (d // 2) + inside] = 255
    s.values[page, 0, 0, inside, :32] = np.nan
    _, lse = s.attend()
    rows = np.flatnonzero(lse.isnan().any(1).cpu().numpy())
    assert len(rows)
    for quiet in ([], [int(rows[0])], rows.tolist()):
        sums = lse.clone()
        sums[quiet] = -torch.inf
        mass = torch.ones(s.pages, s.kv, s.page, device="cuda")
        s.draw(mass, sums)
        after, slack = C.mass_after(np.ones(mass.shape), s.want(lse_in=R.f64(sums)))
        assert np.isnan(after).any() == (len(quiet) < len(rows))
        check(mass, after, slack, "mass")


# ------------------------------------------------------------------ select
def selected(mass, lens, table, sinks, recent, budget, **more):
    kept = torch.full((len(lens), mass.shape[1], budget), -9, dtype=torch.int32, device="cuda")
    new = torch.full((len(lens),), -9, dtype=torch.int32, device="cuda")
    srg.lora_kv_select(dev(mass, torch.float32), ints(lens), dev(table), sinks, recent, kept, new, **more)
    return kept.cpu().numpy(), new.cpu().tolist()


def check_selected(mass, lens, table, sinks, recent, budget, most=None, **more):
    pages, kv, page = mass.shape
    kept, new = selected(mass, lens, table, sinks, recent, budget, **more)
    for s, length in enumerate(lens):
        n = max(0, min(length, most or length))
        ids = table[s][np.arange(n) // page]
        there = (ids >= 0) & (ids < pages)
        for h in range(kv):
            w = np.where(there, mass[np.where(there, ids, 0), h, np.arange(n) % page].astype(np.float32), -np.inf)
            want = C.select(w.tolist(), n, sinks, recent, budget)
            assert kept[s, h].tolist() == want + [-1] * (budget - len(want)), (s, h)
        assert new[s] == min(n, budget)


def paged(rng, lens, kv, page, weights):
    need = [-(-n // page) for n in lens]
    table = np.full((len(lens), max(1, max(need))), -1, dtype=np.int32)
    order, at = rng.permutation(sum(need) + 1), 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return weights((sum(need) + 1, kv, page)), table


@pytest.mark.parametrize("lens,kv,page,sinks,recent,budget", [
    ([1, 2, 0, 3], 1, 16, 0, 0, 1), ([40, 17, 33, 5], 2, 16, 2, 5, 17), ([40, 17, 33], 2, 32, 0, 17, 17),
    ([40, 17, 33], 2, 16, 17, 0, 17), ([40, 18], 1, 16, 0, 0, 17), ([4095, 4096, 4097, 8193], 2, 64, 4, 100, 1000),
    ([9000, 100], 3, 256, 1, 4000, 5001), ([20000], 2, 128, 0, 1, 19999), ([70001], 1, 64, 4, 512, 30000),
    # more long lists than are cut into pieces
    ([70001, 50, 40000, 32769] + [10, 0, 30001] * 10, 1, 64, 4, 512, 30000)])
@pytest.mark.parametrize("kind", ["spread", "ties", "special"])
def test_select(lens, kv, page, sinks, recent, budget, kind):
    rng = np.random.default_rng(sum(lens))
    make = {"spread": lambda shape: np.exp(3 * rng.standard_normal(shape)),
            "ties": lambda shape: rng.integers(0, 3, shape).astype(float),
            "special": lambda shape: rng.choice(
                [np.nan, np.inf, -np.inf, 0.0, -0.0, 1.0, -1.0, 1e-45, -1e-45, 3e38], shape)}[kind]
    mass, table = paged(rng, lens, kv, page, make)
    check_selected(mass, lens, table, sinks, recent, budget)


@pytest.mark.parametrize("lens,kv,page,sinks,recent,budget", [
    ([24577], 1, 64, 0, 0, 1), ([32768], 2, 16, 0, 0, 32767), ([32769, 100, 8192, 8193], 2, 64, 9000, 9000, 20000),
    ([0, 40000, 16385], 3, 32, 4, 512, 16384), ([131072], 1, 256, 0, 70000, 70001), ([131072], 2, 64, 20000, 0, 20000),
    ([30000], 1, 64, 4, 4, 60000), ([131071], 8, 64, 4, 512, 65536)])
@pytest.mark.parametrize("kind", ["spread", "ties", "special", "one digit", "equal"])
def test_select_in_pieces(lens, kv, page, sinks, recent, budget, kind):
    rng = np.random.default_rng(sum(lens))
    make = {"spread": lambda shape: np.exp(3 * rng.standard_normal(shape)),
            "ties": lambda shape: rng.integers(0, 3, shape).astype(float),
            "special": lambda shape: rng.choice(
                [np.nan, np.inf, -np.inf, 0.0, -0.0, 1.0, -1.0, 1e-45, -1e-45, 3e38], shape),
            "one digit": lambda shape: 1 + 2.0 ** -23 * rng.integers(0, 5000, shape),
            "equal": lambda shape: np.full(shape, 0.5)}[kind]
    mass, table = paged(rng, lens, kv, page, make)
    most = table.shape[1] * page
    assert srg.lora_kv_select_workspace_bytes(len(lens), kv, most) > 0
    check_selected(mass, lens, table, sinks, recent, budget)
    ws = srg.kv_select_workspace(len(lens), kv, most).random_()  # whatever it held
    check_selected(mass, lens, table, sinks, recent, budget, workspace=ws)


def test_select_in_as_many_pieces_as_there_are():
    rng = np.random.default_rng(128)
    mass, table = paged(rng, [128 * 8192 - 5], 1, 256, lambda shape: rng.standard_normal(shape))
    assert srg.lora_kv_select_workspace_bytes(1, 1, table.shape[1] * 256) > 0
    check_selected(mass, [128 * 8192 - 5], table, 5, 300, 600000)
    # one more page of the table, and the list is left whole
    table = np.concatenate([table, np.full((1, 1), -1, dtype=np.int32)], axis=1)
    assert srg.lora_kv_select_workspace_bytes(1, 1, table.shape[1] * 256) == 0
    check_selected(mass, [128 * 8192 + 100], table, 5, 300, 600000)


def test_select_of_neighbours_in_every_bit():
    """Weights that differ in one bit, at every place of the number."""
    rng = np.random.default_rng(2)
    bits = np.concatenate([np.uint32(0x3F800000) ^ (np.uint32(1) << np.arange(31, dtype=np.uint32)),
                           rng.integers(0, 0x7F800000, 193, dtype=np.uint32)])
    mass, table = paged(rng, [224], 1, 16, lambda shape: rng.permutation(
        np.resize(bits, np.prod(shape))).view(np.float32).reshape(shape).astype(float))
    for budget in (1, 2, 100, 223):
        check_selected(mass, [224], table, 0, 0, budget)


def test_select_with_bad_pages_and_a_length_past_the_most():
    rng = np.random.default_rng(3)
    mass, table = paged(rng, [100, 64, 90], 2, 16, lambda shape: rng.standard_normal(shape))
    table[0, 1], table[2, 0], table[2, 5] = -1, mass.shape[0], 2 ** 31 - 1
    check_selected(mass, [100, -3, 90], table, 3, 4, 40)
    check_selected(mass, [100, 2 ** 31 - 1, 90], table, 3, 4, 40, most=64, max_seq_len=64)
    mass, table = paged(rng, [50000, 16], 2, 16, lambda shape: rng.standard_normal(shape))
    table[0, 1:3000:7], table[0, 40], table[0, 41] = -1, mass.shape[0], 2 ** 31 - 1
    check_selected(mass, [50000, -3], table, 3, 4, 30000)
    check_selected(mass, [2 ** 31 - 1, 0], table, 3, 4, 30000, most=40000, max_seq_len=40000)


# ------------------------------------------------------------------ compact
class Moves:
    def __init__(self, seed, seqs, lists, n, kv, d, page, span, first=None, new_pages=False, counts=None):
        rng = np.random.default_rng(seed)
        self.d, self.page = d, page
        need = -(-span // page)
        more = -(-(n + (max(first) if first else 0)) // page) if new_pages else 0
        self.pages = seqs * (need + more) + 2
        order = rng.permutation(self.pages).astype(np.int32)
        self.table = order[:seqs * need].reshape(seqs, need)
        self.dst = order[seqs * need:seqs * (need + more)].reshape(seqs, more) if new_pages else None
        self.first = first
        base = np.array(first if first else [0] * seqs)
        self.kept = np.stack([np.stack([np.sort(rng.permutation(span - b)[:n]) for _ in range(lists)]) for b in base])
        self.kept = self.kept.astype(np.int32)
        self.counts = counts if counts is not None else [n] * seqs
        self.cache = rng.integers(0, 256, (self.pages, 2, kv, page * (d // 2 + d // 32)), dtype=np.uint8)
        self.mass = rng.random((self.pages, kv, page)).astype(np.float32)

    def check(self, mass=True):
        cache, weights = dev(self.cache), dev(self.mass)
        srg.lora_kv_compact(dev(self.kept), ints(self.counts), dev(self.table), cache, self.d,
                            mass=weights if mass else None, first=None if self.first is None else ints(self.first),
                            dst_table=None if self.dst is None else dev(self.dst), page_size=self.page)
        places, want = C.compact(C.by_place(self.cache, self.d, self.page), self.mass, self.kept, self.counts,
                                 self.first, self.table, self.dst)
        assert np.array_equal(C.by_place(cache.cpu().numpy(), self.d, self.page), places)
        assert np.array_equal(weights.cpu().numpy(), want if mass else self.mass)


@pytest.mark.parametrize("new_pages", [False, True])
@pytest.mark.parametrize("kw", [
    dict(seqs=1, lists=1, n=1, kv=1, d=64, page=16, span=1), dict(seqs=3, lists=2, n=20, kv=2, d=64, page=16, span=90),
    dict(seqs=2, lists=1, n=33, kv=3, d=128, page=32, span=70), dict(seqs=2, lists=2, n=300, kv=2, d=128, page=64, span=310),
    dict(seqs=1, lists=2, n=2000, kv=2, d=128, page=64, span=3500), dict(seqs=1, lists=1, n=3000, kv=1, d=64, page=256, span=3001),
    dict(seqs=3, lists=4, n=7, kv=4, d=128, page=16, span=60, first=[0, 11, 30]),
    dict(seqs=3, lists=1, n=5, kv=4, d=64, page=128, span=300, first=[127, 128, 130], counts=[5, 0, 3]),
    dict(seqs=4, lists=2, n=50, kv=2, d=64, page=16, span=100, counts=[-1, 2 ** 31 - 1, 17, 0])])
def test_compact(kw, new_pages):
    Moves(1, new_pages=new_pages, **kw).check()


def test_compact_without_mass():
    Moves(2, 2, 2, 40, 2, 128, 16, 90).check(mass=False)


def spoil(m):
    """Pages and starts that are not there."""
    m.table[1, 1], m.table[1, m.table.shape[1] // 2] = -1, m.pages
    m.first[3] = -5
    if m.dst is not None:
        m.dst[2, -3] = m.pages


@pytest.mark.parametrize("seed", range(4))
def test_compact_of_any_list_into_new_pages(seed):
    """Numbers out of order, twice, behind; entries that are skipped."""
    m = Moves(seed, 4, 2, 60, 2, 128 if seed % 2 else 64, 16, 3000, first=[0, 3, 2900, 5], new_pages=True)
    rng = np.random.default_rng(seed)
    m.kept = rng.integers(0, 2900, m.kept.shape).astype(np.int32)
    m.kept[rng.random(m.kept.shape) < 0.1] = -1
    m.kept[rng.random(m.kept.shape) < 0.05] = 2 ** 31 - 1
    spoil(m)
    m.check()


@pytest.mark.parametrize("n", [60, 5000])
@pytest.mark.parametrize("seed", range(2))
def test_compact_in_place_skips_what_is_not_there(seed, n):
    """Ascending lists with entries below 0 behind and numbers far past the table's places."""
    m = Moves(seed, 4, 2, n, 2, 128 if seed % 2 else 64, 16, 3 * n, first=[0, 3, 2 * n - 100, 5])
    rng = np.random.default_rng(seed)
    m.kept = np.sort(np.stack([[rng.permutation(4 * n)[:n] for _ in range(2)] for _ in range(4)]), axis=-1).astype(np.int32)
    m.kept[1, 0, -7:] = -1
    m.kept[2, 1, -1] = 2 ** 31 - 1
    spoil(m)
    m.check()


def runs(*parts):
    """Ascending numbers: of (length, kept of each so many) parts one behind another."""
    out, at = [], 0
    for length, one_of in parts:
        out += range(at, at + length, one_of)
        at += length
    return np.array(out, dtype=np.int32)


@pytest.mark.parametrize("parts", [
    [(11000, 1)],                                  # all stay
    [(1, 1), (5000, 5000), (6000, 1)],             # 5000 out at once, then all behind come far
    [(3000, 1), (1500, 1500), (7000, 1)],          # the far ones start inside a block
    [(1024, 1), (3000, 2), (9000, 2)], [(4000, 4), (30000, 6)], [(2048, 1), (1024, 1024), (6000, 1), (100, 100), (500, 1)],
    [(6000, 1), (40, 40), (2000, 1)],              # never far
    [(1023, 1), (1100, 1100), (4200, 1)], [(200000, 40)],
])
@pytest.mark.parametrize("d,lists", [(64, 1), (128, 2)])
def test_compact_of_long_lists_in_place(parts, d, lists):
    kept = runs(*parts)
    n = len(kept)
    assert n > 4096
    m = Moves(n, 2, lists, n, 2, d, 64, int(kept[-1]) + 3, first=[0, 2])
    m.kept[:] = kept
    rng = np.random.default_rng(n)
    if lists == 2:  # another list for the other head: random gaps
        m.kept[:, 1] = np.sort(rng.permutation(max(int(kept[-1]), n + 1))[:n])
    m.counts = [n, n - 333]
    m.check()


@pytest.mark.parametrize("d,n,tail", [(64, 9000, 3000), (128, 9000, 8900), (64, 20000, 64), (64, 20000, 9999), (64, 4097, 1)])
def test_compact_of_long_lists_in_place_with_entries_below_0_behind(d, n, tail):
    m = Moves(n, 2, 2, n, 2, d, 64, 2 * n + 5, first=[0, 3])
    rng = np.random.default_rng(n)
    for s in range(2):
        for h in range(2):
            m.kept[s, h] = np.sort(rng.permutation(2 * n)[:n])
            m.kept[s, h, n - tail:] = rng.choice([-1, -7, -2 ** 31], tail)
    m.counts = [n, n]
    m.check()


def test_compact_of_a_long_list_with_one_token_out():
    m = Moves(4, 1, 1, 5000, 1, 64, 64, 5001)
    m.kept[:] = np.delete(np.arange(5001), 77)
    m.check()


# ------------------------------------------------------------------ as they are used
def test_a_step_with_drafts_and_an_eviction():
    """Masks and positions, append, attention and mass for trees; the accepted path to its
    places; the heaviest tokens to the front; the next step over what is left."""
    B, hq, kv, d, page, n = 3, 8, 2, 64, 16, 12
    rng = np.random.default_rng(0)
    lens = [70, 41, 90]
    s = Step(1, [x + n for x in lens], [n] * B, hq, kv, d, page, bits="tree")
    parents = [p for _ in range(B) for p in C.random_tree(rng, n)]
    bits = [path for b in range(B) for path in C.ancestors(parents[n * b:n * b + n])]
    T = n * B
    masks = torch.zeros(T, 1, dtype=torch.int64, device="cuda")
    positions = torch.zeros(T, dtype=torch.int32, device="cuda")
    srg.lora_draft_masks(ints(parents), ints(s.start), masks, positions, ints(lens))
    qkv = R.bf16(rng.standard_normal((T, (hq + 2 * kv) * d))).cuda()
    rope = srg.rope_table(256, d)
    cache, q = dev(s.cache), torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")
    places = [int(s.table[b, t // page]) * page + t % page for b in range(B) for t in range(lens[b], lens[b] + n)]
    slots = torch.tensor(places, device="cuda")
    srg.lora_kv_append(qkv, positions, slots, rope, cache, q, page_size=page)
    k, v = (torch.empty(T, kv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    srg.lora_kv_read(slots, cache, k, v, page_size=page)
    heads = R.f64(qkv).reshape(T, -1, d)
    depth = [len(p) - 1 for p in bits]
    turned = R.rotate(heads, R.f64(rope), [lens[i // n] + depth[i] for i in range(T)], False)
    assert np.array_equal(R.f64(k), R.held(turned[:, hq:hq + kv].astype(np.float32).astype(np.float64)))
    for i, place in enumerate(places):
        s.values[place // page, :, :, place % page] = np.stack([R.f64(k)[i], R.f64(v)[i]])
    s.cache, s.q, s.bits, s.max_q, s.words = cache.cpu().numpy(), q.cpu(), bits, n, 1
    out, lse = s.attend()
    want = s.want()
    check(out, want["out"], want["out_slack"], "out")
    old = rng.random((s.pages, kv, page)).astype(np.float32)
    mass = dev(old)
    s.draw(mass, lse)
    after, slack = C.mass_after(old.astype(np.float64), s.want(lse_in=R.f64(lse)))
    check(mass, after, slack, "mass")

    # each sequence accepts the longest path of its tree
    paths = [sorted(max(bits[n * b:n * b + n], key=len)) for b in range(B)]
    accepted = np.zeros((B, 1, n), dtype=np.int32)
    for b, path in enumerate(paths):
        accepted[b, 0, :len(path)] = path
    srg.lora_kv_compact(dev(accepted), ints([len(p) for p in paths]), dev(s.table), cache, d, mass=mass,
                        first=ints(lens), page_size=page)
    now = [x + len(p) for x, p in zip(lens, paths)]
    held = [list(range(x)) + [x + j for j in p] for x, p in zip(lens, paths)]  # by their places before

    # each key head keeps 50 tokens
    budget = 50
    kept = torch.zeros(B, kv, budget, dtype=torch.int32, device="cuda")
    new_lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    srg.lora_kv_select(mass, ints(now), dev(s.table), 2, 8, kept, new_lens)
    srg.lora_kv_compact(kept, new_lens, dev(s.table), cache, d, mass=mass, page_size=page)
    assert new_lens.cpu().tolist() == [min(x, budget) for x in now]

    # one more query a sequence over what is left
    s2 = Step(2, [min(x, budget) for x in now], [1] * B, hq, kv, d, page, bits=None)
    s2.table, s2.cache, s2.pages = s.table, cache.cpu().numpy(), s.pages
    out, _ = s2.attend()
    q2 = R.f64(s2.q)
    for b in range(B):
        for h in range(kv):
            mine = [held[b][t] for t in kept[b, h].cpu().tolist() if t >= 0]
            assert len(mine) == min(now[b], budget)
            ids = s.table[b][np.array(mine) // page]
            keys, values = (s.values[ids, part, h, np.array(mine) % page] for part in (0, 1))
            for i in range(hq // kv):
                row = h * (hq // kv) + i
                score = s2.scale * (keys @ q2[b, row])
                p = np.exp(score - score.max())
                p /= p.sum()
                size = s2.scale * np.abs(q2[b, row]).max() * np.abs(keys).sum(1).max()
                slack = R.attention_slack(p @ values, p @ np.abs(values), size, d, len(mine), np.abs(score).max())
                assert (np.abs(R.f64(out)[b, row] - p @ values) <= slack).all()
