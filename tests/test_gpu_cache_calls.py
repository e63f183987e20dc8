"""Drafted tokens and caches of bounded length as programs call them: captured and
replayed, on other streams, twice, with many rows, with caches past 4 GiB, and what the
binding refuses."""

import numpy as np
import pytest
import torch

import segmented_rank_gemm_amd as srg
from segmented_rank_gemm_amd import cache as binding
from tests import attention_reference as R
from tests import cache_reference as C
from tests.test_gpu_cache import CASES, Step, check, dev, ints

pytestmark = pytest.mark.gpu


class Buffers:
    """The static tensors of a step with drafts and an eviction."""

    def __init__(self, B=3, n=12, hq=8, kv=2, d=64, page=16, per_seq=16, budget=100):
        self.B, self.n, self.T, self.d, self.page, self.budget = B, n, B * n, d, page, budget
        self.g = torch.Generator(device="cuda").manual_seed(1)
        new = lambda *shape, dtype=torch.int32: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
        self.table = torch.randperm(B * per_seq, device="cuda", generator=self.g).int().view(B, per_seq)
        self.fresh_pages = (torch.arange(B * 8, device="cuda").int() + B * per_seq).view(B, 8)
        pages = B * per_seq + B * 8
        self.start = ints([n * b for b in range(B + 1)])
        self.parents, self.positions, self.text, self.lens = new(self.T), new(self.T), new(B), new(B)
        self.masks = new(self.T, 1, dtype=torch.int64)
        self.q = new(self.T, hq, d, dtype=torch.bfloat16)
        self.out, self.lse = new(self.T, hq, d, dtype=torch.bfloat16), new(self.T, hq, dtype=torch.float32)
        self.cache = dev(R.random_cache(np.random.default_rng(2), pages, kv, d, page)[0])
        self.mass = new(*srg.kv_mass_shape(pages, kv, page), dtype=torch.float32)
        self.accepted, self.counts = new(B, 1, 4), new(B)
        self.kept, self.new_lens = new(B, kv, budget), new(B)
        self.ws = srg.kv_tree_attention_workspace(B, n, per_seq * page, hq, kv, d)

    def draw(self, seed):
        g = self.g.manual_seed(seed)
        at = torch.arange(self.T, device="cuda") % self.n
        self.parents.copy_((torch.rand(self.T, device="cuda", generator=g) * at).floor() - (at == 0).int())
        self.text.copy_(torch.randint(0, self.table.shape[1] * self.page - self.n, (self.B,), device="cuda", generator=g))
        self.lens.copy_(self.text + self.n)
        self.q.normal_(generator=g)
        self.mass.exponential_(generator=g)
        for b in range(self.B):
            self.accepted[b, 0, :] = torch.randperm(self.n, device="cuda", generator=g)[:4].sort().values.int()
        self.counts.copy_(torch.randint(0, 5, (self.B,), device="cuda", generator=g))

    def step(self, **more):
        srg.lora_draft_masks(self.parents, self.start, self.masks, self.positions, self.text, **more)
        srg.lora_kv_tree_attention(self.q, self.start, self.lens, self.table, self.cache, self.out, 0.125, self.masks,
                                   self.ws, self.n, lse=self.lse, **more)
        srg.lora_kv_attention_mass(self.q, self.lse, self.start, self.lens, self.table, self.cache, self.mass, 0.125,
                                   self.masks, self.n, **more)
        srg.lora_kv_compact(self.accepted, self.counts, self.table, self.cache, self.d, mass=self.mass, first=self.text, **more)
        srg.lora_kv_select(self.mass, self.lens, self.table, 2, 10, self.kept, self.new_lens, **more)
        srg.lora_kv_compact(self.kept, self.new_lens, self.table, self.cache, self.d, mass=self.mass,
                            dst_table=self.fresh_pages, **more)
        srg.lora_kv_compact(self.kept, self.new_lens, self.table, self.cache, self.d, mass=self.mass, **more)

    def state(self):
        return [t.clone() for t in (self.masks, self.positions, self.out, self.lse, self.mass, self.kept, self.new_lens,
                                    self.cache)]


def test_a_step_captured_and_replayed():
    s = Buffers()
    s.draw(0)
    s.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step()
    for seed in range(1, 6):
        cache = s.cache.clone()
        s.draw(seed)
        graph.replay()
        torch.cuda.synchronize()
        got = s.state()
        s.cache.copy_(cache)
        s.draw(seed)
        s.step()
        torch.cuda.synchronize()
        for a, b in zip(got, s.state()):
            assert torch.equal(a, b), seed


def test_a_long_choice_captured_on_streams_and_with_a_workspace():
    """A list in pieces, with a workspace of its own, the caller's, and a graph's; two at
    once on two streams."""
    kv, page, n = 4, 64, 60000
    pages = -(-n // page)
    table = torch.randperm(pages, device="cuda").int()[None]
    mass, other = (torch.zeros(srg.kv_mass_shape(pages, kv, page), device="cuda").exponential_() for _ in range(2))
    lens, new = ints([n]), torch.zeros(1, dtype=torch.int32, device="cuda")
    kept = lambda: torch.zeros(1, kv, 20000, dtype=torch.int32, device="cuda")  # noqa: E731
    assert srg.lora_kv_select_workspace_bytes(1, kv, pages * page) > 0

    def want(mass, length):
        by_head = mass[table[0].long()].transpose(0, 1).reshape(kv, -1)[:, :length].cpu().numpy()
        return [C.select(by_head[h].tolist(), length, 4, 100, 20000) for h in range(kv)]

    captured, graph = kept(), torch.cuda.CUDAGraph()
    srg.lora_kv_select(mass, lens, table, 4, 100, captured, new)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        srg.lora_kv_select(mass, lens, table, 4, 100, captured, new)
    for length in (n, 50001, 41000):
        lens.fill_(length)
        mass.exponential_()
        graph.replay()
        eager = kept()
        srg.lora_kv_select(mass, lens, table, 4, 100, eager, new, workspace=srg.kv_select_workspace(1, kv, pages * page))
        assert captured[0].tolist() == want(mass, length) and torch.equal(captured, eager)
    streams, lists = [torch.cuda.Stream() for _ in range(2)], [kept(), kept()]
    news = [torch.zeros_like(new), torch.zeros_like(new)]
    torch.cuda.synchronize()
    for _ in range(4):
        for stream, m, k, count in zip(streams, (mass, other), lists, news):
            srg.lora_kv_select(m, lens, table, 4, 100, k, count, stream=stream)
    torch.cuda.synchronize()
    for m, k in zip((mass, other), lists):
        assert k[0].tolist() == want(m, 41000)
    with pytest.raises(srg.LoraError):
        srg.lora_kv_select(mass, lens, table, 4, 100, captured, new, workspace=torch.empty(1000, dtype=torch.uint8, device="cuda"))


def test_on_another_stream():
    s = Buffers()
    cache, side = s.cache.clone(), torch.cuda.Stream()
    s.draw(3)
    s.step()
    want = s.state()
    s.cache.copy_(cache)
    s.draw(3)
    for tensor in (s.masks, s.positions, s.out, s.lse, s.kept, s.new_lens):
        tensor.zero_()
    side.wait_stream(torch.cuda.current_stream())
    s.step(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, s.state()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["ragged", "many rows", "long, in parts", "no masks, many rows", "512 drafts"])
def test_the_same_call_gives_the_same_bits(name):
    s = Step(3, **CASES[name])
    (out, lse), (again, lse2) = s.attend(), s.attend()
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)
    masses = [torch.zeros(s.pages, s.kv, s.page, device="cuda") for _ in range(2)]
    for m in masses:
        s.draw(m, lse)
    assert torch.equal(*masses)


@pytest.mark.parametrize("kw", [
    dict(lens=[70, 33, 50, 64, 40, 45, 60, 35], queries=[32, 31, 30, 32, 17, 20, 32, 5], hq=256, kv=32, d=64, page=16),
    dict(lens=[90, 33, 50, 64, 40, 45, 60, 35], queries=[32, 31, 30, 32, 17, 20, 32, 5], hq=256, kv=32, d=128, page=16,
         bits="any", window=25),
    dict(lens=[70, 33, 50, 64, 40, 45, 60, 35], queries=[32, 31, 30, 32, 17, 20, 32, 5], hq=256, kv=32, d=128, page=64,
         bits=None)])
def test_rows_that_fill_the_device(kw):
    """Enough tiles of 128 rows for the kernel of pieces of prompts."""
    s = Step(6, **kw)
    out, lse = s.attend()
    want = s.want()
    check(lse, want["lse"], want["lse_slack"], "lse")
    check(out, want["out"], want["out_slack"], "out")
    mass = torch.zeros(s.pages, s.kv, s.page, device="cuda")
    s.draw(mass, lse)
    after, slack = C.mass_after(np.zeros(mass.shape), s.want(lse_in=R.f64(lse)))
    check(mass, after, slack, "mass")


def test_sums_beside_plain_attention():
    """Without masks the outputs are lora_kv_attention's, within the bounds of both."""
    s = Step(7, **CASES["no masks, window"])
    out, _ = s.attend()
    plain = torch.zeros_like(out)
    ws = srg.kv_attention_workspace(len(s.lens), s.max_q, s.table.shape[1] * s.page, s.hq, s.kv, s.d)
    srg.lora_kv_attention(s.q.cuda(), ints(s.start), ints(s.lens), dev(s.table), dev(s.cache), plain, s.scale, ws, s.max_q,
                          window=s.window)
    want = s.want()
    check(plain, want["out"], want["out_slack"], "plain")
    check(out, want["out"], want["out_slack"], "with sums")


def test_caches_past_4_gib():
    """Places whose bytes lie past 32-bit offsets: attention and mass read there, moves go there."""
    kv, d, page, pages = 32, 128, 256, 4400  # 1.1 MB a page
    cache = torch.empty(srg.kv_cache_shape(pages, kv, d, page), dtype=torch.uint8, device="cuda")
    assert cache.numel() > 1 << 32
    s = Step(8, [300, 40], [5, 3], kv, kv, d, page, spare=0)
    far = torch.arange(pages - s.pages, pages, device="cuda")
    cache[far] = dev(s.cache)
    out, lse = torch.zeros(s.T, kv, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(s.T, kv, device="cuda")
    table = dev(np.where(s.table >= 0, s.table + pages - s.pages, -1).astype(np.int32))
    mass = torch.zeros(srg.kv_mass_shape(pages, kv, page), device="cuda")
    ws = srg.kv_tree_attention_workspace(2, 5, table.shape[1] * page, kv, kv, d)
    args = (ints(s.start), ints(s.lens), table, cache)
    srg.lora_kv_tree_attention(s.q.cuda(), *args, out, s.scale, s.masks(), ws, 5, lse=lse)
    want = s.want()
    check(out, want["out"], want["out_slack"], "out")
    srg.lora_kv_attention_mass(s.q.cuda(), lse, *args, mass, s.scale, s.masks(), 5)
    after, slack = C.mass_after(np.zeros((s.pages, kv, page)), s.want(lse_in=R.f64(lse)))
    check(mass[far], after, slack, "mass")
    assert float(mass[:pages - s.pages].abs().sum()) == 0
    # the first sequence's places 40.. to the second page of the table and back to the front
    kept = dev(np.arange(40, 300, dtype=np.int32)[None, None])
    before = C.by_place(cache[far].cpu().numpy(), d, page)
    held = mass[far].cpu().numpy()
    srg.lora_kv_compact(kept, ints([260]), table[:1], cache, d, mass=mass, page_size=page)
    places, weights = C.compact(before, held, kept.cpu().numpy(), [260], None, s.table[:1], None)
    assert np.array_equal(C.by_place(cache[far].cpu().numpy(), d, page), places)
    assert np.array_equal(mass[far].cpu().numpy(), weights)


def test_masses_past_4_gib():
    kv, page, pages = 32, 256, 131072 + 40
    mass = torch.empty(srg.kv_mass_shape(pages, kv, page), device="cuda")
    assert mass.numel() * 4 > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(0)
    mass[-40:] = torch.rand(40, kv, page, generator=g, device="cuda")
    table = torch.arange(pages - 40, pages, device="cuda").int()[None]
    kept, new = torch.zeros(1, kv, 3000, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    srg.lora_kv_select(mass, ints([10000]), table, 3, 50, kept, new)
    weights = mass[-40:].transpose(0, 1).reshape(kv, -1)[:, :10000].cpu().numpy()
    for h in range(0, kv, 7):
        assert kept[0, h].tolist() == C.select(weights[h].tolist(), 10000, 3, 50, 3000), h


def test_the_binding_refuses(monkeypatch):
    s = Buffers()
    s.draw(0)
    i32, i64 = torch.int32, torch.int64
    new = lambda *shape, dtype=i32: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731

    def refused(error, call, *args, **kw):
        with pytest.raises(error):
            call(*args, **kw)

    refused(TypeError, srg.lora_draft_masks, s.parents.long(), s.start, s.masks)
    refused(ValueError, srg.lora_draft_masks, s.parents, s.start, s.masks[:-1])
    refused(TypeError, srg.lora_draft_masks, s.parents, s.start, s.masks.int())
    refused(ValueError, srg.lora_draft_masks, s.parents, s.start, new(s.T, 4, dtype=i64)[:, ::2])
    refused(srg.LoraError, srg.lora_draft_masks, s.parents, s.start, new(s.T, 9, dtype=i64))
    refused(srg.LoraError, srg.lora_draft_masks, s.parents, s.start)
    refused(ValueError, srg.lora_draft_masks, s.parents, s.start, s.masks, s.positions, new(s.B + 1))
    tree = dict(q=s.q, query_start=s.start, seq_lens=s.lens, page_table=s.table, cache=s.cache, out=s.out, scale=0.125,
                masks=s.masks, workspace=s.ws, max_query_len=s.n, lse=s.lse)
    for change, error in ((dict(masks=s.masks.int()), TypeError), (dict(masks=s.masks[1:]), ValueError),
                          (dict(lse=s.lse.double()), TypeError), (dict(lse=s.lse[:, 1:]), ValueError),
                          (dict(lse=s.lse.t().contiguous().t()), ValueError), (dict(max_query_len=65), srg.LoraError),
                          (dict(max_query_len=1 << 33), ValueError), (dict(max_seq_len=10000), ValueError),
                          (dict(scale=float("nan")), srg.LoraError), (dict(window=-1), srg.LoraError),
                          (dict(out=s.out[:, 1:]), ValueError), (dict(page_size=32), ValueError),
                          (dict(q=s.q.cpu()), TypeError), (dict(query_start=s.start[1:]), ValueError)):
        refused(error, srg.lora_kv_tree_attention, **{**tree, **change})
    mass = dict(q=s.q, lse=s.lse, query_start=s.start, seq_lens=s.lens, page_table=s.table, cache=s.cache, mass=s.mass,
                scale=0.125, masks=s.masks, max_query_len=s.n)
    for change, error in ((dict(mass=s.mass[1:]), ValueError), (dict(mass=s.mass.double()), TypeError),
                          (dict(lse=None), TypeError), (dict(mass=s.mass.transpose(1, 2)), ValueError)):
        refused(error, srg.lora_kv_attention_mass, **{**mass, **change})
    select = dict(mass=s.mass, seq_lens=s.lens, page_table=s.table, sinks=2, recent=10, kept=s.kept, new_lens=s.new_lens)
    for change, error in ((dict(sinks=-1), srg.LoraError), (dict(recent=99), srg.LoraError), (dict(sinks=1 << 40), ValueError),
                          (dict(kept=s.kept[:, :1]), ValueError), (dict(kept=s.kept.long()), TypeError),
                          (dict(new_lens=s.lens), srg.LoraError), (dict(mass=s.mass[..., :8].contiguous()), srg.LoraError)):
        refused(error, srg.lora_kv_select, **{**select, **change})
    compact = dict(kept=s.kept, counts=s.new_lens, page_table=s.table, cache=s.cache, head_dim=s.d, mass=s.mass)
    for change, error in ((dict(kept=new(s.B, 3, 5)), srg.LoraError), (dict(counts=new(s.B + 1)), ValueError),
                          (dict(head_dim=96), ValueError), (dict(page_size=32), ValueError), (dict(mass=s.mass[1:]), ValueError),
                          (dict(first=new(s.B, dtype=i64)), TypeError), (dict(dst_table=new(s.B, 0)), ValueError),
                          (dict(dst_table=new(s.B + 1, 4)), ValueError), (dict(kept=s.kept[..., ::2]), ValueError)):
        refused(error, srg.lora_kv_compact, **{**compact, **change})
    # tensors of another device than the current one
    monkeypatch.setattr(binding, "_current_device", lambda: 1)
    for call, kw in ((srg.lora_kv_tree_attention, tree), (srg.lora_kv_attention_mass, mass), (srg.lora_kv_select, select),
                     (srg.lora_kv_compact, compact), (srg.lora_draft_masks, dict(parents=s.parents, query_start=s.start, masks=s.masks))):
        refused(ValueError, call, **kw)


def test_masks_without_words_are_not_left_out_masks():
    s = Buffers()
    s.draw(0)
    none = s.masks[:, :0]
    args = (s.q, s.start, s.lens, s.table, s.cache)
    with pytest.raises(ValueError):
        srg.lora_kv_tree_attention(*args, s.out, 0.125, none, s.ws, s.n, lse=s.lse)
    with pytest.raises(ValueError):
        srg.lora_kv_attention_mass(s.q, s.lse, *args[1:], s.mass, 0.125, none, s.n)
    with pytest.raises(ValueError):
        srg.lora_draft_masks(s.parents, s.start, none, s.positions)


class Elsewhere(torch.Tensor):
    """A tensor that says it is on another device."""

    def get_device(self):
        return 1


def test_every_tensor_is_on_the_streams_device(monkeypatch):
    s = Buffers()
    s.draw(0)
    monkeypatch.setattr(binding, "_SEVERAL_DEVICES", True)
    step = dict(q=s.q, query_start=s.start, seq_lens=s.lens, page_table=s.table, cache=s.cache, scale=0.125, masks=s.masks,
                max_query_len=s.n, lse=s.lse)
    one = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    for call, args in (
            (srg.lora_draft_masks, dict(parents=s.parents, query_start=s.start, masks=s.masks, positions=s.positions,
                                        first_positions=s.text)),
            (srg.lora_kv_tree_attention, dict(step, out=s.out, workspace=one)),
            (srg.lora_kv_attention_mass, dict(step, mass=s.mass)),
            (srg.lora_kv_select, dict(mass=s.mass, seq_lens=s.lens, page_table=s.table, sinks=2, recent=10, kept=s.kept,
                                      new_lens=s.new_lens, workspace=one)),
            (srg.lora_kv_compact, dict(kept=s.kept, counts=s.new_lens, page_table=s.table, cache=s.cache, head_dim=s.d,
                                       mass=s.mass, first=torch.zeros_like(s.lens), dst_table=s.fresh_pages))):
        for stream in (None, torch.cuda.current_stream()):
            call(**args, stream=stream)
            for name, value in args.items():
                if isinstance(value, torch.Tensor):
                    with pytest.raises(ValueError, match="device"):
                        call(**{**args, name: value.as_subclass(Elsewhere)}, stream=stream)


def test_rejected_drafts_leave_neither_mass_nor_places():
    """A step as the header has it: the mass between the choice of drafts and their move, without
    the others' rows; the lengths set behind the move; the choice of tokens over these."""
    text, n, page = [70, 41, 90], [12, 7, 12], 16
    s = Step(4, [t + m for t, m in zip(text, n)], n, 8, 2, 64, page)
    _, lse = s.attend()
    want = s.want()
    # the longest path of each tree
    paths = [sorted(max(s.bits[a:b], key=len)) for a, b in zip(s.start, s.start[1:])]
    rejected = torch.ones(s.T, dtype=torch.bool, device="cuda")
    for a, path in zip(s.start, paths):
        rejected[[a + p for p in path]] = False
    lse.masked_fill_(rejected[:, None], -torch.inf)
    mass = torch.zeros(s.pages, s.kv, page, device="cuda")
    s.draw(mass, lse)
    accepted = np.full((3, 1, 12), -1, dtype=np.int32)
    for b, path in enumerate(paths):
        accepted[b, 0, :len(path)] = path
    counts, cache = ints([len(p) for p in paths]), dev(s.cache)
    srg.lora_kv_compact(dev(accepted), counts, dev(s.table), cache, s.d, mass=mass, first=ints(text), page_size=page)
    seq_lens = torch.empty_like(counts)
    torch.add(ints(text), counts, out=seq_lens)
    budget = 40
    kept, new_lens = ints(np.zeros((3, 2, budget))), ints([0] * 3)
    recent = max(len(p) for p in paths)
    srg.lora_kv_select(mass, seq_lens, dev(s.table), 2, recent, kept, new_lens)
    for b, path in enumerate(paths):
        length = text[b] + len(path)
        assert seq_lens[b] == length
        held = mass[torch.from_numpy(s.table[b]).cuda().long().clamp(min=0)].transpose(0, 1).reshape(2, -1)[:, :length]
        # the weights of every accepted row add up to one, each off by its score's and its sum's error
        rows = len(path) * s.hq
        slack = 2 * want["lse_slack"][s.start[b]:s.start[b + 1]].max() * rows
        assert abs(float(held.double().sum()) - rows) <= slack
        for h in range(2):
            assert kept[b, h, budget - recent:].tolist() == list(range(length - recent, length))
            assert kept[b, h].tolist() == C.select(held[h].tolist(), length, 2, recent, budget)


def test_calls_over_nothing():
    new = lambda *shape, dtype=torch.int32: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
    cache, mass = new(2, 2, 1, 16 * 34, dtype=torch.uint8), new(2, 1, 16, dtype=torch.float32)
    srg.lora_draft_masks(new(0), new(3), new(0, 1, dtype=torch.int64))
    q = new(0, 2, 64, dtype=torch.bfloat16)
    for masks in (None, new(0, 1, dtype=torch.int64)):
        srg.lora_kv_tree_attention(q, new(3), new(2), new(2, 1), cache, q, 1.0, masks, None, 4, lse=new(0, 2, dtype=torch.float32))
        srg.lora_kv_attention_mass(q, new(0, 2, dtype=torch.float32), new(3), new(2), new(2, 1), cache, mass, 1.0, masks, 4)
    srg.lora_kv_select(mass, new(0), new(0, 1), 0, 0, new(0, 1, 4), new(0))
    srg.lora_kv_compact(new(0, 1, 4), new(0), new(0, 1), cache, 64, mass=mass)
    srg.lora_kv_compact(new(2, 1, 0), new(2), new(2, 1), cache, 64, mass=mass)
    assert float(mass.sum()) == 0 and int(cache.sum()) == 0
