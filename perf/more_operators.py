"""The operators of drafted tokens and of caches of bounded length, as measured cases.

Four parts of a serving step over the 4-bit paged cache:

* ``tree``: a tree of drafted tokens in front of a model: which drafted tokens each one sees
  (its ancestors) and its position, and attention of the drafted tokens over the cache, in
  which they already stand behind their sequence's tokens; with the logarithm of each row's
  sum of exponentials;
* ``mass``: how much attention each cached token drew in a step, added up by token and key
  head beside the cache, the weight by which tokens are kept;
* ``select``: which tokens of a sequence that has grown past its bound each key head keeps:
  the first few, the last ones and the heaviest of the others;
* ``compact``: the move of kept tokens (or of the drafted tokens that were accepted) to the
  places in front, in the same pages or into new ones.

``run`` computes them with elementary torch operations, or (``own``) through the package.

The cache: uint8 [pages, 2 (k, v), kv_heads, page_bytes]; one page of one head is
page_size rows of head_dim / 2 bytes (two codes a byte, the even element in the low half)
followed by head_dim / 32 rows of page_size scale bytes.  A code is sign, two exponent bits
and one mantissa bit (0, 0.5, 1, 1.5, 2, 3, 4, 6); a scale byte b stands for 2^(b - 127) over
32 elements of one token's head.  The mass: fp32 [pages, kv_heads, page_size].
"""

import math

import torch

own = False

DEVICE = "cuda"
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------------
# The cases.
# --------------------------------------------------------------------------
def listed():
    return [
        # A single user's tree of drafts behind a short text, one key head a query head: latency.
        dict(name="tree 1x26 of 500", op="tree", seqs=1, q_min=26, q_max=26, len_min=500, len_max=500,
             q_heads=32, kv_heads=32, head_dim=128, page=64, window=0),
        # A serving batch, a tree for each sequence.
        dict(name="tree 16x32 to 4096", op="tree", seqs=16, q_min=32, q_max=32, len_min=300, len_max=4096,
             q_heads=64, kv_heads=8, head_dim=128, page=64, window=0),
        # A wide tree over one long document: the long axis has to be split.
        dict(name="tree 1x64 of 32768", op="tree", seqs=1, q_min=64, q_max=64, len_min=32768, len_max=32768,
             q_heads=64, kv_heads=8, head_dim=128, page=64, window=0),
        # Ragged small trees, short heads, a window, and sequences shorter than their trees.
        dict(name="tree drafts in a window", op="tree", seqs=24, q_min=1, q_max=13, len_min=0, len_max=3001,
             q_heads=24, kv_heads=4, head_dim=64, page=16, window=1024),
        # A decode step of a serving batch: one query a sequence.
        dict(name="mass 64 to 8192", op="mass", seqs=64, q_min=1, q_max=1, len_min=17, len_max=8192,
             q_heads=64, kv_heads=8, head_dim=128, page=64, window=0, tree=False),
        # Pieces of prompts behind an earlier part: the matrix products count.
        dict(name="mass pieces of prompts", op="mass", seqs=8, q_min=129, q_max=512, len_min=600, len_max=4608,
             q_heads=64, kv_heads=8, head_dim=128, page=64, window=0, tree=False),
        # A few drafted tokens behind short texts: latency.
        dict(name="mass drafts", op="mass", seqs=4, q_min=3, q_max=9, len_min=100, len_max=700,
             q_heads=16, kv_heads=4, head_dim=64, page=16, window=0, tree=True),
        # A batch whose sequences have doubled past their bound.
        dict(name="select 64 of 8192", op="select", seqs=64, len_min=4097, len_max=8192, kv_heads=8, page=64,
             budget=4096, sinks=4, recent=512),
        # One long document.
        dict(name="select 1 of 131072", op="select", seqs=1, len_min=131072, len_max=131072, kv_heads=8, page=64,
             budget=65536, sinks=4, recent=4096),
        # That document's kept tokens to the front, in place.
        dict(name="compact 1 to 65536 in place", op="compact", seqs=1, len_min=131072, len_max=131072,
             kv_heads=8, head_dim=128, page=64, budget=65536, sinks=4, heads=True, move=False),
        # A batch's into new pages: the old ones may be shared with other sequences.
        dict(name="compact 16 to 4096 into new pages", op="compact", seqs=16, len_min=4097, len_max=8192,
             kv_heads=8, head_dim=128, page=64, budget=4096, sinks=4, heads=True, move=True),
        # The accepted drafts of 64 sequences behind their texts: a few tokens, all heads alike.
        dict(name="compact accepted 64x6", op="compact", seqs=64, len_min=100, len_max=4096, kv_heads=8,
             head_dim=128, page=64, budget=6, sinks=1, heads=False, move=False),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "mass", "mass", "select", "compact"])
    head_dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 32])
    page = rng.choice([16, 32, 64, 128])
    if op == "select":
        seqs = _log(rng, 1, 64)
        len_max = _log(rng, 8, min(131072, 64 * 6144 * 8 // (seqs * kv_heads)))
        budget = _log(rng, 1, len_max)
        recent = rng.randrange(0, budget + 1)
        return dict(op=op, seqs=seqs, len_min=_log(rng, 1, len_max), len_max=len_max, kv_heads=kv_heads, page=page,
                    budget=budget, sinks=rng.randrange(0, min(8, budget - recent) + 1), recent=recent)
    if op == "compact":
        if rng.random() < 0.4:  # accepted drafts
            budget, heads, seqs = rng.randrange(1, 9), False, _log(rng, 1, 64)
            len_max = _log(rng, 64, 4096)
        else:
            seqs, heads = _log(rng, 1, 16), rng.random() < 0.8
            len_max = _log(rng, 8, min(131072, 131072 * 8 * 128 // (seqs * kv_heads * head_dim)))
            budget = max(1, len_max // rng.choice([2, 3, 8]))
        return dict(op=op, seqs=seqs, len_min=_log(rng, max(1, len_max // 2), len_max), len_max=len_max,
                    kv_heads=kv_heads, head_dim=head_dim, page=page, budget=budget, sinks=min(budget, rng.randrange(0, 5)),
                    heads=heads, move=heads and rng.random() < 0.5)
    per_kv = rng.choice([1, 2, 3, 4, 6, 8]) if kv_heads < 32 else 1
    window = rng.choice([0, 0, 0, 700])
    if op == "mass" and rng.random() < 0.4:  # pieces of prompts
        seqs, q_max = _log(rng, 1, 6), _log(rng, 16, 512)
        return dict(op=op, seqs=seqs, q_min=_log(rng, 1, q_max), q_max=q_max, len_min=q_max,
                    len_max=_log(rng, q_max, 4608), q_heads=kv_heads * per_kv, kv_heads=kv_heads, head_dim=head_dim,
                    page=page, window=window, tree=False)
    seqs = _log(rng, 1, 64)
    # some trees have more drafts than a word of the masks has bits
    q_max = min(_log(rng, 1, 200), max(1, 512 // seqs)) if op == "tree" else _log(rng, 1, 16)
    most = min(131072, 32768 * 64 * 64 // (seqs * kv_heads * per_kv * q_max), 64 * 4096 * 8 * 128 // (seqs * kv_heads * head_dim))
    len_max = _log(rng, 1, most)
    case = dict(op=op, seqs=seqs, q_min=_log(rng, 1, q_max), q_max=q_max, len_min=_log(rng, 1, len_max),
                len_max=len_max, q_heads=kv_heads * per_kv, kv_heads=kv_heads, head_dim=head_dim, page=page,
                window=window)
    return dict(case, tree=q_max > 1 and rng.random() < 0.5) if op == "mass" else case


def _spread(low, high, n):
    """n whole numbers from low to high, evenly."""
    return [high if n == 1 else low + (high - low) * i // (n - 1) for i in range(n)]


def _lengths(case):
    """(length, queries) of each sequence, before they are put into the seed's order."""
    n = case["seqs"]
    return _spread(case["len_min"], case["len_max"], n), _spread(case.get("q_min", 0), case.get("q_max", 0), n)


def _pairs(case):
    """(pairs of a query and a key it sees, tokens that some query sees), of trees without the
    ancestors besides the token itself."""
    window, tree = case["window"], case["op"] == "tree" or case["tree"]
    pairs = read = 0
    for length, queries in zip(*_lengths(case)):
        before = length - queries
        if tree:
            earlier = min(max(0, before), window) if window else max(0, before)
            pairs += queries * earlier + min(queries, length)
            read += earlier + min(queries, length)
        else:
            for i in range(queries):
                seen = max(0, before + i + 1)
                pairs += min(seen, window) if window else seen
            read += min(length, window + queries - 1) if window else length
    return pairs, read


def work(case):
    kv = case["kv_heads"]
    lens, queries = _lengths(case)
    if case["op"] == "select":
        over = [n for n in lens if n > case["budget"]]
        kept = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": 4 * kv * (sum(over) + kept) + 8 * len(lens), "flops": kv * sum(over)}
    d = case["head_dim"]
    row = 2 * kv * (d // 2 + d // 32)  # cache bytes of one token
    if case["op"] == "compact":
        lists = kv if case["heads"] else 1
        moved = sum(case["budget"] - (0 if case["move"] else case["sinks"]) for _ in lens)
        return {"bytes": moved * 2 * (row + 4 * kv) + 4 * len(lens) * lists * case["budget"], "flops": 0}
    hq, n = case["q_heads"], sum(queries)
    pairs, read = _pairs(case)
    if case["op"] == "tree":
        words = -(-case["q_max"] // 64)
        # parents read, masks, positions and sums written beside q, the cache and the outputs
        return {"bytes": read * row + n * (4 * hq * d + 4 * hq + 8 * words + 8), "flops": 4 * pairs * hq * d}
    return {"bytes": read * row // 2 + n * (2 * hq * d + 4 * hq) + 8 * kv * read, "flops": 2 * pairs * hq * d}


# --------------------------------------------------------------------------
# Inputs.
# --------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device=DEVICE).manual_seed(seed)


def _pages(need, g, first=1):
    """A page table for sequences of these numbers of pages: pages in the seed's order, from
    `first` on; page 0 is no sequence's (the page that a serving program points unused places at)."""
    ids = (torch.randperm(sum(need), generator=g, device=DEVICE) + first).int().cpu()
    table, at = torch.zeros(len(need), max(1, max(need)), dtype=torch.int32), 0
    for i, n in enumerate(need):
        table[i, :n] = ids[at:at + n]
        at += n
    return table.to(DEVICE), sum(need) + first


def _cache_of(pages, kv, page, d, g):
    """A cache of codes near a normal distribution's and scales over a few powers of two: keys
    of some channels a few times the others'."""
    cache = torch.empty(pages, 2, kv, page * (d // 2 + d // 32), dtype=torch.uint8, device=DEVICE)
    size = (pages, 2, kv, page * (d // 2))
    # magnitudes by the sum of two even draws: small ones more often
    low, high = (torch.randint(0, 4, size, generator=g, device=DEVICE, dtype=torch.uint8) +
                 torch.randint(0, 4, size, generator=g, device=DEVICE, dtype=torch.uint8) +
                 8 * torch.randint(0, 2, size, generator=g, device=DEVICE, dtype=torch.uint8) for _ in range(2))
    cache[..., :page * (d // 2)] = low | (high << 4)
    cache[..., page * (d // 2):] = torch.randint(124, 127, (pages, 2, kv, page * (d // 32)), generator=g,
                                                 device=DEVICE, dtype=torch.uint8)
    return cache


def _parents(queries, g):
    """Trees in the order of their drawing up: the first token is the root, the parent of
    each other one is one of those before it."""
    at = torch.cat([torch.arange(n) for n in queries] + [torch.zeros(0, dtype=torch.int64)]).to(DEVICE)
    pick = (torch.rand(len(at), generator=g, device=DEVICE) * at).floor().int()
    return torch.where(at == 0, -1, torch.minimum(pick, (at - 1).clamp(min=0).int())).int()


def _prepare_attention(case, g):
    d, kv, hq, page = case["head_dim"], case["kv_heads"], case["q_heads"], case["page"]
    lens, queries = _lengths(case)
    order = torch.randperm(len(lens), generator=g, device=DEVICE).tolist()
    lens, queries = [lens[i] for i in order], [queries[i] for i in order]
    table, pages = _pages([-(-n // page) for n in lens], g)
    n, words = sum(queries), -(-case["q_max"] // 64)
    new = lambda *shape, dtype=torch.float32: torch.zeros(*shape, dtype=dtype, device=DEVICE)  # noqa: E731
    s = {"q": torch.randn(n, hq, d, generator=g, device=DEVICE).bfloat16(),
         "start": torch.tensor([0] + queries).cumsum(0).int().to(DEVICE),
         "lens": torch.tensor(lens, dtype=torch.int32, device=DEVICE), "table": table,
         "cache": _cache_of(pages, kv, page, d, g), "scale": d ** -0.5, "q_max": case["q_max"],
         "window": case["window"], "page": page, "tree": case["op"] == "tree" or case["tree"]}
    if s["tree"]:
        s["parents"] = _parents(queries, g)
        s["first"] = (s["lens"] - (s["start"][1:] - s["start"][:-1])).clamp(min=0)
        s["masks"], s["positions"] = new(n, words, dtype=torch.int64), new(n, dtype=torch.int32)
    if case["op"] == "tree":
        s["out"], s["lse"] = new(n, hq, d, dtype=torch.bfloat16), new(n, hq)
        if own:
            import segmented_rank_gemm_amd as srg
            s["workspace"] = srg.kv_tree_attention_workspace(len(lens), case["q_max"], table.shape[1] * page, hq, kv, d)
        return s
    # the sums are attention's, and a tree's masks are made before it
    if s["tree"]:
        s["masks"].copy_(_bits(_reach(s), s))
    s["lse"] = _rows(_lse(_scores(s)).float(), s)
    # what earlier steps left
    s["mass"] = (2 * torch.randn(pages, kv, page, generator=g, device=DEVICE)).exp()
    return s


def _prepare_select(case, g):
    lens, _ = _lengths(case)
    lens = [lens[i] for i in torch.randperm(len(lens), generator=g, device=DEVICE).tolist()]
    table, pages = _pages([-(-n // case["page"]) for n in lens], g)
    kv, page, budget = case["kv_heads"], case["page"], case["budget"]
    # a few tokens draw most of the attention; some draw none at all, and are equal
    mass = (2 * torch.randn(pages, kv, page, generator=g, device=DEVICE)).exp()
    mass = mass * (torch.rand(pages, kv, page, generator=g, device=DEVICE) > 0.05)
    return {"mass": mass, "lens": torch.tensor(lens, dtype=torch.int32, device=DEVICE), "table": table,
            "sinks": case["sinks"], "recent": case["recent"],
            "kept": torch.zeros(len(lens), kv, budget, dtype=torch.int32, device=DEVICE),
            "new_lens": torch.zeros(len(lens), dtype=torch.int32, device=DEVICE)}


def _prepare_compact(case, g):
    lens, _ = _lengths(case)
    lens = [lens[i] for i in torch.randperm(len(lens), generator=g, device=DEVICE).tolist()]
    kv, d, page, budget, sinks = (case[k] for k in ("kv_heads", "head_dim", "page", "budget", "sinks"))
    lists = kv if case["heads"] else 1
    if case["heads"] or case["budget"] > 8:
        first, span = None, lens  # kept tokens of the whole sequence
    else:
        # drafted tokens behind the text: the root, and others that no other one moves to
        first, span = torch.tensor(lens, dtype=torch.int32, device=DEVICE), [8 * budget] * len(lens)
    table, pages = _pages([-(-(n + (0 if first is None else m)) // page) for n, m in zip(lens, span)], g)
    dst, more = _pages([-(-budget // page)] * len(lens), g, pages) if case["move"] else (None, pages)
    # each list: the first `sinks`, then a choice of the others in their order
    mine = torch.tensor([max(m, budget) for m in span], device=DEVICE)
    at = torch.arange(int(mine.max()), device=DEVICE)
    weight = torch.rand(len(lens), lists, len(at), generator=g, device=DEVICE)
    low = sinks if first is None else budget
    weight = torch.where(at < sinks, 2.0, torch.where((at >= low) & (at < mine[:, None, None]), weight, -1.0))
    kept = weight.topk(budget, dim=-1).indices.sort(-1).values.int()
    return {"kept": kept, "counts": torch.tensor([min(budget, m) for m in span], dtype=torch.int32, device=DEVICE),
            "first": first, "table": table, "dst": dst, "head_dim": d, "page": page,
            "cache": torch.randint(0, 256, (more, 2, kv, page * (d // 2 + d // 32)), dtype=torch.uint8, generator=g, device=DEVICE),
            "mass": torch.rand(more, kv, page, generator=g, device=DEVICE)}


def prepare(case, seed):
    g = _generator(seed)
    make = {"tree": _prepare_attention, "mass": _prepare_attention, "select": _prepare_select, "compact": _prepare_compact}
    return dict(make[case["op"]](case, g), op=case["op"])


# --------------------------------------------------------------------------
# The plain form.
# --------------------------------------------------------------------------
def _power(byte):
    """2^(byte - 127) in fp32, from its bits."""
    return (byte.int() << 23).view(torch.float32)


def _held(s, part):
    """fp32 keys (part 0) or values (1) of every sequence: [sequences, kv, longest, d]."""
    page, d = s["page"], s["q"].shape[2]
    held = s["cache"][:, part][s["table"].long()]
    codes = held[..., :page * (d // 2)].unflatten(-1, (page, d // 2))
    scales = held[..., page * (d // 2):].unflatten(-1, (d // 32, page)).transpose(-1, -2)
    both = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)
    levels = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=codes.device)
    values = (levels[both.int()].unflatten(-1, (-1, 32)) * _power(scales)[..., None]).flatten(-2)
    return values.transpose(1, 2).flatten(2, 3)


def _reach(s):
    """Which drafted tokens each one sees: [sequences, q_max, q_max]."""
    start, q_max = s["start"].long(), s["q_max"]
    at = torch.arange(q_max, device=start.device)
    mine = at < (start[1:] - start[:-1])[:, None]
    parents = s["parents"].long()[(start[:-1, None] + at).clamp(max=len(s["parents"]) - 1)]
    parents = torch.where(mine & (parents >= 0) & (parents < at), parents, q_max)
    seen = (at[None, None] == parents[..., None]) | (torch.eye(q_max, device=start.device) > 0) & mine[..., None]
    for _ in range((q_max - 1).bit_length()):  # ancestors of twice as many steps
        seen = torch.matmul(seen.float(), seen.float()) > 0
    return seen


def _bits(reach, s):
    """The rows of `reach` as words of 64 bits, the first drafted token in the lowest."""
    words = s["masks"].shape[1]
    bits = torch.nn.functional.pad(reach, (0, 64 * words - s["q_max"])).unflatten(-1, (words, 64)).long()
    bits = (bits << torch.arange(64, device=bits.device)).sum(-1)
    start = s["start"].long()
    token = torch.arange(len(s["parents"]), device=bits.device)
    seq = torch.searchsorted(start[1:], token, right=True)
    return bits[seq, token - start[seq]]


def _seen(s):
    """Which tokens each query sees: [sequences, q_max, longest]."""
    start, lens, q_max = s["start"].long(), s["lens"].long(), s["q_max"]
    queries = start[1:] - start[:-1]
    row = torch.arange(q_max, device=start.device)
    key = torch.arange(s["table"].shape[1] * s["page"], device=start.device)
    before = (lens - queries)[:, None, None]
    if not s["tree"]:
        place = before + row[:, None]
        seen = (key <= place) & (key < lens[:, None, None])
        return seen & (key > place - s["window"]) if s["window"] else seen
    if s.get("op") == "tree":
        reach = _reach(s)
    else:  # from the masks
        words = s["masks"][(start[:-1, None] + row).clamp(max=len(s["masks"]) - 1)]
        reach = ((words[..., None] >> torch.arange(64, device=words.device)) & 1).flatten(-2)[..., :q_max] > 0
    draft = key - before  # [sequences, 1, longest]: the key's number among the drafted tokens
    drafted = (draft >= 0) & (key < lens[:, None, None])
    mine = torch.gather(reach, 2, draft.clamp(0, q_max - 1).expand(-1, q_max, -1))
    seen = torch.where(drafted, mine, (key < before).expand_as(mine))
    if s["window"]:  # the last ones of those
        seen = seen & (seen.flip(-1).int().cumsum(-1).flip(-1) <= s["window"])
    return seen


def _scores(s):
    """[sequences, kv, q_max * group, longest], -inf where a query does not see a key."""
    (n, hq, d), kv, q_max = s["q"].shape, s["cache"].shape[2], s["q_max"]
    start = s["start"].long()
    row = torch.arange(q_max, device=start.device)
    q = s["q"].float()[(start[:-1, None] + row).clamp(max=n - 1)].unflatten(2, (kv, hq // kv))
    q = q.permute(0, 2, 1, 3, 4).flatten(2, 3)
    there = row < (start[1:] - start[:-1])[:, None]
    seen = (_seen(s) & there[..., None]).repeat_interleave(hq // kv, dim=1)[:, None]
    score = torch.matmul(q, _held(s, 0).transpose(-1, -2).contiguous()) * s["scale"]
    return score.masked_fill(~seen, -math.inf)


def _lse(score):
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    return (score - top).exp().sum(-1).log() + top[..., 0]


def _rows(x, s):
    """[sequences, kv, q_max * group, ...] as the rows [tokens, q_heads, ...] of q."""
    start, group = s["start"].long(), s["q"].shape[1] // s["cache"].shape[2]
    x = x.unflatten(2, (s["q_max"], group)).transpose(1, 2).flatten(2, 3)
    token = torch.arange(s["q"].shape[0], device=start.device)
    seq = torch.searchsorted(start[1:], token, right=True)
    return x[seq, token - start[seq]]


def _plain_tree(s):
    reach = _reach(s)
    s["masks"].copy_(_bits(reach, s))
    start = s["start"].long()
    token = torch.arange(len(s["parents"]), device=start.device)
    seq = torch.searchsorted(start[1:], token, right=True)
    s["positions"].copy_(s["first"][seq] + reach.sum(-1)[seq, token - start[seq]] - 1)
    score = _scores(s)
    top = score.amax(-1, keepdim=True)
    p = (score - torch.where(top == -math.inf, 0.0, top)).exp()
    total = p.sum(-1, keepdim=True)
    s["out"].copy_(_rows(torch.matmul(p, _held(s, 1)) / torch.where(total == 0, 1.0, total), s))
    s["lse"].copy_(_rows((total.log() + torch.where(top == -math.inf, 0.0, top))[..., 0], s))


def _plain_mass(s):
    score = _scores(s)
    start, lens, group = s["start"].long(), s["lens"].long(), s["q"].shape[1] // s["cache"].shape[2]
    n = s["q"].shape[0]
    row = torch.arange(s["q_max"], device=start.device)
    lse = s["lse"][(start[:-1, None] + row).clamp(max=n - 1)].unflatten(2, (-1, group)).transpose(1, 2).flatten(2)
    p = (score - torch.where(lse == -math.inf, 0.0, lse)[..., None]).exp()
    drawn = p.sum(2)                                              # [sequences, kv, longest]
    page, table = s["page"], s["table"].long()
    key = torch.arange(table.shape[1] * page, device=start.device)
    queries = (start[1:] - start[:-1])[:, None]
    there = (key < lens[:, None]) & (queries > 0)
    fresh = key >= lens[:, None] - queries                        # this step's own tokens have no earlier weight
    at = torch.where(there, table[:, key // page], 0)             # no sequence's page otherwise
    old = s["mass"][at, :, key % page].transpose(1, 2)
    now = torch.where(fresh[:, None], drawn, old + drawn)
    s["mass"][at, :, key % page] = torch.where(there[:, None], now, old).transpose(1, 2)


def _plain_select(s):
    (b, kv, budget), page = s["kept"].shape, s["mass"].shape[2]
    lens = s["lens"].long()
    weight = s["mass"][s["table"].long()].transpose(1, 2).flatten(2)  # [sequences, kv, longest]
    key = torch.arange(weight.shape[2], device=lens.device)
    n = lens[:, None]
    always = (key < s["sinks"]) | (key >= n - s["recent"])
    weight = torch.where(weight.isnan(), -math.inf, weight)
    # the tokens that stay anyway, then by weight, then those that are not there; equal ones in their order
    by_weight = torch.argsort(weight, dim=-1, descending=True, stable=True)
    group = torch.where(key >= n, 2, torch.where(always, 0, 1))[:, None].expand_as(by_weight)
    order = by_weight.gather(-1, torch.argsort(group.gather(-1, by_weight), dim=-1, stable=True))
    room = torch.nn.functional.pad(order, (0, max(0, budget - order.shape[-1])), value=len(key))[..., :budget]
    count = n.clamp(max=budget)[..., None]
    room = torch.where(torch.arange(budget, device=lens.device) < count, room, len(key)).sort(-1).values
    s["kept"].copy_(torch.where(room < len(key), room, -1))
    s["new_lens"].copy_(lens.clamp(max=budget))


def _places(s):
    """(from, to): page and place in it of each kept token, [sequences, kv, budget], all heads' lists."""
    page, kept = s["page"], s["kept"].long().expand(-1, s["cache"].shape[2], -1)
    first = 0 if s["first"] is None else s["first"].long()[:, None, None]
    source, to = kept + first, torch.arange(kept.shape[2], device=kept.device).expand_as(kept) + first
    seq = torch.arange(len(kept), device=kept.device)[:, None, None]
    dst = s["table"] if s["dst"] is None else s["dst"]
    return (s["table"].long()[seq, source // page], source % page), (dst.long()[seq, to // page], to % page)


def _plain_compact(s):
    page, d, kv = s["page"], s["head_dim"], s["cache"].shape[2]
    (sp, so), (dp, do) = _places(s)
    codes = s["cache"][..., :page * (d // 2)].unflatten(-1, (page, d // 2))
    scales = s["cache"][..., page * (d // 2):].unflatten(-1, (d // 32, page))
    head = torch.arange(kv, device=sp.device)[:, None]
    part = torch.arange(2, device=sp.device)[:, None, None, None]
    codes[dp, part, head, do] = codes[sp, part, head, so]
    scales[dp, part, head, :, do] = scales[sp, part, head, :, so]
    s["mass"][dp, head, do] = s["mass"][sp, head, so]


def _run_own(s):
    import segmented_rank_gemm_amd as srg
    if s["op"] == "tree":
        srg.lora_draft_masks(s["parents"], s["start"], s["masks"], positions=s["positions"], first_positions=s["first"])
        srg.lora_kv_tree_attention(s["q"], s["start"], s["lens"], s["table"], s["cache"], s["out"], s["scale"],
                                   s["masks"], s["workspace"], s["q_max"], window=s["window"], lse=s["lse"])
    elif s["op"] == "mass":
        srg.lora_kv_attention_mass(s["q"], s["lse"], s["start"], s["lens"], s["table"], s["cache"], s["mass"], s["scale"],
                                   s["masks"] if s["tree"] else None, s["q_max"], window=s["window"])
    elif s["op"] == "select":
        srg.lora_kv_select(s["mass"], s["lens"], s["table"], s["sinks"], s["recent"], s["kept"], s["new_lens"])
    else:
        srg.lora_kv_compact(s["kept"], s["counts"], s["table"], s["cache"], s["head_dim"], mass=s["mass"],
                            first=s["first"], dst_table=s["dst"])


# The compacted cache is returned as it is: its bytes move, nothing is computed from them.
OUTPUTS = {"tree": ("masks", "positions", "out", "lse"), "mass": ("mass",), "select": ("kept", "new_lens"),
           "compact": ("cache", "mass")}


def run(s):
    if own:
        _run_own(s)
    else:
        {"tree": _plain_tree, "mass": _plain_mass, "select": _plain_select, "compact": _plain_compact}[s["op"]](s)
    return [s[k] for k in OUTPUTS[s["op"]]]


# --------------------------------------------------------------------------
# The definitions in 64 bits.
# --------------------------------------------------------------------------
def _exact_sequences(s):
    """For each sequence with queries and tokens: its number, rows, length, keys and values
    [2, kv, length, d] in 64 bits, and which tokens each row does not see."""
    kv, page, d = s["cache"].shape[2], s["page"], s["q"].shape[2]
    levels = list(LEVELS) + [-x for x in LEVELS]
    even, odd = (torch.tensor([levels[b >> k & 15] for b in range(256)], dtype=torch.float64, device=DEVICE) for k in (0, 4))
    start, lens = s["start"].tolist(), s["lens"].tolist()
    for i, length in enumerate(lens):
        rows, pages = start[i + 1] - start[i], -(-length // page)
        if not rows or not length:
            continue
        held = s["cache"][s["table"][i, :pages].long()]
        codes = held[..., :page * d // 2].reshape(pages, 2, kv, page, d // 2)
        power = torch.exp2(held[..., page * d // 2:].reshape(pages, 2, kv, d // 32, page).double() - 127)
        full = torch.stack([even[codes.int()], odd[codes.int()]], dim=-1)
        full = full.reshape(pages, 2, kv, page, d // 32, 32) * power.transpose(-1, -2)[..., None]
        full = full.reshape(pages, 2, kv, page, d).permute(1, 2, 0, 3, 4).reshape(2, kv, -1, d)[:, :, :length]
        before, hidden = length - rows, torch.ones(rows, length, dtype=torch.bool)
        if s["tree"]:
            parents = s["parents"][start[i]:start[i + 1]].tolist()
            for r in range(rows):
                path, node = [], r
                while node >= 0:
                    path.append(node)
                    node = parents[node]
                path = [before + p for p in reversed(path) if before + p >= 0]
                text = max(0, before)
                if s["window"]:
                    path = path[-s["window"]:]
                    text = min(text, s["window"] - len(path))
                hidden[r, path] = False
                hidden[r, max(0, before) - text:max(0, before)] = False
        else:
            for r in range(rows):
                low = max(0, before + r + 1 - s["window"]) if s["window"] else 0
                hidden[r, low:max(0, before + r + 1)] = False
        yield i, slice(start[i], start[i + 1]), length, full, hidden.to(DEVICE)


def _exact_tree(s):
    (n, hq, d), kv = s["q"].shape, s["cache"].shape[2]
    group = hq // kv
    out = torch.zeros(n, hq, d, dtype=torch.float64, device=DEVICE)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device=DEVICE)
    for i, rows, length, full, hidden in _exact_sequences(s):
        blind = hidden.all(1)[:, None]
        for h in range(hq):
            q = s["q"][rows, h].double() * s["scale"]
            score = (q @ full[0, h // group].T.contiguous()).masked_fill(hidden, -math.inf)
            lse[rows, h] = torch.logsumexp(score, -1)
            p = torch.softmax(score, -1).masked_fill(blind, 0.0)
            out[rows, h] = p @ full[1, h // group]
    return [None, None, out, lse]


def _exact_mass(s):
    (n, hq, d), kv, page = s["q"].shape, s["cache"].shape[2], s["page"]
    mass = s["mass"].double()
    for i, rows, length, full, hidden in _exact_sequences(s):
        drawn = torch.zeros(kv, length, dtype=torch.float64, device=DEVICE)
        for h in range(hq):
            q = s["q"][rows, h].double() * s["scale"]
            score = (q @ full[0, h * kv // hq].T.contiguous()).masked_fill(hidden, -math.inf)
            lse = s["lse"][rows, h, None].double()
            drawn[h * kv // hq] += torch.exp(score - lse).masked_fill(lse == -math.inf, 0.0).sum(0)
        key = torch.arange(length, device=DEVICE)
        place = s["table"][i].long()[key // page], slice(None), key % page
        earlier = mass[place] * (key < length - hidden.shape[0]).double()[:, None]
        mass[place] = earlier + drawn.T
    return [mass]


def _exact_compact(s):
    """The mass; the cache's bytes move with it."""
    pages, kv, page = s["mass"].shape
    flat = s["mass"].double().transpose(1, 2).reshape(pages * page, kv)
    moved = flat.clone()
    dst = s["table"] if s["dst"] is None else s["dst"]
    for i, count in enumerate(s["counts"].tolist()):
        base = 0 if s["first"] is None else int(s["first"][i])
        to = base + torch.arange(count, device=DEVICE)
        to = dst[i].long()[to // page] * page + to % page
        for h in range(kv):
            at = base + s["kept"][i, h % s["kept"].shape[1], :count].long()
            moved[to, h] = flat[s["table"][i].long()[at // page] * page + at % page, h]
    return [None, moved.reshape(pages, page, kv).transpose(1, 2)]


def exact(case, seed):
    if case["op"] == "select":  # a choice
        return None
    s = prepare(case, seed)
    return {"tree": _exact_tree, "mass": _exact_mass, "compact": _exact_compact}[case["op"]](s)
