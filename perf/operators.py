"""The operators of an attention layer around the low-rank projections, as measured cases.

Three parts of one layer of a served model, in the order in which it runs them:

* ``norm``: the residual's addition and the root-mean-square norm in front of a projection,
  with the normalised row in bf16 (the low-rank path's x) and in 8 bits with scales (the
  base product's operand);
* ``append``: the rotation by position of the projection's q and k, and the write of k and v
  into a paged cache held in 4 bits; then the read of what those places now hold;
* ``attention``: attention over that cache, from one query a sequence to whole prompts.

``run`` computes them with elementary torch operations, or (``own``) through the package.

The cache: uint8 [pages, 2 (k, v), kv_heads, page_bytes]; one page of one head is
page_size rows of head_dim / 2 bytes (two codes a byte, the even element in the low half)
followed by head_dim / 32 rows of page_size scale bytes.  A code is sign, two exponent bits
and one mantissa bit (0, 0.5, 1, 1.5, 2, 3, 4, 6); a scale byte b stands for 2^(b - 127) over
32 elements of one token's head; b = 255 marks a block that held an infinity or a NaN.
"""

import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-5
ROPE_BASE = 10000.0
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------------
# The cases.
# --------------------------------------------------------------------------
def listed():
    return [
        # One decode step of 16 sequences: a few hundred KB, so the launch counts.
        dict(name="norm decode 16x4096", op="norm", tokens=16, hidden=4096, residual=True, bf16=True,
             group=0),
        # A batch of whole prompts in front of a qkv projection that runs in 8 bits while the
        # low-rank path reads bf16.
        dict(name="norm prompts 8192x8192", op="norm", tokens=8192, hidden=8192, residual=True,
             bf16=True, group=0),
        # In front of a down projection, scales a 128-element group, no residual, 8 bits only;
        # an odd number of tokens.
        dict(name="norm groups 1001x11008", op="norm", tokens=1001, hidden=11008, residual=False,
             bf16=False, group=128),
        # One token for each of 64 sequences at positions all over the table.
        dict(name="append decode 64", op="append", tokens=64, q_heads=64, kv_heads=8, head_dim=128,
             rot_dim=128, interleaved=False, page=64, prompt=0, skip=0),
        # Whole prompts, one key head a query head (4096 wide).
        dict(name="append prompts 4096", op="append", tokens=4096, q_heads=32, kv_heads=32,
             head_dim=128, rot_dim=128, interleaved=False, page=64, prompt=1365, skip=0),
        # Short heads, half of each rotated in neighbouring pairs, small pages, and a padded
        # batch: every seventh token has no place in the cache.
        dict(name="append padded 777", op="append", tokens=777, q_heads=16, kv_heads=4, head_dim=64,
             rot_dim=32, interleaved=True, page=16, prompt=259, skip=7),
        # A single user's next token: latency.
        dict(name="attention 1 of 500", op="attention", seqs=1, q_min=1, q_max=1, len_min=500,
             len_max=500, q_heads=32, kv_heads=32, head_dim=128, page=64, window=0),
        # A serving batch's next tokens, lengths spread over the whole range.
        dict(name="attention 64 to 8192", op="attention", seqs=64, q_min=1, q_max=1, len_min=17,
             len_max=8192, q_heads=64, kv_heads=8, head_dim=128, page=64, window=0),
        # One key head a query head: the most cache bytes a query.
        dict(name="attention 16 heads of their own", op="attention", seqs=16, q_min=1, q_max=1,
             len_min=1900, len_max=2100, q_heads=32, kv_heads=32, head_dim=128, page=16, window=0),
        # One long document: few rows, so the long axis has to be split.
        dict(name="attention 1 of 131072", op="attention", seqs=1, q_min=1, q_max=1, len_min=131072,
             len_max=131072, q_heads=64, kv_heads=8, head_dim=128, page=64, window=0),
        # Prompts taken in pieces of up to 512 tokens behind an earlier part: the matrix
        # products count.
        dict(name="attention pieces of prompts", op="attention", seqs=8, q_min=129, q_max=512,
             len_min=600, len_max=4608, q_heads=64, kv_heads=8, head_dim=128, page=64, window=0),
        # A few drafted tokens a sequence, short heads, a window, and sequences that are shorter
        # than their queries (their first queries see nothing).
        dict(name="attention drafts in a window", op="attention", seqs=24, q_min=1, q_max=5,
             len_min=0, len_max=3001, q_heads=24, kv_heads=4, head_dim=64, page=16, window=1024),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "append", "attention", "attention"])
    if op == "norm":
        group = rng.choice([0, 0, 32, 128])
        hidden = _log(rng, 256, 16384)
        hidden -= hidden % (group or 8)
        return dict(op=op, tokens=_log(rng, 1, min(8192, 8192 * 8192 // hidden)), hidden=hidden,
                    residual=rng.random() < 0.7, bf16=rng.random() < 0.7, group=group)
    head_dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 32])
    per_kv = rng.choice([1, 2, 3, 4, 6, 8]) if kv_heads < 32 else 1
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        rot_dim = rng.choice([head_dim, head_dim, head_dim // 2])
        tokens = _log(rng, 1, 4096)
        return dict(op=op, tokens=tokens, q_heads=kv_heads * per_kv, kv_heads=kv_heads,
                    head_dim=head_dim, rot_dim=rot_dim, interleaved=rng.random() < 0.3, page=page,
                    prompt=rng.choice([0, _log(rng, 1, tokens)]), skip=rng.choice([0, 0, 5]))
    if rng.random() < 0.7:  # next tokens
        seqs = _log(rng, 1, 64)
        q_max = rng.choice([1, 1, 1, 2, 4, 7])
        len_max = _log(rng, 1, min(131072, 512 * 1024 * 8 * 128 // (seqs * kv_heads * head_dim)))
    else:                   # pieces of prompts
        seqs = _log(rng, 1, 6)
        q_max = _log(rng, 16, 512)
        len_max = _log(rng, q_max, 4608)
    return dict(op=op, seqs=seqs, q_min=_log(rng, 1, q_max), q_max=q_max,
                len_min=_log(rng, 1, len_max), len_max=len_max, q_heads=kv_heads * per_kv,
                kv_heads=kv_heads, head_dim=head_dim, page=page, window=rng.choice([0, 0, 0, 700]))


def _spread(low, high, n):
    """n whole numbers from low to high, evenly."""
    return [high if n == 1 else low + (high - low) * i // (n - 1) for i in range(n)]


def _lengths(case):
    """(length, queries) of each sequence, before they are put into the seed's order."""
    n = case["seqs"]
    return _spread(case["len_min"], case["len_max"], n), _spread(case["q_min"], case["q_max"], n)


def _pairs(length, queries, window):
    """(query, key) pairs of one sequence: query i sees the keys up to its own place."""
    total = 0
    for i in range(queries):
        seen = max(0, length - queries + i + 1)
        total += min(seen, window) if window else seen
    return total


def work(case):
    if case["op"] == "norm":
        t, h = case["tokens"], case["hidden"]
        groups = h // case["group"] if case["group"] else 1
        per_row = 2 * h + h + 4 * groups + (4 * h if case["residual"] else 0) + (2 * h if case["bf16"] else 0)
        return {"bytes": t * per_row + 2 * h, "flops": 8 * t * h}
    d, kv, hq = case["head_dim"], case["kv_heads"], case["q_heads"]
    row = 2 * kv * (d // 2 + d // 32)  # cache bytes of one token
    if case["op"] == "append":
        t = case["tokens"]
        kept = t - (t + case["skip"] - 1) // case["skip"] if case["skip"] else t
        # q, k, v read; q, the cache and the values that it holds written; places, angles
        per = 2 * d * (hq + 2 * kv) + 2 * d * hq + 4 * d * kv + 12 + 4 * case["rot_dim"]
        return {"bytes": t * per + 2 * kept * row, "flops": 3 * t * case["rot_dim"] * (hq + kv) + 4 * t * 2 * kv * d}
    lens, queries = _lengths(case)
    window = case["window"]
    read = sum(min(l, window + q - 1) if window else l for l, q in zip(lens, queries))
    pairs = sum(_pairs(l, q, window) for l, q in zip(lens, queries))
    return {"bytes": read * row + 4 * sum(queries) * hq * d, "flops": 4 * pairs * hq * d}


# --------------------------------------------------------------------------
# Inputs.
# --------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device=DEVICE).manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE)


def _angles(rows, rot_dim):
    """cos and sin of every position's angles, the table that a program keeps."""
    freq = ROPE_BASE ** (-torch.arange(0, rot_dim, 2, device=DEVICE, dtype=torch.float64) / rot_dim)
    a = torch.arange(rows, device=DEVICE, dtype=torch.float64)[:, None] * freq
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def _pages(lens, page, g):
    """A page table for sequences of these lengths: pages in the seed's order; page 0 is no
    sequence's (the page that a serving program points unused places at)."""
    need = [-(-l // page) for l in lens]
    order = torch.randperm(sum(need), generator=g, device=DEVICE) + 1
    table = torch.zeros(len(lens), max(1, max(need)), dtype=torch.int32)
    ids, at = order.cpu().to(torch.int32), 0
    for i, n in enumerate(need):
        table[i, :n] = ids[at:at + n]
        at += n
    return table.to(DEVICE), sum(need) + 1


def _prepare_norm(case, g):
    t, h = case["tokens"], case["hidden"]
    # activations with a few channels far larger than the others
    spread = 1 + 15 * (torch.rand(h, generator=g, device=DEVICE) < 0.01)
    s = {"x": (_normal(g, t, h) * spread).bfloat16(),
         "weight": (1 + 0.2 * _normal(g, h)).bfloat16(),
         "residual": (2 * _normal(g, t, h) * spread).bfloat16() if case["residual"] else None}
    s["sum"] = torch.empty_like(s["x"]) if case["residual"] else None
    s["y"] = torch.empty_like(s["x"]) if case["bf16"] else None
    s["y8"] = torch.empty(t, h, dtype=torch.float8_e4m3fn, device=DEVICE)
    s["scales"] = torch.empty(t, h // case["group"] if case["group"] else 1, device=DEVICE)
    return s


def _prepare_append(case, g):
    t, d, kv, hq, page = case["tokens"], case["head_dim"], case["kv_heads"], case["q_heads"], case["page"]
    rows = 131072
    step = max(1, case["prompt"])  # tokens of one sequence: one, or a prompt's
    lens = [min(step, t - at) for at in range(0, t, step)]
    first = torch.randint(0, rows - step, (len(lens),), generator=g, device=DEVICE)
    if case["prompt"]:
        first = torch.zeros_like(first)
    places = [page * 3 if not case["prompt"] else l for l in lens]
    table, pages = _pages(places, page, g)
    i = torch.arange(t, device=DEVICE)
    seq, at = i // step, i % step
    inside = torch.randint(0, page * 3, (t,), generator=g, device=DEVICE) if not case["prompt"] else at
    slots = table[seq, inside // page].long() * page + inside % page
    if case["skip"]:
        slots = torch.where(i % case["skip"] == 0, -1, slots)
    channel = 1 + 5 * (torch.rand((hq + 2 * kv) * d, generator=g, device=DEVICE) < 0.02)
    old = torch.randint(0, 256, (pages, 2, kv, page * (d // 2 + d // 32)), dtype=torch.uint8, generator=g, device=DEVICE)
    old[..., page * (d // 2):] = old[..., page * (d // 2):] % 8 + 124
    return {"qkv": (_normal(g, t, (hq + 2 * kv) * d) * channel).bfloat16(),
            "positions": (first[seq] + at).int(), "slots": slots, "rope": _angles(rows, case["rot_dim"]),
            "cache": old, "interleaved": case["interleaved"], "page": page,
            "q_out": torch.empty(t, hq, d, dtype=torch.bfloat16, device=DEVICE),
            "k_out": torch.empty(t, kv, d, dtype=torch.bfloat16, device=DEVICE),
            "v_out": torch.empty(t, kv, d, dtype=torch.bfloat16, device=DEVICE)}


def _prepare_attention(case, g):
    d, kv, hq, page = case["head_dim"], case["kv_heads"], case["q_heads"], case["page"]
    lens, queries = _lengths(case)
    order = torch.randperm(len(lens), generator=g, device=DEVICE).tolist()
    lens, queries = [lens[i] for i in order], [queries[i] for i in order]
    table, pages = _pages(lens, page, g)
    cache = torch.empty(pages, 2, kv, page * (d // 2 + d // 32), dtype=torch.uint8, device=DEVICE)
    for part in (0, 1):  # keys with a few strong channels, values without
        values = torch.randn(pages, kv, page, d, generator=g, device=DEVICE)
        if part == 0:
            values *= 1 + 3 * (torch.rand(kv, 1, d, generator=g, device=DEVICE) < 0.03)
        codes, scales = _to_codes(values.bfloat16())
        cache[:, part] = torch.cat([_packed(codes).flatten(2), scales.transpose(-1, -2).flatten(2)], dim=-1)
    n = sum(queries)
    start = torch.tensor([0] + queries, dtype=torch.int32).cumsum(0).int()
    s = {"q": _normal(g, n, hq, d).bfloat16(), "start": start.to(DEVICE),
         "lens": torch.tensor(lens, dtype=torch.int32, device=DEVICE), "table": table, "cache": cache,
         "out": torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEVICE), "scale": d ** -0.5,
         "q_max": case["q_max"], "window": case["window"], "page": page}
    if own:
        import segmented_rank_gemm_amd as srg
        s["workspace"] = srg.kv_attention_workspace(len(lens), case["q_max"], table.shape[1] * page, hq, kv, d)
    return s


def prepare(case, seed):
    g = _generator(seed)
    made = {"norm": _prepare_norm, "append": _prepare_append, "attention": _prepare_attention}[case["op"]](case, g)
    return dict(made, op=case["op"])


# --------------------------------------------------------------------------
# The plain form.
# --------------------------------------------------------------------------
def _power(byte):
    """2^(byte - 127) in fp32, from its bits."""
    return (byte.int() << 23).view(torch.float32)


def _to_codes(v):
    """Codes (one a byte, 0..15) and scale bytes of the last axis in blocks of 32: the scale is
    the smallest power of two, from 2^-125 to 2^125, that leaves the largest magnitude at most
    7 (which rounds to 6 like everything from 5 up); codes are the nearest, ties to even."""
    blocks = v.float().unflatten(-1, (-1, 32))
    largest = blocks.abs().amax(-1)
    m, e = torch.frexp(largest)
    byte = torch.where(largest == 0, 2, (e - 3 + (m > 0.875).int() + 127).clamp(2, 252))
    u = blocks * _power(254 - byte)[..., None]
    a = u.abs()
    code = torch.where(a < 2, (a * 2).round(), torch.where(a < 4, a.round() + 2, (a / 2).round() + 4)).clamp(max=7)
    fine = torch.isfinite(largest)
    code = torch.where(fine[..., None], code, 0.0).to(torch.uint8) + (torch.signbit(u) & fine[..., None]).to(torch.uint8) * 8
    return code.flatten(-2), torch.where(fine, byte, 255).to(torch.uint8)


def _packed(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _values(codes, scales):
    """fp32 values of packed codes [..., d / 2] and scale bytes [..., d / 32]."""
    both = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)
    levels = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=codes.device)
    power = torch.where(scales == 255, math.nan, _power(scales))
    return (levels[both.int()].unflatten(-1, (-1, 32)) * power[..., None]).flatten(-2)


def _cache_parts(cache, page, d):
    """Views of a cache: codes [pages, 2, kv, page, d / 2] and scales [pages, 2, kv, d / 32, page]."""
    return (cache[..., :page * (d // 2)].unflatten(-1, (page, d // 2)),
            cache[..., page * (d // 2):].unflatten(-1, (d // 32, page)))


def _plain_norm(s):
    x, w = s["x"].double(), s["weight"].double()
    if s["residual"] is not None:
        s["sum"].copy_((s["x"].float() + s["residual"].float()).bfloat16())
        x = s["sum"].double()
    # in 64 bits: values next to a border between two of 8 bits
    v = x * w / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
    if s["y"] is not None:
        s["y"].copy_(v)
    g = v.unflatten(-1, (s["scales"].shape[1], -1))
    s["scales"].copy_((g.abs().amax(-1) / 448).float().clamp(min=2.0 ** -126))
    s["y8"].copy_((g / s["scales"].double()[..., None]).flatten(-2).clamp(-448, 448).float())


def _rotated(x, rope, interleaved):
    """x [tokens, heads, d] in 64 bits with its first rot_dim elements turned by rope's angles."""
    half = rope.shape[1] // 2
    cos, sin = rope[:, None, :half].double(), rope[:, None, half:].double()
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    turned = (a * cos - b * sin, b * cos + a * sin)
    turned = torch.stack(turned, dim=-1).flatten(-2) if interleaved else torch.cat(turned, dim=-1)
    return torch.cat([turned, rest], dim=-1)


def _plain_append(s):
    (t, hq, d), kv, page = s["q_out"].shape, s["cache"].shape[2], s["page"]
    q, k, v = s["qkv"].view(t, hq + 2 * kv, d).split([hq, kv, kv], dim=1)
    rope = s["rope"][s["positions"]]
    s["q_out"].copy_(_rotated(q.double(), rope, s["interleaved"]))
    k = _rotated(k.double(), rope, s["interleaved"]).float()
    kept = s["slots"] >= 0
    at = torch.where(kept, s["slots"], 0)  # a token without a place leaves page 0 as it is
    codes, scales = _cache_parts(s["cache"], page, d)
    new, scale = _to_codes(torch.stack([k, v.float()], dim=1))
    keep = kept[:, None, None, None]
    codes[at // page, :, :, at % page] = torch.where(keep, _packed(new), codes[at // page, :, :, at % page])
    scales[at // page, :, :, :, at % page] = torch.where(keep, scale, scales[at // page, :, :, :, at % page])
    held = _values(codes[at // page, :, :, at % page], scales[at // page, :, :, :, at % page])
    held = torch.where(keep, held, 0.0)
    s["k_out"].copy_(held[:, 0])
    s["v_out"].copy_(held[:, 1])


def _plain_attention(s):
    (n, hq, d), kv, page = s["q"].shape, s["cache"].shape[2], s["page"]
    codes, scales = _cache_parts(s["cache"], page, d)
    table = s["table"].long()
    start, lens, q_max = s["start"].long(), s["lens"].long(), s["q_max"]
    b, longest = table.shape[0], table.shape[1] * page

    def gathered(part):  # [sequences, kv, longest, d]
        held = _values(codes[table, part], scales[table, part].transpose(-1, -2))
        return held.transpose(1, 2).flatten(2, 3)

    queries = (start[1:] - start[:-1])[:, None]
    row = torch.arange(q_max, device=start.device)
    q = s["q"].float()[(start[:-1, None] + row).clamp(max=n - 1)].view(b, q_max, kv, hq // kv, d)
    q = q.permute(0, 2, 1, 3, 4).flatten(2, 3)
    place = lens[:, None] - queries + row  # the place of each query in its sequence
    key = torch.arange(longest, device=start.device)
    seen = (key <= place[..., None]) & (key < lens[:, None, None])
    if s["window"]:
        seen = seen & (key > place[..., None] - s["window"])
    seen = seen.repeat_interleave(hq // kv, dim=1)[:, None]
    score = torch.matmul(q, gathered(0).transpose(-1, -2)) * s["scale"]
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - torch.where(top == -math.inf, 0.0, top)).exp()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, gathered(1)) / torch.where(total == 0, 1.0, total)
    out = out.unflatten(2, (q_max, hq // kv)).permute(0, 2, 1, 3, 4).reshape(b, q_max, hq, d)
    token = torch.arange(n, device=start.device)
    seq = torch.searchsorted(start[1:], token, right=True)
    s["out"].copy_(out[seq, token - start[seq]])


def _run_own(s):
    import segmented_rank_gemm_amd as srg
    if s["op"] == "norm":
        srg.lora_rms_norm(s["x"], s["weight"], EPS, residual=s["residual"], residual_out=s["sum"],
                          y=s["y"], y8=s["y8"], scales=s["scales"])
    elif s["op"] == "append":
        srg.lora_kv_append(s["qkv"], s["positions"], s["slots"], s["rope"], s["cache"], s["q_out"],
                           interleaved=s["interleaved"])
        srg.lora_kv_read(s["slots"], s["cache"], s["k_out"], s["v_out"])
    else:
        srg.lora_kv_attention(s["q"], s["start"], s["lens"], s["table"], s["cache"], s["out"], s["scale"],
                              s["workspace"], s["q_max"], window=s["window"])


OUTPUTS = {"norm": ("sum", "y", "y8", "scales"), "append": ("q_out", "k_out", "v_out"), "attention": ("out",)}


def run(s):
    if own:
        _run_own(s)
    else:
        {"norm": _plain_norm, "append": _plain_append, "attention": _plain_attention}[s["op"]](s)
    return [s[k] for k in OUTPUTS[s["op"]]]


# --------------------------------------------------------------------------
# The definitions in 64 bits.
# --------------------------------------------------------------------------
def _exact_norm(s):
    total = s["x"].double()
    if s["residual"] is not None:
        total = total + s["residual"].double()
    h = total.bfloat16().double()  # what the next layer reads is what is normalised
    y = h / torch.sqrt((h * h).sum(-1, keepdim=True) / h.shape[1] + EPS) * s["weight"].double()
    n = s["scales"].shape[1]
    scale = y.view(len(y), n, -1).abs().max(-1).values / 448
    y8 = (y.view(len(y), n, -1) / scale[..., None].float().double()).view_as(y)
    return [total if s["residual"] is not None else None, y if s["y"] is not None else None, y8, scale]


def _exact_held(v):
    """What the cache holds for v: the nearest of the scaled levels, ties to the even code."""
    blocks = v.reshape(-1, 32)
    powers = 2.0 ** torch.arange(-125, 126, dtype=torch.float64, device=v.device)
    largest = blocks.abs().max(-1).values
    power = powers[torch.searchsorted(7 * powers, largest).clamp(max=250)][:, None]
    levels = torch.tensor(LEVELS, dtype=torch.float64, device=v.device)
    middles = ((levels[1:] + levels[:-1]) / 2).contiguous()
    low = torch.searchsorted(middles, blocks.abs() / power)               # ties down
    high = torch.searchsorted(middles, blocks.abs() / power, right=True)  # ties up
    code = torch.where(low % 2 == 0, low, high)
    return (torch.sign(blocks) * levels[code] * power).view_as(v)


def _exact_append(s):
    (t, hq, d), kv = s["q_out"].shape, s["cache"].shape[2]
    x = s["qkv"].double().view(t, hq + 2 * kv, d)
    angles = s["rope"].double()[s["positions"]]
    half = angles.shape[1] // 2
    turn = torch.complex(angles[:, :half], angles[:, half:])[:, None]
    first = torch.arange(half, device=x.device) * (2 if s["interleaved"] else 1)
    second = first + (1 if s["interleaved"] else half)
    a, b = x[:, :hq + kv, first], x[:, :hq + kv, second]
    turned = x.clone()
    turned[:, :hq + kv, first] = a * turn.real - b * turn.imag
    turned[:, :hq + kv, second] = b * turn.real + a * turn.imag
    kept = (s["slots"] >= 0).double()[:, None, None]
    k = turned[:, hq:hq + kv].float().double()  # 32 bits, then 4
    return [turned[:, :hq], _exact_held(k) * kept, _exact_held(x[:, hq + kv:]) * kept]


def _exact_attention(s):
    (n, hq, d), kv, page = s["q"].shape, s["cache"].shape[2], s["page"]
    levels = list(LEVELS) + [-x for x in LEVELS]
    even, odd = (torch.tensor([levels[b >> s & 15] for b in range(256)], dtype=torch.float64, device=DEVICE) for s in (0, 4))
    out = torch.zeros(n, hq, d, dtype=torch.float64, device=DEVICE)
    start, lens = s["start"].tolist(), s["lens"].tolist()
    for i, length in enumerate(lens):
        rows, kept = start[i + 1] - start[i], -(-length // page)
        if not length:
            continue
        held = s["cache"][s["table"][i, :kept].long()]
        codes = held[..., :page * d // 2].reshape(kept, 2, kv, page, d // 2)
        power = torch.exp2(held[..., page * d // 2:].reshape(kept, 2, kv, d // 32, page).double() - 127)
        full = torch.stack([even[codes.int()], odd[codes.int()]], dim=-1)
        full = full.reshape(kept, 2, kv, page, d // 32, 32) * power.transpose(-1, -2)[..., None]
        full = full.reshape(kept, 2, kv, page, d).permute(1, 2, 0, 3, 4).reshape(2, kv, -1, d)[:, :, :length]
        place = torch.arange(length - rows, length, device=DEVICE)[:, None]
        key = torch.arange(length, device=DEVICE)
        hidden = key > place
        if s["window"]:
            hidden |= key <= place - s["window"]
        blind = hidden.all(1)
        for h in range(kv):
            q = s["q"][start[i]:start[i + 1], h * (hq // kv):(h + 1) * (hq // kv)].double()
            score = (q @ full[0, h].T.contiguous() * s["scale"]).masked_fill(hidden[:, None], -math.inf)
            e = torch.exp(score - score.max(-1, keepdim=True).values).masked_fill(blind[:, None, None], 0.0)
            mean = e @ full[1, h] / e.sum(-1, keepdim=True).masked_fill(blind[:, None, None], 1.0)
            out[start[i]:start[i + 1], h * (hq // kv):(h + 1) * (hq // kv)] = mean
    return [out]


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "attention": _exact_attention}[case["op"]](s)
