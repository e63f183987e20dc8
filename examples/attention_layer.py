"""One attention layer of a served model with per-adapter low-rank weights, from the
residual stream to the heads' outputs, for a step's tokens: prompts first, then
one token a sequence.

    norm -> 8-bit base product + low-rank step over (q, k, v)
         -> rotation and append to the 4-bit paged cache -> attention over it

The low-rank step reads the norm's bf16 rows, the base product its 8-bit rows and
scales.  The decode step is captured into a HIP graph once and replayed with the
next token's inputs.  Run it from the repository's root on an MI355X:

    python examples/attention_layer.py
"""

from __future__ import annotations

import dataclasses
import os
import sys

import torch

if __package__ in (None, ""):
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import segmented_rank_gemm_amd as srg  # noqa: E402


@dataclasses.dataclass
class Config:
    hidden: int = 4096
    q_heads: int = 32
    kv_heads: int = 8
    head_dim: int = 128
    rank: int = 16
    adapters: int = 4
    page: int = 64
    pages: int = 512
    positions: int = 8192
    eps: float = 1e-5

    @property
    def slices(self):
        return [self.q_heads * self.head_dim, self.kv_heads * self.head_dim, self.kv_heads * self.head_dim]


class Layer:
    """The layer's weights and its cache."""

    def __init__(self, cfg: Config, seed: int = 0):
        self.cfg = cfg
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *shape, scale=1.0: scale * torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
        n = sum(cfg.slices)
        self.norm = (1 + 0.1 * normal(cfg.hidden)).bfloat16()
        base = normal(n, cfg.hidden, scale=cfg.hidden ** -0.5)
        self.base_scales = (base.abs().amax(1, keepdim=True) / 448).t().contiguous()
        self.base8 = (base / self.base_scales.t()).to(torch.float8_e4m3fn)
        self.lora_a = [normal(cfg.adapters, cfg.rank, cfg.hidden, scale=cfg.hidden ** -0.5).bfloat16()
                       for _ in cfg.slices]
        self.lora_b = [normal(cfg.adapters, m, cfg.rank, scale=0.3 * cfg.rank ** -0.5).bfloat16()
                       for m in cfg.slices]
        self.rope = srg.rope_table(cfg.positions, cfg.head_dim)
        self.cache = torch.zeros(srg.kv_cache_shape(cfg.pages, cfg.kv_heads, cfg.head_dim, cfg.page),
                                 dtype=torch.uint8, device="cuda")


class Step:
    """Static buffers for up to `tokens` tokens of `seqs` sequences; run() enqueues
    the layer on the current stream and can be captured into a graph."""

    def __init__(self, layer: Layer, tokens: int, seqs: int, max_query_len: int, max_pages: int):
        cfg = layer.cfg
        self.layer, self.tokens, self.max_query_len = layer, tokens, max_query_len
        new = lambda *shape, dtype=torch.bfloat16: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
        self.x, self.residual, self.h, self.y = (new(tokens, cfg.hidden) for _ in range(4))
        self.y8 = torch.empty(tokens, cfg.hidden, dtype=torch.float8_e4m3fn, device="cuda")
        self.scales = new(tokens, 1, dtype=torch.float32)
        self.qkv = new(tokens, sum(cfg.slices))
        self.q, self.out = (new(tokens, cfg.q_heads, cfg.head_dim) for _ in range(2))
        self.adapter = new(tokens, dtype=torch.int32)
        self.positions = new(tokens, dtype=torch.int32)
        self.slots = new(tokens, dtype=torch.int64)
        self.query_start = new(seqs + 1, dtype=torch.int32)
        self.seq_lens = new(seqs, dtype=torch.int32)
        self.page_table = new(seqs, max_pages, dtype=torch.int32)
        self.meta = srg.LoraMeta(tokens, cfg.adapters)
        self.splits = srg.lora_shrink_default_splits(cfg.hidden, tokens, cfg.adapters, 3, cfg.rank)
        self.buf = new(self.splits, 3, tokens, cfg.rank, dtype=torch.float32)
        self.step_workspace = srg.fused_step_workspace(tokens, cfg.adapters, 3, cfg.rank)
        self.attention_workspace = srg.kv_attention_workspace(
            seqs, max_query_len, max_pages * cfg.page, cfg.q_heads, cfg.kv_heads, cfg.head_dim)

    def run(self) -> None:
        layer, cfg = self.layer, self.layer.cfg
        srg.lora_rms_norm(self.x, layer.norm, cfg.eps, residual=self.residual, residual_out=self.h,
                          y=self.y, y8=self.y8, scales=self.scales)
        self.qkv.copy_(torch._scaled_mm(self.y8, layer.base8.t(), scale_a=self.scales,
                                        scale_b=layer.base_scales, out_dtype=torch.bfloat16))
        srg.lora_fused_step(self.adapter, self.tokens, self.y, layer.lora_a, layer.lora_b, 1.0, self.buf,
                            self.splits, self.qkv, self.meta, self.step_workspace)
        srg.lora_kv_append(self.qkv, self.positions, self.slots, layer.rope, layer.cache, self.q,
                           page_size=cfg.page)
        srg.lora_kv_attention(self.q, self.query_start, self.seq_lens, self.page_table, layer.cache, self.out,
                              cfg.head_dim ** -0.5, self.attention_workspace, self.max_query_len,
                              page_size=cfg.page)

    def place(self, before, counts, table, adapters) -> None:
        """Tokens of each sequence: counts[s] new ones behind before[s] cached ones."""
        seq = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts))
        first = torch.tensor([0] + list(counts)).cumsum(0)
        at = torch.arange(self.tokens) - first[seq] + torch.tensor(before)[seq]
        page = self.layer.cfg.page
        self.positions.copy_(at)
        self.slots.copy_(table[seq, at // page].long() * page + at % page)
        self.adapter.copy_(torch.tensor(adapters)[seq])
        self.query_start.copy_(first)
        self.seq_lens.copy_(torch.tensor(before) + torch.tensor(counts))
        self.page_table.copy_(table)


def run(cfg: Config = Config(), prompts=(200, 37, 129, 64), new_tokens: int = 4, seed: int = 0):
    """Prompts, then new_tokens decode steps through one captured graph.  Returns
    the last step with its layer and the lengths, for a caller to check."""
    layer = Layer(cfg, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    seqs = len(prompts)
    max_pages = (max(prompts) + new_tokens + cfg.page - 1) // cfg.page
    table = torch.randperm(cfg.pages)[:seqs * max_pages].view(seqs, max_pages).int()
    adapters = [s % (cfg.adapters + 1) - 1 for s in range(seqs)]  # some without an adapter
    fill = Step(layer, sum(prompts), seqs, max(prompts), max_pages)
    fill.x.normal_(generator=g), fill.residual.normal_(generator=g)
    fill.place([0] * seqs, list(prompts), table, adapters)
    fill.run()

    step = Step(layer, seqs, seqs, 1, max_pages)
    lens = list(prompts)
    step.place(lens, [1] * seqs, table, adapters)
    side = torch.cuda.Stream()  # warm the step up before its capture
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step.run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run()
    for _ in range(new_tokens):
        step.x.normal_(generator=g), step.residual.normal_(generator=g)
        step.place(lens, [1] * seqs, table, adapters)
        graph.replay()
        lens = [n + 1 for n in lens]
    torch.cuda.synchronize()
    return step, graph, lens


def main() -> None:
    step, graph, lens = run()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(100):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"{len(lens)} sequences of {min(lens)} to {max(lens)} tokens: "
          f"{start.elapsed_time(end) * 10:.1f} us a step, "
          f"|out| up to {step.out.float().abs().max().item():.3f}")


if __name__ == "__main__":
    main()
