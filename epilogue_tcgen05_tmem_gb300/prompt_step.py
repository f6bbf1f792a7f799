"""Example: one attention layer of a decoder that takes in a step of many
requests, prompts and single tokens mixed, each with its own adapter, from the
linear plans and the operators around them.

``PromptLayer.run`` adds the last layer's output to the residual stream and
norms it into E4M3 codes for the QKV projection and 16-bit values for the
adapters beside it; the projection takes the adapters' part as its residual;
queries and keys are normed and rotated, keys and values appended to the paged
cache in one launch; every request's new tokens attend to its cache, all of it
or a sliding window and the first places; the output projection gives the next
layer's input.

    python -m epilogue_tcgen05_tmem_gb300.prompt_step --prompts 2 --length 1000 --steps-in 6 --window 512
"""
from __future__ import annotations

import argparse
from dataclasses import dataclass

from . import ChunkAttention, Plan, add_rms_norm, kv_append, lora


@dataclass
class Requests:
    """The requests of one step: their new tokens packed, one after the other."""
    q_start: "torch.Tensor"        # noqa: F821  int32 [batch + 1]
    context_lens: "torch.Tensor"   # noqa: F821  int32 [batch], places before the new tokens
    block_table: "torch.Tensor"    # noqa: F821  int32 [batch, pages of a sequence]
    adapter: "torch.Tensor"        # noqa: F821  int32 [batch], -1: none
    positions: "torch.Tensor"      # noqa: F821  int64 [tokens]
    slots: "torch.Tensor"          # noqa: F821  int64 [tokens]: where their keys and values go


def pack_requests(lengths, context_lens, block_table, adapters, page_size, max_chunk, device="cuda") -> Requests:
    """``lengths[b]`` new tokens of request b after ``context_lens[b]`` cached ones."""
    import torch
    start, positions, slots = [0], [], []
    for b, (n, ctx) in enumerate(zip(lengths, context_lens, strict=True)):
        if n > max_chunk:
            raise ValueError(f"request {b} has {n} new tokens, more than max_chunk={max_chunk}")
        if ctx + n > len(block_table[b]) * page_size:
            raise ValueError(f"request {b} has {ctx + n} tokens, more than its {len(block_table[b])} pages hold")
        for at in range(ctx, ctx + n):
            positions.append(at)
            slots.append(block_table[b][at // page_size] * page_size + at % page_size)
        start.append(start[-1] + n)
    if len(adapters) != len(lengths):
        raise ValueError(f"{len(adapters)} adapters for {len(lengths)} requests")
    i32, i64 = dict(dtype=torch.int32, device=device), dict(dtype=torch.int64, device=device)
    return Requests(torch.tensor(start, **i32), torch.tensor(context_lens, **i32), torch.tensor(block_table, **i32), torch.tensor(adapters, **i32),
                    torch.tensor(positions, **i64), torch.tensor(slots, **i64))


class PromptLayer:
    """Plans and weights for steps of ``tokens`` new tokens (a linear plan is
    made for its rows) of up to ``max_batch`` requests with up to ``max_chunk``
    each, and a bank of ``adapters`` adapters for the QKV projection."""

    def __init__(self, tokens, hidden, q_heads, kv_heads, head_dim, page_size=16, max_batch=1, max_chunk=1, rank=16, adapters=1,
                 window=0, sinks=0, max_positions=4096, rope_base=10000.0, seed=0):
        import torch
        gen = torch.Generator(device="cuda").manual_seed(seed)
        bf16 = torch.bfloat16

        def normal(*shape, scale=1.0):
            return torch.randn(shape, generator=gen, device="cuda") * scale

        self.q_heads, self.kv_heads, self.head_dim, self.window, self.sinks = q_heads, kv_heads, head_dim, window, sinks
        wide = (q_heads + 2 * kv_heads) * head_dim
        self.qkv = Plan(tokens, wide, hidden, "e4m3", "token_channel", residual=True, residual_pre_act=True)
        self.attention = ChunkAttention(q_heads, kv_heads, head_dim, "bf16", page_size, max_batch, max_chunk)
        self.output = Plan(tokens, hidden, q_heads * head_dim)
        weight = normal(wide, hidden, scale=hidden ** -0.5)
        self.s_qkv = weight.abs().amax(1) / 448.0
        self.w_qkv = (weight / self.s_qkv[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        self.w_output = normal(hidden, q_heads * head_dim, scale=(q_heads * head_dim) ** -0.5).to(bf16)
        self.lora_a = normal(adapters, rank, hidden, scale=hidden ** -0.5).to(bf16)
        self.lora_b = normal(adapters, wide, rank, scale=rank ** -0.5).to(bf16)
        self.lora_scales = 0.5 + torch.rand(adapters, generator=gen, device="cuda")
        self.norm = (1 + 0.1 * normal(hidden)).to(bf16)
        self.q_norm, self.k_norm = (1 + 0.1 * normal(head_dim)).to(bf16), (1 + 0.1 * normal(head_dim)).to(bf16)
        angle = torch.arange(max_positions, dtype=torch.float64)[:, None] * rope_base ** (
            -torch.arange(0, head_dim, 2, dtype=torch.float64) / head_dim)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        # what the steps write, kept for the next call
        self.normed = torch.empty(tokens, hidden, dtype=bf16, device="cuda")
        self.added = torch.empty(tokens, wide, dtype=bf16, device="cuda")
        self.projected = torch.empty(tokens, wide, dtype=bf16, device="cuda")
        self.attended = torch.empty(tokens, q_heads, head_dim, dtype=bf16, device="cuda")
        self.states = torch.empty(tokens, hidden, dtype=bf16, device="cuda")

    def run(self, x, residual, requests: Requests, k_cache, v_cache):
        """x [tokens, hidden] (the last layer's output) and the residual stream,
        which x is added to in place -> this layer's output, of the layer's own
        buffer.  The cache [pages, page_size, kv_heads, head_dim] has the new
        tokens' keys and values afterwards."""
        # the linear plans take pointers: their row count is the plan's
        like = self.states
        for name, t in (("x", x), ("residual", residual)):
            if t.shape != like.shape or t.dtype is not like.dtype or t.device != like.device or t.stride(1) != 1:
                raise ValueError(f"{name} must be {like.dtype} {tuple(like.shape)} on {like.device} with a contiguous last dimension: got "
                                 f"{t.dtype} {tuple(t.shape)} on {t.device}")
        if requests.slots.shape[0] != like.shape[0]:
            raise ValueError(f"the layer's steps have {like.shape[0]} tokens, not {requests.slots.shape[0]}")
        n = add_rms_norm(x, self.norm, residual, quant="e4m3", out=self.normed, sum_out=residual)
        lora(n.out, self.lora_a, self.lora_b, requests.q_start, requests.adapter, self.lora_scales, out=self.added)
        self.qkv.run(n.codes, self.w_qkv, self.projected, s_a=n.scales, s_w=self.s_qkv, residual=self.added)
        heads = self.projected.view(-1, self.q_heads + 2 * self.kv_heads, self.head_dim)
        q, k, v = heads.split([self.q_heads, self.kv_heads, self.kv_heads], 1)
        q = kv_append(k, v, k_cache, v_cache, requests.slots, q=q, cos_sin=self.cos_sin, positions=requests.positions,
                      q_weight=self.q_norm, k_weight=self.k_norm)
        self.attention.run(q, k_cache, v_cache, requests.block_table, requests.context_lens, requests.q_start, self.window, self.sinks,
                           out=self.attended)
        return self.output.run(self.attended.flatten(1), self.w_output, self.states)


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("prompts", 2), ("length", 1000), ("steps-in", 6), ("context", 2000), ("hidden", 2048), ("q-heads", 16), ("kv-heads", 2),
                        ("head-dim", 128), ("window", 0), ("sinks", 0), ("rank", 16), ("adapters", 4), ("page-size", 16), ("repeats", 50)):
        ap.add_argument(f"--{name}", type=int, default=value, help="requests with one new token each" if name == "steps-in" else None)
    a = ap.parse_args(argv)
    import torch
    batch = a.prompts + a.steps_in
    lengths = [a.length] * a.prompts + [1] * a.steps_in
    contexts = [0] * a.prompts + [a.context] * a.steps_in
    pages = -(-max(n + c for n, c in zip(lengths, contexts)) // a.page_size)
    table = torch.randperm(batch * pages).view(batch, pages).tolist()
    requests = pack_requests(lengths, contexts, table, [b % a.adapters for b in range(batch)], a.page_size, max(lengths))
    tokens = sum(lengths)
    layer = PromptLayer(tokens, a.hidden, a.q_heads, a.kv_heads, a.head_dim, a.page_size, batch, max(lengths), a.rank, a.adapters, a.window, a.sinks,
                        max_positions=pages * a.page_size)
    cache = [torch.randn(batch * pages, a.page_size, a.kv_heads, a.head_dim, device="cuda").bfloat16() for _ in range(2)]
    x, residual = (torch.randn(tokens, a.hidden, device="cuda").bfloat16() for _ in range(2))

    def call():
        return layer.run(x, residual, requests, *cache)

    def time(step):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        for _ in range(5):
            step()
        begin.record()
        for _ in range(a.repeats):
            step()
        end.record()
        torch.cuda.synchronize()
        return begin.elapsed_time(end) / a.repeats * 1e3

    calls = time(call)
    # lengths, tables, adapters and slots are read on the device: a captured
    # step replays with whatever its tensors hold by then
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    print(f"{a.prompts} prompts of {a.length} tokens and {a.steps_in} single tokens after {a.context}: {calls:.1f} us a step, "
          f"{time(graph.replay):.1f} us as a captured graph")
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
