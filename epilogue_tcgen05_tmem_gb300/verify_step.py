"""Example: one attention layer and the head of a decoder that verifies drafted
token trees, from the linear plans and the operators between them.

``VerifyLayer.run`` takes the drafted tokens' hidden states: the QKV
projection, the per-head norm and rotation of queries and keys with the append
to the paged cache in one launch, attention of every tree over its sequence's
cache, the output projection with the residual, the head's logits, and each
draft's log probability with the best alternatives.  Nothing is copied between
the steps: the queries, keys and values are parts of the projection's output,
and the attention's output is the next projection's input.

    python -m epilogue_tcgen05_tmem_gb300.verify_step --batch 4 --tree 13 --context 1000
"""
from __future__ import annotations

import argparse
from dataclasses import dataclass

from . import Plan, TokenLogProbs, TreeAttention, kv_append, token_logprobs


@dataclass
class Trees:
    """The drafted trees of one step: packed tokens, sequence after sequence."""
    q_start: "torch.Tensor"        # noqa: F821  int32 [batch + 1]
    context_lens: "torch.Tensor"   # noqa: F821  int32 [batch], cached places before the drafts
    block_table: "torch.Tensor"    # noqa: F821  int32 [batch, pages of a sequence]
    mask: "torch.Tensor"           # noqa: F821  int32 words [tokens, words]: the drafts that each one sees
    positions: "torch.Tensor"      # noqa: F821  int64 [tokens]: the context's length and the depth in the tree
    slots: "torch.Tensor"          # noqa: F821  int64 [tokens]: where their keys and values go


def pack_trees(parents, context_lens, block_table, page_size, max_tree, device="cuda") -> Trees:
    """``parents[b][i]``: the draft before draft i in tree b, -1 for the first.
    A draft sees its ancestors and itself."""
    import torch
    words = (max_tree + 31) // 32
    start, masks, positions, slots = [0], [], [], []
    for b, tree in enumerate(parents):
        if len(tree) > max_tree:
            raise ValueError(f"tree {b} has {len(tree)} drafts, more than max_tree={max_tree}")
        seen, depth = [], []
        for i, parent in enumerate(tree):
            if not -1 <= parent < i:
                raise ValueError(f"draft {i} of tree {b} has parent {parent}: drafts come after their parents")
            seen.append((seen[parent] if parent >= 0 else 0) | 1 << i)
            depth.append(depth[parent] + 1 if parent >= 0 else 0)
        for i, bits in enumerate(seen):
            word = [bits >> 32 * w & 0xFFFFFFFF for w in range(words)]
            masks.append([x - (1 << 32) if x >> 31 else x for x in word])
            positions.append(context_lens[b] + depth[i])
            at = context_lens[b] + i
            slots.append(block_table[b][at // page_size] * page_size + at % page_size)
        start.append(start[-1] + len(tree))
    i32 = dict(dtype=torch.int32, device=device)
    i64 = dict(dtype=torch.int64, device=device)
    return Trees(torch.tensor(start, **i32), torch.tensor(context_lens, **i32), torch.tensor(block_table, **i32),
                 torch.tensor(masks, **i32).reshape(-1, words), torch.tensor(positions, **i64), torch.tensor(slots, **i64))


class VerifyLayer:
    """Plans and weights for up to ``max_batch`` trees of up to ``max_tree``
    drafts, ``tokens`` of them a step (a linear plan is made for its rows)."""

    def __init__(self, tokens, hidden, q_heads, kv_heads, head_dim, vocab, page_size=16, max_batch=1, max_tree=1,
                 max_positions=4096, rope_base=10000.0, seed=0):
        import torch
        gen = torch.Generator(device="cuda").manual_seed(seed)
        bf16 = torch.bfloat16

        def weight(n, k):
            return (torch.randn(n, k, generator=gen, device="cuda") * k ** -0.5).to(bf16)

        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        wide = (q_heads + 2 * kv_heads) * head_dim
        self.qkv = Plan(tokens, wide, hidden)
        self.attention = TreeAttention(q_heads, kv_heads, head_dim, "bf16", page_size, max_batch, max_tree)
        self.output = Plan(tokens, hidden, q_heads * head_dim, residual=True)
        self.head = Plan(tokens, vocab, hidden)
        self.w_qkv, self.w_output, self.w_head = weight(wide, hidden), weight(hidden, q_heads * head_dim), weight(vocab, hidden)
        self.q_norm = 1 + 0.1 * weight(1, head_dim)[0]
        self.k_norm = 1 + 0.1 * weight(1, head_dim)[0]
        angle = torch.arange(max_positions, dtype=torch.float64)[:, None] * rope_base ** (
            -torch.arange(0, head_dim, 2, dtype=torch.float64) / head_dim)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        # what the steps write, kept for the next call
        self.projected = torch.empty(tokens, wide, dtype=bf16, device="cuda")
        self.attended = torch.empty(tokens, q_heads, head_dim, dtype=bf16, device="cuda")
        self.states = torch.empty(tokens, hidden, dtype=bf16, device="cuda")
        self.logits = torch.empty(tokens, vocab, dtype=bf16, device="cuda")

    def run(self, hidden, trees: Trees, k_cache, v_cache, next_tokens=None, top=4) -> TokenLogProbs:
        """hidden [tokens, hidden] of the drafts -> for each the log probability
        of next_tokens (int64 [tokens], -1: none) and the ``top`` alternatives;
        the cache [pages, page_size, kv_heads, head_dim] has the drafts' keys
        and values afterwards."""
        # the linear plans take pointers: their row count is the plan's
        like = self.states
        if hidden.shape != like.shape or hidden.dtype is not like.dtype or hidden.device != like.device or hidden.stride(1) != 1:
            raise ValueError(f"hidden must be {like.dtype} {tuple(like.shape)} on {like.device} with a contiguous last dimension: got "
                             f"{hidden.dtype} {tuple(hidden.shape)} on {hidden.device}")
        if trees.slots.shape[0] != like.shape[0]:
            raise ValueError(f"the layer's steps have {like.shape[0]} drafts, not {trees.slots.shape[0]}")
        self.qkv.run(hidden, self.w_qkv, self.projected)
        heads = self.projected.view(-1, self.q_heads + 2 * self.kv_heads, self.head_dim)
        q, k, v = heads.split([self.q_heads, self.kv_heads, self.kv_heads], 1)
        q = kv_append(k, v, k_cache, v_cache, trees.slots, q=q, cos_sin=self.cos_sin, positions=trees.positions,
                      q_weight=self.q_norm, k_weight=self.k_norm)
        self.attention.run(q, k_cache, v_cache, trees.block_table, trees.context_lens, trees.q_start, mask=trees.mask,
                           out=self.attended)
        self.output.run(self.attended.flatten(1), self.w_output, self.states, residual=hidden)
        self.head.run(self.states, self.w_head, self.logits)
        return token_logprobs(self.logits, next_tokens, top=top)


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("batch", 4), ("tree", 13), ("context", 1000), ("hidden", 2048), ("q-heads", 16), ("kv-heads", 2),
                        ("head-dim", 128), ("vocab", 32000), ("page-size", 16), ("steps", 50)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args(argv)
    import torch
    pages = -(-(a.context + a.tree) // a.page_size)
    table = torch.randperm(a.batch * pages).view(a.batch, pages).tolist()
    # a binary tree of drafts for every sequence
    parents = [[(i - 1) // 2 for i in range(a.tree)] for _ in range(a.batch)]
    trees = pack_trees(parents, [a.context] * a.batch, table, a.page_size, a.tree)
    layer = VerifyLayer(a.batch * a.tree, a.hidden, a.q_heads, a.kv_heads, a.head_dim, a.vocab, a.page_size, a.batch, a.tree,
                        max_positions=a.context + a.tree)
    cache = [torch.randn(a.batch * pages, a.page_size, a.kv_heads, a.head_dim, device="cuda").bfloat16() for _ in range(2)]
    hidden = torch.randn(a.batch * a.tree, a.hidden, device="cuda").bfloat16()
    def call():
        return layer.run(hidden, trees, *cache)

    def time(step):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        for _ in range(5):
            step()
        begin.record()
        for _ in range(a.steps):
            step()
        end.record()
        torch.cuda.synchronize()
        return begin.elapsed_time(end) / a.steps * 1e3

    calls = time(call)
    # lengths, tables, masks and slots are read on the device: a captured step
    # replays with whatever its tensors hold by then
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        best = call()
    print(f"{a.batch} trees of {a.tree} drafts after {a.context} tokens: {calls:.1f} us a step, {time(graph.replay):.1f} us as a captured graph")
    print("best next tokens of the first tree:", best.top_ids[:a.tree, 0].tolist())
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
