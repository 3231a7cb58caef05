"""Decoding over the 4-bit cache: one attention layer and an lm_head, every operator of kv4.py in its place.

    python -m fp8_quantized_skinny_amd.cached_decode [--tokens 256] [--budget 128]

A step takes M = streams * rows activations through
    qkv GEMM -> kv4_append -> kv4_attention -> kv4_attention_weights -> o_proj GEMM
    -> lm_head GEMM -> lm_head_logprobs
with the GEMMs on NVFP4 weights, and continues every stream with its most probable token.  With more
than one row a step also takes the rows - 1 tokens that follow it, given from outside (a template or a
grammar forces them; random here), so that no token of a stream goes into the cache twice.  A cache
that a step would fill past its budget is cut first (kv4_evict) to the slots with the most
accumulated weight, into a second pool of pages; the two pools take turns.

Synthetic weights; there are no positions, norms or MLP, which the calls here have no part in.
"""

import argparse

import numpy as np
import torch

from . import (OP_NVFP4, kv4_append, kv4_attention, kv4_attention_weights, kv4_attention_workspace_bytes, kv4_evict,
               lm_head_logprobs, lm_head_logprobs_workspace_bytes, new_workspace, nvfp4_gemm, workspace_bytes)
from . import workload
from .kv4 import PAGE


class CachedDecoder:
    """streams sequences; every step adds `rows` tokens to each (streams * rows <= 8)."""

    def __init__(self, streams=2, rows=1, hidden=512, Hq=8, Hk=2, D=64, vocab=1000, budget=128, keep=96, sinks=4, recent=32,
                 alternatives=5, seed=0):
        self.B, self.T, self.Hq, self.Hk, self.D = streams, rows, Hq, Hk, D
        self.hidden, self.vocab, self.budget, self.keep, self.sinks, self.recent = hidden, vocab, budget, keep, sinks, recent
        if keep + rows > budget:
            raise ValueError("keep + rows must be within the budget")
        M = streams * rows
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        weights = lambda K, N, s: dev(workload.nvfp4_case(1, K, N, seed=s)["blob"])  # noqa: E731
        self.qkv_width = (Hq + 2 * Hk) * D
        self.w_qkv, self.w_o, self.w_head = weights(hidden, self.qkv_width, seed), weights(Hq * D, hidden, seed + 1), weights(hidden, vocab, seed + 2)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.embedding = (torch.randn((vocab, hidden), generator=g, device="cuda") * 0.5).half()
        # The tokens that follow the last step's rows; the last of each stream is not in the cache yet.
        self.tokens = torch.randint(0, vocab, (streams, rows), generator=g, device="cuda", dtype=torch.int32)
        self.generator = g

        width = -(-budget // PAGE)
        pages = torch.randperm(streams * width, generator=g, device="cuda").to(torch.int32).reshape(streams, width)
        empty = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
        # Two pools of pages, each with its table and accumulated weights; `now` is the one in use.
        self.pools = [torch.zeros((streams * width, Hk, 72 * D), dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.tables = [pages, pages.flip(0).contiguous()]
        self.accs = [torch.zeros((streams, Hk, PAGE * width), device="cuda") for _ in range(2)]
        self.now, self.length = 0, 0
        self.lens = torch.zeros(streams, dtype=torch.int32, device="cuda")
        self.kept, self.new_lens = empty(streams, Hk, keep, dtype=torch.int32), torch.empty_like(self.lens)
        self.qkv, self.y = empty(M, self.qkv_width, dtype=torch.float16), empty(M, hidden, dtype=torch.float16)
        self.logits, self.out = empty(M, vocab, dtype=torch.float16), empty(streams, rows, Hq, D, dtype=torch.float16)
        self.lse = empty(streams, rows, Hq)
        self.logprob, self.entropy = empty(M), empty(M)
        self.top_ids, self.top_logprobs = empty(M, alternatives, dtype=torch.int32), empty(M, alternatives)
        # One workspace serves every call: they run one after another.
        self.workspace = new_workspace(max(
            1, *(workspace_bytes(OP_NVFP4, M, K, N) for K, N in ((hidden, self.qkv_width), (Hq * D, hidden), (hidden, vocab))),
            kv4_attention_workspace_bytes(streams, rows, Hq, Hk, D, width), lm_head_logprobs_workspace_bytes(M, vocab, alternatives)))

    def cache(self):
        """Cache, table and lengths as the calls take them."""
        return self.pools[self.now], self.tables[self.now], self.lens

    def evict(self):
        """Cuts every stream to `keep` slots."""
        to = 1 - self.now
        kv4_evict(*self.cache(), self.accs[self.now], self.pools[to], self.tables[to], self.kept, self.new_lens, self.accs[to],
                  sinks=self.sinks, recent=self.recent)
        self.now = to
        self.lens.copy_(self.new_lens)
        self.length = self.keep

    def step(self):
        """One step; True if the caches were cut before it."""
        B, T, Hq, Hk, D, ws = self.B, self.T, self.Hq, self.Hk, self.D, self.workspace
        cut = self.length + T > self.budget
        if cut:
            self.evict()
        fed = self.tokens[:, -1:]
        if T > 1:
            forced = torch.randint(0, self.vocab, (B, T - 1), generator=self.generator, device="cuda", dtype=torch.int32)
            fed = torch.cat((fed, forced), 1)
        x = self.embedding[fed.flatten().long()]
        nvfp4_gemm(self.w_qkv, x, self.qkv, workspace=ws)
        heads = self.qkv.view(B, T, Hq + 2 * Hk, D)
        q, k, v = heads[:, :, :Hq], heads[:, :, Hq:Hq + Hk], heads[:, :, Hq + Hk:]
        self.lens += T
        self.length += T
        kv4_append(*self.cache(), k, v)
        kv4_attention(q, *self.cache(), self.out, lse=self.lse, workspace=ws)
        acc = self.accs[self.now]
        kv4_attention_weights(q, *self.cache(), self.lse, acc, acc)
        nvfp4_gemm(self.w_o, self.out.view(B * T, Hq * D), self.y, workspace=ws)
        nvfp4_gemm(self.w_head, x + self.y, self.logits, workspace=ws)
        # The log probability of the token that follows each row: for the rows before a
        # stream's last that is the next row's; the last is continued greedily.
        best = self.logits.view(B, T, -1)[:, -1].argmax(-1).to(torch.int32)
        following = torch.cat((fed[:, 1:], best[:, None]), 1)
        lm_head_logprobs(self.logits, following.flatten(), self.logprob, self.entropy, self.top_ids, self.top_logprobs, workspace=ws)
        self.tokens = following
        return cut


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=256)
    p.add_argument("--budget", type=int, default=128)
    a = p.parse_args()
    d = CachedDecoder(budget=a.budget, keep=a.budget * 3 // 4, recent=a.budget // 4)
    total, cuts = 0.0, 0
    for _ in range(a.tokens):
        cuts += d.step()
        total += d.logprob
    torch.cuda.synchronize()
    print(f"{a.tokens} tokens of {d.B} streams, cut {cuts} times to {d.keep} slots; "
          f"mean log probability {(total / a.tokens).mean().item():.4f}, last entropies {[round(e, 3) for e in d.entropy.tolist()]}")


if __name__ == "__main__":
    main()
