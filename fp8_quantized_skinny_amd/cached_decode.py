"""Decoding over the 4-bit cache: one attention layer and an lm_head, every operator of kv4.py in its place.

    python -m fp8_quantized_skinny_amd.cached_decode [--tokens 256] [--budget 128] [--window 0]

A step takes M = streams * rows activations through
    qkv GEMM -> kv4_append -> kv4_attention -> kv4_attention_weights -> o_proj GEMM
    -> lm_head GEMM -> lm_head_logprobs
with the GEMMs on NVFP4 weights, and continues every stream with its most probable token.  With more
than one row a step also takes the rows - 1 tokens that follow it, given from outside (a template or a
grammar forces them; random here), so that no token of a stream goes into the cache twice.  A cache
that a step would fill past its budget is cut first (kv4_evict) to the slots with the most
accumulated weight, into a second pool of pages; the two pools take turns.

With --window a decode with positions, in a cache that keeps all tokens: prompts of different lengths go through
    qkv GEMM -> qk_norm_rope -> kv4_append -> kv4_attention_chunk
and their streams' steps through qk_norm_rope and kv4_attention_window in the place of what cuts the cache.

Synthetic weights; there is no MLP, and no norm but that of the heads, which the calls here have no part in.
"""

import argparse

import numpy as np
import torch

from . import (OP_NVFP4, kv4_append, kv4_attention, kv4_attention_chunk, kv4_attention_chunk_workspace_bytes, kv4_attention_weights,
               kv4_attention_window, kv4_attention_window_workspace_bytes, kv4_attention_workspace_bytes, kv4_evict, lm_head_logprobs,
               lm_head_logprobs_workspace_bytes, new_workspace, nvfp4_gemm, qk_norm_rope, rope_inv_freq, workspace_bytes)
from . import workload
from .kv4 import PAGE

ROWS = 8  # of a GEMM call, at most


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


class WindowDecoder:
    """streams sequences (at most 8) of up to `room` tokens, whose rows see the last `window` tokens and the first `sinks`."""

    def __init__(self, streams=2, hidden=512, Hq=8, Hk=2, D=64, rot=64, vocab=1000, room=1024, window=256, sinks=4, alternatives=5, seed=0):
        self.B, self.Hq, self.Hk, self.D, self.hidden, self.vocab = streams, Hq, Hk, D, hidden, vocab
        self.room, self.window, self.sinks = room, window, sinks
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        weights = lambda K, N, s: dev(workload.nvfp4_case(1, K, N, seed=s)["blob"])  # noqa: E731
        self.qkv_width = (Hq + 2 * Hk) * D
        self.w_qkv, self.w_o, self.w_head = weights(hidden, self.qkv_width, seed), weights(Hq * D, hidden, seed + 1), weights(hidden, vocab, seed + 2)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.embedding = (torch.randn((vocab, hidden), generator=g, device="cuda") * 0.5).half()
        self.q_weight, self.k_weight = (1.0 + 0.1 * torch.randn((2, D), generator=g, device="cuda")).unbind()
        self.inv_freq = dev(rope_inv_freq(rot))
        self.width = -(-room // PAGE)
        self.cache = torch.zeros((streams * self.width, Hk, 72 * D), dtype=torch.uint8, device="cuda")
        self.table = torch.randperm(streams * self.width, generator=g, device="cuda").to(torch.int32).reshape(streams, self.width)
        self.longest = 0
        self.lens = torch.zeros(streams, dtype=torch.int32, device="cuda")
        self.tokens = torch.zeros((streams, 1), dtype=torch.int32, device="cuda")  # that follow the last rows, not in the cache yet
        empty = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
        self.qkv, self.y = empty(streams, self.qkv_width, dtype=torch.float16), empty(streams, hidden, dtype=torch.float16)
        self.logits, self.out = empty(streams, vocab, dtype=torch.float16), empty(streams, 1, Hq, D, dtype=torch.float16)
        self.logprob, self.entropy = empty(streams), empty(streams)
        self.top_ids, self.top_logprobs = empty(streams, alternatives, dtype=torch.int32), empty(streams, alternatives)
        self.workspace = new_workspace(max(
            1, *(workspace_bytes(OP_NVFP4, m, K, N) for m in range(1, ROWS + 1)
                 for K, N in ((hidden, self.qkv_width), (Hq * D, hidden), (hidden, vocab))),
            kv4_attention_window_workspace_bytes(streams, 1, Hq, Hk, D, self.width, window, sinks),
            lm_head_logprobs_workspace_bytes(streams, vocab, alternatives)))

    def heads(self, qkv):
        """Queries, keys and values in a qkv GEMM's output."""
        h = qkv.unflatten(-1, (self.Hq + 2 * self.Hk, self.D))
        return h[..., :self.Hq, :], h[..., self.Hq:self.Hq + self.Hk, :], h[..., self.Hq + self.Hk:, :]

    def rotate(self, q, k, positions):
        qk_norm_rope(q, k, positions, self.inv_freq, q, k, q_weight=self.q_weight, k_weight=self.k_weight)

    def follow(self, x, out):
        """The tokens that follow rows x with attention `out`, and their log probabilities."""
        nvfp4_gemm(self.w_o, out.reshape(self.B, self.Hq * self.D), self.y, workspace=self.workspace)
        nvfp4_gemm(self.w_head, x + self.y, self.logits, workspace=self.workspace)
        self.tokens = self.logits.argmax(-1, keepdim=True).to(torch.int32)
        lm_head_logprobs(self.logits, self.tokens.flatten(), self.logprob, self.entropy, self.top_ids, self.top_logprobs,
                         workspace=self.workspace)

    def prompt(self, prompts):
        """Appends a list of at least one token to each stream; returns the attention of all rows."""
        n, before = [len(p) for p in prompts], self.lens.tolist()
        if len(n) != self.B or min(n) < 1 or max(map(sum, zip(before, n))) > self.room:
            raise ValueError("a prompt of at least one token for each stream, within its room")
        i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
        ends = np.cumsum(n).tolist()
        positions = i32([before[b] + t for b in range(self.B) for t in range(n[b])])
        x = self.embedding[i32(sum(map(list, prompts), [])).long()]
        qkv = torch.empty((len(x), self.qkv_width), dtype=torch.float16, device="cuda")
        for r in range(0, len(x), ROWS):
            nvfp4_gemm(self.w_qkv, x[r:r + ROWS], qkv[r:r + ROWS], workspace=self.workspace)
        q, k, v = self.heads(qkv)
        self.rotate(q, k, positions)
        self.lens += i32(n)
        self.longest = max(map(sum, zip(before, n)))
        for b, end in enumerate(ends):
            rows = slice(end - n[b], end)
            kv4_append(self.cache, self.table[b:b + 1], self.lens[b:b + 1], k[None, rows], v[None, rows])
        out = torch.empty((len(x), self.Hq, self.D), dtype=torch.float16, device="cuda")
        need = kv4_attention_chunk_workspace_bytes(len(x), self.B, self.Hq, self.Hk, self.D, self.width, self.window, self.sinks)
        kv4_attention_chunk(q, i32([0] + ends), self.cache, self.table, self.lens, out, window=self.window, sinks=self.sinks,
                            workspace=new_workspace(need))
        last = torch.tensor(ends, device="cuda") - 1
        self.follow(x[last], out[last])
        return out

    def step(self):
        """One token of every stream."""
        if self.longest == self.room:
            raise ValueError("the streams have no room left")
        x = self.embedding[self.tokens.flatten().long()]
        nvfp4_gemm(self.w_qkv, x, self.qkv, workspace=self.workspace)
        q, k, v = self.heads(self.qkv[:, None])
        self.rotate(q, k, self.lens[:, None])  # the new token's position: as many are before it
        self.lens += 1
        self.longest += 1
        kv4_append(self.cache, self.table, self.lens, k, v)
        kv4_attention_window(q, self.cache, self.table, self.lens, self.out, self.window, self.sinks, workspace=self.workspace)
        self.follow(x, self.out)


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=256)
    p.add_argument("--budget", type=int, default=128)
    p.add_argument("--window", type=int, default=0)
    a = p.parse_args()
    if a.window:
        d = WindowDecoder(window=a.window, room=1024 + a.tokens)
        d.prompt([[i * 7 % d.vocab for i in range(n)] for n in (1000, 300)])
        total = d.logprob.clone()
        for _ in range(a.tokens):
            d.step()
            total += d.logprob
        torch.cuda.synchronize()
        print(f"{a.tokens} tokens of {d.B} streams after prompts of 1000 and 300, within a window of {d.window} and {d.sinks} first tokens; "
              f"mean log probability {(total / (a.tokens + 1)).mean().item():.4f}, last entropies {[round(e, 3) for e in d.entropy.tolist()]}")
        return
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
