"""The 4-bit key/value cache, the norm and rotation before it and the lm_head's log probabilities: Python binding.

The functions have the names of the C ABI in include/skinny.h, which documents
layouts and values; here device buffers are torch tensors and their sizes are
checked (csrc/binding.cpp).  Every call runs in the HIP kernels of libskinny.so.
stream: a torch stream, a raw handle, or None for torch's current stream.

    cache  uint8 [pages, Hk, 72 * D]     one page holds 64 tokens
    table  int32 [B, width]              the pages of each sequence
    lens   int32 [B]                     slots of each sequence, the step's own tokens among them
"""

import numpy as np

from ._lib import lib, native

PAGE = 64
MAX_TOP = 32


def _status(status, where):
    if status:
        from . import SkinnyError
        raise SkinnyError(status, where)


def _buffer(t, dtype, shape, name, device):
    """The address of a contiguous device tensor of exactly this type and shape.  The calls below make this check in
    the extension module itself; here it can be reached without a GPU, for tests of its refusals."""
    return native().buffer(t, dtype, tuple(shape), name, device)


def kv4_append(cache, table, lens, k, v, gk=1.0, gv=1.0, stream=None):
    """Quantizes k and v (fp16 or bf16 [B, T, Hk, D], views allowed) into the newest T slots of each
    sequence: row t goes to slot lens - T + t, and is dropped where that is negative."""
    _status(native().kv4_append(cache, table, lens, k, v, gk, gv, stream), "kv4_append")


def kv4_read(cache, table, lens, k, v, gk=1.0, gv=1.0, stream=None):
    """Writes the newest n slots as held to k and v (fp16 or bf16 [B, n, Hk, D], contiguous),
    right-aligned: row t is slot lens - n + t, zeros where that is negative."""
    _status(native().kv4_read(cache, table, lens, k, v, gk, gv, stream), "kv4_read")
    return k, v


def kv4_attention_workspace_bytes(B, T, Hq, Hk, D, width):
    """Workspace bytes of kv4_attention (0: none needed, or an unsupported shape)."""
    return lib().kv4_attention_workspace_bytes(B, T, Hq, Hk, D, width)


def kv4_attention(q, cache, table, lens, out, lse=None, scale=None, gk=1.0, gv=1.0, workspace=None, stream=None):
    """out = softmax(scale * q . K) . V over the cache, row t of T over the first lens - (T - 1 - t) slots.

    q: fp16 or bf16 [B, T, Hq, D], T = 1..8, views allowed; out: the same shape and type, contiguous;
    lse: fp32 [B, T, Hq] or None; scale: 1 / sqrt(D) by default.
    workspace: from new_workspace(kv4_attention_workspace_bytes(...))."""
    _status(native().kv4_attention(q, cache, table, lens, out, lse, scale, gk, gv, workspace, stream), "kv4_attention")
    return out


def kv4_attention_window_workspace_bytes(B, T, Hq, Hk, D, width, window, sinks=0):
    """Workspace bytes of kv4_attention_window (0: none needed, or an unsupported shape)."""
    return lib().kv4_attention_window_workspace_bytes(B, T, Hq, Hk, D, width, window, sinks)


def kv4_attention_window(q, cache, table, lens, out, window, sinks=0, lse=None, scale=None, gk=1.0, gv=1.0, workspace=None, stream=None):
    """kv4_attention within a sliding window: of its slots s < L (L = lens - (T - 1 - t)) a row sees those with
    s >= L - window and the first `sinks` of the sequence.  window 0: all of them.

    workspace: from new_workspace(kv4_attention_window_workspace_bytes(...)); the rest as kv4_attention."""
    _status(native().kv4_attention_window(q, cache, table, lens, out, window, sinks, lse, scale, gk, gv, workspace, stream),
            "kv4_attention_window")
    return out


def kv4_attention_chunk_workspace_bytes(N, B, Hq, Hk, D, width, window=0, sinks=0):
    """Workspace bytes of kv4_attention_chunk (0: none needed, or an unsupported shape)."""
    return lib().kv4_attention_chunk_workspace_bytes(N, B, Hq, Hk, D, width, window, sinks)


def kv4_attention_chunk(q, starts, cache, table, lens, out, lse=None, scale=None, window=0, sinks=0, gk=1.0, gv=1.0, workspace=None,
                        stream=None):
    """Attention of chunks of new tokens, which the cache holds already: rows starts[b] .. starts[b + 1] - 1 of q are
    sequence b's newest tokens, each over the slots up to its own (with a window, as kv4_attention_window).

    q: fp16 or bf16 [N, Hq, D], views allowed; starts: int32 [B + 1]; out: q's shape and type, contiguous;
    lse: fp32 [N, Hq] or None.  Rows that no sequence has are left as they were.
    workspace: from new_workspace(kv4_attention_chunk_workspace_bytes(...)) with the same window and sinks."""
    _status(native().kv4_attention_chunk(q, starts, cache, table, lens, out, lse, scale, window, sinks, gk, gv, workspace, stream),
            "kv4_attention_chunk")
    return out


def qk_norm_rope(q, k, positions, inv_freq, q_out, k_out, q_weight=None, k_weight=None, eps=1e-6, amplitude=1.0, interleaved=False,
                 stream=None):
    """The norm of each query and key head (over its D values, times a weight; none without weights) and the rotation of
    its first 2 * len(inv_freq) positions by the angles positions * inv_freq, in one pass.

    q, k: fp16 or bf16 [B, T, heads, D] or [N, heads, D], views allowed; positions: int32 [B, T] or [N]; inv_freq: fp32
    [rot / 2], radians per position (see rope_inv_freq); weights: fp32 [D] or None; q_out, k_out: as q and k, or q and k
    themselves; amplitude: a factor of the rotated positions.  Pairs are (i, i + rot / 2), interleaved (2 i, 2 i + 1)."""
    _status(native().qk_norm_rope(q, k, positions, inv_freq, q_out, k_out, q_weight, k_weight, eps, amplitude, interleaved, stream),
            "qk_norm_rope")
    return q_out, k_out


def rope_inv_freq(rot, base=10000.0, factor=1.0, original=0, fast=32.0, slow=1.0):
    """The frequencies of qk_norm_rope, float32 [rot / 2] (host): base ** (-2 i / rot), for contexts `factor` times those
    that a model was trained on divided by factor.  With `original`, the positions it was trained on, only the pairs that turn
    fewer than `slow` times over these are divided by all of it, those of more than `fast` turns stay, and between
    them the share falls in a straight line over the pairs' indices (YaRN: Peng et al., 2023, whose amplitude is 0.1 ln(factor) + 1)."""
    if rot < 0 or rot % 2 or not (1.0 < base < np.inf and 0.0 < factor < np.inf and 0.0 <= original < np.inf and 0.0 < slow < fast < np.inf):
        raise ValueError("rot must be even, base > 1, factor > 0, original >= 0 and fast > slow > 0, all of them finite")
    i = np.arange(rot // 2, dtype=np.float64)
    freq = base ** (-2.0 * i / max(rot, 1))
    stay = np.zeros_like(freq)
    if original:
        # The index at which a pair makes n turns over the original positions.
        at = lambda n: rot * np.log(original / (n * 2.0 * np.pi)) / (2.0 * np.log(base))  # noqa: E731
        low, high = max(np.floor(at(fast)), 0.0), min(np.ceil(at(slow)), rot - 1.0)
        stay = 1.0 - np.clip((i - low) / max(high - low, 1e-3), 0.0, 1.0)
        stay[i >= np.ceil(at(slow))] = 0.0  # also where the first pair itself makes too few turns
    return (freq * stay + freq / factor * (1.0 - stay)).astype(np.float32)


def kv4_attention_weights(q, cache, table, lens, lse, acc, acc_out, scale=None, gk=1.0, stream=None):
    """acc_out = acc + the attention weights of the step's rows, per key/value head and slot.

    q, cache, table, lens, scale, gk: as given to kv4_attention; lse: its output (fp32 [B, T, Hq]);
    acc, acc_out: fp32 [B, Hk, 64 * width], the same tensor or two that do not overlap."""
    _status(native().kv4_attention_weights(q, cache, table, lens, lse, acc, acc_out, scale, gk, stream), "kv4_attention_weights")
    return acc_out


def kv4_evict(cache, table, lens, acc, dst_cache, dst_table, kept, new_lens, new_acc, sinks=0, recent=0, stream=None):
    """Copies, per sequence and head, the kept.shape[2] slots with the greatest accumulated weight to the
    pages of dst_table in dst_cache (the first `sinks` and last `recent` always; ties: the lower slot).

    acc: fp32 [B, Hk, 64 * width]; kept: int32 [B, Hk, keep] (slots, -1 past the new length);
    new_lens: int32 [B]; new_acc: fp32 [B, Hk, 64 * dst width] (weights of the kept slots, then 0).
    No output may share memory with an input or another output (new_lens with lens, new_acc with acc,
    dst_cache with cache); cache and dst_cache may be separate ranges of pages of one tensor."""
    _status(native().kv4_evict(cache, table, lens, acc, dst_cache, dst_table, kept, new_lens, new_acc, sinks, recent, stream),
            "kv4_evict")


def lm_head_logprobs_workspace_bytes(R, V, k):
    """Workspace bytes of lm_head_logprobs (0: none needed, or an unsupported shape)."""
    return lib().lm_head_logprobs_workspace_bytes(R, V, k)


def lm_head_logprobs(logits, tokens, logprob, entropy, top_ids, top_logprobs, workspace=None, stream=None):
    """Log probabilities of tokens (int32 [R]) under logits (fp16, bf16 or fp32 [R, V], rows contiguous),
    the rows' entropies, and their k greatest logits' indices and log probabilities (ties: the lower index).

    logits begin at a multiple of 16 bytes (their rows need not).
    logprob, entropy: fp32 [R]; top_ids: int32 [R, k]; top_logprobs: fp32 [R, k], k = 1..32.
    workspace: from new_workspace(lm_head_logprobs_workspace_bytes(R, V, k)) when that is > 0."""
    _status(native().lm_head_logprobs(logits, tokens, logprob, entropy, top_ids, top_logprobs, workspace, stream),
            "lm_head_logprobs")
    return logprob
