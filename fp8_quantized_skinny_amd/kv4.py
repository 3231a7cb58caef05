"""The 4-bit key/value cache and the lm_head's log probabilities: Python binding.

The functions have the names of the C ABI in include/skinny.h, which documents
layouts and values; here device buffers are torch tensors and their sizes are
checked (csrc/binding.cpp).  Every call runs in the HIP kernels of libskinny.so.
stream: a torch stream, a raw handle, or None for torch's current stream.

    cache  uint8 [pages, Hk, 72 * D]     one page holds 64 tokens
    table  int32 [B, width]              the pages of each sequence
    lens   int32 [B]                     slots of each sequence, the step's own tokens among them
"""

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
