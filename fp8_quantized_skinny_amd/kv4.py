"""The 4-bit key/value cache and the lm_head's log probabilities: Python binding.

The functions have the names of the C ABI in include/skinny.h, which documents
layouts and values; here device buffers are torch tensors and their sizes are
checked.  Every call runs in the HIP kernels of libskinny.so.

    cache  uint8 [pages, Hk, 72 * D]     one page holds 64 tokens
    table  int32 [B, width]              the pages of each sequence
    lens   int32 [B]                     slots of each sequence, the step's own tokens among them
"""

import struct

from ._lib import lib

PAGE = 64
MAX_TOP = 32

_CACHE = struct.Struct("=QQQiiiiiff4x").pack    # kv4_cache
_ROWS = struct.Struct("=Qqqq").pack             # kv4_rows
_TYPES = {}
_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TYPES.update({torch.float16: 0, torch.bfloat16: 1, torch.float32: 2})
        _TORCH = torch
    return _TORCH


def _is_tensor(t, name):
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a CUDA (HIP) torch tensor")


def _device(t, name, device):
    if t.get_device() == device:
        return
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) torch tensor")
    raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{device}")


def _buffer(t, dtype, shape, name, device):
    """The address of a contiguous device tensor of exactly this type and shape."""
    if (isinstance(t, _torch().Tensor) and t.get_device() == device and t.dtype is dtype and t.shape == shape
            and t.is_contiguous()):
        return t.data_ptr()
    _is_tensor(t, name)
    _device(t, name, device)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _rows(t, name, device):
    """kv4_rows of a [B, T, heads, D] view; the C call checks pointer and strides."""
    _is_tensor(t, name)
    _device(t, name, device)
    if t.dtype not in _TYPES or t.dim() != 4:
        raise TypeError(f"{name} must be float16 or bfloat16 [B, T, heads, D]")
    B, T, H, D = t.shape
    if B < 1 or T < 1 or H < 1:
        raise ValueError(f"{name} is empty")
    sb, st, sh, sd = t.stride()
    if sd != 1 and D > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    # A dimension of one entry may have any stride.
    return _ROWS(t.data_ptr(), sb if B > 1 else 0, st if T > 1 else 0, sh if H > 1 else 0)


def _cache(cache, table, lens, gk, gv, torch, device, names=("cache", "table", "lens")):
    """(kv4_cache, B, Hk, D, width)."""
    _is_tensor(cache, names[0])
    _is_tensor(table, names[1])
    if cache.dim() != 3 or cache.shape[2] % 72:
        raise ValueError(f"{names[0]} must be uint8 [pages, Hk, 72 * D]")
    if table.dim() != 2:
        raise ValueError(f"{names[1]} must be int32 [B, width]")
    pages, Hk, block = cache.shape
    B, width = table.shape
    D = block // 72
    c = _buffer(cache, torch.uint8, cache.shape, names[0], device)
    t = _buffer(table, torch.int32, table.shape, names[1], device)
    n = 0 if lens is None else _buffer(lens, torch.int32, (B,), names[2], device)
    return _CACHE(c, t, n, pages, width, B, Hk, D, gk, gv), B, Hk, D, width


def _stream(torch, stream):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())  # current_stream() builds an object
    return stream if isinstance(stream, int) else stream.cuda_stream


def _status(status, where):
    if status:
        from . import SkinnyError
        raise SkinnyError(status, where)


def _scratch(workspace, need, torch, where, device):
    if workspace is None:
        if need:
            raise ValueError(f"{where}: a workspace of at least {need} bytes is required")
        return None, 0
    _is_tensor(workspace, "workspace")
    if workspace.numel() < need:
        raise ValueError(f"{where}: a workspace of at least {need} bytes is required")
    return _buffer(workspace, torch.uint8, workspace.shape, "workspace", device), workspace.numel()


def _kv_shape(t, name, B, T, Hk, D):
    if t.shape != (B, T, Hk, D):
        raise ValueError(f"{name} must be [B, T, Hk, D] = {[B, T, Hk, D]}, got {list(t.shape)}")


def kv4_append(cache, table, lens, k, v, gk=1.0, gv=1.0, stream=None):
    """Quantizes k and v (fp16 or bf16 [B, T, Hk, D], views allowed) into the newest T slots of each
    sequence: row t goes to slot lens - T + t, and is dropped where that is negative."""
    torch = _torch()
    device = torch.cuda.current_device()
    c, B, Hk, D, _ = _cache(cache, table, lens, gk, gv, torch, device)
    kr, vr = _rows(k, "k", device), _rows(v, "v", device)
    T = k.shape[1]
    _kv_shape(k, "k", B, T, Hk, D)
    _kv_shape(v, "v", B, T, Hk, D)
    if k.dtype is not v.dtype:
        raise TypeError("k and v must have one type")
    _status(lib().kv4_append(c, kr, vr, _TYPES[k.dtype], T, _stream(torch, stream)), "kv4_append")


def kv4_read(cache, table, lens, k, v, gk=1.0, gv=1.0, stream=None):
    """Writes the newest n slots as held to k and v (fp16 or bf16 [B, n, Hk, D], contiguous),
    right-aligned: row t is slot lens - n + t, zeros where that is negative."""
    torch = _torch()
    device = torch.cuda.current_device()
    c, B, Hk, D, _ = _cache(cache, table, lens, gk, gv, torch, device)
    _is_tensor(k, "k")
    if k.dim() != 4:
        raise ValueError("k must be [B, n, Hk, D]")
    n = k.shape[1]
    shape = (B, n, Hk, D)
    kp, vp = _buffer(k, k.dtype, shape, "k", device), _buffer(v, k.dtype, shape, "v", device)
    _status(lib().kv4_read(c, kp, vp, _TYPES.get(k.dtype, -1), n, _stream(torch, stream)), "kv4_read")
    return k, v


def kv4_attention_workspace_bytes(B, T, Hq, Hk, D, width):
    """Workspace bytes of kv4_attention (0: none needed, or an unsupported shape)."""
    return lib().kv4_attention_workspace_bytes(B, T, Hq, Hk, D, width)


def _queries(q, B, Hk, D, device):
    qr = _rows(q, "q", device)
    if q.shape[0] != B or q.shape[3] != D:
        raise ValueError(f"q must be [B, T, Hq, D] with B = {B}, D = {D}, got {list(q.shape)}")
    return qr, q.shape[1], q.shape[2]


def kv4_attention(q, cache, table, lens, out, lse=None, scale=None, gk=1.0, gv=1.0, workspace=None, stream=None):
    """out = softmax(scale * q . K) . V over the cache, row t of T over the first lens - (T - 1 - t) slots.

    q: fp16 or bf16 [B, T, Hq, D], T = 1..8, views allowed; out: the same shape and type, contiguous;
    lse: fp32 [B, T, Hq] or None; scale: 1 / sqrt(D) by default.
    workspace: from new_workspace(kv4_attention_workspace_bytes(...))."""
    torch = _torch()
    device = torch.cuda.current_device()
    c, B, Hk, D, width = _cache(cache, table, lens, gk, gv, torch, device)
    qr, T, Hq = _queries(q, B, Hk, D, device)
    op = _buffer(out, q.dtype, q.shape, "out", device)
    lp = None if lse is None else _buffer(lse, torch.float32, (B, T, Hq), "lse", device)
    L = lib()
    ws, wsb = _scratch(workspace, L.kv4_attention_workspace_bytes(B, T, Hq, Hk, D, width), torch, "kv4_attention", device)
    _status(L.kv4_attention(c, qr, _TYPES[q.dtype], T, Hq, D ** -0.5 if scale is None else scale, op, lp, ws, wsb,
                            _stream(torch, stream)), "kv4_attention")
    return out


def kv4_attention_weights(q, cache, table, lens, lse, acc, acc_out, scale=None, gk=1.0, stream=None):
    """acc_out = acc + the attention weights of the step's rows, per key/value head and slot.

    q, cache, table, lens, scale, gk: as given to kv4_attention; lse: its output (fp32 [B, T, Hq]);
    acc, acc_out: fp32 [B, Hk, 64 * width], possibly the same tensor."""
    torch = _torch()
    device = torch.cuda.current_device()
    c, B, Hk, D, width = _cache(cache, table, lens, gk, 1.0, torch, device)
    qr, T, Hq = _queries(q, B, Hk, D, device)
    lp = _buffer(lse, torch.float32, (B, T, Hq), "lse", device)
    shape = (B, Hk, PAGE * width)
    ap, bp = _buffer(acc, torch.float32, shape, "acc", device), _buffer(acc_out, torch.float32, shape, "acc_out", device)
    _status(lib().kv4_attention_weights(c, qr, _TYPES[q.dtype], T, Hq, D ** -0.5 if scale is None else scale, lp, ap, bp,
                                        _stream(torch, stream)), "kv4_attention_weights")
    return acc_out


def kv4_evict(cache, table, lens, acc, dst_cache, dst_table, kept, new_lens, new_acc, sinks=0, recent=0, stream=None):
    """Copies, per sequence and head, the kept.shape[2] slots with the greatest accumulated weight to the
    pages of dst_table in dst_cache (the first `sinks` and last `recent` always; ties: the lower slot).

    acc: fp32 [B, Hk, 64 * width]; kept: int32 [B, Hk, keep] (slots, -1 past the new length);
    new_lens: int32 [B]; new_acc: fp32 [B, Hk, 64 * dst width] (weights of the kept slots, then 0)."""
    torch = _torch()
    device = torch.cuda.current_device()
    c, B, Hk, D, width = _cache(cache, table, lens, 1.0, 1.0, torch, device)
    d, B2, Hk2, D2, dwidth = _cache(dst_cache, dst_table, None, 1.0, 1.0, torch, device, ("dst_cache", "dst_table", ""))
    if (B2, Hk2, D2) != (B, Hk, D):
        raise ValueError("dst_cache and dst_table must have the cache's sequences, heads and head size")
    _is_tensor(kept, "kept")
    if kept.dim() != 3:
        raise ValueError("kept must be int32 [B, Hk, keep]")
    keep = kept.shape[2]
    ap = _buffer(acc, torch.float32, (B, Hk, PAGE * width), "acc", device)
    kp = _buffer(kept, torch.int32, (B, Hk, keep), "kept", device)
    np_ = _buffer(new_lens, torch.int32, (B,), "new_lens", device)
    ap2 = _buffer(new_acc, torch.float32, (B, Hk, PAGE * dwidth), "new_acc", device)
    _status(lib().kv4_evict(c, ap, d, kp, np_, ap2, keep, sinks, recent, _stream(torch, stream)), "kv4_evict")


def lm_head_logprobs_workspace_bytes(R, V, k):
    """Workspace bytes of lm_head_logprobs (0: none needed, or an unsupported shape)."""
    return lib().lm_head_logprobs_workspace_bytes(R, V, k)


def lm_head_logprobs(logits, tokens, logprob, entropy, top_ids, top_logprobs, workspace=None, stream=None):
    """Log probabilities of tokens (int32 [R]) under logits (fp16, bf16 or fp32 [R, V], rows contiguous),
    the rows' entropies, and their k greatest logits' indices and log probabilities (ties: the lower index).

    logprob, entropy: fp32 [R]; top_ids: int32 [R, k]; top_logprobs: fp32 [R, k], k = 1..32.
    workspace: from new_workspace(lm_head_logprobs_workspace_bytes(R, V, k)) when that is > 0."""
    torch = _torch()
    device = torch.cuda.current_device()
    _is_tensor(logits, "logits")
    _is_tensor(top_ids, "top_ids")
    _device(logits, "logits", device)
    if logits.dtype not in _TYPES or logits.dim() != 2:
        raise TypeError("logits must be float16, bfloat16 or float32 [R, V]")
    R, V = logits.shape
    stride = logits.stride(0) if R > 1 else V
    if logits.stride(1) != 1 and V > 1:
        raise ValueError("the rows of logits must be contiguous")
    if top_ids.dim() != 2:
        raise ValueError("top_ids must be int32 [R, k]")
    k = top_ids.shape[1]
    f32 = torch.float32
    args = (_buffer(tokens, torch.int32, (R,), "tokens", device), _buffer(logprob, f32, (R,), "logprob", device),
            _buffer(entropy, f32, (R,), "entropy", device), _buffer(top_ids, torch.int32, (R, k), "top_ids", device),
            _buffer(top_logprobs, f32, (R, k), "top_logprobs", device))
    L = lib()
    ws, wsb = _scratch(workspace, L.lm_head_logprobs_workspace_bytes(R, V, k), torch, "lm_head_logprobs", device)
    _status(L.lm_head_logprobs(logits.data_ptr(), _TYPES[logits.dtype], stride, *args, R, V, k, ws, wsb,
                               _stream(torch, stream)), "lm_head_logprobs")
    return logprob
