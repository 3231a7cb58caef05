"""What is measured of the operators around the decode GEMMs: the 4-bit key/value cache
(append, read, attention, accumulated attention weights, eviction) and the log
probabilities of an lm_head's logits.

`run` computes a case in plain torch operations, or, with `own` set, through the
package's entry points.  Head shapes are those behind the qkv (K 5120, N 7168) and
o_proj (K 6144) GEMMs of the decode path, 48 query and 4 key/value heads of 128, and
other layouts with the same entry points; the vocabulary is the lm_head's (151936).

Conventions of the cache (include/skinny.h has them in full): a page holds 64 tokens;
per page and key/value head there are 72 * D bytes: K codes, K scales, V codes, V scales.
lens counts the step's own T tokens, so row t stands for slot lens - T + t.
"""

import math

import torch

own = False

PAGE = 64
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HEADS = ((48, 4, 128), (24, 4, 256), (32, 8, 128), (16, 16, 64), (8, 1, 128), (28, 4, 64), (5, 1, 256))


def listed():
    attend = dict(op="attend", weights=False, scale=0.0)
    return [
        # One stream, a few hundred tokens in: the smallest attention call, all latency.
        dict(attend, name="attend_one_token", type="f16", B=1, T=1, Hq=48, Hk=4, D=128, shortest=301, longest=301),
        # A speculative round of one stream: the target token and seven drafts over 8K of context.
        dict(attend, name="attend_verify_8k", type="f16", B=1, T=8, Hq=48, Hk=4, D=128, shortest=8197, longest=8197),
        # A server's batch with sequences of very different lengths.
        dict(attend, name="attend_ragged_batch", type="bf16", B=32, T=1, Hq=48, Hk=4, D=128, shortest=1, longest=20000),
        # Long documents, four rows a sequence: the largest cache.
        dict(attend, name="attend_long", type="f16", B=8, T=4, Hq=48, Hk=4, D=128, shortest=120000, longest=131072),
        # A verification round that also adds to the slots' accumulated weights, wide heads.
        dict(attend, name="weights_verify", type="bf16", weights=True, B=3, T=8, Hq=24, Hk=4, D=256, shortest=2000, longest=9000),
        # A batch near its cache budget, decoding one token each with the weights kept.
        dict(attend, name="weights_batch", type="f16", weights=True, B=16, T=1, Hq=48, Hk=4, D=128, shortest=30000, longest=32768),
        # The eight rows of one speculative round written to the cache and read back as held.
        dict(name="append_round", op="append", type="f16", B=1, T=8, Hk=4, D=128, shortest=777, longest=777),
        # A chunk of four prompts written to the cache; the chunk's own attention takes the values as held.
        dict(name="append_prompts", op="append", type="bf16", B=4, T=8192, Hk=4, D=128, shortest=5000, longest=9000),
        # One stream cut to its budget.
        dict(name="evict_one", op="evict", type="f16", B=1, Hk=4, D=128, shortest=4133, longest=4133, keep=1024, sinks=4, recent=128),
        # A batch of long prompts cut to a quarter before the next chunk.
        dict(name="evict_batch", op="evict", type="bf16", B=16, Hk=4, D=128, shortest=20000, longest=32768, keep=8192, sinks=64, recent=1024),
        # The rows of one speculative round: draft tokens' log probabilities and five alternatives.
        dict(name="logprobs_round", op="logprobs", type="f16", R=8, V=151936, k=5, banned=0.0),
        # A prompt scored token by token, with a part of the vocabulary banned.
        dict(name="logprobs_prompt", op="logprobs", type="bf16", R=2048, V=151936, k=20, banned=0.1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("attend", "attend", "weights", "append", "evict", "logprobs"))
    kind = rng.choice(("f16", "bf16"))
    Hq, Hk, D = rng.choice(HEADS)
    B = _log(rng, 1, 48)
    if op in ("attend", "weights"):
        T = rng.choice((1, 1, 2, 3, 4, 5, 8))
        # At most the tokens, heads and rows of the largest listed case of the kind.
        budget = (3e8 if op == "attend" else 1.5e8) / (B * Hk * D)
        longest = _log(rng, 1, max(2, int(min(131072, budget))))
        return dict(op="attend", weights=op == "weights", scale=rng.choice((0.0, 0.0, 0.11)), type=kind, B=B, T=T, Hq=Hq, Hk=Hk, D=D,
                    shortest=rng.choice((0, 1, longest // 2, longest)), longest=longest)
    if op == "append":
        T = _log(rng, 1, max(1, int(min(9000, 1.6e7 / (B * Hk * D)))))
        longest = T + _log(rng, 1, max(1, int(min(9000, 3e8 / (B * Hk * D)))))
        return dict(op="append", type=kind, B=B, T=T, Hk=Hk, D=D, shortest=rng.choice((0, T // 2, T, longest)), longest=longest)
    if op == "evict":
        longest = _log(rng, 64, max(65, int(min(32768, 2.2e8 / (B * Hk * D)))))
        keep = max(1, int(longest * rng.uniform(0.02, 0.3)))
        sinks = rng.randint(0, keep // 4)
        return dict(op="evict", type=kind, B=B, Hk=Hk, D=D, shortest=rng.choice((0, 1, longest // 2, longest)), longest=longest,
                    keep=keep, sinks=sinks, recent=rng.randint(0, keep - sinks))
    kind = rng.choice(("f16", "bf16", "f32"))
    V = rng.choice((151936, 151936, 32000, _log(rng, 40, 200001)))
    R = _log(rng, 1, max(1, min(4096, int(1.5e8 / V))))
    return dict(op="logprobs", type=kind, R=R, V=V, k=rng.randint(1, 32), banned=rng.choice((0.0, 0.1, 0.999)))


def _lens(case, g):
    """Lengths between the shortest and the longest, one of them the longest."""
    lens = torch.randint(case["shortest"], case["longest"] + 1, (case["B"],), generator=g, device="cuda", dtype=torch.int32)
    lens[int(torch.randint(0, case["B"], (1,), generator=g, device="cuda"))] = case["longest"]
    return lens


def _pages(B, width, g, spare=3):
    """A table of pages scattered over a pool of B * width + spare pages."""
    at = torch.randperm(B * width + spare, generator=g, device="cuda")[:B * width]
    return at.to(torch.int32).reshape(B, width), B * width + spare


def _cache(pages, Hk, D, g):
    """A pool of full pages: codes distributed as a normal value's over its group of 16, scales around a half."""
    edges = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 1e9]
    below = [math.erf(e / 3.3 / math.sqrt(2)) for e in edges]
    lut = torch.tensor([next(i for i in range(8) if (j % 128 + 0.5) / 128 < below[i]) + 8 * (j // 128) for j in range(256)],
                       dtype=torch.uint8, device="cuda")
    cache = torch.empty((pages, Hk, 72 * D), dtype=torch.uint8, device="cuda")
    for at in (0, 36 * D):
        low = torch.randint(0, 256, (pages, Hk, 32 * D), generator=g, device="cuda", dtype=torch.uint8)
        high = torch.randint(0, 256, (pages, Hk, 32 * D), generator=g, device="cuda", dtype=torch.uint8)
        cache[..., at:at + 32 * D] = lut[low.int()] | (lut[high.int()] << 4)
        cache[..., at + 32 * D:at + 36 * D] = torch.randint(0x2A, 0x35, (pages, Hk, 4 * D), generator=g, device="cuda", dtype=torch.uint8)
    return cache


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind = TYPES[case["type"]]
    s = dict(case=case)
    if case["op"] == "logprobs":
        R, V, k = case["R"], case["V"], case["k"]
        # Logits of a language model: a wide normal body with a few tokens far above it.
        x = torch.randn((R, V), generator=g, device="cuda") * 2.5
        peaks = torch.randint(0, V, (R, 24), generator=g, device="cuda")
        x.scatter_add_(1, peaks, torch.rand((R, 24), generator=g, device="cuda") * 14.0)
        tokens = torch.where(torch.rand((R,), generator=g, device="cuda") < 0.7, x.argmax(1), torch.randint(0, V, (R,), generator=g, device="cuda"))
        if case["banned"]:
            x.masked_fill_(torch.rand((R, V), generator=g, device="cuda") < case["banned"], float("-inf"))
        s.update(logits=x.to(kind), tokens=tokens.to(torch.int32), logprob=torch.empty(R, device="cuda"), entropy=torch.empty(R, device="cuda"),
                 top_ids=torch.empty((R, k), dtype=torch.int32, device="cuda"), top_logprobs=torch.empty((R, k), device="cuda"))
        if own:  # the scratch buffer that a program keeps; no data of the case goes there before the call
            import fp8_quantized_skinny_amd as sk
            s["workspace"] = sk.new_workspace(sk.lm_head_logprobs_workspace_bytes(R, V, k))
        return s

    B, Hk, D = case["B"], case["Hk"], case["D"]
    width = max(1, -(-case["longest"] // PAGE))
    table, pages = _pages(B, width, g)
    lens = _lens(case, g)
    s.update(table=table, lens=lens, gk=1.0, gv=0.75)
    if case["op"] == "attend":
        T, Hq = case["T"], case["Hq"]
        s["cache"] = _cache(pages, Hk, D, g)
        # The queries lie in the output of a qkv GEMM, beside that step's keys and values.
        qkv = (torch.randn((B, T, (Hq + 2 * Hk) * D), generator=g, device="cuda") * 2.0).to(kind)
        s["q"] = qkv[..., :Hq * D].unflatten(-1, (Hq, D))
        s["out"] = torch.empty((B, T, Hq, D), dtype=kind, device="cuda")
        s["lse"] = torch.empty((B, T, Hq), device="cuda")
        s["scale"] = case["scale"] or 1.0 / math.sqrt(D)
        if case["weights"]:
            s["acc"] = torch.rand((B, Hk, width * PAGE), generator=g, device="cuda").square_() * 4.0
            s["acc_out"] = torch.empty_like(s["acc"])
        if own:  # the scratch buffer that a program keeps; no data of the case goes there before the call
            import fp8_quantized_skinny_amd as sk
            s["workspace"] = sk.new_workspace(sk.kv4_attention_workspace_bytes(B, T, Hq, Hk, D, width))
    elif case["op"] == "append":
        T = case["T"]
        s["cache"] = _cache(pages, Hk, D, g)
        # Keys with a few large channels, as trained models have them; both lie in a qkv GEMM's output.
        kv = torch.randn((B, T, 2 * Hk * D), generator=g, device="cuda")
        kv[..., :Hk * D] *= 0.5 + 4.0 * torch.rand((Hk * D,), generator=g, device="cuda").pow_(6)
        kv = kv.to(kind)
        s["k"], s["v"] = kv[..., :Hk * D].unflatten(-1, (Hk, D)), kv[..., Hk * D:].unflatten(-1, (Hk, D))
        s["k_held"] = torch.empty((B, T, Hk, D), dtype=kind, device="cuda")
        s["v_held"] = torch.empty_like(s["k_held"])
    else:
        keep, dst_width = case["keep"], -(-case["keep"] // PAGE)
        s["cache"] = _cache(pages, Hk, D, g)
        s["acc"] = -torch.rand((B, Hk, width * PAGE), generator=g, device="cuda").log_()
        s["acc"] *= torch.rand((B, Hk, width * PAGE), generator=g, device="cuda") < 0.9  # slots that no row looked at tie at 0
        s["dst_table"], dst_pages = _pages(B, dst_width, g)
        s["dst_cache"] = torch.zeros((dst_pages, Hk, 72 * D), dtype=torch.uint8, device="cuda")
        s["kept"] = torch.empty((B, Hk, keep), dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.empty((B,), dtype=torch.int32, device="cuda")
        s["new_acc"] = torch.empty((B, Hk, dst_width * PAGE), device="cuda")
        s["k_held"] = torch.empty((B, keep, Hk, D), dtype=kind, device="cuda")
        s["v_held"] = torch.empty_like(s["k_held"])
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return {"attend": _attend_own, "append": _append_own, "evict": _evict_own, "logprobs": _logprobs_own}[op](s)
    return {"attend": _attend_plain, "append": _append_plain, "evict": _evict_plain, "logprobs": _logprobs_plain}[op](s)


# ---------------------------------------------------------------- the package's operators
def _attend_own(s):
    import fp8_quantized_skinny_amd as sk
    sk.kv4_attention(s["q"], s["cache"], s["table"], s["lens"], s["out"], lse=s["lse"], scale=s["scale"], gk=s["gk"], gv=s["gv"],
                     workspace=s["workspace"])
    if not s["case"]["weights"]:
        return {"out": s["out"], "lse": s["lse"]}
    sk.kv4_attention_weights(s["q"], s["cache"], s["table"], s["lens"], s["lse"], s["acc"], s["acc_out"], scale=s["scale"], gk=s["gk"])
    return {"out": s["out"], "lse": s["lse"], "acc": s["acc_out"]}


def _append_own(s):
    import fp8_quantized_skinny_amd as sk
    sk.kv4_append(s["cache"], s["table"], s["lens"], s["k"], s["v"], gk=s["gk"], gv=s["gv"])
    sk.kv4_read(s["cache"], s["table"], s["lens"], s["k_held"], s["v_held"], gk=s["gk"], gv=s["gv"])
    return {"k": s["k_held"], "v": s["v_held"]}


def _evict_own(s):
    import fp8_quantized_skinny_amd as sk
    case = s["case"]
    sk.kv4_evict(s["cache"], s["table"], s["lens"], s["acc"], s["dst_cache"], s["dst_table"], s["kept"], s["new_lens"], s["new_acc"],
                 sinks=case["sinks"], recent=case["recent"])
    sk.kv4_read(s["dst_cache"], s["dst_table"], s["new_lens"], s["k_held"], s["v_held"], gk=s["gk"], gv=s["gv"])
    return {"kept": s["kept"], "lens": s["new_lens"], "acc": s["new_acc"], "k": s["k_held"], "v": s["v_held"]}


def _logprobs_own(s):
    import fp8_quantized_skinny_amd as sk
    sk.lm_head_logprobs(s["logits"], s["tokens"], s["logprob"], s["entropy"], s["top_ids"], s["top_logprobs"], workspace=s["workspace"])
    return {"logprob": s["logprob"], "entropy": s["entropy"], "top_ids": s["top_ids"], "top_logprobs": s["top_logprobs"]}


# ---------------------------------------------------------------- plain forms
def _split(cache, D):
    """The four parts of every (page, head) block: K codes and scales, V codes and scales."""
    return cache[..., :32 * D], cache[..., 32 * D:36 * D], cache[..., 36 * D:68 * D], cache[..., 68 * D:]


def _code_values(b):
    """Bytes to the two E2M1 values of each, low nibble first, along the last axis."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=b.device)
    return torch.stack((lut[(b & 15).int()], lut[(b >> 4).int()]), -1).flatten(-2)


def _scale_values(b):
    return b.view(torch.float8_e4m3fn).float()


def _values(cache, table, D):
    """K and V [B, Hk, width * 64, D] in 32 bits, before the tensor scales."""
    kc, ks, vc, vs = _split(cache[table.clamp(min=0).long()].transpose(1, 2), D)
    lead = kc.shape[:3]
    # K codes: 16-byte pieces [D/32][4 quarters of D][16 tokens]; a quarter's bytes run over 4 tiles of 16 tokens.
    k = kc.reshape(*lead, D // 32, 4, 16, 16).permute(0, 1, 2, 4, 5, 3, 6).reshape(*lead, 4, 16, 4, D // 8)
    k = _code_values(k).permute(0, 1, 2, 5, 4, 3, 6).reshape(*lead, PAGE, D)
    # K scales: [4 quarters][16 tokens][4 tiles][D/64].
    f = ks.reshape(*lead, 4, 16, 4, D // 64).permute(0, 1, 2, 5, 4, 3, 6).reshape(*lead, PAGE, D // 16)
    k = k * _scale_values(f.contiguous()).repeat_interleave(16, -1)
    # V codes: 16-byte pieces [D/32][4 token groups][16 columns blocks]; a block's bytes run over [2][2][4] tokens.
    v = vc.reshape(*lead, D // 32, 4, 16, 16).permute(0, 1, 2, 4, 5, 3, 6).reshape(*lead, 4, 16, 4, 4, D // 32)
    v = _code_values(v).permute(0, 1, 2, 5, 3, 6, 4, 7).reshape(*lead, PAGE, D)
    # V scales: [D/16][4 token groups][2][2][4].
    f = vs.reshape(*lead, D // 16, 4, 4, 4).permute(0, 1, 2, 5, 4, 6, 3).reshape(*lead, PAGE, D // 16)
    v = v * _scale_values(f.contiguous()).repeat_interleave(16, -1)
    return k.flatten(2, 3), v.flatten(2, 3)


def _attend_plain(s):
    case = s["case"]
    B, T, Hq, Hk, D = (case[n] for n in ("B", "T", "Hq", "Hk", "D"))
    k, v = _values(s["cache"], s["table"], D)
    q = s["q"].float().reshape(B, T, Hk, Hq // Hk, D).transpose(1, 2).reshape(B, Hk, -1, D)
    x = torch.matmul(q, k.transpose(2, 3)) * (s["scale"] * s["gk"])
    limit = s["lens"][:, None] - (T - 1 - torch.arange(T, device=q.device, dtype=torch.int32))
    seen = torch.arange(k.shape[2], device=q.device) < limit.repeat_interleave(Hq // Hk, 1)[:, None, :, None]
    x = x.masked_fill(~seen, float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.masked_fill(m == float("-inf"), 0.0))
    total = p.sum(-1, keepdim=True)
    some = total.clamp(min=1e-30)
    out = torch.matmul(p, v) / some * s["gv"]
    lse = (m + torch.log(total)).squeeze(-1)
    back = lambda t: t.unflatten(2, (T, Hq // Hk)).transpose(1, 2).flatten(2, 3)  # noqa: E731
    got = {"out": back(out).to(s["out"].dtype), "lse": back(lse)}
    if case["weights"]:
        inside = torch.arange(k.shape[2], device=q.device) < s["lens"][:, None, None]
        got["acc"] = torch.where(inside, s["acc"] + (p / some).sum(2), 0.0)
    return got


def _quantize_plain(x, g):
    """x [..., D] to E2M1 values and E4M3 scales (one for 16), decided in 64 bits: no value lies beside a border by rounding."""
    w = x.double().unflatten(-1, (-1, 16))
    scale = (w.abs().amax(-1, keepdim=True) / (6.0 * g)).clamp(max=448.0)
    # E4M3 to the nearest, ties to even: multiples of 2^(e - 3), e at least -6.
    step = torch.exp2(torch.floor(torch.log2(scale.clamp(min=2.0 ** -6))).clamp(max=8.0) - 3.0)
    scale = (torch.round(scale / step) * step).clamp(max=448.0)
    unit = scale * g
    a = w.abs()
    code = (a > 0.25 * unit).int() + (a >= 0.75 * unit) + (a > 1.25 * unit) + (a >= 1.75 * unit) + (a > 2.5 * unit) + (a >= 3.5 * unit) + (a > 5.0 * unit)
    code = torch.where(scale > 0, code + 8 * torch.signbit(w), 0)
    return code.flatten(-2).to(torch.uint8), scale.squeeze(-1).float().to(torch.float8_e4m3fn).view(torch.uint8)


def _slots(s, n):
    """For the newest n slots of each sequence: whether row t has one, its page and its place in the page, [B, n]."""
    slot = s["lens"][:, None].long() - n + torch.arange(n, device="cuda")
    return slot >= 0, s["table"].gather(1, slot.clamp(min=0) // PAGE).long(), slot.clamp(min=0) % PAGE


def _append_plain(s):
    case = s["case"]
    T, Hk, D = case["T"], case["Hk"], case["D"]
    has, page, at = _slots(s, T)
    cache = s["cache"]
    heads = torch.arange(Hk, device="cuda")[None, :, None]
    page, at = page[has][:, None, None], at[has][:, None, None]
    (kc, ks), (vc, vs) = _quantize_plain(s["k"][has], s["gk"]), _quantize_plain(s["v"][has], s["gv"])
    kc, vc = kc[..., 0::2] | (kc[..., 1::2] << 4), vc[..., 0::2] | (vc[..., 1::2] << 4)
    byte, group = torch.arange(D // 2, device="cuda"), torch.arange(D // 16, device="cuda")
    # The places of a token's bytes in the block (see _values).
    f = at // 16 * (D // 8) + byte % (D // 8)
    cache[page, heads, ((f // 16 * 4 + byte // (D // 8)) * 16 + at % 16) * 16 + f % 16] = kc
    cache[page, heads, 32 * D + ((group // (D // 64) * 16 + at % 16) * 4 + at // 16) * (D // 64) + group % (D // 64)] = ks
    f = (at // 16 * 4 + at % 4) * (D // 32) + byte % (D // 32)
    cache[page, heads, 36 * D + ((f // 16 * 4 + at % 16 // 4) * 16 + byte // (D // 32)) * 16 + f % 16] = vc
    cache[page, heads, 68 * D + (group * 4 + at % 16 // 4) * 16 + at // 16 * 4 + at % 4] = vs
    return _read_plain(s, cache, s["table"], s["lens"], T)


def _read_plain(s, cache, table, lens, n):
    D = s["case"]["D"]
    k, v = _values(cache, table, D)
    has, _, _ = _slots({"lens": lens, "table": table}, n)
    slot = (lens[:, None].long() - n + torch.arange(n, device="cuda")).clamp(min=0)
    pick = lambda t, g: torch.where(has[..., None, None], (t * g).transpose(1, 2).gather(1, slot[..., None, None].expand(-1, -1, t.shape[1], D)), 0.0)  # noqa: E731
    kind = s["k_held"].dtype
    return {"k": pick(k, s["gk"]).to(kind), "v": pick(v, s["gv"]).to(kind)}


def _evict_plain(s):
    case = s["case"]
    B, Hk, D, keep = case["B"], case["Hk"], case["D"], case["keep"]
    acc, lens = s["acc"], s["lens"].long()
    slot = torch.arange(acc.shape[2], device="cuda")
    inside = slot < lens[:, None, None]
    sure = inside & ((slot < case["sinks"]) | (slot >= lens[:, None, None] - case["recent"]))
    # Weights as whole numbers of the same order, the sure ones above all, and the lowest slot first among equals.
    key = torch.where(sure, 0x7fffffff, (acc + 0.0).view(torch.int32).long())
    key = torch.where(inside, (key << 24) + (acc.shape[2] - slot), -1)
    n = min(keep, acc.shape[2])
    best = key.topk(n, dim=2).indices.sort(2).values
    # A sequence that fits keeps its slots; others have `keep` of them, in order.
    new_lens = lens.clamp(max=keep)
    has = torch.arange(n, device="cuda") < new_lens[:, None, None]
    best = torch.where(lens[:, None, None] <= keep, torch.arange(n, device="cuda"), best)
    kept = torch.full((B, Hk, keep), -1, dtype=torch.int32, device="cuda")
    kept[..., :n] = torch.where(has, best, -1).int()
    new_acc = torch.zeros_like(s["new_acc"])
    new_acc[..., :n] = torch.where(has, acc.gather(2, best), 0.0)
    k, v = _values(s["cache"], s["table"], D)
    at = best[..., None].expand(-1, -1, -1, D)
    # Rows are right-aligned: row t of `keep` is slot new_len - keep + t.
    row = torch.arange(keep, device="cuda") - keep + new_lens[:, None]
    pick = lambda t, g: torch.where((row >= 0)[:, None, :, None], (t * g).gather(2, at).gather(2, row.clamp(min=0)[:, None, :, None].expand(-1, Hk, -1, D)), 0.0)  # noqa: E731
    kind = s["k_held"].dtype
    return {"kept": kept, "lens": new_lens.int(), "acc": new_acc, "k": pick(k, s["gk"]).transpose(1, 2).to(kind), "v": pick(v, s["gv"]).transpose(1, 2).to(kind)}


def _logprobs_plain(s):
    x = s["logits"].float()
    # A row without a finite logit has nothing to draw: every probability is 0 and so is the entropy.
    m = x.amax(1, keepdim=True)
    some = m > float("-inf")
    y = x - torch.where(some, m, 0.0)
    e = torch.exp(y)
    total = torch.where(some[:, 0], e.sum(1), 1.0)
    log = torch.log(total)
    entropy = log - torch.where(e > 0, e * y, 0.0).sum(1) / total
    lse = torch.where(some, m, 0.0)[:, 0] + log
    logprob = x.gather(1, s["tokens"].long()[:, None])[:, 0] - lse
    # Whole numbers that order like the logits, the lower index first among equals.
    bits = (x + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7fffffff), bits) * (1 << 18) + ((1 << 18) - 1 - torch.arange(x.shape[1], device="cuda"))
    ids = key.topk(s["case"]["k"], dim=1).indices
    return {"logprob": logprob, "entropy": entropy, "top_ids": ids.int(), "top_logprobs": x.gather(1, ids) - lse[:, None]}


def work(case):
    op = case["op"]
    if op == "logprobs":
        R, V = case["R"], case["V"]
        return {"bytes": R * V * (4 if case["type"] == "f32" else 2) + R * (12 + 8 * case["k"]), "flops": 6 * R * V}
    mean = case["longest"] if case["B"] == 1 else ((case["shortest"] + case["longest"]) * (case["B"] - 1) / 2 + case["longest"]) / case["B"]
    heads = case["B"] * case["Hk"]
    if op == "attend":
        rows = case["B"] * case["T"] * case["Hq"]
        return {"bytes": mean * heads * (case["D"] * 1.125 + 8 * case["weights"]) + rows * (4 * case["D"] + 4),
                "flops": 4 * rows * mean * case["D"]}
    if op == "append":
        return {"bytes": heads * case["T"] * case["D"] * (4 + 1.125 + 4), "flops": 2 * 8 * heads * case["T"] * case["D"]}
    kept = min(case["keep"], mean)
    return {"bytes": heads * (4 * mean + kept * (8 + case["D"] * (2 * 1.125 + 4))), "flops": heads * mean}


# ---------------------------------------------------------------- from the definitions, in 64 bits
def _exact_block(block, D):
    """K and V [64, D] of (page, head) blocks [..., 72 * D], by each value's own place in the block."""
    t, d = torch.arange(PAGE, device="cuda")[:, None], torch.arange(D, device="cuda")[None, :]

    def held(code_at, nibble, scale_at):
        c = (block[..., code_at].int() >> (4 * nibble)) & 15
        mant, ex = (c & 1).double(), ((c >> 1) & 3).double()
        mag = torch.where(ex == 0, mant / 2, (1 + mant / 2) * torch.exp2(ex - 1))
        f = block[..., scale_at].int()
        mant, ex = (f & 7).double(), ((f >> 3) & 15).double()
        scale = torch.where(ex == 0, mant / 512, (1 + mant / 8) * torch.exp2(ex - 7))
        return torch.where(c >= 8, -mag, mag) * scale

    quarter, inside = d // (D // 4), d % (D // 4)
    run = (t // 16) * (D // 8) + inside // 2
    k = held((run // 16) * 1024 + quarter * 256 + (t % 16) * 16 + run % 16, inside % 2,
             32 * D + (quarter * 16 + t % 16) * (D // 16) + (t // 16) * (D // 64) + inside // 16)
    column, inside = d // (D // 16), d % (D // 16)
    order = t // 16 * 4 + t % 4
    run = order * (D // 32) + inside // 2
    v = held(36 * D + (run // 16) * 1024 + (t % 16 // 4) * 256 + column * 16 + run % 16, inside % 2,
             68 * D + (d // 16) * 64 + (t % 16 // 4) * 16 + order)
    return k, v


def _exact_cache(s, cache, table, b, n, D):
    """K and V [Hk, n, D] of the first n slots of sequence b."""
    k, v = _exact_block(cache[table[b, :-(-n // PAGE)].long()], D)
    return tuple(a.transpose(0, 1).flatten(1, 2)[:, :n] * g for a, g in ((k, s["gk"]), (v, s["gv"])))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        got = {"logprob": [], "entropy": [], "top_ids": [], "top_logprobs": []}
        for x, token in zip(s["logits"], s["tokens"].long()):
            x = x.double()
            lp = x - torch.logsumexp(x, 0).clamp(min=-1e300)
            order = torch.sort(x, descending=True, stable=True).indices[:case["k"]]
            got["logprob"].append(lp[token])
            got["entropy"].append(-torch.special.xlogy(lp.exp(), lp.exp()).sum())
            got["top_ids"].append(order.int())
            got["top_logprobs"].append(lp[order])
        return {n: torch.stack(v) for n, v in got.items()}
    lens, D, Hk, B = s["lens"].tolist(), case["D"], case["Hk"], case["B"]
    if case["op"] == "attend":
        T, Hq = case["T"], case["Hq"]
        out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device="cuda")
        lse = torch.full((B, T, Hq), float("-inf"), dtype=torch.float64, device="cuda")
        acc = torch.zeros((B, Hk, s["table"].shape[1] * PAGE), dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            if n == 0:
                continue
            if case["weights"]:
                acc[b, :, :n] = s["acc"][b, :, :n].double()
            k, v = _exact_cache(s, s["cache"], s["table"], b, n, D)
            for t in range(max(0, T - n), T):
                m = n - (T - 1 - t)
                q = s["q"][b, t].double().reshape(Hk, Hq // Hk, D)
                x = s["scale"] * torch.matmul(q, k[:, :m].transpose(1, 2).contiguous())
                lse[b, t] = torch.logsumexp(x, 2).flatten()
                p = torch.softmax(x, 2)
                out[b, t] = torch.matmul(p, v[:, :m].contiguous()).flatten(0, 1)
                if case["weights"]:
                    acc[b, :, :m] += p.sum(1)
        return {"out": out, "lse": lse, **({"acc": acc} if case["weights"] else {})}
    if case["op"] == "append":
        T, got = case["T"], {}
        grid = torch.tensor(sorted({m / 512 for m in range(8)} | {(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)}),
                            dtype=torch.float64, device="cuda")
        fp4 = torch.tensor(E2M1, dtype=torch.float64, device="cuda")

        def nearest(a, points):
            # Of the two neighbours the nearer; at the middle the one with the even index.
            hi = torch.searchsorted(points, a).clamp(1, len(points) - 1)
            up, down = points[hi] - a, a - points[hi - 1]
            return points[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)]

        for name, x, g in (("k", s["k"], s["gk"]), ("v", s["v"], s["gv"])):
            w = x.double().unflatten(-1, (-1, 16))
            scale = nearest((w.abs().amax(-1, keepdim=True) / 6 / g).clamp(max=448.0), grid)
            ratio = torch.where(scale > 0, w.abs() / torch.where(scale > 0, scale * g, 1.0), 0.0)
            held = (torch.sign(w) * nearest(ratio.clamp(max=6.0), fp4) * scale * g).flatten(-2)
            row = torch.arange(T, device="cuda")[None, :] - T + s["lens"][:, None]
            got[name] = torch.where((row >= 0)[..., None, None], held, 0.0)
        return got
    keep = case["keep"]
    got = {"kept": torch.full((B, Hk, keep), -1, dtype=torch.int32, device="cuda"), "lens": s["lens"].clamp(max=keep),
           "acc": torch.zeros(s["new_acc"].shape, dtype=torch.float64, device="cuda"),
           "k": torch.zeros((B, keep, Hk, D), dtype=torch.float64, device="cuda"), "v": torch.zeros((B, keep, Hk, D), dtype=torch.float64, device="cuda")}
    for b, n in enumerate(lens):
        if n == 0:
            continue
        k, v = _exact_cache(s, s["cache"], s["table"], b, n, D)
        for h in range(Hk):
            weight = s["acc"][b, h, :n].double()
            weight[:min(n, case["sinks"])] = float("inf")
            weight[max(0, n - case["recent"]):] = float("inf")
            at = torch.sort(weight, descending=True, stable=True).indices[:keep].sort().values
            m = len(at)
            got["kept"][b, h, :m] = at.int()
            got["acc"][b, h, :m] = s["acc"][b, h, at].double()
            got["k"][b, keep - m:, h], got["v"][b, keep - m:, h] = k[h, at], v[h, at]
    return got
