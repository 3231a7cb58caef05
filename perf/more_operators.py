"""What is measured of the operators that bring a prompt and positions to the 4-bit cache: the
norm of queries and keys with their rotation, the attention of a chunk of new tokens, and
attention within a sliding window.

`run` computes a case in plain torch operations, or, with `own` set, through the package's
entry points.  Head shapes are those behind the qkv (K 5120, N 7168) and o_proj (K 6144) GEMMs
of the decode path, 48 query and 4 key/value heads of 128, and other layouts.

Conventions (include/skinny.h has them in full): a page holds 64 tokens; per page and key/value
head there are 72 * D bytes: K codes, K scales, V codes, V scales.  lens counts the step's own
tokens: row t of a sequence's T has the slots s < L = lens - (T - 1 - t), and with a window of
those the ones with s >= L - window or s < sinks.
"""

import math

import torch

own = False

PAGE = 64
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
HEADS = ((48, 4, 128), (24, 4, 256), (32, 8, 128), (16, 16, 64), (8, 1, 128), (28, 4, 64), (5, 1, 256))


def listed():
    rope = dict(op="rope", eps=1e-6, amplitude=1.0, base=10000.0, norm=True, interleaved=False)
    chunk = dict(op="chunk", window=0, sinks=0, pad=0)
    window = dict(op="window")
    return [
        # The one new token of one stream: all latency.
        dict(rope, name="rope_token", type="f16", B=1, T=1, Hq=48, Hk=4, D=128, rot=128, reach=9000),
        # A step of a server's batch, eight rows a sequence, far positions, an interleaved part of wide heads, scaled frequencies.
        dict(rope, name="rope_batch", type="bf16", B=64, T=8, Hq=24, Hk=4, D=256, rot=64, reach=1000000, interleaved=True, base=1e7, amplitude=1.2),
        # A long prompt at once.
        dict(rope, name="rope_prompt", type="bf16", B=1, T=32768, Hq=48, Hk=4, D=128, rot=128, reach=32768, base=1e6),
        # A short question into a short conversation: latency.
        dict(chunk, name="chunk_question", type="f16", B=1, Hq=48, Hk=4, D=128, least=17, most=17, before_least=284, before=284),
        # A prompt from an empty cache.
        dict(chunk, name="chunk_prompt", type="f16", B=1, Hq=48, Hk=4, D=128, least=8192, most=8192, before_least=0, before=0),
        # The next piece of a long document: few rows, a long axis of keys.
        dict(chunk, name="chunk_document", type="bf16", B=1, Hq=48, Hk=4, D=128, least=512, most=512, before_least=120000, before=120000),
        # A server's batch: prompts of any length, single tokens among them, over contexts of any length, rows behind the last.
        dict(chunk, name="chunk_ragged", type="bf16", B=16, Hq=32, Hk=8, D=128, least=1, most=640, before_least=0, before=9000, pad=37),
        # Prompts of a layer with a sliding window, wide heads.
        dict(chunk, name="chunk_window", type="f16", B=3, Hq=24, Hk=4, D=256, least=1500, most=4100, before_least=0, before=2500, window=1024, sinks=4),
        # One stream deep in a long context.
        dict(window, name="window_token", type="f16", B=1, T=1, Hq=48, Hk=4, D=128, shortest=32000, longest=32000, window=1024, sinks=4),
        # A verification round of a batch, wide heads, an odd window.
        dict(window, name="window_verify", type="bf16", B=8, T=8, Hq=24, Hk=4, D=256, shortest=500, longest=20000, window=2047, sinks=5),
        # A server's batch, some sequences shorter than the window.
        dict(window, name="window_batch", type="bf16", B=48, T=1, Hq=48, Hk=4, D=128, shortest=1, longest=32000, window=4096, sinks=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    op = rng.choice(("rope", "chunk", "chunk", "window"))
    kind = rng.choice(("f16", "bf16"))
    Hq, Hk, D = rng.choice(HEADS)
    if op == "rope":
        B = _log(rng, 1, 64)
        T = _log(rng, 1, int(2.1e8 / (B * (Hq + Hk) * D)))
        return dict(op=op, type=kind, B=B, T=T, Hq=Hq, Hk=Hk, D=D, rot=rng.choice((D, D, D // 2, D // 4, 0)), reach=_log(rng, 100, 1000000),
                    interleaved=rng.random() < 0.4, norm=rng.random() < 0.7, eps=rng.choice((1e-6, 1e-5)), base=rng.choice((1e4, 5e5, 1e7)),
                    amplitude=rng.choice((1.0, 1.0, 1.3)))
    if op == "chunk":
        B = _log(rng, 1, 24)
        # Scores of the plain form (padded to the longest), products and slots within the largest listed case's.
        most = _log(rng, 1, min(8192, math.isqrt(int(min(3e9 / (B * Hq), 3.7e11 / (B * Hq * D))))))
        room = max(1, int(min(3e9 / (B * Hq * most), 3.7e11 / (B * Hq * D * most), 5e8 / (B * Hk * D), 130000)) - most)
        before = _log(rng, 1, room)
        windowed = rng.random() < 0.4
        return dict(op=op, type=kind, B=B, Hq=Hq, Hk=Hk, D=D, least=rng.choice((1, max(1, most // 2), most)), most=most,
                    before_least=rng.choice((0, 0, before // 2, before)), before=before, window=_log(rng, 1, 8192) if windowed else 0,
                    sinks=rng.choice((0, 1, 4, 70)) if windowed else 0, pad=rng.choice((0, 0, 11)))
    T = rng.choice((1, 1, 2, 4, 5, 8))
    B = _log(rng, 1, 64)
    longest = _log(rng, 1, int(min(32768, 7.5e8 / (B * Hk * D), 6e8 / (B * T * Hq))))
    return dict(op=op, type=kind, B=B, T=T, Hq=Hq, Hk=Hk, D=D, shortest=rng.choice((0, 1, longest // 2, longest)), longest=longest,
                window=_log(rng, 1, 8192), sinks=rng.choice((0, 1, 4, 64, 200)))


def _pages(B, width, g, spare=3):
    """A table of pages scattered over a pool of B * width + spare pages."""
    at = torch.randperm(B * width + spare, generator=g, device="cuda")[:B * width]
    return at.to(torch.int32).reshape(B, width), B * width + spare


def _between(lo, hi, B, g):
    """B whole numbers from lo to hi, one of them hi."""
    n = torch.randint(lo, hi + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    n[int(torch.randint(0, B, (1,), generator=g, device="cuda"))] = hi
    return n


def _chunk_lengths(case):
    """The new tokens of a batch's sequences: many short chunks and a few long ones, from the least to the most."""
    B = case["B"]
    return [case["most"] - round((case["most"] - case["least"]) * (1 - ((i + 1) / B) ** 2)) for i in range(B)]


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


def _frequencies(rot, base):
    """The radians per position of each pair; with the largest base those of the slow pairs divided by 8, as long contexts have them."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    if base > 1e6:
        f = torch.where(f * 8192 < 2 * math.pi, f / 8, f)
    return f.float().cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind = TYPES[case["type"]]
    B, Hq, Hk, D = (case[n] for n in ("B", "Hq", "Hk", "D"))
    s = dict(case=case)
    if case["op"] == "rope":
        T = case["T"]
        qkv = torch.randn((B, T, (Hq + 2 * Hk) * D), generator=g, device="cuda")
        # Channels of different sizes, as projections have them; q and k lie in the qkv GEMM's output.
        qkv *= 0.2 + 3.0 * torch.rand(((Hq + 2 * Hk) * D,), generator=g, device="cuda").pow_(4)
        qkv = qkv.to(kind)
        s["q"], s["k"] = qkv[..., :Hq * D].unflatten(-1, (Hq, D)), qkv[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D))
        first = torch.randint(0, max(1, case["reach"] - T), (B, 1), generator=g, device="cuda", dtype=torch.int32)
        s["positions"] = first + torch.arange(T, device="cuda", dtype=torch.int32)
        s["inv_freq"] = _frequencies(case["rot"], case["base"])
        if case["norm"]:
            s["q_weight"], s["k_weight"] = (1.0 + 0.4 * torch.randn((2, D), generator=g, device="cuda")).unbind(0)
        else:
            s["q_weight"] = s["k_weight"] = None
        s["q_out"], s["k_out"] = (torch.empty((B, T, H, D), dtype=kind, device="cuda") for H in (Hq, Hk))
        return s

    if case["op"] == "chunk":
        T = torch.tensor(_chunk_lengths(case), dtype=torch.int32, device="cuda")[torch.randperm(B, generator=g, device="cuda")]
        lens = T + _between(case["before_least"], case["before"], B, g)
        width = -(-(case["most"] + case["before"]) // PAGE)
        s["starts"] = torch.cat((torch.zeros(1, dtype=torch.int32, device="cuda"), T.cumsum(0).int()))
        N = sum(_chunk_lengths(case)) + case["pad"]
        # The queries lie in the output of a qkv GEMM, beside those tokens' keys and values.
        qkv = (torch.randn((N, (Hq + 2 * Hk) * D), generator=g, device="cuda") * 2.0).to(kind)
        s["q"] = qkv[:, :Hq * D].unflatten(-1, (Hq, D))
        s["out"], s["lse"] = torch.zeros((N, Hq, D), dtype=kind, device="cuda"), torch.zeros((N, Hq), device="cuda")
    else:
        T, width = case["T"], max(1, -(-case["longest"] // PAGE))
        lens = _between(case["shortest"], case["longest"], B, g)
        qkv = (torch.randn((B, T, (Hq + 2 * Hk) * D), generator=g, device="cuda") * 2.0).to(kind)
        s["q"] = qkv[..., :Hq * D].unflatten(-1, (Hq, D))
        s["out"], s["lse"] = torch.empty((B, T, Hq, D), dtype=kind, device="cuda"), torch.empty((B, T, Hq), device="cuda")
    s["table"], pages = _pages(B, width, g)
    s.update(cache=_cache(pages, Hk, D, g), lens=lens, gk=1.0, gv=0.75, scale=1.0 / math.sqrt(D))
    if own:  # the scratch buffer that a program keeps; no data of the case goes there before the call
        import fp8_quantized_skinny_amd as sk
        if case["op"] == "chunk":
            s["workspace"] = sk.new_workspace(sk.kv4_attention_chunk_workspace_bytes(N, B, Hq, Hk, D, width, case["window"], case["sinks"]))
        else:
            s["workspace"] = sk.new_workspace(sk.kv4_attention_window_workspace_bytes(B, T, Hq, Hk, D, width, case["window"], case["sinks"]))
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": _rope_own, "chunk": _chunk_own, "window": _window_own}[op](s)
    return {"rope": _rope_plain, "chunk": _chunk_plain, "window": _window_plain}[op](s)


# ---------------------------------------------------------------- the package's operators
def _rope_own(s):
    import fp8_quantized_skinny_amd as sk
    case = s["case"]
    sk.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_out"], s["k_out"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                    eps=case["eps"], amplitude=case["amplitude"], interleaved=case["interleaved"])
    return {"q": s["q_out"], "k": s["k_out"]}


def _chunk_own(s):
    import fp8_quantized_skinny_amd as sk
    sk.kv4_attention_chunk(s["q"], s["starts"], s["cache"], s["table"], s["lens"], s["out"], lse=s["lse"], scale=s["scale"],
                           window=s["case"]["window"], sinks=s["case"]["sinks"], gk=s["gk"], gv=s["gv"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _window_own(s):
    import fp8_quantized_skinny_amd as sk
    sk.kv4_attention_window(s["q"], s["cache"], s["table"], s["lens"], s["out"], s["case"]["window"], s["case"]["sinks"], lse=s["lse"],
                            scale=s["scale"], gk=s["gk"], gv=s["gv"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- plain forms
def _rope_plain(s):
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2
    # Angles in 64 bits: a far position times a frequency has lost its turn in 32.
    angle = s["positions"].double()[..., None] * s["inv_freq"].double()
    c, n = (case["amplitude"] * torch.cos(angle)).float()[:, :, None], (case["amplitude"] * torch.sin(angle)).float()[:, :, None]

    def rotated(x, weight):
        u = x.float()
        if weight is not None:
            u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + case["eps"]) * weight
        if case["interleaved"]:
            a, b = u[..., 0:rot:2], u[..., 1:rot:2]
            y = torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
        else:
            a, b = u[..., :half], u[..., half:rot]
            y = torch.cat((a * c - b * n, b * c + a * n), -1)
        return torch.cat((y, u[..., rot:]), -1).to(x.dtype)
    return {"q": rotated(s["q"], s["q_weight"]), "k": rotated(s["k"], s["k_weight"])}


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
    kc, ks, vc, vs = _split(cache[table.long()].transpose(1, 2), D)
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


def _attend_plain(s, q, T, limit):
    """out [B, T, Hq, D] and lse [B, T, Hq] in 32 bits of rows q [B, T, Hq, D], of which row t sees slots below limit [B, T]."""
    case = s["case"]
    Hk, G = case["Hk"], case["Hq"] // case["Hk"]
    k, v = _values(s["cache"], s["table"], case["D"])
    q = q.float().unflatten(2, (Hk, G)).transpose(1, 2).flatten(2, 3)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"] * s["gk"])
    limit = limit.repeat_interleave(G, 1)[:, None, :, None]
    slot = torch.arange(k.shape[2], device=q.device, dtype=torch.int32)
    hidden = slot >= limit
    if case["window"]:
        hidden |= (slot < limit - case["window"]) & (slot >= case["sinks"])
    x.masked_fill_(hidden, float("-inf"))
    del hidden
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m.masked_fill(m == float("-inf"), 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / total.clamp(min=1e-30) * s["gv"]
    lse = (m + torch.log(total)).squeeze(-1)
    return tuple(t.unflatten(2, (T, G)).transpose(1, 2).flatten(2, 3) for t in (out, lse))


def _chunk_plain(s):
    # Sequences padded to the longest chunk.
    T = s["case"]["most"]
    first, end = s["starts"][:-1, None], s["starts"][1:, None]
    row = first + torch.arange(T, device="cuda", dtype=torch.int32)
    has = row < end
    at = row.clamp(max=s["q"].shape[0] - 1).long()
    out, lse = _attend_plain(s, s["q"][at], T, s["lens"][:, None] - (end - 1 - row))
    got = {"out": torch.zeros_like(s["out"]), "lse": torch.zeros_like(s["lse"])}
    got["out"][at[has]] = out[has].to(s["out"].dtype)
    got["lse"][at[has]] = lse[has]
    return got


def _window_plain(s):
    T = s["case"]["T"]
    out, lse = _attend_plain(s, s["q"], T, s["lens"][:, None] - (T - 1 - torch.arange(T, device="cuda", dtype=torch.int32)))
    return {"out": out.to(s["out"].dtype), "lse": lse}


def _seen(n, window, sinks):
    """How many of the first n slots the newest row sees."""
    return n if not window else min(n, window + min(sinks, max(0, n - window)))


def work(case):
    Hq, Hk, D, B = case["Hq"], case["Hk"], case["D"], case["B"]
    if case["op"] == "rope":
        values = B * case["T"] * (Hq + Hk) * D
        return {"bytes": 4 * values + 4 * B * case["T"], "flops": 10 * values}
    held = 1.125 * D * Hk
    mean = lambda lo, hi: hi if B == 1 else ((lo + hi) * (B - 1) / 2 + hi) / B  # noqa: E731
    if case["op"] == "chunk":
        before, pairs, slots, tokens = mean(case["before_least"], case["before"]), 0.0, 0.0, 0
        for T in _chunk_lengths(case):
            pairs += sum(_seen(before + T * (i + 0.5) / 64, case["window"], case["sinks"]) for i in range(64)) / 64 * T
            slots += min(before + T, _seen(before + 1, case["window"], case["sinks"]) + T - 1)
            tokens += T
        return {"bytes": slots * held + tokens * Hq * (4 * D + 4), "flops": 4 * pairs * Hq * D}
    T = case["T"]
    # Over the lengths of the batch.
    many = [case["longest"]] if B == 1 else [case["longest"]] + [case["shortest"] + (case["longest"] - case["shortest"]) * (i + 0.5) / (B - 1) for i in range(B - 1)]
    seen = sum(_seen(n, case["window"], case["sinks"]) for n in many)
    return {"bytes": seen * held + B * T * Hq * (4 * D + 4), "flops": 4 * seen * T * Hq * D}


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


def _exact_rows(s, q, k, v, first, limits):
    """out and lse of rows q [rows, Hq, D] over slots first .. of one sequence, k and v [Hk, n, D] of those; limits: what each row sees."""
    case = s["case"]
    Hk, n = k.shape[:2]
    rows, G = len(limits), case["Hq"] // Hk
    x = torch.matmul(q.double().reshape(rows, Hk, G, -1).permute(1, 0, 2, 3).reshape(Hk, rows * G, -1), k.transpose(1, 2).contiguous())
    x = (x * s["scale"]).reshape(Hk, rows, G, n)
    slot = torch.tensor(first, device="cuda")
    see = torch.stack([(slot < L) & (((slot >= L - case["window"]) | (slot < case["sinks"])) if case["window"] else (slot >= 0)) for L in limits])
    x = x.masked_fill(~see[None, :, None], float("-inf"))
    some = see.any(1)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(some[None, :, None], lse, 0.0)[..., None])
    out = torch.matmul(p.reshape(Hk, rows * G, n), v).reshape(Hk, rows, G, -1)
    return out.permute(1, 0, 2, 3).flatten(1, 2), lse.permute(1, 0, 2).flatten(1, 2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        got, rot = {}, case["rot"]
        for name, x, w in (("q", s["q"], s["q_weight"]), ("k", s["k"], s["k_weight"])):
            u = torch.empty(x.shape, dtype=torch.float64, device="cuda")
            step = max(1, 4096 // case["B"])
            for t in range(0, case["T"], step):
                y = x[:, t:t + step].double()
                if w is not None:
                    y = y / (y.pow(2).sum(-1, keepdim=True) / case["D"] + case["eps"]).sqrt() * w.double()
                if rot:
                    # A pair is a complex number, and the rotation a product.
                    a = s["positions"][:, t:t + step].double()[..., None, None] * s["inv_freq"].double()
                    pairs = y[..., :rot].unflatten(-1, (-1, 2)) if case["interleaved"] else y[..., :rot].unflatten(-1, (2, -1)).transpose(-1, -2)
                    z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.full_like(a, case["amplitude"]), a)
                    z = torch.view_as_real(z)
                    y[..., :rot] = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
                u[:, t:t + step] = y
            got[name] = u
        return got
    lens, Hq, D, B = s["lens"].tolist(), case["Hq"], case["D"], case["B"]
    starts = s["starts"].tolist() if case["op"] == "chunk" else [b * case["T"] for b in range(B + 1)]
    q = s["q"] if case["op"] == "chunk" else s["q"].flatten(0, 1)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    flat, flat_lse = out.view(-1, Hq, D), lse.view(-1, Hq)
    for b, n in enumerate(lens):
        r0, r1 = starts[b], starts[b + 1]
        held = _exact_block(s["cache"][s["table"][b, :max(1, -(-n // PAGE))].long()], D)
        k, v = (a.transpose(0, 1).flatten(1, 2)[:, :max(n, 1)] * g for a, g in zip(held, (s["gk"], s["gv"])))
        for r in range(r0, r1, 100):
            limits = [n - (r1 - 1 - i) for i in range(r, min(r + 100, r1))]
            low = max(0, limits[0] - case["window"]) if case["window"] else 0
            slots = list(range(min(case["sinks"], low))) + list(range(low, max(limits[-1], low + 1)))
            at = torch.tensor(slots, device="cuda").clamp(max=k.shape[1] - 1)
            flat[r:r + len(limits)], flat_lse[r:r + len(limits)] = _exact_rows(s, q[r:r + len(limits)], k[:, at], v[:, at].contiguous(), slots, limits)
    return {"out": out, "lse": lse}
