"""The cache's calls at the edges that their kernels' parts have, and together in a decode."""

import numpy as np
import pytest
import torch

import fp8_quantized_skinny_amd as sk
from fp8_quantized_skinny_amd.cached_decode import CachedDecoder
from oracle import kv4 as oracle
from test_logprobs import _check, _run

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def _append_one(x, g, D, T=64):
    """Codes and scales, bit for bit as the oracle finds them, of x [T, D] appended as keys and as values."""
    cache = torch.full((2, 1, 72 * D), 0xAB, dtype=torch.uint8, device="cuda")
    table, lens = torch.tensor([[1]], dtype=torch.int32, device="cuda"), torch.tensor([T], dtype=torch.int32, device="cuda")
    rows = x.cuda().view(1, T, 1, D)
    sk.kv4_append(cache, table, lens, rows, rows, gk=g, gv=g)
    codes, scales = oracle.kv_quantize(x.double().numpy(), np.float32(g))
    want = np.full(72 * D, 0xAB, np.uint8)
    for t in range(T):
        oracle.kv_put(want, t, codes[t], scales[t], codes[t], scales[t])
    got = cache.cpu().numpy()
    assert (got[0] == 0xAB).all()
    assert np.array_equal(got[1, 0], want)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("g", [1.0, 3.0, 7.0, 0.375, float(np.float32(0.1)), 2.0 ** -20])
@pytest.mark.parametrize("T", [64, 63])  # a whole page, and a part of one
def test_append_on_and_beside_the_borders(kind, g, T):
    """Groups whose greatest value puts the scale half way between two E4M3 values, or beside that, and
    values on the borders between codes, or one step of the type beside them."""
    D = 64
    rng = np.random.default_rng(1)
    steps = rng.integers(8, 16, (T, D // 16, 1)) + rng.choice([0.0, 0.5], (T, D // 16, 1))  # of an eighth
    amax = 6.0 * g * steps / 8.0 * np.exp2(rng.integers(-3, 3, (T, D // 16, 1)))
    border = rng.choice([0.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], (T, D // 16, 16)) / 6.0
    x = amax * border * rng.choice([-1.0, 1.0], border.shape)
    x[..., :1] = amax
    x = torch.from_numpy(x.reshape(T, D)).to(TYPES[kind])
    beside = torch.from_numpy(rng.integers(-1, 2, (T, D)).astype(np.int16))
    x = torch.where(x == 0, x, (x.view(torch.int16) + beside).view(TYPES[kind]))
    _append_one(x, g, D, T)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_of_extreme_groups(kind, D):
    """The type's greatest and least values, infinities, NaN and zeros of both signs, with great and small g."""
    info = torch.finfo(TYPES[kind])
    rng = np.random.default_rng(D)
    pool = torch.tensor([info.max, -info.max, info.tiny, info.smallest_normal, float("inf"), 0.0, -0.0, 1.0, -3.0], dtype=torch.float64)
    x = pool[torch.from_numpy(rng.integers(0, len(pool), (64, D)))].to(TYPES[kind])
    x[3, :16] = float("nan")
    x[5, 16:32] = 0.0
    x[6, :16] = torch.from_numpy(rng.integers(1, 9, 16).astype(np.int16)).view(TYPES[kind])  # denormals
    for g in (1.0, 1e-30, 1e30, 3e38):
        _append_one(x, g, D)


@pytest.mark.parametrize("weights", ["exp", "equal", "few", "nan"])
@pytest.mark.parametrize("n, keep, sinks, recent", [(70000, 5000, 4, 100), (65536, 33000, 32770, 7), (32769, 1, 0, 0), (98304, 40000, 0, 40000)])
def test_evict_of_more_slots_than_are_held_at_once(n, keep, sinks, recent, weights):
    """Ties, sinks and recent slots that cross the 32768 slots a workgroup holds."""
    rng = np.random.default_rng(n)
    width = -(-n // 64)
    acc = {"exp": lambda: rng.exponential(size=64 * width) * (rng.random(64 * width) < 0.7), "equal": lambda: np.full(64 * width, 0.5),
           "few": lambda: rng.integers(0, 3, 64 * width) * 1.0,
           "nan": lambda: np.where(rng.random(64 * width) < 0.9, np.nan, rng.random(64 * width))}[weights]().astype(np.float32)
    c = lambda pages: torch.zeros((pages, 1, 72 * 64), dtype=torch.uint8, device="cuda")  # noqa: E731
    i32 = lambda a: torch.as_tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    dwidth = -(-keep // 64)
    kept, lens = torch.empty((1, 1, keep), dtype=torch.int32, device="cuda"), i32([0])
    new_acc = torch.empty((1, 1, 64 * dwidth), device="cuda")
    sk.kv4_evict(c(3), i32([[p % 3 for p in range(width)]]), i32([n]), torch.from_numpy(acc).cuda().view(1, 1, -1), c(dwidth),
                 i32([list(range(dwidth))]), kept, lens, new_acc, sinks=sinks, recent=recent)
    want = oracle.kv_evict(acc, n, keep, sinks, recent)
    assert lens.tolist() == [keep] and np.array_equal(kept.cpu().numpy()[0, 0], want)
    assert np.array_equal(new_acc.cpu().numpy()[0, 0, :keep], acc[want], equal_nan=True)


@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("V", [8, 32, 39, 63, 64, 65, 255, 300, 1024])
def test_alternatives_of_few_groups(kind, V):
    """Fewer loads of logits than alternatives, rows that begin inside a 16-byte load, and ties."""
    k = min(32, V)
    g = torch.Generator().manual_seed(V)
    x = (torch.randn((7, V), generator=g) * 3.0).round()  # many ties
    x[1] = torch.randn((V,), generator=g)
    x[2, : V // 2] = float("-inf")
    x = x.to(TYPES[kind])
    tokens = torch.randint(0, V, (7,), generator=g).tolist()
    for stride in (V, V + 1, V + 3):
        _check(x, tokens, k, _run(x, tokens, k, stride))


def test_eviction_and_log_probabilities_replayed_from_a_graph():
    """evict, read and the log probabilities captured together: every replay gives the eager results."""
    B, Hk, D, n, keep, R, V, k = 3, 2, 128, 1000, 200, 4, 30000, 9
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    width, dwidth = -(-n // 64), -(-keep // 64)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = torch.randint(0, 0x30, (B * width, Hk, 72 * D), generator=g, device="cuda").to(torch.uint8)
    table, dtable = torch.arange(B * width, device="cuda").int().view(B, width), torch.arange(B * dwidth, device="cuda").int().view(B, dwidth)
    lens = torch.tensor([n, 150, 777], dtype=torch.int32, device="cuda")
    acc = torch.rand((B, Hk, 64 * width), generator=g, device="cuda")
    dst, kept, new_lens, new_acc = torch.zeros((B * dwidth, Hk, 72 * D), dtype=torch.uint8, device="cuda"), i32(B, Hk, keep), i32(B), torch.zeros((B, Hk, 64 * dwidth), device="cuda")
    held = torch.zeros((2, B, keep, Hk, D), dtype=torch.float16, device="cuda")
    logits, tokens = torch.randn((R, V), generator=g, device="cuda").half(), i32(R) + 7
    lp, ent, ids, top = torch.zeros(R, device="cuda"), torch.zeros(R, device="cuda"), i32(R, k), torch.zeros((R, k), device="cuda")
    ws = sk.new_workspace(sk.lm_head_logprobs_workspace_bytes(R, V, k))

    def step():
        sk.kv4_evict(cache, table, lens, acc, dst, dtable, kept, new_lens, new_acc, sinks=4, recent=32)
        sk.kv4_read(dst, dtable, new_lens, held[0], held[1])
        sk.lm_head_logprobs(logits, tokens, lp, ent, ids, top, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    outs = (dst, kept, new_lens, new_acc, held, lp, ent, ids, top)
    for i in range(4):
        acc.copy_(torch.rand(acc.shape, generator=g, device="cuda"))
        logits.copy_(torch.randn(logits.shape, generator=g, device="cuda"))
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, outs):
            assert torch.equal(a, b), i


def test_the_calls_refuse_wrong_tensors():
    B, Hk, D, width, T, Hq = 2, 2, 64, 12, 2, 4
    cache = torch.zeros((4, Hk, 72 * D), dtype=torch.uint8, device="cuda")
    table, lens = torch.zeros((B, width), dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    k = torch.zeros((B, T, Hk, D), dtype=torch.float16, device="cuda")
    for bad in ((cache.cpu(), table, lens, k, k), (cache, table.long(), lens, k, k), (cache, table, lens.float(), k, k),
                (cache, table, lens, k, k.bfloat16()), (cache, table, lens, k.int(), k), (cache, table, lens, k, None), (3, table, lens, k, k)):
        with pytest.raises(TypeError):
            sk.kv4_append(*bad)
    for bad in ((cache[..., :-8], table, lens, k, k), (cache, table[0], lens, k, k), (cache, table, lens[:1], k, k),
                (cache, table, lens, k[:, :, :1], k), (cache, table, lens, k, k[:, :1]), (cache, table, lens, k.transpose(2, 3), k),
                (cache[:, :, ::2], table, lens, k, k), (cache, table, lens, k[:0], k)):
        with pytest.raises(ValueError):
            sk.kv4_append(*bad)
    with pytest.raises(sk.SkinnyError):
        sk.kv4_append(cache, table, lens, k, k, gk=0.0)
    q = torch.zeros((B, T, Hq, D), dtype=torch.float16, device="cuda")
    need = sk.kv4_attention_workspace_bytes(B, T, Hq, Hk, D, width)
    assert need
    out, lse = torch.empty_like(q), torch.empty((B, T, Hq), device="cuda")
    for ws in (None, sk.new_workspace(need - 1)):
        with pytest.raises(ValueError):
            sk.kv4_attention(q, cache, table, lens, out, workspace=ws)
    ws = sk.new_workspace(need)
    for bad in (dict(lse=lse[..., :2]), dict(out=out.transpose(0, 1)), dict(q=q[..., :32])):
        with pytest.raises(ValueError):
            sk.kv4_attention(**{**dict(q=q, cache=cache, table=table, lens=lens, out=out, workspace=ws), **bad})
    for bad in (dict(lse=lse.half()), dict(out=out.bfloat16()), dict(workspace=ws.int()), dict(scale="x")):
        with pytest.raises(TypeError):
            sk.kv4_attention(**{**dict(q=q, cache=cache, table=table, lens=lens, out=out, workspace=ws), **bad})
    with pytest.raises(sk.SkinnyError):
        sk.kv4_attention(q.float(), cache, table, lens, out.float(), workspace=ws)
    acc = torch.zeros((B, Hk, 64 * width), device="cuda")
    with pytest.raises(ValueError):
        sk.kv4_attention_weights(q, cache, table, lens, lse, acc[..., :64], acc)
    with pytest.raises(ValueError):
        sk.kv4_read(cache, table, lens, k, k[:, :1])
    x, i32 = torch.zeros((3, 100), device="cuda"), lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    f = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    for bad in ((x.t(), i32(3), f(3), f(3), i32(3, 2), f(3, 2)), (x, i32(2), f(3), f(3), i32(3, 2), f(3, 2)), (x, i32(3), f(3), f(3), i32(3, 2), f(3, 3))):
        with pytest.raises((ValueError, sk.SkinnyError)):
            sk.lm_head_logprobs(*bad)
    with pytest.raises(TypeError):
        sk.lm_head_logprobs(x.double(), i32(3), f(3), f(3), i32(3, 2), f(3, 2))
    torch.cuda.synchronize()


@pytest.mark.parametrize("streams, rows", [(2, 1), (1, 4)])
def test_decode_over_a_budgeted_cache(streams, rows):
    """Every step of the example against 64 bits, from the keys and values as the cache holds them."""
    d = CachedDecoder(streams=streams, rows=rows, budget=100, keep=70, sinks=4, recent=16)
    B, T, Hq, Hk, D = d.B, d.T, d.Hq, d.Hk, d.D
    cuts, previous, last_keys = 0, None, None
    for i in range(130 // rows):
        before = d.length
        cut = d.step()
        cuts += cut
        torch.cuda.synchronize()
        assert d.lens.tolist() == [d.length] * B and d.length == (d.keep if cut else before) + T
        k, v = torch.zeros((2, B, d.length, Hk, D), dtype=torch.float16, device="cuda")
        sk.kv4_read(*d.cache(), k, v)
        if cut:  # the kept slots are those of the cache before, in order; the last `recent` and first `sinks` stay
            kept = d.kept.long()
            assert (kept[..., :d.sinks].cpu() == torch.arange(d.sinks)).all() and (kept[..., -d.recent:].cpu() == torch.arange(before - d.recent, before)).all()
            for b in range(B):
                for h in range(Hk):
                    assert torch.equal(k[b, :d.keep, h], last_keys[b, kept[b, h], h])
        last_keys = k.clone()
        q = d.qkv.view(B, T, Hq + 2 * Hk, D)[:, :, :Hq].double().cpu()
        kd, vd = k.double().cpu(), v.double().cpu()
        for b in range(B):
            for t in range(T):
                n = d.length - (T - 1 - t)
                for h in range(Hq):
                    x = kd[b, :n, h // (Hq // Hk)] @ q[b, t, h] / D ** 0.5
                    p, vals = torch.softmax(x, 0), vd[b, :n, h // (Hq // Hk)]
                    # p V: a rounding of p to fp16 and of the result (2^-11 of each), exp's argument (24 bits of the
                    # scores' size; the scores' sums are of D products), so 2^-10 of sum p |v| and the scores' share
                    tol = (p @ vals.abs()) * (2.0 ** -10 + 2.0 ** -20 * (1 + x.abs().max()))
                    assert ((d.out[b, t, h].double().cpu() - p @ vals).abs() <= tol + 2.0 ** -24).all(), (i, b, t, h)
        lp = torch.log_softmax(d.logits.double(), 1).cpu()
        given = d.tokens.flatten().long().cpu()
        tol = 2.0 ** -16 + 2.0 ** -22 * d.logits.abs().max().item()  # as for the log probabilities alone
        assert ((d.logprob.double().cpu() - lp.gather(1, given[:, None])[:, 0]).abs() <= tol).all()
        assert (d.top_ids.view(B, T, -1)[:, -1, 0].cpu() == d.tokens[:, -1].cpu()).all()
        # every row's weights sum to one per query head
        if not cut and previous is not None:
            grown = d.accs[d.now].double().sum().item() - previous
            assert abs(grown - B * T * Hq) <= B * T * Hq * 2.0 ** -12 + 2.0 ** -24 * d.accs[d.now].numel() * d.accs[d.now].max().item()
        previous = d.accs[d.now].double().sum().item()
    assert cuts >= 1
