"""The 4-bit key/value cache against its definition in 64 bits, and the refusals of its calls."""

import struct

import numpy as np
import pytest
import torch

import fp8_quantized_skinny_amd as sk
from fp8_quantized_skinny_amd._lib import lib
from oracle import kv4 as oracle

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


# ---------------------------------------------------------------- the oracle itself
@pytest.mark.parametrize("D", [64, 128, 256])
def test_places_cover_a_block_once(D):
    k, v, nib, ks, vs = oracle.kv_places(D)
    nibbles = np.concatenate([(k * 2 + nib).ravel(), (v * 2 + nib).ravel()])
    scales = np.concatenate([ks[:, ::16].ravel(), vs[:, ::16].ravel()])
    taken = np.concatenate([nibbles, scales * 2, scales * 2 + 1])
    assert np.array_equal(np.sort(taken), np.arange(72 * D * 2))
    # a group of 16 shares a scale byte
    assert (ks.reshape(64, -1, 16) == ks[:, ::16, None]).all() and (vs.reshape(64, -1, 16) == vs[:, ::16, None]).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_token_put_into_a_block_is_held(D):
    rng = np.random.default_rng(0)
    block = rng.integers(0, 256, 72 * D, dtype=np.uint8)
    x, y = rng.standard_normal((2, D))
    before = block.copy()
    oracle.kv_put(block, 21, *oracle.kv_quantize(x, 1.0), *oracle.kv_quantize(y, 0.5))
    k, v = oracle.kv_values(block, D, 1.0, 0.5)
    for got, want in ((k[21], x), (v[21], y)):
        # half an E2M1 gap (1 at most, of 6 units) and a scale off by 2^-4 of itself
        amax = np.abs(want).reshape(-1, 16).max(1).repeat(16)
        assert (np.abs(got - want) <= amax * (1 / 6 * 1.0625 + 0.0625)).all()
    k0, v0 = oracle.kv_values(before, D, 1.0, 0.5)
    others = np.arange(64) != 21
    assert np.array_equal(k[others], k0[others], equal_nan=True) and np.array_equal(v[others], v0[others], equal_nan=True)


# ---------------------------------------------------------------- refusals (no GPU)
A, MIS = 0x10000, 0x10008


def _cache(data=A, table=A, lens=A, pages=8, width=2, B=2, Hk=4, D=128, gk=1.0, gv=1.0):
    return struct.pack("=QQQiiiiiff4x", data, table, lens, pages, width, B, Hk, D, gk, gv)


def _rows(data=A, sequence=4096, row=512, head=128):
    return struct.pack("=Qqqq", data, sequence, row, head)


BAD_CACHES = [(dict(data=0), sk.EINVAL), (dict(table=0), sk.EINVAL), (dict(lens=0), sk.EINVAL), (dict(data=MIS), sk.EALIGN),
              (dict(table=A + 2), sk.EALIGN), (dict(lens=A + 1), sk.EALIGN), (dict(pages=0), sk.ESHAPE), (dict(width=0), sk.ESHAPE),
              (dict(width=1 << 25), sk.ESHAPE), (dict(B=0), sk.ESHAPE), (dict(B=65537), sk.ESHAPE), (dict(Hk=0), sk.ESHAPE),
              (dict(Hk=1025), sk.ESHAPE), (dict(D=96), sk.ESHAPE), (dict(D=512), sk.ESHAPE), (dict(gk=0.0), sk.EINVAL),
              (dict(gv=-1.0), sk.EINVAL), (dict(gk=float("nan")), sk.EINVAL), (dict(gv=float("inf")), sk.EINVAL)]
BAD_ROWS = [(dict(data=0), sk.EINVAL), (dict(data=MIS), sk.EALIGN), (dict(row=-8), sk.EINVAL), (dict(head=4), sk.EALIGN),
            (dict(sequence=4097), sk.EALIGN), (dict(row=12), sk.EALIGN)]


def _calls(cache=None, rows=None, type=0, T=2, Hq=8):
    """Every call that takes a cache, with these arguments."""
    c, r, L = cache if cache is not None else _cache(), rows if rows is not None else _rows(), lib()
    return {
        "append": lambda: L.kv4_append(c, r, r, type, T, None),
        "attention": lambda ws=A, n=1 << 40: L.kv4_attention(c, r, type, T, Hq, 0.1, A, A, ws, n, None),
        "weights": lambda: L.kv4_attention_weights(c, r, type, T, Hq, 0.1, A, A, A, None),
        "read": lambda: L.kv4_read(c, A, A, type, T, None),
        "evict": lambda: L.kv4_evict(c, A, _cache(data=A * 2), A, A, A, 64, 1, 1, None),
    }


@pytest.mark.parametrize("bad, status", BAD_CACHES)
def test_cache_refusals(bad, status):
    for name, call in _calls(cache=_cache(**bad)).items():
        assert call() == status, name


@pytest.mark.parametrize("bad, status", BAD_ROWS)
def test_row_refusals(bad, status):
    calls = _calls(rows=_rows(**bad))
    for name in ("append", "attention", "weights"):
        assert calls[name]() == status, name


def test_type_head_and_row_count_refusals():
    for name, call in _calls(type=2).items():
        if name != "evict":
            assert call() == sk.EINVAL, name
    for bad in (dict(T=0), dict(T=9), dict(Hq=6), dict(Hq=0), dict(Hq=4 * 65)):
        calls = _calls(**bad)
        assert calls["attention"]() == sk.ESHAPE and calls["weights"]() == sk.ESHAPE, bad
    assert _calls(T=0)["append"]() == sk.ESHAPE and _calls(T=0)["read"]() == sk.ESHAPE
    L = lib()
    assert L.kv4_append(None, _rows(), _rows(), 0, 1, None) == sk.EINVAL
    assert L.kv4_append(_cache(), None, _rows(), 0, 1, None) == sk.EINVAL


def test_attention_refusals():
    L, c, r = lib(), _cache(width=64), _rows()
    call = lambda scale=0.1, out=A, lse=A, ws=A, n=1 << 40: L.kv4_attention(c, r, 0, 2, 8, scale, out, lse, ws, n, None)  # noqa: E731
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=scale) == sk.EINVAL
    assert call(out=None) == sk.EINVAL and call(out=MIS) == sk.EALIGN and call(lse=A + 2) == sk.EALIGN
    need = sk.kv4_attention_workspace_bytes(2, 2, 8, 4, 128, 64)
    assert need > sk.WORKSPACE_SYNC_BYTES
    assert call(ws=None, n=0) == sk.EINVAL and call(n=need - 1) == sk.ESIZE and call(ws=MIS) == sk.EALIGN
    assert sk.kv4_attention_workspace_bytes(2, 9, 8, 4, 128, 64) == 0
    for bad in ((None, A, A), (A, None, A), (A, A, None)):
        assert L.kv4_attention_weights(c, r, 0, 2, 8, 0.1, *bad, None) == sk.EINVAL
    assert L.kv4_attention_weights(c, r, 0, 2, 8, 0.1, A, MIS, A, None) == sk.EALIGN


def test_evict_refusals():
    L = lib()

    def call(c=_cache(), acc=A, dst=_cache(data=2 * A, lens=0), kept=A, lens=A, new=A, keep=64, sinks=4, recent=8):
        return L.kv4_evict(c, acc, dst, kept, lens, new, keep, sinks, recent, None)
    assert call(dst=_cache()) == sk.EINVAL                     # in place
    assert call(dst=_cache(data=2 * A, Hk=2)) == sk.ESHAPE
    assert call(keep=129) == sk.ESIZE
    for bad in (dict(keep=0), dict(sinks=-1), dict(recent=-1), dict(sinks=60), dict(recent=61), dict(acc=None), dict(kept=None),
                dict(lens=None), dict(new=None)):
        assert call(**bad) == sk.EINVAL, bad
    assert call(acc=MIS) == sk.EALIGN and call(new=MIS) == sk.EALIGN and call(kept=A + 2) == sk.EALIGN


def test_binding_refuses_host_tensors_and_other_types():
    cache = torch.zeros((4, 2, 72 * 64), dtype=torch.uint8)
    with pytest.raises(TypeError):
        sk.kv4._buffer(cache, torch.uint8, cache.shape, "cache", 0)
    with pytest.raises(TypeError):
        sk.kv4._buffer(np.zeros(3), torch.uint8, (3,), "cache", 0)


# ---------------------------------------------------------------- GPU
gpu = pytest.mark.gpu


def _table(rng, B, width, spare=2):
    pages = B * width + spare
    return rng.permutation(pages)[:B * width].reshape(B, width).astype(np.int32), pages


def _random_cache(rng, pages, Hk, D, garbage=False):
    """Full pages of random codes with scales around a half (garbage: any bytes, NaN scales among them)."""
    cache = rng.integers(0, 256, (pages, Hk, 72 * D), dtype=np.uint8)
    if not garbage:
        for at in (32 * D, 68 * D):
            cache[..., at:at + 4 * D] = rng.integers(0x28, 0x36, (pages, Hk, 4 * D))
    return cache


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


APPENDS = [  # type, D, Hk, T, lens, width, gk, gv
    ("f16", 128, 4, 8, [777], 13, 1.0, 0.75),
    ("bf16", 64, 3, 1, [1, 64, 65, 0], 2, 1.0, 1.0),
    ("f16", 256, 2, 5, [3, 200, 66], 4, 0.5, 3.0),
    ("bf16", 128, 1, 200, [130, 200, 391, 7], 7, 1.0, 0.01),
    ("f16", 64, 16, 64, [64, 128, 100], 2, 1.0, 1.0),
    ("bf16", 256, 1, 130, [192, 131], 3, 1.7, 1.0),
]


@gpu
@pytest.mark.parametrize("kind, D, Hk, T, lens, width, gk, gv", APPENDS)
def test_append_and_read(kind, D, Hk, T, lens, width, gk, gv):
    rng = np.random.default_rng(hash((D, Hk, T)) % 1000)
    B = len(lens)
    table, pages = _table(rng, B, width)
    before = _random_cache(rng, pages, Hk, D, garbage=True)
    # Rows lie in a wider tensor, as in a qkv GEMM's output; values of many sizes, zero groups, exact borders.
    kv = torch.from_numpy(rng.standard_normal((B, T, 2 * Hk * D)) * np.exp2(rng.integers(-9, 9, (B, T, 2 * Hk * D // 16)).repeat(16, 2)))
    kv[:, :, :16] = 0.0
    kv[:, T // 2, -16:] = torch.tensor([6.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.25, -5.0, -0.0, 0.0, 0.2499, 5.01, -1.25, 3.51])
    kv[0, T - 1, 20] = float("inf")
    kv[0, T - 1, 40] = float("nan")
    kv = kv.to(TYPES[kind])
    dev = kv.cuda()
    k, v = dev[..., :Hk * D].unflatten(-1, (Hk, D)), dev[..., Hk * D:].unflatten(-1, (Hk, D))
    cache = _cuda(before)
    args = (cache, _cuda(table), _cuda(np.array(lens, np.int32)))
    sk.kv4_append(*args, k, v, gk=gk, gv=gv)
    kr, vr = torch.full((2, B, T + 3, Hk, D), 7.0, dtype=TYPES[kind], device="cuda")
    sk.kv4_read(*args, kr, vr, gk=gk, gv=gv)

    want = before.copy()
    kk, vv = kv[..., :Hk * D].double().numpy().reshape(B, T, Hk, D), kv[..., Hk * D:].double().numpy().reshape(B, T, Hk, D)
    gk, gv = np.float32(gk), np.float32(gv)
    kc, ks = oracle.kv_quantize(kk, gk)
    vc, vs = oracle.kv_quantize(vv, gv)
    for b, n in enumerate(lens):
        for t in range(T):
            s = n - T + t
            if s >= 0:
                for h in range(Hk):
                    oracle.kv_put(want[table[b, s // 64], h], s % 64, kc[b, t, h], ks[b, t, h], vc[b, t, h], vs[b, t, h])
    assert np.array_equal(cache.cpu().numpy(), want)
    for b, n in enumerate(lens):
        for h in range(Hk):
            held = oracle.kv_held(want, table[b], n, h, D, gk, gv)
            for got, ref in zip((kr, vr), held):
                m = min(n, T + 3)
                full = np.concatenate([np.zeros((T + 3 - m, D)), ref[n - m:]])
                # two roundings: to fp32 and to the type
                full = torch.from_numpy(full.astype(np.float32)).to(TYPES[kind]).double()
                assert torch.equal(got[b, :, h].double().cpu().nan_to_num(1e9), full.nan_to_num(1e9))


ATTENDS = [  # type, D, Hq, Hk, T, lens
    ("f16", 128, 48, 4, 1, [301]),
    ("bf16", 128, 48, 4, 8, [1, 5, 300, 1030, 0]),
    ("f16", 256, 24, 4, 8, [513, 64]),
    ("bf16", 256, 5, 1, 3, [200, 2, 65]),
    ("f16", 64, 16, 16, 1, [63, 64, 65, 1, 0, 129]),
    ("bf16", 64, 28, 4, 5, [700, 4]),
    ("f16", 128, 8, 1, 2, [2500]),
    ("bf16", 128, 32, 8, 4, [128, 127, 131, 1]),
    ("f16", 64, 64, 1, 8, [90]),
    ("bf16", 256, 64, 1, 8, [70, 7]),
    ("f16", 128, 2, 2, 1, [1] * 70),
    ("f16", 128, 12, 1, 1, [40000]),
]


def _attend_inputs(rng, kind, D, Hq, Hk, T, lens, q_size=2.0):
    B, width = len(lens), max(1, -(-max(lens) // 64)) + 1
    table, pages = _table(rng, B, width)
    cache = _random_cache(rng, pages, Hk, D)
    garbage = rng.integers(0, 256, cache.shape, dtype=np.uint8)
    for b, n in enumerate(lens):  # any bytes past the lengths, NaN scales among them
        for p in range(width):
            for h in range(Hk):
                if p * 64 >= n:
                    cache[table[b, p], h] = garbage[table[b, p], h]
                elif (p + 1) * 64 > n:
                    k, v, _, ks, vs = oracle.kv_places(D)
                    for at in (k, v, ks, vs):
                        past = at[n % 64:].ravel()
                        cache[table[b, p], h, past] = garbage[table[b, p], h, past]
                    for at in (ks, vs):
                        cache[table[b, p], h, at[63]] = 0x7F
    table[:, -1] = [-1 if b % 2 else 2 ** 31 - 1 for b in range(B)]
    # (the last column of every row is beyond its length unless the longest fills it)
    q = torch.from_numpy(rng.standard_normal((B, T, (Hq + 2 * Hk) * D)) * q_size).to(TYPES[kind])
    return table, cache, q


def _attend_refs(rows, cache, table, lens, q, Hq, Hk, D, T, scale, gk, gv):
    """Yields (b, t, h, out, lse, weights, spread) of the given (b, t, h); q float64 [B, T, Hq, D]."""
    held = {}
    for b, t, h in rows:
        hk = h // (Hq // Hk)
        if (b, hk) not in held:
            held[b, hk] = oracle.kv_held(cache, table[b], lens[b], hk, D, gk, gv)
        k, v, ok = held[b, hk]
        yield (b, t, h, *oracle.kv_attend(q[b, t, h], k, v, ok, lens[b] - (T - 1 - t), scale))


def _check_rows(kind, got, lse, refs, scale_max):
    for b, t, h, out, ref_lse, _, spread in refs:
        x = got[b, t, h].double().cpu().numpy()
        # weights rounded to fp16 (2^-11) and scores off by a few fp32 roundings of numbers up to scale_max
        tol = spread * (2.0 ** -11 + scale_max * 2.0 ** -20) + np.abs(out) * HALF_STEP[kind] + 2.0 ** -24
        nan = np.isnan(out)  # a row whose query holds an infinity
        assert np.array_equal(np.isnan(x), nan), (b, t, h)
        assert (np.abs(x - out) <= tol)[~nan].all(), (b, t, h, np.abs(x - out).max(), tol.min())
        y = float(lse[b, t, h])
        assert (y == ref_lse) or (np.isnan(y) and np.isnan(ref_lse)) or abs(y - ref_lse) <= 2.0 ** -20 * (scale_max + 1), (b, t, h, y, ref_lse)


@gpu
@pytest.mark.parametrize("kind, D, Hq, Hk, T, lens", ATTENDS)
def test_attention_and_weights(kind, D, Hq, Hk, T, lens):
    rng = np.random.default_rng(D + Hq + T)
    table, cache, qkv = _attend_inputs(rng, kind, D, Hq, Hk, T, lens)
    B, width = table.shape
    scale, gk, gv = float(np.float32(D ** -0.5)), 1.5, 0.75
    dev = qkv.cuda()
    q = dev[..., :Hq * D].unflatten(-1, (Hq, D))
    out = torch.full((B, T, Hq, D), 3.0, dtype=TYPES[kind], device="cuda")
    lse = torch.full((B, T, Hq), 3.0, device="cuda")
    args = (_cuda(cache), _cuda(table), _cuda(np.array(lens, np.int32)))
    ws = sk.new_workspace(sk.kv4_attention_workspace_bytes(B, T, Hq, Hk, D, width), fill=0xFF)
    for _ in range(2):  # a workspace serves again
        sk.kv4_attention(q, *args, out, lse=lse, scale=scale, gk=gk, gv=gv, workspace=ws)
    first = out.clone()
    sk.kv4_attention(q, *args, out, scale=scale, gk=gk, gv=gv, workspace=ws)
    assert torch.equal(first.view(torch.int16), out.view(torch.int16))
    qd = q.double().cpu().numpy()
    rows = [(b, t, h) for b in range(B) for t in range(T) for h in range(Hq)]
    if len(rows) > 400:
        rows = [rows[i] for i in sorted(rng.permutation(len(rows))[:400])]
    refs = list(_attend_refs(rows, cache, table, lens, qd, Hq, Hk, D, T, scale, gk, gv))
    _check_rows(kind, out, lse, refs, 64.0)

    acc = torch.rand((B, Hk, 64 * width), device="cuda") * 4
    acc_out = torch.full_like(acc, 9.0)
    sk.kv4_attention_weights(q, *args, lse, acc, acc_out, scale=scale, gk=gk)
    want = np.zeros((B, Hk, 64 * width))
    for b, n in enumerate(lens):
        want[b, :, :n] = acc[b, :, :n].double().cpu().numpy()
    everything = ((b, t, h) for b in range(B) for t in range(T) for h in range(Hq))
    if B * T * Hq * max(lens) <= 4e6:
        for b, t, h, _, _, w, _ in _attend_refs(everything, cache, table, lens, qd, Hq, Hk, D, T, scale, gk, gv):
            want[b, h // (Hq // Hk), :len(w)] += w
        err = np.abs(acc_out.double().cpu().numpy() - want)
        assert (err <= want * (64 * 2.0 ** -20)).all(), err.max()
    again = acc.clone()  # in place
    sk.kv4_attention_weights(q, *args, lse, again, again, scale=scale, gk=gk)
    assert torch.equal(again, acc_out)


@gpu
def test_a_missing_page_is_skipped():
    rng = np.random.default_rng(5)
    lens, D, Hq, Hk, T = [200, 250], 128, 8, 2, 2
    table, cache, qkv = _attend_inputs(rng, "f16", D, Hq, Hk, T, lens)
    table[0, 1], table[1, 0], table[1, 3] = -1, len(cache), 2 ** 31 - 1
    B, width = table.shape
    q = qkv.cuda()[..., :Hq * D].unflatten(-1, (Hq, D))
    args = (_cuda(cache), _cuda(table), _cuda(np.array(lens, np.int32)))
    out, lse = torch.empty((B, T, Hq, D), dtype=torch.float16, device="cuda"), torch.empty((B, T, Hq), device="cuda")
    ws = sk.new_workspace(sk.kv4_attention_workspace_bytes(B, T, Hq, Hk, D, width))
    sk.kv4_attention(q, *args, out, lse=lse, workspace=ws)
    rows = [(b, t, h) for b in range(B) for t in range(T) for h in range(Hq)]
    refs = list(_attend_refs(rows, cache, table, lens, q.double().cpu().numpy(), Hq, Hk, D, T, D ** -0.5, 1.0, 1.0))
    _check_rows("f16", out, lse, refs, 64.0)
    acc = torch.ones((B, Hk, 64 * width), device="cuda")
    got = torch.empty_like(acc)
    sk.kv4_attention_weights(q, *args, lse, acc, got)
    assert (got[0, :, 64:128] == 1).all() and (got[1, :, :64] == 1).all() and (got[1, :, 250:] == 0).all()
    held = torch.full((2, B, 250, Hk, D), 5.0, dtype=torch.float16, device="cuda")
    sk.kv4_read(*args, held[0], held[1])
    assert (held[:, 0, 50 + 64:50 + 128] == 0).all() and (held[:, 1, :64] == 0).all()
    before = args[0].clone()
    x = torch.ones((B, 150, Hk, D), dtype=torch.float16, device="cuda")
    sk.kv4_append(*args, x, x)  # rows whose page is missing are dropped
    changed = (args[0] != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert set(changed) <= {table[0, 0], table[0, 2], table[0, 3], table[1, 1], table[1, 2]}


@gpu
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_nan_value_reaches_only_the_rows_that_see_it(D):
    rng = np.random.default_rng(6)
    T, Hq, Hk, lens = 8, 12, 2, [100]
    table, cache, qkv = _attend_inputs(rng, "f16", D, Hq, Hk, T, lens)
    _, _, _, _, vs = oracle.kv_places(D)
    cache[table[0, 1], :, vs[97 - 64, 0]] = 0x7F  # slot 97: rows 5, 6 and 7 see it
    q = qkv.cuda()[..., :Hq * D].unflatten(-1, (Hq, D))
    args = (_cuda(cache), _cuda(table), _cuda(np.array(lens, np.int32)))
    out, lse = torch.empty((1, T, Hq, D), dtype=torch.float16, device="cuda"), torch.empty((1, T, Hq), device="cuda")
    sk.kv4_attention(q, *args, out, lse=lse, workspace=sk.new_workspace(sk.kv4_attention_workspace_bytes(1, T, Hq, Hk, D, table.shape[1])))
    assert out[:, 5:, :, :16].isnan().all() and not out[:, :5].isnan().any() and not lse.isnan().any()
    rows = [(0, t, h) for t in range(5) for h in range(Hq)]
    refs = list(_attend_refs(rows, cache, table, lens, q.double().cpu().numpy(), Hq, Hk, D, T, D ** -0.5, 1.0, 1.0))
    _check_rows("f16", out, lse, refs, 64.0)


@gpu
@pytest.mark.parametrize("kind, size", [("f16", 3e4), ("bf16", 1e30), ("bf16", 1e-30), ("f16", 1e-7)])
def test_queries_of_extreme_size(kind, size):
    """Scores far beyond the usual: one slot takes all, or all the same."""
    rng = np.random.default_rng(7)
    lens, D, Hq, Hk, T = [150], 128, 4, 1, 2
    table, cache, qkv = _attend_inputs(rng, kind, D, Hq, Hk, T, lens, q_size=size)
    q = qkv.cuda()[..., :Hq * D].unflatten(-1, (Hq, D))
    scale = float(np.float32(1.0 / size)) if size > 1 else 1.0
    args = (_cuda(cache), _cuda(table), _cuda(np.array(lens, np.int32)))
    out, lse = torch.empty((1, T, Hq, D), dtype=TYPES[kind], device="cuda"), torch.empty((1, T, Hq), device="cuda")
    sk.kv4_attention(q, *args, out, lse=lse, scale=scale, workspace=sk.new_workspace(sk.kv4_attention_workspace_bytes(1, T, Hq, Hk, D, table.shape[1])))
    refs = list(_attend_refs([(0, t, h) for t in range(T) for h in range(Hq)], cache, table, lens, q.double().cpu().numpy(), Hq, Hk, D, T, scale, 1.0, 1.0))
    _check_rows(kind, out, lse, refs, 128.0)


@gpu
def test_offsets_past_32_bits():
    D, Hk, Hq, T, n = 128, 2, 8, 3, 190
    pages = (1 << 32) // (Hk * 72 * D) + 64
    rng = np.random.default_rng(8)
    small, qkv = _random_cache(rng, 4, Hk, D), torch.from_numpy(rng.standard_normal((1, T, Hq, D))).half()
    cache = torch.empty((pages, Hk, 72 * D), dtype=torch.uint8, device="cuda")
    ids = np.array([[pages - 1, pages - 9, pages - 2, pages - 40]], np.int32)
    for i, p in enumerate(ids[0]):
        cache[p] = _cuda(small[i])
    q, lens = qkv.cuda(), _cuda(np.array([n], np.int32))
    x = torch.randn((1, T, Hk, D), device="cuda").half()
    small_args = (_cuda(small), _cuda(np.arange(4, dtype=np.int32)[None]), lens)
    args = (cache, _cuda(ids), lens)
    got = []
    for a in (args, small_args):
        sk.kv4_append(*a, x, x)
        out, lse, held = torch.empty_like(q), torch.empty((1, T, Hq), device="cuda"), torch.empty((2, 1, n, Hk, D), dtype=torch.float16, device="cuda")
        sk.kv4_attention(q, *a, out, lse=lse, workspace=sk.new_workspace(sk.kv4_attention_workspace_bytes(1, T, Hq, Hk, D, 4)))
        sk.kv4_read(*a, held[0], held[1])
        w = torch.zeros((1, Hk, 256), device="cuda")
        sk.kv4_attention_weights(q, *a, lse, w, w)
        dst, kept, m, acc = torch.zeros((2, Hk, 72 * D), dtype=torch.uint8, device="cuda"), torch.empty((1, Hk, 70), dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty((1, Hk, 128), device="cuda")
        sk.kv4_evict(*a, w, dst, _cuda(np.array([[1, 0]], np.int32)), kept, m, acc, sinks=2, recent=8)
        got.append((out, lse, held, w, dst, kept, m, acc))
    for a, b in zip(*got):
        assert torch.equal(a, b)


EVICTS = [  # D, Hk, lens, keep, sinks, recent, weights
    (128, 4, [300, 64, 20], 64, 4, 16, "exp"),
    (64, 2, [1000, 65, 66, 0], 65, 0, 0, "exp"),
    (256, 1, [130], 1, 0, 0, "exp"),
    (128, 2, [500], 100, 100, 0, "exp"),
    (128, 2, [500], 100, 0, 100, "exp"),
    (64, 3, [777], 500, 10, 20, "equal"),
    (64, 3, [777], 300, 10, 20, "zeros"),
    (64, 1, [5000], 4096, 0, 1, "few"),
    (64, 1, [40000], 9000, 4, 64, "wild"),
]


@gpu
@pytest.mark.parametrize("D, Hk, lens, keep, sinks, recent, weights", EVICTS)
def test_evict(D, Hk, lens, keep, sinks, recent, weights):
    rng = np.random.default_rng(keep + sinks)
    B, width = len(lens), max(1, -(-max(lens) // 64))
    table, pages = _table(rng, B, width)
    cache = _random_cache(rng, pages, Hk, D, garbage=True)
    dwidth = -(-keep // 64) + 1
    dtable, dpages = _table(rng, B, dwidth)
    shape = (B, Hk, 64 * width)
    acc = {"exp": lambda: rng.exponential(size=shape) * (rng.random(shape) < 0.8), "equal": lambda: np.full(shape, 2.5),
           "zeros": lambda: (rng.random(shape) < 0.1) * rng.random(shape), "few": lambda: rng.integers(0, 3, shape) * 1.0,
           "wild": lambda: np.where(rng.random(shape) < 0.01, np.nan, np.where(rng.random(shape) < 0.01, np.inf, np.exp2(rng.uniform(-140, 120, shape))))}[weights]().astype(np.float32)
    dst = np.full((dpages, Hk, 72 * D), 0xAB, np.uint8)
    d = _cuda(dst)
    kept = torch.full((B, Hk, keep), 77, dtype=torch.int32, device="cuda")
    new_lens = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    new_acc = torch.full((B, Hk, 64 * dwidth), 77.0, device="cuda")
    sk.kv4_evict(_cuda(cache), _cuda(table), _cuda(np.array(lens, np.int32)), _cuda(acc), d, _cuda(dtable), kept, new_lens, new_acc, sinks=sinks, recent=recent)
    assert new_lens.tolist() == [min(n, keep) for n in lens]
    got, kept, new_acc = d.cpu().numpy(), kept.cpu().numpy(), new_acc.cpu().numpy()
    k, v, nib, ks, vs = oracle.kv_places(D)
    touched = set()
    for b, n in enumerate(lens):
        for h in range(Hk):
            at = oracle.kv_evict(acc[b, h], n, keep, sinks, recent)
            m = len(at)
            assert np.array_equal(kept[b, h], np.concatenate([at, np.full(keep - m, -1)]))
            assert np.array_equal(new_acc[b, h], np.concatenate([acc[b, h, at], np.zeros(64 * dwidth - m, np.float32)]), equal_nan=True)
            for p in range(-(-m // 64)):
                want = np.zeros(72 * D, np.uint8)
                touched.add(dtable[b, p])
                for t, s in enumerate(at[64 * p:64 * p + 64]):
                    src = cache[table[b, s // 64], h]
                    for place in (k, v):
                        want[place[t][::2]] = src[place[s % 64][::2]]
                    for place in (ks, vs):
                        want[place[t][::16]] = src[place[s % 64][::16]]
                assert np.array_equal(got[dtable[b, p], h], want)
    for p in set(range(dpages)) - touched:
        assert (got[p] == 0xAB).all()


@gpu
def test_lens_beyond_the_table_and_below_zero_are_clamped():
    rng = np.random.default_rng(9)
    D, Hk, Hq, T = 64, 1, 4, 2
    table, pages = _table(rng, 2, 2)
    args = lambda lens: (_cuda(cache), _cuda(table), _cuda(np.array(lens, np.int32)))  # noqa: E731
    cache = _random_cache(rng, pages, Hk, D)
    q = torch.randn((2, T, Hq, D), device="cuda").half()
    got = []
    for lens in ([1000, -5], [128, 0]):
        out, lse = torch.empty_like(q), torch.empty((2, T, Hq), device="cuda")
        sk.kv4_attention(q, *args(lens), out, lse=lse, workspace=sk.new_workspace(sk.kv4_attention_workspace_bytes(2, T, Hq, Hk, D, 2)))
        acc = torch.ones((2, Hk, 128), device="cuda")
        sk.kv4_attention_weights(q, *args(lens), lse, acc, acc)
        held = torch.empty((2, 2, 130, Hk, D), dtype=torch.float16, device="cuda")
        sk.kv4_read(*args(lens), held[0], held[1])
        got.append((out, lse, acc, held))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert (got[0][0][1] == 0).all() and (got[0][1][1] == -float("inf")).all() and (got[0][2][1] == 0).all()


@gpu
def test_a_step_replayed_from_a_graph_on_another_stream():
    """append, attention and weights captured together: every replay gives the eager step's results."""
    rng = np.random.default_rng(10)
    D, Hk, Hq, T, lens = 128, 4, 48, 4, [900, 130, 64]
    table, cache, qkv = _attend_inputs(rng, "bf16", D, Hq, Hk, T, lens)
    B, width = table.shape
    args = (_cuda(cache), _cuda(table), _cuda(np.array(lens, np.int32)))
    dev = qkv.cuda()
    heads = lambda a, n: dev[..., a * D:(a + n) * D].unflatten(-1, (n, D))  # noqa: E731
    q, k, v = heads(0, Hq), heads(Hq, Hk), heads(Hq + Hk, Hk)
    ws = sk.new_workspace(sk.kv4_attention_workspace_bytes(B, T, Hq, Hk, D, width))
    out, lse = torch.empty((B, T, Hq, D), dtype=torch.bfloat16, device="cuda"), torch.empty((B, T, Hq), device="cuda")
    acc, acc_out = torch.rand((B, Hk, 64 * width), device="cuda"), torch.empty((B, Hk, 64 * width), device="cuda")

    def step():
        sk.kv4_append(*args, k, v)
        sk.kv4_attention(q, *args, out, lse=lse, workspace=ws)
        sk.kv4_attention_weights(q, *args, lse, acc, acc_out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        dev.copy_(torch.randn(dev.shape, device="cuda"))
        out.fill_(5.0), lse.fill_(5.0), acc_out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, lse, acc_out, args[0])]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (out, lse, acc_out, args[0])):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i
