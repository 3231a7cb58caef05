"""Attention of chunks of new tokens over the 4-bit cache, against its definition in 64 bits."""

import numpy as np
import pytest
import torch

import fp8_quantized_skinny_amd as sk
from fp8_quantized_skinny_amd._lib import lib
from oracle import kv4 as oracle
from test_kv4 import A, BAD_CACHES, HALF_STEP, MIS, TYPES, _attend_inputs, _cache, _cuda, _random_cache

gpu = pytest.mark.gpu


# ---------------------------------------------------------------- refusals (no GPU)
Q, O, W = 0x1000000, 0x2000000, 0x100000000


def _call(c=None, q=Q, row=1024, head=128, starts=0x600000, N=20, type=0, Hq=8, scale=0.1, window=0, sinks=0, out=O, lse=0x5000000, ws=W, n=1 << 40):
    return lib().kv4_attention_chunk(c or _cache(table=0x700000, lens=0x710000, width=100), q, row, head, starts, N, type, Hq, scale, window, sinks, out, lse, ws, n, None)


@pytest.mark.parametrize("bad, status", BAD_CACHES)
def test_cache_refusals(bad, status):
    assert _call(c=_cache(**bad)) == status


@pytest.mark.parametrize("bad, status", [
    (dict(q=None), sk.EINVAL), (dict(q=Q + 8), sk.EALIGN), (dict(row=-8), sk.EINVAL), (dict(head=4), sk.EALIGN), (dict(row=1028), sk.EALIGN),
    (dict(starts=None), sk.EINVAL), (dict(starts=A + 2), sk.EALIGN), (dict(N=0), sk.ESHAPE), (dict(N=1 << 30, Hq=8), sk.ESHAPE),
    (dict(type=2), sk.EINVAL), (dict(Hq=0), sk.ESHAPE), (dict(Hq=6), sk.ESHAPE), (dict(Hq=4 * 65), sk.ESHAPE), (dict(scale=0.0), sk.EINVAL),
    (dict(scale=float("nan")), sk.EINVAL), (dict(window=-1), sk.EINVAL), (dict(sinks=-1), sk.EINVAL), (dict(out=None), sk.EINVAL),
    (dict(out=O + 8), sk.EALIGN), (dict(lse=A + 2), sk.EALIGN), (dict(ws=None), sk.EINVAL), (dict(ws=MIS), sk.EALIGN), (dict(n=1000), sk.ESIZE),
    # what overlaps: out and a part of q, lse and out, an output and the cache, its table, lens, starts or the workspace
    (dict(out=Q + 16), sk.EINVAL), (dict(out=Q, row=2048), sk.EINVAL), (dict(lse=O + 64), sk.EINVAL), (dict(lse=Q), sk.EINVAL), (dict(out=A), sk.EINVAL),
    (dict(lse=0x700000), sk.EINVAL), (dict(lse=0x710004), sk.EINVAL), (dict(lse=0x600008), sk.EINVAL), (dict(out=W + (1 << 17)), sk.EINVAL)])
def test_refusals(bad, status):
    assert _call(**bad) == status


def test_workspaces():
    size = sk.kv4_attention_chunk_workspace_bytes
    # none for few rows over few pages
    assert size(64, 3, 8, 4, 128, 96) == 0 and size(64, 3, 8, 4, 128, 97) > sk.WORKSPACE_SYNC_BYTES and size(64, 3, 8, 4, 128, 5000, 1000, 4) == 0
    assert size(40000, 3, 8, 4, 128, 64) > sk.WORKSPACE_SYNC_BYTES
    # by the pages that can be seen, not by a wide table
    assert size(64, 1, 8, 4, 128, 5000, 6000, 4) == size(64, 1, 8, 4, 128, 300, 6000, 4) < size(64, 1, 8, 4, 128, 5000)
    assert size(64, 1, 8, 4, 128, 100, 6400, 4) == size(64, 1, 8, 4, 128, 100) > 0
    for bad in ((0, 1, 8, 4, 128, 1), (1, 0, 8, 4, 128, 1), (1, 1, 7, 4, 128, 1), (1, 1, 8, 4, 96, 1), (1, 1, 8, 4, 128, 0), (1 << 30, 1, 8, 4, 128, 1),
                (1, 1, 8, 4, 128, 1, -1), (1, 1, 8, 4, 128, 1, 5, -1)):
        assert size(*bad) == 0, bad


# ---------------------------------------------------------------- GPU
CHUNKS = [  # type, D, Hq, Hk, chunks, lens, window, sinks
    ("f16", 128, 48, 4, [17], [301], 0, 0),
    ("bf16", 128, 48, 4, [8, 1, 0, 40, 100], [1000, 5, 300, 40, 64], 0, 0),
    ("f16", 256, 24, 4, [70, 3], [513, 3], 0, 0),
    ("bf16", 256, 5, 1, [130, 2, 61], [200, 2, 65], 0, 0),
    ("f16", 64, 16, 16, [300, 1, 64, 65], [300, 64, 700, 65], 0, 0),   # 300 rows: two tiles
    ("bf16", 64, 28, 4, [50, 9], [700, 4], 0, 0),                       # more new tokens than slots
    ("f16", 128, 8, 1, [33], [2500], 0, 0),                             # a split tile
    ("bf16", 64, 64, 1, [5, 4], [90, 64], 0, 0),
    ("f16", 128, 1, 1, [600, 10], [640, 10], 0, 0),                     # one head: three tiles
    ("f16", 128, 12, 1, [2], [40000], 0, 0),
    ("bf16", 128, 32, 8, [1] * 70, list(range(70)), 0, 0),              # more sequences than lanes
    ("f16", 128, 48, 4, [40, 90], [3010, 500], 1024, 4),
    ("bf16", 128, 8, 2, [300, 7, 1], [700, 600, 64], 100, 70),
    ("f16", 256, 24, 4, [90, 5], [513, 700], 64, 64),
    ("bf16", 256, 4, 1, [200], [400], 1, 0),
    ("f16", 64, 16, 16, [290, 64], [1000, 64], 1, 1),
    ("bf16", 64, 28, 4, [100], [3000], 1900, 130),                      # a window whose tiles are split
    ("f16", 64, 2, 2, [520], [520], 63, 0),
    ("f16", 64, 8, 2, [60, 40], [400, 40], 5000, 9),
    ("bf16", 128, 8, 2, [60, 30], [600, 300], 32, 2 ** 31 - 1),
]


# Three ways: few rows over few pages, few rows over a table of more than 96 pages, and many rows (most of them no sequence's).
WIDE = pytest.mark.parametrize("wide", [False, True, "tall"])


def _inputs(rng, kind, D, Hq, Hk, chunks, lens, wide, pad=3, q_size=2.0):
    """Pages as for the steps of a few rows, a wide table with 100 columns more that name none; packed queries in a qkv
    GEMM's output, `pad` rows before the first and behind the last, and more of these where it is tall."""
    table, cache, _ = _attend_inputs(rng, kind, D, Hq, Hk, 1, lens)
    if wide:
        table = np.concatenate([table, np.full((len(lens), 100), -1, np.int32)], 1)
    N = sum(chunks) + 2 * pad + (500 * len(chunks) * Hk // Hq + 1 if wide == "tall" else 0)
    qkv = torch.from_numpy(rng.standard_normal((N, (Hq + 2 * Hk) * D)) * q_size).to(TYPES[kind])
    starts = pad + np.concatenate([[0], np.cumsum(chunks)]).astype(np.int32)
    return table, cache, qkv, starts


def _refs(rows, cache, table, lens, starts, q, Hq, Hk, D, scale, gk, gv, window, sinks):
    held = {}
    for b, i, h in rows:
        hk = h // (Hq // Hk)
        if (b, hk) not in held:
            held[b, hk] = oracle.kv_held(cache, table[b], lens[b], hk, D, gk, gv)
        k, v, ok = held[b, hk]
        T = starts[b + 1] - starts[b]
        limit = lens[b] - (T - 1 - i)
        yield (starts[b] + i, h, *oracle.kv_attend(q[starts[b] + i, h], k, v, ok & oracle.in_window(len(k), limit, window, sinks), limit, scale))


def _check(kind, out, lse, refs, scale_max=64.0):
    out, lse = out.double().cpu().numpy(), lse.cpu().numpy()
    for r, h, want, ref_lse, _, spread in refs:
        # weights rounded to fp16 (2^-11) and scores off by a few fp32 roundings of numbers up to scale_max
        tol = spread * (2.0 ** -11 + scale_max * 2.0 ** -20) + np.abs(want) * HALF_STEP[kind] + 2.0 ** -24
        x, nan = out[r, h], np.isnan(want)
        assert np.array_equal(np.isnan(x), nan), (r, h)
        assert (np.abs(x - want) <= tol)[~nan].all(), (r, h, np.abs(x - want).max(), tol.min())
        y = float(lse[r, h])
        assert (y == ref_lse) or (np.isnan(y) and np.isnan(ref_lse)) or abs(y - ref_lse) <= 2.0 ** -20 * (scale_max + 1), (r, h, y, ref_lse)


def _some(rng, chunks, Hq, most=300):
    rows = [(b, i, h) for b, n in enumerate(chunks) for i in range(n) for h in range(Hq)]
    if len(rows) > most:
        edge = [(b, i, rng.integers(Hq)) for b, n in enumerate(chunks) if n for i in (0, n - 1)]
        rows = [rows[i] for i in sorted(rng.permutation(len(rows))[:most - len(edge)])] + edge
    return rows


@gpu
@WIDE
@pytest.mark.parametrize("kind, D, Hq, Hk, chunks, lens, window, sinks", CHUNKS)
def test_chunks(kind, D, Hq, Hk, chunks, lens, window, sinks, wide):
    rng = np.random.default_rng(D + Hq + sum(chunks) + window)
    table, cache, qkv, starts = _inputs(rng, kind, D, Hq, Hk, chunks, lens, wide)
    B, width = table.shape
    for b, n in enumerate(lens):  # pages that no row sees: NaN and pages that are none
        for p in range(-(-sinks // 64), max(0, n - chunks[b] + 1 - window) // 64 if window and chunks[b] else 0):
            cache[table[b, p]] = 0xFF
            if p % 2:
                table[b, p] = -1
    N, scale, gk, gv = len(qkv), float(np.float32(D ** -0.5)), 1.5, 0.75
    q = qkv.cuda()[:, :Hq * D].unflatten(-1, (Hq, D))
    out, lse = torch.full((N, Hq, D), 3.0, dtype=TYPES[kind], device="cuda"), torch.full((N, Hq), 3.0, device="cuda")
    args = (_cuda(starts), _cuda(cache), _cuda(table), _cuda(np.array(lens, np.int32)))
    ws = sk.new_workspace(sk.kv4_attention_chunk_workspace_bytes(N, B, Hq, Hk, D, width, window, sinks), fill=0xFF)
    more = dict(scale=scale, window=window, sinks=sinks, gk=gk, gv=gv, workspace=ws)
    for _ in range(2):  # a workspace serves again
        sk.kv4_attention_chunk(q, *args, out, lse=lse, **more)
    assert ws is None or (ws[:sk.WORKSPACE_SYNC_BYTES] == 0).all()
    assert ws is not None or not wide or window
    for t in (out, lse):  # rows that no sequence has
        assert (t[:starts[0]] == 3).all() and (t[starts[-1]:] == 3).all()
    again = torch.full_like(out, 4.0)
    again[:starts[0]], again[starts[-1]:] = 3.0, 3.0
    sk.kv4_attention_chunk(q, *args, again, **more)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))
    same = q.contiguous()  # in place
    sk.kv4_attention_chunk(same, *args, same, **more)
    assert torch.equal(same[starts[0]:starts[-1]].view(torch.int16), out[starts[0]:starts[-1]].view(torch.int16))
    _check(kind, out, lse, _refs(_some(rng, chunks, Hq), cache, table, lens, starts, q.double().cpu().numpy(), Hq, Hk, D, scale, gk, gv, window, sinks))


@gpu
@WIDE
def test_a_prompt_agrees_with_its_last_rows_one_by_one(wide):
    """A long prompt's rows against kv4_attention of the same rows, eight at a time."""
    rng = np.random.default_rng(2)
    D, Hq, Hk, n = 128, 16, 2, 1500
    table, cache, qkv, starts = _inputs(rng, "bf16", D, Hq, Hk, [n], [n], wide, pad=0)
    q = qkv.cuda()[:n, :Hq * D].unflatten(-1, (Hq, D))
    c, t = _cuda(cache), _cuda(table)
    out, lse = torch.empty((n, Hq, D), dtype=torch.bfloat16, device="cuda"), torch.empty((n, Hq), device="cuda")
    ws = sk.new_workspace(sk.kv4_attention_chunk_workspace_bytes(n, 1, Hq, Hk, D, table.shape[1]))
    sk.kv4_attention_chunk(q, _cuda(starts), c, t, _cuda(np.array([n], np.int32)), out, lse=lse, workspace=ws)
    few, few_lse = torch.empty((1, 8, Hq, D), dtype=torch.bfloat16, device="cuda"), torch.empty((1, 8, Hq), device="cuda")
    ws = sk.new_workspace(sk.kv4_attention_workspace_bytes(1, 8, Hq, Hk, D, table.shape[1]))
    for end in list(range(8, 280, 8)) + [512, 1024, n]:
        sk.kv4_attention(q[end - 8:end][None], c, t, _cuda(np.array([end], np.int32)), few, lse=few_lse, workspace=ws)
        # both off by the roundings that _check counts, of values up to 6 * 1.75
        assert (out[end - 8:end].float() - few[0].float()).abs().max() <= 2 * 10.5 * (2.0 ** -8 + 2.0 ** -11)
        assert (lse[end - 8:end] - few_lse[0]).abs().max() <= 2 * 2.0 ** -14


@gpu
@WIDE
def test_a_missing_page_is_skipped(wide):
    rng = np.random.default_rng(5)
    chunks, lens, D, Hq, Hk = [100, 30], [200, 2000], 128, 8, 2
    table, cache, qkv, starts = _inputs(rng, "f16", D, Hq, Hk, chunks, lens, wide)
    table[0, 1], table[0, 3], table[1, 0], table[1, 7:20] = -1, 2 ** 31 - 1, len(cache), -7
    q = qkv.cuda()[:, :Hq * D].unflatten(-1, (Hq, D))
    out, lse = torch.empty(q.shape, dtype=torch.float16, device="cuda"), torch.empty(q.shape[:2], device="cuda")
    ws = sk.new_workspace(sk.kv4_attention_chunk_workspace_bytes(len(qkv), 2, Hq, Hk, D, table.shape[1]))
    sk.kv4_attention_chunk(q, _cuda(starts), _cuda(cache), _cuda(table), _cuda(np.array(lens, np.int32)), out, lse=lse, workspace=ws)
    _check("f16", out, lse, _refs(_some(rng, chunks, Hq), cache, table, lens, starts, q.double().cpu().numpy(), Hq, Hk, D, D ** -0.5, 1.0, 1.0, 0, 0))


@gpu
@WIDE
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window, sinks", [(0, 0), (40, 3)])
def test_a_nan_value_reaches_only_the_rows_that_see_it(D, window, sinks, wide):
    rng = np.random.default_rng(6)
    chunks, lens, Hq, Hk = [70], [200], 12, 2
    table, cache, qkv, starts = _inputs(rng, "f16", D, Hq, Hk, chunks, lens, wide)
    places = oracle.kv_places(D)
    for s, at in ((150, places[4][150 % 64, D - 16]), (2, places[4][2, 0]), (133, places[4][133 % 64, 16])):
        cache[table[0, s // 64], :, at] = 0x7F
    cache[table[0, 2], :, places[3][190 - 128, 0]] = 0xFF  # a NaN key: all of the rows that see it
    q = qkv.cuda()[:, :Hq * D].unflatten(-1, (Hq, D))
    out, lse = torch.empty(q.shape, dtype=torch.float16, device="cuda"), torch.empty(q.shape[:2], device="cuda")
    ws = sk.new_workspace(sk.kv4_attention_chunk_workspace_bytes(len(qkv), 1, Hq, Hk, D, table.shape[1], window, sinks))
    for _ in range(2):
        sk.kv4_attention_chunk(q, _cuda(starts), _cuda(cache), _cuda(table), _cuda(np.array(lens, np.int32)), out, lse=lse, window=window,
                               sinks=sinks, workspace=ws)
    for i in range(70):
        limit = 131 + i
        see = oracle.in_window(200, limit, window, sinks)
        x, want = out[starts[0] + i].isnan(), np.zeros(D, bool)
        want[D - 16:] |= see[150]
        want[:16] |= see[2]
        want[16:32] |= see[133]
        want |= see[190]
        assert (x.cpu().numpy() == want).all(), i
        assert lse[starts[0] + i].isnan().all() == see[190], i


@gpu
@WIDE
def test_starts_that_fall_or_leave_the_rows(wide):
    """Rows never belong to two sequences, and none outside q is touched."""
    rng = np.random.default_rng(7)
    D, Hq, Hk, lens = 64, 4, 2, [70, 80, 90, 100]
    table, cache, qkv, _ = _inputs(rng, "f16", D, Hq, Hk, [50], lens, wide, pad=0)
    N = len(qkv)
    q = qkv.cuda()[:, :Hq * D].unflatten(-1, (Hq, D))
    args = (_cuda(cache), _cuda(table), _cuda(np.array(lens, np.int32)))
    ws = sk.new_workspace(sk.kv4_attention_chunk_workspace_bytes(N, 4, Hq, Hk, D, table.shape[1]))

    def run(starts):
        out, lse = torch.full(q.shape, 3.0, dtype=torch.float16, device="cuda"), torch.full(q.shape[:2], 3.0, device="cuda")
        sk.kv4_attention_chunk(q, _cuda(np.array(starts, np.int32)), *args, out, lse=lse, workspace=ws)
        return out, lse
    for bad, good in (([10, 30, 20, 25, 40], [10, 30, 30, 30, 40]), ([-5, 5, 2 ** 31 - 1, 7, N + 10], [0, 5, N, N, N]),
                      ([-2 ** 31] * 5, [0] * 5), ([N + 10, 10, 20, 30, 40], [N] * 5), ([5, 4, 3, 2, 50], [5, 5, 5, 5, 50])):
        for a, b in zip(run(bad), run(good)):
            assert torch.equal(a, b), bad
    assert (run([0] * 5)[0] == 3).all()


@gpu
@pytest.mark.parametrize("wide", [False, True])
def test_lens_beyond_the_table_and_below_zero_are_clamped(wide):
    rng = np.random.default_rng(9)
    D, Hk, Hq = 64, 1, 4
    table, cache, qkv, starts = _inputs(rng, "f16", D, Hq, Hk, [20, 20], [128, 100], False, pad=0)
    table = np.repeat(table[:, :2], 50 if wide else 1, 1)  # (pages may be named twice)
    n = 64 * table.shape[1]
    q = qkv.cuda()[:, :Hq * D].unflatten(-1, (Hq, D))
    ws = sk.new_workspace(sk.kv4_attention_chunk_workspace_bytes(40, 2, Hq, Hk, D, table.shape[1]))
    assert (ws is not None) == wide
    got = []
    for lens in ([n + 1000, -5], [n, 0]):
        out, lse = torch.empty(q.shape, dtype=torch.float16, device="cuda"), torch.empty(q.shape[:2], device="cuda")
        sk.kv4_attention_chunk(q, _cuda(starts), _cuda(cache), _cuda(table), _cuda(np.array(lens, np.int32)), out, lse=lse, workspace=ws)
        got.append((out, lse))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert (got[0][0][20:] == 0).all() and (got[0][1][20:] == -float("inf")).all()


@gpu
@WIDE
@pytest.mark.parametrize("kind, size", [("f16", 3e4), ("bf16", 1e30), ("bf16", 1e-30), ("f16", 1e-7)])
def test_queries_of_extreme_size(kind, size, wide):
    """Scores far beyond the usual: one slot takes all, or all the same."""
    rng = np.random.default_rng(7)
    chunks, lens, D, Hq, Hk = [40], [150], 128, 4, 1
    table, cache, qkv, starts = _inputs(rng, kind, D, Hq, Hk, chunks, lens, wide, q_size=size)
    qkv[5, :D] = 0.0
    q = qkv.cuda()[:, :Hq * D].unflatten(-1, (Hq, D))
    q.clamp_(-6e4, 6e4) if kind == "f16" else None  # infinite queries are tested by themselves
    scale = float(np.float32(1.0 / size)) if size > 1 else 1.0
    out, lse = torch.empty(q.shape, dtype=TYPES[kind], device="cuda"), torch.empty(q.shape[:2], device="cuda")
    ws = sk.new_workspace(sk.kv4_attention_chunk_workspace_bytes(len(qkv), 1, Hq, Hk, D, table.shape[1]))
    sk.kv4_attention_chunk(q, _cuda(starts), _cuda(cache), _cuda(table), _cuda(np.array(lens, np.int32)), out, lse=lse, scale=scale, workspace=ws)
    _check(kind, out, lse, _refs(_some(rng, chunks, Hq), cache, table, lens, starts, q.double().cpu().numpy(), Hq, Hk, D, scale, 1.0, 1.0, 0, 0), 128.0)


@gpu
@WIDE
def test_infinite_and_nan_queries_stay_in_their_rows(wide):
    rng = np.random.default_rng(8)
    chunks, lens, D, Hq, Hk = [40], [150], 64, 2, 1
    table, cache, qkv, starts = _inputs(rng, "f16", D, Hq, Hk, chunks, lens, wide)
    clean = qkv.clone()
    qkv[10, 3], qkv[20, 5] = float("inf"), float("nan")
    got = []
    for x in (qkv, clean):
        q = x.cuda()[:, :Hq * D].unflatten(-1, (Hq, D))
        out, lse = torch.full(q.shape, 3.0, dtype=torch.float16, device="cuda"), torch.full(q.shape[:2], 3.0, device="cuda")
        ws = sk.new_workspace(sk.kv4_attention_chunk_workspace_bytes(len(qkv), 1, Hq, Hk, D, table.shape[1]))
        sk.kv4_attention_chunk(q, _cuda(starts), _cuda(cache), _cuda(table), _cuda(np.array(lens, np.int32)), out, lse=lse, workspace=ws)
        got.append((out, lse))
    others = torch.ones(got[0][1].shape, dtype=torch.bool)
    others[10, 0] = others[20, 0] = False
    assert torch.equal(got[0][0][others], got[1][0][others]) and torch.equal(got[0][1][others], got[1][1][others])
    assert got[0][0][20, 0].isnan().all() and got[0][1][20, 0].isnan() and got[0][0][10, 0].isnan().all() and got[0][1][10, 0].isnan()


@gpu
@WIDE
def test_offsets_past_32_bits(wide):
    D, Hk, Hq, T, n = 128, 2, 8, 30, 190
    pages = (1 << 32) // (Hk * 72 * D) + 64
    rng = np.random.default_rng(8)
    table, small, qkv, starts = _inputs(rng, "f16", D, Hq, Hk, [T], [n], wide, pad=0)
    N = len(qkv)
    small, none = small[:4], np.full((1, table.shape[1] - 4 if wide else 0), -1, np.int32)
    table = np.concatenate([np.arange(4, dtype=np.int32)[None], none], 1)
    cache = torch.empty((pages, Hk, 72 * D), dtype=torch.uint8, device="cuda")
    ids = np.array([[pages - 1, pages - 9, pages - 2, pages - 40]], np.int32)
    for i, p in enumerate(ids[0]):
        cache[p] = _cuda(small[i])
    ids = np.concatenate([ids, none], 1)
    # Rows far apart: the last of a view whose elements span more than 2^32 bytes.
    far = torch.empty((N, (1 << 32) // (2 * (N - 1)) // 8 * 8 + 4096), dtype=torch.float16, device="cuda")
    far[:, :Hq * D] = qkv.cuda()[:, :Hq * D]
    got = []
    for q, c, t in ((far, cache, ids), (qkv.cuda(), _cuda(small), table)):
        out, lse = torch.zeros((N, Hq, D), dtype=torch.float16, device="cuda"), torch.zeros((N, Hq), device="cuda")
        ws = sk.new_workspace(sk.kv4_attention_chunk_workspace_bytes(N, 1, Hq, Hk, D, t.shape[1]))
        sk.kv4_attention_chunk(q[:, :Hq * D].unflatten(-1, (Hq, D)), _cuda(starts), c, _cuda(t), _cuda(np.array([n], np.int32)), out, lse=lse, workspace=ws)
        got.append((out, lse))
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@gpu
@WIDE
def test_two_calls_at_once_and_replays_of_a_graph(wide):
    """Two streams with a workspace each; a captured call whose starts and lengths change between the replays."""
    rng = np.random.default_rng(10)
    D, Hk, Hq, chunks, lens = 128, 4, 48, [60, 1, 25], [900, 2130, 64]
    table, cache, qkv, starts = _inputs(rng, "bf16", D, Hq, Hk, chunks, lens, wide)
    B, width = table.shape
    N, dev = len(qkv), qkv.cuda()
    q = dev[:, :Hq * D].unflatten(-1, (Hq, D))
    st, ln, c, t = _cuda(starts), _cuda(np.array(lens, np.int32)), _cuda(cache), _cuda(table)
    new = lambda: (torch.zeros((N, Hq, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((N, Hq), device="cuda"),  # noqa: E731
                   sk.new_workspace(sk.kv4_attention_chunk_workspace_bytes(N, B, Hq, Hk, D, width)))
    sets = [new(), new()]
    call = lambda s, stream=None: sk.kv4_attention_chunk(q, st, c, t, ln, s[0], lse=s[1], workspace=s[2], stream=stream)  # noqa: E731
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s, stream in zip(sets, streams):
            call(s, stream)
    torch.cuda.synchronize()
    want = new()
    call(want)
    for s in sets:
        assert torch.equal(s[0].view(torch.int16), want[0].view(torch.int16)) and torch.equal(s[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(sets[0])
    for i, (a, b) in enumerate((([0, 20, 20, 92], [400, 2000, 100]), ([3, 63, 64, 89], lens), ([0, 0, 1, 2], [5, 2176, 1]))):
        dev.copy_(torch.randn(dev.shape, device="cuda"))
        st.copy_(torch.tensor(a, dtype=torch.int32)), ln.copy_(torch.tensor(b, dtype=torch.int32))
        for s in (sets[0], want):
            s[0].fill_(5.0), s[1].fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        call(want)
        torch.cuda.synchronize()
        assert torch.equal(sets[0][0].view(torch.int16), want[0].view(torch.int16)) and torch.equal(sets[0][1].view(torch.int32), want[1].view(torch.int32)), i


@gpu
def test_binding_refuses_what_does_not_fit():
    D, Hq, Hk = 64, 4, 2
    q, cache = torch.zeros((6, Hq, D), dtype=torch.float16, device="cuda"), torch.zeros((4, Hk, 72 * D), dtype=torch.uint8, device="cuda")
    table, lens, starts = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([[0, 1] * 60, [2, 3] * 60], [3, 3], [0, 3, 6]))
    good = dict(q=q, starts=starts, cache=cache, table=table, lens=lens, out=torch.empty_like(q), lse=torch.empty((6, Hq), device="cuda"),
                workspace=sk.new_workspace(sk.kv4_attention_chunk_workspace_bytes(6, 2, Hq, Hk, D, 120)))
    sk.kv4_attention_chunk(**good)
    for name, value, error in (("q", q.float(), (TypeError, sk.SkinnyError)), ("q", q[None], TypeError), ("q", q[:, :, :32], ValueError), ("q", q[:0], ValueError),
                               ("starts", starts[:2], ValueError), ("starts", starts.long(), TypeError), ("out", good["out"][:5], ValueError),
                               ("out", good["out"].bfloat16(), TypeError), ("lse", good["lse"][:, :2], ValueError), ("workspace", None, ValueError),
                               ("workspace", good["workspace"][:-1], ValueError), ("lens", lens.cpu(), TypeError), ("window", -1, sk.SkinnyError),
                               ("q", q.transpose(1, 2), ValueError)):
        with pytest.raises(error):
            sk.kv4_attention_chunk(**{**good, name: value})


@gpu
@pytest.mark.parametrize("D, call", [(64, "chunk"), (128, "chunk"), (256, "chunk"), (64, "window"), (128, "window"), (256, "window")])
def test_many_slots_of_little_weight_count(D, call):
    """One slot in front, and so many of 2^-25.5 of its weight that together they are more than the tolerance: no sum over
    pages may lose them.  Rows and sequences enough that a workgroup has thousands of pages; every fourth page is another."""
    Hk, Hq, pages = 1, 2, 4000
    n = 64 * pages
    cache = np.zeros((3, Hk, 72 * D), np.uint8)
    one, none = np.full(D, 2, np.uint8), np.zeros(D, np.uint8)  # codes of 1.0 and 0
    some = np.where(np.arange(D) < D // 8, 2, 1).astype(np.uint8)  # 1.0, and 0.5 from D / 8 on
    unit = np.full(D // 16, 0x38, np.uint8)  # scales of 1.0
    for t in range(64):
        for p, code in enumerate((one if t == 0 else none, some, none)):
            oracle.kv_put(cache[p, 0], t, code, unit, one, unit)
    ids = np.array([0] + [2 if p % 4 == 0 else 1 for p in range(1, pages)], np.int32)
    # The first slot's score is x, most others' 9 x / 16, the rest's 0: the second is at e^-17.7 of the first's weight.
    value = float(torch.tensor(17.7 * 16 / 7 / D).bfloat16())
    x = value * D
    lens = np.array([n], np.int32)
    if call == "chunk":
        T = 32768
        q = torch.full((T, Hq, D), value, dtype=torch.bfloat16, device="cuda")
        out, lse = torch.empty_like(q), torch.empty((T, Hq), device="cuda")
        ws = sk.new_workspace(sk.kv4_attention_chunk_workspace_bytes(T, 1, Hq, Hk, D, pages))
        sk.kv4_attention_chunk(q, _cuda(np.array([0, T], np.int32)), _cuda(cache), _cuda(ids[None]), _cuda(lens), out, lse=lse, scale=1.0, workspace=ws)
        limits = n - T + 1 + np.arange(T)
    else:
        B = 512
        q = torch.full((B, 1, Hq, D), value, dtype=torch.bfloat16, device="cuda")
        out, lse = torch.empty_like(q), torch.empty((B, 1, Hq), device="cuda")
        ws = sk.new_workspace(sk.kv4_attention_window_workspace_bytes(B, 1, Hq, Hk, D, pages, n))
        sk.kv4_attention_window(q, _cuda(cache), _cuda(ids[None].repeat(B, 0)), _cuda(lens.repeat(B)), out, n, lse=lse, scale=1.0, workspace=ws)
        limits = np.full(B, n)
    light = np.concatenate([[0], np.cumsum(np.repeat(ids == 1, 64))])[limits]
    want = x + np.log1p(light * np.exp(-x * 7 / 16) + (limits - 1 - light) * np.exp(-x))
    assert (want - x > 2.0 ** -9).all()
    # a score's fp32 roundings, the exponential's of numbers up to 64, and the log-sum's own: 2^-24 of 64 each, sixteen of them
    assert (np.abs(lse.double().cpu().numpy().reshape(len(limits), Hq) - want[:, None]) <= 16 * 64 * 2.0 ** -24).all()
    assert (out.double() - 1.0).abs().max().item() <= 2.0 ** -8


@gpu
@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("B, longest", [(300, 190000), (500, 700), (1100, 500), (1500, 100000)])
def test_many_sequences(B, longest, tall):
    """More tiles than the plan has threads, more sequences than it holds at once, and one that is much longer than all
    others, or not; some have no new token, and pages are shared."""
    rng = np.random.default_rng(B)
    D, Hq, Hk = 64, 8, 8
    chunks = rng.integers(0, 4, B)
    lens = np.maximum(chunks, rng.integers(0, 130, B))
    at = B // 2
    chunks[at], lens[at] = 3, longest
    width = max(100, -(-longest // 64))
    cache = _random_cache(rng, 40, Hk, D)
    table = rng.integers(-1, len(cache), (B, width)).astype(np.int32)
    starts = np.concatenate([[2], 2 + np.cumsum(chunks)]).astype(np.int32)
    N = int(starts[-1]) + 3
    used = torch.from_numpy(rng.standard_normal((N, Hq, D)) * 2.0).half()
    N += 500 * B if tall else 0
    q = torch.zeros((N, Hq, D), dtype=torch.float16, device="cuda")
    q[:len(used)] = used
    out, lse = torch.full((N, Hq, D), 3.0, dtype=torch.float16, device="cuda"), torch.full((N, Hq), 3.0, device="cuda")
    ws = sk.new_workspace(sk.kv4_attention_chunk_workspace_bytes(N, B, Hq, Hk, D, width))
    sk.kv4_attention_chunk(q, _cuda(starts), _cuda(cache), _cuda(table), _cuda(lens.astype(np.int32)), out, lse=lse, scale=0.125, workspace=ws)
    for t in (out, lse):
        assert (t[:2] == 3).all() and (t[starts[-1]:] == 3).all()
    some = [(b, i, rng.integers(Hq)) for b in [at, *rng.permutation(B)[:150], 0, B - 1] for i in range(chunks[b])]
    _check("f16", out[:len(used)], lse[:len(used)], _refs(some, cache, table, lens, starts, used.double().numpy(), Hq, Hk, D, 0.125, 1.0, 1.0, 0, 0))
    assert not (out[2:starts[-1]] == 3).all(-1).any()
