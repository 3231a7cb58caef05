"""Chunk attention by tiles of 256 rows, against its definition in 64 bits.

Calls of more than 512 sequences always go that way; here all but a few of them have no row.  Short ones are whole tiles;
tiles of 14 pages and more are cut wherever the workgroups' even shares end."""

import numpy as np
import pytest
import torch

import fp8_quantized_skinny_amd as sk
from oracle import kv4 as oracle
from test_kv4 import TYPES, _attend_inputs, _cuda
from test_kv4_chunk import _check, _refs, _some

pytestmark = pytest.mark.gpu
B = 520


class Call:
    """Chunks of some sequences among B, queries in a qkv GEMM's output with rows of no sequence before and behind them."""

    def __init__(self, rng, kind, D, Hq, Hk, chunks, lens, window=0, sinks=0, pad=3, q_size=2.0):
        self.kind, self.D, self.Hq, self.Hk, self.window, self.sinks = kind, D, Hq, Hk, window, sinks
        table, self.cache, _ = _attend_inputs(rng, kind, D, Hq, Hk, 1, lens)
        self.at = sorted(rng.permutation(B)[:len(chunks)].tolist())
        self.chunks, self.lens = np.zeros(B, int), rng.integers(0, 64 * table.shape[1], B)
        self.table = np.full((B, table.shape[1]), -1, np.int32)
        self.chunks[self.at], self.lens[self.at], self.table[self.at] = chunks, lens, table
        self.starts = pad + np.concatenate([[0], np.cumsum(self.chunks)]).astype(np.int32)
        self.N = int(self.starts[-1]) + pad
        self.qkv = torch.from_numpy(rng.standard_normal((self.N, (Hq + 2 * Hk) * D)) * q_size).to(TYPES[kind])
        self.scale = float(np.float32(D ** -0.5))

    def workspace(self):
        ws = sk.new_workspace(sk.kv4_attention_chunk_workspace_bytes(self.N, B, self.Hq, self.Hk, self.D, self.table.shape[1], self.window, self.sinks), fill=0xFF)
        assert ws is not None  # attention in one launch has none
        return ws

    def args(self, starts=None):
        return (_cuda(self.starts if starts is None else np.array(starts, np.int32)), _cuda(self.cache), _cuda(self.table),
                _cuda(self.lens.astype(np.int32)))

    def queries(self, qkv=None):
        return (self.qkv if qkv is None else qkv).cuda()[:, :self.Hq * self.D].unflatten(-1, (self.Hq, self.D))

    def run(self, q=None, starts=None, out=None, **more):
        q = self.queries() if q is None else q
        out = torch.full(q.shape, 3.0, dtype=q.dtype, device="cuda") if out is None else out
        lse = torch.full(q.shape[:2], 3.0, device="cuda")
        sk.kv4_attention_chunk(q, *self.args(starts), out, lse=lse, window=self.window, sinks=self.sinks,
                               **{"scale": self.scale, "workspace": self.workspace(), **more})
        return out, lse

    def refs(self, rng, gk=1.0, gv=1.0, most=300, q=None):
        rows = _some(rng, self.chunks, self.Hq, most)
        return _refs(rows, self.cache, self.table, self.lens, self.starts, (self.queries() if q is None else q).double().cpu().numpy(), self.Hq, self.Hk,
                     self.D, self.scale, gk, gv, self.window, self.sinks)

    def spoil_unseen(self):
        """Pages that no row sees: NaN, and pages that are none."""
        for b in self.at:
            first = max(0, self.lens[b] - self.chunks[b] + 1 - self.window) // 64 if self.window and self.chunks[b] else 0
            for p in range(-(-self.sinks // 64), first):
                self.cache[self.table[b, p]] = 0xFF
                if p % 2:
                    self.table[b, p] = -1


def _same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


SHORT = ([300, 1, 64, 70], [700, 64, 90, 40])     # more new tokens than slots in the last
LONG = ([260, 9, 130], [2600, 1300, 3000])
HEADS = {64: (12, 2), 128: (16, 4), 256: (6, 1)}


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lengths, window, sinks", [
    (SHORT, 0, 0), (SHORT, 1, 0), (SHORT, 64, 64), (SHORT, 100, 3), (SHORT, 63, 130), (SHORT, 300, 2 ** 31 - 1),
    (LONG, 0, 0), (LONG, 1100, 4), (LONG, 1900, 130), (LONG, 64, 5), (LONG, 100, 1500), (LONG, 2047, 0)])
def test_tiles(kind, D, lengths, window, sinks):
    rng = np.random.default_rng(D + window + sinks % 1000)
    c = Call(rng, kind, D, *HEADS[D], *lengths, window, sinks)
    c.spoil_unseen()
    more = dict(gk=1.5, gv=0.75, workspace=c.workspace())
    out, lse = c.run(**more)
    again, again_lse = c.run(**more)  # the workspace serves again
    assert _same(out, again) and _same(lse, again_lse) and (more["workspace"][:sk.WORKSPACE_SYNC_BYTES] == 0).all()
    for t in (out, lse):  # rows that no sequence has
        assert (t[:c.starts[0]] == 3).all() and (t[c.starts[-1]:] == 3).all()
    q = c.queries().contiguous()  # in place
    rows = slice(c.starts[0], c.starts[-1])
    assert _same(c.run(q=q, out=q, **more)[0][rows], out[rows])
    _check(kind, out, lse, c.refs(rng, 1.5, 0.75))


@pytest.mark.parametrize("kind, D, Hq, Hk, chunks, lens, window, sinks", [
    ("f16", 64, 128, 128, [270, 3], [1500, 70], 0, 0),      # so many heads that tiles are never cut
    ("bf16", 64, 128, 128, [270, 3], [1500, 70], 200, 65),
    ("f16", 128, 64, 1, [11, 5, 4], [2000, 5, 1500], 700, 66),  # 64 query heads a key/value head
    ("bf16", 128, 1, 1, [520], [1800], 1000, 1),            # one
    ("f16", 256, 15, 3, [150, 2], [1700, 1700], 900, 0),
    ("bf16", 64, 28, 4, [130, 64, 63, 65, 128] * 3, [1300, 64, 200, 65, 900] * 3, 130, 200),
    ("f16", 128, 8, 2, [2] * 200, [40 * i % 1700 for i in range(200)], 500, 3)])
def test_tiles_of_other_heads(kind, D, Hq, Hk, chunks, lens, window, sinks):
    rng = np.random.default_rng(D + Hq)
    c = Call(rng, kind, D, Hq, Hk, chunks, lens, window, sinks)
    c.spoil_unseen()
    _check(kind, *c.run(), c.refs(rng))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n, T, window, sinks", [(200, 70, 0, 0), (200, 70, 40, 3), (200, 70, 100, 70), (2200, 70, 0, 0), (2200, 70, 1900, 3), (2200, 70, 1000, 100)])
def test_a_nan_value_reaches_only_the_rows_that_see_it(D, n, T, window, sinks):
    rng = np.random.default_rng(6)
    kind = "bf16" if D == 128 else "f16"
    c = Call(rng, kind, D, *HEADS[D], [T], [n], window, sinks)
    b, (_, _, _, ks, vs) = c.at[0], oracle.kv_places(D)
    # of the newest slots, a first one, one that some rows' windows have left behind, and one in a page that all see whole
    groups = {n - 50: D // 16 - 1, 2: 0, n - T + 3: 1, max(0, n - T - window + 30 if window else 70): 2, n - 150: 0}
    for s, g in groups.items():
        c.cache[c.table[b, s // 64], :, vs[s % 64, 16 * g]] = 0x7F
    bad_key = n - 10
    c.cache[c.table[b, bad_key // 64], :, ks[bad_key % 64, 0]] = 0xFF  # a NaN key: all of the rows that see it
    out, lse = (t[c.starts[0]:c.starts[-1]].isnan().cpu().numpy() for t in c.run())
    for i in range(T):
        see = oracle.in_window(n, n - T + 1 + i, window, sinks)
        want = np.zeros(D, bool)
        for s, g in groups.items():
            want[16 * g:16 * g + 16] |= see[s]
        want |= see[bad_key]
        assert (out[i] == want).all() and (lse[i] == see[bad_key]).all(), i


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window, sinks", [(0, 0), (1500, 100)])
def test_missing_pages_are_skipped(D, window, sinks):
    rng = np.random.default_rng(5)
    c = Call(rng, "bf16", D, *HEADS[D], [100, 30], [200, 2300], window, sinks)
    a, b = c.at
    c.table[a, 1], c.table[a, 3], c.table[b, 0], c.table[b, 12:20], c.table[b, 35] = -1, 2 ** 31 - 1, len(c.cache), -7, -2 ** 31
    _check("bf16", *c.run(), c.refs(rng))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind, size", [("f16", 3e4), ("bf16", 1e30), ("bf16", 1e-30), ("f16", 1e-7)])
def test_queries_of_extreme_size(kind, size, D):
    rng = np.random.default_rng(7)
    c = Call(rng, kind, D, 4, 1, [40], [1150], q_size=size)
    if kind == "f16":
        c.qkv.clamp_(-6e4, 6e4)
    c.qkv[5, :D] = 0.0
    c.scale = float(np.float32(1.0 / size)) if size > 1 else 1.0
    # scores of sqrt(D) times keys of about 1.7: five standard deviations, in powers of two, are below 256 at D = 256
    _check(kind, *c.run(), c.refs(rng), 256.0)


@pytest.mark.parametrize("n", [150, 2000])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_infinite_and_nan_queries_stay_in_their_rows(D, n):
    rng = np.random.default_rng(8)
    c = Call(rng, "f16", D, 2, 1, [140], [n])
    clean = c.run()
    c.qkv[10, 3], c.qkv[20, D + 5] = float("inf"), float("nan")
    got = c.run()
    hit = torch.zeros(clean[1].shape, dtype=torch.bool)
    hit[10, 0] = hit[20, 1] = True
    for a, b in zip(got, clean):
        assert a[hit].isnan().all() and _same(a[~hit], b[~hit])


def test_starts_that_fall_or_leave_the_rows():
    rng = np.random.default_rng(7)
    c = Call(rng, "f16", 64, 4, 2, [50, 60, 40], [700, 80, 1290], pad=0)
    N, q = c.N, c.queries()
    for _ in range(4):
        bad = rng.integers(-20, N + 20, B + 1)
        bad[rng.permutation(B + 1)[:3]] = [-2 ** 31, 2 ** 31 - 1, N]
        bad[:400] = rng.integers(-20, 60, 400)
        good = np.maximum.accumulate(np.clip(bad, 0, N))
        for a, b in zip(c.run(q, bad), c.run(q, good)):
            assert _same(a, b)
    for nothing in ([0] * (B + 1), [N] * (B + 1), [-5] * (B + 1), [N + 9] * (B + 1)):
        out, lse = c.run(q, nothing)
        assert (out == 3).all() and (lse == 3).all()


def test_offsets_past_32_bits():
    """Pages, rows and parts behind 2^32 bytes."""
    D, Hk, Hq, T, n = 128, 2, 8, 80, 1090
    rng = np.random.default_rng(8)
    c = Call(rng, "f16", D, Hq, Hk, [T], [n], pad=0)
    want = c.run()
    pages = (1 << 32) // (Hk * 72 * D) + 64
    far = torch.empty((pages, Hk, 72 * D), dtype=torch.uint8, device="cuda")
    ids = pages - 1 - rng.permutation(60)[:len(c.cache)]
    for p, i in enumerate(ids):
        far[i] = _cuda(c.cache[p])
    table = np.where((c.table >= 0) & (c.table < len(c.cache)), ids[np.clip(c.table, 0, len(c.cache) - 1)], -1).astype(np.int32)
    q = torch.empty((T, (1 << 32) // (2 * (T - 1)) // 8 * 8 + 4096), dtype=torch.float16, device="cuda")
    q[:, :Hq * D] = c.qkv.cuda()[:, :Hq * D]
    out, lse = torch.full((T, Hq, D), 3.0, dtype=torch.float16, device="cuda"), torch.full((T, Hq), 3.0, device="cuda")
    starts, _, _, lens = c.args()
    sk.kv4_attention_chunk(q[:, :Hq * D].unflatten(-1, (Hq, D)), starts, far, _cuda(table), lens, out, lse=lse, scale=c.scale, workspace=c.workspace())
    assert _same(out, want[0]) and _same(lse, want[1])


@pytest.mark.parametrize("D, window, sinks", [(64, 0, 0), (128, 900, 70), (256, 700, 1)])
def test_two_calls_at_once_and_replays_of_a_graph(D, window, sinks):
    """Two streams with a workspace each; a captured call whose starts and lengths change between the replays."""
    rng = np.random.default_rng(10)
    c = Call(rng, "bf16", D, *HEADS[D], [160, 1, 325], [1500, 2130, 964], window, sinks)
    starts, cache, table, lens = c.args()
    dev = c.qkv.cuda()
    q = dev[:, :c.Hq * D].unflatten(-1, (c.Hq, D))
    sets = [(torch.zeros(q.shape, dtype=q.dtype, device="cuda"), torch.zeros(q.shape[:2], device="cuda"), c.workspace()) for _ in range(3)]

    def call(s, stream=None):
        sk.kv4_attention_chunk(q, starts, cache, table, lens, s[0], lse=s[1], window=window, sinks=sinks, workspace=s[2], stream=stream)

    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s, stream in zip(sets, streams):
            call(s, stream)
    torch.cuda.synchronize()
    call(sets[2])
    for s in sets[:2]:
        assert _same(s[0], sets[2][0]) and _same(s[1], sets[2][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(sets[0])
    for _ in range(4):
        dev.copy_(torch.randn(dev.shape, device="cuda"))
        lens.copy_(torch.from_numpy(rng.integers(0, 64 * table.shape[1], B).astype(np.int32)))
        at = np.zeros(B + 1, np.int32)
        at[c.at[1] + 1:], at[c.at[2] + 1:] = rng.integers(0, c.N), c.N
        starts.copy_(torch.from_numpy(at))
        for s in (sets[0], sets[2]):
            s[0].fill_(5.0), s[1].fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        call(sets[2])
        torch.cuda.synchronize()
        assert _same(sets[0][0], sets[2][0]) and _same(sets[0][1], sets[2][1])
