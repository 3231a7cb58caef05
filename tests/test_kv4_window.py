"""Attention within a sliding window over the 4-bit cache, against its definition in 64 bits."""

import numpy as np
import pytest
import torch

import fp8_quantized_skinny_amd as sk
from fp8_quantized_skinny_amd._lib import lib
from oracle import kv4 as oracle
from test_kv4 import A, BAD_CACHES, BAD_ROWS, MIS, TYPES, _attend_inputs, _cache, _check_rows, _cuda, _rows

gpu = pytest.mark.gpu


# ---------------------------------------------------------------- refusals (no GPU)
def _call(c=None, r=None, type=0, T=2, Hq=8, scale=0.1, window=100, sinks=4, out=A, lse=A, ws=A, n=1 << 40):
    return lib().kv4_attention_window(c or _cache(), r or _rows(), type, T, Hq, scale, window, sinks, out, lse, ws, n, None)


@pytest.mark.parametrize("bad, status", BAD_CACHES)
def test_cache_refusals(bad, status):
    assert _call(c=_cache(**bad)) == status


@pytest.mark.parametrize("bad, status", BAD_ROWS)
def test_row_refusals(bad, status):
    assert _call(r=_rows(**bad)) == status


def test_argument_refusals():
    for bad in (dict(type=2), dict(scale=0.0), dict(scale=float("nan")), dict(window=-1), dict(sinks=-1), dict(out=None)):
        assert _call(**bad) == sk.EINVAL, bad
    for bad in (dict(T=0), dict(T=9), dict(Hq=6), dict(Hq=0), dict(Hq=4 * 65)):
        assert _call(**bad) == sk.ESHAPE, bad
    assert _call(out=MIS) == sk.EALIGN and _call(lse=A + 2) == sk.EALIGN
    wide = _cache(width=64)
    need = sk.kv4_attention_window_workspace_bytes(2, 2, 8, 4, 128, 64, 2000, 4)
    assert need > sk.WORKSPACE_SYNC_BYTES
    assert _call(c=wide, window=2000, ws=None, n=0) == sk.EINVAL and _call(c=wide, window=2000, n=need - 1) == sk.ESIZE
    assert _call(c=wide, window=2000, ws=MIS) == sk.EALIGN


def test_workspaces_go_by_the_window():
    size = lambda width, window, sinks=0, T=1: sk.kv4_attention_window_workspace_bytes(2, T, 8, 4, 128, width, window, sinks)  # noqa: E731
    whole = sk.kv4_attention_workspace_bytes(2, 1, 8, 4, 128, 2000)
    assert size(2000, 0) == size(2000, 128000) == size(2000, 2 ** 31 - 1, 2 ** 31 - 1) == whole
    assert size(2000, 64) == 0 and 0 < size(2000, 1024) < whole and size(2000, 1024, 4) == size(30000, 1024, 4)
    assert size(2000, -1) == size(2000, 5, -1) == size(2000, 64, 0, 9) == 0


# ---------------------------------------------------------------- GPU
WINDOWS = [  # type, D, Hq, Hk, T, lens, window, sinks
    ("f16", 128, 48, 4, 1, [3010], 1024, 4),
    ("bf16", 128, 48, 4, 8, [1, 5, 300, 1030, 0, 64, 65], 100, 3),
    ("f16", 256, 24, 4, 8, [513, 64, 700], 64, 64),
    ("bf16", 256, 5, 1, 3, [200, 2, 65], 1, 0),
    ("f16", 64, 16, 16, 1, [63, 64, 65, 1, 0, 129], 1, 1),
    ("bf16", 64, 28, 4, 5, [700, 4], 130, 200),
    ("f16", 128, 8, 1, 2, [2500, 900], 2000, 65),
    ("bf16", 128, 32, 8, 4, [128, 127, 131, 1], 2, 0),
    ("f16", 64, 64, 1, 8, [90, 640], 63, 128),
    ("f16", 128, 2, 2, 1, [191] * 70, 66, 5),
    ("f16", 128, 12, 1, 1, [40000], 20000, 700),
    ("bf16", 128, 8, 2, 3, [400, 40], 0, 9),
    ("f16", 64, 8, 2, 3, [400, 40], 5000, 9),
    ("bf16", 128, 8, 2, 1, [600, 300], 32, 2 ** 31 - 1),
]


@gpu
@pytest.mark.parametrize("kind, D, Hq, Hk, T, lens, window, sinks", WINDOWS)
def test_window(kind, D, Hq, Hk, T, lens, window, sinks):
    rng = np.random.default_rng(D + Hq + T + window)
    table, cache, qkv = _attend_inputs(rng, kind, D, Hq, Hk, T, lens)
    B, width = table.shape
    for b, n in enumerate(lens):  # pages that no row sees: NaN and pages that are none
        for p in range(-(-sinks // 64), max(0, n - T + 1 - window) // 64 if window else 0):
            cache[table[b, p]] = 0xFF
            if p % 2:
                table[b, p] = -1
    scale, gk, gv = float(np.float32(D ** -0.5)), 1.5, 0.75
    q = qkv.cuda()[..., :Hq * D].unflatten(-1, (Hq, D))
    out, lse = torch.full((B, T, Hq, D), 3.0, dtype=TYPES[kind], device="cuda"), torch.full((B, T, Hq), 3.0, device="cuda")
    args = (_cuda(cache), _cuda(table), _cuda(np.array(lens, np.int32)))
    ws = sk.new_workspace(sk.kv4_attention_window_workspace_bytes(B, T, Hq, Hk, D, width, window, sinks), fill=0xFF)
    for _ in range(2):  # a workspace serves again
        sk.kv4_attention_window(q, *args, out, window, sinks, lse=lse, scale=scale, gk=gk, gv=gv, workspace=ws)
    first = out.clone()
    sk.kv4_attention_window(q, *args, out, window, sinks, scale=scale, gk=gk, gv=gv, workspace=ws)
    assert torch.equal(first.view(torch.int16), out.view(torch.int16))
    if window == 0 or window >= 64 * width:  # nothing is left out: kv4_attention, bit for bit
        sk.kv4_attention(q, *args, out, scale=scale, gk=gk, gv=gv, workspace=ws)
        assert torch.equal(first.view(torch.int16), out.view(torch.int16))
    qd = q.double().cpu().numpy()
    rows = [(b, t, h) for b in range(B) for t in range(T) for h in range(Hq)]
    if len(rows) > 300:
        rows = [rows[i] for i in sorted(rng.permutation(len(rows))[:300])]
    _check_rows(kind, out, lse, _refs(rows, cache, table, lens, qd, Hq, Hk, D, T, scale, gk, gv, window, sinks), 64.0)


def _refs(rows, cache, table, lens, q, Hq, Hk, D, T, scale, gk, gv, window, sinks):
    held = {}
    for b, t, h in rows:
        hk = h // (Hq // Hk)
        if (b, hk) not in held:
            held[b, hk] = oracle.kv_held(cache, table[b], lens[b], hk, D, gk, gv)
        k, v, ok = held[b, hk]
        limit = lens[b] - (T - 1 - t)
        yield (b, t, h, *oracle.kv_attend(q[b, t, h], k, v, ok & oracle.in_window(len(k), limit, window, sinks), limit, scale))


@gpu
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_nan_value_reaches_only_the_rows_that_see_it(D):
    rng = np.random.default_rng(6)
    T, Hq, Hk, lens, window, sinks = 8, 12, 2, [300], 128, 10
    table, cache, qkv = _attend_inputs(rng, "f16", D, Hq, Hk, T, lens)
    vs = oracle.kv_places(D)[4]
    # Row t sees the slots from 165 + t on: slot 168 is seen by rows 0 .. 3, 12 by none, and 298 by rows 6 and 7.
    for s in (168, 12, 298):
        cache[table[0, s // 64], :, vs[s % 64, 0]] = 0x7F
    q = qkv.cuda()[..., :Hq * D].unflatten(-1, (Hq, D))
    args = (_cuda(cache), _cuda(table), _cuda(np.array(lens, np.int32)))
    out, lse = torch.empty((1, T, Hq, D), dtype=torch.float16, device="cuda"), torch.empty((1, T, Hq), device="cuda")
    ws = sk.new_workspace(sk.kv4_attention_window_workspace_bytes(1, T, Hq, Hk, D, table.shape[1], window, sinks))
    sk.kv4_attention_window(q, *args, out, window, sinks, lse=lse, workspace=ws)
    for t in range(T):
        assert out[:, t, :, :16].isnan().all() == (t <= 3 or t >= 6) and (4 <= t < 6) == (not out[:, t].isnan().any()), t
    assert not lse.isnan().any()


@gpu
def test_a_step_replayed_from_a_graph():
    rng = np.random.default_rng(10)
    D, Hk, Hq, T, lens, window, sinks = 128, 4, 48, 4, [900, 1330, 64], 700, 5
    table, cache, qkv = _attend_inputs(rng, "bf16", D, Hq, Hk, T, lens)
    B, width = table.shape
    args = (_cuda(cache), _cuda(table), _cuda(np.array(lens, np.int32)))
    dev = qkv.cuda()
    q = dev[..., :Hq * D].unflatten(-1, (Hq, D))
    ws = sk.new_workspace(sk.kv4_attention_window_workspace_bytes(B, T, Hq, Hk, D, width, window, sinks))
    out, lse = torch.empty((B, T, Hq, D), dtype=torch.bfloat16, device="cuda"), torch.empty((B, T, Hq), device="cuda")
    step = lambda: sk.kv4_attention_window(q, *args, out, window, sinks, lse=lse, workspace=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        dev.copy_(torch.randn(dev.shape, device="cuda"))
        args[2].copy_(torch.tensor([[1000, 30, 0], [900, 1330, 64], [1, 1408, 200]][i], dtype=torch.int32))
        out.fill_(5.0), lse.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0].view(torch.int16), out.view(torch.int16)) and torch.equal(got[1].view(torch.int32), lse.view(torch.int32)), i
