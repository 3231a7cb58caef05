"""A NaN among the values of a slot reaches its own group of 16 positions, in the rows that see the slot, and nothing else."""

import numpy as np
import pytest
import torch

import fp8_quantized_skinny_amd as sk
from oracle import kv4 as oracle
from test_kv4 import TYPES, _attend_inputs, _check_rows, _cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call", ["attention", "window", "chunk"])
@pytest.mark.parametrize("width", [0, 10])  # pages more than the lengths fill: split or not
@pytest.mark.parametrize("kind, D, Hq, Hk, T", [("f16", 64, 12, 2, 8), ("bf16", 64, 4, 4, 1), ("bf16", 128, 12, 2, 8), ("f16", 128, 8, 1, 3),
                                                ("f16", 256, 12, 2, 8), ("bf16", 256, 6, 1, 5), ("f16", 128, 16, 1, 1)])
def test_a_nan_value_stays_in_its_group(kind, D, Hq, Hk, T, width, call):
    """Slots in whole pages, in the newest page that all rows see, and among the step's own, of which the first rows see none."""
    rng = np.random.default_rng(D + T)
    n = 300
    table, cache, qkv = _attend_inputs(rng, kind, D, Hq, Hk, T, [n])
    table = np.concatenate([table, np.full((1, width), -1, np.int32)], 1)
    places = oracle.kv_places(D)[4]
    groups = {5: 0, 257: D // 16 - 1, n - 1: 1, n - (T + 1) // 2: 2}
    for s, g in groups.items():
        cache[table[0, s // 64], :, places[s % 64, 16 * g]] = 0x7F
    q = qkv.cuda()[..., :Hq * D].unflatten(-1, (Hq, D))
    args = (_cuda(cache), _cuda(table), _cuda(np.array([n], np.int32)))
    out, lse = torch.empty((1, T, Hq, D), dtype=TYPES[kind], device="cuda"), torch.empty((1, T, Hq), device="cuda")
    scale = float(np.float32(D ** -0.5))
    more, window = dict(lse=lse, scale=scale), 0
    if call == "attention":
        sk.kv4_attention(q, *args, out, workspace=sk.new_workspace(sk.kv4_attention_workspace_bytes(1, T, Hq, Hk, D, table.shape[1])), **more)
    elif call == "window":
        window = 299
        ws = sk.new_workspace(sk.kv4_attention_window_workspace_bytes(1, T, Hq, Hk, D, table.shape[1], window))
        sk.kv4_attention_window(q, *args, out, window, workspace=ws, **more)
    else:
        ws = sk.new_workspace(sk.kv4_attention_chunk_workspace_bytes(T, 1, Hq, Hk, D, table.shape[1]))
        sk.kv4_attention_chunk(q[0], _cuda(np.array([0, T], np.int32)), *args, out[0], lse=lse[0], scale=scale, workspace=ws)
    for t in range(T):
        want = np.zeros(D, bool)
        for s, g in groups.items():
            want[16 * g:16 * g + 16] |= s < n - (T - 1 - t)
        assert (out[0, t].isnan().cpu().numpy() == want).all(), t
    assert not lse.isnan().any()
    # The other positions have their values: 64 bits with zeros in the place of the NaN.
    qd = q.double().cpu().numpy()
    refs = []
    for t in range(T):
        for h in range(Hq):
            k, v, ok = oracle.kv_held(cache, table[0], n, h // (Hq // Hk), D, 1.0, 1.0)
            limit = n - (T - 1 - t)
            see = ok & oracle.in_window(n, limit, window, 0)
            r = oracle.kv_attend(qd[0, t, h], k, np.nan_to_num(v), see, limit, scale)
            nan = out[0, t, h].isnan().cpu().numpy()
            refs.append((0, t, h, np.where(nan, np.nan, r[0]), *r[1:]))
    _check_rows(kind, out, lse, refs, 64.0)
