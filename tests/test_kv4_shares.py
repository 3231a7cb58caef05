"""Attention of more sequences than a wavefront has lanes, with more segments than the CUs hold shares, against 64 bits."""

import numpy as np
import pytest
import torch

import fp8_quantized_skinny_amd as sk
from test_kv4 import TYPES, _attend_inputs, _attend_refs, _check_rows, _cuda

pytestmark = pytest.mark.gpu


def _lens(kind, B, longest, rng):
    lens = {"ragged": lambda: rng.integers(0, longest + 1, B), "equal": lambda: np.full(B, longest), "short": lambda: np.ones(B, int)}[kind]()
    lens[rng.integers(0, B)] = longest
    if kind == "short":  # long ones on both sides of a wavefront's 64, and last
        lens[[1, min(B - 1, 63), min(B - 1, 64), B - 1]] = longest
    return [int(n) for n in lens]


@pytest.mark.parametrize("lengths", ["ragged", "equal", "short"])
@pytest.mark.parametrize("kind, D, Hq, Hk, T, B, longest", [("f16", 64, 8, 4, 1, 130, 700), ("bf16", 128, 12, 1, 1, 70, 1500), ("f16", 64, 6, 6, 3, 200, 600),
                                                            ("bf16", 256, 24, 2, 2, 65, 330), ("f16", 128, 24, 1, 2, 300, 400)])
def test_many_sequences(kind, D, Hq, Hk, T, B, longest, lengths):
    rng = np.random.default_rng(B + D)
    lens = _lens(lengths, B, longest, rng)
    table, cache, qkv = _attend_inputs(rng, kind, D, Hq, Hk, T, lens)
    scale, gk, gv = float(np.float32(D ** -0.5)), 1.5, 0.75
    dev = qkv.cuda()
    q = dev[..., :Hq * D].unflatten(-1, (Hq, D))
    args = (_cuda(cache), _cuda(table), _cuda(np.array(lens, np.int32)))
    need = sk.kv4_attention_workspace_bytes(B, T, Hq, Hk, D, table.shape[1])
    assert need > 0  # its sequences are split
    out, lse = torch.full((B, T, Hq, D), 3.0, dtype=TYPES[kind], device="cuda"), torch.full((B, T, Hq), 3.0, device="cuda")
    sk.kv4_attention(q, *args, out, lse=lse, scale=scale, gk=gk, gv=gv, workspace=sk.new_workspace(need, fill=0xFF))
    rows = [(b, t, h) for b in range(B) for t in range(T) for h in range(Hq)]
    some = [rows[i] for i in sorted(rng.permutation(len(rows))[:250])] + [r for r in rows if r[0] in (0, 1, 63, 64, B - 1) and r[2] in (0, Hq - 1)]
    _check_rows(kind, out, lse, _attend_refs(some, cache, table, lens, q.double().cpu().numpy(), Hq, Hk, D, T, scale, gk, gv), 64.0)
    # a row that sees nothing, and no others, has lse -inf
    limit = torch.tensor(lens)[:, None] - (T - 1 - torch.arange(T))
    assert torch.equal((lse.cpu() == -float("inf")).all(-1), limit <= 0) and torch.equal((lse.cpu() == -float("inf")).any(-1), limit <= 0)
