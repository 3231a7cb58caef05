"""Many slots of little weight beside one of much: no sum over a workgroup's pages may lose them."""

import numpy as np
import pytest
import torch

import fp8_quantized_skinny_amd as sk
from oracle import kv4 as oracle

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call", ["attention", "window", "window and sinks"])
@pytest.mark.parametrize("T, Hq", [(1, 2), (8, 6)])  # one and three tiles of rows
@pytest.mark.parametrize("D", [64, 128, 256])
def test_light_slots_count(D, T, Hq, call):
    """Slot 0 has the weight, the others 2^-25.5 of it each, less than half a step of a sum that holds slot 0's.  So many
    sequences that a share is half of one: the wavefront with slot 0 has 500 pages, and the lane 8000 slots, 1.6e-4 of the sum."""
    B, Hk, pages = 512, 1, 4000
    n = 64 * pages
    cache = np.zeros((2, Hk, 72 * D), np.uint8)
    heavy = np.full(D, 2, np.uint8)  # codes of 1.0
    light = np.where(np.arange(D) < D // 8, 2, 1).astype(np.uint8)  # 1.0, and 0.5 from D / 8 on
    unit = np.full(D // 16, 0x38, np.uint8)  # scales of 1.0
    for p in range(2):
        for t in range(64):
            oracle.kv_put(cache[p, 0], t, heavy if p == t == 0 else light, unit, heavy, unit)
    width = pages + 1  # the last column is past the lengths: a window of n slots leaves none of them out
    table = torch.ones((B, width), dtype=torch.int32, device="cuda")
    table[:, 0] = 0
    # The first slot's score is x, the others' 9 x / 16, at e^-17.7 of its weight.
    value = float(torch.tensor(17.7 * 16 / 7 / D).bfloat16())
    x = value * D
    q = torch.full((B, T, Hq, D), value, dtype=torch.bfloat16, device="cuda")
    args = (q, torch.from_numpy(cache).cuda(), table, torch.full((B,), n, dtype=torch.int32, device="cuda"))
    out, lse = torch.empty_like(q), torch.empty((B, T, Hq), device="cuda")
    more = dict(lse=lse, scale=1.0)
    seen = n - T + 1 + np.arange(T)
    if call == "attention":
        ws = sk.new_workspace(sk.kv4_attention_workspace_bytes(B, T, Hq, Hk, D, width))
        sk.kv4_attention(*args, out, workspace=ws, **more)
    else:
        window, sinks = (n, 0) if call == "window" else (n - 64, 1)
        if sinks:
            seen = np.minimum(seen, window + 1)  # slot 0, and the window without it
        ws = sk.new_workspace(sk.kv4_attention_window_workspace_bytes(B, T, Hq, Hk, D, width, window, sinks))
        sk.kv4_attention_window(*args, out, window, sinks, workspace=ws, **more)
    want = x + np.log1p((seen - 1) * np.exp(-x * 7 / 16))
    # a score's fp32 roundings, the exponential's of numbers up to 64, and the log-sum's own: 2^-24 of 64 each, sixteen of them
    assert np.abs(lse.double().cpu().numpy() - want[None, :, None]).max() <= 16 * 64 * 2.0 ** -24
    assert (out.double() - 1.0).abs().max().item() <= 2.0 ** -8  # rounded to bf16
