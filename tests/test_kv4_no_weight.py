"""A row whose scores are all -inf has no weight on any slot: out 0, lse -inf, and nothing added to the slots."""

import pytest
import torch

import fp8_quantized_skinny_amd as sk

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D, Hq, Hk, T, n, width", [(128, 8, 2, 1, 1, 1), (64, 4, 4, 3, 65, 2), (256, 12, 1, 2, 300, 5), (128, 48, 4, 3, 1000, 40)])
def test_scores_of_minus_infinity(kind, D, Hq, Hk, T, n, width):
    G = Hq // Hk
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    cache = torch.zeros((width, Hk, 72 * D), dtype=torch.uint8, device="cuda")
    cache[..., :32 * D] = 0xFF                      # every key is -6 * 0.5
    cache[..., 32 * D:36 * D] = 0x30
    cache[..., 36 * D:68 * D] = 0x21
    cache[..., 68 * D:] = 0x38
    args = (cache, torch.arange(width, device="cuda").int()[None].contiguous(), torch.tensor([n], dtype=torch.int32, device="cuda"))
    q = torch.randn((1, T, Hq, D), generator=g, device="cuda").to(kind)
    q[0, T - 1, ::G, 3] = float("inf")              # one row of every key/value head
    rows = torch.zeros((T, Hq), dtype=torch.bool)
    rows[T - 1, ::G] = True
    out, lse = torch.full_like(q, 7.0), torch.full((1, T, Hq), 7.0, device="cuda")
    sk.kv4_attention(q, *args, out, lse=lse, workspace=sk.new_workspace(sk.kv4_attention_workspace_bytes(1, T, Hq, Hk, D, width)))
    assert (out[0].cpu()[rows] == 0).all() and (lse[0].cpu()[rows] == -float("inf")).all()
    assert out[0].cpu()[~rows].isfinite().all() and lse[0].cpu()[~rows].isfinite().all()

    acc = torch.rand((1, Hk, 64 * width), generator=g, device="cuda")
    got = torch.full_like(acc, 7.0)
    sk.kv4_attention_weights(q, *args, lse, acc, got)
    # All keys are alike, so a row's weights are 1 / (the slots it sees); each head has T * G - 1 rows left.
    want = acc.double().cpu()
    want[..., n:] = 0.0
    for t in range(T):
        see = n - (T - 1 - t)
        if see > 0:
            want[..., :see] += (G - (1 if t == T - 1 else 0)) / see
    # exp's argument is off by a few roundings of scores and lse, both below 256 here: 2^-24 * 256 * 4, and the sums' T * G + 1
    tol = want * (2.0 ** -14 + (T * G + 1) * 2.0 ** -24)
    assert ((got.double().cpu() - want).abs() <= tol).all()
