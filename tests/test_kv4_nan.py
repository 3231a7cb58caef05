"""A NaN among a row's scores makes that row NaN, however its sequence is shared out over workgroups.

Every other row keeps its bits: rows are columns of the products, and a share's plan does not go by values."""

import numpy as np
import pytest
import torch

import fp8_quantized_skinny_amd as sk
from oracle import kv4 as oracle

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}

# type, D, Hq, Hk, T, slots, and the pages of the table past those.  Rows of one tile are split from nine pages on and
# rows of several from five; 57 pages in shares of eight, and 13 in shares of four, leave one page to the last share.
SHAPES = [("f16", 128, 12, 2, 1, 57 * 64 - 63, 0), ("bf16", 64, 4, 1, 2, 57 * 64 - 63, 0), ("f16", 128, 48, 4, 3, 13 * 64 - 63, 0),
          ("bf16", 128, 24, 1, 2, 13 * 64 - 63, 9), ("f16", 256, 24, 2, 2, 13 * 64 - 63, 0), ("bf16", 256, 12, 1, 8, 300, 5),
          ("f16", 64, 16, 16, 8, 1000, 1),
          # not split: the table holds no more than one share
          ("f16", 128, 12, 2, 1, 8 * 64 - 63, 0), ("bf16", 128, 48, 4, 3, 4 * 64 - 63, 0), ("f16", 256, 24, 2, 2, 193, 0), ("bf16", 64, 8, 2, 4, 65, 0)]


class Case:
    def __init__(self, kind, D, Hq, Hk, T, n, spare):
        rng = np.random.default_rng(n + D)
        self.D, self.Hq, self.Hk, self.T, self.n, self.width = D, Hq, Hk, T, n, -(-n // 64) + spare
        cache = rng.integers(0, 256, (self.width, Hk, 72 * D), dtype=np.uint8)
        for at in (32 * D, 68 * D):
            cache[..., at:at + 4 * D] = rng.integers(0x28, 0x36, (self.width, Hk, 4 * D))
        self.cache = torch.from_numpy(cache).cuda()
        self.table = torch.arange(self.width, device="cuda").int()[None].contiguous()
        self.lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        self.q = torch.from_numpy(rng.standard_normal((1, T, Hq, D))).to(TYPES[kind]).cuda()
        self.acc = torch.rand((1, Hk, 64 * self.width), device="cuda")
        _, _, _, self.k_scales, self.v_scales = oracle.kv_places(D)

    def run(self):
        args = (self.cache, self.table, self.lens)
        out, lse = torch.full_like(self.q, 7.0), torch.full((1, self.T, self.Hq), 7.0, device="cuda")
        ws = sk.new_workspace(sk.kv4_attention_workspace_bytes(1, self.T, self.Hq, self.Hk, self.D, self.width), fill=0xFF)
        sk.kv4_attention(self.q, *args, out, lse=lse, workspace=ws)
        acc = torch.empty_like(self.acc)
        sk.kv4_attention_weights(self.q, *args, lse, self.acc, acc)
        return out[0].cpu(), lse[0].cpu(), acc[0].cpu()


def _check(case, before, after, rows):
    """rows [T, Hq]: those that become NaN, in out, lse and the weights of the slots they see; nothing else changes."""
    out, lse, acc = after
    assert out[rows].isnan().all() and lse[rows].isnan().all()
    bits = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
    assert torch.equal(bits(out[~rows]), bits(before[0][~rows])) and torch.equal(bits(lse[~rows]), bits(before[1][~rows]))
    assert not before[0].isnan().any() and not before[1].isnan().any()
    G = case.Hq // case.Hk
    for h in range(case.Hk):
        seen = torch.zeros(64 * case.width, dtype=torch.bool)
        for t in range(case.T):
            if rows[t, h * G:(h + 1) * G].any():
                seen[:case.n - (case.T - 1 - t)] = True
        assert acc[h, seen].isnan().all() and torch.equal(bits(acc[h, ~seen]), bits(before[2][h, ~seen]))


@pytest.mark.parametrize("kind, D, Hq, Hk, T, n, spare", SHAPES)
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_an_invalid_query(kind, D, Hq, Hk, T, n, spare, value):
    """An infinity meets keys of both signs and zeros, so its scores' maximum or sum is no number either."""
    c = Case(kind, D, Hq, Hk, T, n, spare)
    before = c.run()
    rows = torch.zeros((T, Hq), dtype=torch.bool)
    rows[T // 2, Hq // 2] = rows[T - 1, 0] = True
    c.q[0, T // 2, Hq // 2, 5] = c.q[0, T - 1, 0, D - 1] = value
    _check(c, before, c.run(), rows)


@pytest.mark.parametrize("kind, D, Hq, Hk, T, n, spare", SHAPES)
def test_a_nan_key_in_the_newest_slot(kind, D, Hq, Hk, T, n, spare):
    """Only the last row sees it; the slot is the only one of its page."""
    c = Case(kind, D, Hq, Hk, T, n, spare)
    before = c.run()
    c.cache[(n - 1) // 64, 0, int(c.k_scales[(n - 1) % 64, 0])] = 0x7F
    rows = torch.zeros((T, Hq), dtype=torch.bool)
    rows[T - 1, :Hq // Hk] = True
    _check(c, before, c.run(), rows)


@pytest.mark.parametrize("kind, D, Hq, Hk, T, n, spare", SHAPES)
@pytest.mark.parametrize("part", ["first", "middle", "last"])
def test_pages_of_nan_keys(kind, D, Hq, Hk, T, n, spare, part):
    """Whole pages, and with them whole shares, in which every score is NaN; all rows see some of them."""
    c = Case(kind, D, Hq, Hk, T, n, spare)
    before = c.run()
    np_, width = -(-n // 64), max(1, min(8, -(-n // 64) // 2))
    p0 = {"first": 0, "middle": (np_ - width) // 2, "last": np_ - width}[part]
    at = torch.from_numpy(np.unique(c.k_scales)).cuda()
    c.cache[p0:p0 + width, Hk - 1, at] = 0xFF
    rows = torch.zeros((T, Hq), dtype=torch.bool)
    rows[:, -(Hq // Hk):] = True
    if p0 * 64 >= n - (T - 1):  # rows before the last see no slot of the page
        for t in range(T):
            rows[t] &= p0 * 64 < n - (T - 1 - t)
    _check(c, before, c.run(), rows)
