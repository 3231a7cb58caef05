"""Prompts and steps of streams with positions, within a window: the operators together, as they are used."""

import numpy as np
import pytest
import torch

import fp8_quantized_skinny_amd as sk
from fp8_quantized_skinny_amd.cached_decode import WindowDecoder
from oracle import kv4 as oracle

pytestmark = pytest.mark.gpu


def _attend(q, k, v, limit, window, sinks, scale, G):
    """[Hq, D] of one token's queries over the slots that it sees, and what bounds the error, in 64 bits."""
    s = torch.arange(limit)
    see = (s >= limit - window) | (s < sinks)
    k, v = (a[:limit][see].repeat_interleave(G, 1) for a in (k, v))  # [n, Hq, D]
    x = (k * q).sum(-1) * scale
    p = torch.softmax(x, 0)[..., None]
    return (p * v).sum(0), (p * v.abs()).sum(0) * (2.0 ** -10 + 2.0 ** -20 * (1 + x.abs().amax(0)[:, None]))


@pytest.mark.parametrize("streams, D, window, sinks, lengths", [(2, 64, 100, 4, (333, 71)), (3, 128, 64, 0, (1, 200, 64)), (1, 64, 1000, 9, (500,))])
def test_prompts_and_steps_within_a_window(streams, D, window, sinks, lengths):
    """Prompts, steps and prompts again: norm, rotation, append and both attentions against 64 bits, from the qkv products
    and the keys and values as the cache holds them."""
    d = WindowDecoder(streams=streams, D=D, rot=D, room=640, window=window, sinks=sinks)
    B, Hq, Hk, G, rng = d.B, d.Hq, d.Hk, d.Hq // d.Hk, np.random.default_rng(D)
    told = [[] for _ in range(B)]
    seen = []  # (queries as rotated, attention, stream, position)

    def held():
        longest = d.lens.max().item()
        k, v = torch.zeros((2, B, longest, Hk, D), dtype=torch.float16, device="cuda")
        sk.kv4_read(d.cache, d.table, d.lens, k, v)
        n = d.lens.tolist()
        return [(k[b, longest - n[b]:].double().cpu(), v[b, longest - n[b]:].double().cpu()) for b in range(B)]

    rotate = d.rotate

    def watched(q, k, positions):
        """The norm and rotation of the first and the last row against the definition."""
        pos = positions.flatten().tolist()  # before the lengths that a step's positions are grow
        before = [a.reshape(-1, a.shape[-2], D).double().cpu().numpy() for a in (q, k)]
        rotate(q, k, positions)
        for x, y, w in ((before[0], q, d.q_weight), (before[1], k, d.k_weight)):
            y = y.reshape(-1, y.shape[-2], D).double().cpu().numpy()
            for r in (0, len(pos) - 1):
                for h in range(x.shape[1]):
                    want, size = oracle.norm_rope(x[r, h], w.cpu().numpy(), 1e-6, pos[r], d.inv_freq.cpu().numpy(), 1.0, False)
                    # one rounding to fp16; 20 fp32 roundings before it, as in the operator's own test
                    assert (np.abs(y[r, h] - want) <= np.abs(want) * 2.0 ** -11 + size * 20 * 2.0 ** -24 + 2.0 ** -25).all()
        seen.append((q.reshape(-1, Hq, D).double().cpu(), pos))

    d.rotate = watched

    def check(out, who):
        q, pos = seen.pop()
        kv = held()
        for r in rng.permutation(len(pos))[:24].tolist() + [len(pos) - 1]:
            want, tol = _attend(q[r], *kv[who[r]], pos[r] + 1, window, sinks, D ** -0.5, G)
            assert ((out[r].double().cpu() - want).abs() <= tol + 2.0 ** -24).all(), (r, pos[r])

    def prompt(n):
        ps = [rng.integers(0, d.vocab, m).tolist() for m in n]
        places = [len(told[b]) + i for b in range(B) for i in range(n[b])]
        for b in range(B):
            told[b] += ps[b]
        out = d.prompt(ps)
        assert seen[-1][1] == places
        check(out, [b for b in range(B) for _ in ps[b]])

    def step():
        for b in range(B):
            told[b] += d.tokens[b].tolist()
        d.step()
        assert seen[-1][1] == [len(p) - 1 for p in told]
        check(d.out[:, 0], list(range(B)))

    prompt(lengths)
    for _ in range(5):
        step()
    prompt([2 + b for b in range(B)])
    for _ in range(3):
        step()
    assert d.lens.tolist() == [len(p) for p in told]
    lp = torch.log_softmax(d.logits.double(), 1).gather(1, d.tokens.long())[:, 0]
    assert ((d.logprob.double() - lp).abs() <= 2.0 ** -16 + 2.0 ** -22 * d.logits.abs().max().item()).all()

    with pytest.raises(ValueError):
        d.prompt([[1] * 640] * B)
    with pytest.raises(ValueError):
        d.prompt([[]] * B)
