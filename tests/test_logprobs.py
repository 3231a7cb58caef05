"""lm_head_logprobs against its definition in 64 bits, and its refusals."""

import numpy as np
import pytest
import torch

import fp8_quantized_skinny_amd as sk
from fp8_quantized_skinny_amd._lib import lib
from oracle import kv4 as oracle

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
A = 0x10000


def test_refusals():
    def call(x=A, type=0, stride=100, tokens=A, lp=A, ent=A, ids=A, top=A, R=2, V=100, k=5, ws=A, n=1 << 40):
        return lib().lm_head_logprobs(x, type, stride, tokens, lp, ent, ids, top, R, V, k, ws, n, None)
    for name in ("x", "tokens", "lp", "ent", "ids", "top"):
        assert call(**{name: None}) == sk.EINVAL, name
    assert call(type=3) == sk.EINVAL and call(type=-1) == sk.EINVAL and call(stride=99) == sk.EINVAL
    for bad in (dict(R=0), dict(V=0), dict(k=0), dict(k=33), dict(V=4, k=5), dict(R=1 << 24), dict(V=(1 << 24) + 1)):
        assert call(**bad) == sk.ESHAPE, bad
    assert call(x=A + 8) == sk.EALIGN and call(tokens=A + 2) == sk.EALIGN and call(top=A + 1) == sk.EALIGN
    need = sk.lm_head_logprobs_workspace_bytes(8, 151936, 5)
    if need:
        big = dict(R=8, V=151936, stride=151936)
        assert call(**big, ws=None, n=0) == sk.EINVAL and call(**big, n=need - 1) == sk.ESIZE and call(**big, ws=A + 8) == sk.EALIGN
    assert sk.lm_head_logprobs_workspace_bytes(8, 4, 5) == 0


def _run(x, tokens, k, stride=None):
    R, V = x.shape
    if stride:
        wide = torch.full((R, stride), 50.0, dtype=x.dtype, device="cuda")
        wide[:, :V] = x.cuda()
        x = wide[:, :V]
    else:
        x = x.cuda()
    out = (torch.full((R,), 9.0, device="cuda"), torch.full((R,), 9.0, device="cuda"),
           torch.full((R, k), 9, dtype=torch.int32, device="cuda"), torch.full((R, k), 9.0, device="cuda"))
    ws = sk.new_workspace(sk.lm_head_logprobs_workspace_bytes(R, V, k), fill=0xFF)
    for _ in range(2):
        sk.lm_head_logprobs(x, torch.tensor(tokens, dtype=torch.int32, device="cuda"), *out, workspace=ws)
    return [t.cpu().numpy() for t in out]


def _check(x, tokens, k, got):
    lp, ent, ids, top = got
    for r in range(len(x)):
        row = x[r].double().numpy()
        a, b, c, d = oracle.logprobs(row, tokens[r], k)
        assert np.array_equal(ids[r], c), (r, ids[r], c)
        finite = row[np.isfinite(row)]
        # lse is off by the sum's roundings (at most V of 2^-24 in each of the partial sums: a few hundred terms
        # each, hence 2^-16 at worst), exp's, and the last subtractions of numbers up to the greatest logit
        size = np.abs(finite).max() if len(finite) else 0.0
        tol = 2.0 ** -16 + 2.0 ** -22 * size
        for g, w in [(lp[r], a), *zip(top[r], d)]:
            assert (np.isnan(g) and np.isnan(w)) or g == w or abs(g - w) <= tol + abs(w) * 2.0 ** -22, (r, g, w)
        assert (np.isnan(ent[r]) and np.isnan(b)) or abs(ent[r] - b) <= 2.0 ** -15 * (1 + b), (r, ent[r], b)


SHAPES = [("f16", 8, 151936, 5, None), ("bf16", 3, 151936, 20, None), ("f32", 2, 32000, 1, 32001), ("bf16", 5, 40, 32, 43),
          ("f16", 300, 1001, 7, 1003), ("f32", 4, 1, 1, None), ("bf16", 2, 200001, 32, 200005), ("f16", 1, 33, 32, None),
          ("f16", 600, 2048, 32, None)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind, R, V, k, stride", SHAPES)
def test_rows(kind, R, V, k, stride):
    g = torch.Generator().manual_seed(V + k)
    x = torch.randn((R, V), generator=g) * 2.5
    x += (torch.rand((R, V), generator=g) < 24 / V) * 14.0 * torch.rand((R, V), generator=g)
    x = x.to(TYPES[kind])
    tokens = torch.randint(0, V, (R,), generator=g).tolist()
    _check(x, tokens, k, _run(x, tokens, k, stride))


def _special(V, kind, g):
    """Rows that a running maximum, a threshold or a tie can go wrong at."""
    low = torch.finfo(TYPES[kind]).min
    inf, nan = float("inf"), float("nan")
    base = torch.randn((V,), generator=g)
    rows = [torch.zeros(V), torch.full((V,), -inf), torch.full((V,), low), torch.arange(V) * 0.01, -torch.arange(V) * 0.01,
            (torch.arange(V) % 7).float(), (torch.arange(V) % 2) * 1.0 - 0.5]
    one = torch.full((V,), -inf); one[V - 1] = 3.0; rows.append(one)
    first = torch.full((V,), -inf); first[0] = -2.0; rows.append(first)
    lows = torch.full((V,), low); lows[V // 2] = 1.0; rows.append(lows)
    few = torch.full((V,), -inf); few[torch.randperm(V, generator=g)[:4]] = torch.tensor([1.0, 2.0, 2.0, -5.0])[:min(4, V)]; rows.append(few)
    withnan = base.clone(); withnan[V // 3] = nan; rows.append(withnan)
    rows.append(torch.full((V,), nan))
    withinf = base.clone(); withinf[V // 2] = inf; rows.append(withinf)
    signed = torch.zeros(V); signed[::2] = -0.0; rows.append(signed)
    late = base.clone() * 0.1; late[V - V // 4:] += torch.arange(V // 4) * 0.001 + 5; rows.append(late)
    small = torch.full((V,), nan); small[:3] = torch.tensor([1.0, 1.0, 0.5]); rows.append(small)
    return torch.stack(rows).to(TYPES[kind])


@pytest.mark.gpu
@pytest.mark.parametrize("kind, V, k", [("f16", 33, 32), ("bf16", 5000, 20), ("f32", 70001, 32), ("f16", 151936, 5), ("bf16", 4096, 1)])
def test_special_rows(kind, V, k):
    g = torch.Generator().manual_seed(V)
    x = _special(V, kind, g)
    tokens = [(i * 7919) % V for i in range(len(x))]
    tokens[3], tokens[4] = -1, V  # outside: NaN
    with np.errstate(all="ignore"):
        _check(x, tokens, k, _run(x, tokens, k, V + 3))


@pytest.mark.gpu
def test_many_rows_agree_with_few():
    """A row's results go by the row: alone (its columns split) or among thousands."""
    g = torch.Generator().manual_seed(1)
    x = (torch.randn((3000, 700), generator=g) * 3).to(torch.bfloat16)
    tokens = torch.randint(0, 700, (3000,), generator=g).tolist()
    many, few = _run(x, tokens, 6), _run(x[:2], tokens[:2], 6)
    _check(x[::97], tokens[::97], 6, [t[::97] for t in many])
    assert np.array_equal(many[2][:2], few[2])
