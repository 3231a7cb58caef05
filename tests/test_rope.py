"""The norm of query and key heads with the rotation of their positions, against its definition in 64 bits."""

import struct

import numpy as np
import pytest
import torch

import fp8_quantized_skinny_amd as sk
from fp8_quantized_skinny_amd._lib import lib
from oracle import kv4 as oracle

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half a step of the type's least numbers
gpu = pytest.mark.gpu


# ---------------------------------------------------------------- refusals (no GPU)
A = 0x10000


def _rows(data=A, sequence=0, row=0, head=128):
    return struct.pack("=Qqqq", data, sequence, row, head)


def _call(q=None, k=None, positions=0x900000, freq=0x910000, qw=0x920000, kw=0x930000, type=0, B=1, T=1, Hq=8, Hk=2, D=128, rot=128, inter=0,
          eps=1e-6, amp=1.0, qo=None, ko=None):
    q, k = q or _rows(), k or _rows(A + 0x8000)
    qo, ko = qo or _rows(A + 0x10000), ko or _rows(A + 0x18000)
    return lib().qk_norm_rope(q, k, positions, freq, qw, kw, type, B, T, Hq, Hk, D, rot, inter, eps, amp, qo, ko, None)


@pytest.mark.parametrize("bad, status", [
    (dict(type=2), sk.EINVAL), (dict(type=-1), sk.EINVAL), (dict(D=96), sk.ESHAPE), (dict(D=512), sk.ESHAPE), (dict(B=0), sk.ESHAPE),
    (dict(T=0), sk.ESHAPE), (dict(Hq=0), sk.ESHAPE), (dict(Hk=0), sk.ESHAPE), (dict(Hq=65537), sk.ESHAPE), (dict(rot=144), sk.ESHAPE),
    (dict(rot=-16), sk.ESHAPE), (dict(rot=24), sk.ESHAPE), (dict(rot=8), sk.ESHAPE), (dict(B=1 << 16, T=1 << 15), sk.ESHAPE),
    (dict(B=1 << 20, T=1 << 10, Hq=64), sk.ESHAPE), (dict(positions=None), sk.EINVAL), (dict(freq=None), sk.EINVAL), (dict(inter=2), sk.EINVAL),
    (dict(eps=-1.0), sk.EINVAL), (dict(eps=float("nan")), sk.EINVAL), (dict(amp=float("inf")), sk.EINVAL), (dict(positions=A + 2), sk.EALIGN),
    (dict(freq=A + 1), sk.EALIGN), (dict(qw=A + 2), sk.EALIGN), (dict(kw=A + 2), sk.EALIGN), (dict(q=_rows(0)), sk.EINVAL),
    (dict(k=_rows(A + 8)), sk.EALIGN), (dict(qo=_rows(head=-8)), sk.EINVAL), (dict(ko=_rows(row=4)), sk.EALIGN)])
def test_refusals(bad, status):
    assert _call(**bad) == status


@pytest.mark.parametrize("bad", [
    dict(qo=_rows(A + 0x100)),                                    # q_out over a part of q
    dict(qo=_rows(A + 0x8000 - 0x700)),                           # q_out over k
    dict(ko=_rows(A + 0x700)),                                    # k_out over q
    dict(qo=_rows(A + 0x20000), ko=_rows(A + 0x20000 + 0x700)),   # one output over the other
    dict(qo=_rows(head=256)),                                     # q's pointer, other strides
    dict(qo=_rows(A + 0x20000, head=64)),                         # heads of an output over each other
    dict(qo=_rows(A + 0x20000, head=0)),
    dict(T=2, q=_rows(row=4096), qo=_rows(A + 0x20000, row=896)),  # tokens of an output over each other
    dict(T=2, q=_rows(row=1280), k=_rows(A + 2048, row=1280), qo=_rows(A + 2048, row=1280), ko=_rows(A + 0x20000, row=256)),
    dict(qo=_rows(0x900000 - 2048 + 16)), dict(ko=_rows(0x930000)), dict(ko=_rows(0x910000)),
])
def test_outputs_that_overlap_are_refused(bad):
    assert _call(**bad) == sk.EINVAL


def test_frequencies():
    assert np.allclose(sk.rope_inv_freq(8, 10000.0), [1.0, 0.1, 0.01, 0.001])
    assert np.allclose(sk.rope_inv_freq(8, 10000.0, factor=4.0), np.array([1.0, 0.1, 0.01, 0.001]) / 4)
    f, plain = sk.rope_inv_freq(128, 10000.0, factor=8.0, original=4096), sk.rope_inv_freq(128, 10000.0)
    turns = plain * 4096 / (2 * np.pi)
    assert f.dtype == np.float32 and np.allclose(f[turns > 40], plain[turns > 40]) and np.allclose(f[turns < 0.8], plain[turns < 0.8] / 8)
    assert (np.diff(plain / f) >= -1e-6).all() and len(sk.rope_inv_freq(0)) == 0
    for bad in (dict(rot=7), dict(rot=-2), dict(rot=8, base=1.0), dict(rot=8, factor=0.0), dict(rot=8, original=-1), dict(rot=8, fast=1.0)):
        with pytest.raises(ValueError):
            sk.rope_inv_freq(**bad)


# ---------------------------------------------------------------- GPU
CASES = [  # type, B, T, Hq, Hk, D, rot, interleaved, norm, amplitude, greatest position
    ("f16", 1, 1, 48, 4, 128, 128, False, True, 1.0, 9000),
    ("bf16", 3, 5, 24, 4, 256, 64, True, True, 1.25, 1 << 20),
    ("f16", 2, 7, 5, 1, 256, 256, False, True, 1.0, 1 << 30),
    ("bf16", 1, 130, 28, 4, 64, 64, False, False, 1.0, 4096),
    ("f16", 9, 1, 16, 16, 64, 16, False, True, 0.5, 100),
    ("bf16", 1, 3, 1, 1, 128, 96, False, True, 1.0, 131072),
    ("f16", 2, 2, 3, 7, 128, 48, True, False, 1.0, 2000),
    ("f16", 1, 400, 48, 4, 128, 128, True, True, 1.0, 32768),
    ("bf16", 2, 300, 48, 4, 128, 128, False, True, 1.0, 1000000),
    ("bf16", 1, 4, 8, 2, 128, 0, False, True, 1.0, 10),
    ("f16", 1, 4, 8, 2, 64, 0, True, False, 3.0, 10),
    ("f16", 5, 200, 24, 4, 256, 32, False, False, 1.0, 50000),
    ("f16", 1, 900, 27, 5, 64, 64, False, True, 1.0, 50000),
    ("bf16", 1, 1400, 8, 1, 128, 64, False, True, 1.0, 50000),
]


def _inputs(rng, kind, B, T, Hq, Hk, D, rot, norm, top):
    qkv = rng.standard_normal((B, T, (Hq + 2 * Hk) * D)) * np.exp2(rng.integers(-4, 4, (Hq + 2 * Hk) * D))
    qkv = torch.from_numpy(qkv).to(TYPES[kind])
    pos = rng.integers(0, top + 1, (B, T)).astype(np.int32)
    pos[0, 0] = top
    w = (1.0 + 0.5 * rng.standard_normal((2, D))).astype(np.float32) if norm else (None, None)
    return qkv, pos, sk.rope_inv_freq(rot, 10000.0 if top < 1 << 21 else 1e6), w


def _views(qkv, Hq, Hk, D):
    return qkv[..., :Hq * D].unflatten(-1, (Hq, D)), qkv[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D))


def _check(kind, got, x, weight, pos, freq, amplitude, interleaved, eps, rng):
    """A result is rounded once (half a step of the type); before that the value u has about six fp32 roundings (the sum of
    squares' error is a mean of them), a product with cos or sin has theirs: 2^-24 of a turn in the angle (2 pi 2^-24 of the
    value), three roundings and the sine's own 2^-22."""
    B, T, H, D = x.shape
    at = [(b, t, h) for b in range(B) for t in range(T) for h in range(H)]
    if len(at) > 300:
        at = [at[i] for i in rng.permutation(len(at))[:300]] + [(0, 0, 0), (B - 1, T - 1, H - 1)]
    y, x = got.double().cpu().numpy(), x.double().cpu().numpy()
    for b, t, h in at:
        want, size = oracle.norm_rope(x[b, t, h], weight, eps, pos[b, t], freq, amplitude, interleaved)
        tol = np.abs(want) * HALF_STEP[kind] + size * (20 * 2.0 ** -24) + TINY[kind]
        err = np.abs(y[b, t, h] - want)
        assert (err <= tol).all(), (b, t, h, (err / tol).max())


@gpu
@pytest.mark.parametrize("kind, B, T, Hq, Hk, D, rot, interleaved, norm, amplitude, top", CASES)
def test_norm_and_rotation(kind, B, T, Hq, Hk, D, rot, interleaved, norm, amplitude, top):
    rng = np.random.default_rng(D + T + rot)
    qkv, pos, freq, (qw, kw) = _inputs(rng, kind, B, T, Hq, Hk, D, rot, norm, top)
    dev = qkv.cuda()
    q, k = _views(dev, Hq, Hk, D)
    cuda = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    args = dict(q_weight=cuda(qw), k_weight=cuda(kw), eps=1e-5, amplitude=amplitude, interleaved=interleaved)
    qo, ko = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda"), torch.full(k.shape, 7.0, dtype=q.dtype, device="cuda")
    sk.qk_norm_rope(q, k, cuda(pos), cuda(freq), qo, ko, **args)
    assert torch.equal(dev.view(torch.int16).cpu(), qkv.view(torch.int16))
    _check(kind, qo, q, qw, pos, freq, amplitude, interleaved, 1e-5, rng)
    _check(kind, ko, k, kw, pos, freq, amplitude, interleaved, 1e-5, rng)
    # In place in the qkv buffer: the same bits, and the values stay as they were.
    values = dev[..., (Hq + Hk) * D:].clone()
    sk.qk_norm_rope(q, k, cuda(pos), cuda(freq), q, k, **args)
    for a, b in ((q, qo), (k, ko), (dev[..., (Hq + Hk) * D:], values)):
        assert torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))
    if B == 1:  # the same of packed rows, into outputs whose heads lie apart
        q3, k3 = _views(qkv.cuda()[0], Hq, Hk, D)
        wide = torch.full((Hq + Hk, T, D), 3.0, dtype=q.dtype, device="cuda").transpose(0, 1)
        sk.qk_norm_rope(q3, k3, cuda(pos[0]), cuda(freq), wide[:, :Hq], wide[:, Hq:], **args)
        assert torch.equal(wide[:, :Hq].contiguous().view(torch.int16), qo[0].view(torch.int16))
        assert torch.equal(wide[:, Hq:].contiguous().view(torch.int16), ko[0].view(torch.int16))


@gpu
def test_one_weight_alone_negative_positions_and_values_without_a_number():
    rng = np.random.default_rng(3)
    Hq, Hk, D, rot = 4, 2, 128, 64
    qkv, _, freq, (qw, _) = _inputs(rng, "f16", 1, 6, Hq, Hk, D, rot, True, 100)
    pos = np.array([[-5, 0, 2 ** 31 - 1, -2 ** 31, 7, 8]], np.int32)
    qkv[0, 4, 100] = float("inf")   # of the part that does not turn, where nothing is normed: it stays by itself
    qkv[0, 5, Hq * D + 3] = float("nan")
    q, k = _views(qkv.cuda(), Hq, Hk, D)
    for weights in (dict(q_weight=torch.from_numpy(qw).cuda()), dict(k_weight=torch.from_numpy(qw).cuda())):
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        sk.qk_norm_rope(q, k, torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda(), qo, ko, eps=0.0, **weights)
        normed = "q_weight" in weights
        _check("f16", qo[:, :4], q[:, :4], qw if normed else None, pos, freq, 1.0, False, 0.0, rng)
        _check("f16", ko[:, :5], k[:, :5], None if normed else qw, pos, freq, 1.0, False, 0.0, rng)
        bad = qo[0, 4, 0]
        if normed:  # x / inf, and inf / inf
            assert bad[100].isnan() and (bad[:100] == 0).all()
        else:
            assert bad[100] == float("inf") and bad.isfinite().sum() == D - 1
        bad = ko[0, 5, 0].isnan()
        assert bad.all() if not normed else (bad[3] and bad[35] and bad.sum() == 2)


@gpu
def test_rows_of_zeros_need_an_epsilon():
    x = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16, device="cuda")
    w, pos, freq = torch.ones(64, device="cuda"), torch.zeros((1, 2), dtype=torch.int32, device="cuda"), torch.ones(32, device="cuda")
    q, k = torch.empty_like(x), torch.empty_like(x)
    sk.qk_norm_rope(x, x, pos, freq, q, k, q_weight=w, k_weight=w, eps=1e-6)
    assert (q == 0).all() and (k == 0).all()


@gpu
def test_binding_refuses_what_does_not_fit():
    T, Hq, Hk, D = 2, 4, 2, 64
    q, k = (torch.zeros((1, T, H, D), dtype=torch.float16, device="cuda") for H in (Hq, Hk))
    pos, freq, w = torch.zeros((1, T), dtype=torch.int32, device="cuda"), torch.ones(16, device="cuda"), torch.ones(D, device="cuda")
    good = dict(q=q, k=k, positions=pos, inv_freq=freq, q_out=q.clone(), k_out=k.clone(), q_weight=w, k_weight=w)
    sk.qk_norm_rope(**good)
    for name, value, error in (("q", q.float(), TypeError), ("k", k.bfloat16(), TypeError), ("q_out", q.bfloat16(), TypeError),
                               ("k", k[:, :1], ValueError), ("k", k[..., :32], ValueError), ("q_out", q[:, :, :2], ValueError),
                               ("positions", pos[:, :1], ValueError), ("positions", pos.long(), TypeError), ("inv_freq", freq.double(), TypeError),
                               ("inv_freq", freq[None], ValueError), ("q_weight", w[:32], ValueError), ("k_weight", w.half(), TypeError),
                               ("q", q.cpu(), TypeError), ("q", q.transpose(2, 3), ValueError), ("q", q[0], ValueError), ("k", k[:0], ValueError)):
        with pytest.raises(error):
            sk.qk_norm_rope(**{**good, name: value})
    for name, value in (("q_out", q[:, :1].expand(1, T, Hq, D)),
                        ("inv_freq", torch.ones(40, device="cuda")), ("inv_freq", torch.ones(20, device="cuda")), ("eps", -1.0)):
        with pytest.raises(sk.SkinnyError):
            sk.qk_norm_rope(**{**good, name: value})
