"""Which views qk_norm_rope takes as outputs beside others of the same buffer: no two may share an element."""

import itertools
import random
import struct

import numpy as np
import pytest
import torch

import fp8_quantized_skinny_amd as sk
from fp8_quantized_skinny_amd._lib import lib

D = 64
BASE, FAR = 0x100000, 0x40000000
gpu = pytest.mark.gpu


def _rows(at, sequence, row, head):
    return struct.pack("=Qqqq", at, sequence, row, head)


def _tokens(at, B, T, H, sequence, row, head):
    """The elements of a view, in units of the eight that strides are multiples of."""
    starts = [at + b * sequence + t * row + h * head for b in range(B) for t in range(T) for h in range(H)]
    return [s // 8 + i for s in starts for i in range(D // 8)]


def _refused(B, T, at, sequence, row, output, H=(1, 1), head=(D, D)):
    """The status of a call whose k_out lies `at` elements behind q (output: behind q_out) with the same strides."""
    q = _rows(BASE, sequence, row, head[0])
    beside = _rows(BASE + 2 * at, sequence, row, head[1])
    apart = [_rows(FAR + i * 0x4000000, T * 4096, 4096, D) for i in range(2)]
    args = (apart[0], apart[1], q, beside) if output else (q, apart[0], apart[1], beside)
    return lib().qk_norm_rope(args[0], args[1], 0x900000, 0x910000, None, None, 0, B, T, *H, D, D, 0, 1e-6, 1.0, args[2], args[3], None)


# Tokens of one view on another's of the next sequence: B, T, the distance, and steps of the sequence and the row.
CROSSING = [(2, 2, 160, 448, 608), (2, 2, 128, 384, 256), (2, 2, 160, 384, 224), (3, 4, 64, 448, 128), (5, 2, 64, 128, 576), (4, 3, 448, 192, 1024)]


@pytest.mark.parametrize("output", [False, True])
@pytest.mark.parametrize("B, T, at, sequence, row", CROSSING)
def test_tokens_that_cross_are_refused(B, T, at, sequence, row, output):
    assert set(_tokens(0, B, T, 1, sequence, row, D)) & set(_tokens(at, B, T, 1, sequence, row, D))
    assert _refused(B, T, at, sequence, row, output) == sk.EINVAL


def test_every_overlap_of_random_steps_is_refused():
    rng, crossed = random.Random(0), 0
    while crossed < 3000:
        B, T, H = rng.randint(1, 5), rng.randint(1, 5), (rng.randint(1, 2), rng.randint(1, 2))
        head = (D * rng.randint(1, 2), D * rng.randint(1, 2))
        sequence, row = (8 * rng.randint(8, 160) for _ in range(2))
        at = 8 * rng.randint(0, 200)
        if not set(_tokens(0, B, T, H[0], sequence, row, head[0])) & set(_tokens(at, B, T, H[1], sequence, row, head[1])):
            continue
        crossed += 1
        assert _refused(B, T, at, sequence, row, rng.random() < 0.5, H, head) == sk.EINVAL, (B, T, at, sequence, row, H, head)


# Views of one buffer that share nothing: slices of ordinary layouts, and steps that cross without meeting.
APART = [("BTHD", 3, 4), ("TBHD", 3, 4), ("BHTD", 3, 4), ("THBD", 3, 4), ("HBTD", 2, 5), ("HTBD", 2, 5)]


def _reference(x, w, pos, freq):
    u = x.double()
    u = u * w.double() / (u.square().mean(-1, keepdim=True) + float(np.float32(1e-6))).sqrt()
    angle = pos.double()[..., None, None] * freq.double()
    a, b = u[..., :D // 2], u[..., D // 2:]
    size = (a.abs() + b.abs()).repeat(1, 1, 1, 2)
    return torch.cat((a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()), -1), size


def _check(q, k, qo, ko):
    B, T = q.shape[:2]
    g = torch.Generator().manual_seed(1)
    pos = torch.randint(0, 1000, (B, T), generator=g, dtype=torch.int32)
    freq, (qw, kw) = torch.from_numpy(sk.rope_inv_freq(D)), 1.0 + 0.1 * torch.randn((2, D), generator=g)
    want = [_reference(x.cpu(), w, pos, freq) for x, w in ((q, qw), (k, kw))]
    sk.qk_norm_rope(q, k, pos.cuda(), freq.cuda(), qo, ko, q_weight=qw.cuda(), k_weight=kw.cuda())
    for got, (y, size) in zip((qo, ko), want):
        # rounded once to fp16, after some twenty roundings of fp32
        assert ((got.double().cpu() - y).abs() <= y.abs() * 2.0 ** -11 + size * 20 * 2.0 ** -24 + 2.0 ** -25).all()


@gpu
@pytest.mark.parametrize("order, B, T", APART)
def test_slices_of_one_buffer_serve(order, B, T):
    """q, k and their outputs as neighbouring heads of a buffer in any order of its dimensions, and in place."""
    Hq, Hk = 3, 2
    sizes = dict(B=B, T=T, H=2 * (Hq + Hk), D=D)
    buffer = torch.randn([sizes[c] for c in order], generator=torch.Generator().manual_seed(0)).half().cuda()
    views = buffer.permute(*(order.index(c) for c in "BTHD")).split([Hq, Hk, Hq, Hk], 2)
    _check(*views)
    _check(views[0], views[1], views[0], views[1])


@gpu
@pytest.mark.parametrize("order, B, T", [*APART, ("BTHD", 1, 1), ("BTHD", 1, 7), ("BTHD", 7, 1)])
def test_heads_in_turn_serve(order, B, T):
    """A head's query, key and value behind one another, and the next head's behind these."""
    sizes = dict(B=B, T=T, H=3, D=3 * D)
    buffer = torch.randn([sizes[c] for c in order], generator=torch.Generator().manual_seed(0)).half().cuda()
    q, k, v = buffer.permute(*(order.index(c) for c in "BTHD")).split(D, 3)
    values = v.clone()
    _check(q, k, torch.empty_like(q), torch.empty_like(k))
    _check(q, k, q, k)
    _check(q, k[:, :, :2], q, k[:, :, :2])
    assert torch.equal(v, values)


@gpu
@pytest.mark.parametrize("B, T, at, sequence, row", [(2, 2, 192, 384, 960), (3, 2, 128, 256, 832), (2, 3, 64, 1000, 256), (4, 5, 128, 1408, 256)])
def test_steps_that_cross_without_meeting_serve(B, T, at, sequence, row):
    for a, b in itertools.combinations((0, at), 2):
        assert not set(_tokens(a, B, T, 1, sequence, row, D)) & set(_tokens(b, B, T, 1, sequence, row, D))
    buffer = torch.randn(8192, generator=torch.Generator().manual_seed(0)).half().cuda()
    q, k = (torch.as_strided(buffer, (B, T, 1, D), (sequence, row, D, 1), x) for x in (0, at))
    _check(q, k, torch.empty((B, T, 1, D), dtype=torch.float16, device="cuda"), torch.empty((B, T, 1, D), dtype=torch.float16, device="cuda"))
    _check(q, k, q, k)
