"""Calls that need more workgroups than a grid holds are refused before any launch (no GPU)."""

import struct

import pytest

import fp8_quantized_skinny_amd as sk
from fp8_quantized_skinny_amd._lib import lib

A = 0x10000


def _cache(data=A, width=2, B=2, Hk=4, D=128):
    return struct.pack("=QQQiiiiiff4x", data, A, A, 8, width, B, Hk, D, 1.0, 1.0)


ROWS = struct.pack("=Qqqq", A, 4096, 512, 128)


def test_append_and_read():
    L = lib()
    assert L.kv4_append(_cache(B=65536, Hk=256), ROWS, ROWS, 0, 1, None) == sk.ESHAPE       # 2^24 workgroups
    assert L.kv4_append(_cache(B=64, Hk=64, width=1 << 20), ROWS, ROWS, 0, 1 << 20, None) == sk.ESHAPE
    assert L.kv4_read(_cache(B=65536, Hk=256), A, A, 0, 1, None) == sk.ESHAPE


@pytest.mark.parametrize("B, Hk, T, Hq", [(65536, 256, 1, 256), (65536, 128, 8, 128 * 64)])
def test_attention(B, Hk, T, Hq):
    L = lib()
    for width in (1, 64):
        assert L.kv4_attention(_cache(B=B, Hk=Hk, width=width), ROWS, 0, T, Hq, 0.1, A, A, A, 1 << 62, None) == sk.ESHAPE
    assert L.kv4_attention_weights(_cache(B=65536, Hk=256), ROWS, 0, 1, 256, 0.1, A, A, A, None) == sk.ESHAPE


def test_evict():
    call = lambda B, Hk, keep=64: lib().kv4_evict(_cache(B=B, Hk=Hk), A, _cache(data=2 * A, B=B, Hk=Hk, width=1 << 12), A, A, A, keep, 1, 1, None)  # noqa: E731
    assert call(65536, 64) == sk.ESHAPE                     # 2^22 of 1024 threads
    assert call(4096, 64, keep=64 << 12) == sk.ESHAPE
