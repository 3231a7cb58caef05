"""kv4_attention's plan counts the pages of a whole table in 32 bits; larger tables are refused (no GPU: before any launch)."""

import struct

import pytest

import fp8_quantized_skinny_amd as sk
from fp8_quantized_skinny_amd._lib import lib

A = 0x10000


@pytest.mark.parametrize("B, width", [(65536, 32768), (65536, (1 << 25) - 1), (64, (1 << 25) - 1), (65535, 32768), (128, 1 << 24)])
@pytest.mark.parametrize("D, T, Hq", [(128, 1, 1), (64, 8, 4), (256, 8, 8)])
def test_attention_refuses_tables_past_32_bits(B, width, D, T, Hq):
    assert B * (width + 1) >= 1 << 31
    cache = struct.pack("=QQQiiiiiff4x", A, A, A, 8, width, B, 1, D, 1.0, 1.0)
    rows = struct.pack("=Qqqq", A, 4096, 512, 256)
    assert sk.kv4_attention_workspace_bytes(B, T, Hq, 1, D, width) == 0
    assert lib().kv4_attention(cache, rows, 0, T, Hq, 0.1, A, A, A, 1 << 62, None) == sk.ESHAPE


def test_tables_within_32_bits_have_a_plan():
    for B, width in ((65535, 32767), (1, (1 << 25) - 1), (63, (1 << 25) - 1)):
        assert B * (width + 1) < 1 << 31
        assert sk.kv4_attention_workspace_bytes(B, 1, 1, 1, 128, width) > 0
