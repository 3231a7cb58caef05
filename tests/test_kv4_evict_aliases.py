"""kv4_evict refuses outputs that lie on its inputs or on each other: workgroups read the one while others write the other."""

import struct

import pytest
import torch

import fp8_quantized_skinny_amd as sk
from fp8_quantized_skinny_amd._lib import lib

B, HK, D, PAGES, WIDTH, DPAGES, DWIDTH, KEEP = 2, 4, 128, 8, 2, 6, 2, 64
BLOCK = HK * 72 * D
# Buffers of the call in order, with their bytes.
SIZES = dict(cache=PAGES * BLOCK, table=4 * B * WIDTH, lens=4 * B, acc=4 * B * HK * 64 * WIDTH, dst=DPAGES * BLOCK, dst_table=4 * B * DWIDTH,
             kept=4 * B * HK * KEEP, new_lens=4 * B, new_acc=4 * B * HK * 64 * DWIDTH)
INPUTS, OUTPUTS = ("cache", "table", "lens", "acc", "dst_table"), ("dst", "kept", "new_lens", "new_acc")


def _call(at):
    cache = struct.pack("=QQQiiiiiff4x", at["cache"], at["table"], at["lens"], PAGES, WIDTH, B, HK, D, 1.0, 1.0)
    dst = struct.pack("=QQQiiiiiff4x", at["dst"], at["dst_table"], 0, DPAGES, DWIDTH, B, HK, D, 1.0, 1.0)
    return lib().kv4_evict(cache, at["acc"], dst, at["kept"], at["new_lens"], at["new_acc"], KEEP, 4, 8, None)


def _apart():
    at, p = {}, 1 << 20
    for name, size in SIZES.items():
        at[name] = p
        p += (size // 4096 + 2) * 4096
    return at


PAIRS = [(o, i) for o in OUTPUTS for i in INPUTS] + [(o, p) for k, o in enumerate(OUTPUTS) for p in OUTPUTS[k + 1:]]


@pytest.mark.parametrize("output, other", PAIRS)
def test_overlapping_buffers(output, other):
    """The same address, and the last 16 bytes of either under the first of the other (no GPU: refused before any launch)."""
    assert len(set(_apart().values())) == len(SIZES)
    for at, to in ((output, other), (other, output)):
        where = _apart()
        where[at] = where[to]
        assert _call(where) == sk.EINVAL
        where = _apart()
        where[at] = where[to] + (SIZES[to] - 1) // 16 * 16
        assert _call(where) == sk.EINVAL


@pytest.mark.gpu
def test_parts_of_one_allocation_serve_and_aliases_do_not():
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    n, keep = 100, 40
    pool = torch.randint(0, 0x30, (8, 1, 72 * 64), generator=g, device="cuda").to(torch.uint8)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    table, lens, acc = i32([[1, 3]]), i32([n]), torch.rand((1, 1, 128), generator=g, device="cuda")
    got = []
    for src, dst, dst_table in ((pool, torch.zeros_like(pool[:2]), i32([[1]])), (pool[:4], pool[4:], i32([[2]]))):
        kept, new_lens, new_acc = i32([[[7] * keep]]), i32([7]), torch.full((1, 1, 64), 7.0, device="cuda")
        sk.kv4_evict(src, table, lens, acc, dst, dst_table, kept, new_lens, new_acc, sinks=2, recent=3)
        got.append((dst[dst_table.long()].clone(), kept, new_lens, new_acc))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    wide = torch.full((1, 1, 128), 7.0, device="cuda")
    for bad in (dict(new_lens=lens), dict(new_acc=acc, dst_table=i32([[2, 3]])), dict(dst_cache=pool[3:]), dict(dst_cache=pool[1:3])):
        call = dict(cache=pool[:4], table=table, lens=lens, acc=acc, dst_cache=pool[4:], dst_table=i32([[2, 3]]), kept=i32([[[7] * keep]]),
                    new_lens=i32([7]), new_acc=wide)
        before = pool.clone()
        with pytest.raises(sk.SkinnyError) as e:
            sk.kv4_evict(**{**call, **bad})
        assert e.value.status == sk.EINVAL
        assert torch.equal(pool, before) and lens.tolist() == [n]
