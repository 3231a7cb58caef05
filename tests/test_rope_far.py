"""Angles of the farthest positions: right to 2^-24 of a turn at every position, for frequencies up to 1."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import fp8_quantized_skinny_amd as sk

pytestmark = pytest.mark.gpu
TURN = Fraction("0.159154943091895335768883763372514362034459645740456448747667344058896797634226535")  # 1 / 2 pi

# Positions and frequencies whose angle is next to a multiple of pi, so that bf16 shows its sine to 2^-8 of next to
# nothing.  Were both products rounded to fp64, they would be off by 2^-23.8 of a turn.
NEAR = [(2138457421, 0.9854873418807983), (2139601407, 0.9059668779373169), (2134062455, 0.8244434595108032),
        (2132079581, 0.8125160932540894), (2145235406, 0.997768223285675)]
FAR = [(2 ** 31 - 1, 1.0), (-2 ** 31, 1.0), (2 ** 30 + 1, 0.75), (123456789, 0.1), (1, 1.0), (-7, 0.3333333432674408), (0, 1.0), (2 ** 31 - 1, 1e-30)]


def _angle(position, freq):
    """Radians within half a turn, of a float32 frequency."""
    turns = position * Fraction(float(np.float32(freq))) * TURN
    return 2.0 * np.pi * float(turns - round(turns))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_far_angles(D, interleaved):
    pairs = [*NEAR, *FAR, *[(-p, f) for p, f in NEAR]]
    pos = torch.tensor([p for p, _ in pairs], dtype=torch.int32, device="cuda")
    freq = torch.tensor([f for _, f in pairs], dtype=torch.float32, device="cuda")
    freq = torch.nn.functional.pad(freq, (0, 32 - len(pairs)), value=1.0)  # rot 64: token n is looked at in pair n
    x = torch.zeros((len(pairs), 1, D), dtype=torch.bfloat16, device="cuda")
    at = [(2 * n, 2 * n + 1) if interleaved else (n, n + 32) for n in range(len(pairs))]
    for n, (i, _) in enumerate(at):
        x[n, 0, i] = 1.0
    q, k = torch.empty_like(x), torch.empty_like(x)
    sk.qk_norm_rope(x, x, pos, freq, q, k, interleaved=interleaved)
    for y in (q, k):
        y = y[:, 0].double().cpu().numpy()
        for n, (i, j) in enumerate(at):
            angle = _angle(*pairs[n])
            for got, want in ((y[n, i], np.cos(angle)), (y[n, j], np.sin(angle))):
                # the angle, the sine's own 2^-22 of it, and one rounding to bf16
                assert abs(got - want) <= 2.0 * np.pi * 2.0 ** -24 + abs(want) * (2.0 ** -22 + 2.0 ** -8) + 2.0 ** -134, (n, pairs[n], got, want)
