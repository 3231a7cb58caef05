"""The example's streams: every step's rows are tokens that the cache does not hold yet, in the stream's order."""

import pytest
import torch

import fp8_quantized_skinny_amd as sk
from fp8_quantized_skinny_amd.cached_decode import CachedDecoder

pytestmark = pytest.mark.gpu


def _qkv_of(d, tokens):
    """What the qkv GEMM makes of one token per stream, in a call of the decoder's own M (a row's sums do not go by the others)."""
    x = d.embedding[tokens.long()][:, None].expand(-1, d.T, -1).reshape(d.B * d.T, -1).contiguous()
    y = torch.empty_like(d.qkv)
    sk.nvfp4_gemm(d.w_qkv, x, y, workspace=d.workspace)
    return y.view(d.B, d.T, -1)[:, 0]


@pytest.mark.parametrize("streams, rows", [(1, 4), (2, 3), (2, 1), (1, 8)])
def test_no_token_of_a_stream_is_appended_twice(streams, rows):
    d = CachedDecoder(streams=streams, rows=rows, budget=100, keep=70, sinks=4, recent=16)
    continued = previous = None
    for step in range(100 // rows):
        d.step()
        torch.cuda.synchronize()
        fed = d.qkv.view(d.B, d.T, -1)
        if continued is not None:
            # the first row is the token that the stream was continued with
            assert torch.equal(fed[:, 0], _qkv_of(d, continued)), step
            # and the rows are not those that the last step ended with
            again = (fed[:, :-1] == previous[:, 1:]).all(-1)
            assert not again.any() or rows == 1, step
        # what a row is scored with is the row after it
        for t in range(rows - 1):
            assert torch.equal(fed[:, t + 1], _qkv_of(d, d.tokens[:, t])), (step, t)
        continued, previous = d.tokens[:, -1].clone(), fed.clone()
