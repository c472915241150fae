"""Rotations of more than 2^31 elements, which the library cuts into several launches: bit for bit single
fp32 operations in all parts, and nothing between the rows of a strided output is touched."""
import pytest
import torch

import microscaling_fp4_weight_amd as mx
from gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,rot,interleaved", [(96, 24, False), (80, 12, True), (128, 128, False)])
def test_rope_past_31_bits(dim, rot, interleaved):
    heads, gap = 64, 8
    tokens = 3221225472 // (heads * dim)  # below 2^32 elements; 24 of 96, pair by pair: 2.8e9 units of work
    gen = torch.Generator(device=DEV).manual_seed(dim)
    few = torch.randn((4099, heads, dim), generator=gen, device=DEV).bfloat16()
    x = torch.empty((tokens, heads, dim), dtype=torch.bfloat16, device=DEV)
    for t in range(0, tokens, len(few)):
        part = x[t:t + len(few)]
        part.copy_(few[:len(part)]).mul_(1 + t / tokens)
    positions = torch.randint(0, 777, (tokens,), generator=gen, device=DEV, dtype=torch.int32)
    table = mx.mxkv_rope_table(777, rot)
    whole = torch.full((tokens, heads, dim + gap), 3.0, dtype=torch.bfloat16, device=DEV)
    y = whole[..., :dim]
    mx.mxkv_rope(x, positions, table, interleaved=interleaved, y=y)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    for t in range(0, tokens, 1 << 16):
        at = slice(t, t + (1 << 16))
        c, s = table[positions[at].long()][:, None].chunk(2, dim=-1)
        p, q = x[at, :, a].float(), x[at, :, b].float()
        assert torch.equal(y[at, :, a], (p * c - q * s).bfloat16()), t
        assert torch.equal(y[at, :, b], (q * c + p * s).bfloat16()), t
        assert torch.equal(y[at, :, rot:], x[at, :, rot:]) and (whole[at, :, dim:] == 3.0).all(), t
