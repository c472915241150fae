"""What a new token's slot holds reaches the rows that see it, and no others: values past bf16's range, and what a
non-finite value or key leaves behind when it is written."""
import numpy as np
import pytest
import torch

import microscaling_fp4_weight_amd as mx
from gpu_util import DEV
from test_gpu_kv import dev, host, ints, make_cache

pytestmark = pytest.mark.gpu

HELD, PAGE, BAD = 75, 16, 7  # cached tokens, page size, the new token that is poked


def tree(rng, new):
    m = np.eye(new, dtype=bool)
    for i in range(1, new):
        m[i] |= m[rng.integers(0, i)]
    return m


def masks(rng, new):
    """(mask argument, who sees whom): causal, and a tree."""
    m = tree(rng, new)
    return [(None, np.tril(np.ones((new, new), dtype=bool))), (torch.from_numpy(m[None]).to(DEV), m)]


def case(dim, q_heads, new=20, element="fp4", seed=0):
    rng = np.random.default_rng(dim + q_heads + seed)
    cache, _ = make_cache(rng, 6, 2, PAGE, dim, element, "e8m0", 16)
    table = ints([[3, 1, 4, 0, 5, 2]])
    q = dev(rng.standard_normal((1, new, q_heads, dim)), "bf16")
    at = table[0, (HELD + BAD) // PAGE].item(), (HELD + BAD) % PAGE
    return rng, cache, q, dict(block_table=table, lens=ints([HELD]), block=16, element=element), at


@pytest.mark.parametrize("q_heads", [2, 6, 12])
@pytest.mark.parametrize("dim", [64, 80, 128, 256])
@pytest.mark.parametrize("element,code,scale", [("fp4", 0x77, 0xFE), ("fp4", 0xFE, 0xFD), ("fp4", 0x62, 0xFE), ("fp8", 0x7E, 0xFE),
                                                ("fp8", 0xFE, 0xF8), ("fp8", 0x7E, 0xF7)])
def test_values_past_the_range_of_bf16(element, code, scale, dim, q_heads):
    rng, cache, q, kind, (page, place) = case(dim, q_heads, element=element)
    for mask, sees in masks(rng, 20):
        want = mx.mxkv_attention(q, cache, mask=mask, **kind)
        for parts in ((2, 3), (0, 1), (0, 1, 2, 3)):
            poked = mx.KVCache(*(t.clone() for t in cache))
            for t in parts:
                poked[t][page, :, place] = (code, scale)[t % 2]
            got = mx.mxkv_attention(q, poked, mask=mask, **kind)
            hidden = torch.from_numpy(~sees[:, BAD]).to(DEV)
            assert torch.equal(got[0, hidden], want[0, hidden]), (mask is None, parts)
            if parts == (2, 3):  # elements of code 0x6 and more are past 2^128, whatever their weight
                assert not torch.isfinite(got[0, ~hidden].float()).all(-1).any()


@pytest.mark.parametrize("dim", [64, 80, 128, 256])
@pytest.mark.parametrize("element,code,scale,value", [("fp4", 0x11, 0xFE, 2.0 ** 126), ("fp4", 0x22, 0xFD, 2.0 ** 126), ("fp8", 0x38, 0xFD, 2.0 ** 126),
                                                      ("fp8", 0x01, 0xF8, 2.0 ** 112)])
def test_large_values_that_are_finite(element, code, scale, value, dim):
    """A block scale of a size that could pass the range under other codes: rows that see the token get their part of it."""
    rng, cache, q, kind, (page, place) = case(dim, 6, element=element)
    for mask, sees in masks(rng, 20):
        want, lse = mx.mxkv_attention(q, cache, mask=mask, return_lse=True, **kind)
        poked = mx.KVCache(*(t.clone() for t in cache))
        for t in (2, 3):
            poked[t][page, :, place] = (code, scale)[t % 2]
        got = mx.mxkv_attention(q, poked, mask=mask, **kind)
        hidden = torch.from_numpy(~sees[:, BAD]).to(DEV)
        assert torch.equal(got[0, hidden], want[0, hidden])
        k, _ = mx.mxkv_read(cache, ints([page * PAGE + place]), block=16, element=element, out_dtype=torch.float32)
        score = np.einsum("thd,hd->th", host(q[0]).astype(np.float64), np.repeat(host(k[0]), 3, axis=0).astype(np.float64)) * dim ** -0.5
        part = np.exp(score - host(lse[0])) * value  # next to which the other values are nothing
        rows = sees[:, BAD]
        # two roundings to bf16 at most (p and the result), and fp32 scores
        assert np.all(np.abs(host(got[0])[rows] / part[rows][..., None] - 1) <= 2.0 ** -7 + 2.0 ** -10)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dim", [64, 80, 128, 256])
@pytest.mark.parametrize("element", ["fp4", "fp8"])
def test_tokens_written_from_values_that_are_not_finite(element, dim, bad):
    rng, cache, q, kind, (page, place) = case(dim, 6, element=element)
    x = dev(rng.standard_normal((2, 1, 2, dim)), "bf16")
    x[:, :, :, 5] = bad
    for mask, sees in masks(rng, 20):
        want = mx.mxkv_attention(q, cache, mask=mask, **kind)
        poked = mx.KVCache(*(t.clone() for t in cache))
        mx.mxkv_write(x[0], x[1], poked, ints([page * PAGE + place]), block=16, element=element)
        got = mx.mxkv_attention(q, poked, mask=mask, **kind)
        hidden = torch.from_numpy(~sees[:, BAD]).to(DEV)
        assert torch.equal(got[0, hidden], want[0, hidden])


@pytest.mark.parametrize("q_heads", [2, 6, 12])
@pytest.mark.parametrize("dim", [64, 80, 128, 256])
@pytest.mark.parametrize("element", ["fp4", "fp8"])
def test_a_seen_nan_is_nan_whatever_its_weight(element, dim, q_heads):
    """A NaN value under a score far below the row's maximum, so that its weight is 0: the rows that see it are NaN, as
    they are where nobody hides it, and the others keep their bits."""
    new = 20
    rng, cache, q, kind, (page, place) = case(dim, q_heads, element=element)
    q[:] = 40.0 * torch.sign(q[:, :1, :1])
    poked = mx.KVCache(*(t.clone() for t in cache))
    low = torch.where(q[0, 0, 0] > 0, -6.0, 6.0).bfloat16().expand(1, 2, dim).contiguous()  # scores of -240 dim^0.5
    mx.mxkv_write(low, low, poked, ints([page * PAGE + place]), block=16, element=element)
    free = mx.KVCache(*(t.clone() for t in poked))
    poked[3][page, :, place] = 0xFF
    nobody = np.ones((new, new), dtype=bool)
    for mask, sees in [*masks(rng, new), (torch.from_numpy(nobody[None]).to(DEV), nobody)]:
        want = mx.mxkv_attention(q, free, mask=mask, **kind)
        got = mx.mxkv_attention(q, poked, mask=mask, **kind)
        hidden = torch.from_numpy(~sees[:, BAD]).to(DEV)
        assert torch.isfinite(want.float()).all() and torch.equal(got[0, hidden], want[0, hidden])
        assert torch.isnan(got[0, ~hidden]).all()


@pytest.mark.parametrize("element,scale", [("fp4", 0xFE), ("fp8", 0xFE), ("fp8", 0xF9)])
@pytest.mark.parametrize("dim", [64, 80, 128, 256])
def test_keys_that_score_minus_infinity_have_no_weight(element, scale, dim):
    """Keys past the range of fp32 on the side where scores are -inf, the first of a sequence among them: the
    same bits as with keys whose scores are finite and have no weight either."""
    rng, cache, q, kind, _ = case(dim, 6, element=element)
    q = q.abs() + 0.01
    first = kind["block_table"][0, 0].item()
    results = []
    for byte in (scale, 0x90):
        poked = mx.KVCache(*(t.clone() for t in cache))
        for place in (0, 1, 2, 3, 9):
            poked[0][first, :, place] = 0xFF if element == "fp4" else 0xFE  # -6, -448
            poked[1][first, :, place] = byte
        results.append(mx.mxkv_attention(q, poked, return_lse=True, **kind))
    assert torch.isfinite(results[1][0].float()).all()
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])


@pytest.mark.parametrize("dim", [64, 80, 128, 256])
def test_a_seen_nan_is_nan_among_tokens_of_no_weight(dim):
    """Every fourth or thirty-second token far below the row's maximum, one of them of NaN values."""
    rng, cache, q, kind, _ = case(dim, 6)
    q[:] = 40.0 * torch.sign(q[:, :1, :1])
    low = torch.where(q[0, 0, 0] > 0, -6.0, 6.0).bfloat16()
    table = kind["block_table"][0]
    for step in (4, 32):
        poked = mx.KVCache(*(t.clone() for t in cache))
        tokens = torch.arange(2, HELD + 20, step, device=DEV)
        slots = table[tokens // PAGE] * PAGE + (tokens % PAGE).int()
        rows = low.expand(len(tokens), 2, dim).contiguous()
        mx.mxkv_write(rows, rows, poked, slots, block=16)
        assert torch.isfinite(mx.mxkv_attention(q, poked, **kind).float()).all()
        at = int(slots[1])
        poked[3][at // PAGE, :, at % PAGE] = 0xFF
        assert torch.isnan(mx.mxkv_attention(q, poked, **kind)).all()
