"""What the attention over the cache may lose: fp32 work rounded once to bf16 at the end, for every head
size, number of rows and format.  Elements whose terms nearly cancel show every other rounding."""
import numpy as np
import pytest
import torch

import kv_util as ku
import microscaling_fp4_weight_amd as mx
from gpu_util import DEV
from test_gpu_kv import KINDS, check_attention, dev, host, ints, make_cache, sequence

pytestmark = pytest.mark.gpu


def check(seed, lens, new, q_heads, heads, dim, element="fp4", fmt="e8m0", block=32, page=16, q_size=1.5):
    rng = np.random.default_rng(seed)
    each = [-(-(n + new) // page) for n in lens]
    cache, values = make_cache(rng, sum(each), heads, page, dim, element, fmt, block)
    order, table, at = rng.permutation(sum(each)), np.zeros((len(lens), max(each)), dtype=int), 0
    for b, n in enumerate(each):
        table[b, :n] = order[at:at + n]
        at += n
    q = ku.to_type((rng.standard_normal((len(lens), new, q_heads, dim)) * q_size).astype(np.float32), "bf16")
    out = mx.mxkv_attention(dev(q, "bf16"), cache, ints(table), ints(lens), block=block, fmt=fmt, element=element)
    out = host(out).astype(np.float64)
    for b, cached in enumerate(lens):
        held = cached + new
        see = np.arange(held)[None] <= cached + np.arange(new)[:, None]
        ref, _, mass, most = ku.attention(q[b], *sequence(values, table[b], held, page), see, dim ** -0.5)
        # An exponent is off by d (fp32 sums of dim exact products and a few factors), which p and its sum both
        # have, and the exponential by a few units of 2^-24: e.  What is left of p after two parts of 8 bits is
        # 2^-16; adding up `held` terms in any order rounds each at most `held` times by 2^-24, in the
        # sum of p too; the result is rounded to bf16.
        d = (dim + 16) * 2.0 ** -24 * most
        e = (2 * d + 2.0 ** -18)[..., None]
        tol = mass * (2.0 ** -16 + e + 2 * held * 2.0 ** -24) * 1.01 + ku.U8 * np.abs(ref) + 1e-30
        worst = np.max(np.abs(out[b] - ref) / tol)
        assert worst <= 1, f"sequence {b}: {np.mean(np.abs(out[b] - ref) > tol):.2%} of the outputs off, worst {worst:.2f} of the bound"


@pytest.mark.parametrize("new", [1, 4, 9])
@pytest.mark.parametrize("dim", [64, 80, 128, 256])
def test_rows(dim, new):
    """One, two and four row tiles of a wave, and the kernel of other head sizes."""
    check(dim + new, [33, 7, 60], new, 16, 2, dim, block=16)


@pytest.mark.parametrize("element,fmt,block", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_formats(dim, element, fmt, block):
    if block > dim:
        pytest.skip("a block is no longer than a head")
    check(dim, [37, 20], 5, 8, 2, dim, element, fmt, block)


@pytest.mark.parametrize("q_size", [0.1, 1.5, 12.0])
@pytest.mark.parametrize("new", [1, 8])
def test_cut_sequences(new, q_size):
    """Sequences that several workgroups share, with flat and with nearly one-hot weights."""
    check(new, [700, 2500], new, 8, 2, 128, page=64, q_size=q_size)


@pytest.mark.parametrize("g", [(1e-32, 1e-32), (1e-32, 3.0), (1e-25, 1e25), (1e30, 1e-30), (1e30, 1e30)])
@pytest.mark.parametrize("dim", [64, 80, 128, 256])
def test_per_tensor_scales_far_from_one(dim, g):
    """Scores are the same whatever part of a key's size its per-tensor scale carries."""
    for element in ("fp4", "fp8"):
        check_attention(np.random.default_rng(dim), [100, 9], 4, 8, 2, dim, element, block=16, g=g)
