"""Calls that are given a stream: the tensors that they make themselves are memory of that stream, also where
the current stream is busy with the memory that it would hand out.  On the CPU by stand-ins for the library
and the allocator's stream, on the GPU by two streams at once."""
import contextlib
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import microscaling_fp4_weight_amd as mx
from microscaling_fp4_weight_amd import kv

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class Library:
    """Stands in for the library: every call succeeds and is remembered."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 256 if name.endswith("workspace_size") or name == "mx_scale_bytes" else 0
        return call


@pytest.fixture
def made(monkeypatch):
    """The streams that tensors were made on, in order; CPU tensors pass for a GPU's."""
    on, current = [], [SimpleNamespace(cuda_stream=11, device_index=0)]
    usual = current[0]

    def set_stream(s):
        current[0] = s

    def noted(make):
        def call(*args, **kw):
            on.append(None if current[0] is usual else current[0])
            kw.pop("device", None)
            return make(*args, **kw)
        return call

    library = Library()
    monkeypatch.setattr(torch.cuda, "device", contextlib.nullcontext)
    monkeypatch.setattr(torch.cuda, "set_stream", set_stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[0])
    for name in ("empty", "empty_like", "zeros"):
        monkeypatch.setattr(torch, name, noted(getattr(torch, name)))
    new_empty = torch.Tensor.new_empty
    monkeypatch.setattr(torch.Tensor, "new_empty", noted(new_empty))
    monkeypatch.setattr(kv, "_entry", lambda: library)
    monkeypatch.setattr(kv, "_on_gpu", lambda t: 0)
    monkeypatch.setattr(kv, "_same_device", lambda *a: None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: current[0].cuda_stream, raising=False)
    monkeypatch.setattr(mx, "lib", lambda: library)
    monkeypatch.setattr(mx, "_need_gpu", lambda **kw: None)
    yield SimpleNamespace(on=on, calls=library.calls)
    assert current[0] is usual


def kv_calls():
    z = torch.zeros
    cache = kv.KVCache(*(z((3, 2, 16, w), dtype=torch.uint8) for w in (32, 2, 32, 2)))
    x, i, table = z((4, 2, 64), dtype=BF16), z(4, dtype=I32), z((8, 64))
    q, pages, lens = z((2, 1, 4, 64), dtype=BF16), z((2, 3), dtype=I32), z(2, dtype=I32)
    return {"table": (1, lambda **kw: mx.mxkv_rope_table(8, 64, **kw)),
            "rope": (1, lambda **kw: mx.mxkv_rope(x, i, table, **kw)),
            "write": (0, lambda **kw: mx.mxkv_write(x, x, cache, i, **kw)),
            "read": (2, lambda **kw: mx.mxkv_read(cache, i, **kw)),
            "attention": (2, lambda **kw: mx.mxkv_attention(q, cache, pages, lens, **kw)),
            "attention and lse": (3, lambda **kw: mx.mxkv_attention(q, cache, pages, lens, return_lse=True, **kw))}


@pytest.mark.parametrize("name", list(kv_calls()))
def test_cache_calls_make_their_tensors_on_the_given_stream(made, name):
    count, call = kv_calls()[name]
    side = SimpleNamespace(cuda_stream=77, device_index=0)
    made.on.clear()
    call(stream=side)
    assert made.on == [side] * count and made.calls[-1][1][-1] == 77
    made.on.clear()
    call()
    assert made.on == [None] * count and made.calls[-1][1][-1] == 11


def weight_calls():
    z = torch.zeros
    x, codes, bytes8 = z((4, 64), dtype=BF16), z((4, 32), dtype=torch.uint8), z((4, 64), dtype=torch.uint8)
    scales = z(512, dtype=torch.uint8)
    return {"quantize": (2, lambda **kw: mx.mx_quantize(x, 32, "e8m0", **kw)),
            "quantize, tiled": (2, lambda **kw: mx.mx_quantize(x, 32, "e8m0", layout="tiled", **kw)),
            "dequantize": (1, lambda **kw: mx.mx_dequantize(codes, scales, 64, 32, "e8m0", **kw)),
            "error": (2, lambda **kw: mx.mx_quant_error(x, 32, "e8m0", **kw)),
            "statistics": (2, lambda **kw: mx.mx_tensor_stats(x, **kw)),
            "quantize to FP8": (2, lambda **kw: mx.mx_quantize_fp8(x, 32, "e8m0", **kw)),
            "dequantize from FP8": (1, lambda **kw: mx.mx_dequantize_fp8(bytes8, scales, 32, "e8m0", **kw)),
            "product with FP8": (1, lambda **kw: mx.mx_gemm_fp8(x, bytes8, scales, 32, "e8m0", **kw)),
            "product": (2, lambda **kw: mx.mx_gemm(x, codes, scales, 32, "e8m0", mode="a4", **kw)),
            "product, static scratch": (1, lambda **kw: mx.mx_gemm_static(x, codes, scales, 32, "e8m0", mode="a4", **kw))}


@pytest.mark.parametrize("name", list(weight_calls()))
def test_weight_calls_make_their_tensors_on_the_given_stream(made, name, monkeypatch):
    count, call = weight_calls()[name]
    monkeypatch.setattr(mx, "_need_bytes", lambda *a: None)  # the stand-in's sizes are no sizes
    side = SimpleNamespace(cuda_stream=77, device_index=0)
    made.on.clear()
    call(stream=side)
    assert made.on == [side] * count and made.calls[-1][1][-1] == 77
    made.on.clear()
    call()
    assert made.on == [None] * count and made.calls[-1][1][-1] == 11


def test_the_current_stream_given_is_as_none_given(made):
    for count, call in kv_calls().values():
        made.on.clear()
        call(stream=SimpleNamespace(cuda_stream=11, device_index=0))
        assert made.on == [None] * count and made.calls[-1][1][-1] == 11


def test_cache_calls_refuse_a_stream_of_another_gpu(made):
    for name, (_, call) in kv_calls().items():
        before = len(made.calls)
        with pytest.raises(ValueError, match="stream on GPU 1"):
            call(stream=SimpleNamespace(cuda_stream=77, device_index=1))
        assert all(c[0].endswith("workspace_size") for c in made.calls[before:]), name


@pytest.mark.gpu
def test_attention_on_two_streams_without_a_workspace():
    """Both calls wait behind a long kernel when they return; what the current stream allocates and fills then
    is neither their workspaces nor their results."""
    from test_gpu_kv import dev, ints, make_cache
    rng = np.random.default_rng(2)
    cache, _ = make_cache(rng, 80, 2, 32, 128, "fp4", "e8m0", 32)
    table = ints(rng.permutation(80).reshape(2, 40))
    qs, lens = [dev(rng.standard_normal((2, 4, 16, 128)), "bf16") for _ in range(2)], [ints([1000, 777]), ints([400, 1201])]
    want = [mx.mxkv_attention(q, cache, table, n, return_lse=True) for q, n in zip(qs, lens)]
    need = mx.mxkv_attention_workspace_size(cache, 2, 4, 16, 40)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for side, q, n in zip(sides, qs, lens):
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                torch.cuda._sleep(20_000_000)
            got.append(mx.mxkv_attention(q, cache, table, n, return_lse=True, stream=side))
        filled = [torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
        for side in sides:
            torch.cuda.current_stream().wait_stream(side)
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
        assert all((f == 0xFF).all() for f in filled)


@pytest.mark.gpu
def test_rotate_write_and_read_on_a_stream():
    from test_gpu_kv import dev, ints
    rng = np.random.default_rng(3)
    x, slots, pos = dev(rng.standard_normal((40, 2, 128)), "bf16"), ints(rng.permutation(48)[:40]), ints(rng.integers(0, 99, 40))
    caches = [mx.mxkv_alloc(3, 2, 16, 128) for _ in range(2)]
    side = torch.cuda.Stream()
    results = []
    for cache, stream in zip(caches, (None, side)):
        side.wait_stream(torch.cuda.current_stream())
        if stream is not None:
            with torch.cuda.stream(side):
                torch.cuda._sleep(20_000_000)
        table = mx.mxkv_rope_table(99, 128, stream=stream)
        mx.mxkv_write(x, x, cache, slots, positions=pos, table=table, stream=stream)
        results.append([table, mx.mxkv_rope(x, pos, table, stream=stream), *mx.mxkv_read(cache, slots, stream=stream)])
        filled = [torch.full_like(t, 7.0) for t in results[-1]]
    torch.cuda.current_stream().wait_stream(side)
    for a, b, f in zip(*results, filled):
        assert torch.equal(a, b) and (f == 7.0).all()


@pytest.mark.gpu
def test_weight_calls_on_a_stream():
    """The error split and the statistics (whose results are zeroed first) and a product with its workspace, behind a
    long kernel, with the current stream's memory filled meanwhile."""
    from test_gpu_kv import dev
    x = dev(np.random.default_rng(4).standard_normal((128, 512)), "bf16")
    side = torch.cuda.Stream()
    results = []
    for stream in (None, side):
        side.wait_stream(torch.cuda.current_stream())
        if stream is not None:
            with torch.cuda.stream(side):
                torch.cuda._sleep(20_000_000)
        codes, scales = mx.mx_quantize(x, 32, "e8m0", stream=stream)
        bytes8, scales8 = mx.mx_quantize_fp8(x, 32, "e8m0", stream=stream)
        results.append([codes, scales, bytes8, scales8, mx.mx_dequantize(codes, scales, 512, 32, "e8m0", stream=stream),
                        mx.mx_quant_error(x, 32, "e8m0", stream=stream), mx.mx_tensor_stats(x, stream=stream),
                        mx.mx_dequantize_fp8(bytes8, scales8, 32, "e8m0", stream=stream),
                        mx.mx_gemm(x, codes, scales, 32, "e8m0", mode="a4", stream=stream),
                        mx.mx_gemm_fp8(x, bytes8, scales8, 32, "e8m0", stream=stream)])
        filled = [torch.full_like(t, 7) for t in results[-1]]
        filled += [torch.full((mx.mx_gemm_workspace_size(128, 128, 512, 32, "a4"),), 7, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert all((f == 7).all() for f in filled)
