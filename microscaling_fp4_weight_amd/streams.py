"""Tensors that a call makes itself when it is given a stream."""
from __future__ import annotations

import torch


def made_on(stream, make, *args, **kw) -> torch.Tensor:
    """make(*args, **kw), a new tensor, in memory of `stream` (None: the current one), on which the call's
    kernels run.  Memory of the current stream could still be in use there, or be given to others there as
    soon as the call returns, while the kernels are still to run.  The current stream is recorded as a user:
    a result that is dropped is not given to others before that stream's work on it is done."""
    if stream is None or stream.cuda_stream == torch._C._cuda_getCurrentRawStream(stream.device_index):
        return make(*args, **kw)
    current = torch.cuda.current_stream(stream.device_index)
    with torch.cuda.device(stream.device_index):
        torch.cuda.set_stream(stream)  # as torch.cuda.stream does, in less of the host's time
        try:
            t = make(*args, **kw)
        finally:
            torch.cuda.set_stream(current)
    if t.is_cuda:
        t.record_stream(current)
    return t
