"""Memory of the forms that allocate."""

from __future__ import annotations


def new(like, shape, dtype, stream, returned=True):
    """An uninitialised tensor beside `like` for a call on `stream` (None: the current one).

    The caching allocator hands memory out for a stream, and takes it back once its tensor is gone, whatever
    other streams still have to do with it. So what a call on another stream writes is allocated for that
    stream; what it returns is also known to be used on the caller's, as before that stream could be named."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    import torch
    if not like.is_cuda:
        raise ValueError("tensors must be on the GPU")
    at = int(getattr(stream, "cuda_stream", stream))
    own = torch.cuda.ExternalStream(at, device=like.device) if at else torch.cuda.default_stream(like.device)
    with torch.cuda.stream(own):
        t = like.new_empty(shape, dtype=dtype)
    if returned:
        t.record_stream(torch.cuda.current_stream(like.device))
    return t
