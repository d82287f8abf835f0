"""Whose memory the tensors are that a call makes.

torch's allocator keeps its free blocks by stream: a block is handed out again
on the stream it was asked for, whose own order keeps earlier and later users
apart, and on no other.  A call that launches on a stream of the caller's
choice therefore asks for its outputs and workspaces on that stream: taken
from the current one, a block could still be read by work queued there, or be
handed out there again while the launch is pending.
"""

from __future__ import annotations


def as_torch_stream(stream):
    """A stream argument (a torch stream, an object with a cuda_stream, or a
    raw handle) as a torch stream of the current device."""
    import torch

    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = stream if isinstance(stream, int) else int(stream.cuda_stream)
    # (ExternalStream makes a new stream of handle 0)
    return torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()


def empty_on(stream):
    """torch.empty whose tensors belong to the stream."""
    import torch

    owner = as_torch_stream(stream)

    def empty(*size, **kw):
        with torch.cuda.stream(owner):
            return torch.empty(*size, **kw)

    return empty
