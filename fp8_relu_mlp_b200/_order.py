"""Order between torch's current stream and a stream that an object of this
package was given: its buffers are filled, and its inputs written, on the
current stream."""
from __future__ import annotations

import torch


def as_stream(stream, device):
    """torch's form of a stream; an int is a handle, another object has one."""
    if hasattr(stream, "wait_stream"):
        return stream
    return torch.cuda.ExternalStream(getattr(stream, "cuda_stream", stream), device)


def after_current(stream, device):
    """What is launched on ``stream`` from here on waits for the current
    stream's work so far (by an event: the host does not wait, and both
    streams may be in a graph capture)."""
    s, current = as_stream(stream, device), torch.cuda.current_stream(device)
    if s.cuda_stream != current.cuda_stream:
        s.wait_stream(current)


def current_after(stream, device):
    """What comes next on the current stream waits for ``stream``'s work so far."""
    s, current = as_stream(stream, device), torch.cuda.current_stream(device)
    if s.cuda_stream != current.cuda_stream:
        current.wait_stream(s)


def used_on(stream, device, *groups):
    """Tensors of ``groups`` that are freed go back to the allocator once
    ``stream`` has done what it was given until then."""
    s = as_stream(stream, device)
    for t in (t for group in groups for t in group):
        if t is not None and t.is_cuda:
            t.record_stream(s)
