"""A stream that an object of this package was given, next to torch's current
one."""
from __future__ import annotations

import torch


def as_stream(stream, device):
    """torch's form of a stream; an int is a handle."""
    return stream if hasattr(stream, "synchronize") else torch.cuda.ExternalStream(stream, device)


def used_on(stream, device, *groups):
    """Tensors of ``groups`` that are freed go back to the allocator once
    ``stream`` has done what it was given until then."""
    s = as_stream(stream, device)
    for t in (t for group in groups for t in group):
        if t is not None and t.is_cuda:
            t.record_stream(s)
