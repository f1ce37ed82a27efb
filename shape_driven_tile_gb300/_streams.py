"""Outputs that a call allocates for itself, on the stream that writes them."""
from __future__ import annotations

import torch


def handle(stream) -> int:
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def empty(shape, dtype, device, stream=None):
    """An uninitialised output of a call on `stream` (None: the current one).

    The caching allocator orders a block's users by the stream that it was allocated on.  A block
    of the current stream may still be read there by work that was queued earlier, and is handed
    out again there while another stream writes it; so the block comes from `stream`, and is noted
    as used on the current stream, where the caller (who lets it wait for `stream`) reads it.
    """
    if stream is not None:
        here, to = torch.cuda.current_stream(device), handle(stream)
        if to != here.cuda_stream:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(to, device=device) if to else torch.cuda.default_stream(device)
            with torch.cuda.stream(stream):
                t = torch.empty(shape, dtype=dtype, device=device)
            t.record_stream(here)
            return t
    return torch.empty(shape, dtype=dtype, device=device)
