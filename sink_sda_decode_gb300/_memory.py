"""Memory that a call makes for itself: results and workspaces."""
from __future__ import annotations

import torch


def empties(dev, stream, *specs, results: bool = True) -> list[torch.Tensor]:
    """torch.empty(shape, dtype) per spec, for a call whose kernels run on `stream`
    (None: the current one).

    Made on `stream`, so that blocks which are free there are given: one that was
    freed on the current stream may still be in use by work queued there, which
    `stream` does not wait for.  `results` are read on the current stream, which is
    recorded: their memory is not given away on `stream` while work that was queued
    here before they were dropped still reads it.
    """
    here = None if stream is None else torch.cuda.current_stream(dev)
    if here is None or stream.cuda_stream == here.cuda_stream:
        return [torch.empty(shape, dtype=dtype, device=dev) for shape, dtype in specs]
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=dev)
    with torch.cuda.stream(stream):
        made = [torch.empty(shape, dtype=dtype, device=dev) for shape, dtype in specs]
    if results:
        for t in made:
            t.record_stream(here)
    return made


def empty(shape, dtype, dev, stream) -> torch.Tensor:
    """One result."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    return empties(dev, stream, (shape, dtype))[0]


def workspace(nbytes: int, dev, stream) -> torch.Tensor:
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    return empties(dev, stream, (nbytes, torch.uint8), results=False)[0]
