"""Helpers of the sequence operators' GPU tests: outputs between canary bands,
strided placements, conversions."""
import numpy as np
import torch

import depthwise_convolution_forward_gb300 as gc
from depthwise_convolution_forward_gb300 import inputs

DEV = torch.device("cuda:0")
GUARD = 4096  # bytes of canary on each side of an output


class Guarded:
    """An uninitialised (0xFF: NaN in every float type) output of `shape`
    between two canary bands.  `stride` places it as a strided tensor inside its
    buffer; the elements between its rows are canaries too."""

    def __init__(self, shape, dtype, stride=None, offset=0):
        self.shape = tuple(shape)
        es = torch.empty(0, dtype=dtype).element_size()
        if stride is None:
            stride = torch.empty(self.shape, device="meta").stride()
        n = sum((s - 1) * st for s, st in zip(self.shape, stride)) + 1 if all(self.shape) else 0
        g = GUARD // es
        self.buf = torch.full(((n + offset + 2 * g) * es,), 0xFF, dtype=torch.uint8, device=DEV)
        self.t = self.buf.view(dtype)[g + offset:].as_strided(self.shape, stride)

    def check(self):
        """The bytes outside the output are untouched; returns the output."""
        torch.cuda.synchronize()
        keep = self.t.clone()
        self.t.view(torch.uint8 if self.t.element_size() == 1 else
                    torch.int16 if self.t.element_size() == 2 else torch.int32).fill_(-1 if self.t.element_size() > 1 else 255)
        assert bool((self.buf == 0xFF).all()), "wrote outside the output"
        self.t.copy_(keep)
        return keep


def host(t):
    return None if t is None else t.detach().cpu().double().numpy()


def f64(*ts):
    return [host(t) for t in ts]


def code(dtype):
    return gc.DTYPE_CODES[dtype]


def randn(g, *shape, dtype="f32", std=1.0):
    return (torch.randn(shape, generator=g) * std).to(inputs.DTYPES[dtype]).to(DEV)


def place(t, stride, offset=0):
    """A copy of t with the given strides inside a buffer of NaNs."""
    n = sum((s - 1) * st for s, st in zip(t.shape, stride)) + 1
    buf = torch.full((n + offset,), float("nan"), dtype=t.dtype, device=t.device)
    v = buf[offset:].as_strided(t.shape, stride)
    v.copy_(t)
    return v


def same_bits(a, b):
    return bool(torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)))


def as_array(lens):
    return None if lens is None else np.asarray(lens)
