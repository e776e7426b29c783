"""Argument marshalling shared by the bindings of the operators around the experts.

Those operators' smallest calls take a few microseconds on the GPU, so the host's part
counts: a pointer is passed as a plain int, the current stream is read as a raw handle, and
the device is switched only if it is another one.
"""

import contextlib

import torch
from torch.autograd import forward_ad

_HERE = contextlib.nullcontext()


def on_device(device):
    """A context in which ``device`` is the current one."""
    return _HERE if torch._C._cuda_getDevice() == device.index else torch.cuda.device(device)


def stream_of(device):
    """The raw handle of the device's current stream."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def ptr(t):
    """The address of a tensor, None for none or for an empty one."""
    return t.data_ptr() or None if t is not None else None


def ready(t, dtype=None):
    """The tensor in ``dtype``, contiguous and starting on 16 bytes: itself where it is so already."""
    if dtype is not None and t.dtype != dtype:
        t = t.to(dtype)
    if not t.is_contiguous():
        return t.contiguous()
    return t.clone() if t.data_ptr() & 15 else t


def refuse_gradients(why, *tensors):
    """ValueError if a gradient of one of the tensors would be asked for (None: no tensor)."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise ValueError(why)


def check_tensor(name, t, dtypes, dims, device=None):
    """Type, device, dtype and number of dimensions; ``device``: the one it has to be on.  A tangent of forward-mode
    differentiation, which needs no requires_grad and would be lost, is refused."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if forward_ad._current_level >= 0 and forward_ad.unpack_dual(t).tangent is not None:
        raise ValueError("%s has a forward-mode tangent: this operator has no forward-mode derivative" % name)
    if not t.is_cuda:
        raise ValueError("%s must be on a HIP device (got %s)" % (name, t.device))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, not on %s" % (name, t.device, device))
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s (got %s)" % (name, " or ".join(str(d) for d in dtypes), t.dtype))
    if t.dim() not in dims:
        raise ValueError("%s must have %s dimensions (got %s)" % (name, " or ".join(map(str, dims)), tuple(t.shape)))
