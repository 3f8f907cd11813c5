"""Helpers of the GPU tests of the operators around the scan: seeded arrays in
either type, upload, and elementwise bars.

A bar is u |ref| + c 2^-24 mag: u is half a step of the output's type (2^-8
bfloat16; float32's is inside c), mag the sum of the magnitudes of the terms
that the value is made of, c the number of float32 roundings on the longest
path to it.  Each test derives its c beside its call."""
import numpy as np
import torch

import _gpu
from selective_state_space_09_amd import inputs

U = {"bf16": 2.0 ** -8, "f32": 0.0}
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E = 2.0 ** -24


def normal(rng, shape, t="f32", mul=1.0, add=0.0):
    a = (rng.standard_normal(shape, dtype=np.float32) * np.float32(mul) + np.float32(add)).astype(np.float32)
    return inputs.f32_to_bf16_bits(a) if t == "bf16" else a


def wide(a):
    return None if a is None else (inputs.bf16_bits_to_f32(a) if a.dtype == np.uint16 else a).astype(np.float64)


def within(got, ref, t, c, mag, what):
    got = _gpu.to_host64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    err = np.abs(got - ref)
    lim = U[t] * np.abs(ref) + c * E * np.broadcast_to(mag, ref.shape) + 1e-38
    bad = np.argwhere(~(err <= lim))
    if len(bad):
        i = tuple(bad[0])
        raise AssertionError(f"{what}: {len(bad)} of {ref.size} outside the bar, first at {i}: got {got[i]}, "
                             f"ref {ref[i]}, error {err[i]:.3g}, bar {lim[i]:.3g}")


def rows_in(a, ld, col, fill=0):
    """The rows of a as columns col.. of wider device rows (`fill` elsewhere):
    (the view, the whole buffer)."""
    t = _gpu.to_dev(a)
    buf = torch.full(tuple(t.shape[:-1]) + (ld,), fill, dtype=t.dtype, device="cuda")
    view = buf[..., col:col + t.shape[-1]]
    view.copy_(t)
    return view, buf
