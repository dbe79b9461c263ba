"""Shared by the GPU tests of the layer steps: the built library, element-wise
comparison against bounds, and the rounding units the bounds count."""
import numpy as np
import pytest
import torch

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# largest relative error of one rounding to the type (half a step)
UNIT = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
F32 = UNIT["f32"]


def library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_sequence_sca_b200 import build, lib
    build.build()
    lib.load()
    return lib


def host(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def within(got, want, bound, what):
    """|got - want| <= bound everywhere (and got finite where want is)."""
    got = host(got) if isinstance(got, torch.Tensor) else np.asarray(got)
    assert got.shape == want.shape, f"{what}: shape {got.shape} for {want.shape}"
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    over = np.abs(got - want) - bound
    i = np.unravel_index(np.argmax(over), over.shape)
    assert over[i] <= 0, f"{what}{i}: {got[i]!r} for {want[i]!r}, off by {abs(got[i] - want[i]):.3e}, " \
                         f"bound {np.broadcast_to(bound, over.shape)[i]:.3e}"
