"""One rounding of float64 values to float32 or bf16, for the tests."""
import numpy as np


def to_bf16(v):
    """float64 values rounded once to bf16 (ties to even, subnormals too, overflow to infinity), as float64."""
    v = np.asarray(v, np.float64)
    m, e = np.frexp(np.where(np.isfinite(v), v, 0.0))
    step = np.ldexp(1.0, np.maximum(e - 8, -133))
    r = np.rint(np.where(np.isfinite(v), v, 0.0) / step) * step
    r = np.where(np.abs(r) >= 2.0 ** 128, np.copysign(np.inf, r), r)
    return np.where(np.isfinite(v), r, v)


def to_f32(v):
    with np.errstate(over="ignore", under="ignore"):
        return np.asarray(v, np.float64).astype(np.float32).astype(np.float64)
