"""Helpers of the operator tests: seeded inputs on the GPU, comparison against
the fp64 oracle with an elementwise bound."""
import numpy as np
import torch

U = 2.0 ** -24            # half a step of fp32, relative
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
HALF = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}     # half a step, relative
TINY = {"fp32": 1e-37, "bf16": 1e-37, "fp16": 2.0 ** -24}              # and among the smallest values


def dev(x, dtype="fp32"):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to("cuda", DT[dtype])


def host(t):
    return t.double().cpu().numpy()


def within(got, want, bound, dtype="fp32", label=""):
    """|got - want| <= bound + the rounding of the result to dtype, element by element."""
    got = host(got)
    room = bound + HALF[dtype] * (np.abs(want) + bound) + TINY[dtype]
    off = np.abs(got - want)
    assert np.isfinite(got).all(), label
    worst = (off / room).max() if off.size else 0.0
    print(f"[bound] {label}: {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0, f"{label}: {worst:.3f} times the bound"


def cu_tensor(cu):
    return None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
