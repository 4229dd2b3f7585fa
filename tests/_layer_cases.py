"""Seeded inputs and comparisons of the loss, embedding and residual norm tests.

Tolerances count roundings.  A value rounded to bf16 is off by at most 2^-8 of
itself (half a step); fp32 arithmetic adds a few 2^-24 for each operation, of
the size of the terms that meet, which each test bounds from the oracle."""
import numpy as np

import workloads as WL
from _cache_cases import bf16, dev_bf16, dev_i32  # noqa: F401

HALF = 2.0 ** -8   # half a step of bf16, relative


def f64(t):
    """A bf16 or float32 device tensor in fp64 on the host."""
    import torch
    t = t.detach().contiguous()
    if t.dtype == torch.bfloat16:
        return WL.bf16_to_f32(t.view(torch.int16).cpu().numpy().view(np.uint16)).astype(np.float64)
    return t.cpu().numpy().astype(np.float64)


def close(got, want, tol, where):
    got = f64(got) if not isinstance(got, np.ndarray) else got
    assert got.shape == want.shape, (where, got.shape, want.shape)
    err, tol = np.abs(got - want), np.broadcast_to(tol, want.shape)
    ok = err <= tol
    assert np.all(ok), (f"{where}: {np.argwhere(~ok)[:3].tolist()} of {int((~ok).sum())}, off by up to "
                        f"{np.nanmax(np.where(ok, 0, err / np.maximum(tol, 1e-300))):.3g} tolerances")


def dev_f32(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda()


def replayed(call, outputs, refill, rounds=3):
    """Captures ``call()`` in a graph and replays it ``rounds`` times, each time
    after ``refill(i)`` wrote new inputs; between replays the same call runs
    eagerly and the device is synchronised.  ``outputs(i)`` checks a replay."""
    import torch
    refill(0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = call()
    for i in range(rounds):
        refill(i)
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        eager = call()
        torch.cuda.synchronize()
        outputs(i, got, eager)
