"""GPU parity of the rotary positions against the fp64 oracle.

Tolerance: the angle's fraction of a turn is rounded to fp32 once (at most
2^-25 of a turn, 2^-22.3 rad), cos and sin are fp32 to a few ulp and the
rotation is two products and a sum, so before the output's rounding a value
is within 2^-20 of its pair's length; the rounding to bf16 adds at most
2^-8 of the value (half a step)."""
import numpy as np
import pytest

import workloads as WL
from _cache_cases import bf16, dev_bf16, dev_i32
from oracle import cache as oc

pytestmark = pytest.mark.gpu


def _close(got, want, size, where):
    err = np.abs(got - want)
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * size
    assert np.all(err <= tol), f"{where}: {np.argwhere(err > tol)[:3].tolist()} off by up to {np.max(err / np.maximum(tol, 1e-300)):.3g} tolerances"


def _f64(t):
    import torch
    return WL.bf16_to_f32(t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)).astype(np.float64)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,H,D,r", [
    (1, 1, 64, 64),       # one token, one head
    (37, 3, 128, 128),
    (5, 28, 128, 64),     # half of the head
    (5, 4, 128, 6),       # a few pairs: the element path
    (70, 2, 256, 256),
    (9, 3, 50, 22),       # a head size without any alignment
    (3, 2, 7, 6),         # odd head size: the last dimension is copied
    (2500, 2, 64, 32),    # many tokens
])
def test_rotary_parity(T, H, D, r, layout):
    import torch

    import masked_token_logits_amd as mtl
    rng = np.random.default_rng(T * 1000 + H * 100 + D + r)
    print(f"[case] rotary T={T} H={H} D={D} r={r} {layout}", flush=True)
    x, xf = bf16(rng, (T, H, D))
    pos = rng.integers(0, 131072, T)
    rot = mtl.Rotary(D, r, layout=layout)
    got = rot(dev_bf16(x), dev_i32(pos))
    torch.cuda.synchronize()
    want, size = oc.rotate(xf, pos, oc.rotary_theta(r), layout)
    _close(_f64(got), want, size, "rotated")
    assert np.array_equal(_f64(got)[..., r:], xf[..., r:])


@pytest.mark.parametrize("scaling,kw", [("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
                                        ("ramp", dict(factor=16.0, original_len=4096, fast=32.0, slow=1.0))])
def test_rotary_scalings(scaling, kw):
    import torch

    import masked_token_logits_amd as mtl
    rng = np.random.default_rng(7)
    T, H, D = 33, 2, 128
    x, xf = bf16(rng, (T, H, D))
    pos = rng.integers(0, 1 << 20, T)
    rot = mtl.Rotary(D, scaling=scaling, **kw)
    got = rot(dev_bf16(x), dev_i32(pos))
    torch.cuda.synchronize()
    mag = 0.1 * np.log(kw["factor"]) + 1.0 if scaling == "ramp" else 1.0
    want, size = oc.rotate(xf, pos, oc.rotary_theta(D, scaling=scaling, **kw), "half", mag)
    _close(_f64(got), want, size, scaling)


def test_rotary_far_and_negative_positions():
    """Angles of positions up to the int32 limits keep their fraction: fp64
    holds position * turns to 2^-22 of a turn there."""
    import torch

    import masked_token_logits_amd as mtl
    rng = np.random.default_rng(8)
    pos = np.array([0, -1, 2 ** 24 + 1, -(2 ** 24) - 3, 10 ** 9 + 7, 2 ** 31 - 1, -2 ** 31])
    x, xf = bf16(rng, (len(pos), 2, 64))
    rot = mtl.Rotary(64)
    got = rot(dev_bf16(x), dev_i32(pos))
    torch.cuda.synchronize()
    want, size = oc.rotate(xf, pos, oc.rotary_theta(64), "half")
    # the host's pow and the device's share theta to 2^-52 relative: 2^31 radians of angle move by 2^-20
    err = np.abs(_f64(got) - want)
    assert np.all(err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * size)


@pytest.mark.parametrize("layout,r", [("half", 64), ("interleaved", 64), ("half", 20)])
def test_rotary_in_place_strided_and_broadcast(layout, r):
    """A slice of a fused projection in place, [H, T, D] outputs, an expanded
    input, and a base address of odd alignment give what contiguous tensors give, bit for
    bit, and nothing around them is written."""
    import torch

    import masked_token_logits_amd as mtl
    rng = np.random.default_rng(9)
    T, H, D = 21, 3, 64
    x, _ = bf16(rng, (T, 3 * H, D))
    pos = dev_i32(rng.integers(0, 9000, T))
    rot = mtl.Rotary(D, r, layout=layout)
    fused = dev_bf16(x)
    ref = rot(fused[:, H:2 * H].contiguous(), pos)
    before = fused.clone()
    out = rot(fused[:, H:2 * H], pos, out=fused[:, H:2 * H])
    assert out.data_ptr() == fused[:, H:2 * H].data_ptr()
    assert torch.equal(out, ref)
    assert torch.equal(fused[:, :H], before[:, :H]) and torch.equal(fused[:, 2 * H:], before[:, 2 * H:])
    turned = torch.zeros((H, T, D), dtype=torch.bfloat16, device="cuda")
    rot(before[:, H:2 * H], pos, out=turned.transpose(0, 1))
    assert torch.equal(turned.transpose(0, 1), ref)
    one = before[:, H:H + 1].expand(T, H, D)
    assert torch.equal(rot(one, pos), rot(one.contiguous(), pos))
    flat = torch.zeros(T * H * D + 1, dtype=torch.bfloat16, device="cuda")
    off = flat[1:].view(T, H, D)
    off.copy_(before[:, H:2 * H])
    assert torch.equal(rot(off, pos), ref)


def test_rotary_transpose_is_the_gradient():
    """<y', R x> = <R^T y', x> up to roundings, R^T R = m^2, and the oracle's
    transposed rotation; differences: R is linear, so R(x + e) - R(x) = R e."""
    import torch

    import masked_token_logits_amd as mtl
    rng = np.random.default_rng(10)
    T, H, D, r = 40, 3, 128, 96
    pos = rng.integers(0, 100000, T)
    x, xf = bf16(rng, (T, H, D))
    g, gf = bf16(rng, (T, H, D))
    rot = mtl.Rotary(D, r, magnitude=1.25)
    gx = rot(dev_bf16(g), dev_i32(pos), transpose=True)
    y = rot(dev_bf16(x), dev_i32(pos))
    torch.cuda.synchronize()
    want, size = oc.rotate(gf, pos, oc.rotary_theta(r), "half", 1.25, transpose=True)
    _close(_f64(gx), want, size, "transposed")
    # both sides carry one bf16 rounding of each term: 2^-8 relative, independent, six deviations
    lhs, rhs = np.sum(gf * _f64(y)), np.sum(_f64(gx) * xf)
    dev = 6 * 2.0 ** -8 * np.sqrt(np.sum((gf * _f64(y)) ** 2) + np.sum((_f64(gx) * xf) ** 2))
    assert abs(lhs - rhs) <= dev
    # the derivative along e by differences of the oracle, against the kernel's
    e = rng.standard_normal(xf.shape)
    theta = oc.rotary_theta(r)
    num = np.sum(gf * (oc.rotate(xf + e, pos, theta, "half", 1.25)[0] - oc.rotate(xf - e, pos, theta, "half", 1.25)[0])) / 2
    assert abs(num - np.sum(_f64(gx) * e)) <= 6 * 2.0 ** -8 * np.sqrt(np.sum((_f64(gx) * e) ** 2))


def test_rotary_nan_and_inf_stay_in_their_pair():
    import torch

    import masked_token_logits_amd as mtl
    x = torch.ones((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    x[0, 1, 3] = float("nan")
    x[1, 0, 5] = float("inf")
    y = mtl.Rotary(64)(x, dev_i32([3, 4])).float().cpu()
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[0, 1, [3, 35]] = True
    want[1, 0, [5, 37]] = True
    assert torch.equal(bad, want)


def test_rotary_no_tokens():
    import torch

    import masked_token_logits_amd as mtl
    x = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    assert mtl.Rotary(64)(x, dev_i32([])).shape == (0, 2, 64)


@pytest.mark.parametrize("T,H,D,r", [(5, 1, 64, 32), (9, 3, 128, 128), (3, 40, 64, 64), (17, 2, 512, 512), (2, 5, 256, 48),
                                     (11, 7, 72, 16), (6, 3, 72, 70), (4, 5, 64, 2), (3, 33, 128, 50)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_alignment_changes_nothing(T, H, D, r, layout):
    """Aligned heads go in 16-byte pieces, several tokens to a workgroup where heads are few; the same values
    one element off go one by one, to the same bits."""
    import torch

    import masked_token_logits_amd as mtl
    g = torch.Generator(device="cuda").manual_seed(T + D)
    rot = mtl.Rotary(D, r, layout=layout)
    x = torch.randn(T, H, D, generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.randint(-1000, 200000, (T,), generator=g, device="cuda", dtype=torch.int32)
    off = torch.empty(T * H * D + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, H, D)
    off.copy_(x)
    for transpose in (False, True):
        y = rot(x, pos, transpose=transpose)
        z = rot(off, pos, out=torch.empty(T * H * D + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, H, D),
                transpose=transpose)
        assert torch.equal(y, z)
        inplace = x.clone()
        assert rot(inplace, pos, out=inplace, transpose=transpose) is inplace and torch.equal(inplace, y)


@pytest.mark.parametrize("T,H,D,r", [(9, 1, 8, 8), (300, 1, 16, 16), (5, 8, 8, 4), (3, 33, 16, 16), (70, 3, 16, 2),
                                     (1, 300, 8, 8), (11, 2, 24, 16), (4, 5, 24, 24)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_small_heads(T, H, D, r, layout):
    """Heads of one 16-byte unit, of one piece of two and of a piece and a half, one head and several tokens to a
    workgroup: the oracle's values both ways, the element path's bits, and nothing written around the output."""
    import torch

    import masked_token_logits_amd as mtl
    rng = np.random.default_rng(T * 1000 + H * 100 + D + r)
    print(f"[case] rotary small T={T} H={H} D={D} r={r} {layout}", flush=True)
    x, xf = bf16(rng, (T, H, D))
    pos = rng.integers(-1000, 131072, T)
    rot = mtl.Rotary(D, r, layout=layout)
    n = T * H * D
    tx, tp = dev_bf16(x), dev_i32(pos)
    off = torch.zeros(n + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, H, D)
    off.copy_(tx)
    for transpose in (False, True):
        flat = torch.full((n + 128,), 7.0, dtype=torch.bfloat16, device="cuda")
        y = rot(tx, tp, out=flat[64:64 + n].view(T, H, D), transpose=transpose)
        torch.cuda.synchronize()
        want, size = oc.rotate(xf, pos, oc.rotary_theta(r), layout, transpose=transpose)
        _close(_f64(y), want, size, "small heads")
        assert np.array_equal(_f64(y)[..., r:], xf[..., r:])
        assert torch.all(flat[:64] == 7) and torch.all(flat[64 + n:] == 7)
        z = torch.empty(n + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, H, D)
        assert torch.equal(rot(off, tp, out=z, transpose=transpose), y)
        inplace = tx.clone()
        assert torch.equal(rot(inplace, tp, out=inplace, transpose=transpose), y)
