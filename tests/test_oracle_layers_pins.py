"""The fp64 oracle of the loss, the embedding and the residual norm, pinned
against torch's fp64 autograd and against differences."""
import numpy as np
import pytest
import torch

from oracle import layers as ol

# fp64 on both sides: a few hundred operations of 2^-53 each
CLOSE = dict(rtol=1e-10, atol=1e-12)


def _loss_inputs(rng, L=23, d=16, V=37):
    H, W = rng.standard_normal((L, d)), rng.standard_normal((V, d))
    mask = (rng.random(L) < 0.6).astype(np.uint8)
    t = rng.integers(-3, V + 3, L).astype(np.int32)
    return H, W, mask, t, rng.random(L)


def test_loss_against_autograd():
    H, W, mask, t, w = _loss_inputs(np.random.default_rng(1))
    o = ol.loss(W, H, mask, t, w, grad=3.0)
    h, v = torch.tensor(H, requires_grad=True), torch.tensor(W, requires_grad=True)
    ok = torch.tensor((mask != 0) & (t >= 0) & (t < len(W)))
    ce = torch.nn.functional.cross_entropy((h @ v.T)[ok], torch.tensor(t[ok.numpy()]).long(), reduction="none")
    total = (ce * torch.tensor(w)[ok]).sum()
    (3.0 * total).backward()
    assert 0 < len(o["idx"]) < len(H)
    np.testing.assert_allclose(o["loss"], total.item(), **CLOSE)
    np.testing.assert_allclose(o["losses"][o["idx"]], ce.detach().numpy(), **CLOSE)
    np.testing.assert_allclose(o["d_hidden"], h.grad.numpy(), **CLOSE)
    np.testing.assert_allclose(o["d_W"], v.grad.numpy(), **CLOSE)


def test_loss_against_differences():
    rng = np.random.default_rng(2)
    H, W, mask, t, w = _loss_inputs(rng)
    o = ol.loss(W, H, mask, t, w)
    dH, dW, e = rng.standard_normal(H.shape), rng.standard_normal(W.shape), 1e-5
    up, down = (ol.loss(W + s * e * dW, H + s * e * dH, mask, t, w)["loss"] for s in (1, -1))
    # central differences: the third derivative's share is e^2, rounding 2^-53 / e
    np.testing.assert_allclose((up - down) / (2 * e), (o["d_hidden"] * dH).sum() + (o["d_W"] * dW).sum(), rtol=1e-6)


def test_loss_without_rows():
    H, W, mask, t, w = _loss_inputs(np.random.default_rng(3))
    o = ol.loss(W, H, 0 * mask, t, w)
    assert o["loss"] == 0 and not o["d_hidden"].any() and not o["d_W"].any() and not o["lse"].any()


def test_lookup_against_autograd():
    rng = np.random.default_rng(4)
    table, tok, g = rng.standard_normal((11, 8)), rng.integers(-2, 14, 50), rng.standard_normal((50, 8))
    ok = (tok >= 0) & (tok < 11)
    v = torch.tensor(table, requires_grad=True)
    out = 2.5 * v[torch.tensor(np.where(ok, tok, 0))] * torch.tensor(ok)[:, None]
    out.backward(torch.tensor(g))
    np.testing.assert_allclose(ol.lookup(table, tok, 2.5), out.detach().numpy(), **CLOSE)
    got, size = ol.lookup_grad(tok, g, 11, 2.5)
    np.testing.assert_allclose(got, v.grad.numpy(), **CLOSE)
    assert np.all(size >= np.abs(got) - 1e-12)


@pytest.mark.parametrize("update", [True, False])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("groups", [0, 1, 3, 12])
@pytest.mark.parametrize("pre", [True, False])
def test_residual_norm_against_autograd(update, post, groups, pre):
    if not update and (post or groups or not pre):
        pytest.skip("no such call")
    rng = np.random.default_rng(5)
    T, d, eps, scale = 12, 16, 1e-3, 0.7
    x, y, dn, dx = (rng.standard_normal((T, d)) for _ in range(4))
    wp, wq, gate = rng.standard_normal(d), rng.standard_normal(d), rng.standard_normal((groups or 1, d))
    t = {k: torch.tensor(v, requires_grad=True) for k, v in dict(x=x, y=y, pre=wp, post=wq, gate=gate).items()}
    norm = lambda v, w: w * v * torch.rsqrt(v.pow(2).mean(1, keepdim=True) + eps)  # noqa: E731
    u = norm(t["y"], t["post"]) if post else t["y"]
    if groups:
        u = u * torch.repeat_interleave(t["gate"], T // groups, 0)
    xo = t["x"] + scale * u if update else t["x"]
    n = norm(xo, t["pre"]) if pre else None
    total = (xo * torch.tensor(dx)).sum()
    if pre:
        total = total + (n * torch.tensor(dn)).sum()
    total.backward()
    a = (y if update else None, wp if pre else None, wq if post else None, gate if groups else None, eps, scale)
    ox, on, _ = ol.residual_norm(x, *a)
    np.testing.assert_allclose(ox, xo.detach().numpy(), **CLOSE)
    if pre:
        np.testing.assert_allclose(on, n.detach().numpy(), **CLOSE)
    got = ol.residual_norm_grad(ox, *a, dn if pre else None, dx)
    for k, there in dict(x=True, y=update, pre=pre, post=post, gate=groups > 0).items():
        assert (got[k] is not None) == there
        if there:
            np.testing.assert_allclose(got[k][0], t[k].grad.numpy(), **CLOSE)
            assert np.all(got[k][1] >= np.abs(got[k][0]) - 1e-9)
