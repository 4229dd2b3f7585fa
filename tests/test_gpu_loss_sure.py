"""Sure targets at large logits.  The target's logit and lse come from sums in different orders, so their difference is
off by several steps of the logit in either direction, where the true gradient is 0: whatever it is, the probability
stays between 0 and 1."""
import numpy as np
import pytest

from _layer_cases import HALF, dev_bf16, dev_f32, f64
from test_gpu_loss import _dev, bf16_of

pytestmark = pytest.mark.gpu

CASES = [(64, 1024, 512), (300, 1024, 512), (64, 1544, 33000), (300, 1024, 33000), (20, 4096, 33000)]


def _sure(L, d, V, top):
    """Rows along their target's entry of a positive head: (inputs, z, the most that lse - z may be off, others' gap)."""
    rng = np.random.default_rng(L + d + V)
    W, Wf = bf16_of(0.5 + rng.random((V, d), dtype=np.float32))
    t = rng.permutation(V)[:L]
    H, Hf = bf16_of(2.0 ** top / (Wf[t] ** 2).sum(axis=1, keepdims=True) * Wf[t])
    a = dict(H=H, Hf=Hf, W=W, Wf=Wf, mask=np.ones(L, np.uint8), t=t.astype(np.int32), w=np.ones(L, np.float32))
    z = (Hf * Wf[t]).sum(axis=1)
    others = Hf @ Wf.T
    others[np.arange(L), t] = -np.inf
    assert (z - others.max(axis=1)).min() > 150     # every other probability is below fp32's smallest number
    # two logits, d 2^-24 sum |h w| each in any order, their difference's rounding, and lse's own 2^-17
    return a, 2 * d * 2.0 ** -24 * z + 2.0 ** -24 * z + 2.0 ** -17


@pytest.mark.parametrize("top", [14, 20, 30])
@pytest.mark.parametrize("L,d,V", CASES)
def test_gradients_of_sure_targets(L, d, V, top):
    """dz at the target lies in [-grad, 0] and is 0 elsewhere, so each gradient is a share of one row, of one sign."""
    import torch

    import masked_token_logits_amd as mtl
    print(f"[case] sure L={L} d={d} V={V} top={top}", flush=True)
    a, off = _sure(L, d, V, top)
    x, head, grad = _dev(a), mtl.MaskedLoss(dev_bf16(a["W"])), 3.0
    args = (x["hidden"], x["mask"], x["targets"])
    lse = head(*args)[2]
    dh, dW = head.backward(*args, lse, grad=dev_f32([grad]))
    torch.cuda.synchronize()
    most = np.minimum(off, 1.0)[:, None] * grad * (1 + 2 * HALF)
    dh, dW = f64(dh), f64(dW)
    assert np.isfinite(dh).all() and np.isfinite(dW).all()
    share = dh / a["Wf"][a["t"]]
    assert (share <= 0).all() and (share >= -most).all(), (share.min(), share.max())
    share = dW[a["t"]] / a["Hf"]
    assert (share <= 0).all() and (share >= -most).all(), (share.min(), share.max())
    assert not np.delete(dW, a["t"], axis=0).any()


@pytest.mark.parametrize("top", [14, 20, 30])
@pytest.mark.parametrize("L,d,V", CASES)
def test_losses_of_sure_targets(L, d, V, top):
    """No cross entropy is below 0."""
    import torch

    import masked_token_logits_amd as mtl
    print(f"[case] sure losses L={L} d={d} V={V} top={top}", flush=True)
    a, off = _sure(L, d, V, top)
    x = _dev(a)
    loss, losses, lse = mtl.MaskedLoss(dev_bf16(a["W"]))(x["hidden"], x["mask"], x["targets"])
    torch.cuda.synchronize()
    losses, loss = f64(losses), f64(loss)[0]
    assert (losses >= 0).all() and (losses <= off).all(), (losses.min(), losses.max())
    assert abs(loss - losses.sum()) <= 2.0 ** -24 * losses.sum()


# the forward product's kernels (128 x 128 tiles whose K starts at their own stage, with and without a tail; few rows;
# persistent, K in steps of 64 and of 32; streaming), and heads of one entry and one tile
ORDERS = [(64, 1024, 512), (300, 4096, 700), (90, 1544, 2000), (40, 1000, 300), (20, 4096, 33000), (32, 1544, 33000),
          (90, 2048, 33000), (90, 2080, 33000), (64, 1544, 33000), (300, 2048, 40000)]


@pytest.mark.parametrize("top", [14, 20, 28, 30])
@pytest.mark.parametrize("L,d,V", ORDERS)
def test_target_logits_are_the_products(L, d, V, top):
    """The target's logit is summed as the product sums it, so the loss of a sure target does not see the logit's own
    rounding: it is 0 but for the sum of exponentials and its logarithm, 2^-17, and so is its gradient."""
    import torch

    import masked_token_logits_amd as mtl
    print(f"[case] order L={L} d={d} V={V} top={top}", flush=True)
    a, _ = _sure(L, d, V, top)
    x, head = _dev(a), mtl.MaskedLoss(dev_bf16(a["W"]))
    args = (x["hidden"], x["mask"], x["targets"])
    loss, losses, lse = head(*args)
    dh, dW = head.backward(*args, lse)
    torch.cuda.synchronize()
    assert (f64(losses) >= 0).all() and (f64(losses) <= 2.0 ** -17).all(), f64(losses).max()
    # z - lse, both rounded to the logit's own steps: at these sizes 0 or, where lse is a step lower, above it
    assert not dh.any() and not dW.any()


@pytest.mark.parametrize("L,d,V", ORDERS + [(1, 4096, 1), (1, 4096, 3871), (5, 2048, 462)])
def test_losses_of_almost_sure_targets(L, d, V):
    """l = ln(1 + sum of exp(z_v - z_t) over the others): the logits' errors, e each, count by 1 - p_t, and the sum of
    exponentials (2^-20 of itself, a few rescalings) and its logarithm add 2^-18."""
    import torch

    import masked_token_logits_amd as mtl
    from oracle import layers as ol
    print(f"[case] almost sure L={L} d={d} V={V}", flush=True)
    rng = np.random.default_rng(L + d + V)
    W, Wf = bf16_of(rng.standard_normal((V, d)).astype(np.float32) * 1.3 / np.sqrt(d))
    t = rng.integers(0, V, L)
    far = np.linspace(14.0, 34.0, L)[:, None]
    H, Hf = bf16_of(rng.standard_normal((L, d)) + far * Wf[t] / (Wf[t] ** 2).sum(axis=1, keepdims=True))
    a = dict(H=H, W=W, mask=np.ones(L, np.uint8), t=t.astype(np.int32), w=np.ones(L, np.float32))
    x = _dev(a)
    losses = f64(mtl.MaskedLoss(dev_bf16(W))(x["hidden"], x["mask"], x["targets"])[1])
    o = ol.loss(Wf, Hf, a["mask"], a["t"])
    e = d * 2.0 ** -24 * (np.abs(Hf) @ np.abs(Wf).T).max(axis=1)
    rest = 1.0 - o["p"][np.arange(L), t]
    err = np.abs(losses - o["losses"])
    assert (err <= 2 * e * rest + 2.0 ** -18 + 2.0 ** -23 * o["losses"]).all(), (err - 2 * e * rest).max()
