"""The loss's kernels by their number of rows and tiles, and what is given back of dz's rounding at the targets.

Which kernel takes a product goes by the counted rows M on the device (256 are few, 257 are not) and by its tiles of
256 x 256; every case states its M.  Tolerances: those of test_gpu_loss, and for the targets' part the ones derived at
test_targets_are_given_back."""
import numpy as np
import pytest

from _layer_cases import HALF, bf16, close, dev_bf16, dev_f32, f64
from oracle import layers as ol
from test_gpu_loss import _check_backward, _check_forward, _dev, _errors, _inputs, bf16_of

pytestmark = pytest.mark.gpu


CASES = [  # L, d, V, accumulate
    (256, 128, 33000, False),   # the most few rows, and one more, against a large head
    (257, 128, 33000, False),
    (257, 136, 33000, True),
    (256, 136, 33000, True),
    (600, 128, 33000, False),   # several row tiles of dz and of d_W, K whole and with a tail
    (600, 136, 33000, False),
    (513, 264, 33000, True),
    (256, 64, 700, False),      # the same number of rows against a small head
    (257, 64, 700, False),
    (600, 39048, 300, False),   # 3 x 153 tiles of d_hidden, more than cuts: whole ones start late and wrap around
    (8456, 2056, 300, False),   # 34 x 9 of them, in two groups of row tiles
    (8456, 264, 1300, False),   # 34 row tiles of dz
]


@pytest.mark.parametrize("L,d,V,accumulate", CASES)
def test_rows_and_tiles(L, d, V, accumulate):
    import torch

    import masked_token_logits_amd as mtl
    rng = np.random.default_rng(L + d + V)
    print(f"[case] paths L={L} d={d} V={V} accumulate={accumulate}", flush=True)
    a = _inputs(rng, L, d, V, 1.0, strays=False)
    x, head, grad = _dev(a), mtl.MaskedLoss(dev_bf16(a["W"])), dev_f32([2.5])
    args = (x["hidden"], x["mask"], x["targets"])
    got = head(*args, weights=x["weights"])
    old, of = bf16(rng, (V, d), 0.01) if accumulate else (None, None)
    call = lambda: head.backward(*args, got[2], weights=x["weights"], grad=grad, accumulate=accumulate,  # noqa: E731
                                 d_W=dev_bf16(old) if accumulate else None)
    dh, dW = call()
    again = call()
    torch.cuda.synchronize()
    assert torch.equal(dh, again[0]) and torch.equal(dW, again[1])
    o = ol.loss(a["Wf"], a["Hf"], a["mask"], a["t"], a["w"], 2.5)
    assert len(o["idx"]) == L
    _check_forward(got, a, o)
    _check_backward(dh, dW, a, o, 2.5, old=of)


def _half_ulp(x):
    """Half the distance of neighbouring bf16 values around x."""
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126))) - 8)


@pytest.mark.parametrize("L,d,V,accumulate", [
    (100, 256, 2000, False), (100, 256, 2000, True), (256, 136, 2311, False),     # small heads, by pieces
    (102, 256, 33000, False), (102, 264, 33000, True), (256, 128, 33000, True),   # large heads
    (300, 256, 2000, False), (300, 128, 33000, False),                            # many rows: d_hidden alone
])
def test_targets_are_given_back(L, d, V, accumulate):
    """Rows without hope (p almost 0 at the target, a target each), and a gradient of the loss halfway between two bf16
    numbers but for 2 percent: dz's rounding at the target is 2^-8 of it, where the result's own is at most half its
    step.  So the targets' terms get fp32 tolerances, (terms + 3) 2^-24 of them (their products, their sums and dz
    itself), and the others those of test_gpu_loss.  In an emulation on the CPU the values come to 0.98 tolerances; without
    what is given back 39 percent of d_W's rows and more lie outside (of d_hidden 0.1 to 8), with its sign turned 81 (15
    to 41)."""
    import torch

    import masked_token_logits_amd as mtl
    rng = np.random.default_rng(L + d + V)
    print(f"[case] targets L={L} d={d} V={V} accumulate={accumulate}", flush=True)
    grad = float(np.float32(1 + 0.98 * 2.0 ** -8))
    a = _inputs(rng, L, d, V, 1.0, strays=False)
    a["t"] = rng.permutation(V)[:L].astype(np.int32)
    Wt = a["Wf"][a["t"]]
    a["H"], a["Hf"] = bf16_of(a["Hf"] * 0.1 - 30.0 * Wt / (Wt ** 2).sum(axis=1, keepdims=True))
    a["weighted"] = False
    x = _dev(a)
    head = mtl.MaskedLoss(dev_bf16(a["W"]), piece=512 if V < 4096 else 16384)
    args = (x["hidden"], x["mask"], x["targets"])
    lse = head(*args)[2]
    old, of = bf16(rng, (V, d), 2.0 ** -9) if accumulate else (None, np.zeros((V, d)))
    dh, dW = head.backward(*args, lse, grad=dev_f32([grad]), accumulate=accumulate, d_W=dev_bf16(old) if accumulate else None)
    torch.cuda.synchronize()
    o = ol.loss(a["Wf"], a["Hf"], a["mask"], a["t"], None, grad)
    rows, t, W, H = np.arange(L), a["t"], a["Wf"], a["Hf"]
    assert len(o["idx"]) == L and o["p"][rows, t].max() < 2.0 ** -24
    off = (grad * (2 * _errors(a, o) + 2.0 ** -16))[:, None] * o["p"]
    rest = o["dz"].copy()
    rest[rows, t] = 0.0
    fp32 = (V + 3) * 2.0 ** -24 * (np.abs(o["dz"]) @ np.abs(W))
    tol = _half_ulp(o["d_hidden"]) * (1 + 2.0 ** -6) + 6.5 * HALF * np.sqrt(rest ** 2 @ W ** 2) + off @ np.abs(W) + fp32
    close(dh, o["d_hidden"], tol, "d_hidden")
    if L <= 256:
        want = (o["d_W"] + of)[t]
        fp32 = (L + 3) * 2.0 ** -24 * (np.abs(o["dz"]).T @ np.abs(H))[t]
        tol = (_half_ulp(want) * (1 + 2.0 ** -6) + 6.5 * HALF * np.sqrt((rest ** 2).T @ H ** 2)[t]
               + (off.T @ np.abs(H))[t] + fp32)
        close(f64(dW)[t], want, tol, "d_W")
