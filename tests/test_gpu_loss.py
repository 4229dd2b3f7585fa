"""GPU parity of the masked cross entropy and its gradients against the fp64 oracle.

Tolerances.  A logit is an fp32 sum of d exact products: off by at most
d 2^-24 sum |h w| =: e (any order).  lse is off by the largest e of its row, and
by 2^-17: base-2 exponentials and the sums of them are within 2^-20 of
themselves, rescaled a few times, and the final logarithm of a number of a few
units adds 2^-21 of |lse| <= 64.  With those, dz is off by coef p (2 e + 2^-16)
and by its rounding to bf16, at most 2^-8 of itself.  These roundings are
independent of each other and centred, so by Hoeffding's inequality a sum of
terms r_k with |r_k| <= 2^-8 |a_k| stays within 6.5 * 2^-8 sqrt(sum a_k^2) but
for one in 10^9 values; the rest adds up in the worst case.  The fp32 sums of
the two gradient products add (terms) 2^-24 of the terms' absolute sum, and the
output half a step of bf16."""
import numpy as np
import pytest

from _layer_cases import HALF, bf16, close, dev_bf16, dev_f32, dev_i32, f64, replayed
from oracle import layers as ol

pytestmark = pytest.mark.gpu


def _inputs(rng, L, d, V, ratio, strays=True, lean=8.0):
    H, Hf = bf16(rng, (L, d))
    W, Wf = bf16(rng, (V, d), 1.3 / np.sqrt(d))
    t = rng.integers(0, V, L)
    H, Hf = bf16_of(Hf + lean * rng.random((L, 1)) * Wf[t] / (Wf[t] ** 2).sum(axis=1, keepdims=True))
    if strays and L > 4:
        at = rng.integers(0, L, max(L // 16, 2))
        t[at] = rng.choice([-100, -1, V, 2 ** 31 - 1], len(at))
    mask = (rng.random(L) < ratio).astype(np.uint8) * rng.integers(1, 256, L).astype(np.uint8)
    w = (rng.random(L) + 0.1).astype(np.float32) / L
    return dict(H=H, W=W, mask=mask, t=t.astype(np.int32), w=w, Hf=Hf, Wf=Wf)


def bf16_of(x):
    import workloads as WL
    b = WL.bf16_round(x.astype(np.float32))
    return b, WL.bf16_to_f32(b).astype(np.float64)


def _dev(a):
    import torch
    return dict(hidden=dev_bf16(a["H"]), mask=torch.from_numpy(a["mask"].copy()).cuda(), targets=dev_i32(a["t"]),
                weights=dev_f32(a["w"]))


def _errors(a, o):
    """e of every counted row's largest logit error, and of dz, without its rounding."""
    d = a["Hf"].shape[1]
    e = d * 2.0 ** -24 * (np.abs(a["Hf"][o["idx"]]) @ np.abs(a["Wf"]).T).max(axis=1, initial=0.0)
    return e


def _check_forward(got, a, o):
    loss, losses, lse = got
    e = np.zeros(len(a["t"]))
    e[o["idx"]] = _errors(a, o) + 2.0 ** -17
    close(lse, o["lse"], e, "lse")
    close(losses, o["losses"], 2 * e, "losses")
    w = a["w"].astype(np.float64) if a.get("weighted", True) else np.ones(len(e))
    size = (w * (np.abs(o["losses"]) * 2.0 ** -23 + 2 * e)).sum()
    close(loss, np.array([o["loss"]]), size + 2.0 ** -24 * abs(o["loss"]), "loss")


def _check_backward(d_hidden, d_W, a, o, grad=1.0, old=None):
    H, W, idx, dz = a["Hf"][o["idx"]], a["Wf"], o["idx"], o["dz"]
    w = a["w"].astype(np.float64)[idx] if a.get("weighted", True) else np.ones(len(idx))
    off = (abs(grad) * w * (2 * _errors(a, o) + 2.0 ** -16))[:, None] * o["p"]
    step = 6.5 * HALF
    if d_hidden is not None:
        tol = np.zeros_like(a["Hf"])
        tol[idx] = (HALF * np.abs(o["d_hidden"][idx]) + step * np.sqrt((dz ** 2) @ (W ** 2)) + off @ np.abs(W)
                    + len(W) * 2.0 ** -24 * (np.abs(dz) @ np.abs(W)))
        close(d_hidden, o["d_hidden"], tol, "d_hidden")
    if d_W is not None:
        want = o["d_W"] + (old if old is not None else 0.0)
        tol = (HALF * np.abs(want) + step * np.sqrt((dz ** 2).T @ (H ** 2)) + off.T @ np.abs(H)
               + (len(idx) + 1) * 2.0 ** -24 * (np.abs(dz).T @ np.abs(H) + (np.abs(old) if old is not None else 0.0)))
        close(d_W, want, tol, "d_W")


CASES = [  # L, d, V, ratio, piece
    (1, 8, 1, 1.0, None),           # one position, one token: p = 1
    (1, 64, 300, 1.0, 256),
    (5, 8, 3, 1.0, None),           # fewer entries than any tile
    (40, 72, 257, 0.5, 256),        # d a multiple of 8 only, a piece of one entry
    (33, 96, 700, 0.9, 256),        # d a multiple of 32 only
    (100, 128, 1000, 0.5, 512),
    (300, 256, 4096, 0.5, None),
    (257, 64, 513, 1.0, 256),       # one row and one entry over a tile
    (512, 320, 2311, 1.0, 1024),    # odd vocabulary, all masked
    (700, 200, 777, 0.7, 256),
    (1100, 64, 300, 0.02, None),    # few rows of many positions
    (130, 1024, 640, 1.0, None),
    (32, 72, 70001, 0.9, 8192),     # the readout's few rows
    (7, 128, 140000, 1.0, None),
    (40, 72, 70001, 0.9, 8192),     # few rows of a large head
    (600, 128, 65537, 0.3, 16384),  # two tiles of them
    (260, 64, 66000, 1.0, None),    # just over few
    (257, 136, 900, 1.0, 256),      # few and over with a d that is no multiple of 32
    (300, 40, 500, 0.7, None),
    (60, 1544, 5000, 1.0, None),    # one row tile, seven column tiles whose cuts do not line up
    (20, 66056, 300, 1.0, None),    # more column tiles than compute units
    (200, 784, 34000, 0.5, 16384),  # one row tile against a large head, four column tiles in three pieces
]


@pytest.mark.parametrize("L,d,V,ratio,piece", CASES)
def test_parity(L, d, V, ratio, piece):
    import torch

    import masked_token_logits_amd as mtl
    rng = np.random.default_rng(L + d + V)
    print(f"[case] loss L={L} d={d} V={V} ratio={ratio} piece={piece}", flush=True)
    a = _inputs(rng, L, d, V, ratio)
    x, grad = _dev(a), dev_f32([2.5])
    head = mtl.MaskedLoss(dev_bf16(a["W"]), piece=piece)
    got = head(x["hidden"], x["mask"], x["targets"], weights=x["weights"])
    torch.cuda.synchronize()
    o = ol.loss(a["Wf"], a["Hf"], a["mask"], a["t"], a["w"], 2.5)
    _check_forward(got, a, o)
    dh, dW = head.backward(x["hidden"], x["mask"], x["targets"], got[2], weights=x["weights"], grad=grad)
    torch.cuda.synchronize()
    _check_backward(dh, dW, a, o, 2.5)
    again = head.backward(x["hidden"], x["mask"], x["targets"], got[2], weights=x["weights"], grad=grad)
    assert torch.equal(dh, again[0]) and torch.equal(dW, again[1])
    assert all(torch.equal(p, q) for p, q in zip(got, head(x["hidden"], x["mask"], x["targets"], weights=x["weights"])))


def test_without_weights_and_with_a_bool_mask():
    import torch

    import masked_token_logits_amd as mtl
    a = _inputs(np.random.default_rng(2), 90, 128, 500, 0.5)
    a["weighted"] = False
    x, head = _dev(a), mtl.MaskedLoss(dev_bf16(a["W"]))
    got = head(x["hidden"], x["mask"] != 0, x["targets"])
    dh, dW = head.backward(x["hidden"], x["mask"] != 0, x["targets"], got[2])
    torch.cuda.synchronize()
    o = ol.loss(a["Wf"], a["Hf"], a["mask"], a["t"])
    _check_forward(got, a, o)
    _check_backward(dh, dW, a, o)


@pytest.mark.parametrize("what", ["mask", "targets", "weights"])
def test_nothing_to_learn(what):
    """No masked position, no target, or no weight: zero gradients, and outputs that are written."""
    import torch

    import masked_token_logits_amd as mtl
    a = _inputs(np.random.default_rng(3), 200, 64, 700, 0.5, strays=False)
    x, head = _dev(a), mtl.MaskedLoss(dev_bf16(a["W"]), piece=256)
    x[what].fill_({"mask": 0, "targets": -100, "weights": 0.0}[what])
    out = [torch.full((n,), 9.0, device="cuda") for n in (1, 200, 200)]
    loss, losses, lse = head(x["hidden"], x["mask"], x["targets"], weights=x["weights"], out=out)
    assert loss is out[0] and lse is out[2]
    dh = torch.full((200, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    dW = torch.full((700, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    head.backward(x["hidden"], x["mask"], x["targets"], lse, weights=x["weights"], d_hidden=dh, d_W=dW)
    assert loss.item() == 0 and not dh.any() and not dW.any()
    if what != "weights":
        assert not losses.any() and not lse.any()
    dW.fill_(9.0)
    head.backward(x["hidden"], x["mask"], x["targets"], lse, weights=x["weights"], d_W=dW, accumulate=True)
    assert (dW == 9).all()


def test_either_gradient_and_accumulation():
    import torch

    import masked_token_logits_amd as mtl
    rng = np.random.default_rng(4)
    a = _inputs(rng, 150, 192, 900, 0.6)
    x, head = _dev(a), mtl.MaskedLoss(dev_bf16(a["W"]), piece=512)
    args = (x["hidden"], x["mask"], x["targets"])
    lse = head(*args, weights=x["weights"])[2]
    dh, dW = head.backward(*args, lse, weights=x["weights"])
    h2, w2 = head.backward(*args, lse, weights=x["weights"], need=("hidden",))
    h3, w3 = head.backward(*args, lse, weights=x["weights"], need=("W",))
    assert w2 is None and h3 is None and torch.equal(h2, dh) and torch.equal(w3, dW)
    old, of = bf16(rng, (900, 192), 0.01)
    _, w4 = head.backward(*args, lse, weights=x["weights"], d_W=dev_bf16(old), accumulate=True)
    _check_backward(None, w4, a, ol.loss(a["Wf"], a["Hf"], a["mask"], a["t"], a["w"]), old=of)


@pytest.mark.parametrize("L,d,V", [(700, 192, 900), (420, 136, 34000), (40, 264, 33300)])
def test_accumulation(L, d, V):
    """Many and few rows, small and large heads: added once, rounded once."""
    import masked_token_logits_amd as mtl
    rng = np.random.default_rng(L)
    a = _inputs(rng, L, d, V, 0.8)
    x, head = _dev(a), mtl.MaskedLoss(dev_bf16(a["W"]))
    args = (x["hidden"], x["mask"], x["targets"])
    lse = head(*args, weights=x["weights"])[2]
    old, of = bf16(rng, (V, d), 0.01)
    dh, dW = head.backward(*args, lse, weights=x["weights"], d_W=dev_bf16(old), accumulate=True)
    _check_backward(dh, dW, a, ol.loss(a["Wf"], a["Hf"], a["mask"], a["t"], a["w"]), old=of)


def test_sure_and_hopeless_rows():
    """Logits tens apart: probabilities of 1 and of almost 0 at the target."""
    import torch

    import masked_token_logits_amd as mtl
    rng = np.random.default_rng(5)
    a = _inputs(rng, 64, 256, 400, 1.0, strays=False)
    Hf = a["Hf"].copy()
    for i in range(64):
        w = a["Wf"][a["t"][i]]
        Hf[i] = Hf[i] * 0.1 + (60.0 if i % 2 else -60.0) * w / (w ** 2).sum()
    a["H"], a["Hf"] = bf16_of(Hf)
    x, head = _dev(a), mtl.MaskedLoss(dev_bf16(a["W"]))
    got = head(x["hidden"], x["mask"], x["targets"], weights=x["weights"])
    dh, dW = head.backward(x["hidden"], x["mask"], x["targets"], got[2], weights=x["weights"])
    torch.cuda.synchronize()
    o = ol.loss(a["Wf"], a["Hf"], a["mask"], a["t"], a["w"])
    _check_forward(got, a, o)
    _check_backward(dh, dW, a, o)


@pytest.mark.parametrize("top", [10, 20, 40])
def test_large_logits(top):
    """Logits of up to 2^top that fp32 holds exactly, one hidden value and one weight each, and apart by
    at least 2^-7 of that: no probability passes 1."""
    import torch

    import masked_token_logits_amd as mtl
    L, d, V = 300, 64, 128
    i, v, k = np.arange(L)[:, None], np.arange(V)[:, None], np.arange(d)[None, :]
    Hf = np.where(i % d == k, 2.0 ** (top - i % 4) * np.where(i % 8 < 4, 1.0, -1.0), 0.0)
    H, Hf = bf16_of(Hf)
    W, Wf = bf16_of((1.0 + (v * 37 + k * 11) % V) / V)
    t = ((np.arange(L) * 13) % V).astype(np.int32)
    best = (Hf @ Wf.T).argmax(axis=1)
    t[::3] = best[::3]
    a = dict(H=H, Hf=Hf, W=W, Wf=Wf, mask=np.ones(L, np.uint8), t=t, w=(np.ones(L) / L).astype(np.float32))
    x, head = _dev(a), mtl.MaskedLoss(dev_bf16(a["W"]))
    got = head(x["hidden"], x["mask"], x["targets"], weights=x["weights"])
    dh, dW = head.backward(x["hidden"], x["mask"], x["targets"], got[2], weights=x["weights"])
    torch.cuda.synchronize()
    o = ol.loss(a["Wf"], a["Hf"], a["mask"], a["t"], a["w"])
    # the logits are exact; lse and the difference round to half a step of the largest, and lse is within 2^-17 besides
    e = 2.0 ** -17 + 2.0 ** -24 * np.abs(o["lse"])
    close(got[2], o["lse"], e, "lse")
    close(got[1], o["losses"], e + 2.0 ** -24 * np.abs(o["losses"]), "losses")
    # a probability below 1 that counts is of logits up to 2^10 alone, where e is below 2^-13
    off = np.where(o["p"] < 1 - 2.0 ** -20, np.minimum(e, 2.0 ** -13)[:, None] * 2, 2.0 ** -16) * o["p"] / L
    # fp32 and bf16 have no normal numbers below 2^-126: a probability, dz, a product, a sum or an output there may
    # be zero instead, each off by less than that (this was left out at first: gradients of e-38 came out as 0)
    step = HALF * np.abs(o["dz"]) + 2 * 2.0 ** -126
    tol_h = (V + 2) * 2.0 ** -126 + (step + off) @ np.abs(a["Wf"]) + HALF * np.abs(o["d_hidden"]) + V * 2.0 ** -24 * (np.abs(o["dz"]) @ np.abs(a["Wf"]))
    close(dh, o["d_hidden"], tol_h, "d_hidden")
    tol_w = (L + 2) * 2.0 ** -126 + (step + off).T @ np.abs(Hf) + HALF * np.abs(o["d_W"]) + L * 2.0 ** -24 * (np.abs(o["dz"]).T @ np.abs(Hf))
    close(dW, o["d_W"], tol_w, "d_W")


def test_values_that_do_not_count_are_not_read_into_results():
    """NaN hidden states, weights and lse at positions that do not count change nothing."""
    import torch

    import masked_token_logits_amd as mtl
    a = _inputs(np.random.default_rng(6), 300, 128, 600, 0.5)
    x, head = _dev(a), mtl.MaskedLoss(dev_bf16(a["W"]), piece=256)
    args = (x["hidden"], x["mask"], x["targets"])
    got = head(*args, weights=x["weights"])
    want = head.backward(*args, got[2], weights=x["weights"])
    idle = torch.from_numpy(np.setdiff1d(np.arange(300), ol.counted(a["mask"], a["t"], 600))).cuda()
    x["hidden"][idle], x["weights"][idle] = float("nan"), float("nan")
    again = head(*args, weights=x["weights"])
    assert all(torch.equal(p, q) for p, q in zip(got, again))
    again[2][idle] = float("nan")
    back = head.backward(*args, again[2], weights=x["weights"])
    assert torch.equal(want[0], back[0]) and torch.equal(want[1], back[1])


def test_gradient_against_differences():
    """The loss's directional derivative by the oracle's forward pass."""
    import masked_token_logits_amd as mtl
    rng = np.random.default_rng(7)
    a = _inputs(rng, 60, 64, 300, 0.7)
    x, head = _dev(a), mtl.MaskedLoss(dev_bf16(a["W"]))
    args = (x["hidden"], x["mask"], x["targets"])
    dh, dW = head.backward(*args, head(*args, weights=x["weights"])[2], weights=x["weights"])
    toH, toW, e = rng.standard_normal(a["Hf"].shape), rng.standard_normal(a["Wf"].shape), 1e-5
    up, down = (ol.loss(a["Wf"] + s * toW, a["Hf"] + s * toH, a["mask"], a["t"], a["w"])["loss"] for s in (e, -e))
    terms = np.concatenate([(f64(dh) * toH).ravel(), (f64(dW) * toW).ravel()])
    # two roundings to bf16 of each term's parts, one of the operand and one of the gradient
    assert abs(terms.sum() - (up - down) / (2 * e)) <= 2 * HALF * np.abs(terms).sum() + 1e-6


def test_readout_and_loss_agree():
    """The readout's log-sum-exp of the same rows."""
    import torch

    import masked_token_logits_amd as mtl
    a = _inputs(np.random.default_rng(8), 200, 256, 2000, 0.5, strays=False)
    x, W = _dev(a), dev_bf16(a["W"])
    lse = mtl.MaskedLoss(W)(x["hidden"], x["mask"], x["targets"])[2]
    rd = mtl.MaskedReadout(W, 200, 4)
    out = rd.outputs()
    rd.step(x["hidden"], x["mask"].clone(), torch.zeros(200, dtype=torch.int32, device="cuda"), 0, out=out)
    M = int(out["m_out"].item())
    # the same GEMM; slices may be cut elsewhere
    np.testing.assert_allclose(f64(lse)[f64(out["row_idx"])[:M].astype(int)], f64(out["row_lse"])[:M], atol=2.0 ** -17)


def test_captured_and_replayed():
    import torch

    import masked_token_logits_amd as mtl
    sets = [_inputs(np.random.default_rng(60 + i), 260, 128, 900, r) for i, r in enumerate((0.5, 0.0, 1.0))]
    devs = [_dev(s) for s in sets]
    buf = {k: v.clone() for k, v in devs[0].items()}
    W = dev_bf16(sets[0]["W"])
    head = mtl.MaskedLoss(W, piece=256)

    def refill(i):
        for k, v in devs[i].items():
            buf[k].copy_(v)
        W.copy_(dev_bf16(sets[i]["W"]))

    def call():
        args = (buf["hidden"], buf["mask"], buf["targets"])
        got = head(*args, weights=buf["weights"])
        return list(got) + list(head.backward(*args, got[2], weights=buf["weights"]))

    def check(i, got, eager):
        assert all(torch.equal(p, q) for p, q in zip(got, eager))
        o = ol.loss(sets[i]["Wf"], sets[i]["Hf"], sets[i]["mask"], sets[i]["t"], sets[i]["w"])
        _check_forward(got[:3], sets[i], o)
        _check_backward(got[3], got[4], sets[i], o)

    replayed(call, check, refill)


def test_streams():
    import torch

    import masked_token_logits_amd as mtl
    sets = [_inputs(np.random.default_rng(70 + i), 300, 128, 1500, 0.5) for i in range(2)]
    devs, heads = [_dev(s) for s in sets], []
    Ws = [dev_bf16(s["W"]) for s in sets]
    torch.cuda.synchronize()
    heads = [mtl.MaskedLoss(W, piece=512, stream=torch.cuda.Stream()) for W in Ws]
    for _ in range(3):
        out = []
        for h, x in zip(heads, devs):
            args = (x["hidden"], x["mask"], x["targets"])
            got = h(*args, weights=x["weights"])
            out.append((got, h.backward(*args, got[2], weights=x["weights"])))
    torch.cuda.synchronize()
    for (got, back), a in zip(out, sets):
        o = ol.loss(a["Wf"], a["Hf"], a["mask"], a["t"], a["w"])
        _check_forward(got, a, o)
        _check_backward(*back, a, o)
