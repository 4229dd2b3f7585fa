"""NaN and infinity in places that count: a row whose logits hold a NaN has a NaN log-sum-exp, loss and gradient, one
with an infinite logit and no NaN an infinite log-sum-exp, on every path of the forward product; other rows keep their
bits.  And the readout's statistics of logits from 2^29 on, which it takes from the same sums."""
import numpy as np
import pytest

from _layer_cases import bf16, close, dev_bf16, f64
from oracle import layers as ol
from test_gpu_loss import _check_forward, _dev, _inputs, bf16_of

pytestmark = pytest.mark.gpu

# the forward product's kernels: 128 x 128 tiles; few rows; persistent, K in steps of 64 and of 32; streaming (K odd)
PATHS = {"small": (90, 64, 700), "few": (20, 64, 33000), "persistent": (90, 64, 33000), "narrow": (90, 96, 33000),
         "streaming": (90, 72, 33000), "many": (600, 64, 33000)}


def _run(a, W=None, H=None):
    import torch

    import masked_token_logits_amd as mtl
    x = _dev(a)
    if H is not None:
        x["hidden"] = H
    head = mtl.MaskedLoss(dev_bf16(a["W"]) if W is None else W)
    args = (x["hidden"], x["mask"], x["targets"])
    got = head(*args, weights=x["weights"])
    back = head.backward(*args, got[2], weights=x["weights"])
    torch.cuda.synchronize()
    return got, back


@pytest.mark.parametrize("path", PATHS)
def test_hidden_rows(path):
    """A NaN or infinite hidden state makes its own row's results so, and all of d_W."""
    import torch
    L, d, V = PATHS[path]
    print(f"[case] hidden rows {path}", flush=True)
    a = _inputs(np.random.default_rng(L + d), L, d, V, 1.0, strays=False)
    want, want_back = _run(a)
    H = dev_bf16(a["H"])
    nan, one, inf = 3, 11, 17
    H[nan], H[one, 5], H[inf, 7] = float("nan"), float("nan"), float("inf")
    got, (dh, dW) = _run(a, H=H)
    rows = np.arange(L)
    bad = np.isin(rows, (nan, one, inf))
    for k, name in ((1, "losses"), (2, "lse")):
        g = f64(got[k])
        assert np.isnan(g[[nan, one]]).all(), (name, g[[nan, one]])
        assert np.array_equal(g[~bad], f64(want[k])[~bad]), name
    assert np.isposinf(f64(got[2])[inf]) and not np.isfinite(f64(got[1])[inf])      # logits of both signs
    assert np.isnan(f64(got[0])[0])
    assert torch.isnan(dh[bad]).all() and torch.equal(dh[~bad], want_back[0][~bad])
    assert torch.isnan(dW).all()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("first,count", [(0, 64), (0, 1), (64, 64), (128, 256), (-64, 64), (-1, 1), (-1, -1)])
def test_head_rows(path, first, count):
    """NaN entries of the head, from one to a tile of them (and the whole head), reach every row that counts: none is
    left out because all that a lane sees of a tile is NaN."""
    import torch
    L, d, V = PATHS[path]
    print(f"[case] head rows {path} {first} {count}", flush=True)
    a = _inputs(np.random.default_rng(L + d + 1), L, d, V, 0.7)
    W = dev_bf16(a["W"])
    if count < 0:
        W[:] = float("nan")
    else:
        W[first: first + count if first + count else None] = float("nan")
    got, (dh, dW) = _run(a, W=W)
    counts = np.isin(np.arange(L), ol.counted(a["mask"], a["t"], V))
    for k, name in ((1, "losses"), (2, "lse")):
        assert np.array_equal(np.isnan(f64(got[k])), counts), name
        assert not f64(got[k])[~counts].any(), name
    assert np.isnan(f64(got[0])[0])
    assert torch.isnan(dh[counts]).all() and not dh[~counts].any()
    assert torch.isnan(dW).all()


@pytest.mark.parametrize("path", PATHS)
def test_head_rows_of_infinity(path):
    """An entry whose logits are -inf everywhere adds nothing to lse; one of +inf makes lse infinite."""
    L, d, V = PATHS[path]
    print(f"[case] infinite entries {path}", flush=True)
    a = _inputs(np.random.default_rng(L + d + 2), L, d, V, 1.0, strays=False, lean=0.0)
    a["H"], Hf = bf16_of(np.abs(a["Hf"]) + 0.25)
    low, high = [0, 1, 65, V - 1], V // 2
    a["t"][:] = 2
    W = dev_bf16(a["W"])
    W[low] = float("-inf")
    got, (dh, dW) = _run(a, W=W)
    rest = np.setdiff1d(np.arange(V), low)
    b = dict(a, Hf=Hf, Wf=a["Wf"][rest], t=np.full_like(a["t"], int(np.searchsorted(rest, 2))))
    _check_forward(got, b, ol.loss(b["Wf"], Hf, a["mask"], b["t"], a["w"]))
    W[high] = float("inf")
    lse = f64(_run(a, W=W)[0][2])
    assert np.isposinf(lse).all(), lse


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("top", [28, 29, 30, 60, 110])
def test_nan_among_large_logits(path, top):
    """Logits of 2^top: lse is their largest; with a NaN among them it is NaN."""
    L, d, V = PATHS[path]
    print(f"[case] large {path} {top}", flush=True)
    rng = np.random.default_rng(L + top)
    sign = np.where(rng.random((L, 1)) < 0.5, 1.0, -1.0)
    H, Hf = bf16_of(np.where(np.arange(d) == 0, sign * 2.0 ** top, 0.0))
    W, Wf = bf16_of(np.where(np.arange(d) == 0, rng.integers(64, 129, (V, 1)) / 128.0, 1.0))
    a = dict(H=H, Hf=Hf, W=W, Wf=Wf, mask=np.ones(L, np.uint8), t=rng.integers(0, V, L).astype(np.int32),
             w=(np.ones(L) / L).astype(np.float32))
    got, (dh, dW) = _run(a)
    o = ol.loss(Wf, Hf, a["mask"], a["t"], a["w"])
    # exact logits, and lse and the difference rounded to half a step of the largest (and by 2^-17 below 2^29)
    e = 2.0 ** -17 + 2.0 ** -24 * np.abs(o["lse"])
    close(got[2], o["lse"], e, "lse")
    close(got[1], o["losses"], e + 2.0 ** -24 * np.abs(o["losses"]), "losses")
    assert np.isfinite(f64(dh)).all() and np.isfinite(f64(dW)).all()
    Wn = dev_bf16(W)
    Wn[V // 3] = float("nan")
    got = _run(a, W=Wn)[0]
    assert np.isnan(f64(got[2])).all() and np.isnan(f64(got[0])[0])


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("top", [27, 29])
def test_readout_of_large_logits(path, top):
    """The readout's confidence and log-sum-exp where the largest logit, 2^top, occurs three times."""
    import torch

    import masked_token_logits_amd as mtl
    L, d, V = PATHS[path]
    print(f"[case] readout large {path} {top}", flush=True)
    rng = np.random.default_rng(top)
    H = bf16_of(np.where(np.arange(d) == 0, 2.0 ** top, 0.0) * np.ones((L, 1)))[0]
    w = rng.integers(64, 128, V) / 128.0
    at = [V // 5, V // 2, V - 1]
    w[at] = 1.0
    W = dev_bf16(bf16_of(np.where(np.arange(d) == 0, w[:, None], 1.0))[0])
    rd = mtl.MaskedReadout(W, L, 4)
    out = rd.outputs()
    rd.step(dev_bf16(H), torch.ones(L, dtype=torch.uint8, device="cuda"), torch.zeros(L, dtype=torch.int32, device="cuda"),
            0, out=out)
    torch.cuda.synchronize()
    assert int(out["m_out"].item()) == L
    assert (out["row_tok"][:L].cpu().numpy() == at[0]).all()
    # base-2 exponentials and their sums, within 2^-20 of themselves
    close(f64(out["row_conf"])[:L], np.full(L, 1 / 3), 2.0 ** -20, "conf")
    want = 2.0 ** top + np.log(3.0)
    close(f64(out["row_lse"])[:L], np.full(L, want), 2.0 ** -17 + 2.0 ** -24 * want, "lse")


def test_readout_keeps_nan():
    """A NaN entry of the head makes every row's confidence NaN, wherever it stands."""
    import torch

    import masked_token_logits_amd as mtl
    for path, (L, d, V) in PATHS.items():
        for first, last in ((0, 64), (V - 1, V)):
            print(f"[case] readout nan {path} {first}", flush=True)
            a = _inputs(np.random.default_rng(9), L, d, V, 1.0, strays=False)
            W = dev_bf16(a["W"])
            W[first:last] = float("nan")
            rd = mtl.MaskedReadout(W, L, 4)
            out = rd.outputs()
            rd.step(dev_bf16(a["H"]), torch.ones(L, dtype=torch.uint8, device="cuda"),
                    torch.zeros(L, dtype=torch.int32, device="cuda"), 0, out=out)
            torch.cuda.synchronize()
            assert int(out["m_out"].item()) == L
            assert torch.isnan(out["row_conf"][:L]).all() and torch.isnan(out["row_lse"][:L]).all(), path
