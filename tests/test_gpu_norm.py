"""GPU parity of the residual update and norms against the fp64 oracle.

Tolerances.  A row's mean of squares is an fp32 sum of at most 8192 squares,
16 in a row in each thread and then a tree of at most 9 + 3 levels, so it is
within 2^-19 of itself, its root within 2^-20; the products behind it are a few
2^-24.  So before the output's rounding x' is within 2^-18 of the size of its
terms, n within 2^-17 of pre / rms times that size (x' enters twice), and the
gradients within 2^-16 of the size of theirs, which the oracle gives with every
sum of terms taken of their absolute values.  Sums over T tokens add T / 1024
fp32 additions in a row and two levels of at most 256 behind: below 2^-15 for
the T here.  A bf16 output adds half a step, 2^-8 of itself."""
import numpy as np
import pytest

from _layer_cases import HALF, bf16, close, dev_bf16, f64, replayed
from oracle import layers as ol

pytestmark = pytest.mark.gpu

X, N, G, S = 2.0 ** -18, 2.0 ** -17, 2.0 ** -16, 2.0 ** -15


def _inputs(rng, T, d, pre, post, groups, size=1.0):
    a = {}
    a["x"] = bf16(rng, (T, d), 4 * size)
    a["y"] = bf16(rng, (T, d), size)
    a["pre"] = bf16(rng, (d,)) if pre else None
    a["post"] = bf16(rng, (d,)) if post else None
    a["gate"] = bf16(rng, (groups, d)) if groups else None
    a["d_n"] = bf16(rng, (T, d)) if pre else None
    a["d_x"] = bf16(rng, (T, d))
    dev = {k: None if v is None else dev_bf16(v[0]) for k, v in a.items()}
    return dev, {k: None if v is None else v[1] for k, v in a.items()}


def _layer(dev, eps, scale, **kw):
    import masked_token_logits_amd as mtl
    d = dev["x"].shape[1]
    return mtl.ResidualNorm(pre=dev["pre"], post=dev["post"], eps=eps, scale=scale, d=d, device="cuda", **kw)


def _check_forward(got, h, eps, scale, update=True):
    x, n = got
    ox, on, size = ol.residual_norm(h["x"], h["y"] if update else None, h["pre"], h["post"], h["gate"], eps, scale)
    assert (x is not None) == update and (n is not None) == (h["pre"] is not None)
    if update:
        close(x, ox, HALF * np.abs(ox) + X * size, "x'")
    if n is not None:
        close(n, on, HALF * np.abs(on) + N * np.abs(h["pre"]) * size / ol.rms(ox, eps), "n")


def _check_backward(got, h, eps, scale, update=True, d_x=True):
    want = ol.residual_norm_grad(h["x"], h["y"] if update else None, h["pre"], h["post"], h["gate"], eps, scale, h["d_n"],
                                 h["d_x"] if d_x else None)
    for k, w in want.items():
        g = got["d_" + k]
        assert (g is not None) == (w is not None), k
        if w is not None:
            close(g, w[0], (HALF * np.abs(w[0]) + G * w[1]) if k in "xy" else (S + G) * w[1], "d_" + k)


CASES = [  # T, d, pre, post, groups
    (1, 8, 1, 0, 0),          # one token, one piece
    (1, 4096, 1, 1, 1),
    (3, 64, 1, 1, 1),
    (37, 1024, 1, 1, 37),     # a gate for every token
    (5, 1032, 1, 0, 5),       # just over a workgroup's width
    (64, 3584, 1, 1, 4),
    (2, 8192, 1, 1, 2),       # the widest
    (9, 8184, 0, 1, 3),
    (1500, 256, 1, 1, 1500),  # more gate rows than workgroups of the sums
    (2600, 72, 1, 1, 1300),
    (4099, 520, 1, 0, 0),     # several tokens to a workgroup, the last with fewer
    (2100, 2056, 0, 0, 7),    # no norm at all
    (3000, 128, 1, 1, 0),
]


@pytest.mark.parametrize("T,d,pre,post,groups", CASES)
def test_parity(T, d, pre, post, groups):
    import torch
    rng = np.random.default_rng(T * 7 + d)
    eps, scale = 1e-5, 0.75
    dev, h = _inputs(rng, T, d, pre, post, groups)
    print(f"[case] norm T={T} d={d} pre={pre} post={post} groups={groups}", flush=True)
    layer = _layer(dev, eps, scale)
    got = layer(dev["x"], dev["y"], gate=dev["gate"])
    torch.cuda.synchronize()
    _check_forward(got, h, eps, scale)
    back = layer.backward(dev["x"], dev["d_n"], y=dev["y"], d_x=dev["d_x"], gate=dev["gate"])
    torch.cuda.synchronize()
    _check_backward(back, h, eps, scale)
    again = layer.backward(dev["x"], dev["d_n"], y=dev["y"], d_x=dev["d_x"], gate=dev["gate"])
    for k, v in back.items():       # no result depends on timing
        assert v is None or torch.equal(v, again[k]), k


@pytest.mark.parametrize("T,d", [(1, 64), (33, 4096), (1200, 320)])
def test_norm_alone(T, d):
    import torch
    dev, h = _inputs(np.random.default_rng(T + d), T, d, 1, 0, 0)
    layer = _layer(dev, 1e-6, 1.0)
    got = layer(dev["x"])
    back = layer.backward(dev["x"], dev["d_n"])
    torch.cuda.synchronize()
    _check_forward(got, h, 1e-6, 1.0, update=False)
    _check_backward(back, h, 1e-6, 1.0, update=False, d_x=False)


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** -12, 2.0 ** 40])
def test_sizes_of_values(size):
    """Squares from far below fp32's smallest to far above ordinary values."""
    import torch
    eps = 1e-5
    dev, h = _inputs(np.random.default_rng(11), 21, 512, 1, 1, 3, size)
    layer = _layer(dev, eps, 1.0)
    got = layer(dev["x"], dev["y"], gate=dev["gate"])
    back = layer.backward(dev["x"], dev["d_n"], y=dev["y"], d_x=dev["d_x"], gate=dev["gate"])
    torch.cuda.synchronize()
    _check_forward(got, h, eps, 1.0)
    _check_backward(back, h, eps, 1.0)


def test_rows_of_zeros_infinities_and_nan_stay_rows():
    """A row's values reach its own outputs and the sums over tokens only."""
    import torch
    eps = 1e-5
    dev, h = _inputs(np.random.default_rng(12), 8, 256, 1, 1, 0)
    h["x"][3], h["y"][3] = 0.0, 0.0
    dev["x"][3], dev["y"][3] = 0.0, 0.0
    dev["x"][5, 7], dev["y"][6, 9] = float("inf"), float("nan")
    layer = _layer(dev, eps, 1.0)
    x, n = layer(dev["x"], dev["y"])
    back = layer.backward(dev["x"], dev["d_n"], y=dev["y"], d_x=dev["d_x"])
    torch.cuda.synchronize()
    ox, on, size = ol.residual_norm(h["x"], h["y"], h["pre"], h["post"], None, eps, 1.0)
    fine = [0, 1, 2, 3, 4, 7]
    close(f64(x)[fine], ox[fine], HALF * np.abs(ox[fine]) + X * size[fine], "x'")
    close(f64(n)[fine], on[fine], (HALF * np.abs(on) + N * np.abs(h["pre"]) * size / ol.rms(ox, eps))[fine], "n")
    assert f64(x)[3].max() == 0 and f64(n)[3].max() == 0 and np.isnan(f64(n)[6]).all()
    want = ol.residual_norm_grad(h["x"], h["y"], h["pre"], h["post"], None, eps, 1.0, h["d_n"], h["d_x"])
    for k in "xy":
        close(f64(back["d_" + k])[fine], want[k][0][fine], (HALF * np.abs(want[k][0]) + G * want[k][1])[fine], "d_" + k)


def test_in_place():
    import torch
    eps = 1e-5
    dev, h = _inputs(np.random.default_rng(13), 300, 640, 1, 1, 3)
    layer = _layer(dev, eps, 0.5)
    x, n = layer(dev["x"], dev["y"], gate=dev["gate"])
    kept = dev["x"].clone()
    x2, n2 = layer(kept, dev["y"], gate=dev["gate"], x_out=kept)
    assert x2 is kept and torch.equal(x, x2) and torch.equal(n, n2)
    back = layer.backward(dev["x"], dev["d_n"], y=dev["y"], d_x=dev["d_x"], gate=dev["gate"])
    for over in ("d_x", "d_n"):
        a = {k: dev[k].clone() for k in ("d_x", "d_n", "y")}
        b = layer.backward(dev["x"], a["d_n"], y=a["y"], d_x=a["d_x"], gate=dev["gate"], d_x_out=a[over], d_y_out=a["y"])
        assert b["d_x"] is a[over] and b["d_y"] is a["y"]
        for k, v in back.items():
            assert torch.equal(v, b[k]), (over, k)


def test_no_tokens():
    import torch
    dev, _ = _inputs(np.random.default_rng(14), 1, 64, 1, 1, 1)
    layer = _layer(dev, 1e-5, 1.0)
    none = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    x, n = layer(none, none, gate=dev["gate"])
    assert x.shape == n.shape == (0, 64)
    back = layer.backward(none, none, y=none, gate=dev["gate"])
    assert not back["d_pre"].any() and not back["d_post"].any() and not back["d_gate"].any()


def test_gradient_against_differences():
    """The directional derivative of sum(n d_n) + sum(x' d_x) by the oracle's own
    forward pass; the gradients are bf16, so half a step of each term."""
    rng = np.random.default_rng(15)
    eps, scale, e = 1e-5, 0.5, 1e-6
    dev, h = _inputs(rng, 16, 128, 1, 1, 4)
    layer = _layer(dev, eps, scale)
    y, pre, post, gate = h["y"], h["pre"], h["post"], h["gate"]
    base = h["x"] - (ol.residual_norm(0 * h["x"], y, None, post, gate, eps, scale)[0])
    got = {k: f64(v) for k, v in layer.backward(dev["x"], dev["d_n"], y=dev["y"], d_x=dev["d_x"], gate=dev["gate"]).items()}
    to = {k: rng.standard_normal(v.shape) for k, v in dict(x=base, y=y, pre=pre, post=post, gate=gate).items()}

    def value(s):
        x, n, _ = ol.residual_norm(base + s * to["x"], y + s * to["y"], pre + s * to["pre"], post + s * to["post"],
                                   gate + s * to["gate"], eps, scale)
        return (n * h["d_n"]).sum() + (x * h["d_x"]).sum()

    slope, terms = (value(e) - value(-e)) / (2 * e), {k: got["d_" + k] * v for k, v in to.items()}
    tol = sum((HALF if k in "xy" else S) * np.abs(v).sum() for k, v in terms.items()) + 1e-6 * abs(slope)
    assert abs(sum(v.sum() for v in terms.values()) - slope) <= tol


def test_captured_and_replayed():
    import torch
    eps, scale = 1e-5, 0.5
    sets = [_inputs(np.random.default_rng(20 + i), 1100, 384, 1, 1, 2) for i in range(3)]
    buf = {k: v.clone() for k, v in sets[0][0].items()}
    layer = _layer(buf, eps, scale)

    def refill(i):
        for k, v in sets[i][0].items():
            buf[k].copy_(v)

    def call():
        x, n = layer(buf["x"], buf["y"], gate=buf["gate"])
        g = layer.backward(buf["x"], buf["d_n"], y=buf["y"], d_x=buf["d_x"], gate=buf["gate"])
        return [x, n] + [g[k] for k in sorted(g)]

    def check(i, got, eager):
        for a, b in zip(got, eager):
            assert torch.equal(a, b)
        _check_forward(got[:2], sets[i][1], eps, scale)

    replayed(call, check, refill)


def test_streams():
    """An object's own stream, and two streams at once."""
    import torch
    eps = 1e-5
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = [_inputs(np.random.default_rng(30 + i), 900, 512, 1, 1, 3) for i in range(2)]
    torch.cuda.synchronize()
    layers = [_layer(dev, eps, 1.0, stream=s) for (dev, _), s in zip(sets, streams)]
    got = []
    for _ in range(4):
        got = [(la(dev["x"], dev["y"], gate=dev["gate"]),
                la.backward(dev["x"], dev["d_n"], y=dev["y"], d_x=dev["d_x"], gate=dev["gate"])) for la, (dev, _) in zip(layers, sets)]
    torch.cuda.synchronize()
    for (f, b), (_, h) in zip(got, sets):
        _check_forward(f, h, eps, 1.0)
        _check_backward(b, h, eps, 1.0)


@pytest.mark.parametrize("pre,groups", [(0, 0), (1, 0), (0, 3), (1, 3), (1, 600)])
@pytest.mark.parametrize("d", [64, 2056])
def test_y_reaches_no_gradient_of_its_own_without_a_norm(d, pre, groups):
    """Without a norm behind the block d_y = scale gate d_x: an infinite or NaN y changes nothing but its gate's gradient."""
    import torch
    dev, _ = _inputs(np.random.default_rng(d + groups), 600, d, pre, 0, groups)
    layer = _layer(dev, 1e-5, 0.5)
    want = layer.backward(dev["x"], dev["d_n"], y=dev["y"], d_x=dev["d_x"], gate=dev["gate"])
    dev["y"][3, 7], dev["y"][5], dev["y"][8, 0] = float("nan"), float("inf"), float("-inf")
    got = layer.backward(dev["x"], dev["d_n"], y=dev["y"], d_x=dev["d_x"], gate=dev["gate"])
    torch.cuda.synchronize()
    for k in ("d_x", "d_y") + (("d_pre",) if pre else ()):
        assert torch.equal(got[k], want[k]), k
    assert torch.isfinite(got["d_y"]).all()
    if groups:
        run = 600 // groups
        bad = np.zeros((groups, d), bool)
        bad[5 // run], bad[3 // run, 7], bad[8 // run, 0] = True, True, True
        g = f64(got["d_gate"])
        assert np.array_equal(~np.isfinite(g), bad) and np.array_equal(g[~bad], f64(want["d_gate"])[~bad])
