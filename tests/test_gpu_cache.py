"""GPU parity of the 8-bit block cache (write, attention, accumulated weights,
eviction) against the fp64 oracle.

Tolerances, from the arithmetic:
- write: scales and value bytes are decided by exact comparisons and one
  rounding, so they are equal.  A rotated key is an fp32 number within 2^-20
  of its pair's length of the exact one, so its byte is equal unless a
  rounding boundary is that near.
- attention: a probability is rounded to fp16 for its product with v, a
  relative error of at most 2^-11; those roundings are independent, so a
  dimension's sum is held to six times their root of squares.  Scores are
  fp32 sums of D exact products: with A = scale max_j sum_i |q_i k_ji|, a
  score is within dS = (D + 8) 2^-24 A, which moves every probability by that
  relatively.  The output's rounding adds 2^-8 of the value.
    |d out| <= 6 2^-11 Q + (2 dS + 2^-20) B + 2^-8 |out|
    |d lse| <= dS + 2^-21 (|lse| + A + 1)
- weights: exp of such a score, summed in fp32 over n terms:
    |d w| <= (dS + 2^-21 (|lse| + A + 1) + n 2^-24) (w - decay w0) + 2^-22 |w|
- eviction moves bytes and weights: equal."""
import numpy as np
import pytest

import workloads as WL
from _cache_cases import bf16, cache, cu_of, dev_bf16, dev_i32, host, on_gpu, tables
from oracle import cache as oc

pytestmark = pytest.mark.gpu


def _batch(bc, cu, lens, table, **kw):
    return bc.batch(dev_i32(cu), dev_i32(lens), dev_i32(table), **kw)


# ---- write ----------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("D,heads,lens,new,r,layout", [
    (64, 2, [1], [1], 64, "half"),                         # one token in an empty cache
    (128, 3, [33, 70, 5], [1, 1, 1], 128, "half"),         # one token each, blocks partly full
    (128, 1, [64, 95, 200], [32, 33, 170], 64, "interleaved"),
    (256, 2, [77, 32], [77, 32], 256, "half"),             # a prompt from the start
    (64, 2, [40, 0, 31], [7, 0, 31], 10, "half"),          # a sequence without new tokens, few rotated dims
    (128, 2, [50, 64], [20, 32], 0, "half"),               # no rotation
    (128, 5, [90, 31], [70, 31], 64, "half"),              # half of each head, several heads of a workgroup
    (256, 1, [33], [33], 96, "half"),
    (64, 3, [40], [40], 22, "interleaved"),                # pairs that end inside a piece
    (128, 2, [45], [45], 40, "half"),                      # partners that no pieces hold
])
def test_write_parity(D, heads, lens, new, r, layout):
    import torch

    import masked_token_logits_amd as mtl
    rng = np.random.default_rng(D + heads + sum(lens))
    print(f"[case] write D={D} heads={heads} lens={lens} new={new} r={r} {layout}", flush=True)
    table, pages = tables(rng, lens, extra=1)
    old = [a - b for a, b in zip(lens, new)]
    c = cache(rng, pages, heads, D, old, table)
    cu, T = cu_of(new), sum(new)
    k, kf = bf16(rng, (T, heads, D), 2.0)
    v, vf = bf16(rng, (T, heads, D), 0.3)
    pos = rng.integers(0, 131072, T)
    bc = on_gpu(c)
    rot = mtl.Rotary(D, r, layout=layout) if r else None
    bc.write(_batch(bc, cu, lens, table), dev_bf16(k), dev_bf16(v), dev_i32(old),
             positions=dev_i32(pos) if r else None, rotary=rot)
    torch.cuda.synchronize()
    want, loose = oc.write(c, cu, lens, table, old, kf, vf, pos, oc.rotary_theta(r) if r else None, layout)
    got = host(bc)
    np.testing.assert_array_equal(got["k_scale"], want["k_scale"])
    np.testing.assert_array_equal(got["v_scale"], want["v_scale"])
    np.testing.assert_array_equal(got["v"], want["v"])
    off = got["k"] != want["k"]
    assert not np.any(off & ~loose), np.argwhere(off & ~loose)[:5].tolist()
    assert off.sum() <= max(2, 1e-3 * off.size)


def test_write_overwrites_the_middle_of_a_block():
    """A decoding block's keys are rewritten at every step: tokens around them
    stay, requantised only if the scale grows, and writing the same again
    changes nothing."""
    import torch
    rng = np.random.default_rng(20)
    D, heads, lens, new, start = 64, 2, [90, 61], [32, 5], [40, 3]
    table, pages = tables(rng, lens)
    c = cache(rng, pages, heads, D, lens, table)
    for std in (0.01, 50.0):      # below the old scale, far above it
        k, kf = bf16(rng, (37, heads, D), std)
        v, vf = bf16(rng, (37, heads, D), std)
        bc = on_gpu(c)
        b = _batch(bc, cu_of(new), lens, table)
        for _ in range(2):
            bc.write(b, dev_bf16(k), dev_bf16(v), dev_i32(start))
            torch.cuda.synchronize()
            want, _ = oc.write(c, cu_of(new), lens, table, start, kf, vf)
            got = host(bc)
            for name in want:
                np.testing.assert_array_equal(got[name], want[name], err_msg=f"{name} std={std}")


def test_write_extremes():
    """Zeros, the largest and smallest bf16 values, NaN and infinity."""
    import torch
    rng = np.random.default_rng(21)
    D, heads, lens = 64, 1, [32, 32, 32, 32]
    table, pages = tables(rng, lens)
    c = cache(rng, pages, heads, D)
    x, _ = bf16(rng, (128, heads, D))
    x[:32] = 0
    x[32:64, :, ::2] = 0x7F7F            # largest
    x[64:96] = x[64:96] & 0x807F         # subnormals
    x[96, 0, 0], x[97, 0, 1], x[98, 0, 2] = 0x7FC0, 0x7F80, 0xFF80
    xf = WL.bf16_to_f32(x).astype(np.float64)
    bc = on_gpu(c)
    bc.write(_batch(bc, cu_of(lens), lens, table), dev_bf16(x), dev_bf16(x), dev_i32([0] * 4))
    torch.cuda.synchronize()
    want, _ = oc.write(c, cu_of(lens), lens, table, [0] * 4, xf, xf)
    got = host(bc)
    for name in ("k_scale", "v_scale"):
        np.testing.assert_array_equal(got[name], want[name])
    for name in ("k", "v"):
        nan_g, nan_w = (got[name] & 0x7F) == 0x7F, (want[name] & 0x7F) == 0x7F
        np.testing.assert_array_equal(nan_g, nan_w)
        np.testing.assert_array_equal(got[name][~nan_w], want[name][~nan_w])


def test_write_leaves_the_rest_alone():
    """Bad pages, negative starts, slots behind the table and tokens behind the
    last sequence write nothing."""
    import torch
    rng = np.random.default_rng(22)
    D, heads, lens, new, start = 64, 2, [40, 64, 60, 10], [40, 40, 8, 6], [0, 40, 60, -1]
    table = np.array([[3, -1], [5, 999], [0, 1], [2, 4]], np.int32)   # second blocks of 0 and 1 are no pages
    c = cache(rng, 7, heads, D)
    T = sum(new) + 5
    k, kf = bf16(rng, (T, heads, D))
    v, vf = bf16(rng, (T, heads, D))
    bc = on_gpu(c)
    bc.write(_batch(bc, cu_of(new), lens, table), dev_bf16(k), dev_bf16(v), dev_i32(start))
    torch.cuda.synchronize()
    want, _ = oc.write(c, cu_of(new), lens, table, start, kf, vf)
    got = host(bc)
    for name in want:
        np.testing.assert_array_equal(got[name], want[name], err_msg=name)
    assert np.array_equal(got["k"][[2, 4, 6]], c["k"][[2, 4, 6]])


def test_write_strided_inputs():
    import torch

    import masked_token_logits_amd as mtl
    rng = np.random.default_rng(23)
    D, heads, lens = 64, 2, [50, 3]
    table, pages = tables(rng, lens)
    c = cache(rng, pages, heads, D)
    T = 53
    fused, _ = bf16(rng, (T, 3 * heads * D + 1))
    f = dev_bf16(fused)
    k = f[:, 1:1 + heads * D].unflatten(1, (heads, D))                  # odd alignment
    v = f[:, 2 * heads * D:3 * heads * D].unflatten(1, (heads, D)).transpose(0, 1).contiguous().transpose(0, 1)
    pos = dev_i32(rng.integers(0, 5000, T))
    rot = mtl.Rotary(D)
    res = []
    for kk, vv in ((k, v), (k.contiguous(), v.contiguous())):
        bc = on_gpu(c)
        bc.write(_batch(bc, cu_of(lens), lens, table), kk, vv, dev_i32([0, 0]), positions=pos, rotary=rot)
        torch.cuda.synchronize()
        res.append(host(bc))
    for name in res[0]:
        np.testing.assert_array_equal(res[0][name], res[1][name])
    one = k[:, :1].expand(T, heads, D)                                  # one head for all
    bc = on_gpu(c)
    bc.write(_batch(bc, cu_of(lens), lens, table), one, one, dev_i32([0, 0]))
    torch.cuda.synchronize()
    g = host(bc)
    np.testing.assert_array_equal(g["k"][table[0, :2], 0], g["k"][table[0, :2], 1])

@pytest.mark.parametrize("D,heads,lens,new,r,layout", [
    (128, 2, [45, 64], [40, 30], 64, "half"),              # in pieces, tokens of the first block held
    (64, 3, [40], [33], 22, "interleaved"),                # pairs that end inside a piece
    (128, 2, [45], [45], 40, "half"),                      # the general kernel
    (64, 1, [33], [33], 64, "half"),                       # nothing behind the rotated dimensions
])
@pytest.mark.parametrize("magnitude", [0.25, 0.5, 1.25])
def test_write_magnitude(D, heads, lens, new, r, layout, magnitude):
    """A magnitude shrinks or stretches only the rotated dimensions: those behind them, here the loudest, fit
    the block's scale as they are.  Besides parity, every finite key is read back to within half a step of e4m3
    (2^-4 of it, or 2^-10 of the scale below its normal range)."""
    import torch

    import masked_token_logits_amd as mtl
    rng = np.random.default_rng(D + heads + sum(lens))
    print(f"[case] write magnitude={magnitude} D={D} heads={heads} lens={lens} new={new} r={r} {layout}", flush=True)
    table, pages = tables(rng, lens, extra=1)
    old = [a - b for a, b in zip(lens, new)]
    c = cache(rng, pages, heads, D, old, table)
    cu, T = cu_of(new), sum(new)
    k, kf = bf16(rng, (T, heads, D), 2.0)
    if r < D:
        k[..., D - 1], kf[..., D - 1] = 0x4416, 600.0
    v, vf = bf16(rng, (T, heads, D), 0.3)
    pos = rng.integers(0, 131072, T)
    bc = on_gpu(c)
    rot = mtl.Rotary(D, r, layout=layout, magnitude=magnitude)
    bc.write(_batch(bc, cu, lens, table), dev_bf16(k), dev_bf16(v), dev_i32(old), positions=dev_i32(pos), rotary=rot)
    torch.cuda.synchronize()
    got = host(bc)
    y, size = oc.rotate(kf, pos, oc.rotary_theta(r), layout, magnitude)
    for s, (n, st) in enumerate(zip(new, old)):
        for h in range(heads):
            x, _ = oc.read_tokens(got, "k", table[s], h, lens[s])
            at = slice(int(cu[s]), int(cu[s]) + n)
            e = 2.0 ** (got["k_scale"][table[s, np.arange(st, lens[s]) // 32], h].astype(float) - 127)[:, None]
            err, tol = np.abs(x[st:] - y[at, h]), np.maximum(2.0 ** -4 * np.abs(y[at, h]), 2.0 ** -10 * e) + 2.0 ** -20 * size[at, h]
            assert np.all(err <= tol), f"sequence {s} head {h}: {np.argwhere(~(err <= tol))[:3].tolist()}"
    want, loose = oc.write(c, cu, lens, table, old, kf, vf, pos, oc.rotary_theta(r), layout, magnitude)
    np.testing.assert_array_equal(got["k_scale"], want["k_scale"])
    np.testing.assert_array_equal(got["v_scale"], want["v_scale"])
    np.testing.assert_array_equal(got["v"], want["v"])
    off = got["k"] != want["k"]
    assert not np.any(off & ~loose), np.argwhere(off & ~loose)[:5].tolist()
    assert off.sum() <= max(2, 1e-3 * off.size)


# ---- attention ------------------------------------------------------------------------------------------------

def _dS(r, D):
    return (D + 8) * 2.0 ** -24 * r["A"]


def _check_attention(out, lse, r, D, where):
    out = WL.bf16_to_f32(out.cpu().view(__import__("torch").int16).numpy().view(np.uint16)).astype(np.float64)
    lse = lse.cpu().numpy().astype(np.float64)
    real = ~np.isnan(r["lse"])
    dS = _dS(r, D)
    tol = 6 * 2.0 ** -11 * r["Q"] + (2 * dS[..., None] + 2.0 ** -20) * r["B"] + 2.0 ** -8 * np.abs(r["out"])
    err = np.abs(out - r["out"])
    bad = real[..., None] & ~(err <= tol)
    assert not bad.any(), f"{where}: out {np.argwhere(bad)[:3].tolist()}, {np.nanmax(np.where(bad, err / tol, 0)):.3g} tolerances"
    empty = real & np.isneginf(r["lse"])
    assert np.all(np.isneginf(lse[empty])) and np.all(out[empty] == 0), where
    seen = real & ~empty
    err = np.abs(lse[seen] - r["lse"][seen])
    tol = (dS + 2.0 ** -21 * (np.abs(r["lse"]) + r["A"] + 1))[seen]
    assert np.all(err <= tol), f"{where}: lse off by {np.max(err / tol):.3g} tolerances"


ATTEND = [
    # D, kv heads, q heads, lens, new, causal
    (64, 1, 1, [1], [1], 0),                           # one token
    (128, 2, 2, [31, 32, 33], [1, 1, 1], 0),           # around a block's end
    (128, 2, 8, [700, 1, 65], [1, 1, 1], 0),           # single tokens, shared heads
    (128, 1, 7, [200, 64], [32, 32], 0),               # a decoding block, 224 rows
    (64, 3, 3, [130, 77], [33, 5], 1),                 # causal, more than one tile of rows
    (256, 2, 4, [97, 40], [20, 40], 1),
    (256, 1, 1, [300], [3], 0),
    (128, 1, 4, [100, 0, 50], [3, 4, 0], 0),           # an empty cache, a sequence without queries
    (64, 1, 2, [5, 40], [9, 70], 1),                   # more queries than tokens: rows that see nothing
    (128, 1, 28, [96], [40], 1),                       # 1120 rows
    (64, 2, 2, [4000], [2], 0),                        # long
]


@pytest.mark.parametrize("D,heads,Hq,lens,new,causal", ATTEND)
def test_attention_parity(D, heads, Hq, lens, new, causal):
    import torch
    rng = np.random.default_rng(D + Hq + sum(lens) + sum(new))
    print(f"[case] attend D={D} heads={heads}/{Hq} lens={lens} new={new} causal={causal}", flush=True)
    table, pages = tables(rng, lens, extra=1)
    c = cache(rng, pages, heads, D, lens, table)     # NaN behind every sequence
    cu, T = cu_of(new), sum(new) + 3                  # three tokens belong to no sequence
    q, qf = bf16(rng, (T, Hq, D))
    scale = 1.5 / np.sqrt(D)
    bc = on_gpu(c)
    out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    o, l = bc.attend(_batch(bc, cu, lens, table), dev_bf16(q), scale=scale, causal=bool(causal), out=out, lse=lse)
    torch.cuda.synchronize()
    assert o is out and l is lse
    assert torch.all(out[-3:] == 7) and torch.all(lse[-3:] == 7)      # left as they were
    r = oc.attend(c, cu, lens, table, qf, float(np.float32(scale)), bool(causal))
    _check_attention(out, lse, r, D, "attention")
    # the tight bounds on the host's maxima change nothing
    o2, l2 = bc.attend(_batch(bc, cu, lens, table, max_new=max(max(new), 1), max_len=max(max(lens), 1)), dev_bf16(q),
                       scale=scale, causal=bool(causal), lse=True)
    n = sum(new)
    r2 = {k: v[:n] for k, v in r.items()}
    _check_attention(o2[:n], l2[:n], r2, D, "tight bounds")


@pytest.mark.parametrize("case", ["sharp", "equal", "outlier", "growing"])
def test_attention_score_shapes(case):
    """Scores of one winner, all alike, one far larger, and ever larger along
    the cache (the running maximum is replaced again and again)."""
    import torch
    rng = np.random.default_rng(30)
    D, heads, Hq, lens, new = 128, 1, 4, [515], [9]
    table, pages = tables(rng, lens)
    c = cache(rng, pages, heads, D, lens, table)
    q, qf = bf16(rng, (9, Hq, D), {"sharp": 12.0, "equal": 0.0, "outlier": 1.0, "growing": 1.0}[case])
    if case == "outlier":
        q[..., 5], qf[..., 5] = 0x4500, 2048.0
    if case == "growing":
        q[:], qf[:] = 0x3F80, 1.0
        for j in range(table.shape[1]):
            c["k"][table[0, j], 0] = oc.e4m3_bytes(np.array([1.0 + j]))[0]
            c["k"][table[0, j], 0, ::5] = oc.e4m3_bytes(np.array([2.0]))[0]
            c["k_scale"][table[0, j], 0] = 124
        for p in range(pages):
            c["v"][p, 0][(c["v"][p, 0] & 0x7F) == 0x7F] = 0x7F
    bc = on_gpu(c)
    o, l = bc.attend(_batch(bc, cu_of(new), lens, table), dev_bf16(q), lse=True)
    torch.cuda.synchronize()
    r = oc.attend(c, cu_of(new), lens, table, qf, float(np.float32(D ** -0.5)), False)
    _check_attention(o, l, r, D, case)


def test_attention_value_scales_far_apart():
    """Blocks whose values' scales differ by up to 2^20, ever larger and then
    ever smaller along the cache: every block counts for what it is."""
    import torch
    rng = np.random.default_rng(33)
    D, heads, Hq, lens, new = 64, 1, 2, [330, 330], [3, 3]
    table, pages = tables(rng, lens)
    c = cache(rng, pages, heads, D, lens, table)
    c["v_scale"][table[0, :11], 0] = 110 + 2 * np.arange(11)
    c["v_scale"][table[1, :11], 0] = 130 - 2 * np.arange(11)
    q, qf = bf16(rng, (6, Hq, D))
    bc = on_gpu(c)
    o, l = bc.attend(_batch(bc, cu_of(new), lens, table), dev_bf16(q), lse=True)
    torch.cuda.synchronize()
    r = oc.attend(c, cu_of(new), lens, table, qf, float(np.float32(D ** -0.5)), False)
    _check_attention(o, l, r, D, "scales")


def test_attention_strides_bad_pages_and_bounds():
    """q out of a fused projection; a table whose entries are partly no pages
    (their tokens are absent); lengths beyond the bound are cut."""
    import torch
    rng = np.random.default_rng(31)
    D, heads, Hq, lens, new = 64, 2, 4, [100, 64, 40], [5, 3, 2]
    table, pages = tables(rng, lens)
    table[0, 1], table[2, :] = -7, pages
    c = cache(rng, pages, heads, D, lens, table)
    x, xf = bf16(rng, (10, 3 * Hq, D))
    q = dev_bf16(x)[:, Hq:2 * Hq]
    bc = on_gpu(c)
    b = _batch(bc, cu_of(new), lens, table)
    o, l = bc.attend(b, q, lse=True)
    torch.cuda.synchronize()
    r = oc.attend(c, cu_of(new), lens, table, xf[:, Hq:2 * Hq], float(np.float32(D ** -0.5)), False)
    _check_attention(o, l, r, D, "bad pages")
    turned = q.transpose(0, 1).contiguous().transpose(0, 1)            # [H, T, D] in memory
    assert torch.equal(bc.attend(b, turned), o)
    wild = _batch(bc, cu_of(new), [2 ** 31 - 1, 64, -5], table, max_len=96)
    o2, l2 = bc.attend(wild, q, lse=True)
    torch.cuda.synchronize()
    r = oc.attend(c, cu_of(new), [96, 64, 0], table, xf[:, Hq:2 * Hq], float(np.float32(D ** -0.5)), False)
    _check_attention(o2, l2, r, D, "cut")


def test_attention_nan_stays_where_it_is_seen():
    """A NaN key or value token reaches the queries that see it and no other;
    a NaN query only its own row."""
    import torch
    rng = np.random.default_rng(32)
    D, heads, lens, new = 64, 1, [70], [40]
    table, pages = tables(rng, lens)
    q, _ = bf16(rng, (40, 1, D))
    for name, token, causal in (("k", 69, True), ("v", 69, True), ("v", 45, True), ("k", 50, True), ("v", 3, False)):
        c = cache(rng, pages, heads, D, lens, table)
        c[name][table[0, token // 32], 0, oc.places(D, name == "k")[token % 32]] = 0x7F
        bc = on_gpu(c)
        o = bc.attend(_batch(bc, cu_of(new), lens, table), dev_bf16(q), causal=causal).float().cpu().numpy()
        sees = np.arange(40) + 30 >= token if causal else np.ones(40, bool)
        np.testing.assert_array_equal(np.isnan(o[:, 0]).all(1), sees, err_msg=f"{name} {token}")
        np.testing.assert_array_equal(np.isnan(o[:, 0]).any(1), sees, err_msg=f"{name} {token}")
    c = cache(rng, pages, heads, D, lens, table)
    q[7, 0, 11] = 0x7FC0
    bc = on_gpu(c)
    o, l = bc.attend(_batch(bc, cu_of(new), lens, table), dev_bf16(q), lse=True)
    bad = np.isnan(o.float().cpu().numpy()[:, 0]).all(1)
    assert bad.sum() == 1 and bad[7] and np.array_equal(np.isnan(l.cpu().numpy()[:, 0]), bad)


def _check_faint(out, r, D, where):
    """Outputs made by tokens of faint probability, where what fp16 has of it below its normal range counts too.
    A probability is held in units in which the largest of its run is at least 2^7; below 2^-14 of them fp16 numbers
    are 2^-24 apart, so that each of at most two roundings moves it by 2^-25, which is 2^-32 of the largest:
    2^-31 V more than the tolerance above."""
    import torch
    out = WL.bf16_to_f32(out.cpu().view(torch.int16).numpy().view(np.uint16)).astype(np.float64)
    tol = 6 * 2.0 ** -11 * r["Q"] + (2 * _dS(r, D)[..., None] + 2.0 ** -20) * r["B"] + 2.0 ** -8 * np.abs(r["out"])
    err, tol = np.abs(out - r["out"]), tol + 2.0 ** -31 * r["V"]
    assert np.all(err <= tol), f"{where}: {np.argwhere(~(err <= tol))[:3].tolist()}, {np.max(err / tol):.3g} tolerances"


@pytest.mark.parametrize("D,Hq,new,extra", [(64, 2, 70, 80000), (128, 1, 140, 80000), (256, 5, 30, 80000),
                                            (64, 1, 3, 0)])
@pytest.mark.parametrize("step", [1.0, 1.875, 2.0])
def test_attention_values_of_faint_tokens(D, Hq, new, extra, step):
    """The most attended tokens have values of 0, and what there is comes from those of the block before them, whose
    scores lie up to 2^-23 lower: the reference moves far while their probabilities wait for their product."""
    import torch
    rng = np.random.default_rng(36)
    lens = [128]
    print(f"[case] faint D={D} heads=1/{Hq} new={new} step={step}", flush=True)
    table, pages = tables(rng, lens)
    c = cache(rng, pages, 1, D)
    q, qf = np.full((new, Hq, D), 0x3F80, np.uint16), np.ones((new, Hq, D))
    for name in "kv":
        c[name + "_scale"][:] = 127
    for j, (key, loud) in enumerate(((0.0, False), (0.0, True), (step, False), (step, False))):
        c["k"][table[0, j]] = oc.e4m3_bytes(np.array([key]))[0]
        if not loud:
            c["v"][table[0, j]] = 0
    bc = on_gpu(c)
    wide = np.concatenate([table, np.full((1, extra), -1, np.int32)], 1)
    o, l = bc.attend(_batch(bc, cu_of([new]), lens, wide), dev_bf16(q), scale=8.0 / D, lse=True)
    torch.cuda.synchronize()
    r = oc.attend(c, cu_of([new]), lens, table, qf, 8.0 / D, False)
    _check_faint(o, r, D, "faint")
    assert np.all(np.abs(l.cpu().numpy() - r["lse"]) <= _dS(r, D) + 2.0 ** -21 * (np.abs(r["lse"]) + r["A"] + 1))


# ---- accumulated weights --------------------------------------------------------------------------------------

@pytest.mark.parametrize("decay", [1.0, 0.5, 0.0])
@pytest.mark.parametrize("D,heads,Hq,lens,new,causal", [
    (128, 2, 8, [700, 1, 65], [1, 1, 1], 0),
    (128, 1, 7, [200, 64], [32, 32], 0),
    (64, 3, 3, [130, 77], [33, 5], 1),
    (256, 2, 4, [97, 40], [20, 40], 1),
    (64, 1, 2, [5, 40, 0, 9], [9, 70, 2, 0], 1),       # rows that see nothing, an empty cache, no queries
])
def test_weigh_parity(D, heads, Hq, lens, new, causal, decay):
    import torch
    rng = np.random.default_rng(D + Hq + sum(lens))
    print(f"[case] weigh D={D} heads={heads}/{Hq} lens={lens} new={new} causal={causal} decay={decay}", flush=True)
    table, pages = tables(rng, lens, extra=1)
    if lens[0] == 700:
        table[0, 3] = -1                               # a hole: its weights stay
    c = cache(rng, pages, heads, D, lens, table)
    cu, T = cu_of(new), sum(new) + 2
    q, qf = bf16(rng, (T, Hq, D))
    w0 = rng.random((len(lens), heads, table.shape[1] * 32)).astype(np.float32)
    if decay == 0.0:
        w0[:, :, ::3] = np.nan                         # not read
    bc = on_gpu(c)
    b = _batch(bc, cu, lens, table)
    lse = torch.full((T, Hq), float("nan"), device="cuda")
    bc.attend(b, dev_bf16(q), causal=bool(causal), lse=lse)
    w = torch.from_numpy(w0.copy()).cuda()
    bc.weigh(b, dev_bf16(q), lse, w, causal=bool(causal), decay=decay)
    torch.cuda.synchronize()
    lh = lse.cpu().numpy()
    scale = float(np.float32(D ** -0.5))
    want = oc.weigh(c, cu, lens, table, qf, lh, scale, bool(causal), w0, decay)
    r = oc.attend(c, cu, lens, table, qf, scale, bool(causal))
    rel = np.nanmax(np.where(np.isfinite(r["lse"]), _dS(r, D) + 2.0 ** -21 * (np.abs(r["lse"]) + r["A"] + 1), 0))
    got = w.cpu().numpy().astype(np.float64)
    for s, n in enumerate(lens):
        np.testing.assert_array_equal(got[s, :, n:], w0[s, :, n:].astype(np.float64))
        x, y = got[s, :, :n], want[s, :, :n]
        add = y - (decay * w0[s, :, :n] if decay else 0)
        tol = (rel + T * Hq * 2.0 ** -24) * np.abs(add) + 2.0 ** -22 * np.abs(y)
        same = np.isnan(x) & np.isnan(y)                # the hole, where decay is 0
        assert np.all(same | (np.abs(x - y) <= tol)), f"sequence {s}"

@pytest.mark.parametrize("D,heads,Hq,S", [(64, 2, 4, 2), (128, 1, 3, 2), (256, 1, 1, 2),   # few workgroups
                                          (64, 16, 16, 16), (128, 32, 32, 8)])             # of eight blocks
def test_weigh_nan_queries_reach_what_they_see(D, heads, Hq, S):
    """Under a causal mask a NaN query (whose lse is NaN) makes the tokens that it sees NaN, in its key head, and
    leaves the others to the queries that see them."""
    import torch
    rng = np.random.default_rng(51 + D)
    lens = [80] * S
    new = [70] * (S - 1) + [80]
    print(f"[case] weigh nan D={D} heads={heads}/{Hq} S={S}", flush=True)
    table, pages = tables(rng, lens)
    c = cache(rng, pages, heads, D, lens, table)
    q, qf = bf16(rng, (sum(new), Hq, D))
    cu = cu_of(new)
    hit = [(0, 20, 0), (0, 50, Hq - 1), (S - 1, 3, 0)]            # sequence, query, head
    for s, i, h in hit:
        q[cu[s] + i, h, 5], qf[cu[s] + i, h, 5] = 0x7FC0, np.nan
    w0 = rng.random((S, heads, table.shape[1] * 32)).astype(np.float32)
    bc = on_gpu(c)
    b = _batch(bc, cu, lens, table, max_len=96)
    _, lse = bc.attend(b, dev_bf16(q), causal=True, lse=True)
    w = torch.from_numpy(w0.copy()).cuda()
    bc.weigh(b, dev_bf16(q), lse, w, causal=True)
    torch.cuda.synchronize()
    lh = lse.cpu().numpy()
    scale = float(np.float32(D ** -0.5))
    want = oc.weigh(c, cu, lens, table, qf, lh, scale, True, w0, 1.0)
    r = oc.attend(c, cu, lens, table, qf, scale, True)
    rel = np.nanmax(np.where(np.isfinite(r["lse"]), _dS(r, D) + 2.0 ** -21 * (np.abs(r["lse"]) + r["A"] + 1), 0))
    got = w.cpu().numpy().astype(np.float64)
    nan = np.zeros((S, heads, 80), bool)
    for s, i, h in hit:
        nan[s, h // (Hq // heads), :80 - new[s] + i + 1] = True
    np.testing.assert_array_equal(np.isnan(got[..., :80]), nan)
    x, y = got[..., :80][~nan], want[..., :80][~nan]
    tol = (rel + sum(new) * Hq * 2.0 ** -24) * np.abs(y - w0[..., :80][~nan]) + 2.0 ** -22 * np.abs(y)
    assert np.all(np.abs(x - y) <= tol)


# ---- eviction -------------------------------------------------------------------------------------------------

def _evict(rng, lens, keep, sink, recent, pool, heads=2, D=64, w=None, max_keep=None, bad=False):
    import torch
    table, pages0 = tables(rng, lens, extra=1)
    out_blocks = (max(max(keep), 1) + 31) // 32
    pages = pages0 + len(lens) * out_blocks
    table = np.where(table == pages0, -1, table)
    table_out = (pages0 + rng.permutation(len(lens) * out_blocks).reshape(len(lens), out_blocks)).astype(np.int32)
    if bad:
        table[0, 0], table_out[-1, 0] = pages, -3
    c = cache(rng, pages, heads, D, lens, table)
    if w is None:
        w = rng.random((len(lens), heads, table.shape[1] * 32)).astype(np.float32)
        w[rng.random(w.shape) < 0.3] = 0
    bc = on_gpu(c)
    most = max_keep or out_blocks * 32
    kept = torch.full((len(lens), heads, most), -5, dtype=torch.int32, device="cuda")
    wout = torch.full((len(lens), heads, out_blocks * 32), -5.0, device="cuda")
    lens_out = torch.full((len(lens),), -5, dtype=torch.int32, device="cuda")
    bc.evict(_batch(bc, [0] * (len(lens) + 1), lens, table), torch.from_numpy(w).cuda(), dev_i32(keep),
             dev_i32(table_out), sink=sink, recent=recent, pool=pool, lens_out=lens_out, kept=kept, weights_out=wout)
    torch.cuda.synchronize()
    cut = [min(k, most) for k in keep]
    want, n, kk, ww = oc.evict(c, lens, table, w, cut, sink, recent, pool, table_out)
    np.testing.assert_array_equal(lens_out.cpu().numpy(), n)
    for s in range(len(lens)):
        for h in range(heads):
            got = kept[s, h].cpu().numpy()
            np.testing.assert_array_equal(got[:n[s]], kk[s][h], err_msg=f"kept {s} {h}")
            assert np.all(got[n[s]:] == -5)
            gw = wout[s, h].cpu().numpy()
            np.testing.assert_array_equal(gw[:n[s]], ww[s][h])
            assert np.all(gw[n[s]:] == -5)
    got = host(bc)
    for name in want:
        np.testing.assert_array_equal(got[name], want[name], err_msg=name)


@pytest.mark.parametrize("lens,keep,sink,recent,pool", [
    ([1], [1], 0, 0, 1),
    ([100, 31, 64], [50, 31, 33], 0, 0, 1),
    ([100, 31, 64], [50, 40, 0], 4, 8, 3),             # more than there are; none
    ([300, 0, 33], [65, 5, 32], 2, 40, 7),             # an empty cache
    ([200], [10], 20, 20, 3),                          # sink alone fills it
    ([200], [30], 20, 20, 63),                         # sink and a part of recent
    ([2000], [999], 4, 64, 5),
])
def test_evict_parity(lens, keep, sink, recent, pool):
    print(f"[case] evict lens={lens} keep={keep} sink={sink} recent={recent} pool={pool}", flush=True)
    _evict(np.random.default_rng(sum(lens) + sum(keep)), lens, keep, sink, recent, pool)


@pytest.mark.parametrize("D,heads", [(128, 3), (256, 1)])
def test_evict_head_sizes(D, heads):
    _evict(np.random.default_rng(40), [130, 95], [70, 33], 1, 4, 3, heads=heads, D=D)


@pytest.mark.parametrize("kind", ["equal", "zeros", "specials", "few values"])
def test_evict_ties_and_special_weights(kind):
    rng = np.random.default_rng(41)
    w = np.zeros((2, 2, 160), np.float32)
    if kind == "equal":
        w[:] = 0.25
    if kind == "zeros":
        w[:, :, ::2] = -0.0
    if kind == "specials":
        w = rng.standard_normal(w.shape).astype(np.float32)
        w[:, :, 3::11], w[:, :, 4::13], w[:, :, 5::17] = np.nan, np.inf, -np.inf
    if kind == "few values":
        w = rng.integers(0, 3, w.shape).astype(np.float32)
    _evict(rng, [128, 77], [51, 40], 0, 0, 1, w=w)
    _evict(rng, [128, 77], [51, 40], 3, 5, 3, w=w)


@pytest.mark.parametrize("kind", ["spread", "equal", "few values", "specials"])
def test_evict_long_rows(kind):
    """Rows of several selection chunks, ending on, before and behind a chunk's
    end, one of them short; ties across chunks."""
    rng = np.random.default_rng(44)
    lens, keep = [20001, 8192, 8193, 100, 0], [5003, 8000, 1, 99, 4]
    w = rng.random((5, 1, 626 * 32 + 32)).astype(np.float32)
    if kind == "equal":
        w[:] = 0.5
    if kind == "few values":
        w = rng.integers(0, 4, w.shape).astype(np.float32)
    if kind == "specials":
        w = rng.standard_normal(w.shape).astype(np.float32) * np.exp(20 * rng.standard_normal(w.shape)).astype(np.float32)
        w[:, :, 3::11], w[:, :, 4::13], w[:, :, 5::17] = np.nan, np.inf, -np.inf
    print(f"[case] evict long rows {kind}", flush=True)
    _evict(rng, lens, keep, 4, 32, 3, heads=1, w=w)
    _evict(rng, lens, keep, 0, 0, 63, heads=1, w=w)


def test_evict_bad_pages_and_cut_keep():
    _evict(np.random.default_rng(42), [100, 90], [64, 60], 4, 0, 1, bad=True)
    _evict(np.random.default_rng(43), [100, 90], [64, 60], 4, 0, 1, max_keep=37)


# ---- scale bytes that no write leaves ---------------------------------------------------------------------------

@pytest.mark.parametrize("D,heads,Hq,lens,new,causal,extra", [
    (64, 40, 40, [1300, 330], [1, 2], False, 0),           # few rows, several blocks to a wave
    (128, 1, 4, [300], [9], True, 0),
    (64, 40, 80, [700], [70], False, 1000),                # many
    (256, 1, 5, [400], [30], True, 30000),
])
@pytest.mark.parametrize("kind", ["low", "high"])
def test_attention_outermost_scale_bytes(D, heads, Hq, lens, new, causal, extra, kind):
    """Scale bytes 0 and 255 count as 1 and 254, wherever along the cache they stand."""
    import torch
    rng = np.random.default_rng(34)
    print(f"[case] scale bytes {kind} D={D} heads={heads}/{Hq} lens={lens} new={new} causal={causal} {extra}", flush=True)
    table, pages = tables(rng, lens)
    c = cache(rng, pages, heads, D, lens, table)
    if kind == "low":                                      # so that runs of blocks begin with some
        for s, n in enumerate(lens):
            blocks = np.arange((n + 31) // 32)
            c["v_scale"][table[s, blocks[blocks % 3 < 2]]] = 0
            c["k_scale"][table[s, blocks[::4]]] = 0
    else:                                                  # values within 1, for sums that bf16 holds
        for p in range(pages):
            c["v"][p] = np.where((c["v"][p] & 0x7F) == 0x7F, c["v"][p], (c["v"][p] & 0x87) | 0x28)
        for s in range(len(lens)):
            c["v_scale"][table[s, [1, 6]]] = 255
    q, qf = bf16(rng, (sum(new), Hq, D))
    bc = on_gpu(c)
    wide = np.concatenate([table, np.full((len(lens), extra), -1, np.int32)], 1)
    o, l = bc.attend(_batch(bc, cu_of(new), lens, wide), dev_bf16(q), causal=causal, lse=True)
    torch.cuda.synchronize()
    r = oc.attend(c, cu_of(new), lens, table, qf, float(np.float32(D ** -0.5)), causal)
    _check_faint(o, r, D, f"scale bytes {kind}")            # the most attended tokens may be those without values
    assert np.all(np.abs(l.cpu().numpy() - r["lse"]) <= _dS(r, D) + 2.0 ** -21 * (np.abs(r["lse"]) + r["A"] + 1))


def test_weigh_write_and_evict_outermost_scale_bytes():
    """The same where the other calls read them: keys of accumulated weights, the tokens that a write holds, the
    blocks that an eviction moves."""
    import torch
    rng = np.random.default_rng(35)
    D, heads, lens, new, start = 64, 2, [100, 78], [20, 11], [80, 67]
    table, pages = tables(rng, lens)
    table_out = (pages + np.arange(4).reshape(2, 2)).astype(np.int32)
    c = cache(rng, pages + 4, heads, D)
    for name in "kv":                                      # values within 1, none of them NaN
        c[name] = (c[name] & 0x87) | 0x28
    c["k_scale"][table[0, :3]], c["v_scale"][table[0, :4]] = 0, 0
    q, qf = bf16(rng, (31, 2, D))
    bc = on_gpu(c)
    b = _batch(bc, cu_of(new), lens, table)
    _, lse = bc.attend(b, dev_bf16(q), lse=True)
    w = torch.zeros(2, heads, table.shape[1] * 32, device="cuda")
    bc.weigh(b, dev_bf16(q), lse, w)
    torch.cuda.synchronize()
    scale = float(np.float32(D ** -0.5))
    want = oc.weigh(c, cu_of(new), lens, table, qf, lse.cpu().numpy(), scale, False, np.zeros(w.shape, np.float32), 1.0)
    r = oc.attend(c, cu_of(new), lens, table, qf, scale, False)
    rel = (_dS(r, D) + 2.0 ** -21 * (np.abs(r["lse"]) + r["A"] + 1)).max() + 31 * 2.0 ** -24
    got = w.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - want) <= rel * np.abs(want))
    c["v_scale"][table[1, :3], 0], c["k_scale"][table[1, 2], 1] = 255, 255
    bc = on_gpu(c)
    x, xf = bf16(rng, (31, heads, D))
    bc.write(b, dev_bf16(x), dev_bf16(x), dev_i32(start))
    torch.cuda.synchronize()
    want, _ = oc.write(c, cu_of(new), lens, table, start, xf, xf)
    got = host(bc)
    for name in want:
        np.testing.assert_array_equal(got[name], want[name], err_msg=f"write {name}")
    w = rng.random((2, heads, table.shape[1] * 32)).astype(np.float32)
    bc.evict(b, torch.from_numpy(w).cuda(), dev_i32([50, 60]), dev_i32(table_out))
    torch.cuda.synchronize()
    moved = oc.evict(got, lens, table, w, [50, 60], 0, 0, 1, table_out)[0]
    got = host(bc)
    for name in moved:
        np.testing.assert_array_equal(got[name], moved[name], err_msg=f"evict {name}")
