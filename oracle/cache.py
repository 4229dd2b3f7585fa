"""fp64 CPU oracle of rotary positions and the 8-bit block cache (test
infrastructure only).

Written from the definitions in include/dllm_rotary.h and
include/dllm_cache.h, one token, block and head at a time.  Sparse-dLLM
(Sparse-dLLM: Accelerating Diffusion LLMs with Dynamic Cache Eviction,
Method and Pseudocode) scores a cached key by the attention it receives,
max-pools the scores and keeps the best; the pages give no numerics, which
the headers fix.  A cache here is a dict of NumPy arrays: k, v [pages, heads,
32 * D] uint8 and k_scale, v_scale [pages, heads] uint8.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 32
SCALE_MIN, SCALE_MAX = 27, 254
ROOT2 = np.float32(1.41421366)


def rotary_theta(r: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0, original_len: int = 0,
                 fast: float = 32.0, slow: float = 1.0) -> np.ndarray:
    """Angle per position of each of the r / 2 pairs."""
    theta = []
    for i in range(r // 2):
        b = base * factor ** (r / (r - 2.0)) if scaling == "base" else base
        t = b ** (-2.0 * i / r)
        if scaling == "linear":
            t /= factor
        if scaling == "ramp":
            n = original_len * t / (2.0 * math.pi)
            g = min(max((n - slow) / (fast - slow), 0.0), 1.0)
            t = g * t + (1.0 - g) * t / factor
        theta.append(t)
    return np.array(theta)


def rotate(x: np.ndarray, pos: np.ndarray, theta: np.ndarray, layout: str, magnitude: float = 1.0,
           transpose: bool = False):
    """x [T, H, D] fp64 -> (rotated x, length of each dimension's pair)."""
    y, size = x.copy(), np.abs(x)
    n = len(theta)
    for i in range(n):
        a, b = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
        ang = pos.astype(np.float64) * theta[i]
        c, s = magnitude * np.cos(ang)[:, None], magnitude * np.sin(ang)[:, None]
        if transpose:
            s = -s
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        size[..., a] = size[..., b] = magnitude * np.hypot(x[..., a], x[..., b])
    return y, size


def _e4m3_values() -> np.ndarray:
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = math.nan if e == 15 and m == 7 else m / 512.0 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        out[b] = -v if b & 128 else v
    return out


E4M3 = _e4m3_values()


def e4m3_bytes(x: np.ndarray) -> np.ndarray:
    """Bytes of the e4m3 values nearest to x, ties to the even byte; NaN for
    what is not finite.  |x| <= 448 up to the roundings of a scale's bound:
    what is larger was given a scale that does not hold it."""
    x = np.asarray(x, dtype=np.float64)
    out = np.full(x.shape, 0x7F, np.uint8)
    ok = np.isfinite(x)
    a = np.abs(x[ok])
    if a.max(initial=0) > 448.0 * (1 + 2.0 ** -20):
        raise ValueError(f"{a.max()} is beyond e4m3's largest value")
    a = np.minimum(a, 448.0)
    grid = E4M3[:127]                                     # ascending
    i = np.clip(np.searchsorted(grid, a), 1, 126)
    lo, hi = grid[i - 1], grid[i]
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 0))
    out[ok] = np.where(up, i, i - 1).astype(np.uint8) | (np.signbit(x[ok]).astype(np.uint8) << 7)
    return out


def near_tie(x: np.ndarray, width: np.ndarray) -> np.ndarray:
    """Whether a boundary between two e4m3 values lies within `width` of x."""
    grid = E4M3[:127]
    edge = (grid[1:] + grid[:-1]) / 2
    a = np.abs(x)
    i = np.clip(np.searchsorted(edge, a), 1, len(edge) - 1)
    return np.minimum(np.abs(a - edge[i - 1]), np.abs(a - edge[i])) <= width


def k_place(t: int, d: int, D: int) -> int:
    """Where a key block holds dimension d of token t."""
    h, rest = divmod(d, D // 2)
    return ((rest // 16) * 2 + h) * 512 + t * 16 + rest % 16


def v_place(t: int, d: int, D: int) -> int:
    return ((d // 32) * 2 + (t // 4) % 2) * 512 + (d % 32) * 16 + (t // 8) * 4 + t % 4


def places(D: int, key: bool) -> np.ndarray:
    """[32, D]: place of every token and dimension."""
    f = k_place if key else v_place
    return np.array([[f(t, d, D) for d in range(D)] for t in range(BLOCK)])


def stored_scale(cache: dict, name: str, page: int, head: int) -> int:
    """A block's scale byte; 0 and 255 count as 1 and 254."""
    return min(max(int(cache[name + "_scale"][page, head]), 1), 254)


def read_block(cache: dict, name: str, page: int, head: int) -> np.ndarray:
    """[32, D] fp64."""
    D = cache[name].shape[2] // BLOCK
    raw = E4M3[cache[name][page, head]][places(D, name == "k")]
    return raw * 2.0 ** (stored_scale(cache, name, page, head) - 127)


def read_tokens(cache: dict, name: str, table: np.ndarray, head: int, n: int) -> tuple[np.ndarray, np.ndarray]:
    """The first n tokens of a sequence [n, D], and which of them have a page."""
    D = cache[name].shape[2] // BLOCK
    x, ok = np.zeros((n, D)), np.zeros(n, bool)
    for j in range((n + BLOCK - 1) // BLOCK):
        page, m = int(table[j]), min(BLOCK, n - j * BLOCK)
        if 0 <= page < cache[name].shape[0]:
            x[j * BLOCK:j * BLOCK + m] = read_block(cache, name, page, head)[:m]
            ok[j * BLOCK:j * BLOCK + m] = True
    return x, ok


def scale_byte(big: float) -> int:
    """127 + the smallest e with big <= 448 * 2^e, clamped to the range a write chooses from."""
    if big <= 0:
        return SCALE_MIN
    e = math.ceil(math.log2(big)) - 10
    while big > 448.0 * 2.0 ** e:
        e += 1
    return min(max(e + 127, SCALE_MIN), SCALE_MAX)


def write(cache: dict, cu, lens, table, start, k: np.ndarray, v: np.ndarray, pos=None, theta=None, layout="half",
          magnitude: float = 1.0):
    """The cache after a write of k, v [T, heads, D] (fp64 values of bf16
    data).  Returns (cache, loose): loose [pages, heads, 32 * D] marks key
    bytes whose unrounded value lies so near a rounding boundary that fp32
    may decide either way."""
    new = {n: a.copy() for n, a in cache.items()}
    heads, D = k.shape[1:]
    loose = np.zeros(cache["k"].shape, bool)
    yk, size = (rotate(k, pos, theta, layout, magnitude) if theta is not None else (k, np.zeros_like(k)))
    gain = np.float32(1)
    if theta is not None:
        gain = np.float32(ROOT2 * np.float32(magnitude))
        if 2 * len(theta) < D:                 # some dimensions are stored as they are
            gain = max(gain, np.float32(1))
    for s in range(len(lens)):
        n, st = int(cu[s + 1] - cu[s]), int(start[s])
        if st < 0 or n == 0:
            continue
        for blk in range(st // BLOCK, (st + n - 1) // BLOCK + 1):
            if blk >= table.shape[1] or not 0 <= int(table[s, blk]) < cache["k"].shape[0]:
                continue
            page, slots = int(table[s, blk]), blk * BLOCK + np.arange(BLOCK)
            fresh = (slots >= st) & (slots < st + n)
            held = (slots < int(lens[s])) & ~fresh
            at = int(cu[s]) + slots[fresh] - st
            for h in range(heads):
                for name, y, x, g in (("k", yk, k, gain), ("v", v, v, np.float32(1))):
                    fin = np.where(np.isfinite(x[at, h]), np.abs(x[at, h]), 0)
                    byte = scale_byte(float(np.float32(fin.max(initial=0)) * g))
                    if held.any():
                        byte = min(max(byte, stored_scale(cache, name, page, h)), SCALE_MAX)
                    rows = np.zeros((BLOCK, D))
                    rows[held] = read_block(cache, name, page, h)[held] * 2.0 ** (127 - byte)
                    rows[fresh] = y[at, h] * 2.0 ** (127 - byte)
                    put = np.where((fresh | held)[:, None], e4m3_bytes(rows), 0)
                    pl = places(D, name == "k")
                    new[name][page, h, pl] = put
                    new[name + "_scale"][page, h] = byte
                    if name == "k" and theta is not None:
                        wide = np.zeros((BLOCK, D))
                        wide[fresh] = size[at, h] * 2.0 ** (127 - byte) * 2.0 ** -20
                        loose[page, h, pl] = near_tie(rows, wide) & fresh[:, None]
    return new, loose


def attend(cache: dict, cu, lens, table, q: np.ndarray, scale: float, causal: bool):
    """q [T, q_heads, D] fp64.  Returns a dict with out, lse and, for error
    bounds, per query (and dimension): B = sum p |v|, Q = sqrt(sum p^2 v^2) and
    V = (largest p) sum |v|, each over sum p, and A = scale max_j sum_i |q_i k_ji|."""
    T, Hq, D = q.shape
    heads = cache["k"].shape[1]
    r = {n: np.full((T, Hq, D), np.nan) for n in ("out", "B", "Q", "V")}
    r["lse"], r["A"] = (np.full((T, Hq), np.nan) for _ in range(2))
    for s in range(len(lens)):
        n, length = int(cu[s + 1] - cu[s]), int(lens[s])
        for h in range(heads):
            k, ok = read_tokens(cache, "k", table[s], h, length)
            v, _ = read_tokens(cache, "v", table[s], h, length)
            for i in range(n):
                see = ok & (np.arange(length) <= length - n + i) if causal else ok
                for g in range(Hq // heads):
                    t, hq = int(cu[s]) + i, h * (Hq // heads) + g
                    if not see.any():
                        for name in ("out", "B", "Q", "V"):
                            r[name][t, hq] = 0
                        r["lse"][t, hq], r["A"][t, hq] = -np.inf, 0
                        continue
                    ks, vs = k[see], v[see]
                    z = scale * (ks @ q[t, hq])
                    top = z.max()
                    p = np.exp(z - top)
                    tot = p.sum()
                    r["out"][t, hq] = p @ vs / tot
                    r["lse"][t, hq] = top + math.log(tot)
                    r["B"][t, hq] = p @ np.abs(vs) / tot
                    r["Q"][t, hq] = np.sqrt((p * p) @ (vs * vs)) / tot
                    r["V"][t, hq] = np.abs(vs).sum(0) / tot
                    r["A"][t, hq] = scale * (np.abs(ks) @ np.abs(q[t, hq])).max()
    return r


def weigh(cache: dict, cu, lens, table, q: np.ndarray, lse: np.ndarray, scale: float, causal: bool,
          weights: np.ndarray, decay: float) -> np.ndarray:
    out = weights.astype(np.float64).copy()
    heads = cache["k"].shape[1]
    group = q.shape[1] // heads
    for s in range(len(lens)):
        n, length = int(cu[s + 1] - cu[s]), int(lens[s])
        for h in range(heads):
            k, ok = read_tokens(cache, "k", table[s], h, length)
            got = np.zeros(length)
            for i in range(n):
                see = ok & (np.arange(length) <= length - n + i) if causal else ok
                for g in range(group):
                    t, hq = int(cu[s]) + i, h * group + g
                    if lse[t, hq] != -np.inf:
                        got[see] += np.exp(scale * (k[see] @ q[t, hq]) - float(lse[t, hq]))
            old = decay * out[s, h, :length] if decay else 0.0
            out[s, h, :length] = np.where(ok, old + got, out[s, h, :length])
    return out


def select(w: np.ndarray, keep: int, sink: int, recent: int, pool: int) -> np.ndarray:
    """The kept tokens of one sequence and head, ascending."""
    length = len(w)
    n = min(max(keep, 0), length)
    first = min(sink, n)
    last = min(recent, n - first)
    w = np.where(np.isnan(w), -np.inf, w)
    pooled = [max(w[max(0, j - pool // 2):j + pool // 2 + 1]) for j in range(length)]
    between = sorted(range(first, length - last), key=lambda j: (-pooled[j], j))[:n - first - last]
    return np.array(sorted(list(range(first)) + between + list(range(length - last, length))), dtype=np.int64)


def evict(cache: dict, lens, table, weights: np.ndarray, keep, sink: int, recent: int, pool: int, table_out):
    """Returns (cache, lens_out, kept[s][h], weights_out[s][h])."""
    new = {n: a.copy() for n, a in cache.items()}
    heads, D = cache["k"].shape[1], cache["k"].shape[2] // BLOCK
    pages = cache["k"].shape[0]
    lens_out, kept, wout = [], [], []
    for s in range(len(lens)):
        length = int(lens[s])
        kept.append([select(weights[s, h, :length], int(keep[s]), sink, recent, pool) for h in range(heads)])
        wout.append([weights[s, h][kept[s][h]] for h in range(heads)])
        n = len(kept[s][0])
        lens_out.append(n)
        for h in range(heads):
            for blk in range((n + BLOCK - 1) // BLOCK):
                to = int(table_out[s, blk])
                if not 0 <= to < pages:
                    continue
                js = kept[s][h][blk * BLOCK:(blk + 1) * BLOCK]
                src = [int(table[s, j // BLOCK]) for j in js]
                for name in "kv":
                    pl = places(D, name == "k")
                    es = [stored_scale(cache, name, p, h) if 0 <= p < pages else 0 for p in src]
                    top = max(max(es), SCALE_MIN)
                    put = np.zeros((BLOCK, D), np.uint8)
                    for t, (j, p, e) in enumerate(zip(js, src, es)):
                        if 0 <= p < pages:
                            raw = cache[name][p, h][pl[j % BLOCK]]
                            put[t] = raw if e == top else e4m3_bytes(E4M3[raw] * 2.0 ** (e - top))
                    new[name][to, h, pl] = put
                    new[name + "_scale"][to, h] = top
    return new, np.array(lens_out), kept, wout
