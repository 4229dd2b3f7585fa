"""Seeded inputs of the block cache and rotary tests."""
import numpy as np

import workloads as WL
from oracle import cache as oc


def bf16(rng, shape, std=1.0):
    """(bf16 bits, their fp64 values)."""
    b = WL.bf16_round((rng.standard_normal(shape) * std).astype(np.float32))
    return b, WL.bf16_to_f32(b).astype(np.float64)


def tables(rng, lens, extra=0, spare=2):
    """Block tables of scattered pages, `extra` blocks more than the longest
    sequence needs; unused entries are no page at all.  Returns (table, pages)."""
    S = len(lens)
    blocks = max((max(lens) + 31) // 32, 1) + extra
    pages = S * blocks + spare
    order = rng.permutation(pages)[:S * blocks].reshape(S, blocks).astype(np.int32)
    for s, n in enumerate(lens):
        order[s, (n + 31) // 32:] = rng.choice([-1, pages, 2 ** 31 - 1])
    return order, pages


def cache(rng, pages, heads, D, lens=None, table=None, spread=3):
    """A cache of random finite values, its blocks' scales apart by up to
    2^spread; bytes at or behind each sequence's length are NaN."""
    c = {}
    for name in "kv":
        raw = rng.standard_normal((pages, heads, 32 * D)) * 80
        c[name] = oc.e4m3_bytes(np.clip(raw, -448, 448))
        c[name + "_scale"] = rng.integers(120, 121 + spread, (pages, heads)).astype(np.uint8)
    if table is not None:
        for s, n in enumerate(lens):
            for j in range(table.shape[1]):
                if 0 <= table[s, j] < pages:
                    dead = np.arange(32) + 32 * j >= n
                    for name in "kv":
                        c[name][int(table[s, j])][:, oc.places(D, name == "k")[dead]] = 0x7F
    return c


def on_gpu(c):
    import torch

    import masked_token_logits_amd as mtl
    t = {n: torch.from_numpy(a.copy()).cuda() for n, a in c.items()}
    return mtl.BlockCache.over(t["k"], t["v"], t["k_scale"], t["v_scale"])


def host(cache):
    return {n: getattr(cache, n).cpu().numpy() for n in ("k", "v", "k_scale", "v_scale")}


def dev_bf16(bits):
    import torch
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def dev_i32(x):
    import torch
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def cu_of(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
