"""The operators of cached block decoding, as cases that can be timed and compared: rotary positions, the write into
the 8-bit block cache, attention over that cache, the accumulation of attention weights and the eviction by them.

``run`` computes them in plain torch (``own`` false) or through the package's public entry points (``own`` true).
A cache block is 32 tokens of one head: 32 * D bytes of e4m3 values and one power-of-two scale, held as its exponent
plus 127.  Byte (c, h, t, j) of a key block [D/32][2][32][16] is token t, dimension h * D/2 + 16 c + j; byte
(c, h, r, b) of a value block is token 8 (b / 4) + 4 h + b % 4, dimension 32 c + r."""
import math
import random

import torch

own = False

BLOCK = 32
LOWEST, HIGHEST = 27, 254  # exponent bytes that a write chooses from
ROOT2 = 1.41421366  # the float32 above the square root of two


def listed():
    return [
        # the queries of one 32-token decoding block: the smallest call, where only latency counts
        dict(name="rotary block", op="rotary", T=32, H=32, D=128, r=128, layout="half", scaling="none", factor=1.0, fused=0),
        # the queries of a long prompt, a slice of the fused projection's output, half of each head rotated, positions stretched
        dict(name="rotary prompt", op="rotary", T=8192, H=28, D=128, r=64, layout="interleaved", scaling="ramp", factor=8.0, fused=1),
        # one new token in each of 64 sequences: blocks that are partly full keep their other tokens
        dict(name="write one token", op="write", S=64, n=1, len=4096, ragged=1, Hkv=8, D=128, r=128, layout="half"),
        # the prompt of a long-context sequence, written at once
        dict(name="write prompt", op="write", S=1, n=131072, len=131072, ragged=0, Hkv=4, D=128, r=128, layout="half"),
        # serving single tokens: 16 sequences of different lengths
        dict(name="attend one token", op="attend", S=16, n=1, len=4096, ragged=1, Hq=32, Hkv=8, D=128, causal=0),
        # one denoising step of a 32-token block against a 4096-token cache, every head with its own keys
        dict(name="attend block", op="attend", S=1, n=32, len=4096, ragged=0, Hq=32, Hkv=32, D=128, causal=0),
        # the same at long context with shared key heads
        dict(name="attend block long", op="attend", S=1, n=32, len=131072, ragged=0, Hq=28, Hkv=4, D=128, causal=0),
        # the refresh of a whole sequence: every position attends to every other
        dict(name="attend all", op="attend", S=1, n=8192, len=8192, ragged=0, Hq=28, Hkv=4, D=128, causal=0),
        # the weights that one block's step gives to each cached token
        dict(name="weigh block", op="weigh", S=4, n=32, len=8192, ragged=1, Hq=28, Hkv=4, D=128, causal=0),
        # the weights of a prompt under a causal mask
        dict(name="weigh prompt", op="weigh", S=1, n=4096, len=4096, ragged=0, Hq=32, Hkv=32, D=128, causal=1),
        # half of a 4096-token cache evicted, as block decoding does once a block
        dict(name="evict half", op="evict", S=1, len=4096, ragged=0, keep=2048, Hkv=32, D=128, sink=0, recent=32, pool=3),
        # long contexts of different lengths cut down to a budget
        dict(name="evict long", op="evict", S=4, len=131072, ragged=1, keep=16385, Hkv=4, D=128, sink=4, recent=64, pool=3),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "write", "attend", "attend", "weigh", "evict"])
    D = rng.choice([64, 128, 128, 256])
    Hq, Hkv = rng.choice([(32, 32), (28, 4), (32, 8), (8, 1), (12, 12), (6, 2)])
    layout = rng.choice(["half", "interleaved"])
    r = rng.choice([D, D // 2, D // 4, 2 * rng.randint(1, D // 2)])
    if op == "rotary":
        return dict(op=op, T=_log(rng, 1, 16384 * 128 // D), H=Hq, D=D, r=r, layout=layout,
                    scaling=rng.choice(["none", "linear", "base", "ramp"]) if r > 2 else "none",
                    factor=rng.choice([2.0, 8.0, 10.0]), fused=rng.randint(0, 1))
    S = _log(rng, 1, 64)
    if op == "write":
        n = _log(rng, 1, max(1, 131072 * 512 // (S * Hkv * D)))
        return dict(op=op, S=S, n=n, len=n + rng.randint(0, 4000), ragged=1, Hkv=Hkv, D=D, r=r, layout=layout)
    if op == "evict":
        length = _log(rng, 1, max(1, min(131072, 131072 * 2048 // (S * Hkv * D))))
        return dict(op=op, S=S, len=length, ragged=rng.randint(0, 1), keep=rng.randint(1, length), Hkv=Hkv, D=D,
                    sink=rng.choice([0, 1, 4]), recent=rng.choice([0, 32, 100]), pool=rng.choice([1, 3, 7]))
    length = _log(rng, 1, max(1, min(131072, 131072 * 2048 // (S * Hkv * D))))
    most = (8192 * 8192 * 28 * 128 if op == "attend" else 4096 * 4096 * 32 * 128) // 2  # a quarter to a half of the listed
    n = _log(rng, 1, max(1, min(length, most // (S * length * Hq * D))))
    return dict(op=op, S=S, n=n, len=length, ragged=rng.randint(0, 1), Hq=Hq, Hkv=Hkv, D=D, causal=rng.randint(0, 1))


def _counts(case):
    """Lengths after the call and new tokens of each sequence: plain numbers that the case alone decides."""
    S, top, n = case["S"], case["len"], case.get("n", 0)
    lens = [max(min(n, top), top - (s * 3 * top) // (4 * S)) if case["ragged"] else top for s in range(S)]
    random.Random(S * 1000003 + top).shuffle(lens)
    new = [min(n, x) if not case["ragged"] or n == 1 else max(1, min(x, n) - (s % 3)) for s, x in enumerate(lens)]
    return lens, new


def _frequencies(case, dev):
    """Angle for each position step [r/2] and the magnitude, in 64 bits."""
    r, base, factor = case["r"], 10000.0, case.get("factor", 1.0)
    scaling = case.get("scaling", "none")
    if scaling == "base":
        base = base * factor ** (r / (r - 2))
    theta = base ** (-torch.arange(0, r, 2, dtype=torch.float64, device=dev) / r)
    if scaling == "linear":
        theta = theta / factor
    if scaling == "ramp":
        gamma = ((4096 * theta / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        theta = theta * (gamma + (1 - gamma) / factor)
    return theta, 0.1 * math.log(factor) + 1.0 if scaling == "ramp" else 1.0


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rnd = lambda *shape: torch.randn(*shape, generator=g, device=dev)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    s, op, D = dict(case=case), case["op"], case["D"]
    if op == "rotary":
        T, H = case["T"], case["H"]
        x = rnd(T, (3 if case["fused"] else 1) * H, D).to(torch.bfloat16)
        s["x"] = x[:, :H]
        s["pos"] = (torch.arange(T, device=dev) + torch.randint(0, 100000, (1,), generator=g, device=dev)).to(torch.int32)
        return s
    S, H = case["S"], case["Hkv"]
    lens, new = _counts(case)
    cap = (max(lens) + BLOCK - 1) // BLOCK  # blocks a sequence may have
    cap_out = (case.get("keep", 0) + BLOCK - 1) // BLOCK
    pages = S * (cap + cap_out)
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)  # blocks lie anywhere in the pool
    s["table"], s["table_out"] = order[: S * cap].view(S, cap).contiguous(), order[S * cap:].view(S, cap_out).contiguous()
    # e4m3 bytes as a write leaves them: normal values up to the top binade of their block, and scales around 2^-7
    for k in "kv":
        fill = rnd(pages, H, BLOCK * D).mul_(80).clamp_(-448, 448).to(torch.float8_e4m3fn)
        s[k], s[k + "_scale"] = fill.view(torch.uint8), torch.randint(119, 122, (pages, H), generator=g, device=dev, dtype=torch.uint8)
    s["lens"], s["lens_host"], s["new_host"] = i32(lens), lens, new
    s["cu"] = i32([sum(new[:i]) for i in range(S + 1)])
    T = sum(new)
    if op == "write":
        chan = torch.exp(0.7 * rnd(1, H, D))  # keys with louder channels
        s["k_new"], s["v_new"] = (rnd(T, H, D) * chan).to(torch.bfloat16), rnd(T, H, D).to(torch.bfloat16)
        s["start"] = i32([a - b for a, b in zip(lens, new)])
        s["pos"] = torch.cat([torch.arange(a - b, a, dtype=torch.int32, device=dev) for a, b in zip(lens, new)])
    elif op in ("attend", "weigh"):
        loud = torch.exp(0.5 * rnd(1, case["Hq"], 1))  # heads from diffuse to sharp
        s["q"] = (rnd(T, case["Hq"], D) * loud).to(torch.bfloat16)
        if op == "weigh":
            s["lse"] = _attend_plain(s)[1]
            s["weights"] = torch.rand(S, H, cap * BLOCK, generator=g, device=dev)
    else:
        w = torch.exp(2 * rnd(S, H, cap * BLOCK))
        s["weights"] = torch.where(w < 0.05, torch.zeros_like(w), w)  # tokens that no query saw: equal weights
        s["keep"] = i32([case["keep"]] * S)
        s["lens_out"] = torch.zeros(S, dtype=torch.int32, device=dev)
        s["weights_out"] = torch.zeros(S, H, cap_out * BLOCK, device=dev)
        s["kept"] = torch.full((S, H, case["keep"]), -1, dtype=torch.int32, device=dev)
    return s


# ---- plain forms ----------------------------------------------------------------------------------------------

def _tokens_k(b, D):
    """Key blocks [..., 32 D] in the cache's order -> [..., 32, D]."""
    n = b.dim() - 1
    return b.unflatten(-1, (D // 32, 2, 32, 16)).permute(*range(n), n + 2, n + 1, n, n + 3).flatten(n + 1)


def _tokens_v(b, D):
    n = b.dim() - 1
    return b.unflatten(-1, (D // 32, 2, 32, 4, 4)).permute(*range(n), n + 3, n + 1, n + 4, n, n + 2).flatten(n + 3).flatten(n, n + 2)


def _blocks_k(x):
    """[..., 32, D] -> [..., 32 D] in the cache's order."""
    n, D = x.dim() - 2, x.shape[-1]
    return x.unflatten(-1, (2, D // 32, 16)).permute(*range(n), n + 2, n + 1, n, n + 3).flatten(n)


def _blocks_v(x):
    n, D = x.dim() - 2, x.shape[-1]
    return x.unflatten(-1, (D // 32, 32)).unflatten(-3, (4, 2, 4)).permute(*range(n), n + 3, n + 1, n + 4, n, n + 2).flatten(n)


def _value(b):
    return b.contiguous().view(torch.float8_e4m3fn).float()


def _scale(b):
    return torch.exp2(b.double() - 127).float()


def _gathered(s, name):
    """Keys or values of every sequence [S, Hkv, tokens, D] in 32 bits."""
    D, table = s["case"]["D"], s["table"].long()
    tok = _tokens_k if name == "k" else _tokens_v
    x = _value(tok(s[name][table], D)) * _scale(s[name + "_scale"][table])[..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _rotate(x, pos, case):
    """x [T, H, D] rotated in 32 bits, angles in 64."""
    theta, mag = _frequencies(case, x.device)
    a = pos.double()[:, None, None] * theta
    c, sn, r = (torch.cos(a) * mag).float(), (torch.sin(a) * mag).float(), case["r"]
    x = x.float()
    if case["layout"] == "half":
        p, q = x[..., : r // 2], x[..., r // 2: r]
        y = torch.cat([p * c - q * sn, q * c + p * sn], -1)
    else:
        p, q = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([p * c - q * sn, q * c + p * sn], -1).flatten(-2)
    return torch.cat([y, x[..., r:]], -1)


def _padded(s):
    """For each sequence and row of the longest: the token, and whether there is one; for each token: its sequence and row."""
    cu, top = s["cu"].long(), max(s["new_host"])
    row = torch.arange(top, device=cu.device)
    at = cu[:-1, None] + row
    t = torch.arange(sum(s["new_host"]), device=cu.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    return at.clamp(max=len(t) - 1), row < (cu[1:] - cu[:-1])[:, None], seq, t - cu[seq]


def _scores(s):
    """Scaled and masked scores [S, Hkv, rows * G, tokens]."""
    c = s["case"]
    at, real, seq, row = _padded(s)
    q = s["q"].float()[at]  # [S, rows, Hq, D]
    q = q.unflatten(2, (c["Hkv"], c["Hq"] // c["Hkv"])).permute(0, 2, 1, 3, 4).flatten(2, 3)
    k = _gathered(s, "k")
    sc = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(c["D"]))
    key = torch.arange(k.shape[2], device=q.device)
    lens = s["lens"].long()[:, None, None]
    end = lens - (s["cu"][1:] - s["cu"][:-1]).long()[:, None, None] + torch.arange(at.shape[1], device=q.device)[None, :, None] + 1 if c["causal"] else lens
    seen = ((key < end) & real[:, :, None]).repeat_interleave(c["Hq"] // c["Hkv"], 1)[:, None]
    return sc.masked_fill(~seen, -math.inf), seq, row


def _attend_plain(s):
    c = s["case"]
    sc, seq, row = _scores(s)
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(top == -math.inf, torch.zeros_like(top), top))
    del sc
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _gathered(s, "v")) / torch.where(total == 0, torch.ones_like(total), total)
    back = lambda x: x.unflatten(2, (-1, c["Hq"] // c["Hkv"])).permute(0, 2, 1, 3, 4).flatten(2, 3)[seq, row]  # noqa: E731
    return back(o).to(torch.bfloat16), back(top + torch.log(total))[..., 0]


def _weigh_plain(s):
    c = s["case"]
    sc, seq, row = _scores(s)
    at, real, _, _ = _padded(s)
    lse = s["lse"][at].unflatten(2, (c["Hkv"], -1)).permute(0, 2, 1, 3).flatten(2)[..., None]
    lse = torch.where(real.repeat_interleave(c["Hq"] // c["Hkv"], 1)[:, None, :, None], lse, torch.zeros_like(lse))
    s["weights"] += torch.exp(sc - lse).sum(-2)
    return s["weights"]


def _write_plain(s):
    c, dev = s["case"], s["k"].device
    S, D, cap = c["S"], c["D"], s["table"].shape[1]
    lens, start = s["lens"].long()[:, None], s["start"].long()[:, None]
    new = (s["cu"][1:] - s["cu"][:-1]).long()[:, None]
    slot = torch.arange(cap * BLOCK, device=dev)[None]
    fresh = (slot >= start) & (slot < start + new)  # [S, slots]
    token = (s["cu"][:-1].long()[:, None] + slot - start).clamp(0, s["k_new"].shape[0] - 1)
    held = (slot < lens) & ~fresh
    touched = fresh.unflatten(1, (cap, BLOCK)).any(-1)[..., None]  # [S, cap, 1]
    table = s["table"].long()
    for name, x, gain in (("k", s["k_new"], ROOT2), ("v", s["v_new"], 1.0)):
        tok, blk = (_tokens_k, _blocks_k) if name == "k" else (_tokens_v, _blocks_v)
        sc, y = s[name + "_scale"], _rotate(x, s["pos"], c) if name == "k" else x.float()
        big = x.float().abs().amax(-1)[token].masked_fill(~fresh[..., None], 0)  # [S, slots, H]
        big = big.unflatten(1, (cap, BLOCK)).amax(2) * torch.tensor(gain, device=dev)
        m, e = torch.frexp(big)  # big = m 2^e, 0.5 <= m < 1; 448 = 0.875 2^9
        want = torch.where(big > 0, e.long() - 9 + (m > 0.875), torch.full_like(e.long(), -127)) + 127
        kept = torch.where(held.unflatten(1, (cap, BLOCK)).any(-1)[..., None], sc[table].long(), torch.zeros_like(want))
        byte = torch.maximum(want, kept).clamp(LOWEST, HIGHEST)  # [S, cap, H]
        old = _value(tok(s[name][table], D)) * torch.exp2((sc[table].long() - byte).double()).float()[..., None, None]
        put = y[token].unflatten(1, (cap, BLOCK)).transpose(2, 3) * torch.exp2((127 - byte).double()).float()[..., None, None]
        at = lambda mask: mask.unflatten(1, (cap, BLOCK))[:, :, None, :, None]  # noqa: E731
        z = torch.where(at(fresh), put, torch.where(at(held), old, torch.zeros_like(old)))
        z = blk(z.to(torch.float8_e4m3fn).view(torch.uint8))
        s[name][table] = torch.where(touched[..., None], z, s[name][table])
        sc[table] = torch.where(touched, byte, sc[table].long()).to(torch.uint8)
    return _cache_of(s)


def _cache_of(s):
    f8 = torch.float8_e4m3fn
    return {"k": s["k"].view(f8), "v": s["v"].view(f8), "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _evict_plain(s):
    c, dev = s["case"], s["k"].device
    S, H, D, keep, w = c["S"], c["Hkv"], c["D"], c["keep"], s["weights"]
    slots, out_slots = w.shape[2], s["weights_out"].shape[2]
    slot = torch.arange(slots, device=dev)
    lens = s["lens"].long()[:, None, None]
    n = torch.minimum(lens, torch.full_like(lens, keep))
    first = n.clamp(max=c["sink"])
    last = (n - first).clamp(max=c["recent"])
    pooled = torch.where(slot < lens, w, torch.full_like(w, -math.inf))
    pooled = torch.nn.functional.pad(pooled, (c["pool"] // 2, c["pool"] // 2), value=-math.inf).unfold(-1, c["pool"], 1).amax(-1)
    pooled = torch.where((slot < first) | ((slot >= lens - last) & (slot < lens)), torch.full_like(pooled, math.inf), pooled)
    pooled = torch.where(slot < lens, pooled, torch.full_like(pooled, -math.inf))
    best = torch.sort(pooled, dim=-1, descending=True, stable=True)[1][..., :keep]
    ok = torch.arange(best.shape[-1], device=dev) < n
    kept = torch.sort(torch.where(ok, best, torch.full_like(best, slots)), dim=-1)[0]  # ascending, the unused behind
    kept = torch.nn.functional.pad(kept, (0, out_slots - kept.shape[-1]), value=slots)
    real = kept < slots
    src = kept.clamp(max=slots - 1)
    s["lens_out"].copy_(n[:, 0, 0])
    s["kept"].copy_(torch.where(real, kept, torch.full_like(kept, -1))[..., :keep])
    s["weights_out"].copy_(torch.where(real, torch.gather(w, 2, src), torch.zeros_like(s["weights_out"])))
    page = torch.gather(s["table"].long()[:, None].expand(S, H, -1), 2, src // BLOCK)  # [S, H, out_slots]
    head = torch.arange(H, device=dev)[None, :, None]
    used = (slot[: out_slots: BLOCK] < n)[:, 0, :, None]  # [S, cap_out, 1]
    to = s["table_out"].long()
    for name in "kv":
        tok, blk = (_tokens_k, _blocks_k) if name == "k" else (_tokens_v, _blocks_v)
        x = _value(tok(s[name], D)[page, head, src % BLOCK])  # [S, H, out_slots, D]
        e = torch.where(real, s[name + "_scale"][page, head].long(), torch.zeros_like(src))
        byte = e.unflatten(2, (-1, BLOCK)).amax(-1)  # [S, H, cap_out]
        z = (x * torch.exp2((e - byte.repeat_interleave(BLOCK, 2)).double()).float()[..., None]).masked_fill(~real[..., None], 0)
        z = blk(z.to(torch.float8_e4m3fn).view(torch.uint8).unflatten(2, (-1, BLOCK))).transpose(1, 2)
        s[name][to] = torch.where(used[..., None], z, s[name][to])
        s[name + "_scale"][to] = torch.where(used, byte.transpose(1, 2).to(torch.uint8), s[name + "_scale"][to])
    return {**_cache_of(s), "lens": s["lens_out"], "kept": s["kept"], "weights": s["weights_out"]}


# ---- one pass -------------------------------------------------------------------------------------------------

def _handles(s):
    """What a program makes once for its cache, batch and rotary positions."""
    import masked_token_logits_amd as mtl
    c = s["case"]
    if "r" in c:
        more = dict(original_len=4096) if c.get("scaling") == "ramp" else {}
        s["rotary"] = mtl.Rotary(c["D"], c["r"], layout=c["layout"], scaling=c.get("scaling", "none"), factor=c.get("factor", 1.0), **more)
    if "k" in s:
        s["cache"] = mtl.BlockCache.over(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["batch"] = s["cache"].batch(s["cu"], s["lens"], s["table"], max_new=max(1, *s["new_host"]), max_len=max(s["lens_host"]))
    s["ready"] = True


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        if "ready" not in s:
            _handles(s)
        if op == "rotary":
            return s["rotary"](s["x"], s["pos"])
        if op == "write":
            s["cache"].write(s["batch"], s["k_new"], s["v_new"], s["start"], positions=s["pos"], rotary=s["rotary"])
            return _cache_of(s)
        if op == "attend":
            return s["cache"].attend(s["batch"], s["q"], causal=bool(c["causal"]), lse=True)
        if op == "weigh":
            s["cache"].weigh(s["batch"], s["q"], s["lse"], s["weights"], causal=bool(c["causal"]))
            return s["weights"]
        s["cache"].evict(s["batch"], s["weights"], s["keep"], s["table_out"], sink=c["sink"], recent=c["recent"],
                         pool=c["pool"], lens_out=s["lens_out"], weights_out=s["weights_out"], kept=s["kept"])
        return {**_cache_of(s), "lens": s["lens_out"], "kept": s["kept"], "weights": s["weights_out"]}
    if op == "rotary":
        return _rotate(s["x"], s["pos"], c).to(torch.bfloat16)
    return {"write": _write_plain, "attend": _attend_plain, "weigh": _weigh_plain, "evict": _evict_plain}[op](s)


def _pairs(lens, new, causal):
    """Query-key pairs that are not masked."""
    if not causal:
        return sum(a * b for a, b in zip(lens, new))
    return sum(sum(max(0, a - b + i + 1) for i in range(b)) for a, b in zip(lens, new))


def work(case):
    D, op = case["D"], case["op"]
    if op == "rotary":
        T, H = case["T"], case["H"]
        return {"bytes": 4 * T * H * D + 4 * T, "flops": 3 * T * H * case["r"]}
    lens, new = _counts(case)
    H, T = case["Hkv"], sum(new)
    if op == "write":
        held = sum(min(BLOCK, (a - b) % BLOCK) for a, b in zip(lens, new))  # tokens beside the new ones in the first block
        return {"bytes": 2 * H * D * (3 * T + held) + 8 * T, "flops": H * D * (6 * T)}
    if op == "evict":
        kept = sum(min(a, case["keep"]) for a in lens)
        return {"bytes": 4 * H * sum(lens) + H * kept * (4 * D + 8), "flops": H * sum(lens) * case["pool"]}
    pairs, Hq = _pairs(lens, new, case["causal"]), case["Hq"]
    if op == "weigh":
        return {"bytes": H * sum(lens) * (D + 8) + T * Hq * (2 * D + 4), "flops": 2 * pairs * Hq * D}
    return {"bytes": 2 * H * sum(lens) * D + T * Hq * (4 * D + 4), "flops": 4 * pairs * Hq * D}


# ---- the definitions in 64 bits, apart from the plain forms ----------------------------------------------------

def _e4m3(dev):
    """The value of each of the 256 bytes, from the format's definition (sign, 4 exponent bits of bias 7, 3 bits)."""
    b = torch.arange(256, device=dev)
    e, m, sign = (b >> 3) & 15, (b & 7).double(), 1.0 - 2.0 * (b >> 7).double()
    v = torch.where(e == 0, m / 512, (1 + m / 8) * torch.exp2((e - 7).double()))
    return torch.where((b & 127) == 127, torch.full_like(v, math.nan), sign * v)


def _places(D, dev, key):
    """Where in a block [32 D] the value of token t and dimension d stands: [32, D]."""
    t, d = torch.arange(32, device=dev)[:, None], torch.arange(D, device=dev)[None]
    if key:
        return ((d % (D // 2)) // 16 * 2 + d // (D // 2)) * 512 + t * 16 + d % 16
    return (d // 32 * 2 + (t // 4) % 2) * 512 + (d % 32) * 16 + (t // 8) * 4 + t % 4


def _read64(s, name, seq, head, n, table="table"):
    """n tokens of one sequence and head in 64 bits [n, D]."""
    D, dev = s["case"]["D"], s[name].device
    pages = s[table][seq, : (n + 31) // 32].long()
    x = _e4m3(dev)[s[name][pages, head].long()][:, _places(D, dev, name == "k")]
    return (x * torch.exp2(s[name + "_scale"][pages, head].double() - 127)[:, None, None]).reshape(-1, D)[:n]


def _rotated64(x, pos, case):
    """Rotation as a product of complex numbers."""
    r, mag = case["r"], 1.0
    i = torch.arange(r // 2, dtype=torch.float64, device=x.device)
    f, scaling = case.get("factor", 1.0), case.get("scaling", "none")
    base = 10000.0 * (f ** (r / (r - 2)) if scaling == "base" else 1.0)
    theta = torch.exp(-2 * i / r * math.log(base)) / (f if scaling == "linear" else 1.0)
    if scaling == "ramp":
        share = torch.clamp((4096 * theta / (2 * math.pi) - 1) / 31, 0, 1)
        theta, mag = share * theta + (1 - share) * theta / f, 1 + 0.1 * math.log(f)
    first, second = (torch.arange(r // 2), torch.arange(r // 2) + r // 2) if case["layout"] == "half" else (2 * torch.arange(r // 2), 2 * torch.arange(r // 2) + 1)
    x = x.double()
    turn = torch.polar(torch.full_like(theta, mag).expand(len(pos), -1).contiguous(), pos.double()[:, None] * theta)
    z = torch.complex(x[..., first], x[..., second]) * turn[:, None]
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _nearest_e4m3(x):
    """The e4m3 value nearest to each x (|x| <= 448), ties to the even code, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    op, D, dev = case["op"], case["D"], s["x"].device if "x" in s else s["k"].device
    if op == "rotary":
        return _rotated64(s["x"], s["pos"], case)
    lens, new = s["lens_host"], s["new_host"]
    if op in ("attend", "weigh"):
        group = case["Hq"] // case["Hkv"]
        out = torch.zeros(sum(new), case["Hq"], D, dtype=torch.float64, device=dev)
        lse = torch.full((sum(new), case["Hq"]), -math.inf, dtype=torch.float64, device=dev)
        weights = s["weights"].double() if op == "weigh" else None
        at = 0
        for b, (length, n) in enumerate(zip(lens, new)):
            for h in range(case["Hkv"]):
                k = _read64(s, "k", b, h, length)
                v = _read64(s, "v", b, h, length) if op == "attend" else None
                for i in range(h * group, (h + 1) * group):
                    z = s["q"][at: at + n, i].double() @ k.T / math.sqrt(D)
                    if case["causal"]:
                        z += torch.full_like(z, -math.inf).triu(length - n + 1)
                    if op == "weigh":
                        weights[b, h, :length] += torch.exp(z - s["lse"][at: at + n, i].double()[:, None]).sum(0)
                    else:
                        lse[at: at + n, i] = torch.logsumexp(z, 1)
                        out[at: at + n, i] = torch.softmax(z, 1) @ v
            at += n
        return weights if op == "weigh" else (out, lse)
    if op == "evict":
        return _evicted64(s)
    held = {"k_scale": None, "v_scale": None}  # whole numbers
    for name, y, gain in (("k", _rotated64(s["k_new"], s["pos"], case), ROOT2), ("v", s["v_new"].double(), 1.0)):
        pool, x, at = _e4m3(dev)[s[name].long()], s[name + "_new"], 0
        for b, (length, n) in enumerate(zip(lens, new)):
            begin, first = length - n, (length - n) // 32
            blocks, stay = (length + 31) // 32 - first, begin - 32 * first  # `stay` tokens of the first block are not new
            pages = s["table"][b, first: first + blocks].long()
            rows = torch.zeros(blocks * 32, case["Hkv"], D, dtype=torch.float64, device=dev)
            rows[stay: stay + n] = y[at: at + n]
            size = torch.zeros(blocks * 32, case["Hkv"], dtype=torch.float64, device=dev)
            size[stay: stay + n] = x[at: at + n].double().abs().amax(-1) * gain
            need = torch.ceil(torch.log2(size.view(blocks, 32, -1).amax(1).clamp(min=2.0 ** -80) / 448)) + 127  # [blocks, H]
            if stay:
                had = s[name + "_scale"][pages[0]].double()
                need[0] = torch.maximum(need[0], had)
                old = _e4m3(dev)[s[name][pages[0]].long()][:, _places(D, dev, name == "k")] * torch.exp2(had - 127)[:, None, None]
                rows[:stay] = old[:, :stay].transpose(0, 1)
            z = _nearest_e4m3(rows.view(blocks, 32, -1, D) * torch.exp2(127 - need)[:, None, :, None]).transpose(1, 2)
            pool[pages[:, None, None, None], torch.arange(case["Hkv"], device=dev)[None, :, None, None], _places(D, dev, name == "k")] = z
            at += n
        held[name] = pool
    return held


def _evicted64(s):
    """The pool after an eviction and the kept weights, one sequence and head at a time."""
    case, D, dev = s["case"], s["case"]["D"], s["k"].device
    pool = {name: _e4m3(dev)[s[name].long()] for name in "kv"}
    weights = torch.zeros_like(s["weights_out"], dtype=torch.float64)
    for b, length in enumerate(s["lens_host"]):
        n = min(case["keep"], length)
        first = min(case["sink"], n)
        last = min(case["recent"], n - first)
        blocks = (n + 31) // 32
        for h in range(case["Hkv"]):
            w = s["weights"][b, h, :length]
            around = w.clone()
            for d in range(1, case["pool"] // 2 + 1):
                around[d:] = torch.maximum(around[d:], w[: max(0, length - d)])
                around[: max(0, length - d)] = torch.maximum(around[: max(0, length - d)], w[d:])
            middle = torch.sort(around[first: length - last], descending=True, stable=True)[1][: n - first - last] + first
            keep = torch.zeros(length, dtype=torch.bool, device=dev)
            keep[:first], keep[length - last:], keep[middle] = True, True, True
            at = torch.nonzero(keep)[:, 0]
            weights[b, h, :n] = w[at].double()
            page = s["table"][b].long()[at // 32]
            to = s["table_out"][b, :blocks].long()
            for name in "kv":
                x = torch.zeros(blocks * 32, D, dtype=torch.float64, device=dev)
                x[:n] = _read64(s, name, b, h, length)[at]
                e = torch.zeros(blocks * 32, dtype=torch.float64, device=dev)
                e[:n] = s[name + "_scale"][page, h].double()
                z = _nearest_e4m3(x.view(blocks, 32, D) * torch.exp2(127 - e.view(blocks, 32).amax(1))[:, None, None])
                pool[name][to[:, None, None], h, _places(D, dev, name == "k")] = z
    return {"k": pool["k"], "v": pool["v"], "k_scale": None, "v_scale": None, "lens": None, "kept": None, "weights": weights}
