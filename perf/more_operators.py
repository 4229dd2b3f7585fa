"""The operators at the two ends of a masked diffusion model and between its blocks, as cases that can be timed and
compared: the cross entropy of masked positions over the whole vocabulary with its gradients, the embedding lookup with
its gradient, and the residual update with the norms around a block, with its gradients.

``run`` computes them in plain torch (``own`` false) or through the package's public entry points (``own`` true)."""
import math

import torch

own = False

EPS = 1e-5


def listed():
    return [
        # likelihood of a short sequence: the smallest call of the loss, where only latency counts
        dict(name="score short", op="score", L=512, d=256, V=4096, ratio=0.5, weighted=0, ignored=0),
        # likelihood of a long, mostly masked sequence
        dict(name="score long", op="score", L=8192, d=4096, V=126464, ratio=0.9, weighted=1, ignored=1),
        # a training step's loss and gradients at low mask ratio: few rows against the whole head
        dict(name="train few", op="train", L=1024, d=4096, V=126464, ratio=0.1, weighted=1, ignored=0),
        # the same at the mean mask ratio of a batch, with padded targets
        dict(name="train many", op="train", L=8192, d=3584, V=152064, ratio=0.5, weighted=1, ignored=1),
        # the tokens of one 32-token decoding block: the smallest call of all
        dict(name="lookup block", op="lookup", T=32, d=4096, V=126464, scaled=0, masked=0.5),
        # a long context's tokens, scaled by the root of the hidden size
        dict(name="lookup prompt", op="lookup", T=131072, d=4096, V=126464, scaled=1, masked=0.5),
        # the table's gradient from a short, odd batch
        dict(name="lookup grad short", op="scatter", T=509, d=256, V=4096, scaled=1, masked=0.3),
        # the table's gradient of a training batch: half of its tokens are the mask token
        dict(name="lookup grad long", op="scatter", T=65536, d=4096, V=126464, scaled=0, masked=0.5),
        # one decoding block between two layers: a plain residual update and the next norm
        dict(name="norm block", op="norm", T=32, d=4096, post=0, groups=0, scale=1.0),
        # a long batch with a norm behind the block, a gate for each of 8 sequences and a residual scale
        dict(name="norm long", op="norm", T=65536, d=3584, post=1, groups=8, scale=0.5),
        # gradients of the plain update, odd number of tokens
        dict(name="norm grad short", op="norm grad", T=509, d=4096, post=0, groups=0, scale=1.0),
        # gradients of the update with everything in it
        dict(name="norm grad long", op="norm grad", T=32768, d=3584, post=1, groups=4, scale=0.5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["score", "train", "train", "lookup", "scatter", "norm", "norm grad"])
    d = 8 * _log(rng, 8, 512) if rng.random() < 0.5 else rng.choice([256, 512, 1024, 2048, 3584, 4096])
    if op in ("score", "train"):
        V, ratio = _log(rng, 50, 152064), rng.choice([0.0, 0.1, 0.5, 0.9, 1.0, rng.random()])
        most = 4096 * 3584 * 152064 // (1 if op == "train" else 2)
        L = _log(rng, 1, max(1, min(16384, int(most / (V * d * max(ratio, 0.25))))))
        return dict(op=op, L=L, d=d, V=V, ratio=ratio, weighted=rng.randint(0, 1), ignored=rng.randint(0, 1))
    if op in ("lookup", "scatter"):
        return dict(op=op, T=_log(rng, 1, 65536), d=d, V=_log(rng, 50, 152064), scaled=rng.randint(0, 1),
                    masked=rng.choice([0.0, 0.1, 0.5, 0.9, 1.0]))
    groups = rng.choice([0, 1, _log(rng, 2, 64), -1])  # no gate, one, one a sequence, one a token
    rows = _log(rng, 1, 32768 // max(groups, 1))
    T = rows * max(groups, 1)
    return dict(op=op, T=T, d=d, post=rng.randint(0, 1), groups=T if groups < 0 else groups, scale=rng.choice([1.0, 0.5, 0.1]))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rnd = lambda *shape: torch.randn(*shape, generator=g, device=dev)  # noqa: E731
    uni = lambda *shape: torch.rand(*shape, generator=g, device=dev)  # noqa: E731
    bf = lambda x: x.to(torch.bfloat16)  # noqa: E731
    s, op, d = dict(case=case), case["op"], case["d"]
    if op in ("score", "train"):
        L, V = case["L"], case["V"]
        W = s["W"] = torch.randn(V, d, generator=g, device=dev, dtype=torch.bfloat16).mul_(0.02 * math.sqrt(4096 / d))
        t = (uni(L) * V).long().clamp(max=V - 1)
        w = W[t].float()
        # hidden states of a partly trained model: each leans towards its target, from not at all to almost surely
        s["hidden"] = bf(rnd(L, d) + w * (16 * uni(L, 1) / w.square().sum(-1, keepdim=True).clamp(min=1e-3)))
        s["mask"] = (uni(L) < case["ratio"]).to(torch.uint8)
        if case["ignored"]:
            t = torch.where(uni(L) < 0.05, torch.full_like(t, -100), t)
        s["targets"] = t.to(torch.int32)
        # each token counts by the inverse of the ratio that its sequence was masked with
        s["weights"] = 1.0 / (L * (0.1 + 0.9 * uni(L))) if case["weighted"] else None
        s["grad"] = torch.full((1,), 1.0 + 1023.0 * case["weighted"], device=dev)  # the scale of the loss
        return s
    if op in ("lookup", "scatter"):
        T, V = case["T"], case["V"]
        tok = torch.exp(uni(T) * math.log(V)).long().clamp(max=V) - 1  # a few tokens are frequent, most are rare
        tok = torch.randperm(V, generator=g, device=dev)[tok]
        s["tokens"] = torch.where(uni(T) < case["masked"], torch.full_like(tok, V - 1), tok).to(torch.int32)
        s["scale"] = math.sqrt(d) if case["scaled"] else 1.0
        if op == "lookup":
            s["table"] = torch.randn(V, d, generator=g, device=dev, dtype=torch.bfloat16)
        else:
            s["table"] = torch.empty(V, d, device=dev, dtype=torch.bfloat16)
            s["d_out"] = bf(rnd(T, d) * torch.exp(rnd(T, 1)))
        return s
    T = case["T"]
    x = rnd(T, d) * torch.exp(0.5 * rnd(T, 1)) * 4
    x[:, : max(1, d // 512)] *= 30  # a residual stream has a few loud channels
    s["x"], s["y"] = bf(x), bf(rnd(T, d) * torch.exp(0.5 * rnd(T, 1)))
    s["pre"] = bf(1 + 0.1 * rnd(d))
    s["post"] = bf(1 + 0.1 * rnd(d)) if case["post"] else None
    s["gate"] = bf(0.5 * rnd(case["groups"], d)) if case["groups"] else None
    if op == "norm grad":
        s["d_n"], s["d_x"] = bf(rnd(T, d)), bf(rnd(T, d))
    return s


# ---- plain forms ----------------------------------------------------------------------------------------------

def _loss_plain(s):
    hidden, mask, targets, W = s["hidden"], s["mask"], s["targets"].long(), s["W"].float()
    V, L = W.shape[0], mask.shape[0]
    at = torch.nonzero((mask != 0) & (targets >= 0) & (targets < V))[:, 0]
    h, t = hidden[at].float(), targets[at]
    w = s["weights"][at] if s["weights"] is not None else torch.ones_like(at, dtype=torch.float32)
    z = h @ W.T
    top = z.amax(-1, keepdim=True)
    lse = (top + torch.log(torch.exp(z - top).sum(-1, keepdim=True)))[:, 0]
    row = lse - z.gather(1, t[:, None])[:, 0]
    full = lambda v: torch.zeros(L, device=v.device).index_put((at,), v)  # noqa: E731
    out = {"loss": (row * w).double().sum().float()[None], "losses": full(row), "lse": full(lse)}
    if s["case"]["op"] == "train":
        p = torch.exp(z - lse[:, None])
        del z
        p[torch.arange(len(at), device=p.device), t] -= 1
        p *= (w * s["grad"])[:, None]
        out["d_W"] = (p.T @ h).to(torch.bfloat16)
        out["d_hidden"] = torch.zeros_like(hidden).index_put((at,), (p @ W).to(torch.bfloat16))
    return out


def _norm_plain(s):
    c = s["case"]
    x, y = s["x"].float(), s["y"].float()
    u = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * s["post"].float() if c["post"] else y
    if c["groups"]:
        u = (u.view(c["groups"], -1, c["d"]) * s["gate"].float()[:, None]).view_as(u)
    x = x + c["scale"] * u
    n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["pre"].float()
    return {"x": x.to(torch.bfloat16), "n": n.to(torch.bfloat16)}


def _norm_grad_plain(s):
    c = s["case"]
    x, y, dn, pre = s["x"].float(), s["y"].float(), s["d_n"].float(), s["pre"].float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    dnw = dn * pre
    dx = s["d_x"].float() + r * (dnw - x * (r * r) * (dnw * x).mean(-1, keepdim=True))
    out = {"d_x": dx.to(torch.bfloat16), "d_pre": (dn * x * r).double().sum(0).float()}
    q = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) if c["post"] else None
    u = y * q * s["post"].float() if c["post"] else y
    du = c["scale"] * dx
    if c["groups"]:
        out["d_gate"] = (du * u).view(c["groups"], -1, c["d"]).double().sum(1).float()
        du = (du.view(c["groups"], -1, c["d"]) * s["gate"].float()[:, None]).view_as(du)
    if c["post"]:
        out["d_post"] = (du * y * q).double().sum(0).float()
        duw = du * s["post"].float()
        du = q * (duw - y * (q * q) * (duw * y).mean(-1, keepdim=True))
    out["d_y"] = du.to(torch.bfloat16)
    return out


def _lookup_plain(s):
    return (s["table"][s["tokens"].long()].float() * s["scale"]).to(torch.bfloat16)


def _scatter_plain(s):
    sums = torch.zeros(s["table"].shape, device=s["table"].device)
    sums.index_add_(0, s["tokens"].long(), s["d_out"].float())
    return (sums * s["scale"]).to(torch.bfloat16)


# ---- one pass -------------------------------------------------------------------------------------------------

def _handles(s):
    """What a program makes once for its head, table and norms."""
    import masked_token_logits_amd as mtl
    c = s["case"]
    if c["op"] in ("score", "train"):
        s["head"] = mtl.MaskedLoss(s["W"])
    elif c["op"] in ("lookup", "scatter"):
        s["embedding"] = mtl.Embedding(s["table"], scale=s["scale"])
    else:
        s["layer"] = mtl.ResidualNorm(pre=s["pre"], post=s["post"], eps=EPS, scale=c["scale"])
    s["ready"] = True


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        if "ready" not in s:
            _handles(s)
        if op in ("score", "train"):
            loss, losses, lse = s["head"](s["hidden"], s["mask"], s["targets"], weights=s["weights"])
            out = {"loss": loss, "losses": losses, "lse": lse}
            if op == "train":
                out["d_hidden"], out["d_W"] = s["head"].backward(s["hidden"], s["mask"], s["targets"], lse,
                                                                 weights=s["weights"], grad=s["grad"])
            return out
        if op == "lookup":
            return s["embedding"](s["tokens"])
        if op == "scatter":
            return s["embedding"].backward(s["tokens"], s["d_out"])
        if op == "norm":
            x, n = s["layer"](s["x"], s["y"], gate=s["gate"])
            return {"x": x, "n": n}
        got = s["layer"].backward(s["x"], s["d_n"], y=s["y"], d_x=s["d_x"], gate=s["gate"])
        return {k: v for k, v in got.items() if v is not None}
    plain = {"score": _loss_plain, "train": _loss_plain, "lookup": _lookup_plain, "scatter": _scatter_plain,
             "norm": _norm_plain, "norm grad": _norm_grad_plain}
    return plain[op](s)


def _rows(case):
    """Masked rows with a target, as many as are expected."""
    return case["L"] * case["ratio"] * (0.95 if case["ignored"] else 1.0)


def work(case):
    op, d = case["op"], case["d"]
    if op in ("score", "train"):
        M, L, V = _rows(case), case["L"], case["V"]
        read = 2 * V * d + 2 * M * d + L * (5 + 4 * case["weighted"])
        if op == "score":
            return {"bytes": read + 8 * L, "flops": 2 * M * V * d}
        # the logits are not kept: their product, and one for each gradient; both gradients are written whole
        return {"bytes": read + 8 * L + 2 * V * d + 2 * L * d, "flops": 6 * M * V * d}
    if op == "lookup":
        known = min(case["V"], case["T"])  # rows of the table that are read, at most
        return {"bytes": 4 * case["T"] + 2 * d * (case["T"] + known), "flops": case["T"] * d}
    if op == "scatter":
        return {"bytes": 4 * case["T"] + 2 * d * (case["T"] + case["V"]), "flops": 2 * case["T"] * d}
    T, G = case["T"], case["groups"]
    if op == "norm":
        return {"bytes": 2 * d * (4 * T + 1 + case["post"] + G), "flops": T * d * (8 + 4 * case["post"])}
    return {"bytes": 2 * d * (6 * T + 1 + case["post"] + G) + 4 * d * (1 + case["post"] + G), "flops": T * d * (16 + 10 * case["post"])}


# ---- the definitions in 64 bits, apart from the plain forms ----------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op, d, dev = case["op"], case["d"], torch.device("cuda")
    if op in ("score", "train"):
        return _loss64(s)
    if op == "lookup":
        return torch.index_select(s["table"], 0, s["tokens"].long()).double().mul_(s["scale"])
    if op == "scatter":
        # runs of equal tokens in sorted order, as differences of running sums
        tok, order = torch.sort(s["tokens"].long(), stable=True)
        run = torch.cat([torch.zeros(1, d, dtype=torch.float64, device=dev), torch.cumsum(s["d_out"].double()[order], 0)])
        ids, count = torch.unique_consecutive(tok, return_counts=True)
        end = torch.cumsum(count, 0)
        out = torch.zeros(case["V"], d, dtype=torch.float64, device=dev)
        out[ids] = (run[end] - run[end - count]) * s["scale"]
        return out
    T, G = case["T"], case["groups"]
    wide = {k: s[k].double() for k in ("x", "y", "pre", "post", "gate", "d_n", "d_x") if s.get(k) is not None}
    norm = lambda v, w: w * v / torch.sqrt((v * v).sum(1, keepdim=True) / d + EPS)  # noqa: E731
    names = ["y", "pre"] + [k for k in ("post", "gate") if k in wide]

    def branch():
        u = norm(wide["y"], wide["post"]) if case["post"] else wide["y"]
        return case["scale"] * u * (torch.repeat_interleave(wide["gate"], T // G, 0) if G else 1.0)

    if op == "norm":
        x = wide["x"] + branch()
        return {"x": x, "n": norm(x, wide["pre"])}
    base = wide["x"] - branch()  # the stream before the update: x is the one behind it
    leaves = [base.requires_grad_()] + [wide[k].requires_grad_() for k in names]
    x = base + branch()
    got = torch.autograd.grad((norm(x, wide["pre"]) * wide["d_n"]).sum() + (x * wide["d_x"]).sum(), leaves)
    return {"d_" + k: v for k, v in zip(["x"] + names, got)}


def _loss64(s):
    case, V, L, d = s["case"], s["case"]["V"], s["case"]["L"], s["case"]["d"]
    dev, piece = s["W"].device, 16384
    t = s["targets"].long()
    at = torch.where((s["mask"] > 0) & (t >= 0) & (t < V))[0]
    h, t = s["hidden"].index_select(0, at).double(), t[at]
    w = s["weights"].double()[at] if s["weights"] is not None else torch.ones(len(at), dtype=torch.float64, device=dev)
    lse = torch.full((len(at),), -math.inf, dtype=torch.float64, device=dev)
    for v in range(0, V, piece):
        lse = torch.logaddexp(lse, torch.logsumexp(h @ s["W"][v: v + piece].double().T, 1))
    row = lse - (h * s["W"][t].double()).sum(1)
    whole = lambda v: torch.zeros(L, dtype=torch.float64, device=dev).index_copy_(0, at, v)  # noqa: E731
    out = {"loss": torch.dot(row, w)[None], "losses": whole(row), "lse": whole(lse)}
    if case["op"] == "train":
        coef, dh = w * s["grad"].double(), torch.zeros_like(h)
        dW = torch.empty(V, d, dtype=torch.float64, device=dev)
        for v in range(0, V, piece):
            part = s["W"][v: v + piece].double()
            p = torch.exp(h @ part.T - lse[:, None]) - (t[:, None] == torch.arange(v, v + len(part), device=dev)).double()
            p = coef[:, None] * p
            dh += p @ part
            dW[v: v + piece] = p.T @ h
        out["d_hidden"] = torch.zeros(L, d, dtype=torch.float64, device=dev).index_copy_(0, at, dh)
        out["d_W"] = dW
    return out
