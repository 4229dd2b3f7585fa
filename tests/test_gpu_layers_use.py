"""The loss, the embedding and the residual norm together, as a training step
and a denoising step of a small masked diffusion model use them: rows looked
up, residual updates around the framework's FFN, the last norm, the loss of the
masked positions, and the gradients back to every weight; and the same head in
readout and loss."""
import numpy as np
import pytest
import torch

import masked_token_logits_amd as mtl
from _layer_cases import dev_bf16, dev_i32, replayed

pytestmark = pytest.mark.gpu

EPS = 1e-5


def _model(seed, V=700, d=256, L=300):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
    m = dict(table=rnd(V, d), post=1 + rnd(d, std=0.1), pre=1 + rnd(d, std=0.1), last=1 + rnd(d, std=0.1),
             gate=rnd(3, d, std=0.5), block=rnd(d, d, std=d ** -0.5), head=rnd(V, d, std=2 * d ** -0.5))
    tokens = torch.randint(0, V - 1, (L,), generator=g, device="cuda", dtype=torch.int32)
    mask = (torch.rand(L, generator=g, device="cuda") < 0.5).to(torch.uint8)
    seen = torch.where(mask != 0, torch.full_like(tokens, V - 1), tokens)     # V - 1 is the mask token
    weights = torch.rand(L, generator=g, device="cuda") / L
    return m, tokens, seen, mask, weights


def _step(m, tokens, seen, mask, weights, scale=0.5):
    """One training step: the loss and the gradient of every weight.  The block
    between the norms is a matrix, in torch."""
    emb = mtl.Embedding(m["table"], scale=2.0)
    layer = mtl.ResidualNorm(pre=m["last"], post=m["post"], eps=EPS, scale=scale)
    first = mtl.ResidualNorm(pre=m["pre"], eps=EPS)
    head = mtl.MaskedLoss(m["head"], piece=256)
    x = emb(seen)
    _, n = first(x)
    y = n @ m["block"]
    x1, h = layer(x, y, gate=m["gate"])
    loss, losses, lse = head(h, mask, tokens, weights=weights)
    d_h, d_head = head.backward(h, mask, tokens, lse, weights=weights)
    g = layer.backward(x1, d_h, y=y, gate=m["gate"])
    d_y = g["d_y"]
    d_n = d_y @ m["block"].t().contiguous()
    g0 = first.backward(x, d_n, d_x=g["d_x"])
    d_table = emb.backward(seen, g0["d_x"])
    return dict(loss=loss, head=d_head, last=g["d_pre"], post=g["d_post"], gate=g["d_gate"],
                block=n.t().contiguous() @ d_y, pre=g0["d_pre"], table=d_table)


def _reference(m, tokens, seen, mask, weights, scale=0.5):
    """The same in fp64 by torch's autograd, on the CPU."""
    w = {k: v.double().cpu().requires_grad_() for k, v in m.items()}
    seen, tokens, keep = seen.cpu().long(), tokens.cpu().long(), mask.cpu() != 0
    norm = lambda v, s: s * v * torch.rsqrt(v.pow(2).mean(1, keepdim=True) + EPS)  # noqa: E731
    x = 2.0 * w["table"][seen]
    y = norm(x, w["pre"]) @ w["block"]
    x = x + scale * torch.repeat_interleave(w["gate"], len(seen) // 3, 0) * norm(y, w["post"])
    h = norm(x, w["last"])
    ce = torch.nn.functional.cross_entropy((h @ w["head"].T)[keep], tokens[keep], reduction="none")
    loss = (ce * weights.cpu().double()[keep]).sum()
    loss.backward()
    return dict(loss=loss.detach()[None], **{k: v.grad for k, v in w.items()})


def test_training_step_against_autograd():
    """A handful of tensors are rounded to bf16 on the way, each off by up to
    2^-9 of itself on average less than half of that, and the gradients pass
    through at most six of them: in the 2-norm 6 * 2^-9 of the gradient."""
    args = _model(1)
    got, want = _step(*args), _reference(*args)
    for k, w in want.items():
        off = (got[k].double().cpu() - w).norm() / w.norm()
        assert off <= (2.0 ** -9 if k == "loss" else 6 * 2.0 ** -9), (k, off.item())


def test_training_step_captured():
    sets = [_model(s) for s in (2, 3, 4)]
    m, *rest = sets[0]
    m, rest = {k: v.clone() for k, v in m.items()}, [t.clone() for t in rest]

    def refill(i):
        for k, v in sets[i][0].items():
            m[k].copy_(v)
        for a, b in zip(rest, sets[i][1:]):
            a.copy_(b)

    # the two products of the block are torch's; the rest is captured with them
    def call():
        return list(_step(m, *rest).values())

    def check(i, got, eager):
        assert all(torch.equal(a, b) for a, b in zip(got, eager))

    replayed(call, check, refill)


def test_tied_table_takes_both_gradients():
    """A table that is also the head: the head's gradient first, the lookup's on top."""
    V, d, L = 500, 128, 200
    m, tokens, seen, mask, weights = _model(5, V, d, L)
    head, emb = mtl.MaskedLoss(m["head"]), mtl.Embedding(m["head"])
    h = m["table"][:L].contiguous()
    lse = head(h, mask, tokens, weights=weights)[2]
    _, d_head = head.backward(h, mask, tokens, lse, weights=weights, need=("W",))
    d_out = (m["table"][:L] * 0.01).contiguous()
    alone = emb.backward(seen, d_out)
    both = emb.backward(seen, d_out, d_table=d_head.clone(), accumulate=True)
    hit = torch.zeros(V, dtype=torch.bool, device="cuda")
    hit[seen.long()] = True
    assert torch.equal(both[~hit], d_head[~hit])
    want = d_head.double() + alone.double()
    # one rounding here, one in `alone`
    assert ((both.double() - want).abs() <= 2.0 ** -8 * (want.abs() + alone.double().abs()))[hit].all()


def test_denoising_step_around_the_ffn():
    """Lookup, update, norm, FFN, update in place, last norm, readout: against the
    same step from separate torch operations in fp32, rounded where this one is."""
    V, d, F, L = 900, 256, 512, 64
    m, tokens, seen, mask, _ = _model(6, V, d, L)
    g = torch.Generator(device="cuda").manual_seed(7)
    rnd = lambda *s: (torch.randn(*s, generator=g, device="cuda") * s[-1] ** -0.5).to(torch.bfloat16)  # noqa: E731
    ffn = mtl.SwiGLUFFN(rnd(F, d), rnd(F, d), rnd(d, F), chunk=64)
    emb = mtl.Embedding(m["table"])
    first, last = mtl.ResidualNorm(pre=m["pre"], eps=EPS), mtl.ResidualNorm(pre=m["last"], eps=EPS)
    x = emb(seen)
    before = x.clone()
    _, n = first(x)
    y = ffn(n)
    x_out, h = last(x, y, x_out=x)
    assert x_out is x
    norm = lambda v, w: w.float() * v * torch.rsqrt(v.pow(2).mean(1, keepdim=True) + EPS)  # noqa: E731
    s = before.float() + y.float()
    assert ((x.float() - s).abs() <= 2.0 ** -8 * s.abs() + 1e-6).all()
    want = norm(s, m["last"])
    assert ((h.float() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -16 * want.abs().amax()).all()
    rd = mtl.MaskedReadout(m["head"], L, 4)
    out, left, toks = rd.outputs(), mask.clone(), seen.clone()
    rd.step(h, left, toks, 4, out=out)
    loss, losses, lse = mtl.MaskedLoss(m["head"])(h, mask, out["row_tok"][: L].new_full((L,), 0))
    M = int(out["m_out"].item())
    at = out["row_idx"][:M].long()
    # the readout's log-sum-exp of the same rows: fp32 sums cut at other places
    assert ((lse[at] - out["row_lse"][:M]).abs() <= 2.0 ** -17 * out["row_lse"][:M].abs().clamp(min=1)).all()
    assert int((left != mask).sum()) == 4


def test_two_graphs_at_once():
    """Two captured steps with workspaces of their own, replayed on two streams."""
    sets = [_model(s) for s in (8, 9)]
    want = [_step(*a) for a in sets]
    torch.cuda.synchronize()
    graphs, held, streams = [], [], [torch.cuda.Stream() for _ in sets]
    for a, s in zip(sets, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            held.append(_step(*a))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for w, h in zip(want, held):
        for k in w:
            assert torch.equal(w[k], h[k]), k


def test_stream_of_another_device_is_refused():
    if torch.cuda.device_count() > 1:
        pytest.skip("one device's test")
    s = torch.cuda.Stream()
    w = torch.zeros(64, dtype=torch.bfloat16)
    for make in (lambda: mtl.ResidualNorm(pre=w, stream=s), lambda: mtl.Embedding(w.view(8, 8), stream=s),
                 lambda: mtl.MaskedLoss(w.view(8, 8), stream=s)):
        with pytest.raises(ValueError):
            make()


def test_inputs_of_another_device_are_refused():
    m, tokens, seen, mask, weights = _model(10)
    head, emb, layer = mtl.MaskedLoss(m["head"]), mtl.Embedding(m["table"]), mtl.ResidualNorm(pre=m["pre"])
    h = m["table"][:300].contiguous()
    for call in (lambda: head(h.cpu(), mask, tokens), lambda: head(h, mask, tokens.cpu()), lambda: emb(seen.cpu()),
                 lambda: emb.backward(seen, h.cpu()), lambda: layer(h.cpu()), lambda: layer(h, h, gate=m["gate"].cpu())):
        with pytest.raises(ValueError):
            call()


def test_long_sequences_and_64_bit_offsets():
    """Hidden states of more than 4 GiB, the counted rows at their end."""
    L, d, V = 1 << 20, 2304, 300
    g = torch.Generator(device="cuda").manual_seed(11)
    W = (torch.randn(V, d, generator=g, device="cuda") * d ** -0.5).to(torch.bfloat16)
    hidden = torch.zeros((L, d), dtype=torch.bfloat16, device="cuda")
    rows = torch.randn(5, d, generator=g, device="cuda").to(torch.bfloat16)
    at = torch.tensor([3, L - 1000, L - 7, L - 2, L - 1], device="cuda")
    hidden[at] = rows
    mask = torch.zeros(L, dtype=torch.uint8, device="cuda")
    mask[at] = 1
    targets = torch.full((L,), 7, dtype=torch.int32, device="cuda")
    head = mtl.MaskedLoss(W, piece=256)
    loss, losses, lse = head(hidden, mask, targets)
    d_hidden, d_W = head.backward(hidden, mask, targets, lse)
    few = mtl.MaskedLoss(W, piece=256)
    ones, t5 = torch.ones(5, dtype=torch.uint8, device="cuda"), targets[:5].contiguous()
    l5, ls5, lse5 = few(rows, ones, t5)
    h5, w5 = few.backward(rows, ones, t5, lse5)
    assert torch.equal(losses[at], ls5) and torch.equal(lse[at], lse5) and torch.equal(loss, l5)
    assert torch.equal(d_hidden[at], h5) and torch.equal(d_W, w5)
    assert int((d_hidden != 0).any(1).sum()) == 5 and int((losses != 0).sum()) == 5
