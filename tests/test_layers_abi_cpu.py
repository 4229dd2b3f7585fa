"""The host side of the norm, embedding and loss C ABI and their binding:
argument refusals before any HIP call, workspace sizes, and the tensor checks
of ResidualNorm, Embedding and MaskedLoss.  No GPU."""
import pytest
import torch

import masked_token_logits_amd as mtl

FAKE = 0x7F0000000000   # aligned, never dereferenced
STEP = 1 << 32          # buffers that far apart never overlap
E = mtl


def _at(i):
    return FAKE + i * STEP


def _norm(**kw):
    a = dict(pre=_at(0), post=_at(1), d=64, eps=1e-5, scale=1.0)
    a.update(kw)
    return mtl.dllm_norm(a["pre"], a["post"], a["d"], a["eps"], a["scale"])


def _forward(norm=None, **kw):
    a = dict(norm=norm or _norm(), x=_at(2), y=_at(3), T=12, gate=_at(4), groups=3, x_out=_at(5), n=_at(6))
    a.update(kw)
    return mtl.dllm_residual_norm(**a)


def _backward(norm=None, **kw):
    a = dict(norm=norm or _norm(), x=_at(2), y=_at(3), T=12, gate=_at(4), groups=3, d_n=_at(7), d_x_out=_at(8),
             d_x=_at(9), d_y=_at(10), d_pre=_at(11), d_post=_at(12), d_gate=_at(13), workspace=_at(14),
             workspace_bytes=1 << 30)
    a.update(kw)
    return mtl.dllm_residual_norm_backward(**a)


BAD_NORMS = [dict(d=0), dict(d=-8), dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=float("inf"))]


def test_residual_norm_refused():
    for bad in BAD_NORMS + [dict(scale=float("nan")), dict(scale=float("inf"))]:
        assert _forward(_norm(**bad)) == E.DLLM_ERR_INVALID_ARG, bad
    for kw in (dict(norm=_norm(pre=None)), dict(n=None), dict(x=None), dict(y=None), dict(x_out=None), dict(T=-1),
               dict(T=1 << 31), dict(groups=0), dict(gate=None), dict(groups=-1), dict(groups=5), dict(groups=24),
               dict(n=_at(2)), dict(n=_at(5)), dict(x_out=_at(3)), dict(x_out=_at(2) + 16), dict(n=_at(4) - 16),
               dict(y=None, x_out=None)):
        assert _forward(**kw) == E.DLLM_ERR_INVALID_ARG, kw
    for kw in (dict(norm=_norm(d=60)), dict(norm=_norm(d=mtl.DLLM_NORM_DIM_MAX + 8)), dict(x=_at(2) + 2),
               dict(norm=_norm(pre=_at(0) + 8)), dict(n=_at(6) + 4), dict(gate=_at(4) + 2)):
        assert _forward(**kw) == E.DLLM_ERR_UNSUPPORTED, kw
    assert _forward(T=0, groups=1) == E.DLLM_OK
    if not torch.cuda.is_available():
        assert _forward() == E.DLLM_ERR_HIP
        assert _forward(x_out=_at(2)) == E.DLLM_ERR_HIP                                    # in place
        assert _forward(_norm(post=None), y=None, x_out=None, gate=None, groups=0) == E.DLLM_ERR_HIP
        assert _forward(_norm(pre=None), n=None) == E.DLLM_ERR_HIP


def test_residual_norm_backward_refused():
    for bad in BAD_NORMS + [dict(scale=float("nan"))]:
        assert _backward(_norm(**bad)) == E.DLLM_ERR_INVALID_ARG, bad
    for kw in (dict(norm=_norm(pre=None)), dict(d_n=None), dict(x=None), dict(y=None), dict(d_y=None), dict(d_x=None),
               dict(T=-1), dict(groups=5), dict(gate=None), dict(norm=_norm(post=None)),
               dict(gate=None, groups=0), dict(d_x=_at(2)), dict(d_x=_at(3)), dict(d_y=_at(9)), dict(d_y=_at(7)),
               dict(d_pre=_at(12) + 16), dict(d_gate=_at(2)), dict(d_post=_at(14)), dict(d_x=_at(8) + 16),
               dict(norm=_norm(pre=None), d_n=None, d_pre=None, d_x_out=None)):
        assert _backward(**kw) == E.DLLM_ERR_INVALID_ARG, kw
    need = mtl.dllm_residual_norm_backward_workspace_bytes(_norm(), 12, 3)
    assert need > 0
    for kw in (dict(workspace=None), dict(workspace_bytes=need - 1), dict(workspace=_at(14) + 16)):
        assert _backward(**kw) == E.DLLM_ERR_WORKSPACE, kw
    for kw in (dict(norm=_norm(d=60)), dict(d_x=_at(9) + 2), dict(d_pre=_at(11) + 4)):
        assert _backward(**kw) == E.DLLM_ERR_UNSUPPORTED, kw
    assert _backward(T=0, groups=1) == E.DLLM_OK
    for groups in (0, 1):
        assert mtl.dllm_residual_norm_backward_workspace_bytes(_norm(), 0, groups) > 0
    for bad in (dict(norm=_norm(d=60)), dict(norm=_norm(d=0)), dict(T=-1), dict(groups=-1), dict(groups=7)):
        a = dict(norm=_norm(), T=12, groups=3)
        a.update(bad)
        assert mtl.dllm_residual_norm_backward_workspace_bytes(**a) == 0
    if not torch.cuda.is_available():
        assert _backward(workspace_bytes=need) == E.DLLM_ERR_HIP
        assert _backward(d_x=_at(8), d_y=_at(3)) == E.DLLM_ERR_HIP
        assert _backward(d_x=_at(7), d_pre=None, d_post=None, d_gate=None) == E.DLLM_ERR_HIP


def test_workspace_is_apart_from_the_inputs():
    """A workspace that holds an input would be written while the input is still read."""
    for i in (0, 1, 2, 3, 4, 7, 8):
        assert _backward(workspace=_at(i)) == E.DLLM_ERR_INVALID_ARG, i
    for i in (1, 2):
        assert _embed_backward(workspace=_at(i)) == E.DLLM_ERR_INVALID_ARG, i
    for i in range(5):
        assert _loss(workspace=_at(i)) == E.DLLM_ERR_INVALID_ARG, i
    for i in (0, 1, 2, 3, 4, 7, 9):
        assert _loss_backward(workspace=_at(i)) == E.DLLM_ERR_INVALID_ARG, i


def test_most_places_of_a_table_gradient():
    most = (1 << 30) - 1
    assert mtl.dllm_embed_backward_workspace_bytes(100, 8, most) > 0
    assert mtl.dllm_embed_backward_workspace_bytes(100, 8, most + 1) == 0
    assert _embed_backward(T=most + 1, d=8) == E.DLLM_ERR_INVALID_ARG


def _embed(**kw):
    a = dict(table=_at(0), V=100, d=64, tokens=_at(1), T=10, scale=1.0, out=_at(2))
    a.update(kw)
    return mtl.dllm_embed(**a)


def _embed_backward(**kw):
    a = dict(tokens=_at(1), T=10, d_out=_at(2), V=100, d=64, scale=1.0, accumulate=0, d_table=_at(3), workspace=_at(4),
             workspace_bytes=1 << 30)
    a.update(kw)
    return mtl.dllm_embed_backward(**a)


def test_embed_refused():
    sizes = (dict(V=0), dict(V=(1 << 31) - 1024), dict(d=0), dict(T=-1), dict(T=(1 << 31) - 1024), dict(scale=float("nan")),
             dict(scale=float("-inf")))
    for kw in sizes + (dict(table=None), dict(tokens=None), dict(out=None), dict(out=_at(0) + 16), dict(out=_at(1) - 16)):
        assert _embed(**kw) == E.DLLM_ERR_INVALID_ARG, kw
    for kw in (dict(d=60), dict(d=1 << 20), dict(table=_at(0) + 8), dict(out=_at(2) + 2), dict(tokens=_at(1) + 2)):
        assert _embed(**kw) == E.DLLM_ERR_UNSUPPORTED, kw
    assert _embed(T=0, tokens=None, out=None) == E.DLLM_OK
    for kw in sizes + (dict(tokens=None), dict(d_out=None), dict(d_table=None), dict(accumulate=2), dict(accumulate=-1),
                       dict(d_table=_at(2) + 16), dict(d_table=_at(1) - 128), dict(workspace=_at(3))):
        assert _embed_backward(**kw) == E.DLLM_ERR_INVALID_ARG, kw
    for kw in (dict(d=60), dict(d_table=_at(3) + 2), dict(d_out=_at(2) + 4), dict(tokens=_at(1) + 1)):
        assert _embed_backward(**kw) == E.DLLM_ERR_UNSUPPORTED, kw
    need = mtl.dllm_embed_backward_workspace_bytes(100, 64, 10)
    assert need > 0
    for kw in (dict(workspace=None), dict(workspace_bytes=need - 1), dict(workspace=_at(4) + 64)):
        assert _embed_backward(**kw) == E.DLLM_ERR_WORKSPACE, kw
    assert mtl.dllm_embed_backward_workspace_bytes(100, 64, 0) > 0
    for bad in ((0, 64, 10), (100, 60, 10), (100, 64, -1)):
        assert mtl.dllm_embed_backward_workspace_bytes(*bad) == 0
    if not torch.cuda.is_available():
        assert _embed() == E.DLLM_ERR_HIP
        assert _embed_backward(workspace_bytes=need) == E.DLLM_ERR_HIP


def _loss_struct(**kw):
    a = dict(W_lm=_at(0), hidden=_at(1), mask=_at(2), targets=_at(3), weights=_at(4), V=1000, d=64, L=50)
    a.update(kw)
    return mtl.dllm_loss(*(a[n] for n, _ in mtl.dllm_loss._fields_))


def _loss(p=None, **kw):
    a = dict(p=p or _loss_struct(), loss=_at(5), losses=_at(6), lse=_at(7), workspace=_at(8), workspace_bytes=1 << 31)
    a.update(kw)
    return mtl.dllm_loss_forward(**a)


def _loss_backward(p=None, **kw):
    a = dict(p=p or _loss_struct(), lse=_at(7), grad=_at(9), d_hidden=_at(10), d_W=_at(11), accumulate=0, piece=256,
             workspace=_at(8), workspace_bytes=1 << 31)
    a.update(kw)
    return mtl.dllm_loss_backward(**a)


def test_loss_refused():
    for call in (_loss, _loss_backward):
        for bad in (dict(V=0), dict(V=(1 << 31) - 1024), dict(d=0), dict(L=0), dict(L=-1), dict(W_lm=None), dict(hidden=None),
                    dict(mask=None), dict(targets=None)):
            assert call(_loss_struct(**bad)) == E.DLLM_ERR_INVALID_ARG, (call, bad)
        for bad in (dict(d=60), dict(d=1 << 20), dict(W_lm=_at(0) + 8), dict(hidden=_at(1) + 2), dict(targets=_at(3) + 2),
                    dict(weights=_at(4) + 1)):
            assert call(_loss_struct(**bad)) == E.DLLM_ERR_UNSUPPORTED, (call, bad)
        assert call(p=_loss_struct(), workspace=None) == E.DLLM_ERR_WORKSPACE
        assert call(p=_loss_struct(), workspace=_at(8) + 16) == E.DLLM_ERR_WORKSPACE
    for kw in (dict(loss=None), dict(losses=None), dict(lse=None), dict(lse=_at(6) + 4), dict(loss=_at(7) + 8),
               dict(losses=_at(1)), dict(lse=_at(4)), dict(lse=_at(8)), dict(workspace=_at(0))):
        assert _loss(**kw) == E.DLLM_ERR_INVALID_ARG, kw
    need = mtl.dllm_loss_forward_workspace_bytes(1000, 64, 50)
    assert _loss(workspace_bytes=need - 1) == E.DLLM_ERR_WORKSPACE
    for kw in (dict(lse=None), dict(d_hidden=None, d_W=None), dict(accumulate=2), dict(piece=-256), dict(piece=100),
               dict(d_hidden=_at(1)), dict(d_W=_at(0)), dict(d_W=_at(10) + 16), dict(d_hidden=_at(8)), dict(workspace=_at(7))):
        assert _loss_backward(**kw) == E.DLLM_ERR_INVALID_ARG, kw
    for kw in (dict(d_W=_at(11) + 2), dict(d_hidden=_at(10) + 8), dict(lse=_at(7) + 2), dict(grad=_at(9) + 1)):
        assert _loss_backward(**kw) == E.DLLM_ERR_UNSUPPORTED, kw
    back = mtl.dllm_loss_backward_workspace_bytes(1000, 64, 50, 256)
    assert _loss_backward(workspace_bytes=back - 1) == E.DLLM_ERR_WORKSPACE
    if not torch.cuda.is_available():
        assert _loss(workspace_bytes=need) == E.DLLM_ERR_HIP
        assert _loss_backward(workspace_bytes=back) == E.DLLM_ERR_HIP
        assert _loss_backward(_loss_struct(weights=None), grad=None, d_hidden=None) == E.DLLM_ERR_HIP


def test_loss_workspace_does_not_hold_the_logits():
    """The backward workspace is bounded by the piece, not by the vocabulary."""
    V, d, L = 152064, 3584, 8192
    a, b = (mtl.dllm_loss_backward_workspace_bytes(v, d, L, 8192) for v in (V, 4 * V))
    # the piece's dz in bf16, the rows' gradient in fp32 and the rows themselves, and a fixed part
    assert a == b and a < L * 8192 * 2 + L * d * 6 + (1 << 28)
    assert mtl.dllm_loss_backward_workspace_bytes(V, d, L) < (1 << 30) + L * d * 6 + (1 << 28)
    assert mtl.dllm_loss_backward_workspace_bytes(V, d, 131072) < 131072 * 8192 * 2 + 131072 * d * 6 + (1 << 28)
    for bad in ((0, d, L, 0), (V, 60, L, 0), (V, d, 0, 0), (V, d, L, 100), (V, d, L, -256)):
        assert mtl.dllm_loss_backward_workspace_bytes(*bad) == 0
    assert mtl.dllm_loss_forward_workspace_bytes(V, 60, L) == 0


# ---- the binding's checks, on CPU tensors ---------------------------------------------------------------------

def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_residual_norm_checks():
    with pytest.raises(ValueError):
        mtl.ResidualNorm()
    with pytest.raises(TypeError):
        mtl.ResidualNorm(pre=torch.zeros(64))
    with pytest.raises(ValueError):
        mtl.ResidualNorm(pre=bf(64), post=bf(72))
    with pytest.raises(ValueError):
        mtl.ResidualNorm(pre=bf(64), eps=-1.0)
    with pytest.raises(ValueError):
        mtl.ResidualNorm(pre=bf(64), scale=float("nan"))
    for d in (4, 60, mtl.DLLM_NORM_DIM_MAX + 8):
        with pytest.raises(mtl.DllmError):
            mtl.ResidualNorm(pre=bf(d))
    both, pre, none = mtl.ResidualNorm(pre=bf(64), post=bf(64)), mtl.ResidualNorm(pre=bf(64)), mtl.ResidualNorm(d=64, device="cpu")
    x, y = bf(12, 64), bf(12, 64)
    for layer, args, kw in ((both, (x,), {}), (none, (x,), {}), (pre, (x,), dict(gate=bf(1, 64))), (both, (x, bf(11, 64)), {}),
                            (both, (x, y), dict(gate=bf(5, 64))), (both, (x, y), dict(gate=bf(64))),
                            (both, (x, y), dict(gate=bf(24, 64))), (none, (x, y), dict(n_out=bf(12, 64))),
                            (both, (bf(64, 12).t(), y), {}), (both, (x, y), dict(x_out=bf(12, 72))), (both, (bf(64),), {}),
                            (pre, (x,), dict(x_out=bf(12, 64)))):
        with pytest.raises(ValueError):
            layer(*args, **kw)
    with pytest.raises(TypeError):
        both(x.float(), y)
    for layer, kw in ((both, dict(d_n=None, y=y)), (none, dict(d_n=x, y=y)), (none, dict(y=y)), (both, dict(d_n=x)),
                      (both, dict(d_n=x, y=y, gate=bf(5, 64))), (both, dict(d_n=bf(11, 64), y=y)),
                      (pre, dict(d_n=x, d_y_out=y))):
        with pytest.raises(ValueError):
            layer.backward(x, **kw)
    for call in (lambda: both(x, y), lambda: pre(x), lambda: both.backward(x, x, y=y), lambda: none.backward(x, y=y, d_x=x)):
        with pytest.raises(mtl.DllmError) as e:     # a valid call off the GPU
            call()
        assert e.value.status == E.DLLM_ERR_UNSUPPORTED


def test_embedding_checks():
    for bad in (bf(64), bf(0, 64), bf(64, 10).t()):
        with pytest.raises(ValueError):
            mtl.Embedding(bad)
    with pytest.raises(TypeError):
        mtl.Embedding(torch.zeros(4, 64))
    with pytest.raises(mtl.DllmError):
        mtl.Embedding(bf(4, 60))
    with pytest.raises(ValueError):
        mtl.Embedding(bf(4, 64), scale=float("inf"))
    emb, tok = mtl.Embedding(bf(10, 64)), torch.zeros(5, dtype=torch.int32)
    with pytest.raises(TypeError):
        emb(tok.long())
    for args in ((tok[None],), (tok, bf(4, 64))):
        with pytest.raises(ValueError):
            emb(*args)
    for args, kw in (((tok, bf(4, 64)), {}), ((tok, bf(5, 72)), {}), ((tok, bf(5, 64)), dict(accumulate=True)),
                     ((tok, bf(5, 64)), dict(d_table=bf(9, 64)))):
        with pytest.raises(ValueError):
            emb.backward(*args, **kw)
    for call in (lambda: emb(tok), lambda: emb.backward(tok, bf(5, 64))):
        with pytest.raises(mtl.DllmError) as e:
            call()
        assert e.value.status == E.DLLM_ERR_UNSUPPORTED


def test_masked_loss_checks():
    for bad in (bf(64), bf(0, 64), bf(64, 10).t()):
        with pytest.raises(ValueError):
            mtl.MaskedLoss(bad)
    with pytest.raises(TypeError):
        mtl.MaskedLoss(torch.zeros(4, 64))
    with pytest.raises(mtl.DllmError):
        mtl.MaskedLoss(bf(4, 60))
    for piece in (0, 100, -256):
        with pytest.raises(ValueError):
            mtl.MaskedLoss(bf(10, 64), piece=piece)
    head = mtl.MaskedLoss(bf(10, 64))
    H, m, t, w, lse = bf(7, 64), torch.zeros(7, dtype=torch.uint8), torch.zeros(7, dtype=torch.int32), torch.zeros(7), torch.zeros(7)
    for args, kw in (((H.float(), m, t), {}), ((H, m.int(), t), {}), ((H, m, t.long()), {}), ((H, m, t), dict(weights=w.double()))):
        with pytest.raises(TypeError):
            head(*args, **kw)
    for args, kw in (((bf(0, 64), m[:0], t[:0]), {}), ((H, m[:6], t), {}), ((H, m, t[:6]), {}), ((H, m, t), dict(weights=w[:6])),
                     ((bf(7, 72), m, t), {}), ((H, m, t), dict(out=(w, w, w))), ((H, m, t), dict(out=(w[:1], w)))):
        with pytest.raises(ValueError):
            head(*args, **kw)
    for kw in (dict(need=()), dict(need=("table",)), dict(accumulate=True), dict(grad=torch.zeros(2)), dict(d_W=bf(9, 64)),
               dict(d_hidden=bf(6, 64))):
        with pytest.raises(ValueError):
            head.backward(H, m, t, lse, **kw)
    with pytest.raises(TypeError):
        head.backward(H, m, t, lse.double())
    for call in (lambda: head(H, m.bool(), t), lambda: head.backward(H, m, t, lse)):
        with pytest.raises(mtl.DllmError) as e:
            call()
        assert e.value.status == E.DLLM_ERR_UNSUPPORTED


@pytest.mark.parametrize("form", [tuple, list, iter])
def test_masked_loss_keeps_its_outputs_for_the_stream(form, monkeypatch):
    """Outputs are among the tensors that a call on another stream keeps alive, in whatever form they come."""
    head, kept = mtl.MaskedLoss(bf(10, 64)), []
    monkeypatch.setattr(head, "_call", lambda where, tensors, make: kept.extend(tensors))
    out = [torch.zeros(1), torch.zeros(7), torch.zeros(7)]
    got = head(bf(7, 64), torch.zeros(7, dtype=torch.uint8), torch.zeros(7, dtype=torch.int32), out=form(out))
    assert all(any(t is k for k in kept) for t in out) and all(g is t for g, t in zip(got, out))
