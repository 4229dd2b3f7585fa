"""GPU parity of the embedding and its gradient against the fp64 oracle.

Tolerances.  A looked-up value is one fp32 product (2^-24) and half a step of
bf16.  A gradient is an fp32 sum: 32 additions in a row in a chunk, then the
chunks' shares, a sixteenth of them in a row and 16 more: for the counts here
(at most 20000 of a token, 625 chunks) below 100 additions, 100 * 2^-24 < 2^-17
of the sum of the terms' absolute values, the product with the scale and half a
step of bf16."""
import numpy as np
import pytest

from _layer_cases import HALF, bf16, close, dev_bf16, dev_i32, f64, replayed
from oracle import layers as ol

pytestmark = pytest.mark.gpu

SUM = 2.0 ** -17


def _tokens(rng, T, V, masked, strays=True):
    """Frequent and rare tokens, the last one most of all, and some that have no row."""
    tok = np.minimum(np.exp(rng.random(T) * np.log(V)).astype(np.int64), V) - 1
    tok = np.where(rng.random(T) < masked, V - 1, tok)
    if strays and T > 3:
        at = rng.integers(0, T, max(T // 16, 3))
        tok[at] = rng.choice([-1, V, -2 ** 31, 2 ** 31 - 1, V + 5], len(at))
    return tok.astype(np.int32)


@pytest.mark.parametrize("T,V,d,scale", [(1, 1, 8, 1.0), (7, 50, 64, 8.0), (33, 1000, 4096, 1.0), (1000, 37, 72, 0.3),
                                         (3, 5, 8200, 2.0), (5000, 4096, 256, 16.0)])
def test_lookup(T, V, d, scale):
    import torch

    import masked_token_logits_amd as mtl
    rng = np.random.default_rng(T + V + d)
    table, tf = bf16(rng, (V, d))
    tok = _tokens(rng, T, V, 0.3)
    got = mtl.Embedding(dev_bf16(table), scale=scale)(dev_i32(tok))
    torch.cuda.synchronize()
    want = ol.lookup(tf, tok, scale)
    close(got, want, 0 if scale == 1.0 else (HALF + 2.0 ** -23) * np.abs(want), "rows")


def test_lookup_copies_bits_and_writes_into_a_given_tensor():
    import torch

    import masked_token_logits_amd as mtl
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16).reshape(16, 4096)   # every bf16, NaNs among them
    tok = np.array([3, 15, 0, 15, 99, 8], dtype=np.int32)
    big = torch.full((8, 4096), 7, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    out = mtl.Embedding(dev_bf16(bits))(dev_i32(tok), out=big[1:7])
    torch.cuda.synchronize()
    got = out.view(torch.int16).cpu().numpy().view(np.uint16)
    assert np.array_equal(got, np.where((tok < 16)[:, None], bits[np.minimum(tok, 15)], 0))
    assert (big.view(torch.int16)[[0, 7]] == 7).all()


CASES = [  # T, V, d, scale, share of the last token
    (1, 1, 8, 1.0, 0.0),
    (1, 100, 64, 2.0, 0.0),
    (31, 10, 64, 1.0, 0.5),        # one chunk
    (32, 1, 8, 1.0, 1.0),          # a run that is exactly a chunk
    (33, 1, 520, 1.0, 1.0),        # and one place more; just over a wave's columns
    (64, 2, 128, 0.5, 0.5),
    (509, 4096, 256, 16.0, 0.3),
    (1025, 300, 1032, 1.0, 0.9),
    (4096, 5000, 72, 1.0, 0.5),
    (20001, 40, 16, 1.0, 0.8),     # long runs
    (9000, 130000, 24, 1.0, 0.1),  # many rows without a token
    (16384, 700, 8, 1.0, 0.2),     # the most that are ranked in one launch
    (16385, 700, 8, 1.0, 0.2),     # sorted by one digit
    (18000, 1500, 16, 2.0, 0.0),   # by two
    (17001, 1 << 21, 8, 1.0, 0.5), # by three, most rows without a token
]


@pytest.mark.parametrize("T,V,d,scale,masked", CASES)
def test_gradient(T, V, d, scale, masked):
    import torch

    import masked_token_logits_amd as mtl
    rng = np.random.default_rng(T + V + d)
    print(f"[case] scatter T={T} V={V} d={d} masked={masked}", flush=True)
    tok = _tokens(rng, T, V, masked, strays=T > 40)
    g, gf = bf16(rng, (T, d))
    emb = mtl.Embedding(torch.empty((V, d), dtype=torch.bfloat16, device="cuda"), scale=scale)
    want, size = ol.lookup_grad(tok, gf, V, scale)
    got = emb.backward(dev_i32(tok), dev_bf16(g), d_table=torch.full((V, d), 9.0, dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    close(got, want, HALF * np.abs(want) + SUM * size, "d_table")
    old, of = bf16(rng, (V, d))
    more = emb.backward(dev_i32(tok), dev_bf16(g), d_table=dev_bf16(old), accumulate=True)
    torch.cuda.synchronize()
    close(more, of + want, HALF * np.abs(of + want) * (size > 0) + SUM * (size + np.abs(of) * (size > 0)), "accumulated")
    again = emb.backward(dev_i32(tok), dev_bf16(g))
    assert torch.equal(got, again)      # no result depends on timing


def test_gradient_of_no_tokens():
    import torch

    import masked_token_logits_amd as mtl
    for tok in (np.zeros(0, np.int32), np.full(100, -1, np.int32), np.full(70, 50, np.int32)):
        emb = mtl.Embedding(torch.empty((50, 64), dtype=torch.bfloat16, device="cuda"))
        g = torch.ones((len(tok), 64), dtype=torch.bfloat16, device="cuda")
        d = torch.full((50, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        assert (emb.backward(dev_i32(tok), g, d_table=d, accumulate=True) == 3).all()
        assert not emb.backward(dev_i32(tok), g, d_table=d).any()
        assert emb(dev_i32(tok)).shape == (len(tok), 64)


def test_nan_reaches_its_own_row_only():
    import torch

    import masked_token_logits_amd as mtl
    rng = np.random.default_rng(3)
    tok = rng.integers(0, 20, 400).astype(np.int32)
    g, _ = bf16(rng, (400, 64))
    d = dev_bf16(g)
    at = int(np.nonzero(tok == 4)[0][2])
    d[at, 5] = float("nan")
    got = f64(mtl.Embedding(torch.empty((20, 64), dtype=torch.bfloat16, device="cuda")).backward(dev_i32(tok), d))
    assert np.isnan(got[4, 5]) and np.isnan(got).sum() == 1


def test_offsets_beyond_32_bits():
    """A table of more than 4 GiB: rows at its end."""
    import torch

    import masked_token_logits_amd as mtl
    V, d = 1 << 19, 4608
    table = torch.zeros((V, d), dtype=torch.bfloat16, device="cuda")
    table[V - 1], table[V - 2] = 3.0, 5.0
    tok = dev_i32([V - 1, 0, V - 2, V - 1])
    emb = mtl.Embedding(table)
    out = emb(tok)
    assert (out[0] == 3).all() and (out[1] == 0).all() and (out[2] == 5).all()
    emb.backward(tok, out, d_table=table)
    assert (table[V - 1] == 6).all() and (table[V - 2] == 5).all() and not table[: V - 2].any()


def test_captured_and_replayed():
    import torch

    import masked_token_logits_amd as mtl
    T, V, d = 2000, 500, 128
    sets = []
    for i in range(3):
        rng = np.random.default_rng(40 + i)
        sets.append((dev_i32(_tokens(rng, T, V, 0.2 * i)), dev_bf16(bf16(rng, (T, d))[0])))
    tok, g = sets[0][0].clone(), sets[0][1].clone()
    emb = mtl.Embedding(dev_bf16(bf16(np.random.default_rng(1), (V, d))[0]), scale=3.0)

    def refill(i):
        tok.copy_(sets[i][0])
        g.copy_(sets[i][1])

    def check(i, got, eager):
        for a, b in zip(got, eager):
            assert torch.equal(a, b)
        want, size = ol.lookup_grad(tok.cpu().numpy(), f64(g), V, 3.0)
        close(got[1], want, HALF * np.abs(want) + SUM * size, "d_table")

    replayed(lambda: [emb(tok), emb.backward(tok, g)], check, refill)


def test_streams():
    import torch

    import masked_token_logits_amd as mtl
    rng = np.random.default_rng(50)
    T, V, d = 3000, 200, 256
    sets = [(dev_i32(_tokens(rng, T, V, 0.5)), dev_bf16(bf16(rng, (T, d))[0])) for _ in range(2)]
    torch.cuda.synchronize()
    embs = [mtl.Embedding(torch.empty((V, d), dtype=torch.bfloat16, device="cuda"), stream=torch.cuda.Stream()) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [e.backward(*s) for e, s in zip(embs, sets)]
    torch.cuda.synchronize()
    for out, (tok, g) in zip(got, sets):
        want, size = ol.lookup_grad(tok.cpu().numpy(), f64(g), V)
        close(out, want, HALF * np.abs(want) + SUM * size, "d_table")
