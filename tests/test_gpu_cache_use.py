"""The block cache's operators as a program uses them: one after another with the
FFN and the readout, the same call twice, captured and replayed, on streams of
their own, in pools past 32-bit offsets, with many sequences and with work cut
into many parts.  Parity is held to the tolerances of test_gpu_cache.py, whose
derivations cover these sizes too; everything else here is equality, for a call's
result depends on its inputs alone."""
import numpy as np
import pytest

import workloads as WL
from _cache_cases import bf16, cache, cu_of, dev_bf16, dev_i32, host, on_gpu, tables
from oracle import cache as oc
from test_gpu_cache import _batch, _check_attention, _dS

pytestmark = pytest.mark.gpu


def _attend_against_oracle(rng, D, heads, Hq, lens, new, causal, where, change=None, extra=0):
    import torch
    table, pages = tables(rng, lens)
    table = np.concatenate([table, np.full((len(lens), extra), -1, np.int32)], 1)
    if change == "holes":
        table[:, 1::3] = -1
    c = cache(rng, pages, heads, D, lens, table)
    if change == "scales":                       # values' scales 2^40 apart, ever larger
        for s in range(len(lens)):
            for j in range(table.shape[1]):
                if 0 <= table[s, j] < pages:
                    c["v_scale"][table[s, j]] = 100 + min(2 * j, 40)
    T = sum(new)
    q, qf = bf16(rng, (T, Hq, D))
    bc = on_gpu(c)
    b = _batch(bc, cu_of(new), lens, table)
    o, l = bc.attend(b, dev_bf16(q), causal=causal, lse=True)
    torch.cuda.synchronize()
    r = oc.attend(c, cu_of(new), lens, table, qf, float(np.float32(D ** -0.5)), causal)
    _check_attention(o, l, r, D, where)
    for _ in range(2):                           # the same call, the same bits
        o2, l2 = bc.attend(b, dev_bf16(q), causal=causal, lse=True)
        assert torch.equal(o2, o) and torch.equal(l2, l)


@pytest.mark.parametrize("D,heads,Hq,lens,new,causal,change", [
    (64, 1, 2, [2500], [70], False, None),             # 140 rows along 79 blocks: a tile in many parts
    (128, 1, 4, [3001], [40], False, "holes"),         # 160 rows
    (128, 2, 16, [1500, 33, 700], [20, 33, 25], False, "scales"),
    (256, 1, 5, [1100], [30], True, "holes"),          # 150 rows
    (256, 1, 3, [900, 50], [50, 60], False, "scales"),
    (64, 1, 1, [600], [600], True, None),              # causal tiles of different lengths
    (128, 1, 3, [257, 255], [257, 255], True, None),
    (128, 1, 1, [5000], [33], False, "scales"),        # 33 rows: the kernel for few rows
    (128, 2, 8, [2000], [32], False, "holes"),         # 128 rows: its last
    (64, 2, 2, [1999], [97], True, None),
    (256, 2, 4, [1500], [30], True, None),
])
@pytest.mark.parametrize("extra", [0, 30000])
def test_attention_in_parts(D, heads, Hq, lens, new, causal, change, extra):
    """With room in the table for a million tokens a call of more than 128 rows of a head is
    taken for a large one, without it for a small one."""
    print(f"[case] parts D={D} heads={heads}/{Hq} lens={lens} new={new} causal={causal} {change} {extra}", flush=True)
    _attend_against_oracle(np.random.default_rng(D + sum(lens) + sum(new)), D, heads, Hq, lens, new, causal, "parts", change,
                           extra)


@pytest.mark.parametrize("S,n,extra", [(63, 1, 0), (64, 1, 0), (65, 1, 0), (300, 1, 0), (300, 9, 0), (65, 9, 1000),
                                       (300, 9, 1000)])
def test_attention_many_sequences(S, n, extra):
    """Around the number of sequences that one wave, or one workgroup, looks through at
    a time; some have no tokens or no queries; 9 queries of 16 heads make 144 rows."""
    rng = np.random.default_rng(S + n)
    lens = [int(x) for x in rng.integers(0, 100, S)]
    new = [int(x) for x in rng.integers(0, n + 1, S)]
    lens[0] = new[1] = 0
    new[S - 1], lens[S - 1] = n, 90
    print(f"[case] sequences S={S} n={n}", flush=True)
    _attend_against_oracle(rng, 64, 1, 16, lens, new, n > 1, "sequences", extra=extra)


@pytest.mark.parametrize("D,heads,Hq,S,causal", [(64, 16, 16, 17, True), (64, 16, 48, 17, False), (128, 32, 32, 8, True),
                                                 (128, 32, 64, 9, False), (256, 16, 16, 16, True)])
def test_weigh_many_workgroups(D, heads, Hq, S, causal):
    """Enough heads and sequences for workgroups of eight blocks, with odd numbers of
    blocks, a hole, and queries that see nothing; twice, to the same bits."""
    import torch
    rng = np.random.default_rng(D + heads + S)
    lens = [int(x) for x in rng.integers(1, 290, S)]
    new = [int(x) for x in rng.integers(0, 40, S)]
    lens[0], new[0], lens[1], new[1], lens[2], new[2] = 289, 289, 20, 70, 256, 1
    print(f"[case] weigh many D={D} heads={heads}/{Hq} S={S} causal={causal}", flush=True)
    table, pages = tables(rng, lens)
    table[0, 4] = -1
    assert S * heads * -(-((max(lens) + 31) // 32) // 8) >= 256
    c = cache(rng, pages, heads, D, lens, table)
    T = sum(new)
    q, qf = bf16(rng, (T, Hq, D))
    w0 = rng.random((S, heads, table.shape[1] * 32)).astype(np.float32)
    bc = on_gpu(c)
    b = _batch(bc, cu_of(new), lens, table)
    _, lse = bc.attend(b, dev_bf16(q), causal=causal, lse=True)
    w = torch.from_numpy(w0.copy()).cuda()
    bc.weigh(b, dev_bf16(q), lse, w, causal=causal, decay=0.5)
    w2 = torch.from_numpy(w0.copy()).cuda()
    bc.weigh(b, dev_bf16(q), lse, w2, causal=causal, decay=0.5)
    torch.cuda.synchronize()
    assert torch.equal(w, w2)
    scale = float(np.float32(D ** -0.5))
    want = oc.weigh(c, cu_of(new), lens, table, qf, lse.cpu().numpy(), scale, causal, w0, 0.5)
    r = oc.attend(c, cu_of(new), lens, table, qf, scale, causal)
    rel = np.nanmax(np.where(np.isfinite(r["lse"]), _dS(r, D) + 2.0 ** -21 * (np.abs(r["lse"]) + r["A"] + 1), 0))
    got = w.cpu().numpy().astype(np.float64)
    for s, n in enumerate(lens):
        np.testing.assert_array_equal(got[s, :, n:], w0[s, :, n:].astype(np.float64))
        x, y = got[s, :, :n], want[s, :, :n]
        tol = (rel + T * Hq * 2.0 ** -24) * np.abs(y - 0.5 * w0[s, :, :n]) + 2.0 ** -22 * np.abs(y)
        assert np.all(np.abs(x - y) <= tol), f"sequence {s}"


def test_weigh_sums_to_the_number_of_queries():
    """What a query gives away is one in all: the sum of a head's weights is the number of
    its queries that see a token."""
    import torch
    rng = np.random.default_rng(50)
    D, heads, Hq, lens, new = 128, 2, 6, [1000, 70], [50, 90]
    table, pages = tables(rng, lens)
    bc = on_gpu(cache(rng, pages, heads, D, lens, table))
    b = _batch(bc, cu_of(new), lens, table)
    q = dev_bf16(bf16(rng, (140, Hq, D))[0])
    for causal in (False, True):
        _, lse = bc.attend(b, q, causal=causal, lse=True)
        w = torch.zeros(2, heads, table.shape[1] * 32, device="cuda")
        bc.weigh(b, q, lse, w, causal=causal)
        seen = torch.tensor([50, 70 if causal else 90], dtype=torch.float64, device="cuda")[:, None] * (Hq // heads)
        # a score is the same fp32 number in both, within (D + 8) 2^-24 of |q| |k| scale < 400
        assert torch.all((w.double().sum(-1) - seen).abs() <= seen * 2 * (D + 8) * 2.0 ** -24 * 400)


# ---- one after another ------------------------------------------------------------------------------------------

class _Layer:
    """Buffers of one layer's cache calls; run() queues a decoding block's: positions, write,
    attention, accumulated weights, eviction, and attention over what is left."""

    def __init__(self, seed, stream=None):
        import torch

        import masked_token_logits_amd as mtl
        rng = np.random.default_rng(seed)
        self.D, self.H, self.Hq, self.S, self.n = 64, 2, 4, 2, 32
        lens = [200, 137]
        self.table_h, pages = tables(rng, lens, spare=0)
        self.table_out_h = (pages + rng.permutation(2 * 4).reshape(2, 4)).astype(np.int32)
        old = [a - self.n for a in lens]
        self.host_cache = cache(rng, pages + 8, self.H, self.D, old, self.table_h)
        self.lens_h, self.old, self.keep_h = lens, old, [100, 128]
        self.bc = on_gpu(self.host_cache)
        self.bc.stream = stream
        self.rot = mtl.Rotary(self.D, stream=stream)
        self.b = self.bc.batch(dev_i32(cu_of([self.n] * 2)), dev_i32(lens), dev_i32(self.table_h), max_new=self.n)
        self.q, self.qf = bf16(rng, (64, self.Hq, self.D))
        self.k, self.kf = bf16(rng, (64, self.H, self.D))
        self.v, self.vf = bf16(rng, (64, self.H, self.D))
        self.pos_h = np.concatenate([np.arange(self.n) + o for o in old])
        self.tq, self.tk, self.tv = (dev_bf16(x) for x in (self.q, self.k, self.v))
        self.start, self.pos = dev_i32(old), dev_i32(self.pos_h)
        self.weights = torch.zeros(2, self.H, self.table_h.shape[1] * 32, device="cuda")
        self.keep, self.table_out = dev_i32(self.keep_h), dev_i32(self.table_out_h)
        self.lens_out = torch.zeros(2, dtype=torch.int32, device="cuda")
        self.kept = torch.zeros(2, self.H, 128, dtype=torch.int32, device="cuda")
        self.weights_out = torch.zeros(2, self.H, 128, device="cuda")
        self.b2 = self.bc.batch(self.b.cu, self.lens_out, self.table_out, max_new=self.n)
        self.start0 = [t.clone() for t in self._state()]

    def _state(self):
        return [self.bc.k, self.bc.v, self.bc.k_scale, self.bc.v_scale, self.weights, self.lens_out, self.kept,
                self.weights_out]

    def reset(self):
        for t, t0 in zip(self._state(), self.start0):
            t.copy_(t0)

    def run(self):
        qr = self.rot(self.tq, self.pos)
        self.bc.write(self.b, self.tk, self.tv, self.start, positions=self.pos, rotary=self.rot)
        out, lse = self.bc.attend(self.b, qr, lse=True)
        self.bc.weigh(self.b, qr, lse, self.weights)
        self.bc.evict(self.b, self.weights, self.keep, self.table_out, sink=1, recent=self.n, pool=3,
                      lens_out=self.lens_out, kept=self.kept, weights_out=self.weights_out)
        out2 = self.bc.attend(self.b2, qr)
        return qr, out, lse, out2

    def results(self, outs):
        return [t.clone() for t in list(outs) + self._state()]


def _same(a, b):
    import torch
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_a_block_through_a_layer():
    """Every step against the oracle on the inputs that it had, then the attention's output through the FFN and
    the readout that the package has beside them."""
    import torch

    import masked_token_logits_amd as mtl
    L = _Layer(60)
    qr, out, lse, out2 = L.run()
    torch.cuda.synchronize()
    bits = lambda t: t.cpu().view(torch.int16).numpy().view(np.uint16)
    qrf = WL.bf16_to_f32(bits(qr)).astype(np.float64)
    want, _ = oc.rotate(L.qf, L.pos_h, oc.rotary_theta(64), "half")
    assert np.all(np.abs(qrf - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * np.abs(L.qf).max())
    cu = cu_of([32, 32])
    stored, _ = oc.write(L.host_cache, cu, L.lens_h, L.table_h, L.old, L.kf, L.vf, L.pos_h, oc.rotary_theta(64), "half")
    got = host(L.bc)
    used = L.table_h[:, :7][L.table_h[:, :7] < len(got["k"])]
    used = used[used >= 0]
    for name in ("v", "k_scale", "v_scale"):
        np.testing.assert_array_equal(got[name][used], stored[name][used], err_msg=name)
    scale = float(np.float32(64 ** -0.5))
    r = oc.attend(got, cu, L.lens_h, L.table_h, qrf, scale, False)
    _check_attention(out, lse, r, 64, "over the whole cache")
    w = L.weights.cpu().numpy()
    wants, n, kept, ww = oc.evict(got, L.lens_h, L.table_h, w, L.keep_h, 1, 32, 3, L.table_out_h)
    np.testing.assert_array_equal(L.lens_out.cpu().numpy(), n)
    for s in range(2):
        for h in range(L.H):
            np.testing.assert_array_equal(L.kept[s, h, :n[s]].cpu().numpy(), kept[s][h])
            np.testing.assert_array_equal(L.weights_out[s, h, :n[s]].cpu().numpy(), ww[s][h])
    for name in wants:
        np.testing.assert_array_equal(got[name], wants[name], err_msg=name)
    r2 = oc.attend(got, cu, n, L.table_out_h, qrf, scale, False)
    _check_attention(out2, torch.from_numpy(r2["lse"].astype(np.float32)).cuda(), r2, 64, "over what is left")
    # one more block into the evicted cache, where the pages have room
    rng = np.random.default_rng(61)
    d, F, V = 256, 512, 1000
    hidden = out2.reshape(64, d)
    dev = lambda shape, std: dev_bf16(bf16(rng, shape, std)[0])
    ffn = mtl.SwiGLUFFN(dev((F, d), 0.05), dev((F, d), 0.05), dev((d, F), 0.05), 64)
    rd = mtl.MaskedReadout(dev((V, d), 0.05), 64, 4)
    o = rd.outputs()
    mask, tokens = torch.ones(64, dtype=torch.uint8, device="cuda"), torch.full((64,), V, dtype=torch.int32, device="cuda")
    rd.step(ffn(hidden), mask, tokens, 4, out=o)
    torch.cuda.synchronize()
    assert int(o["n_out"]) == 4 and int(mask.sum()) == 60 and int((tokens < V).sum()) == 4
    rd.close()


def test_graphs_replay_to_the_same_bits():
    """Two layers' calls captured in a graph each, replayed in turn with eager work between, and once with other
    lengths in the buffers that they read."""
    import torch
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        layers = [_Layer(70), _Layer(71)]
        eager = []
        for L in layers:
            outs = L.run()
            eager.append(L.results(outs))
            L.reset()
        s.synchronize()
        graphs = []
        for L in layers:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                outs = L.run()
            graphs.append((g, outs))
        for turn in range(4):
            for L, (g, outs), want in zip(layers, graphs, eager):
                L.reset()
                g.replay()
                junk = torch.randn(1 << 20, device="cuda").sum()       # eager work between
                assert _same(L.results(outs), want), f"replay {turn}"
                if turn % 2:
                    s.synchronize()
                assert torch.isfinite(junk)
        for L, (g, outs) in zip(layers, graphs):                       # shorter sequences, the same graph
            L.b.lens.copy_(dev_i32([150, 137]))
            L.keep.copy_(dev_i32([40, 0]))
            L.reset()
            want = L.results(L.run())
            L.reset()
            g.replay()
            got = L.results(outs)
            assert int(L.lens_out[0]) == 40 and int(L.lens_out[1]) == 0
            assert _same(got, want)
        s.synchronize()


def test_streams():
    """Objects with a stream of their own, called while another is current; the current stream of the moment where
    they have none; and inputs dropped at once."""
    import torch
    want = _Layer(80)
    want = want.results(want.run())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    L = _Layer(80, stream=s)
    torch.cuda.synchronize()
    outs = L.run()
    for name in ("tq", "tk", "tv", "pos", "start", "b", "keep"):
        setattr(L, name, None)                                         # still being read
    junk = [torch.full((64, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(20)]
    s.synchronize()
    assert _same(L.results(outs), want) and len(junk) == 20
    L = _Layer(80)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        outs = L.run()
        s.synchronize()
        assert _same(L.results(outs), want)


def test_pool_past_32_bit_offsets():
    """Pages whose bytes lie 4 GiB and more behind the pool's start, and a batch whose new tokens lie as far
    apart: the same bits as in a small pool."""
    import torch

    import masked_token_logits_amd as mtl
    rng = np.random.default_rng(90)
    D, H, Hq, lens, new = 128, 2, 4, [100, 75], [20, 33]
    far = (5 << 30) // (H * 32 * D)
    table, pages = tables(rng, lens)
    c = cache(rng, pages, H, D, [a - b for a, b in zip(lens, new)], table)
    bad = (table < 0) | (table >= pages)
    q, k, v = (dev_bf16(bf16(rng, (53, h, D))[0]) for h in (Hq, H, H))
    keep, start = dev_i32([40, 64]), dev_i32([a - b for a, b in zip(lens, new)])
    res = []
    for base in (0, far):
        n = base + pages + 4
        t = {}
        for name in "kv":
            t[name] = torch.empty((n, H, 32 * D), dtype=torch.uint8, device="cuda")
            t[name][base:base + pages] = torch.from_numpy(c[name]).cuda()
            t[name + "_scale"] = torch.empty((n, H), dtype=torch.uint8, device="cuda")
            t[name + "_scale"][base:base + pages] = torch.from_numpy(c[name + "_scale"]).cuda()
        bc = mtl.BlockCache.over(t["k"], t["v"], t["k_scale"], t["v_scale"])
        b = bc.batch(dev_i32(cu_of(new)), dev_i32(lens), dev_i32(np.where(bad, -1, table + base)))
        bc.write(b, k, v, start)
        o, l = bc.attend(b, q, lse=True)
        w = torch.zeros(2, H, table.shape[1] * 32, device="cuda")
        bc.weigh(b, q, l, w)
        table_out = dev_i32((base + pages + np.arange(4)).reshape(2, 2))
        lens_out, kept, wout = bc.evict(b, w, keep, table_out)
        o2 = bc.attend(bc.batch(dev_i32(cu_of(new)), lens_out, table_out), q)
        res.append([o, l, w, lens_out, kept[0, :, :40], kept[1], o2] +
                   [t[name][base:].clone() for name in ("k", "v", "k_scale", "v_scale")])
        del t, bc
    assert _same(*res)


def test_nothing_to_do():
    """No new tokens at all, or none of the sequences has any: nothing is written."""
    import torch
    rng = np.random.default_rng(91)
    D, H, lens = 64, 2, [40, 0]
    table, pages = tables(rng, lens)
    c = cache(rng, pages, H, D, lens, table)
    bc = on_gpu(c)
    for T, cu in ((0, [0, 0, 0]), (5, [0, 0, 0]), (5, [5, 5, 5])):
        b = bc.batch(dev_i32(cu), dev_i32(lens), dev_i32(table))
        x = torch.randn(T, H, D, device="cuda").to(torch.bfloat16)
        bc.write(b, x, x, dev_i32([3, 0]))
        out = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
        _, lse = bc.attend(b, x, out=out, lse=True)
        w = torch.rand(2, H, table.shape[1] * 32, device="cuda")
        w0 = w.clone()
        bc.weigh(b, x, lse, w, decay=1.0)
        assert torch.all(out == 7) and torch.equal(w, w0)
    got = host(bc)
    for name in c:
        np.testing.assert_array_equal(got[name], c[name], err_msg=name)


def test_a_new_cache_is_filled_before_its_stream_writes():
    """A cache made with a stream while the current one is busy: the first write, queued at once, comes behind the
    fill of the pool."""
    import torch

    import masked_token_logits_amd as mtl
    rng = np.random.default_rng(92)
    D, H, pages = 64, 2, 4096
    k, v = (dev_bf16(bf16(rng, (40, H, D))[0]) for _ in "kv")
    cu, lens, table, start = dev_i32([0, 40]), dev_i32([40]), dev_i32([[pages - 1, 0]]), dev_i32([0])
    busy = torch.randn(4096, 4096, device="cuda").to(torch.bfloat16)
    s = torch.cuda.Stream()
    res = []
    for stream in (None, s):
        torch.cuda.synchronize()
        if stream is not None:
            for _ in range(30):
                busy = torch.mm(busy, busy).clamp_(-1, 1)
        bc = mtl.BlockCache(pages, H, D, stream=stream)
        bc.write(bc.batch(cu, lens, table), k, v, start)
        torch.cuda.synchronize()
        res.append([t.clone() for t in (bc.k, bc.v, bc.k_scale, bc.v_scale)])
    assert _same(*res)
    assert torch.any(res[0][0][pages - 1]) and not torch.any(res[0][0][1:pages - 1]) and torch.all(res[0][2][1:pages - 1] == 127)
