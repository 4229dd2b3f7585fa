"""The host side of the rotary and block cache C ABI and their binding:
frequencies against the oracle, argument refusals before any HIP call, and
the tensor checks of Rotary, CacheBatch and BlockCache.  No GPU."""
import numpy as np
import pytest
import torch

import masked_token_logits_amd as mtl
from masked_token_logits_amd import _abi
from oracle import cache as oc

FAKE = 0x7F0000000000   # aligned, never dereferenced
E = mtl


@pytest.mark.parametrize("r", [2, 6, 64, 128, 512])
@pytest.mark.parametrize("scaling,kw", [("none", {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
                                        ("ramp", dict(factor=16.0, original_len=4096, fast=32.0, slow=1.0))])
def test_frequencies(r, scaling, kw):
    if scaling == "base" and r == 2:
        pytest.skip("refused, below")
    st, turns = mtl.dllm_rotary_frequencies(r, 10000.0, _abi.ROTARY_SCALINGS[scaling], kw.get("factor", 1.0),
                                            kw.get("original_len", 0), kw.get("fast", 32.0), kw.get("slow", 1.0))
    assert st == E.DLLM_OK
    # pow on both sides is within an ulp or two, the rest is a handful of fp64 operations
    np.testing.assert_allclose(np.array(turns) * 2 * np.pi, oc.rotary_theta(r, 10000.0, scaling, **kw), rtol=2.0 ** -48)


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=3), dict(rotary_dim=514), dict(base=1.0), dict(base=float("inf")),
    dict(scaling=4), dict(scaling=-1), dict(scaling=1, factor=0.5), dict(scaling=1, factor=float("nan")),
    dict(scaling=2, factor=2.0, rotary_dim=2), dict(scaling=3, factor=2.0, original_len=0),
    dict(scaling=3, factor=2.0, original_len=10, fast=1.0, slow=1.0),
])
def test_frequencies_refused(kw):
    a = dict(rotary_dim=64)
    a.update(kw)
    assert mtl.dllm_rotary_frequencies(**a)[0] == E.DLLM_ERR_INVALID_ARG


def _plan(**kw):
    a = dict(turns=FAKE, magnitude=1.0, rotary_dim=64, layout=0)
    a.update(kw)
    return mtl.dllm_rotary_plan(**a)


def _rotary(plan=None, **kw):
    a = dict(plan=plan or _plan(), x=FAKE, T=4, H=2, D=64, x_token=128, x_head=64, positions=FAKE, transpose=0,
             y=FAKE + 4096, y_token=128, y_head=64)
    a.update(kw)
    return mtl.dllm_rotary(**a)


def test_rotary_refused():
    for bad in (_plan(turns=None), _plan(magnitude=0.0), _plan(magnitude=float("nan")), _plan(rotary_dim=65),
                _plan(rotary_dim=0), _plan(rotary_dim=66), _plan(layout=2)):
        assert _rotary(bad) == E.DLLM_ERR_INVALID_ARG
    for kw in (dict(x=None), dict(y=None), dict(positions=None), dict(T=-1), dict(T=1 << 31), dict(H=0), dict(D=0),
               dict(transpose=2), dict(x_token=-1), dict(y_head=-64),
               dict(y_token=64), dict(y_head=32), dict(y_token=0),      # outputs that share elements
               dict(y=FAKE, y_token=256)):                              # in place with other strides
        assert _rotary(**kw) == E.DLLM_ERR_INVALID_ARG, kw
    assert _rotary(D=514, y_token=1028, y_head=514) == E.DLLM_ERR_UNSUPPORTED
    assert _rotary(T=0, x=None) == E.DLLM_OK
    if not torch.cuda.is_available():
        assert _rotary() == E.DLLM_ERR_HIP
        assert _rotary(y_token=64, y_head=256) == E.DLLM_ERR_HIP        # [H, T, D] in memory


def _cache(**kw):
    a = dict(k=FAKE, v=FAKE + (1 << 30), k_scale=FAKE + 1, v_scale=FAKE + 3, pages=100, kv_heads=4, head_dim=128)
    a.update(kw)
    return mtl.dllm_cache(**a)


def _batch(**kw):
    a = dict(cu=FAKE, lens=FAKE + 64, table=FAKE + 128, S=3, table_blocks=10, max_new=8, max_len=320)
    a.update(kw)
    return mtl.dllm_cache_batch(**a)


BAD_CACHES = [(dict(k=None), 1), (dict(v_scale=None), 1), (dict(pages=0), 1), (dict(kv_heads=0), 1),
              (dict(head_dim=96), 2), (dict(head_dim=0), 2), (dict(pages=1 << 31), 2), (dict(k=FAKE + 8), 2)]
BAD_BATCHES = [dict(cu=None), dict(lens=None), dict(table=None), dict(S=0), dict(S=65536), dict(table_blocks=0),
               dict(max_new=0), dict(max_len=0), dict(max_len=321), dict(table_blocks=1 << 26)]


def _write(cache=None, batch=None, **kw):
    a = dict(cache=cache or _cache(), batch=batch or _batch(), T=20, k=FAKE, k_token=512, k_head=128, v=FAKE,
             v_token=512, v_head=128, start=FAKE, positions=FAKE, plan=_plan())
    a.update(kw)
    return mtl.dllm_cache_write(**a)


def _attend(cache=None, batch=None, **kw):
    a = dict(cache=cache or _cache(), batch=batch or _batch(), T=20, q=FAKE, q_token=1024, q_head=128, q_heads=8,
             scale=0.1, causal=0, out=FAKE, lse=None, workspace=FAKE, workspace_bytes=1 << 40)
    a.update(kw)
    return mtl.dllm_cache_attention(**a)


def _weigh(cache=None, batch=None, **kw):
    a = dict(cache=cache or _cache(), batch=batch or _batch(), T=20, q=FAKE, q_token=1024, q_head=128, q_heads=8,
             scale=0.1, causal=0, lse=FAKE, decay=1.0, weights=FAKE)
    a.update(kw)
    return mtl.dllm_cache_weigh(**a)


def _evict(cache=None, batch=None, **kw):
    a = dict(cache=cache or _cache(), batch=batch or _batch(), weights=FAKE, keep=FAKE + 512, max_keep=64, sink=0,
             recent=0, pool=3, table_out=FAKE + 1024, out_blocks=2, lens_out=FAKE + 2048, kept=FAKE + 4096,
             weights_out=FAKE + 8192, workspace=FAKE, workspace_bytes=1 << 40)
    a.update(kw)
    return mtl.dllm_cache_evict(**a)


@pytest.mark.parametrize("call", [_write, _attend, _weigh, _evict])
def test_cache_and_batch_refused(call):
    for kw, st in BAD_CACHES:
        assert call(cache=_cache(**kw)) == st, kw
    for kw in BAD_BATCHES:
        assert call(batch=_batch(**kw)) == E.DLLM_ERR_INVALID_ARG, kw
    if not torch.cuda.is_available():
        assert call() == E.DLLM_ERR_HIP


def test_write_refused():
    for kw in (dict(k=None), dict(v=None), dict(start=None), dict(positions=None), dict(T=-1), dict(T=1 << 31),
               dict(k_token=-1), dict(v_head=-1), dict(plan=_plan(rotary_dim=130)), dict(plan=_plan(turns=None))):
        assert _write(**kw) == E.DLLM_ERR_INVALID_ARG, kw
    assert _write(k_token=1 << 31) == E.DLLM_ERR_UNSUPPORTED
    assert _write(cache=_cache(kv_heads=65536)) == E.DLLM_ERR_UNSUPPORTED
    assert _write(T=0, k=None) == E.DLLM_OK


def test_attention_and_weigh_refused():
    for call in (_attend, _weigh):
        for kw in (dict(q=None), dict(T=-1), dict(q_heads=0), dict(q_heads=6), dict(scale=0.0), dict(scale=-1.0),
                   dict(scale=float("nan")), dict(scale=float("inf")), dict(causal=2), dict(q_token=-8)):
            assert call(**kw) == E.DLLM_ERR_INVALID_ARG, kw
        for kw in (dict(q_token=1020), dict(q_head=4), dict(q=FAKE + 2), dict(q_token=1 << 31)):
            assert call(**kw) == E.DLLM_ERR_UNSUPPORTED, kw
    assert _attend(out=None) == E.DLLM_ERR_INVALID_ARG
    assert _attend(out=FAKE + 8) == E.DLLM_ERR_UNSUPPORTED
    assert _attend(T=0, q=None) == E.DLLM_OK
    for kw in (dict(workspace=None), dict(workspace_bytes=8), dict(workspace=FAKE + 16)):
        assert _attend(**kw) == E.DLLM_ERR_WORKSPACE, kw
    for kw in (dict(lse=None), dict(weights=None), dict(decay=-0.1), dict(decay=1.5), dict(decay=float("nan"))):
        assert _weigh(**kw) == E.DLLM_ERR_INVALID_ARG, kw
    assert mtl.dllm_cache_attention_workspace_bytes(_cache(), _batch(), 8) > 0
    assert mtl.dllm_cache_attention_workspace_bytes(_cache(), _batch(), 6) == 0
    assert mtl.dllm_cache_attention_workspace_bytes(_cache(head_dim=80), _batch(), 8) == 0


def test_evict_refused():
    for kw in (dict(weights=None), dict(keep=None), dict(table_out=None), dict(lens_out=None), dict(kept=None),
               dict(sink=-1), dict(recent=-1), dict(pool=0), dict(pool=2), dict(pool=65), dict(max_keep=0),
               dict(max_keep=65), dict(out_blocks=0), dict(weights_out=FAKE), dict(lens_out=FAKE + 64),
               dict(lens_out=FAKE + 512), dict(table_out=FAKE + 128)):
        assert _evict(**kw) == E.DLLM_ERR_INVALID_ARG, kw
    for kw in (dict(workspace=None), dict(workspace_bytes=8), dict(workspace=FAKE + 16)):
        assert _evict(**kw) == E.DLLM_ERR_WORKSPACE, kw
    assert mtl.dllm_cache_evict_workspace_bytes(_cache(), _batch()) > 0
    assert mtl.dllm_cache_evict_workspace_bytes(_cache(pages=0), _batch()) == 0


# ---- the binding's tensor checks (CPU tensors) ----------------------------------------------------------------

def _objects():
    cache = mtl.BlockCache(12, 2, 64, device="cpu")
    i = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return cache, cache.batch(i(0, 3, 5), i(40, 33), torch.zeros((2, 3), dtype=torch.int32)), i


def test_rotary_object_checks():
    for kw in (dict(layout="other"), dict(scaling="other"), dict(rotary_dim=130), dict(magnitude=0.0)):
        with pytest.raises(ValueError):
            mtl.Rotary(128, device="cpu", **kw)
    with pytest.raises(mtl.DllmError):
        mtl.Rotary(128, rotary_dim=5, device="cpu")
    rot = mtl.Rotary(64, device="cpu")
    x, pos = torch.zeros((5, 2, 64), dtype=torch.bfloat16), torch.zeros(5, dtype=torch.int32)
    for a in ((x.float(), pos), (x, pos.long())):
        with pytest.raises(TypeError):
            rot(*a)
    for a in ((x[..., :32], pos), (x[0], pos), (x, pos[:4]), (x.transpose(1, 2).contiguous().transpose(1, 2), pos),
              (x, pos, x[:4]), (x, pos, x.view(torch.int16))):
        with pytest.raises(ValueError):
            rot(*a)


def test_attention_in_place_refused():
    cache, batch, _ = _objects()
    q = torch.zeros((5, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        cache.attend(batch, q, out=q)


def test_streams_of_another_device_refused():
    import types
    other = types.SimpleNamespace(device=torch.device("cuda", 1))
    c = mtl.BlockCache(4, 2, 64, device="cpu")
    for make in (lambda: mtl.Rotary(64, device="cpu", stream=other),
                 lambda: mtl.BlockCache(4, 2, 64, device="cpu", stream=other),
                 lambda: mtl.BlockCache.over(c.k, c.v, c.k_scale, c.v_scale, stream=other)):
        with pytest.raises(ValueError):
            make()


def test_batch_checks():
    cache, _, i = _objects()
    t = torch.zeros((2, 3), dtype=torch.int32)
    for a in ((i(0, 3), i(4, 4), t), (i(0, 3, 5), i(4), t), (i(0, 3, 5), i(4, 4), t[0]),
              (i(0, 3, 5), i(4, 4), torch.zeros((3, 2), dtype=torch.int32).t())):
        with pytest.raises(ValueError):
            cache.batch(*a)
    with pytest.raises(TypeError):
        cache.batch(i(0, 3, 5).long(), i(4, 4), t)
    for kw in (dict(max_len=97), dict(max_len=0), dict(max_new=0)):
        with pytest.raises(ValueError):
            cache.batch(i(0, 3, 5), i(4, 4), t, **kw)


def test_cache_object_checks():
    cache, batch, i = _objects()
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError):
        mtl.BlockCache(4, 2, 96, device="cpu")
    with pytest.raises(ValueError):
        mtl.BlockCache.over(cache.k, cache.v[:4], cache.k_scale, cache.v_scale)
    with pytest.raises(TypeError):
        mtl.BlockCache.over(cache.k, cache.v, cache.k_scale.int(), cache.v_scale)
    k = bf(5, 2, 64)
    for a, kw in (((bf(5, 3, 64), k, i(0, 0)), {}), ((k, bf(4, 2, 64), i(0, 0)), {}), ((k, k, i(0)), {}),
                  ((k, k, i(0, 0)), dict(positions=i(0, 1, 2, 3, 4))),
                  ((k, k, i(0, 0)), dict(positions=i(0, 1), rotary=mtl.Rotary(64, device="cpu"))),
                  ((k, k, i(0, 0)), dict(positions=i(0, 1, 2, 3, 4), rotary=mtl.Rotary(128, device="cpu")))):
        with pytest.raises(ValueError):
            cache.write(batch, *a, **kw)
    with pytest.raises(TypeError):
        cache.write(None, k, k, i(0, 0))
    q = bf(5, 4, 64)
    f32 = lambda *s: torch.zeros(s)  # noqa: E731
    for kw in (dict(q=bf(5, 3, 64)), dict(q=bf(5, 4, 32)), dict(out=bf(5, 4, 32)), dict(lse=f32(5, 3))):
        with pytest.raises(ValueError):
            cache.attend(batch, **{**dict(q=q), **kw})
    with pytest.raises(TypeError):
        cache.attend(batch, q, out=f32(5, 4, 64))
    for lse, w in ((f32(5, 3), f32(2, 2, 96)), (f32(5, 4), f32(2, 2, 95)), (f32(5, 4), f32(2, 4, 96))):
        with pytest.raises(ValueError):
            cache.weigh(batch, q, lse, w)
    w, to = f32(2, 2, 96), torch.zeros((2, 2), dtype=torch.int32)
    for a, kw in (((w[:1], i(1, 1), to), {}), ((w, i(1), to), {}), ((w, i(1, 1), to[0]), {}),
                  ((w, i(1, 1), to), dict(kept=torch.zeros((2, 2, 65), dtype=torch.int32))),
                  ((w, i(1, 1), to), dict(weights_out=f32(2, 2, 96))), ((w, i(1, 1), to), dict(lens_out=i(1)))):
        with pytest.raises(ValueError):
            cache.evict(batch, *a, **kw)
    if not torch.cuda.is_available():   # valid calls pass the checks and reach the library
        for f in (lambda: cache.write(batch, k, k, i(0, 0)), lambda: cache.attend(batch, q, lse=True),
                  lambda: cache.weigh(batch, q, f32(5, 4), w), lambda: cache.evict(batch, w, i(1, 1), to)):
            with pytest.raises(mtl.DllmError) as e:
                f()
            assert e.value.status in (E.DLLM_ERR_HIP, E.DLLM_ERR_UNSUPPORTED, E.DLLM_ERR_WORKSPACE)


# ---- the oracle against other statements of the same things ----------------------------------------------------

def test_oracle_e4m3_against_torch():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(oc.E4M3, v)
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(20000) * 100, rng.standard_normal(20000) * 0.01, oc.E4M3[:127],
                        (oc.E4M3[:126] + oc.E4M3[1:127]) / 2])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(oc.e4m3_bytes(x), want)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_oracle_places(D):
    for key in (True, False):
        assert sorted(oc.places(D, key).ravel()) == list(range(32 * D))
    assert oc.k_place(5, D // 2 + 17, D) == (1 * 2 + 1) * 512 + 5 * 16 + 1
    assert oc.v_place(13, 33, D) == (1 * 2 + 1) * 512 + 1 * 16 + 1 * 4 + 1


def test_oracle_attention_against_torch():
    rng = np.random.default_rng(2)
    from _cache_cases import cache as make
    c = make(rng, 6, 1, 64)
    table, q = np.array([[4, 1, 0]], np.int32), rng.standard_normal((4, 2, 64))
    r = oc.attend(c, [0, 4], [70], table, q, 0.2, True)
    k, _ = oc.read_tokens(c, "k", table[0], 0, 70)
    v, _ = oc.read_tokens(c, "v", table[0], 0, 70)
    z = torch.from_numpy(0.2 * np.einsum("thd,jd->thj", q, k))
    z[:, :] += torch.full((4, 70), -np.inf, dtype=torch.float64).triu(67)[:, None]
    np.testing.assert_allclose(r["out"], (torch.softmax(z, -1) @ torch.from_numpy(v)).numpy(), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(r["lse"], torch.logsumexp(z, -1).numpy(), rtol=1e-13)
    w = oc.weigh(c, [0, 4], [70], table, q, r["lse"], 0.2, True, np.zeros((1, 1, 96)), 1.0)
    np.testing.assert_allclose(w[0, 0, :70], torch.softmax(z, -1).sum((0, 1)).numpy(), rtol=1e-10)


def test_oracle_select():
    w = np.array([5, 1, 1, 9, 1, 1, 1, 4, 1, 2.0])
    assert oc.select(w, 3, 0, 0, 1).tolist() == [0, 3, 7]
    assert oc.select(w, 4, 0, 0, 3).tolist() == [0, 2, 3, 4]      # 9 lifts its neighbours
    assert oc.select(w, 4, 1, 2, 1).tolist() == [0, 3, 8, 9]
    assert oc.select(np.ones(6), 3, 0, 0, 1).tolist() == [0, 1, 2]
    assert oc.select(w, 99, 2, 2, 3).tolist() == list(range(10))


def test_oracle_refuses_what_a_scale_does_not_hold():
    oc.e4m3_bytes(np.array([448.0, -448.0 * (1 + 2.0 ** -21), np.inf, np.nan]))
    with pytest.raises(ValueError):
        oc.e4m3_bytes(np.array([1.0, -449.0]))


class _Library:
    """Stands in for the loaded library: workspace sizes are 256, and kernel launches are noted."""

    def __init__(self):
        self.launched = []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_bytes"):
                return 256
            self.launched.append(name)
            return E.DLLM_OK
        return call


def test_objects_off_the_gpu_launch_nothing(monkeypatch):
    """Objects of another device than a GPU are refused before the library gets their pointers, whether or not there is a
    GPU whose kernels would take them for their own."""
    cache, batch, i = _objects()
    rot = mtl.Rotary(64, device="cpu")
    k, q = torch.zeros((5, 2, 64), dtype=torch.bfloat16), torch.zeros((5, 4, 64), dtype=torch.bfloat16)
    w, lse, to = torch.zeros((2, 2, 96)), torch.zeros((5, 4)), torch.zeros((2, 2), dtype=torch.int32)
    lib = _Library()
    with monkeypatch.context() as m:
        m.setattr(_abi, "load", lambda *a: lib)
        m.setattr(_abi, "dllm_status_string", str)
        for f in (lambda: rot(k, i(0, 1, 2, 3, 4)), lambda: rot(k, i(0, 1, 2, 3, 4), out=k, transpose=True),
                  lambda: cache.write(batch, k, k, i(0, 0)),
                  lambda: cache.write(batch, k, k, i(0, 0), positions=i(0, 1, 2, 3, 4), rotary=rot),
                  lambda: cache.attend(batch, q, lse=True), lambda: cache.weigh(batch, q, lse, w),
                  lambda: cache.evict(batch, w, i(1, 1), to)):
            with pytest.raises(mtl.DllmError) as e:
                f()
            assert e.value.status == E.DLLM_ERR_UNSUPPORTED
    assert lib.launched == []


def test_batch_of_another_device_refused():
    cache, _, i = _objects()
    other = mtl.BlockCache(12, 2, 64, device="meta")
    meta = lambda *s: torch.zeros(s, dtype=torch.int32, device="meta")  # noqa: E731
    batch = other.batch(meta(3), meta(2), meta(2, 3))
    k, q = torch.zeros((5, 2, 64), dtype=torch.bfloat16), torch.zeros((5, 4, 64), dtype=torch.bfloat16)
    w, lse, to = torch.zeros((2, 2, 96)), torch.zeros((5, 4)), torch.zeros((2, 2), dtype=torch.int32)
    for f in (lambda: cache.write(batch, k, k, i(0, 0)), lambda: cache.attend(batch, q),
              lambda: cache.weigh(batch, q, lse, w), lambda: cache.evict(batch, w, i(1, 1), to)):
        with pytest.raises(ValueError, match="batch"):
            f()


def test_attention_outputs_that_overlap_the_queries_refused():
    cache, batch, _ = _objects()
    flat = torch.zeros(4096 * 8, dtype=torch.bfloat16)
    n = 5 * 4 * 64
    at = lambda i: flat[i:i + n].view(5, 4, 64)  # noqa: E731
    fused = flat[:3 * n].view(5, 12, 64)[:, 4:8]
    spread = flat[:5 * 6000].view(5, 6000)[:, :256].view(5, 4, 64)      # rows far apart, room between them
    turned = flat[:n].view(4, 5, 64).transpose(0, 1)
    one = flat[:64].view(1, 1, 64).expand(5, 4, 64)
    f32 = flat.view(torch.float32)
    for q, kw in ((at(0), dict(out=at(256))), (at(256), dict(out=at(0))), (fused, dict(out=at(256))),
                  (fused, dict(out=at(768 * 4 + 448))), (spread, dict(out=at(24000 - n + 8))), (turned, dict(out=at(n - 64))),
                  (one, dict(out=at(0))), (at(0), dict(lse=f32[100:120].view(5, 4))),
                  (at(n), dict(out=at(4 * n), lse=f32[2 * n + 8:2 * n + 28].view(5, 4)))):
        with pytest.raises(ValueError, match="overlap"):
            cache.attend(batch, q, **kw)
    for q, kw in ((at(0), dict(out=at(n))), (at(n), dict(out=at(0))), (fused, dict(out=at(768 * 4 + 512))), (spread, dict(out=at(256))),
                  (spread, dict(out=at(6000 - n))), (one, dict(out=at(64))), (at(0), dict(lse=f32[n // 2:n // 2 + 20].view(5, 4)))):
        with pytest.raises(mtl.DllmError):                              # on to the call, which needs a GPU
            cache.attend(batch, q, **kw)
