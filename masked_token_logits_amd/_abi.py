"""ctypes binding of libdllm_readout.so (argument marshalling only).

The functions carry the C names and C argument order; device buffers may be
given as torch tensors (their data pointers are passed) or plain integers.
Every step of the readout runs in the library's HIP kernels; there is no
Python or CPU fallback, and loading fails loudly when the library is absent.
"""
from __future__ import annotations

import ctypes as C
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdllm_readout.so")

DLLM_OK = 0
DLLM_ERR_INVALID_ARG = 1
DLLM_ERR_UNSUPPORTED = 2
DLLM_ERR_WORKSPACE = 3
DLLM_ERR_HIP = 4
DLLM_K_MAX_LIMIT = 4096
DLLM_BATCH_MAX = 128
DLLM_NOALLOC_SCRATCH_BYTES = 32 << 20

DLLM_SCORE_CONF = 0
DLLM_SCORE_MARGIN = 1
DLLM_SCORE_NEG_ENTROPY = 2
SCORES = {"conf": DLLM_SCORE_CONF, "margin": DLLM_SCORE_MARGIN, "neg_entropy": DLLM_SCORE_NEG_ENTROPY}

EXPORTED = (
    "dllm_masked_readout_workspace_bytes",
    "dllm_masked_readout_create",
    "dllm_masked_readout_step",
    "dllm_masked_readout_step_ex",
    "dllm_masked_readout_step_batch",
    "dllm_masked_readout_destroy",
    "dllm_status_string",
    "dllm_masked_readout_set_slices",
    "dllm_masked_readout_set_gemm_events",
    "dllm_masked_readout_step_noalloc",
    "dllm_ffn_workspace_bytes",
    "dllm_ffn_pack_gate_up",
    "dllm_ffn_swiglu_chunked",
    "dllm_probe_source_bytes",
    "dllm_probe_wall_clock_khz",
    "dllm_probe_gemm_mix",
    "dllm_rotary_frequencies",
    "dllm_rotary",
    "dllm_cache_write",
    "dllm_cache_attention_workspace_bytes",
    "dllm_cache_attention",
    "dllm_cache_weigh",
    "dllm_cache_evict_workspace_bytes",
    "dllm_cache_evict",
    "dllm_residual_norm",
    "dllm_residual_norm_backward_workspace_bytes",
    "dllm_residual_norm_backward",
    "dllm_embed",
    "dllm_embed_backward_workspace_bytes",
    "dllm_embed_backward",
    "dllm_loss_forward_workspace_bytes",
    "dllm_loss_forward",
    "dllm_loss_backward_workspace_bytes",
    "dllm_loss_backward",
)

DLLM_ROTARY_HALF = 0
DLLM_ROTARY_INTERLEAVED = 1
ROTARY_LAYOUTS = {"half": DLLM_ROTARY_HALF, "interleaved": DLLM_ROTARY_INTERLEAVED}
DLLM_ROTARY_PLAIN = 0
DLLM_ROTARY_LINEAR = 1
DLLM_ROTARY_BASE = 2
DLLM_ROTARY_RAMP = 3
ROTARY_SCALINGS = {"none": DLLM_ROTARY_PLAIN, "linear": DLLM_ROTARY_LINEAR, "base": DLLM_ROTARY_BASE,
                   "ramp": DLLM_ROTARY_RAMP}
DLLM_ROTARY_DIM_MAX = 512
DLLM_CACHE_BLOCK = 32
DLLM_NORM_DIM_MAX = 8192


class dllm_step_out(C.Structure):
    _fields_ = [
        ("n_out", C.c_void_p),
        ("m_out", C.c_void_p),
        ("sel_idx", C.c_void_p),
        ("sel_tok", C.c_void_p),
        ("sel_conf", C.c_void_p),
        ("row_idx", C.c_void_p),
        ("row_tok", C.c_void_p),
        ("row_conf", C.c_void_p),
        ("row_lse", C.c_void_p),
        ("row_margin", C.c_void_p),
        ("row_entropy", C.c_void_p),
    ]


class dllm_seq(C.Structure):
    _fields_ = [
        ("k", C.c_int32),
        ("win_lo", C.c_int32),
        ("win_hi", C.c_int32),
    ]


class dllm_policy(C.Structure):
    _fields_ = [
        ("score", C.c_int32),
        ("use_threshold", C.c_int32),
        ("tau", C.c_float),
    ]


class dllm_rotary_plan(C.Structure):
    _fields_ = [
        ("turns", C.c_void_p),
        ("magnitude", C.c_float),
        ("rotary_dim", C.c_int32),
        ("layout", C.c_int32),
    ]


class dllm_cache(C.Structure):
    _fields_ = [
        ("k", C.c_void_p),
        ("v", C.c_void_p),
        ("k_scale", C.c_void_p),
        ("v_scale", C.c_void_p),
        ("pages", C.c_int64),
        ("kv_heads", C.c_int32),
        ("head_dim", C.c_int32),
    ]


class dllm_cache_batch(C.Structure):
    _fields_ = [
        ("cu", C.c_void_p),
        ("lens", C.c_void_p),
        ("table", C.c_void_p),
        ("S", C.c_int32),
        ("table_blocks", C.c_int32),
        ("max_new", C.c_int32),
        ("max_len", C.c_int32),
    ]


class dllm_norm(C.Structure):
    _fields_ = [
        ("pre", C.c_void_p),
        ("post", C.c_void_p),
        ("d", C.c_int64),
        ("eps", C.c_float),
        ("scale", C.c_float),
    ]


class dllm_loss(C.Structure):
    _fields_ = [
        ("W_lm", C.c_void_p),
        ("hidden", C.c_void_p),
        ("mask", C.c_void_p),
        ("targets", C.c_void_p),
        ("weights", C.c_void_p),
        ("V", C.c_int64),
        ("d", C.c_int64),
        ("L", C.c_int64),
    ]


_lib = None


def load(path: str = LIB_PATH):
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m masked_token_logits_amd.build`")
    # The library must share the process's HIP runtime with PyTorch, which
    # allocates the buffers: with torch loaded first, the dynamic linker
    # resolves the library's libamdhip64 to torch's copy.  Loaded the other
    # way round, the process holds two runtimes and the library's sees no
    # device.
    try:
        import torch  # noqa: F401
    except ImportError:  # pragma: no cover - the library still loads (host-only uses)
        pass
    lib = C.CDLL(path)
    lib.dllm_masked_readout_workspace_bytes.restype = C.c_size_t
    lib.dllm_masked_readout_workspace_bytes.argtypes = [C.c_int64, C.c_int64, C.c_int64, C.c_int32]
    lib.dllm_masked_readout_create.restype = C.c_int
    lib.dllm_masked_readout_create.argtypes = [C.POINTER(C.c_void_p), C.c_void_p, C.c_int64, C.c_int64,
                                               C.c_int64, C.c_int32, C.c_void_p, C.c_size_t, C.c_void_p]
    lib.dllm_masked_readout_step.restype = C.c_int
    lib.dllm_masked_readout_step.argtypes = [C.c_void_p, C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p,
                                             C.c_int32, C.c_int64, C.c_int64, C.c_int64,
                                             C.POINTER(dllm_step_out)]
    lib.dllm_masked_readout_step_ex.restype = C.c_int
    lib.dllm_masked_readout_step_ex.argtypes = [C.c_void_p, C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p,
                                                C.c_int32, C.c_int64, C.c_int64, C.c_int64,
                                                C.POINTER(dllm_policy), C.POINTER(dllm_step_out)]
    lib.dllm_masked_readout_step_batch.restype = C.c_int
    lib.dllm_masked_readout_step_batch.argtypes = [C.c_void_p, C.c_int32, C.c_void_p, C.c_int64, C.c_void_p,
                                                   C.c_void_p, C.POINTER(dllm_seq), C.c_int64,
                                                   C.POINTER(dllm_policy), C.POINTER(dllm_step_out)]
    lib.dllm_masked_readout_destroy.restype = C.c_int
    lib.dllm_masked_readout_destroy.argtypes = [C.c_void_p]
    lib.dllm_status_string.restype = C.c_char_p
    lib.dllm_status_string.argtypes = [C.c_int]
    lib.dllm_masked_readout_set_slices.restype = C.c_int
    lib.dllm_masked_readout_set_slices.argtypes = [C.c_void_p, C.c_int32]
    lib.dllm_masked_readout_set_gemm_events.restype = C.c_int
    lib.dllm_masked_readout_set_gemm_events.argtypes = [C.c_void_p, C.c_void_p, C.c_void_p]
    lib.dllm_masked_readout_step_noalloc.restype = C.c_int
    lib.dllm_masked_readout_step_noalloc.argtypes = [C.c_void_p, C.c_int64, C.c_int64, C.c_void_p, C.c_int64,
                                                     C.c_void_p, C.c_void_p, C.c_int32, C.c_int64, C.c_int64,
                                                     C.c_int64, C.POINTER(dllm_policy), C.POINTER(dllm_step_out),
                                                     C.c_void_p]
    lib.dllm_probe_source_bytes.restype = C.c_size_t
    lib.dllm_probe_source_bytes.argtypes = []
    lib.dllm_probe_wall_clock_khz.restype = C.c_int64
    lib.dllm_probe_wall_clock_khz.argtypes = []
    lib.dllm_probe_gemm_mix.restype = C.c_int
    lib.dllm_probe_gemm_mix.argtypes = [C.c_int32, C.c_void_p, C.c_int32, C.c_void_p, C.c_int32, C.c_void_p,
                                        C.c_void_p]
    lib.dllm_ffn_workspace_bytes.restype = C.c_size_t
    lib.dllm_ffn_workspace_bytes.argtypes = [C.c_int64, C.c_int64]
    lib.dllm_ffn_pack_gate_up.restype = C.c_int
    lib.dllm_ffn_pack_gate_up.argtypes = [C.c_void_p, C.c_void_p, C.c_int64, C.c_int64, C.c_void_p, C.c_void_p]
    lib.dllm_ffn_swiglu_chunked.restype = C.c_int
    lib.dllm_ffn_swiglu_chunked.argtypes = [C.c_void_p, C.c_int64, C.c_int64, C.c_void_p, C.c_void_p, C.c_int64,
                                            C.c_int64, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]
    P, i32, i64, f32 = C.c_void_p, C.c_int32, C.c_int64, C.c_float
    plan_p, cache_p, batch_p = C.POINTER(dllm_rotary_plan), C.POINTER(dllm_cache), C.POINTER(dllm_cache_batch)
    lib.dllm_rotary_frequencies.restype = C.c_int
    lib.dllm_rotary_frequencies.argtypes = [i32, C.c_double, i32, C.c_double, i64, C.c_double, C.c_double,
                                            C.POINTER(C.c_double)]
    lib.dllm_rotary.restype = C.c_int
    lib.dllm_rotary.argtypes = [plan_p, P, i64, i32, i32, i64, i64, P, i32, P, i64, i64, P]
    lib.dllm_cache_write.restype = C.c_int
    lib.dllm_cache_write.argtypes = [cache_p, batch_p, i64, P, i64, i64, P, i64, i64, P, P, plan_p, P]
    lib.dllm_cache_attention_workspace_bytes.restype = C.c_size_t
    lib.dllm_cache_attention_workspace_bytes.argtypes = [cache_p, batch_p, i32]
    lib.dllm_cache_attention.restype = C.c_int
    lib.dllm_cache_attention.argtypes = [cache_p, batch_p, i64, P, i64, i64, i32, f32, i32, P, P, P, C.c_size_t, P]
    lib.dllm_cache_weigh.restype = C.c_int
    lib.dllm_cache_weigh.argtypes = [cache_p, batch_p, i64, P, i64, i64, i32, f32, i32, P, f32, P, P]
    lib.dllm_cache_evict_workspace_bytes.restype = C.c_size_t
    lib.dllm_cache_evict_workspace_bytes.argtypes = [cache_p, batch_p]
    lib.dllm_cache_evict.restype = C.c_int
    lib.dllm_cache_evict.argtypes = [cache_p, batch_p, P, P, i32, i32, i32, i32, P, i32, P, P, P, P, C.c_size_t, P]
    norm_p, loss_p, size = C.POINTER(dllm_norm), C.POINTER(dllm_loss), C.c_size_t
    lib.dllm_residual_norm.restype = C.c_int
    lib.dllm_residual_norm.argtypes = [norm_p, P, P, i64, P, i64, P, P, P]
    lib.dllm_residual_norm_backward_workspace_bytes.restype = size
    lib.dllm_residual_norm_backward_workspace_bytes.argtypes = [norm_p, i64, i64]
    lib.dllm_residual_norm_backward.restype = C.c_int
    lib.dllm_residual_norm_backward.argtypes = [norm_p, P, P, i64, P, i64, P, P, P, P, P, P, P, P, size, P]
    lib.dllm_embed.restype = C.c_int
    lib.dllm_embed.argtypes = [P, i64, i64, P, i64, f32, P, P]
    lib.dllm_embed_backward_workspace_bytes.restype = size
    lib.dllm_embed_backward_workspace_bytes.argtypes = [i64, i64, i64]
    lib.dllm_embed_backward.restype = C.c_int
    lib.dllm_embed_backward.argtypes = [P, i64, P, i64, i64, f32, i32, P, P, size, P]
    lib.dllm_loss_forward_workspace_bytes.restype = size
    lib.dllm_loss_forward_workspace_bytes.argtypes = [i64, i64, i64]
    lib.dllm_loss_forward.restype = C.c_int
    lib.dllm_loss_forward.argtypes = [loss_p, P, P, P, P, size, P]
    lib.dllm_loss_backward_workspace_bytes.restype = size
    lib.dllm_loss_backward_workspace_bytes.argtypes = [i64, i64, i64, i64]
    lib.dllm_loss_backward.restype = C.c_int
    lib.dllm_loss_backward.argtypes = [loss_p, P, P, P, P, i32, i64, P, size, P]
    _lib = lib
    return lib


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class DllmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {dllm_status_string(status)} (status {status})")


def dllm_status_string(status: int) -> str:
    return load().dllm_status_string(int(status)).decode()


def dllm_masked_readout_workspace_bytes(L_max: int, d: int, V: int, k_max: int) -> int:
    return int(load().dllm_masked_readout_workspace_bytes(L_max, d, V, k_max))


def dllm_masked_readout_create(W_lm, V: int, d: int, L_max: int, k_max: int, workspace,
                               workspace_bytes: int, stream=None) -> tuple[int, int | None]:
    """Returns (status, handle)."""
    h = C.c_void_p()
    st = load().dllm_masked_readout_create(C.byref(h), _ptr(W_lm), V, d, L_max, k_max, _ptr(workspace),
                                           workspace_bytes, _stream(stream))
    return st, h.value


def dllm_masked_readout_step(handle, hidden, L: int, mask, tokens, k: int, win_lo: int, win_hi: int,
                             block: int = 0, out: dict | None = None) -> int:
    """``out`` maps dllm_step_out field names to device buffers (optional)."""
    so = None
    if out:
        so = dllm_step_out(**{key: _ptr(v) for key, v in out.items()})
    return load().dllm_masked_readout_step(handle, _ptr(hidden), L, _ptr(mask), _ptr(tokens), k, win_lo, win_hi,
                                           block, C.byref(so) if so is not None else None)


def make_policy(score="conf", tau: float | None = None) -> dllm_policy:
    """dllm_policy for a score name ("conf", "margin", "neg_entropy") or
    dllm_score value; ``tau`` None = top-k, otherwise the threshold rule."""
    sc = SCORES[score] if isinstance(score, str) else int(score)
    if tau is None:
        return dllm_policy(sc, 0, 0.0)
    return dllm_policy(sc, 1, float(tau))


def dllm_masked_readout_step_ex(handle, hidden, L: int, mask, tokens, k: int, win_lo: int, win_hi: int,
                                block: int = 0, policy: dllm_policy | None = None,
                                out: dict | None = None) -> int:
    so = None
    if out:
        so = dllm_step_out(**{key: _ptr(v) for key, v in out.items()})
    return load().dllm_masked_readout_step_ex(handle, _ptr(hidden), L, _ptr(mask), _ptr(tokens), k, win_lo,
                                              win_hi, block, C.byref(policy) if policy is not None else None,
                                              C.byref(so) if so is not None else None)


def dllm_masked_readout_step_noalloc(W_lm, V: int, d: int, hidden, L: int, mask, tokens, k: int, win_lo: int,
                                     win_hi: int, block: int = 0, policy: dllm_policy | None = None,
                                     out: dict | None = None, stream=None) -> int:
    """The handle-free step on the library's static device scratch."""
    so = None
    if out:
        so = dllm_step_out(**{key: _ptr(v) for key, v in out.items()})
    return load().dllm_masked_readout_step_noalloc(_ptr(W_lm), V, d, _ptr(hidden), L, _ptr(mask), _ptr(tokens), k,
                                                   win_lo, win_hi, block,
                                                   C.byref(policy) if policy is not None else None,
                                                   C.byref(so) if so is not None else None, _stream(stream))


def dllm_probe_source_bytes() -> int:
    return int(load().dllm_probe_source_bytes())


def dllm_probe_wall_clock_khz() -> int:
    return int(load().dllm_probe_wall_clock_khz())


def dllm_probe_gemm_mix(mode: int, src, stages: int, sink, grid: int, clocks=None, stream=None) -> int:
    return load().dllm_probe_gemm_mix(int(mode), _ptr(src), int(stages), _ptr(sink), int(grid), _ptr(clocks),
                                      _stream(stream))


def dllm_masked_readout_step_batch(handle, B: int, hidden, L: int, mask, tokens, seqs, block: int = 0,
                                   policy: dllm_policy | None = None, out: dict | None = None) -> int:
    """``seqs``: B (k, win_lo, win_hi) triples (or a dllm_seq array)."""
    if not isinstance(seqs, C.Array):
        arr = (dllm_seq * max(len(seqs), 1))()
        for i, (k, lo, hi) in enumerate(seqs):
            arr[i] = dllm_seq(int(k), int(lo), int(hi))
        seqs = arr
    so = None
    if out:
        so = dllm_step_out(**{key: _ptr(v) for key, v in out.items()})
    return load().dllm_masked_readout_step_batch(handle, int(B), _ptr(hidden), int(L), _ptr(mask), _ptr(tokens),
                                                 seqs, int(block),
                                                 C.byref(policy) if policy is not None else None,
                                                 C.byref(so) if so is not None else None)


def dllm_ffn_workspace_bytes(chunk: int, F: int) -> int:
    return int(load().dllm_ffn_workspace_bytes(chunk, F))


def dllm_ffn_pack_gate_up(W_gate, W_up, F: int, d: int, W_gu, stream=None) -> int:
    return load().dllm_ffn_pack_gate_up(_ptr(W_gate), _ptr(W_up), F, d, _ptr(W_gu), _stream(stream))


def dllm_ffn_swiglu_chunked(X, L: int, d: int, W_gu, W_down, F: int, chunk: int, Y, workspace,
                            workspace_bytes: int, stream=None) -> int:
    return load().dllm_ffn_swiglu_chunked(_ptr(X), L, d, _ptr(W_gu), _ptr(W_down), F, chunk, _ptr(Y),
                                          _ptr(workspace), workspace_bytes, _stream(stream))


def dllm_masked_readout_destroy(handle) -> int:
    return load().dllm_masked_readout_destroy(handle)


def dllm_masked_readout_set_slices(handle, slices: int) -> int:
    return load().dllm_masked_readout_set_slices(handle, slices)


def dllm_masked_readout_set_gemm_events(handle, ev_before, ev_after) -> int:
    return load().dllm_masked_readout_set_gemm_events(handle, ev_before, ev_after)


def _ref(struct):
    return C.byref(struct) if struct is not None else None


def dllm_rotary_frequencies(rotary_dim: int, base: float = 10000.0, scaling: int = DLLM_ROTARY_PLAIN,
                            factor: float = 1.0, original_len: int = 0, fast: float = 32.0,
                            slow: float = 1.0) -> tuple[int, list[float]]:
    """Returns (status, turns per position of each pair)."""
    turns = (C.c_double * max(int(rotary_dim) // 2, 1))()
    st = load().dllm_rotary_frequencies(rotary_dim, base, scaling, factor, original_len, fast, slow, turns)
    return st, list(turns)


def dllm_rotary(plan, x, T: int, H: int, D: int, x_token: int, x_head: int, positions, transpose: int, y,
                y_token: int, y_head: int, stream=None) -> int:
    return load().dllm_rotary(_ref(plan), _ptr(x), T, H, D, x_token, x_head, _ptr(positions), transpose, _ptr(y),
                              y_token, y_head, _stream(stream))


def dllm_cache_write(cache, batch, T: int, k, k_token: int, k_head: int, v, v_token: int, v_head: int, start,
                     positions=None, plan=None, stream=None) -> int:
    return load().dllm_cache_write(_ref(cache), _ref(batch), T, _ptr(k), k_token, k_head, _ptr(v), v_token, v_head,
                                   _ptr(start), _ptr(positions), _ref(plan), _stream(stream))


def dllm_cache_attention_workspace_bytes(cache, batch, q_heads: int) -> int:
    return int(load().dllm_cache_attention_workspace_bytes(_ref(cache), _ref(batch), q_heads))


def dllm_cache_attention(cache, batch, T: int, q, q_token: int, q_head: int, q_heads: int, scale: float, causal: int,
                         out, lse, workspace, workspace_bytes: int, stream=None) -> int:
    return load().dllm_cache_attention(_ref(cache), _ref(batch), T, _ptr(q), q_token, q_head, q_heads, scale, causal,
                                       _ptr(out), _ptr(lse), _ptr(workspace), workspace_bytes, _stream(stream))


def dllm_cache_weigh(cache, batch, T: int, q, q_token: int, q_head: int, q_heads: int, scale: float, causal: int, lse,
                     decay: float, weights, stream=None) -> int:
    return load().dllm_cache_weigh(_ref(cache), _ref(batch), T, _ptr(q), q_token, q_head, q_heads, scale, causal,
                                   _ptr(lse), decay, _ptr(weights), _stream(stream))


def dllm_cache_evict_workspace_bytes(cache, batch) -> int:
    return int(load().dllm_cache_evict_workspace_bytes(_ref(cache), _ref(batch)))


def dllm_cache_evict(cache, batch, weights, keep, max_keep: int, sink: int, recent: int, pool: int, table_out,
                     out_blocks: int, lens_out, kept, weights_out, workspace, workspace_bytes: int, stream=None) -> int:
    return load().dllm_cache_evict(_ref(cache), _ref(batch), _ptr(weights), _ptr(keep), max_keep, sink, recent, pool,
                                   _ptr(table_out), out_blocks, _ptr(lens_out), _ptr(kept), _ptr(weights_out),
                                   _ptr(workspace), workspace_bytes, _stream(stream))


def dllm_residual_norm(norm, x, y, T: int, gate, groups: int, x_out, n, stream=None) -> int:
    return load().dllm_residual_norm(_ref(norm), _ptr(x), _ptr(y), T, _ptr(gate), groups, _ptr(x_out), _ptr(n),
                                     _stream(stream))


def dllm_residual_norm_backward_workspace_bytes(norm, T: int, groups: int) -> int:
    return int(load().dllm_residual_norm_backward_workspace_bytes(_ref(norm), T, groups))


def dllm_residual_norm_backward(norm, x, y, T: int, gate, groups: int, d_n, d_x_out, d_x, d_y, d_pre, d_post, d_gate,
                                workspace, workspace_bytes: int, stream=None) -> int:
    return load().dllm_residual_norm_backward(_ref(norm), _ptr(x), _ptr(y), T, _ptr(gate), groups, _ptr(d_n),
                                              _ptr(d_x_out), _ptr(d_x), _ptr(d_y), _ptr(d_pre), _ptr(d_post),
                                              _ptr(d_gate), _ptr(workspace), workspace_bytes, _stream(stream))


def dllm_embed(table, V: int, d: int, tokens, T: int, scale: float, out, stream=None) -> int:
    return load().dllm_embed(_ptr(table), V, d, _ptr(tokens), T, scale, _ptr(out), _stream(stream))


def dllm_embed_backward_workspace_bytes(V: int, d: int, T: int) -> int:
    return int(load().dllm_embed_backward_workspace_bytes(V, d, T))


def dllm_embed_backward(tokens, T: int, d_out, V: int, d: int, scale: float, accumulate: int, d_table, workspace,
                        workspace_bytes: int, stream=None) -> int:
    return load().dllm_embed_backward(_ptr(tokens), T, _ptr(d_out), V, d, scale, accumulate, _ptr(d_table),
                                      _ptr(workspace), workspace_bytes, _stream(stream))


def dllm_loss_forward_workspace_bytes(V: int, d: int, L: int) -> int:
    return int(load().dllm_loss_forward_workspace_bytes(V, d, L))


def dllm_loss_forward(p, loss, losses, lse, workspace, workspace_bytes: int, stream=None) -> int:
    return load().dllm_loss_forward(_ref(p), _ptr(loss), _ptr(losses), _ptr(lse), _ptr(workspace), workspace_bytes,
                                    _stream(stream))


def dllm_loss_backward_workspace_bytes(V: int, d: int, L: int, piece: int = 0) -> int:
    return int(load().dllm_loss_backward_workspace_bytes(V, d, L, piece))


def dllm_loss_backward(p, lse, grad, d_hidden, d_W, accumulate: int, piece: int, workspace, workspace_bytes: int,
                       stream=None) -> int:
    return load().dllm_loss_backward(_ref(p), _ptr(lse), _ptr(grad), _ptr(d_hidden), _ptr(d_W), accumulate, piece,
                                     _ptr(workspace), workspace_bytes, _stream(stream))
