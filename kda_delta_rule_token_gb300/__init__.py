"""Python binding of the GB300 KDA token-step library (libkda.so).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI of ``include/kda.h``.  The functions carry the C
names; tensors are PyTorch CUDA tensors (PyTorch supplies device memory and
streams).  There is no fallback: if libkda.so is missing or a call fails, an
exception is raised.
"""
from __future__ import annotations

import ctypes
import os

from . import build as _build_mod

__all__ = [
    "KDAError", "load", "kda_create", "kda_destroy", "kda_strerror", "kda_last_error_detail",
    "kda_decode_step", "kda_decode_step_bf16state", "kda_prefill", "kda_prefill_varlen", "kda_prefill_workspace_bytes", "kda_sync_status",
    "kda_launch_count", "kda_bind_lowrank", "kda_lowrank", "kda_lowrank_workspace_bytes",
    "kda_decode_step_lowrank", "kda_decode_lowrank_workspace_bytes", "kda_lowrank_noalloc",
    "LOWRANK_NOALLOC_SCRATCH_BYTES", "kda_bind_projections", "kda_project_qkvg", "kda_project_o",
    "kda_project_o_workspace_bytes", "kda_attn_create", "kda_attn_destroy", "kda_attn_bind_cache",
    "kda_attn_plan", "kda_attn_append", "kda_attn_workspace_bytes", "kda_attn_decode", "kda_attn_prefill",
    "kda_attn_decode_shared", "kda_attn_shared_workspace_bytes", "kda_attn_fork", "kda_attn_fork_workspace_bytes", "kda_attn_copy_pages",
    "kda_attn_sync_status", "kda_beam_select", "kda_beam_select_workspace_bytes", "kda_beam_reorder", "KDA_CACHE_BF16", "KDA_CACHE_E4M3", "KDA_OK", "KDA_ERR_INVALID_ARG", "KDA_ERR_ALIGNMENT",
    "KDA_ERR_UNSUPPORTED", "KDA_ERR_CUDA", "KDA_ERR_TIMEOUT", "HEAD_DIM", "CHUNK",
]

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_ALIGNMENT, KDA_ERR_UNSUPPORTED, KDA_ERR_CUDA, \
    KDA_ERR_TIMEOUT = range(6)
KDA_CACHE_BF16, KDA_CACHE_E4M3 = range(2)
HEAD_DIM = 128
CHUNK = 64
LOWRANK_NOALLOC_SCRATCH_BYTES = 4 << 20   # KDA_LOWRANK_NOALLOC_SCRATCH_BYTES of include/kda.h

_lib = None


class KDAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = ""
        if _lib is not None:
            d = _lib.kda_last_error_detail()
            detail = d.decode() if d else ""
        msg = f"{where}: {kda_strerror(status)}" + (f" [{detail}]" if detail else "")
        super().__init__(msg)


class _Config(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("chunk_size", ctypes.c_int), ("l2_eps", ctypes.c_float),
                ("rms_eps", ctypes.c_float)]


class _AttnConfig(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int), ("num_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("page_size", ctypes.c_int), ("cache_type", ctypes.c_int),
                ("rotary_dim", ctypes.c_int), ("rope_interleaved", ctypes.c_int),
                ("rms_eps", ctypes.c_float), ("softmax_scale", ctypes.c_float)]


def library_path() -> str:
    return _build_mod.LIB


def load(path: str | None = None):
    """Load libkda.so (built by ``build.build()``); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or library_path()
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build the CUDA library first "
            "(python -m kda_delta_rule_token_gb300.build)")
    lib = ctypes.CDLL(path)
    vp, sz, i32, u64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_uint64
    lib.kda_create.argtypes = [ctypes.POINTER(_Config), vp, vp, vp, vp, ctypes.POINTER(vp)]
    lib.kda_create.restype = i32
    lib.kda_destroy.argtypes = [vp]
    lib.kda_destroy.restype = None
    lib.kda_strerror.argtypes = [i32]
    lib.kda_strerror.restype = ctypes.c_char_p
    lib.kda_last_error_detail.argtypes = []
    lib.kda_last_error_detail.restype = ctypes.c_char_p
    lib.kda_decode_step.argtypes = [vp, i32] + [vp] * 11
    lib.kda_decode_step.restype = i32
    lib.kda_decode_step_bf16state.argtypes = [vp, i32] + [vp] * 11
    lib.kda_decode_step_bf16state.restype = i32
    lib.kda_prefill_workspace_bytes.argtypes = [vp, i32, i32]
    lib.kda_prefill_workspace_bytes.restype = sz
    lib.kda_prefill.argtypes = [vp, i32, i32] + [vp] * 10 + [sz, vp]
    lib.kda_prefill.restype = i32
    lib.kda_prefill_varlen.argtypes = [vp, i32, vp, i32] + [vp] * 10
    lib.kda_prefill_varlen.restype = i32
    lib.kda_sync_status.argtypes = [vp, vp]
    lib.kda_sync_status.restype = i32
    lib.kda_launch_count.argtypes = []
    lib.kda_launch_count.restype = u64
    lib.kda_bind_lowrank.argtypes = [vp, i32, i32, vp, vp, vp]
    lib.kda_bind_lowrank.restype = i32
    lib.kda_lowrank_workspace_bytes.argtypes = [vp, i32]
    lib.kda_lowrank_workspace_bytes.restype = sz
    lib.kda_lowrank.argtypes = [vp, i32, vp, vp, vp, vp, sz, vp]
    lib.kda_lowrank.restype = i32
    lib.kda_decode_lowrank_workspace_bytes.argtypes = [vp, i32]
    lib.kda_decode_lowrank_workspace_bytes.restype = sz
    lib.kda_decode_step_lowrank.argtypes = [vp, i32] + [vp] * 10 + [sz, vp]
    lib.kda_decode_step_lowrank.restype = i32
    lib.kda_lowrank_noalloc.argtypes = [vp, i32, vp, vp, vp, vp]
    lib.kda_lowrank_noalloc.restype = i32
    lib.kda_bind_projections.argtypes = [vp, i32, vp, vp]
    lib.kda_bind_projections.restype = i32
    lib.kda_project_qkvg.argtypes = [vp, i32, vp, vp, vp, vp, vp, i32, vp]
    lib.kda_project_qkvg.restype = i32
    lib.kda_project_o_workspace_bytes.argtypes = [vp, i32]
    lib.kda_project_o_workspace_bytes.restype = sz
    lib.kda_project_o.argtypes = [vp, i32, vp, vp, vp, sz, vp]
    lib.kda_project_o.restype = i32
    i64 = ctypes.c_longlong
    lib.kda_attn_create.argtypes = [ctypes.POINTER(_AttnConfig), ctypes.POINTER(ctypes.c_double),
                                    vp, vp, vp, vp, ctypes.POINTER(vp)]
    lib.kda_attn_create.restype = i32
    lib.kda_attn_destroy.argtypes = [vp]
    lib.kda_attn_destroy.restype = None
    lib.kda_attn_bind_cache.argtypes = [vp, i32, vp, vp]
    lib.kda_attn_bind_cache.restype = i32
    lib.kda_attn_plan.argtypes = [vp, i32, i32, vp, vp, vp, i32, vp, vp, i32] + [vp] * 6
    lib.kda_attn_plan.restype = i32
    lib.kda_attn_append.argtypes = [vp, i32, vp, i64, vp, i64, vp, i64] + [vp] * 4
    lib.kda_attn_append.restype = i32
    lib.kda_attn_workspace_bytes.argtypes = [vp]
    lib.kda_attn_workspace_bytes.restype = sz
    lib.kda_attn_decode.argtypes = [vp, i32, vp, vp, i32, vp, vp, vp, i32, vp, vp, sz, vp]
    lib.kda_attn_decode.restype = i32
    lib.kda_attn_prefill.argtypes = [vp, i32, i32, vp, vp, vp, i32, vp, vp, vp, i32, vp, vp, sz, vp]
    lib.kda_attn_prefill.restype = i32
    lib.kda_attn_shared_workspace_bytes.argtypes = [vp, i32]
    lib.kda_attn_shared_workspace_bytes.restype = sz
    lib.kda_attn_decode_shared.argtypes = [vp, i32, vp, vp, i32, vp, i32, vp, vp, vp, vp, i32, vp, vp, sz, vp]
    lib.kda_attn_decode_shared.restype = i32
    lib.kda_attn_fork_workspace_bytes.argtypes = [vp, i32, i32]
    lib.kda_attn_fork_workspace_bytes.restype = sz
    lib.kda_attn_fork.argtypes = [vp, i32, vp, vp, vp, i32, vp, vp, i32] + [vp] * 8 + [sz, vp]
    lib.kda_attn_fork.restype = i32
    lib.kda_attn_copy_pages.argtypes = [vp, i32, vp, vp, vp, vp]
    lib.kda_attn_copy_pages.restype = i32
    lib.kda_attn_sync_status.argtypes = [vp, vp]
    lib.kda_attn_sync_status.restype = i32
    lib.kda_beam_select_workspace_bytes.argtypes = [vp] + [i32] * 4
    lib.kda_beam_select_workspace_bytes.restype = sz
    lib.kda_beam_select.argtypes = [vp, i32, i32, i32, vp, i32, i64, vp, vp, i32, i32, i32, vp, vp, vp, vp, sz, vp]
    lib.kda_beam_select.restype = i32
    lib.kda_beam_reorder.argtypes = [vp, i32, vp, vp, vp, vp, vp, i32, vp]
    lib.kda_beam_reorder.restype = i32
    lib.kda_testing_bounded_wait.argtypes = [vp, ctypes.c_uint, vp]
    lib.kda_testing_bounded_wait.restype = i32
    _lib = lib
    return lib


def _check(status: int, where: str):
    if status != KDA_OK:
        raise KDAError(status, where)


def _p(t):
    """Device address of a tensor (None -> NULL); ints pass through."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_current = None   # the current stream's handle, found on first use


def _find_current():
    global _current
    import torch
    c = torch._C
    if hasattr(c, "_cuda_getCurrentRawStream") and hasattr(c, "_cuda_getDevice"):
        # The handle alone: building a torch.cuda.Stream object around it takes
        # 3 us, a third of a small call's time on the host.
        _current = lambda: c._cuda_getCurrentRawStream(c._cuda_getDevice())   # noqa: E731
    else:
        _current = lambda: torch.cuda.current_stream().cuda_stream            # noqa: E731


def _stream(stream):
    if stream is None:
        if _current is None:
            _find_current()
        return _current()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def kda_strerror(status: int) -> str:
    return load().kda_strerror(int(status)).decode()


def kda_last_error_detail() -> str:
    d = load().kda_last_error_detail()
    return d.decode() if d else ""


def kda_launch_count() -> int:
    return int(load().kda_launch_count())


def kda_create(num_heads, conv_w, dt_bias, A_log, rms_gamma, *, head_dim=HEAD_DIM,
               chunk_size=CHUNK, l2_eps=1e-6, rms_eps=1e-6) -> int:
    """Returns an opaque context handle (int).  Parameters are borrowed."""
    cfg = _Config(int(num_heads), int(head_dim), int(chunk_size), float(l2_eps), float(rms_eps))
    out = ctypes.c_void_p()
    _check(load().kda_create(ctypes.byref(cfg), _p(conv_w), _p(dt_bias), _p(A_log),
                             _p(rms_gamma), ctypes.byref(out)), "kda_create")
    return out.value


def kda_destroy(ctx: int) -> None:
    load().kda_destroy(ctx)


def kda_decode_step(ctx, B, q, k, v, z, beta_logit, gate_logit, conv_state, S, o,
                    o_pre=None, stream=None) -> None:
    _check(load().kda_decode_step(ctx, int(B), _p(q), _p(k), _p(v), _p(z), _p(beta_logit),
                                  _p(gate_logit), _p(conv_state), _p(S), _p(o), _p(o_pre),
                                  _stream(stream)), "kda_decode_step")


def kda_decode_step_bf16state(ctx, B, q, k, v, z, beta_logit, gate_logit, conv_state, S, o,
                              o_pre=None, stream=None) -> None:
    """kda_decode_step with S held as bf16 (a 16-bit tensor of raw patterns)."""
    _check(load().kda_decode_step_bf16state(ctx, int(B), _p(q), _p(k), _p(v), _p(z), _p(beta_logit),
                                            _p(gate_logit), _p(conv_state), _p(S), _p(o), _p(o_pre),
                                            _stream(stream)), "kda_decode_step_bf16state")


def kda_prefill_workspace_bytes(ctx, B, T) -> int:
    return int(load().kda_prefill_workspace_bytes(ctx, int(B), int(T)))


def kda_prefill(ctx, B, T, q, k, v, z, beta_logit, gate_logit, conv_state, S, o,
                workspace=None, workspace_bytes=0, stream=None) -> None:
    if workspace is not None and not isinstance(workspace, int) and workspace_bytes == 0:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check(load().kda_prefill(ctx, int(B), int(T), _p(q), _p(k), _p(v), _p(z), _p(beta_logit),
                              _p(gate_logit), _p(conv_state), _p(S), _p(o), _p(workspace),
                              int(workspace_bytes), _stream(stream)), "kda_prefill")


def kda_prefill_varlen(ctx, B, cu_seqlens, total_T, q, k, v, z, beta_logit, gate_logit, conv_state,
                       S, o, stream=None) -> None:
    """Packed sequences: cu_seqlens is a device int32 tensor of B + 1 offsets."""
    _check(load().kda_prefill_varlen(ctx, int(B), _p(cu_seqlens), int(total_T), _p(q), _p(k), _p(v),
                                     _p(z), _p(beta_logit), _p(gate_logit), _p(conv_state), _p(S),
                                     _p(o), _stream(stream)), "kda_prefill_varlen")


def _nbytes(buf, given):
    if buf is None or isinstance(buf, int) or given:
        return int(given)
    return buf.nbytes


def kda_bind_lowrank(ctx, hidden, rank, W_fa, W_fb, W_bp) -> None:
    _check(load().kda_bind_lowrank(ctx, int(hidden), int(rank), _p(W_fa), _p(W_fb), _p(W_bp)),
           "kda_bind_lowrank")


def kda_lowrank_workspace_bytes(ctx, N) -> int:
    return int(load().kda_lowrank_workspace_bytes(ctx, int(N)))


def kda_lowrank(ctx, N, x, z, beta_logit, workspace, workspace_bytes=0, stream=None) -> None:
    _check(load().kda_lowrank(ctx, int(N), _p(x), _p(z), _p(beta_logit), _p(workspace),
                              _nbytes(workspace, workspace_bytes), _stream(stream)), "kda_lowrank")


def kda_lowrank_noalloc(ctx, N, x, z, beta_logit, stream=None) -> None:
    """The front-end with its scratch in the library's static device array
    (no workspace argument; see kda.h)."""
    _check(load().kda_lowrank_noalloc(ctx, int(N), _p(x), _p(z), _p(beta_logit), _stream(stream)),
           "kda_lowrank_noalloc")


def kda_decode_lowrank_workspace_bytes(ctx, B) -> int:
    return int(load().kda_decode_lowrank_workspace_bytes(ctx, int(B)))


def kda_decode_step_lowrank(ctx, B, x, q, k, v, gate_logit, conv_state, S, o, o_pre, workspace,
                            workspace_bytes=0, stream=None) -> None:
    _check(load().kda_decode_step_lowrank(ctx, int(B), _p(x), _p(q), _p(k), _p(v), _p(gate_logit),
                                          _p(conv_state), _p(S), _p(o), _p(o_pre), _p(workspace),
                                          _nbytes(workspace, workspace_bytes), _stream(stream)),
           "kda_decode_step_lowrank")


def kda_bind_projections(ctx, hidden, W_qkvg, W_o) -> None:
    """W_qkvg [4*H*d, hidden] and W_o [hidden, H*d]: bf16 tensors (or their int16 views)."""
    _check(load().kda_bind_projections(ctx, int(hidden), _p(W_qkvg), _p(W_o)), "kda_bind_projections")


def kda_project_qkvg(ctx, N, x, q, k, v, gate_logit, qkv_f32=False, stream=None) -> None:
    _check(load().kda_project_qkvg(ctx, int(N), _p(x), _p(q), _p(k), _p(v), _p(gate_logit),
                                   1 if qkv_f32 else 0, _stream(stream)), "kda_project_qkvg")


def kda_project_o_workspace_bytes(ctx, N) -> int:
    return int(load().kda_project_o_workspace_bytes(ctx, int(N)))


def kda_project_o(ctx, N, o, y, workspace, workspace_bytes=0, stream=None) -> None:
    _check(load().kda_project_o(ctx, int(N), _p(o), _p(y), _p(workspace),
                                _nbytes(workspace, workspace_bytes), _stream(stream)), "kda_project_o")


def kda_sync_status(ctx, stream=None) -> int:
    """Synchronise and return the status code (does not raise)."""
    return int(load().kda_sync_status(ctx, _stream(stream)))


def kda_attn_create(num_q_heads, num_kv_heads, *, page_size, cache_type=KDA_CACHE_BF16,
                    rotary_dim=HEAD_DIM, rope_interleaved=False, inv_freq=None, q_gamma=None,
                    k_gamma=None, k_scale=None, v_scale=None, rms_eps=1e-6,
                    softmax_scale=HEAD_DIM ** -0.5, head_dim=HEAD_DIM) -> int:
    """Returns an opaque handle (int) of one softmax-attention layer (kda_attn.h).
    inv_freq: a sequence of rotary_dim / 2 radians per position (host numbers,
    copied).  The device tensors are borrowed."""
    freqs = None
    if inv_freq is not None:
        freqs = [float(f) for f in inv_freq]
        if len(freqs) != int(rotary_dim) // 2:
            raise ValueError(f"inv_freq has {len(freqs)} values, rotary_dim {rotary_dim} needs {int(rotary_dim) // 2}")
        freqs = (ctypes.c_double * max(1, len(freqs)))(*freqs)
    cfg = _AttnConfig(int(num_q_heads), int(num_kv_heads), int(head_dim), int(page_size), int(cache_type),
                      int(rotary_dim), 1 if rope_interleaved else 0, float(rms_eps), float(softmax_scale))
    out = ctypes.c_void_p()
    _check(load().kda_attn_create(ctypes.byref(cfg), freqs, _p(q_gamma), _p(k_gamma), _p(k_scale),
                                  _p(v_scale), ctypes.byref(out)), "kda_attn_create")
    return out.value


def kda_attn_destroy(attn: int) -> None:
    load().kda_attn_destroy(attn)


def kda_attn_bind_cache(attn, num_pages, k_cache, v_cache) -> None:
    """Caches [num_pages, kv heads, page_size, 128]: bf16 or e4m3 tensors (or their raw views)."""
    _check(load().kda_attn_bind_cache(attn, int(num_pages), _p(k_cache), _p(v_cache)), "kda_attn_bind_cache")


def _pitch(table, given):
    """Row length of a block table [B, max_pages]: given, or the tensor's."""
    if given is not None:
        return int(given)
    if table.dim() == 2:
        (rows, width), (pitch, step) = table.shape, table.stride()
        if step == 1 or width == 1:
            if pitch >= width:
                return pitch
            if rows == 1:
                return width
    raise ValueError(f"block_table must be [B, max_pages] with dense rows: shape {tuple(table.shape)}, strides {table.stride()}")


def _dense(t, name):
    """The address of a tensor that the library takes as dense."""
    if t is not None and not isinstance(t, int) and not t.is_contiguous():
        raise ValueError(f"{name} must be dense: shape {tuple(t.shape)}, strides {t.stride()}")
    return _p(t)


def kda_attn_plan(attn, B, N, cache_lens, new_lens, free_pages, free_count, block_table, cu_new, kv_lens,
                  positions, slots, info, *, free_capacity=None, max_pages=None, stream=None) -> None:
    cap = free_pages.numel() if free_capacity is None else int(free_capacity)
    _check(load().kda_attn_plan(attn, B, N, _p(cache_lens), _p(new_lens), _p(free_pages), cap,
                                _p(free_count), _p(block_table), _pitch(block_table, max_pages), _p(cu_new),
                                _p(kv_lens), _p(positions), _p(slots), _p(info), _stream(stream)),
           "kda_attn_plan")


def _token_stride(t, given):
    """Elements from one token's heads to the next's: given, or the [N, heads, 128] tensor's."""
    if given is not None:
        return int(given)
    st = t.stride()
    heads = t.shape[-2]
    if st[-1] != 1 or (st[-2] != HEAD_DIM and heads != 1):
        raise ValueError(f"heads must be dense rows of {HEAD_DIM} elements: strides {tuple(st)}")
    return st[0] if t.shape[0] != 1 else heads * HEAD_DIM   # of one token any stride will do


def kda_attn_append(attn, N, q, k, v, positions, slots, q_out, *, q_stride=None, k_stride=None,
                    v_stride=None, stream=None) -> None:
    _check(load().kda_attn_append(attn, N, _p(q), _token_stride(q, q_stride), _p(k), _token_stride(k, k_stride),
                                  _p(v), _token_stride(v, v_stride), _p(positions), _p(slots),
                                  _dense(q_out, "q_out"), _stream(stream)), "kda_attn_append")


def kda_attn_workspace_bytes(attn) -> int:
    return int(load().kda_attn_workspace_bytes(attn))


def _is_f32(o, given):
    return int(bool(given)) if given is not None else int(o.element_size() == 4)


def kda_attn_decode(attn, B, q, block_table, kv_lens, o, workspace, *, max_pages=None, gate_logit=None,
                    o_f32=None, lse=None, workspace_bytes=0, stream=None) -> None:
    _check(load().kda_attn_decode(attn, B, _dense(q, "q"), _p(block_table), _pitch(block_table, max_pages),
                                  _p(kv_lens), _dense(gate_logit, "gate_logit"), _dense(o, "o"),
                                  _is_f32(o, o_f32), _dense(lse, "lse"), _p(workspace),
                                  _nbytes(workspace, workspace_bytes), _stream(stream)), "kda_attn_decode")


def kda_attn_shared_workspace_bytes(attn, B) -> int:
    return int(load().kda_attn_shared_workspace_bytes(attn, int(B)))


def kda_attn_decode_shared(attn, B, q, block_table, kv_lens, groups, cu_groups, prefix_lens, o, workspace, *, max_pages=None,
                           gate_logit=None, o_f32=None, lse=None, workspace_bytes=0, stream=None) -> None:
    """kda_attn_decode where group g's requests, cu_groups[g] to cu_groups[g + 1] - 1, share their first prefix_lens[g] keys."""
    f32 = _is_f32(o, o_f32)
    table, pitch = _table(block_table, "block_table", B, max_pages)
    offsets = groups if 0 < groups <= B else -1   # (no offsets of no groups, or of so many that the library refuses the call)
    _check(load().kda_attn_decode_shared(attn, B, _values(q, "q", B, 1), table, pitch,
                                         _words(kv_lens, "kv_lens", B), int(groups), _words(cu_groups, "cu_groups", offsets + 1),
                                         _words(prefix_lens, "prefix_lens", offsets), _values(gate_logit, "gate_logit", B, 0),
                                         _values(o, "o", B, 1 - f32), f32, _words(lse, "lse", B), _p(workspace),
                                         _nbytes(workspace, workspace_bytes), _stream(stream)),
           "kda_attn_decode_shared")


def kda_attn_prefill(attn, B, N, cu_new, q, block_table, kv_lens, o, workspace, *, max_pages=None,
                     gate_logit=None, o_f32=None, lse=None, workspace_bytes=0, stream=None) -> None:
    _check(load().kda_attn_prefill(attn, B, N, _p(cu_new), _dense(q, "q"), _p(block_table),
                                   _pitch(block_table, max_pages), _p(kv_lens), _dense(gate_logit, "gate_logit"),
                                   _dense(o, "o"), _is_f32(o, o_f32), _dense(lse, "lse"), _p(workspace),
                                   _nbytes(workspace, workspace_bytes), _stream(stream)), "kda_attn_prefill")


def kda_attn_fork_workspace_bytes(attn, B, max_pages) -> int:
    return int(load().kda_attn_fork_workspace_bytes(attn, int(B), int(max_pages)))


def kda_attn_fork(attn, B, rows, kv_lens, block_table, page_refs, free_pages, free_count, new_table, new_lens,
                  copy_src, copy_dst, copy_rows, info, workspace, *, free_capacity=None, max_pages=None,
                  workspace_bytes=0, stream=None) -> None:
    """Requests take over one another's pages (kda_attn.h).  Both tables have rows of the same pitch."""
    cap = free_pages.numel() if free_capacity is None else int(free_capacity)
    old, pitch = _table(block_table, "block_table", B, max_pages)
    new, new_pitch = _table(new_table, "new_table", B, max_pages)
    if new_pitch != pitch:
        raise ValueError(f"rows of block_table are {pitch} apart, those of new_table {new_pitch}")
    _check(load().kda_attn_fork(attn, B, _words(rows, "rows", B), _words(kv_lens, "kv_lens", B), old, pitch,
                                _words(page_refs, "page_refs", 0), _words(free_pages, "free_pages", cap), cap,
                                _words(free_count, "free_count", 1), new, _words(new_lens, "new_lens", B),
                                _words(copy_src, "copy_src", B), _words(copy_dst, "copy_dst", B),
                                _words(copy_rows, "copy_rows", B), _words(info, "info", 4), _p(workspace),
                                _nbytes(workspace, workspace_bytes), _stream(stream)), "kda_attn_fork")


def kda_attn_copy_pages(attn, n, src, dst, rows, *, stream=None) -> None:
    _check(load().kda_attn_copy_pages(attn, n, _words(src, "src", n), _words(dst, "dst", n), _words(rows, "rows", n),
                                      _stream(stream)), "kda_attn_copy_pages")


def kda_attn_sync_status(attn, stream=None) -> int:
    """Synchronise and return the status code (does not raise)."""
    return int(load().kda_attn_sync_status(attn, _stream(stream)))


def _words(t, name, count, size=4):
    """The address of a dense tensor of at least `count` elements of `size` bytes."""
    if t is None or t.__class__ is int:
        return t
    if t.numel() >= count and t.element_size() == size and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must have {count} dense elements of {size} bytes: shape {tuple(t.shape)}, strides {t.stride()}, {t.dtype}")


_kinds = {}   # of torch's types: 1 what the library takes as bf16, 0 as fp32; found on first use


def _bf16(t, name):
    """Whether a tensor is bf16 (or its raw view), or fp32.  Others, fp16 among them, are refused: the library
    would take them for one of these."""
    kind = _kinds.get(t.dtype)
    if kind is None:
        if not _kinds:
            import torch
            _kinds.update({torch.float32: 0, torch.bfloat16: 1, torch.int16: 1, torch.uint16: 1})
            return _bf16(t, name)
        raise ValueError(f"{name} must be fp32 or bf16 (or bf16's raw view): {t.dtype}")
    return kind


def _values(t, name, B, bf16):
    """The address of a dense tensor of at least B rows, bf16 (or its raw view) or fp32."""
    if t is None or t.__class__ is int:
        return t
    if _bf16(t, name) == bf16 and t.is_contiguous() and t.shape[0] >= B:
        return t.data_ptr()
    raise ValueError(f"{name} must have {B} dense rows of {'bf16' if bf16 else 'fp32'}: shape {tuple(t.shape)}, strides {t.stride()}, {t.dtype}")


def _table(t, name, B, given):
    """The address of an int32 block table of at least B rows, and its pitch (_pitch)."""
    if t.__class__ is int:
        return t, int(given)
    if t.element_size() != 4 or (t.shape[0] < B and t.dim() == 2):
        raise ValueError(f"{name} must have {B} rows of int32: shape {tuple(t.shape)}, {t.dtype}")
    return t.data_ptr(), _pitch(t, given)


def kda_beam_select_workspace_bytes(ctx, groups, beams, vocab, num) -> int:
    return int(load().kda_beam_select_workspace_bytes(ctx, int(groups), int(beams), int(vocab), int(num)))


def kda_beam_select(ctx, groups, beams, logits, scores, num, out_scores, out_tokens, out_rows, workspace, *,
                    done=None, end_token=0, keep_places=False, workspace_bytes=0, stream=None) -> None:
    """The num best continuations of every group (kda_beam.h).  logits [groups * beams, vocab]: fp32 or bf16
    (or its raw view), rows at any stride; done: bytes or truth values."""
    if logits.dim() != 2:
        raise ValueError(f"logits must be [{groups * beams}, vocab]: shape {tuple(logits.shape)}")
    (rows, vocab), (stride, step) = logits.shape, logits.stride()
    if rows < groups * beams or (step != 1 and vocab != 1):
        raise ValueError(f"logits must be [{groups * beams}, vocab] with dense rows: shape {(rows, vocab)}, strides {(stride, step)}")
    if rows == 1:
        stride = vocab   # of one row any stride will do
    _check(load().kda_beam_select(ctx, int(groups), int(beams), vocab, logits.data_ptr(), _bf16(logits, "logits"), stride,
                                  _words(scores, "scores", groups * beams), _words(done, "done", groups * beams, 1),
                                  int(end_token), int(num), 1 if keep_places else 0,
                                  _words(out_scores, "out_scores", groups * num), _words(out_tokens, "out_tokens", groups * num),
                                  _words(out_rows, "out_rows", groups * num), _p(workspace),
                                  _nbytes(workspace, workspace_bytes), _stream(stream)), "kda_beam_select")


def kda_beam_reorder(ctx, B, rows, S, conv_state, *, S_out=None, conv_out=None, stream=None) -> None:
    """S[b], conv_state[b] <- S[rows[b]], conv_state[rows[b]] in place, or into S_out and conv_out (kda_beam.h)."""
    size = S.element_size()
    if size not in (2, 4):
        raise ValueError(f"S must be fp32 or bf16: {S.dtype}")
    S_at, conv_at = _sequences(S, "S", B, size), _sequences(conv_state, "conv_state", B, 4)
    _check(load().kda_beam_reorder(ctx, int(B), _words(rows, "rows", B), S_at, conv_at,
                                   S_at if S_out is None else _sequences(S_out, "S_out", B, size),
                                   conv_at if conv_out is None else _sequences(conv_out, "conv_out", B, 4), int(size == 2),
                                   _stream(stream)), "kda_beam_reorder")


def _sequences(t, name, B, size):
    """The address of a dense tensor of at least B sequences' values of `size` bytes."""
    if t.element_size() == size and t.is_contiguous() and t.shape[0] >= B:
        return t.data_ptr()
    raise ValueError(f"{name} must hold {B} dense sequences of values of {size} bytes: shape {tuple(t.shape)}, strides {t.stride()}, {t.dtype}")


def kda_testing_bounded_wait(ctx, limit_us, stream=None) -> None:
    """Test hook (not part of the public API): launch a kernel whose bounded
    wait runs out after ``limit_us`` microseconds; the next kda_sync_status
    reports KDA_ERR_TIMEOUT."""
    _check(load().kda_testing_bounded_wait(ctx, int(limit_us), _stream(stream)),
           "kda_testing_bounded_wait")
