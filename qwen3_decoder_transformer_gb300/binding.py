"""ctypes binding of the C ABI in include/qwen3.h. Argument marshalling only: every step of the
forward pass runs in the CUDA library; torch tensors only provide device memory and streams.

The library must have been built (``__graft_entry__.build()``); loading fails loudly otherwise.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import numpy as np
import torch

from .build import LIB, tensors_path

_vp = ctypes.c_void_p
_i32p = ctypes.POINTER(ctypes.c_int)

EPI_BF16, EPI_SWIGLU, EPI_RESIDUAL, EPI_F32 = 0, 1, 2, 3
ALL_ROWS = 1


class Qwen3Error(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what} (code {code})")
        self.code = code


class Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "n_layers", "hidden", "n_q_heads", "n_kv_heads", "head_dim", "intermediate", "vocab",
        "tie_embeddings", "max_positions")] + [("rope_theta", ctypes.c_float), ("rms_eps", ctypes.c_float),
                                               ("sliding_window", ctypes.c_int32), ("rolling_cache", ctypes.c_int32)]

    @classmethod
    def from_dict(cls, c: dict) -> "Config":
        return cls(c["n_layers"], c["hidden"], c["n_q_heads"], c["n_kv_heads"], c["head_dim"],
                   c["intermediate"], c["vocab"], int(c["tie_embeddings"]), c.get("max_positions", 40960),
                   float(c["rope_theta"]), float(c["rms_eps"]), int(c.get("sliding_window", 0)),
                   int(c.get("rolling_cache", 0)))


_LAYER = ("in_norm", "q_proj", "k_proj", "v_proj", "o_proj", "q_norm", "k_norm", "post_norm", "gate_proj",
          "up_proj", "down_proj")


class Weights(ctypes.Structure):
    _fields_ = [("embed", _vp), ("lm_head", _vp), ("final_norm", _vp)] + [(n, ctypes.POINTER(_vp)) for n in _LAYER]


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB):
        raise RuntimeError(f"CUDA library not built ({LIB}); run __graft_entry__.build() first")
    L = ctypes.CDLL(LIB)
    i, sz, cp = ctypes.c_int, ctypes.c_size_t, ctypes.c_char_p
    L.qwen3_strerror.restype = cp
    L.qwen3_strerror.argtypes = [i]
    L.qwen3_validate_config.argtypes = [ctypes.POINTER(Config)]
    L.qwen3_init.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(Weights), i, i, i, _vp, ctypes.POINTER(_vp)]
    L.qwen3_prefill.argtypes = [_vp, _vp, i, i, _vp, i, _vp]
    L.qwen3_decode_step.argtypes = [_vp, _vp, i, _vp, _vp]
    L.qwen3_prefill_host.argtypes = [_vp, _vp, i, i, _vp, i, _vp]
    L.qwen3_length.argtypes = [_vp, _i32p, _i32p]
    L.qwen3_set_length.argtypes = [_vp, i, i, _vp]
    L.qwen3_kv_view.argtypes = [_vp, i, ctypes.POINTER(_vp), ctypes.POINTER(_vp), ctypes.POINTER(ctypes.c_int64)]
    L.qwen3_set_tap.argtypes = [_vp, i, _vp, _vp]
    L.qwen3_get_error.argtypes = [_vp, _vp]
    L.qwen3_set_timing.argtypes = [_vp, i]
    L.qwen3_kernel_times.argtypes = [_vp, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64), _i32p]
    L.qwen3_kernel_class_name.restype = cp
    L.qwen3_kernel_class_name.argtypes = [i]
    L.qwen3_launch_count.argtypes = [_vp, i, i, i, i]
    L.qwen3_free.restype = None
    L.qwen3_free.argtypes = [_vp]
    L.qwen3_op_embed.argtypes = [_vp, i, i, _vp, i, _vp, _vp, _vp]
    L.qwen3_op_rmsnorm.argtypes = [_vp, _vp, i, i, i, i, ctypes.c_float, _vp, _vp]
    L.qwen3_op_gemm.argtypes = [_vp, _vp, i, i, i, i, _vp, i, _vp, i, _vp, _vp]
    L.qwen3_op_pack_gate_up.argtypes = [_vp, _vp, i, i, _vp, _vp]
    L.qwen3_gemm_norm_supported.argtypes = [i, i]
    L.qwen3_gemm_norm_part_floats.restype = sz
    L.qwen3_gemm_norm_part_floats.argtypes = [i]
    L.qwen3_op_gemm_residual_norm.argtypes = [_vp, _vp, i, i, i, _vp, _vp, ctypes.c_float, _vp, _vp, _vp, _vp]
    L.qwen3_gemm_skinny_splits.argtypes = [i, i]
    L.qwen3_op_gemm_skinny.argtypes = [_vp, _vp, i, i, i, i, _vp, _vp, _vp, _vp]
    L.qwen3_op_rope_table.argtypes = [ctypes.c_float, i, i, _vp, _vp]
    L.qwen3_op_qknorm_rope_append.argtypes = [_vp, i, i, i, i, i, _vp, _vp, _vp, _vp, ctypes.c_float, _vp, _vp,
                                              _vp, i, _vp]
    L.qwen3_op_attention_prefill.argtypes = [_vp, _vp, _vp, i, i, i, i, i, i, _vp, _vp, i, i, i, i, i, _vp, _vp,
                                             _vp, _vp]
    L.qwen3_attention_prefill_workspace.restype = sz
    L.qwen3_attention_prefill_workspace.argtypes = [i, i, i, i, i, i]
    L.qwen3_attention_decode_workspace.restype = sz
    L.qwen3_attention_decode_workspace.argtypes = [i, i, i, i, i, i]
    L.qwen3_op_attention_decode.argtypes = [_vp, _vp, _vp, i, i, i, i, i, _vp, _vp, i, i, _vp, _vp, _vp, _vp]
    L.qwen3_op_attention_decode_noalloc.argtypes = [_vp, _vp, _vp, i, i, i, i, i, _vp, _vp, _vp, _vp]
    L.qwen3_op_greedy.argtypes = [_vp, ctypes.c_int64, i, i, i, _vp, _vp, _vp, _vp]
    L.qwen3_greedy_workspace.restype = sz
    L.qwen3_greedy_workspace.argtypes = [i]
    L.qwen3_prefill_padded.argtypes = [_vp, _vp, _i32p, i, i, _vp, i, _vp]
    L.qwen3_share_prefix.argtypes = [_vp, i, _vp]
    L.qwen3_generate.argtypes = [_vp, _vp, _i32p, i, i, i, i, _vp, _i32p, _vp]
    L.qwen3_op_token_logprobs.argtypes = [_vp, i, ctypes.c_int64, i, i, _vp, i, _vp, _vp, _vp, _vp, _vp, _vp]
    L.qwen3_attention_decode_shared_workspace.restype = sz
    L.qwen3_attention_decode_shared_workspace.argtypes = [i, i, i, i, i]
    L.qwen3_op_attention_decode_shared.argtypes = [_vp, _vp, _vp, i, i, _vp, _vp, i, i, i, i, i, _vp, i, _vp, _vp, sz,
                                                   _vp, _vp, _vp]
    L.qwen3_attention_sink_rows.argtypes = [i]
    L.qwen3_op_attention_prefill_sinks.argtypes = [_vp, _vp, _vp, i, i, i, i, i, i, _vp, i, i, i, i, _vp, _vp, _vp]
    L.qwen3_op_attention_decode_sinks.argtypes = [_vp, _vp, _vp, i, i, i, i, i, _vp, i, i, i, i, _vp, _vp, _vp]
    i64 = ctypes.c_int64
    L.qwen3_paged4_page_bytes.restype = sz
    L.qwen3_paged4_page_bytes.argtypes = [i, i]
    L.qwen3_op_append_paged4.argtypes = [_vp, i64, i, _vp, _vp, i, i, i, i, _vp, _vp, ctypes.c_float, _vp, i, _vp, _vp, _vp,
                                         _vp, i, i, _vp, i, _vp, _vp]
    L.qwen3_op_read_paged4.argtypes = [_vp, _vp, i, i, _vp, i, _vp, _vp, i, i, i, i, _vp, _vp, _vp, _vp]
    L.qwen3_attention_decode_paged4_workspace.restype = sz
    L.qwen3_attention_decode_paged4_workspace.argtypes = [i, i, i, i]
    L.qwen3_op_attention_decode_paged4.argtypes = [_vp, _vp, _vp, i, i, _vp, i, _vp, i, i, i, i, _vp, sz, _vp, _vp, _vp]
    L.qwen3_attention_packed_plan_bytes.restype = sz
    L.qwen3_attention_packed_plan_bytes.argtypes = [i, i]
    L.qwen3_op_attention_packed_plan.argtypes = [_vp, _vp, i, i, i, _vp, sz, _vp, _vp]
    L.qwen3_op_attention_prefill_packed.argtypes = [_vp, i64, _vp, i64, _vp, i64, i, i, i, i, i, _vp, sz, i, _vp, _vp, _vp]
    for name in ("append_paged4", "read_paged4", "attention_decode_paged4", "attention_prefill_packed"):
        getattr(L, f"qwen3_op_{name}_block").argtypes = [ctypes.c_char_p, _vp]
    _lib = L
    return L


def strerror(code: int) -> str:
    return lib().qwen3_strerror(code).decode()


def check(rc: int):
    if rc != 0:
        raise Qwen3Error(rc, strerror(rc))


def _p(t) -> _vp:
    if t is None:
        return _vp(None)
    if isinstance(t, np.ndarray):
        return _vp(t.ctypes.data)
    return _vp(t.data_ptr())


def _stream(stream=None) -> _vp:
    s = torch.cuda.current_stream() if stream is None else stream
    return _vp(s.cuda_stream)


class _DeviceArray:
    def __init__(self, ptr: int, shape, typestr: str):
        self.__cuda_array_interface__ = {"data": (ptr, False), "shape": tuple(shape), "typestr": typestr,
                                         "version": 3, "strides": None}


def device_view(ptr: int, shape, dtype) -> torch.Tensor:
    """A torch tensor that aliases device memory owned by the library (no copy)."""
    if dtype == torch.bfloat16:
        return torch.as_tensor(_DeviceArray(ptr, shape, "<i2"), device="cuda").view(torch.bfloat16)
    typestr = {torch.float32: "<f4", torch.int32: "<i4"}[dtype]
    return torch.as_tensor(_DeviceArray(ptr, shape, typestr), device="cuda")


def validate_config(cfg: dict) -> int:
    c = Config.from_dict(cfg)
    return lib().qwen3_validate_config(ctypes.byref(c))


class Model:
    """A Qwen3 decoder context: KV cache, scratch and packed weights owned by the library.

    ``weights`` holds bf16 CUDA tensors in nn.Linear layout (synth.make_weights format); they are
    borrowed and kept alive by this object.
    """

    def __init__(self, cfg: dict, weights: dict, max_batch: int, capacity: int, max_tokens: int = 0,
                 stream=None):
        self.cfg = cfg
        self._w = weights
        L = cfg["n_layers"]
        self._arrays = {}
        for name in _LAYER:
            arr = (_vp * L)(*[t.data_ptr() for t in weights[name]])
            self._arrays[name] = arr
        lm = weights.get("lm_head")
        self._ws = Weights(_p(weights["embed"]), _p(lm), _p(weights["final_norm"]),
                           *[ctypes.cast(self._arrays[n], ctypes.POINTER(_vp)) for n in _LAYER])
        self._cfg = Config.from_dict(cfg)
        self.ctx = _vp()
        check(lib().qwen3_init(ctypes.byref(self._cfg), ctypes.byref(self._ws), max_batch, capacity, max_tokens,
                               _stream(stream), ctypes.byref(self.ctx)))
        self.max_batch, self.capacity = max_batch, capacity

    def close(self):
        if self.ctx:
            lib().qwen3_free(self.ctx)
            self.ctx = _vp()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def prefill(self, ids: torch.Tensor, logits: torch.Tensor, all_rows: bool = False, stream=None):
        B, T = ids.shape
        check(lib().qwen3_prefill(self.ctx, _p(ids), B, T, _p(logits), ALL_ROWS if all_rows else 0,
                                  _stream(stream)))

    def prefill_padded(self, ids: torch.Tensor, real, logits: torch.Tensor, all_rows: bool = False, stream=None):
        """ids [B, T] left-padded; real[b] = number of real tokens at the end of row b."""
        B, T = ids.shape
        r = (ctypes.c_int32 * B)(*[int(x) for x in real])
        check(lib().qwen3_prefill_padded(self.ctx, _p(ids), r, B, T, _p(logits), ALL_ROWS if all_rows else 0,
                                         _stream(stream)))

    def share_prefix(self, batch: int, stream=None):
        check(lib().qwen3_share_prefix(self.ctx, batch, _stream(stream)))

    def generate(self, ids: torch.Tensor, real, max_new: int, stop_id: int, out: torch.Tensor, stream=None) -> int:
        """Greedy generation; out [B, max_new] int32 receives the tokens. Returns the columns written."""
        B, T = ids.shape
        r = (ctypes.c_int32 * B)(*[int(x) for x in real]) if real is not None else None
        steps = ctypes.c_int32()
        check(lib().qwen3_generate(self.ctx, _p(ids), r, B, T, max_new, stop_id, _p(out), ctypes.byref(steps),
                                   _stream(stream)))
        return steps.value

    def decode_step(self, ids: torch.Tensor, logits: torch.Tensor, stream=None):
        check(lib().qwen3_decode_step(self.ctx, _p(ids), ids.shape[0], _p(logits), _stream(stream)))

    def prefill_host(self, ids: np.ndarray, logits: np.ndarray, all_rows: bool = False, stream=None):
        B, T = ids.shape
        check(lib().qwen3_prefill_host(self.ctx, _p(ids), B, T, _p(logits), ALL_ROWS if all_rows else 0,
                                       _stream(stream)))

    def length(self):
        n, b = ctypes.c_int(), ctypes.c_int()
        check(lib().qwen3_length(self.ctx, ctypes.byref(n), ctypes.byref(b)))
        return n.value, b.value

    def set_length(self, length: int, batch: int, stream=None):
        check(lib().qwen3_set_length(self.ctx, length, batch, _stream(stream)))

    def kv_view(self, layer: int):
        k, v = _vp(), _vp()
        dims = (ctypes.c_int64 * 4)()
        check(lib().qwen3_kv_view(self.ctx, layer, ctypes.byref(k), ctypes.byref(v), dims))
        shape = tuple(dims)
        return device_view(k.value, shape, torch.bfloat16), device_view(v.value, shape, torch.bfloat16)

    def set_tap(self, layer: int, t_in: torch.Tensor | None = None, t_out: torch.Tensor | None = None):
        check(lib().qwen3_set_tap(self.ctx, layer, _p(t_in), _p(t_out)))

    def get_error(self, stream=None) -> int:
        return lib().qwen3_get_error(self.ctx, _stream(stream))

    def set_timing(self, enable: bool):
        check(lib().qwen3_set_timing(self.ctx, int(enable)))

    def kernel_times(self) -> dict:
        n = ctypes.c_int(32)
        ms = (ctypes.c_double * 32)()
        cnt = (ctypes.c_int64 * 32)()
        check(lib().qwen3_kernel_times(self.ctx, ms, cnt, ctypes.byref(n)))
        return {lib().qwen3_kernel_class_name(i).decode(): (ms[i], cnt[i]) for i in range(n.value)}

    def launch_count(self, B: int, T: int, decode: bool = False, all_rows: bool = False) -> int:
        return lib().qwen3_launch_count(self.ctx, B, T, ALL_ROWS if all_rows else 0, int(decode))


# ------------------------------------------------------------------------------ single operations

def op_embed(E, ids, out, err, stream=None):
    V, d = E.shape
    check(lib().qwen3_op_embed(_p(E), V, d, _p(ids), ids.numel(), _p(out), _p(err), _stream(stream)))


def op_rmsnorm(x, gamma, eps, out, rows=None, in_stride=1, in_offset=0, stream=None):
    n = gamma.numel()
    rows = out.numel() // n if rows is None else rows
    check(lib().qwen3_op_rmsnorm(_p(x), _p(gamma), rows, n, in_stride, in_offset, eps, _p(out), _stream(stream)))


def op_gemm(A, B, epi, C, R=None, err=None, stream=None):
    M, K = A.shape
    N = B.shape[0]
    check(lib().qwen3_op_gemm(_p(A), _p(B), M, N, K, epi, _p(C), C.shape[1], _p(R),
                              R.shape[1] if R is not None else 0, _p(err), _stream(stream)))


def gemm_norm_supported(M, N) -> bool:
    return bool(lib().qwen3_gemm_norm_supported(M, N))


def gemm_norm_part_floats(M) -> int:
    return lib().qwen3_gemm_norm_part_floats(M)


def op_gemm_residual_norm(A, B, X, gamma, eps, Y, part, err=None, stream=None):
    """X [M, N] += A B^T in place (bf16 rounding as QWEN3_EPI_RESIDUAL), Y = RMSNorm(X; gamma)."""
    M, K = A.shape
    N = B.shape[0]
    check(lib().qwen3_op_gemm_residual_norm(_p(A), _p(B), M, N, K, _p(X), _p(gamma), eps, _p(Y), _p(part), _p(err),
                                            _stream(stream)))


def gemm_skinny_splits(N, K) -> int:
    return lib().qwen3_gemm_skinny_splits(N, K)


def op_gemm_skinny(A, B, splits, slices=None, out=None, err=None, stream=None):
    M, K = A.shape
    N = B.shape[0]
    check(lib().qwen3_op_gemm_skinny(_p(A), _p(B), M, N, K, splits, _p(slices), _p(out), _p(err), _stream(stream)))


def op_pack_gate_up(gate, up, out, stream=None):
    F, d = gate.shape
    check(lib().qwen3_op_pack_gate_up(_p(gate), _p(up), F, d, _p(out), _stream(stream)))


def op_rope_table(theta, dh, n_pos, out, stream=None):
    check(lib().qwen3_op_rope_table(theta, dh, n_pos, _p(out), _stream(stream)))


def op_qknorm_rope_append(qkv, B, T, Hq, Hkv, dh, q_gamma, k_gamma, table, len0, eps, q_out, k_cache, v_cache,
                          stream=None):
    cap = k_cache.shape[2]
    check(lib().qwen3_op_qknorm_rope_append(_p(qkv), B, T, Hq, Hkv, dh, _p(q_gamma), _p(k_gamma), _p(table),
                                            _p(len0), eps, _p(q_out), _p(k_cache), _p(v_cache), cap,
                                            _stream(stream)))


def attention_prefill_workspace(B, T, Hq, Hkv, dh, kv_chunks) -> int:
    return lib().qwen3_attention_prefill_workspace(B, T, Hq, Hkv, dh, kv_chunks)


def op_attention_prefill(q, k_cache, v_cache, len0, out, err=None, kv_split=0, kv_chunks=1, work=None,
                         seq_meta=None, window=0, ring=0, heads_per_cta=0, stream=None):
    B, Hq, T, dh = q.shape
    Hkv, cap = k_cache.shape[1], k_cache.shape[2]
    check(lib().qwen3_op_attention_prefill(_p(q), _p(k_cache), _p(v_cache), B, T, Hq, Hkv, dh, cap, _p(len0),
                                           _p(seq_meta), window, ring, heads_per_cta, kv_split, kv_chunks, _p(work),
                                           _p(out), _p(err), _stream(stream)))


def attention_decode_workspace(B, Hq, dh, cap, window=0, ring=0) -> int:
    return lib().qwen3_attention_decode_workspace(B, Hq, dh, cap, window, ring)


def op_attention_decode(q, k_cache, v_cache, len0, work, out, seq_meta=None, window=0, ring=0, err=None,
                        stream=None):
    B, Hq, dh = q.shape
    Hkv, cap = k_cache.shape[1], k_cache.shape[2]
    check(lib().qwen3_op_attention_decode(_p(q), _p(k_cache), _p(v_cache), B, Hq, Hkv, dh, cap, _p(len0),
                                          _p(seq_meta), window, ring, _p(work), _p(out), _p(err), _stream(stream)))


_greedy_work = {}


def greedy_workspace(B) -> int:
    return lib().qwen3_greedy_workspace(B)


def op_greedy(logits, next_ids, stop_id=-1, done=None, work="auto", stream=None):
    """work: "auto" (a zeroed scratch buffer kept per device and size, reused across calls on one stream),
    None (one CTA per row), or a caller tensor of greedy_workspace(B) bytes, zero before its first use."""
    B, V = logits.shape
    if isinstance(work, str):
        key = (logits.device, greedy_workspace(B))
        if key not in _greedy_work:
            _greedy_work[key] = torch.zeros(max(1, key[1] // 4), dtype=torch.int32, device=logits.device)
        work = _greedy_work[key]
    check(lib().qwen3_op_greedy(_p(logits), logits.stride(0), B, V, stop_id, _p(done), _p(next_ids), _p(work),
                                _stream(stream)))


# The operators below check their tensors: a wrong type, shape, layout or device raises ValueError before anything
# is launched (sizes that the library itself refuses raise Qwen3Error). A decode step calls them in a launch-bound
# loop, so a call's tensors are compared in one expression, and what is wrong is worked out only when that fails.

_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32


def _want(ok, what: str):
    if not ok:
        raise ValueError(what)


def _dense(name, t, dtype, shape, device: int) -> int:
    """Address of t, which must be a contiguous tensor of this type and shape on CUDA device `device` (-1: the host)."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == device
            and t.is_contiguous()):
        return t.data_ptr()
    got = (f"{t.dtype} {tuple(t.shape)} on {t.device}, strides {t.stride()}" if isinstance(t, torch.Tensor)
           else type(t).__name__)
    raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(shape)} on CUDA device {device}, not {got}")


def _launch(fn, args, device: int, stream):
    """Call an entry point with `device` as the current CUDA device, on its current stream unless one is given."""
    if device < 0:
        raise ValueError("the tensors must be on a CUDA device")
    if stream is None and torch._C._cuda_getDevice() == device:
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(device))
    else:
        _want(stream is None or stream.device.index == device, "the stream belongs to another device")
        with torch.cuda.device(device):
            rc = fn(*args, (torch.cuda.current_stream() if stream is None else stream).cuda_stream)
    if rc:
        check(rc)


LOGPROB_MAX_TOP = 32


def op_token_logprobs(logits, tokens=None, logprob=None, entropy=None, top_ids=None, top_logprobs=None, err=None,
                      stream=None):
    """Log probabilities of `tokens` [M] int32 under logits [M, V] (fp32 or bf16, unit stride along V) into logprob [M],
    each row's entropy (nats) into entropy [M], and its largest alternatives, largest first, into top_ids [M, k] int32
    and top_logprobs [M, k]; outputs are fp32, and those left out are not computed. err: device int (bit 1: a token id
    outside the vocabulary)."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits must be a tensor [M, V]")
    f32 = logits.dtype is _F32
    if not f32 and logits.dtype is not _BF16:
        raise ValueError("logits must be fp32 or bf16")
    M, V = logits.shape
    dev = logits.get_device()
    ld, unit = logits.stride()
    if V < 1 or (V > 1 and unit != 1):
        raise ValueError("logits must be dense along the vocabulary")
    if M > 1 << 27 or V >= 1 << 31:
        raise ValueError("at most 2^27 rows of fewer than 2^31 logits")
    if M <= 1:
        ld = V
    if ld < V:
        raise ValueError("rows of the logits overlap")
    if (tokens is None) != (logprob is None):
        raise ValueError("tokens and logprob go together")
    k = 0
    if top_ids is not None or top_logprobs is not None:
        t = top_logprobs if top_ids is None else top_ids
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError("top_ids and top_logprobs must be tensors [M, k]")
        k = t.shape[1]
        if k > V or k > LOGPROB_MAX_TOP:
            raise ValueError("at most 32 alternatives, and no more than the vocabulary")
    row, top = (M,), (M, k)
    p_tok = p_lp = p_ent = p_ids = p_tops = p_err = None
    if tokens is not None:
        p_tok = _dense("tokens", tokens, _I32, row, dev)
        p_lp = _dense("logprob", logprob, _F32, row, dev)
    if entropy is not None:
        p_ent = _dense("entropy", entropy, _F32, row, dev)
    if top_ids is not None:
        p_ids = _dense("top_ids", top_ids, _I32, top, dev)
    if top_logprobs is not None:
        p_tops = _dense("top_logprobs", top_logprobs, _F32, top, dev)
    if err is not None:
        p_err = _dense("err", err, _I32, (1,), dev)
    if M == 0:
        return
    _launch(lib().qwen3_op_token_logprobs,
            (logits.data_ptr(), 0 if f32 else 1, ld, M, V, p_tok, k, p_lp, p_ent, p_ids, p_tops, p_err), dev, stream)


def _attention_tensors(q, what, k_cache, v_cache, len0, out, out_shape, dev):
    """Check the tensors of an attention call: q (its shape as `what` says), caches [B, Hkv, cap, dh], len0 [1] (one
    length for all) or [B], out of out_shape. Returns Hkv, cap and the library's len_stride."""
    try:
        shape = k_cache.shape
        n, = len0.shape
        B, Hkv, cap, dh = shape
        if (q.dtype is _BF16 and k_cache.dtype is _BF16 and v_cache.dtype is _BF16 and out.dtype is _BF16
                and len0.dtype is _I32 and v_cache.shape == shape and out.shape == out_shape
                and B == q.shape[0] and dh == q.shape[-1] and (n == 1 or n == B) and Hkv >= 1 and cap >= 1
                and q.shape[1] % Hkv == 0 and k_cache.get_device() == dev and v_cache.get_device() == dev
                and out.get_device() == dev and len0.get_device() == dev and q.is_contiguous()
                and k_cache.is_contiguous() and v_cache.is_contiguous() and out.is_contiguous() and len0.is_contiguous()):
            return Hkv, cap, 0 if n == 1 else 1
    except (AttributeError, ValueError):  # not tensors, or not of these numbers of dimensions
        pass
    _dense(f"q {what}", q, _BF16, q.shape, dev)
    _want(isinstance(k_cache, torch.Tensor) and k_cache.dim() == 4, "k_cache must be a tensor [B, Hkv, cap, dh]")
    shape = k_cache.shape
    _want(shape[0] == q.shape[0] and shape[3] == q.shape[-1], "the caches do not match the queries' batch and head_dim")
    _want(shape[1] >= 1 and shape[2] >= 1 and q.shape[1] % shape[1] == 0,
          "query heads must be a multiple of kv heads, with at least one slot")
    _dense("k_cache", k_cache, _BF16, shape, dev)
    _dense("v_cache", v_cache, _BF16, shape, dev)
    _want(isinstance(len0, torch.Tensor) and len0.dim() == 1 and len0.shape[0] in (1, q.shape[0]),
          "len0 must be a tensor [1] (one length for all) or [B]")
    _dense("len0", len0, _I32, len0.shape, dev)
    _dense("out", out, _BF16, out_shape, dev)
    raise ValueError("the tensors do not fit the call")


def attention_decode_shared_workspace(B, Hq, Hkv, dh, prefix_len) -> int:
    return lib().qwen3_attention_decode_shared_workspace(B, Hq, Hkv, dh, prefix_len)


def op_attention_decode_shared(q, k_prefix, v_prefix, k_cache, v_cache, len0, work, out, prefix_len=None, seq_meta=None,
                               err=None, stream=None):
    """Decode attention of q [B, Hq, dh] over a prefix shared by the batch (k_prefix, v_prefix [Hkv, P, dh], the first
    prefix_len rows of it; None: no prefix) and each sequence's own cache [B, Hkv, cap, dh], slots 0..len0, into out
    [B, Hq*dh]. work: attention_decode_shared_workspace bytes of scratch of any type (None without a prefix)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a tensor [B, Hq, dh]")
    B, Hq, dh = q.shape
    dev = q.get_device()
    Hkv, cap, stride = _attention_tensors(q, "[B, Hq, dh]", k_cache, v_cache, len0, out, (B, Hq * dh), dev)
    p_k = p_v = p_work = p_meta = p_err = None
    rows = n = 0
    if k_prefix is not None:
        if not isinstance(k_prefix, torch.Tensor) or k_prefix.dim() != 3:
            raise ValueError("k_prefix must be a tensor [Hkv, P, dh]")
        rows = k_prefix.shape[1]
        n = rows if prefix_len is None else prefix_len
        if not 0 <= n <= rows:
            raise ValueError("prefix_len is not within the prefix")
        shape = (Hkv, rows, dh)
        p_k = _dense("k_prefix", k_prefix, _BF16, shape, dev)
        p_v = _dense("v_prefix", v_prefix, _BF16, shape, dev)
    else:
        _want(v_prefix is None and not prefix_len, "v_prefix and prefix_len go with k_prefix")
    if B == 0:
        return
    size = 0
    if n > 0:  # the library refuses scratch that is too small
        if not isinstance(work, torch.Tensor) or work.get_device() != dev or not work.is_contiguous():
            raise ValueError("work must be contiguous scratch on the same device, of attention_decode_shared_workspace "
                             "bytes")
        p_work, size = work.data_ptr(), work.nbytes
    if seq_meta is not None:
        p_meta = _dense("seq_meta", seq_meta, _I32, (2 + B,), dev)
    if err is not None:
        p_err = _dense("err", err, _I32, (1,), dev)
    _launch(lib().qwen3_op_attention_decode_shared,
            (q.data_ptr(), p_k, p_v, rows, n, k_cache.data_ptr(), v_cache.data_ptr(), B, Hq, Hkv, dh, cap,
             len0.data_ptr(), stride, p_meta, p_work, size, out.data_ptr(), p_err), dev, stream)


def _int32(v) -> int:
    """v, or the nearest 32-bit integer, for the library to refuse or to take as no limit (a plain conversion would
    drop its upper bits)."""
    return v if -1 << 31 <= v < 1 << 31 else (1 << 31) - 1 if v > 0 else -1 << 31


def attention_sink_rows(sinks) -> int:
    """Cache rows in front of the ring of a rolling buffer with this many sink tokens."""
    return lib().qwen3_attention_sink_rows(_int32(sinks))


def op_attention_prefill_sinks(q, k_cache, v_cache, len0, out, window, sinks, rolling=False, err=None, stream=None):
    """Attention of the new tokens q [B, Hq, T, dh] in slots len0 .. len0+T-1 of the caches [B, Hkv, cap, dh] with a
    sliding window and sink tokens, into out [B*T, Hq*dh]; len0 [1] or [B]."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a tensor [B, Hq, T, dh]")
    B, Hq, T, dh = q.shape
    dev = q.get_device()
    Hkv, cap, stride = _attention_tensors(q, "[B, Hq, T, dh]", k_cache, v_cache, len0, out, (B * T, Hq * dh), dev)
    p_err = None if err is None else _dense("err", err, _I32, (1,), dev)
    if B == 0 or T == 0:
        return
    _launch(lib().qwen3_op_attention_prefill_sinks,
            (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), B, T, Hq, Hkv, dh, cap, len0.data_ptr(), stride,
             _int32(window), _int32(sinks), 1 if rolling else 0, out.data_ptr(), p_err), dev, stream)


def op_attention_decode_sinks(q, k_cache, v_cache, len0, out, window, sinks, rolling=False, err=None, stream=None):
    """The single-token form of op_attention_prefill_sinks: q [B, Hq, dh], out [B, Hq*dh]."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a tensor [B, Hq, dh]")
    B, Hq, dh = q.shape
    dev = q.get_device()
    Hkv, cap, stride = _attention_tensors(q, "[B, Hq, dh]", k_cache, v_cache, len0, out, (B, Hq * dh), dev)
    p_err = None if err is None else _dense("err", err, _I32, (1,), dev)
    if B == 0:
        return
    _launch(lib().qwen3_op_attention_decode_sinks,
            (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), B, Hq, Hkv, dh, cap, len0.data_ptr(), stride,
             _int32(window), _int32(sinks), 1 if rolling else 0, out.data_ptr(), p_err), dev, stream)


# ------------------------------------------------------------------ the paged 4-bit cache and packed batches
#
# The extension module _tensors (csrc/tensors.cpp) looks the tensors over and packs their arguments in one block each (the args
# structs of the header); what is wrong with them is worked out here (the _why functions) only when it finds something.

_U8 = torch.uint8
PAGE_SIZES = (16, 32, 64, 128, 256)
_tensors = None
_PAGE_OF = {(p * (dh // 2 + dh // 16), dh): p for p in PAGE_SIZES for dh in (64, 128)}  # by page bytes and head_dim


def _checks():
    global _tensors
    if _tensors is None:
        path = tensors_path()
        if not os.path.exists(path):
            raise RuntimeError(f"extension not built for this PyTorch and Python ({path}); run __graft_entry__.build() first")
        loader = importlib.machinery.ExtensionFileLoader("_tensors", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_tensors", loader))
        loader.exec_module(module)
        _tensors = module
    return _tensors


def paged4_page_bytes(page_size, dh) -> int:
    """Bytes of a page of page_size tokens of one kv head (0: not a page size or head_dim of the cache)."""
    return lib().qwen3_paged4_page_bytes(_int32(page_size), _int32(dh))


def _why_pages(k_pages, v_pages, page_table, dh, dev):
    """Find what is wrong with a paged cache (k_pages, v_pages [n_pages, Hkv, page bytes] uint8, page_table [sequences,
    max_pages] int32). Returns n_pages, Hkv, the page size and max_pages."""
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        _want(isinstance(t, torch.Tensor) and t.dim() == 3, f"{name} must be a tensor [n_pages, Hkv, page bytes]")
    _want(dh in (64, 128), "head_dim must be 64 or 128")
    n, Hkv, size = k_pages.shape
    page = _PAGE_OF.get((size, dh))
    _want(page is not None, "a page must hold 16, 32, 64, 128 or 256 tokens of paged4_page_bytes")
    _dense("k_pages", k_pages, _U8, (n, Hkv, size), dev)
    _dense("v_pages", v_pages, _U8, (n, Hkv, size), dev)
    _want(isinstance(page_table, torch.Tensor) and page_table.dim() == 2, "page_table must be a tensor [sequences, max_pages]")
    _dense("page_table", page_table, _I32, page_table.shape, dev)
    _want(n >= 1 and Hkv >= 1 and page_table.shape[1] >= 1, "the cache needs a page, a kv head and a page a sequence")
    return n, Hkv, page, page_table.shape[1]


def _why_bounds(cu, start, sequences, dev):
    _dense("cu", cu, _I32, (sequences + 1,), dev)
    _dense("start", start, _I32, (sequences,), dev)


def _why_append(qkv, cu, start, cos_sin, k_pages, v_pages, page_table, q_out, k_out, q_gamma, k_gamma, err):
    _want(isinstance(qkv, torch.Tensor) and qkv.dim() == 2, "qkv must be a tensor [N, (Hq + 2 Hkv) dh]")
    _want(isinstance(q_out, torch.Tensor) and q_out.dim() == 3, "q_out must be a tensor [N, Hq, dh]")
    N, Hq, dh = q_out.shape
    dev = qkv.get_device()
    _, Hkv, _, _ = _why_pages(k_pages, v_pages, page_table, dh, dev)
    _want(Hq >= 1 and Hq % Hkv == 0, "query heads must be a multiple of kv heads")
    width = (Hq + 2 * Hkv) * dh
    _want(qkv.dtype is _BF16 and qkv.shape == (N, width) and qkv.stride(1) == 1,
          f"qkv must be bf16 rows {(N, width)}, dense along a row")
    _why_bounds(cu, start, page_table.shape[0], dev)
    _dense("q_out", q_out, _BF16, (N, Hq, dh), dev)
    _want(isinstance(cos_sin, torch.Tensor) and cos_sin.dim() == 2, "cos_sin must be a tensor [positions, dh]")
    _dense("cos_sin", cos_sin, _BF16, (cos_sin.shape[0], dh), dev)
    if k_out is not None:
        _dense("k_out", k_out, _BF16, (N, Hkv, dh), dev)
    for name, g in (("q_gamma", q_gamma), ("k_gamma", k_gamma)):
        if g is not None:
            _dense(name, g, _BF16, (dh,), dev)
    if err is not None:
        _dense("err", err, _I32, (1,), dev)
    raise ValueError("the tensors do not fit the call")


def op_append_paged4(qkv, cu, start, cos_sin, k_pages, v_pages, page_table, q_out, k_out=None, q_gamma=None, k_gamma=None,
                     eps=1e-6, err=None, stream=None):
    """Head norms (with gammas), rotation and append to the paged 4-bit cache of the rows qkv [N, (Hq + 2 Hkv) dh] (unit
    stride along a row): rows cu[s] .. cu[s+1]-1 take the slots start[s] .. of sequence s. Writes q_out [N, Hq, dh], k_out
    [N, Hkv, dh] (None: not wanted) and the pages; rows from cu[-1] on are left as they were. err: device int (bit 4: a
    page id or a position out of range)."""
    block = _checks().append_paged4(qkv, cu, start, cos_sin, k_pages, v_pages, page_table, q_out, k_out, q_gamma, k_gamma, eps, err)
    if block is None:
        _why_append(qkv, cu, start, cos_sin, k_pages, v_pages, page_table, q_out, k_out, q_gamma, k_gamma, err)
    if block:
        _launch(lib().qwen3_op_append_paged4_block, (block,), qkv.get_device(), stream)


def _why_read(k_pages, v_pages, page_table, cu, start, k_out, v_out, err):
    _want(isinstance(k_out, torch.Tensor) and k_out.dim() == 3, "k_out must be a tensor [N, Hkv, dh]")
    N, _, dh = k_out.shape
    dev = k_out.get_device()
    _, Hkv, _, _ = _why_pages(k_pages, v_pages, page_table, dh, dev)
    _why_bounds(cu, start, page_table.shape[0], dev)
    _dense("k_out", k_out, _BF16, (N, Hkv, dh), dev)
    _dense("v_out", v_out, _BF16, (N, Hkv, dh), dev)
    if err is not None:
        _dense("err", err, _I32, (1,), dev)
    raise ValueError("the tensors do not fit the call")


def op_read_paged4(k_pages, v_pages, page_table, cu, start, k_out, v_out, err=None, stream=None):
    """Slots start[s] .. of sequence s of the paged 4-bit cache into the rows cu[s] .. cu[s+1]-1 of k_out and v_out
    [N, Hkv, dh] bf16."""
    block = _checks().read_paged4(k_pages, v_pages, page_table, cu, start, k_out, v_out, err)
    if block is None:
        _why_read(k_pages, v_pages, page_table, cu, start, k_out, v_out, err)
    if block:
        _launch(lib().qwen3_op_read_paged4_block, (block,), k_out.get_device(), stream)


def attention_decode_paged4_workspace(B, Hq, Hkv, dh) -> int:
    return lib().qwen3_attention_decode_paged4_workspace(B, Hq, Hkv, dh)


def _why_decode_paged4(q, k_pages, v_pages, page_table, len0, work, out, err):
    _want(isinstance(q, torch.Tensor) and q.dim() == 3, "q must be a tensor [B, Hq, dh]")
    B, Hq, dh = q.shape
    dev = q.get_device()
    _, Hkv, _, _ = _why_pages(k_pages, v_pages, page_table, dh, dev)
    _want(Hq >= 1 and Hq % Hkv == 0 and Hq // Hkv <= 8, "query heads must be 1 to 8 times the kv heads")
    _want(page_table.shape[0] == B, "page_table must have a row for each sequence")
    _dense("q", q, _BF16, (B, Hq, dh), dev)
    _dense("len0", len0, _I32, (B,), dev)
    _dense("out", out, _BF16, (B, Hq * dh), dev)
    _want(isinstance(work, torch.Tensor) and work.get_device() == dev and work.is_contiguous(),
          "work must be contiguous scratch on the same device, of attention_decode_paged4_workspace bytes")
    if err is not None:
        _dense("err", err, _I32, (1,), dev)
    raise ValueError("the tensors do not fit the call")


def op_attention_decode_paged4(q, k_pages, v_pages, page_table, len0, work, out, err=None, stream=None):
    """Decode attention of q [B, Hq, dh] over the slots 0..len0[b] of each sequence of the paged 4-bit cache, into out
    [B, Hq*dh]. work: attention_decode_paged4_workspace bytes of scratch of any type."""
    block = _checks().attention_decode_paged4(q, k_pages, v_pages, page_table, len0, work, out, err)
    if block is None:
        _why_decode_paged4(q, k_pages, v_pages, page_table, len0, work, out, err)
    if block:
        _launch(lib().qwen3_op_attention_decode_paged4_block, (block,), q.get_device(), stream)


def attention_packed_plan_bytes(Nq, S) -> int:
    """Bytes of the work list of a packed batch of Nq query rows in S sequences."""
    return lib().qwen3_attention_packed_plan_bytes(_int32(Nq), _int32(S))


def op_attention_packed_plan(cu_q, cu_k, Nq, Nk, plan, err=None, stream=None):
    """Write the work list of a packed batch (query rows cu_q [S + 1], key rows cu_k [S + 1]) into plan, contiguous scratch of
    attention_packed_plan_bytes; made once for all layers. err: device int (bit 4: bounds out of order or range)."""
    _want(isinstance(cu_q, torch.Tensor) and cu_q.dim() == 1 and cu_q.shape[0] >= 1, "cu_q must be a tensor [S + 1]")
    dev = cu_q.get_device()
    n = cu_q.shape[0]
    _dense("cu_q", cu_q, _I32, (n,), dev)
    _dense("cu_k", cu_k, _I32, (n,), dev)
    _want(isinstance(plan, torch.Tensor) and plan.get_device() == dev and plan.is_contiguous(),
          "plan must be contiguous scratch on the same device, of attention_packed_plan_bytes")
    p_err = None if err is None else _dense("err", err, _I32, (1,), dev)
    _launch(lib().qwen3_op_attention_packed_plan,
            (cu_q.data_ptr(), cu_k.data_ptr(), n - 1, _int32(Nq), _int32(Nk), plan.data_ptr(), plan.nbytes, p_err), dev, stream)


def _why_packed(q, k, v, plan, out, err):
    _want(isinstance(q, torch.Tensor) and q.dim() == 3, "q must be a tensor [Nq, Hq, dh]")
    Nq, Hq, dh = q.shape
    dev = q.get_device()
    for name, t in (("q", q), ("k", k), ("v", v)):
        _want(isinstance(t, torch.Tensor) and t.dim() == 3 and t.dtype is _BF16 and t.get_device() == dev and t.shape[2] == dh
              and t.stride(2) == 1 and (t.shape[1] == 1 or t.stride(1) == dh),
              f"{name} must be a bf16 tensor [rows, heads, dh], dense along heads and dims")
    _want(v.shape == k.shape and k.shape[1] >= 1 and Hq >= 1 and Hq % k.shape[1] == 0,
          "k and v must have the same rows and heads, and query heads must be a multiple of them")
    _dense("out", out, _BF16, (Nq, Hq * dh), dev)
    _want(isinstance(plan, torch.Tensor) and plan.get_device() == dev and plan.is_contiguous(),
          "plan must be the contiguous work list that op_attention_packed_plan wrote, on the same device")
    if err is not None:
        _dense("err", err, _I32, (1,), dev)
    raise ValueError("the tensors do not fit the call")


def op_attention_prefill_packed(q, k, v, plan, longest, out, err=None, stream=None):
    """Causal attention over packed sequences: q [Nq, Hq, dh], k and v [Nk, Hkv, dh] (rows may be further apart, as views of
    packed qkv rows are), plan as op_attention_packed_plan wrote it for these Nq and Nk; out [Nq, Hq*dh]. longest = keys of
    the longest sequence, a hint for the launch (any value is right)."""
    block = _checks().attention_prefill_packed(q, k, v, plan, longest, out, err)
    if block is None:
        _why_packed(q, k, v, plan, out, err)
    if block:
        _launch(lib().qwen3_op_attention_prefill_packed_block, (block,), q.get_device(), stream)
