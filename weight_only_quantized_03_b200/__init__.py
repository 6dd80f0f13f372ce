"""Python binding of libqg, weight-only-quantized decode kernels for B200.

Argument marshalling only: every function here forwards torch tensors' device
pointers, shapes and the current CUDA stream to the C ABI of the same name
(include/qg.h) and raises QGError when it returns a non-zero status. No
computation happens in Python and there is no fallback: importing this module
fails if libqg.so is missing.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# QG_LIBRARY may name the diagnostic build next to it (libqg_timeline.so)
_NAME = os.environ.get("QG_LIBRARY", "libqg.so")
if _NAME not in ("libqg.so", "libqg_timeline.so"):
    raise ImportError(f"QG_LIBRARY={_NAME!r}: expected libqg.so or libqg_timeline.so")
LIB_PATH = os.path.join(_HERE, _NAME)

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python weight_only_quantized_03_b200/build.py`"
    )
lib = ctypes.CDLL(LIB_PATH)

QG_OK = 0
QG_ERR_INVALID_ARGUMENT = 1
QG_ERR_UNSUPPORTED_SHAPE = 2
QG_ERR_MISALIGNED = 3
QG_ERR_WORKSPACE_TOO_SMALL = 4
QG_ERR_CUDA = 5
QG_ERR_TIMEOUT = 6
QG_F32 = 0
QG_BF16 = 1
QG_KV_BF16 = 0
QG_KV_INT8 = 1
QG_KV_BLOCK = 16

_vp = ctypes.c_void_p
_i = ctypes.c_int
_f = ctypes.c_float
_d = ctypes.c_double
_sz = ctypes.c_size_t
_ll = ctypes.c_longlong


class QGError(RuntimeError):
    def __init__(self, name, status, msg):
        super().__init__(f"{name} returned {status}: {msg}")
        self.status = status


class qg_affine8_matrix(ctypes.Structure):
    _fields_ = [("w", _vp), ("scales", _vp), ("biases", _vp)]


class qg_qwen3_layer(ctypes.Structure):
    _fields_ = [("input_norm", _vp), ("post_norm", _vp), ("q_norm", _vp), ("k_norm", _vp)] + [
        (n, qg_affine8_matrix) for n in ("q", "k", "v", "o", "gate", "up", "down")]


class qg_qwen3_config(ctypes.Structure):
    _fields_ = [("hidden", _i), ("layers", _i), ("heads", _i), ("kv_heads", _i),
                ("head_dim", _i), ("ffn", _i), ("vocab", _i), ("eps", _f), ("theta", _d)]


class qg_qwen3_weights(ctypes.Structure):
    _fields_ = [("embed", qg_affine8_matrix), ("final_norm", _vp),
                ("layers", ctypes.POINTER(qg_qwen3_layer))]


class qg_whisper_config(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int), ("heads", ctypes.c_int), ("ffn", ctypes.c_int),
                ("eps", ctypes.c_float)]


class qg_whisper_layer(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("ln1_g", "ln1_b", "q", "q_b", "k", "v", "v_b", "o", "o_b", "ln2_g", "ln2_b",
                 "fc1", "fc1_b", "fc2", "fc2_b")]


class qg_paged_kv(ctypes.Structure):
    _fields_ = [("k_pages", _vp), ("v_pages", _vp), ("k_scales", _vp), ("v_scales", _vp),
                ("num_pages", _i), ("page_size", _i), ("kv_heads", _i), ("head_dim", _i),
                ("dtype", _i)]


class qg_code_predictor_weights(ctypes.Structure):
    _fields_ = [("input_proj", qg_affine8_matrix),
                ("code_embed", ctypes.POINTER(qg_affine8_matrix)),
                ("heads", ctypes.POINTER(qg_affine8_matrix)),
                ("layers", ctypes.POINTER(qg_qwen3_layer)), ("final_norm", _vp), ("groups", _i)]


_SIGS = {
    "qg_last_error": (ctypes.c_char_p, []),
    "qg_abi_version": (_i, []),
    "qg_kernel_launch_count": (ctypes.c_ulonglong, []),
    "qg_gemv_affine8_g64": (_i, [_vp, _vp, _vp, _vp, _i, _vp, _i, _vp, _i, _i, _i, _vp]),
    "qg_gemv_q4_0": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _vp]),
    "qg_gemm_q4_0_workspace_size": (_sz, [_i, _i, _i]),
    "qg_gemm_q4_0": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _vp, _sz, _vp]),
    "qg_gemm_q4_0_error": (_i, [_i, _i, _vp, ctypes.POINTER(ctypes.c_uint), _vp]),
    "qg_rmsnorm": (_i, [_vp, _vp, _f, _vp, _i, _i, _i, _vp]),
    "qg_rmsnorm_perhead": (_i, [_vp, _i, _vp, _f, _vp, _i, _i, _i, _i, _vp]),
    "qg_rope_neox": (_i, [_vp, _i, _vp, _d, _i, _i, _i, _i, _vp]),
    "qg_silu_mul": (_i, [_vp, _vp, _vp, _i, _i, _vp]),
    "qg_residual_add": (_i, [_vp, _vp, _i, _vp]),
    "qg_embed_affine8_g64": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _vp]),
    "qg_decode_attention_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "qg_decode_attention": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _sz,
                                 _vp]),
    "qg_decode_attention_static_scratch_capacity": (_sz, []),
    "qg_decode_attention_static_scratch": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i,
                                                _f, _vp]),
    "qg_decode_step_workspace_size": (_sz, [ctypes.POINTER(qg_qwen3_config), _i, _i]),
    "qg_decode_step": (_i, [ctypes.POINTER(qg_qwen3_config), ctypes.POINTER(qg_qwen3_weights),
                            _vp, _vp, _i, _vp, _vp, _vp, _i, _vp, _sz, _vp]),
    "qg_decode_step_inspect": (_i, [ctypes.POINTER(qg_qwen3_config), _i, _i,
                                    ctypes.POINTER(ctypes.c_size_t)]),
    "qg_decode_step_inspect_f32": (_i, [ctypes.POINTER(qg_qwen3_config), _i, _i,
                                        ctypes.POINTER(ctypes.c_size_t)]),
    "qg_code_predict_workspace_size": (_sz, [ctypes.POINTER(qg_qwen3_config), _i]),
    "qg_gemm_q4_0_ex": (_i, [_vp, _vp, _i, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _sz, _vp]),
    "qg_gemm_q4_0_stall_test": (_i, [_vp, _vp, _vp, _i, _i, _i, _vp, _sz, _vp]),
    "qg_gemm_affine8_g64": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _vp, _sz, _vp]),
    "qg_prefill_workspace_size": (_sz, [ctypes.POINTER(qg_qwen3_config), _i]),
    "qg_prefill": (_i, [ctypes.POINTER(qg_qwen3_config), ctypes.POINTER(qg_qwen3_weights), _vp,
                        _vp, _i, _vp, _i, _i, _vp, _vp, _sz, _vp]),
    "qg_prefill_inspect": (_i, [ctypes.POINTER(qg_qwen3_config), _i,
                                ctypes.POINTER(ctypes.c_size_t)]),
    "qg_layernorm": (_i, [_vp, _vp, _vp, _f, _vp, _i, _i, _i, _vp]),
    "qg_attention_rows": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp]),
    "qg_whisper_encoder_layer_workspace_size": (_sz, [ctypes.POINTER(qg_whisper_config), _i]),
    "qg_whisper_encoder_layer": (_i, [ctypes.POINTER(qg_whisper_config),
                                      ctypes.POINTER(qg_whisper_layer), _vp, _i, _vp, _sz, _vp]),
    "qg_whisper_encoder_layer_inspect": (_i, [ctypes.POINTER(qg_whisper_config), _i,
                                              ctypes.POINTER(ctypes.c_size_t)]),
    "qg_timeline_available": (_i, []),
    "qg_timeline_begin": (_i, [_vp, _i]),
    "qg_timeline_end": (_i, [ctypes.POINTER(ctypes.c_int), _i]),
    "qg_code_predict_trace_layout": (_i, [ctypes.POINTER(qg_qwen3_config), _i, _i,
                                          ctypes.POINTER(ctypes.c_size_t)]),
    "qg_code_predict_traced": (_i, [ctypes.POINTER(qg_qwen3_config),
                                    ctypes.POINTER(qg_code_predictor_weights), _vp, _vp, _vp,
                                    _vp, _i, _vp, _sz, _vp, _sz, _vp]),
    "qg_code_predict": (_i, [ctypes.POINTER(qg_qwen3_config),
                             ctypes.POINTER(qg_code_predictor_weights), _vp, _vp, _vp, _vp, _i,
                             _vp, _sz, _vp]),
    "qg_token_logprob_workspace_size": (_sz, [_i, _i]),
    "qg_token_logprob": (_i, [_vp, _i, _i, _vp, _vp, _vp, _sz, _vp]),
    "qg_sample_workspace_size": (_sz, [_i, _i, _i]),
    "qg_sample": (_i, [_vp, _i, _i, _vp, _i, _f, _f, _i, _vp, _vp, _vp, _sz, _vp]),
    "qg_paged_kv_append": (_i, [_vp, _vp, _i, _vp, _vp, _vp, _ll, _vp, _ll, _vp, _ll, _i, _vp, _vp,
                                _f, _d, _i, _vp, _i, _i, _i, _i, _vp]),
    "qg_paged_kv_gather": (_i, [_vp, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _vp]),
    "qg_paged_attention_workspace_size": (_sz, [_i]),
    "qg_paged_attention": (_i, [_vp, _vp, _i, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _f, _vp, _sz,
                                _vp]),
    "qg_sample_filtered": (_i, [_vp, _ll, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "qg_step_graphs_enable": (None, [_i]),
    "qg_step_graphs_clear": (None, []),
    "qg_argmax_workspace_size": (_sz, [_i, _i]),
    "qg_argmax_f32": (_i, [_vp, _i, _i, _vp, _vp, _sz, _vp]),
    "qg_unpack_affine8": (_i, [_vp, _vp, _i, _i, _vp]),
    "qg_dequant_affine8_g64": (_i, [_vp, _vp, _vp, _vp, _i, _i, _vp]),
    "qg_dequant_q4_0": (_i, [_vp, _vp, _i, _i, _vp]),
}

for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def last_error() -> str:
    return lib.qg_last_error().decode()


def _call(name, *args):
    st = getattr(lib, name)(*args)
    if st != QG_OK:
        raise QGError(name, st, last_error())


def _p(t):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _current_device():
    """Index of the current device (tensors on one exist, so CUDA is up)."""
    return torch._C._cuda_getDevice()


def _raw_stream(stream, dev):
    """``_stream`` without building a stream object."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return _stream(stream)


def _dt(t):
    dt = t.dtype
    if dt is torch.float32:
        return QG_F32
    if dt is torch.bfloat16:
        return QG_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


# ------------------------------------------------------------------ ops ----

def qg_gemv_affine8_g64(w, scales, biases, x, y, residual=None, stream=None):
    """y[B,N] = dequant(w, scales, biases)[N,K] @ x[B,K] (+ residual). w is
    int32/uint32-viewed [N, K/4]; scales/biases int16/bf16 bits [N, K/64]."""
    N, K = w.shape[0], w.shape[1] * 4
    B = x.shape[0] if x.dim() == 2 else 1
    _call("qg_gemv_affine8_g64", _p(w), _p(scales), _p(biases), _p(x), _dt(x), _p(y), _dt(y),
          _p(residual), N, K, B, _stream(stream))


def qg_gemv_q4_0(blocks, x, y, bias=None, stream=None):
    N = blocks.shape[0]
    K = blocks.shape[1] // 18 * 32
    B = x.shape[0] if x.dim() == 2 else 1
    _call("qg_gemv_q4_0", _p(blocks), _p(x), _p(bias), _p(y), N, K, B, _stream(stream))


def qg_gemm_q4_0_workspace_size(M, N, K):
    return int(lib.qg_gemm_q4_0_workspace_size(M, N, K))


def qg_gemm_q4_0(blocks, A, C, bias=None, ws=None, stream=None):
    N = blocks.shape[0]
    K = blocks.shape[1] // 18 * 32
    M = A.shape[0]
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _call("qg_gemm_q4_0", _p(blocks), _p(A), _p(bias), _p(C), M, N, K, _p(ws), nbytes,
          _stream(stream))


def qg_gemm_q4_0_ex(blocks, A, C, bias=None, residual=None, gelu=False, ws=None, stream=None):
    """C = epilogue(bf16(A) @ bf16(W)^T + bias (+ residual)), A fp32 or bf16
    [M, K], C fp32 or bf16 [M, N]; gelu applies gelu_tanh."""
    N = blocks.shape[0]
    K = blocks.shape[1] // 18 * 32
    M = A.shape[0]
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _call("qg_gemm_q4_0_ex", _p(blocks), _p(A), _dt(A), _p(bias), _p(residual), _p(C), _dt(C),
          1 if gelu else 0, M, N, K, _p(ws), nbytes, _stream(stream))


def qg_gemm_affine8_g64(w, scales, biases, x, y, residual=None, ws=None, stream=None):
    """y[T, N] = x[T, K] (bf16) @ dequant(w)[N, K]^T (+ residual) on the
    tensor cores; ws holds the 4-byte error word."""
    N, K = w.shape[0], w.shape[1] * 4
    T = x.shape[0]
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _call("qg_gemm_affine8_g64", _p(w), _p(scales), _p(biases), _p(x), _p(y), _dt(y),
          _p(residual), N, K, T, _p(ws), nbytes, _stream(stream))


def qg_layernorm(x, gamma, beta, eps, y, stream=None):
    _call("qg_layernorm", _p(x), _p(gamma), _p(beta), eps, _p(y), _dt(y), x.shape[0],
          x.shape[1], _stream(stream))


def qg_attention_rows(q, k, v, out, H, Hkv, causal=False, stream=None):
    """q, out bf16 [B, T, H*D]; k, v bf16 [B, S, Hkv*D] (a leading batch
    dimension may be omitted)."""
    if q.dim() == 2:
        q, k, v, out = q[None], k[None], v[None], out[None]
    B, T = q.shape[0], q.shape[1]
    S = k.shape[1]
    D = q.shape[2] // H
    _call("qg_attention_rows", _p(q), _p(k), _p(v), _p(out), B, T, S, H, Hkv, D,
          1 if causal else 0, _stream(stream))


def qg_gemm_q4_0_error(M, K, ws, stream=None):
    """(status, code) of the device error word of the last GEMM on ``ws``."""
    code = ctypes.c_uint(0)
    st = lib.qg_gemm_q4_0_error(M, K, _p(ws), ctypes.byref(code), _stream(stream))
    return st, code.value


def qg_rmsnorm(x, w, eps, y, stream=None):
    rows, dim = x.shape
    _call("qg_rmsnorm", _p(x), _p(w), float(eps), _p(y), _dt(y), rows, dim, _stream(stream))


def qg_rmsnorm_perhead(x, w, eps, y, heads, stream=None):
    rows = x.shape[0]
    D = x.shape[1] // heads
    _call("qg_rmsnorm_perhead", _p(x), _dt(x), _p(w), float(eps), _p(y), _dt(y), rows, heads, D,
          _stream(stream))


def qg_rope_neox(x, pos, theta, heads, rotary_dim=None, stream=None):
    rows = x.shape[0]
    D = x.shape[1] // heads
    _call("qg_rope_neox", _p(x), _dt(x), _p(pos), float(theta), rows, heads, D,
          D if rotary_dim is None else rotary_dim, _stream(stream))


def qg_silu_mul(gate, up, out, stream=None):
    _call("qg_silu_mul", _p(gate), _p(up), _p(out), _dt(out), gate.numel(), _stream(stream))


def qg_residual_add(x, delta, stream=None):
    _call("qg_residual_add", _p(x), _p(delta), x.numel(), _stream(stream))


def qg_embed_affine8_g64(w, scales, biases, tokens, x, stream=None):
    _call("qg_embed_affine8_g64", _p(w), _p(scales), _p(biases), _p(tokens), _p(x), w.shape[0],
          w.shape[1] * 4, tokens.numel(), _stream(stream))


def qg_decode_attention_workspace_size(B, H, Hkv, D, cap):
    return int(lib.qg_decode_attention_workspace_size(B, H, Hkv, D, cap))


def qg_decode_attention(q, k_cache, v_cache, kv_len, out, H, Hkv, scale, ws, stream=None):
    """q [B, H*D] fp32; caches [B, Hkv, cap, D] bf16; kv_len int32 [B]."""
    B, _, cap, D = k_cache.shape
    _call("qg_decode_attention", _p(q), _p(k_cache), _p(v_cache), _p(kv_len), _p(out), _dt(out),
          B, H, Hkv, D, cap, float(scale), _p(ws), ws.numel() * ws.element_size(),
          _stream(stream))


def qg_argmax_workspace_size(B, V):
    return int(lib.qg_argmax_workspace_size(B, V))


def qg_argmax_f32(logits, out, ws, stream=None):
    """out[b] (int32, device) = first strict maximum of logits[b] (fp32
    [B, V]), NaNs skipped, 0 when nothing beats -inf."""
    B, V = logits.shape
    _call("qg_argmax_f32", _p(logits), B, V, _p(out), _p(ws), ws.numel() * ws.element_size(),
          _stream(stream))


def qg_token_logprob(logits, tokens, out, ws, stream=None):
    """out[b] (fp32, device) = log-softmax of logits[b] (fp32 [B, V]) at
    tokens[b] (int32, device)."""
    B, V = logits.shape
    _call("qg_token_logprob", _p(logits), B, V, _p(tokens), _p(out), _p(ws),
          ws.numel() * ws.element_size(), _stream(stream))


def qg_sample_workspace_size(B, V, top_k):
    return int(lib.qg_sample_workspace_size(B, V, top_k))


def qg_sample(logits, out, ws, past=None, penalty=1.0, temperature=1.0, top_k=0, r=None,
              stream=None):
    """out[b] (int32, device): repetition penalty over past[b] (int32 [B, P],
    -1 = empty), then greedy (top_k 0 or temperature 0) or a top-k draw with
    the uniform numbers r (fp32 [B]) from the temperature softmax."""
    B, V = logits.shape
    P = 0 if past is None else past.shape[1]
    _call("qg_sample", _p(logits), B, V, _p(past), P, float(penalty), float(temperature),
          int(top_k), _p(r), _p(out), _p(ws), ws.numel() * ws.element_size(), _stream(stream))


def qg_sample_filtered(logits, u, out, temperature=None, top_k=None, top_p=None, min_p=None,
                       kept=None, logprob=None, stream=None):
    """out[b] (int32 [B]): a token of logits[b] (fp32 [B, V], rows may lie
    apart) drawn with the uniform number u[b] after temperature, top_k, top_p
    and min_p, each a device tensor [B] (fp32; top_k int32) or None for off.
    kept (int32) and logprob (fp32), when given, get the number of tokens
    kept and the drawn one's log-probability among them."""
    B, V = logits.shape
    dev = _current_device()
    if logits.dtype is not torch.float32:
        raise TypeError(f"logits must be float32, not {logits.dtype}")
    ld = _rows_of("logits", logits, V)
    floats, ints = (u, temperature, top_p, min_p, logprob), (out, top_k, kept)
    for some, dt in ((floats, torch.float32), (ints, torch.int32)):
        for t in some:
            if t is not None and (t.dtype is not dt or t.dim() != 1 or t.numel() != B
                                  or not t.is_contiguous() or t.get_device() != dev):
                _check_device(dev, ("u", u), ("out", out), ("temperature", temperature),
                              ("top_k", top_k), ("top_p", top_p), ("min_p", min_p),
                              ("kept", kept), ("logprob", logprob))
                names = ("u", "temperature", "top_p", "min_p", "logprob", "out", "top_k", "kept")
                name = [n for n, x in zip(names, floats + ints) if x is t][0]
                raise ValueError(f"{name} must be a contiguous {dt} tensor of {B} values")
    if logits.get_device() != dev:
        _check_device(dev, ("logits", logits))
    st = _sample(logits.data_ptr(), ld, B, V, _p(temperature), _p(top_k), _p(top_p), _p(min_p),
                 u.data_ptr(), out.data_ptr(), _p(kept), _p(logprob), _raw_stream(stream, dev))
    if st:
        raise QGError("qg_sample_filtered", st, last_error())


def qg_decode_attention_static_scratch_capacity():
    return int(lib.qg_decode_attention_static_scratch_capacity())


def qg_decode_attention_static_scratch(q, k_cache, v_cache, kv_len, out, H, Hkv, scale,
                                       stream=None):
    """qg_decode_attention with the library's fixed scratch (no workspace)."""
    B, _, cap, D = k_cache.shape
    _call("qg_decode_attention_static_scratch", _p(q), _p(k_cache), _p(v_cache), _p(kv_len),
          _p(out), _dt(out), B, H, Hkv, D, cap, float(scale), _stream(stream))


def qg_unpack_affine8(w, out, stream=None):
    _call("qg_unpack_affine8", _p(w), _p(out), w.shape[0], w.shape[1] * 4, _stream(stream))


def qg_dequant_affine8_g64(w, scales, biases, out, stream=None):
    _call("qg_dequant_affine8_g64", _p(w), _p(scales), _p(biases), _p(out), w.shape[0],
          w.shape[1] * 4, _stream(stream))


def qg_dequant_q4_0(blocks, out, stream=None):
    _call("qg_dequant_q4_0", _p(blocks), _p(out), blocks.shape[0], blocks.shape[1] // 18 * 32,
          _stream(stream))


# ------------------------------------------------------------ paged cache ----
# A serving loop makes these calls once a layer and token, so their checks
# are written to cost little: plain loops, no keyword dictionaries.

_PAGED_KV = struct.Struct("@PPPPiiiii").pack  # the fields of qg_paged_kv


_append, _gather = lib.qg_paged_kv_append, lib.qg_paged_kv_gather
_attend, _sample = lib.qg_paged_attention, lib.qg_sample_filtered
_f32, _bf16, _i32 = torch.float32, torch.bfloat16, torch.int32
_TYPES = {_f32: QG_F32, _bf16: QG_BF16}


def _check_device(dev, *named):
    """Every given tensor of the (name, tensor) pairs is on CUDA device ``dev``."""
    for name, t in named:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, not on the current device cuda:{dev}")


def _check_index(dev, name, t, n):
    """A contiguous int32 tensor of n values on device ``dev``."""
    if t.dtype is not torch.int32 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n} values")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on the current device cuda:{dev}")


def _rows_of(name, t, width):
    """Row stride (elements) of [rows, width] whose rows may lie apart."""
    shape = t.shape
    if len(shape) == 2 and shape[1] == width:
        ld, one = t.stride()
        if one == 1 or shape[0] == 0:
            return ld if shape[0] > 1 else max(ld, width)
    raise ValueError(f"{name} must be [rows, {width}] with unit stride along a row, got "
                     f"{tuple(shape)} with strides {t.stride()}")


_BF16_BITS = (_bf16, torch.int16, torch.uint16)  # bf16 values, or their bits


def _check_norm(w, D):
    """A norm weight of D bf16 values (float16 has another meaning per bit)."""
    if w.dtype not in _BF16_BITS or w.numel() != D or not w.is_contiguous():
        raise ValueError(f"q_norm and k_norm must be contiguous, {D} bf16 values (or their bits as "
                         f"int16), not {w.dtype} {tuple(w.shape)}")


class PagedKV:
    """A pool of K/V pages of one layer (``qg_paged_kv``): ``k_pages`` and
    ``v_pages`` [num_pages, kv_heads, page_size, head_dim], bfloat16, or int8
    with fp32 ``k_scales`` and ``v_scales`` [num_pages, kv_heads,
    page_size / 16]. The tensors are borrowed and kept alive."""

    def __init__(self, k_pages, v_pages, k_scales=None, v_scales=None):
        shape, dtype = k_pages.shape, k_pages.dtype
        if len(shape) != 4 or v_pages.shape != shape or v_pages.dtype is not dtype:
            raise ValueError("k_pages and v_pages must be [num_pages, kv_heads, page_size, "
                             "head_dim] of one type")
        int8 = dtype is torch.int8
        if not int8 and dtype is not _bf16:
            raise TypeError(f"pages must be bfloat16 or int8, not {dtype}")
        P, Hkv, size, D = shape
        self.device_index = dev = k_pages.get_device()
        ks = vs = 0
        if int8:
            blocks = (P, Hkv, size // QG_KV_BLOCK)
            for name, s in (("k_scales", k_scales), ("v_scales", v_scales)):
                if s is None:
                    raise ValueError(f"{name} goes with int8 pages only, and they need it")
                if s.dtype is not _f32 or s.shape != blocks or not s.is_contiguous() \
                        or s.get_device() != dev:
                    raise ValueError(f"{name} must be contiguous fp32 {list(blocks)} on the "
                                     f"pages' device")
            ks, vs = k_scales.data_ptr(), v_scales.data_ptr()
        elif k_scales is not None or v_scales is not None:
            raise ValueError("k_scales and v_scales go with int8 pages only")
        if not (k_pages.is_contiguous() and v_pages.is_contiguous()
                and v_pages.get_device() == dev):
            raise ValueError("k_pages and v_pages must be contiguous, on one device")
        self.k_pages, self.v_pages, self.k_scales, self.v_scales = (k_pages, v_pages, k_scales,
                                                                    v_scales)
        self.kv_heads, self.page_size, self.head_dim = Hkv, size, D
        # the C struct qg_paged_kv (read during a call only)
        self.c_kv = _PAGED_KV(k_pages.data_ptr(), v_pages.data_ptr(), ks, vs, P, size, Hkv, D,
                              QG_KV_INT8 if int8 else QG_KV_BF16)

    @classmethod
    def empty(cls, num_pages, page_size, kv_heads, head_dim, dtype=torch.int8, device="cuda"):
        """A pool of new pages (contents not initialised)."""
        shape = (num_pages, kv_heads, page_size, head_dim)
        pages = [torch.empty(shape, dtype=dtype, device=device) for _ in range(2)]
        if dtype == torch.int8:
            pages += [torch.empty(shape[:2] + (page_size // QG_KV_BLOCK,), device=device)
                      for _ in range(2)]
        return cls(*pages)

    def _batch(self, page_table, lens, lens_name, row_start, T, dev):
        """(B, max_pages), after checking the batch's index tensors."""
        if self.device_index != dev:
            raise ValueError(f"the pages are on device {self.device_index}, not on the current "
                             f"device cuda:{dev}")
        shape = page_table.shape
        if len(shape) != 2:
            raise ValueError("page_table must be [B, max_pages]")
        B, most = shape
        if page_table.dtype is not _i32 or not page_table.is_contiguous() \
                or page_table.get_device() != dev:
            _check_index(dev, "page_table", page_table, B * most)
        if lens is not None and (lens.dtype is not _i32 or lens.numel() != B
                                 or not lens.is_contiguous() or lens.get_device() != dev):
            _check_index(dev, lens_name, lens, B)
        if row_start is None:
            if T != B:
                raise ValueError(f"{T} rows of {B} sequences need row_start")
        elif row_start.dtype is not _i32 or row_start.numel() != B + 1 \
                or not row_start.is_contiguous() or row_start.get_device() != dev:
            _check_index(dev, "row_start", row_start, B + 1)
        return B, most


def qg_paged_kv_append(kv, page_table, kv_len, k, v, row_start=None, q=None, q_out=None,
                       q_norm=None, k_norm=None, eps=1e-6, theta=1e6, rotary_dim=None,
                       stream=None):
    """Norm (optional) and rotate q [T, H*D] and k [T, Hkv*D], append k and v
    to the pages of ``kv`` (a PagedKV) and write the rotated q to q_out
    [T, H*D] (fp32 or bf16; q itself if the types match). Rows of q, k and v
    (fp32 or bf16, one type) may lie apart, as slices of one projection do.
    q_norm and k_norm: D bf16 values (or their bits as int16).
    page_table int32 [B, max_pages]; kv_len int32 [B] counts the new rows;
    row_start int32 [B+1], or None for one row per sequence. ``rotary_dim``
    None: the whole head."""
    dev = _current_device()
    D = kv.head_dim
    W = kv.kv_heads * D
    dt = k.dtype
    if kv_len is None:
        raise ValueError("kv_len is needed")
    k_ld, v_ld = _rows_of("k", k, W), _rows_of("v", v, W)
    T = k.shape[0]
    if v.shape[0] != T or v.dtype is not dt:
        raise ValueError("v must have k's rows and type")
    B, most = kv._batch(page_table, kv_len, "kv_len", row_start, T, dev)
    H, q_ld, qdt, q_at, out_at = 0, 0, QG_BF16, None, None
    if q is not None:
        shape = q.shape
        Q = shape[-1]
        if shape[0] != T or q.dtype is not dt or Q % D:
            raise ValueError(f"q must be [{T}, H * {D}] of k's type")
        H, q_ld = Q // D, _rows_of("q", q, Q)
        if q_out is None or q_out.shape != shape or not q_out.is_contiguous():
            raise ValueError("q_out must be contiguous with q's shape")
        qdt = _TYPES.get(q_out.dtype)
        if qdt is None:
            _dt(q_out)
        q_at, out_at = q.data_ptr(), q_out.data_ptr()
    for t in (k, v, q, q_out, q_norm, k_norm):
        if t is not None and t.get_device() != dev:
            _check_device(dev, ("k", k), ("v", v), ("q", q), ("q_out", q_out), ("q_norm", q_norm),
                          ("k_norm", k_norm))
    for w in (q_norm, k_norm):
        if w is not None:
            _check_norm(w, D)
    xdt = _TYPES.get(dt)
    if xdt is None:
        _dt(k)
    st = _append(kv.c_kv, page_table.data_ptr(), most, kv_len.data_ptr(),
                 None if row_start is None else row_start.data_ptr(), q_at, q_ld, k.data_ptr(),
                 k_ld, v.data_ptr(), v_ld, xdt, None if q_norm is None else q_norm.data_ptr(),
                 None if k_norm is None else k_norm.data_ptr(), eps, theta,
                 D if rotary_dim is None else rotary_dim, out_at, qdt, B, T, H,
                 _raw_stream(stream, dev))
    if st:
        raise QGError("qg_paged_kv_append", st, last_error())


def qg_paged_kv_gather(kv, page_table, first, row_start, k_out=None, v_out=None, stream=None):
    """Cached rows as values: packed row i of sequence b is its token
    first[b] + i (first int32 [B] or None: from 0; row_start int32 [B+1] or
    None: one row each). k_out, v_out contiguous [T, Hkv*D], fp32 or bf16."""
    one = k_out if k_out is not None else v_out
    if one is None:
        return
    dev = _current_device()
    shape, dt = one.shape, one.dtype
    T = shape[0]
    B, most = kv._batch(page_table, first, "first", row_start, T, dev)
    good = len(shape) == 2 and shape[1] == kv.kv_heads * kv.head_dim
    for t in (k_out, v_out):
        if t is not None:
            if t is not one and t.shape != shape or t.dtype is not dt or not t.is_contiguous():
                good = False
            elif t.get_device() != dev:
                _check_device(dev, ("k_out", k_out), ("v_out", v_out))
    if not good:
        raise ValueError(f"k_out and v_out must be contiguous [{T}, "
                         f"{kv.kv_heads * kv.head_dim}] of one type")
    st = _gather(kv.c_kv, page_table.data_ptr(), most, None if first is None else first.data_ptr(),
                 None if row_start is None else row_start.data_ptr(),
                 None if k_out is None else k_out.data_ptr(),
                 None if v_out is None else v_out.data_ptr(), _dt(one), B, T,
                 _raw_stream(stream, dev))
    if st:
        raise QGError("qg_paged_kv_gather", st, last_error())


def qg_paged_attention_workspace_size(head_dim):
    return int(lib.qg_paged_attention_workspace_size(head_dim))


def qg_paged_attention(kv, page_table, kv_len, q, out, H, scale, ws, row_start=None, stream=None):
    """out [T, H*D] (fp32 or bf16) = causal softmax attention of the rows q
    [T, H*D] (fp32 or bf16) over their sequences' cached tokens in the pages
    of ``kv`` (a PagedKV). page_table int32 [B, max_pages]; kv_len int32 [B]
    counts the rows' own tokens; row_start int32 [B+1], or None for one row
    per sequence; ws of qg_paged_attention_workspace_size(D) bytes."""
    dev = _current_device()
    shape = q.shape
    T = shape[0]
    if kv_len is None:
        raise ValueError("kv_len is needed")
    B, most = kv._batch(page_table, kv_len, "kv_len", row_start, T, dev)
    if len(shape) != 2 or shape[1] != H * kv.head_dim or out.shape != shape or \
            not (q.is_contiguous() and out.is_contiguous()):
        raise ValueError(f"q and out must be contiguous [T, {H} * {kv.head_dim}]")
    if q.get_device() != dev or out.get_device() != dev or ws.get_device() != dev:
        _check_device(dev, ("q", q), ("out", out), ("ws", ws))
    st = _attend(kv.c_kv, page_table.data_ptr(), most, kv_len.data_ptr(),
                 None if row_start is None else row_start.data_ptr(), q.data_ptr(), _dt(q),
                 out.data_ptr(), _dt(out), B, T, H, scale, ws.data_ptr(), ws.nbytes,
                 _raw_stream(stream, dev))
    if st:
        raise QGError("qg_paged_attention", st, last_error())


# ---------------------------------------------------------- decode step ----

class Qwen3Model:
    """Device-resident packed Qwen3 weights plus the C structs that point at
    them. ``weights`` is the host dict layout of ``qg_synth.qwen3_weights``
    (numpy arrays); everything is uploaded once to ``device``."""

    def __init__(self, cfg: dict, weights: dict, device="cuda"):
        self.cfg = dict(cfg)
        self._keep = []

        def up(a):
            t = torch.from_numpy(a.view({2: "int16", 4: "int32"}[a.dtype.itemsize])).to(device)
            self._keep.append(t)
            return t.data_ptr()

        def mat(triple):
            w, s, b = triple
            return qg_affine8_matrix(up(w), up(s), up(b))

        self.c_cfg = qg_qwen3_config(cfg["hidden"], cfg["layers"], cfg["heads"], cfg["kv_heads"],
                                     cfg["head_dim"], cfg["ffn"], cfg["vocab"], cfg["eps"],
                                     cfg["theta"])
        L = cfg["layers"]
        self.c_layers = (qg_qwen3_layer * max(L, 1))()
        for i, lw in enumerate(weights["layers"]):
            cl = self.c_layers[i]
            cl.input_norm = up(lw["input_norm"])
            cl.post_norm = up(lw["post_norm"])
            cl.q_norm = up(lw["q_norm"])
            cl.k_norm = up(lw["k_norm"])
            for n in ("q", "k", "v", "o", "gate", "up", "down"):
                setattr(cl, n, mat(lw[n]))
        self.c_weights = qg_qwen3_weights(mat(weights["embed"]), up(weights["final_norm"]),
                                          ctypes.cast(self.c_layers, ctypes.POINTER(qg_qwen3_layer)))
        self.device = device

    def workspace_size(self, B, cap):
        return int(lib.qg_decode_step_workspace_size(ctypes.byref(self.c_cfg), B, cap))

    def new_state(self, B, cap):
        """Zeroed KV caches [layers, B, kv_heads, cap, head_dim] bf16, a
        workspace and a logits
        buffer for batch B."""
        c = self.cfg
        shape = (c["layers"], B, c["kv_heads"], cap, c["head_dim"])
        return dict(
            k_cache=torch.zeros(shape, dtype=torch.bfloat16, device=self.device),
            v_cache=torch.zeros(shape, dtype=torch.bfloat16, device=self.device),
            ws=torch.zeros(self.workspace_size(B, cap), dtype=torch.uint8, device=self.device),
            logits=torch.empty((B, c["vocab"]), dtype=torch.float32, device=self.device),
            B=B, cap=cap)

    def residual(self, state):
        """The fp32 residual stream [B, hidden] after the last layer of the
        latest step (the head of the step workspace, per include/qg.h)."""
        n = state["B"] * self.cfg["hidden"]
        return state["ws"][: 4 * n].view(torch.float32).view(state["B"], self.cfg["hidden"])

    def intermediates(self, state):
        """The last decoder layer's values after a step
        (``qg_decode_step_inspect`` and ``_inspect_f32``): dict of torch views
        into the workspace -- bf16 ``xn`` [B, hidden], ``attn``
        [B, heads*head_dim], ``xn2`` [B, hidden], ``h`` [B, ffn]; fp32
        ``q_proj`` [B, heads*head_dim], ``k_proj``, ``v_proj``
        [B, kv_heads*head_dim], ``x_attn`` [B, hidden], ``gate``, ``up``
        [B, ffn]."""
        c, B = self.cfg, state["B"]
        ws = state["ws"]
        off = (ctypes.c_size_t * 4)()
        _call("qg_decode_step_inspect", ctypes.byref(self.c_cfg), B, state["cap"], off)
        off32 = (ctypes.c_size_t * 6)()
        _call("qg_decode_step_inspect_f32", ctypes.byref(self.c_cfg), B, state["cap"], off32)

        def view(o, n, dt=torch.bfloat16):
            size = 2 if dt == torch.bfloat16 else 4
            return ws[o:o + size * B * n].view(dt).view(B, n)
        HD, KD, h, F = c["heads"] * c["head_dim"], c["kv_heads"] * c["head_dim"], c["hidden"], c["ffn"]
        f32 = torch.float32
        return {"xn": view(off[0], h), "attn": view(off[1], HD), "xn2": view(off[2], h),
                "h": view(off[3], F), "q_proj": view(off32[0], HD, f32),
                "k_proj": view(off32[1], KD, f32), "v_proj": view(off32[2], KD, f32),
                "x_attn": view(off32[3], h, f32), "gate": view(off32[4], F, f32),
                "up": view(off32[5], F, f32)}

    def prefill_workspace(self, T):
        n = int(lib.qg_prefill_workspace_size(ctypes.byref(self.c_cfg), T))
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def qg_prefill(self, state, tokens, p0, ws, logits=None, stream=None, layers=None):
        """The prompt rows ``tokens`` (device int32 [T]) of sequence 0 of
        ``state`` at positions p0 .. p0+T-1; the last row's logits into
        ``logits`` ([vocab]) when given. ``layers`` runs only the first that
        many layers."""
        cfg = self.c_cfg
        if layers is not None:
            cfg = qg_qwen3_config.from_buffer_copy(self.c_cfg)
            cfg.layers = layers
        _call("qg_prefill", ctypes.byref(cfg), ctypes.byref(self.c_weights),
              _p(state["k_cache"]), _p(state["v_cache"]), state["cap"], _p(tokens),
              tokens.shape[0], p0, _p(logits), _p(ws), ws.numel(), _stream(stream))

    def prefill_intermediates(self, ws, T):
        """The last layer's values after qg_prefill (qg_prefill_inspect)."""
        off = (ctypes.c_size_t * 12)()
        _call("qg_prefill_inspect", ctypes.byref(self.c_cfg), T, off)
        c = self.cfg
        HD, KD, h, F = c["heads"] * c["head_dim"], c["kv_heads"] * c["head_dim"], c["hidden"], c["ffn"]
        bf, f32 = torch.bfloat16, torch.float32
        spec = [("x", h, f32), ("xn", h, bf), ("q_proj", HD, f32), ("k_proj", KD, f32),
                ("v_proj", KD, f32), ("q_rope", HD, bf), ("att", HD, bf), ("x_attn", h, f32),
                ("xn2", h, bf), ("gate", F, f32), ("up", F, f32), ("h", F, bf)]
        out = {}
        for i, (name, n, dt) in enumerate(spec):
            size = 2 if dt == bf else 4
            out[name] = ws[off[i]:off[i] + size * T * n].view(dt).view(T, n)
        return out

    def qg_decode_step(self, state, tokens, positions, stream=None, layers=None):
        """tokens, positions: device int32 [B]. Writes state['logits'].
        ``layers`` runs only the first that many layers (then the head)."""
        cfg = self.c_cfg
        if layers is not None:
            cfg = qg_qwen3_config.from_buffer_copy(self.c_cfg)
            cfg.layers = layers
        _call("qg_decode_step", ctypes.byref(cfg), ctypes.byref(self.c_weights),
              _p(state["k_cache"]), _p(state["v_cache"]), state["cap"], _p(tokens),
              _p(positions), _p(state["logits"]), state["B"], _p(state["ws"]),
              state["ws"].numel(), _stream(stream))


class CodePredictor:
    """Device-resident packed code-predictor weights (the host dict layout of
    ``qg_synth.code_predictor_weights``) and ``qg_code_predict``."""

    def __init__(self, cfg: dict, weights: dict, device="cuda"):
        self.cfg = dict(cfg)
        self._keep = []

        def up(a):
            t = torch.from_numpy(a.view({2: "int16", 4: "int32"}[a.dtype.itemsize])).to(device)
            self._keep.append(t)
            return t.data_ptr()

        def mat(triple):
            w, s, b = triple
            return qg_affine8_matrix(up(w), up(s), up(b))

        self.c_cfg = qg_qwen3_config(cfg["hidden"], cfg["layers"], cfg["heads"], cfg["kv_heads"],
                                     cfg["head_dim"], cfg["ffn"], cfg["vocab"], cfg["eps"],
                                     cfg["theta"])
        G = len(weights["heads"])
        self.groups = G
        self.c_embed = (qg_affine8_matrix * G)(*[mat(t) for t in weights["code_embed"]])
        self.c_heads = (qg_affine8_matrix * G)(*[mat(t) for t in weights["heads"]])
        L = cfg["layers"]
        self.c_layers = (qg_qwen3_layer * max(L, 1))()
        for i, lw in enumerate(weights["layers"]):
            cl = self.c_layers[i]
            cl.input_norm = up(lw["input_norm"])
            cl.post_norm = up(lw["post_norm"])
            cl.q_norm = up(lw["q_norm"])
            cl.k_norm = up(lw["k_norm"])
            for n in ("q", "k", "v", "o", "gate", "up", "down"):
                setattr(cl, n, mat(lw[n]))
        self.c_weights = qg_code_predictor_weights(
            mat(weights["input_proj"]), ctypes.cast(self.c_embed, ctypes.POINTER(qg_affine8_matrix)),
            ctypes.cast(self.c_heads, ctypes.POINTER(qg_affine8_matrix)),
            ctypes.cast(self.c_layers, ctypes.POINTER(qg_qwen3_layer)), up(weights["final_norm"]), G)
        self.device = device

    def workspace(self, B):
        n = int(lib.qg_code_predict_workspace_size(ctypes.byref(self.c_cfg), B))
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def qg_code_predict(self, lm_hidden, code0, codes, ws, logits=None, stream=None):
        """lm_hidden fp32 [B, hidden], code0 int32 [B] (device) -> codes int32
        [groups, B]; logits fp32 [groups, B, vocab] when given."""
        B = lm_hidden.shape[0]
        _call("qg_code_predict", ctypes.byref(self.c_cfg), ctypes.byref(self.c_weights),
              _p(lm_hidden), _p(code0), _p(codes), _p(logits), B, _p(ws),
              ws.numel(), _stream(stream))

    def trace_layout(self, B):
        """(total bytes, bytes per group, offset of slot 0 in a group, bytes
        per slot) of the trace of ``qg_code_predict_traced``."""
        out = (ctypes.c_size_t * 4)()
        _call("qg_code_predict_trace_layout", ctypes.byref(self.c_cfg), B, self.groups, out)
        return tuple(int(v) for v in out)

    def step_offsets(self, B):
        """Offsets of the step buffers inside a trace slot (the workspace
        head, cap 1): ``qg_decode_step_inspect`` and ``_inspect_f32``."""
        off = (ctypes.c_size_t * 4)()
        _call("qg_decode_step_inspect", ctypes.byref(self.c_cfg), B, 1, off)
        off32 = (ctypes.c_size_t * 6)()
        _call("qg_decode_step_inspect_f32", ctypes.byref(self.c_cfg), B, 1, off32)
        return list(off), list(off32)

    def qg_code_predict_traced(self, lm_hidden, code0, codes, ws, trace, logits=None,
                               stream=None):
        """qg_code_predict that also fills ``trace`` (uint8, trace_layout()[0]
        bytes) with every group's layer values."""
        B = lm_hidden.shape[0]
        _call("qg_code_predict_traced", ctypes.byref(self.c_cfg), ctypes.byref(self.c_weights),
              _p(lm_hidden), _p(code0), _p(codes), _p(logits), B, _p(ws), ws.numel(),
              _p(trace), trace.numel(), _stream(stream))


class WhisperEncoderLayer:
    """Device-resident weights of one Whisper encoder layer (the host dict of
    ``qg_synth.whisper_layer_weights``) and ``qg_whisper_encoder_layer``."""

    NAMES = ("ln1_g", "ln1_b", "q", "q_b", "k", "v", "v_b", "o", "o_b", "ln2_g", "ln2_b", "fc1",
             "fc1_b", "fc2", "fc2_b")

    def __init__(self, cfg: dict, weights: dict, device="cuda"):
        self.cfg = dict(cfg)
        self._keep = {}
        for n in self.NAMES:
            a = weights[n]
            t = torch.from_numpy(a if a.dtype == "uint8" else a.astype("float32")).to(device)
            self._keep[n] = t
        self.c_cfg = qg_whisper_config(cfg["d_model"], cfg["heads"], cfg["ffn"], cfg["eps"])
        self.c_w = qg_whisper_layer(*[self._keep[n].data_ptr() for n in self.NAMES])
        self.device = device

    def tensor(self, name):
        return self._keep[name]

    def workspace(self, M):
        n = int(lib.qg_whisper_encoder_layer_workspace_size(ctypes.byref(self.c_cfg), M))
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def qg_whisper_encoder_layer(self, x, ws, stream=None):
        """x fp32 [M, d_model] in place."""
        _call("qg_whisper_encoder_layer", ctypes.byref(self.c_cfg), ctypes.byref(self.c_w), _p(x),
              x.shape[0], _p(ws), ws.numel(), _stream(stream))

    def intermediates(self, ws, M):
        """Views into the workspace after a call: bf16 ``xl``, ``q``, ``k``,
        ``v``, ``ctx``, ``xl2`` [M, d], ``mid`` [M, ffn]; fp32 ``xa`` [M, d];
        and the six matmuls' error words (``err``, int32)."""
        off = (ctypes.c_size_t * 9)()
        _call("qg_whisper_encoder_layer_inspect", ctypes.byref(self.c_cfg), M, off)
        d, F = self.cfg["d_model"], self.cfg["ffn"]

        def view(o, n, dt=torch.bfloat16):
            size = 2 if dt == torch.bfloat16 else 4
            return ws[o:o + size * M * n].view(dt).view(M, n)
        out = {name: view(off[i], d) for i, name in enumerate(("xl", "q", "k", "v", "ctx"))}
        out["xa"] = view(off[5], d, torch.float32)
        out["xl2"] = view(off[6], d)
        out["mid"] = view(off[7], F)
        out["err"] = ws[off[8]:off[8] + 6 * 256].view(torch.int32).view(6, 64)[:, 0]
        return out
