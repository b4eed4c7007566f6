"""Python binding of the C ABI in ``include/moe_gb300.h``.

Argument marshalling only: every function takes torch tensors (device memory from
PyTorch), checks dtype / shape / device, and passes raw pointers plus the current CUDA
stream to the library of the same name.  All arithmetic runs in the CUDA kernels of
``libmoe_gb300.so``; there is no other implementation behind these calls, and the
library must be built (``deepseek_moe_layer_gb300.build``) before use.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

MOE_OK, MOE_ERR_INVALID, MOE_ERR_CUDA, MOE_ERR_TIMEOUT, MOE_ERR_NODEVICE = 0, -1, -2, -3, -4
MOE_DTYPE_F32, MOE_DTYPE_BF16 = 0, 1

# Every symbol the public header declares.
EXPORTS = ("moe_last_error", "moe_version", "moe_device_status", "moe_route_deepseek",
           "moe_permute", "moe_router_logits", "moe_grouped_swiglu",
           "moe_grouped_swiglu_workspace_bytes", "moe_combine", "moe_forward",
           "moe_forward_workspace_bytes", "moe_set_phase_events", "moe_forward_noalloc",
           "moe_route_softmax", "moe_shared_gate", "moe_combine_gated", "moe_forward_ex",
           "moe_forward_ex_workspace_bytes", "moe_watchdog_selftest", "moe_indexer_topk",
           "moe_set_fault", "moe_get_fault", "moe_route_softmax_grouped", "moe_quantize_blocks",
           "moe_matmul_blocks", "moe_cache_append", "moe_indexer_scores",
           "moe_latent_attention", "moe_latent_attention_workspace_bytes")
MOE_ROUTE_DEEPSEEK, MOE_ROUTE_SOFTMAX, MOE_ROUTE_SOFTMAX_GROUPED = 0, 1, 2
MOE_BITS_E4M3 = 0x108  # expert weights: e4m3 codes with an fp32 scale per 128 x 128 block


class MoeError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"{msg} (code {code})")
        self.code = code


class RouteParams(ctypes.Structure):
    _fields_ = [("top_k", ctypes.c_int32), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("norm_topk_prob", ctypes.c_int32),
                ("routed_scaling_factor", ctypes.c_float)]


class ExpertWeights(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("group_size", ctypes.c_int32),
                ("gate", ctypes.c_void_p), ("up", ctypes.c_void_p), ("down", ctypes.c_void_p),
                ("gate_scale", ctypes.c_void_p), ("gate_bias", ctypes.c_void_p),
                ("up_scale", ctypes.c_void_p), ("up_bias", ctypes.c_void_p),
                ("down_scale", ctypes.c_void_p), ("down_bias", ctypes.c_void_p)]


class LayerArgs(ctypes.Structure):
    _fields_ = [("route_kind", ctypes.c_int32), ("x", ctypes.c_void_p), ("T", ctypes.c_int64),
                ("d", ctypes.c_int32), ("I", ctypes.c_int32), ("E", ctypes.c_int32),
                ("w_router", ctypes.c_void_p), ("logit_offset", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("params", RouteParams),
                ("experts", ctypes.POINTER(ExpertWeights)),
                ("shared", ctypes.POINTER(ExpertWeights)), ("w_shared_gate", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("inds_out", ctypes.c_void_p),
                ("scores_out", ctypes.c_void_p), ("logits_out", ctypes.c_void_p)]


class AppendArgs(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("T", ctypes.c_int64), ("ldx", ctypes.c_int64),
                ("W", ctypes.c_int32), ("slots", ctypes.c_void_p), ("cache", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("norm_weight", ctypes.c_void_p), ("norm_bias", ctypes.c_void_p),
                ("norm_cols", ctypes.c_int32), ("eps", ctypes.c_float),
                ("positions", ctypes.c_void_p), ("inv_freq", ctypes.c_void_p),
                ("rope_cols", ctypes.c_int32), ("rope_at", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("q", ctypes.c_void_p),
                ("q_out", ctypes.c_void_p), ("H", ctypes.c_int32), ("q_token", ctypes.c_int64),
                ("q_head", ctypes.c_int64), ("q_out_token", ctypes.c_int64),
                ("q_out_head", ctypes.c_int64)]


class PagedCache(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_void_p), ("pages", ctypes.c_int64), ("page", ctypes.c_int32),
                ("table", ctypes.c_void_p), ("sequences", ctypes.c_int32),
                ("width", ctypes.c_int32)]


_lock = threading.Lock()
_lib = None


def lib(path: str | None = None):
    """The loaded CUDA library (built on first use if the sources are newer)."""
    global _lib
    with _lock:
        if _lib is None:
            so = path or _build.build()
            if not os.path.exists(so):
                raise MoeError(MOE_ERR_NODEVICE, f"CUDA library missing: {so}")
            L = ctypes.CDLL(so)
            P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
            L.moe_last_error.restype = ctypes.c_char_p
            L.moe_version.restype = i32
            L.moe_device_status.argtypes = [i32, P]
            L.moe_route_deepseek.argtypes = [P, ctypes.c_int, i64, i32, P,
                                             ctypes.POINTER(RouteParams), P, P, P]
            L.moe_permute.argtypes = [P, i64, i32, i32, P, P, P, P, P]
            L.moe_router_logits.argtypes = [P, i64, i32, P, i32, P, P, P]
            L.moe_grouped_swiglu.argtypes = [P, i64, i32, i32, i32, i32, P, P,
                                             ctypes.POINTER(ExpertWeights),
                                             ctypes.POINTER(ExpertWeights), P, P, sz, P]
            L.moe_grouped_swiglu_workspace_bytes.argtypes = [i64, i32, i32, i32, i32, i32]
            L.moe_grouped_swiglu_workspace_bytes.restype = sz
            L.moe_combine.argtypes = [P, P, P, P, i64, i32, i32, P, P]
            L.moe_forward.argtypes = [P, i64, i32, i32, i32, P, P, P,
                                      ctypes.POINTER(RouteParams), ctypes.POINTER(ExpertWeights),
                                      ctypes.POINTER(ExpertWeights), P, P, P, P, P, sz, P]
            L.moe_forward_workspace_bytes.argtypes = [i64, i32, i32, i32, i32, i32]
            L.moe_forward_workspace_bytes.restype = sz
            L.moe_set_phase_events.argtypes = [ctypes.POINTER(ctypes.c_void_p), i32]
            L.moe_forward_noalloc.argtypes = [P, i64, i32, i32, i32, P, P, P,
                                              ctypes.POINTER(RouteParams),
                                              ctypes.POINTER(ExpertWeights),
                                              ctypes.POINTER(ExpertWeights), P, P, P, P, P]
            L.moe_route_softmax.argtypes = [P, ctypes.c_int, i64, i32, i32, P, P, P]
            L.moe_shared_gate.argtypes = [P, i64, i32, P, P, P]
            L.moe_combine_gated.argtypes = [P, P, P, P, P, i64, i32, i32, P, P]
            L.moe_forward_ex.argtypes = [ctypes.POINTER(LayerArgs), P, sz, P]
            L.moe_forward_ex_workspace_bytes.argtypes = [ctypes.POINTER(LayerArgs)]
            L.moe_forward_ex_workspace_bytes.restype = sz
            L.moe_watchdog_selftest.argtypes = [i64, P]
            L.moe_indexer_topk.argtypes = [P, ctypes.c_int, i64, i32, i64, P, i32, P, P, i64, P]
            L.moe_set_fault.argtypes = [i32, i32]
            L.moe_route_softmax_grouped.argtypes = [P, ctypes.c_int, i64, i32, P,
                                                    ctypes.POINTER(RouteParams), P, P, P]
            L.moe_quantize_blocks.argtypes = [P, ctypes.c_int, i64, i32, i64, i32, P, P, P]
            L.moe_matmul_blocks.argtypes = [P, P, i64, i64, P, P, i32, i32, ctypes.c_int, P, P]
            L.moe_cache_append.argtypes = [ctypes.POINTER(AppendArgs), P]
            L.moe_indexer_scores.argtypes = [P, P, i64, i32, ctypes.POINTER(PagedCache), P, P, P,
                                             i32, P, i64, P]
            L.moe_latent_attention.argtypes = [P, i64, i32, i64, i64, ctypes.POINTER(PagedCache), P,
                                               P, ctypes.c_float, P, i32, P, P, P, sz, P]
            L.moe_latent_attention_workspace_bytes.argtypes = [i64, i64]
            L.moe_latent_attention_workspace_bytes.restype = sz
            L.moe_get_fault.argtypes = [ctypes.POINTER(i32), ctypes.POINTER(i32)]
            for name in ("moe_device_status", "moe_route_deepseek", "moe_permute",
                         "moe_router_logits", "moe_grouped_swiglu", "moe_combine",
                         "moe_forward", "moe_set_phase_events", "moe_forward_noalloc",
                         "moe_route_softmax", "moe_shared_gate", "moe_combine_gated",
                         "moe_forward_ex", "moe_watchdog_selftest", "moe_indexer_topk",
                         "moe_set_fault", "moe_get_fault", "moe_route_softmax_grouped",
                         "moe_quantize_blocks", "moe_matmul_blocks", "moe_cache_append",
                         "moe_indexer_scores", "moe_latent_attention"):
                getattr(L, name).restype = ctypes.c_int
            _lib = L
    return _lib


def _check(rc):
    if rc != MOE_OK:
        raise MoeError(rc, lib().moe_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _raw_stream(t, stream):
    """cudaStream_t (an int) for a call on tensor t: `stream`, or the current one.  The library
    launches on the current device, so t has to be there."""
    if not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    dev = torch._C._cuda_getDevice()
    if t.get_device() != dev:
        raise ValueError(f"tensors are on {t.device}, but the current device is cuda:{dev}")
    # (the raw query: torch.cuda.current_stream() alone costs as much as the launch)
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev)


def _torch_stream(stream):
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(stream.cuda_stream)


def _empty(shape, dtype, device, stream, returned=True):
    """Memory that a call on `stream` writes.  It comes from that stream's pool: what the current
    one's pool hands out may still be in use there by work queued before.  A result that is
    `returned` is also marked as used by the caller's stream, so that its memory is not written
    again before what the caller does with it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    stream = _torch_stream(stream)
    if stream.device != device:
        return torch.empty(shape, dtype=dtype, device=device)
    caller = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned and caller != stream:
        t.record_stream(caller)
    return t


def _need(t, dtype, name, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _need_out(t, dtype, name, shape, device):
    _need(t, dtype, name, device)
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, not {tuple(t.shape)}")


def route_params(top_k, n_group, topk_group, norm_topk_prob, routed_scaling_factor):
    return RouteParams(int(top_k), int(n_group), int(topk_group), int(bool(norm_topk_prob)),
                       float(routed_scaling_factor))


def _is_scaled(w):
    return w is not None and int(w.get("bits", 16)) == MOE_BITS_E4M3


def expert_weights(w: dict | None, shape=None, device=None):
    """ExpertWeights from a dict: bits 16 -> gate/up/down bf16; bits 8 or 4 -> gate/up/down
    int32 (packed uint32 words) plus gate_s/gate_b/up_s/up_b/down_s/down_b fp16 and an
    optional 'group' (inputs per scale: 32, 64 or 128; default 64); bits MOE_BITS_E4M3 ->
    gate/up/down float8_e4m3fn plus gate_s/up_s/down_s fp32 [.., rows/128, inputs/128], which
    are held against shape (E, d, I) and device where given: gate, up [E, I, d], down [E, d, I]
    (E = 1: without it, too)."""
    if w is None:
        return None
    bits = int(w.get("bits", 16))
    if bits == 16:
        for k in ("gate", "up", "down"):
            _need(w[k], torch.bfloat16, k)
        return ExpertWeights(16, 0, w["gate"].data_ptr(), w["up"].data_ptr(), w["down"].data_ptr(),
                             None, None, None, None, None, None)
    if bits == MOE_BITS_E4M3:
        for k in ("gate", "up", "down"):
            q, sc = w[k], w[k + "_s"]
            _need(q, torch.float8_e4m3fn, k, device)
            _need(sc, torch.float32, k + "_s", q.device)
            if shape is not None:
                E, d, I = shape
                full = (E, d, I) if k == "down" else (E, I, d)
                if q.shape != full and not (E == 1 and q.shape == full[1:]):
                    raise ValueError(f"{k}: shape {tuple(q.shape)}, expected {full}")
            want = tuple(q.shape[:-2]) + (-(-q.shape[-2] // 128), -(-q.shape[-1] // 128))
            if tuple(sc.shape) != want:
                raise ValueError(f"{k}_s: shape {tuple(sc.shape)}, expected {want}")
        return ExpertWeights(MOE_BITS_E4M3, 128, w["gate"].data_ptr(), w["up"].data_ptr(),
                             w["down"].data_ptr(), w["gate_s"].data_ptr(), None,
                             w["up_s"].data_ptr(), None, w["down_s"].data_ptr(), None)
    for k in ("gate", "up", "down"):
        _need(w[k], torch.int32, k)
    for k in ("gate_s", "gate_b", "up_s", "up_b", "down_s", "down_b"):
        _need(w[k], torch.float16, k)
    if bits not in (4, 8):
        raise ValueError(f"bits = {bits}: expert weights are bf16 (16), affine 8 / 4-bit or "
                         "MOE_BITS_E4M3")
    return ExpertWeights(bits, int(w.get("group", 64)), w["gate"].data_ptr(), w["up"].data_ptr(),
                         w["down"].data_ptr(), w["gate_s"].data_ptr(), w["gate_b"].data_ptr(),
                         w["up_s"].data_ptr(), w["up_b"].data_ptr(), w["down_s"].data_ptr(),
                         w["down_b"].data_ptr())


def _ref(s):
    return None if s is None else ctypes.byref(s)


# ---------------------------------------------------------------------------------------
# the calls
# ---------------------------------------------------------------------------------------

def route_deepseek(logits, bias, top_k, n_group, topk_group, norm_topk_prob,
                   routed_scaling_factor, inds=None, scores=None, stream=None):
    """logits [..., E] fp32/bf16, bias [E] fp32 -> (inds int32 [..., K], scores fp32 [..., K])."""
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("logits must be fp32 or bf16")
    _need(logits, logits.dtype, "logits")
    if bias.dim() != 1 or bias.shape[0] != logits.shape[-1]:
        raise ValueError("bias must have rank 1 and length E (the last dim of logits)")
    _need(bias, torch.float32, "bias", logits.device)
    E = logits.shape[-1]
    rows = logits.numel() // E if E else 0
    shape = tuple(logits.shape[:-1]) + (int(top_k),)
    if inds is None:
        inds = _empty(shape, torch.int32, logits.device, stream)
    if scores is None:
        scores = _empty(shape, torch.float32, logits.device, stream)
    p = route_params(top_k, n_group, topk_group, norm_topk_prob, routed_scaling_factor)
    dt = MOE_DTYPE_F32 if logits.dtype == torch.float32 else MOE_DTYPE_BF16
    _check(lib().moe_route_deepseek(_ptr(logits), dt, rows, E, _ptr(bias), ctypes.byref(p),
                                    _ptr(inds), _ptr(scores), _stream(stream)))
    return inds, scores


def route_softmax(logits, top_k, inds=None, scores=None, stream=None):
    """Softmax route: logits [..., E] fp32/bf16 -> (inds int32, scores fp32) [..., K]."""
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("logits must be fp32 or bf16")
    _need(logits, logits.dtype, "logits")
    E = logits.shape[-1]
    rows = logits.numel() // E if E else 0
    shape = tuple(logits.shape[:-1]) + (int(top_k),)
    if inds is None:
        inds = _empty(shape, torch.int32, logits.device, stream)
    if scores is None:
        scores = _empty(shape, torch.float32, logits.device, stream)
    dt = MOE_DTYPE_F32 if logits.dtype == torch.float32 else MOE_DTYPE_BF16
    _check(lib().moe_route_softmax(_ptr(logits), dt, rows, E, int(top_k), _ptr(inds),
                                   _ptr(scores), _stream(stream)))
    return inds, scores


def route_softmax_grouped(logits, top_k, n_group, topk_group, norm_topk_prob,
                          routed_scaling_factor, bias=None, inds=None, scores=None, stream=None):
    """Group-limited softmax gate: probabilities over all experts, groups ranked by their best
    expert, weights renormalised only with norm_topk_prob; logits [..., E] fp32/bf16, bias [E]
    fp32 or None -> (inds int32, scores fp32) [..., K]."""
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("logits must be fp32 or bf16")
    if not logits.is_contiguous():
        raise ValueError("logits must be contiguous")
    E = logits.shape[-1]
    if bias is not None:
        if bias.dim() != 1 or bias.shape[0] != E:
            raise ValueError("bias must have rank 1 and length E (the last dim of logits)")
        _need(bias, torch.float32, "bias", logits.device)
    rows = logits.numel() // E if E else 0
    shape = (*logits.shape[:-1], int(top_k))
    if inds is None:
        inds = _empty(shape, torch.int32, logits.device, stream)
    else:
        _need_out(inds, torch.int32, "inds", shape, logits.device)
    if scores is None:
        scores = _empty(shape, torch.float32, logits.device, stream)
    else:
        _need_out(scores, torch.float32, "scores", shape, logits.device)
    p = route_params(top_k, n_group, topk_group, norm_topk_prob, routed_scaling_factor)
    dt = MOE_DTYPE_F32 if logits.dtype == torch.float32 else MOE_DTYPE_BF16
    _check((_lib or lib()).moe_route_softmax_grouped(
        logits.data_ptr(), dt, rows, E, None if bias is None else bias.data_ptr(),
        ctypes.byref(p), inds.data_ptr(), scores.data_ptr(), _raw_stream(logits, stream)))
    return inds, scores


def quantize_blocks(x, block_rows=1, codes=None, scales=None, stream=None):
    """x [rows, n] fp32/bf16 (rows may be strided) -> (codes float8_e4m3fn [rows, n], scales
    fp32 [ceil(rows/block_rows), ceil(n/128)]); block_rows 1 (activations) or 128 (weights)."""
    if x.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("x must be fp32 or bf16")
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError("x must be [rows, n] with unit stride along n")
    rows, n = x.shape
    if block_rows not in (1, 128):
        raise ValueError(f"block_rows = {block_rows} (1 or 128)")
    blocks = (-(-rows // block_rows), -(-n // 128))
    if codes is None:
        codes = _empty((rows, n), torch.float8_e4m3fn, x.device, stream)
    else:
        _need_out(codes, torch.float8_e4m3fn, "codes", (rows, n), x.device)
    if scales is None:
        scales = _empty(blocks, torch.float32, x.device, stream)
    else:
        _need_out(scales, torch.float32, "scales", blocks, x.device)
    _check((_lib or lib()).moe_quantize_blocks(
        x.data_ptr(), MOE_DTYPE_F32 if x.dtype == torch.float32 else MOE_DTYPE_BF16, rows, n,
        x.stride(0) if rows > 1 else n, block_rows, codes.data_ptr(), scales.data_ptr(),
        _raw_stream(x, stream)))
    return codes, scales


def matmul_blocks(a, a_scale, w, w_scale, out_dtype=torch.bfloat16, out=None, stream=None):
    """Block-scaled e4m3 product a w^T: a float8_e4m3fn [M, K] (rows may be strided), a_scale
    fp32 [M, ceil(K/128)], w float8_e4m3fn [N, K], w_scale fp32 [ceil(N/128), ceil(K/128)] ->
    bf16 or fp32 [M, N]."""
    if a.dtype != torch.float8_e4m3fn:
        raise TypeError(f"a: dtype {a.dtype}, expected {torch.float8_e4m3fn}")
    if a.dim() != 2 or (a.shape[1] > 1 and a.stride(1) != 1):
        raise ValueError("a must be [M, K] with unit stride along K")
    M, K = a.shape
    if w.dim() != 2 or w.shape[1] != K:
        raise ValueError(f"w must be [N, {K}]")
    N, kb, dev = w.shape[0], -(-K // 128), a.device
    _need(w, torch.float8_e4m3fn, "w", dev)
    _need_out(a_scale, torch.float32, "a_scale", (M, kb), dev)
    _need_out(w_scale, torch.float32, "w_scale", (-(-N // 128), kb), dev)
    if out is None:
        out = _empty((M, N), out_dtype, dev, stream)
    else:
        out_dtype = out.dtype
        _need_out(out, out_dtype, "out", (M, N), dev)
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("out must be fp32 or bf16")
    _check((_lib or lib()).moe_matmul_blocks(
        a.data_ptr(), a_scale.data_ptr(), M, a.stride(0) if M > 1 else K, w.data_ptr(),
        w_scale.data_ptr(), N, K, MOE_DTYPE_F32 if out_dtype == torch.float32 else MOE_DTYPE_BF16,
        out.data_ptr(), _raw_stream(a, stream)))
    return out


def shared_gate(x, w_gate, stream=None):
    """gate[t] = sigmoid(x[t] . w_gate): bf16 x [T, d], w_gate [d] -> fp32 [T]."""
    _need(x, torch.bfloat16, "x")
    _need(w_gate, torch.bfloat16, "w_gate", x.device)
    T, d = x.shape
    g = _empty(T, torch.float32, x.device, stream)
    _check(lib().moe_shared_gate(_ptr(x), T, d, _ptr(w_gate), _ptr(g), _stream(stream)))
    return g


def combine_gated(expert_out, scores, inv_perm, shared_out, gate, stream=None):
    """y[t] = sum_k scores[t,k] expert_out[inv_perm[t*K+k]] + gate[t] shared_out[t]."""
    _need(expert_out, torch.bfloat16, "expert_out")
    _need(scores, torch.float32, "scores")
    _need(inv_perm, torch.int32, "inv_perm")
    _need(gate, torch.float32, "gate")
    T, K = scores.shape
    d = expert_out.shape[1]
    y = _empty((T, d), torch.bfloat16, expert_out.device, stream)
    _check(lib().moe_combine_gated(_ptr(expert_out), _ptr(scores), _ptr(inv_perm),
                                   _ptr(shared_out), _ptr(gate), T, K, d, _ptr(y),
                                   _stream(stream)))
    return y


def indexer_topk(scores, k, lengths=None, want_mask=False, inds=None, mask=None,
                 stream=None):
    """DSA indexer selection: scores [rows, n] fp32/bf16 (rows may be strided: the row
    stride is taken from the tensor) -> int32 [rows, k] ascending positions padded with -1,
    and with want_mask also the uint8 [rows, n] selection mask."""
    if scores.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("scores must be fp32 or bf16")
    if scores.dim() != 2 or (scores.shape[1] > 1 and scores.stride(1) != 1):
        raise ValueError("scores must be [rows, n] with unit stride along n")
    rows, n = scores.shape
    ld = scores.stride(0) if rows > 1 else n
    if lengths is not None:
        _need(lengths, torch.int32, "lengths", scores.device)
        if lengths.shape != (rows,):
            raise ValueError("lengths must be [rows]")
    if inds is None:
        inds = _empty((rows, int(k)), torch.int32, scores.device, stream)
    if want_mask and mask is None:
        mask = _empty((rows, n), torch.uint8, scores.device, stream)
    dt = MOE_DTYPE_F32 if scores.dtype == torch.float32 else MOE_DTYPE_BF16
    _check(lib().moe_indexer_topk(_ptr(scores), dt, rows, n, ld, _ptr(lengths), int(k),
                                  _ptr(inds), _ptr(mask), n if mask is not None else 0,
                                  _stream(stream)))
    return (inds, mask) if want_mask else inds


def _fits(t, dtype, shape, dev):
    """Whether t is a contiguous tensor of this type, shape and device (an index; -1: the host).  The
    calls below ask this first and look for what is wrong only where it is not so: a check by
    check costs a call as much as its launch."""
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == dev and t.is_contiguous())


def _address(t):
    """The address of a tensor that a caller may leave out, never 0: the library takes NULL for "not
    given", and torch gives 0 as an empty tensor's address."""
    return t.data_ptr() or 256


def _too_large(*sizes):
    """Of sizes that do not fit an int32_t: ctypes cuts those down to their lowest 32 bits, silently."""
    return ValueError(f"sizes {sizes} do not fit 32 bits")


def _need_vector(t, dtype, name, n, device):
    _need(t, dtype, name, device)
    if t.shape != (n,):
        raise ValueError(f"{name} must be [{n}], not {tuple(t.shape)}")


def cache_append(x, slots, cache, scales=None, norm_weight=None, norm_bias=None, eps=1e-6,
                 positions=None, inv_freq=None, rope_at=0, interleaved=True, q=None, q_out=None,
                 stream=None):
    """Rows of new tokens into a paged cache: x bf16 [T, W] (rows may be strided) -> row slots[t]
    (int64 [T]; outside the cache: not written) of cache [pages, page, W], bf16, or float8_e4m3fn with
    fp32 scales [pages, page, W/128].  The first len(norm_weight) columns are normalised (fp32
    weight: RMS; with a bias: layer norm), 2 len(inv_freq) columns from rope_at on are rotated by
    positions (int32 [T]) * inv_freq (fp32), in pairs of neighbours (interleaved) or of halves.
    q bf16 [T, H, 2 len(inv_freq)] (tokens and heads may be strided) is rotated too, into q_out (a new
    tensor, or given: q itself, a slice of wider queries).  Returns cache, or (cache, q_out) with q."""
    if x.dtype is not torch.bfloat16:
        raise TypeError(f"x: dtype {x.dtype}, expected {torch.bfloat16}")
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError("x must be [T, W] with unit stride along W")
    T, W = x.shape
    dev = x.get_device()
    if not _fits(slots, torch.int64, (T,), dev):
        _need_vector(slots, torch.int64, "slots", T, x.device)
    if cache.dim() != 3 or cache.shape[2] != W:
        raise ValueError(f"cache must be [pages, page, {W}], not {tuple(cache.shape)}")
    pages, page, _ = cache.shape
    _need(cache, torch.bfloat16 if scales is None else torch.float8_e4m3fn, "cache", x.device)
    if scales is not None:
        if W % 128:
            raise ValueError(f"rows of an e4m3 cache must have a multiple of 128 columns, not {W}")
        _need_out(scales, torch.float32, "scales", (pages, page, W // 128), x.device)
    n = R = at = 0
    weight = bias = pos = freq = None
    if norm_weight is not None:
        n = norm_weight.numel()
        if not _fits(norm_weight, torch.float32, (n,), dev):
            _need_vector(norm_weight, torch.float32, "norm_weight", n, x.device)
        weight = norm_weight.data_ptr()
        if norm_bias is not None:
            if not _fits(norm_bias, torch.float32, (n,), dev):
                _need_vector(norm_bias, torch.float32, "norm_bias", n, x.device)
            bias = norm_bias.data_ptr()
    elif norm_bias is not None:
        raise ValueError("norm_bias given without norm_weight")
    if inv_freq is not None:
        half = inv_freq.numel()
        if not _fits(inv_freq, torch.float32, (half,), dev):
            _need_vector(inv_freq, torch.float32, "inv_freq", half, x.device)
        if positions is None:
            raise ValueError("inv_freq given without positions")
        if not _fits(positions, torch.int32, (T,), dev):
            _need_vector(positions, torch.int32, "positions", T, x.device)
        R, at, pos, freq = 2 * half, rope_at, positions.data_ptr(), inv_freq.data_ptr()
    H, src, dst, st = 0, None, None, (0, 0, 0, 0)
    if q is not None:
        if inv_freq is None:
            raise ValueError("q given without inv_freq")
        if q_out is None:
            q_out = _empty(q.shape, torch.bfloat16, x.device, stream)
        for t, name in ((q, "q"), (q_out, "q_out")):
            if t.dtype is not torch.bfloat16:
                raise TypeError(f"{name}: dtype {t.dtype}, expected {torch.bfloat16}")
            if t.dim() != 3 or t.shape != (T, q.shape[1], R) or t.stride(2) != 1:
                raise ValueError(f"{name} must be [{T}, H, {R}] with unit stride along its columns")
            if t.get_device() != dev:
                raise ValueError(f"{name} is on {t.device}, expected {x.device}")
        H, src, dst = q.shape[1], q.data_ptr(), q_out.data_ptr()
        # (the stride of an axis of one is arbitrary)
        (q0, q1, _), (o0, o1, _) = q.stride(), q_out.stride()
        st = (q0 if T > 1 else 0, q1 if H > 1 else 0, o0 if T > 1 else 0, o1 if H > 1 else 0)
    elif q_out is not None:
        raise ValueError("q_out given without q")
    if (W | n | R | H | (at if at >= 0 else ~at)) >> 31:
        raise _too_large(W, n, R, H, at)
    a = AppendArgs(x.data_ptr(), T, x.stride(0) if T > 1 else W, W, slots.data_ptr(),
                   cache.data_ptr(), None if scales is None else _address(scales), pages * page,
                   weight, bias, n, eps, pos, freq, R, at, int(bool(interleaved)), src, dst, H, *st)
    _check((_lib or lib()).moe_cache_append(ctypes.byref(a), _raw_stream(x, stream)))
    return cache if q is None else (cache, q_out)


def _paged_cache(rows, dtype, name, width, table, lengths, cu_tokens, T, device, dev):
    if rows.dim() != 3 or rows.shape[2] != width:
        raise ValueError(f"{name} must be [pages, page, {width}], not {tuple(rows.shape)}")
    pages, page, _ = rows.shape
    if not _fits(rows, dtype, (pages, page, width), dev):
        _need(rows, dtype, name, device)
    if table.dim() != 2:
        raise ValueError("block_table must be [sequences, pages]")
    B, wide = table.shape
    if not _fits(table, torch.int32, (B, wide), dev):
        _need(table, torch.int32, "block_table", device)
    if not _fits(lengths, torch.int32, (T,), dev):
        _need_vector(lengths, torch.int32, "lengths", T, device)
    if cu_tokens is not None:
        _need_vector(cu_tokens, torch.int32, "cu_tokens", B + 1, device)
    elif B != T:
        raise ValueError(f"block_table has {B} rows for {T} tokens, and cu_tokens is None")
    if (page | B | wide) >> 31:
        raise _too_large(page, B, wide)
    return PagedCache(rows.data_ptr(), pages, page, table.data_ptr(), B, wide)


def indexer_scores(q, weights, keys, block_table, lengths, n, key_scales=None, cu_tokens=None,
                   out=None, stream=None):
    """The indexer's scores of the cached positions: q [T, H, 128] and keys [pages, page, 128] bf16, or
    both float8_e4m3fn with fp32 key_scales [pages, page, 1] (or [pages, page]); weights fp32 [T, H];
    block_table int32 [B, pages of a sequence]; lengths int32 [T], the positions each token may see;
    cu_tokens int32 [B + 1], or None for one token per sequence -> fp32 [T, n] (rows of a given `out` may
    be strided), s_j sum_h weights[t, h] max(q[t, h] . k_j, 0) for j < lengths[t], -inf for the others."""
    dtype = torch.bfloat16 if key_scales is None else torch.float8_e4m3fn
    if q.dim() != 3 or q.shape[2] != 128:
        raise ValueError(f"q must be [T, H, 128], not {tuple(q.shape)}")
    T, H, _ = q.shape
    device, dev = q.device, q.get_device()
    if not _fits(q, dtype, (T, H, 128), dev):
        _need(q, dtype, "q")
    if not _fits(weights, torch.float32, (T, H), dev):
        _need_out(weights, torch.float32, "weights", (T, H), device)
    c = _paged_cache(keys, dtype, "keys", 128, block_table, lengths, cu_tokens, T, device, dev)
    if key_scales is not None:
        _need(key_scales, torch.float32, "key_scales", device)
        if key_scales.shape not in (keys.shape[:2], (*keys.shape[:2], 1)):
            raise ValueError(f"key_scales must be {(*keys.shape[:2], 1)}, not {tuple(key_scales.shape)}")
    n = int(n)
    if (n | H) >> 31:
        raise _too_large(n, H)
    if out is None:
        out = _empty((T, n), torch.float32, device, stream)
        ld = n
    else:
        if out.dtype is not torch.float32:
            raise TypeError(f"out: dtype {out.dtype}, expected {torch.float32}")
        if out.shape != (T, n) or (n > 1 and out.stride(1) != 1) or out.get_device() != dev:
            raise ValueError(f"out must be [{T}, {n}] on {device} with unit stride along its rows")
        ld = out.stride(0) if T > 1 else n
    _check((_lib or lib()).moe_indexer_scores(
        q.data_ptr(), weights.data_ptr(), T, H, ctypes.byref(c),
        None if key_scales is None else _address(key_scales),
        None if cu_tokens is None else cu_tokens.data_ptr(), lengths.data_ptr(), n, out.data_ptr(),
        ld, _raw_stream(q, stream)))
    return out


def latent_attention(q, cache, block_table, lengths, scale, inds=None, cu_tokens=None, out=None,
                     want_lse=False, ws=None, stream=None):
    """Attention over cached latent rows, absorbed form: q bf16 [T, H, 576] (tokens and heads may be
    strided), cache bf16 [pages, page, 576], block_table int32 [B, pages of a sequence], lengths int32 [T]
    (positions each token may see), cu_tokens int32 [B + 1] or None for one token per sequence, inds int32
    [T, k] (selected positions, as indexer_topk gives them) or None for all -> bf16 [T, H, 512], and
    with want_lse also the fp32 [T, H] log-sum-exp of the scaled scores."""
    if q.dtype is not torch.bfloat16:
        raise TypeError(f"q: dtype {q.dtype}, expected {torch.bfloat16}")
    if q.dim() != 3 or q.shape[2] != 576 or q.stride(2) != 1:
        raise ValueError(f"q must be [T, H, 576] with unit stride along its columns, not {tuple(q.shape)}")
    T, H, _ = q.shape
    device, dev = q.device, q.get_device()
    c = _paged_cache(cache, torch.bfloat16, "cache", 576, block_table, lengths, cu_tokens, T, device, dev)
    k, chosen = 0, None
    if inds is not None:
        if inds.dim() != 2 or inds.shape[0] != T:
            raise ValueError(f"inds must be [{T}, k], not {tuple(inds.shape)}")
        k, chosen = inds.shape[1], _address(inds) if T else None
    if (k | H) >> 31:
        raise _too_large(k, H)
    if inds is not None:
        _need(inds, torch.int32, "inds", device)
    if out is None:
        out = _empty((T, H, 512), torch.bfloat16, device, stream)
    else:
        _need_out(out, torch.bfloat16, "out", (T, H, 512), device)
    lse = _empty((T, H), torch.float32, device, stream) if want_lse else None
    L = _lib or lib()
    if ws is None:
        need = L.moe_latent_attention_workspace_bytes(T, k if inds is not None else c.width * c.page)
        ws = _empty((max(need, 256),), torch.uint8, device, stream, returned=False)
    else:
        _need(ws, torch.uint8, "ws", device)
    q0, q1, _ = q.stride()
    _check(L.moe_latent_attention(
        q.data_ptr(), T, H, q0 if T > 1 else 0, q1 if H > 1 else 0, ctypes.byref(c),
        None if cu_tokens is None else cu_tokens.data_ptr(), lengths.data_ptr(), scale, chosen, k,
        out.data_ptr(), None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.numel(),
        _raw_stream(q, stream)))
    return (out, lse) if want_lse else out


def permute(inds, E, stream=None):
    """inds int32 [T, K] -> (counts [E], offsets [E+1], perm [P], inv_perm [P]), int32."""
    _need(inds, torch.int32, "inds")
    T, K = inds.shape
    dev = inds.device
    counts = _empty(E, torch.int32, dev, stream)
    offsets = _empty(E + 1, torch.int32, dev, stream)
    perm = _empty(T * K, torch.int32, dev, stream)
    inv = _empty(T * K, torch.int32, dev, stream)
    _check(lib().moe_permute(_ptr(inds), T, K, E, _ptr(counts), _ptr(offsets), _ptr(perm),
                             _ptr(inv), _stream(stream)))
    return counts, offsets, perm, inv


def router_logits(x, w_router, logit_offset=None, stream=None):
    """x bf16 [T, d], w_router bf16 [E, d] -> fp32 logits [T, E]."""
    _need(x, torch.bfloat16, "x")
    _need(w_router, torch.bfloat16, "w_router", x.device)
    T, d = x.shape
    E = w_router.shape[0]
    if logit_offset is not None:
        _need(logit_offset, torch.float32, "logit_offset", x.device)
    out = _empty((T, E), torch.float32, x.device, stream)
    _check(lib().moe_router_logits(_ptr(x), T, d, _ptr(w_router), E, _ptr(logit_offset),
                                   _ptr(out), _stream(stream)))
    return out


def grouped_swiglu_workspace_bytes(T, d, I, E, K, has_shared):
    return lib().moe_grouped_swiglu_workspace_bytes(T, d, I, E, K, int(bool(has_shared)))


def grouped_swiglu(x, offsets, perm, K, experts, shared=None, I=None, ws=None, stream=None):
    """Expert SwiGLU over the dispatched tokens; returns bf16 [P (+T), d] in slot order."""
    _need(x, torch.bfloat16, "x")
    T, d = x.shape
    E = offsets.numel() - 1
    I = I if I is not None else (experts["gate"].shape[1])
    P = T * K
    if _is_scaled(experts):
        ew = expert_weights(experts, (E, d, I), x.device)
        sw = expert_weights(shared, (1, d, I), x.device)
        _need(offsets, torch.int32, "offsets", x.device)
        _need(perm, torch.int32, "perm", x.device)
        if perm.numel() < P:
            raise ValueError(f"perm holds {perm.numel()} pairs, not T * K = {P}")
        st = _raw_stream(x, stream)
    else:
        ew, sw = expert_weights(experts), expert_weights(shared)
        st = _stream(stream)
    out = _empty((P + (T if shared is not None else 0), d), torch.bfloat16, x.device, stream)
    need = grouped_swiglu_workspace_bytes(T, d, I, E, K, shared is not None)
    if ws is None:
        ws = _empty(max(need, 256), torch.uint8, x.device, stream, returned=False)
    _check(lib().moe_grouped_swiglu(_ptr(x), T, d, I, E, K, _ptr(offsets), _ptr(perm),
                                    ctypes.byref(ew), _ref(sw), _ptr(out), _ptr(ws),
                                    ws.numel(), st))
    return out


def combine(expert_out, scores, inv_perm, shared_out=None, stream=None):
    """y[t] = sum_k scores[t,k] expert_out[inv_perm[t*K+k]] (+ shared_out[t]), bf16 [T, d]."""
    _need(expert_out, torch.bfloat16, "expert_out")
    _need(scores, torch.float32, "scores")
    _need(inv_perm, torch.int32, "inv_perm")
    T, K = scores.shape
    d = expert_out.shape[1]
    y = _empty((T, d), torch.bfloat16, expert_out.device, stream)
    _check(lib().moe_combine(_ptr(expert_out), _ptr(scores), _ptr(inv_perm), _ptr(shared_out),
                             T, K, d, _ptr(y), _stream(stream)))
    return y


def forward_workspace_bytes(T, d, I, E, top_k, has_shared):
    return lib().moe_forward_workspace_bytes(T, d, I, E, top_k, int(bool(has_shared)))


class MoELayer:
    """The whole layer on device-resident weights: ``layer(x) -> y``.

    Holds the weights, the gate parameters and a reusable workspace; each call is one
    ``moe_forward`` on the current stream (or ``stream``).  Calls share the workspace: on several
    streams their caller has to order them.  With ``want_intermediates`` it also returns the
    selected experts, their weights and the router logits.
    """

    def __init__(self, w_router, bias, experts, shared, top_k, n_group, topk_group,
                 norm_topk_prob, routed_scaling_factor, logit_offset=None,
                 route_kind=MOE_ROUTE_DEEPSEEK, w_shared_gate=None):
        _need(w_router, torch.bfloat16, "w_router")
        self.dev = w_router.device
        if bias is not None:
            _need(bias, torch.float32, "bias", self.dev)
        if w_shared_gate is not None:
            _need(w_shared_gate, torch.bfloat16, "w_shared_gate", self.dev)
        self.route_kind, self.w_shared_gate = int(route_kind), w_shared_gate
        # the DeepSeek body goes through moe_forward, anything else through moe_forward_ex
        self.ex = self.route_kind != MOE_ROUTE_DEEPSEEK or w_shared_gate is not None
        self.w_router, self.bias, self.logit_offset = w_router, bias, logit_offset
        self.experts, self.shared = experts, shared
        self.E, self.d = w_router.shape
        grouped = self.route_kind == MOE_ROUTE_SOFTMAX_GROUPED
        if grouped and bias is not None and bias.shape != (self.E,):
            raise ValueError(f"bias must be [{self.E}], not {tuple(bias.shape)}")
        self.I = experts["gate"].shape[1]
        self.params = route_params(top_k, n_group, topk_group, norm_topk_prob,
                                   routed_scaling_factor)
        self.scaled = _is_scaled(experts)
        of = lambda E: ((E, self.d, self.I), self.dev) if self.scaled else ()  # noqa: E731
        self.ew, self.sw = expert_weights(experts, *of(self.E)), expert_weights(shared, *of(1))
        self.ws, self.ws_stream = None, None

    def _args(self, x, y, inds, scores, logits):
        a = LayerArgs()
        a.route_kind = self.route_kind
        a.x, a.T, a.d, a.I, a.E = x.data_ptr(), x.shape[0], self.d, self.I, self.E
        a.w_router = self.w_router.data_ptr()
        a.logit_offset = None if self.logit_offset is None else self.logit_offset.data_ptr()
        a.bias = None if self.bias is None else self.bias.data_ptr()
        a.params = self.params
        a.experts = ctypes.pointer(self.ew)
        a.shared = ctypes.pointer(self.sw) if self.sw is not None else None
        a.w_shared_gate = None if self.w_shared_gate is None else self.w_shared_gate.data_ptr()
        a.y = None if y is None else y.data_ptr()
        a.inds_out = None if inds is None else inds.data_ptr()
        a.scores_out = None if scores is None else scores.data_ptr()
        a.logits_out = None if logits is None else logits.data_ptr()
        return a

    def workspace(self, T, stream=None):
        if self.ex:
            a = LayerArgs()
            a.route_kind, a.T, a.d, a.I, a.E = self.route_kind, T, self.d, self.I, self.E
            a.params = self.params
            a.shared = ctypes.pointer(self.sw) if self.sw is not None else None
            a.w_shared_gate = None if self.w_shared_gate is None else 1
            need = lib().moe_forward_ex_workspace_bytes(ctypes.byref(a))
        else:
            need = forward_workspace_bytes(T, self.d, self.I, self.E, self.params.top_k,
                                           self.shared is not None)
        used = None
        if self.dev.type == "cuda":
            used = (stream.cuda_stream if stream is not None
                    else torch._C._cuda_getCurrentRawStream(self.dev.index))
        if self.ws is None or self.ws.numel() < need:
            self.ws = _empty(max(need, 256), torch.uint8, self.dev, stream, returned=False)
            self.ws_stream = used
        elif used != self.ws_stream:
            # the memory must outlive this call when a later one needs more
            self.ws.record_stream(_torch_stream(stream) or torch.cuda.current_stream(self.dev))
        return self.ws

    def __call__(self, x, y=None, want_intermediates=False, stream=None):
        _need(x, torch.bfloat16, "x", self.dev)
        T, d = x.shape
        K = self.params.top_k
        if self.scaled:
            if d != self.d:
                raise ValueError(f"x must be [T, {self.d}], not {tuple(x.shape)}")
            if y is not None:
                _need_out(y, torch.bfloat16, "y", (T, d), self.dev)
            st = _raw_stream(x, stream)
        else:
            st = _stream(stream)
        ws = self.workspace(T, stream)
        if y is None:
            y = _empty((T, d), torch.bfloat16, self.dev, stream)
        inds = scores = logits = None
        if want_intermediates:
            inds = _empty((T, K), torch.int32, self.dev, stream)
            scores = _empty((T, K), torch.float32, self.dev, stream)
            logits = _empty((T, self.E), torch.float32, self.dev, stream)
        if self.ex:
            a = self._args(x, y, inds, scores, logits)
            _check(lib().moe_forward_ex(ctypes.byref(a), _ptr(ws), ws.numel(), st))
            return (y, inds, scores, logits) if want_intermediates else y
        _check(lib().moe_forward(_ptr(x), T, d, self.I, self.E, _ptr(self.w_router),
                                 _ptr(self.bias), _ptr(self.logit_offset),
                                 ctypes.byref(self.params), ctypes.byref(self.ew), _ref(self.sw),
                                 _ptr(y), _ptr(inds), _ptr(scores), _ptr(logits), _ptr(ws),
                                 ws.numel(), st))
        if want_intermediates:
            return y, inds, scores, logits
        return y


PHASES = ("router", "route", "permute", "gather", "gate_up", "down", "combine")


def set_phase_events(events):
    """Record torch.cuda.Event objects (8: start + one after each of PHASES) inside the
    next moe_forward calls on their stream; None stops recording."""
    if not events:
        _check(lib().moe_set_phase_events(None, 0))
        return
    for e in events:
        if not e.cuda_event:  # torch creates the CUDA event at its first record
            e.record()
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _check(lib().moe_set_phase_events(arr, len(events)))


def device_status(clear=True, stream=None):
    """MOE_OK, or raises MoeError(MOE_ERR_TIMEOUT) if a kernel gave up a wait."""
    _check(lib().moe_device_status(int(bool(clear)), _stream(stream)))


def watchdog_selftest(limit_ns=20_000_000, stream=None):
    """Launches a wait that nothing completes, bounded by limit_ns; afterwards
    device_status() raises MoeError(MOE_ERR_TIMEOUT)."""
    _check(lib().moe_watchdog_selftest(int(limit_ns), _stream(stream)))


MOE_FAULT_NONE, MOE_FAULT_LAUNCH = 0, 1


def set_fault(kind=MOE_FAULT_NONE, at=0):
    """Test hook: with MOE_FAULT_LAUNCH the at-th kernel launch of every later call reports
    MOE_ERR_CUDA instead of launching; MOE_FAULT_NONE turns it off."""
    _check(lib().moe_set_fault(int(kind), int(at)))


def get_fault():
    """(kind, at) of the fault hook (MOE_FAULT in the environment sets the initial state)."""
    k, a = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().moe_get_fault(ctypes.byref(k), ctypes.byref(a)))
    return k.value, a.value
