"""Thin Python binding of libdcu (``include/dcu.h``): argument marshalling only.

Every step of the DCU path runs in the CUDA kernels of ``libdcu.so``; this
module converts torch tensors to device pointers and raises ``DcuError`` on a
non-zero return code.  It fails loudly when the library is missing: there is
no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdcu.so")

# ---- constants mirrored from include/dcu.h
DCU_OK, DCU_EINVAL, DCU_ENOMEM, DCU_ECUDA, DCU_ECAPACITY, DCU_ESTATE, DCU_EDEVICE = 0, -1, -2, -3, -4, -5, -6
DCU_ST_BAD_KEY, DCU_ST_BAD_TOKEN, DCU_ST_TIMEOUT = 1, 2, 4
DCU_ST_BAD_PAGE, DCU_ST_NO_PAGE, DCU_ST_BAD_ROW = 8, 16, 32
DCU_F32, DCU_BF16 = 0, 1
DCU_FRECHET, DCU_THRESHOLD, DCU_FACTOR, DCU_APD = 0, 1, 2, 3
DCU_WINDOW_INCLUSIVE, DCU_WINDOW_HALFOPEN = 0, 1
(DCU_T_H, DCU_T_K, DCU_T_V, DCU_T_D, DCU_T_S, DCU_T_S_PREV, DCU_T_BUDGET, DCU_T_SEL, DCU_T_SEL_COUNT,
 DCU_T_CONF, DCU_T_ARGMAX, DCU_T_ATTN, DCU_T_STALE, DCU_T_APD_TAU, DCU_T_APD_C, DCU_T_APD_H) = range(16)
DCU_SELECT_INPUT, DCU_SELECT_VALUE = 0, 1
DCU_OPT_FUSED_EPILOGUE, DCU_OPT_L2_PREFETCH, DCU_OPT_ATTENTION, DCU_OPT_GEMM_SMEM_KB = 1, 2, 3, 4
DCU_OPT_GEMM_PASS_SWEEP = 5
DCU_ATTN_TCGEN05, DCU_ATTN_MMA_SYNC = 0, 1
(DCU_K_REFRESH, DCU_K_BUDGET, DCU_K_SELECT, DCU_K_GATHER, DCU_K_GEMM, DCU_K_EPILOGUE, DCU_K_ATTN, DCU_K_SCATTER,
 DCU_K_LMHEAD, DCU_K_COMMIT, DCU_K_COUNT) = range(11)

_i32, _i64, _f32, _f64, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double, ctypes.c_void_p


class dcu_cfg(ctypes.Structure):
    _fields_ = [("n_layers", _i32), ("d_model", _i32), ("n_heads", _i32), ("n_kv_heads", _i32),
                ("head_dim", _i32), ("d_ffn", _i32), ("vocab", _i32), ("mask_id", _i32),
                ("max_batch", _i32), ("max_seq", _i32), ("dtype", _i32), ("rms_eps", _f32),
                ("rope_theta", _f32), ("window_mode", _i32)]


class dcu_pages(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("page_stride", _i64), ("slot_stride", _i64), ("head_stride", _i64),
                ("n_pages", _i32), ("page_size", _i32), ("n_kv_heads", _i32), ("head_dim", _i32), ("dtype", _i32)]


_PP = ctypes.POINTER(_vp)


class dcu_weights(ctypes.Structure):
    _fields_ = [("embed", _vp), ("final_norm", _vp), ("lm_head", _vp),
                ("attn_norm", _PP), ("wq", _PP), ("wk", _PP), ("wv", _PP), ("wo", _PP),
                ("ffn_norm", _PP), ("w_gate", _PP), ("w_up", _PP), ("w_down", _PP)]


class DcuError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libdcu error {code}: {msg}")
        self.code = code


_LIB = None

# name -> (restype, argtypes)
_SIGS = {
    "dcu_create": (_i32, [ctypes.POINTER(dcu_weights), ctypes.POINTER(dcu_cfg), ctypes.POINTER(_vp)]),
    "dcu_destroy": (None, [_vp]),
    "dcu_last_error": (ctypes.c_char_p, [_vp]),
    "dcu_full_forward": (_i32, [_vp, _vp, _i32, _i32, _vp]),
    "dcu_step": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _vp]),
    "commit_select": (_i32, [_vp, _i32, _f32, _vp, _vp, _vp, _vp, _vp]),
    "commit_select_block": (_i32, [_vp, _i32, _f32, _i32, _i32, _vp, _vp, _vp, _vp, _vp]),
    "dcu_status": (_i32, [_vp, _vp, ctypes.POINTER(_i32)]),
    "dcu_budget_split": (_i32, [_vp, _i32, _i32, _i32, _i32, _vp, _vp]),
    "dcu_select_tokens": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp]),
    "dcu_cosine_distance": (_i32, [_vp, _vp, _vp, _i64, _i32, _i32, _vp, _vp]),
    "dcu_commit_rule": (_i32, [_i32, _f32, _vp, _vp, _vp, _vp, _i32, _i32, _vp, _vp, _vp]),
    "dcu_commit_rule_block": (_i32, [_i32, _f32, _i32, _i32, _vp, _vp, _vp, _vp, _i32, _i32, _vp, _vp, _vp]),
    "dcu_selftest_wait_timeout": (_i32, [_vp, _vp]),
    "dcu_tensor_bytes": (_i32, [_vp, _i32, ctypes.POINTER(_i64)]),
    "dcu_get_tensor": (_i32, [_vp, _i32, _i32, _vp, _i64, _vp]),
    "dcu_set_tensor": (_i32, [_vp, _i32, _i32, _vp, _i64, _vp]),
    "dcu_profile_enable": (_i32, [_vp, _i32]),
    "dcu_profile_read": (_i32, [_vp, _i32, ctypes.POINTER(_f64), ctypes.POINTER(_i64), _i32]),
    "dcu_kernel_class_name": (ctypes.c_char_p, [_i32]),
    "dcu_launch_count": (_i64, [_vp]),
    "dcu_set_graphs": (_i32, [_vp, _i32]),
    "dcu_set_refresh": (_i32, [_vp, _i32, _i32, _i32]),
    "dcu_set_select_from": (_i32, [_vp, _i32]),
    "dcu_set_option": (_i32, [_vp, _i32, _i32]),
    "dcu_set_apd": (_i32, [_vp, _f32, _f32, _f32]),
    "dcu_linear": (_i32, [_vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp]),
    "dcu_page_table": (_i32, [_vp, _i32, _i32, _i32, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp]),
    "dcu_slot_map": (_i32, [_vp, _i32, _i32, _i32, _i32, _vp, _vp, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _vp]),
    "dcu_rope_table": (_i32, [_vp, _i32, _i32, _f32, _vp]),
    "dcu_paged_write": (_i32, [_vp, _i32, _vp, _vp, _vp, _vp, _i32, _i32, ctypes.POINTER(dcu_pages), _vp, _vp, _vp]),
    "dcu_paged_attention": (_i32, [_vp, _i32, _vp, _i32, _vp, _vp, _i32, _i32, ctypes.POINTER(dcu_pages), _f32, _vp,
                                   _vp, _i64, _vp, _vp]),
    "dcu_paged_attention_workspace": (_i32, [ctypes.POINTER(dcu_pages), ctypes.POINTER(_i64)]),
    "dcu_lm_confidence_noalloc": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _f32, _vp, _vp, _vp]),
}


def lib():
    """Loads libdcu.so (raises if it is not built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run `python -m dynamic_layer_wise_b200.build` "
                               "(the DCU path has no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


def _err(handle) -> str:
    m = lib().dcu_last_error(handle)
    return m.decode() if m else ""


def _check(rc: int, handle=None):
    if rc != DCU_OK:
        raise DcuError(rc, _err(handle))


def _ptr(t) -> _vp:
    if t is None:
        return _vp(0)
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return _vp(t.data_ptr())


def _stream(stream) -> _vp:
    if stream is None:
        return _vp(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return _vp(stream.cuda_stream)
    return _vp(int(stream))


_LAYER_KEYS = ("attn_norm", "wq", "wk", "wv", "wo", "ffn_norm", "w_gate", "w_up", "w_down")


class Context:
    """Owns a dcu_ctx handle and keeps the weight tensors it points to alive."""

    def __init__(self, handle, weights, arrays, cfg: dict):
        self.handle = handle
        self._weights = weights
        self._arrays = arrays
        self.cfg = dict(cfg)

    def close(self):
        if self.handle:
            lib().dcu_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def dcu_create(weights: dict, cfg: dict) -> Context:
    """weights: {'embed', 'final_norm', 'lm_head', 'layers': [ {attn_norm, wq, ...}, ... ]} of CUDA
    tensors; cfg: the fields of dcu_cfg (dtype as 'bf16' | 'f32' or DCU_*)."""
    c = dict(cfg)
    if isinstance(c.get("dtype"), str):
        c["dtype"] = {"bf16": DCU_BF16, "f32": DCU_F32}[c["dtype"]]
    c.setdefault("mask_id", c["vocab"] - 1)
    c.setdefault("rms_eps", 1e-5)
    c.setdefault("rope_theta", 10000.0)
    c.setdefault("window_mode", DCU_WINDOW_INCLUSIVE)
    cs = dcu_cfg(**{k: c[k] for k, _ in dcu_cfg._fields_})
    L = c["n_layers"]
    layers = weights["layers"]
    if len(layers) != L:
        raise ValueError("weights['layers'] must have n_layers entries")
    arrays = {}
    for k in _LAYER_KEYS:
        arr = (_vp * L)(*[_ptr(layers[l][k]).value for l in range(L)])
        arrays[k] = arr
    w = dcu_weights(_ptr(weights["embed"]), _ptr(weights["final_norm"]), _ptr(weights["lm_head"]),
                    *[ctypes.cast(arrays[k], _PP) for k in _LAYER_KEYS])
    h = _vp(0)
    rc = lib().dcu_create(ctypes.byref(w), ctypes.byref(cs), ctypes.byref(h))
    _check(rc, None)
    return Context(h, weights, arrays, c)


def dcu_full_forward(ctx: Context, token_ids, stream=None):
    B, N = token_ids.shape
    assert token_ids.dtype == torch.int32
    _check(lib().dcu_full_forward(ctx.handle, _ptr(token_ids), B, N, _stream(stream)), ctx.handle)


def dcu_step(ctx: Context, token_ids, key_positions, n_keys, B_layer: int, B_window: int, stream=None):
    for t in (token_ids, key_positions, n_keys):
        assert t.dtype == torch.int32
    _check(lib().dcu_step(ctx.handle, _ptr(token_ids), _ptr(key_positions), _ptr(n_keys), int(B_layer),
                          int(B_window), _stream(stream)), ctx.handle)


def commit_select(ctx: Context, rule: int, param: float, masked, token_ids, out_positions, out_count, stream=None):
    assert masked.dtype == torch.uint8 and token_ids.dtype == torch.int32
    assert out_positions.dtype == torch.int32 and out_count.dtype == torch.int32
    _check(lib().commit_select(ctx.handle, int(rule), float(param), _ptr(masked), _ptr(token_ids),
                               _ptr(out_positions), _ptr(out_count), _stream(stream)), ctx.handle)


def commit_select_block(ctx: Context, rule: int, param: float, gen_start: int, block_len: int, masked, token_ids,
                        out_positions, out_count, stream=None):
    assert masked.dtype == torch.uint8 and token_ids.dtype == torch.int32
    assert out_positions.dtype == torch.int32 and out_count.dtype == torch.int32
    _check(lib().commit_select_block(ctx.handle, int(rule), float(param), int(gen_start), int(block_len),
                                     _ptr(masked), _ptr(token_ids), _ptr(out_positions), _ptr(out_count),
                                     _stream(stream)), ctx.handle)


def dcu_status(ctx: Context, stream=None) -> int:
    bits = _i32(0)
    rc = lib().dcu_status(ctx.handle, _stream(stream), ctypes.byref(bits))
    if rc not in (DCU_OK, DCU_EDEVICE):
        _check(rc, ctx.handle)
    return int(bits.value)


def dcu_budget_split(s_prev, B_layer: int, uniform: bool, budgets=None, stream=None):
    B, L = s_prev.shape
    if budgets is None:
        budgets = torch.empty((B, L), dtype=torch.int32, device=s_prev.device)
    _check(lib().dcu_budget_split(_ptr(s_prev), B, L, int(B_layer), int(bool(uniform)), _ptr(budgets),
                                  _stream(stream)))
    return budgets


def dcu_select_tokens(d, key_positions, n_keys, budgets, B_window: int, window_mode: int = 0, status=None,
                      stream=None):
    B, N = d.shape
    idx = torch.empty((B, N), dtype=torch.int32, device=d.device)
    count = torch.empty((B,), dtype=torch.int32, device=d.device)
    s = torch.empty((B,), dtype=torch.float32, device=d.device)
    _check(lib().dcu_select_tokens(_ptr(d), _ptr(key_positions), _ptr(n_keys), _ptr(budgets), B, N, int(B_window),
                                   int(window_mode), _ptr(idx), _ptr(count), _ptr(s), _ptr(status),
                                   _stream(stream)))
    return idx, count, s


def dcu_cosine_distance(x, y, gain, stream=None):
    rows, D = x.shape
    dt = {torch.bfloat16: DCU_BF16, torch.float32: DCU_F32}[x.dtype]
    d = torch.empty((rows,), dtype=torch.float32, device=x.device)
    _check(lib().dcu_cosine_distance(_ptr(x), _ptr(y), _ptr(gain), rows, D, dt, _ptr(d), _stream(stream)))
    return d


def dcu_commit_rule(rule: int, param: float, conf, argmax, masked, token_ids, out_positions, out_count, stream=None):
    B, N = conf.shape
    _check(lib().dcu_commit_rule(int(rule), float(param), _ptr(conf), _ptr(argmax), _ptr(masked), _ptr(token_ids),
                                 B, N, _ptr(out_positions), _ptr(out_count), _stream(stream)))


def dcu_commit_rule_block(rule: int, param: float, gen_start: int, block_len: int, conf, argmax, masked, token_ids,
                          out_positions, out_count, stream=None):
    B, N = conf.shape
    _check(lib().dcu_commit_rule_block(int(rule), float(param), int(gen_start), int(block_len), _ptr(conf),
                                       _ptr(argmax), _ptr(masked), _ptr(token_ids), B, N, _ptr(out_positions),
                                       _ptr(out_count), _stream(stream)))


def dcu_selftest_wait_timeout(status, stream=None):
    """One bounded device wait that must expire: sets DCU_ST_TIMEOUT in status."""
    assert status.dtype == torch.int32
    _check(lib().dcu_selftest_wait_timeout(_ptr(status), _stream(stream)))


_KIND_DTYPE = {DCU_T_D: torch.float32, DCU_T_S: torch.float32, DCU_T_S_PREV: torch.float32,
               DCU_T_BUDGET: torch.int32, DCU_T_SEL: torch.int32, DCU_T_SEL_COUNT: torch.int32,
               DCU_T_CONF: torch.float32, DCU_T_ARGMAX: torch.int32, DCU_T_STALE: torch.uint8,
               DCU_T_APD_TAU: torch.float32, DCU_T_APD_C: torch.float32, DCU_T_APD_H: torch.float32}


def _kind_dtype(ctx: Context, kind: int):
    if kind in (DCU_T_H, DCU_T_K, DCU_T_V, DCU_T_ATTN):
        return torch.bfloat16 if ctx.cfg["dtype"] == DCU_BF16 else torch.float32
    return _KIND_DTYPE[kind]


def dcu_get_tensor(ctx: Context, kind: int, layer: int = 0, stream=None):
    n = _i64(0)
    _check(lib().dcu_tensor_bytes(ctx.handle, kind, ctypes.byref(n)), ctx.handle)
    dt = _kind_dtype(ctx, kind)
    out = torch.empty(n.value // torch.tensor([], dtype=dt).element_size(), dtype=dt, device="cuda")
    _check(lib().dcu_get_tensor(ctx.handle, kind, layer, _ptr(out), n.value, _stream(stream)), ctx.handle)
    return out


def dcu_set_tensor(ctx: Context, kind: int, layer: int, src, stream=None):
    src = src.contiguous()
    _check(lib().dcu_set_tensor(ctx.handle, kind, layer, _ptr(src), src.numel() * src.element_size(),
                                _stream(stream)), ctx.handle)


def dcu_profile_enable(ctx: Context, max_launches: int):
    _check(lib().dcu_profile_enable(ctx.handle, int(max_launches)), ctx.handle)


def dcu_profile_read(ctx: Context, kernel_class: int, reset: bool = True):
    ms, n = _f64(0.0), _i64(0)
    _check(lib().dcu_profile_read(ctx.handle, kernel_class, ctypes.byref(ms), ctypes.byref(n), int(reset)),
           ctx.handle)
    return ms.value, n.value


def dcu_kernel_class_name(k: int) -> str:
    return lib().dcu_kernel_class_name(k).decode()


def dcu_launch_count(ctx: Context) -> int:
    return int(lib().dcu_launch_count(ctx.handle))


def dcu_lm_confidence_noalloc(h_rows, final_norm, lm_head, rms_eps: float = 1e-5, stream=None):
    """Confidence and argmax of final-layer rows with no device allocation by the
    library (the outputs are allocated here, by the caller side)."""
    m, D = h_rows.shape
    V = lm_head.shape[0]
    dt = {torch.bfloat16: DCU_BF16, torch.float32: DCU_F32}[h_rows.dtype]
    if lm_head.dtype != h_rows.dtype or lm_head.dim() != 2 or lm_head.shape[1] != D:
        raise ValueError("lm_head must be [V][D] in the dtype of h_rows")
    if final_norm.dtype != torch.float32 or final_norm.numel() != D:
        raise ValueError("final_norm must be float32 [D]")
    conf = torch.empty(m, dtype=torch.float32, device=h_rows.device)
    amax = torch.empty(m, dtype=torch.int32, device=h_rows.device)
    _check(lib().dcu_lm_confidence_noalloc(_ptr(h_rows), _ptr(final_norm), _ptr(lm_head), m, D, V, dt,
                                           float(rms_eps), _ptr(conf), _ptr(amax), _stream(stream)))
    return conf, amax


def dcu_linear(X, W, stream=None):
    """Y = X W^T in fp32 (X [M][K], W [Nout][K], bf16 or float32)."""
    M, K = X.shape
    Nout = W.shape[0]
    dt = {torch.bfloat16: DCU_BF16, torch.float32: DCU_F32}[X.dtype]
    Y = torch.empty((M, Nout), dtype=torch.float32, device=X.device)
    _check(lib().dcu_linear(_ptr(X), _ptr(W), M, K, Nout, dt, _ptr(Y), _stream(stream)))
    return Y


def dcu_set_graphs(ctx: Context, on: bool):
    _check(lib().dcu_set_graphs(ctx.handle, int(bool(on))), ctx.handle)


def dcu_set_refresh(ctx: Context, gen_start: int, prompt_interval: int, gen_interval: int):
    """Periodic full refresh of the prompt / generated positions (0 disables an interval)."""
    _check(lib().dcu_set_refresh(ctx.handle, int(gen_start), int(prompt_interval), int(gen_interval)), ctx.handle)


def dcu_set_select_from(ctx: Context, source: int):
    """DCU_SELECT_INPUT (layer-input distance, default) or DCU_SELECT_VALUE (Value distance)."""
    _check(lib().dcu_set_select_from(ctx.handle, int(source)), ctx.handle)


def dcu_set_option(ctx: Context, option: int, value: int):
    """Performance option of the context (DCU_OPT_FUSED_EPILOGUE, DCU_OPT_L2_PREFETCH, DCU_OPT_ATTENTION)."""
    _check(lib().dcu_set_option(ctx.handle, int(option), int(value)), ctx.handle)


def dcu_set_apd(ctx: Context, alpha: float, beta: float, tau0: float = 0.9):
    """Adaptive parallel decoding: enables rule DCU_APD with its alpha, beta and initial tau."""
    _check(lib().dcu_set_apd(ctx.handle, float(alpha), float(beta), float(tau0)), ctx.handle)


# ---- paged K/V caches
# Outputs and workspaces that these calls allocate belong to the stream they run
# on; the caller keeps the inputs alive until that stream has passed the call.

_DTYPE_CODE = {torch.bfloat16: DCU_BF16, torch.float32: DCU_F32}
_I32 = torch.int32


# handle of a device's current stream without the Stream object around it (3 us of a call)
_current_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run(device, stream, call, args):
    """call(raw stream, *args) with `device` and `stream` (None: the device's current stream) current."""
    if device.type != "cuda":
        raise ValueError(f"expected CUDA tensors, got tensors on {device}")
    if stream is None and device.index == torch.cuda.current_device():
        return call(_current_raw(device.index), *args)
    if stream is None:
        with torch.cuda.device(device):
            return call(_current_raw(device.index), *args)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else \
            torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError(f"stream of {stream.device} for tensors of {device}")
    with torch.cuda.stream(stream):
        return call(stream.cuda_stream, *args)


def _arg(t, name: str, dtype, shape, device):
    """Address of a contiguous tensor of `dtype`, `shape` and `device`."""
    if isinstance(t, torch.Tensor):
        if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
            return t.data_ptr()
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got "
                         f"{t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")
    raise TypeError(f"{name}: expected a torch.Tensor")


def _opt(t, name: str, dtype, shape, device):
    return None if t is None else _arg(t, name, dtype, shape, device)


def _dims(t, name: str, n: int):
    """Shape of a tensor argument with n dimensions."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dim() != n:
        raise ValueError(f"{name}: expected {n} dimensions, got shape {tuple(t.shape)}")
    return t.shape


# ctypes passes the low 32 bits of an integer.  Sizes are OR-ed together and compared with this once a call.
_MAX = 0x7fffffff


def _too_large():
    raise ValueError("sizes above 2^31 - 1 are not supported")


def _pages(k_pages, v_pages, device) -> dcu_pages:
    """dcu_pages of K and V tensors [n_pages][page_size][n_kv_heads][head_dim] (any strides but the last)."""
    n, p, h, d = shape = _dims(k_pages, "k_pages", 4)
    if _dims(v_pages, "v_pages", 4) != shape or v_pages.dtype != k_pages.dtype or k_pages.dtype not in _DTYPE_CODE:
        raise ValueError("k_pages and v_pages must have one shape and both be bfloat16 or both float32")
    if k_pages.device != device or v_pages.device != device:
        raise ValueError(f"k_pages and v_pages: expected tensors on {device}, got {k_pages.device}, {v_pages.device}")
    sn, sp, sh, sd = strides = k_pages.stride()
    if v_pages.stride() != strides and any(m > 1 and a != b for m, a, b in zip(shape, strides, v_pages.stride())):
        raise ValueError("k_pages and v_pages must have the same strides")
    if (sd != 1 and d != 1) or 0 in shape:
        raise ValueError(f"k_pages: expected [n_pages][page_size][n_kv_heads][head_dim] with a contiguous last "
                         f"dimension, got {tuple(shape)} with strides {strides}")
    if (n | p | h | d) > _MAX:
        _too_large()
    return dcu_pages(k_pages.data_ptr(), v_pages.data_ptr(), sn if n > 1 else 0, sp if p > 1 else 0,
                     sh if h > 1 else 0, n, p, h, d, _DTYPE_CODE[k_pages.dtype])


def dcu_page_table(lens, page_size: int, max_pages: int, n_pages: int, pool=None, first=None, status=None,
                   stream=None):
    """Block table of B requests from their lengths (int32 [B]) over the free pages `pool` (int32; None: page i is
    entry i), beginning at entry `first` (int32 [1]; None: 0).  Returns (table [B][max_pages], held [B], next [1])."""
    B, = _dims(lens, "lens", 1)
    dev = lens.device
    n_pool = n_pages if pool is None else _dims(pool, "pool", 1)[0]
    if max_pages <= 0:
        raise ValueError("max_pages must be positive")
    if (B | page_size | max_pages | n_pages | n_pool) > _MAX:
        _too_large()
    return _run(dev, stream, _page_table, (
        lens, _arg(lens, "lens", _I32, (B,), dev), B, page_size, max_pages, n_pages,
        _opt(pool, "pool", _I32, (n_pool,), dev), n_pool, _opt(first, "first", _I32, (1,), dev),
        _opt(status, "status", _I32, (1,), dev)))


def _page_table(raw, lens, p_lens, B, page_size, max_pages, n_pages, p_pool, n_pool, p_first, p_status):
    table = lens.new_empty(B, max_pages)
    held = torch.empty_like(lens)
    nxt = lens.new_empty(1)
    _check(lib().dcu_page_table(p_lens, B, page_size, max_pages, n_pages, p_pool, n_pool, p_first, table.data_ptr(),
                                held.data_ptr(), nxt.data_ptr(), p_status, raw))
    return table, held, nxt


def dcu_slot_map(table, count, page_size: int, n_pages: int, max_rows: int, pos=None, first=None, status=None,
                 stream=None):
    """Packed rows of B sequences (count int32 [B]) at positions pos (int32 [B][N], e.g. idx of dcu_select_tokens)
    or first[b], first[b] + 1, ... (int32 [B]; None: from 0).  Returns (row_start [B + 1], row_pos, slot [max_rows]);
    entries at and after row_start[B] are not written."""
    B, max_pages = _dims(table, "table", 2)
    dev = table.device
    N = 0 if pos is None else _dims(pos, "pos", 2)[1]
    if pos is not None and not N:  # its address is NULL, which the library takes for no positions
        raise ValueError("pos: expected at least one column")
    if max_rows < 0:
        raise ValueError("max_rows must not be negative")
    if (B | max_pages | page_size | n_pages | N | max_rows) > _MAX:
        _too_large()
    return _run(dev, stream, _slot_map, (
        count, _arg(table, "table", _I32, (B, max_pages), dev), B, max_pages, page_size, n_pages,
        _arg(count, "count", _I32, (B,), dev), _opt(pos, "pos", _I32, (B, N), dev), N,
        _opt(first, "first", _I32, (B,), dev), max_rows, _opt(status, "status", _I32, (1,), dev)))


def _slot_map(raw, count, p_table, B, max_pages, page_size, n_pages, p_count, p_pos, N, p_first, max_rows, p_status):
    row_start = count.new_empty(B + 1)
    row_pos = count.new_empty(max_rows)
    slot = torch.empty_like(row_pos)
    _check(lib().dcu_slot_map(p_table, B, max_pages, page_size, n_pages, p_count, p_pos, N, p_first, max_rows,
                              row_start.data_ptr(), row_pos.data_ptr(), slot.data_ptr(), p_status, raw))
    return row_start, row_pos, slot


def dcu_rope_table(max_pos: int, head_dim: int, theta: float = 10000.0, device="cuda", stream=None):
    """(cos, sin) of pos * theta^(-2j / head_dim): float32 [max_pos][head_dim / 2][2]."""
    if max_pos <= 0 or head_dim <= 0 or head_dim % 2:
        raise ValueError("max_pos and head_dim must be positive, head_dim even")
    if (max_pos | head_dim) > _MAX:
        _too_large()
    dev = torch.device(device)
    if dev.type != "cuda":
        raise ValueError("expected a CUDA device")
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())

    def call(raw):
        tab = torch.empty(max_pos, head_dim // 2, 2, dtype=torch.float32, device=dev)
        _check(lib().dcu_rope_table(tab.data_ptr(), max_pos, head_dim, theta, raw))
        return tab

    return _run(dev, stream, call, ())


def dcu_paged_write(qkv, row_start, row_pos, slot, rope, k_pages, v_pages, n_heads: int, q=None, status=None,
                    stream=None):
    """RoPE and K/V write of packed QKV rows (float32 [T][(n_heads + 2 n_kv_heads) * head_dim], e.g. of dcu_linear)
    into the pages (k_pages, v_pages: [n_pages][page_size][n_kv_heads][head_dim], any strides but the last), the
    first row_start[-1] rows.  rope: of dcu_rope_table, None for no rotation.  Returns q [T][n_heads][head_dim]
    (the given tensor when q is not None)."""
    T, width = _dims(qkv, "qkv", 2)
    dev = qkv.device
    pages = _pages(k_pages, v_pages, dev)
    hd = pages.head_dim
    if width != (n_heads + 2 * pages.n_kv_heads) * hd:
        raise ValueError(f"qkv: expected {(n_heads + 2 * pages.n_kv_heads) * hd} columns, got {width}")
    n_start, = _dims(row_start, "row_start", 1)
    if n_start < 1:
        raise ValueError("row_start: expected at least one entry")
    max_pos = 0 if rope is None else _dims(rope, "rope", 3)[0]
    if rope is not None and not max_pos:  # its address is NULL, which the library takes for no rotation
        raise ValueError("rope: expected at least one position")
    if (T | max_pos | n_heads) > _MAX:
        _too_large()
    if q is not None:
        _arg(q, "q", k_pages.dtype, (T, n_heads, hd), dev)
    return _run(dev, stream, _paged_write, (
        k_pages, q, _arg(qkv, "qkv", torch.float32, (T, width), dev), T,
        _arg(row_start, "row_start", _I32, (n_start,), dev) + 4 * (n_start - 1),
        _arg(row_pos, "row_pos", _I32, (T,), dev), _arg(slot, "slot", _I32, (T,), dev),
        _opt(rope, "rope", torch.float32, (max_pos, hd // 2, 2), dev), max_pos, n_heads, pages,
        _opt(status, "status", _I32, (1,), dev)))


def _paged_write(raw, k_pages, q, p_qkv, T, p_rows, p_pos, p_slot, p_rope, max_pos, n_heads, pages, p_status):
    if q is None:
        q = k_pages.new_empty(T, n_heads, pages.head_dim)
    _check(lib().dcu_paged_write(p_qkv, T, p_rows, p_pos, p_slot, p_rope, max_pos, n_heads, pages, q.data_ptr(),
                                 p_status, raw))
    return q


def dcu_paged_attention(q, row_start, kv_len, table, k_pages, v_pages, scale: float | None = None, out=None,
                        workspace=None, status=None, stream=None):
    """Attention of packed query rows q [T][n_heads][head_dim] (rows row_start[b] .. row_start[b + 1] belong to
    sequence b; row_start int32 [B + 1]) over the kv_len[b] (int32 [B]) cached keys of their sequence, through the
    block table (int32 [B][max_pages]).  scale defaults to head_dim^-1/2.  Returns out [T][n_heads][head_dim]; rows
    at and after row_start[B] are not written.  workspace: uint8, dcu_paged_attention_workspace bytes (None: allocated
    for the call)."""
    T, H, hd = _dims(q, "q", 3)
    dev = q.device
    pages = _pages(k_pages, v_pages, dev)
    B, max_pages = _dims(table, "table", 2)
    if (T | H | B | max_pages) > _MAX:
        _too_large()
    if out is not None:
        _arg(out, "out", q.dtype, (T, H, hd), dev)
    if workspace is not None:
        _arg(workspace, "workspace", torch.uint8, (_dims(workspace, "workspace", 1)[0],), dev)
    return _run(dev, stream, _paged_attention, (
        q, out, workspace, _arg(q, "q", k_pages.dtype, (T, H, pages.head_dim), dev), T,
        _arg(row_start, "row_start", _I32, (B + 1,), dev), B, _arg(kv_len, "kv_len", _I32, (B,), dev),
        _arg(table, "table", _I32, (B, max_pages), dev), max_pages, H, pages, hd ** -0.5 if scale is None else scale,
        _opt(status, "status", _I32, (1,), dev)))


def _paged_attention(raw, q, out, workspace, p_q, T, p_start, B, p_len, p_table, max_pages, H, pages, scale, p_status):
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = torch.empty(_workspace_bytes(pages), dtype=torch.uint8, device=q.device)
    _check(lib().dcu_paged_attention(p_q, T, p_start, B, p_len, p_table, max_pages, H, pages, scale, out.data_ptr(),
                                     workspace.data_ptr(), workspace.numel(), p_status, raw))
    return out


def _workspace_bytes(pages: dcu_pages) -> int:
    n = _i64(0)
    _check(lib().dcu_paged_attention_workspace(pages, n))
    return n.value


def dcu_paged_attention_workspace(k_pages, v_pages) -> int:
    """Bytes of the workspace tensor of dcu_paged_attention over these pages, on their device."""
    return _workspace_bytes(_pages(k_pages, v_pages, k_pages.device))
