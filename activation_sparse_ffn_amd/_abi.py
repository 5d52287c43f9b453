"""ctypes binding of libsfx (include/sfx.h).

Argument marshalling only: each function takes torch tensors, checks dtype /
contiguity / device, passes raw pointers and the current HIP stream to the C entry
point of the same name, and raises SfxError on a negative status.  Every step of
the computation runs in the library's kernels; there is no fallback.
"""
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsfx.so")

SFX_F32, SFX_F16, SFX_BF16, SFX_Q4G32 = 0, 1, 2, 3
SFX_RELU, SFX_REGLU, SFX_RELU2 = 0, 1, 2
SFX_MAX_B = 64
SFX_MAX_GROUPS = 1024
ACTS = {"relu": SFX_RELU, "reglu": SFX_REGLU, "relu2": SFX_RELU2}
WDT = {torch.float32: SFX_F32, torch.float16: SFX_F16, torch.bfloat16: SFX_BF16}

EXPORTS = ("sfx_status_str", "sfx_abi_version", "sfx_predict_ws", "sfx_predict", "sfx_compact_ws",
           "sfx_compact", "sfx_sparse_up", "sfx_sparse_down_ws", "sfx_sparse_down", "sfx_tam_ws",
           "sfx_tam_update", "sfx_ffn_step_ws", "sfx_ffn_step", "sfx_sparse_down_noalloc",
           "sfx_ffn_pipeline_ws", "sfx_ffn_pipeline", "sfx_stream_read", "sfx_predict_q4",
           "sfx_topk_now_update", "sfx_hot_update", "sfx_count_active", "sfx_select_kth_ws",
           "sfx_select_kth", "sfx_hot_first_order_ws", "sfx_hot_first_order", "sfx_gather_rows",
           "sfx_dense_ffn_ws", "sfx_dense_ffn", "sfx_linear_q4", "sfx_kv_cache_bytes", "sfx_kv_append_q4",
           "sfx_kv_read_q4", "sfx_kv_lens_q4", "sfx_attn_q4_ws", "sfx_attn_q4", "sfx_norm_q8", "sfx_linear_q8",
           "sfx_kv_cache_q8_bytes", "sfx_kv_append_q8", "sfx_kv_blank_q8", "sfx_kv_read_q8", "sfx_attn_q8_ws",
           "sfx_attn_q8")
HOT_MAX_MATS = 8
SFX_DOWN_SCRATCH_BYTES = 17 << 20


class SfxLayer(ctypes.Structure):
    """Mirror of `sfx_layer` in include/sfx.h (one layer of a fused step)."""
    _fields_ = [("x", ctypes.c_void_p), ("W1", ctypes.c_void_p), ("W2", ctypes.c_void_p),
                ("Wa", ctypes.c_void_p), ("Wa_scales", ctypes.c_void_p), ("ba", ctypes.c_void_p),
                ("Wl", ctypes.c_void_p), ("Wl_scales", ctypes.c_void_p), ("Wd", ctypes.c_void_p),
                ("Wd_scales", ctypes.c_void_p), ("threshold", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("scores", ctypes.c_void_p), ("tok_bits", ctypes.c_void_p), ("union_bits", ctypes.c_void_p),
                ("idx", ctypes.c_void_p), ("count", ctypes.c_void_p), ("hact", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("xp", ctypes.c_void_p)]


class SfxError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({status_str(status)})")


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libsfx (once).  Raises if the library has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libsfx is not built ({path} missing): run "
                           "`python -m activation_sparse_ffn_amd.build`")
    lib = ctypes.CDLL(path)
    P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.sfx_status_str.restype = ctypes.c_char_p
    lib.sfx_status_str.argtypes = [I]
    lib.sfx_abi_version.restype = I
    lib.sfx_abi_version.argtypes = []
    lib.sfx_predict_ws.restype = Z
    lib.sfx_predict_ws.argtypes = [I, I, I, I, I]
    lib.sfx_predict.restype = I
    lib.sfx_predict.argtypes = [P, I, I, I, I, I, P, P, P, P, P, Z]
    lib.sfx_compact_ws.restype = Z
    lib.sfx_compact_ws.argtypes = [I, I]
    lib.sfx_compact.restype = I
    lib.sfx_compact.argtypes = [P, I, I, P, F, P, P, P, I, P, P, Z]
    lib.sfx_sparse_up.restype = I
    lib.sfx_sparse_up.argtypes = [P, I, I, I, I, I, P, P, P, P, P, P, P, P, I, P]
    lib.sfx_sparse_down_ws.restype = Z
    lib.sfx_sparse_down_ws.argtypes = [I, I, I, I]
    lib.sfx_sparse_down.restype = I
    lib.sfx_sparse_down.argtypes = [P, I, I, I, I, P, P, P, P, I, P, P, P, Z]
    lib.sfx_sparse_down_noalloc.restype = I
    lib.sfx_sparse_down_noalloc.argtypes = [P, I, I, I, I, P, P, P, P, I, P, P]
    lib.sfx_tam_ws.restype = Z
    lib.sfx_tam_ws.argtypes = [I, I]
    lib.sfx_tam_update.restype = I
    lib.sfx_tam_update.argtypes = [P, I, I, P, F, F, I, P, P, P, P, P, P, P, Z]
    lib.sfx_topk_now_update.restype = I
    lib.sfx_topk_now_update.argtypes = [P, I, I, P, I, P, P, P, P, P]
    lib.sfx_hot_update.restype = I
    lib.sfx_hot_update.argtypes = [P, I, I, I, P, P, P, P, P, P, I, P, P, P]
    lib.sfx_count_active.restype = I
    lib.sfx_count_active.argtypes = [P, I, I, P, P]
    lib.sfx_select_kth_ws.restype = Z
    lib.sfx_select_kth_ws.argtypes = []
    lib.sfx_select_kth.restype = I
    lib.sfx_select_kth.argtypes = [P, Z, P, Z, P, P, Z]
    lib.sfx_hot_first_order_ws.restype = Z
    lib.sfx_hot_first_order_ws.argtypes = [I]
    lib.sfx_hot_first_order.restype = I
    lib.sfx_hot_first_order.argtypes = [P, I, P, P, P, P, Z]
    lib.sfx_gather_rows.restype = I
    lib.sfx_gather_rows.argtypes = [P, I, I, Z, P, P, P]
    lib.sfx_dense_ffn_ws.restype = Z
    lib.sfx_dense_ffn_ws.argtypes = [I, I, I, I]
    lib.sfx_dense_ffn.restype = I
    lib.sfx_dense_ffn.argtypes = [P, I, I, I, I, I, P, P, P, P, P, P, P, P, P, P, P, Z]
    lib.sfx_ffn_step_ws.restype = Z
    lib.sfx_ffn_step_ws.argtypes = [I, I, I, I, I, I]
    lib.sfx_ffn_step.restype = I
    lib.sfx_ffn_step.argtypes = [P, I, I, I, I, I, I, I, P, P, Z]
    lib.sfx_predict_q4.restype = I
    lib.sfx_predict_q4.argtypes = [P, I, I, I, I, P, P, P, P, P, P, P, Z]
    lib.sfx_stream_read.restype = I
    lib.sfx_stream_read.argtypes = [P, P, Z, P]
    lib.sfx_ffn_pipeline_ws.restype = Z
    lib.sfx_ffn_pipeline_ws.argtypes = [I, I, I, I, I, I]
    lib.sfx_ffn_pipeline.restype = I
    lib.sfx_ffn_pipeline.argtypes = [P, I, I, I, I, I, I, I, P, P, Z]
    lib.sfx_linear_q4.restype = I
    lib.sfx_linear_q4.argtypes = [P, I, I, I, I, I, P, Z, P, P, P, I, P, Z]
    lib.sfx_kv_cache_bytes.restype = Z
    lib.sfx_kv_cache_bytes.argtypes = [I, I, I, I]
    lib.sfx_kv_append_q4.restype = I
    lib.sfx_kv_append_q4.argtypes = [P, I, I, I, I, I, I, P, Z, P, Z, P, Z, P, P, P, I, I, I, I, I, P, I, I, P, P]
    lib.sfx_kv_read_q4.restype = I
    lib.sfx_kv_read_q4.argtypes = [P, I, I, I, I, P, P, I, I, P, I, I, P, P, P]
    lib.sfx_kv_lens_q4.restype = I
    lib.sfx_kv_lens_q4.argtypes = [P, I, P, I, I, I, P, I, I, P, P]
    lib.sfx_attn_q4_ws.restype = Z
    lib.sfx_attn_q4_ws.argtypes = [I, I, I, I, I]
    lib.sfx_attn_q4.restype = I
    lib.sfx_attn_q4.argtypes = [P, I, I, I, I, I, P, Z, I, P, I, I, P, P, P, F, P, P, P, Z]
    lib.sfx_norm_q8.restype = I
    lib.sfx_norm_q8.argtypes = [P, I, I, I, I, I, I, F, P, Z, P, Z, P, Z, P, P, P, P, Z]
    lib.sfx_linear_q8.restype = I
    lib.sfx_linear_q8.argtypes = [P, I, I, I, I, P, Z, P, P, P, P, I, P, Z]
    lib.sfx_kv_cache_q8_bytes.restype = Z
    lib.sfx_kv_cache_q8_bytes.argtypes = [I, I, I, I]
    lib.sfx_kv_append_q8.restype = I
    lib.sfx_kv_append_q8.argtypes = [P, I, I, I, I, I, I, P, Z, P, Z, P, Z, P, P, P, I, I, I, I, I, P, I, I, P, P]
    lib.sfx_kv_blank_q8.restype = I
    lib.sfx_kv_blank_q8.argtypes = [P, I, I, P, P, I, I, I, I, P, I, I, P]
    lib.sfx_kv_read_q8.restype = I
    lib.sfx_kv_read_q8.argtypes = [P, I, I, I, I, P, P, I, I, P, I, I, P, P, P]
    lib.sfx_attn_q8_ws.restype = Z
    lib.sfx_attn_q8_ws.argtypes = [I, I, I, I, I, I]
    lib.sfx_attn_q8.restype = I
    lib.sfx_attn_q8.argtypes = [P, I, I, I, I, I, I, I, P, Z, P, I, P, I, I, P, P, P, I, F, P, P, P, Z]
    _lib = lib
    return lib


def status_str(status: int) -> str:
    return load().sfx_status_str(int(status)).decode()


def abi_version() -> int:
    return load().sfx_abi_version()


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch tensor")
    if not t.is_cuda:
        raise ValueError("tensor must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(status, where):
    if status != 0:
        raise SfxError(status, where)


def _wdt_of(t: torch.Tensor) -> int:
    if t.dtype == torch.uint8:
        return SFX_Q4G32
    if t.dtype not in WDT:
        raise TypeError(f"unsupported weight dtype {t.dtype}")
    return WDT[t.dtype]


def _need(t, dtype, where):
    if t.dtype != dtype:
        raise TypeError(f"{where}: expected {dtype}, got {t.dtype}")


# ------------------------------------------------------------------------- workspaces

def workspace(nbytes: int, device=None) -> torch.Tensor:
    """Zero-filled device workspace of at least `nbytes` (the library keeps its
    control words at zero between calls)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


def sfx_predict_ws(wdt: int, B: int, d: int, h: int, f: int) -> int:
    return load().sfx_predict_ws(wdt, B, d, h, f)


def sfx_compact_ws(B: int, f: int) -> int:
    return load().sfx_compact_ws(B, f)


def sfx_sparse_down_ws(wdt: int, B: int, d: int, kmax: int) -> int:
    return load().sfx_sparse_down_ws(wdt, B, d, kmax)


def sfx_tam_ws(G: int, K: int) -> int:
    return load().sfx_tam_ws(G, K)


# ------------------------------------------------------------------------- entry points

def sfx_predict(x, W1, W2, scores, ws, stream=None):
    """scores[B][f] = W2 relu(W1 x_b).  x [B][d], W1 [h][d], W2 [f][h] (same dtype)."""
    B, d = x.shape
    h, f = W1.shape[0], W2.shape[0]
    if W1.shape[1] != d or W2.shape[1] != h or tuple(scores.shape) != (B, f):
        raise ValueError("sfx_predict: shape mismatch")
    if W1.dtype != x.dtype or W2.dtype != x.dtype:
        raise TypeError("sfx_predict: x, W1, W2 must share a dtype")
    _need(scores, torch.float32, "scores")
    ptrs = (_ptr(x), _ptr(W1), _ptr(W2), _ptr(scores), _ptr(ws))
    st = load().sfx_predict(_stream(stream), _wdt_of(x), B, d, h, f, *ptrs, ws.numel() if ws is not None else 0)
    _check(st, "sfx_predict")


def sfx_predict_q4(x, W1, W1_scales, W2, W2_scales, scores, ws, stream=None):
    """scores[B][f] = W2 relu(W1 x_b) with int4 W1 [h][d/2] / W2 [f][h/2] codes and
    fp16 scales; x [B][d] fp16."""
    B, d = x.shape
    h, f = W1.shape[0], W2.shape[0]
    if W1.shape[1] * 2 != d or W2.shape[1] * 2 != h or tuple(scores.shape) != (B, f):
        raise ValueError("sfx_predict_q4: shape mismatch")
    _need(x, torch.float16, "x")
    _need(scores, torch.float32, "scores")
    for t, n in ((W1, "W1"), (W2, "W2")):
        _need(t, torch.uint8, n)
    for t, n in ((W1_scales, "W1_scales"), (W2_scales, "W2_scales")):
        _need(t, torch.float16, n)
    p = (_ptr(x), _ptr(W1), _ptr(W1_scales), _ptr(W2), _ptr(W2_scales), _ptr(scores), _ptr(ws))
    st = load().sfx_predict_q4(_stream(stream), B, d, h, f, *p, ws.numel() if ws is not None else 0)
    _check(st, "sfx_predict_q4")


def sfx_compact(scores, threshold, union_bits, idx, count, ws, tok_bits=None, stream=None):
    """Union of {score >= threshold} over tokens -> ascending idx, device count."""
    B, f = scores.shape
    _need(scores, torch.float32, "scores")
    for t, n in ((union_bits, "union_bits"), (count, "count"), (idx, "idx")):
        if t.dtype not in (torch.int32, torch.uint32):
            raise TypeError(f"{n} must be int32/uint32")
    p = (_ptr(scores), _ptr(tok_bits), _ptr(union_bits), _ptr(idx), _ptr(count), _ptr(ws))
    st = load().sfx_compact(_stream(stream), B, f, p[0], float(threshold), p[1], p[2], p[3], idx.numel(), p[4],
                            p[5], ws.numel() if ws is not None else 0)
    _check(st, "sfx_compact")


def sfx_sparse_up(x, Wa, ba, idx, count, hact, act="relu", Wa_scales=None, Wl=None, Wl_scales=None,
                  stream=None):
    """hact[kmax][B] for the listed neurons (rows < count written)."""
    B, d = x.shape
    f = Wa.shape[0]
    wdt = _wdt_of(Wa)
    kmax = idx.numel()
    if hact.numel() < kmax * B:
        raise ValueError("hact too small")
    _need(hact, torch.float32, "hact")
    if ba is not None:
        _need(ba, torch.float32, "ba")
    p = (_ptr(x), _ptr(Wa), _ptr(Wa_scales), _ptr(ba), _ptr(Wl), _ptr(Wl_scales), _ptr(idx), _ptr(count))
    st = load().sfx_sparse_up(_stream(stream), wdt, ACTS[act], B, d, f, *p, kmax, _ptr(hact))
    _check(st, "sfx_sparse_up")


def sfx_sparse_down(Wd, idx, count, hact, y, ws, Wd_scales=None, stream=None):
    """y[B][d] = sum_j hact[j][b] Wd[idx_j] (overwritten)."""
    B, d = y.shape
    f = Wd.shape[0]
    wdt = _wdt_of(Wd)
    kmax = idx.numel()
    _need(y, torch.float32, "y")
    _need(hact, torch.float32, "hact")
    p = (_ptr(Wd), _ptr(Wd_scales), _ptr(idx), _ptr(count))
    q = (_ptr(hact), _ptr(y), _ptr(ws))
    st = load().sfx_sparse_down(_stream(stream), wdt, B, d, f, *p, kmax, *q, ws.numel() if ws is not None else 0)
    _check(st, "sfx_sparse_down")


def sfx_dense_ffn_ws(wdt: int, B: int, d: int, f: int) -> int:
    return load().sfx_dense_ffn_ws(wdt, B, d, f)


def sfx_dense_ffn(x, Wa, ba, Wd, hact, y, ws, act="relu", Wa_scales=None, Wl=None, Wl_scales=None,
                  Wd_scales=None, stream=None):
    """The FFN over every neuron: hact[f][B] and y[B][d] (both overwritten)."""
    B, d = x.shape
    f = Wa.shape[0]
    wdt = _wdt_of(Wa)
    if hact.numel() < f * B or tuple(y.shape) != (B, d):
        raise ValueError("sfx_dense_ffn: hact [f][B] and y [B][d] expected")
    _need(hact, torch.float32, "hact")
    _need(y, torch.float32, "y")
    if ba is not None:
        _need(ba, torch.float32, "ba")
    p = (_ptr(x), _ptr(Wa), _ptr(Wa_scales), _ptr(ba), _ptr(Wl), _ptr(Wl_scales), _ptr(Wd), _ptr(Wd_scales),
         _ptr(hact), _ptr(y), _ptr(ws))
    st = load().sfx_dense_ffn(_stream(stream), wdt, ACTS[act], B, d, f, *p, ws.numel() if ws is not None else 0)
    _check(st, "sfx_dense_ffn")


def sfx_sparse_down_noalloc(Wd, idx, count, hact, y, Wd_scales=None, stream=None):
    """sfx_sparse_down without a workspace: the library's static scratch is used
    (shared by every call on the GPU, so calls must not overlap)."""
    B, d = y.shape
    f = Wd.shape[0]
    wdt = _wdt_of(Wd)
    kmax = idx.numel()
    _need(y, torch.float32, "y")
    _need(hact, torch.float32, "hact")
    p = (_ptr(Wd), _ptr(Wd_scales), _ptr(idx), _ptr(count))
    st = load().sfx_sparse_down_noalloc(_stream(stream), wdt, B, d, f, *p, kmax, _ptr(hact), _ptr(y))
    _check(st, "sfx_sparse_down_noalloc")


def sfx_tam_update(union_bits, lam, eps, K, score, hot_bits, entered_bits, left_bits, topk, topk_count,
                   ws=None, stream=None):
    """One TAM step for L layers.  union_bits [L][G], score [L][G] fp32, bit sets [L][ceil(G/32)]."""
    L, G = union_bits.shape
    _need(score, torch.float32, "score")
    p = (_ptr(score), _ptr(hot_bits), _ptr(entered_bits), _ptr(left_bits), _ptr(topk) if K > 0 else None,
         _ptr(topk_count), _ptr(ws))
    st = load().sfx_tam_update(_stream(stream), L, G, _ptr(union_bits), float(lam), float(eps), int(K), *p,
                               ws.numel() if ws is not None else 0)
    _check(st, "sfx_tam_update")


def sfx_topk_now_update(union_bits, K, hot_bits, entered_bits, left_bits, topk, topk_count, stream=None):
    """The Top-K reload rule on this step's activity alone (no score state).
    union_bits [L][G], bit sets [L][ceil(G/32)], topk [L][K], topk_count [L]."""
    L, G = union_bits.shape
    st = load().sfx_topk_now_update(_stream(stream), L, G, _ptr(union_bits), int(K), _ptr(hot_bits),
                                    _ptr(entered_bits), _ptr(left_bits), _ptr(topk) if K > 0 else None,
                                    _ptr(topk_count))
    _check(st, "sfx_topk_now_update")


def sfx_hot_update(G, K, entered_bits, left_bits, slot_of, group_of, copies, ncopies, group_bytes=(),
                   src=None, dst=None, stream=None):
    """Hot-region slots and the copy of entering groups for L layers.
    entered_bits / left_bits [L][ceil(G/32)], slot_of [L][G], group_of [L][K],
    copies [L][K][2], ncopies [L] (int32 device tensors); group_bytes: host sizes
    of one group per matrix; src / dst: device int64 tensors [L][nmat] of
    matrix addresses (None when group_bytes is empty)."""
    L = entered_bits.shape[0]
    nmat = len(group_bytes)
    gb = (ctypes.c_size_t * max(nmat, 1))(*[int(v) for v in group_bytes])
    st = load().sfx_hot_update(_stream(stream), L, int(G), int(K), _ptr(entered_bits), _ptr(left_bits),
                               _ptr(slot_of), _ptr(group_of), _ptr(copies), _ptr(ncopies), nmat,
                               gb if nmat > 0 else None, _ptr(src) if nmat > 0 else None,
                               _ptr(dst) if nmat > 0 else None)
    _check(st, "sfx_hot_update")


# ------------------------------------------------------------------------- calibration

def sfx_count_active(tok_bits, f, counts, stream=None):
    """counts [f] int32 += active tokens per neuron; tok_bits [B][ceil(f/32)]."""
    B = tok_bits.shape[0]
    _check(load().sfx_count_active(_stream(stream), B, int(f), _ptr(tok_bits), _ptr(counts)), "sfx_count_active")


def sfx_select_kth(values, k, out, ws=None, stream=None):
    """out[0] = k-th smallest (0-based) of the fp32 values, exact."""
    _need(values, torch.float32, "values")
    if ws is None:
        ws = workspace(load().sfx_select_kth_ws(), values.device)
    st = load().sfx_select_kth(_stream(stream), values.numel(), _ptr(values), int(k), _ptr(out), _ptr(ws),
                               ws.numel())
    _check(st, "sfx_select_kth")


def sfx_hot_first_order(counts, perm, group=None, ws=None, stream=None):
    """perm [f] int32 = hot-first neuron table from counts [f] (and group ids)."""
    f = counts.numel()
    if group is not None and ws is None:
        ws = workspace(load().sfx_hot_first_order_ws(f), counts.device)
    st = load().sfx_hot_first_order(_stream(stream), f, _ptr(counts), _ptr(group), _ptr(perm), _ptr(ws),
                                    ws.numel() if ws is not None else 0)
    _check(st, "sfx_hot_first_order")


def sfx_gather_rows(src, idx, dst, stream=None):
    """dst row r = src row idx[r]; rows along the first dimension."""
    if src.dtype != dst.dtype or src.shape[1:] != dst.shape[1:] or dst.shape[0] != idx.numel():
        raise ValueError("dst must be [len(idx)] + src row shape, same dtype")
    row_bytes = src[0].numel() * src.element_size()
    st = load().sfx_gather_rows(_stream(stream), dst.shape[0], src.shape[0], row_bytes, _ptr(src), _ptr(idx),
                                _ptr(dst))
    _check(st, "sfx_gather_rows")


# ------------------------------------------------------------------------- fused step

def sfx_ffn_step_ws(wdt: int, act: int, B: int, d: int, h: int, f: int) -> int:
    """Workspace bytes of the fused step, 0 when the shape is not built for it."""
    return load().sfx_ffn_step_ws(wdt, act, B, d, h, f)


TORCH_OF = {SFX_F16: torch.float16, SFX_BF16: torch.bfloat16}


def _check_layer(i: int, e: dict, B: int, d: int, h: int, f: int, wdt: int, act: int):
    """Raise unless layer entry `e` holds what the fused kernel reads and writes:
    the kernel cannot check device-resident descriptors, so a missing, short or
    misaligned buffer must be caught here."""
    W = (f + 31) // 32
    wt = TORCH_OF.get(wdt)
    if wt is None:
        raise TypeError("fused step: weights must be fp16 or bf16")
    need = ["x", "W1", "W2", "Wa", "Wd", "scores", "union_bits", "idx", "count", "hact", "y"]
    if act == SFX_REGLU:
        need.append("Wl")
    for n in need:
        if e.get(n) is None:
            raise ValueError(f"layer {i}: '{n}' is required")
    shapes = {"x": (B, d), "xp": (B, d), "W1": (h, d), "W2": (f, h), "Wa": (f, d), "Wl": (f, d), "Wd": (f, d)}
    for n, shp in shapes.items():
        t = e.get(n)
        if t is None:
            continue
        if t.dtype != wt:
            raise TypeError(f"layer {i}: '{n}' is {t.dtype}, expected {wt}")
        if tuple(t.shape) != shp:
            raise ValueError(f"layer {i}: '{n}' has shape {tuple(t.shape)}, expected {shp}")
    # outputs and the bias: dtype and at least the elements the kernel touches
    sizes = {"ba": (torch.float32, f), "scores": (torch.float32, B * f), "hact": (torch.float32, f * B),
             "y": (torch.float32, B * d), "tok_bits": ((torch.int32, torch.uint32), B * W),
             "union_bits": ((torch.int32, torch.uint32), W), "idx": ((torch.int32,), f),
             "count": ((torch.int32,), 1)}
    for n, (dt, numel) in sizes.items():
        t = e.get(n)
        if t is None:
            continue
        dts = dt if isinstance(dt, tuple) else (dt,)
        if t.dtype not in dts:
            raise TypeError(f"layer {i}: '{n}' is {t.dtype}, expected {dts}")
        if t.numel() < numel:
            raise ValueError(f"layer {i}: '{n}' holds {t.numel()} elements, needs >= {numel}")
    for n, t in e.items():
        if not isinstance(t, torch.Tensor):
            continue
        align = 4 if n in ("tok_bits", "union_bits", "idx", "count", "ba") else 16
        if t.data_ptr() % align != 0:
            raise ValueError(f"layer {i}: '{n}' is not {align}-byte aligned")


def layer_descriptors(layers, B: int, d: int, h: int, f: int, wdt: int, act, device=None) -> torch.Tensor:
    """Device array of `sfx_layer` descriptors.  `layers` is a list of dicts of
    tensors (x, W1, W2, Wa, ba, Wl, Wd, scores, tok_bits, union_bits, idx, count,
    hact, y) plus a float `threshold`; missing optional entries (ba, Wl for ReLU,
    tok_bits) are NULL.  Every entry is checked against the shape (B, d, h, f) first."""
    a = ACTS[act] if isinstance(act, str) else int(act)
    arr = (SfxLayer * len(layers))()
    for i, e in enumerate(layers):
        _check_layer(i, e, B, d, h, f, wdt, a)
        for name, _ in SfxLayer._fields_:
            if name in ("threshold", "reserved"):
                continue
            t = e.get(name)
            setattr(arr[i], name, _ptr(t).value if t is not None else None)
        arr[i].threshold = float(e["threshold"])
    raw = torch.frombuffer(bytearray(bytes(arr)), dtype=torch.uint8)
    return raw.to(device or "cuda")


def sfx_ffn_step(wdt: int, act, B: int, d: int, h: int, f: int, descs: torch.Tensor, ws, stream=None):
    """Every layer's predict -> compact -> up -> down in one launch."""
    L = descs.numel() // ctypes.sizeof(SfxLayer)
    a = ACTS[act] if isinstance(act, str) else int(act)
    p = (_ptr(descs), _ptr(ws))
    st = load().sfx_ffn_step(_stream(stream), wdt, a, B, d, h, f, L, p[0], p[1], ws.numel())
    _check(st, "sfx_ffn_step")


def sfx_ffn_pipeline_ws(wdt: int, act: int, B: int, d: int, h: int, f: int) -> int:
    """Workspace bytes of the Live Pipeline step, 0 when the shape is not built for it."""
    return load().sfx_ffn_pipeline_ws(wdt, act, B, d, h, f)


def sfx_ffn_pipeline(wdt: int, act, B: int, d: int, h: int, f: int, descs: torch.Tensor, ws, stream=None):
    """Every layer's step with layer l+1's predictor (on its input xp) overlapped with
    layer l's FFN, in one launch."""
    L = descs.numel() // ctypes.sizeof(SfxLayer)
    a = ACTS[act] if isinstance(act, str) else int(act)
    p = (_ptr(descs), _ptr(ws))
    st = load().sfx_ffn_pipeline(_stream(stream), wdt, a, B, d, h, f, L, p[0], p[1], ws.numel())
    _check(st, "sfx_ffn_pipeline")


# ------------------------------------------------------------------------- int4 attention half

_F16, _BF16, _U8, _I32, _FP32 = torch.float16, torch.bfloat16, torch.uint8, torch.int32, torch.float32


def _device_error(where, *tensors):
    """Raise for tensors that are not all on one GPU."""
    for t in tensors:
        if t is not None and not t.is_cuda:
            raise ValueError(f"{where}: tensors must be on the GPU")
    raise ValueError(f"{where}: tensors are on different devices")


def _run_on(dev, stream, fn, args, where):
    """Call `fn(stream, *args)` with device `dev` current, on its current stream unless
    `stream`, one of its streams, is given."""
    if stream is not None and stream.device_index != dev:
        raise ValueError(f"{where}: the stream is on device {stream.device_index}, the tensors on {dev}")
    if dev == torch._C._cuda_getDevice():
        st = fn(torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream, *args)
    else:
        with torch.cuda.device(dev):
            st = fn(torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream, *args)
    if st != 0:
        raise SfxError(st, where)


def _rows(t, where, name):
    """Row stride of a 2-D tensor whose rows are dense (rows may be apart)."""
    n, d = t.shape
    s0, s1 = t.stride()
    if d > 1 and s1 != 1:
        raise ValueError(f"{where}: the rows of {name} must be dense")
    return s0 if n > 1 else d


def _head_rows(t, where, name):
    """Token stride of [tokens][heads][D] with dense heads (tokens may be apart)."""
    T, H, D = t.shape
    s0, s1, s2 = t.stride()
    if (D > 1 and s2 != 1) or (H > 1 and s1 != D):
        raise ValueError(f"{where}: the heads of {name} must be dense")
    return s0 if T > 1 else H * D


def _not_dense(where, t, name, dtype):
    """Raise for a tensor that is not of `dtype` or not contiguous."""
    if t.dtype != dtype:
        raise TypeError(f"{where}: {name} is {t.dtype}, expected {dtype}")
    raise ValueError(f"{where}: {name} must be contiguous")


def sfx_linear_q4(x, W, W_scales, y, bias=None, accumulate=False, stream=None):
    """y[B][n] (+)= x W^T + bias with int4 W: codes [n][d/2] uint8, W_scales
    [n][d/group] fp16 (group 32, 64 or 128).  x [B][d] fp16 / bf16, y fp32; the rows of
    x and y may be apart (slices of wider tensors)."""
    w = "sfx_linear_q4"
    if x.dim() != 2 or W.dim() != 2 or W_scales.dim() != 2 or y.dim() != 2:
        raise ValueError(f"{w}: x, W, W_scales and y must be 2-D")
    B, d = x.shape
    n, dw = W.shape
    ns, groups = W_scales.shape
    if dw * 2 != d or y.shape != (B, n):
        raise ValueError(f"{w}: shape mismatch")
    if ns != n or groups < 1 or d % groups != 0:
        raise ValueError(f"{w}: W_scales must be [n][d / group]")
    xdt = x.dtype
    if xdt is not _F16 and xdt is not _BF16:
        raise TypeError(f"{w}: x must be fp16 or bf16")
    if y.dtype is not _FP32:
        raise TypeError(f"{w}: y is {y.dtype}, expected {_FP32}")
    if W.dtype is not _U8 or not W.is_contiguous():
        _not_dense(w, W, "W", _U8)
    if W_scales.dtype is not _F16 or not W_scales.is_contiguous():
        _not_dense(w, W_scales, "W_scales", _F16)
    dev = x.get_device()
    if dev < 0 or W.get_device() != dev or W_scales.get_device() != dev or y.get_device() != dev:
        _device_error(w, x, W, W_scales, y)
    pb = None
    if bias is not None:
        if bias.numel() != n:
            raise ValueError(f"{w}: bias must hold {n} values")
        if bias.dtype is not _FP32 or not bias.is_contiguous():
            _not_dense(w, bias, "bias", _FP32)
        if bias.get_device() != dev:
            _device_error(w, x, bias)
        pb = bias.data_ptr()
    _run_on(dev, stream, (_lib or load()).sfx_linear_q4,
            (SFX_F16 if xdt is _F16 else SFX_BF16, d // groups, B, n, d, x.data_ptr(),
             d if x.is_contiguous() else _rows(x, w, "x"), W.data_ptr(), W_scales.data_ptr(), pb, 1 if accumulate else 0,
             y.data_ptr(), n if y.is_contiguous() else _rows(y, w, "y")), w)


def kv_cache_q4(num_pages: int, Hkv: int, page: int, D: int, device="cuda") -> torch.Tensor:
    """Uninitialised int4 key/value cache of one layer: uint8 [num_pages][Hkv][page/8][9 D]."""
    if load().sfx_kv_cache_bytes(Hkv, D, page, num_pages) == 0:
        raise SfxError(-2, "kv_cache_q4")
    return torch.empty(num_pages, Hkv, page // 8, 9 * D, dtype=torch.uint8, device=device)


def _cache_shape(cache, table, D, Hkv, w):
    """(page, num_pages, max_pages, B) of a cache and its page table."""
    if cache.dim() != 4 or table.dim() != 2:
        raise ValueError(f"{w}: cache must be [pages][{Hkv}][page/8][{9 * D}], table [B][max pages]")
    num_pages, hc, octets, nine_d = cache.shape
    if hc != Hkv or nine_d != 9 * D:
        raise ValueError(f"{w}: cache must be [pages][{Hkv}][page/8][{9 * D}]")
    if cache.dtype is not _U8 or not cache.is_contiguous():
        _not_dense(w, cache, "cache", _U8)
    if table.dtype is not _I32 or not table.is_contiguous():
        _not_dense(w, table, "table", _I32)
    B, max_pages = table.shape
    return octets * 8, num_pages, max_pages, B


def _tokens(t, T, dev, w, name):
    if t.numel() != T:
        raise ValueError(f"{w}: {name} must hold {T} entries")
    if t.dtype is not _I32 or not t.is_contiguous():
        _not_dense(w, t, name, _I32)
    if t.get_device() != dev:
        _device_error(w, t)
    return t.data_ptr()


def sfx_kv_append_q4(q, k, v, pos, table, cache, q_out, seq=None, cos_sin=None, interleaved=False, stream=None):
    """Rotate q [T][Hq][D] and k [T][Hkv][D] by the angles of `cos_sin` [max_pos][rot], store
    k and v as int4 at (seq[t], pos[t]) of the paged cache and write the rotated queries
    to q_out (fp16 / bf16).  q and q_out may be None (keys and values only)."""
    w = "sfx_kv_append_q4"
    if k.dim() != 3 or v.dim() != 3:
        raise ValueError(f"{w}: k and v must be [T][Hkv][D]")
    shape = k.shape
    T, Hkv, D = shape
    xdt = k.dtype
    if v.shape != shape or v.dtype is not xdt:
        raise ValueError(f"{w}: k and v must have one shape and dtype")
    if xdt not in WDT:
        raise TypeError(f"{w}: unsupported dtype {xdt}")
    dev = k.get_device()
    if dev < 0 or v.get_device() != dev or table.get_device() != dev or cache.get_device() != dev:
        _device_error(w, k, v, table, cache)
    Hq, ldq, pq, pqo, qdt = 0, 0, None, None, 0
    if q is not None:
        shape = q.shape
        if len(shape) != 3 or shape[0] != T or shape[2] != D or q.dtype is not xdt:
            raise ValueError(f"{w}: q must be [{T}][Hq][{D}] in k's dtype")
        Hq = shape[1]
        if q_out is None or q_out.shape != shape:
            raise ValueError(f"{w}: q_out must have q's shape")
        odt = q_out.dtype
        if odt is not _F16 and odt is not _BF16:
            raise TypeError(f"{w}: q_out must be fp16 or bf16")
        if not q_out.is_contiguous():
            _not_dense(w, q_out, "q_out", odt)
        qdt = SFX_F16 if odt is _F16 else SFX_BF16
        if q.get_device() != dev or q_out.get_device() != dev:
            _device_error(w, k, q, q_out)
        pq, ldq, pqo = q.data_ptr(), _head_rows(q, w, "q"), q_out.data_ptr()
    rot, max_pos, pcs = 0, 0, None
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            raise ValueError(f"{w}: cos_sin must be [positions][rot]")
        if cos_sin.dtype is not _FP32 or not cos_sin.is_contiguous():
            _not_dense(w, cos_sin, "cos_sin", _FP32)
        if cos_sin.get_device() != dev:
            _device_error(w, k, cos_sin)
        max_pos, rot = cos_sin.shape
        pcs = cos_sin.data_ptr()
    page, num_pages, max_pages, B = _cache_shape(cache, table, D, Hkv, w)
    _run_on(dev, stream, (_lib or load()).sfx_kv_append_q4,
            (WDT[xdt], qdt, T, Hq, Hkv, D, pq, ldq, k.data_ptr(), _head_rows(k, w, "k"), v.data_ptr(),
             _head_rows(v, w, "v"), _tokens(pos, T, dev, w, "pos"),
             None if seq is None else _tokens(seq, T, dev, w, "seq"), pcs, rot, max_pos, 1 if interleaved else 0, B,
             max_pages, table.data_ptr(), page, num_pages, cache.data_ptr(), pqo), w)


def sfx_kv_read_q4(pos, table, cache, k_out, v_out, seq=None, stream=None):
    """Values held at (seq[t], pos[t]): k_out, v_out [T][Hkv][D] (fp32, fp16 or bf16)."""
    w = "sfx_kv_read_q4"
    odt, shape = k_out.dtype, k_out.shape
    if len(shape) != 3 or v_out.shape != shape or v_out.dtype is not odt:
        raise ValueError(f"{w}: k_out and v_out must be [T][Hkv][D] of one dtype")
    if odt not in WDT:
        raise TypeError(f"{w}: unsupported dtype {odt}")
    if not k_out.is_contiguous() or not v_out.is_contiguous():
        raise ValueError(f"{w}: k_out and v_out must be contiguous")
    T, Hkv, D = shape
    dev = k_out.get_device()
    if dev < 0 or v_out.get_device() != dev or table.get_device() != dev or cache.get_device() != dev:
        _device_error(w, k_out, v_out, table, cache)
    page, num_pages, max_pages, B = _cache_shape(cache, table, D, Hkv, w)
    _run_on(dev, stream, (_lib or load()).sfx_kv_read_q4,
            (WDT[odt], T, Hkv, D, _tokens(pos, T, dev, w, "pos"),
             None if seq is None else _tokens(seq, T, dev, w, "seq"), B, max_pages, table.data_ptr(), page,
             num_pages, cache.data_ptr(), k_out.data_ptr(), v_out.data_ptr()),
            w)


def sfx_kv_lens_q4(pos, table, page: int, num_pages: int, lens, starts=None, window=0, max_pos=0, stream=None):
    """lens [B] = pos + 1 where a token at pos [B] is stored by sfx_kv_append_q4 (with angles for
    `max_pos` positions; 0: no angles), else 0; with a window, starts [B] = max(0, lens - window)."""
    w = "sfx_kv_lens_q4"
    if table.dim() != 2:
        raise ValueError(f"{w}: table must be [B][max pages]")
    if table.dtype is not _I32 or not table.is_contiguous():
        _not_dense(w, table, "table", _I32)
    B, max_pages = table.shape
    dev = table.get_device()
    if dev < 0:
        _device_error(w, table)
    _run_on(dev, stream, (_lib or load()).sfx_kv_lens_q4,
            (B, _tokens(pos, B, dev, w, "pos"), max_pos, window, max_pages, table.data_ptr(), page, num_pages,
             _tokens(lens, B, dev, w, "lens"), None if starts is None else _tokens(starts, B, dev, w, "starts")), w)


def sfx_attn_q4_ws(B: int, Hq: int, Hkv: int, D: int, max_len: int) -> int:
    """Workspace bytes of sfx_attn_q4 for page tables of up to `max_len` positions."""
    return load().sfx_attn_q4_ws(B, Hq, Hkv, D, max_len)


def sfx_attn_q4(q, cache, table, lens, out, ws, starts=None, scale=None, lse=None, stream=None):
    """Attention of one token per sequence over the int4 cache: q [B][Hq][D] (fp16 / bf16,
    sequences may be apart), out [B][Hq][D] in q's dtype; positions [starts[b], lens[b]);
    scale defaults to D ** -0.5; lse [B][Hq] fp32 optional."""
    w = "sfx_attn_q4"
    if q.dim() != 3 or cache.dim() != 4:
        raise ValueError(f"{w}: q must be [B][Hq][D], cache [pages][Hkv][page/8][9 D]")
    shape = q.shape
    B, Hq, D = shape
    qdt = q.dtype
    if qdt is not _F16 and qdt is not _BF16:
        raise TypeError(f"{w}: q must be fp16 or bf16")
    if out.shape != shape:
        raise ValueError(f"{w}: out must have q's shape")
    if out.dtype is not qdt or not out.is_contiguous():
        _not_dense(w, out, "out", qdt)
    Hkv = cache.shape[1]
    page, num_pages, max_pages, Bt = _cache_shape(cache, table, D, Hkv, w)
    if Bt != B:
        raise ValueError(f"{w}: table must have {B} rows")
    if lens.numel() != B:
        raise ValueError(f"{w}: lens must hold {B} entries")
    if lens.dtype is not _I32 or not lens.is_contiguous():
        _not_dense(w, lens, "lens", _I32)
    dev = q.get_device()
    if (dev < 0 or cache.get_device() != dev or table.get_device() != dev or out.get_device() != dev or
            lens.get_device() != dev):
        _device_error(w, q, cache, table, lens, out)
    pl = pw = None
    nws = 0
    if lse is not None:
        if lse.shape != (B, Hq):
            raise ValueError(f"{w}: lse must be [{B}][{Hq}]")
        if lse.dtype is not _FP32 or not lse.is_contiguous():
            _not_dense(w, lse, "lse", _FP32)
        if lse.get_device() != dev:
            _device_error(w, q, lse)
        pl = lse.data_ptr()
    if ws is not None:
        if ws.get_device() != dev:
            _device_error(w, q, ws)
        if not ws.is_contiguous():
            raise ValueError(f"{w}: ws must be contiguous")
        pw, nws = ws.data_ptr(), ws.nbytes
    _run_on(dev, stream, (_lib or load()).sfx_attn_q4,
            (SFX_F16 if qdt is _F16 else SFX_BF16, B, Hq, Hkv, D, q.data_ptr(),
             Hq * D if q.is_contiguous() else _head_rows(q, w, "q"), max_pages,
             table.data_ptr(), page, num_pages, cache.data_ptr(),
             None if starts is None else _tokens(starts, B, dev, w, "starts"), lens.data_ptr(),
             D ** -0.5 if scale is None else float(scale), out.data_ptr(), pl, pw, nws), w)


# ------------------------------------------------------------------------- 8-bit layer half

_I8 = torch.int8


def _dense(t, dtype, dev, w, name):
    """Pointer of a contiguous tensor of `dtype` on `dev`."""
    if t.dtype is not dtype or not t.is_contiguous():
        _not_dense(w, t, name, dtype)
    if t.get_device() != dev:
        _device_error(w, t)
    return t.data_ptr()


def sfx_norm_q8(x, q=None, s=None, weight=None, eps=1e-5, residual=None, residual_out=None, y=None, norm=True, stream=None):
    """h = x + residual (written to residual_out, in place if that is None); n = h's
    root-mean-square norm times `weight` (norm=False: n = h); int8 codes q [T][d] with a scale
    s [T] per row, and / or y = n.  x, residual and y [T][d] fp32, fp16 or bf16 (rows may be
    apart), weight [d] fp32."""
    w = "sfx_norm_q8"
    if x.dim() != 2:
        raise ValueError(f"{w}: x must be [T][d]")
    T, d = shape = x.shape
    xdt = x.dtype
    if xdt not in WDT:
        raise TypeError(f"{w}: unsupported dtype {xdt}")
    dev = x.get_device()
    if dev < 0:
        _device_error(w, x)
    rdt = ydt = ldr = ldro = ldy = 0
    pr = pro = py = pq = ps = pw = None
    if residual is not None:
        ro = residual if residual_out is None else residual_out
        dt = residual.dtype
        if residual.shape != shape or ro is not residual and (ro.shape != shape or ro.dtype is not dt):
            raise ValueError(f"{w}: residual and residual_out must be [{T}][{d}] of one dtype")
        if dt not in WDT:
            raise TypeError(f"{w}: unsupported dtype {dt}")
        if residual.get_device() != dev or ro.get_device() != dev:
            _device_error(w, x, residual, ro)
        rdt, pr = WDT[dt], residual.data_ptr()
        ldr = d if residual.is_contiguous() else _rows(residual, w, "residual")
        pro, ldro = (pr, ldr) if ro is residual else (ro.data_ptr(), d if ro.is_contiguous() else _rows(ro, w, "residual_out"))
    elif residual_out is not None:
        raise ValueError(f"{w}: residual_out without a residual")
    if y is not None:
        if y.shape != shape:
            raise ValueError(f"{w}: y must be [{T}][{d}]")
        dt = y.dtype
        if dt not in WDT:
            raise TypeError(f"{w}: unsupported dtype {dt}")
        if y.get_device() != dev:
            _device_error(w, x, y)
        ydt, py, ldy = WDT[dt], y.data_ptr(), d if y.is_contiguous() else _rows(y, w, "y")
    if (q is None) != (s is None):
        raise ValueError(f"{w}: q and s go together")
    if q is not None:
        if q.shape != shape or s.numel() != T:
            raise ValueError(f"{w}: q must be [{T}][{d}] and s hold {T} values")
        if q.dtype is not _I8 or not q.is_contiguous():
            _not_dense(w, q, "q", _I8)
        if s.dtype is not _FP32 or not s.is_contiguous():
            _not_dense(w, s, "s", _FP32)
        if q.get_device() != dev or s.get_device() != dev:
            _device_error(w, x, q, s)
        pq, ps = q.data_ptr(), s.data_ptr()
    if weight is not None:
        if weight.numel() != d:
            raise ValueError(f"{w}: weight must hold {d} values")
        if weight.dtype is not _FP32 or not weight.is_contiguous():
            _not_dense(w, weight, "weight", _FP32)
        if weight.get_device() != dev:
            _device_error(w, x, weight)
        pw = weight.data_ptr()
    _run_on(dev, stream, (_lib or load()).sfx_norm_q8,
            (WDT[xdt], rdt, ydt, T, d, 1 if norm else 0, eps, x.data_ptr(),
             d if x.is_contiguous() else _rows(x, w, "x"), pr, ldr, pro, ldro, pw, pq, ps, py, ldy), w)


def sfx_linear_q8(x, x_scales, W, W_scales, y, bias=None, accumulate=False, stream=None):
    """y [T][n] (+)= (x_scales x) (W_scales W)^T + bias for int8 x [T][d] and W [n][d] with fp32
    scales [T] and [n]; y fp32, fp16 or bf16.  The rows of x and y may be apart."""
    w = "sfx_linear_q8"
    if x.dim() != 2 or W.dim() != 2 or y.dim() != 2:
        raise ValueError(f"{w}: x, W and y must be 2-D")
    T, d = x.shape
    n, dw = W.shape
    if dw != d or y.shape != (T, n) or x_scales.numel() != T or W_scales.numel() != n:
        raise ValueError(f"{w}: shape mismatch")
    if x.dtype is not _I8:
        raise TypeError(f"{w}: x is {x.dtype}, expected {_I8}")
    ydt = y.dtype
    if ydt not in WDT:
        raise TypeError(f"{w}: unsupported dtype {ydt}")
    if W.dtype is not _I8 or not W.is_contiguous():
        _not_dense(w, W, "W", _I8)
    if x_scales.dtype is not _FP32 or not x_scales.is_contiguous():
        _not_dense(w, x_scales, "x_scales", _FP32)
    if W_scales.dtype is not _FP32 or not W_scales.is_contiguous():
        _not_dense(w, W_scales, "W_scales", _FP32)
    dev = x.get_device()
    if (dev < 0 or y.get_device() != dev or W.get_device() != dev or x_scales.get_device() != dev or
            W_scales.get_device() != dev):
        _device_error(w, x, x_scales, W, W_scales, y)
    pb = None
    if bias is not None:
        if bias.numel() != n:
            raise ValueError(f"{w}: bias must hold {n} values")
        pb = _dense(bias, _FP32, dev, w, "bias")
    _run_on(dev, stream, (_lib or load()).sfx_linear_q8,
            (WDT[ydt], T, n, d, x.data_ptr(), d if x.is_contiguous() else _rows(x, w, "x"), x_scales.data_ptr(),
             W.data_ptr(), W_scales.data_ptr(), pb, 1 if accumulate else 0, y.data_ptr(),
             n if y.is_contiguous() else _rows(y, w, "y")), w)


def kv_cache_q8(num_pages: int, Hkv: int, page: int, D: int, device="cuda") -> torch.Tensor:
    """Uninitialised int8 key/value cache of one layer: uint8 [num_pages][Hkv][page/16][32 D + 16]."""
    if load().sfx_kv_cache_q8_bytes(Hkv, D, page, num_pages) == 0:
        raise SfxError(-2, "kv_cache_q8")
    return torch.empty(num_pages, Hkv, page // 16, 32 * D + 16, dtype=torch.uint8, device=device)


def _cache8_shape(cache, table, D, Hkv, w):
    """(page, num_pages, max_pages, B) of an int8 cache and its page table."""
    if cache.dim() != 4 or table.dim() != 2:
        raise ValueError(f"{w}: cache must be [pages][{Hkv}][page/16][{32 * D + 16}], table [B][max pages]")
    num_pages, hc, blocks, size = cache.shape
    if hc != Hkv or size != 32 * D + 16:
        raise ValueError(f"{w}: cache must be [pages][{Hkv}][page/16][{32 * D + 16}]")
    if cache.dtype is not _U8 or not cache.is_contiguous():
        _not_dense(w, cache, "cache", _U8)
    if table.dtype is not _I32 or not table.is_contiguous():
        _not_dense(w, table, "table", _I32)
    B, max_pages = table.shape
    return blocks * 16, num_pages, max_pages, B


def sfx_kv_append_q8(q, k, v, lens, table, cache, q_out, q_start=None, cos_sin=None, interleaved=False, stream=None):
    """Rotate q [T][Hq][D] and k [T][Hkv][D] by the angles of `cos_sin` [max_pos][rot], store k and
    v as int8 at the last positions of the sequences (rows q_start[b] .. q_start[b + 1] - 1 of
    sequence b, which has lens[b] positions with them; without q_start one row each) and
    write the rotated queries to q_out (fp16 / bf16).  q and q_out may be None."""
    w = "sfx_kv_append_q8"
    if k.dim() != 3 or v.dim() != 3:
        raise ValueError(f"{w}: k and v must be [T][Hkv][D]")
    shape = k.shape
    T, Hkv, D = shape
    xdt = k.dtype
    if v.shape != shape or v.dtype is not xdt:
        raise ValueError(f"{w}: k and v must have one shape and dtype")
    if xdt not in WDT:
        raise TypeError(f"{w}: unsupported dtype {xdt}")
    dev = k.get_device()
    if dev < 0 or v.get_device() != dev or table.get_device() != dev or cache.get_device() != dev:
        _device_error(w, k, v, table, cache)
    Hq, ldq, pq, pqo, qdt = 0, 0, None, None, 0
    if q is not None:
        shape = q.shape
        if len(shape) != 3 or shape[0] != T or shape[2] != D or q.dtype is not xdt:
            raise ValueError(f"{w}: q must be [{T}][Hq][{D}] in k's dtype")
        Hq = shape[1]
        if q_out is None or q_out.shape != shape:
            raise ValueError(f"{w}: q_out must have q's shape")
        odt = q_out.dtype
        if odt is not _F16 and odt is not _BF16:
            raise TypeError(f"{w}: q_out must be fp16 or bf16")
        qdt = SFX_F16 if odt is _F16 else SFX_BF16
        if not q_out.is_contiguous():
            _not_dense(w, q_out, "q_out", odt)
        if q.get_device() != dev or q_out.get_device() != dev:
            _device_error(w, k, q, q_out)
        pq, ldq, pqo = q.data_ptr(), Hq * D if q.is_contiguous() else _head_rows(q, w, "q"), q_out.data_ptr()
    rot, max_pos, pcs = 0, 0, None
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            raise ValueError(f"{w}: cos_sin must be [positions][rot]")
        max_pos, rot = cos_sin.shape
        if cos_sin.dtype is not _FP32 or not cos_sin.is_contiguous():
            _not_dense(w, cos_sin, "cos_sin", _FP32)
        if cos_sin.get_device() != dev:
            _device_error(w, k, cos_sin)
        pcs = cos_sin.data_ptr()
    page, num_pages, max_pages, B = _cache8_shape(cache, table, D, Hkv, w)
    if lens.numel() != B:
        raise ValueError(f"{w}: lens must hold {B} entries")
    if lens.dtype is not _I32 or not lens.is_contiguous():
        _not_dense(w, lens, "lens", _I32)
    if lens.get_device() != dev:
        _device_error(w, k, lens)
    _run_on(dev, stream, (_lib or load()).sfx_kv_append_q8,
            (WDT[xdt], qdt, T, Hq, Hkv, D, pq, ldq, k.data_ptr(), Hkv * D if k.is_contiguous() else _head_rows(k, w, "k"),
             v.data_ptr(), Hkv * D if v.is_contiguous() else _head_rows(v, w, "v"),
             None if q_start is None else _tokens(q_start, B + 1, dev, w, "q_start"), lens.data_ptr(), pcs, rot, max_pos,
             1 if interleaved else 0, B, max_pages, table.data_ptr(), page, num_pages, cache.data_ptr(), pqo), w)


def sfx_kv_blank_q8(x, lens, table, page: int, num_pages: int, q_start=None, max_q=1, max_pos=0, stream=None):
    """Zeroes the rows of x [T][n] (fp16 / bf16) that are no token of a call: those that sfx_kv_append_q8 does not
    store (with angles for `max_pos` positions; 0: no angles) and those past a sequence's first max_q."""
    w = "sfx_kv_blank_q8"
    if x.dim() != 2 or table.dim() != 2:
        raise ValueError(f"{w}: x must be [T][n], table [B][max pages]")
    if x.dtype is not _F16 and x.dtype is not _BF16:
        raise TypeError(f"{w}: x must be fp16 or bf16")
    if not x.is_contiguous():
        _not_dense(w, x, "x", x.dtype)
    if table.dtype is not _I32 or not table.is_contiguous():
        _not_dense(w, table, "table", _I32)
    B, max_pages = table.shape
    dev = x.get_device()
    if dev < 0 or table.get_device() != dev:
        _device_error(w, x, table)
    _run_on(dev, stream, (_lib or load()).sfx_kv_blank_q8,
            (x.shape[0], x.shape[1], None if q_start is None else _tokens(q_start, B + 1, dev, w, "q_start"),
             _tokens(lens, B, dev, w, "lens"), max_pos, max_q, B, max_pages, table.data_ptr(), page, num_pages, x.data_ptr()), w)


def sfx_kv_read_q8(pos, table, cache, k_out, v_out, seq=None, stream=None):
    """Values held at (seq[t], pos[t]): k_out, v_out [T][Hkv][D] (fp32, fp16 or bf16)."""
    w = "sfx_kv_read_q8"
    odt, shape = k_out.dtype, k_out.shape
    if len(shape) != 3 or v_out.shape != shape or v_out.dtype is not odt:
        raise ValueError(f"{w}: k_out and v_out must be [T][Hkv][D] of one dtype")
    if odt not in WDT:
        raise TypeError(f"{w}: unsupported dtype {odt}")
    if not k_out.is_contiguous() or not v_out.is_contiguous():
        raise ValueError(f"{w}: k_out and v_out must be contiguous")
    T, Hkv, D = shape
    dev = k_out.get_device()
    if dev < 0 or v_out.get_device() != dev or table.get_device() != dev or cache.get_device() != dev:
        _device_error(w, k_out, v_out, table, cache)
    page, num_pages, max_pages, B = _cache8_shape(cache, table, D, Hkv, w)
    if pos.numel() != T:
        raise ValueError(f"{w}: pos must hold {T} entries")
    if pos.dtype is not _I32 or not pos.is_contiguous():
        _not_dense(w, pos, "pos", _I32)
    if pos.get_device() != dev:
        _device_error(w, k_out, pos)
    _run_on(dev, stream, (_lib or load()).sfx_kv_read_q8,
            (WDT[odt], T, Hkv, D, pos.data_ptr(),
             None if seq is None else _tokens(seq, T, dev, w, "seq"), B, max_pages, table.data_ptr(), page,
             num_pages, cache.data_ptr(), k_out.data_ptr(), v_out.data_ptr()),
            w)


def sfx_attn_q8_ws(B: int, max_q: int, Hq: int, Hkv: int, D: int, max_len: int) -> int:
    """Workspace bytes of sfx_attn_q8 for page tables of up to `max_len` positions."""
    return load().sfx_attn_q8_ws(B, max_q, Hq, Hkv, D, max_len)


def sfx_attn_q8(q, cache, table, lens, out, ws, q_start=None, max_q=1, starts=None, window=0, scale=None, lse=None,
                stream=None):
    """Causal attention of the last tokens of each sequence over the int8 cache: q [T][Hq][D]
    (fp16 / bf16, tokens may be apart), rows q_start[b] .. q_start[b + 1] - 1 (at most max_q) of
    sequence b with lens[b] positions; without q_start one row each.  out [T][Hq][D] in q's
    dtype; `window` positions back (0: all), none before starts[b]; scale defaults to
    D ** -0.5; lse [T][Hq] fp32 optional."""
    w = "sfx_attn_q8"
    if q.dim() != 3 or cache.dim() != 4:
        raise ValueError(f"{w}: q must be [T][Hq][D], cache [pages][Hkv][page/16][32 D + 16]")
    shape = q.shape
    T, Hq, D = shape
    qdt = q.dtype
    if qdt is not _F16 and qdt is not _BF16:
        raise TypeError(f"{w}: q must be fp16 or bf16")
    if out.shape != shape:
        raise ValueError(f"{w}: out must have q's shape")
    if out.dtype is not qdt or not out.is_contiguous():
        _not_dense(w, out, "out", qdt)
    Hkv = cache.shape[1]
    page, num_pages, max_pages, B = _cache8_shape(cache, table, D, Hkv, w)
    if q_start is None and B != T:
        raise ValueError(f"{w}: table must have {T} rows")
    if lens.numel() != B:
        raise ValueError(f"{w}: lens must hold {B} entries")
    if lens.dtype is not _I32 or not lens.is_contiguous():
        _not_dense(w, lens, "lens", _I32)
    dev = q.get_device()
    if (dev < 0 or cache.get_device() != dev or table.get_device() != dev or out.get_device() != dev or
            lens.get_device() != dev):
        _device_error(w, q, cache, table, lens, out)
    pl = pw = None
    nws = 0
    if lse is not None:
        if lse.shape != (T, Hq):
            raise ValueError(f"{w}: lse must be [{T}][{Hq}]")
        pl = _dense(lse, _FP32, dev, w, "lse")
    if ws is not None:
        if ws.get_device() != dev:
            _device_error(w, q, ws)
        if not ws.is_contiguous():
            raise ValueError(f"{w}: ws must be contiguous")
        pw, nws = ws.data_ptr(), ws.nbytes
    _run_on(dev, stream, (_lib or load()).sfx_attn_q8,
            (SFX_F16 if qdt is _F16 else SFX_BF16, T, B, max_q, Hq, Hkv, D, q.data_ptr(),
             Hq * D if q.is_contiguous() else _head_rows(q, w, "q"),
             None if q_start is None else _tokens(q_start, B + 1, dev, w, "q_start"), max_pages,
             table.data_ptr(), page, num_pages, cache.data_ptr(),
             None if starts is None else _tokens(starts, B, dev, w, "starts"), lens.data_ptr(), window,
             D ** -0.5 if scale is None else float(scale), out.data_ptr(), pl, pw, nws), w)


STREAM_READ_OUT_WORDS = 16384


def sfx_stream_read(buf: torch.Tensor, out: torch.Tensor, stream=None):
    """Measurement helper: read `buf` once (the streaming-read ceiling)."""
    if out.numel() < STREAM_READ_OUT_WORDS or out.element_size() != 4:
        raise ValueError("out must hold 16384 32-bit words")
    st = load().sfx_stream_read(_stream(stream), _ptr(buf), buf.numel() * buf.element_size(), _ptr(out))
    _check(st, "sfx_stream_read")
