"""ctypes binding of the C ABI in include/moe.h (libmoe_mi355x.so).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  Functions take torch tensors on the GPU (PyTorch supplies device
memory and streams) and return the library status, raising ``MoeError`` on
anything but MOE_OK.  The library is loaded from this package's directory;
there is no other implementation to fall back to.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_mi355x.so")

MOE_OK, MOE_ERR_INVALID, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_DEVICE = range(5)
SCORE = {"sigmoid": 0, "sqrt_softplus": 1, "softmax": 2}
DTYPE = {"f32": 0, "bf16": 1, "q8b32": 2, "f8b128": 3}
PATH = {"auto": 0, "decode": 1, "prefill": 2}
DECODE_MAX_TOKENS = 8


class MoeError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__("%s (status %d)" % (msg, status))
        self.status = status


class moe_config(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int32), ("d_model", ctypes.c_int32),
                ("n_expert", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("d_ff", ctypes.c_int32), ("n_shared", ctypes.c_int32),
                ("d_ff_shared", ctypes.c_int32), ("score", ctypes.c_int32),
                ("route_scale", ctypes.c_float), ("act_dtype", ctypes.c_int32),
                ("w_dtype", ctypes.c_int32), ("path", ctypes.c_int32)]


class moe_groups(ctypes.Structure):
    _fields_ = [("n_group", ctypes.c_int32), ("topk_group", ctypes.c_int32),
                ("group_top", ctypes.c_int32), ("normalise", ctypes.c_int32)]


class moe_mat(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


class moe_weights(ctypes.Structure):
    _fields_ = [("w_router", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("gate", moe_mat), ("up", moe_mat), ("down", moe_mat),
                ("s_gate", moe_mat), ("s_up", moe_mat), ("s_down", moe_mat)]


STAGES = ("router", "select", "permute", "gate_up", "down", "combine")
STAGE_EVENTS = 2 * len(STAGES)  # [2s] start of stage s's first kernel, [2s+1] end of its last
DECODE_STAGES = ("router", "select", "gate_up", "down")  # stages the decode path launches kernels for


class moe_debug(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("topk_idx", ctypes.c_void_p),
                ("topk_w", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
                ("perm_rows", ctypes.c_void_p), ("inv_perm", ctypes.c_void_p),
                ("stage_events", ctypes.POINTER(ctypes.c_void_p))]


EXPORTS = ("moe_workspace_bytes", "moe_route", "moe_select", "moe_permute", "moe_expert_ffn",
           "moe_combine", "moe_layer_forward", "moe_layer_forward_noalloc", "moe_topk_rows",
           "moe_prefetch_experts", "moe_select_grouped", "moe_route_grouped", "moe_layer_forward_grouped",
           "moe_quantize_rows", "moe_block_matmul", "moe_block_matmul_workspace_bytes", "moe_status_str")
STATIC_SCRATCH_BYTES = 64 << 20  # MOE_STATIC_SCRATCH_BYTES
TOPK_ROWS_MAX_N = 65536  # MOE_TOPK_ROWS_MAX_N
PREFETCH_MAX_IDS = 65536  # MOE_PREFETCH_MAX_IDS
PREFETCH_MAX_WORKGROUPS = 4096  # MOE_PREFETCH_MAX_WORKGROUPS
PREFETCH_GATE, PREFETCH_UP, PREFETCH_DOWN = 1, 2, 4  # bits of moe_prefetch_experts' `which`

_lib = None


def load(path: str = LIB_PATH):
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise ImportError("libmoe_mi355x.so is not built (run __graft_entry__.build() or "
                          "python sparse_moe_layer_02_amd/build.py); there is no fallback path")
    lib = ctypes.CDLL(path)
    P, C = ctypes.c_void_p, ctypes.POINTER(moe_config)
    W = ctypes.POINTER(moe_weights)
    lib.moe_workspace_bytes.argtypes = [C]
    lib.moe_workspace_bytes.restype = ctypes.c_size_t
    lib.moe_route.argtypes = [C, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.moe_select.argtypes = [C, P, P, P, P, P]
    lib.moe_permute.argtypes = [C, P, P, P, P, P, ctypes.c_size_t, P]
    lib.moe_expert_ffn.argtypes = [C, P, W, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.moe_combine.argtypes = [C, P, P, P, P]
    lib.moe_layer_forward.argtypes = [C, P, W, P, ctypes.POINTER(moe_debug), P, ctypes.c_size_t, P]
    lib.moe_layer_forward_noalloc.argtypes = [C, P, W, P, ctypes.POINTER(moe_debug), P]
    I = ctypes.c_int32
    lib.moe_topk_rows.argtypes = [P, I, I, I, P, P, ctypes.POINTER(ctypes.c_void_p), P]
    lib.moe_prefetch_experts.argtypes = [C, W, P, I, I, I, I, ctypes.POINTER(ctypes.c_void_p), P]
    G = ctypes.POINTER(moe_groups)
    S, D = ctypes.c_size_t, ctypes.POINTER(moe_debug)
    lib.moe_select_grouped.argtypes = [C, G, P, P, P, P, P]
    lib.moe_route_grouped.argtypes = [C, G, P, P, P, P, P, P, P, S, P]
    lib.moe_layer_forward_grouped.argtypes = [C, G, P, W, P, I, D, P, S, P]
    lib.moe_quantize_rows.argtypes = [P, I, I, I, ctypes.c_int64, P, P, P]
    lib.moe_block_matmul.argtypes = [P, I, P, P, P, I, I, I, P, I, P, S, P]
    lib.moe_block_matmul_workspace_bytes.argtypes = [I, I, I]
    lib.moe_status_str.argtypes = [ctypes.c_int]
    lib.moe_status_str.restype = ctypes.c_char_p
    for name in EXPORTS[1:-1]:
        getattr(lib, name).restype = ctypes.c_int
    lib.moe_block_matmul_workspace_bytes.restype = ctypes.c_size_t
    if path == LIB_PATH:
        _lib = lib
    return lib


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

def make_config(T, d, E, k, F, n_shared=1, Fs=None, score="sigmoid", route_scale=1.0, act="bf16",
                w="bf16", path="auto") -> moe_config:
    return moe_config(n_tokens=T, d_model=d, n_expert=E, top_k=k, d_ff=F, n_shared=n_shared,
                      d_ff_shared=F if Fs is None else Fs, score=SCORE.get(score, score),
                      route_scale=route_scale, act_dtype=DTYPE.get(act, act),
                      w_dtype=DTYPE.get(w, w), path=PATH.get(path, path))


def config_from(cfg: dict, T=None, path="auto") -> moe_config:
    """A moe_config from a workload dict (keys T, d, E, k, F, Fs, n_shared, score, scale, act, w)."""
    return make_config(cfg["T"] if T is None else T, cfg["d"], cfg["E"], cfg["k"], cfg["F"],
                       cfg["n_shared"], cfg["Fs"], cfg["score"], cfg["scale"], cfg["act"], cfg["w"], path)


def ptr(t) -> int | None:
    """Device address of a tensor (None passes through as NULL)."""
    if t is None:
        return None
    return t.data_ptr()


def mat(m) -> moe_mat:
    """moe_mat from a tensor or a (quants, scales) pair of tensors."""
    if m is None:
        return moe_mat(None, None)
    if isinstance(m, (tuple, list)):
        return moe_mat(ptr(m[0]), ptr(m[1]))
    return moe_mat(ptr(m), None)


def make_weights(W: dict) -> moe_weights:
    """moe_weights from a dict of device tensors (keys as in the header)."""
    return moe_weights(ptr(W["w_router"]), ptr(W.get("bias")), mat(W["gate"]), mat(W["up"]),
                       mat(W["down"]), mat(W.get("s_gate")), mat(W.get("s_up")), mat(W.get("s_down")))


def _stream(stream):
    if stream is not None:
        return stream
    import torch
    try:  # the handle alone, without building a Stream object (2.8 us less per call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    except AttributeError:
        return torch.cuda.current_stream().cuda_stream


def _check(st, lib=None):
    if st != MOE_OK:
        lib = lib or load()
        raise MoeError(st, lib.moe_status_str(st).decode())
    return st


# ---------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ---------------------------------------------------------------------------

def moe_workspace_bytes(cfg: moe_config) -> int:
    return load().moe_workspace_bytes(ctypes.byref(cfg))


def moe_status_str(status: int) -> str:
    return load().moe_status_str(status).decode()


def moe_route(cfg, x, w_router, bias, logits, topk_idx, topk_w, ws, stream=None):
    lib = load()
    return _check(lib.moe_route(ctypes.byref(cfg), ptr(x), ptr(w_router), ptr(bias), ptr(logits),
                                ptr(topk_idx), ptr(topk_w), ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                _stream(stream)), lib)


def moe_select(cfg, logits, bias, topk_idx, topk_w, stream=None):
    lib = load()
    return _check(lib.moe_select(ctypes.byref(cfg), ptr(logits), ptr(bias), ptr(topk_idx), ptr(topk_w),
                                 _stream(stream)), lib)


def moe_permute(cfg, topk_idx, offsets, perm_rows, inv_perm, ws, stream=None):
    lib = load()
    return _check(lib.moe_permute(ctypes.byref(cfg), ptr(topk_idx), ptr(offsets), ptr(perm_rows),
                                  ptr(inv_perm), ptr(ws), ws.numel() * ws.element_size(), _stream(stream)), lib)


def moe_expert_ffn(cfg, x, weights: moe_weights, offsets, perm_rows, topk_w, slot_out, shared_out, ws,
                   stream=None):
    lib = load()
    return _check(lib.moe_expert_ffn(ctypes.byref(cfg), ptr(x), ctypes.byref(weights), ptr(offsets),
                                     ptr(perm_rows), ptr(topk_w), ptr(slot_out), ptr(shared_out), ptr(ws),
                                     ws.numel() * ws.element_size(), _stream(stream)), lib)


def moe_combine(cfg, slot_out, shared_out, y, stream=None):
    lib = load()
    return _check(lib.moe_combine(ctypes.byref(cfg), ptr(slot_out), ptr(shared_out), ptr(y),
                                  _stream(stream)), lib)


def moe_layer_forward(cfg, x, weights: moe_weights, y, ws, debug: dict | None = None, stream=None,
                      stage_events=None):
    """``stage_events``: optional ctypes array of STAGE_EVENTS hipEvent_t handles
    (start and end timestamps of each stage's kernels)."""
    lib = load()
    dbg = _debug_struct(debug, stage_events)
    return _check(lib.moe_layer_forward(ctypes.byref(cfg), ptr(x), ctypes.byref(weights), ptr(y),
                                        ctypes.byref(dbg) if dbg else None, ptr(ws),
                                        ws.numel() * ws.element_size(), _stream(stream)), lib)


def _debug_struct(debug, stage_events):
    if not debug and stage_events is None:
        return None
    debug = debug or {}
    dbg = moe_debug(*(ptr(debug.get(k)) for k in ("logits", "topk_idx", "topk_w", "offsets", "perm_rows",
                                                  "inv_perm")))
    if stage_events is not None:
        dbg.stage_events = ctypes.cast(stage_events, ctypes.POINTER(ctypes.c_void_p))
    return dbg


def moe_layer_forward_noalloc(cfg, x, weights: moe_weights, y, debug: dict | None = None, stream=None,
                              stage_events=None):
    """moe_layer_forward over the library's static device scratch (no workspace
    argument; configs needing more than STATIC_SCRATCH_BYTES are refused)."""
    lib = load()
    dbg = _debug_struct(debug, stage_events)
    return _check(lib.moe_layer_forward_noalloc(ctypes.byref(cfg), ptr(x), ctypes.byref(weights), ptr(y),
                                                ctypes.byref(dbg) if dbg else None, _stream(stream)), lib)


def moe_topk_rows(scores, k, idx, vals=None, stream=None, events=None):
    """Row top-k of ``scores`` [rows, n] fp32 into ``idx`` [rows, k] int32 (ascending
    candidate index) and ``vals`` [rows, k] fp32 (optional).  ``events``: optional
    ctypes array of 2 hipEvent_t handles (dispatch start and end timestamps)."""
    lib = load()
    rows, n = scores.shape
    ev = None if events is None else ctypes.cast(events, ctypes.POINTER(ctypes.c_void_p))
    return _check(lib.moe_topk_rows(ptr(scores), rows, n, k, ptr(idx), ptr(vals), ev,
                                    _stream(stream)), lib)


def moe_prefetch_experts(cfg, weights: moe_weights, ids, which=3, rows=0, workgroups=256, stream=None,
                         events=None):
    """Read the weights of the experts in ``ids`` (int32 device tensor, any shape;
    e.g. moe_route's topk_idx for the next layer's router on this layer's input)
    of the layer ``weights``: ``which`` bit 0 gate, 1 up, 2 down; ``rows`` > 0: only
    the leading rows of each matrix.  Writes nothing.  ``events``: optional ctypes
    array of 2 hipEvent_t handles."""
    lib = load()
    ev = None if events is None else ctypes.cast(events, ctypes.POINTER(ctypes.c_void_p))
    return _check(lib.moe_prefetch_experts(ctypes.byref(cfg), ctypes.byref(weights), ptr(ids), ids.numel(),
                                           which, rows, workgroups, ev, _stream(stream)), lib)


# ---------------------------------------------------------------------------
# expert groups and the 8-bit operators.  These take typed tensors and check
# their shapes, types and layout against each other; the launch goes to the
# tensors' device.
# ---------------------------------------------------------------------------

def make_groups(n_group=1, topk_group=1, group_top=1, normalise=True) -> moe_groups:
    return moe_groups(n_group, topk_group, group_top, int(normalise))


def _invalid(msg):
    raise MoeError(MOE_ERR_INVALID, "invalid argument: " + msg)


def _call(fn, device, stream, *args):
    """fn(*args, stream) with ``device`` current; the current stream if ``stream`` is None."""
    import torch
    if device.type != "cuda":
        _invalid("tensors must be on the GPU")
    if torch.cuda.current_device() != device.index:
        with torch.cuda.device(device):
            return _check(fn(*args, _stream(stream)))
    return _check(fn(*args, _stream(stream)))


def _row_dtype(t):
    """DTYPE of activation rows: float32, or bf16 (as bfloat16, or its bits)."""
    import torch
    dt = t.dtype
    if dt is torch.float32:
        return 0
    if dt is not torch.bfloat16 and dt is not torch.int16:
        _invalid("expected float32 or bfloat16 rows, got %s" % dt)
    return 1


def _is_f8(t):
    import torch
    return t.dtype is torch.float8_e4m3fn or t.dtype is torch.uint8


def _dense(t, shape, msg, dtype=None):
    if t.shape != shape or not t.is_contiguous() or (dtype is not None and t.dtype is not dtype):
        _invalid("%s must be contiguous %s%s, got %s %s" % (msg, shape, "" if dtype is None else " %s" % dtype,
                                                           tuple(t.shape), t.dtype))


def _same_device(first, *rest):
    d = first.device
    for t in rest:
        if t is not None and t.device != d:
            _invalid("tensors on different devices")


def scale_ld(cols: int) -> int:
    """Bytes of one row's scales (MOE_F8_SCALE_LD)."""
    return (cols + 511) // 512 * 4


def _selection_args(cfg, bias, topk_idx, topk_w):
    import torch
    shape = (cfg.n_tokens, cfg.top_k)
    _dense(topk_idx, shape, "topk_idx", torch.int32)
    _dense(topk_w, shape, "topk_w", torch.float32)
    if bias is not None:
        _dense(bias, (cfg.n_expert,), "bias", torch.float32)


def _rows_match(cfg, x):
    _dense(x, (cfg.n_tokens, cfg.d_model), "x")
    if _row_dtype(x) != cfg.act_dtype:
        _invalid("x is not of the config's activation type")


def _ref(groups):
    return None if groups is None else ctypes.byref(groups)


def _bytes(ws):
    return 0 if ws is None else ws.numel() * ws.element_size()


def moe_select_grouped(cfg, groups, logits, bias, topk_idx, topk_w, stream=None):
    """Selection from ``logits`` [T, E] fp32 with expert groups (``make_groups``; None: flat)."""
    import torch
    _dense(logits, (cfg.n_tokens, cfg.n_expert), "logits", torch.float32)
    _selection_args(cfg, bias, topk_idx, topk_w)
    _same_device(logits, bias, topk_idx, topk_w)
    return _call(load().moe_select_grouped, logits.device, stream, ctypes.byref(cfg), _ref(groups), ptr(logits),
                 ptr(bias), ptr(topk_idx), ptr(topk_w))


def moe_route_grouped(cfg, groups, x, w_router, bias, logits, topk_idx, topk_w, ws, stream=None):
    """Router product and selection with expert groups; ``ws`` is needed only if ``logits`` is None."""
    import torch
    _rows_match(cfg, x)
    _dense(w_router, (cfg.n_expert, cfg.d_model), "w_router", torch.float32)
    if logits is not None:
        _dense(logits, (cfg.n_tokens, cfg.n_expert), "logits", torch.float32)
    _selection_args(cfg, bias, topk_idx, topk_w)
    _same_device(x, w_router, bias, logits, topk_idx, topk_w, ws)
    return _call(load().moe_route_grouped, x.device, stream, ctypes.byref(cfg), _ref(groups), ptr(x), ptr(w_router),
                 ptr(bias), ptr(logits), ptr(topk_idx), ptr(topk_w), ptr(ws), _bytes(ws))


def moe_layer_forward_grouped(cfg, groups, x, weights: moe_weights, y, ws, debug: dict | None = None, stream=None,
                              stage_events=None):
    """moe_layer_forward with expert groups; y float32, or (f8b128 weights) bfloat16."""
    _rows_match(cfg, x)
    _dense(y, (cfg.n_tokens, cfg.d_model), "y")
    _same_device(x, y, ws)
    dbg = _debug_struct(debug, stage_events)
    return _call(load().moe_layer_forward_grouped, x.device, stream, ctypes.byref(cfg), _ref(groups), ptr(x),
                 ctypes.byref(weights), ptr(y), _row_dtype(y), ctypes.byref(dbg) if dbg else None, ptr(ws), _bytes(ws))


def moe_quantize_rows(x, q, scale, stream=None):
    """Rows ``x`` [rows, cols] (float32 or bfloat16, unit column stride) to e4m3 codes ``q`` [rows, cols]
    (float8_e4m3fn or uint8) and e8m0 scale bytes ``scale`` [rows, scale_ld(cols)] uint8."""
    import torch
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        _invalid("x must be [rows, cols] with adjacent columns")
    rows, cols = x.shape
    dt = _row_dtype(x)
    if not _is_f8(q):
        _invalid("q must be float8_e4m3fn or uint8")
    _dense(q, (rows, cols), "q")
    _dense(scale, (rows, scale_ld(cols)), "scale", torch.uint8)
    _same_device(x, q, scale)
    return _call(load().moe_quantize_rows, x.device, stream, ptr(x), dt, rows, cols, x.stride(0) if rows > 1 else -(-cols // 16) * 16,
                 ptr(q), ptr(scale))


def moe_block_matmul_workspace_bytes(x_dtype, m, k) -> int:
    return load().moe_block_matmul_workspace_bytes(DTYPE.get(x_dtype, x_dtype), m, k)


def block_matmul_workspace(x, n):
    """A workspace tensor for moe_block_matmul of rows ``x`` with n weight rows (None if none is needed)."""
    import torch
    del n  # the workspace holds the quantised rows only
    if _is_f8(x):
        return None
    size = moe_block_matmul_workspace_bytes(_row_dtype(x), *x.shape)
    return torch.empty(size, dtype=torch.uint8, device=x.device)


def moe_block_matmul(x, x_scale, w, w_scale, out, ws=None, stream=None):
    """out [m, n] (float32 or bfloat16) = x [m, k] w[n, k]^T with e4m3 operands: ``x`` codes with their
    ``x_scale`` bytes (moe_quantize_rows), or float32 / bfloat16 rows (x_scale None, ``ws`` needed); ``w`` codes
    with ``w_scale`` [ceil(n/128), ceil(k/128)] float32."""
    import torch
    if x.dim() != 2 or w.dim() != 2:
        _invalid("x and w must have two dimensions")
    (m, k), n = x.shape, w.shape[0]
    _dense(x, (m, k), "x")
    if not _is_f8(w):
        _invalid("w must be float8_e4m3fn or uint8")
    _dense(w, (n, k), "w")
    _dense(w_scale, (-(-n // 128), -(-k // 128)), "w_scale", torch.float32)
    _dense(out, (m, n), "out")
    if _is_f8(x):
        xdt = 3
        if x_scale is None:
            _invalid("e4m3 rows need their scale bytes")
        _dense(x_scale, (m, scale_ld(k)), "x_scale", torch.uint8)
    else:
        xdt = _row_dtype(x)
        if x_scale is not None:
            _invalid("x_scale goes with e4m3 rows only")
    _same_device(x, x_scale, w, w_scale, out, ws)
    return _call(load().moe_block_matmul, x.device, stream, ptr(x), xdt, ptr(x_scale), ptr(w), ptr(w_scale), m, n, k,
                 ptr(out), _row_dtype(out), ptr(ws), _bytes(ws))


def workspace(cfg: moe_config, device="cuda"):
    """A workspace tensor of moe_workspace_bytes(cfg) bytes (zero-filled, although
    the library needs no initialisation)."""
    import torch
    n = moe_workspace_bytes(cfg)
    if n == 0:
        raise MoeError(MOE_ERR_INVALID, "invalid config")
    return torch.zeros(n, dtype=torch.uint8, device=device)
