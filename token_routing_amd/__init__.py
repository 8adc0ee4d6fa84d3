"""token_routing_amd -- MoE grouped GEMM on AMD MI355X (gfx950).

A thin ctypes binding over libmoegg.so (``include/moegg.h``).  The functions
here have the C entry points' names and only marshal arguments: every step
of routing and every GEMM runs in the library's HIP kernels.  PyTorch is used
for device memory and the current stream; outputs that the caller does not
pass are allocated with torch.

There is no fallback: if libmoegg.so is missing or fails to load, the first
call raises OSError, and every call raises MoeggError on a non-OK status.
"""

from __future__ import annotations

import ctypes
import os

import torch

PERMUTE_X = 1
PERMUTE_Y = 2
FUSE_MUL_POST = 4
DW_FP32_OUT = 8
GATED_SILU = 32
GATED_GELU = 64
GATED_HALVES = 128

DERR_EXPERT_ID = 1
DERR_M_SIZES = 2
DERR_GATHER = 4
DERR_LOGIT = 8
DERR_RANK = 16

MAX_EXPERTS = 1024
MAX_GROUPS = 16
MAX_TOPK = 64
MAX_LORA_RANK = 256

GATE_SIGMOID = 1
GATE_RENORM = 2

LORA_FP32_GRAD = 1
LORA_ALL_ROWS = 4

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoegg.so")

STATUS = {0: "OK", 1: "EINVAL", 2: "ESHAPE", 3: "EUNSUPPORTED", 4: "EWORKSPACE", 5: "EHIP"}


class MoeggError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)} ({_status_string(status)})")


class MoeggGroup(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("w", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("m", ctypes.c_int32), ("n", ctypes.c_int32), ("k", ctypes.c_int32),
                ("ldx", ctypes.c_int32), ("ldw", ctypes.c_int32), ("ldy", ctypes.c_int32)]


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmoegg.so (raises OSError if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise OSError(f"{path} is not built; run `python -m token_routing_amd.build`")
    lib = ctypes.CDLL(path)
    vp, i32, i64, u32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32,
                             ctypes.c_size_t)
    lib.moegg_status_string.argtypes = [ctypes.c_int]
    lib.moegg_status_string.restype = ctypes.c_char_p
    lib.moegg_version.argtypes = []
    lib.moegg_version.restype = i32
    lib.moegg_route_workspace_bytes.argtypes = [i64, i32]
    lib.moegg_route_workspace_bytes.restype = sz
    lib.moegg_route.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]
    lib.moegg_route.restype = ctypes.c_int
    lib.moegg_route_noalloc.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.moegg_route_noalloc.restype = ctypes.c_int
    lib.moegg_grouped_gemm_fwd.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, u32, vp,
                                           vp, vp]
    lib.moegg_grouped_gemm_fwd.restype = ctypes.c_int
    lib.moegg_grouped_gemm_dX.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, u32, vp, vp,
                                          sz, vp, vp]
    lib.moegg_grouped_gemm_dX.restype = ctypes.c_int
    lib.moegg_grouped_gemm_dX_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    lib.moegg_grouped_gemm_dX_workspace_bytes.restype = sz
    lib.moegg_grouped_gemm_dW.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, u32, vp, vp,
                                          sz, vp, vp]
    lib.moegg_grouped_gemm_dW.restype = ctypes.c_int
    lib.moegg_grouped_gemm_dW_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    lib.moegg_grouped_gemm_dW_workspace_bytes.restype = sz
    lib.moegg_grouped_gemm_dW_gather_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    lib.moegg_grouped_gemm_dW_gather_workspace_bytes.restype = sz
    lib.moegg_grouped_gemm_groups.argtypes = [ctypes.POINTER(MoeggGroup), i32, i32, vp]
    lib.moegg_grouped_gemm_groups.restype = ctypes.c_int
    lib.moegg_combine.argtypes = [vp, vp, vp, i64, i32, i32, i64, u32, vp, vp, vp]
    lib.moegg_combine.restype = ctypes.c_int
    lib.moegg_combine_bwd.argtypes = [vp, vp, vp, vp, i64, i32, i32, i64, vp, vp, vp, vp]
    lib.moegg_combine_bwd.restype = ctypes.c_int
    f32 = ctypes.c_float
    lib.moegg_gate.argtypes = [vp, i32, i64, vp, i64, i32, i32, i32, i32, f32, u32, vp, vp, vp, vp,
                               vp]
    lib.moegg_gate.restype = ctypes.c_int
    lib.moegg_gate_bwd.argtypes = [vp, i32, i64, vp, vp, vp, i64, i32, i32, f32, u32, vp, vp, vp]
    lib.moegg_gate_bwd.restype = ctypes.c_int
    lib.moegg_permute.argtypes = [vp, i32, vp, vp, vp, vp, i64, i32, i32, i32, i64, vp, vp, vp, vp]
    lib.moegg_permute.restype = ctypes.c_int
    lib.moegg_permute_bwd.argtypes = [vp, i32, vp, vp, vp, i64, i32, i32, i64, vp, vp, vp, vp]
    lib.moegg_permute_bwd.restype = ctypes.c_int
    lib.moegg_unpermute.argtypes = [vp, i32, vp, vp, vp, i64, i32, i32, i64, vp, vp, vp]
    lib.moegg_unpermute.restype = ctypes.c_int
    lib.moegg_unpermute_bwd.argtypes = [vp, i32, vp, vp, vp, vp, vp, i64, i32, i32, i32, i64, vp,
                                        vp, vp, vp]
    lib.moegg_unpermute_bwd.restype = ctypes.c_int
    lib.moegg_lora_workspace_bytes.argtypes = [i64, i32, i32, i32, i32]
    lib.moegg_lora_workspace_bytes.restype = sz
    lib.moegg_lora_bwd_workspace_bytes.argtypes = [i64, i32, i32, i32, i32]
    lib.moegg_lora_bwd_workspace_bytes.restype = sz
    lib.moegg_lora_fwd.argtypes = [vp, i64, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, i32,
                                   vp, i64, vp, i64, vp, vp, sz, vp, vp]
    lib.moegg_lora_fwd.restype = ctypes.c_int
    lib.moegg_lora_fwd_all_rows.argtypes = lib.moegg_lora_fwd.argtypes
    lib.moegg_lora_fwd_all_rows.restype = ctypes.c_int
    lib.moegg_lora_bwd.argtypes = [vp, i64, vp, i64, vp, vp, vp, vp, vp, vp, vp, i32, i64, i32,
                                   i32, i32, i32, vp, i64, vp, i64, vp, vp, u32, vp, sz, vp, vp]
    lib.moegg_lora_bwd.restype = ctypes.c_int
    lib.moegg_quant_rows.argtypes = [vp, i32, i64, i64, i32, vp, vp, vp]
    lib.moegg_quant_rows.restype = ctypes.c_int
    lib.moegg_grouped_gemm_i8.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, u32,
                                          vp, vp, vp]
    lib.moegg_grouped_gemm_i8.restype = ctypes.c_int
    lib.moegg_pack8.argtypes = [vp, i32, i64, i64, i32, vp, vp, vp]
    lib.moegg_pack8.restype = ctypes.c_int
    lib.moegg_unpack8.argtypes = [vp, vp, i64, i32, vp, i32, i64, vp]
    lib.moegg_unpack8.restype = ctypes.c_int
    lib.moegg_gated_fwd.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, u32, vp, vp, vp, vp,
                                    vp, sz, vp, vp]
    lib.moegg_gated_fwd.restype = ctypes.c_int
    lib.moegg_gated_fwd_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, u32]
    lib.moegg_gated_fwd_workspace_bytes.restype = sz
    lib.moegg_gated_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, u32, vp,
                                    vp, vp, sz, vp, vp]
    lib.moegg_gated_bwd.restype = ctypes.c_int
    lib.moegg_gated_bwd_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    lib.moegg_gated_bwd_workspace_bytes.restype = sz
    lib.moegg_grouped_gemm_dW_packed.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, u32,
                                                 vp, vp, sz, vp, vp]
    lib.moegg_grouped_gemm_dW_packed.restype = ctypes.c_int
    lib.moegg_grouped_gemm_dW_packed_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, u32]
    lib.moegg_grouped_gemm_dW_packed_workspace_bytes.restype = sz
    _lib = lib
    return lib


def _status_string(status: int) -> str:
    try:
        return load_library().moegg_status_string(status).decode()
    except OSError:
        return "library not loaded"


def _check(status: int, what: str) -> None:
    if status != 0:
        raise MoeggError(status, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _device_tensor(t, dtype, name):
    if t is None:
        return None
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor")
    return t


def route_workspace_bytes(num_slots: int, num_experts: int) -> int:
    return int(load_library().moegg_route_workspace_bytes(num_slots, num_experts))


def moe_route(topk_ids: torch.Tensor, num_experts: int, block_m: int = 128, *, out=None,
              workspace=None, error_flags=None, stream=None):
    """Expert histogram, offsets and stable gather/scatter indices (moegg_route).

    topk_ids: int32 CUDA tensor [T, topk] (or [S]).  Returns a dict of int32
    CUDA tensors m_sizes [E], offsets / padded_offsets / tile_offsets [E+1],
    gather [S], scatter [S].
    """
    lib = load_library()
    ids = _device_tensor(topk_ids, torch.int32, "topk_ids")
    topk = ids.shape[-1] if ids.dim() == 2 else 1
    T = ids.numel() // topk
    S, E = T * topk, int(num_experts)
    dev = ids.device
    if out is None:
        out = {"m_sizes": torch.empty(E, dtype=torch.int32, device=dev),
               "offsets": torch.empty(E + 1, dtype=torch.int32, device=dev),
               "padded_offsets": torch.empty(E + 1, dtype=torch.int32, device=dev),
               "tile_offsets": torch.empty(E + 1, dtype=torch.int32, device=dev),
               "gather": torch.empty(S, dtype=torch.int32, device=dev),
               "scatter": torch.empty(S, dtype=torch.int32, device=dev)}
    need = route_workspace_bytes(S, E)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _check(lib.moegg_route(
        _ptr(ids), T, topk, E, int(block_m), _ptr(out["m_sizes"]), _ptr(out["offsets"]),
        _ptr(out.get("padded_offsets")), _ptr(out.get("tile_offsets")), _ptr(out["gather"]),
        _ptr(out.get("scatter")), _ptr(workspace), workspace.numel(), _ptr(error_flags),
        _stream(stream)), "moegg_route")
    return out


ROUTE_NOALLOC_MAX_BYTES = 1 << 20


def moe_route_noalloc(topk_ids: torch.Tensor, num_experts: int, block_m: int = 128, *, out,
                      error_flags=None, stream=None):
    """moe_route without a workspace (moegg_route_noalloc): the library keeps
    the per-chunk counts in its own static device array, so the call
    allocates nothing.  `out` holds the output tensors, as moe_route returns
    them (m_sizes and offsets required; padded_offsets, tile_offsets and
    scatter optional); calls that overlap on one GPU race."""
    lib = load_library()
    ids = _device_tensor(topk_ids, torch.int32, "topk_ids")
    topk = ids.shape[-1] if ids.dim() == 2 else 1
    T = ids.numel() // topk
    _check(lib.moegg_route_noalloc(
        _ptr(ids), T, topk, int(num_experts), int(block_m), _ptr(out["m_sizes"]),
        _ptr(out["offsets"]), _ptr(out.get("padded_offsets")), _ptr(out.get("tile_offsets")),
        _ptr(out["gather"]), _ptr(out.get("scatter")), _ptr(error_flags), _stream(stream)),
        "moegg_route_noalloc")
    return out


def grouped_gemm_fwd(X, W, m_sizes, gather_idx, topk_weights, topk: int, flags: int, *,
                     Y=None, error_flags=None, stream=None):
    """Y = grouped X W_e^T with the permute_x / permute_y / fuse_mul_post fusions.

    X: bf16 [T, K] (PERMUTE_X) or [T*topk, K]; W: bf16 [E, N, K]; m_sizes int32
    [E]; gather_idx int32 [T*topk]; topk_weights fp32 [T*topk] (slot order).
    Returns Y bf16 [T*topk, N], or [T*topk, N/2] with GATED_SILU (W rows in
    (gate, linear) pairs).
    """
    lib = load_library()
    E, N, K = W.shape
    S = gather_idx.numel() if gather_idx is not None else X.shape[0]
    T = S // topk
    if Y is None:
        Y = torch.empty(S, N // 2 if (flags & GATED_SILU) else N, dtype=torch.bfloat16,
                        device=X.device)
    _check(lib.moegg_grouped_gemm_fwd(
        _ptr(_device_tensor(X, torch.bfloat16, "X")), _ptr(_device_tensor(W, torch.bfloat16, "W")),
        _ptr(_device_tensor(m_sizes, torch.int32, "m_sizes")),
        _ptr(_device_tensor(gather_idx, torch.int32, "gather_idx")),
        _ptr(_device_tensor(topk_weights, torch.float32, "topk_weights")), T, topk, E, N, K,
        int(flags), _ptr(_device_tensor(Y, torch.bfloat16, "Y")), _ptr(error_flags),
        _stream(stream)), "moegg_grouped_gemm_fwd")
    return Y

def dx_workspace_bytes(num_tokens: int, topk: int, num_experts: int, N: int, K: int) -> int:
    """Workspace bytes that let grouped_gemm_dX balance its last round (current device)."""
    return int(load_library().moegg_grouped_gemm_dX_workspace_bytes(num_tokens, topk,
                                                                       num_experts, N, K))


def _workspace(need: int, workspace, device):
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    if workspace is None:
        return None, 0
    workspace = _device_tensor(workspace, torch.uint8, "workspace")
    return workspace, workspace.numel()


def grouped_gemm_dX(dY, W, m_sizes, gather_idx, topk: int, flags: int, *, dX=None,
                    workspace=None, split: bool = True, error_flags=None, stream=None):
    """dX = grouped dY_e W_e; flags are the forward's permute flags. Returns bf16 [S, K].

    split: let the library balance the last round of tiles (fp32 partials in
    `workspace`, a uint8 CUDA tensor of dx_workspace_bytes(...) bytes,
    allocated here when not given).  split=False passes no workspace.
    """
    lib = load_library()
    E, N, K = W.shape
    S = dY.shape[0]
    if dX is None:
        dX = torch.empty(S, K, dtype=torch.bfloat16, device=dY.device)
    need = dx_workspace_bytes(S // topk, topk, E, N, K) if split else 0
    ws, ws_bytes = _workspace(need, workspace if split else None, dY.device)
    _check(lib.moegg_grouped_gemm_dX(
        _ptr(_device_tensor(dY, torch.bfloat16, "dY")), _ptr(_device_tensor(W, torch.bfloat16, "W")),
        _ptr(_device_tensor(m_sizes, torch.int32, "m_sizes")),
        _ptr(_device_tensor(gather_idx, torch.int32, "gather_idx")), S // topk, topk, E, N, K,
        int(flags), _ptr(_device_tensor(dX, torch.bfloat16, "dX")), _ptr(ws), ws_bytes,
        _ptr(error_flags), _stream(stream)), "moegg_grouped_gemm_dX")
    return dX

def dw_workspace_bytes(num_tokens: int, topk: int, num_experts: int, N: int, K: int) -> int:
    """Workspace bytes that let grouped_gemm_dW split hot experts' reductions (0: none)."""
    return int(load_library().moegg_grouped_gemm_dW_workspace_bytes(num_tokens, topk,
                                                                       num_experts, N, K))


def dw_gather_workspace_bytes(num_tokens: int, topk: int, num_experts: int, N: int,
                              K: int) -> int:
    """Workspace bytes with which grouped_gemm_dW under PERMUTE_X also copies X's rows
    into expert order before the reduction (the split area plus S * K * 2)."""
    return int(load_library().moegg_grouped_gemm_dW_gather_workspace_bytes(
        num_tokens, topk, num_experts, N, K))


def grouped_gemm_dW(X, dY, m_sizes, gather_idx, topk: int, flags: int, *, dW=None,
                    workspace=None, split: bool = True, error_flags=None, stream=None):
    """dW[e] = dY_e^T X_e (ragged per expert). Returns [E, N, K] bf16 (fp32 with DW_FP32_OUT).

    split: pass the library a workspace (`workspace`, a uint8 CUDA tensor,
    allocated here when not given: dw_gather_workspace_bytes(...) bytes under
    PERMUTE_X, else dw_workspace_bytes(...)).  It cuts hot experts'
    reductions into chunks with fp32 partials there and, under PERMUTE_X
    with room for them, copies X's rows into expert order first.
    split=False passes no workspace: one launch, rows gathered inside it.
    """
    lib = load_library()
    S, N = dY.shape
    K = X.shape[1]
    E = m_sizes.numel()
    if dW is None:
        dt = torch.float32 if (flags & DW_FP32_OUT) else torch.bfloat16
        dW = torch.empty(E, N, K, dtype=dt, device=dY.device)
    ws_bytes = 0
    if not split:
        workspace = None
    elif workspace is None:
        if flags & PERMUTE_X:
            need = dw_gather_workspace_bytes(S // topk, topk, E, N, K)
        else:
            need = dw_workspace_bytes(S // topk, topk, E, N, K)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dY.device)
    if workspace is not None:
        workspace = _device_tensor(workspace, torch.uint8, "workspace")
        ws_bytes = workspace.numel()
    _check(lib.moegg_grouped_gemm_dW(
        _ptr(_device_tensor(X, torch.bfloat16, "X")), _ptr(_device_tensor(dY, torch.bfloat16, "dY")),
        _ptr(_device_tensor(m_sizes, torch.int32, "m_sizes")),
        _ptr(_device_tensor(gather_idx, torch.int32, "gather_idx")), S // topk, topk, E, N, K,
        int(flags), _ptr(dW), _ptr(workspace), ws_bytes, _ptr(error_flags), _stream(stream)),
        "moegg_grouped_gemm_dW")
    return dW


def grouped_gemm_groups(groups, trans_b: int = 0, *, outputs=None, stream=None):
    """Independent GEMMs y_g = x_g @ w_g in one launch.

    groups: list of (x [m, k], w [k, n] (trans_b=0) or [n, k] (trans_b=1)) bf16
    CUDA tensors.  Returns the list of y [m, n] bf16.
    """
    lib = load_library()
    if not 1 <= len(groups) <= MAX_GROUPS:
        raise ValueError("1..16 groups")
    arr = (MoeggGroup * len(groups))()
    ys = []
    for i, (x, w) in enumerate(groups):
        for t, name in ((x, "x"), (w, "w")):
            if not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 2 or t.stride(1) != 1:
                raise ValueError(f"group {i}: {name} must be a row-major bf16 CUDA matrix")
        m, k = x.shape
        n = w.shape[0] if trans_b else w.shape[1]
        y = outputs[i] if outputs is not None else torch.empty(m, n, dtype=torch.bfloat16,
                                                               device=x.device)
        ys.append(y)
        arr[i] = MoeggGroup(x.data_ptr(), w.data_ptr(), y.data_ptr(), m, n, k, x.stride(0),
                            w.stride(0), y.stride(0))
    _check(lib.moegg_grouped_gemm_groups(arr, len(groups), int(trans_b), _stream(stream)),
           "moegg_grouped_gemm_groups")
    return ys


COMBINE_FP32_OUT = 16


def combine(Y, topk: int, scatter_idx=None, topk_weights=None, *, num_tokens=None,
            fp32_out: bool = False, out=None, error_flags=None, stream=None):
    """Top-k combine (moegg_combine): out[t] = sum_j w[t*k+j] * Y[row(t*k+j)].

    Y: bf16 [rows, N]; scatter_idx: int32 [T*k] (Y in expert-sorted order) or
    None (Y in slot order); topk_weights: float32 [T*k] or None (weight 1).
    Returns out [T, N], bf16 (fp32 with fp32_out).
    """
    lib = load_library()
    Y = _device_tensor(Y, torch.bfloat16, "Y")
    scatter_idx = _device_tensor(scatter_idx, torch.int32, "scatter_idx")
    topk_weights = _device_tensor(topk_weights, torch.float32, "topk_weights")
    S = scatter_idx.numel() if scatter_idx is not None else Y.shape[0]
    T = S // topk if num_tokens is None else int(num_tokens)
    N = Y.shape[1]
    if out is None:
        out = torch.empty(T, N, dtype=torch.float32 if fp32_out else torch.bfloat16,
                          device=Y.device)
    _check(lib.moegg_combine(_ptr(Y), _ptr(scatter_idx), _ptr(topk_weights), T, topk, N,
                             Y.shape[0], COMBINE_FP32_OUT if fp32_out else 0, _ptr(out),
                             _ptr(error_flags), _stream(stream)), "moegg_combine")
    return out


def combine_bwd(dOut, Y, topk: int, scatter_idx=None, topk_weights=None, *, want_dw=True,
                dY=None, dw=None, error_flags=None, stream=None):
    """Backward of combine (moegg_combine_bwd): returns (dY bf16 [rows, N], dw float32 [T*k]
    or None).  Y (the forward input) is read only for dw."""
    lib = load_library()
    dOut = _device_tensor(dOut, torch.bfloat16, "dOut")
    Y = _device_tensor(Y, torch.bfloat16, "Y")
    scatter_idx = _device_tensor(scatter_idx, torch.int32, "scatter_idx")
    topk_weights = _device_tensor(topk_weights, torch.float32, "topk_weights")
    T, N = dOut.shape
    rows = Y.shape[0] if Y is not None else T * topk
    if dY is None:
        dY = torch.empty(rows, N, dtype=torch.bfloat16, device=dOut.device)
    if want_dw and dw is None:
        dw = torch.empty(T * topk, dtype=torch.float32, device=dOut.device)
    _check(lib.moegg_combine_bwd(_ptr(dOut), _ptr(Y), _ptr(scatter_idx), _ptr(topk_weights), T,
                                 topk, N, rows, _ptr(dY), _ptr(dw if want_dw else None),
                                 _ptr(error_flags), _stream(stream)), "moegg_combine_bwd")
    return dY, (dw if want_dw else None)


# The entry points below check shapes and devices as well, run on the device
# that holds their tensors, and allocate outputs (and workspaces) on the stream
# that they launch on.

def _run(device, stream, call):
    """call(stream handle) with `device` current and, when given, `stream` current."""
    index = device.index
    if index is None or device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, not on {device}")
    if stream is None:
        if index == torch.cuda.current_device():
            return call(torch._C._cuda_getCurrentRawStream(index))
        with torch.cuda.device(index):
            return call(torch._C._cuda_getCurrentRawStream(index))
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    with torch.cuda.stream(stream):        # makes the stream's device current as well
        return call(stream.cuda_stream)


def _dtype_code(t, name):
    code = DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, not {t.dtype}")
    return code


def _refuse(t, name, dtype, shape, index):
    if t.dtype != dtype or t.get_device() != index:
        raise ValueError(f"{name} must be a {dtype} tensor on cuda:{index}, not {t.dtype} on "
                         f"{t.device}")
    raise ValueError(f"{name} must be contiguous of shape {tuple(shape)}, not {tuple(t.shape)} "
                     f"with strides {t.stride()}")


def _arg(t, name, dtype, shape, index):
    """Address of a contiguous tensor of this type and shape on GPU `index`."""
    if t is None:
        return None
    if (t.dtype is dtype and t.shape == shape and t.get_device() == index
            and t.is_contiguous()):
        return t.data_ptr()
    _refuse(t, name, dtype, shape, index)


def _out(t, name, dtype, shape, device):
    """An output tensor, allocated unless given, and its address."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=device)
        return t, t.data_ptr()
    return t, _arg(t, name, dtype, shape, device.index)


def _slots_arg(t, name, dtype, slots, index):
    """Address of a contiguous per-slot tensor: [slots] or [T, topk]."""
    if t is None:
        return None
    if (t.dtype is dtype and t.numel() == slots and t.get_device() == index
            and t.is_contiguous()):
        return t.data_ptr()
    _refuse(t, name, dtype, (slots,), index)


def _dw_out(dw, wanted, slots, device):
    """The slots' weight gradient and its address, or None twice."""
    if not wanted:
        return None, None
    if dw is None:
        return _out(None, "dw", torch.float32, (slots,), device)
    return dw, _slots_arg(dw, "dw", torch.float32, slots, device.index)


def _rows_arg(t, name, dtype, shape, index):
    """Address and row stride of a matrix whose rows are contiguous."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index:
        _refuse(t, name, dtype, shape, index)
    rows, cols = shape
    if t.is_contiguous():
        return t.data_ptr(), cols
    ld, step = t.stride()
    if rows == 1:
        ld = max(ld, cols)
    if (step != 1 and cols > 1) or ld < cols:
        raise ValueError(f"{name} must have contiguous rows that do not overlap, not strides "
                         f"{t.stride()}")
    return t.data_ptr(), ld


def _flag_arg(t, index):
    return None if t is None else _slots_arg(t, "error_flags", torch.int32, 1, index)


def moe_gate(logits, topk: int, *, bias=None, n_groups: int = 1, topk_groups: int = 1,
             scale: float = 1.0, sigmoid: bool = False, renorm: bool = False,
             want_scores: bool = False, ids=None, weights=None, scores=None, error_flags=None,
             stream=None):
    """Top-k expert ids and weights from router logits (moegg_gate).

    logits: [T, E] bf16, fp16 or fp32, rows contiguous (any row stride); bias:
    fp32 [E] added for the pick alone.  sigmoid / renorm / scale and the groups
    as in the header.  Returns (ids int32 [T, topk], weights fp32 [T, topk],
    scores fp32 [T, E] or None).  ids feeds moe_route, weights (flattened) the
    GEMMs and combines; places without an expert hold id -1 and weight 0.
    """
    lib = load_library()
    dev = logits.device
    index = dev.index
    T, E = logits.shape
    ptr, ld = _rows_arg(logits, "logits", logits.dtype, (T, E), index)
    code = _dtype_code(logits, "logits")
    topk = int(topk)

    def call(stream_ptr):
        i, i_ptr = _out(ids, "ids", torch.int32, (T, topk), dev)
        w, w_ptr = _out(weights, "weights", torch.float32, (T, topk), dev)
        s = s_ptr = None
        if want_scores or scores is not None:
            s, s_ptr = _out(scores, "scores", torch.float32, (T, E), dev)
        _check(lib.moegg_gate(
            ptr, code, ld, _arg(bias, "bias", torch.float32, (E,), index), T, E, topk, int(n_groups),
            int(topk_groups), float(scale),
            (GATE_SIGMOID if sigmoid else 0) | (GATE_RENORM if renorm else 0),
            i_ptr, w_ptr, s_ptr, _flag_arg(error_flags, index), stream_ptr), "moegg_gate")
        return i, w, s

    if topk < 1 or topk > E:
        raise ValueError(f"topk must be between 1 and {E}")
    return _run(dev, stream, call)


def moe_gate_bwd(logits, ids, dweights, *, dscores=None, scale: float = 1.0,
                 sigmoid: bool = False, renorm: bool = False, dlogits=None, error_flags=None,
                 stream=None):
    """Gradient of moe_gate's weights (and scores, with dscores) in the logits
    (moegg_gate_bwd), for the ids it picked.  Returns dlogits [T, E] of the
    logits' type."""
    lib = load_library()
    dev = logits.device
    index = dev.index
    T, E = logits.shape
    ptr, ld = _rows_arg(logits, "logits", logits.dtype, (T, E), index)
    code = _dtype_code(logits, "logits")
    topk = ids.shape[-1]

    def call(stream_ptr):
        d, d_ptr = _out(dlogits, "dlogits", logits.dtype, (T, E), dev)
        _check(lib.moegg_gate_bwd(
            ptr, code, ld, _arg(ids, "ids", torch.int32, (T, topk), index),
            _arg(dweights, "dweights", torch.float32, (T, topk), index),
            _arg(dscores, "dscores", torch.float32, (T, E), index), T, E, topk, float(scale),
            (GATE_SIGMOID if sigmoid else 0) | (GATE_RENORM if renorm else 0),
            d_ptr, _flag_arg(error_flags, index),
            stream_ptr), "moegg_gate_bwd")
        return d

    return _run(dev, stream, call)


def permute(X, scatter_idx, topk: int, topk_weights=None, *, offsets=None, padded_offsets=None,
            block_m=None, rows=None, Xs=None, row_map=None, error_flags=None, stream=None):
    """Token rows into expert order (moegg_permute): Xs[row(s)] = w[s] * X[t].

    X: [T, K] bf16, fp16 or fp32; scatter_idx int32 [T*topk] (moe_route);
    topk_weights fp32 [T*topk] or None.  With offsets and padded_offsets
    (moe_route) the block-padded layout, pad rows cleared; a new Xs then needs
    `rows` or the block_m that was routed with.  Returns (Xs [rows, K],
    row_map int32 [T*topk]); rows past the last expert's are left as they were
    (a new Xs leaves them uninitialised).  Without padding the map is
    scatter_idx itself, its buffer and its entries as they are, unless a
    row_map is given to write it to: give one where scatter_idx is written again
    before the backward, or may hold rows past Xs (a written map has -1 there).
    """
    lib = load_library()
    dev = X.device
    index = dev.index
    T, K = X.shape
    S = T * topk
    code = _dtype_code(X, "X")
    E = 0 if offsets is None else offsets.numel() - 1
    if Xs is not None:
        rows = Xs.shape[0]
    elif rows is None:
        if padded_offsets is not None and block_m is None:
            raise ValueError("the padded layout needs rows, block_m or Xs")
        rows = S + (E * (int(block_m) - 1) if padded_offsets is not None else 0)

    def call(stream_ptr):
        out, out_ptr = _out(Xs, "Xs", X.dtype, (rows, K), dev)
        if row_map is None and padded_offsets is None:
            m, m_ptr = scatter_idx, None
        else:
            m, m_ptr = _out(row_map, "row_map", torch.int32, (S,), dev)
        _check(lib.moegg_permute(
            _arg(X, "X", X.dtype, (T, K), index), code,
            _slots_arg(scatter_idx, "scatter_idx", torch.int32, S, index),
            _slots_arg(topk_weights, "topk_weights", torch.float32, S, index),
            _arg(offsets, "offsets", torch.int32, (E + 1,), index),
            _arg(padded_offsets, "padded_offsets", torch.int32, (E + 1,), index), T, topk, E, K,
            rows, out_ptr, m_ptr, _flag_arg(error_flags, index), stream_ptr), "moegg_permute")
        return out, m

    return _run(dev, stream, call)


def permute_bwd(dXs, X, topk: int, row_map, topk_weights=None, *, want_dw: bool = True, dX=None,
                dw=None, error_flags=None, stream=None):
    """Gradient of permute (moegg_permute_bwd): (dX [T, K], dw fp32 [T*topk] or None).
    X (the forward's input) is read only for dw; dX may be X."""
    lib = load_library()
    dev = dXs.device
    index = dev.index
    rows, K = dXs.shape
    S = row_map.numel()
    T = S // topk
    code = _dtype_code(dXs, "dXs")

    def call(stream_ptr):
        out, out_ptr = _out(dX, "dX", dXs.dtype, (T, K), dev)
        g, g_ptr = _dw_out(dw, want_dw, S, dev)
        _check(lib.moegg_permute_bwd(
            _arg(dXs, "dXs", dXs.dtype, (rows, K), index), code,
            _arg(X, "X", dXs.dtype, (T, K), index),
            _slots_arg(row_map, "row_map", torch.int32, T * topk, index),
            _slots_arg(topk_weights, "topk_weights", torch.float32, S, index), T, topk, K, rows,
            out_ptr, g_ptr, _flag_arg(error_flags, index), stream_ptr), "moegg_permute_bwd")
        return out, g

    return _run(dev, stream, call)


def unpermute(Y, topk: int, row_map, topk_weights=None, *, base=None, out=None, error_flags=None,
              stream=None):
    """Expert-ordered rows back to token order (moegg_unpermute):
    out[t] = base[t] + sum_j w[s] * Y[row_map[s]].  base may be out."""
    lib = load_library()
    dev = Y.device
    index = dev.index
    rows, K = Y.shape
    S = row_map.numel()
    T = S // topk
    code = _dtype_code(Y, "Y")

    def call(stream_ptr):
        o, o_ptr = _out(out, "out", Y.dtype, (T, K), dev)
        _check(lib.moegg_unpermute(
            _arg(Y, "Y", Y.dtype, (rows, K), index), code,
            _slots_arg(row_map, "row_map", torch.int32, T * topk, index),
            _slots_arg(topk_weights, "topk_weights", torch.float32, S, index),
            _arg(base, "base", Y.dtype, (T, K), index), T, topk, K, rows,
            o_ptr, _flag_arg(error_flags, index), stream_ptr), "moegg_unpermute")
        return o

    return _run(dev, stream, call)


def unpermute_bwd(dOut, Y, topk: int, row_map, topk_weights=None, *, offsets=None,
                  padded_offsets=None, rows=None, want_dw: bool = True, dY=None, dw=None,
                  error_flags=None, stream=None):
    """Gradient of unpermute (moegg_unpermute_bwd): (dY [rows, K], dw fp32 [T*topk] or None).

    Y (the forward's input) is read only for dw and may be None without it
    (`rows` or dY then say how many rows dY has); dY may be Y.  With offsets and
    padded_offsets the pad rows of dY are cleared; rows no slot maps to are
    left as they were.
    """
    lib = load_library()
    dev = dOut.device
    index = dev.index
    T, K = dOut.shape
    S = T * topk
    code = _dtype_code(dOut, "dOut")
    E = 0 if offsets is None else offsets.numel() - 1
    if dY is not None:
        rows = dY.shape[0]
    elif Y is not None:
        rows = Y.shape[0]
    elif rows is None:
        raise ValueError("without Y and dY, rows is needed")

    def call(stream_ptr):
        out, out_ptr = _out(dY, "dY", dOut.dtype, (rows, K), dev)
        g, g_ptr = _dw_out(dw, want_dw, S, dev)
        _check(lib.moegg_unpermute_bwd(
            _arg(dOut, "dOut", dOut.dtype, (T, K), index), code,
            _arg(Y, "Y", dOut.dtype, (rows, K), index),
            _slots_arg(row_map, "row_map", torch.int32, S, index),
            _slots_arg(topk_weights, "topk_weights", torch.float32, S, index),
            _arg(offsets, "offsets", torch.int32, (E + 1,), index),
            _arg(padded_offsets, "padded_offsets", torch.int32, (E + 1,), index), T, topk, E, K,
            rows, out_ptr, g_ptr, _flag_arg(error_flags, index), stream_ptr),
            "moegg_unpermute_bwd")
        return out, g

    return _run(dev, stream, call)


def lora_workspace_bytes(num_rows: int, num_adapters: int, R: int, K: int, N: int) -> int:
    """Workspace bytes of lora_fwd."""
    return int(load_library().moegg_lora_workspace_bytes(num_rows, num_adapters, R, K, N))


def lora_bwd_workspace_bytes(num_rows: int, num_adapters: int, R: int, K: int, N: int) -> int:
    """Workspace bytes of lora_bwd."""
    return int(load_library().moegg_lora_bwd_workspace_bytes(num_rows, num_adapters, R, K, N))


def _workspace_arg(workspace, need, device):
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        return workspace, workspace.data_ptr()
    return workspace, _slots_arg(workspace, "workspace", torch.uint8, workspace.numel(),
                                 device.index)


def lora_fwd(X, A, B, m_sizes, gather_idx=None, *, ranks=None, scales=None, base=None, Y=None,
             H=None, want_h: bool = False, workspace=None, error_flags=None, stream=None):
    """Low-rank adapters of many requests on a shared projection's output
    (moegg_lora_fwd): Y[i] = base[i] + scales[a] * (X[i] A_a^T) B_a^T.

    X: [T, K] bf16 or fp16, A: [L, R, K], B: [L, N, R]; m_sizes int32 [L] and
    gather_idx int32 [T] from moe_route over the rows' adapter ids (None: rows
    are in adapter order already); ranks int32 [L] or None (R); scales fp32 [L]
    or None (1).  base [T, N]: the projection's output; None adds to Y in
    place.  X, base and Y may have any row stride.  A row without an adapter
    (an id that moe_route dropped) gets its base row in a new Y, and keeps what
    a given Y holds.  Returns (Y, H): H is fp32 [T, R] in adapter order for
    lora_bwd, None unless given or want_h (rows at positions past the last
    adapter's are left as they were).
    """
    lib = load_library()
    dev = X.device
    index = dev.index
    L, R, K = A.shape
    T, N = X.shape[0], B.shape[1]
    dt = X.dtype
    code = _dtype_code(X, "X")
    if base is None and Y is None:
        raise ValueError("base or Y is needed")

    def call(stream_ptr):
        y = torch.empty(T, N, dtype=dt, device=dev) if Y is None else Y
        h = h_ptr = None
        if want_h or H is not None:
            h, h_ptr = _out(H, "H", torch.float32, (T, R), dev)
        need = lib.moegg_lora_workspace_bytes(T, L, R, K, N)
        ws, ws_ptr = _workspace_arg(workspace, need, dev)
        x_ptr, ldx = _rows_arg(X, "X", dt, (T, K), index)
        y_ptr, ldy = _rows_arg(y, "Y", dt, (T, N), index)
        b_ptr, ldb = (None, ldy) if base is None else _rows_arg(base, "base", dt, (T, N), index)
        forward = lib.moegg_lora_fwd_all_rows if Y is None else lib.moegg_lora_fwd
        _check(forward(
            x_ptr, ldx, _arg(A, "A", dt, (L, R, K), index), _arg(B, "B", dt, (L, N, R), index),
            _arg(m_sizes, "m_sizes", torch.int32, (L,), index),
            _arg(gather_idx, "gather_idx", torch.int32, (T,), index),
            _arg(ranks, "ranks", torch.int32, (L,), index),
            _arg(scales, "scales", torch.float32, (L,), index), code, T, L, R, K, N, b_ptr, ldb,
            y_ptr, ldy, h_ptr, ws_ptr, ws.numel(),
            _flag_arg(error_flags, index), stream_ptr), "moegg_lora_fwd")
        return y, h

    return _run(dev, stream, call)


def lora_bwd(X, dY, A, B, H, m_sizes, gather_idx=None, *, ranks=None, scales=None, base=None,
             dX=None, dA=None, dB=None, want_dx: bool = True, want_weights: bool = True,
             fp32_grads: bool = False, workspace=None, error_flags=None, stream=None):
    """Gradients of lora_fwd (moegg_lora_bwd): (dX [T, K], dA [L, R, K], dB [L, N, R]).

    base [T, K]: the shared projection's input gradient, which dX adds to; None
    adds to the dX given.  Rows without an adapter get their base row in a new
    dX, and keep what a given dX holds.  A given dX may not overlap X or dY
    unless want_weights=False.  want_dx=False or want_weights=False leave dX or dA
    and dB out (None in their place).  fp32_grads writes dA and dB in fp32.
    """
    lib = load_library()
    dev = dY.device
    index = dev.index
    L, R, K = A.shape
    T, N = dY.shape
    dt = dY.dtype
    code = _dtype_code(dY, "dY")
    if want_dx and base is None and dX is None:
        raise ValueError("base or dX is needed (or want_dx=False)")
    wt = torch.float32 if fp32_grads else dt

    def call(stream_ptr):
        dx, x_ptr, ldx, dx_ptr, lddx, b_ptr, ldb = None, None, K, None, K, None, K
        da = db = da_ptr = db_ptr = None
        if want_dx:
            dx = torch.empty(T, K, dtype=dt, device=dev) if dX is None else dX
            dx_ptr, lddx = _rows_arg(dx, "dX", dt, (T, K), index)
            if base is not None:
                b_ptr, ldb = _rows_arg(base, "base", dt, (T, K), index)
        if want_weights:
            da, da_ptr = _out(dA, "dA", wt, (L, R, K), dev)
            db, db_ptr = _out(dB, "dB", wt, (L, N, R), dev)
            x_ptr, ldx = _rows_arg(X, "X", dt, (T, K), index)
        dy_ptr, lddy = _rows_arg(dY, "dY", dt, (T, N), index)
        need = lib.moegg_lora_bwd_workspace_bytes(T, L, R, K, N)
        ws, ws_ptr = _workspace_arg(workspace, need, dev)
        _check(lib.moegg_lora_bwd(
            x_ptr, ldx, dy_ptr, lddy, _arg(A, "A", dt, (L, R, K), index),
            _arg(B, "B", dt, (L, N, R), index),
            _arg(H, "H", torch.float32, (T, R), index) if want_weights else None,
            _arg(m_sizes, "m_sizes", torch.int32, (L,), index),
            _arg(gather_idx, "gather_idx", torch.int32, (T,), index),
            _arg(ranks, "ranks", torch.int32, (L,), index),
            _arg(scales, "scales", torch.float32, (L,), index), code, T, L, R, K, N, b_ptr, ldb,
            dx_ptr, lddx, da_ptr, db_ptr,
            (LORA_FP32_GRAD if fp32_grads else 0) | (LORA_ALL_ROWS if dX is None else 0),
            ws_ptr, ws.numel(), _flag_arg(error_flags, index), stream_ptr), "moegg_lora_bwd")
        return dx, da, db

    return _run(dev, stream, call)


PACK_BLOCK = 32
QUANT_MAX_ROWS = (1 << 24) - 1      # of one moegg_quant_rows


def quant_rows(X, *, Q=None, scales=None, stream=None):
    """Rows in 8-bit integers with a scale each (moegg_quant_rows).

    X: [..., K] bf16, fp16 or fp32; a matrix may have any row stride, more
    dimensions (weights [E, N, K]) are contiguous.  Returns (Q int8 [..., Kq],
    scales fp32 [...]) with Kq = K rounded up to a multiple of 16, the columns
    from K on zero: what grouped_gemm_i8 takes for tokens and for weights.  Rows
    past QUANT_MAX_ROWS take a launch for each so many.
    """
    lib = load_library()
    dev = X.device
    index = dev.index
    lead, K = X.shape[:-1], X.shape[-1]
    rows = lead.numel()
    code = _dtype_code(X, "X")
    if X.dim() == 2:
        x_ptr, ldx = _rows_arg(X, "X", X.dtype, (rows, K), index)
    else:
        x_ptr, ldx = _arg(X, "X", X.dtype, X.shape, index), K

    def call(stream_ptr):
        q, q_ptr = _out(Q, "Q", torch.int8, lead + ((K + 15) // 16 * 16,), dev)
        s, s_ptr = _out(scales, "scales", torch.float32, lead, dev)
        if rows <= QUANT_MAX_ROWS:
            _check(lib.moegg_quant_rows(x_ptr, code, ldx, rows, K, q_ptr, s_ptr, stream_ptr),
                   "moegg_quant_rows")
            return q, s
        size = X.element_size()
        spans = sorted([(x_ptr, ((rows - 1) * ldx + K) * size), (q_ptr, q.numel()),
                        (s_ptr, 4 * rows)])
        if any(a + n > b for (a, n), (b, _) in zip(spans, spans[1:])):
            raise ValueError("Q and scales must overlap neither X nor each other")
        for at in range(0, rows, QUANT_MAX_ROWS):
            _check(lib.moegg_quant_rows(x_ptr + at * ldx * size, code, ldx,
                                        min(QUANT_MAX_ROWS, rows - at), K,
                                        q_ptr + at * q.shape[-1], s_ptr + 4 * at, stream_ptr),
                   "moegg_quant_rows")
        return q, s

    return _run(dev, stream, call)


def grouped_gemm_i8(Xq, x_scales, Wq, w_scales, m_sizes, gather_idx, topk_weights, topk: int,
                    flags: int, *, Y=None, error_flags=None, stream=None):
    """grouped_gemm_fwd on 8-bit integers with a scale for each token and output channel
    (moegg_grouped_gemm_i8).

    Xq int8 [T, Kq] (PERMUTE_X) or [T*topk, Kq] and x_scales fp32, Wq int8 [E, N, Kq]
    and w_scales fp32 [E, N], as quant_rows gives them; the others as in
    grouped_gemm_fwd.  flags: also GATED_SILU or GATED_GELU, with GATED_HALVES
    for W's gate rows first instead of (gate, linear) pairs.  Returns Y bf16
    [T*topk, N], [T*topk, N/2] when gated.
    """
    lib = load_library()
    dev = Xq.device
    index = dev.index
    E, N, K = Wq.shape
    S = gather_idx.numel() if gather_idx is not None else Xq.shape[0]
    T = S // topk
    x_rows = T if flags & PERMUTE_X else T * topk
    cols = N // 2 if flags & (GATED_SILU | GATED_GELU) else N

    def call(stream_ptr):
        y, y_ptr = _out(Y, "Y", torch.bfloat16, (T * topk, cols), dev)
        _check(lib.moegg_grouped_gemm_i8(
            _arg(Xq, "Xq", torch.int8, (x_rows, K), index),
            _slots_arg(x_scales, "x_scales", torch.float32, x_rows, index),
            _arg(Wq, "Wq", torch.int8, (E, N, K), index),
            _arg(w_scales, "w_scales", torch.float32, (E, N), index),
            _arg(m_sizes, "m_sizes", torch.int32, (E,), index),
            _slots_arg(gather_idx, "gather_idx", torch.int32, T * topk, index),
            _slots_arg(topk_weights, "topk_weights", torch.float32, T * topk, index), T, topk, E, N,
            K, int(flags), y_ptr, _flag_arg(error_flags, index), stream_ptr),
            "moegg_grouped_gemm_i8")
        return y

    return _run(dev, stream, call)


def _packed_shapes(rows, cols):
    padded = (cols + PACK_BLOCK - 1) // PACK_BLOCK * PACK_BLOCK
    return (rows, padded), (rows, padded // PACK_BLOCK)


def pack8(X, *, Q=None, scales=None, stream=None):
    """An activation in 8.25 bits a value (moegg_pack8): blocks of 32 neighbours
    of a row share a power of two.

    X: [rows, cols] bf16, fp16 or fp32, any row stride.  Returns (Q int8 [rows,
    Cp], scales uint8 [rows, Cp / 32]), Cp = cols rounded up to a multiple of 32.
    """
    lib = load_library()
    dev = X.device
    index = dev.index
    rows, cols = X.shape
    code = _dtype_code(X, "X")
    x_ptr, ldx = _rows_arg(X, "X", X.dtype, (rows, cols), index)
    q_shape, s_shape = _packed_shapes(rows, cols)

    def call(stream_ptr):
        q, q_ptr = _out(Q, "Q", torch.int8, q_shape, dev)
        s, s_ptr = _out(scales, "scales", torch.uint8, s_shape, dev)
        _check(lib.moegg_pack8(x_ptr, code, ldx, rows, cols, q_ptr, s_ptr, stream_ptr),
               "moegg_pack8")
        return q, s

    return _run(dev, stream, call)


def unpack8(Q, scales, cols: int, dtype=torch.bfloat16, *, X=None, stream=None):
    """The values of pack8's (Q, scales) (moegg_unpack8): [rows, cols] of `dtype`,
    exact in bf16 and fp32.  A given X may have any row stride."""
    lib = load_library()
    dev = Q.device
    index = dev.index
    rows, cols = Q.shape[0], int(cols)
    dtype = dtype if X is None else X.dtype
    q_shape, s_shape = _packed_shapes(rows, cols)

    def call(stream_ptr):
        x = torch.empty(rows, cols, dtype=dtype, device=dev) if X is None else X
        x_ptr, ldx = _rows_arg(x, "X", dtype, (rows, cols), index)
        _check(lib.moegg_unpack8(
            _arg(Q, "Q", torch.int8, q_shape, index),
            _arg(scales, "scales", torch.uint8, s_shape, index), rows, cols, x_ptr,
            _dtype_code(x, "X"), ldx, stream_ptr), "moegg_unpack8")
        return x

    return _run(dev, stream, call)


def _chunked(cols, *tensors):
    """Whether rows of `cols` elements of 16 bits are whole, aligned 16-byte chunks."""
    return cols % 8 == 0 and all(t.data_ptr() % 16 == 0 for t in tensors)


def _optional_workspace(workspace, need, device):
    """(workspace, address, bytes): allocated when needed and not given."""
    if workspace is None and need == 0:
        return None, None, 0
    workspace, ptr = _workspace_arg(workspace, need, device)
    return workspace, ptr, workspace.numel()


def gated_fwd(X, W, m_sizes, gather_idx, topk: int, flags: int, *, keep=None, H=None, kept=None,
              workspace=None, error_flags=None, stream=None):
    """The gated block's first half with what its backward needs (moegg_gated_fwd):
    H = act(g) * u of the grouped product X W_e^T, gate columns g and linear u.

    X: bf16 [T, K] (PERMUTE_X) or [T*topk, K]; W: bf16 [E, 2 I, K], its rows in
    (gate, linear) pairs or with GATED_HALVES the I gate rows first; flags:
    PERMUTE_X, GATED_SILU or GATED_GELU, GATED_HALVES.  keep: None, "bf16" (A =
    X W_e^T, [T*topk, 2 I]) or "packed" (g and u in 8.25 bits a value: codes int8
    [T*topk, 2 Ip] and scales uint8 [T*topk, 2 Ip / 32], the gate's and then the
    linear part's, Ip = I rounded up to a multiple of 32).  Returns (H bf16
    [T*topk, I], kept): the A, the pair, or None; `kept` may give its buffers.
    """
    lib = load_library()
    dev = X.device
    index = dev.index
    E, N, K = W.shape
    S = gather_idx.numel() if gather_idx is not None else X.shape[0]
    T = S // topk
    S, I = T * topk, N // 2
    if N % 2:
        raise ValueError(f"W must have an even number of rows per expert, not {N}")
    if keep not in (None, "bf16", "packed"):
        raise ValueError(f"keep must be None, 'bf16' or 'packed', not {keep!r}")
    if kept is not None and (keep is None or isinstance(kept, torch.Tensor) != (keep == "bf16")):
        raise ValueError(f"kept does not fit keep={keep!r}: a tensor for 'bf16', a pair for 'packed'")
    padded = (I + PACK_BLOCK - 1) // PACK_BLOCK * PACK_BLOCK

    def call(stream_ptr):
        h, h_ptr = _out(H, "H", torch.bfloat16, (S, I), dev)
        out = a_ptr = q_ptr = s_ptr = None
        if keep == "bf16":
            out, a_ptr = _out(kept, "kept", torch.bfloat16, (S, N), dev)
        elif keep == "packed":
            q, s = (None, None) if kept is None else kept
            q, q_ptr = _out(q, "kept[0]", torch.int8, (S, 2 * padded), dev)
            s, s_ptr = _out(s, "kept[1]", torch.uint8, (S, 2 * padded // PACK_BLOCK), dev)
            out = (q, s)
        need = 0 if _chunked(K, X, W) else lib.moegg_gated_fwd_workspace_bytes(T, topk, E, I, K,
                                                                               int(flags))
        ws, ws_ptr, ws_bytes = _optional_workspace(workspace, need, dev)
        _check(lib.moegg_gated_fwd(
            _arg(X, "X", torch.bfloat16, (T if flags & PERMUTE_X else S, K), index),
            _arg(W, "W", torch.bfloat16, (E, N, K), index),
            _arg(m_sizes, "m_sizes", torch.int32, (E,), index),
            _slots_arg(gather_idx, "gather_idx", torch.int32, S, index), T, topk, E, I, K,
            int(flags), h_ptr, a_ptr, q_ptr, s_ptr, ws_ptr, ws_bytes,
            _flag_arg(error_flags, index), stream_ptr), "moegg_gated_fwd")
        return h, out

    return _run(dev, stream, call)


def gated_bwd(dY, W, kept, m_sizes, gather_idx, topk: int, flags: int, *, want_h: bool = True,
              dA=None, H=None, workspace=None, error_flags=None, stream=None):
    """From the down projection's output gradient to that of gated_fwd's A (moegg_gated_bwd).

    dY: bf16 [T*topk, N] (slot order with PERMUTE_Y, the flag of the down
    projection's forward); W: bf16 [E, N, I], the down projection's weight;
    kept: what gated_fwd returned, A or the packed pair; the other flags as
    there.  Returns (dA bf16 [T*topk, 2 I], the dY of the first projections'
    grouped_gemm_dX and grouped_gemm_dW; H bf16 [T*topk, I] from the kept values,
    the X of the down projection's grouped_gemm_dW, or None).  dA may be A.
    """
    lib = load_library()
    dev = dY.device
    index = dev.index
    E, N, I = W.shape
    T = dY.shape[0] // topk
    S = T * topk
    padded = (I + PACK_BLOCK - 1) // PACK_BLOCK * PACK_BLOCK
    if kept is None:
        raise ValueError("kept must be what gated_fwd kept: a tensor or a packed pair")

    def call(stream_ptr):
        a_ptr = q_ptr = s_ptr = None
        if isinstance(kept, torch.Tensor):
            a_ptr = _arg(kept, "kept", torch.bfloat16, (S, 2 * I), index)
        else:
            q_ptr = _arg(kept[0], "kept[0]", torch.int8, (S, 2 * padded), index)
            s_ptr = _arg(kept[1], "kept[1]", torch.uint8, (S, 2 * padded // PACK_BLOCK), index)
        da, da_ptr = _out(dA, "dA", torch.bfloat16, (S, 2 * I), dev)
        h = h_ptr = None
        if want_h or H is not None:
            h, h_ptr = _out(H, "H", torch.bfloat16, (S, I), dev)
        need = 0
        if not (_chunked(N, dY) and _chunked(I, W)):
            need = lib.moegg_gated_bwd_workspace_bytes(T, topk, E, N, I)
        ws, ws_ptr, ws_bytes = _optional_workspace(workspace, need, dev)
        _check(lib.moegg_gated_bwd(
            _arg(dY, "dY", torch.bfloat16, (S, N), index),
            _arg(W, "W", torch.bfloat16, (E, N, I), index),
            _arg(m_sizes, "m_sizes", torch.int32, (E,), index),
            _slots_arg(gather_idx, "gather_idx", torch.int32, S, index), a_ptr, q_ptr, s_ptr, T,
            topk, E, N, I, int(flags), da_ptr, h_ptr, ws_ptr, ws_bytes,
            _flag_arg(error_flags, index), stream_ptr), "moegg_gated_bwd")
        return da, h

    return _run(dev, stream, call)


def dw_packed_workspace_bytes(num_tokens: int, topk: int, num_experts: int, N: int, K: int,
                              flags: int) -> int:
    """Workspace bytes of grouped_gemm_dW_packed with these flags."""
    return int(load_library().moegg_grouped_gemm_dW_packed_workspace_bytes(
        num_tokens, topk, num_experts, N, K, int(flags)))


def grouped_gemm_dW_packed(Xq, x_scales, dY, m_sizes, gather_idx, topk: int, flags: int, *, K: int,
                           dW=None, workspace=None, error_flags=None, stream=None):
    """grouped_gemm_dW with X as pack8 keeps it (moegg_grouped_gemm_dW_packed).

    Xq int8 [T or T*topk, Cp] and x_scales uint8: a packed X of K columns; the
    others as in grouped_gemm_dW.  The rows are expanded in `workspace` (a uint8
    CUDA tensor of dw_packed_workspace_bytes(...) bytes, allocated here when not
    given).  Returns [E, N, K] bf16 (fp32 with DW_FP32_OUT).
    """
    lib = load_library()
    dev = dY.device
    index = dev.index
    N, E, K = dY.shape[1], m_sizes.numel(), int(K)
    T = dY.shape[0] // topk
    S = T * topk
    q_shape, s_shape = _packed_shapes(T if flags & PERMUTE_X else S, K)

    def call(stream_ptr):
        w, w_ptr = _out(dW, "dW", torch.float32 if flags & DW_FP32_OUT else torch.bfloat16,
                        (E, N, K), dev)
        need = lib.moegg_grouped_gemm_dW_packed_workspace_bytes(T, topk, E, N, K, int(flags))
        ws, ws_ptr = _workspace_arg(workspace, need, dev)
        _check(lib.moegg_grouped_gemm_dW_packed(
            _arg(Xq, "Xq", torch.int8, q_shape, index),
            _arg(x_scales, "x_scales", torch.uint8, s_shape, index),
            _arg(dY, "dY", torch.bfloat16, (S, N), index),
            _arg(m_sizes, "m_sizes", torch.int32, (E,), index),
            _slots_arg(gather_idx, "gather_idx", torch.int32, S, index), T, topk, E, N, K,
            int(flags), w_ptr, ws_ptr, ws.numel(), _flag_arg(error_flags, index), stream_ptr),
            "moegg_grouped_gemm_dW_packed")
        return w

    return _run(dev, stream, call)
