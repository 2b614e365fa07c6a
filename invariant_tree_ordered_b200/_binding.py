"""ctypes binding of ``libtbik.so`` (argument marshalling only).

Every step of the computation runs in the library's CUDA kernels; this module
only turns torch tensors into device pointers and sizes, allocates workspaces
with torch (the library itself never allocates), and raises on a non-zero
status.  There is no fallback: if the library cannot be loaded, importing the
functions raises.
"""
from __future__ import annotations

import ctypes
import os
import re
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libtbik.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "tbik.h")

TBIK_OK = 0
TBIK_ERR_ARG = 1
TBIK_ERR_SHAPE = 2
TBIK_ERR_ALIGN = 3
TBIK_ERR_WORKSPACE = 4
TBIK_ERR_CUDA = 5
TBIK_ERR_TIMEOUT = 6
TBIK_ERR_TARGET = 7
TBIK_ERR_POSITION = 8
TBIK_ERR_UNSUPPORTED = 9
TBIK_ERR_PAGE = 10
TBIK_ERR_VALUE = 11

EXACT = 0x1
TC = 0x2
NONINV = 0x4
B_KN = 0x00
B_NK = 0x10
OUT_F32 = 0x000
OUT_BF16 = 0x100
SWIGLU_OUT = 0x200
DEBUG_WITHHOLD_ACC_ARRIVE = 0x1
DEBUG_TILE128 = 0x2
VOCAB_LEAF = 64
T_MAX = 8

_lock = threading.Lock()
_lib = None


class TbikError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: tbik status {status} ({status_string(status)})")


class RopeSwigluArgs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p),
        ("pos", ctypes.c_void_p), ("table", ctypes.c_void_p),
        ("tokens", ctypes.c_int), ("heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("max_pos", ctypes.c_int),
        ("g", ctypes.c_void_p), ("u", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("n", ctypes.c_longlong), ("in_f32", ctypes.c_int),
    ]


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load ``libtbik.so`` (raises OSError if it is missing: build it first)."""
    global _lib
    if _lib is not None and path is LIB_PATH:
        return _lib
    with _lock:
        if _lib is not None and path == LIB_PATH:
            return _lib
        if not os.path.exists(path):
            raise OSError(f"{path} not found: run `python -m invariant_tree_ordered_b200.build`")
        lib = ctypes.CDLL(path)
        vp, i32, u32, sz, f32, f64, ull = (ctypes.c_void_p, ctypes.c_int, ctypes.c_uint, ctypes.c_size_t,
                                            ctypes.c_float, ctypes.c_double, ctypes.c_ulonglong)
        sigs = {
            "tbik_version": (ctypes.c_char_p, []),
            "tbik_status_string": (ctypes.c_char_p, [i32]),
            "tbik_gemm_workspace": (sz, [i32, i32, i32, i32, i32, u32]),
            "tbik_gemm": (i32, [vp, vp, vp, i32, i32, i32, i32, i32, u32, vp, sz, vp]),
            "tbik_gemm_residual": (i32, [vp, vp, vp, vp, i32, i32, i32, i32, i32, u32, vp, sz, vp]),
            "tbik_rmsnorm_residual": (i32, [vp, vp, vp, vp, vp, i32, i32, f32, i32, vp]),
            "tbik_rope_table": (i32, [vp, i32, i32, f64, vp]),
            "tbik_rope_swiglu_fp32": (i32, [ctypes.POINTER(RopeSwigluArgs), vp]),
            "tbik_logprob_workspace": (sz, [i32, i32, i32, i32, i32, u32]),
            "tbik_logprob": (i32, [vp, vp, vp, vp, i32, i32, i32, i32, i32, u32, vp, sz, vp]),
            "tbik_attention": (i32, [vp, vp, vp, vp, i32, i32, i32, i32, i32, vp]),
            "tbik_attention_tc_workspace": (sz, [i32, i32, i32, i32, i32]),
            "tbik_attention_tc": (i32, [vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, sz, vp]),
            "tbik_embedding": (i32, [vp, vp, vp, i32, i32, i32, vp]),
            "tbik_transpose": (i32, [vp, vp, i32, i32, vp]),
            "tbik_tree_combine": (i32, [vp, vp, ctypes.c_longlong, i32, u32, vp, vp]),
            "tbik_logprob_partial_workspace": (sz, [i32, i32, i32, i32, i32, u32]),
            "tbik_logprob_partial": (i32, [vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, u32, vp, sz, vp]),
            "tbik_logprob_combine": (i32, [vp, vp, vp, i32, i32, i32, vp]),
            "tbik_cache_extend": (i32, [vp] * 6 + [i32] * 5 + [vp]),
            "tbik_cache_fork_workspace": (sz, [i32]),
            "tbik_cache_fork": (i32, [vp] * 7 + [i32] * 8 + [vp, sz, vp]),
            "tbik_cache_free": (i32, [vp] * 4 + [i32] * 5 + [vp]),
            "tbik_cache_compact_workspace": (sz, [i32]),
            "tbik_cache_compact": (i32, [vp] * 6 + [i32] * 7 + [vp, sz, vp]),
            "tbik_cache_copy": (i32, [vp] * 4 + [i32] * 6 + [vp, sz, vp]),
            "tbik_cache_append": (i32, [vp] * 9 + [i32] * 8 + [vp]),
            "tbik_cache_attention_workspace": (sz, [i32] * 8),
            "tbik_cache_attention": (i32, [vp] * 8 + [i32] * 11 + [vp, sz, vp]),
            "tbik_sample": (i32, [vp] * 7 + [i32] * 3 + [vp]),
            "tbik_get_error": (i32, [vp]),
            "tbik_debug_set": (i32, [u32, ull]),
        }
        for name, (res, args) in sigs.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        if path == LIB_PATH:
            _lib = lib
        return lib


def declared_functions(header: str = HEADER):
    """Names of the functions ``include/tbik.h`` declares."""
    with open(header) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(tbik_[a-z0-9_]+)\s*\(", text)))


def status_string(status: int) -> str:
    try:
        return load_library().tbik_status_string(status).decode()
    except OSError:
        return "library not loaded"


def _check(status: int, what: str):
    if status != TBIK_OK:
        raise TbikError(status, what)


# ------------------------------------------------------------ torch plumbing

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _need_out(t, dtype, shape, name="out"):
    """A caller-provided output: a contiguous CUDA tensor of this dtype and shape."""
    _need(t, dtype, name)
    if t.shape != shape and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _need(t, dtype, name):
    try:
        if t.is_cuda and t.dtype is dtype and t.is_contiguous():
            return
    except AttributeError:
        pass
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _workspace(nbytes: int, device, workspace):
    torch = _torch()
    if nbytes == (1 << 64) - 1 or nbytes < 0:
        raise TbikError(TBIK_ERR_SHAPE, "workspace query")
    if nbytes == 0:
        return workspace, 0
    if workspace is not None:
        return workspace, workspace.numel() * workspace.element_size()
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws, nbytes


# ---------------------------------------------------------------- entry points

def gemm_workspace(M, N, K, T, leaf, mode) -> int:
    return int(load_library().tbik_gemm_workspace(M, N, K, T, leaf, mode))


def gemm(A, B, *, T: int = 1, leaf: int = 256, tc: bool = True, noninv: bool = False, b_nk: bool = False,
         out_bf16: bool = False, swiglu: bool = False, residual=None, out=None, workspace=None, stream=None):
    """C = A @ B with the K reduction in tree order (see tbik_gemm in tbik.h).
    swiglu: B holds gate/up columns interleaved in blocks of 32 and C is the
    bf16 SwiGLU [M, N/2] of the fp32 roots (TBIK_SWIGLU_OUT).
    residual: bf16 [M, N]; C = bf16(root + residual) (tbik_gemm_residual);
    ``out`` may be the residual tensor itself (in place)."""
    torch = _torch()
    lib = load_library()
    _need(A, torch.bfloat16, "A")
    _need(B, torch.bfloat16, "B")
    M, K = A.shape
    N = B.shape[0] if b_nk else B.shape[1]
    kb = B.shape[1] if b_nk else B.shape[0]
    if kb != K:
        raise ValueError("inner dimensions differ")
    mode = (TC if tc else EXACT) | (NONINV if noninv else 0) | (B_NK if b_nk else B_KN)
    if residual is not None:
        if swiglu:
            raise ValueError("residual and swiglu outputs are exclusive")
        _need(residual, torch.bfloat16, "residual")
        if tuple(residual.shape) != (M, N):
            raise ValueError("residual must be [M, N]")
        if out is None:
            out = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
        _need_out(out, torch.bfloat16, (M, N))
        ws, wsb = _workspace(lib.tbik_gemm_workspace(M, N, K, T, leaf, mode | OUT_BF16), A.device, workspace)
        _check(lib.tbik_gemm_residual(_ptr(A), _ptr(B), _ptr(residual), _ptr(out), M, N, K, T, leaf, mode,
                                      _ptr(ws), wsb, _stream_handle(stream)), "tbik_gemm_residual")
        return out
    mode |= OUT_BF16 if out_bf16 else OUT_F32
    if swiglu:
        mode |= SWIGLU_OUT
    out_dtype = torch.bfloat16 if (swiglu or out_bf16) else torch.float32
    out_shape = (M, N // 2) if swiglu else (M, N)
    if out is None:
        out = torch.empty(out_shape, dtype=out_dtype, device=A.device)
    _need_out(out, out_dtype, out_shape)
    ws, wsb = _workspace(lib.tbik_gemm_workspace(M, N, K, T, leaf, mode), A.device, workspace)
    _check(lib.tbik_gemm(_ptr(A), _ptr(B), _ptr(out), M, N, K, T, leaf, mode, _ptr(ws), wsb,
                         _stream_handle(stream)), "tbik_gemm")
    return out


def rmsnorm_residual(x, res, gamma, *, eps: float = 1e-6, T: int = 1, y=None, res_out=None, want_res_out=True,
                     stream=None):
    torch = _torch()
    lib = load_library()
    for t, n in ((x, "x"), (res, "res"), (gamma, "gamma")):
        if t is not None or n != "res":  # res None: no residual input, r = f32(x)
            _need(t, torch.bfloat16, n)
    if x.dim() != 2:
        raise ValueError("x must be [tokens, H]")
    tokens, H = x.shape
    if res is not None and res.shape != x.shape:
        raise ValueError("res must have the shape of x")
    if tuple(gamma.shape) != (H,):
        raise ValueError("gamma must be [H]")
    if y is None:
        y = torch.empty_like(x)
    _need_out(y, torch.bfloat16, x.shape, "y")
    if res_out is None and want_res_out:
        res_out = torch.empty_like(x)
    if res_out is not None:
        _need_out(res_out, torch.bfloat16, x.shape, "res_out")
    _check(lib.tbik_rmsnorm_residual(_ptr(x), _ptr(res), _ptr(gamma), _ptr(y), _ptr(res_out), tokens, H,
                                     float(eps), T, _stream_handle(stream)), "tbik_rmsnorm_residual")
    return y, res_out


def rope_table(max_pos: int, head_dim: int = 128, base: float = 1e6, device="cuda", stream=None):
    torch = _torch()
    lib = load_library()
    t = torch.empty((max_pos, head_dim // 2, 2), dtype=torch.float32, device=device)
    _check(lib.tbik_rope_table(_ptr(t), max_pos, head_dim, float(base), _stream_handle(stream)), "tbik_rope_table")
    return t


def rope_swiglu(*, q=None, k=None, pos=None, table=None, q_out=None, k_out=None, g=None, u=None, out=None,
                stream=None):
    """RoPE on q/k and/or SwiGLU on g/u in one call (see tbik_rope_swiglu_fp32)."""
    torch = _torch()
    lib = load_library()
    a = RopeSwigluArgs()
    if q is not None or k is not None:
        ref = q if q is not None else k
        _need(ref, torch.bfloat16, "q/k")
        _need(pos, torch.int32, "pos")
        _need(table, torch.float32, "table")
        if ref.dim() != 3:
            raise ValueError("q and k must be [tokens, heads, head_dim]")
        tokens, heads, hd = ref.shape
        for t, n in ((q, "q"), (k, "k")):
            if t is not None:
                _need(t, torch.bfloat16, n)
                if t.shape != ref.shape:
                    raise ValueError("q and k must share one shape")
        if pos.numel() != tokens:
            raise ValueError("pos must hold one position per token")
        if table.dim() != 3 or tuple(table.shape[1:]) != (hd // 2, 2):
            raise ValueError("table must be [max_pos, head_dim/2, 2]")
        if q is not None and q_out is None:
            q_out = torch.empty_like(q)
        if k is not None and k_out is None:
            k_out = torch.empty_like(k)
        if q is not None:
            _need_out(q_out, torch.bfloat16, ref.shape, "q_out")
        if k is not None:
            _need_out(k_out, torch.bfloat16, ref.shape, "k_out")
        a.q, a.k, a.q_out, a.k_out = _ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out)
        a.pos, a.table = _ptr(pos), _ptr(table)
        a.tokens, a.heads, a.head_dim, a.max_pos = tokens, heads, hd, table.shape[0]
    if g is not None:
        if g.dtype not in (torch.bfloat16, torch.float32) or u.dtype != g.dtype:
            raise TypeError("g and u must both be bf16 or both fp32")
        _need(g, g.dtype, "g")
        _need(u, g.dtype, "u")
        if u.shape != g.shape:
            raise ValueError("g and u must share one shape")
        if out is None:
            out = torch.empty(g.shape, dtype=torch.bfloat16, device=g.device)
        _need_out(out, torch.bfloat16, g.shape)
        a.g, a.u, a.out, a.n, a.in_f32 = _ptr(g), _ptr(u), _ptr(out), g.numel(), int(g.dtype == torch.float32)
    _check(lib.tbik_rope_swiglu_fp32(ctypes.byref(a), _stream_handle(stream)), "tbik_rope_swiglu_fp32")
    return q_out, k_out, out


# keys per tree leaf: the exact mode's chunk and the tensor-core mode's leaf (two 64-key MMA chunks)
ATTENTION_CHUNK = 64
ATTENTION_TC_LEAF = 128


def attention_tc_workspace(batch, seq, heads, head_dim, chunk=ATTENTION_TC_LEAF) -> int:
    n = load_library().tbik_attention_tc_workspace(batch, seq, heads, head_dim, chunk)
    if n == (1 << 64) - 1:
        raise TbikError(TBIK_ERR_SHAPE, "tbik_attention_tc_workspace: unsupported shape")
    return n


def attention(q, k, v, *, out=None, chunk=None, tc: bool = False, workspace=None, stream=None):
    """Causal attention with the key reduction in tree order; q, k, v bf16
    [batch, seq, heads, head_dim].  tc=False: tbik_attention (exact order on
    the CUDA cores, leaves of `chunk` = 64 keys); tc=True: tbik_attention_tc
    (tensor cores, leaves of 128 keys; a workspace is allocated when none is
    given)."""
    if chunk is None:
        chunk = ATTENTION_TC_LEAF if tc else ATTENTION_CHUNK
    torch = _torch()
    lib = load_library()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, torch.bfloat16, n)
    if q.dim() != 4 or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must share the shape [batch, seq, heads, head_dim]")
    B, S, NH, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    _need_out(out, torch.bfloat16, q.shape)
    if not tc:
        _check(lib.tbik_attention(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, S, NH, D, chunk, _stream_handle(stream)),
               "tbik_attention")
        return out
    need = attention_tc_workspace(B, S, NH, D, chunk)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    wsp, wsn = (_ptr(workspace), workspace.numel() * workspace.element_size()) if workspace is not None else (None, 0)
    _check(lib.tbik_attention_tc(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, S, NH, D, chunk, wsp, wsn,
                                 _stream_handle(stream)), "tbik_attention_tc")
    return out


def embedding(ids, table, *, out=None, stream=None):
    """Rows of ``table`` (bf16 [V, d]) at ``ids`` (int32 [tokens]) (see tbik_embedding)."""
    torch = _torch()
    lib = load_library()
    _need(ids, torch.int32, "ids")
    _need(table, torch.bfloat16, "table")
    V, d = table.shape
    if out is None:
        out = torch.empty((ids.numel(), d), dtype=torch.bfloat16, device=table.device)
    _need_out(out, torch.bfloat16, (ids.numel(), d))
    _check(lib.tbik_embedding(_ptr(ids), _ptr(table), _ptr(out), ids.numel(), V, d, _stream_handle(stream)),
           "tbik_embedding")
    return out


def transpose(x, *, out=None, stream=None):
    """bf16 [rows, cols] -> [cols, rows] (see tbik_transpose)."""
    torch = _torch()
    lib = load_library()
    _need(x, torch.bfloat16, "x")
    rows, cols = x.shape
    if out is None:
        out = torch.empty((cols, rows), dtype=torch.bfloat16, device=x.device)
    _need_out(out, torch.bfloat16, (cols, rows))
    _check(lib.tbik_transpose(_ptr(x), _ptr(out), rows, cols, _stream_handle(stream)), "tbik_transpose")
    return out


def logprob_workspace(M, V, H, T, leaf, mode) -> int:
    return int(load_library().tbik_logprob_workspace(M, V, H, T, leaf, mode))


def _logprob_shapes(hidden, W, targets):
    if hidden.dim() != 2 or W.dim() != 2 or W.shape[1] != hidden.shape[1]:
        raise ValueError("hidden must be [M, H] and W_lm [V, H]")
    if targets.numel() != hidden.shape[0]:
        raise ValueError("targets must hold one index per row of hidden")


def logprob(hidden, W, targets, *, T: int = 1, leaf: int = 256, tc: bool = True, noninv: bool = False, out=None,
            workspace=None, stream=None):
    torch = _torch()
    lib = load_library()
    _need(hidden, torch.bfloat16, "hidden")
    _need(W, torch.bfloat16, "W_lm")
    _need(targets, torch.int32, "targets")
    M, H = hidden.shape
    V = W.shape[0]
    _logprob_shapes(hidden, W, targets)
    mode = (TC if tc else EXACT) | (NONINV if noninv else 0)
    if out is None:
        out = torch.empty(M, dtype=torch.float32, device=hidden.device)
    _need_out(out, torch.float32, (M,))
    ws, wsb = _workspace(lib.tbik_logprob_workspace(M, V, H, T, leaf, mode), hidden.device, workspace)
    _check(lib.tbik_logprob(_ptr(hidden), _ptr(W), _ptr(targets), _ptr(out), M, V, H, T, leaf, mode, _ptr(ws), wsb,
                            _stream_handle(stream)), "tbik_logprob")
    return out


# ------------------------------------------- shard level across GPUs (TP)

def vocab_shard(V: int, T: int, t: int):
    """Shard t of T of the padded vocabulary (tbik.h, vocabulary-parallel
    logprob): (v0, Vs, Lvs) = first vocabulary index, real columns, leaves."""
    step = VOCAB_LEAF * T_MAX
    vpad = ((V + step - 1) // step) * step
    if T not in (1, 2, 4, 8) or not 0 <= t < T:
        raise ValueError("T must be 1, 2, 4 or 8 and 0 <= t < T")
    width = vpad // T
    v0 = t * width
    vs = max(0, min(V - v0, width))
    return v0, vs, width // VOCAB_LEAF


def tree_combine(partials, *, noninv: bool = False, out_bf16: bool = False, residual=None, out=None, stream=None):
    """tbik_tree_combine: the shard level of the tree over fp32 partials [T, ...]
    gathered in rank order (left to right with noninv).  Returns fp32 or bf16
    of shape partials.shape[1:]; residual (bf16, that shape) is added to the
    fp32 root before the bf16 rounding."""
    torch = _torch()
    lib = load_library()
    _need(partials, torch.float32, "partials")
    T = partials.shape[0]
    shape = tuple(partials.shape[1:])
    mn = partials[0].numel()
    if residual is not None:
        out_bf16 = True
        _need_out(residual, torch.bfloat16, shape, "residual")
    dtype = torch.bfloat16 if out_bf16 else torch.float32
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=partials.device)
    _need_out(out, dtype, shape)
    mode = (NONINV if noninv else 0) | (OUT_BF16 if out_bf16 else 0)
    _check(lib.tbik_tree_combine(_ptr(partials), _ptr(out), mn, T, mode, _ptr(residual), _stream_handle(stream)),
           "tbik_tree_combine")
    return out


def logprob_partial(hidden, W_shard, targets, *, v0: int, Lvs: int, leaf: int = 256, tc: bool = True, out=None,
                    workspace=None, stream=None):
    """tbik_logprob_partial: one vocabulary shard's per-row (m, s, z, own),
    fp32 [M, 4].  W_shard holds vocabulary rows [v0, v0 + Vs) (Vs may be 0)."""
    torch = _torch()
    lib = load_library()
    _need(hidden, torch.bfloat16, "hidden")
    _need(W_shard, torch.bfloat16, "W_shard")
    _need(targets, torch.int32, "targets")
    M, H = hidden.shape
    Vs = W_shard.shape[0]
    if W_shard.dim() != 2 or (Vs > 0 and W_shard.shape[1] != H):
        raise ValueError("W_shard must be [Vs, H]")
    if targets.numel() != M:
        raise ValueError("targets must hold one index per row of hidden")
    mode = TC if tc else EXACT
    if out is None:
        out = torch.empty((M, 4), dtype=torch.float32, device=hidden.device)
    _need_out(out, torch.float32, (M, 4))
    ws, wsb = _workspace(lib.tbik_logprob_partial_workspace(M, Vs, Lvs, H, leaf, mode), hidden.device, workspace)
    wptr = _ptr(W_shard) if Vs > 0 else None
    _check(lib.tbik_logprob_partial(_ptr(hidden), wptr, _ptr(targets), _ptr(out), M, Vs, v0, Lvs, H, leaf, mode,
                                    _ptr(ws), wsb, _stream_handle(stream)), "tbik_logprob_partial")
    return out


def logprob_combine(parts, targets, V: int, *, out=None, stream=None):
    """tbik_logprob_combine: parts fp32 [T, M, 4] (shard summaries in rank
    order) -> logprob fp32 [M]."""
    torch = _torch()
    lib = load_library()
    _need(parts, torch.float32, "parts")
    _need(targets, torch.int32, "targets")
    if parts.dim() != 3 or parts.shape[2] != 4:
        raise ValueError("parts must be [T, M, 4]")
    T, M = parts.shape[0], parts.shape[1]
    if targets.numel() != M:
        raise ValueError("targets must hold one index per row")
    if out is None:
        out = torch.empty(M, dtype=torch.float32, device=parts.device)
    _need_out(out, torch.float32, (M,))
    _check(lib.tbik_logprob_combine(_ptr(parts), _ptr(targets), _ptr(out), M, V, T, _stream_handle(stream)),
           "tbik_logprob_combine")
    return out


# ------------------------------------------------ paged 8-bit key/value cache

def cache_pages(num_pages: int, kv_heads: int, head_dim: int, page: int, layers: int = 1, device="cuda"):
    """An empty pool (tbik.h, paged 8-bit key/value cache): (pages e4m3 [layers, 2, num_pages, kv_heads, page/8,
    head_dim/16, 8, 16], scales fp32 [layers, 2, num_pages, kv_heads], refs int32 [num_pages])."""
    torch = _torch()
    if page not in (16, 32, 64, 128) or head_dim not in (64, 128):
        raise ValueError("page must be 16, 32, 64 or 128 and head_dim 64 or 128")
    pages = torch.zeros((layers, 2, num_pages, kv_heads, page // 8, head_dim // 16, 8, 16), dtype=torch.uint8,
                        device=device).view(torch.float8_e4m3fn)
    scales = torch.ones((layers, 2, num_pages, kv_heads), dtype=torch.float32, device=device)
    return pages, scales, torch.zeros(num_pages, dtype=torch.int32, device=device)


def cache_table(slots: int, max_pages: int, device="cuda"):
    """Empty slots: (table int32 [slots, max_pages] of -1, lens int32 [slots] of 0)."""
    torch = _torch()
    return (torch.full((slots, max_pages), -1, dtype=torch.int32, device=device),
            torch.zeros(slots, dtype=torch.int32, device=device))


def _on_device(first, others, stream, fn, args, what):
    """Calls the library on `first`'s device and stream (its current one by default), whatever the current device
    is; every tensor of the call has to be there."""
    torch = _torch()
    index = first.get_device()
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError("all tensors must be on one device")
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if index == torch._C._cuda_getDevice():
        status = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            status = fn(*args, handle)
    if status != TBIK_OK:
        raise TbikError(status, what)


def _new(shape, dtype, device, stream):
    """A tensor for a call on `stream`: it belongs to that stream's memory, so that what the call drops at its end (a
    workspace) is not handed to another stream while the kernels run."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _need_i32(t, name, n=None):
    torch = _torch()
    if t is None:
        return None
    _need(t, torch.int32, name)
    if n is not None and t.numel() != n:
        raise ValueError(f"{name} must hold {n} values, got {t.numel()}")
    return t.data_ptr()


def _pool(pages, scales, layered):
    """(layers, num_pages, kv_heads, page, head_dim) of a pool; one layer's has no leading dimension."""
    torch = _torch()
    _need(pages, torch.float8_e4m3fn, "pages")
    _need(scales, torch.float32, "scales")
    s, c, k = pages.shape, scales.shape, 1 if layered else 0
    if len(s) != 7 + k or s[k] != 2 or s[k + 5] != 8 or s[k + 6] != 16:
        raise ValueError("pages must be [%s2, num_pages, kv_heads, page/8, head_dim/16, 8, 16]" % ("layers, " if layered else ""))
    layers, num_pages, kv_heads = s[0] if layered else 1, s[k + 1], s[k + 2]
    if len(c) != 3 + k or c[k] != 2 or c[k + 1] != num_pages or c[k + 2] != kv_heads or (layered and c[0] != layers):
        raise ValueError("scales must be [%s2, num_pages, kv_heads]" % ("layers, " if layered else ""))
    return layers, num_pages, kv_heads, s[k + 3] * 8, s[k + 4] * 16


def _meta(table, lens, refs):
    """(slots, max_pages, num_pages) of the bookkeeping."""
    torch = _torch()
    _need(table, torch.int32, "table")
    _need(lens, torch.int32, "lens")
    _need(refs, torch.int32, "refs")
    if table.dim() != 2:
        raise ValueError("table must be [slots, max_pages]")
    if lens.numel() != table.shape[0]:
        raise ValueError("lens must hold one length per slot")
    return table.shape[0], table.shape[1], refs.numel()


def cache_extend(table, lens, refs, n_new, *, page: int, rows=None, start=None, stream=None):
    """Room for n_new[b] more tokens of each sequence (slots `rows`, default 0, 1, ...): returns start int32 [batch],
    the position of each sequence's first new token, or -1 for all when the call is refused (tbik_cache_extend)."""
    torch = _torch()
    lib = load_library()
    slots, max_pages, num_pages = _meta(table, lens, refs)
    _need(n_new, torch.int32, "n_new")
    batch = n_new.numel()
    rp = _need_i32(rows, "rows", batch)
    if start is None:
        start = _new(batch, torch.int32, table.device, stream)
    _need_out(start, torch.int32, (batch,), "start")
    _on_device(table, (lens, refs, n_new, rows, start), stream, lib.tbik_cache_extend,
               (table.data_ptr(), lens.data_ptr(), refs.data_ptr(), rp, n_new.data_ptr(), start.data_ptr(), batch,
                slots, max_pages, num_pages, page), "tbik_cache_extend")
    return start


def _bytes_on(nbytes, device, workspace, stream):
    """(tensor, pointer, bytes) of the caller's workspace, or of a new one."""
    torch = _torch()
    if nbytes == (1 << 64) - 1:
        raise TbikError(TBIK_ERR_SHAPE, "workspace query")
    if workspace is None:
        if nbytes == 0:
            return None, None, 0
        workspace = _new(nbytes, torch.uint8, device, stream)
    elif not workspace.is_contiguous():  # the bytes of an expanded tensor are fewer than its elements
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def cache_fork(pages, scales, table, lens, refs, parents, children, *, workspace=None, stream=None):
    """children[i] (empty slots) become copies of parents[i] (tbik_cache_fork); pages and scales of all layers,
    [layers, 2, ...]."""
    torch = _torch()
    lib = load_library()
    layers, num_pages, kv_heads, page, head_dim = _pool(pages, scales, True)
    slots, max_pages, n_refs = _meta(table, lens, refs)
    if n_refs != num_pages:
        raise ValueError("refs must hold one count per page")
    _need(parents, torch.int32, "parents")
    count = parents.numel()
    cp = _need_i32(children, "children", count)
    ws, wsp, wsb = _bytes_on(lib.tbik_cache_fork_workspace(count), pages.device, workspace, stream)
    _on_device(pages, (scales, table, lens, refs, parents, children, ws), stream, lib.tbik_cache_fork,
               (pages.data_ptr(), scales.data_ptr(), table.data_ptr(), lens.data_ptr(), refs.data_ptr(),
                parents.data_ptr(), cp, count, layers, slots, max_pages, num_pages, kv_heads, head_dim, page, wsp, wsb),
               "tbik_cache_fork")


def cache_free(table, lens, refs, rows, *, page: int, stream=None):
    """Gives up the pages of the sequences in slots `rows` (tbik_cache_free)."""
    torch = _torch()
    lib = load_library()
    slots, max_pages, num_pages = _meta(table, lens, refs)
    _need(rows, torch.int32, "rows")
    _on_device(table, (lens, refs, rows), stream, lib.tbik_cache_free,
               (table.data_ptr(), lens.data_ptr(), refs.data_ptr(), rows.data_ptr(), rows.numel(), slots, max_pages,
                num_pages, page), "tbik_cache_free")


def cache_compact(pages, scales, table, lens, refs, *, live=None, workspace=None, stream=None):
    """Live pages to the front of the pool (tbik_cache_compact); returns their number as int32 [1] (-1: refused)."""
    torch = _torch()
    lib = load_library()
    layers, num_pages, kv_heads, page, head_dim = _pool(pages, scales, True)
    slots, max_pages, n_refs = _meta(table, lens, refs)
    if n_refs != num_pages:
        raise ValueError("refs must hold one count per page")
    if live is None:
        live = _new(1, torch.int32, pages.device, stream)
    _need_out(live, torch.int32, (1,), "live")
    ws, wsp, wsb = _bytes_on(lib.tbik_cache_compact_workspace(num_pages), pages.device, workspace, stream)
    _on_device(pages, (scales, table, lens, refs, live, ws), stream, lib.tbik_cache_compact,
               (pages.data_ptr(), scales.data_ptr(), table.data_ptr(), lens.data_ptr(), refs.data_ptr(),
                live.data_ptr(), layers, slots, max_pages, num_pages, kv_heads, head_dim, page, wsp, wsb),
               "tbik_cache_compact")
    return live


def cache_copy(pages, scales, src, dst, *, workspace=None, stream=None):
    """Page dst[i] = page src[i] in all layers (tbik_cache_copy); no bookkeeping."""
    torch = _torch()
    lib = load_library()
    layers, num_pages, kv_heads, page, head_dim = _pool(pages, scales, True)
    _need(src, torch.int32, "src")
    count = src.numel()
    dp = _need_i32(dst, "dst", count)
    ws, wsp, wsb = _bytes_on(lib.tbik_cache_fork_workspace(count), pages.device, workspace, stream)
    _on_device(pages, (scales, src, dst, ws), stream, lib.tbik_cache_copy,
               (pages.data_ptr(), scales.data_ptr(), src.data_ptr(), dp, count, layers, num_pages, kv_heads, head_dim,
                page, wsp, wsb), "tbik_cache_copy")


def _packed(x, name, table, start, cu, rows):
    """(tokens, batch, slots, max_pages) of a call on packed tokens."""
    torch = _torch()
    if x.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    _need(table, torch.int32, "table")
    if table.dim() != 2:
        raise ValueError("table must be [slots, max_pages]")
    _need(start, torch.int32, "start")
    batch, tokens = start.numel(), x.shape[0]
    if cu is None and tokens != batch:
        raise ValueError("without cu there is one token per sequence")
    if rows is None and batch > table.shape[0]:
        raise ValueError("more sequences than slots")
    return tokens, batch, table.shape[0], table.shape[1]


def cache_append(k, v, pages, scales, table, refs, start, *, cu=None, rows=None, stream=None):
    """Writes new tokens of one layer into its pages [2, num_pages, ...] (tbik_cache_append): k, v bf16 [tokens,
    kv_heads, head_dim], sequence b's tokens cu[b] .. cu[b+1]-1 (cu None: one token each) at positions start[b], ..."""
    torch = _torch()
    lib = load_library()
    _need(k, torch.bfloat16, "k")
    _need(v, torch.bfloat16, "v")
    _, num_pages, kv_heads, page, head_dim = _pool(pages, scales, False)
    tokens, batch, slots, max_pages = _packed(k, "k", table, start, cu, rows)
    if v.shape != k.shape or k.shape[1] != kv_heads or k.shape[2] != head_dim:
        raise ValueError("k and v must be [tokens, kv_heads, head_dim] of the pool")
    rfp = _need_i32(refs, "refs", num_pages)
    cup, rp = _need_i32(cu, "cu", batch + 1), _need_i32(rows, "rows", batch)
    _on_device(pages, (k, v, scales, table, refs, start, cu, rows), stream, lib.tbik_cache_append,
               (k.data_ptr(), v.data_ptr(), pages.data_ptr(), scales.data_ptr(), table.data_ptr(), rfp,
                start.data_ptr(), cup, rp, tokens, batch, slots, max_pages, num_pages, kv_heads, head_dim, page),
               "tbik_cache_append")


def cache_attention_workspace(tokens, batch, max_q, max_keys, heads, kv_heads, head_dim, page) -> int:
    n = load_library().tbik_cache_attention_workspace(tokens, batch, max_q, max_keys, heads, kv_heads, head_dim, page)
    if n == (1 << 64) - 1:
        raise TbikError(TBIK_ERR_SHAPE, "tbik_cache_attention_workspace: unsupported shape")
    return n


_attention_bytes = {}


def cache_attention(q, pages, scales, table, start, *, cu=None, rows=None, max_q=None, max_keys=None, out=None,
                    workspace=None, stream=None):
    """Attention of new queries over one layer's pages [2, num_pages, ...] (tbik_cache_attention): q bf16 [tokens,
    heads, head_dim], packed like cache_append's tokens, query t of sequence b at position start[b] + t over the keys
    at positions up to its own.  max_q and max_keys bound the tokens of a sequence in this call and the keys that any
    query sees (default: all tokens; what a table row can hold); tight bounds keep the workspace and the grid small."""
    torch = _torch()
    lib = load_library()
    _need(q, torch.bfloat16, "q")
    _, num_pages, kv_heads, page, head_dim = _pool(pages, scales, False)
    tokens, batch, slots, max_pages = _packed(q, "q", table, start, cu, rows)
    heads = q.shape[1]
    if q.shape[2] != head_dim:
        raise ValueError("q must have the head_dim of the pool")
    if max_q is None:
        max_q = 1 if cu is None else max(tokens, 1)
    if max_keys is None:
        max_keys = max_pages * page
    cup, rp = _need_i32(cu, "cu", batch + 1), _need_i32(rows, "rows", batch)
    key = (q.get_device(), tokens, batch, max_q, max_keys, heads, kv_heads, head_dim, page)
    nbytes = _attention_bytes.get(key)
    if nbytes is None:  # a function of the sizes and the device
        with torch.cuda.device(key[0]):
            nbytes = lib.tbik_cache_attention_workspace(*key[1:])
        if len(_attention_bytes) < 4096:
            _attention_bytes[key] = nbytes
    if out is None:
        # tokens outside every sequence are left as they are: zeros in a new tensor
        if stream is None:
            out = torch.empty_like(q) if cu is None else torch.zeros_like(q)
        else:
            out = _new(q.shape, q.dtype, q.device, stream)
            if cu is not None:
                with torch.cuda.stream(stream):
                    out.zero_()
    else:
        _need_out(out, torch.bfloat16, q.shape)
    ws, wsp, wsb = _bytes_on(nbytes, q.device, workspace, stream)
    _on_device(pages, (q, scales, table, start, cu, rows, out, ws), stream, lib.tbik_cache_attention,
               (q.data_ptr(), pages.data_ptr(), scales.data_ptr(), table.data_ptr(), start.data_ptr(), cup, rp,
                out.data_ptr(), tokens, batch, slots, max_pages, num_pages, heads, kv_heads, head_dim, page, max_q,
                max_keys, wsp, wsb), "tbik_cache_attention")
    return out


# -------------------------------------------------------------------- sampling

def sample(logits, u, *, temperature=None, top_k=None, top_p=None, min_p=None, out=None, stream=None):
    """One token per row of logits (fp32 or bf16 [batch, vocab]) from given numbers u (fp32 [batch], in [0, 1)):
    temperature, top-k, top-p, min-p, then the inverse of the running sum in index order (tbik_sample).  The settings
    are device tensors of one value per row (fp32; top_k int32), or None."""
    torch = _torch()
    lib = load_library()
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("logits must be fp32 or bf16")
    _need(logits, logits.dtype, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be [batch, vocab]")
    batch, vocab = logits.shape
    ptrs = []
    for t, name in ((u, "u"), (temperature, "temperature"), (top_k, "top_k"), (top_p, "top_p"), (min_p, "min_p")):
        if t is None and name != "u":
            ptrs.append(None)
            continue
        _need(t, torch.int32 if name == "top_k" else torch.float32, name)
        if t.numel() != batch:
            raise ValueError(f"{name} must hold one value per row")
        ptrs.append(t.data_ptr())
    if out is None:
        out = _new(batch, torch.int32, logits.device, stream)
    _need_out(out, torch.int32, (batch,))
    _on_device(logits, (u, temperature, top_k, top_p, min_p, out), stream, lib.tbik_sample,
               (logits.data_ptr(), *ptrs, out.data_ptr(), batch, vocab, int(logits.dtype == torch.bfloat16)), "tbik_sample")
    return out


def get_error(stream=None) -> int:
    return int(load_library().tbik_get_error(_stream_handle(stream)))


def debug_set(flags: int = 0, wait_limit_ns: int = 0):
    _check(load_library().tbik_debug_set(flags, wait_limit_ns), "tbik_debug_set")


_noalloc_ready = False


def logprob_noalloc(hidden, W, targets, *, T: int = 1, leaf: int = 256, noninv: bool = False, out=None,
                    stream=None):
    """tbik_logprob_noalloc: tensor-core logprob whose scratch is the library's
    fixed device array, for callers that cannot allocate a workspace.  Only the
    output (when not given) is allocated here, by torch."""
    global _noalloc_ready
    torch = _torch()
    lib = load_library()
    if not _noalloc_ready:
        vp, i32, u32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint
        lib.tbik_logprob_noalloc.restype = i32
        lib.tbik_logprob_noalloc.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, u32, vp]
        _noalloc_ready = True
    _need(hidden, torch.bfloat16, "hidden")
    _need(W, torch.bfloat16, "W_lm")
    _need(targets, torch.int32, "targets")
    M, H = hidden.shape
    V = W.shape[0]
    _logprob_shapes(hidden, W, targets)
    mode = TC | (NONINV if noninv else 0)
    if out is None:
        out = torch.empty(M, dtype=torch.float32, device=hidden.device)
    _need_out(out, torch.float32, (M,))
    _check(lib.tbik_logprob_noalloc(_ptr(hidden), _ptr(W), _ptr(targets), _ptr(out), M, V, H, T, leaf, mode,
                                    _stream_handle(stream)), "tbik_logprob_noalloc")
    return out

