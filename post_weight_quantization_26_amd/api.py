"""Torch-facing wrappers of the C ABI: AWQ per-layer search on one MI355X.

PyTorch provides device memory and the current HIP stream; every computation
runs in the HIP library through the C ABI. Tensors must live on the GPU and be
contiguous. Defaults follow the AutoAWQ configuration the roadmap page prints
in section 9 (zero point on, group 128, 4 bits).
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import numpy as np
import torch

from . import _lib as L

_DT = {torch.float32: L.AWQ_F32, torch.bfloat16: L.AWQ_BF16, torch.float16: L.AWQ_F16}

DEFAULT_BITS = 4
DEFAULT_GROUP = 128
DEFAULT_ZERO_POINT = True


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dev(t: torch.Tensor, name: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _dtype(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return _DT[t.dtype]


def _groups(K: int, group: int) -> int:
    """Groups of K channels; a size the library would refuse before it divides."""
    if group < 1:
        raise L.AwqError(L.AWQ_E_UNSUPPORTED, f"group_size {group} not supported (32, 64 or 128)")
    return K // group


def workspace_bytes(op: int, T: int, N: int, K: int, n_grid: int, dtype: torch.dtype) -> int:
    return int(L.lib().awq_workspace_bytes(op, T, N, K, n_grid, _DT[dtype]))


def workspace_bytes_batch(op: int, T: int, N: int, K: int, n_grid: int, batch: int,
                          dtype: torch.dtype) -> int:
    return int(L.lib().awq_workspace_bytes_batch(op, T, N, K, n_grid, batch, _DT[dtype]))


def _workspace(ws: Optional[torch.Tensor], need: int, device) -> torch.Tensor:
    if ws is not None:
        return ws
    return torch.empty(max(need, 256), dtype=torch.uint8, device=device)


def qconfig(bits=DEFAULT_BITS, group=DEFAULT_GROUP, zero_point=DEFAULT_ZERO_POINT,
            split_e=False, fused=False) -> L.QConfig:
    return L.QConfig(int(bits), int(group), int(bool(zero_point)),
                     (L.AWQ_SEARCH_SPLIT_E if split_e else 0) |
                     (L.AWQ_SEARCH_FUSED if fused else 0))


def _direct_op(op: int, split_e: bool, fused: bool = False) -> int:
    """The workspace op of a direct search, in its split or fused form when asked."""
    if fused:
        return {L.AWQ_OP_SEARCH_SCALE: L.AWQ_OP_SEARCH_SCALE_FUSED,
                L.AWQ_OP_SEARCH_CLIP: L.AWQ_OP_SEARCH_CLIP_FUSED}.get(op, op)
    if not split_e:
        return op
    return {L.AWQ_OP_SEARCH_SCALE: L.AWQ_OP_SEARCH_SCALE_SPLIT_E,
            L.AWQ_OP_SEARCH_CLIP: L.AWQ_OP_SEARCH_CLIP_SPLIT_E}.get(op, op)


def act_stats(X: torch.Tensor, ws: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Per-input-channel mean |x| over tokens: X [T, K] -> abar [K] float32."""
    _dev(X, "X")
    T, K = X.shape
    abar = out if out is not None else torch.empty(K, dtype=torch.float32, device=X.device)
    ws = _workspace(ws, workspace_bytes(L.AWQ_OP_STATS, T, 1, K, 1, X.dtype), X.device)
    L.check(L.lib().awq_act_stats(_ptr(X), _dtype(X), T, K, _ptr(abar), _ptr(ws), ws.numel(),
                                  _stream()))
    return abar


def act_stats_noalloc(X: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """act_stats through the entry point that allocates nothing (its partials
    live in a static device array shared by all such calls on a GPU; calls
    that overlap on one GPU race). ``out`` lets the caller avoid torch's
    allocation too."""
    _dev(X, "X")
    T, K = X.shape
    abar = out if out is not None else torch.empty(K, dtype=torch.float32, device=X.device)
    L.check(L.lib().awq_act_stats_noalloc(_ptr(X), _dtype(X), T, K, _ptr(abar), _stream()))
    return abar


def act_stats_accumulate(X: torch.Tensor, sums: torch.Tensor,
                         ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """sums[j] += Σ_t |x_tj| for one calibration batch X [T, K]; sums is a
    float64 [K] device tensor the caller zeroes before the first batch."""
    _dev(X, "X")
    _dev(sums, "sums")
    T, K = X.shape
    if sums.dtype != torch.float64 or sums.numel() != K:
        raise ValueError("sums must be a float64 tensor of K elements")
    ws = _workspace(ws, workspace_bytes(L.AWQ_OP_STATS, T, 1, K, 1, X.dtype), X.device)
    L.check(L.lib().awq_act_stats_accumulate(_ptr(X), _dtype(X), T, K, _ptr(sums), _ptr(ws),
                                             ws.numel(), _stream()))
    return sums


def act_stats_finalize(sums: torch.Tensor, count: int,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """abar_j = fl32(sums_j / count), count = all calibration tokens."""
    _dev(sums, "sums")
    K = sums.numel()
    abar = out if out is not None else torch.empty(K, dtype=torch.float32, device=sums.device)
    L.check(L.lib().awq_act_stats_finalize(_ptr(sums), count, K, _ptr(abar), _stream()))
    return abar


def scale_table(abar: torch.Tensor, alphas: Sequence[float]) -> torch.Tensor:
    """s[a][j] = abar_j^alpha_a / sqrt(max abar^alpha_a * min abar^alpha_a), float32."""
    _dev(abar, "abar")
    n = len(alphas)
    out = torch.empty((n, abar.numel()), dtype=torch.float32, device=abar.device)
    L.check(L.lib().awq_scale_table(_ptr(abar), abar.numel(), L.float_array(alphas), n, _ptr(out),
                                    _stream()))
    return out


_METHODS = ("direct", "gram")


def _method(method: str, G: Optional[torch.Tensor] = None) -> bool:
    if method not in _METHODS:
        raise ValueError(f"method must be one of {_METHODS}")
    if G is not None:
        if method != "gram":
            raise ValueError("a prepared Gram matrix G goes with method='gram'")
        _dev(G, "G")
    return method == "gram"


def gram_bytes(K: int) -> int:
    return int(L.lib().awq_gram_bytes(K))


def gram_build(X: torch.Tensor, ws: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """G = XᵀX of a bf16 layer input [T, K], in the layout the Gram searches
    read (a uint8 device buffer of gram_bytes(K) bytes). Pass it as ``G=`` to
    search_scale, search_clip and search_scale_group (method "gram") of every
    layer that reads X, instead of building it in each search."""
    _dev(X, "X")
    T, K = X.shape
    nbytes = gram_bytes(K)
    G = out if out is not None else torch.empty(nbytes, dtype=torch.uint8, device=X.device)
    ws = _workspace(ws, workspace_bytes(L.AWQ_OP_GRAM_BUILD, T, 1, K, 1, X.dtype), X.device)
    L.check(L.lib().awq_gram_build(_ptr(X), _dtype(X), T, K, _ptr(G), G.numel() * G.element_size(),
                                   _ptr(ws), ws.numel(), _stream()))
    return G


def search_scale(X: torch.Tensor, W: torch.Tensor, abar: torch.Tensor, alphas: Sequence[float],
                 bits: int = DEFAULT_BITS, group: int = DEFAULT_GROUP,
                 zero_point: bool = DEFAULT_ZERO_POINT, want_row_sums: bool = False,
                 ws: Optional[torch.Tensor] = None, method: str = "direct",
                 G: Optional[torch.Tensor] = None, split_e: bool = False,
                 fused: bool = False) -> dict:
    """Grid search over alpha. Returns alpha_best, index, s_best [K], mse (numpy
    [n_alpha]) and, if asked, row_sums [n_alpha, N] float64 on the GPU.
    method "direct" measures X·Eᵀ per candidate; "gram" (bf16 only) uses the
    activations' Gram matrix, E·G·Eᵀ per candidate row, built in the call or
    taken from ``G`` (gram_build(X)). split_e (direct method): candidates go
    to the matrix cores as hi + lo 16-bit halves (twice the GEMM work).
    fused (direct method, 16-bit, N a multiple of 256): the search GEMM forms
    the candidates itself from W and per-group parameters; same results."""
    gram = _method(method, G)
    _dev(X, "X"), _dev(W, "W"), _dev(abar, "abar")
    if X.dtype != W.dtype:
        raise ValueError("X and W must share a dtype")
    T, K = X.shape
    N = W.shape[0]
    n = len(alphas)
    op = (L.AWQ_OP_SEARCH_SCALE_GRAM_G if G is not None else
          L.AWQ_OP_SEARCH_SCALE_GRAM if gram else
          _direct_op(L.AWQ_OP_SEARCH_SCALE, split_e, fused))
    ws = _workspace(ws, workspace_bytes(op, T, N, K, n, X.dtype), X.device)
    s_best = torch.empty(K, dtype=torch.float32, device=X.device)
    rows = torch.empty((n, N), dtype=torch.float64, device=X.device) if want_row_sums else None
    a_best = ctypes.c_float(0.0)
    mse = (ctypes.c_double * n)()
    grid = L.float_array(alphas)
    fn = (L.lib().awq_search_scale_gram_g if G is not None else
          L.lib().awq_search_scale_gram if gram else L.lib().awq_search_scale)
    L.check(fn(_ptr(G if G is not None else X), _ptr(W), _dtype(X), T, N, K, _ptr(abar), grid, n,
               qconfig(bits, group, zero_point, split_e, fused), _ptr(s_best),
               ctypes.byref(a_best), mse, _ptr(rows), _ptr(ws), ws.numel(), _stream()))
    mse_np = np.array(mse[:], dtype=np.float64)
    g32 = np.asarray(alphas, dtype=np.float32)
    idx = int(np.flatnonzero(g32 == np.float32(a_best.value))[0])
    return dict(alpha_best=np.float32(a_best.value), index=idx, s_best=s_best, mse=mse_np,
                row_sums=rows)


def search_scale_group(X: torch.Tensor, Ws: Sequence[torch.Tensor], abar: torch.Tensor,
                       alphas: Sequence[float], bits: int = DEFAULT_BITS,
                       group: int = DEFAULT_GROUP, zero_point: bool = DEFAULT_ZERO_POINT,
                       want_row_sums: bool = False, ws: Optional[torch.Tensor] = None,
                       method: str = "direct", G: Optional[torch.Tensor] = None,
                       split_e: bool = False) -> dict:
    """One alpha search for linears that read the same X (one shared s): the
    error is averaged over all their outputs. Same result dict as
    ``search_scale``; row_sums [n_alpha, sum N] keeps the layers in order.
    method "gram" (bf16) scores all layers through one G = XᵀX (or ``G``)."""
    gram = _method(method, G)
    _dev(X, "X"), _dev(abar, "abar")
    if not 1 <= len(Ws) <= 16:
        raise ValueError("a group holds 1 to 16 layers")
    for i, W in enumerate(Ws):
        _dev(W, f"Ws[{i}]")
        if W.dtype != X.dtype or W.shape[1] != X.shape[1]:
            raise ValueError(f"Ws[{i}] must be [N, K] with X's dtype and K")
    T, K = X.shape
    Ns = [int(W.shape[0]) for W in Ws]
    N = sum(Ns)
    n = len(alphas)
    op = (L.AWQ_OP_SEARCH_SCALE_GRAM_G if G is not None else
          L.AWQ_OP_SEARCH_SCALE_GRAM if gram else _direct_op(L.AWQ_OP_SEARCH_SCALE, split_e))
    ws = _workspace(ws, workspace_bytes(op, T, N, K, n, X.dtype), X.device)
    s_best = torch.empty(K, dtype=torch.float32, device=X.device)
    rows = torch.empty((n, N), dtype=torch.float64, device=X.device) if want_row_sums else None
    a_best = ctypes.c_float(0.0)
    mse = (ctypes.c_double * n)()
    wptrs = (ctypes.c_void_p * len(Ws))(*[W.data_ptr() for W in Ws])
    nvals = (ctypes.c_int64 * len(Ws))(*Ns)
    fn = (L.lib().awq_search_scale_group_gram_g if G is not None else
          L.lib().awq_search_scale_group_gram if gram else L.lib().awq_search_scale_group)
    L.check(fn(_ptr(G if G is not None else X), wptrs, nvals, len(Ws), _dtype(X), T, K, _ptr(abar), L.float_array(alphas),
               n, qconfig(bits, group, zero_point, split_e), _ptr(s_best), ctypes.byref(a_best),
               mse,
               _ptr(rows), _ptr(ws), ws.numel(), _stream()))
    mse_np = np.array(mse[:], dtype=np.float64)
    g32 = np.asarray(alphas, dtype=np.float32)
    idx = int(np.flatnonzero(g32 == np.float32(a_best.value))[0])
    return dict(alpha_best=np.float32(a_best.value), index=idx, s_best=s_best, mse=mse_np,
                row_sums=rows)


def fold_norm(gamma: torch.Tensor, s: torch.Tensor, beta: Optional[torch.Tensor] = None) -> None:
    """In place: gamma /= s (and beta /= s) per channel, for the normalisation
    that produces the searched layer's input."""
    _dev(gamma, "gamma"), _dev(s, "s")
    if beta is not None:
        _dev(beta, "beta")
        if beta.dtype != gamma.dtype or beta.numel() != gamma.numel():
            raise ValueError("beta must match gamma")
    if s.dtype != torch.float32 or s.numel() != gamma.numel():
        raise ValueError("s must be float32 with one value per channel")
    L.check(L.lib().awq_fold_norm(_ptr(gamma), _ptr(beta), _dtype(gamma), gamma.numel(), _ptr(s),
                                  _stream()))


def fold_linear(W_prev: torch.Tensor, s: torch.Tensor, bias: Optional[torch.Tensor] = None) -> None:
    """In place: row j of W_prev [K, K_prev] (and bias[j]) /= s[j], for the
    linear whose outputs are the searched layer's inputs."""
    _dev(W_prev, "W_prev"), _dev(s, "s")
    K, K_prev = W_prev.shape
    if bias is not None:
        _dev(bias, "bias")
        if bias.dtype != W_prev.dtype or bias.numel() != K:
            raise ValueError("bias must be [K] with W_prev's dtype")
    if s.dtype != torch.float32 or s.numel() != K:
        raise ValueError("s must be float32 with one value per output channel of W_prev")
    L.check(L.lib().awq_fold_linear(_ptr(W_prev), _ptr(bias), _dtype(W_prev), K, K_prev, _ptr(s),
                                    _stream()))


def search_clip(X: torch.Tensor, W: torch.Tensor, s: torch.Tensor, ratios: Sequence[float],
                bits: int = DEFAULT_BITS, group: int = DEFAULT_GROUP,
                zero_point: bool = DEFAULT_ZERO_POINT, want_row_sums: bool = False,
                ws: Optional[torch.Tensor] = None, method: str = "direct",
                G: Optional[torch.Tensor] = None, split_e: bool = False,
                fused: bool = False) -> dict:
    """Per-output-channel clip-ratio search with s fixed. Returns ratio_best [N]
    (GPU), mse_clip (float) and optionally row_sums [n_ratio, N]. method, G,
    split_e and fused as in search_scale."""
    gram = _method(method, G)
    _dev(X, "X"), _dev(W, "W"), _dev(s, "s")
    if X.dtype != W.dtype:
        raise ValueError("X and W must share a dtype")
    T, K = X.shape
    N = W.shape[0]
    n = len(ratios)
    op = (L.AWQ_OP_SEARCH_CLIP_GRAM_G if G is not None else
          L.AWQ_OP_SEARCH_CLIP_GRAM if gram else
          _direct_op(L.AWQ_OP_SEARCH_CLIP, split_e, fused))
    ws = _workspace(ws, workspace_bytes(op, T, N, K, n, X.dtype), X.device)
    r_best = torch.empty(N, dtype=torch.float32, device=X.device)
    rows = torch.empty((n, N), dtype=torch.float64, device=X.device) if want_row_sums else None
    mse_clip = ctypes.c_double(0.0)
    fn = (L.lib().awq_search_clip_gram_g if G is not None else
          L.lib().awq_search_clip_gram if gram else L.lib().awq_search_clip)
    L.check(fn(_ptr(G if G is not None else X), _ptr(W), _dtype(X), T, N, K, _ptr(s), L.float_array(ratios), n,
               qconfig(bits, group, zero_point, split_e, fused), _ptr(r_best),
               ctypes.byref(mse_clip),
               _ptr(rows),
               _ptr(ws), ws.numel(), _stream()))
    return dict(ratio_best=r_best, mse_clip=float(mse_clip.value), row_sums=rows)


def quantize_pack(W: torch.Tensor, s: torch.Tensor, ratio: Optional[torch.Tensor] = None,
                  bits: int = DEFAULT_BITS, group: int = DEFAULT_GROUP,
                  zero_point: bool = DEFAULT_ZERO_POINT, ws: Optional[torch.Tensor] = None,
                  out=None):
    """Packed layer: qweight [K, N·b/32] int32, qzeros [K/g, N·b/32] int32,
    scales [K/g, N] float16 (b = bits, 4 or 3; codes packed densely along the
    output dim, lowest bits first)."""
    _dev(W, "W"), _dev(s, "s")
    if ratio is not None:
        _dev(ratio, "ratio")
    N, K = W.shape
    if out is None:
        nw = N * int(bits) // 32
        qweight = torch.empty((K, nw), dtype=torch.int32, device=W.device)
        qzeros = torch.empty((_groups(K, group), nw), dtype=torch.int32, device=W.device)
        scales = torch.empty((_groups(K, group), N), dtype=torch.float16, device=W.device)
    else:
        qweight, qzeros, scales = out
    ws = _workspace(ws, workspace_bytes(L.AWQ_OP_PACK, 1, N, K, 1, W.dtype), W.device)
    L.check(L.lib().awq_quantize_pack(_ptr(W), _dtype(W), N, K, _ptr(s), _ptr(ratio),
                                      qconfig(bits, group, zero_point), _ptr(qweight),
                                      _ptr(qzeros), _ptr(scales), _ptr(ws), ws.numel(), _stream()))
    return qweight, qzeros, scales


def w4a16_workspace_bytes(T: int, N: int, K: int, dtype: torch.dtype) -> int:
    return int(L.lib().awq_w4a16_workspace_bytes(T, N, K, _DT[dtype]))


def w3a16_workspace_bytes(T: int, N: int, K: int, dtype) -> int:
    return int(L.lib().awq_w3a16_workspace_bytes(T, N, K, _DT[dtype]))


def w4a16_matmul(X: torch.Tensor, qweight: torch.Tensor, qzeros: torch.Tensor,
                 scales: torch.Tensor, group: int = DEFAULT_GROUP,
                 ws: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                 bits: int = 4, on_the_fly: bool = False):
    """Y = X·Ŵᵀ for a packed layer (bits 4: qweight [K, N/8], qzeros
    [K/g, N/8]; bits 3: [K, 3N/32] and [K/g, 3N/32]; scales [K/g, N] float16)
    and activations X [T, K] (bf16 or float16, already divided by s). Returns
    Y [T, N] in X's dtype. on_the_fly (4 bits, T > 16): the GEMM dequantises
    as it goes and takes no workspace (same result, slower)."""
    _dev(X, "X"), _dev(qweight, "qweight"), _dev(qzeros, "qzeros"), _dev(scales, "scales")
    if bits not in (3, 4):
        raise ValueError("bits must be 3 or 4")
    T, K = X.shape
    N = scales.shape[1]
    cols = N * bits // 32
    G = _groups(K, group)
    if qweight.shape != (K, cols) or qzeros.shape != (G, cols) or scales.shape != (G, N):
        raise ValueError("packed layer shapes do not match X and the group size")
    Y = out if out is not None else torch.empty((T, N), dtype=X.dtype, device=X.device)
    if bits == 4:
        fn, need = L.lib().awq_w4a16_matmul, w4a16_workspace_bytes(T, N, K, X.dtype)
    else:
        fn, need = L.lib().awq_w3a16_matmul, w3a16_workspace_bytes(T, N, K, X.dtype)
    if on_the_fly and bits == 4 and T > 16:
        L.check(fn(_ptr(X), _dtype(X), T, N, K, _ptr(qweight), _ptr(qzeros), _ptr(scales),
                   int(group), _ptr(Y), None, 0, _stream()))
        return Y
    ws = _workspace(ws, need, X.device)
    L.check(fn(_ptr(X), _dtype(X), T, N, K, _ptr(qweight), _ptr(qzeros), _ptr(scales), int(group),
               _ptr(Y), _ptr(ws), ws.numel(), _stream()))
    return Y


def _check_on(device: int, names: Sequence[str], tensors) -> None:
    """Each tensor is a contiguous one on GPU number ``device``."""
    for name, t in zip(names, tensors):
        if isinstance(t, torch.Tensor) and t.get_device() == device and t.is_contiguous():
            continue
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        raise ValueError(f"{name} is on {t.device}, not on GPU {device}")


def _out(t: Optional[torch.Tensor], shape, dtype, like: torch.Tensor, name: str) -> torch.Tensor:
    """The caller's output buffer, checked, or a new one."""
    if t is None:
        return like.new_empty(shape, dtype=dtype)
    _check_on(like.get_device(), (name,), (t,))
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {tuple(shape)} {dtype}")
    return t


def _both(pair, name: str, of: str) -> None:
    """Two buffers that are filled together: in place of a missing one a new one would be
    filled and lost."""
    if len(pair) != 2 or any(t is None for t in pair):
        raise ValueError(f"{name} must be ({of}), both given")


def _call(device: int, fn, *args) -> None:
    """One call of the library on the current stream of GPU number ``device``,
    which need not be the current GPU."""
    if device == torch.cuda.current_device():
        L.check(fn(*args, torch._C._cuda_getCurrentRawStream(device)))
        return
    with torch.cuda.device(device):
        L.check(fn(*args, torch._C._cuda_getCurrentRawStream(device)))


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def w4a16_lora_workspace_bytes(T: int, N: int, K: int, L_: int, r: int,
                               dtype: torch.dtype) -> int:
    """Workspace of w4a16_lora_matmul for L_ adapters of rank r."""
    return int(L.lib().awq_w4a16_lora_workspace_bytes(T, N, K, L_, r, _DT[dtype]))


def w4a16_lora_backward_workspace_bytes(T: int, N: int, K: int, L_: int, r: int,
                                        dtype: torch.dtype) -> int:
    """Workspace of w4a16_lora_backward for L_ adapters of rank r."""
    return int(L.lib().awq_w4a16_lora_backward_workspace_bytes(T, N, K, L_, r, _DT[dtype]))


_LORA_NAMES = ("qweight", "qzeros", "scales", "A", "B", "scaling", "ids")


def _lora_args(V: torch.Tensor, V_cols: str, qweight, qzeros, scales, A, B, scaling, ids,
               group: int):
    """Checks what the forward and the backward call share; (T, N, K, L, r)."""
    _dev(V, V_cols)
    _check_on(V.get_device(), _LORA_NAMES, (qweight, qzeros, scales, A, B, scaling, ids))
    vs, qs, ss, az = V.shape, qweight.shape, scales.shape, A.shape
    if len(vs) != 2 or len(qs) != 2 or len(ss) != 2 or len(az) != 3:
        raise ValueError(f"{V_cols}, qweight and scales must have 2 dimensions, A 3")
    T, K, N = vs[0], qs[0], ss[1]
    n, r = az[0], az[1]
    G = _groups(K, group)
    if qs[1] * 8 != N or qzeros.shape != (G, N // 8) or \
            ss[0] != G or vs[1] != (K if V_cols == "X" else N):
        raise ValueError(f"packed layer shapes do not match {V_cols} and the group size")
    if qweight.dtype != torch.int32 or qzeros.dtype != torch.int32 or \
            scales.dtype != torch.float16:
        raise ValueError("qweight and qzeros must be int32, scales float16")
    if az[2] != K or B.shape != (n, N, r) or scaling.shape != (n,) or ids.shape != (T,):
        raise ValueError("adapters must be A [L, r, K], B [L, N, r], scaling [L], ids [T]")
    if A.dtype != V.dtype or B.dtype != V.dtype:
        raise ValueError(f"A and B must share {V_cols}'s dtype")
    if scaling.dtype != torch.float32 or ids.dtype != torch.int32:
        raise ValueError("scaling must be float32 and ids int32")
    return T, N, K, n, r


def w4a16_lora_matmul(X: torch.Tensor, qweight: torch.Tensor, qzeros: torch.Tensor,
                      scales: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                      scaling: torch.Tensor, ids: torch.Tensor, group: int = DEFAULT_GROUP,
                      ws: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                      h: Optional[torch.Tensor] = None, x8=None) -> torch.Tensor:
    """Low-rank adapters of many requests beside a packed 4-bit layer:
    Y[t] = Ŵ·x_t + scaling[a]·B[a]·(A[a]·x_t) with a = ids[t]; an id outside
    [0, L) means no adapter. X [T, K] (already divided by s) and the 4-bit
    layer as in w4a16_matmul, A [L, r, K] and B [L, N, r] in X's dtype,
    scaling [L] float32, ids [T] int32. Adapters of the unquantised layer
    enter with A times s, channel by channel. For training: ``h`` [T, r]
    float32 receives A[a]·x_t and ``x8`` = (codes, steps) the checkpoint of X
    that act_pack8 would make, both for w4a16_lora_backward. Returns Y [T, N] in X's dtype."""
    T, N, K, n, r = _lora_args(X, "X", qweight, qzeros, scales, A, B, scaling, ids, group)
    Y = _out(out, (T, N), X.dtype, X, "out")
    codes = steps = None
    if h is not None:
        _out(h, (T, r), torch.float32, X, "h")
    if x8 is not None:
        codes = _out(x8[0], (T, K), torch.int8, X, "x8 codes")
        steps = _out(x8[1], (T, K // 128), torch.float32, X, "x8 steps")
    device = X.get_device()
    if ws is None:
        ws = _workspace(ws, w4a16_lora_workspace_bytes(T, N, K, n, r, X.dtype), X.device)
    else:
        _check_on(device, ("ws",), (ws,))
    _call(device, L.lib().awq_w4a16_lora_matmul, X.data_ptr(), _dtype(X), T, N, K,
          qweight.data_ptr(), qzeros.data_ptr(), scales.data_ptr(), int(group), A.data_ptr(),
          B.data_ptr(), scaling.data_ptr(), ids.data_ptr(), n, r, Y.data_ptr(), _at(h),
          _at(codes), _at(steps), ws.data_ptr(), ws.nbytes)
    return Y


def w4a16_lora_backward(dY: torch.Tensor, X, h: torch.Tensor, qweight: torch.Tensor,
                        qzeros: torch.Tensor, scales: torch.Tensor, A: torch.Tensor,
                        B: torch.Tensor, scaling: torch.Tensor, ids: torch.Tensor,
                        group: int = DEFAULT_GROUP, ws: Optional[torch.Tensor] = None, out=None,
                        want_dx: bool = True):
    """The gradient of w4a16_lora_matmul: (dX [T, K], dA [L, r, K], dB
    [L, N, r]) in dY's dtype from dY [T, N], the ``h`` that the forward call
    wrote and X, its input or that input's checkpoint (codes, steps). dX
    takes Ŵ rounded to dY's dtype at every T; it is None with want_dx False.
    ``out`` = (dX, dA, dB) gives the buffers."""
    T, N, K, n, r = _lora_args(dY, "dY", qweight, qzeros, scales, A, B, scaling, ids, group)
    steps = None
    if isinstance(X, (tuple, list)):
        X, steps = X
        _dev(steps, "steps")
        _dev(X, "X")
        if X.dtype != torch.int8 or steps.dtype != torch.float32 or steps.shape != (T, K // 128):
            raise ValueError("a checkpoint is (codes [T, K] int8, steps [T, K / 128] float32)")
    else:
        _dev(X, "X")
        if X.dtype != dY.dtype:
            raise ValueError("X must share dY's dtype or be a checkpoint")
    if X.shape != (T, K):
        raise ValueError("X must be [T, K]")
    _dev(h, "h")
    device = dY.get_device()
    _check_on(device, ("X", "h"), (X, h))
    if steps is not None:
        _check_on(device, ("steps",), (steps,))
    if h.shape != (T, r) or h.dtype != torch.float32:
        raise ValueError("h must be [T, r] float32")
    dX, dA, dB = out if out is not None else (None, None, None)
    dX = _out(dX, (T, K), dY.dtype, dY, "dX") if want_dx else None
    dA = _out(dA, (n, r, K), dY.dtype, dY, "dA")
    dB = _out(dB, (n, N, r), dY.dtype, dY, "dB")
    if ws is None:
        ws = _workspace(ws, w4a16_lora_backward_workspace_bytes(T, N, K, n, r, dY.dtype),
                        dY.device)
    else:
        _check_on(device, ("ws",), (ws,))
    _call(device, L.lib().awq_w4a16_lora_backward, dY.data_ptr(), X.data_ptr(), _at(steps),
          h.data_ptr(), _dtype(dY), T, N, K, qweight.data_ptr(), qzeros.data_ptr(),
          scales.data_ptr(), int(group), A.data_ptr(), B.data_ptr(), scaling.data_ptr(),
          ids.data_ptr(), n, r, _at(dX), dA.data_ptr(), dB.data_ptr(), ws.data_ptr(), ws.nbytes)
    return dX, dA, dB


def act_pack8(X: torch.Tensor, out=None):
    """An 8-bit checkpoint of activations X [T, K] (bf16, float16 or float32,
    K a multiple of 128): (codes [T, K] int8, steps [T, K / 128] float32)
    with x ≈ code·step, step = max |x| / 127 over a token's 128 channels."""
    _dev(X, "X")
    T, K = X.shape
    codes, steps = out if out is not None else (None, None)
    codes = _out(codes, (T, K), torch.int8, X, "codes")
    steps = _out(steps, (T, K // 128), torch.float32, X, "steps")
    _call(X.get_device(), L.lib().awq_act_pack8, X.data_ptr(), _dtype(X), T, K, codes.data_ptr(),
          steps.data_ptr())
    return codes, steps


def act_unpack8(codes: torch.Tensor, steps: torch.Tensor, dtype: torch.dtype,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The activations that a checkpoint of act_pack8 stands for, code·step
    rounded once to ``dtype``."""
    _dev(codes, "codes"), _dev(steps, "steps")
    T, K = codes.shape
    if codes.dtype != torch.int8 or steps.dtype != torch.float32 or steps.shape != (T, K // 128):
        raise ValueError("a checkpoint is (codes [T, K] int8, steps [T, K / 128] float32)")
    X = _out(out, (T, K), dtype, codes, "out")
    device = codes.get_device()
    _check_on(device, ("steps",), (steps,))
    _call(device, L.lib().awq_act_unpack8, codes.data_ptr(), steps.data_ptr(), _dtype(X), T, K,
          X.data_ptr())
    return X


def quantize_rows8(X: torch.Tensor, s: Optional[torch.Tensor] = None, out=None):
    """Rows of X [T, K] (bf16, float16 or float32) in 8 bits with one step per
    row: (codes [T, K] int8, steps [T] float32), x·s ≈ code·step, step = max
    |x·s| / 127. A token's activations for w8a8_matmul, or, with output
    channels as rows and the scales ``s`` [K] float32 of a search, the 8-bit
    layer of W·diag(s) (its input is divided by s, as for the packed layer)."""
    _dev(X, "X")
    if X.dim() != 2:
        raise ValueError("X must be [T, K]")
    T, K = X.shape
    device = X.get_device()
    if s is not None:
        _check_on(device, ("s",), (s,))
        if s.dtype != torch.float32 or s.shape != (K,):
            raise ValueError("s must be float32 with one value per channel")
    codes, steps = out if out is not None else (None, None)
    codes = _out(codes, (T, K), torch.int8, X, "codes")
    steps = _out(steps, (T,), torch.float32, X, "steps")
    _call(device, L.lib().awq_quantize_rows8, X.data_ptr(), _dtype(X), T, K, _at(s),
          codes.data_ptr(), steps.data_ptr())
    return codes, steps


def _rows8(codes: torch.Tensor, steps: torch.Tensor, names=("codes", "steps")):
    """Checks 8-bit rows (codes [R, K] int8, steps [R] float32); (R, K, GPU number)."""
    _dev(codes, names[0])
    device = codes.get_device()
    _check_on(device, names[1:], (steps,))
    shape = codes.shape
    if len(shape) != 2 or codes.dtype != torch.int8 or steps.dtype != torch.float32 or \
            steps.shape != shape[:1]:
        raise ValueError(f"{names[0]} must be [rows, K] int8 and {names[1]} [rows] float32")
    return shape[0], shape[1], device


def dequantize_rows8(codes: torch.Tensor, steps: torch.Tensor, dtype: torch.dtype,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values that 8-bit rows stand for, code·step rounded once to ``dtype``."""
    T, K, device = _rows8(codes, steps)
    X = _out(out, (T, K), dtype, codes, "out")
    _call(device, L.lib().awq_dequantize_rows8, codes.data_ptr(), steps.data_ptr(), _dtype(X), T,
          K, X.data_ptr())
    return X


def _norm_weight(X: torch.Tensor, gamma: torch.Tensor, beta: Optional[torch.Tensor]) -> None:
    K = X.shape[1]
    _check_on(X.get_device(), ("gamma",), (gamma,))
    if gamma.shape != (K,) or (gamma.dtype != X.dtype and gamma.dtype != torch.float32):
        raise ValueError("gamma must be [K] in X's dtype or float32")
    if beta is not None:
        _check_on(X.get_device(), ("beta",), (beta,))
        if beta.shape != (K,) or beta.dtype != gamma.dtype:
            raise ValueError("beta must match gamma")


def layer_norm(X: torch.Tensor, gamma: torch.Tensor, beta: Optional[torch.Tensor] = None,
               eps: float = 1e-5, rms: bool = False, out: Optional[torch.Tensor] = None,
               stats: Optional[torch.Tensor] = None, rows8=None, want_y: bool = True):
    """The norm that precedes a layer (whose gamma and beta fold_norm divides):
    y = (x - mean)·r·gamma + beta with r = 1 / sqrt(mean (x - mean)² + eps)
    over each row of X [T, K]; with ``rms`` the mean is taken as 0. gamma and
    beta [K] in X's dtype or float32. ``stats`` [T, 2] float32 receives (mean,
    r) for layer_norm_backward, ``rows8`` = (codes [T, K] int8, steps [T]
    float32) the 8-bit rows of y for w8a8_matmul. Returns Y in X's dtype, or
    None with want_y False."""
    _dev(X, "X")
    if X.dim() != 2:
        raise ValueError("X must be [T, K]")
    T, K = X.shape
    _norm_weight(X, gamma, beta)
    Y = _out(out, (T, K), X.dtype, X, "out") if want_y else None
    codes = steps = None
    if stats is not None:
        _out(stats, (T, 2), torch.float32, X, "stats")
    if rows8 is not None:
        _both(rows8, "rows8", "codes, steps")
        codes = _out(rows8[0], (T, K), torch.int8, X, "rows8 codes")
        steps = _out(rows8[1], (T,), torch.float32, X, "rows8 steps")
    _call(X.get_device(), L.lib().awq_layer_norm, X.data_ptr(), _dtype(X), T, K, gamma.data_ptr(),
          _at(beta), _dtype(gamma), float(eps), int(bool(rms)), _at(Y), _at(stats), _at(codes),
          _at(steps))
    return Y


def layer_norm_backward_workspace_bytes(T: int, K: int) -> int:
    return int(L.lib().awq_layer_norm_backward_workspace_bytes(T, K))


def layer_norm_backward(dY: torch.Tensor, X: torch.Tensor, stats: torch.Tensor,
                        gamma: torch.Tensor, rms: bool = False, want_beta: bool = True,
                        ws: Optional[torch.Tensor] = None, out=None):
    """The gradient of layer_norm: (dX [T, K] in X's dtype, dgamma [K], dbeta
    [K] in gamma's dtype) from dY, the X and the ``stats`` of the forward call;
    dbeta is None with want_beta False. ``out`` = (dX, dgamma, dbeta) gives
    the buffers."""
    _dev(dY, "dY")
    if dY.dim() != 2:
        raise ValueError("dY must be [T, K]")
    T, K = dY.shape
    device = dY.get_device()
    _check_on(device, ("X", "stats"), (X, stats))
    if X.shape != dY.shape or X.dtype != dY.dtype:
        raise ValueError("X must share dY's shape and dtype")
    if stats.shape != (T, 2) or stats.dtype != torch.float32:
        raise ValueError("stats must be [T, 2] float32")
    _norm_weight(X, gamma, None)
    dX, dgamma, dbeta = out if out is not None else (None, None, None)
    dX = _out(dX, (T, K), dY.dtype, dY, "dX")
    dgamma = _out(dgamma, (K,), gamma.dtype, dY, "dgamma")
    dbeta = _out(dbeta, (K,), gamma.dtype, dY, "dbeta") if want_beta else None
    if ws is None:
        ws = _workspace(ws, layer_norm_backward_workspace_bytes(T, K), dY.device)
    else:
        _check_on(device, ("ws",), (ws,))
    _call(device, L.lib().awq_layer_norm_backward, dY.data_ptr(), X.data_ptr(), stats.data_ptr(),
          _dtype(dY), T, K, gamma.data_ptr(), _dtype(gamma), int(bool(rms)), dX.data_ptr(),
          dgamma.data_ptr(), _at(dbeta), ws.data_ptr(), ws.nbytes)
    return dX, dgamma, dbeta


_ACTS = {"silu": L.AWQ_ACT_SILU, "gelu": L.AWQ_ACT_GELU}


def _act(act: str) -> int:
    if act not in _ACTS:
        raise ValueError(f"act must be one of {tuple(_ACTS)}")
    return _ACTS[act]


def w8a8_workspace_bytes(T: int, N: int, K: int, layers: int = 1) -> int:
    """Workspace of w8a8_matmul (layers 1) or w8a8_gated_matmul (2)."""
    return int(L.lib().awq_w8a8_workspace_bytes(T, N, K, layers))


def w8a8_backward_workspace_bytes(T: int, N: int, K: int, layers: int = 1) -> int:
    """Workspace of w8a8_backward (layers 1) or w8a8_gated_backward (2)."""
    return int(L.lib().awq_w8a8_backward_workspace_bytes(T, N, K, layers))


def _w8_ws(ws: Optional[torch.Tensor], need: int, like: torch.Tensor):
    """(address, bytes) of the caller's workspace or of a new one, kept alive by the third."""
    if ws is not None:
        _check_on(like.get_device(), ("ws",), (ws,))
    elif need:
        ws = torch.empty(need, dtype=torch.uint8, device=like.device)
    return (None, 0, None) if ws is None else (ws.data_ptr(), ws.nbytes, ws)


def _pair(gate, up, K: Optional[int], device: int):
    """Checks a gated pair's layers; (N, K)."""
    N, Kg, on = _rows8(*gate, ("gate codes", "gate steps"))
    Nu, Ku, on_u = _rows8(*up, ("up codes", "up steps"))
    if on != device or on_u != device:
        raise ValueError(f"the layers are not on GPU {device}")
    if Nu != N or Ku != Kg or (K is not None and K != Kg):
        raise ValueError("gate and up must be [N, K] with the input's K")
    return N, Kg


def w8a8_matmul(codes: torch.Tensor, steps: torch.Tensor, qweight: torch.Tensor,
                wsteps: torch.Tensor, dtype: torch.dtype, bias: Optional[torch.Tensor] = None,
                ws: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y[t][n] = steps[t]·wsteps[n]·Σ_k codes[t][k]·qweight[n][k] + bias[n] for
    8-bit rows (quantize_rows8 or layer_norm's rows8) and an 8-bit layer
    (quantize_rows8 of W [N, K]). The sum is exact; Y [T, N] is rounded once to
    ``dtype`` (bf16 or float16), which bias [N] shares."""
    T, K, device = _rows8(codes, steps)
    N, Kw, on = _rows8(qweight, wsteps, ("qweight", "wsteps"))
    if on != device:
        raise ValueError(f"qweight is not on GPU {device}")
    if Kw != K:
        raise ValueError("qweight must be [N, K] with the rows' K")
    if bias is not None:
        _check_on(device, ("bias",), (bias,))
        if bias.shape != (N,) or bias.dtype != dtype:
            raise ValueError("bias must be [N] in dtype")
    Y = _out(out, (T, N), dtype, codes, "out")
    at, nbytes, _keep = _w8_ws(ws, w8a8_workspace_bytes(T, N, K), codes)
    _call(device, L.lib().awq_w8a8_matmul, codes.data_ptr(), steps.data_ptr(), T, N, K,
          qweight.data_ptr(), wsteps.data_ptr(), _at(bias), _dtype(Y), Y.data_ptr(), at, nbytes)
    return Y


def w8a8_gated_matmul(codes: torch.Tensor, steps: torch.Tensor, gate, up, dtype: torch.dtype,
                      act: str = "silu", ws: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, pre=None) -> torch.Tensor:
    """H = act(G)·U of two 8-bit layers of one input, ``gate`` and ``up`` =
    (codes [N, K] int8, steps [N] float32), G and U their products as in
    w8a8_matmul, held in float32 until H is rounded once. act "silu" or "gelu"
    (g·Φ(g)). ``pre`` = (G, U) [T, N] buffers in ``dtype`` receive the
    products, for w8a8_gated_backward."""
    T, K, device = _rows8(codes, steps)
    N, _ = _pair(gate, up, K, device)
    kind = _act(act)
    H = _out(out, (T, N), dtype, codes, "out")
    G = U = None
    if pre is not None:
        _both(pre, "pre", "G, U")
        G = _out(pre[0], (T, N), dtype, codes, "pre G")
        U = _out(pre[1], (T, N), dtype, codes, "pre U")
    at, nbytes, _keep = _w8_ws(ws, w8a8_workspace_bytes(T, N, K, 2), codes)
    _call(device, L.lib().awq_w8a8_gated_matmul, codes.data_ptr(), steps.data_ptr(), T, N, K,
          gate[0].data_ptr(), gate[1].data_ptr(), up[0].data_ptr(), up[1].data_ptr(), kind,
          _dtype(H), H.data_ptr(), _at(G), _at(U), at, nbytes)
    return H


def w8a8_backward(dY: torch.Tensor, qweight: torch.Tensor, wsteps: torch.Tensor,
                  ws: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of w8a8_matmul with respect to the values that its 8-bit
    rows stand for: dX [T, K] in dY's dtype from dY [T, N]. dY times the steps
    is rounded to fp16 under a power of two per row (2^-11 of a term), for
    either dtype; sums are float32."""
    N, K, device = _rows8(qweight, wsteps, ("qweight", "wsteps"))
    _check_on(device, ("dY",), (dY,))
    if dY.dim() != 2 or dY.shape[1] != N:
        raise ValueError("dY must be [T, N]")
    T = dY.shape[0]
    dX = _out(out, (T, K), dY.dtype, dY, "out")
    at, nbytes, _keep = _w8_ws(ws, w8a8_backward_workspace_bytes(T, N, K), dY)
    _call(device, L.lib().awq_w8a8_backward, dY.data_ptr(), _dtype(dY), T, N, K,
          qweight.data_ptr(), wsteps.data_ptr(), dX.data_ptr(), at, nbytes)
    return dX


def w8a8_gated_backward(dH: torch.Tensor, pre, gate, up, act: str = "silu",
                        ws: Optional[torch.Tensor] = None, out=None):
    """The gradient of w8a8_gated_matmul: (dX [T, K], dG, dU [T, N]) in dH's
    dtype from dH [T, N] and the ``pre`` = (G, U) that the forward call kept; dX
    with respect to the values that the 8-bit rows stand for, dG and dU those
    of the two products, which times the steps are rounded for dX as in
    w8a8_backward. ``out`` = (dX, dG, dU) gives the buffers."""
    _dev(dH, "dH")
    device = dH.get_device()
    N, K = _pair(gate, up, None, device)
    if dH.dim() != 2 or dH.shape[1] != N:
        raise ValueError("dH must be [T, N]")
    T = dH.shape[0]
    G, U = pre
    _check_on(device, ("pre G", "pre U"), (G, U))
    if G.shape != dH.shape or U.shape != dH.shape or G.dtype != dH.dtype or U.dtype != dH.dtype:
        raise ValueError("pre must be (G, U), each [T, N] in dH's dtype")
    kind = _act(act)
    dX, dG, dU = out if out is not None else (None, None, None)
    dX = _out(dX, (T, K), dH.dtype, dH, "dX")
    dG = _out(dG, (T, N), dH.dtype, dH, "dG")
    dU = _out(dU, (T, N), dH.dtype, dH, "dU")
    at, nbytes, _keep = _w8_ws(ws, w8a8_backward_workspace_bytes(T, N, K, 2), dH)
    _call(device, L.lib().awq_w8a8_gated_backward, dH.data_ptr(), G.data_ptr(), U.data_ptr(),
          _dtype(dH), T, N, K, gate[0].data_ptr(), gate[1].data_ptr(), up[0].data_ptr(),
          up[1].data_ptr(), kind, dX.data_ptr(), dG.data_ptr(), dU.data_ptr(), at, nbytes)
    return dX, dG, dU


def profile_enable(on: bool = True) -> None:
    L.lib().awq_profile_enable(1 if on else 0)


def profile_reset() -> None:
    L.lib().awq_profile_reset()


def profile_read(kind: str):
    """(total milliseconds, launches) of one kernel kind since the last reset."""
    ms = ctypes.c_double(0.0)
    n = ctypes.c_int64(0)
    L.check(L.lib().awq_profile_read(L.KERNEL_KINDS[kind], ctypes.byref(ms), ctypes.byref(n)))
    return ms.value, n.value
