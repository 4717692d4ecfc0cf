"""MI355X-native randomized per-sample gradient-norm estimation (libdpnorm).

For a linear-like layer with hooked activations A_i (T x d) and output
gradients G_i (T x p) of sample i, the squared per-sample gradient norm is
||A_i^T G_i||_F^2; the Hutchinson estimate with a shared Gaussian projection
P (p x k, entries of variance 1/k) is ||A_i^T (G_i P)||_F^2. Estimates are
summed over layers per sample and turned into clip factors min(C/sqrt(n), 1)
('Efficient DP-SGD for LLMs with Randomized Clipping', papernotes.org note,
方法详解 › 整体框架 and 关键设计 › Hutchinson).

This module is a thin binding: it checks torch tensors, takes their device
pointers, allocates the workspace the library asks for and calls the C ABI
of libdpnorm.so on torch's current HIP stream. Every step of the computation
runs in the library's HIP kernels; there is no other code path, and calls
fail loudly if the library is not built or no GPU is present.
"""
from __future__ import annotations

import ctypes as C
from typing import List, Optional, Sequence, Tuple

import torch

from . import _lib

__all__ = ["DpnormError", "hutch", "hutch_grouped", "hutchpp", "exact", "clip_factors", "hutchpp_split", "KernelTimer",
           "embed_lookup", "EmbedOrder", "embed_order", "embed_norm", "embed_grad", "attention_forward", "attention_backward",
           "layernorm_forward", "layernorm_backward", "layernorm_norm",
           "lib", "hutch_workspace", "hutch_grouped_workspace", "hutchpp_workspace", "exact_workspace"]


class DpnormError(RuntimeError):
    """A libdpnorm call returned a non-OK status."""

    def __init__(self, status: int, what: str):
        self.status = status
        msg = lib().dpnorm_status_string(status)
        super().__init__(f"{what}: {msg.decode() if msg else status}")


def lib() -> C.CDLL:
    return _lib.load()


def _check(status: int, what: str) -> None:
    if status != _lib.OK:
        raise DpnormError(status, what)


def _code(dtype: torch.dtype) -> int:
    if dtype == torch.bfloat16:
        return _lib.BF16
    if dtype == torch.float32:
        return _lib.F32
    raise TypeError(f"libdpnorm takes bfloat16 or float32 inputs, got {dtype}")


def _need(t: torch.Tensor, name: str, ndim: int, dtype: Optional[torch.dtype] = None) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (libdpnorm runs on the GPU only)")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


# The current stream's handle by device index; without the Stream object that
# torch.cuda.current_stream makes, which takes 2 us, a sixth of a small call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _stream(device: torch.device) -> int:
    return _raw_stream(device.index)


def _workspace(nbytes: int, device: torch.device) -> Tuple[Optional[torch.Tensor], int]:
    if nbytes == 0:
        return None, 0
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws, ws.data_ptr()


def _out(out: Optional[torch.Tensor], B: int, device: torch.device, accumulate: bool, name: str = "out"):
    if out is None:
        if accumulate:
            raise ValueError("accumulate=True needs an existing output tensor")
        return torch.empty(B, dtype=torch.float32, device=device)
    _need(out, name, 1, torch.float32)
    if out.shape[0] != B:
        raise ValueError(f"{name} must have {B} entries")
    return out


def _layer_array(layers: Sequence[Tuple[torch.Tensor, torch.Tensor, torch.Tensor]]):
    if len(layers) == 0:
        raise ValueError("at least one layer is needed")
    A0, G0, P0 = layers[0]
    _need(A0, "A", 3)
    dtype, device = A0.dtype, A0.device
    B, T = A0.shape[0], A0.shape[1]
    k = P0.shape[1] if P0.dim() == 2 else -1
    arr = (_lib.Layer * len(layers))()
    for j, (A, G, P) in enumerate(layers):
        _need(A, f"layers[{j}].A", 3, dtype)
        _need(G, f"layers[{j}].G", 3, dtype)
        _need(P, f"layers[{j}].P", 2, dtype)
        if A.device != device or G.device != device or P.device != device:
            raise ValueError("all tensors of a call must be on one device")
        if A.shape[:2] != (B, T) or G.shape[:2] != (B, T):
            raise ValueError(f"layers[{j}]: A and G must be [B={B}][T={T}][*]")
        if P.shape[0] != G.shape[2] or P.shape[1] != k:
            raise ValueError(f"layers[{j}]: P must be [p={G.shape[2]}][k={k}]")
        arr[j] = _lib.Layer(A.data_ptr(), G.data_ptr(), P.data_ptr(), A.shape[2], G.shape[2])
    return arr, dtype, device, B, T, k


def hutch(A: torch.Tensor, G: torch.Tensor, P: torch.Tensor, out: Optional[torch.Tensor] = None,
          accumulate: bool = False, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """n_hat_i = ||A_i^T (G_i P)||_F^2 for every sample (dpnorm_hutch).

    A [B][T][d], G [B][T][p], P [p][k], all bfloat16 or all float32, on the
    GPU and contiguous. Returns float32 [B]; with accumulate=True the
    estimates are added to ``out`` (the per-sample layer sum).
    """
    arr, dtype, device, B, T, k = _layer_array([(A, G, P)])
    L = lib()
    nbytes = C.c_size_t(0)
    _check(L.dpnorm_hutch_workspace(_code(dtype), B, T, A.shape[2], G.shape[2], k, C.byref(nbytes)),
           "dpnorm_hutch_workspace")
    n = _out(out, B, device, accumulate)
    ws, wsp = _given_workspace(workspace, nbytes.value, device)
    _check(L.dpnorm_hutch(A.data_ptr(), G.data_ptr(), P.data_ptr(), _code(dtype), B, T, A.shape[2], G.shape[2], k,
                          n.data_ptr(), int(accumulate), wsp, nbytes.value, _stream(device)), "dpnorm_hutch")
    return n


def hutch_workspace(dtype: torch.dtype, B: int, T: int, d: int, p: int, k: int) -> int:
    nbytes = C.c_size_t(0)
    _check(lib().dpnorm_hutch_workspace(_code(dtype), B, T, d, p, k, C.byref(nbytes)), "dpnorm_hutch_workspace")
    return nbytes.value


def hutch_grouped_workspace(layers, dtype: torch.dtype, B: int, T: int, k: int) -> int:
    """Workspace bytes of dpnorm_hutch_grouped for layer tensors or (d, p) pairs.

    Given the (A, G, P) tensors, the size is that of the call's own plan, in
    which layers sharing one A tensor share one pass over it. Given (d, p)
    pairs, it is the size without that sharing; a call with such a workspace
    still succeeds and then streams each A separately if it must.
    """
    arr = (_lib.Layer * len(layers))()
    for j, y in enumerate(layers):
        if isinstance(y[0], torch.Tensor):
            arr[j] = _lib.Layer(y[0].data_ptr(), y[1].data_ptr(), y[2].data_ptr(), y[0].shape[2], y[1].shape[2])
        else:
            arr[j] = _lib.Layer(None, None, None, int(y[0]), int(y[1]))
    nbytes = C.c_size_t(0)
    _check(lib().dpnorm_hutch_grouped_workspace(arr, len(layers), _code(dtype), B, T, k, C.byref(nbytes)),
           "dpnorm_hutch_grouped_workspace")
    return nbytes.value


def hutch_grouped(layers: Sequence[Tuple[torch.Tensor, torch.Tensor, torch.Tensor]],
                  out: Optional[torch.Tensor] = None, accumulate: bool = False, C_clip: Optional[float] = None,
                  clip_out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  timer: Optional["KernelTimer"] = None):
    """Per-sample sum over layers of the Hutchinson estimates (dpnorm_hutch_grouped).

    ``layers`` is a sequence of (A, G, P) triples sharing B, T, k and dtype.
    Returns n [B] float32, or (n, c) when ``C_clip`` is given, with
    c = min(C / sqrt(n), 1). ``workspace`` (uint8, GPU) may be passed to
    reuse one allocation across calls; ``timer`` records HIP events between
    the call's launches.
    """
    arr, dtype, device, B, T, k = _layer_array(layers)
    L = lib()
    nbytes = C.c_size_t(0)
    _check(L.dpnorm_hutch_grouped_workspace(arr, len(layers), _code(dtype), B, T, k, C.byref(nbytes)),
           "dpnorm_hutch_grouped_workspace")
    n = _out(out, B, device, accumulate)
    c = None
    if C_clip is not None:
        c = _out(clip_out, B, device, False, "clip_out") if clip_out is not None else torch.empty_like(n)
    if workspace is None:
        ws, wsp = _workspace(nbytes.value, device)
        ws_bytes = nbytes.value
    else:
        # the library decides whether a smaller workspace still fits a plan
        # without shared-input passes (see hutch_grouped_workspace)
        if not workspace.is_cuda:
            raise ValueError("workspace must be a GPU tensor")
        ws, wsp = workspace, workspace.data_ptr()
        ws_bytes = workspace.numel() * workspace.element_size()
    args = (arr, len(layers), _code(dtype), B, T, k, n.data_ptr(), int(accumulate),
            c.data_ptr() if c is not None else None, float(C_clip) if C_clip is not None else 1.0,
            wsp, ws_bytes, _stream(device))
    if timer is None:
        _check(L.dpnorm_hutch_grouped(*args), "dpnorm_hutch_grouped")
    else:
        tr = timer._trace()
        _check(L.dpnorm_hutch_grouped_traced(*args, C.byref(tr)), "dpnorm_hutch_grouped_traced")
        timer._record(tr)
    return (n, c) if c is not None else n


def random_signs(p: int, k: int, device="cuda", generator: Optional[torch.Generator] = None) -> torch.Tensor:
    """Uniformly random 32-bit words [p][ceil(k/32)] (int32 storage): the
    bit-packed i.i.d. Rademacher signs of a +-1 projection (see hutch_sign)."""
    return torch.randint(-2 ** 31, 2 ** 31, (p, (k + 31) // 32), dtype=torch.int32, device=device,
                         generator=generator)


def _sign_layer_array(layers, k: int):
    if len(layers) == 0:
        raise ValueError("at least one layer is needed")
    A0 = layers[0][0]
    _need(A0, "A", 3)
    dtype, device = A0.dtype, A0.device
    B, T = A0.shape[0], A0.shape[1]
    if not 1 <= k <= 64:
        raise ValueError("k must be in 1..64")
    arr = (_lib.Layer * len(layers))()
    for j, (A, G, S) in enumerate(layers):
        _need(A, f"layers[{j}].A", 3, dtype)
        _need(G, f"layers[{j}].G", 3, dtype)
        _need(S, f"layers[{j}].S_bits", 2, torch.int32)
        if A.device != device or G.device != device or S.device != device:
            raise ValueError("all tensors of a call must be on one device")
        if A.shape[:2] != (B, T) or G.shape[:2] != (B, T):
            raise ValueError(f"layers[{j}]: A and G must be [B={B}][T={T}][*]")
        if tuple(S.shape) != (G.shape[2], (k + 31) // 32):
            raise ValueError(f"layers[{j}]: S_bits must be [p={G.shape[2]}][{(k + 31) // 32}] int32 words")
        arr[j] = _lib.Layer(A.data_ptr(), G.data_ptr(), S.data_ptr(), A.shape[2], G.shape[2])
    return arr, dtype, device, B, T


def hutch_sign(A: torch.Tensor, G: torch.Tensor, S_bits: torch.Tensor, k: int, out: Optional[torch.Tensor] = None,
               accumulate: bool = False, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """n_hat_i = ||A_i^T (G_i S)||_F^2 / k with S in {-1,+1}^{p x k} stored as
    bits (dpnorm_hutch_sign): S_bits is int32 [p][ceil(k/32)], bit j % 32 of
    word j // 32 of row v set for S[v][j] = -1."""
    _sign_layer_array([(A, G, S_bits)], k)
    B, T = A.shape[0], A.shape[1]
    L = lib()
    nbytes = C.c_size_t(0)
    _check(L.dpnorm_hutch_workspace(_code(A.dtype), B, T, A.shape[2], G.shape[2], k, C.byref(nbytes)),
           "dpnorm_hutch_workspace")
    n = _out(out, B, A.device, accumulate)
    ws, wsp = _given_workspace(workspace, nbytes.value, A.device)
    _check(L.dpnorm_hutch_sign(A.data_ptr(), G.data_ptr(), S_bits.data_ptr(), _code(A.dtype), B, T, A.shape[2],
                               G.shape[2], k, n.data_ptr(), int(accumulate), wsp, nbytes.value, _stream(A.device)),
           "dpnorm_hutch_sign")
    return n


def hutch_sign_grouped(layers, k: int, out: Optional[torch.Tensor] = None, accumulate: bool = False,
                       C_clip: Optional[float] = None, clip_out: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None):
    """hutch_grouped with +-1 projections (dpnorm_hutch_sign_grouped): layers
    are (A, G, S_bits) triples. Returns n, or (n, c) when C_clip is given."""
    arr, dtype, device, B, T = _sign_layer_array(layers, k)
    L = lib()
    nbytes = C.c_size_t(0)
    _check(L.dpnorm_hutch_grouped_workspace(arr, len(layers), _code(dtype), B, T, k, C.byref(nbytes)),
           "dpnorm_hutch_grouped_workspace")
    n = _out(out, B, device, accumulate)
    c = None
    if C_clip is not None:
        c = _out(clip_out, B, device, False, "clip_out") if clip_out is not None else torch.empty_like(n)
    if workspace is None:
        ws, wsp = _workspace(nbytes.value, device)
        ws_bytes = nbytes.value
    else:
        if not workspace.is_cuda:
            raise ValueError("workspace must be a GPU tensor")
        ws, wsp = workspace, workspace.data_ptr()
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(L.dpnorm_hutch_sign_grouped(arr, len(layers), _code(dtype), B, T, k, n.data_ptr(), int(accumulate),
                                       c.data_ptr() if c is not None else None,
                                       float(C_clip) if C_clip is not None else 1.0, wsp, ws_bytes,
                                       _stream(device)), "dpnorm_hutch_sign_grouped")
    return (n, c) if c is not None else n


def routes_exact(d: int, p: int, k: int) -> bool:
    """True when norms_routed computes a layer's exact norm (min(d, p) <= k)."""
    return min(d, p) <= k


def norms_routed(layers, k: int, out: Optional[torch.Tensor] = None, accumulate: bool = False,
                 C_clip: Optional[float] = None, clip_out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, return_routes: bool = False):
    """Per-sample sum over layers of the exact norm (layers with min(d, p) <= k)
    or the Hutchinson estimate (the others), dpnorm_norms_routed. ``layers``
    are (A, G, P) triples; P may be None for exactly routed layers, else it
    is [p][k] of the inputs' type. Returns n, (n, c) with C_clip, and the
    per-layer routes (1 exact, 0 estimated) last when return_routes."""
    if len(layers) == 0:
        raise ValueError("at least one layer is needed")
    A0 = layers[0][0]
    _need(A0, "A", 3)
    dtype, device = A0.dtype, A0.device
    B, T = A0.shape[0], A0.shape[1]
    arr = (_lib.Layer * len(layers))()
    for j, (A, G, P) in enumerate(layers):
        _need(A, f"layers[{j}].A", 3, dtype)
        _need(G, f"layers[{j}].G", 3, dtype)
        if A.shape[:2] != (B, T) or G.shape[:2] != (B, T):
            raise ValueError(f"layers[{j}]: A and G must be [B={B}][T={T}][*]")
        if P is None:
            if not routes_exact(A.shape[2], G.shape[2], k):
                raise ValueError(f"layers[{j}]: P is needed (min(d, p) > k)")
        else:
            _need(P, f"layers[{j}].P", 2, dtype)
            if tuple(P.shape) != (G.shape[2], k):
                raise ValueError(f"layers[{j}]: P must be [p={G.shape[2]}][k={k}]")
        arr[j] = _lib.Layer(A.data_ptr(), G.data_ptr(), P.data_ptr() if P is not None else None, A.shape[2],
                            G.shape[2])
    L = lib()
    nbytes = C.c_size_t(0)
    _check(L.dpnorm_norms_routed_workspace(arr, len(layers), _code(dtype), B, T, k, C.byref(nbytes)),
           "dpnorm_norms_routed_workspace")
    n = _out(out, B, device, accumulate)
    c = None
    if C_clip is not None:
        c = _out(clip_out, B, device, False, "clip_out") if clip_out is not None else torch.empty_like(n)
    ws, wsp = _given_workspace(workspace, nbytes.value, device)
    routes = (C.c_int32 * len(layers))()
    _check(L.dpnorm_norms_routed(arr, len(layers), _code(dtype), B, T, k, n.data_ptr(), int(accumulate),
                                 c.data_ptr() if c is not None else None,
                                 float(C_clip) if C_clip is not None else 1.0, routes, wsp, nbytes.value,
                                 _stream(device)), "dpnorm_norms_routed")
    res = (n, c) if c is not None else (n,)
    if return_routes:
        res = res + (list(routes),)
    return res if len(res) > 1 else res[0]


def read_probe(buf: torch.Tensor) -> None:
    """Calibration: stream the whole of ``buf`` (a contiguous GPU tensor whose
    size is a multiple of 16384 bytes) once with the stage kernels' direct
    global-to-LDS loads (dpnorm_read_probe); time it to get that path's read
    rate."""
    if not buf.is_cuda or not buf.is_contiguous():
        raise ValueError("buf must be a contiguous GPU tensor")
    _check(lib().dpnorm_read_probe(buf.data_ptr(), buf.numel() * buf.element_size(), _stream(buf.device)),
           "dpnorm_read_probe")


_ROUTES = {"auto": _lib.EXACT_AUTO, "explicit": _lib.EXACT_EXPLICIT, "gram": _lib.EXACT_GRAM}


def _given_workspace(workspace: Optional[torch.Tensor], nbytes: int, device: torch.device):
    if workspace is None:
        return _workspace(nbytes, device)
    if not workspace.is_cuda or workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError(f"workspace must be a GPU tensor of at least {nbytes} bytes")
    return workspace, workspace.data_ptr()


def hutchpp_workspace(dtype: torch.dtype, B: int, T: int, d: int, p: int, k: int) -> int:
    nbytes = C.c_size_t(0)
    _check(lib().dpnorm_hutchpp_workspace(_code(dtype), B, T, d, p, k, C.byref(nbytes)), "dpnorm_hutchpp_workspace")
    return nbytes.value


def exact_workspace(dtype: torch.dtype, B: int, T: int, d: int, p: int, route: str = "auto") -> int:
    nbytes = C.c_size_t(0)
    _check(lib().dpnorm_exact_workspace(_code(dtype), B, T, d, p, _ROUTES[route], C.byref(nbytes)),
           "dpnorm_exact_workspace")
    return nbytes.value


def hutchpp(A: torch.Tensor, G: torch.Tensor, S: torch.Tensor, P: torch.Tensor, k: Optional[int] = None,
            out: Optional[torch.Tensor] = None, accumulate: bool = False, return_parts: bool = False,
            workspace: Optional[torch.Tensor] = None, return_residuals: bool = False):
    """Hutch++ estimate with total budget k (dpnorm_hutchpp).

    S [p][m_s] is the sketch and P [p][m_t] the tail projection, with
    (m_s, m_t) = hutchpp_split(k); by default k = 2 m_s + m_t from the
    shapes. Returns n [B], or (n, head, tail, rank) with return_parts;
    return_residuals appends resid [B][m_s], the relative residual of each
    sketch column that the rank rule compared with its threshold.
    ``workspace`` (uint8, GPU) may be passed to reuse one allocation.
    """
    _need(A, "A", 3)
    dtype, device = A.dtype, A.device
    _need(G, "G", 3, dtype)
    _need(S, "S", 2, dtype)
    _need(P, "P", 2, dtype)
    B, T, d = A.shape
    p = G.shape[2]
    if G.shape[:2] != (B, T) or S.shape[0] != p or P.shape[0] != p:
        raise ValueError("shapes must be A [B][T][d], G [B][T][p], S [p][m_s], P [p][m_t]")
    if k is None:
        k = 2 * S.shape[1] + P.shape[1]
    ms, mt = hutchpp_split(k)
    if S.shape[1] != ms or P.shape[1] != mt:
        raise ValueError(f"budget {k} needs S with {ms} and P with {mt} columns")
    L = lib()
    nbytes = C.c_size_t(0)
    _check(L.dpnorm_hutchpp_workspace(_code(dtype), B, T, d, p, k, C.byref(nbytes)), "dpnorm_hutchpp_workspace")
    n = _out(out, B, device, accumulate)
    head = torch.empty(B, dtype=torch.float32, device=device) if return_parts else None
    tail = torch.empty(B, dtype=torch.float32, device=device) if return_parts else None
    rank = torch.empty(B, dtype=torch.int32, device=device) if return_parts else None
    resid = torch.empty(B, ms, dtype=torch.float32, device=device) if return_residuals else None
    ws, wsp = _given_workspace(workspace, nbytes.value, device)
    ptr = lambda t: t.data_ptr() if t is not None else None
    _check(L.dpnorm_hutchpp(A.data_ptr(), G.data_ptr(), S.data_ptr(), P.data_ptr(), _code(dtype), B, T, d, p, k,
                            n.data_ptr(), int(accumulate), ptr(head), ptr(tail), ptr(rank), ptr(resid), wsp,
                            nbytes.value, _stream(device)), "dpnorm_hutchpp")
    out_ = (n, head, tail, rank) if return_parts else (n,)
    if return_residuals:
        out_ = out_ + (resid,)
    return out_ if len(out_) > 1 else n


def exact(A: torch.Tensor, G: torch.Tensor, route: str = "auto", out: Optional[torch.Tensor] = None,
          accumulate: bool = False, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Exact n_i = ||A_i^T G_i||_F^2 (dpnorm_exact); route 'auto', 'explicit' or 'gram'."""
    _need(A, "A", 3)
    dtype, device = A.dtype, A.device
    _need(G, "G", 3, dtype)
    B, T, d = A.shape
    p = G.shape[2]
    if G.shape[:2] != (B, T):
        raise ValueError("A and G must be [B][T][*]")
    r = _ROUTES[route]
    L = lib()
    nbytes = C.c_size_t(0)
    _check(L.dpnorm_exact_workspace(_code(dtype), B, T, d, p, r, C.byref(nbytes)), "dpnorm_exact_workspace")
    n = _out(out, B, device, accumulate)
    ws, wsp = _given_workspace(workspace, nbytes.value, device)
    _check(L.dpnorm_exact(A.data_ptr(), G.data_ptr(), _code(dtype), B, T, d, p, r, n.data_ptr(), int(accumulate), wsp,
                          nbytes.value, _stream(device)), "dpnorm_exact")
    return n


def clip_factors(n: torch.Tensor, C_clip: float, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """c_i = min(C / sqrt(n_i), 1) (dpnorm_clip_factors); ``out`` may be ``n``."""
    _need(n, "n", 1, torch.float32)
    c = torch.empty_like(n) if out is None else out
    _need(c, "out", 1, torch.float32)
    _check(lib().dpnorm_clip_factors(n.data_ptr(), n.shape[0], float(C_clip), c.data_ptr(), _stream(n.device)),
           "dpnorm_clip_factors")
    return c


def hutchpp_split(k: int) -> Tuple[int, int]:
    """Hutch++ budget split (m_s, m_t) used by the library."""
    ms, mt = C.c_int64(0), C.c_int64(0)
    _check(lib().dpnorm_hutchpp_split(k, C.byref(ms), C.byref(mt)), "dpnorm_hutchpp_split")
    return ms.value, mt.value


# ---------------------------------------------------------------------------
# Around the linear layers: the embedding table, causal attention and norm layers. The calls
# run on the current stream of the tensors' device; temporaries come from
# torch's allocator on that stream.
# ---------------------------------------------------------------------------
def _run(device: torch.device, name: str, *args) -> None:
    """One library call on `device` and its current stream."""
    if torch.cuda.current_device() == device.index:
        status = getattr(lib(), name)(*args, _stream(device))
    else:
        with torch.cuda.device(device):
            status = getattr(lib(), name)(*args, _stream(device))
    if status != _lib.OK:
        raise DpnormError(status, name)


def _one_device(device: torch.device, *tensors) -> None:
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError("all tensors of a call must be on one device")


_INDEX = {torch.int64: _lib.I64, torch.int32: _lib.I32}


def _index(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in _INDEX:
        raise TypeError(f"{name} must be int32 or int64, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (libdpnorm runs on the GPU only)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _INDEX[t.dtype]


def embed_lookup(tokens: torch.Tensor, W: torch.Tensor, scale: float = 1.0,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """scale * W[tokens], rounded once to W's type (dpnorm_embed_lookup).

    tokens: int32 or int64 of any shape; W [V][d] bfloat16 or float32. An id
    outside [0, V) gives a zero row. Returns tokens.shape + (d,).
    """
    it = _index(tokens, "tokens")
    _need(W, "W", 2)
    code = _code(W.dtype)
    V, d = W.shape
    shape = (*tokens.shape, d)
    if out is None:
        out = torch.empty(shape, dtype=W.dtype, device=W.device)
    else:
        _need(out, "out", len(shape), W.dtype)
        if out.shape != shape:
            raise ValueError(f"out must be {list(shape)}")
    _one_device(W.device, tokens, out)
    n = tokens.numel()
    if n * d > 0:
        _run(W.device, "dpnorm_embed_lookup", tokens.data_ptr(), it, W.data_ptr(), code, n, V, d, scale, out.data_ptr())
    return out


class EmbedOrder:
    """The order of a batch's ids [B][T] for a table of V rows
    (dpnorm_embed_order), read by embed_norm and embed_grad. It describes the
    ids at the time of the call that made it."""

    def __init__(self, B: int, T: int, V: int, data: torch.Tensor):
        self.B, self.T, self.V, self.data = B, T, V, data


def embed_order(tokens: torch.Tensor, V: int) -> EmbedOrder:
    """Groups the positions of tokens [B][T] by id, for any number of
    embed_norm and embed_grad calls on the same ids."""
    it = _index(tokens, "tokens")
    if tokens.dim() != 2:
        raise ValueError(f"tokens must have 2 dimensions, got shape {tuple(tokens.shape)}")
    B, T = tokens.shape
    if B * T == 0:
        if not 1 <= V <= 1 << 30:
            raise ValueError("V must be in 1 .. 2^30")
        return EmbedOrder(B, T, V, torch.empty(0, dtype=torch.uint8, device=tokens.device))
    ob, wb = C.c_size_t(0), C.c_size_t(0)
    _check(lib().dpnorm_embed_order_sizes(B, T, V, C.byref(ob), C.byref(wb)), "dpnorm_embed_order_sizes")
    data = torch.empty(ob.value, dtype=torch.uint8, device=tokens.device)
    ws, wsp = _workspace(wb.value, tokens.device)
    _run(tokens.device, "dpnorm_embed_order", tokens.data_ptr(), it, B, T, V, data.data_ptr(), ob.value, wsp, wb.value)
    return EmbedOrder(B, T, V, data)


def _embed_ids(tokens, G: torch.Tensor, V: Optional[int]):
    """(tok pointer, index type, order pointer, ordered, V) of a norm or gradient call."""
    _need(G, "G", 3)
    if isinstance(tokens, EmbedOrder):
        if V is not None and V != tokens.V:
            raise ValueError(f"the order is of a table of {tokens.V} rows, not {V}")
        shape, V, res = (tokens.B, tokens.T), tokens.V, (None, 0, tokens.data.data_ptr(), 1, tokens.V)
        _one_device(G.device, tokens.data)
    else:
        it = _index(tokens, "tokens")
        if tokens.dim() != 2:
            raise ValueError(f"tokens must have 2 dimensions, got shape {tuple(tokens.shape)}")
        if V is None:
            raise ValueError("V (the rows of the table) is needed with token ids")
        shape, res = tokens.shape, (tokens.data_ptr(), it, None, 0, V)
        _one_device(G.device, tokens)
    if tuple(G.shape[:2]) != tuple(shape):
        raise ValueError(f"G must be [B={shape[0]}][T={shape[1]}][*]")
    return res


def embed_norm(tokens, G: torch.Tensor, V: Optional[int] = None, scale: float = 1.0, out: Optional[torch.Tensor] = None,
               accumulate: bool = False, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Exact squared per-sample gradient norm of an embedding table
    (dpnorm_embed_norm): n_i = scale^2 sum_v ||sum_{t: tokens[i, t] = v} G[i, t]||^2.

    tokens: the ids [B][T] (then V, the table's rows, is needed) or their
    EmbedOrder. G [B][T][d]: the gradient of the lookup's output. Returns
    float32 [B]; with accumulate=True the norms are added to ``out``.
    """
    tok, it, order, ordered, V = _embed_ids(tokens, G, V)
    code, (B, T, d), device = _code(G.dtype), G.shape, G.device
    n = _out(out, B, device, accumulate)
    _one_device(device, n)
    if B * T * d == 0:
        return n if accumulate else n.zero_()
    nbytes = C.c_size_t(0)
    _check(lib().dpnorm_embed_norm_workspace(code, B, T, V, d, ordered, C.byref(nbytes)), "dpnorm_embed_norm_workspace")
    ws, wsp = _given_workspace(workspace, nbytes.value, device)
    _run(device, "dpnorm_embed_norm", tok, it, order, G.data_ptr(), code, B, T, V, d, scale, n.data_ptr(), int(accumulate),
         wsp, nbytes.value)
    return n


def embed_grad(tokens, G: torch.Tensor, V: Optional[int] = None, scale: float = 1.0,
               weights: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, accumulate: bool = False,
               workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of an embedding table [V][d] in G's type (dpnorm_embed_grad):
    scale * sum_i weights_i sum_{t: tokens[i, t] = v} G[i, t] in row v.

    tokens, V, G as for embed_norm; weights: float32 [B] (clip factors), or
    None for 1. With accumulate=True the rows of the ids that occur are added
    to ``out`` and its other rows are left as they are.
    """
    tok, it, order, ordered, V = _embed_ids(tokens, G, V)
    code, (B, T, d), device = _code(G.dtype), G.shape, G.device
    if weights is not None:
        _need(weights, "weights", 1, torch.float32)
        if weights.shape[0] != B:
            raise ValueError(f"weights must have {B} entries")
    if out is None:
        if accumulate:
            raise ValueError("accumulate=True needs an existing output tensor")
        out = torch.empty(V, d, dtype=G.dtype, device=device)
    else:
        _need(out, "out", 2, G.dtype)
        if tuple(out.shape) != (V, d):
            raise ValueError(f"out must be [V={V}][d={d}]")
    _one_device(device, weights, out)
    if B * T * d == 0:
        return out if accumulate else out.zero_()
    nbytes = C.c_size_t(0)
    _check(lib().dpnorm_embed_grad_workspace(code, B, T, V, d, ordered, C.byref(nbytes)), "dpnorm_embed_grad_workspace")
    ws, wsp = _given_workspace(workspace, nbytes.value, device)
    _run(device, "dpnorm_embed_grad", tok, it, order, G.data_ptr(), code, B, T, V, d, scale,
         weights.data_ptr() if weights is not None else None, out.data_ptr(), int(accumulate), wsp, nbytes.value)
    return out


def _heads(t: torch.Tensor, name: str, dtype: torch.dtype, device: torch.device, shape) -> _lib.AttnTensor:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device or device.type != "cuda":
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor (libdpnorm runs on the GPU only)")
        raise ValueError("all tensors of a call must be on one device")
    if t.shape != shape:
        raise ValueError(f"{name} must be [N][heads][D] = {list(shape)}, got {list(t.shape)}")
    st, sh, sd = t.stride()
    if sd != 1 and shape[2] > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return _lib.AttnTensor(t.data_ptr(), st, sh)


def _attn_shape(q, k, v, cu_seqlens, sequences, scale, clear):
    """The shape record, and q's, k's and v's."""
    for t, name in ((q, "q"), (k, "k")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if t.dim() != 3:
            raise ValueError(f"{name} must be [N][heads][D], got shape {tuple(t.shape)}")
    code, dtype, device = _code(q.dtype), q.dtype, q.device
    N, Hq, D = q.shape
    Hkv = k.shape[1]
    if Hkv == 0 or Hq % Hkv != 0:
        raise ValueError(f"{Hq} query heads are not a multiple of {Hkv} key heads")
    kv = torch.Size((N, Hkv, D))
    tq, tk, tv = _heads(q, "q", dtype, device, q.shape), _heads(k, "k", dtype, device, kv), _heads(v, "v", dtype, device, kv)
    if cu_seqlens is not None:
        if sequences is not None:
            raise ValueError("give cu_seqlens or sequences, not both")
        _need(cu_seqlens, "cu_seqlens", 1, torch.int32)
        if cu_seqlens.device != device or cu_seqlens.shape[0] < 1:
            raise ValueError("cu_seqlens must be the S + 1 row offsets on the tensors' device")
        S, cup = cu_seqlens.shape[0] - 1, cu_seqlens.data_ptr()
    else:
        S, cup = (1 if sequences is None else int(sequences)), None
        if S < 1 or N % S != 0:
            raise ValueError(f"{N} rows are not a multiple of {S} sequences")
    if scale is None:
        scale = D ** -0.5 if D else 1.0
    return _lib.AttnShape(code, N, S, Hq, Hkv, D, cup, scale, int(clear)), tq, tk, tv


def _attn_scores(cap: Optional[float], slopes: Optional[torch.Tensor], prefix: Optional[torch.Tensor],
                 shape: _lib.AttnShape, device: torch.device) -> Optional[_lib.AttnScores]:
    """The record of changed scores; None where they are not."""
    if slopes is None and prefix is None and not cap:
        return None
    sp = pp = None
    if slopes is not None:
        _need(slopes, "slopes", 1, torch.float32)
        if slopes.shape[0] != shape.Hq:
            raise ValueError(f"slopes must have an entry for each of the {shape.Hq} query heads")
        sp = slopes.data_ptr()
    if prefix is not None:
        _need(prefix, "prefix", 1, torch.int32)
        if prefix.shape[0] != shape.S:
            raise ValueError(f"prefix must have an entry for each of the {shape.S} sequences")
        pp = prefix.data_ptr()
    _one_device(device, slopes, prefix)
    return _lib.AttnScores(cap or 0.0, sp, pp)


def attention_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
                      sequences: Optional[int] = None, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                      lse: Optional[torch.Tensor] = None, cap: Optional[float] = None, slopes: Optional[torch.Tensor] = None,
                      prefix: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Causal attention of packed sequences (dpnorm_attention_forward).

    q [N][Hq][D], k and v [N][Hkv][D], bfloat16 or float32, token and head
    strides of any multiples of 16 bytes; Hq a multiple of Hkv. cu_seqlens: int32 [S + 1] row offsets on
    the GPU; without it the N rows are ``sequences`` (default 1) sequences of
    equal length. scale defaults to 1 / sqrt(D). Returns (o [N][Hq][D],
    lse float32 [Hq][N]). Sums are float32; bfloat16 calls round the softmax
    weights to bfloat16 before they multiply v. Rows that belong to no sequence are left as they
    are in a given ``out`` and ``lse`` (give both or neither), and are zero
    where the call makes them.

    Scores may be changed before the softmax (dpnorm_attention_scores_forward):
    cap, in 1/1024 .. 1024, makes a score s cap * tanh(s / cap); slopes, float32
    [Hq] on the GPU, of up to 2^32, adds -slopes[h] * |t - u| for row t and key u (below zero,
    |slope| (length - 1) is at most 2^14; a steeper one gives NaN in its head and sequence);
    prefix, int32 [S] on the GPU, lets every row of a sequence see its first prefix[s] rows.
    """
    if (out is None) != (lse is None):
        raise ValueError("give out and lse both, or neither")
    shape, tq, tk, tv = _attn_shape(q, k, v, cu_seqlens, sequences, scale, out is None)
    N, Hq, D = q.shape
    device = q.device
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        lse = torch.empty((Hq, N), dtype=torch.float32, device=device)
    else:
        _need(lse, "lse", 2, torch.float32)
        if tuple(lse.shape) != (Hq, N) or lse.device != device:
            raise ValueError(f"lse must be [Hq={Hq}][N={N}] on q's device")
    to = _heads(out, "out", q.dtype, device, q.shape)
    scores = _attn_scores(cap, slopes, prefix, shape, device)
    if N > 0 and shape.S > 0:
        if scores is None:
            _run(device, "dpnorm_attention_forward", shape, tq, tk, tv, to, lse.data_ptr())
        else:
            _run(device, "dpnorm_attention_scores_forward", shape, scores, tq, tk, tv, to, lse.data_ptr())
    elif shape.clear_rest:
        out.zero_(), lse.zero_()
    return out, lse


def attention_backward(do: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                       lse: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None, sequences: Optional[int] = None,
                       scale: Optional[float] = None, out: Optional[Sequence[torch.Tensor]] = None,
                       workspace: Optional[torch.Tensor] = None, cap: Optional[float] = None,
                       slopes: Optional[torch.Tensor] = None,
                       prefix: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(dq, dk, dv) of attention_forward for the output gradient ``do``
    (dpnorm_attention_backward, dpnorm_attention_scores_backward). q, k, v,
    cu_seqlens, sequences, scale, cap, slopes and prefix are the forward call's, o and lse its results. Sums are float32; bfloat16 calls
    round p and ds to bfloat16 before they multiply rows. ``out``: three tensors to write
    to. Rows that belong to no sequence are left as they are in ``out``, and
    are zero where the call makes it.
    """
    shape, tq, tk, tv = _attn_shape(q, k, v, cu_seqlens, sequences, scale, out is None)
    N, Hq, D = q.shape
    dtype, device = q.dtype, q.device
    tdo, to = _heads(do, "do", dtype, device, q.shape), _heads(o, "o", dtype, device, q.shape)
    _need(lse, "lse", 2, torch.float32)
    if tuple(lse.shape) != (Hq, N) or lse.device != device:
        raise ValueError(f"lse must be [Hq={Hq}][N={N}] on q's device")
    if out is None:
        dq, dk, dv = (torch.empty_like(t, memory_format=torch.contiguous_format) for t in (q, k, v))
    else:
        dq, dk, dv = out
    tdq, tdk, tdv = (_heads(t, n, dtype, device, x.shape) for t, n, x in ((dq, "dq", q), (dk, "dk", k), (dv, "dv", k)))
    scores = _attn_scores(cap, slopes, prefix, shape, device)
    if N > 0 and shape.S > 0:
        nbytes = C.c_size_t(0)
        _check(lib().dpnorm_attention_scores_backward_workspace(shape, scores, C.byref(nbytes)),
               "dpnorm_attention_scores_backward_workspace")
        ws, wsp = _given_workspace(workspace, nbytes.value, device)
        rest = (tdo, tq, tk, tv, to, lse.data_ptr(), tdq, tdk, tdv, wsp, nbytes.value)
        if scores is None:
            _run(device, "dpnorm_attention_backward", shape, *rest)
        else:
            _run(device, "dpnorm_attention_scores_backward", shape, scores, *rest)
    elif shape.clear_rest:
        dq.zero_(), dk.zero_(), dv.zero_()
    return dq, dk, dv


def _normed(x: torch.Tensor, w: torch.Tensor, b: Optional[torch.Tensor]) -> int:
    """Checks rows x [..., d] and their gain and bias; the type's code."""
    _rows_of(x, "x")
    d, dtype = x.shape[-1], x.dtype
    for t, name in ((w, "weight"), (b, "bias")):
        if t is None and name == "bias":
            break
        _need(t, name, 1, dtype)
        if t.shape[0] != d:
            raise ValueError(f"{name} must have the {d} entries of a row")
        if t.device != x.device:
            raise ValueError("all tensors of a call must be on one device")
    return _code(dtype)


def _rows_of(t: torch.Tensor, name: str, like: Optional[torch.Tensor] = None) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dim() < 1:
        raise ValueError(f"{name} must have rows: [..., d]")
    _need(t, name, t.dim(), like.dtype if like is not None else None)
    if like is not None and t.shape != like.shape:
        raise ValueError(f"{name} must be {list(like.shape)}, got {list(t.shape)}")


def layernorm_forward(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
                      rms: bool = False, out: Optional[torch.Tensor] = None
                      ) -> Tuple[torch.Tensor, Optional[torch.Tensor], torch.Tensor]:
    """Layer norm (or, with rms=True, RMS norm) of the rows of x
    (dpnorm_layernorm_forward): (x - mean) rstd weight + bias.

    x [..., d], weight and bias [d], bfloat16 or float32, contiguous; d a
    multiple of 8 (bfloat16) or 4 (float32) up to 32768. Returns (y, mean, rstd), the
    statistics float32 [...], which layernorm_backward reads; RMS norm has
    no bias and its mean is None. Sums are float32; y is rounded once.
    """
    if rms and bias is not None:
        raise ValueError("RMS norm has no bias")
    code = _normed(x, weight, bias)
    d = x.shape[-1]
    if out is None:
        out = torch.empty_like(x)
    else:
        _rows_of(out, "out", x)
        _one_device(x.device, out)
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    mean = None if rms else torch.empty_like(rstd)
    n = rstd.numel()
    if n > 0:
        _run(x.device, "dpnorm_layernorm_forward", x.data_ptr(), weight.data_ptr(), bias.data_ptr() if bias is not None else None, code,
             int(rms), n, d, eps, out.data_ptr(), mean.data_ptr() if mean is not None else None, rstd.data_ptr())
    return out, mean, rstd


def layernorm_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, mean: Optional[torch.Tensor], rstd: torch.Tensor,
                       bias: bool = True, weights: Optional[torch.Tensor] = None, need_dx: bool = True, need_dw: bool = True,
                       workspace: Optional[torch.Tensor] = None
                       ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(dx, dweight, dbias) of layernorm_forward for the output's gradient dy
    (dpnorm_layernorm_backward); mean (None: RMS norm) and rstd are the forward
    call's. dbias is None for RMS norm and with bias=False; need_dx=False and
    need_dw=False leave out the others.

    weights: float32 [B] factors of the samples (clip factors) for dweight and
    dbias, x then being [B, ..., d]; they do not change dx. Sums are float32,
    each result is rounded once, and results are reproducible bit for bit.
    """
    code = _normed(x, weight, None)
    _rows_of(dy, "dy", x)
    d, device = x.shape[-1], x.device
    rms = mean is None
    bias = bias and not rms
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        if t is not None:
            _need(t, name, x.dim() - 1, torch.float32)
            if t.shape != x.shape[:-1]:
                raise ValueError(f"{name} must be {list(x.shape[:-1])}, got {list(t.shape)}")
    N, B = rstd.numel(), 1
    if weights is not None:
        _need(weights, "weights", 1, torch.float32)
        B = weights.shape[0]
        if x.dim() < 2 or x.shape[0] != B:
            raise ValueError(f"weights are of {B} samples, x must be [{B}, ..., d]")
    if not (need_dx or need_dw or bias):
        raise ValueError("no gradient is wanted")
    _one_device(device, dy, mean, rstd, weights)
    dx = torch.empty_like(x) if need_dx else None
    dw = torch.empty_like(weight) if need_dw else None
    db = torch.empty_like(weight) if bias else None
    if N * d == 0:
        for t in (dw, db):
            if t is not None:
                t.zero_()
        return dx, dw, db
    nbytes = C.c_size_t(0)
    _check(lib().dpnorm_layernorm_backward_workspace(code, int(rms), B, N // B, d, C.byref(nbytes)), "dpnorm_layernorm_backward_workspace")
    need = nbytes.value if need_dw or bias else 0
    ws, wsp = _given_workspace(workspace, need, device)
    ptr = lambda t: t.data_ptr() if t is not None else None
    _run(device, "dpnorm_layernorm_backward", dy.data_ptr(), x.data_ptr(), weight.data_ptr(), ptr(mean), rstd.data_ptr(), code, int(rms),
         B, N // B, d, ptr(weights), ptr(dx), ptr(dw), ptr(db), wsp, need)
    return dx, dw, db


def layernorm_norm(x: torch.Tensor, G: torch.Tensor, eps: float = 1e-5, rms: bool = False, gain: bool = True, bias: bool = True,
                   out: Optional[torch.Tensor] = None, accumulate: bool = False,
                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Exact squared per-sample gradient norm of a layer norm's gain and bias
    (dpnorm_layernorm_norm): n_i = ||sum_t G[i, t] h[i, t]||^2 + ||sum_t G[i, t]||^2
    with h the normalised rows of x.

    x [B][T][d] the norm's input, G [B][T][d] the gradient of its output.
    gain, bias: whose gradients count (RMS norm has no bias). Returns
    float32 [B]; with accumulate=True the norms are added to ``out``.
    """
    _need(x, "x", 3)
    _need(G, "G", 3, x.dtype)
    if G.shape != x.shape:
        raise ValueError(f"G must be {list(x.shape)}, got {list(G.shape)}")
    parts = (_lib.LN_GAIN if gain else 0) | (_lib.LN_BIAS if bias and not rms else 0)
    if parts == 0:
        raise ValueError("neither the gain's gradient nor a bias's is wanted")
    code, (B, T, d), device = _code(x.dtype), x.shape, x.device
    n = _out(out, B, device, accumulate)
    _one_device(device, G, n)
    if B * T * d == 0:
        return n if accumulate else n.zero_()
    nbytes = C.c_size_t(0)
    _check(lib().dpnorm_layernorm_norm_workspace(code, int(rms), B, T, d, C.byref(nbytes)), "dpnorm_layernorm_norm_workspace")
    ws, wsp = _given_workspace(workspace, nbytes.value, device)
    _run(device, "dpnorm_layernorm_norm", x.data_ptr(), G.data_ptr(), code, int(rms), B, T, d, eps, parts, n.data_ptr(), int(accumulate),
         wsp, nbytes.value)
    return n


class KernelTimer:
    """HIP events recorded by the library between the launches of one call.

    After each traced call, ``last`` lists (kernel kind, milliseconds) for the
    call's launches once the stream has reached the last event.
    """

    def __init__(self, capacity: int = 64):
        self.capacity = capacity
        self._events = (C.c_void_p * capacity)()
        self._kinds = (C.c_int32 * capacity)()
        L = lib()
        for j in range(capacity):
            ev = C.c_void_p()
            _check(L.dpnorm_event_create(C.byref(ev)), "dpnorm_event_create")
            self._events[j] = ev
        self._count = 0

    def _trace(self) -> _lib.Trace:
        return _lib.Trace(C.cast(self._events, C.POINTER(C.c_void_p)), C.cast(self._kinds, C.POINTER(C.c_int32)),
                          self.capacity, 0)

    def _record(self, tr: _lib.Trace) -> None:
        self._count = int(tr.count)

    def last(self) -> List[Tuple[str, float]]:
        L = lib()
        if self._count == 0:
            return []
        _check(L.dpnorm_event_synchronize(self._events[self._count - 1]), "dpnorm_event_synchronize")
        res = []
        for j in range(1, self._count):
            ms = C.c_float(0.0)
            _check(L.dpnorm_event_elapsed_ms(self._events[j - 1], self._events[j], C.byref(ms)),
                   "dpnorm_event_elapsed_ms")
            res.append((_lib.KERNEL_NAMES.get(self._kinds[j - 1], "?"), ms.value))
        return res

    def close(self) -> None:
        L = lib()
        for j in range(self.capacity):
            if self._events[j]:
                L.dpnorm_event_destroy(self._events[j])
                self._events[j] = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
