"""Block-scaled FP8 operators (C ABI in include/wq_block.h).

E4M3 codes with one fp32 scale for each 128 codes along K (activations: of a
row; weights: of 128 rows).  The operators of a decoder layer's feed-forward
part, from the residual stream to the experts' outputs:

  add_rmsnorm_quantize   residual addition + RMS norm -> codes, scales
  quantize_act           bf16 rows -> codes, scales
  silu_mul_quantize      silu(gate) * up -> codes, scales
  linear                 codes . weight^T (+ bias) -> bf16
  grouped_linear         the same for rows sorted by expert, ragged counts

and ``quantize_weight`` for the weights, which is done once.  As in ``wq``,
each function checks what the C side cannot see (types, shapes, strides,
devices), allocates the outputs that were not passed in, and forwards device
pointers and torch's current stream; all compute runs in libwq.so and there is
no fallback path.  Tensors of other types, shapes, strides or devices than
stated raise; nothing is converted or copied silently.
"""

import ctypes

import torch

from . import wq

BLOCK = 128

_U8, _F32, _BF16, _I32 = torch.uint8, torch.float32, torch.bfloat16, torch.int32
_stream_of = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)

_L = None


def _lib():
    global _L
    if _L is None:
        L = wq.lib()
        P, I64, SZ, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
        L.wq_block_quantize_weight.argtypes = [P, I64, I64, I64, P, P, P]
        L.wq_block_quantize_act.argtypes = [P, I64, I64, I64, P, P, P]
        L.wq_block_silu_mul_quantize.argtypes = [P, I64, I64, I64, P, P, P]
        L.wq_block_add_rmsnorm_quantize.argtypes = [P, I64, P, P, F, I64, I64, P, P, P, P, P]
        L.wq_block_linear_workspace.argtypes = [I64, I64, I64]
        L.wq_block_linear_workspace.restype = SZ
        L.wq_block_linear.argtypes = [P, P, I64, I64, P, P, P, I64, P, P, SZ, P]
        L.wq_block_grouped_linear.argtypes = [P, P, I64, I64, P, P, I64, I64, P, P, I64, P, P]
        _L = L
    return _L


def blocks(n):
    """Scale blocks that cover n elements."""
    return (n + BLOCK - 1) // BLOCK


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _tensor(t, name, dtype, shape, device):
    """`t` is a contiguous tensor of this type and shape on `device`."""
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s (got %s %s, strides %s, on %s)" % (
            name, dtype, tuple(shape), device, t.dtype, tuple(t.shape), t.stride(), t.device))
    return t


def _rows(t, name, dtype):
    """`t` is a GPU matrix whose rows are contiguous; returns (M, K, row stride)."""
    if t.dtype is not dtype or t.dim() != 2 or not t.is_cuda:
        raise ValueError("%s must be a %s matrix on the GPU (got %s of shape %s on %s)" % (
            name, dtype, t.dtype, tuple(t.shape), t.device))
    M, K = t.shape
    ld, one = t.stride()
    if M == 1:
        ld = K  # a single row's stride says nothing
    _need(one == 1 or K == 1, "%s must have contiguous rows (strides %s)" % (name, t.stride()))
    return M, K, ld


def _call(fn, name, device, *args):
    """Enqueue on `device`'s current stream."""
    index = device.index
    if index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return wq._check(fn(*args, _stream_of(index)), name)
    status = fn(*args, _stream_of(index))
    if status:
        wq._check(status, name)


def _codes(out, M, K, device):
    """The (codes, scales) output buffers of a quantizing operator."""
    if out is None:
        return (torch.empty((M, K), dtype=_U8, device=device),
                torch.empty((M, blocks(K)), dtype=_F32, device=device))
    xq, xs = out
    _tensor(xq, "codes", _U8, (M, K), device)
    _tensor(xs, "scales", _F32, (M, blocks(K)), device)
    return xq, xs


# ---------------------------------------------------------------- quantizers


def quantize_weight(W):
    """Quantize bf16 W[N, K] (or E stacked weights [E, N, K]) on its device.

    Returns the weight dict that ``linear`` (or ``grouped_linear``) takes:
    ``codes`` uint8 of W's shape, ``scales`` float32 [(E,) ceil(N/128),
    ceil(K/128)], and the sizes ``E``, ``N``, ``K``."""
    _need(W.dim() in (2, 3) and W.dtype is _BF16 and W.is_cuda, "W must be a bf16 tensor [N, K] or [E, N, K] on the GPU")
    N, K = W.shape[-2:]
    E = 1 if W.dim() == 2 else W.shape[0]
    _tensor(W, "W", _BF16, W.shape, W.device)
    codes = torch.empty(W.shape, dtype=_U8, device=W.device)
    scales = torch.empty(tuple(W.shape[:-2]) + (blocks(N), blocks(K)), dtype=_F32, device=W.device)
    _call(_lib().wq_block_quantize_weight, "wq_block_quantize_weight", W.device,
          W.data_ptr(), E, N, K, codes.data_ptr(), scales.data_ptr())
    return {"E": E, "N": N, "K": K, "codes": codes, "scales": scales}


def quantize_act(X, out=None):
    """Quantize bf16 rows X[M, K] -> (codes uint8 [M, K], scales float32
    [M, ceil(K/128)]).  Rows may be strided (a multiple of 8 elements)."""
    M, K, ld = _rows(X, "X", _BF16)
    xq, xs = _codes(out, M, K, X.device)
    _call(_lib().wq_block_quantize_act, "wq_block_quantize_act", X.device,
          X.data_ptr(), ld, M, K, xq.data_ptr(), xs.data_ptr())
    return xq, xs


def silu_mul_quantize(GU, out=None):
    """silu(gate) * up of GU[M, 2 K] = [gate | up], quantized -> (codes
    [M, K], scales).  Rows may be strided (a multiple of 8 elements)."""
    M, K2, ld = _rows(GU, "GU", _BF16)
    _need(K2 % 2 == 0, "GU must have an even number of columns (got %d)" % K2)
    K = K2 // 2
    xq, xs = _codes(out, M, K, GU.device)
    _call(_lib().wq_block_silu_mul_quantize, "wq_block_silu_mul_quantize", GU.device,
          GU.data_ptr(), ld, M, K, xq.data_ptr(), xs.data_ptr())
    return xq, xs


def add_rmsnorm_quantize(X, gain, eps=1e-5, residual=None, out=None, residual_out=None, y_out=None):
    """h = X + residual; y = h * rsqrt(mean h^2 + eps) * gain, quantized.

    X bf16 [M, K] (rows may be strided by a multiple of 8 elements), gain bf16
    [K], residual bf16 [M, K] or None.  Returns (codes, scales, residual_out,
    y_out).  residual_out receives bf16(h): with a residual it is allocated
    unless passed in (it may be ``residual`` itself); without one it is None
    unless passed in.  y_out receives bf16(y) where it is passed in."""
    M, K, ld = _rows(X, "X", _BF16)
    dev = X.device
    _tensor(gain, "gain", _BF16, (K,), dev)
    xq, xs = _codes(out, M, K, dev)
    r = ro = yo = None
    if residual is not None:
        r = _tensor(residual, "residual", _BF16, (M, K), dev).data_ptr()
        if residual_out is None:
            residual_out = torch.empty((M, K), dtype=_BF16, device=dev)
    if residual_out is not None:
        ro = _tensor(residual_out, "residual_out", _BF16, (M, K), dev).data_ptr()
    if y_out is not None:
        yo = _tensor(y_out, "y_out", _BF16, (M, K), dev).data_ptr()
    _call(_lib().wq_block_add_rmsnorm_quantize, "wq_block_add_rmsnorm_quantize", dev,
          X.data_ptr(), ld, r, gain.data_ptr(), eps, M, K, xq.data_ptr(), xs.data_ptr(), ro, yo)
    return xq, xs, residual_out, y_out


# ---------------------------------------------------------------- products


def linear(Xq, Xs, q, bias=None, out=None):
    """Y = deq(Xq, Xs) . deq(q)^T (+ bias), bf16 [M, N].

    Xq uint8 [M, K] and Xs float32 [M, ceil(K/128)] from any quantizing
    operator above, q a ``quantize_weight`` result of one [N, K] weight, bias
    bf16 [N] or None."""
    W, Ws = q["codes"], q["scales"]
    dev = W.device
    N, K = W.shape
    M = Xq.shape[0]
    _tensor(Xq, "Xq", _U8, (M, K), dev)
    _tensor(Xs, "Xs", _F32, (M, blocks(K)), dev)
    _weight(q, (N, K), (blocks(N), blocks(K)))
    b = None if bias is None else _tensor(bias, "bias", _BF16, (N,), dev).data_ptr()
    if out is None:
        out = torch.empty((M, N), dtype=_BF16, device=dev)
    else:
        _tensor(out, "out", _BF16, (M, N), dev)
    L = _lib()
    need = L.wq_block_linear_workspace(M, N, K)
    ws = wq.workspace(need, dev).data_ptr() if need else None
    _call(L.wq_block_linear, "wq_block_linear", dev, Xq.data_ptr(), Xs.data_ptr(), M, K, W.data_ptr(),
          Ws.data_ptr(), b, N, out.data_ptr(), ws, need)
    return out


def grouped_linear(Xq, Xs, q, offsets, rows=None, out=None):
    """Y[t] = X[rows[t]] . W[e]^T for offsets[e] <= t < offsets[e+1], bf16.

    q: a ``quantize_weight`` result of [E, N, K] weights; offsets int32 [E+1]
    on the device, nondecreasing from 0; rows int32 [T] on the device (source
    row of each sorted row) or None (sorted row t is X's row t).  Rows of the
    output from offsets[E] on are not written.  Nothing is read back to the
    host, so the call can be captured in a graph."""
    W, Ws = q["codes"], q["scales"]
    dev = W.device
    _need(W.dim() == 3, "grouped_linear takes stacked weights [E, N, K]")
    E, N, K = W.shape
    M = Xq.shape[0]
    _tensor(Xq, "Xq", _U8, (M, K), dev)
    _tensor(Xs, "Xs", _F32, (M, blocks(K)), dev)
    _weight(q, (E, N, K), (E, blocks(N), blocks(K)))
    _tensor(offsets, "offsets", _I32, (E + 1,), dev)
    T = M if rows is None else rows.numel()
    r = None if rows is None else _tensor(rows, "rows", _I32, (T,), dev).data_ptr()
    if out is None:
        out = torch.empty((T, N), dtype=_BF16, device=dev)
    else:
        _tensor(out, "out", _BF16, (T, N), dev)
    _call(_lib().wq_block_grouped_linear, "wq_block_grouped_linear", dev, Xq.data_ptr(), Xs.data_ptr(), M, K, r,
          offsets.data_ptr(), T, E, W.data_ptr(), Ws.data_ptr(), N, out.data_ptr())
    return out


def _weight(q, shape, scale_shape):
    W, Ws = q["codes"], q["scales"]
    _need(W.is_cuda, "the weight must be on the GPU")
    _tensor(W, "weight codes", _U8, shape, W.device)
    _tensor(Ws, "weight scales", _F32, scale_shape, W.device)
