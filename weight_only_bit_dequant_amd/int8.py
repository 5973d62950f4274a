"""8-bit integer operators (C ABI in include/wq_int8.h).

Codes int8 in [-127, 127] with one fp32 scale a row: of activations one for each
token, of weights one for each output channel.

  quantize_act        bf16 rows -> codes, scales
  silu_mul_quantize   silu(gate) * up -> codes, scales
  linear              codes . weight^T (+ bias) -> bf16
  grouped_linear      the same for rows sorted by expert, ragged counts

and ``quantize_weight`` for the weights, which is done once.  Allocation, checks
and streams are as in ``block``: tensors of other types, shapes, strides or
devices than stated raise, nothing is converted or copied silently, all compute
runs in libwq.so and there is no fallback path.
"""

import ctypes

import torch

from . import wq

_I8, _F32, _BF16 = torch.int8, torch.float32, torch.bfloat16

_L = None
_C = None  # the compiled entry points (csrc/wq_int8_py.cpp), bound to the loaded library


def _lib():
    """The C functions by ctypes (``quantize_weight`` and tests)."""
    global _L
    if _L is None:
        L = wq.lib()
        P, I64 = ctypes.c_void_p, ctypes.c_int64
        L.wq_int8_quantize_weight.argtypes = [P, I64, I64, I64, P, P, P]
        L.wq_int8_quantize_act.argtypes = [P, I64, I64, I64, P, P, P]
        L.wq_int8_silu_mul_quantize.argtypes = [P, I64, I64, I64, P, P, P]
        L.wq_int8_linear.argtypes = [P, P, I64, I64, P, P, P, I64, P, P]
        L.wq_int8_grouped_linear.argtypes = [P, P, I64, I64, P, P, I64, I64, P, P, I64, P, P]
        _L = L
    return _L


def _calls():
    global _C
    if _C is None:
        L = _lib()
        from . import _int8_call  # raises if it has not been built

        _int8_call.bind(*[ctypes.cast(f, ctypes.c_void_p).value for f in (
            L.wq_int8_quantize_act, L.wq_int8_silu_mul_quantize, L.wq_int8_linear, L.wq_int8_grouped_linear)])
        _C = _int8_call
    return _C


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _matrix(t, name):
    _need(isinstance(t, torch.Tensor) and t.dim() == 2, "%s must be a matrix" % name)
    return t.shape


def _codes(M, K, device):
    """New (codes, scales) buffers of a quantizing operator."""
    return torch.empty((M, K), dtype=_I8, device=device), torch.empty((M,), dtype=_F32, device=device)


# ---------------------------------------------------------------- quantizers


def quantize_weight(W):
    """Quantize bf16 W[N, K] (or E stacked weights [E, N, K]) on its device.

    Returns the weight dict that ``linear`` (or ``grouped_linear``) takes:
    ``codes`` int8 of W's shape, ``scales`` float32 [(E,) N], and the sizes
    ``E``, ``N``, ``K``."""
    _need(isinstance(W, torch.Tensor) and W.dim() in (2, 3) and W.dtype is _BF16 and W.is_cuda and W.is_contiguous(),
          "W must be a contiguous bf16 tensor [N, K] or [E, N, K] on the GPU")
    N, K = W.shape[-2:]
    _need(K > 0 or W.shape[:-1].numel() == 0, "W must have columns (rows of none would be left without scales)")
    E = 1 if W.dim() == 2 else W.shape[0]
    codes = torch.empty(W.shape, dtype=_I8, device=W.device)
    scales = torch.empty(W.shape[:-1], dtype=_F32, device=W.device)
    with torch.cuda.device(W.device):
        wq._check(_lib().wq_int8_quantize_weight(W.data_ptr(), E, N, K, codes.data_ptr(), scales.data_ptr(),
                                                 wq._stream(W.device)), "wq_int8_quantize_weight")
    return {"E": E, "N": N, "K": K, "codes": codes, "scales": scales}


def quantize_act(X, out=None):
    """Quantize bf16 rows X[M, K] -> (codes int8 [M, K], scales float32 [M]).
    Rows may be strided (a multiple of 8 elements)."""
    if out is None:
        out = _codes(*_matrix(X, "X"), X.device)
    xq, xs = out
    status = _calls().quantize_act(X, xq, xs)
    if status:
        wq._check(status, "wq_int8_quantize_act")
    return xq, xs


def silu_mul_quantize(GU, out=None):
    """silu(gate) * up of GU[M, 2 K] = [gate | up], quantized -> (codes
    [M, K], scales [M]).  Rows may be strided (a multiple of 8 elements)."""
    if out is None:
        M, K2 = _matrix(GU, "GU")
        out = _codes(M, K2 // 2, GU.device)
    xq, xs = out
    status = _calls().silu_mul_quantize(GU, xq, xs)
    if status:
        wq._check(status, "wq_int8_silu_mul_quantize")
    return xq, xs


# ---------------------------------------------------------------- products


def linear(Xq, Xs, q, bias=None, out=None):
    """Y = deq(Xq, Xs) . deq(q)^T (+ bias), bf16 [M, N].

    Xq int8 [M, K] and Xs float32 [M] from a quantizing operator above, q a
    ``quantize_weight`` result of one [N, K] weight, bias bf16 [N] or None.
    K < 2^17, so that the sums are exact."""
    W = q["codes"]
    if out is None:
        out = torch.empty((_matrix(Xq, "Xq")[0], W.shape[0]), dtype=_BF16, device=W.device)
    status = _calls().linear(Xq, Xs, W, q["scales"], bias, out)
    if status:
        wq._check(status, "wq_int8_linear")
    return out


def grouped_linear(Xq, Xs, q, offsets, rows=None, out=None):
    """Y[t] = X[rows[t]] . W[e]^T for offsets[e] <= t < offsets[e+1], bf16.

    q: a ``quantize_weight`` result of [E, N, K] weights; offsets int32 [E+1]
    on the device, nondecreasing from 0; rows int32 [T] on the device (source
    row of each sorted row) or None (sorted row t is X's row t), both as
    ``experts.route`` gives them.  Rows of the output from offsets[E] on are not
    written.  Nothing is read back to the host, so the call can be captured in a
    graph."""
    W = q["codes"]
    if out is None:
        _need(W.dim() == 3, "grouped_linear takes stacked weights [E, N, K]")
        T = _matrix(Xq, "Xq")[0] if rows is None else rows.numel()
        out = torch.empty((T, W.shape[1]), dtype=_BF16, device=W.device)
    status = _calls().grouped_linear(Xq, Xs, W, q["scales"], offsets, rows, out)
    if status:
        wq._check(status, "wq_int8_grouped_linear")
    return out
