"""The experts' routing (C ABI in include/wq_experts.h).

  route     logits -> each token's experts and weights, and the order that sorts
            all choices by expert, as ``block.grouped_linear`` and
            ``int8.grouped_linear`` take it
  combine   weighted sum of each token's rows of those products' output

Allocation, checks and streams are as in ``block``: tensors of other types,
shapes, strides or devices than stated raise, nothing is converted or copied
silently, all compute runs in libwq.so and there is no fallback path.  Nothing
is read back to the host, so the calls can be captured in a graph.
"""

import collections
import ctypes

import torch

from . import wq

_I32, _F32, _BF16 = torch.int32, torch.float32, torch.bfloat16

_SCORES = {"softmax": 0, "sigmoid": 1}
_GROUP_SCORES = {"max": False, "top2": True}

_L = None
_C = None  # the compiled entry points (csrc/wq_experts_py.cpp), bound to the loaded library

#: What ``route`` returns: ids int32 [M, top], weights float32 [M, top], offsets
#: int32 [E + 1], rows int32 [M * top], places int32 [M, top].
Routing = collections.namedtuple("Routing", "ids weights offsets rows places")


def _lib():
    """The C functions by ctypes (the workspace's size and tests)."""
    global _L
    if _L is None:
        L = wq.lib()
        P, I64, I, F, Z = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.wq_experts_route_workspace.argtypes, L.wq_experts_route_workspace.restype = [I64, I64], Z
        L.wq_experts_route.argtypes = [P, I, I64, I64, I64, I64, I, P, I64, I64, I, I, F, P, P, P, P, P, P, P, Z, P]
        L.wq_experts_combine.argtypes = [P, I64, I64, P, P, I64, I64, P, P, P]
        _L = L
    return _L


def _calls():
    global _C
    if _C is None:
        L = _lib()
        from . import _experts_call  # raises if it has not been built

        _experts_call.bind(*[ctypes.cast(f, ctypes.c_void_p).value for f in (L.wq_experts_route, L.wq_experts_combine)])
        _C = _experts_call
    return _C


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def buffers(M, E, top, device):
    """New output buffers of ``route`` for M tokens and E experts."""
    return Routing(torch.empty((M, top), dtype=_I32, device=device), torch.empty((M, top), dtype=_F32, device=device),
                   torch.empty((E + 1,), dtype=_I32, device=device), torch.empty((M * top,), dtype=_I32, device=device),
                   torch.empty((M, top), dtype=_I32, device=device))


def workspace_bytes(M, E):
    """Bytes of the workspace that ``route`` needs for M tokens and E experts, or fewer of either (0: none)."""
    return _lib().wq_experts_route_workspace(M, E)


def route(logits, top, score="softmax", bias=None, groups=1, keep_groups=None, group_score="max", renormalize=True,
          scale=1.0, valid=None, out=None, workspace=None):
    """Route M tokens by their logits [M, E] (float32 or bf16; rows may be
    strided) to ``top`` experts each.

    score: "softmax" (over all E) or "sigmoid".  bias: float32 [E], added to the
    scores for the choice alone, not for the weights.  groups, keep_groups: only
    experts of the ``keep_groups`` best (default: all) of ``groups`` groups of
    consecutive experts are picked; a group counts by its largest choice
    (group_score "max") or the sum of its two largest ("top2").  renormalize:
    each token's weights are divided by their sum.  scale multiplies them.
    valid: bool [M]; a token without it gets no expert.

    Ties go to the lowest index; an expert with a logit of -infinity is never
    picked, and where fewer than ``top`` can be, the rest has id -1, weight 0 and
    place -1.  A NaN is picked first and gives weights of NaN.

    Returns a Routing: ids and weights of each token, largest choice first;
    offsets and rows, the choices sorted by expert (tokens of an expert in their
    order; rows from offsets[E] on are not written); places, where each choice
    went among the sorted.  out: five such buffers to fill; workspace: uint8, at
    least ``workspace_bytes(M, E)``, for a caller that keeps one."""
    _need(isinstance(logits, torch.Tensor) and logits.dim() == 2, "logits must be a matrix")
    M, E = logits.shape
    _need(score in _SCORES, "score must be one of %s" % ", ".join(_SCORES))
    _need(group_score in _GROUP_SCORES, "group_score must be one of %s" % ", ".join(_GROUP_SCORES))
    if out is None:
        _need(isinstance(top, int) and 1 <= top <= E, "top must be 1 to the number of experts")
        out = buffers(M, E, top, logits.device)
    ids, weights, offsets, rows, places = out
    if workspace is None:
        need = _lib().wq_experts_route_workspace(M, E)
        if need:
            workspace = torch.empty((need,), dtype=torch.uint8, device=logits.device)
    status = _calls().route(logits, top, _SCORES[score], bias, groups, groups if keep_groups is None else keep_groups,
                            _GROUP_SCORES[group_score], renormalize, scale, valid, ids, weights, offsets, rows, places,
                            workspace)
    if status:
        wq._check(status, "wq_experts_route")
    return Routing(ids, weights, offsets, rows, places)


def combine(Y, places, weights, base=None, out=None):
    """out[m] = sum_j weights[m, j] * Y[places[m, j]] (+ base[m]), bf16 [M, N].

    Y bf16 [T, N], the sorted rows of a grouped product; places int32 [M, top]
    and weights float32 [M, top] as ``route`` gives them (a place outside [0, T)
    counts as none); base bf16 [M, N] or None (a shared expert's output, a
    residual).  out may be ``base``."""
    if out is None:
        _need(isinstance(places, torch.Tensor) and places.dim() == 2, "places must be a matrix [M, top]")
        _need(isinstance(Y, torch.Tensor) and Y.dim() == 2, "Y must be a matrix")
        out = torch.empty((places.shape[0], Y.shape[1]), dtype=_BF16, device=Y.device)
    status = _calls().combine(Y, places, weights, base, out)
    if status:
        wq._check(status, "wq_experts_combine")
    return out
