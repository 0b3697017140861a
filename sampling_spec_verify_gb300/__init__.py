"""Speculative-sampling verify on GB300: Python binding of the C ABI.

The functions here only marshal arguments: every step of the verify, overlap
and E2E-TV computations runs in the CUDA kernels of ``libspec_verify.so``.
PyTorch provides device memory and streams.  There is no CPU fallback: if the
library is missing, every call raises.

Entry points (same names as the C ABI, see include/spec_verify.h):

* ``verify``          -- batched draft/verify step (acceptance, residual
                         correction, bonus token, greedy at T == 0);
* ``verify_ragged``   -- the same with a length of its own per row, over
                         flattened tensors and row offsets;
* ``verify_relaxed``  -- LOSSY relaxed acceptance (target top-k rank and
                         log-probability gap);
* ``tree_mask``, ``tree_verify_greedy`` -- candidate trees: the attention
                         mask of a parent map, and the greedy verify that
                         commits one path;
* ``overlap``         -- alpha = sum min(p, q), TV, prefix survival, E[tau];
* ``e2e_tv_fwd_bwd``  -- E2E-TV loss and its draft-logit gradient;
* ``diagnostics``     -- alpha, target entropy, cross-entropy, KL and the
                         target-only acceptance p(argmax q) per position;
* ``truncate_logits`` -- top-k / top-p truncation, to apply identically to
                         target and draft logits before ``verify``;
* ``schedule_lengths`` -- verify lengths maximising tau * SPS(B) over prefix
                         survivals and a throughput table;
* ``linear_cross_entropy``, ``linear_cross_entropy_fwd_bwd`` -- cross entropy
                         of a vocabulary head from hidden states, without
                         storing its logits, and its gradients (their
                         memory: ``linear_loss_workspace_bytes``);
* ``topk_distill``, ``topk_distill_fwd_bwd`` -- distillation of draft logits
                         from a teacher's top logits, and its gradient;
* ``linear_topk_distill``, ``linear_topk_distill_fwd_bwd`` -- the same from
                         hidden states, through the head;
* ``tree_attention``  -- attention of a pass's rows (a chain, a tree, one token)
                         over a paged cache and the pass's own keys;
* ``plan_cache``      -- block tables, free pages and slots from request lengths;
* ``commit_cache``    -- keys and values of committed rows into their slots;
* ``adjust_logits``   -- penalties for repeated tokens, biases and grammar masks.
"""

from __future__ import annotations

import ctypes
import os
import struct
import threading
from dataclasses import dataclass
from typing import Optional

import torch

__all__ = [
    "SpecError", "lib", "verify", "verify_ragged", "verify_relaxed", "tree_mask", "tree_verify_greedy", "overlap", "e2e_tv_fwd_bwd", "diagnostics", "truncate_logits", "schedule_lengths", "linear_cross_entropy",
    "linear_loss_workspace_bytes", "release_workspaces",
    "linear_cross_entropy_fwd_bwd", "topk_distill", "topk_distill_fwd_bwd", "linear_topk_distill",
    "linear_topk_distill_fwd_bwd", "selftest_bounded_wait", "launch_shape", "kernel_launches", "set_kernel_override",
    "set_launch_override", "VerifyOutput", "OverlapOutput", "E2EOutput", "DiagOutput", "TreeOutput", "HostVerifier",
    "LinearLossOutput", "DistillOutput",
    "tree_attention", "plan_cache", "commit_cache", "adjust_logits", "AttentionOutput", "CachePlan",
    "DEV_BAD_TOKEN", "DEV_BAD_LOGITS", "DEV_BAD_UNIFORM", "DEV_TIMEOUT", "DEV_EMPTY_RESIDUAL", "DEV_BAD_OFFSETS",
    "DEV_BAD_PAGE", "DEV_NO_PAGES",
    "SPEC_OK", "SPEC_ERR_INVALID_ARG", "SPEC_ERR_UNSUPPORTED", "SPEC_ERR_CUDA",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libspec_verify.so")

SPEC_OK, SPEC_ERR_INVALID_ARG, SPEC_ERR_UNSUPPORTED, SPEC_ERR_CUDA = 0, 1, 2, 3
SPEC_F32, SPEC_BF16, SPEC_F16 = 0, 1, 2
SPEC_MEAN, SPEC_SUM = 0, 1
DEV_BAD_TOKEN, DEV_BAD_LOGITS, DEV_BAD_UNIFORM, DEV_TIMEOUT, DEV_EMPTY_RESIDUAL = 1, 2, 4, 8, 16
DEV_BAD_OFFSETS, DEV_BAD_PAGE, DEV_NO_PAGES = 32, 64, 128

_lib = None


class SpecError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        msg = lib().spec_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{what}: {msg} (status {status})")


def lib():
    """The loaded C library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'` "
            "(or sampling_spec_verify_gb300.build.build())")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.spec_abi_version.restype = i32
    L.spec_kernel_launches.restype = ctypes.c_ulonglong
    L.spec_kernel_launches.argtypes = []
    L.spec_status_string.restype = ctypes.c_char_p
    L.spec_status_string.argtypes = [i32]
    L.spec_verify_workspace_bytes.restype = sz
    L.spec_verify_workspace_bytes.argtypes = [i32, i32, i32]
    L.spec_verify.restype = i32
    L.spec_verify.argtypes = [vp, vp, i32, i32, i32, i32, f32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.spec_overlap_workspace_bytes.restype = sz
    L.spec_overlap_workspace_bytes.argtypes = [i32, i32, i32]
    L.spec_overlap.restype = i32
    L.spec_overlap.argtypes = [vp, vp, i32, i32, i32, i32, i32, f32, vp, vp, vp, vp, vp, vp, sz, vp]
    L.spec_e2e_tv_workspace_bytes.restype = sz
    L.spec_e2e_tv_workspace_bytes.argtypes = [i32, i32, i32]
    L.spec_e2e_tv_fwd_bwd.restype = i32
    L.spec_e2e_tv_fwd_bwd.argtypes = [vp, vp, i32, i32, i32, i32, i32, f32, f32, vp, vp, vp, vp, vp, sz, vp]
    L.spec_diagnostics_workspace_bytes.restype = sz
    L.spec_diagnostics_workspace_bytes.argtypes = [i32, i32, i32]
    L.spec_diagnostics.restype = i32
    L.spec_diagnostics.argtypes = [vp, vp, i32, i32, i32, i32, i32, f32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.spec_truncate_logits.restype = i32
    L.spec_truncate_logits.argtypes = [vp, vp, i32, i32, i32, f32, i32, f32, vp, vp]
    L.spec_schedule_lengths.restype = i32
    L.spec_schedule_lengths.argtypes = [vp, i32, i32, vp, i32, vp, vp, vp, vp]
    L.spec_verify_ragged_workspace_bytes.restype = sz
    L.spec_verify_ragged_workspace_bytes.argtypes = [i32, i32, i32]
    L.spec_verify_ragged.restype = i32
    L.spec_verify_ragged.argtypes = [vp, vp, i32, i32, vp, i32, i32, f32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.spec_verify_relaxed.restype = i32
    L.spec_verify_relaxed.argtypes = [vp, vp, i32, i32, i32, i32, f32, i32, f32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.spec_tree_mask.restype = i32
    L.spec_tree_mask.argtypes = [vp, i32, i32, vp, vp, vp, vp]
    L.spec_tree_verify_workspace_bytes.restype = sz
    L.spec_tree_verify_workspace_bytes.argtypes = [i32, i32, i32]
    L.spec_tree_verify_greedy.restype = i32
    L.spec_tree_verify_greedy.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.spec_selftest_bounded_wait.restype = i32
    L.spec_selftest_bounded_wait.argtypes = [ctypes.c_uint64, vp, vp]
    L.spec_launch_shape.restype = i32
    L.spec_launch_shape.argtypes = [i32, i32, i32] + [ctypes.POINTER(i32)] * 5
    L.spec_set_launch_override.restype = None
    L.spec_set_launch_override.argtypes = [i32, i32]
    L.spec_set_kernel_override.restype = None
    L.spec_set_kernel_override.argtypes = [i32]
    head = [vp, vp, i32, i32, i32, i32]                 # hidden, weight, dtype, N, V, H
    tail = [vp, vp, sz, vp]                             # status, workspace, bytes, stream
    L.spec_linear_loss_workspace_bytes.restype = sz
    L.spec_linear_loss_workspace_bytes.argtypes = [i32] * 7
    L.spec_linear_loss_workspace_least.restype = sz
    L.spec_linear_loss_workspace_least.argtypes = [i32] * 7
    L.spec_linear_cross_entropy.restype = i32
    L.spec_linear_cross_entropy.argtypes = head + [f32, vp, i32, vp, i32, vp, vp, vp] + tail
    L.spec_linear_cross_entropy_fwd_bwd.restype = i32
    L.spec_linear_cross_entropy_fwd_bwd.argtypes = head + [f32, f32, vp, i32, vp, i32, vp, vp, vp, vp, vp, i32] + tail
    L.spec_linear_topk_distill.restype = i32
    L.spec_linear_topk_distill.argtypes = head + [i32, f32, vp, vp, vp, i32, vp, vp, vp] + tail
    L.spec_linear_topk_distill_fwd_bwd.restype = i32
    L.spec_linear_topk_distill_fwd_bwd.argtypes = head + [i32, f32, f32, vp, vp, vp, i32, vp, vp, vp, vp, vp,
                                                          i32] + tail
    L.spec_topk_distill_workspace_bytes.restype = sz
    L.spec_topk_distill_workspace_bytes.argtypes = [i32, i32, i32]
    L.spec_topk_distill.restype = i32
    L.spec_topk_distill.argtypes = [vp, i32, i32, i32, i32, f32, vp, vp, vp, vp, i32, vp, vp] + tail
    L.spec_topk_distill_fwd_bwd.restype = i32
    L.spec_topk_distill_fwd_bwd.argtypes = [vp, i32, i32, i32, i32, f32, f32, vp, vp, vp, vp, i32, vp, vp, vp,
                                            i32] + tail
    L.spec_tree_attention_workspace_bytes.restype = sz
    L.spec_tree_attention_workspace_bytes.argtypes = [i32] * 5
    L.spec_tree_attention.restype = i32
    L.spec_tree_attention.argtypes = [vp, vp, vp, sz, vp]
    L.spec_plan_cache.restype = i32
    L.spec_plan_cache.argtypes = [vp] * 5 + [i32] * 5 + [vp] * 7
    L.spec_commit_cache.restype = i32
    L.spec_commit_cache.argtypes = [vp, vp, vp]
    L.spec_adjust_logits.restype = i32
    L.spec_adjust_logits.argtypes = [vp, vp, vp]
    _lib = L
    return L


# ---------------------------------------------------------------------------
# helpers
# ---------------------------------------------------------------------------

def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    if t.dtype == torch.float32:
        return SPEC_F32
    raise TypeError(f"logits must be bfloat16 or float32, got {t.dtype}")


def _need(t: torch.Tensor, name: str, dtype=None, shape=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")


def _need_current(device, stream: Optional[torch.cuda.Stream]):
    """The library launches on the current device: tensors and stream have to be there."""
    current = torch.cuda.current_device()
    if device.index != current:
        raise ValueError(f"tensors are on {device}, but cuda:{current} is the current device: "
                         f"call under torch.cuda.device({device.index})")
    if stream is not None and stream.device_index != current:
        raise ValueError(f"stream belongs to cuda:{stream.device_index}, the tensors are on {device}")


def _stream_handle(stream: Optional[torch.cuda.Stream], device):
    _need_current(device, stream)
    s = torch.cuda.current_stream(device) if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream), s


_WS = {}
_LOCKS = {}


def _held(device, handle: int):
    """Lock of the buffers cached for a stream.  A call is several launches that use
    one workspace, and ctypes lets other threads run meanwhile: a call holds the lock
    from the look-up of its buffers to its last launch, so that two threads on one
    stream (the default one, say) cannot mix their launches over it."""
    key = (device.index, handle)
    return _LOCKS.get(key) or _LOCKS.setdefault(key, threading.Lock())


def _workspace(nbytes: int, device, stream) -> torch.Tensor:
    """A zero-filled workspace cached per (device, stream).  The library
    leaves it zero-filled after every completed call."""
    key = (device.index, stream.cuda_stream)
    ws = _WS.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
        _WS[key] = ws
    return ws


def _check(status: int, what: str):
    if status != SPEC_OK:
        raise SpecError(status, what)


def kernel_launches() -> int:
    """Kernels the library has launched in this process (host-side count)."""
    return int(lib().spec_kernel_launches())


def set_kernel_override(kernel: int = 0) -> None:
    """Sweep kernel of later calls: 0 automatic, 1 the single-read sweep,
    2 the two-pass sweep where it applies."""
    lib().spec_set_kernel_override(int(kernel))


def set_launch_override(cluster_ctas: int = 0, stages: int = 0) -> None:
    """Force the CTAs per cluster (1..16) and shared-memory stages (1 or 2)
    of later launches; 0 = automatic."""
    lib().spec_set_launch_override(int(cluster_ctas), int(stages))


def launch_shape(dtype: torch.dtype, units: int, V: int):
    """(cluster CTAs, threads per CTA, dynamic shared bytes, clusters, stages)
    of a verify sweep over `units` (row, position) pairs."""
    v = [ctypes.c_int() for _ in range(5)]
    code = SPEC_BF16 if dtype == torch.bfloat16 else SPEC_F32
    _check(lib().spec_launch_shape(code, units, V, *[ctypes.byref(x) for x in v]), "spec_launch_shape")
    return tuple(x.value for x in v)


# ---------------------------------------------------------------------------
# verify
# ---------------------------------------------------------------------------

@dataclass
class VerifyOutput:
    tokens: torch.Tensor       # int32 [B, K+1]
    n_accepted: torch.Tensor   # int32 [B]
    alpha: Optional[torch.Tensor]  # float32 [B, K]
    status: torch.Tensor       # int32 [1] device status word


def verify(target: torch.Tensor, draft: Optional[torch.Tensor], draft_tokens: torch.Tensor,
           u_accept: Optional[torch.Tensor], u_final: Optional[torch.Tensor], temperature: float, *,
           want_alpha: bool = True, out: Optional[VerifyOutput] = None,
           workspace: Optional[torch.Tensor] = None,
           stream: Optional[torch.cuda.Stream] = None) -> VerifyOutput:
    """Batched verify of K drafted tokens per row (see spec_verify in the C
    header).  target [B, K+1, V], draft [B, K, V] (bf16 or fp32),
    draft_tokens int32 [B, K], u_accept float32 [B, K], u_final float32 [B]."""
    L = lib()
    _need(target, "target")
    B, K1, V = target.shape
    K = K1 - 1
    dev = target.device
    greedy = float(temperature) == 0.0
    if draft is not None:
        _need(draft, "draft", dtype=target.dtype, shape=(B, K, V), device=dev)
    _need(draft_tokens, "draft_tokens", dtype=torch.int32, shape=(B, K), device=dev)
    if not greedy:
        _need(u_accept, "u_accept", dtype=torch.float32, shape=(B, K), device=dev)
        _need(u_final, "u_final", dtype=torch.float32, shape=(B,), device=dev)
    want_alpha = want_alpha and draft is not None
    if out is None:
        out = VerifyOutput(
            torch.empty((B, K + 1), dtype=torch.int32, device=dev),
            torch.empty((B,), dtype=torch.int32, device=dev),
            torch.empty((B, K), dtype=torch.float32, device=dev) if want_alpha else None,
            torch.zeros((1,), dtype=torch.int32, device=dev))
    sh, s = _stream_handle(stream, dev)
    need = L.spec_verify_workspace_bytes(B, K, V)
    with _held(dev, s.cuda_stream):
        ws = workspace if workspace is not None else _workspace(need, dev, s)
        st = L.spec_verify(_ptr(target), _ptr(draft), _dtype_code(target), B, K, V, float(temperature),
                           _ptr(draft_tokens), _ptr(u_accept), _ptr(u_final), _ptr(out.tokens),
                           _ptr(out.n_accepted), _ptr(out.alpha), _ptr(out.status), _ptr(ws),
                           ws.numel() * ws.element_size(), sh)
    _check(st, "spec_verify")
    return out


def verify_ragged(target: torch.Tensor, draft: Optional[torch.Tensor], row_offsets: torch.Tensor,
                  draft_tokens: Optional[torch.Tensor], u_accept: Optional[torch.Tensor], u_final: torch.Tensor,
                  temperature: float, *, want_alpha: bool = True, workspace: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> VerifyOutput:
    """Verify with a length of its own per row (see spec_verify_ragged in
    the C header).  target [units, V]: row r's drafted positions then its
    bonus position at rows row_offsets[r] .. row_offsets[r+1]-1; draft
    [units - B, V], draft_tokens and u_accept [units - B] in the same
    flattened order; row_offsets int32 [B + 1]; u_final [B].  Returns tokens
    [units] (flattened like target), n_accepted [B], alpha [units - B]."""
    L = lib()
    _need(target, "target")
    units, V = target.shape
    dev = target.device
    _need(row_offsets, "row_offsets", dtype=torch.int32, device=dev)
    B = row_offsets.numel() - 1
    nd = units - B
    _need(u_final, "u_final", dtype=torch.float32, shape=(B,), device=dev)
    if nd > 0:
        _need(draft, "draft", dtype=target.dtype, shape=(nd, V), device=dev)
        _need(draft_tokens, "draft_tokens", dtype=torch.int32, shape=(nd,), device=dev)
        _need(u_accept, "u_accept", dtype=torch.float32, shape=(nd,), device=dev)
    out = VerifyOutput(torch.empty((units,), dtype=torch.int32, device=dev),
                       torch.empty((B,), dtype=torch.int32, device=dev),
                       torch.empty((nd,), dtype=torch.float32, device=dev) if want_alpha and nd > 0 else None,
                       torch.zeros((1,), dtype=torch.int32, device=dev))
    sh, s = _stream_handle(stream, dev)
    need = L.spec_verify_ragged_workspace_bytes(B, units, V)
    with _held(dev, s.cuda_stream):
        ws = workspace if workspace is not None else _workspace(need, dev, s)
        st = L.spec_verify_ragged(_ptr(target), _ptr(draft), _dtype_code(target), B, _ptr(row_offsets), units, V,
                                  float(temperature), _ptr(draft_tokens), _ptr(u_accept), _ptr(u_final),
                                  _ptr(out.tokens), _ptr(out.n_accepted), _ptr(out.alpha), _ptr(out.status), _ptr(ws),
                                  ws.numel() * ws.element_size(), sh)
    _check(st, "spec_verify_ragged")
    return out


def verify_relaxed(target: torch.Tensor, draft: torch.Tensor, draft_tokens: torch.Tensor, u_final: torch.Tensor,
                   temperature: float, top_k: int = 0, delta: float = float("inf"), *, want_alpha: bool = True,
                   workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> VerifyOutput:
    """LOSSY verify: a draft is accepted while it ranks in the target's
    top_k (0: no rank condition) and its log-probability lies within delta
    of the target's largest (inf: no gap condition); the first rejection
    draws from the full target.  Shapes as ``verify``, without u_accept."""
    L = lib()
    _need(target, "target")
    B, K1, V = target.shape
    K = K1 - 1
    dev = target.device
    _need(draft, "draft", dtype=target.dtype, shape=(B, K, V), device=dev)
    _need(draft_tokens, "draft_tokens", dtype=torch.int32, shape=(B, K), device=dev)
    _need(u_final, "u_final", dtype=torch.float32, shape=(B,), device=dev)
    if K == 0:
        draft = draft_tokens = None  # an empty tensor may have no storage
    out = VerifyOutput(torch.empty((B, K + 1), dtype=torch.int32, device=dev),
                       torch.empty((B,), dtype=torch.int32, device=dev),
                       torch.empty((B, K), dtype=torch.float32, device=dev) if want_alpha else None,
                       torch.zeros((1,), dtype=torch.int32, device=dev))
    sh, s = _stream_handle(stream, dev)
    need = L.spec_verify_workspace_bytes(B, K, V)
    with _held(dev, s.cuda_stream):
        ws = workspace if workspace is not None else _workspace(need, dev, s)
        st = L.spec_verify_relaxed(_ptr(target), _ptr(draft), _dtype_code(target), B, K, V, float(temperature),
                                   int(top_k), float(delta), _ptr(draft_tokens), _ptr(u_final), _ptr(out.tokens),
                                   _ptr(out.n_accepted), _ptr(out.alpha), _ptr(out.status), _ptr(ws),
                                   ws.numel() * ws.element_size(), sh)
    _check(st, "spec_verify_relaxed")
    return out


def tree_mask(parent: torch.Tensor, *, status: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None):
    """Tree attention mask of parent maps [B, N] (int32, parent[i] < i, -1
    on the prefix): (mask uint8 [B, N, N], depth int32 [B, N])."""
    L = lib()
    _need(parent, "parent", dtype=torch.int32)
    B, N = parent.shape
    dev = parent.device
    mask = torch.empty((B, N, N), dtype=torch.uint8, device=dev)
    depth = torch.empty((B, N), dtype=torch.int32, device=dev)
    sh, _ = _stream_handle(stream, dev)
    _check(L.spec_tree_mask(_ptr(parent), B, N, _ptr(mask), _ptr(depth), _ptr(status), sh), "spec_tree_mask")
    return mask, depth


@dataclass
class TreeOutput:
    path: torch.Tensor        # int32 [B, N]
    tokens: torch.Tensor      # int32 [B, N + 1]
    n_accepted: torch.Tensor  # int32 [B]
    status: torch.Tensor


def tree_verify_greedy(target: torch.Tensor, parent: torch.Tensor, node_tokens: torch.Tensor, *,
                       workspace: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> TreeOutput:
    """Greedy verify of candidate trees: target [B, N + 1, V] (slot 0 after
    the prefix, slot i + 1 after node i), parent and node_tokens [B, N]."""
    L = lib()
    _need(target, "target")
    B, N1, V = target.shape
    N = N1 - 1
    dev = target.device
    _need(parent, "parent", dtype=torch.int32, shape=(B, N), device=dev)
    _need(node_tokens, "node_tokens", dtype=torch.int32, shape=(B, N), device=dev)
    out = TreeOutput(torch.empty((B, N), dtype=torch.int32, device=dev),
                     torch.empty((B, N + 1), dtype=torch.int32, device=dev),
                     torch.empty((B,), dtype=torch.int32, device=dev),
                     torch.zeros((1,), dtype=torch.int32, device=dev))
    sh, s = _stream_handle(stream, dev)
    need = L.spec_tree_verify_workspace_bytes(B, N, V)
    with _held(dev, s.cuda_stream):
        ws = workspace if workspace is not None else _workspace(need, dev, s)
        st = L.spec_tree_verify_greedy(_ptr(target), _dtype_code(target), B, N, V, _ptr(parent), _ptr(node_tokens),
                                       _ptr(out.path), _ptr(out.tokens), _ptr(out.n_accepted), _ptr(out.status),
                                       _ptr(ws), ws.numel() * ws.element_size(), sh)
    _check(st, "spec_tree_verify_greedy")
    return out


# ---------------------------------------------------------------------------
# overlap
# ---------------------------------------------------------------------------

@dataclass
class OverlapOutput:
    alpha: torch.Tensor
    tv: Optional[torch.Tensor]
    prefix_survival: Optional[torch.Tensor]
    expected_accepted: Optional[torch.Tensor]
    status: torch.Tensor


def overlap(target: torch.Tensor, draft: torch.Tensor, temperature: float, *, K: Optional[int] = None,
            want_tv: bool = True, want_survival: bool = True, out: Optional[OverlapOutput] = None,
            workspace: Optional[torch.Tensor] = None,
            stream: Optional[torch.cuda.Stream] = None) -> OverlapOutput:
    """Per-position overlap statistics.  target [B, KT, V] with KT >= K (the
    first K positions are used), draft [B, K, V]."""
    L = lib()
    _need(target, "target")
    _need(draft, "draft", dtype=target.dtype)
    B, KT, V = target.shape
    K = draft.shape[1] if K is None else K
    if tuple(draft.shape) != (B, K, V) or KT < K:
        raise ValueError("draft must be [B, K, V] with K <= target.shape[1]")
    dev = target.device
    if out is None:
        f = lambda *shape: torch.empty(shape, dtype=torch.float32, device=dev)  # noqa: E731
        out = OverlapOutput(f(B, K), f(B, K) if want_tv else None, f(B, K) if want_survival else None,
                            f(B) if want_survival else None, torch.zeros((1,), dtype=torch.int32, device=dev))
    sh, s = _stream_handle(stream, dev)
    need = L.spec_overlap_workspace_bytes(B, K, V)
    with _held(dev, s.cuda_stream):
        ws = workspace if workspace is not None else _workspace(need, dev, s)
        st = L.spec_overlap(_ptr(target), _ptr(draft), _dtype_code(target), B, K, KT, V, float(temperature),
                            _ptr(out.alpha), _ptr(out.tv), _ptr(out.prefix_survival),
                            _ptr(out.expected_accepted), _ptr(out.status), _ptr(ws),
                            ws.numel() * ws.element_size(), sh)
    _check(st, "spec_overlap")
    return out


# ---------------------------------------------------------------------------
# E2E-TV
# ---------------------------------------------------------------------------

@dataclass
class E2EOutput:
    loss: torch.Tensor            # float32 [1]
    alpha: Optional[torch.Tensor]  # float32 [B, K]
    grad: torch.Tensor            # float32 [B, K, V]
    status: torch.Tensor


def e2e_tv_fwd_bwd(target: torch.Tensor, draft: torch.Tensor, temperature: float, grad_scale: float = 1.0, *,
                   K: Optional[int] = None, want_alpha: bool = True, out: Optional[E2EOutput] = None,
                   workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> E2EOutput:
    """E2E-TV loss mean_b sum_j prod_{k<=j} alpha_{b,k} and grad_scale times
    its gradient with respect to the draft logits (target held constant)."""
    L = lib()
    _need(target, "target")
    _need(draft, "draft", dtype=target.dtype)
    B, KT, V = target.shape
    K = draft.shape[1] if K is None else K
    if tuple(draft.shape) != (B, K, V) or KT < K:
        raise ValueError("draft must be [B, K, V] with K <= target.shape[1]")
    dev = target.device
    if out is None:
        out = E2EOutput(torch.empty((1,), dtype=torch.float32, device=dev),
                        torch.empty((B, K), dtype=torch.float32, device=dev) if want_alpha else None,
                        torch.empty((B, K, V), dtype=torch.float32, device=dev),
                        torch.zeros((1,), dtype=torch.int32, device=dev))
    sh, s = _stream_handle(stream, dev)
    need = L.spec_e2e_tv_workspace_bytes(B, K, V)
    with _held(dev, s.cuda_stream):
        ws = workspace if workspace is not None else _workspace(need, dev, s)
        st = L.spec_e2e_tv_fwd_bwd(_ptr(target), _ptr(draft), _dtype_code(target), B, K, KT, V, float(temperature),
                                   float(grad_scale), _ptr(out.loss), _ptr(out.alpha), _ptr(out.grad),
                                   _ptr(out.status), _ptr(ws), ws.numel() * ws.element_size(), sh)
    _check(st, "spec_e2e_tv_fwd_bwd")
    return out


# ---------------------------------------------------------------------------
# diagnostics
# ---------------------------------------------------------------------------

@dataclass
class DiagOutput:
    alpha: Optional[torch.Tensor]              # float32 [B, K]: sum_v min(p, q)
    entropy: Optional[torch.Tensor]            # H(p), nats
    cross_entropy: Optional[torch.Tensor]      # -sum_v p log q
    kl: Optional[torch.Tensor]                 # KL(p || q)
    alpha_target_only: Optional[torch.Tensor]  # p(argmax q)
    status: torch.Tensor


def diagnostics(target: torch.Tensor, draft: torch.Tensor, temperature: float, *, K: Optional[int] = None,
                out: Optional[DiagOutput] = None, workspace: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> DiagOutput:
    """Per-position alpha, entropy of p, cross-entropy and KL of q against p,
    and the acceptance p(argmax q) of a point-mass drafter, p and q at
    temperature T > 0.  target [B, KT, V] with KT >= K, draft [B, K, V].
    Fields of ``out`` left as None are not computed."""
    L = lib()
    _need(target, "target")
    _need(draft, "draft", dtype=target.dtype)
    B, KT, V = target.shape
    K = draft.shape[1] if K is None else K
    if tuple(draft.shape) != (B, K, V) or KT < K:
        raise ValueError("draft must be [B, K, V] with K <= target.shape[1]")
    dev = target.device
    if out is None:
        f = lambda: torch.empty((B, K), dtype=torch.float32, device=dev)  # noqa: E731
        out = DiagOutput(f(), f(), f(), f(), f(), torch.zeros((1,), dtype=torch.int32, device=dev))
    sh, s = _stream_handle(stream, dev)
    need = L.spec_diagnostics_workspace_bytes(B, K, V)
    with _held(dev, s.cuda_stream):
        ws = workspace if workspace is not None else _workspace(need, dev, s)
        st = L.spec_diagnostics(_ptr(target), _ptr(draft), _dtype_code(target), B, K, KT, V, float(temperature),
                                _ptr(out.alpha), _ptr(out.entropy), _ptr(out.cross_entropy), _ptr(out.kl),
                                _ptr(out.alpha_target_only), _ptr(out.status), _ptr(ws),
                                ws.numel() * ws.element_size(), sh)
    _check(st, "spec_diagnostics")
    return out


# ---------------------------------------------------------------------------
# top-k / top-p truncation
# ---------------------------------------------------------------------------

def truncate_logits(logits: torch.Tensor, temperature: float, top_k: int = 0, top_p: float = 1.0, *,
                    out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Top-k then top-p truncation of every row of ``logits`` [..., V]
    (dropped logits become -inf).  Apply it with the same arguments to the
    target and the draft logits of a verify step.  ``out`` may be ``logits``
    (in place); ``status`` is an optional int32 [1] device word."""
    L = lib()
    _need(logits, "logits")
    V = logits.shape[-1]
    rows = logits.numel() // V if V else 0
    if out is None:
        out = torch.empty_like(logits)
    elif out.shape != logits.shape or out.dtype != logits.dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor of the shape and dtype of logits")
    sh, _ = _stream_handle(stream, logits.device)
    st = L.spec_truncate_logits(_ptr(logits), _ptr(out), _dtype_code(logits), rows, V, float(temperature),
                                int(top_k), float(top_p), _ptr(status), sh)
    _check(st, "spec_truncate_logits")
    return out


# ---------------------------------------------------------------------------
# verify-length scheduling
# ---------------------------------------------------------------------------

def schedule_lengths(survival: torch.Tensor, sps: torch.Tensor, *, status: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None):
    """Verify lengths l_r maximising tau * SPS(B) for prefix survivals
    ``survival`` [R, L] (float32, e.g. ``overlap(...).prefix_survival``) and
    a throughput table ``sps`` [>= R * (1 + L) + 1] (float32, SPS(B) at index
    B).  Returns (lengths int32 [R], objective float32 [2] = {Theta, tau})."""
    L_ = lib()
    _need(survival, "survival", dtype=torch.float32)
    _need(sps, "sps", dtype=torch.float32, device=survival.device)
    R, L = survival.shape
    dev = survival.device
    lengths = torch.empty((R,), dtype=torch.int32, device=dev)
    objective = torch.empty((2,), dtype=torch.float32, device=dev)
    sh, _ = _stream_handle(stream, dev)
    st = L_.spec_schedule_lengths(_ptr(survival), R, L, _ptr(sps), sps.numel(), _ptr(lengths), _ptr(objective),
                                  _ptr(status), sh)
    _check(st, "spec_schedule_lengths")
    return lengths, objective


# ---------------------------------------------------------------------------
# losses for training a drafter
# ---------------------------------------------------------------------------

_SCRATCH = {}
_STATUS = {}
_STATUS_WORDS = 1024
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _loss_stream(given, device):
    """Handle of a training-loss call's stream.  (A call of few rows takes as long
    as its host side; the stream object alone would be 2 us of 29.)"""
    _need_current(device, given)
    return _raw_stream(device.index) if given is None else given.cuda_stream


def _loss_buffers(device, handle, given, nbytes, workspace, empties):
    """(status word, workspace, empty tensors) of a training-loss call, on its
    stream; the caller holds the stream's lock (``_held``).  Status words come
    zeroed from a block per (device, stream), one for each call; workspaces are
    cached per (device, stream) and never zeroed, so they are not the ones of
    the other calls.  Inside a stream capture nothing is cached: the memory
    belongs to the graph."""
    if given is not None:
        with torch.cuda.stream(given):
            return _buffers_here(device, handle, nbytes, workspace, empties)
    return _buffers_here(device, handle, nbytes, workspace, empties)


def _buffers_here(device, handle, nbytes, workspace, empties):
    key = (device.index, handle)
    capturing = torch.cuda.is_current_stream_capturing()  # of the call's own stream
    made = [torch.empty(shape, dtype=dtype, device=device) for shape, dtype in empties]
    status = None
    if made:
        if capturing:
            status = torch.zeros((1,), dtype=torch.int32, device=device)
        else:
            block = _STATUS.get(key)
            if not block:
                with torch.inference_mode(False):  # later calls may not be in it, and own their words too
                    block = list(torch.zeros((_STATUS_WORDS, 1), dtype=torch.int32, device=device).unbind())
                _STATUS[key] = block
            status = block.pop()
    if workspace is None:
        if capturing:
            workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        else:
            workspace = _SCRATCH.get(key)
            if workspace is None or workspace.numel() < nbytes:
                _SCRATCH.pop(key, None)
                workspace = None  # the old one goes before the new one comes
                workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
                _SCRATCH[key] = workspace
    return status, workspace, made


def release_workspaces() -> None:
    """Gives up the workspaces that the training losses have cached, one a stream
    and as large as its largest call's (up to 4 GB and more).  Later calls
    allocate anew.  (The other calls' zero-filled ones are small and stay: a
    captured graph may hold their addresses.)"""
    for key in list(_SCRATCH):
        with _LOCKS[key]:
            _SCRATCH.pop(key, None)


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


class _Nothing:
    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_LOSS_DTYPES = {torch.float32: SPEC_F32, torch.bfloat16: SPEC_BF16, torch.float16: SPEC_F16}


def _reduction_code(reduction: str) -> int:
    if reduction not in ("mean", "sum"):
        raise ValueError(f"reduction must be 'mean' or 'sum', got {reduction!r}")
    return SPEC_MEAN if reduction == "mean" else SPEC_SUM


def _grad_code(grad_dtype, dtype, name: str):
    grad_dtype = dtype if grad_dtype is None else grad_dtype
    if grad_dtype not in (dtype, torch.float32):
        raise TypeError(f"grad_dtype must be float32 or the dtype of {name}, got {grad_dtype}")
    return grad_dtype, _LOSS_DTYPES[grad_dtype]


def _need_out(t: Optional[torch.Tensor], name: str, dtype, shape, device):
    if t is not None:
        _need(t, f"out.{name}", dtype=dtype, shape=shape, device=device)


@dataclass
class LinearLossOutput:
    loss: torch.Tensor                    # float32 [1]
    row_loss: torch.Tensor                # float32 [N]
    lse: torch.Tensor                     # float32 [N]: log of the normaliser, every row
    grad_hidden: Optional[torch.Tensor]   # [N, H]
    grad_weight: Optional[torch.Tensor]   # [V, H]
    status: torch.Tensor                  # int32 [1] device status word


@dataclass
class DistillOutput:
    loss: torch.Tensor            # float32 [1]
    row_loss: torch.Tensor        # float32 [N]
    grad: Optional[torch.Tensor]  # [N, V]
    status: torch.Tensor          # int32 [1] device status word


def _linear_loss(what, hidden, weight, ids, logits, ignore_index, temperature, grad_scale, row_weight, reduction,
                 want_hidden, want_weight, grad_dtype, out, workspace, stream):
    L = lib()
    _need(hidden, "hidden")
    if hidden.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"hidden must be bfloat16 or float16, got {hidden.dtype}")
    if hidden.dim() != 2:
        raise ValueError("hidden must be [N, H]")
    N, H = hidden.shape
    dev = hidden.device
    _need(weight, "weight", dtype=hidden.dtype, device=dev)
    if weight.dim() != 2 or weight.shape[1] != H:
        raise ValueError(f"weight must be [V, {H}], got {tuple(weight.shape)}")
    V = weight.shape[0]
    if logits is None:
        k = 1
        _need(ids, "labels", dtype=torch.int32, shape=(N,), device=dev)
        ignore_index = int(ignore_index)
        if not -2 ** 31 <= ignore_index < 2 ** 31:
            raise ValueError(f"ignore_index must be an int32 value, as the labels are, got {ignore_index}")
    else:
        _need(ids, "teacher_ids", dtype=torch.int32, device=dev)
        if ids.dim() != 2 or ids.shape[0] != N:
            raise ValueError(f"teacher_ids must be [{N}, k], got {tuple(ids.shape)}")
        k = ids.shape[1]
        _need(logits, "teacher_logits", dtype=torch.float32, shape=(N, k), device=dev)
    if row_weight is not None:
        _need(row_weight, "row_weight", dtype=torch.float32, shape=(N,), device=dev)
    grads = want_hidden or want_weight
    gdt, gcode = _grad_code(grad_dtype, hidden.dtype, "hidden")
    red = _reduction_code(reduction)
    empties = []
    if out is None:
        empties = [((1,), torch.float32), ((N,), torch.float32), ((N,), torch.float32)]
        empties += [((N, H), gdt)] * want_hidden + [((V, H), gdt)] * want_weight
    else:
        _need(out.loss, "out.loss", dtype=torch.float32, shape=(1,), device=dev)
        _need_out(out.row_loss, "row_loss", torch.float32, (N,), dev)
        _need_out(out.lse, "lse", torch.float32, (N,), dev)
        _need_out(out.status, "status", torch.int32, (1,), dev)
        if grads:
            if (out.grad_hidden is None) == want_hidden or (out.grad_weight is None) == want_weight:
                raise ValueError("out must hold exactly the gradients that are asked for")
            _need_out(out.grad_hidden, "grad_hidden", gdt, (N, H), dev)
            _need_out(out.grad_weight, "grad_weight", gdt, (V, H), dev)
    if workspace is not None:
        _need(workspace, "workspace", device=dev)
    handle = _loss_stream(stream, dev)
    need = L.spec_linear_loss_workspace_bytes(_LOSS_DTYPES[hidden.dtype], N, V, H, k, int(want_hidden),
                                              int(want_weight))
    with _held(dev, handle):
        status, ws, made = _loss_buffers(dev, handle, stream, need, workspace, empties)
        if out is None:
            out = LinearLossOutput(made[0], made[1], made[2], made[3] if want_hidden else None,
                                   made[-1] if want_weight else None, status)
        dims = (_at(hidden), _at(weight), _LOSS_DTYPES[hidden.dtype], N, V, H)
        rows = (_at(row_weight), red, _at(out.loss), _at(out.row_loss), _at(out.lse))
        end = (_at(out.status), _at(ws), ws.nbytes, handle)
        t, gs = float(temperature), float(grad_scale)
        if logits is None:
            if grads:
                st = L.spec_linear_cross_entropy_fwd_bwd(*dims, t, gs, _at(ids), ignore_index, *rows,
                                                         _at(out.grad_hidden), _at(out.grad_weight), gcode, *end)
            else:
                st = L.spec_linear_cross_entropy(*dims, t, _at(ids), ignore_index, *rows, *end)
        elif grads:
            st = L.spec_linear_topk_distill_fwd_bwd(*dims, k, t, gs, _at(ids), _at(logits), *rows,
                                                    _at(out.grad_hidden), _at(out.grad_weight), gcode, *end)
        else:
            st = L.spec_linear_topk_distill(*dims, k, t, _at(ids), _at(logits), *rows, *end)
    _check(st, what)
    return out


def linear_loss_workspace_bytes(N: int, V: int, H: int, dtype: torch.dtype = torch.bfloat16, k: int = 1, *,
                                want_grad_hidden: bool = True, want_grad_weight: bool = True,
                                least: bool = False) -> int:
    """Workspace of a loss through the head (k = 1: cross entropy), in bytes: the
    size that a call takes by itself, or the least one that it works with.  A
    call with gradients prefers to keep the probabilities of batches up to 4 GB
    between its passes; given a smaller ``workspace`` it goes through the vocabulary in
    pieces that fit, and computes the logits twice."""
    f = lib().spec_linear_loss_workspace_least if least else lib().spec_linear_loss_workspace_bytes
    size = f(_LOSS_DTYPES.get(dtype, -1), N, V, H, k, int(want_grad_hidden), int(want_grad_weight))
    if size == 0:
        raise ValueError("sizes or dtype beyond what the losses through the head take")
    return size


def linear_cross_entropy(hidden: torch.Tensor, weight: torch.Tensor, labels: torch.Tensor, temperature: float = 1.0, *,
                         row_weight: Optional[torch.Tensor] = None, ignore_index: int = -100,
                         reduction: str = "mean", out: Optional[LinearLossOutput] = None,
                         workspace: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None) -> LinearLossOutput:
    """Cross entropy of softmax(hidden weight^T / temperature) against labels
    without storing the logits (see spec_linear_cross_entropy in the C
    header).  hidden [N, H] and weight [V, H] (bf16 or fp16, H a multiple of
    8), labels int32 [N], row_weight float32 [N].  ``row_loss`` is unweighted
    (minus the label's log-probability); ``loss`` is the weighted sum, over
    the rows whose label is not ``ignore_index``, divided by their number
    unless reduction is "sum"."""
    return _linear_loss("spec_linear_cross_entropy", hidden, weight, labels, None, ignore_index, temperature, 0.0,
                        row_weight, reduction, False, False, None, out, workspace, stream)


def linear_cross_entropy_fwd_bwd(hidden: torch.Tensor, weight: torch.Tensor, labels: torch.Tensor,
                                 temperature: float = 1.0, grad_scale: float = 1.0, *,
                                 row_weight: Optional[torch.Tensor] = None, ignore_index: int = -100,
                                 reduction: str = "mean", want_grad_hidden: bool = True,
                                 want_grad_weight: bool = True, grad_dtype: Optional[torch.dtype] = None,
                                 out: Optional[LinearLossOutput] = None, workspace: Optional[torch.Tensor] = None,
                                 stream: Optional[torch.cuda.Stream] = None) -> LinearLossOutput:
    """``linear_cross_entropy`` and grad_scale times its gradients with respect
    to hidden and weight (of ``grad_dtype``: float32 or, by default, the dtype
    of hidden).  A frozen head saves its product with
    ``want_grad_weight=False``."""
    if not (want_grad_hidden or want_grad_weight):
        raise ValueError("no gradient asked for: call linear_cross_entropy")
    return _linear_loss("spec_linear_cross_entropy_fwd_bwd", hidden, weight, labels, None, ignore_index, temperature,
                        grad_scale, row_weight, reduction, want_grad_hidden, want_grad_weight, grad_dtype, out,
                        workspace, stream)


def linear_topk_distill(hidden: torch.Tensor, weight: torch.Tensor, teacher_ids: torch.Tensor,
                        teacher_logits: torch.Tensor, temperature: float = 1.0, *,
                        row_weight: Optional[torch.Tensor] = None, reduction: str = "mean",
                        out: Optional[LinearLossOutput] = None, workspace: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> LinearLossOutput:
    """KL(t || q) of the teacher's renormalised top logits against
    q = softmax(hidden weight^T / temperature), without storing the logits (see
    spec_linear_topk_distill in the C header).  teacher_ids int32 [N, k] (-1:
    unused slot) and teacher_logits float32 [N, k], k <= 256."""
    if teacher_logits is None:
        raise TypeError("teacher_logits must be a torch.Tensor")
    return _linear_loss("spec_linear_topk_distill", hidden, weight, teacher_ids, teacher_logits, -1, temperature, 0.0,
                        row_weight, reduction, False, False, None, out, workspace, stream)


def linear_topk_distill_fwd_bwd(hidden: torch.Tensor, weight: torch.Tensor, teacher_ids: torch.Tensor,
                                teacher_logits: torch.Tensor, temperature: float = 1.0, grad_scale: float = 1.0, *,
                                row_weight: Optional[torch.Tensor] = None, reduction: str = "mean",
                                want_grad_hidden: bool = True, want_grad_weight: bool = True,
                                grad_dtype: Optional[torch.dtype] = None, out: Optional[LinearLossOutput] = None,
                                workspace: Optional[torch.Tensor] = None,
                                stream: Optional[torch.cuda.Stream] = None) -> LinearLossOutput:
    """``linear_topk_distill`` and grad_scale times its gradients, as
    ``linear_cross_entropy_fwd_bwd`` gives them."""
    if teacher_logits is None:
        raise TypeError("teacher_logits must be a torch.Tensor")
    if not (want_grad_hidden or want_grad_weight):
        raise ValueError("no gradient asked for: call linear_topk_distill")
    return _linear_loss("spec_linear_topk_distill_fwd_bwd", hidden, weight, teacher_ids, teacher_logits, -1,
                        temperature, grad_scale, row_weight, reduction, want_grad_hidden, want_grad_weight,
                        grad_dtype, out, workspace, stream)


def _distill(what, student, ids, logits, lse, temperature, grad_scale, row_weight, reduction, want_grad, grad_dtype,
             out, workspace, stream):
    L = lib()
    _need(student, "student")
    if student.dtype not in _LOSS_DTYPES:
        raise TypeError(f"student must be bfloat16, float16 or float32, got {student.dtype}")
    if student.dim() != 2:
        raise ValueError("student must be [N, V]")
    N, V = student.shape
    dev = student.device
    _need(ids, "teacher_ids", dtype=torch.int32, device=dev)
    if ids.dim() != 2 or ids.shape[0] != N:
        raise ValueError(f"teacher_ids must be [{N}, k], got {tuple(ids.shape)}")
    k = ids.shape[1]
    _need(logits, "teacher_logits", dtype=torch.float32, shape=(N, k), device=dev)
    if lse is not None:
        _need(lse, "teacher_lse", dtype=torch.float32, shape=(N,), device=dev)
    if row_weight is not None:
        _need(row_weight, "row_weight", dtype=torch.float32, shape=(N,), device=dev)
    gdt, gcode = _grad_code(grad_dtype, student.dtype, "student")
    red = _reduction_code(reduction)
    empties = []
    if out is None:
        empties = [((1,), torch.float32), ((N,), torch.float32)] + [((N, V), gdt)] * want_grad
    else:
        _need(out.loss, "out.loss", dtype=torch.float32, shape=(1,), device=dev)
        _need_out(out.row_loss, "row_loss", torch.float32, (N,), dev)
        _need_out(out.status, "status", torch.int32, (1,), dev)
        if want_grad:
            _need(out.grad, "out.grad", dtype=gdt, shape=(N, V), device=dev)
    if workspace is not None:
        _need(workspace, "workspace", device=dev)
    handle = _loss_stream(stream, dev)
    need = L.spec_topk_distill_workspace_bytes(N, V, k)
    with _held(dev, handle):
        status, ws, made = _loss_buffers(dev, handle, stream, need, workspace, empties)
        if out is None:
            out = DistillOutput(made[0], made[1], made[2] if want_grad else None, status)
        end = (_at(out.status), _at(ws), ws.nbytes, handle)
        common = (_at(ids), _at(logits), _at(lse), _at(row_weight), red, _at(out.loss), _at(out.row_loss))
        dims = (_at(student), _LOSS_DTYPES[student.dtype], N, V, k, float(temperature))
        if want_grad:
            st = L.spec_topk_distill_fwd_bwd(*dims, float(grad_scale), *common, _at(out.grad), gcode, *end)
        else:
            st = L.spec_topk_distill(*dims, *common, *end)
    _check(st, what)
    return out


def topk_distill(student: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor,
                 temperature: float = 1.0, *, teacher_lse: Optional[torch.Tensor] = None,
                 row_weight: Optional[torch.Tensor] = None, reduction: str = "mean",
                 out: Optional[DistillOutput] = None, workspace: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> DistillOutput:
    """KL(t || q) of a teacher's top logits against q = softmax(student /
    temperature) (see spec_topk_distill in the C header).  student [N, V]
    (bf16, fp16 or fp32), teacher_ids int32 [N, k] (-1: unused slot),
    teacher_logits float32 [N, k], k <= 256.  Without ``teacher_lse`` the
    listed logits are renormalised; with it (float32 [N], logsumexp of the
    teacher's whole row / temperature) the remaining mass of both sides counts
    as one more token."""
    return _distill("spec_topk_distill", student, teacher_ids, teacher_logits, teacher_lse, temperature, 0.0,
                    row_weight, reduction, False, None, out, workspace, stream)


def topk_distill_fwd_bwd(student: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor,
                         temperature: float = 1.0, grad_scale: float = 1.0, *,
                         teacher_lse: Optional[torch.Tensor] = None, row_weight: Optional[torch.Tensor] = None,
                         reduction: str = "mean", grad_dtype: Optional[torch.dtype] = None,
                         out: Optional[DistillOutput] = None, workspace: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None) -> DistillOutput:
    """``topk_distill`` and grad_scale times its gradient with respect to the
    student logits (of ``grad_dtype``: float32 or, by default, the student's
    dtype)."""
    return _distill("spec_topk_distill_fwd_bwd", student, teacher_ids, teacher_logits, teacher_lse, temperature,
                    grad_scale, row_weight, reduction, True, grad_dtype, out, workspace, stream)


# ---------------------------------------------------------------------------
# a decoding step around the verify: attention, cache, sampling rules
# ---------------------------------------------------------------------------

def _need_strided(t: torch.Tensor, name: str, dtype=None, dims=None, device=None):
    """Like ``_need`` for tensors whose rows may lie apart: the last dimension is contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if dims is not None and t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {tuple(t.shape)}")
    if device is not None and t.get_device() != device.index:
        raise ValueError(f"{name} must be on {device}")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")


def _strides(t: torch.Tensor):
    """Strides of all dimensions but the last; one of size 1 is never stepped along."""
    shape, strides = t.shape, t.stride()[:-1]
    return strides if min(shape) > 1 else [s if n > 1 else shape[-1] for n, s in zip(shape, strides)]


def _need_pass(t: torch.Tensor, name: str, dtype, shape, ragged: bool, lead: int, device):
    """Strides of a pass's rows [*, B, T, heads, D] (``lead`` dimensions before them) or,
    ragged, [*, rows, heads, D]: (lead..., row, head).  (A call of few rows takes as
    long as its host side: what is right is looked at once, the reason of a refusal
    is found afterwards.)"""
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != device.index
            or t.stride(-1) != 1):
        _need_strided(t, name, dtype=dtype, dims=len(shape), device=device)
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    s = t.stride()
    if ragged:
        rows, row, head = shape[-3], s[-3], s[-2]
    else:
        B, T = shape[-4], shape[-3]
        if B > 1 and T > 1 and s[-4] != T * s[-3]:
            raise ValueError(f"the rows of {name} must be evenly spaced over requests")
        rows, row, head = B * T, s[-3] if T > 1 else s[-4], s[-2]
    D = shape[-1]  # a dimension of size 1 is never stepped along
    return (*(x if n > 1 else D for n, x in zip(shape[:lead], s)), row if rows > 1 else D, head if shape[-2] > 1 else D)


def _pass_shape(B_offsets: Optional[torch.Tensor], max_rows: Optional[int], lead_shape, name: str, device):
    """(B, T, rows) of a pass, from [B, T] or from row offsets and the most rows of a request."""
    if B_offsets is None:
        if max_rows is not None:
            raise ValueError("max_rows goes with row_offsets")
        B, T = lead_shape
        return (B, T, B * T) if B * T else (0, max(T, 1), 0)
    _need(B_offsets, "row_offsets", dtype=torch.int32, device=device)
    if B_offsets.dim() != 1 or B_offsets.numel() < 1:
        raise ValueError("row_offsets must be [B + 1]")
    if max_rows is None or int(max_rows) < 1:
        raise ValueError(f"row_offsets of {name} need max_rows >= 1, the most rows of a request")
    return B_offsets.numel() - 1, int(max_rows), lead_shape[0]


def _need_mask(mask: Optional[torch.Tensor], B: int, T: int, device):
    if mask is not None:
        _need(mask, "mask", dtype=torch.uint8, device=device)
        if mask.numel() != B * T * T or (B and tuple(mask.shape) != (B, T, T)):
            raise ValueError(f"mask must be [{B}, {T}, {T}], got {tuple(mask.shape)}")


# spec_attention_t, spec_commit_t and spec_adjust_t as the C compiler lays them out:
# pointers, then strides, then sizes (packing costs a tenth of a ctypes.Structure)
_ATTENTION = struct.Struct("@11P13q10if0q")
_COMMIT = struct.Struct("@7P15q10i0q")
_ADJUST = struct.Struct("@14P7i0q")


def _or0(t: Optional[torch.Tensor]):
    return 0 if t is None else t.data_ptr()


_KV_DTYPES = {torch.bfloat16: SPEC_BF16, torch.float16: SPEC_F16}


@dataclass
class AttentionOutput:
    out: torch.Tensor             # as q, contiguous
    lse: Optional[torch.Tensor]   # float32, q's shape without the last dimension
    status: torch.Tensor          # int32 [1] device status word


def tree_attention(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, k_cache: torch.Tensor,
                   v_cache: torch.Tensor, block_table: torch.Tensor, context_lens: torch.Tensor, *,
                   mask: Optional[torch.Tensor] = None, row_offsets: Optional[torch.Tensor] = None,
                   max_rows: Optional[int] = None, scale: Optional[float] = None, want_lse: bool = False,
                   out: Optional[AttentionOutput] = None, workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> AttentionOutput:
    """Attention of a pass's rows (a chain, a tree, or one token a request) over
    a paged cache and the pass's own keys and values (see spec_tree_attention in
    the C header).  q [B, T, Hq, D], k_new and v_new [B, T, Hkv, D] (bf16 or
    fp16), or [rows, heads, D] with ``row_offsets`` int32 [B + 1] and
    ``max_rows``; k_cache and v_cache [pages, page_size, Hkv, D]; block_table
    int32 [B, width]; context_lens int32 [B]; mask uint8 [B, T, T] (``tree_mask``
    of the rows' parent map; None: a chain).  ``scale`` is 1 / sqrt(D) unless
    given.  Only the last dimension has to be contiguous; the others lie
    multiples of 8 elements apart.  The result carries no gradient, whatever the
    arguments require."""
    L = lib()
    ragged = row_offsets is not None
    _need_strided(q, "q", dims=3 if ragged else 4)
    if q.dtype not in _KV_DTYPES:
        raise TypeError(f"q must be bfloat16 or float16, got {q.dtype}")
    dev, dt = q.device, q.dtype
    Hq, D = q.shape[-2:]
    B, T, rows = _pass_shape(row_offsets, max_rows, q.shape[:-2], "q", dev)
    _need_strided(k_cache, "k_cache", dtype=dt, dims=4, device=dev)
    _need_strided(v_cache, "v_cache", dtype=dt, dims=4, device=dev)
    pages, page, Hkv, last = k_cache.shape
    if last != D or v_cache.shape != k_cache.shape:
        raise ValueError(f"k_cache and v_cache must be [pages, page_size, Hkv, {D}], got {tuple(k_cache.shape)} "
                         f"and {tuple(v_cache.shape)}")
    q_shape = q.shape
    q_stride = _need_pass(q, "q", dt, q_shape, ragged, 0, dev)
    shape = (*q_shape[:-2], Hkv, D)
    kn_stride = _need_pass(k_new, "k_new", dt, shape, ragged, 0, dev)
    vn_stride = _need_pass(v_new, "v_new", dt, shape, ragged, 0, dev)
    _need(context_lens, "context_lens", dtype=torch.int32, device=dev)
    _need_strided(block_table, "block_table", dtype=torch.int32, dims=2, device=dev)
    width = block_table.shape[1]
    if (rows or ragged) and (context_lens.shape != (B,) or block_table.shape[0] != B):
        raise ValueError(f"context_lens and block_table must have {B} rows")
    _need_mask(mask, B, T, dev)
    empties = []
    if out is None:
        empties = [(q_shape, dt), (q_shape[:-1], torch.float32)] if want_lse else [(q_shape, dt)]
    else:
        _need(out.out, "out.out", dtype=dt, shape=q.shape, device=dev)
        if want_lse and out.lse is None:
            raise ValueError("want_lse: out.lse is missing")
        _need_out(out.lse, "lse", torch.float32, q.shape[:-1], dev)
        _need_out(out.status, "status", torch.int32, (1,), dev)
    if workspace is not None:
        _need(workspace, "workspace", device=dev)
    handle = _loss_stream(stream, dev)
    need = L.spec_tree_attention_workspace_bytes(B, T, Hq, Hkv, D)
    with _held(dev, handle):
        status, ws, made = _loss_buffers(dev, handle, stream, need, workspace, empties)
        if out is None:
            out = AttentionOutput(made[0], made[1] if want_lse else None, status)
        a = _ATTENTION.pack(q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                            out.out.data_ptr(), _or0(out.lse), block_table.data_ptr(), context_lens.data_ptr(),
                            _or0(row_offsets), _or0(mask), *q_stride, *kn_stride, *vn_stride, *_strides(k_cache),
                            *_strides(v_cache), block_table.stride(0) if B > 1 else width, B, T, rows, Hq, Hkv, D,
                            pages, page, width, _KV_DTYPES[dt], D ** -0.5 if scale is None else float(scale))
        st = L.spec_tree_attention(a, _at(out.status), ws.data_ptr(), ws.nbytes, handle)
    _check(st, "spec_tree_attention")
    return out


@dataclass
class CachePlan:
    block_table: torch.Tensor   # int32 [B, width]
    free_pages: torch.Tensor    # int32 [capacity]
    free_count: torch.Tensor    # int32 [1]
    context_lens: torch.Tensor  # int32 [B]: lengths after the step
    slots: torch.Tensor         # int32 [B, max_new]: places of the appended tokens, then -1
    status: torch.Tensor        # int32 [1] device status word


def plan_cache(context_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor,
               free_pages: torch.Tensor, free_count: torch.Tensor, page_size: int, max_new: int, *,
               out: Optional[CachePlan] = None, stream: Optional[torch.cuda.Stream] = None) -> CachePlan:
    """Block tables, free pages and slots of the tokens that a step appends
    (``new_lens`` int32 [B], e.g. n_accepted + 1; at most ``max_new``) or takes back
    (negative; -context_lens: the request is done), from lengths alone and without
    the host (see spec_plan_cache in the C header).  context_lens int32 [B],
    block_table int32 [B, width], free_pages int32 [capacity] a stack of
    free_count int32 [1] pages.  ``out.block_table`` and ``out.free_pages`` may
    be the inputs (in place)."""
    L = lib()
    _need(block_table, "block_table", dtype=torch.int32)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, width]")
    B, width = block_table.shape
    dev = block_table.device
    T = int(max_new)
    if T < 0:
        raise ValueError(f"max_new must not be negative, got {T}")
    _need(context_lens, "context_lens", dtype=torch.int32, shape=(B,), device=dev)
    _need(new_lens, "new_lens", dtype=torch.int32, shape=(B,), device=dev)
    _need(free_pages, "free_pages", dtype=torch.int32, device=dev)
    if free_pages.dim() != 1:
        raise ValueError("free_pages must be [capacity]")
    _need(free_count, "free_count", dtype=torch.int32, shape=(1,), device=dev)
    shapes = [(B, width), tuple(free_pages.shape), (1,), (B,), (B, T)]
    if out is not None:
        for t, name, shape in zip((out.block_table, out.free_pages, out.free_count, out.context_lens, out.slots),
                                  ("block_table", "free_pages", "free_count", "context_lens", "slots"), shapes):
            _need(t, f"out.{name}", dtype=torch.int32, shape=shape, device=dev)
        _need_out(out.status, "status", torch.int32, (1,), dev)
    handle = _loss_stream(stream, dev)
    with _held(dev, handle):
        if out is None:
            # no workspace is needed: any tensor stands for it
            status, _, made = _loss_buffers(dev, handle, stream, 0, block_table, [((B, T), torch.int32)])
            with _Nothing() if stream is None else torch.cuda.stream(stream):
                like = torch.empty_like
                out = CachePlan(like(block_table), like(free_pages), like(free_count), like(context_lens), made[0], status)
        st = L.spec_plan_cache(_at(context_lens), _at(new_lens), _at(block_table), _at(free_pages), _at(free_count), B,
                               T, width, free_pages.numel(), int(page_size), _at(out.block_table), _at(out.free_pages),
                               _at(out.free_count), _at(out.context_lens), _at(out.slots), _at(out.status), handle)
    _check(st, "spec_plan_cache")
    return out


def commit_cache(k_new: torch.Tensor, v_new: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 slots: torch.Tensor, *, path: Optional[torch.Tensor] = None,
                 row_offsets: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> None:
    """Copies the keys and values of a pass's committed rows into the cache (see
    spec_commit_cache in the C header): place i of a request, at ``slots`` int32
    [B, S] (``plan_cache``'s), takes row i or, with ``path`` int32 [B, >= S - 1]
    (``tree_verify_greedy``'s), row 0 and then the rows of the accepted nodes.
    k_new and v_new [B, T, Hkv, D] or, with ``row_offsets`` int32 [B + 1], [rows,
    Hkv, D]; k_cache and v_cache [pages, page_size, Hkv, D].  All of them may have
    one more dimension in front, the model's layers.  ``status`` is an optional
    int32 [1] device word."""
    L = lib()
    ragged = row_offsets is not None
    _need_strided(k_cache, "k_cache")
    dt, dev = k_cache.dtype, k_cache.device
    if dt not in _KV_DTYPES:
        raise TypeError(f"k_cache must be bfloat16 or float16, got {dt}")
    if k_cache.dim() not in (4, 5):
        raise ValueError("k_cache must be [pages, page_size, Hkv, D], or [layers, pages, page_size, Hkv, D]")
    lead = k_cache.dim() - 4
    _need_strided(v_cache, "v_cache", dtype=dt, dims=4 + lead, device=dev)
    if v_cache.shape != k_cache.shape:
        raise ValueError(f"v_cache must have shape {tuple(k_cache.shape)}, got {tuple(v_cache.shape)}")
    layers = k_cache.shape[0] if lead else 1
    pages, page, Hkv, D = k_cache.shape[lead:]
    _need_strided(k_new, "k_new", dtype=dt, dims=lead + (3 if ragged else 4), device=dev)
    rows_shape = tuple(k_new.shape[lead:-2])
    shape = (*k_cache.shape[:lead], *rows_shape, Hkv, D)
    kn_stride = _need_pass(k_new, "k_new", dt, shape, ragged, lead, dev)
    vn_stride = _need_pass(v_new, "v_new", dt, shape, ragged, lead, dev)
    B, T, rows = _pass_shape(row_offsets, max(rows_shape[0], 1) if ragged else None, rows_shape, "k_new", dev)
    _need(slots, "slots", dtype=torch.int32, device=dev)
    if slots.dim() != 2 or ((rows or ragged) and slots.shape[0] != B):
        raise ValueError(f"slots must be [{B}, S], got {tuple(slots.shape)}")
    S = slots.shape[1]
    if path is not None:
        _need_strided(path, "path", dtype=torch.int32, dims=2, device=dev)
        if path.shape[0] != slots.shape[0] or path.shape[1] < S - 1:
            raise ValueError(f"path must be [{slots.shape[0]}, {max(S - 1, 0)}] or wider, got {tuple(path.shape)}")
    if status is not None:
        _need(status, "status", dtype=torch.int32, shape=(1,), device=dev)
    handle = _loss_stream(stream, dev)
    one = () if lead else (D,)  # the single layer's stride
    a = _COMMIT.pack(k_new.data_ptr(), v_new.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), slots.data_ptr(),
                     _or0(path) if S > 1 else 0, _or0(row_offsets), *one, *kn_stride, *one, *vn_stride, *one,
                     *_strides(k_cache), *one, *_strides(v_cache),
                     0 if path is None else path.stride(0) if path.shape[0] > 1 else path.shape[1],
                     layers, B, T, rows, S, Hkv, D, pages, page, _KV_DTYPES[dt])
    _check(L.spec_commit_cache(a, _at(status), handle), "spec_commit_cache")


def adjust_logits(logits: torch.Tensor, tokens: torch.Tensor, history: torch.Tensor, history_lens: torch.Tensor, *,
                  prompt_lens: Optional[torch.Tensor] = None, repetition: Optional[torch.Tensor] = None,
                  frequency: Optional[torch.Tensor] = None, presence: Optional[torch.Tensor] = None,
                  bias_ids: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                  allowed: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
                  row_offsets: Optional[torch.Tensor] = None, max_rows: Optional[int] = None,
                  out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Penalties for repeated tokens, biases and grammar masks on a pass's logits
    (see spec_adjust_logits in the C header), before ``truncate_logits`` and the
    verify.  logits [B, T, V] (bf16 or fp32) follow the pass's rows, whose tokens
    are ``tokens`` int32 [B, T] (-1: not counted, such as a first row that the history
    holds); or [rows, V] and [rows] with ``row_offsets`` int32 [B + 1] and ``max_rows``.  history int32 [B, width] holds history_lens int32
    [B] tokens, the first prompt_lens of them the prompt's; repetition, frequency
    and presence float32 [B]; bias_ids int32 [B, n] and bias float32 [B, n];
    allowed int32 [B, T, ceil(V / 32)] bits; mask uint8 [B, T, T] (a tree; None: a
    chain).  ``out`` may be ``logits`` (in place); ``status`` is an optional int32
    [1] device word.  The result carries no gradient, whatever the arguments require."""
    L = lib()
    ragged = row_offsets is not None
    _need(logits, "logits")
    if logits.dim() != (2 if ragged else 3):
        raise ValueError("logits must be [B, T, V], or [rows, V] with row_offsets")
    code = _dtype_code(logits)
    dev, V = logits.device, logits.shape[-1]
    at = tuple(logits.shape[:-1])
    B, T, rows = _pass_shape(row_offsets, max_rows, at, "logits", dev)
    n = B if rows or ragged else at[0]
    _need(tokens, "tokens", dtype=torch.int32, shape=at, device=dev)
    _need(history, "history", dtype=torch.int32, device=dev)
    if history.dim() != 2 or history.shape[0] != n:
        raise ValueError(f"history must be [{n}, width], got {tuple(history.shape)}")
    _need(history_lens, "history_lens", dtype=torch.int32, shape=(n,), device=dev)
    if prompt_lens is not None:
        _need(prompt_lens, "prompt_lens", dtype=torch.int32, shape=(n,), device=dev)
    for t, name in ((repetition, "repetition"), (frequency, "frequency"), (presence, "presence")):
        if t is not None:
            _need(t, name, dtype=torch.float32, shape=(n,), device=dev)
    if (bias_ids is None) != (bias is None):
        raise ValueError("bias_ids and bias go together")
    biases = 0
    if bias is not None:
        _need(bias_ids, "bias_ids", dtype=torch.int32, device=dev)
        if bias_ids.dim() != 2 or bias_ids.shape[0] != n:
            raise ValueError(f"bias_ids must be [{n}, entries], got {tuple(bias_ids.shape)}")
        biases = bias_ids.shape[1]
        _need(bias, "bias", dtype=torch.float32, shape=(n, biases), device=dev)
    if allowed is not None:
        _need(allowed, "allowed", dtype=torch.int32, shape=(*at, (V + 31) // 32), device=dev)
    _need_mask(mask, B, T, dev)
    if out is None:
        with _Nothing() if stream is None else torch.cuda.stream(stream):
            out = torch.empty_like(logits)
    else:
        _need(out, "out", dtype=logits.dtype, shape=logits.shape, device=dev)
    if status is not None:
        _need(status, "status", dtype=torch.int32, shape=(1,), device=dev)
    handle = _loss_stream(stream, dev)
    a = _ADJUST.pack(logits.data_ptr(), out.data_ptr(), tokens.data_ptr(), history.data_ptr(), history_lens.data_ptr(),
                     *map(_or0, (prompt_lens, repetition, frequency, presence, bias_ids, bias, allowed, row_offsets, mask)),
                     B, T, rows, V, history.shape[1], biases, code)
    _check(L.spec_adjust_logits(a, _at(status), handle), "spec_adjust_logits")
    return out


# ---------------------------------------------------------------------------
# host-buffer convenience: one verify step from pinned host memory
# ---------------------------------------------------------------------------

def selftest_bounded_wait(limit_ns: int = 2_000_000, *, status: Optional[torch.Tensor] = None,
                          device="cuda", stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Failure-path self-test of the library's bounded wait (see
    spec_selftest_bounded_wait in the C header): a warp waits on an
    mbarrier that nothing completes and gives up after ``limit_ns``; a thread
    of another warp reports it.  Returns
    the int32 status word, which holds DEV_TIMEOUT once the stream has run the
    test."""
    L = lib()
    if status is None:
        status = torch.zeros((1,), dtype=torch.int32, device=torch.device(device))
    _need(status, "status", dtype=torch.int32, shape=(1,))
    sh, _ = _stream_handle(stream, status.device)
    _check(L.spec_selftest_bounded_wait(int(limit_ns), _ptr(status), sh), "spec_selftest_bounded_wait")
    return status


class HostVerifier:
    """Runs verify steps whose inputs and outputs live in (pinned) host
    memory: each ``run`` copies the step's inputs to the device, launches the
    verify kernel and copies tokens, accepted counts and overlaps back, all on
    one stream, then waits for the stream."""

    def __init__(self, B: int, K: int, V: int, dtype=torch.bfloat16, device="cuda",
                 stream: Optional[torch.cuda.Stream] = None):
        self.device = torch.device(device)
        self.stream = stream or torch.cuda.Stream(self.device)
        d = self.device
        self.target = torch.empty((B, K + 1, V), dtype=dtype, device=d)
        self.draft = torch.empty((B, K, V), dtype=dtype, device=d)
        self.tokens_in = torch.empty((B, K), dtype=torch.int32, device=d)
        self.ua = torch.empty((B, K), dtype=torch.float32, device=d)
        self.uf = torch.empty((B,), dtype=torch.float32, device=d)
        self.out = VerifyOutput(torch.empty((B, K + 1), dtype=torch.int32, device=d),
                                torch.empty((B,), dtype=torch.int32, device=d),
                                torch.empty((B, K), dtype=torch.float32, device=d),
                                torch.zeros((1,), dtype=torch.int32, device=d))
        self.ws = torch.zeros(max(lib().spec_verify_workspace_bytes(B, K, V), 256), dtype=torch.uint8, device=d)
        self.h2d_bytes = sum(t.numel() * t.element_size()
                             for t in (self.target, self.draft, self.tokens_in, self.ua, self.uf))
        self.d2h_bytes = sum(t.numel() * t.element_size() for t in (self.out.tokens, self.out.n_accepted,
                                                                   self.out.alpha))

    def run(self, target_h, draft_h, tokens_h, ua_h, uf_h, temperature, tokens_out_h, n_acc_out_h, alpha_out_h):
        with torch.cuda.stream(self.stream):
            self.target.copy_(target_h, non_blocking=True)
            self.draft.copy_(draft_h, non_blocking=True)
            self.tokens_in.copy_(tokens_h, non_blocking=True)
            self.ua.copy_(ua_h, non_blocking=True)
            self.uf.copy_(uf_h, non_blocking=True)
            verify(self.target, self.draft, self.tokens_in, self.ua, self.uf, temperature,
                   out=self.out, workspace=self.ws, stream=self.stream)
            tokens_out_h.copy_(self.out.tokens, non_blocking=True)
            n_acc_out_h.copy_(self.out.n_accepted, non_blocking=True)
            alpha_out_h.copy_(self.out.alpha, non_blocking=True)
        self.stream.synchronize()
