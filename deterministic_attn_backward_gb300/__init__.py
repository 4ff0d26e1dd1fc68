"""Deterministic attention backward for GB300 (sm_103a).

Thin Python binding over the C ABI of ``libdab.so`` (``include/dab.h``):
argument marshalling only.  Every step of the forward and backward runs in the
library's CUDA kernels; if the library is missing this module raises instead of
falling back to anything else.  PyTorch is used for device memory and streams.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import inputs  # noqa: F401  (seeded input generators)

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdab.so")

MASKS = {"full": 0, "causal": 1}
SCHEDS = {"serial": 0, "descending": 1, "descending_q": 1, "shift": 2, "atomic": 3, "auto": 4}
SCHED_NAMES = ("serial", "descending_q", "shift", "atomic")
STATUS = {0: "DAB_OK", 1: "DAB_ERR_INVALID_ARG", 2: "DAB_ERR_UNSUPPORTED", 3: "DAB_ERR_WORKSPACE",
          4: "DAB_ERR_CUDA", 5: "DAB_ERR_TIMEOUT", 6: "DAB_ERR_DEVICE_BOUNDS"}
DAB_BWD_SKIP_PREPROCESS = 0x1
DAB_BWD_SKIP_CONVERT = 0x2
DAB_BWD_SKIP_MAIN = 0x4
DAB_BWD_PLAIN_ADD = 0x8
DAB_BWD_SEPARATE_CONVERT = 0x10
DAB_BWD_SHARE_GPU = 0x20

EXPORTED = (
    "dab_attn_fwd", "dab_bwd_workspace_size", "dab_attn_bwd", "dab_check_status",
    "dab_status_string", "dab_attn_bwd_ex", "dab_bwd_preprocess", "dab_bwd_workspace_layout",
    "dab_sched_units_per_head", "dab_sched_unit_steps", "dab_sched_step", "dab_sched_rank",
    "dab_sched_contributors", "dab_sched_gang_size", "dab_dag_simulate", "dab_dag_critical_path",
    "dab_dag_simulate_ways", "dab_sched_select", "dab_attn_bwd_host", "dab_bwd_host_workspace_size",
    "dab_attn_fwd_block", "dab_attn_bwd_block", "dab_bwd_block_workspace_size",
    "dab_selftest_mma", "dab_last_error_string", "dab_attn_bwd_noalloc", "dab_mma_peak",
    "dab_mma_peak_grid", "dab_noalloc_check_status", "dab_fwd_limit_workspace_size",
    "dab_attn_fwd_limit", "dab_bwd_limit_workspace_size", "dab_attn_bwd_limit",
    "dab_embed_fwd", "dab_embed_bwd_workspace_size", "dab_embed_bwd",
    "dab_grad_workspace_size", "dab_grad_norm", "dab_grad_clip",
)


class DabError(RuntimeError):
    def __init__(self, code: int, what: str):
        detail = ""
        if code == 4 and _lib is not None:
            detail = " (" + _lib.dab_last_error_string().decode() + ")"
        super().__init__(f"{what}: {STATUS.get(code, code)}{detail}")
        self.code = code


class BwdOpts(ctypes.Structure):
    _fields_ = [("spin_timeout_ns", ctypes.c_uint64), ("flags", ctypes.c_uint32),
                ("grid", ctypes.c_int32)]


class WsLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("status", "sem", "D", "lse2", "dqacc", "total")]


class Grad(ctypes.Structure):
    """dab_grad_t: one tensor of a gradient list."""
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libdab.so (raises OSError if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise OSError(f"{path} is missing: build it with "
                      "`python -m deterministic_attn_backward_gb300.build`")
    lib = ctypes.CDLL(path)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.dab_attn_fwd.argtypes = [vp] * 5 + [i] * 4 + [f, i, vp, sz, vp]
    lib.dab_attn_fwd.restype = i
    lib.dab_bwd_workspace_size.argtypes = [i] * 6
    lib.dab_bwd_workspace_size.restype = sz
    lib.dab_attn_bwd.argtypes = [vp] * 9 + [i] * 4 + [f, i, i, vp, sz, vp]
    lib.dab_attn_bwd.restype = i
    lib.dab_attn_bwd_ex.argtypes = [vp] * 9 + [i] * 4 + [f, i, i, vp, sz, vp, ctypes.POINTER(BwdOpts)]
    lib.dab_attn_bwd_ex.restype = i
    lib.dab_bwd_preprocess.argtypes = [vp] * 3 + [i] * 6 + [vp, sz, vp]
    lib.dab_bwd_preprocess.restype = i
    lib.dab_bwd_workspace_layout.argtypes = [i] * 6 + [ctypes.POINTER(WsLayout)]
    lib.dab_bwd_workspace_layout.restype = i
    lib.dab_check_status.argtypes = [vp, vp]
    lib.dab_check_status.restype = i
    lib.dab_status_string.argtypes = [i]
    lib.dab_status_string.restype = ctypes.c_char_p
    lib.dab_last_error_string.argtypes = []
    lib.dab_last_error_string.restype = ctypes.c_char_p
    lib.dab_sched_units_per_head.argtypes = [i, i, i]
    lib.dab_sched_units_per_head.restype = i
    lib.dab_sched_unit_steps.argtypes = [i, i, i, i]
    lib.dab_sched_unit_steps.restype = i
    ip = ctypes.POINTER(ctypes.c_int)
    lib.dab_sched_step.argtypes = [i, i, i, i, i, ip, ip]
    lib.dab_sched_step.restype = i
    lib.dab_sched_rank.argtypes = [i, i, i, i, i]
    lib.dab_sched_rank.restype = i
    lib.dab_sched_contributors.argtypes = [i, i, i]
    lib.dab_sched_contributors.restype = i
    lib.dab_sched_gang_size.argtypes = [i, i, i]
    lib.dab_sched_gang_size.restype = i
    dp = ctypes.POINTER(ctypes.c_double)
    lib.dab_dag_simulate.argtypes = [i, i, i, i, i, ctypes.c_double, ctypes.c_double, i, dp, dp]
    lib.dab_dag_simulate.restype = i
    lib.dab_dag_simulate_ways.argtypes = [i, i, i, i, i, ctypes.c_double, ctypes.c_double, i, i, dp, dp]
    lib.dab_dag_simulate_ways.restype = i
    lib.dab_sched_select.argtypes = [i] * 5
    lib.dab_sched_select.restype = i
    lib.dab_bwd_host_workspace_size.argtypes = [i] * 7
    lib.dab_bwd_host_workspace_size.restype = sz
    lib.dab_attn_bwd_host.argtypes = [vp] * 9 + [i] * 4 + [f, i, i, vp, sz, i, vp]
    lib.dab_attn_bwd_host.restype = i
    lib.dab_attn_fwd_block.argtypes = [vp] * 5 + [i] * 4 + [f, vp, i, vp, sz, vp]
    lib.dab_attn_fwd_block.restype = i
    lib.dab_bwd_block_workspace_size.argtypes = [i] * 5
    lib.dab_bwd_block_workspace_size.restype = sz
    lib.dab_attn_bwd_block.argtypes = [vp] * 9 + [i] * 4 + [f, vp, i, i, vp, sz, vp]
    lib.dab_attn_bwd_block.restype = i
    lib.dab_fwd_limit_workspace_size.argtypes = [i]
    lib.dab_fwd_limit_workspace_size.restype = sz
    lib.dab_attn_fwd_limit.argtypes = [vp] * 5 + [i] * 4 + [f, vp, i, vp, sz, vp]
    lib.dab_attn_fwd_limit.restype = i
    lib.dab_bwd_limit_workspace_size.argtypes = [i] * 5
    lib.dab_bwd_limit_workspace_size.restype = sz
    lib.dab_attn_bwd_limit.argtypes = [vp] * 9 + [i] * 4 + [f, vp, i, i, vp, sz, vp]
    lib.dab_attn_bwd_limit.restype = i
    i64 = ctypes.c_int64
    lib.dab_embed_fwd.argtypes = [vp, i, vp, i, vp, i, i64, i64, i, f, vp, sz, vp]
    lib.dab_embed_fwd.restype = i
    lib.dab_embed_bwd_workspace_size.argtypes = [i64, i64, i]
    lib.dab_embed_bwd_workspace_size.restype = sz
    lib.dab_embed_bwd.argtypes = [vp, i, vp, i, vp, i, i64, i64, i, f, i64, i, vp, sz, vp]
    lib.dab_embed_bwd.restype = i
    lib.dab_grad_workspace_size.argtypes = [ctypes.POINTER(Grad), i]
    lib.dab_grad_workspace_size.restype = sz
    lib.dab_grad_norm.argtypes = [ctypes.POINTER(Grad), i, vp, vp, sz, vp]
    lib.dab_grad_norm.restype = i
    lib.dab_grad_clip.argtypes = [ctypes.POINTER(Grad), i, f, vp, vp, vp, sz, vp]
    lib.dab_grad_clip.restype = i
    lib.dab_dag_critical_path.argtypes = [i, i, i, ctypes.c_double, ctypes.c_double, i]
    lib.dab_dag_critical_path.restype = ctypes.c_double
    lib.dab_attn_bwd_noalloc.argtypes = [vp] * 9 + [i] * 4 + [f, i, i, vp]
    lib.dab_attn_bwd_noalloc.restype = i
    lib.dab_noalloc_check_status.argtypes = [vp]
    lib.dab_noalloc_check_status.restype = i
    lib.dab_selftest_mma.argtypes = [i] + [vp] * 10
    lib.dab_selftest_mma.restype = i
    lib.dab_mma_peak.argtypes = [i, vp, vp]
    lib.dab_mma_peak.restype = i
    lib.dab_mma_peak_grid.argtypes = []
    lib.dab_mma_peak_grid.restype = i
    _lib = lib
    return lib


def _check(code: int, what: str):
    if code != 0:
        raise DabError(code, what)


def _mask(mask) -> int:
    return MASKS[mask] if isinstance(mask, str) else int(mask)


def _sched(sched) -> int:
    return SCHEDS[sched] if isinstance(sched, str) else int(sched)


def _stream(device: torch.device) -> int:
    # the current stream's handle without a Stream object around it (2 us less a call)
    index = device.index
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if index is None else index)


def _shape(q: torch.Tensor):
    if q.dim() != 4:
        raise ValueError("expected [B, H, S, d] tensors")
    return tuple(int(x) for x in q.shape)


def _dev_bf16(t: torch.Tensor, device) -> torch.Tensor:
    if t.dtype != torch.bfloat16:
        raise TypeError("expected bfloat16 tensors")
    if t.device == device and t.is_contiguous():
        return t
    return t.to(device, non_blocking=True).contiguous()


def default_scale(d: int) -> float:
    return 1.0 / float(d) ** 0.5


def workspace_size(B, H, S, d, mask="full", sched="serial") -> int:
    return int(load_library().dab_bwd_workspace_size(B, H, S, d, _mask(mask), _sched(sched)))


def workspace_layout(B, H, S, d, mask="full", sched="serial") -> WsLayout:
    L = WsLayout()
    _check(load_library().dab_bwd_workspace_layout(B, H, S, d, _mask(mask), _sched(sched),
                                                   ctypes.byref(L)), "dab_bwd_workspace_layout")
    return L


def block_workspace_size(B, H, S, d, sched="descending_q") -> int:
    n = int(load_library().dab_bwd_block_workspace_size(B, H, S, d, _sched(sched)))
    if n == 0:
        raise DabError(1, "dab_bwd_block_workspace_size")
    return n


def limit_workspace_size(B, H, S, d, sched="descending_q") -> int:
    n = int(load_library().dab_bwd_limit_workspace_size(B, H, S, d, _sched(sched)))
    if n == 0:
        raise DabError(1, "dab_bwd_limit_workspace_size")
    return n


def new_workspace(B, H, S, d, mask="full", sched="serial", device="cuda", block=False,
                  limit=False) -> torch.Tensor:
    """Device workspace of the backward; `block` and `limit`: of the one under a
    block mask or key limits (the latter also serves the forward)."""
    if limit:
        n = limit_workspace_size(B, H, S, d, sched)
    else:
        n = block_workspace_size(B, H, S, d, sched) if block else workspace_size(B, H, S, d, mask, sched)
    return torch.empty(n, dtype=torch.uint8, device=device)


def _tiles(tiles, S, dev):
    """Block mask as a contiguous uint8 [S/128, S/128] CUDA tensor."""
    t = torch.as_tensor(tiles)
    if tuple(t.shape) != (S // 128, S // 128):
        raise ValueError("tiles must be [S/128, S/128]")
    return (t != 0).to(device=dev, dtype=torch.uint8).contiguous()


def prefix_limits(lengths, parents=None) -> torch.Tensor:
    """Key limits (int32 [sum(lengths)], on the CPU) of packed segments.

    Segment n has lengths[n] tokens and sees itself (causally) and all of
    segment parents[n] with everything that one sees; a parent of -1, or no
    `parents` at all, is a sequence of its own.  A segment's descendants
    follow it before any other segment (depth-first order).  One prompt and
    its answers: prefix_limits([prompt, a, b, c], [-1, 0, 0, 0])."""
    lengths = [int(x) for x in lengths]
    parents = [-1] * len(lengths) if parents is None else [int(x) for x in parents]
    if len(parents) != len(lengths):
        raise ValueError("one parent for each segment")
    if any(x < 0 for x in lengths):
        raise ValueError("segment lengths must not be negative")
    end, path, at = [0] * len(lengths), [], 0
    for n, (x, parent) in enumerate(zip(lengths, parents)):
        if parent < -1 or parent >= n:
            raise ValueError("a segment's parent comes before it (or is -1)")
        while path and path[-1] != parent:      # leave the subtrees that end here
            end[path.pop()] = at
        if parent >= 0 and not path:
            raise ValueError("a segment's descendants follow it before any other segment")
        path.append(n)
        at += x
    for n in path:
        end[n] = at
    if at >= 2 ** 31:
        raise ValueError("too many tokens")
    return torch.repeat_interleave(torch.tensor(end, dtype=torch.int32), torch.tensor(lengths, dtype=torch.int64))


# The checks of the calls below cost as much as the calls when they go through
# tensors' slower accessors: dtypes are compared as objects, devices by index.
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_WHOLE = (torch.int64, torch.int16, torch.int8, torch.uint8)


def _ready(t, dtype, index) -> bool:
    return t.dtype is dtype and t.get_device() == index and t.is_contiguous()


def _workspace(t, index):
    """(address, bytes) of a workspace that the caller gave."""
    if not _ready(t, _U8, index):
        raise ValueError("a workspace must be a contiguous uint8 tensor on the call's device")
    return t.data_ptr(), t.numel()


def _run(index, fn, *args):
    """fn(*args, stream) with the device current and its current stream; raises
    on a status that is not DAB_OK."""
    if index == torch._C._cuda_getDevice():
        code = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            code = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if code:
        raise DabError(code, fn.__name__)


def _copied(t, dev):
    """t on the device, contiguous, with the values it has now: the copy from pinned
    memory is asynchronous, so it is taken from a snapshot that the caller cannot
    refill meanwhile (from other host memory it is staged before the call returns).
    A graph under capture copies from the caller's pinned memory in every replay."""
    if t.device.type == "cpu" and t.is_pinned() and not torch.cuda.is_current_stream_capturing():
        t = torch.empty(t.shape, dtype=t.dtype, pin_memory=True).copy_(t)
    return t.to(dev, non_blocking=True).contiguous()


def _own_bf16(t, index, dev):
    if t.dtype is not _BF16:
        raise TypeError("expected bfloat16 tensors")
    return t if _ready(t, _BF16, index) else _copied(t, dev)


def _limit(limit, mask, S, dev):
    """Key limits as a contiguous int32 [S] CUDA tensor."""
    t = limit if isinstance(limit, torch.Tensor) else torch.as_tensor(limit)
    if mask != "causal" and _mask(mask) != MASKS["causal"]:
        raise ValueError('limit goes with mask="causal"')
    if t.shape != (S,):
        raise ValueError("limit must be [S]")
    if t.dtype is not _I32:
        if t.dtype not in _WHOLE:
            raise TypeError("limit must hold whole numbers")
        t = t.clamp(0, S).to(_I32) if t.dtype is torch.int64 else t.to(_I32)    # narrower ones fit as they are
    return t if t.device == dev and t.is_contiguous() else _copied(t, dev)


def attn_fwd(q, k, v, mask="full", scale=None, workspace=None, out=None, lse=None, tiles=None, limit=None,
             tokens=None):
    """O (bf16 [B,H,S,d]) and LSE (f32 [B,H,S]) on q's CUDA device.
    `tiles`: optional block mask [S/128, S/128] (dab_attn_fwd_block).
    `limit`: key limits [S] of packed sequences and shared prefixes (int32, or
    other signed whole numbers or uint8, which are converted), with
    mask="causal": key c is visible to the queries c <= q < limit[c]
    (dab_attn_fwd_limit; see prefix_limits).  `tokens`: with limit, how many rows
    of a head are in use; those behind them are not read, and stay as they are in
    out and lse (0 in new tensors)."""
    lib = load_library()
    if limit is not None:
        return _attn_fwd_limit(q, k, v, mask, scale, workspace, out, lse, tiles, limit, tokens)
    if tokens is not None:
        raise ValueError("tokens goes with limit")
    B, H, S, d = _shape(q)
    dev = q.device if q.is_cuda else torch.device("cuda")
    q, k, v = (_dev_bf16(t, dev) for t in (q, k, v))
    o = out if out is not None else torch.empty_like(q)
    lse_t = lse if lse is not None else torch.empty((B, H, S), dtype=torch.float32, device=dev)
    ws_ptr, ws_n = (workspace.data_ptr(), workspace.numel()) if workspace is not None else (None, 0)
    sc = float(scale if scale is not None else default_scale(d))
    if tiles is None:
        _check(lib.dab_attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                lse_t.data_ptr(), B, H, S, d, sc, _mask(mask), ws_ptr, ws_n,
                                _stream(dev)), "dab_attn_fwd")
    else:
        t = _tiles(tiles, S, dev)
        _check(lib.dab_attn_fwd_block(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                      lse_t.data_ptr(), B, H, S, d, sc, t.data_ptr(), _mask(mask),
                                      ws_ptr, ws_n, _stream(dev)), "dab_attn_fwd_block")
    return o, lse_t


def _given(t, shape, dtype, index, what):
    """An output that the caller gave: it is written in place."""
    if t.shape != shape or not _ready(t, dtype, index):
        raise ValueError(f"{what} must be contiguous {dtype} {list(shape)} on the call's device")
    return t


def _tokens(tokens, S):
    if tokens is None:
        return S
    if not 0 <= tokens <= S:
        raise ValueError("tokens must be from 0 to S")
    return int(tokens)


def _attn_fwd_limit(q, k, v, mask, scale, workspace, out, lse, tiles, limit, tokens):
    """dab_attn_fwd_limit; CPU tensors are copied to the current device."""
    lib = _lib or load_library()
    if tiles is not None:
        raise ValueError("tiles and limit do not go together")
    shape = q.shape
    if len(shape) != 4 or k.shape != shape or v.shape != shape:
        raise ValueError("q, k and v must have one shape [B, H, S, d]")
    B, H, S, d = shape
    index = q.get_device() if q.is_cuda else torch.cuda.current_device()
    dev = q.device if q.is_cuda else torch.device("cuda", index)
    if not (_ready(q, _BF16, index) and _ready(k, _BF16, index) and _ready(v, _BF16, index)):
        q, k, v = (_own_bf16(t, index, dev) for t in (q, k, v))
    lim = _limit(limit, mask, S, dev)
    tokens = _tokens(tokens, S)
    new = torch.empty if tokens == S else torch.zeros
    out = new(shape, dtype=_BF16, device=dev) if out is None else _given(out, shape, _BF16, index, "out")
    if lse is None:
        lse = new((B, H, S), dtype=_F32, device=dev)
    else:
        _given(lse, (B, H, S), _F32, index, "lse")
    if workspace is None:
        workspace = torch.empty(max(256, lib.dab_fwd_limit_workspace_size(S)), dtype=_U8, device=dev)
    ws, ws_bytes = _workspace(workspace, index)
    _run(index, lib.dab_attn_fwd_limit, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
         B, H, S, d, default_scale(d) if scale is None else scale, lim.data_ptr(), tokens, ws, ws_bytes)
    return out, lse


def host_workspace_size(B, H, S, d, mask="full", sched="serial", chunks=0) -> int:
    n = load_library().dab_bwd_host_workspace_size(B, H, S, d, _mask(mask), _sched(sched), chunks)
    if n == 0:
        raise DabError(1, "dab_bwd_host_workspace_size")
    return n


def new_host_workspace(B, H, S, d, mask="full", sched="serial", chunks=0, device="cuda"):
    """Device workspace of the host-buffer path (dab_attn_bwd_host)."""
    return torch.empty(host_workspace_size(B, H, S, d, mask, sched, chunks), dtype=torch.uint8,
                       device=device)


def _attn_bwd_host(q, k, v, o, lse, dout, mask, sched, scale, workspace, out, chunks):
    """CPU tensors through dab_attn_bwd_host (copies overlapped with the
    computation inside the library); returns once the gradients are in host
    memory.  Pinned inputs and outputs give asynchronous copies."""
    lib = load_library()
    B, H, S, d = _shape(q)
    dev = torch.device("cuda", torch.cuda.current_device())
    q, k, v, o, dout = (t.contiguous() if t.dtype == torch.bfloat16 else t.to(torch.bfloat16).contiguous()
                        for t in (q, k, v, o, dout))
    lse = lse.contiguous()
    if lse.dtype != torch.float32:
        raise TypeError("lse must be float32")
    if workspace is None:
        workspace = new_host_workspace(B, H, S, d, mask, sched, chunks, dev)
    if out is None:
        out = tuple(torch.empty(q.shape, dtype=torch.bfloat16, pin_memory=True) for _ in range(3))
    dq, dk, dv = out
    _check(lib.dab_attn_bwd_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                 dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, S, d,
                                 float(scale if scale is not None else default_scale(d)), _mask(mask),
                                 _sched(sched), workspace.data_ptr(), workspace.numel(), chunks,
                                 _stream(dev)), "dab_attn_bwd_host")
    torch.cuda.current_stream(dev).synchronize()
    return dq, dk, dv


def attn_bwd(q, k, v, o, lse, dout, mask="full", sched="serial", scale=None, workspace=None,
             out=None, opts: BwdOpts | None = None, chunks: int = 0, tiles=None, limit=None, tokens=None):
    """dQ, dK, dV (bf16 [B,H,S,d]) through the C ABI.

    Device tensors are used in place (dab_attn_bwd / dab_attn_bwd_ex).  CPU
    tensors go through dab_attn_bwd_host, which copies them to the device
    and the gradients back, overlapped with the computation in `chunks`
    groups of heads (0 = the library's default); `workspace` is then the
    device workspace of new_host_workspace() and `out` host tensors.
    `tiles`, `limit`, `tokens`: as for attn_fwd (device tensors only).
    """
    lib = load_library()
    if limit is not None:
        return _attn_bwd_limit(q, k, v, o, lse, dout, mask, sched, scale, workspace, out, opts, tiles, limit, tokens)
    if tokens is not None:
        raise ValueError("tokens goes with limit")
    B, H, S, d = _shape(q)
    host = not q.is_cuda
    if tiles is not None:
        return _attn_bwd_block(q, k, v, o, lse, dout, mask, sched, scale, workspace, out, tiles)
    if host:
        if opts is not None:
            raise ValueError("opts apply to device tensors only")
        return _attn_bwd_host(q, k, v, o, lse, dout, mask, sched, scale, workspace, out, chunks)
    dev = q.device
    q, k, v, o, dout = (_dev_bf16(t, dev) for t in (q, k, v, o, dout))
    lse = lse.to(dev, non_blocking=True).contiguous()
    if lse.dtype != torch.float32:
        raise TypeError("lse must be float32")
    if workspace is None:
        workspace = new_workspace(B, H, S, d, mask, sched, dev)
    if out is None:
        out = (torch.empty_like(q), torch.empty_like(q), torch.empty_like(q))
    dq, dk, dv = out
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
            dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, S, d,
            float(scale if scale is not None else default_scale(d)), _mask(mask), _sched(sched),
            workspace.data_ptr(), workspace.numel(), _stream(dev))
    if opts is None:
        _check(lib.dab_attn_bwd(*args), "dab_attn_bwd")
    else:
        _check(lib.dab_attn_bwd_ex(*args, ctypes.byref(opts)), "dab_attn_bwd_ex")
    return dq, dk, dv


def _attn_bwd_block(q, k, v, o, lse, dout, mask, sched, scale, workspace, out, tiles):
    """dab_attn_bwd_block on CUDA tensors (mask: "full" or "causal")."""
    lib = load_library()
    B, H, S, d = _shape(q)
    dev = q.device
    q, k, v, o, dout = (_dev_bf16(t, dev) for t in (q, k, v, o, dout))
    t = _tiles(tiles, S, dev)
    if workspace is None:
        workspace = new_workspace(B, H, S, d, sched=sched, device=dev, block=True)
    if out is None:
        out = (torch.empty_like(q), torch.empty_like(q), torch.empty_like(q))
    dq, dk, dv = out
    _check(lib.dab_attn_bwd_block(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                  dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, S, d,
                                  float(scale if scale is not None else default_scale(d)), t.data_ptr(),
                                  _mask(mask), _sched(sched), workspace.data_ptr(), workspace.numel(),
                                  _stream(dev)), "dab_attn_bwd_block")
    return dq, dk, dv


def _attn_bwd_limit(q, k, v, o, lse, dout, mask, sched, scale, workspace, out, opts, tiles, limit, tokens):
    """dab_attn_bwd_limit on CUDA tensors."""
    lib = _lib or load_library()
    if tiles is not None or opts is not None:
        raise ValueError("limit goes without tiles and opts")
    if not q.is_cuda:
        raise ValueError("limit applies to device tensors only")
    shape = q.shape
    if len(shape) != 4 or k.shape != shape or v.shape != shape or o.shape != shape or dout.shape != shape:
        raise ValueError("q, k, v, o and dout must have one shape [B, H, S, d]")
    B, H, S, d = shape
    if lse.shape != (B, H, S):
        raise ValueError("lse must be [B, H, S]")
    index, dev = q.get_device(), q.device
    if not (_ready(q, _BF16, index) and _ready(k, _BF16, index) and _ready(v, _BF16, index)
            and _ready(o, _BF16, index) and _ready(dout, _BF16, index)):
        q, k, v, o, dout = (_own_bf16(t, index, dev) for t in (q, k, v, o, dout))
    if not _ready(lse, _F32, index):
        if lse.dtype is not _F32:
            raise TypeError("lse must be float32")
        lse = _copied(lse, dev)
    lim = _limit(limit, mask, S, dev)
    if workspace is None:
        workspace = new_workspace(B, H, S, d, mask, sched, dev, limit=True)
    ws, ws_bytes = _workspace(workspace, index)
    tokens = _tokens(tokens, S)
    if out is None:
        new = torch.empty_like if tokens == S else torch.zeros_like
        dq, dk, dv = new(q), new(q), new(q)
    else:
        dq, dk, dv = (_given(t, shape, _BF16, index, "out") for t in out)
    _run(index, lib.dab_attn_bwd_limit, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
         dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, S, d,
         default_scale(d) if scale is None else scale, lim.data_ptr(), tokens, _sched(sched), ws, ws_bytes)
    return dq, dk, dv


# --------------------------------------------- the rest of a training step
_FLOATS = {torch.bfloat16: 0, torch.float32: 1}
_INDEXES = {torch.int32: 2, torch.int64: 3}


def _float_type(t, index, what):
    """The library's number for t's dtype, t being a contiguous tensor on the device."""
    code = _FLOATS.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} must be bfloat16 or float32")
    if index < 0 or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous CUDA tensor on the call's device")
    return code


def _ids(ids, index, dev):
    """(ids on the device, contiguous; the library's number for their dtype)."""
    code = _INDEXES.get(ids.dtype)
    if code is None:
        raise TypeError("ids must be int32 or int64")
    if ids.get_device() != index or not ids.is_contiguous():
        ids = _copied(ids, dev)
    return ids, code


def embed_fwd(ids, table, scale=1.0, dtype=None, out=None, workspace=None) -> torch.Tensor:
    """scale * table[ids] (dab_embed_fwd): ids int32 or int64 of any shape, table
    [rows, width] bfloat16 or float32, the result ids.shape + [width] in `dtype`
    (the table's if not given) or in `out`.  A token outside the table gives
    zeros and, with a `workspace` (256 bytes or more), check_status() says so."""
    lib = _lib or load_library()
    index, dev = table.get_device(), table.device
    table_type = _float_type(table, index, "table")
    if table.dim() != 2:
        raise ValueError("table must be [rows, width]")
    ids, ids_type = _ids(ids, index, dev)
    rows, width = table.shape
    shape = (*ids.shape, width)
    if out is None:
        out = torch.empty(shape, dtype=dtype or table.dtype, device=dev)
    elif out.shape != shape or (dtype is not None and out.dtype is not dtype):
        raise ValueError("out must be ids.shape + [width], in `dtype`")
    ws, ws_bytes = (None, 0) if workspace is None else _workspace(workspace, index)
    _run(index, lib.dab_embed_fwd, ids.data_ptr(), ids_type, table.data_ptr(), table_type, out.data_ptr(),
         _float_type(out, index, "out"), ids.numel(), rows, width, scale, ws, ws_bytes)
    return out


def embed_workspace_size(n, rows, width) -> int:
    size = int(load_library().dab_embed_bwd_workspace_size(n, rows, width))
    if size == 0:
        raise DabError(1, "dab_embed_bwd_workspace_size")
    return size


def new_embed_workspace(n, rows, width, device="cuda") -> torch.Tensor:
    """Device workspace of embed_bwd for n tokens of a [rows, width] table."""
    return torch.empty(embed_workspace_size(n, rows, width), dtype=torch.uint8, device=device)


def embed_bwd(ids, dout, rows=None, scale=1.0, dtype=None, out=None, accumulate=False, padding=None,
              workspace=None) -> torch.Tensor:
    """The table's gradient [rows, width] (dab_embed_bwd): row v is scale * the sum
    of dout over the tokens equal to v, in a fixed order (the same bits in every
    call).  dout: ids.shape + [width].  The result is a new tensor of `rows` rows
    in `dtype` (dout's if not given), or `out`, overwritten or with accumulate=True
    added to.  Tokens equal to `padding` get no gradient."""
    lib = _lib or load_library()
    index, dev = dout.get_device(), dout.device
    dout_type = _float_type(dout, index, "dout")
    ids, ids_type = _ids(ids, index, dev)
    if dout.dim() < 1 or dout.shape[:-1] != ids.shape:
        raise ValueError("dout must be ids.shape + [width]")
    width = dout.shape[-1]
    if out is None:
        if accumulate or rows is None:
            raise ValueError("give out (to accumulate) or rows")
        out = torch.empty((rows, width), dtype=dtype or dout.dtype, device=dev)
    elif (out.dim() != 2 or out.shape[1] != width or (rows is not None and out.shape[0] != rows)
          or (dtype is not None and out.dtype is not dtype)):
        raise ValueError("out must be [rows, width], in `dtype`")
    rows, n = out.shape[0], ids.numel()
    if workspace is None:
        workspace = new_embed_workspace(n, rows, width, dev)
    ws, ws_bytes = _workspace(workspace, index)
    _run(index, lib.dab_embed_bwd, ids.data_ptr(), ids_type, dout.data_ptr(), dout_type, out.data_ptr(),
         _float_type(out, index, "out"), n, rows, width, scale, -1 if padding is None else padding,
         1 if accumulate else 0, ws, ws_bytes)
    return out


class GradList:
    """A list of gradient tensors as the library takes it, with a workspace of
    its own: made once for gradients that stay where they are and passed to
    grad_norm() and clip_grads() in every step.  `out`: where the clipped
    gradients go (in place if not given).  One list serves one stream at a time,
    which need not be the one it was made on, and outlives the graphs that
    captured a call with it."""

    def __init__(self, grads, out=None):
        lib = load_library()
        # aliases: the memory stays, also when a tensor is given another
        self.grads = [g.detach() for g in grads]
        self.out = self.grads if out is None else [o.detach() for o in out]
        if len(self.out) != len(self.grads):
            raise ValueError("one out tensor for each gradient")
        self.index = self.grads[0].get_device() if self.grads else torch.cuda.current_device()
        for g, o in zip(self.grads, self.out):
            _float_type(g, self.index, "every gradient")
            _float_type(o, self.index, "every out tensor")
            if o.shape != g.shape or o.dtype != g.dtype:
                raise ValueError("an out tensor must have its gradient's shape and dtype")
        self.array = (Grad * len(self.grads))(*[
            Grad(g.data_ptr(), o.data_ptr(), g.numel(), _FLOATS[g.dtype], 0) for g, o in zip(self.grads, self.out)])
        size = lib.dab_grad_workspace_size(self.array, len(self.grads))
        if size == 0:
            raise DabError(1, "dab_grad_workspace_size")
        self.device = torch.device("cuda", self.index)
        self.stream = torch._C._cuda_getCurrentRawStream(self.index)    # that the workspace belongs to
        self.workspace = torch.empty(size, dtype=_U8, device=self.device)
        self.args = (self.array, len(self.grads))
        self.ws = (self.workspace.data_ptr(), size)

    def _used(self):
        """Before a call: keeps the workspace's memory from being handed out, once the
        list is dropped, before the current stream is done with it."""
        if torch._C._cuda_getCurrentRawStream(self.index) != self.stream:
            self.workspace.record_stream(torch.cuda.current_stream(self.device))


def grad_norm(grads, out=None) -> torch.Tensor:
    """The 2-norm of all gradients together (dab_grad_norm), a float32 scalar on
    the device: the same bits in every call.  grads: a GradList, or tensors."""
    lib = _lib or load_library()
    if not isinstance(grads, GradList):
        grads = GradList(grads)
    norm = torch.empty((), dtype=_F32, device=grads.device) if out is None else _scalar(out, grads.index, "out")
    grads._used()
    _run(grads.index, lib.dab_grad_norm, *grads.args, norm.data_ptr(), *grads.ws)
    return norm


def clip_grads(grads, max_norm, norm=None) -> torch.Tensor:
    """Scales the gradients by min(1, max_norm / (norm + 1e-6)) in place, or into
    the GradList's out tensors, and returns the norm before (dab_grad_clip).
    `norm`: a float32 scalar to use instead of the gradients' own, such as the
    norm over several ranks."""
    lib = _lib or load_library()
    if not isinstance(grads, GradList):
        grads = GradList(grads)
    given = None if norm is None else _scalar(norm, grads.index, "norm").data_ptr()
    total = torch.empty((), dtype=_F32, device=grads.device)
    grads._used()
    _run(grads.index, lib.dab_grad_clip, *grads.args, max_norm, given, total.data_ptr(), *grads.ws)
    return total


def _scalar(t, index, what):
    if t.numel() != 1 or not _ready(t, _F32, index):
        raise ValueError(f"{what} must be one float32 on the gradients' device")
    return t


def bwd_preprocess(o, lse, dout, mask, sched, workspace):
    lib = load_library()
    B, H, S, d = _shape(o)
    _check(lib.dab_bwd_preprocess(o.data_ptr(), lse.data_ptr(), dout.data_ptr(), B, H, S, d,
                                  _mask(mask), _sched(sched), workspace.data_ptr(),
                                  workspace.numel(), _stream(o.device)), "dab_bwd_preprocess")


def check_status(workspace: torch.Tensor) -> int:
    """Synchronise the current stream and return the workspace status code."""
    return int(load_library().dab_check_status(workspace.data_ptr(), _stream(workspace.device)))


# ------------------------------------------------------------ schedules (host)
def sched_units_per_head(sched, mask, N) -> int:
    return load_library().dab_sched_units_per_head(_sched(sched), _mask(mask), N)


def sched_unit_steps(sched, mask, N, u) -> int:
    return load_library().dab_sched_unit_steps(_sched(sched), _mask(mask), N, u)


def sched_unit(sched, mask, N, u):
    """[(kv_tile, q_tile), ...] of unit u, in execution order."""
    lib = load_library()
    kv, qt = ctypes.c_int(), ctypes.c_int()
    out = []
    for t in range(sched_unit_steps(sched, mask, N, u)):
        _check(lib.dab_sched_step(_sched(sched), _mask(mask), N, u, t, ctypes.byref(kv),
                                  ctypes.byref(qt)), "dab_sched_step")
        out.append((kv.value, qt.value))
    return out


def sched_rank(sched, mask, N, i, j) -> int:
    return load_library().dab_sched_rank(_sched(sched), _mask(mask), N, i, j)


def sched_contributors(mask, N, j) -> int:
    return load_library().dab_sched_contributors(_mask(mask), N, j)


def sched_gang_size(sched, mask, N) -> int:
    return load_library().dab_sched_gang_size(_sched(sched), _mask(mask), N)


def dag_simulate(sched, mask, N, heads, ctas, wc=1.0, wr=0.0, reducer_depth=0, ways=1):
    """(status, makespan, busy_fraction) of the schedule's DAG model."""
    mk, busy = ctypes.c_double(), ctypes.c_double()
    rc = load_library().dab_dag_simulate_ways(_sched(sched), _mask(mask), N, heads, ctas, wc, wr,
                                              reducer_depth, ways, ctypes.byref(mk),
                                              ctypes.byref(busy))
    return rc, mk.value, busy.value


def sched_select(mask, B: int, H: int, S: int, ctas: int) -> str:
    """The deterministic schedule the library runs for DAB_SCHED_AUTO on
    `ctas` CTAs (the SM count of the device)."""
    r = load_library().dab_sched_select(_mask(mask), B, H, S, ctas)
    if r < 0:
        raise DabError(1, "dab_sched_select")
    return SCHED_NAMES[r]


def dag_critical_path(sched, mask, N, wc=1.0, wr=0.0, reducer_depth=0) -> float:
    return load_library().dab_dag_critical_path(_sched(sched), _mask(mask), N, wc, wr, reducer_depth)


def selftest_mma(d: int, x, y, z, pm):
    """Run the tensor-core operand self-test; returns (out0, out1, out2, out3)."""
    lib = load_library()
    dev = x.device
    out0 = torch.empty((128, 128), dtype=torch.float32, device=dev)
    out1 = torch.empty((128, d), dtype=torch.float32, device=dev)
    out2 = torch.empty((128, d), dtype=torch.float32, device=dev)
    out3 = torch.empty((128, 128 if d == 128 else 64), dtype=torch.float32, device=dev)
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    _check(lib.dab_selftest_mma(d, x.data_ptr(), y.data_ptr(), z.data_ptr(), pm.data_ptr(),
                                out0.data_ptr(), out1.data_ptr(), out2.data_ptr(), out3.data_ptr(),
                                ws.data_ptr(), _stream(dev)), "dab_selftest_mma")
    _check(check_status(ws), "selftest device status")
    return out0, out1, out2, out3


def mma_peak(iters: int = 100000, device=None) -> dict:
    """Dense bf16 tensor throughput of the library's own tcgen05 path: one
    timed launch of `iters` x 4 MMAs (128 x 256 x 16) per SM, after one
    untimed warm-up launch.  Returns {"tflops", "ms", "grid", "iters"}."""
    lib = load_library()
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    stream = _stream(dev)
    grid = lib.dab_mma_peak_grid()
    _check(lib.dab_mma_peak(max(1, iters // 10), ws.data_ptr(), stream), "dab_mma_peak")
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    _check(lib.dab_mma_peak(iters, ws.data_ptr(), stream), "dab_mma_peak")
    e1.record()
    e1.synchronize()
    _check(check_status(ws), "dab_mma_peak device status")
    ms = e0.elapsed_time(e1)
    flops = float(grid) * iters * 4 * 2 * 128 * 256 * 16
    return {"tflops": flops / (ms * 1e-3) / 1e12, "ms": ms, "grid": grid, "iters": iters}
