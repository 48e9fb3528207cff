"""Python binding of the C ABI: argument marshalling only.

Every step of the verification runs in the CUDA kernels of libspecverify;
PyTorch provides device memory and the current stream.  Function names and
argument order follow include/spec_verify.h.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import numpy as np
import torch

from . import _native

SV_F32 = 0
SV_BF16 = 1
REQ_BAD_TOKEN = 1
REQ_BAD_LOGITS = 2
REQ_BAD_DRAFT_LEN = 4
REQ_TIMEOUT = 8
REQ_BAD_TREE = 16
MAX_K = 31


class VerifyError(RuntimeError):
    def __init__(self, code):
        msg = _native.lib().spec_verify_status_string(int(code)).decode()
        super().__init__("spec_verify failed (%d): %s" % (code, msg))
        self.code = int(code)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SV_BF16
    if t.dtype == torch.float32:
        return SV_F32
    raise TypeError("logits must be torch.bfloat16 or torch.float32, got %s" % t.dtype)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(t: torch.Tensor, name, device, dtype=None, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != device:
        raise ValueError("%s must be on %s (got %s)" % (name, device, t.device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s (got %s)" % (name, dtype, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s (got %s)" % (name, tuple(shape), tuple(t.shape)))


# ---------------------------------------------------------------------------
# workspaces: one per (device, stream), grown on demand, zero-filled once
# ---------------------------------------------------------------------------

_workspaces = {}


def workspace(B: int, K: int, V: int, device: torch.device, *, need: Optional[int] = None):
    """The (device, stream)'s workspace, grown to the bytes a (B, K, V) call
    needs (or to ``need`` bytes when given)."""
    lib = _native.lib()
    if need is None:
        need = int(lib.spec_verify_workspace_size(B, K, V))
    if need == 0 and B > 0:
        raise ValueError("unsupported shape B=%d K=%d V=%d" % (B, K, V))
    stream = torch.cuda.current_stream(device)
    key = (device.index, stream.cuda_stream)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < need:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
        rc = lib.spec_verify_workspace_init(_p(ws), ws.numel(), _stream(device))
        if rc:
            raise VerifyError(rc)
        _workspaces[key] = ws
    return ws


@dataclass
class VerifyOutputs:
    tokens: torch.Tensor           # [B, K+1] int32
    accept_len: torch.Tensor       # [B] int32
    cu_accept: Optional[torch.Tensor] = None   # [B+1]
    packed: Optional[torch.Tensor] = None      # [B*(K+1)]
    batch_id: Optional[torch.Tensor] = None    # [B*(K+1)]
    accept_prob: Optional[torch.Tensor] = None  # [B, K] fp32
    status: Optional[torch.Tensor] = None      # [B]
    cut: Optional[torch.Tensor] = None         # [B, R] fp32 (filtered calls)


def alloc_outputs(B, K, device, *, packed=True, accept_prob=True, status=True):
    i32 = dict(dtype=torch.int32, device=device)
    return VerifyOutputs(
        tokens=torch.empty((B, K + 1), **i32), accept_len=torch.empty((B,), **i32),
        cu_accept=torch.empty((B + 1,), **i32) if packed else None,
        packed=torch.empty((B * (K + 1),), **i32) if packed else None,
        batch_id=torch.empty((B * (K + 1),), **i32) if packed else None,
        accept_prob=torch.empty((B, K), dtype=torch.float32, device=device) if accept_prob else None,
        status=torch.empty((B,), **i32) if status else None)


def _validate_batch(target_logits, draft_tokens, draft_lens):
    if target_logits.dim() != 3:
        raise ValueError("target_logits must be [B, K+1, V]")
    B, K1, V = target_logits.shape
    K = K1 - 1
    device = target_logits.device
    if device.type != "cuda":
        raise ValueError("target_logits must be a CUDA tensor")
    _check(target_logits, "target_logits", device)
    if K > 0 or draft_tokens is not None:
        _check(draft_tokens, "draft_tokens", device, torch.int32, (B, K))
    if draft_lens is not None:
        _check(draft_lens, "draft_lens", device, torch.int32, (B,))
    return B, K, V, device


def _check_mask(token_mask, B, K, V, device):
    if token_mask is not None:
        _check(token_mask, "token_mask", device, torch.int32, (B, K + 1, (V + 31) // 32))


def spec_verify_sample(target_logits, draft_logits, draft_tokens, uniforms, temperature,
                       out: Optional[VerifyOutputs] = None, *, draft_lens=None,
                       packed=True, accept_prob=True, status=True,
                       token_mask=None, top_k=0, top_p=1.0, cut=False) -> VerifyOutputs:
    """Rejection-sampling verification of one batch (see spec_verify.h).

    target_logits [B, K+1, V] bf16/fp32 CUDA; draft_logits [B, K, V] same
    dtype or None (one-hot drafts); draft_tokens [B, K] int32; uniforms
    [B, K+1] fp32; temperature >= 0 (0 = greedy rule); token_mask
    [B, K+1, ceil(V/32)] int32 grammar masks or None (bit j % 32 of word
    j // 32 set = token j allowed at that position); top_k (0 = off) and
    top_p (1.0 = off) filter every sampled distribution; cut=True (filtered
    calls) also returns out.cut [B, R], each row's lowest kept logit (R =
    K+1 target rows, then K draft rows with draft logits)."""
    B, K, V, device = _validate_batch(target_logits, draft_tokens, draft_lens)
    if draft_logits is not None:
        _check(draft_logits, "draft_logits", device, target_logits.dtype, (B, K, V))
    _check(uniforms, "uniforms", device, torch.float32, (B, K + 1))
    _check_mask(token_mask, B, K, V, device)
    if out is None:
        out = alloc_outputs(B, K, device, packed=packed, accept_prob=accept_prob, status=status)
    filtered = top_k != 0 or top_p != 1.0
    if filtered and cut and out.cut is None:
        R = K + 1 + (K if draft_logits is not None else 0)
        out.cut = torch.empty((B, R), dtype=torch.float32, device=device)
    ws = workspace(B, K, V, device)
    lib = _native.lib()
    head = (_p(target_logits), _p(draft_logits), _p(draft_tokens), _p(uniforms),
            ctypes.c_float(float(temperature)))
    mid = (_p(out.tokens), _p(out.accept_len), _dtype_code(target_logits), B, K, V,
           _p(draft_lens), _p(out.cu_accept), _p(out.packed), _p(out.batch_id),
           _p(out.accept_prob))
    end = (_p(out.status), _p(ws), ws.numel(), _stream(device))
    tail = mid + end
    if filtered:
        rc = lib.spec_verify_sample_filtered(*head, int(top_k), ctypes.c_float(float(top_p)),
                                             _p(token_mask), *mid,
                                             _p(out.cut if cut else None), *end)
    elif token_mask is None:
        rc = lib.spec_verify_sample(*head, *tail)
    else:
        rc = lib.spec_verify_sample_masked(*head, _p(token_mask), *tail)
    if rc:
        raise VerifyError(rc)
    return out


def spec_verify_greedy(target_logits, draft_tokens, out: Optional[VerifyOutputs] = None, *,
                       draft_lens=None, packed=True, status=True,
                       token_mask=None) -> VerifyOutputs:
    """Greedy verification: accept while the draft equals the target argmax
    (over the tokens token_mask allows, when given)."""
    B, K, V, device = _validate_batch(target_logits, draft_tokens, draft_lens)
    _check_mask(token_mask, B, K, V, device)
    if out is None:
        out = alloc_outputs(B, K, device, packed=packed, accept_prob=False, status=status)
    ws = workspace(B, K, V, device)
    lib = _native.lib()
    tail = (_p(out.tokens), _p(out.accept_len), _dtype_code(target_logits), B, K, V,
            _p(draft_lens), _p(out.cu_accept), _p(out.packed), _p(out.batch_id), _p(out.status),
            _p(ws), ws.numel(), _stream(device))
    if token_mask is None:
        rc = lib.spec_verify_greedy(_p(target_logits), _p(draft_tokens), *tail)
    else:
        rc = lib.spec_verify_greedy_masked(_p(target_logits), _p(draft_tokens), _p(token_mask),
                                           *tail)
    if rc:
        raise VerifyError(rc)
    return out


@dataclass
class TreeOutputs:
    tokens: torch.Tensor      # [B, max_depth+1]
    accept_len: torch.Tensor  # [B]
    path: Optional[torch.Tensor] = None
    status: Optional[torch.Tensor] = None


def tree_depth(parent) -> int:
    """Depth of a host-side parent array (parent of node n at index n-1)."""
    d = [0]
    for n, p in enumerate(np.asarray(parent, dtype=np.int64).reshape(-1), start=1):
        if p < 0 or p >= n:
            raise ValueError("parent of node %d must be an earlier node (got %d)" % (n, p))
        d.append(d[p] + 1)
    return max(d)


def _tree_args(target_logits, tree_parent, tree_tokens, max_depth):
    """(B, N, V, device, parent tensor, parent stride, max_depth).  tree_parent:
    a CUDA int32 tensor [N] (one tree) or [B, N] (a tree per request) - then
    max_depth must be given - or a host array [N] / [B, N], copied to the
    device, whose depth is the default max_depth."""
    if target_logits.dim() != 3:
        raise ValueError("target_logits must be [B, N+1, V]")
    B, N1, V = target_logits.shape
    N = N1 - 1
    device = target_logits.device
    _check(target_logits, "target_logits", device)
    if not (isinstance(tree_parent, torch.Tensor) and tree_parent.device == device):
        host = np.ascontiguousarray(np.asarray(tree_parent, dtype=np.int32))
        if max_depth is None:
            max_depth = max(tree_depth(r) for r in host.reshape(-1, N)) if N else 0
        tree_parent = torch.from_numpy(host).to(device)
    if max_depth is None:
        raise ValueError("max_depth is required with a device-side tree_parent")
    if tuple(tree_parent.shape) == (N,):
        stride = 0
    elif tuple(tree_parent.shape) == (B, N):
        stride = N
    else:
        raise ValueError("tree_parent must be [N] or [B, N] (N = %d)" % N)
    _check(tree_parent, "tree_parent", device, torch.int32)
    _check(tree_tokens, "tree_tokens", device, torch.int32, (B, N))
    return B, N, V, device, tree_parent, stride, int(max_depth)


def _tree_outputs(B, D1, device, path, status):
    i32 = dict(dtype=torch.int32, device=device)
    return TreeOutputs(tokens=torch.empty((B, D1), **i32), accept_len=torch.empty((B,), **i32),
                       path=torch.empty((B, D1), **i32) if path else None,
                       status=torch.empty((B,), **i32) if status else None)


def spec_verify_tree(target_logits, tree_parent, tree_tokens, max_depth=None,
                     out: Optional[TreeOutputs] = None, *, path=True, status=True) -> TreeOutputs:
    """Greedy tree verification.  tree_parent [N] or [B, N] (parent of node n
    at index n-1; device tensor, or host array copied to the device);
    tree_tokens [B, N] int32 CUDA."""
    B, N, V, device, par, stride, max_depth = _tree_args(target_logits, tree_parent, tree_tokens,
                                                         max_depth)
    if out is None:
        out = _tree_outputs(B, max_depth + 1, device, path, status)
    rc = _native.lib().spec_verify_tree(
        _p(target_logits), _p(par), stride, _p(tree_tokens), _p(out.tokens), _p(out.accept_len),
        _dtype_code(target_logits), B, N, V, max_depth, _p(out.path), _p(out.status),
        _stream(device))
    if rc:
        raise VerifyError(rc)
    return out


def spec_verify_tree_sample(target_logits, tree_parent, tree_tokens, uniforms, temperature,
                            max_depth=None, out: Optional[TreeOutputs] = None, *, path=True,
                            status=True) -> TreeOutputs:
    """Lossless tree verification by rejection sampling (see spec_verify.h):
    tree_parent as for spec_verify_tree, tree_tokens [B, N] int32, uniforms
    [B, N+1] fp32 (column n: node n's test, column 0: the final draw);
    temperature 0 runs the greedy walk."""
    B, N, V, device, par, stride, max_depth = _tree_args(target_logits, tree_parent, tree_tokens,
                                                         max_depth)
    _check(uniforms, "uniforms", device, torch.float32, (B, N + 1))
    if out is None:
        out = _tree_outputs(B, max_depth + 1, device, path, status)
    lib = _native.lib()
    ws = workspace(B, N, V, device, need=int(lib.spec_verify_tree_workspace_size(B, N, V)))
    rc = lib.spec_verify_tree_sample(
        _p(target_logits), _p(par), stride, _p(tree_tokens), _p(uniforms),
        ctypes.c_float(float(temperature)), _p(out.tokens), _p(out.accept_len),
        _dtype_code(target_logits), B, N, V, max_depth, _p(out.path), _p(out.status), _p(ws),
        ws.numel(), _stream(device))
    if rc:
        raise VerifyError(rc)
    return out


def spec_verify_typical(target_logits, draft_tokens, uniforms, temperature, eps=0.09, delta=0.3,
                        out: Optional[VerifyOutputs] = None, *, draft_lens=None, packed=True,
                        accept_prob=True, status=True) -> VerifyOutputs:
    """Typical acceptance (see spec_verify.h): x_i passes while p_i(x_i) >
    min(eps, delta * exp(-H(p_i))); the token after the accepted ones is
    drawn from the target distribution there with uniforms[:, K]."""
    B, K, V, device = _validate_batch(target_logits, draft_tokens, draft_lens)
    _check(uniforms, "uniforms", device, torch.float32, (B, K + 1))
    if out is None:
        out = alloc_outputs(B, K, device, packed=packed, accept_prob=accept_prob, status=status)
    ws = workspace(B, K, V, device)
    rc = _native.lib().spec_verify_typical(
        _p(target_logits), _p(draft_tokens), _p(uniforms), ctypes.c_float(float(temperature)),
        ctypes.c_float(float(eps)), ctypes.c_float(float(delta)), _p(out.tokens),
        _p(out.accept_len), _dtype_code(target_logits), B, K, V, _p(draft_lens), _p(out.cu_accept),
        _p(out.packed), _p(out.batch_id), _p(out.accept_prob), _p(out.status), _p(ws), ws.numel(),
        _stream(device))
    if rc:
        raise VerifyError(rc)
    return out


def spec_verify_tree_typical(target_logits, tree_parent, tree_tokens, uniforms, temperature,
                             eps=0.09, delta=0.3, max_depth=None,
                             out: Optional[TreeOutputs] = None, *, path=True,
                             status=True) -> TreeOutputs:
    """Typical acceptance over a candidate tree: tree_parent as for
    spec_verify_tree, tree_tokens [B, N] int32, uniforms [B] fp32 for the
    final draw."""
    B, N, V, device, par, stride, max_depth = _tree_args(target_logits, tree_parent, tree_tokens,
                                                         max_depth)
    _check(uniforms, "uniforms", device, torch.float32, (B,))
    if out is None:
        out = _tree_outputs(B, max_depth + 1, device, path, status)
    lib = _native.lib()
    ws = workspace(B, N, V, device, need=int(lib.spec_verify_tree_workspace_size(B, N, V)))
    rc = lib.spec_verify_tree_typical(
        _p(target_logits), _p(par), stride, _p(tree_tokens), _p(uniforms),
        ctypes.c_float(float(temperature)), ctypes.c_float(float(eps)),
        ctypes.c_float(float(delta)), _p(out.tokens), _p(out.accept_len),
        _dtype_code(target_logits), B, N, V, max_depth, _p(out.path), _p(out.status),
        _p(ws), ws.numel(), _stream(device))
    if rc:
        raise VerifyError(rc)
    return out


def set_wait_limit_ns(limit_ns: int) -> None:
    """The longest a kernel waits for staged logits before the call reports
    REQ_TIMEOUT (default 2 s; 0 gives up at once).  Process-wide."""
    _native.lib().spec_verify_set_wait_limit_ns(int(limit_ns))


def wait_limit_ns() -> int:
    return int(_native.lib().spec_verify_wait_limit_ns())


@dataclass
class NgramOutputs:
    drafts: torch.Tensor      # [B, K], -1 after the drafts
    draft_lens: torch.Tensor  # [B]
    match: Optional[torch.Tensor] = None
    status: Optional[torch.Tensor] = None


def spec_ngram_propose(tokens, lens, K=5, n_min=1, n_max=4, out: Optional[NgramOutputs] = None,
                       *, match=True, status=True) -> NgramOutputs:
    """n-gram (prompt-lookup) proposer (see spec_verify.h): tokens [B, L]
    int32 contexts, lens [B] int32.  The drafts feed spec_verify_sample as
    one-hot drafts with draft_lens = out.draft_lens."""
    if tokens.dim() != 2:
        raise ValueError("tokens must be [B, L]")
    B, L = tokens.shape
    device = tokens.device
    if device.type != "cuda":
        raise ValueError("tokens must be a CUDA tensor")
    _check(tokens, "tokens", device, torch.int32)
    _check(lens, "lens", device, torch.int32, (B,))
    if out is None:
        i32 = dict(dtype=torch.int32, device=device)
        out = NgramOutputs(drafts=torch.empty((B, K), **i32), draft_lens=torch.empty((B,), **i32),
                           match=torch.empty((B,), **i32) if match else None,
                           status=torch.empty((B,), **i32) if status else None)
    rc = _native.lib().spec_ngram_propose(_p(tokens), _p(lens), B, L, int(n_min), int(n_max),
                                          int(K), _p(out.drafts), _p(out.draft_lens),
                                          _p(out.match), _p(out.status), _stream(device))
    if rc:
        raise VerifyError(rc)
    return out


# ---------------------------------------------------------------------------
# draft training and tree drafting: a teacher's top logits, distillation, beams
# ---------------------------------------------------------------------------

MAX_TOP = 128


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# The current stream's handle without the Stream object around it (2 us of a
# 15 us call), where this PyTorch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _short(answer, make):
    """make(*outputs) of the compiled binding's answer to a plain call."""
    if type(answer) is tuple:
        return make(*answer)
    raise VerifyError(answer)


def _launch(device, fn, *args):
    """fn(*args, stream) on the device's current stream, with the device current."""
    index = device.index
    if torch.cuda.current_device() == index:
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, _raw_stream(index))
    if rc:
        raise VerifyError(rc)


def _need(t, name, device, dtype, shape):
    """_check, quick where nothing is wrong."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.device == device and t.is_contiguous()):
        _check(t, name, device, dtype, shape)


def _rows(logits, name, shape):
    """(dims..., device, dtype code) of a [B, P, V] / [B, W, V] CUDA logit tensor."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 3:
        raise ValueError("%s must be a %s tensor" % (name, shape))
    device = logits.device
    if device.type != "cuda":
        raise ValueError("%s must be a CUDA tensor" % name)
    if not logits.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return (*logits.shape, device, _dtype_code(logits))


def _count(k):
    """A record's or selection's size; refused here, before it sizes an output."""
    k = int(k)
    if not 1 <= k <= MAX_TOP:
        raise VerifyError(2)
    return k


def _written(*tensors):
    """Tell autograd that caller-given tensors were written in place: a backward pass that
    saved one of them then refuses to run on the new contents."""
    for t in tensors:
        if t is not None and not t.is_inference():
            torch.autograd.graph.increment_version(t)


def _given(out, device, **like):
    """Check caller-given output tensors: name -> (dtype, shape), None fields are left out."""
    for name, (dtype, shape) in like.items():
        t = getattr(out, name)
        if t is not None:
            _need(t, "out." + name, device, dtype, shape)


@dataclass
class TopLogits:
    ids: torch.Tensor      # [B, P, k] int32, -1 past the last finite logit
    logits: torch.Tensor   # [B, P, k] fp32, -inf past it
    lse: torch.Tensor      # [B, P] fp32
    status: Optional[torch.Tensor] = None  # [B, P]


def spec_top_logits(logits, k, temperature=1.0, out: Optional[TopLogits] = None, *, lens=None,
                    status=True) -> TopLogits:
    """The k largest logits of each row and its log-sum-exp (see
    spec_verify.h): logits [B, P, V] bf16/fp32 CUDA, 1 <= k <= 128, temperature
    > 0 (of the log-sum-exp), lens [B] int32 or None (rows i >= lens[b] are not
    read: pass accept_len to record a verify call's accepted positions)."""
    if out is None:
        r = _native.binding().top_logits(logits, k, temperature, lens, bool(status))
        if r is not None:
            return _short(r, TopLogits)
    B, P, V, device, code = _rows(logits, "logits", "[B, P, V]")
    k = _count(k)
    given = out is not None
    if lens is not None:
        _need(lens, "lens", device, torch.int32, (B,))
    if not given:
        shape = (B, P, k)
        out = TopLogits(torch.empty(shape, dtype=torch.int32, device=device),
                        torch.empty(shape, dtype=torch.float32, device=device),
                        torch.empty((B, P), dtype=torch.float32, device=device),
                        torch.empty((B, P), dtype=torch.int32, device=device) if status else None)
    else:
        _given(out, device, ids=(torch.int32, (B, P, k)), logits=(torch.float32, (B, P, k)),
               lse=(torch.float32, (B, P)), status=(torch.int32, (B, P)))
    _launch(device, _native.lib().spec_top_logits, logits.data_ptr(), k, float(temperature),
            _addr(lens), out.ids.data_ptr(), out.logits.data_ptr(), out.lse.data_ptr(),
            _addr(out.status), code, B, P, V)
    if given:
        _written(out.ids, out.logits, out.lse, out.status)
    return out


@dataclass
class DistillOutputs:
    loss: torch.Tensor                     # [B, P] fp32
    stats: Optional[torch.Tensor] = None   # [B, P, 4] fp32, for spec_distill_grad
    grad: Optional[torch.Tensor] = None    # [B, P, V]
    status: Optional[torch.Tensor] = None  # [B, P]


def _distill_args(student_logits, top_ids, top_logits, top_lse, lens, grad_loss):
    B, P, V, device, code = _rows(student_logits, "student_logits", "[B, P, V]")
    if not isinstance(top_ids, torch.Tensor) or top_ids.dim() != 3:
        raise ValueError("top_ids must be a [B, P, k] tensor")
    k = top_ids.shape[2]
    _need(top_ids, "top_ids", device, torch.int32, (B, P, k))
    _need(top_logits, "top_logits", device, torch.float32, (B, P, k))
    if top_lse is not None:
        _need(top_lse, "top_lse", device, torch.float32, (B, P))
    if lens is not None:
        _need(lens, "lens", device, torch.int32, (B,))
    if grad_loss is not None:
        _need(grad_loss, "grad_loss", device, torch.float32, (B, P))
    return B, P, V, k, device, code


def spec_distill(student_logits, top_ids, top_logits, temperature=1.0,
                 out: Optional[DistillOutputs] = None, *, top_lse=None, lens=None, grad_loss=None,
                 stats=True, status=True) -> DistillOutputs:
    """The distillation loss of each row from a teacher's top logits (see
    spec_verify.h): student_logits [B, P, V] bf16/fp32 CUDA; top_ids,
    top_logits [B, P, k] and top_lse [B, P] as spec_top_logits returns them
    (top_lse None: the teacher renormalised over its record); lens [B] int32
    or None.  With grad_loss [B, P] fp32 the same pass also writes out.grad,
    the gradient of (grad_loss * loss).sum() in the student's type, for
    ``student_logits.backward(out.grad)``; out.grad may be student_logits (an
    operation that saved those logits for its own backward pass then refuses it,
    as after any write in place)."""
    if out is None:
        r = _native.binding().distill(student_logits, top_ids, top_logits, temperature, top_lse,
                                      lens, grad_loss, bool(stats), bool(status))
        if r is not None:
            return _short(r, DistillOutputs)
    B, P, V, k, device, code = _distill_args(student_logits, top_ids, top_logits, top_lse, lens,
                                             grad_loss)
    given = out is not None
    if not given:
        f32 = torch.float32
        out = DistillOutputs(
            torch.empty((B, P), dtype=f32, device=device),
            torch.empty((B, P, 4), dtype=f32, device=device) if stats else None,
            torch.empty((B, P, V), dtype=student_logits.dtype, device=device)
            if grad_loss is not None else None,
            torch.empty((B, P), dtype=torch.int32, device=device) if status else None)
    else:
        _given(out, device, loss=(torch.float32, (B, P)), stats=(torch.float32, (B, P, 4)),
               grad=(student_logits.dtype, (B, P, V)), status=(torch.int32, (B, P)))
    _launch(device, _native.lib().spec_distill, student_logits.data_ptr(), top_ids.data_ptr(),
            top_logits.data_ptr(), _addr(top_lse), _addr(lens), _addr(grad_loss),
            float(temperature), out.loss.data_ptr(), _addr(out.stats),
            _addr(out.grad) if grad_loss is not None else None, _addr(out.status),
            code, B, P, V, k)
    if given:
        _written(out.loss, out.stats, out.grad if grad_loss is not None else None, out.status)
    return out


def spec_distill_grad(student_logits, top_ids, top_logits, temperature, stats, grad_loss,
                      grad=None, *, top_lse=None, lens=None) -> torch.Tensor:
    """The backward pass alone: the gradient of (grad_loss * loss).sum() by
    student_logits, from the stats of a spec_distill call on the same inputs.
    grad: the tensor to write ([B, P, V], the student's type; student_logits
    itself is allowed), or None for a new one."""
    if grad is None:
        r = _native.binding().distill_grad(student_logits, top_ids, top_logits, temperature,
                                           stats, grad_loss, top_lse, lens)
        if r is not None:
            return _short(r, lambda g: g)
    if grad_loss is None or stats is None:
        raise ValueError("stats and grad_loss are required")
    B, P, V, k, device, code = _distill_args(student_logits, top_ids, top_logits, top_lse, lens,
                                             grad_loss)
    _need(stats, "stats", device, torch.float32, (B, P, 4))
    given = grad is not None
    if not given:
        grad = torch.empty((B, P, V), dtype=student_logits.dtype, device=device)
    else:
        _need(grad, "grad", device, student_logits.dtype, (B, P, V))
    _launch(device, _native.lib().spec_distill_grad, student_logits.data_ptr(),
            top_ids.data_ptr(), top_logits.data_ptr(), _addr(top_lse), _addr(lens),
            stats.data_ptr(), grad_loss.data_ptr(), float(temperature), grad.data_ptr(),
            code, B, P, V, k)
    if given:
        _written(grad)
    return grad


@dataclass
class BeamOutputs:
    tokens: torch.Tensor   # [B, n] int32, -1 past the last candidate
    parents: torch.Tensor  # [B, n] int32, the beam of each
    scores: torch.Tensor   # [B, n] fp32, descending
    status: Optional[torch.Tensor] = None  # [B]


def spec_beam_select(logits, scores, n, out: Optional[BeamOutputs] = None, *,
                     status=True) -> BeamOutputs:
    """One step of beam selection (see spec_verify.h): logits [B, W, V]
    bf16/fp32 CUDA, scores [B, W] fp32 (-inf: a finished beam, not read); the
    n best continuations by scores + log_softmax(logits), best first (equal scores
    by beam, in a beam by logit, then by token)."""
    if out is None:
        r = _native.binding().beam_select(logits, scores, n, bool(status))
        if r is not None:
            return _short(r, BeamOutputs)
    B, W, V, device, code = _rows(logits, "logits", "[B, W, V]")
    n = _count(n)
    _need(scores, "scores", device, torch.float32, (B, W))
    given = out is not None
    if not given:
        shape = (B, n)
        out = BeamOutputs(torch.empty(shape, dtype=torch.int32, device=device),
                          torch.empty(shape, dtype=torch.int32, device=device),
                          torch.empty(shape, dtype=torch.float32, device=device),
                          torch.empty((B,), dtype=torch.int32, device=device) if status else None)
    else:
        _given(out, device, tokens=(torch.int32, (B, n)), parents=(torch.int32, (B, n)),
               scores=(torch.float32, (B, n)), status=(torch.int32, (B,)))
    lib = _native.lib()
    need = lib.spec_beam_workspace_size(code, B, W, V, n)
    # scratch of this call alone (stream-ordered, and a captured graph's own)
    ws = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _launch(device, lib.spec_beam_select, logits.data_ptr(), scores.data_ptr(),
            out.tokens.data_ptr(), out.parents.data_ptr(), out.scores.data_ptr(),
            _addr(out.status), code, B, W, V, n, _addr(ws), need)
    if given:
        _written(out.tokens, out.parents, out.scores, out.status)
    return out


_Strides = ctypes.c_int64 * 5


def spec_beam_reorder(state, parents, out=None, *, lens=None, status=None) -> torch.Tensor:
    """Move per-beam states along a selection's parents (see spec_verify.h):
    out[g, b, w, h, l] = state[g, b, parents[b, w], h, l] for l < lens[b].

    state [G, B, W, H, L, D] CUDA of any type, the last dimension contiguous,
    the others at any strides (a permuted view of a cache is fine; a dimension
    the state does not have is 1); parents [B, W_out] int32 (-1 leaves a slot as
    it is); lens [B] int32 or None; out [G, B, W_out, H, L, D] of the same
    type (None: a new tensor of zeros; no entry of it may overlap one of the
    state's, interleaved parts of one cache are fine); status: an int32 [B]
    tensor to receive the request status, or None."""
    if out is not None and status is None:
        r = _native.binding().beam_reorder(state, parents, out, lens)
        if r is not None:
            if r:
                raise VerifyError(r)
            return out
    if not isinstance(state, torch.Tensor) or state.dim() != 6:
        raise ValueError("state must be a [G, B, W, H, L, D] tensor")
    device = state.device
    if device.type != "cuda":
        raise ValueError("state must be a CUDA tensor")
    G, B, W, H, L, D = state.shape
    if not isinstance(parents, torch.Tensor) or parents.dim() != 2:
        raise ValueError("parents must be a [B, W_out] tensor")
    W_out = parents.shape[1]
    _need(parents, "parents", device, torch.int32, (B, W_out))
    if lens is not None:
        _need(lens, "lens", device, torch.int32, (B,))
    if status is not None:
        _need(status, "status", device, torch.int32, (B,))
    shape = (G, B, W_out, H, L, D)
    given = out is not None
    if not given:
        out = torch.zeros(shape, dtype=state.dtype, device=device)
    elif not isinstance(out, torch.Tensor) or out.device != device:
        raise ValueError("out must be a tensor on %s" % device)
    elif out.dtype != state.dtype:
        raise TypeError("out must be %s (got %s)" % (state.dtype, out.dtype))
    elif out.shape != shape:
        raise ValueError("out must have shape %s (got %s)" % (shape, tuple(out.shape)))
    if D == 0:
        raise ValueError("state must have entries of at least one element")
    size = state.element_size()
    a0, a1, a2, a3, a4, a5 = state.stride()
    b0, b1, b2, b3, b4, b5 = out.stride()
    if D > 1 and (a5 != 1 or b5 != 1):
        raise ValueError("the last dimension of %s must be contiguous"
                         % ("state" if a5 != 1 else "out"))
    _launch(device, _native.lib().spec_beam_reorder, state.data_ptr(),
            _Strides(a0 * size, a1 * size, a2 * size, a3 * size, a4 * size), _addr(parents),
            _addr(lens), out.data_ptr(),
            _Strides(b0 * size, b1 * size, b2 * size, b3 * size, b4 * size), _addr(status), G, B,
            W, W_out, H, L, D * size)
    _written(out if given else None, status)
    return out
