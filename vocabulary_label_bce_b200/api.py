"""torch-facing calls of the fused large-vocabulary BCE (device tensors in, device tensors out).

PyTorch supplies device memory and the current stream; all arithmetic runs in
libcutbce's kernels (see include/cutbce.h).
"""
from __future__ import annotations

import functools
import inspect
from typing import Optional

import torch

from . import binding as B

__all__ = ["forward", "backward", "forward_backward", "cut_bce", "Workspace", "embed", "embed_forward",
           "embed_backward", "distill_loss", "distill_forward", "distill_backward", "distill_forward_backward",
           "preference_loss", "preference_forward", "preference_backward", "preference_forward_backward"]


class Workspace:
    """Caches one device workspace per (device, size); grows on demand."""

    def __init__(self):
        self._buf: dict[int, torch.Tensor] = {}

    def get(self, nbytes: int, device: torch.device) -> torch.Tensor:
        idx = device.index if device.index is not None else torch.cuda.current_device()
        buf = self._buf.get(idx)
        if buf is None or buf.numel() < nbytes:
            buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
            self._buf[idx] = buf
        return buf


_WS = Workspace()


def _mask_u8(mask: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    if mask is None:
        return None
    return mask.to(torch.uint8).contiguous() if mask.dtype != torch.uint8 else mask.contiguous()


def _flat(H, targets, mask):
    # [B, N, D] activations and [B, N, L] ids are flattened to T = B*N rows
    if H.dim() == 3:
        H = H.reshape(-1, H.shape[-1])
    if targets.dim() == 3:
        targets = targets.reshape(-1, targets.shape[-1])
    if mask is not None and mask.dim() == 2:
        mask = mask.reshape(-1)
    return H.contiguous(), targets.to(torch.int32).contiguous(), _mask_u8(mask)


def forward_backward(H: torch.Tensor, E: torch.Tensor, targets: torch.Tensor, mask: Optional[torch.Tensor] = None,
                     reduction: str = "mean", grad_loss: Optional[torch.Tensor] = None, want_loss: bool = True,
                     want_dH: bool = True, want_dE: bool = True, workspace: Optional[torch.Tensor] = None):
    """Loss (0-d float64) and gradients dH [T, D], dE [V, D] (float32); None for what was not asked."""
    H2, tg, m = _flat(H, targets, mask)
    E = E.contiguous()
    prob = B.make_problem(H2, E, tg, m, reduction)
    outs = (B.OUT_LOSS if want_loss else 0) | (B.OUT_DH if want_dH else 0) | (B.OUT_DE if want_dE else 0)
    ws = workspace if workspace is not None else _WS.get(B.cutbce_workspace_size_for(prob, outs), H2.device)
    loss = torch.empty((), dtype=torch.float64, device=H2.device) if want_loss else None
    dH = torch.empty(H2.shape, dtype=torch.float32, device=H2.device) if want_dH else None
    dE = torch.empty(E.shape, dtype=torch.float32, device=E.device) if want_dE else None
    g = grad_loss.to(torch.float32).reshape(()) if grad_loss is not None else None
    B.cutbce_forward_backward(prob, g, loss, dH, dE, ws)
    if dH is not None and H.dim() == 3:
        dH = dH.reshape(H.shape)
    return loss, dH, dE


def forward(H, E, targets, mask=None, reduction: str = "mean", workspace=None) -> torch.Tensor:
    H2, tg, m = _flat(H, targets, mask)
    E = E.contiguous()
    prob = B.make_problem(H2, E, tg, m, reduction)
    ws = workspace if workspace is not None else _WS.get(B.cutbce_workspace_size_for(prob, B.OUT_LOSS), H2.device)
    loss = torch.empty((), dtype=torch.float64, device=H2.device)
    B.cutbce_forward(prob, ws, loss)
    return loss


def backward(H, E, targets, mask=None, reduction: str = "mean", grad_loss=None, want_dH=True, want_dE=True,
             workspace=None):
    H2, tg, m = _flat(H, targets, mask)
    E = E.contiguous()
    prob = B.make_problem(H2, E, tg, m, reduction)
    outs = (B.OUT_DH if want_dH else 0) | (B.OUT_DE if want_dE else 0)
    ws = workspace if workspace is not None else _WS.get(B.cutbce_workspace_size_for(prob, outs), H2.device)
    dH = torch.empty(H2.shape, dtype=torch.float32, device=H2.device) if want_dH else None
    dE = torch.empty(E.shape, dtype=torch.float32, device=E.device) if want_dE else None
    g = grad_loss.to(torch.float32).reshape(()) if grad_loss is not None else None
    B.cutbce_backward(prob, g, dH, dE, ws)
    if dH is not None and H.dim() == 3:
        dH = dH.reshape(H.shape)
    return dH, dE


class _CutBCE(torch.autograd.Function):
    """Custom VJP in the paper's sense (section III-B): the forward keeps only H, E and
    the sparse ids; the backward recomputes every logit tile on chip."""

    @staticmethod
    def forward(ctx, H, E, targets, mask, reduction):
        ctx.save_for_backward(H, E, targets, mask if mask is not None else torch.empty(0))
        ctx.has_mask = mask is not None
        ctx.reduction = reduction
        return forward(H.detach(), E.detach(), targets, mask, reduction).to(torch.float32)

    @staticmethod
    def backward(ctx, grad):
        H, E, targets, mask = ctx.saved_tensors
        m = mask if ctx.has_mask else None
        dH, dE = backward(H.detach(), E.detach(), targets, m, ctx.reduction, grad_loss=grad,
                          want_dH=ctx.needs_input_grad[0], want_dE=ctx.needs_input_grad[1])
        dH = dH.to(H.dtype) if dH is not None else None
        dE = dE.to(E.dtype) if dE is not None else None
        return dH, dE, None, None, None


def cut_bce(H, E, targets, mask=None, reduction: str = "mean") -> torch.Tensor:
    """Differentiable fused BCE loss over the full vocabulary (autograd-aware)."""
    return _CutBCE.apply(H, E, targets, mask, reduction)


# ---------------------------------------------------------------- item rows and softmax losses
# These calls run on the device of their tensors and on that device's current
# stream, and take their workspace from torch's caching allocator per call, so
# calls on several streams, and captured graphs, never share one.

_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on_cuda(t: torch.Tensor) -> None:
    if not t.is_cuda:
        raise ValueError(f"tensors must be on a CUDA device, not {t.device}")


def _there(call):
    """The call, made on the device of its first tensor."""
    name = next(iter(inspect.signature(call).parameters))

    @functools.wraps(call)
    def wrapped(*args, **kw):
        first = args[0] if args else kw.get(name)
        if first is not None and first.is_cuda and first.get_device() != _current_device():
            with torch.cuda.device(first.device):
                return call(*args, **kw)
        return call(*args, **kw)
    return wrapped


def _plain(t: torch.Tensor) -> torch.Tensor:
    """t without its graph, contiguous."""
    return (t.detach() if t.requires_grad else t).contiguous()


def _ids32(ids: torch.Tensor, name: str = "ids") -> torch.Tensor:
    if ids.dtype == torch.int32:
        return ids.contiguous()
    if ids.dtype not in (torch.int64, torch.int16, torch.int8, torch.uint8):
        raise ValueError(f"{name} must be integers, not {ids.dtype}")
    if ids.dtype == torch.int64:
        ids = ids.clamp(-2, 2 ** 31 - 1)          # a far value stays out of range instead of wrapping
    return ids.to(torch.int32).contiguous()


def _counts(mask: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """The mask as the library takes it; one of another type counts where it is not zero."""
    return mask if mask is None or mask.dtype in (torch.uint8, torch.bool) else mask != 0


def _scalar_grad(g: Optional[torch.Tensor], like: torch.Tensor) -> Optional[torch.Tensor]:
    if g is None:
        return None
    if g.device != like.device or g.numel() != 1:
        raise ValueError("grad_loss must be one value on the device of H")
    return _as(g.detach(), torch.float32).reshape(())


def _as(t: Optional[torch.Tensor], dtype: torch.dtype) -> Optional[torch.Tensor]:
    return t if t is None or t.dtype == dtype else t.to(dtype)


def _workspace(nbytes: int, like: torch.Tensor, given: Optional[torch.Tensor]) -> torch.Tensor:
    if given is None:
        return like.new_empty(nbytes, dtype=torch.uint8)
    if given.dtype != torch.uint8 or given.device != like.device or not given.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the device of the inputs")
    return given


def embed_forward(E: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, status: Optional[torch.Tensor] = None):
    """scale * E[ids] (any shape of ids; -1 gives a zero row), in E's dtype (bf16 or fp32).

    An id out of range gives a zero row too, and sets `status` (an int32 tensor of one value) if there is one."""
    _on_cuda(E)
    if E.get_device() != _current_device():
        with torch.cuda.device(E.device):
            return embed_forward(E, ids, scale, status)
    if E.dim() != 2:
        raise ValueError("E must be [V, D]")
    E, ids = _plain(E), _ids32(ids)
    # (a tuple of two numbers is the quickest way to an uninitialised tensor)
    X = E.new_empty((ids.shape[0], E.shape[1]) if ids.dim() == 1 else ids.shape + E.shape[1:])
    if ids.numel() > 0:
        B.cutbce_embed_forward(E, ids, X, scale, status)
    return X


@_there
def embed_backward(dX: torch.Tensor, ids: torch.Tensor, V: int, scale: float = 1.0,
                   grad_dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
                   accumulate: bool = False, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dE [V, D] of embed_forward: dE[v] = scale * sum of dX over the entries with id v.

    `out` (contiguous, [V, D]) is written instead of a new tensor; with accumulate the
    sums are added to it and rows without an entry keep their value.  An id out of range adds
    nothing and sets the status of the workspace (binding.cutbce_read_status)."""
    D = dX.shape[-1]
    if dX.shape[:-1] != ids.shape:
        raise ValueError("dX must be ids.shape + [D]")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if out is not None and tuple(out.shape) != (V, D):
        raise ValueError(f"out must be [{V}, {D}]")
    _on_cuda(dX)
    if ids.numel() == 0:
        if out is None:
            return torch.zeros((V, D), dtype=grad_dtype, device=dX.device)
        return out if accumulate else out.zero_()
    dE = out if out is not None else dX.new_empty((V, D), dtype=grad_dtype)
    ws = _workspace(B.cutbce_embed_workspace_size(ids.numel(), V, D), dX, workspace)
    B.cutbce_embed_backward(_plain(dX).view(-1, D), _ids32(ids), dE, ws, scale, accumulate)
    return dE


class _Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, E, ids, scale, status):
        ids = _ids32(ids)
        ctx.save_for_backward(ids)
        ctx.shape, ctx.dtype, ctx.scale = E.shape, E.dtype, scale
        return embed_forward(E, ids, scale, status)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dX):
        (ids,) = ctx.saved_tensors
        return embed_backward(dX, ids, ctx.shape[0], ctx.scale, grad_dtype=ctx.dtype), None, None, None


def _hold_leaves(*tensors):
    """The gradient nodes of the leaves among `tensors`, each marked with the stream it was made on.

    torch keeps a leaf's gradient node, with its stream, while any autograd graph of the leaf lives.
    A backward pass that is captured into a CUDA graph while an eager graph on another stream lives
    would wait across streams and break the capture at its end: it is refused here, at its forward."""
    if not torch.is_grad_enabled():
        return None
    held = []
    for t in tensors:
        if t.requires_grad and t.is_leaf and t.device.type == "cuda":
            node = torch.autograd.graph.get_gradient_edge(t).node
            here = torch.cuda.current_stream(t.device).cuda_stream
            if node.metadata.setdefault("cutbce_stream", here) != here and torch.cuda.is_current_stream_capturing():
                raise RuntimeError("a tensor of this call is also held by an autograd graph that was made on another "
                                   "stream: drop that graph (its loss), or make it on the stream that is captured")
            held.append(node)
    return held


def embed(E: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Differentiable embed_forward; the gradient with respect to E is dense, in E's dtype."""
    held = _hold_leaves(E)  # noqa: F841  (alive until the graph holds them)
    return _Embed.apply(E, ids, float(scale), status)


def _rows(H: torch.Tensor, *rest: Optional[torch.Tensor]):
    """H [.., D] and per-position tensors flattened to T rows."""
    lead = H.dim() - 1
    size = H.shape[:lead]
    for t in rest:
        if t is not None and t.shape[:lead] != size:
            raise ValueError(f"leading sizes {tuple(t.shape[:lead])} and {tuple(size)} do not fit")
    if lead == 1:
        return [_plain(H)] + [None if t is None else _plain(t) for t in rest]
    return [_plain(H).view(-1, H.shape[-1])] + [None if t is None else _plain(t).view((-1,) + t.shape[lead:]) for t in rest]


def _distill_problem(H, E, ids, logits, mask, weights, temperature, reduction):
    """The problem and the tensors it points to (to be kept until the launch)."""
    _on_cuda(H)
    if logits.shape != ids.shape:
        raise ValueError("teacher ids and logits must have one shape")
    H2, ids2, lg, m, w = _rows(H, _ids32(ids), _as(logits, torch.float32), _counts(mask), _as(weights, torch.float32))
    E2 = _plain(E)
    keep = (H2, E2, ids2, lg, m, w)
    return B.make_distill_problem(H2, E2, ids2, lg, m, w, temperature, reduction), keep


def _preference_problem(H, E, ids, offsets, ref_logp, mask, beta, reduction):
    _on_cuda(H)
    H2, ids2, m = _rows(H, _ids32(ids), _counts(mask))
    if offsets is None:
        if H.dim() != 3:
            raise ValueError("without offsets H must be [2P, N, D]")
        offsets = torch.arange(0, H2.shape[0] + 1, H.shape[1], dtype=torch.int32, device=H.device)
    E2 = _plain(E)
    off = _ids32(offsets, "offsets")
    ref = None if ref_logp is None else _as(_plain(ref_logp), torch.float32).view(-1)
    keep = (H2, E2, ids2, off, ref, m)
    return B.make_preference_problem(H2, E2, ids2, off, ref, m, beta, reduction), keep


def _grad_outputs(H, E, want_dH, want_dE, grad_dtype, dE_out, accumulate_dE):
    if accumulate_dE and dE_out is None:
        raise ValueError("accumulate_dE needs dE_out")
    if dE_out is not None and tuple(dE_out.shape) != tuple(E.shape):
        raise ValueError("dE_out must have E's shape")
    if not want_dH and not want_dE:
        raise ValueError("neither gradient is wanted")
    B._same_device(H, dE_out)
    dH = torch.empty(H.shape, dtype=grad_dtype, device=H.device) if want_dH else None
    dE = None
    if want_dE:
        dE = dE_out if dE_out is not None else torch.empty(E.shape, dtype=grad_dtype, device=E.device)
    return dH, dE, B.make_grad_options(dH, dE, B.ACCUMULATE_DE if accumulate_dE else 0)


def _bits(dH, dE) -> int:
    return (B.OUT_DH if dH is not None else 0) | (B.OUT_DE if dE is not None else 0)


def _loss_lse(H):
    """Uninitialised loss (0-d float64) and log-sum-exps (float32, H.shape[:-1])."""
    lse = H.new_empty(H.shape[0] if H.dim() == 2 else H.shape[:-1], dtype=torch.float32)
    return H.new_empty((), dtype=torch.float64), lse


def _lse_rows(lse: torch.Tensor, H: torch.Tensor) -> torch.Tensor:
    if lse.dtype != torch.float32 or lse.shape != H.shape[:-1] or lse.device != H.device:
        raise ValueError("lse must be the float32 tensor of a forward on the same inputs")
    return lse.contiguous()


@_there
def distill_forward(H, E, teacher_ids, teacher_logits, mask=None, weights=None, temperature: float = 1.0,
                    reduction: str = "mean", workspace: Optional[torch.Tensor] = None):
    """Distillation loss (0-d float64) and the rows' log-sum-exps of z / temperature (float32, H.shape[:-1]).

    H [T, D] or [B, N, D] and E [V, D] bf16; teacher_ids [.., K] (-1 empty) and teacher_logits [.., K]
    the teacher's top items and logits of each position; mask: not 0 = counts; weights a factor per position."""
    prob, keep = _distill_problem(H, E, teacher_ids, teacher_logits, mask, weights, temperature, reduction)
    ws = _workspace(B.cutbce_distill_workspace_size(prob, B.OUT_LOSS), H, workspace)
    loss, lse = _loss_lse(H)
    B.cutbce_distill_forward(prob, loss, lse, ws)
    return loss, lse


@_there
def distill_backward(H, E, teacher_ids, teacher_logits, lse, mask=None, weights=None, temperature: float = 1.0,
                     reduction: str = "mean", grad_loss=None, want_dH: bool = True, want_dE: bool = True,
                     grad_dtype: torch.dtype = torch.float32, dE_out=None, accumulate_dE: bool = False,
                     workspace: Optional[torch.Tensor] = None):
    """(dH, dE) given the lse of distill_forward on the same inputs."""
    prob, keep = _distill_problem(H, E, teacher_ids, teacher_logits, mask, weights, temperature, reduction)
    dH, dE, opts = _grad_outputs(H, E, want_dH, want_dE, grad_dtype, dE_out, accumulate_dE)
    ws = _workspace(B.cutbce_distill_workspace_size(prob, _bits(dH, dE)), H, workspace)
    g = _scalar_grad(grad_loss, H)
    B.cutbce_distill_backward(prob, opts, _lse_rows(lse, H), g, dH, dE, ws)
    return dH, dE


@_there
def distill_forward_backward(H, E, teacher_ids, teacher_logits, mask=None, weights=None, temperature: float = 1.0,
                             reduction: str = "mean", grad_loss=None, want_dH: bool = True, want_dE: bool = True,
                             grad_dtype: torch.dtype = torch.float32, dE_out=None, accumulate_dE: bool = False,
                             workspace: Optional[torch.Tensor] = None):
    """(loss, lse, dH, dE) in one call; None for a gradient that is not wanted.

    dE_out ([V, D], contiguous) is written instead of a new tensor, or added to with accumulate_dE."""
    prob, keep = _distill_problem(H, E, teacher_ids, teacher_logits, mask, weights, temperature, reduction)
    dH, dE, opts = _grad_outputs(H, E, want_dH, want_dE, grad_dtype, dE_out, accumulate_dE)
    ws = _workspace(B.cutbce_distill_workspace_size(prob, B.OUT_LOSS | _bits(dH, dE)), H, workspace)
    loss, lse = _loss_lse(H)
    g = _scalar_grad(grad_loss, H)
    B.cutbce_distill_forward_backward(prob, opts, g, loss, lse, dH, dE, ws)
    return loss, lse, dH, dE


@_there
def preference_forward(H, E, ids, offsets=None, ref_logp=None, mask=None, beta: float = 0.1, reduction: str = "mean",
                       workspace: Optional[torch.Tensor] = None):
    """Preference loss (0-d float64), the sequences' log-probabilities (float32 [2P]) and the rows'
    log-sum-exps (float32).

    H [T, D] with offsets [2P + 1] of the packed sequences (2p chosen, 2p + 1 rejected), or H [2P, N, D]
    without; ids: the item that followed each position (-1: does not count); ref_logp [2P]: the
    sequences' log-probabilities under the reference model (the second output of this call with
    that model's H and E), or None for 0."""
    prob, keep = _preference_problem(H, E, ids, offsets, ref_logp, mask, beta, reduction)
    ws = _workspace(B.cutbce_preference_workspace_size(prob, B.OUT_LOSS), H, workspace)
    loss, lse = _loss_lse(H)
    logp = H.new_empty(2 * prob.P, dtype=torch.float32)
    B.cutbce_preference_forward(prob, loss, logp, lse, ws)
    return loss, logp, lse


@_there
def preference_backward(H, E, ids, lse, offsets=None, ref_logp=None, mask=None, beta: float = 0.1,
                        reduction: str = "mean", grad_loss=None, want_dH: bool = True, want_dE: bool = True,
                        grad_dtype: torch.dtype = torch.float32, dE_out=None, accumulate_dE: bool = False,
                        workspace: Optional[torch.Tensor] = None):
    """(dH, dE) given the lse of preference_forward on the same inputs."""
    prob, keep = _preference_problem(H, E, ids, offsets, ref_logp, mask, beta, reduction)
    dH, dE, opts = _grad_outputs(H, E, want_dH, want_dE, grad_dtype, dE_out, accumulate_dE)
    ws = _workspace(B.cutbce_preference_workspace_size(prob, _bits(dH, dE)), H, workspace)
    g = _scalar_grad(grad_loss, H)
    B.cutbce_preference_backward(prob, opts, _lse_rows(lse, H), g, dH, dE, ws)
    return dH, dE


@_there
def preference_forward_backward(H, E, ids, offsets=None, ref_logp=None, mask=None, beta: float = 0.1,
                                reduction: str = "mean", grad_loss=None, want_dH: bool = True, want_dE: bool = True,
                                grad_dtype: torch.dtype = torch.float32, dE_out=None, accumulate_dE: bool = False,
                                workspace: Optional[torch.Tensor] = None):
    """(loss, logp, lse, dH, dE) in one call; None for a gradient that is not wanted."""
    prob, keep = _preference_problem(H, E, ids, offsets, ref_logp, mask, beta, reduction)
    dH, dE, opts = _grad_outputs(H, E, want_dH, want_dE, grad_dtype, dE_out, accumulate_dE)
    ws = _workspace(B.cutbce_preference_workspace_size(prob, B.OUT_LOSS | _bits(dH, dE)), H, workspace)
    loss, lse = _loss_lse(H)
    logp = H.new_empty(2 * prob.P, dtype=torch.float32)
    g = _scalar_grad(grad_loss, H)
    B.cutbce_preference_forward_backward(prob, opts, g, loss, logp, lse, dH, dE, ws)
    return loss, logp, lse, dH, dE


def _no_grad_for(**tensors):
    for name, t in tensors.items():
        if t is not None and t.requires_grad:
            raise ValueError(f"{name} gets no gradient: detach it")


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, E, ids, logits, mask, weights, temperature, reduction):
        loss, lse = distill_forward(H, E, ids, logits, mask, weights, temperature, reduction)
        ctx.save_for_backward(H, E, ids, logits, mask, weights, lse)
        ctx.args = temperature, reduction
        return loss.to(torch.float32)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        H, E, ids, logits, mask, weights, lse = ctx.saved_tensors
        dH, dE = distill_backward(H, E, ids, logits, lse, mask, weights, *ctx.args, grad_loss=grad,
                                  want_dH=ctx.needs_input_grad[0], want_dE=ctx.needs_input_grad[1], grad_dtype=H.dtype)
        return dH, dE, None, None, None, None, None, None


def distill_loss(H, E, teacher_ids, teacher_logits, mask=None, weights=None, temperature: float = 1.0,
                 reduction: str = "mean") -> torch.Tensor:
    """Differentiable distillation loss (float32); gradients with respect to H and E, in bf16."""
    _no_grad_for(teacher_logits=teacher_logits, weights=weights)
    held = _hold_leaves(H, E)  # noqa: F841
    return _Distill.apply(H, E, teacher_ids, teacher_logits, mask, weights, float(temperature), reduction)


class _Preference(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, E, ids, offsets, ref_logp, mask, beta, reduction):
        loss, logp, lse = preference_forward(H, E, ids, offsets, ref_logp, mask, beta, reduction)
        ctx.save_for_backward(H, E, ids, offsets, ref_logp, mask, lse)
        ctx.args = beta, reduction
        ctx.mark_non_differentiable(logp)
        return loss.to(torch.float32), logp

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, _):
        H, E, ids, offsets, ref_logp, mask, lse = ctx.saved_tensors
        dH, dE = preference_backward(H, E, ids, lse, offsets, ref_logp, mask, *ctx.args, grad_loss=grad,
                                     want_dH=ctx.needs_input_grad[0], want_dE=ctx.needs_input_grad[1],
                                     grad_dtype=H.dtype)
        return dH, dE, None, None, None, None, None, None


def preference_loss(H, E, ids, offsets=None, ref_logp=None, mask=None, beta: float = 0.1, reduction: str = "mean"):
    """Differentiable preference loss (float32) and the sequences' log-probabilities (float32 [2P],
    not differentiable); gradients with respect to H and E, in bf16."""
    _no_grad_for(ref_logp=ref_logp)
    held = _hold_leaves(H, E)  # noqa: F841
    return _Preference.apply(H, E, ids, offsets, ref_logp, mask, float(beta), reduction)
