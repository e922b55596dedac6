"""The router's training operators: the losses on the router's logits and the
backward passes of route() and combine() (include/moe_training.h).

The same thin binding as the package's other functions: tensors are checked,
outputs allocated unless given, and raw pointers and the current HIP stream
forwarded. The functions take and give gradients themselves; nothing is
registered with autograd.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import MOE_DTYPE_BF16, MOE_DTYPE_F32, _BF16, _check, _need, _ptr, _stream, lib

MOE_SCORE_SIGMOID = 0
MOE_SCORE_SOFTMAX = 1

try:
    _current_device = torch._C._cuda_getDevice
except AttributeError:   # older torch: the public query (slower)
    _current_device = torch.cuda.current_device

_F32 = (torch.float32,)
_I32 = (torch.int32,)
_MASK = (torch.uint8, torch.bool)


def _new(shape, dtype, dev):
    # empty_strided is torch's cheapest allocation (1.2 us against 1.6 for empty)
    strides = (1,) if len(shape) == 1 else (shape[1], 1)
    return torch.empty_strided(shape, strides, dtype=dtype, device=dev)


def _out(t, name, dtype, shape, dev):
    """An output: the caller's, checked, or a new one."""
    if t is None:
        return _new(shape, dtype, dev)
    _need(t, name, _BF16 if dtype == torch.bfloat16 else (dtype,), shape, dev)
    return t


def _scratch(workspace, nbytes, dev):
    """The workspace's pointer and length; a new one where none is given."""
    if workspace is None:
        if nbytes == 0:
            return None, None, 0
        workspace = _new((nbytes,), torch.uint8, dev)
    elif not workspace.is_cuda or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % dev)
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _call(fn, dev, *args):
    """The library call on dev and its current stream. The library launches on
    the current device, so another one is made current for the call."""
    if dev.index == _current_device():
        _check(fn, getattr(lib(), fn)(*args, _stream(dev)))
        return
    with torch.cuda.device(dev):
        _check(fn, getattr(lib(), fn)(*args, _stream(dev)))


def _table(logits, token_mask):
    """Checks [T,E] logits and their mask; returns (device, T, E)."""
    dev = logits.device
    _need(logits, "logits", _F32, None, dev)
    if logits.dim() != 2:
        raise ValueError("logits must be [T,E]")
    T, E = logits.shape
    _need(token_mask, "token_mask", _MASK, (T,), dev)
    return dev, T, E


def _sequences(seq_offsets, dev):
    if seq_offsets is None:
        return 1
    _need(seq_offsets, "seq_offsets", _I32, None, dev)
    if seq_offsets.dim() != 1 or seq_offsets.shape[0] < 2:
        raise ValueError("seq_offsets must be [S+1] with S >= 1")
    return seq_offsets.shape[0] - 1


def _scalars(t, name, n, dtypes, dev):
    _need(t, name, dtypes, None, dev)
    if t.numel() != n:
        raise ValueError("%s must hold %d value%s" % (name, n, "" if n == 1 else "s"))


def _gradient(d_logits, accumulate, T, E, dev):
    if d_logits is None:
        if accumulate:
            raise ValueError("accumulate needs d_logits to add to")
        return _new((T, E), torch.float32, dev)
    _need(d_logits, "d_logits", _F32, (T, E), dev)
    return d_logits


def balance_loss_workspace_bytes(T: int, E: int, S: int = 1) -> int:
    return int(lib().moe_balance_loss_workspace_bytes(T, E, S))


def balance_loss(logits: torch.Tensor, topk_ids: torch.Tensor, token_mask: torch.Tensor, *,
                 score: int = MOE_SCORE_SIGMOID, seq_offsets: Optional[torch.Tensor] = None, losses=None,
                 counts=None, probs=None, tokens=None, workspace: Optional[torch.Tensor] = None):
    """moe_balance_loss. logits [T,E] fp32, topk_ids [T,k] int32, token_mask
    [T]; seq_offsets [S+1] int32 (None: one sequence). Returns (losses [2]
    fp32: balance and z, counts [S,E] int32, probs [S,E] fp32, tokens [S+2]
    int32: valid tokens per sequence, in all, and sequences that have one)."""
    dev, T, E = _table(logits, token_mask)
    S = _sequences(seq_offsets, dev)
    _need(topk_ids, "topk_ids", _I32, None, dev)
    if topk_ids.dim() != 2 or topk_ids.shape[0] != T:
        raise ValueError("topk_ids must be [T,k] with logits' T")
    k = topk_ids.shape[1]
    losses = _out(losses, "losses", torch.float32, (2,), dev)
    counts = _out(counts, "counts", torch.int32, (S, E), dev)
    probs = _out(probs, "probs", torch.float32, (S, E), dev)
    tokens = _out(tokens, "tokens", torch.int32, (S + 2,), dev)
    workspace, ws, ws_len = _scratch(workspace, balance_loss_workspace_bytes(T, E, S), dev)
    _call("moe_balance_loss", dev,
          logits.data_ptr(), topk_ids.data_ptr(), token_mask.data_ptr(), _ptr(seq_offsets), score, T, E, k, S,
          losses.data_ptr(), counts.data_ptr(), probs.data_ptr(), tokens.data_ptr(), ws, ws_len)
    return losses, counts, probs, tokens


def balance_loss_backward(d_losses: torch.Tensor, logits: torch.Tensor, token_mask: torch.Tensor,
                          counts: torch.Tensor, tokens: torch.Tensor, k: int, *, score: int = MOE_SCORE_SIGMOID,
                          seq_offsets: Optional[torch.Tensor] = None, d_logits: Optional[torch.Tensor] = None,
                          accumulate: bool = False):
    """moe_balance_loss_backward. d_losses [2] fp32 (gradients of balance and
    z); counts and tokens from balance_loss; k its picks per token. Returns
    d_logits [T,E] fp32 (written, or added to with accumulate)."""
    dev, T, E = _table(logits, token_mask)
    S = _sequences(seq_offsets, dev)
    _scalars(d_losses, "d_losses", 2, _F32, dev)
    _need(counts, "counts", _I32, (S, E), dev)
    _need(tokens, "tokens", _I32, (S + 2,), dev)
    d_logits = _gradient(d_logits, accumulate, T, E, dev)
    _call("moe_balance_loss_backward", dev,
          d_losses.data_ptr(), logits.data_ptr(), token_mask.data_ptr(), _ptr(seq_offsets), counts.data_ptr(),
          tokens.data_ptr(), score, T, E, k, S, int(bool(accumulate)), d_logits.data_ptr())
    return d_logits


def distill_loss_workspace_bytes(T: int, E: int) -> int:
    return int(lib().moe_distill_loss_workspace_bytes(T, E))


def _teacher(teacher_ids, teacher_logits, T, dev):
    _need(teacher_ids, "teacher_ids", _I32, None, dev)
    if teacher_ids.dim() != 2 or teacher_ids.shape[0] != T:
        raise ValueError("teacher_ids must be [T,K] with logits' T")
    K = teacher_ids.shape[1]
    _need(teacher_logits, "teacher_logits", _F32, (T, K), dev)
    return K


def distill_loss(logits: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor,
                 token_mask: torch.Tensor, *, score: int = MOE_SCORE_SIGMOID, temperature: float = 1.0, loss=None,
                 token_loss=None, tokens=None, workspace: Optional[torch.Tensor] = None):
    """moe_distill_loss. logits [T,E] fp32 (the student's), teacher_ids [T,K]
    int32 and teacher_logits [T,K] fp32, token_mask [T]. Returns (loss [1]
    fp32, token_loss [T] fp32, tokens [1] int32)."""
    dev, T, E = _table(logits, token_mask)
    K = _teacher(teacher_ids, teacher_logits, T, dev)
    loss = _out(loss, "loss", torch.float32, (1,), dev)
    token_loss = _out(token_loss, "token_loss", torch.float32, (T,), dev)
    tokens = _out(tokens, "tokens", torch.int32, (1,), dev)
    workspace, ws, ws_len = _scratch(workspace, distill_loss_workspace_bytes(T, E), dev)
    _call("moe_distill_loss", dev,
          logits.data_ptr(), teacher_ids.data_ptr(), teacher_logits.data_ptr(), token_mask.data_ptr(), score,
          float(temperature), T, E, K, loss.data_ptr(), token_loss.data_ptr(), tokens.data_ptr(), ws, ws_len)
    return loss, token_loss, tokens


def distill_loss_backward(d_loss: torch.Tensor, logits: torch.Tensor, teacher_ids: torch.Tensor,
                          teacher_logits: torch.Tensor, token_mask: torch.Tensor, tokens: torch.Tensor, *,
                          score: int = MOE_SCORE_SIGMOID, temperature: float = 1.0,
                          d_logits: Optional[torch.Tensor] = None, accumulate: bool = False):
    """moe_distill_loss_backward. d_loss [1] fp32; tokens from distill_loss.
    Returns d_logits [T,E] fp32 (written, or added to with accumulate)."""
    dev, T, E = _table(logits, token_mask)
    K = _teacher(teacher_ids, teacher_logits, T, dev)
    _scalars(d_loss, "d_loss", 1, _F32, dev)
    _scalars(tokens, "tokens", 1, _I32, dev)
    d_logits = _gradient(d_logits, accumulate, T, E, dev)
    _call("moe_distill_loss_backward", dev,
          d_loss.data_ptr(), logits.data_ptr(), teacher_ids.data_ptr(), teacher_logits.data_ptr(),
          token_mask.data_ptr(), tokens.data_ptr(), score, float(temperature), T, E, K, int(bool(accumulate)),
          d_logits.data_ptr())
    return d_logits


def route_backward_workspace_bytes(T: int, H: int, E: int, hidden_dtype: int, logits_in: bool = False) -> int:
    return int(lib().moe_route_backward_workspace_bytes(T, H, E, hidden_dtype, int(bool(logits_in))))


def route_backward(d_topk_w: Optional[torch.Tensor], hidden: Optional[torch.Tensor], W: Optional[torch.Tensor],
                   logits: Optional[torch.Tensor], topk_ids: Optional[torch.Tensor],
                   topk_w: Optional[torch.Tensor], token_mask: torch.Tensor, scale: float = 1.0, *,
                   d_aux: Optional[torch.Tensor] = None, need_hidden: bool = True, need_W: bool = True,
                   d_logits=None, d_hidden=None, d_W=None, workspace: Optional[torch.Tensor] = None):
    """moe_route_backward. d_topk_w [T,k] fp32 (None: only d_aux's gradient,
    and logits, topk_ids and topk_w are unused), d_aux [T,E] fp32 or None;
    hidden, W, scale as given to route() (hidden None: logits-in mode), logits,
    topk_ids, topk_w its outputs. Returns (d_logits [T,E] fp32, d_hidden [T,H]
    in hidden's type, d_W [E,H] fp32); d_hidden and d_W are None in logits-in
    mode or when not needed. d_logits may be d_aux."""
    dev = token_mask.device
    _need(token_mask, "token_mask", _MASK, None, dev)
    if token_mask.dim() != 1:
        raise ValueError("token_mask must be [T]")
    T = token_mask.shape[0]
    if d_topk_w is None and d_aux is None:
        raise ValueError("one of d_topk_w and d_aux is required")
    table = d_aux if d_topk_w is None else logits
    if table is None or table.dim() != 2:
        raise ValueError("logits (d_aux without d_topk_w) must be [T,E]")
    E = table.shape[1]
    k = 1
    if d_topk_w is not None:
        _need(d_topk_w, "d_topk_w", _F32, None, dev)
        if d_topk_w.dim() != 2 or d_topk_w.shape[0] != T:
            raise ValueError("d_topk_w must be [T,k] with T = len(token_mask)")
        k = d_topk_w.shape[1]
        _need(logits, "logits", _F32, (T, E), dev)
        _need(topk_ids, "topk_ids", _I32, (T, k), dev)
        _need(topk_w, "topk_w", _F32, (T, k), dev)
    if d_aux is not None:
        _need(d_aux, "d_aux", _F32, (T, E), dev)
    d_logits = _out(d_logits, "d_logits", torch.float32, (T, E), dev)
    H, dtype = 16, MOE_DTYPE_BF16
    if hidden is None:
        need_hidden = need_W = False
    else:
        _need(hidden, "hidden", _F32 + _BF16, None, dev)
        if hidden.dim() != 2 or hidden.shape[0] != T:
            raise ValueError("hidden must be [T,H] with T = len(token_mask)")
        H = hidden.shape[1]
        dtype = MOE_DTYPE_F32 if hidden.dtype == torch.float32 else MOE_DTYPE_BF16
    if need_hidden:
        _need(W, "W", _F32, (E, H), dev)
        if d_hidden is None:
            d_hidden = torch.empty_like(hidden)
        else:
            _need(d_hidden, "d_hidden", _F32 if dtype == MOE_DTYPE_F32 else _BF16, (T, H), dev)
    else:
        d_hidden = None
    if need_W:
        d_W = _out(d_W, "d_W", torch.float32, (E, H), dev)
    else:
        d_W = None
    workspace, ws, ws_len = _scratch(workspace, route_backward_workspace_bytes(T, H, E, dtype, hidden is None), dev)
    _call("moe_route_backward", dev,
          _ptr(d_topk_w), _ptr(d_aux), _ptr(hidden), dtype, _ptr(W), _ptr(logits), _ptr(topk_ids), _ptr(topk_w),
          token_mask.data_ptr(), float(scale), T, H, E, k, d_logits.data_ptr(), _ptr(d_hidden), _ptr(d_W), ws, ws_len)
    return d_logits, d_hidden, d_W


def combine_backward_workspace_bytes(T: int, R: int, H: int) -> int:
    return int(lib().moe_combine_backward_workspace_bytes(T, R, H))


def combine_backward(d_out: torch.Tensor, expert_out: torch.Tensor, slots: torch.Tensor, topk_w: torch.Tensor,
                     norm_w: torch.Tensor, gain_center: float, eps: float, *, rows: Optional[int] = None,
                     need_norm_w: bool = True, d_expert_out=None, d_topk_w=None, d_norm_w=None,
                     workspace: Optional[torch.Tensor] = None):
    """moe_combine_backward. d_out [T,H] bf16; expert_out, slots, topk_w,
    norm_w, gain_center, eps and rows as given to combine(). Returns
    (d_expert_out [R,H] bf16 with R = rows or expert_out.shape[0], d_topk_w
    [T,k] fp32, d_norm_w [H] fp32 or None)."""
    dev = slots.device
    _need(expert_out, "expert_out", _BF16, None, dev)
    if expert_out.dim() != 2:
        raise ValueError("expert_out must be [R,H]")
    R, H = expert_out.shape
    if rows is not None:
        if rows < 0 or rows > R:
            raise ValueError("rows must be within [0, expert_out.shape[0]]")
        R = rows
    _need(slots, "slots", _I32, None, dev)
    if slots.dim() != 2:
        raise ValueError("slots must be [T,k]")
    T, k = slots.shape
    _need(d_out, "d_out", _BF16, (T, H), dev)
    _need(topk_w, "topk_w", _F32, (T, k), dev)
    _need(norm_w, "norm_w", _F32, (H,), dev)
    d_expert_out = _out(d_expert_out, "d_expert_out", torch.bfloat16, (R, H), dev)
    d_topk_w = _out(d_topk_w, "d_topk_w", torch.float32, (T, k), dev)
    d_norm_w = _out(d_norm_w, "d_norm_w", torch.float32, (H,), dev) if need_norm_w else None
    workspace, ws, ws_len = _scratch(workspace, combine_backward_workspace_bytes(T, R, H), dev)
    _call("moe_combine_backward", dev,
          d_out.data_ptr(), expert_out.data_ptr(), R, slots.data_ptr(), topk_w.data_ptr(), norm_w.data_ptr(),
          float(gain_center), float(eps), T, H, k, d_expert_out.data_ptr(), d_topk_w.data_ptr(), _ptr(d_norm_w), ws,
          ws_len)
    return d_expert_out, d_topk_w, d_norm_w
