"""Greyhound-style functional API (the names and signatures of
``greyhound.nn.functional``) over the C ABI, with PyTorch autograd.

Every loss is computed by the library's kernels in the forward call, together
with its gradients (they come out of the same passes); ``backward`` returns
them, multiplied on the device by the upstream gradient.  PyTorch only holds
the tensors: there is no other implementation behind these functions.

* ``cross_entropy(logits, target, ignore_index, reduction, z_loss_multiplier)``
* ``chunked_linear_cross_entropy(inputs, weight, target, ignore_index, reduction,
  z_loss_multiplier, grad_weight_accum_dtype)``
* ``chunked_linear_loss(inputs, weight, loss_and_grad_fn, *loss_args, chunk_size,
  grad_weight_accum_dtype, **loss_kwargs)``
* ``autograd_loss_and_logits_grad(loss_fn)``: adapts a PyTorch scalar loss to
  the ``(loss, grad_logits)`` contract of ``chunked_linear_loss``
* ``selective_log_softmax(logits, index)`` (forward only)
* ``token_logprobs(logits, index, top_k, temperature, ignore_index)``,
  ``topk_distillation(logits, teacher_index, teacher_logits, ...)`` and its linear
  form ``chunked_linear_topk_distillation`` (no Greyhound counterparts)

Data parallel (one process per GPU, a batch split over the ranks of a
``torch.distributed`` group):

* ``data_parallel_cross_entropy`` and ``data_parallel_chunked_linear_cross_entropy``
  return the whole batch's loss on every rank and, in backward, this rank's share
  of its gradients: the valid-token counts are summed over the ranks first (one
  int64 all-reduce), every shard divides by that total, the shards' losses are
  summed (one scalar all-reduce) and so are the weight gradients (fp32
  accumulators summed in fp32 and rounded once, for fp32 accumulation).
"""
from __future__ import annotations

import math

import torch
from torch.autograd.function import once_differentiable

from . import (gh_ce_fwd, gh_ce_fwd_bwd, gh_chunked_linear_loss, gh_distill_count, gh_linear_ce,
               gh_scale_grad, gh_selective_log_softmax, gh_token_logprobs, gh_token_logprobs_vjp, gh_topk_distill)

_PKG = __name__.rpartition(".")[0]

__all__ = ["cross_entropy", "chunked_linear_cross_entropy", "chunked_linear_loss",
           "autograd_loss_and_logits_grad", "selective_log_softmax", "token_logprobs", "topk_distillation",
           "chunked_linear_topk_distillation", "data_parallel_cross_entropy",
           "data_parallel_chunked_linear_cross_entropy"]


def _scaled(grad, g):
    """grad * g for the scalar upstream gradient g, the product in float32 and
    rounded once (g itself rounded to a bf16 gradient's type would scale every
    element wrongly, by up to 2^-8).

    The product is always formed on the device: testing ``g == 1`` first would
    read g back to the host, which stalls the stream on every backward and is
    not allowed while a CUDA graph is being captured."""
    if grad is None:
        return None
    if not grad.is_cuda or (g.requires_grad and torch.is_grad_enabled()):  # (g may be differentiated further)
        wide = torch.promote_types(grad.dtype, torch.float32)
        return (grad.to(wide) * g.to(wide)).to(grad.dtype)
    return gh_scale_grad(grad, g.float())


class _CrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, target, ignore_index, reduction, z):
        V = logits.shape[-1]
        x = logits.reshape(-1, V).contiguous()
        t = target.reshape(-1).contiguous()
        ctx.shape = logits.shape
        if ctx.needs_input_grad[0]:
            loss, grad = gh_ce_fwd_bwd(x, t, ignore_index, reduction, z)
            ctx.save_for_backward(grad)
        else:
            loss, _ = gh_ce_fwd(x, t, ignore_index, reduction, z)
        return loss

    @staticmethod
    def backward(ctx, g):
        (grad,) = ctx.saved_tensors
        return _scaled(grad, g).view(ctx.shape), None, None, None, None


def cross_entropy(logits, target, ignore_index: int = -100, reduction: str = "mean",
                  z_loss_multiplier: float = 0.0):
    """Cross-entropy of ``logits`` [..., V] (float32 or bfloat16, CUDA) against
    ``target`` [...] (int64) with ``ignore_index``, ``"mean"``/``"sum"`` reduction
    and the z-loss ``z_loss_multiplier * lse**2``.  Returns a float32 scalar; its
    backward gives the logits gradient computed in the forward pass."""
    return _CrossEntropy.apply(logits, target, ignore_index, reduction, float(z_loss_multiplier))


class _LinearCE(torch.autograd.Function):
    @staticmethod
    def forward(ctx, inputs, weight, target, ignore_index, reduction, z, accum):
        loss, dX, dW = gh_linear_ce(inputs.contiguous(), weight.contiguous(), target.contiguous(), ignore_index,
                                    reduction, z, 0, accum)
        ctx.save_for_backward(dX, dW)
        return loss

    @staticmethod
    def backward(ctx, g):
        dX, dW = ctx.saved_tensors
        return (_scaled(dX, g) if ctx.needs_input_grad[0] else None,
                _scaled(dW, g) if ctx.needs_input_grad[1] else None, None, None, None, None, None)


def chunked_linear_cross_entropy(inputs, weight, target, ignore_index: int = -100, reduction: str = "mean",
                                 z_loss_multiplier: float = 0.0, grad_weight_accum_dtype: str = "fp32"):
    """Cross-entropy of ``inputs @ weight.T`` (bf16 [BT, D] and [V, D], CUDA)
    computed in row chunks without materialising the logits; the backward gives
    grad_inputs and grad_weight (accumulated in fp32 or in the weight dtype)."""
    return _LinearCE.apply(inputs, weight, target, ignore_index, reduction, float(z_loss_multiplier),
                           grad_weight_accum_dtype)


class _ChunkedLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, inputs, weight, loss_and_grad_fn, chunk, accum, args, kwargs):
        loss, dX, dW = gh_chunked_linear_loss(inputs.contiguous(), weight.contiguous(), loss_and_grad_fn, *args,
                                              chunk=chunk, accum=accum, **kwargs)
        ctx.save_for_backward(dX, dW)
        return loss

    @staticmethod
    def backward(ctx, g):
        dX, dW = ctx.saved_tensors
        return (_scaled(dX, g) if ctx.needs_input_grad[0] else None,
                _scaled(dW, g) if ctx.needs_input_grad[1] else None, None, None, None, None, None)


def chunked_linear_loss(inputs, weight, loss_and_grad_fn, *loss_args, chunk_size=None,
                        grad_weight_accum_dtype: str = "fp32", **loss_kwargs):
    """``inputs @ weight.T`` in row chunks followed by the caller's
    ``loss_and_grad_fn(logits_chunk, *chunk_args, **chunk_kwargs) -> (loss,
    grad_logits)``; tensor arguments whose leading dimension is BT are sliced to
    the chunk's rows.  Returns the sum of the chunk losses."""
    return _ChunkedLoss.apply(inputs, weight, loss_and_grad_fn, int(chunk_size or 0), grad_weight_accum_dtype,
                              loss_args, loss_kwargs)


def autograd_loss_and_logits_grad(loss_fn):
    """Adapt a PyTorch scalar loss ``loss_fn(logits, *args, **kwargs)`` to the
    ``(loss, grad_logits)`` contract: the loss is evaluated on an fp32 copy of
    the chunk logits and differentiated by autograd; the gradient comes back in
    the logits dtype."""
    def loss_and_grad(logits, *args, **kwargs):
        with torch.enable_grad():
            x = logits.detach().float().requires_grad_(True)
            loss = loss_fn(x, *args, **kwargs)
            (g,) = torch.autograd.grad(loss, x)
        return loss.detach(), g.to(logits.dtype)
    return loss_and_grad


def selective_log_softmax(logits, index):
    """``log_softmax(logits)`` gathered at ``index`` (forward only): float32 [...]."""
    return gh_selective_log_softmax(logits.contiguous(), index.contiguous())


def _dense_rows(logits):
    """[..., V] logits as [rows, V] with dense rows (a copy only where the layout needs one)."""
    x = logits if logits.dim() == 2 else logits.reshape(-1, logits.shape[-1])
    if (x.shape[1] > 1 and x.stride(1) != 1) or (x.shape[0] > 1 and x.stride(0) < x.shape[1]):
        x = x.contiguous()
    return x


def _rows_of(t, name, lead, *tail):
    """A companion of logits [*lead, V] as [rows, *tail], row by row: it has the
    logits' leading shape, or is flat already (dimensions of 1 apart).  Any other
    shape of as many elements would pair the wrong rows."""
    rows, n = math.prod(lead), t.dim() - len(tail)

    def ones_dropped(shape):
        return [d for d in shape if d != 1]

    if (n < 0 or tuple(t.shape[n:]) != tail
            or ones_dropped(t.shape[:n]) not in (ones_dropped(lead), ones_dropped((rows,)))):
        raise ValueError(f"{name}: shape {[*lead, *tail]} or {[rows, *tail]}, not {list(t.shape)}")
    return t.reshape(rows, *tail).contiguous()


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, index, top_k, temperature, ignore_index):
        x = _dense_rows(logits)
        t = _rows_of(index, "index", logits.shape[:-1])
        logprob, entropy, lse, top_logprob, top_index = gh_token_logprobs(x, t, top_k, temperature, ignore_index)
        ctx.save_for_backward(x, t, lse, entropy)
        ctx.conf = (logits.shape, temperature, ignore_index)
        lead = logits.shape[:-1]
        logprob, entropy = logprob.view(lead), entropy.clone().view(lead)
        if top_logprob is None:
            return logprob, entropy
        top_logprob, top_index = top_logprob.view(*lead, top_k), top_index.view(*lead, top_k)
        ctx.mark_non_differentiable(top_logprob, top_index)
        return logprob, entropy, top_logprob, top_index

    @staticmethod
    @once_differentiable
    def backward(ctx, g_logprob, g_entropy, *unused):
        x, t, lse, entropy = ctx.saved_tensors
        shape, temperature, ignore_index = ctx.conf
        grad = gh_token_logprobs_vjp(x, t, lse, entropy, g_logprob.reshape(-1).float().contiguous(),
                                     g_entropy.reshape(-1).float().contiguous(), temperature, ignore_index)
        return grad.reshape(shape), None, None, None, None


def token_logprobs(logits, index, top_k: int = 0, temperature: float = 1.0, ignore_index: int = -100):
    """Log-probabilities of ``index`` [...] (or flat) under ``logits`` [..., V]
    (float32 or bfloat16, CUDA) over ``temperature``, and the rows' entropies:
    float32 [...] each, both differentiable.  With ``top_k`` also the most probable
    alternatives' log-probabilities (float32) and ids (int64) [..., top_k], which
    carry no gradient.  Rows whose index is ``ignore_index`` give 0, 0, -inf and
    -1 and a zero gradient."""
    return _TokenLogprobs.apply(logits, index, int(top_k), float(temperature), int(ignore_index))


class _TopkDistillation(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, teacher_index, teacher_logits, temperature, renormalize, reduction):
        x = _dense_rows(logits)
        lead, K = logits.shape[:-1], teacher_index.shape[-1]
        ids = _rows_of(teacher_index, "teacher_index", lead, K)
        values = _rows_of(teacher_logits.float(), "teacher_logits", lead, K)
        ctx.shape = logits.shape
        loss, grad = gh_topk_distill(x, ids, values, temperature, renormalize, reduction,
                                     with_grad=ctx.needs_input_grad[0])
        if grad is not None:
            ctx.save_for_backward(grad)
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        (grad,) = ctx.saved_tensors
        return _scaled(grad, g).reshape(ctx.shape), None, None, None, None, None


def topk_distillation(logits, teacher_index, teacher_logits, temperature: float = 1.0, renormalize: bool = True,
                      reduction: str = "mean"):
    """Distillation of ``logits`` [..., V] (float32 or bfloat16, CUDA) from a
    teacher's stored entries ``teacher_index`` (int64) and ``teacher_logits``
    [..., K] (or flat, [rows, K]): ``temperature**2`` times the Kullback-Leibler sum over the entries
    (see ``gh_topk_distill``).  Returns a float32 scalar; its backward gives the
    logits gradient computed in the forward pass (the teacher gets none)."""
    return _TopkDistillation.apply(logits, teacher_index, teacher_logits, float(temperature), bool(renormalize),
                                   reduction)


def chunked_linear_topk_distillation(inputs, weight, teacher_index, teacher_logits, temperature: float = 1.0,
                                     renormalize: bool = True, reduction: str = "mean", chunk_size=None,
                                     grad_weight_accum_dtype: str = "fp32"):
    """``topk_distillation`` of ``inputs @ weight.T`` (bf16 [BT, D] and [V, D],
    CUDA) in row chunks without materialising the logits (``chunked_linear_loss``
    with the distillation in place on each chunk): ``teacher_index`` and
    ``teacher_logits`` are [BT, K]; a mean divides by all chunks' rows with an
    entry.  The chunk logits are bf16, as for any ``chunked_linear_loss``."""
    lead, K = inputs.shape[:-1], teacher_index.shape[-1]
    ids = _rows_of(teacher_index, "teacher_index", lead, K)
    values = _rows_of(teacher_logits.float(), "teacher_logits", lead, K)
    total = gh_distill_count(ids, values, weight.shape[0])

    def loss_and_grad(logits, ids, values):
        return gh_topk_distill(logits, ids, values, temperature, renormalize, reduction, n_valid_total=total,
                               grad=logits)

    return chunked_linear_loss(inputs, weight, loss_and_grad, ids, values, chunk_size=chunk_size,
                               grad_weight_accum_dtype=grad_weight_accum_dtype)


def _ops(ops):
    """The library's entry points (``ops`` stands in for them in host-only tests
    of the collective steps)."""
    if ops is not None:
        return ops
    import importlib
    return importlib.import_module(_PKG)


def _all_reduce_sum(t, group):
    import torch.distributed as dist
    dist.all_reduce(t.view(-1), op=dist.ReduceOp.SUM, group=group)
    return t


class _DPCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, target, ignore_index, reduction, z, group, ops):
        V = logits.shape[-1]
        x = logits.reshape(-1, V).contiguous()
        t = target.reshape(-1).contiguous()
        n = _all_reduce_sum(ops.gh_count_valid(t, V, ignore_index), group)
        loss, grad = ops.gh_ce_fwd_bwd_shard(x, t, n, ignore_index, reduction, z)
        loss = _all_reduce_sum(loss, group)
        ctx.shape = logits.shape
        ctx.save_for_backward(grad)
        return loss

    @staticmethod
    def backward(ctx, g):
        (grad,) = ctx.saved_tensors
        return _scaled(grad, g).view(ctx.shape), None, None, None, None, None, None


def data_parallel_cross_entropy(logits, target, ignore_index: int = -100, reduction: str = "mean",
                                z_loss_multiplier: float = 0.0, group=None, ops=None):
    """``cross_entropy`` of the whole batch whose shard ``logits`` / ``target``
    this rank holds (the mean divides by the valid count over all ranks)."""
    return _DPCrossEntropy.apply(logits, target, ignore_index, reduction, float(z_loss_multiplier), group,
                                 _ops(ops))


class _DPLinearCE(torch.autograd.Function):
    @staticmethod
    def forward(ctx, inputs, weight, target, ignore_index, reduction, z, accum, group, ops, slices, comm_sms):
        import torch.distributed as dist
        t = target.contiguous()
        n = _all_reduce_sum(ops.gh_count_valid(t, weight.shape[0], ignore_index), group)
        if accum == "fp32":
            # every shard's fp32 accumulator is summed in fp32 and the batch's sum
            # is rounded to the weight dtype once; the sum of each range of
            # weight rows starts as soon as the last chunk has computed it, while
            # the other ranges are still being computed
            V, D = weight.shape
            dW32 = torch.empty((V, D), dtype=torch.float32, device=weight.device)
            works = []

            def on_slice(v0, v1):
                works.append(dist.all_reduce(dW32[v0:v1], op=dist.ReduceOp.SUM, group=group, async_op=True))

            max_sms = 0
            if weight.is_cuda and comm_sms > 0:
                max_sms = max(2, torch.cuda.get_device_properties(weight.device).multi_processor_count - comm_sms)
            loss, dX, _ = ops.gh_linear_ce_shard_f32(inputs.contiguous(), weight.contiguous(), t, n, ignore_index,
                                                     reduction, z, 0, grad_weight_f32=dW32, on_slice=on_slice,
                                                     dw_slices=max(1, int(slices)), max_sms=max_sms)
            for w in works:
                w.wait()
            dW = ops.gh_cast_f32_to_bf16(dW32)
        else:
            # "weight": each shard rounds between its chunks; the shards' sums are
            # added in the weight dtype
            loss, dX, dW = ops.gh_linear_ce_shard(inputs.contiguous(), weight.contiguous(), t, n, ignore_index,
                                                  reduction, z, 0, accum)
            dW = _all_reduce_sum(dW, group)
        loss = _all_reduce_sum(loss, group)
        ctx.save_for_backward(dX, dW)
        return loss

    @staticmethod
    def backward(ctx, g):
        dX, dW = ctx.saved_tensors
        return (_scaled(dX, g) if ctx.needs_input_grad[0] else None,
                _scaled(dW, g) if ctx.needs_input_grad[1] else None, None, None, None, None, None, None, None,
                None, None)


def data_parallel_chunked_linear_cross_entropy(inputs, weight, target, ignore_index: int = -100,
                                               reduction: str = "mean", z_loss_multiplier: float = 0.0,
                                               grad_weight_accum_dtype: str = "fp32", group=None, ops=None,
                                               overlap_slices: int = 4, comm_sms: int = 16):
    """``chunked_linear_cross_entropy`` of the whole batch whose rows ``inputs`` /
    ``target`` this rank holds, with the weight replicated: the weight gradient
    is summed over the ranks, in fp32 and rounded once for
    ``grad_weight_accum_dtype="fp32"``, in the weight dtype for ``"weight"``.

    For fp32 accumulation the last chunk's weight-gradient contraction runs in
    ``overlap_slices`` ranges of weight rows on all but ``comm_sms`` SMs, and
    each range's all-reduce is issued (asynchronously) as soon as it is
    enqueued, so the communication of the first ranges overlaps the
    computation of the rest."""
    return _DPLinearCE.apply(inputs, weight, target, ignore_index, reduction, float(z_loss_multiplier),
                             grad_weight_accum_dtype, group, _ops(ops), int(overlap_slices), int(comm_sms))
