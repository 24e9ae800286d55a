"""Drop-in autograd wrapper: a ``torch.autograd.Function`` whose forward and
backward are the library's kernels (the pages' PyTorch integration,
paper.rainbus.top summary, reproducibility notes; paperlayer.ai summary,
section 2).  The backward recomputes P, so only Q, K, V and the lengths are
saved."""
from __future__ import annotations

import math

import torch


class _SigmoidAttentionFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, seqlens_q, seqlens_k, alpha, bias):
        from . import fwd
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        out = fwd(q, k, v, seqlens_q, seqlens_k, alpha, bias)
        ctx.save_for_backward(q, k, v, seqlens_q, seqlens_k)
        ctx.alpha, ctx.bias = alpha, bias
        return out

    @staticmethod
    def backward(ctx, dout):
        from . import bwd
        q, k, v, nq, nk = ctx.saved_tensors
        dq, dk, dv = bwd(q, k, v, dout.contiguous(), nq, nk, ctx.alpha, ctx.bias)
        return dq, dk, dv, None, None, None, None


class _SigmoidAttentionBiasFn(torch.autograd.Function):
    """As _SigmoidAttentionFn with one bias per sample (float32 [Z] tensor); its
    gradient is db_z = sum over heads and valid (i, j) of dS_ij."""

    @staticmethod
    def forward(ctx, q, k, v, seqlens_q, seqlens_k, alpha, bias_z):
        from . import fwd_bias
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        bias_z = bias_z.detach().to(torch.float32).contiguous()
        out = fwd_bias(q, k, v, seqlens_q, seqlens_k, alpha, bias_z)
        ctx.save_for_backward(q, k, v, seqlens_q, seqlens_k, bias_z)
        ctx.alpha = alpha
        return out

    @staticmethod
    def backward(ctx, dout):
        from . import bwd_bias
        q, k, v, nq, nk, bias_z = ctx.saved_tensors
        dq, dk, dv, db = bwd_bias(q, k, v, dout.contiguous(), nq, nk, ctx.alpha, bias_z,
                                  want_dbias=ctx.needs_input_grad[6])
        return dq, dk, dv, None, None, None, db


class _SpanAttentionFn(torch.autograd.Function):
    """The masked attention (``fwd_span`` / ``bwd_span``).  Gradients for q, k and
    v; the bias and the slopes are constants here.  A gradient of the gradient is
    refused: it would leave out how dQ, dK and dV depend on q, k and v."""

    @staticmethod
    def forward(ctx, q, k, v, seqlens, spans, slopes, alpha, bias, cap):
        from . import fwd_span
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        out = fwd_span(q, k, v, seqlens, alpha, bias, spans=spans, cap=cap, slopes=slopes)
        bias_z = bias if isinstance(bias, torch.Tensor) else None
        ctx.save_for_backward(q, k, v, seqlens, spans, slopes, bias_z)
        ctx.alpha, ctx.bias, ctx.cap = alpha, None if bias_z is not None else bias, cap
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        from . import bwd_span
        q, k, v, n, spans, slopes, bias_z = ctx.saved_tensors
        grads = bwd_span(q, k, v, dout.contiguous(), n, ctx.alpha, ctx.bias if bias_z is None else bias_z,
                         spans=spans, cap=ctx.cap, slopes=slopes)
        return (*grads, None, None, None, None, None, None)


class SigmoidAttention(torch.nn.Module):
    """sigma(alpha Q K^T + b) V over padded [Z, L, H, D] batches.

    ``alpha`` defaults to 1/sqrt(D).  The bias follows the pages' b = -log n
    (paperlayer.ai summary, section 3; gist.science summary, section 2.A):

    * default: one scalar, ``bias`` or -ln(L) with n the padded length;
    * ``per_sample_bias=True``: b_z = -ln n_k(z), each sample's true length
      (computed on the device by the library, ``log_length_bias``);
    * ``learnable_bias=True``: a scalar parameter trained through
      db = sum_z db_z, created here with the initial value ``bias``, or -ln
      ``max_len`` (the padded length the module will see) when ``bias`` is not
      given, so that an optimiser built from ``parameters()`` before the first
      call already holds it.

    ``cap`` > 0 caps the scores, cap tanh(alpha q . k / cap), and ``slopes`` (one
    number per head, float32 whatever the module is cast to) takes slopes[h] |i - j|
    off them; both are constants.  A call
    with ``spans`` (``mask_spans``: causal, prefix, document and window masks), or
    with k and v of fewer heads, which groups of query heads share, runs the
    masked attention as well; it needs one length per sample for queries and
    keys, and a bias that is not learned.

    To capture a forward and backward in a CUDA graph, warm up on a side stream
    and drop every output of an eager pass over the same leaves before the
    capture: PyTorch keeps a leaf's gradient node, and the stream it was made on,
    for as long as such an output lives, and a captured backward must not wait
    on a stream outside the capture."""

    def __init__(self, alpha: float | None = None, bias: float | None = None,
                 per_sample_bias: bool = False, learnable_bias: bool = False,
                 max_len: int | None = None, cap: float = 0.0, slopes=None):
        super().__init__()
        if learnable_bias and (cap or slopes is not None):
            raise ValueError("a learned bias goes with neither cap nor slopes")
        self.cap = float(cap)
        if self.cap < 0 or not math.isfinite(self.cap):
            raise ValueError("cap must be 0 or a positive finite number")
        self.register_buffer("slopes", None if slopes is None else
                             torch.as_tensor(slopes, dtype=torch.float32).detach().clone().reshape(-1),
                             persistent=False)
        if per_sample_bias and learnable_bias:
            raise ValueError("choose per_sample_bias or learnable_bias, not both")
        self.alpha, self.bias = alpha, bias
        self.per_sample_bias = per_sample_bias
        self.learnable_bias = learnable_bias
        self.b = None
        if learnable_bias:
            if bias is None and max_len is None:
                raise ValueError("learnable_bias needs an initial value: give bias, or max_len "
                                 "for b = -ln(max_len)")
            init = float(bias) if bias is not None else -math.log(max_len)
            self.b = torch.nn.Parameter(torch.tensor(init))

    def _apply(self, fn, recurse=True):
        """Moves of the module.  The slopes follow to the device but stay float32,
        what the kernels take, with the values they were given: a model cast to bf16
        would otherwise round them to 8 bits."""
        slopes = self.slopes
        super()._apply(fn, recurse)
        if slopes is not None:
            to = self.slopes.device
            self.slopes = slopes.to(to) if not slopes.is_meta else torch.empty_like(slopes, device=to)
        return self

    def forward(self, q, k, v, seqlens_q, seqlens_k=None, spans=None):
        if spans is not None or self.cap or self.slopes is not None or k.shape[2] != q.shape[2]:
            return self._masked(q, k, v, seqlens_q, seqlens_k, spans)
        if seqlens_k is None:
            seqlens_k = seqlens_q
        Z, L, D = q.shape[0], q.shape[1], q.shape[-1]
        alpha = float(1.0 / math.sqrt(D) if self.alpha is None else self.alpha)
        if self.per_sample_bias:
            from . import log_length_bias
            bias_z = log_length_bias(seqlens_k)
            return _SigmoidAttentionBiasFn.apply(q, k, v, seqlens_q, seqlens_k, alpha, bias_z)
        if self.learnable_bias:
            bias_z = self.b.to(device=q.device, dtype=torch.float32).expand(Z)
            return _SigmoidAttentionBiasFn.apply(q, k, v, seqlens_q, seqlens_k, alpha, bias_z)
        bias = -math.log(L) if self.bias is None else self.bias
        return _SigmoidAttentionFn.apply(q, k, v, seqlens_q, seqlens_k, alpha, float(bias))

    def _masked(self, q, k, v, seqlens, seqlens_k, spans):
        if seqlens_k is not None and seqlens_k is not seqlens:
            raise ValueError("the masked attention takes one length per sample, for queries and keys")
        if self.learnable_bias:
            raise ValueError("the masked attention has no gradient for a learned bias")
        alpha = float(1.0 / math.sqrt(q.shape[-1]) if self.alpha is None else self.alpha)
        if self.per_sample_bias:
            from . import log_length_bias
            bias = log_length_bias(seqlens)
        else:
            bias = float(-math.log(q.shape[1]) if self.bias is None else self.bias)
        slopes = None if self.slopes is None else self.slopes.to(q.device)
        return _SpanAttentionFn.apply(q, k, v, seqlens, spans, slopes, alpha, bias, self.cap)
