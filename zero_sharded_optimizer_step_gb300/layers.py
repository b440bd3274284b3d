"""The library's training operators as differentiable torch functions: the
embedding lookup, dropout, and linear layers whose operands are quantised to
MXFP4 (include/zero.h, "training operators").

Buffer management and autograd wiring only; every computation is a call of
the binding on the current stream.  Outputs and workspaces come from torch's
allocator.  A model's parameters are the optimizer's (ZeroAdam's views of
its flat buffer, say); the gradients that backward() leaves in `.grad` go into
a rank's gradient buffer, or `embed_grad` and `Mx4Linear.weight_grad` write them
there directly.  The lookup and dropout can be differentiated any number of
times, the linear layer once: an attempt at more raises.

A 4-bit product whose waits on the device run out stores nothing, and its call
has long returned: where a program reads its losses it also asks for the count
(`zero_mx4_timeouts()`, 0 when all is well), which waits for the device.

    h = embed(table, tokens, pad=0)
    h = dropout(h, 0.1, seed, offset)
    y = layer(h)                     # layer = Mx4Linear(weight)
    h = dropout(y, 0.1, seed, offset + 1, residual=h)
    ...
    opt.step(); layer.refresh()      # the weight changed: quantise it again
"""
from __future__ import annotations

import torch

from . import binding as z

_DT = {torch.float32: z.ZERO_F32, torch.bfloat16: z.ZERO_BF16, torch.float16: z.ZERO_F16}


def _rows_apart(x: torch.Tensor) -> bool:
    """Whether x's rows are runs of consecutive elements that do not overlap."""
    return not (x.shape[1] > 1 and x.stride(1) != 1 or
                x.shape[0] > 1 and x.stride(0) < x.shape[1])


def _gradient(dy: torch.Tensor) -> torch.Tensor:
    """An output's gradient as the library can take it.  torch hands on what the
    next operation's gradient looks like: expanded over the rows after a sum
    over them, say."""
    return dy if _rows_apart(dy) else dy.contiguous()


def _matrix(name: str, x: torch.Tensor) -> torch.Tensor:
    """x itself if the library can take it as rows of elements."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if x.dtype not in _DT:
        raise ValueError("%s must be fp32, bf16 or fp16, not %s" % (name, x.dtype))
    if x.dim() != 2:
        raise ValueError("%s must have two dimensions, not %d" % (name, x.dim()))
    if not _rows_apart(x):
        raise ValueError("%s must have consecutive elements in its rows" % name)
    return x


def _stride(x: torch.Tensor) -> int:
    return max(x.stride(0), x.shape[1]) if x.shape[0] > 1 else x.shape[1]


def _tokens(tokens: torch.Tensor, device) -> torch.Tensor:
    if not isinstance(tokens, torch.Tensor) or tokens.dtype not in (torch.int32, torch.int64):
        raise ValueError("tokens must be an int32 or int64 tensor")
    if tokens.device != device:
        raise ValueError("tokens must be on %s" % device)
    return tokens.contiguous()


def _same(name: str, x: torch.Tensor, like: torch.Tensor) -> None:
    if x.device != like.device or x.dtype != like.dtype or x.shape != like.shape:
        raise ValueError("%s must match in device, dtype and shape" % name)


# ----------------------------------------------------------------- embedding

def embed_grad(dy: torch.Tensor, tokens: torch.Tensor, grad: torch.Tensor, scale: float = 1.0,
               pad: int = -1, accumulate: bool = False) -> torch.Tensor:
    """The table's gradient from dy (a row a token) into `grad` (a row a table
    row: a view of a rank's gradient buffer, say); accumulate adds to it."""
    _matrix("dy", dy)
    _matrix("grad", grad)
    tokens = _tokens(tokens, grad.device)
    if dy.device != grad.device or dy.shape[1] != grad.shape[1] or dy.shape[0] != tokens.numel():
        raise ValueError("dy must have a row of grad's width for every token, on its device")
    rows, dim = grad.shape
    n = tokens.numel()
    with torch.cuda.device(grad.device):
        need = z.zero_embed_grad_workspace(rows, dim, n)
        ws = torch.empty(need, dtype=torch.uint8, device=grad.device)
        z.zero_embed_grad(dy, _DT[dy.dtype], _stride(dy), tokens, tokens.element_size(), n, pad,
                          scale, grad, _DT[grad.dtype], rows, dim, _stride(grad), accumulate, ws,
                          need)
    return grad


class _Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, tokens, scale, pad, bad):
        flat = _tokens(tokens, table.device).reshape(-1)
        out = torch.empty(flat.numel(), table.shape[1], dtype=table.dtype, device=table.device)
        with torch.cuda.device(table.device):
            z.zero_embed(table, _DT[table.dtype], table.shape[0], table.shape[1], _stride(table),
                         flat, flat.element_size(), flat.numel(), pad, scale, out, table.shape[1],
                         bad)
        ctx.save_for_backward(flat)
        ctx.like, ctx.scale, ctx.pad = table, scale, pad
        return out.view(*tokens.shape, table.shape[1])

    @staticmethod
    def backward(ctx, dy):
        (flat,) = ctx.saved_tensors
        dy = dy.reshape(flat.numel(), ctx.like.shape[1])
        grad = (_EmbedGrad.apply if torch.is_grad_enabled() else _table_grad)(
            dy, flat, ctx.like, ctx.scale, ctx.pad)
        return grad, None, None, None, None


def _table_grad(dy, flat, like, scale, pad):
    grad = torch.empty(like.shape, dtype=like.dtype, device=like.device)
    return embed_grad(_gradient(dy), flat, grad, scale, pad)


class _EmbedGrad(torch.autograd.Function):
    """The lookup's transpose; its own gradient is the lookup again."""
    @staticmethod
    def forward(ctx, dy, flat, like, scale, pad):
        ctx.save_for_backward(flat)
        ctx.scale, ctx.pad = scale, pad
        return _table_grad(dy, flat, like, scale, pad)

    @staticmethod
    def backward(ctx, g):
        (flat,) = ctx.saved_tensors
        return _Embed.apply(_gradient(g), flat, ctx.scale, ctx.pad, None), None, None, None, None


def embed(table: torch.Tensor, tokens: torch.Tensor, scale: float = 1.0, pad: int = -1,
          bad: torch.Tensor | None = None) -> torch.Tensor:
    """scale * table[tokens], rows of zeros for the token `pad` and for ids
    outside the table; those are counted in `bad` (one int64 on the device)."""
    _matrix("table", table)
    if bad is not None and (bad.dtype != torch.int64 or bad.device != table.device):
        raise ValueError("bad must be an int64 tensor on the table's device")
    return _Embed.apply(table, tokens, float(scale), int(pad), bad)


# ------------------------------------------------------------------- dropout

def _drop(x, residual, p, seed, offset):
    x = x.contiguous()
    out = torch.empty_like(x)
    with torch.cuda.device(x.device):
        z.zero_dropout(x, residual, out, _DT[x.dtype], x.numel(), p, seed, offset)
    return out


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, seed, offset):
        ctx.args = p, seed, offset
        return _drop(x, residual, p, seed, offset)

    @staticmethod
    def backward(ctx, dy):
        dx = None
        if ctx.needs_input_grad[0]:
            # the same map of dy; where a graph of it is wanted, differentiable again
            dx = (_Dropout.apply if torch.is_grad_enabled() else _drop)(dy, None, *ctx.args)
        return dx, dy if ctx.needs_input_grad[1] else None, None, None, None


def dropout(x: torch.Tensor, p: float, seed: int, offset: int,
            residual: torch.Tensor | None = None) -> torch.Tensor:
    """residual + x with elements dropped by probability p and the others
    divided by 1 - p.  (seed, offset) names the stream of random words: give
    every call of a step an offset of its own.  The mask is made again in the
    backward pass, not stored."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype not in _DT:
        raise ValueError("x must be an fp32, bf16 or fp16 CUDA tensor")
    if not 0.0 <= p <= 1.0:
        raise ValueError("p must be in [0, 1]")
    if residual is not None:
        _same("residual", residual, x)
        residual = residual.contiguous()
    return _Dropout.apply(x, residual, float(p), int(seed) & (2 ** 64 - 1),
                          int(offset) & (2 ** 64 - 1))


# -------------------------------------------------------------- 4-bit products

class Mx4Matrix:
    """A matrix quantised to MXFP4, blocks along its rows."""

    def __init__(self, rows: int, cols: int, device):
        self.rows, self.cols = rows, cols
        self.q = torch.empty(z.zero_mx4_bytes(rows, cols), dtype=torch.uint8, device=device)

    def values(self, dtype: torch.dtype = torch.float32) -> torch.Tensor:
        out = torch.empty(self.rows, self.cols, dtype=dtype, device=self.q.device)
        with torch.cuda.device(out.device):
            z.zero_mx4_dequantize(self.q, self.rows, self.cols, out, _DT[dtype], self.cols)
        return out


def mx4_quantize(x: torch.Tensor, rows: bool = True, cols: bool = True):
    """(x quantised along its rows, its transpose quantised along x's columns),
    either None where not asked for."""
    _matrix("x", x)
    R, C = x.shape
    q = Mx4Matrix(R, C, x.device) if rows else None
    qt = Mx4Matrix(C, R, x.device) if cols else None
    if not (rows or cols):
        return q, qt
    with torch.cuda.device(x.device):
        z.zero_mx4_quantize(x, _DT[x.dtype], R, C, _stride(x), q.q if q else None,
                            qt.q if qt else None)
    return q, qt


def mx4_matmul(a: Mx4Matrix, b: Mx4Matrix, dtype: torch.dtype = torch.bfloat16,
               out: torch.Tensor | None = None, alpha: float = 1.0,
               accumulate: bool = False) -> torch.Tensor:
    """alpha * A B^T, into (or added to) `out` if that is given."""
    if a.cols != b.cols or a.q.device != b.q.device:
        raise ValueError("the matrices must have as many columns and one device")
    if out is None:
        if accumulate:
            raise ValueError("there is nothing to add to")
        out = torch.empty(a.rows, b.rows, dtype=dtype, device=a.q.device)
    _matrix("out", out)
    if out.shape != (a.rows, b.rows) or out.device != a.q.device:
        raise ValueError("out must be %d by %d on %s" % (a.rows, b.rows, a.q.device))
    with torch.cuda.device(out.device):
        z.zero_mx4_matmul(a.q, a.rows, b.q, b.rows, a.cols, alpha, accumulate, out,
                          _DT[out.dtype], _stride(out))
    return out


class _Once(torch.autograd.Function):
    """A gradient that depends on what `links` do and cannot be differentiated.
    (torch's once_differentiable does not tie it to them: a derivative with
    respect to given inputs would leave it out and say nothing.)"""
    @staticmethod
    def forward(ctx, grad, *links):
        return grad.clone()

    @staticmethod
    def backward(ctx, g):
        raise RuntimeError("Mx4Linear can be differentiated once: its gradients have none")


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, layer, grads):
        ctx.set_materialize_grads(False)
        ctx.layer, ctx.dtype = layer, x.dtype
        # needs_input_grad tells what the tensors ask for, not whether a
        # backward pass can follow (and here, inside, gradients are always off)
        q, ctx.xt = mx4_quantize(x, True, grads and ctx.needs_input_grad[1])
        # the weight as it was quantised for this forward pass
        ctx.wt = layer.wt if ctx.needs_input_grad[0] else None
        link = None
        if grads:                        # leads back to x and the weight, and holds neither
            link = x.new_empty(0)
            ctx.save_for_backward(link)
        return mx4_matmul(q, layer.w, x.dtype), link

    @staticmethod
    def backward(ctx, dy, _):
        dx = dw = None
        if dy is not None:
            q, qt = mx4_quantize(_gradient(dy), ctx.needs_input_grad[0], ctx.needs_input_grad[1])
            if q is not None:
                dx = mx4_matmul(q, ctx.wt, ctx.dtype)
            if qt is not None:
                dw = mx4_matmul(qt, ctx.xt, ctx.layer.weight.dtype)
            if torch.is_grad_enabled():      # a graph of the gradients is wanted
                (link,) = ctx.saved_tensors
                dx, dw = (None if g is None else _Once.apply(g, dy, link) for g in (dx, dw))
        return dx, dw, None, None


class Mx4Linear:
    """y = x W^T with x, W and, in the backward pass, dy quantised to MXFP4 and
    the products summed in fp32.  The gradients are those of the product of
    the quantised operands, passed straight through the quantisation.

    weight: [n, k]; quantised here, along both of its dimensions, and again by
    refresh(), which belongs after every change of it (an optimizer step)."""

    def __init__(self, weight: torch.Tensor):
        self.weight = weight
        self.w = self.wt = None
        self.refresh()

    def refresh(self) -> None:
        with torch.no_grad():
            self.w, self.wt = mx4_quantize(self.weight.detach())

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        n, k = self.weight.shape
        if x.dim() < 1 or x.shape[-1] != k or x.device != self.weight.device:
            raise ValueError("x must have rows of %d elements on %s" % (k, self.weight.device))
        rows = x.reshape(-1, k)
        _matrix("x", rows)
        return _Linear.apply(rows, self.weight, self, torch.is_grad_enabled())[0].view(
            *x.shape[:-1], n)

    def weight_grad(self, x: torch.Tensor, dy: torch.Tensor, grad: torch.Tensor,
                    accumulate: bool = False) -> torch.Tensor:
        """The weight's gradient from the layer's input and its output's
        gradient, into `grad` ([n, k]: a view of a rank's gradient buffer)."""
        _, xt = mx4_quantize(x, False, True)
        _, dyt = mx4_quantize(dy, False, True)
        return mx4_matmul(dyt, xt, out=grad, accumulate=accumulate)
