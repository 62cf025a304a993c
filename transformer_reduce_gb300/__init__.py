"""transformer_reduce_gb300 -- fused softmax and LayerNorm reduce kernels of a
Transformer layer, forward and backward, for NVIDIA GB300 (sm_103a).

The compute is hand-written CUDA in ``libls_reduce.so`` behind a C ABI
(``include/ls_reduce.h``).  ``transformer_reduce_gb300._lib`` mirrors that ABI
one-for-one (raw pointers); the functions below are the PyTorch-facing
convenience layer: they check shapes, allocate outputs with torch, and pass
pointers and the current CUDA stream to the library.  There is no fallback:
if the library is missing or a call fails, they raise.
"""
from __future__ import annotations

import array
import bisect
import operator

from . import _lib as _lib_module
from ._lib import (LS_BF16, LS_ERR_CUDA, ls_cross_entropy_bw, ls_cross_entropy_fw,
                   ls_softmax_bw_masked_scaled, ls_softmax_fw_scaled, LS_ERR_INVALID_ARG, LS_ERR_MISALIGNED,  # noqa: F401
                   LS_ERR_UNSUPPORTED, LS_ERR_WORKSPACE, LS_F16, LS_F32, LS_OK, LsError,
                   ls_layernorm_bw_dgamma_dbeta, ls_layernorm_bw_dgamma_dbeta_workspace_size,
                   ls_layernorm_bw, ls_layernorm_bw_dinp, ls_layernorm_bw_workspace_size,
                   ls_layernorm_fw, ls_rmsnorm_bw_dgamma,
                   ls_rmsnorm_bw_dinp, ls_rmsnorm_fw, ls_softmax_bw, ls_softmax_bw_masked,
                   ls_softmax_fw, load, status_string)
from ._lib import (ls_grad_clip, ls_grad_norm, ls_grad_norm_workspace_size, ls_qk_norm_rope_bw,
                   ls_qk_norm_rope_bw_workspace_size, ls_qk_norm_rope_fw, ls_softmax_bw_relpos,
                   ls_softmax_bw_relpos_workspace_size, ls_softmax_fw_relpos)

__all__ = [
    "softmax_fw", "softmax_bw", "softmax_bw_masked", "layernorm_fw", "layernorm_bw_dinp",
    "layernorm_bw_dgamma_dbeta", "dgamma_dbeta_workspace", "layernorm_bw", "rmsnorm_fw", "rmsnorm_bw_dinp",
    "rmsnorm_bw_dgamma", "cross_entropy_fw", "cross_entropy_bw", "LsError", "load",
    "ls_cross_entropy_fw", "ls_cross_entropy_bw", "ls_softmax_fw_scaled",
    "ls_softmax_bw_masked_scaled",
    "ls_softmax_fw", "ls_softmax_bw", "ls_softmax_bw_masked", "ls_layernorm_fw", "ls_layernorm_bw_dinp",
    "ls_layernorm_bw_dgamma_dbeta", "ls_layernorm_bw_dgamma_dbeta_workspace_size",
    "ls_layernorm_bw", "ls_layernorm_bw_workspace_size", "ls_rmsnorm_fw", "ls_rmsnorm_bw_dinp", "ls_rmsnorm_bw_dgamma",
    "relpos_buckets", "softmax_fw_relpos", "softmax_bw_relpos", "softmax_relpos_workspace",
    "rope_tables", "qk_norm_rope_fw", "qk_norm_rope_bw", "qk_norm_rope_workspace",
    "grad_norm", "grad_clip", "grad_norm_workspace",
    "ls_softmax_fw_relpos", "ls_softmax_bw_relpos", "ls_softmax_bw_relpos_workspace_size",
    "ls_qk_norm_rope_fw", "ls_qk_norm_rope_bw", "ls_qk_norm_rope_bw_workspace_size",
    "ls_grad_norm", "ls_grad_clip", "ls_grad_norm_workspace_size",
]


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


_DTYPE_CODES = {}


def ls_dtype(t) -> int:
    if not _DTYPE_CODES:
        torch = _torch()
        _DTYPE_CODES.update({torch.float32: LS_F32, torch.float16: LS_F16,
                             torch.bfloat16: LS_BF16})
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported storage dtype {t.dtype} (float32, float16, bfloat16)")
    return code


def _stream(t) -> int:
    torch = _torch()
    return torch.cuda.current_stream(t.device).cuda_stream


def _dev(*ts):
    """The one CUDA device all given tensors live on (None entries skipped);
    every tensor must be contiguous."""
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must live on a CUDA device (there is no CPU path)")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"tensors on different devices ({dev} and {t.device})")
    return dev


def _want(name, t, shape, dtype):
    """Reject a tensor whose shape or dtype differs from what the kernels will
    read or write through its pointer (they trust the sizes they are given)."""
    if t is None:
        return
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} of shape {list(shape)}, "
                         f"got {t.dtype} of shape {list(t.shape)}")


def _workspace(name, t):
    torch = _torch()
    if t.dtype != torch.float32 or t.dim() != 1:
        raise ValueError(f"{name} must be a 1-D float32 tensor")


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _ok(status: int, where: str):
    if status != LS_OK:
        raise LsError(status, where)


def _call(where: str, dev, fn, *args):
    """Run one library call with ``dev`` as the current device (the library
    launches on the current device, on the stream it is given)."""
    torch = _torch()
    if dev.index == torch.cuda.current_device():
        _ok(fn(*args), where)
        return
    with torch.cuda.device(dev):
        _ok(fn(*args), where)


def _same_device(*ts):
    """The index of the one CUDA device of all given tensors (None skipped), all
    contiguous; as _dev, in one call per tensor and property."""
    index = -1
    for t in ts:
        if t is not None:
            i = t.get_device()
            if i < 0 or (index >= 0 and i != index) or not t.is_contiguous():
                return _dev(*ts).index  # says which of them is wrong
            index = i
    return index


def _launch(where: str, index: int, *args):
    """Calls the library on device ``index``'s current stream, which is passed
    after the given arguments, with that device current."""
    torch = _torch()
    fn = getattr(_lib_module._lib or load(), where)
    if index == torch.cuda.current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status != LS_OK:
        raise LsError(status, where)


def _raw_stream(index: int) -> int:
    """Handle of the current stream of device ``index`` (without building a
    Stream object where torch can say it directly)."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


def _rows_hidden(x, name="x"):
    if x.dim() != 2:
        raise ValueError(f"{name} must be [rows, hidden]")
    return x.shape


def softmax_fw(scores, mask=None, causal: bool = False, out=None, scale=None):
    """Softmax over the last axis of scale * scores [B,H,Tq,Tk] plus an
    additive mask [B,Tk] (broadcast over heads and queries), future keys
    j > i + Tk - Tq masked when ``causal`` (Tq <= Tk).  ``scale`` None is 1.
    ``out`` may be ``scores`` (in place)."""
    torch = _torch()
    if scores.dim() != 4:
        raise ValueError("scores must be [B, H, Tq, Tk]")
    B, H, Tq, Tk = scores.shape
    _want("mask", mask, (B, Tk), scores.dtype)
    _want("out", out, scores.shape, scores.dtype)
    out = torch.empty_like(scores) if out is None else out
    dev = _dev(scores, mask, out)
    if scale is None:
        _call("ls_softmax_fw", dev, ls_softmax_fw, _ptr(out), _ptr(scores), _ptr(mask), B, H, Tq,
              Tk, causal, ls_dtype(scores), _stream(scores))
    else:
        _call("ls_softmax_fw_scaled", dev, ls_softmax_fw_scaled, _ptr(out), _ptr(scores),
              _ptr(mask), B, H, Tq, Tk, causal, float(scale), ls_dtype(scores), _stream(scores))
    return out


def softmax_bw(dout, out_fw, dinp=None):
    """Gradient of the softmax input from the output gradient ``dout`` and the
    forward output ``out_fw`` (both [B,H,Tq,Tk]).  ``dinp`` may be ``dout``."""
    torch = _torch()
    if dout.dim() != 4:
        raise ValueError("dout must be [B, H, Tq, Tk]")
    _want("out_fw", out_fw, dout.shape, dout.dtype)
    _want("dinp", dinp, dout.shape, dout.dtype)
    B, H, Tq, Tk = dout.shape
    dinp = torch.empty_like(dout) if dinp is None else dinp
    dev = _dev(dout, out_fw, dinp)
    _call("ls_softmax_bw", dev, ls_softmax_bw, _ptr(dinp), _ptr(dout), _ptr(out_fw), B, H, Tq, Tk,
          ls_dtype(dout), _stream(dout))
    return dinp


def softmax_bw_masked(dout, out_fw, mask=None, causal: bool = False, dinp=None, scale=None):
    """Softmax backward that reads only visible keys (mask != -inf, not in the
    causal future) and writes 0 on the others; with ``scale`` the gradient of
    the scores of ``softmax_fw(..., scale=scale)``."""
    torch = _torch()
    if dout.dim() != 4:
        raise ValueError("dout must be [B, H, Tq, Tk]")
    B, H, Tq, Tk = dout.shape
    _want("out_fw", out_fw, dout.shape, dout.dtype)
    _want("mask", mask, (B, Tk), dout.dtype)
    _want("dinp", dinp, dout.shape, dout.dtype)
    dinp = torch.empty_like(dout) if dinp is None else dinp
    dev = _dev(dout, out_fw, mask, dinp)
    if scale is None:
        _call("ls_softmax_bw_masked", dev, ls_softmax_bw_masked, _ptr(dinp), _ptr(dout),
              _ptr(out_fw), _ptr(mask), B, H, Tq, Tk, causal, ls_dtype(dout), _stream(dout))
    else:
        _call("ls_softmax_bw_masked_scaled", dev, ls_softmax_bw_masked_scaled, _ptr(dinp),
              _ptr(dout), _ptr(out_fw), _ptr(mask), B, H, Tq, Tk, causal, float(scale),
              ls_dtype(dout), _stream(dout))
    return dinp


def _stats(rows, x, **named):
    torch = _torch()
    for name, t in named.items():
        _want(name, t, (rows,), torch.float32)


def layernorm_fw(x, gamma, beta, eps: float = 1e-8, y=None, mean=None, rstd=None):
    """LayerNorm of x [rows, hidden]; returns (y, mean, rstd), the statistics fp32."""
    torch = _torch()
    rows, hidden = _rows_hidden(x)
    _want("gamma", gamma, (hidden,), x.dtype)
    _want("beta", beta, (hidden,), x.dtype)
    _want("y", y, x.shape, x.dtype)
    _stats(rows, x, mean=mean, rstd=rstd)
    y = torch.empty_like(x) if y is None else y
    mean = torch.empty(rows, device=x.device, dtype=torch.float32) if mean is None else mean
    rstd = torch.empty(rows, device=x.device, dtype=torch.float32) if rstd is None else rstd
    dev = _dev(x, gamma, beta, y, mean, rstd)
    _call("ls_layernorm_fw", dev, ls_layernorm_fw, _ptr(y), _ptr(mean), _ptr(rstd), _ptr(x),
          _ptr(gamma), _ptr(beta), rows, hidden, float(eps), ls_dtype(x), _stream(x))
    return y, mean, rstd


def layernorm_bw_dinp(dy, x, gamma, mean, rstd, dx=None):
    """Input gradient of LayerNorm from dy, x and the saved fp32 mean / rstd."""
    torch = _torch()
    rows, hidden = _rows_hidden(x)
    _want("dy", dy, x.shape, x.dtype)
    _want("gamma", gamma, (hidden,), x.dtype)
    _stats(rows, x, mean=mean, rstd=rstd)
    _want("dx", dx, x.shape, x.dtype)
    dx = torch.empty_like(x) if dx is None else dx
    dev = _dev(dy, x, gamma, mean, rstd, dx)
    _call("ls_layernorm_bw_dinp", dev, ls_layernorm_bw_dinp, _ptr(dx), _ptr(dy), _ptr(x),
          _ptr(gamma), _ptr(mean), _ptr(rstd), rows, hidden, ls_dtype(x), _stream(x))
    return dx


def dgamma_dbeta_workspace(rows: int, hidden: int, device):
    """A workspace tensor of the size ls_layernorm_bw_dgamma_dbeta needs."""
    torch = _torch()
    n = ls_layernorm_bw_dgamma_dbeta_workspace_size(rows, hidden)
    return torch.empty(max(n, 16) // 4, device=device, dtype=torch.float32)


def layernorm_bw_dgamma_dbeta(dy, x, mean, rstd, workspace=None, dgamma=None, dbeta=None):
    """gamma / beta gradients (fp32 [hidden]) summed over all rows, in a fixed
    order (bitwise reproducible)."""
    torch = _torch()
    rows, hidden = _rows_hidden(x)
    _want("dy", dy, x.shape, x.dtype)
    _stats(rows, x, mean=mean, rstd=rstd)
    _want("dgamma", dgamma, (hidden,), torch.float32)
    _want("dbeta", dbeta, (hidden,), torch.float32)
    if workspace is None:
        workspace = dgamma_dbeta_workspace(rows, hidden, x.device)
    _workspace("workspace", workspace)
    dgamma = torch.empty(hidden, device=x.device, dtype=torch.float32) if dgamma is None else dgamma
    dbeta = torch.empty(hidden, device=x.device, dtype=torch.float32) if dbeta is None else dbeta
    dev = _dev(dy, x, mean, rstd, workspace, dgamma, dbeta)
    _call("ls_layernorm_bw_dgamma_dbeta", dev, ls_layernorm_bw_dgamma_dbeta, _ptr(dgamma),
          _ptr(dbeta), _ptr(dy), _ptr(x), _ptr(mean), _ptr(rstd), rows, hidden, _ptr(workspace),
          workspace.numel() * workspace.element_size(), ls_dtype(x), _stream(x))
    return dgamma, dbeta


def layernorm_bw(dy, x, gamma, mean, rstd, workspace=None, dx=None, dgamma=None, dbeta=None):
    """Whole LayerNorm backward in one pass over dy and x: returns
    (dx, dgamma, dbeta), the parameter gradients fp32 in a fixed order."""
    torch = _torch()
    rows, hidden = _rows_hidden(x)
    _want("dy", dy, x.shape, x.dtype)
    _want("gamma", gamma, (hidden,), x.dtype)
    _stats(rows, x, mean=mean, rstd=rstd)
    _want("dx", dx, x.shape, x.dtype)
    _want("dgamma", dgamma, (hidden,), torch.float32)
    _want("dbeta", dbeta, (hidden,), torch.float32)
    if workspace is None:
        n = ls_layernorm_bw_workspace_size(rows, hidden)
        workspace = torch.empty(max(n, 16) // 4, device=x.device, dtype=torch.float32)
    _workspace("workspace", workspace)
    dx = torch.empty_like(x) if dx is None else dx
    dgamma = torch.empty(hidden, device=x.device, dtype=torch.float32) if dgamma is None else dgamma
    dbeta = torch.empty(hidden, device=x.device, dtype=torch.float32) if dbeta is None else dbeta
    dev = _dev(dy, x, gamma, mean, rstd, workspace, dx, dgamma, dbeta)
    _call("ls_layernorm_bw", dev, ls_layernorm_bw, _ptr(dx), _ptr(dgamma), _ptr(dbeta), _ptr(dy),
          _ptr(x), _ptr(gamma), _ptr(mean), _ptr(rstd), rows, hidden, _ptr(workspace),
          workspace.numel() * workspace.element_size(), ls_dtype(x), _stream(x))
    return dx, dgamma, dbeta


def rmsnorm_fw(x, gamma, eps: float = 1e-6, y=None, rstd=None):
    """RMSNorm of x [rows, hidden]: y = x * rsqrt(mean(x^2) + eps) * gamma;
    returns (y, rstd), rstd fp32."""
    torch = _torch()
    rows, hidden = _rows_hidden(x)
    _want("gamma", gamma, (hidden,), x.dtype)
    _want("y", y, x.shape, x.dtype)
    _stats(rows, x, rstd=rstd)
    y = torch.empty_like(x) if y is None else y
    rstd = torch.empty(rows, device=x.device, dtype=torch.float32) if rstd is None else rstd
    dev = _dev(x, gamma, y, rstd)
    _call("ls_rmsnorm_fw", dev, ls_rmsnorm_fw, _ptr(y), _ptr(rstd), _ptr(x), _ptr(gamma), rows,
          hidden, float(eps), ls_dtype(x), _stream(x))
    return y, rstd


def rmsnorm_bw_dinp(dy, x, gamma, rstd, dx=None):
    """Input gradient of RMSNorm from dy, x and the saved fp32 rstd."""
    torch = _torch()
    rows, hidden = _rows_hidden(x)
    _want("dy", dy, x.shape, x.dtype)
    _want("gamma", gamma, (hidden,), x.dtype)
    _stats(rows, x, rstd=rstd)
    _want("dx", dx, x.shape, x.dtype)
    dx = torch.empty_like(x) if dx is None else dx
    dev = _dev(dy, x, gamma, rstd, dx)
    _call("ls_rmsnorm_bw_dinp", dev, ls_rmsnorm_bw_dinp, _ptr(dx), _ptr(dy), _ptr(x), _ptr(gamma),
          _ptr(rstd), rows, hidden, ls_dtype(x), _stream(x))
    return dx


def rmsnorm_bw_dgamma(dy, x, rstd, workspace=None, dgamma=None):
    """gamma gradient of RMSNorm (fp32 [hidden]), fixed summation order."""
    torch = _torch()
    rows, hidden = _rows_hidden(x)
    _want("dy", dy, x.shape, x.dtype)
    _stats(rows, x, rstd=rstd)
    _want("dgamma", dgamma, (hidden,), torch.float32)
    if workspace is None:
        workspace = dgamma_dbeta_workspace(rows, hidden, x.device)
    _workspace("workspace", workspace)
    dgamma = torch.empty(hidden, device=x.device, dtype=torch.float32) if dgamma is None else dgamma
    dev = _dev(dy, x, rstd, workspace, dgamma)
    _call("ls_rmsnorm_bw_dgamma", dev, ls_rmsnorm_bw_dgamma, _ptr(dgamma), _ptr(dy), _ptr(x),
          _ptr(rstd), rows, hidden, _ptr(workspace), workspace.numel() * workspace.element_size(),
          ls_dtype(x), _stream(x))
    return dgamma


def cross_entropy_fw(logits, target, loss=None, lse=None):
    """Per-row softmax cross entropy of logits [rows, vocab] against int32
    target [rows] (negative = ignored row); returns (loss, lse), fp32."""
    torch = _torch()
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, vocab]")
    rows, vocab = logits.shape
    _want("target", target, (rows,), torch.int32)
    _stats(rows, logits, loss=loss, lse=lse)
    loss = torch.empty(rows, device=logits.device, dtype=torch.float32) if loss is None else loss
    lse = torch.empty(rows, device=logits.device, dtype=torch.float32) if lse is None else lse
    dev = _dev(logits, target, loss, lse)
    _call("ls_cross_entropy_fw", dev, ls_cross_entropy_fw, _ptr(loss), _ptr(lse), _ptr(logits),
          _ptr(target), rows, vocab, ls_dtype(logits), _stream(logits))
    return loss, lse


def cross_entropy_bw(logits, target, lse, dloss, dlogits=None):
    """Gradient dloss * (softmax(logits) - onehot(target)) per row, from the
    forward's lse; ``dlogits`` may be ``logits`` (in place)."""
    torch = _torch()
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, vocab]")
    rows, vocab = logits.shape
    _want("target", target, (rows,), torch.int32)
    _stats(rows, logits, lse=lse, dloss=dloss)
    _want("dlogits", dlogits, logits.shape, logits.dtype)
    dlogits = torch.empty_like(logits) if dlogits is None else dlogits
    dev = _dev(logits, target, lse, dloss, dlogits)
    _call("ls_cross_entropy_bw", dev, ls_cross_entropy_bw, _ptr(dlogits), _ptr(logits),
          _ptr(target), _ptr(lse), _ptr(dloss), rows, vocab, ls_dtype(logits), _stream(logits))
    return dlogits


# ----------------------------------------------------------------------------
# softmax with a learned relative position bias
# ----------------------------------------------------------------------------
def relpos_buckets(num_buckets: int = 32, max_distance: int = 128, bidirectional: bool = True,
                   device="cuda"):
    """The usual bucket map: int32 [2 * max_distance + 1], the bucket of each
    clipped distance -max_distance ... max_distance from query to key.  Near
    distances have buckets of their own, farther ones share them in ratios up
    to max_distance; with ``bidirectional`` half of the buckets are for keys
    after the query, otherwise those keys share bucket 0 (distance 0).

    Found in whole numbers: distance n is past step t of the k wide buckets
    when log(n/e) / log(max_distance/e) * k >= t, that is when
    n^k e^t >= max_distance^t e^k (e: the distances with their own bucket).
    Any other int32 map of this length can be given to the softmax instead."""
    torch = _torch()
    half = num_buckets // 2 if bidirectional else num_buckets
    e = half // 2
    if e < 1 or max_distance <= e:
        raise ValueError("relpos_buckets needs num_buckets >= 4 (2 without bidirectional) and "
                         "max_distance above the number of single distances")
    k = half - e
    side, t = [], 0
    for n in range(max_distance + 1):
        if n < e:
            side.append(n)
            continue
        while t + 1 < k and n ** k * e ** (t + 1) >= max_distance ** (t + 1) * e ** k:
            t += 1
        side.append(e + t)
    after = [half + b for b in side[1:]] if bidirectional else [0] * max_distance
    return torch.tensor(side[::-1] + after, dtype=torch.int32, device=device)


def _relpos(bucket):
    """max_distance of a bucket map."""
    n = bucket.numel()
    if bucket.dim() != 1 or n % 2 == 0 or bucket.dtype != _torch().int32:
        raise ValueError("buckets must be a 1-D int32 tensor of 2 * max_distance + 1 ids")
    return n // 2


def softmax_fw_relpos(scores, table, buckets, mask=None, causal: bool = False, scale=None,
                      out=None):
    """Softmax over the last axis of scale * scores [B,H,Tq,Tk] plus the learned
    bias ``table[buckets[r + R], h]`` of the clipped distance r = j - (i + Tk -
    Tq) in [-R, R], plus an additive mask [B,Tk]; future keys masked when
    ``causal``.  ``table`` is [num_buckets, H] in the scores' dtype, ``buckets``
    int32 [2R + 1] (see relpos_buckets).  ``out`` may be ``scores``."""
    if scores.dim() != 4:
        raise ValueError("scores must be [B, H, Tq, Tk]")
    B, H, Tq, Tk = scores.shape
    dtype = scores.dtype
    if table.dim() != 2:
        raise ValueError("table must be [num_buckets, H]")
    nb, heads = table.shape
    if heads != H or table.dtype != dtype:
        _want("table", table, (nb, H), dtype)
    R = _relpos(buckets)
    if mask is not None and (mask.dtype != dtype or mask.shape != (B, Tk)):
        _want("mask", mask, (B, Tk), dtype)
    if out is None:
        out = _torch().empty_like(scores)
    else:
        _want("out", out, scores.shape, dtype)
    dev = _same_device(scores, table, buckets, mask, out)
    _launch("ls_softmax_fw_relpos", dev, out.data_ptr(), scores.data_ptr(), _ptr(mask),
            table.data_ptr(), buckets.data_ptr(), B, H, Tq, Tk, nb, R, 1 if causal else 0,
            1.0 if scale is None else float(scale), ls_dtype(scores))
    return out


def softmax_relpos_workspace(H: int, max_distance: int, device):
    """A workspace tensor of the size ls_softmax_bw_relpos needs."""
    n = ls_softmax_bw_relpos_workspace_size(H, max_distance)
    return _torch().empty(max(n, 16) // 4, device=device, dtype=_torch().float32)


def softmax_bw_relpos(dout, out_fw, buckets, num_buckets: int, mask=None, causal: bool = False,
                      scale=None, workspace=None, dinp=None, dtable=None):
    """Gradients of ``softmax_fw_relpos``: (dscores, dtable), dtable fp32
    [num_buckets, H] in a fixed summation order.  What ``dout`` and ``out_fw``
    hold at invisible keys never matters; ``dinp`` may be ``dout``."""
    f32 = _torch().float32
    if dout.dim() != 4:
        raise ValueError("dout must be [B, H, Tq, Tk]")
    B, H, Tq, Tk = shape = dout.shape
    dtype = dout.dtype
    if out_fw.shape != shape or out_fw.dtype != dtype:
        _want("out_fw", out_fw, shape, dtype)
    R = _relpos(buckets)
    if mask is not None and (mask.dtype != dtype or mask.shape != (B, Tk)):
        _want("mask", mask, (B, Tk), dtype)
    if workspace is None:
        n = max(ls_softmax_bw_relpos_workspace_size(H, R), 16) // 4
        workspace = dout.new_empty(n, dtype=f32)
    else:
        _workspace("workspace", workspace)
        n = workspace.numel()
    if dinp is None:
        dinp = _torch().empty_like(dout)
    else:
        _want("dinp", dinp, shape, dtype)
    if dtable is None:
        dtable = dout.new_empty((num_buckets, H), dtype=f32)
    else:
        _want("dtable", dtable, (num_buckets, H), f32)
    dev = _same_device(dout, out_fw, buckets, mask, workspace, dinp, dtable)
    _launch("ls_softmax_bw_relpos", dev, dinp.data_ptr(), dtable.data_ptr(), dout.data_ptr(),
            out_fw.data_ptr(), _ptr(mask), buckets.data_ptr(), B, H, Tq, Tk, num_buckets, R,
            1 if causal else 0, 1.0 if scale is None else float(scale), workspace.data_ptr(),
            4 * n, ls_dtype(dout))
    return dinp, dtable


# ----------------------------------------------------------------------------
# per-head norm of queries and keys with the position rotation
# ----------------------------------------------------------------------------
def rope_tables(max_pos: int, rot: int, base: float = 10000.0, device="cuda"):
    """Cosine and sine tables, fp32 [max_pos, rot / 2], of the angles
    position * base^(-2p / rot), computed in float64 and rounded once."""
    torch = _torch()
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and at least 2")
    p = torch.arange(0, rot, 2, device=device, dtype=torch.float64)
    angle = torch.arange(max_pos, device=device, dtype=torch.float64)[:, None] * base ** (-p / rot)
    return angle.cos().float(), angle.sin().float()


def _heads(name, t):
    """Shape and token stride of a [tokens, heads, D] tensor whose heads and
    features are dense (a slice of a packed projection is)."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, D]")
    n, h, d = t.shape
    st, sh, sd = t.stride()
    if (d > 1 and sd != 1) or (h > 1 and sh != d):
        raise ValueError(f"{name} must have dense heads and features")
    if n <= 1 or h == 0:
        return n, h, d, h * d
    if st < h * d:
        raise ValueError(f"{name} must not overlap itself (token stride {st} < {h * d})")
    return n, h, d, st


def _like_heads(name, t, x):
    """Token stride of t, which has to have x's shape and dtype."""
    if t.shape != x.shape or t.dtype != x.dtype:
        raise ValueError(f"{name} must be {x.dtype} of shape {list(x.shape)}, "
                         f"got {t.dtype} of shape {list(t.shape)}")
    return _heads(name, t)[3]


def _both_heads(q, k, gamma_q, gamma_k):
    """(tokens, Hq, Hk, D, token strides of q and k) of the two sides."""
    tokens, Hq, D, qs = _heads("q", q)
    dtype, shape = q.dtype, k.shape
    if len(shape) != 3 or shape[0] != tokens or shape[2] != D or k.dtype != dtype:
        raise ValueError(f"k must be {dtype} of shape [{tokens}, heads, {D}], "
                         f"got {k.dtype} of shape {list(shape)}")
    _, Hk, _, ks = _heads("k", k)
    want = (D,)
    if gamma_q.shape != want or gamma_q.dtype != dtype or \
            gamma_k.shape != want or gamma_k.dtype != dtype:
        _want("gamma_q", gamma_q, want, dtype)
        _want("gamma_k", gamma_k, want, dtype)
    return tokens, Hq, Hk, D, qs, ks


def _rotation(cos, sin, positions, tokens, D):
    """(rot, max_pos) of the rotation tables; (0, 0) without them."""
    torch = _torch()
    if cos is None and sin is None and positions is None:
        return 0, 0
    if cos is None or sin is None or positions is None:
        raise ValueError("cos, sin and positions go together")
    if cos.dim() != 2 or 2 * cos.shape[1] > D:
        raise ValueError(f"cos must be [max_pos, rot / 2] with rot <= {D}")
    max_pos, half = shape = cos.shape
    f32 = torch.float32
    if cos.dtype != f32 or sin.dtype != f32 or sin.shape != shape or \
            positions.dtype != torch.int32 or positions.shape != (tokens,):
        _want("cos", cos, shape, f32)
        _want("sin", sin, shape, f32)
        _want("positions", positions, (tokens,), torch.int32)
    return 2 * half, max_pos


def _one_device(strided, dense):
    """The one device (its index) of all tensors; the dense ones must be contiguous."""
    index = _same_device(*dense)
    for t in strided:
        if t.get_device() != index:
            if not t.is_cuda:
                raise ValueError("tensors must live on a CUDA device (there is no CPU path)")
            raise ValueError(f"tensors on different devices (cuda:{index} and {t.device})")
    return index


def qk_norm_rope_fw(q, k, gamma_q, gamma_k, cos=None, sin=None, positions=None,
                    interleaved: bool = False, eps: float = 1e-6, q_out=None, k_out=None,
                    q_rstd=None, k_rstd=None):
    """RMSNorm of every head of q [tokens, Hq, D] and k [tokens, Hk, D] (gamma_q
    and gamma_k [D]) and, with ``cos`` / ``sin`` (fp32 [max_pos, rot / 2], see
    rope_tables) and ``positions`` (int32 [tokens]), the rotation of the first
    rot features; pairs are (p, p + rot / 2), or neighbours when
    ``interleaved``.  Returns (q_out, k_out, q_rstd, k_rstd), the statistics
    fp32.  Tokens may be strided (slices of a packed projection); the outputs
    may be the inputs (in place, same strides) where q and k do not overlap."""
    f32 = _torch().float32
    tokens, Hq, Hk, D, qs, ks = _both_heads(q, k, gamma_q, gamma_k)
    rot, max_pos = _rotation(cos, sin, positions, tokens, D)
    qos, kos = Hq * D, Hk * D
    if q_out is None:
        q_out = q.new_empty((tokens, Hq, D))
    else:
        qos = _like_heads("q_out", q_out, q)
    if k_out is None:
        k_out = k.new_empty((tokens, Hk, D))
    else:
        kos = _like_heads("k_out", k_out, k)
    if q_rstd is None:
        q_rstd = q.new_empty((tokens, Hq), dtype=f32)
    else:
        _want("q_rstd", q_rstd, (tokens, Hq), f32)
    if k_rstd is None:
        k_rstd = q.new_empty((tokens, Hk), dtype=f32)
    else:
        _want("k_rstd", k_rstd, (tokens, Hk), f32)
    dev = _one_device((q, k, q_out, k_out),
                      (gamma_q, gamma_k, cos, sin, positions, q_rstd, k_rstd))
    _launch("ls_qk_norm_rope_fw", dev, q_out.data_ptr(), k_out.data_ptr(), q_rstd.data_ptr(),
            k_rstd.data_ptr(), q.data_ptr(), k.data_ptr(), gamma_q.data_ptr(),
            gamma_k.data_ptr(), _ptr(cos), _ptr(sin), _ptr(positions), tokens, Hq, Hk, D, rot,
            max_pos, qos, kos, qs, ks, 1 if interleaved else 0, float(eps), ls_dtype(q))
    return q_out, k_out, q_rstd, k_rstd


def qk_norm_rope_workspace(tokens: int, Hq: int, Hk: int, D: int, device):
    """A workspace tensor of the size ls_qk_norm_rope_bw needs."""
    n = ls_qk_norm_rope_bw_workspace_size(tokens, Hq, Hk, D)
    return _torch().empty(max(n, 16) // 4, device=device, dtype=_torch().float32)


def qk_norm_rope_bw(dq_out, dk_out, q, k, gamma_q, gamma_k, q_rstd, k_rstd, cos=None, sin=None,
                    positions=None, interleaved: bool = False, workspace=None, dq=None, dk=None,
                    dgamma_q=None, dgamma_k=None):
    """Gradients of ``qk_norm_rope_fw`` from those of its outputs, its inputs and
    its saved statistics: (dq, dk, dgamma_q, dgamma_k), the gamma gradients
    fp32 [D] in a fixed summation order.  ``dq`` and ``dk`` may be ``dq_out``
    and ``dk_out``, or slices of a packed gradient."""
    f32 = _torch().float32
    tokens, Hq, Hk, D, qs, ks = _both_heads(q, k, gamma_q, gamma_k)
    dqos, dkos = _like_heads("dq_out", dq_out, q), _like_heads("dk_out", dk_out, k)
    if q_rstd.shape != (tokens, Hq) or q_rstd.dtype != f32 or \
            k_rstd.shape != (tokens, Hk) or k_rstd.dtype != f32:
        _want("q_rstd", q_rstd, (tokens, Hq), f32)
        _want("k_rstd", k_rstd, (tokens, Hk), f32)
    rot, max_pos = _rotation(cos, sin, positions, tokens, D)
    if workspace is None:
        n = max(ls_qk_norm_rope_bw_workspace_size(tokens, Hq, Hk, D), 16) // 4
        workspace = q.new_empty(n, dtype=f32)
    else:
        _workspace("workspace", workspace)
        n = workspace.numel()
    dqs, dks = Hq * D, Hk * D
    if dq is None:
        dq = q.new_empty((tokens, Hq, D))
    else:
        dqs = _like_heads("dq", dq, q)
    if dk is None:
        dk = k.new_empty((tokens, Hk, D))
    else:
        dks = _like_heads("dk", dk, k)
    if dgamma_q is None:
        dgamma_q = q.new_empty(D, dtype=f32)
    else:
        _want("dgamma_q", dgamma_q, (D,), f32)
    if dgamma_k is None:
        dgamma_k = q.new_empty(D, dtype=f32)
    else:
        _want("dgamma_k", dgamma_k, (D,), f32)
    dev = _one_device((q, k, dq_out, dk_out, dq, dk),
                      (gamma_q, gamma_k, q_rstd, k_rstd, cos, sin, positions, workspace,
                       dgamma_q, dgamma_k))
    _launch("ls_qk_norm_rope_bw", dev, dq.data_ptr(), dk.data_ptr(), dgamma_q.data_ptr(),
            dgamma_k.data_ptr(), dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(), k.data_ptr(),
            gamma_q.data_ptr(), gamma_k.data_ptr(), q_rstd.data_ptr(), k_rstd.data_ptr(),
            _ptr(cos), _ptr(sin), _ptr(positions), tokens, Hq, Hk, D, rot, max_pos, dqs, dks,
            dqos, dkos, qs, ks, 1 if interleaved else 0, workspace.data_ptr(), 4 * n, ls_dtype(q))
    # a side without heads has no gradient to sum, and the library leaves its pointers alone
    if not Hq:
        dgamma_q.zero_()
    if not Hk:
        dgamma_k.zero_()
    return dq, dk, dgamma_q, dgamma_k


# ----------------------------------------------------------------------------
# global gradient norm and clipping
# ----------------------------------------------------------------------------
_DTYPE = operator.attrgetter("dtype")


def _list_device(name, tensors):
    """The index of the one CUDA device of a list's dense tensors."""
    Tensor = _torch().Tensor
    try:
        devices = set(map(Tensor.get_device, tensors))
        if len(devices) == 1 and all(map(Tensor.is_contiguous, tensors)):
            index = devices.pop()
            if index >= 0:
                return index
    except TypeError:  # something that only looks like a tensor, or none
        for i, t in enumerate(tensors):
            if not hasattr(t, "data_ptr"):
                raise TypeError(f"{name}[{i}] is no tensor but {t!r}") from None
    return _dev(*tensors).index  # says what is wrong


def _each(method, tensors):
    """``t.method()`` of every tensor of a list, as a list."""
    try:
        return list(map(getattr(_torch().Tensor, method), tensors))
    except TypeError:  # something that only looks like a tensor
        return [getattr(t, method)() for t in tensors]


def _grad_lists(grads):
    """(tensors, device index, pointers, element counts, dtypes, and dtype codes
    as a host array) of a list of dense tensors."""
    grads = list(grads)
    if not grads:
        raise ValueError("an empty list has no device: give at least one gradient")
    index = _list_device("grads", grads)
    dtypes = list(map(_DTYPE, grads))
    try:
        codes = array.array("i", map(_DTYPE_CODES.__getitem__, dtypes))
    except KeyError:  # the first call, or an unsupported dtype
        codes = array.array("i", map(ls_dtype, grads))
    return grads, index, _each("data_ptr", grads), _each("numel", grads), dtypes, codes


def _at(a) -> int:
    return a.buffer_info()[0]


def grad_norm_workspace(count: int, device):
    """A workspace tensor of the size ls_grad_norm and ls_grad_clip need for
    ``count`` gradients."""
    n = ls_grad_norm_workspace_size(count)
    return _torch().empty(max(n, 16) // 4, device=device, dtype=_torch().float32)


def _norm_outputs(grads, index, workspace, norm):
    f32 = _torch().float32
    _want("norm", norm, (1,), f32)
    if workspace is None:
        n = ls_grad_norm_workspace_size(len(grads))
        workspace = grads[0].new_empty(max(n, 16) // 4, dtype=f32)
    _workspace("workspace", workspace)
    norm = grads[0].new_empty(1, dtype=f32) if norm is None else norm
    if _same_device(workspace, norm) != index:
        raise ValueError(f"workspace and norm must be on {grads[0].device}")
    return workspace, norm


def grad_norm(grads, workspace=None, norm=None):
    """Global norm sqrt(sum g^2) over a list of contiguous gradients (fp32, fp16
    and bf16 may be mixed), fp32 [1] on their device."""
    grads, index, ptrs, sizes, _, codes = _grad_lists(grads)
    workspace, norm = _norm_outputs(grads, index, workspace, norm)
    ptrs, sizes = array.array("Q", ptrs), array.array("q", sizes)
    _launch("ls_grad_norm", index, _ptr(norm), _at(ptrs), _at(sizes), _at(codes), len(grads),
            _ptr(workspace), workspace.numel() * 4)
    return norm


def _overlap(out, grads, nbytes):
    """Which output (a pointer; None: none) overlaps another output, or a
    gradient that is not its own in place."""
    spans = sorted((p, p + n, i) for i, (p, n) in enumerate(zip(out, nbytes)) if n)
    for (_, end, i), (beg, _, j) in zip(spans, spans[1:]):
        if beg < end:
            return f"out[{max(i, j)}] overlaps out[{min(i, j)}]"
    starts = [s[0] for s in spans]
    for j, (p, n) in enumerate(zip(grads, nbytes)):
        k = bisect.bisect_left(starts, p + n) - 1  # the last output that begins before its end
        if n and out[j] != p and k >= 0 and spans[k][1] > p:
            return f"out[{spans[k][2]}] overlaps grads[{j}]"
    return None


def grad_clip(grads, max_norm: float, out=None, eps: float = 1e-6, workspace=None, norm=None):
    """Multiplies a list of gradients by min(1, max_norm / (norm + eps)), norm
    being ``grad_norm(grads)``; returns (out, norm).  ``out`` None clips in
    place; otherwise it is a list of tensors with the gradients' element counts
    and dtypes, any of which may be its own gradient.  Outputs that overlap one
    another or other entries' gradients are refused."""
    grads, index, ptrs, sizes, dtypes, codes = _grad_lists(grads)
    if out is None:
        out, optrs = grads, ptrs
    else:
        out = list(out)
        if len(out) != len(grads):
            raise ValueError(f"out must hold {len(grads)} tensors, got {len(out)}")
        out_index = _list_device("out", out)
        if _each("numel", out) != sizes or list(map(_DTYPE, out)) != dtypes:
            for i, (o, g) in enumerate(zip(out, grads)):
                _want(f"out[{i}]", o, g.shape, g.dtype)
        if out_index != index:
            raise ValueError(f"out must be on {grads[0].device}")
        optrs = _each("data_ptr", out)
    if len(set(optrs)) < len(out):
        held = [p for p, n in zip(optrs, sizes) if n]
        if len(set(held)) < len(held):
            raise ValueError("a tensor is in out twice")
    workspace, norm = _norm_outputs(grads, index, workspace, norm)
    same = optrs is ptrs
    ptrs, sizes = array.array("Q", ptrs), array.array("q", sizes)
    optrs = ptrs if same else array.array("Q", optrs)
    try:
        _launch("ls_grad_clip", index, _ptr(norm), _at(optrs), _at(ptrs), _at(sizes), _at(codes),
                len(grads), float(max_norm), float(eps), _ptr(workspace), workspace.numel() * 4)
    except LsError as e:
        why = e.status == LS_ERR_INVALID_ARG and \
            _overlap(optrs, ptrs, [n * g.element_size() for n, g in zip(sizes, grads)])
        if why:
            raise ValueError(why) from None
        raise
    return out, norm
