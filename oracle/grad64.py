"""Gradient of block-sparse attention and rotary positions, in float64, by their definitions.

Attention: which key tokens a query token sees is built token by token from the block lists
(`visible`), and the gradient is the formulas' on dense float64 matrices, one head at a time.
`attention_backward` also returns, per output, the sums that rounding errors are measured by.
Rotary: complex multiplication and autograd.  Works on any torch device.
"""
from __future__ import annotations

from typing import Dict, Optional, Sequence

import torch

__all__ = ["visible", "attention_backward", "rope", "rope_backward"]

F64 = torch.float64


def visible(shape, block_idx, cur_idx, h: int, device) -> torch.Tensor:
    """bool [n_cur, n_cur + (n_sink + n_hist) * T]: the key tokens each query token of head h
    attends to, in the order current chunk, sinks, history."""
    T, B = shape.T, shape.block
    nb = -(-T // B)
    ncur = shape.n_cur_frames * T
    t = torch.arange(ncur, device=device)
    q_blk = t // T * nb + t % T // B
    def chosen(lists, n_blocks, tokens):
        kept = torch.zeros(shape.n_cur_frames * nb, n_blocks, dtype=torch.bool, device=device)
        kept.scatter_(1, torch.as_tensor(lists[h]).long().to(device), True)
        k = torch.arange(tokens, device=device)
        return kept[q_blk][:, k // T * nb + k % T // B]
    ones = lambda n: torch.ones(ncur, n, dtype=torch.bool, device=device)
    cur = chosen(cur_idx, shape.n_cur_frames * nb, ncur) if cur_idx is not None else ones(ncur)
    hist = chosen(block_idx, shape.n_hist * nb, shape.n_hist * T) if shape.n_hist else ones(0)
    return torch.cat([cur, ones(shape.n_sink * T), hist], 1)


def attention_backward(shape, q, k_cur, v_cur, k_cache, v_cache, hist_slots: Sequence[int],
                       sink_slots: Sequence[int], block_idx, cur_idx, dout,
                       out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                       heads: Optional[Sequence[int]] = None) -> Dict[str, Dict[str, torch.Tensor]]:
    """{name: {"ref", "rand", "abs"}} for dq, dk_cur, dv_cur, dk_cache, dv_cache.

    ref: the gradient.  With t the terms of an element's sum (over keys or queries): rand =
    sqrt(sum t^2), abs = sum |t| plus the size of what cancels inside dS.  out and lse: the
    forward pass's rounded results, which the recomputation starts from; without them the
    exact ones.  Frames of the cache that no list names have gradient zero."""
    T, d, ncur = shape.T, shape.d, shape.n_cur_frames * shape.T
    frames = list(sink_slots) + list(hist_slots)
    dev = q.device
    shapes = dict(dq=q, dk_cur=q, dv_cur=q, dk_cache=k_cache, dv_cache=k_cache)
    res = {n: {w: torch.zeros(t.shape, dtype=F64, device=dev) for w in ("ref", "rand", "abs")}
           for n, t in shapes.items()}
    def put(name, w, h, cur, cached):
        res[name + "_cur"][w][:, h] = cur
        if frames:
            res[name + "_cache"][w][frames, :, h] = cached.view(len(frames), T, d)
    for h in (range(shape.H) if heads is None else heads):
        def keys(cur, cache):
            parts = [cur[:, h]]
            if frames:
                parts.append(cache[frames][:, :, h].reshape(-1, d))
            return torch.cat(parts).to(F64)
        k, v = keys(k_cur, k_cache), keys(v_cur, v_cache)
        qh, g = q[:, h].to(F64), dout[:, h].to(F64)
        see = visible(shape, block_idx, cur_idx, h, dev)
        s = (qh @ k.T * shape.scale).masked_fill(~see, float("-inf"))
        m = torch.logsumexp(s, 1) if lse is None else lse[h].to(F64)
        p = torch.where(m[:, None] > -float("inf"), torch.exp(s - m[:, None]), 0.0)
        o = p @ v if out is None else out[:, h].to(F64)
        ds = p * (g @ v.T - (g * o).sum(1, keepdim=True)) * shape.scale
        size = p * (g.abs() @ v.abs().T + (g * o).abs().sum(1, keepdim=True)) * shape.scale
        res["dq"]["ref"][:, h] = ds @ k
        res["dq"]["rand"][:, h] = (ds.square() @ k.square()).sqrt()
        res["dq"]["abs"][:, h] = size @ k.abs()
        for name, w, val in (("dk", "ref", ds.T @ qh), ("dv", "ref", p.T @ g),
                             ("dk", "rand", (ds.square().T @ qh.square()).sqrt()),
                             ("dv", "rand", (p.square().T @ g.square()).sqrt()),
                             ("dk", "abs", size.T @ qh.abs()), ("dv", "abs", p.T @ g.abs())):
            put(name, w, h, val[:ncur], val[ncur:])
    return res


def _positions(n_frames, height, width, frame_pos, device):
    f = torch.as_tensor([int(p) for p in (frame_pos or range(n_frames))], dtype=F64, device=device)
    i = torch.arange(height, dtype=F64, device=device)
    j = torch.arange(width, dtype=F64, device=device)
    return torch.stack(torch.meshgrid(f, i, j, indexing="ij"), -1).view(n_frames, height * width, 3)


def rope(x, weight, height, width, pairs, halves=False, norm=None, base=10000.0, eps=1e-6,
         frame_pos=None):
    """x [frames, T, H, d] in float64 -> normed and turned, differentiable."""
    F, T, H, d = x.shape
    if norm is not None:
        over = 3 if norm == "head" else (2, 3)
        x = x / torch.sqrt(x.square().mean(over, keepdim=True) + eps)
        x = x * (weight if norm == "head" else weight.view(H, d))
    at = _positions(F, height, width, frame_pos, x.device)
    ang = torch.zeros(F, T, d // 2, dtype=F64, device=x.device)
    p = 0
    for axis, n in enumerate(pairs):
        for i in range(n):
            ang[:, :, p] = at[:, :, axis] * float(base) ** (-i / n)
            p += 1
    a, b = (x[..., :d // 2], x[..., d // 2:]) if halves else (x[..., 0::2], x[..., 1::2])
    z = torch.complex(a, b) * torch.polar(torch.ones_like(ang), ang)[:, :, None, :]
    if halves:
        return torch.cat([z.real, z.imag], -1)
    return torch.stack([z.real, z.imag], -1).reshape(x.shape)


def rope_backward(x, weight, dout, *args, **kw):
    """(dx, dweight or None) by autograd through `rope`."""
    x = x.detach().to(F64).requires_grad_(True)
    w = None if weight is None else weight.detach().to(F64).requires_grad_(True)
    (rope(x, w, *args, **kw) * dout.to(F64)).sum().backward()
    return x.grad, None if w is None else w.grad
