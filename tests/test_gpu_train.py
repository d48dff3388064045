"""One attention layer of a chunk, trained: projections -> norm and rotary positions (queries and
keys, into cache slots for an earlier chunk) -> lf_forward_chunk -> gradient of the attention,
cache included -> gradient of positions and norm, back to the projections.  Against float64
autograd through the whole layer (oracle/grad64.py's rotary positions, dense attention under the
lists that the layer chose).

Tolerance.  The layer rounds to bf16 where its tensors are stored or enter a tensor-core product:
rotated queries, rotated keys, P, the output, P and dS of the gradient, its result, and the
projections' gradient: eight roundings, each of at most 2^-8 of what it rounds.  Two of them, in
queries and keys, enter through the exponent: scores of order one have an error of at most
2^-8 (|q| |k| scale summed like independent terms, here near one), so a probability is off by no
more than twice its own share.  Together, as norms of independent errors added up without relying
on their independence: (6 + 2 * 2) * 2^-8 = 3.9 % of the gradient's norm.  Differences of the
float64 layer check the autograd itself.
"""
import math
from types import SimpleNamespace

import pytest
import torch

import block_sparse_attention_46_b200 as lf
from oracle import grad64 as R

pytestmark = pytest.mark.gpu

LIMIT = 10 * 2.0 ** -8
H, D, GRID, FC, FH = 3, 128, (9, 13), 2, 4
T = GRID[0] * GRID[1]
PAIRS = (24, 20, 20)
SLOTS_HIST, SLOTS_SINK, N_SLOTS = [5, 0, 3], [6], 7          # three history frames, one sink


def _shape():
    return SimpleNamespace(H=H, d=D, T=T, block=64, n_cur_frames=FC, n_hist=3, n_sink=1,
                           n_slots=N_SLOTS, k_f=2, k_b=1, scale=1 / math.sqrt(D), k_c=3)


def _inputs():
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    bf = torch.bfloat16
    return dict(cur=rand(FC, T, 3, H, D).to(bf), old=rand(FH, T, 3, H, D).to(bf),
                wq=1 + 0.2 * rand(H * D), wk=1 + 0.2 * rand(H * D),
                grad=rand(FC * T, H, D).to(bf))


def _rope(frames, norm="row"):
    return lf.make_rope(H, D, frames, *GRID, PAIRS if norm else (0, 0, 0), norm=norm)


def _layer(inp, sh):
    """Forward and backward through the library: projections' and weights' gradients, lists."""
    bf, dev = torch.bfloat16, "cuda"
    slots = SLOTS_HIST + SLOTS_SINK
    pos_old, pos_cur = [0, 1, 2, 3], [4, 5]
    k_cache, v_cache = (torch.zeros(N_SLOTS, T, H, D, dtype=bf, device=dev) for _ in range(2))
    lf.lf_rope_frames(_rope(FH), inp["old"][:, :, 1], k_cache, pos_old, inp["wk"], out_slots=slots)
    lf.lf_rope_frames(_rope(FH, None), inp["old"][:, :, 2], v_cache, out_slots=slots)
    q, k, v = (torch.empty(FC, T, H, D, dtype=bf, device=dev) for _ in range(3))
    lf.lf_rope_frames(_rope(FC), inp["cur"][:, :, 0], q, pos_cur, inp["wq"])
    lf.lf_rope_frames(_rope(FC), inp["cur"][:, :, 1], k, pos_cur, inp["wk"])
    lf.lf_rope_frames(_rope(FC, None), inp["cur"][:, :, 2], v)
    q, k, v = (t.view(FC * T, H, D) for t in (q, k, v))
    out, lse = torch.empty_like(q), torch.empty(H, FC * T, device=dev)
    _, nqb, kf, kb = lf.derived(sh)
    bidx = torch.empty(H, nqb, kf * kb, dtype=torch.int32, device=dev)
    cidx = torch.empty(H, nqb, lf.current_blocks(sh), dtype=torch.int32, device=dev)
    lf.lf_forward_chunk(sh, q, k, v, k_cache, v_cache, SLOTS_HIST, SLOTS_SINK, out, lse, bidx,
                        cur_idx_out=cidx)
    dq, dk, dv = (torch.empty_like(q) for _ in range(3))
    dkc, dvc = torch.zeros_like(k_cache), torch.zeros_like(v_cache)
    lf.lf_block_sparse_attn_backward(sh, q, k, v, k_cache, v_cache, SLOTS_HIST, SLOTS_SINK, bidx,
                                     out, inp["grad"], lse, dq, dk, dv, dkc, dvc, cur_idx=cidx)
    dcur, dold = torch.zeros_like(inp["cur"]), torch.zeros_like(inp["old"])
    dw = [torch.empty_like(inp["wq"]) for _ in range(3)]
    fr = lambda t: t.view(FC, T, H, D)
    lf.lf_rope_frames_backward(_rope(FC), inp["cur"][:, :, 0], fr(dq), dcur[:, :, 0], pos_cur, inp["wq"], dw[0])
    lf.lf_rope_frames_backward(_rope(FC), inp["cur"][:, :, 1], fr(dk), dcur[:, :, 1], pos_cur, inp["wk"], dw[1])
    lf.lf_rope_frames_backward(_rope(FC, None), None, fr(dv), dcur[:, :, 2])
    lf.lf_rope_frames_backward(_rope(FH), inp["old"][:, :, 1], dkc, dold[:, :, 1], pos_old, inp["wk"], dw[2],
                               out_slots=slots)
    lf.lf_rope_frames_backward(_rope(FH, None), None, dvc, dold[:, :, 2], out_slots=slots)
    return dict(cur=dcur, old=dold, wq=dw[0], wk=dw[1] + dw[2]), out, bidx, cidx


def _layer64(x, sh, bidx, cidx):
    """The layer in float64, differentiable: its output [tokens, H, d]."""
    turn = lambda t, w, pos: R.rope(t, w, *GRID, PAIRS, norm="row", frame_pos=pos)
    q = turn(x["cur"][:, :, 0], x["wq"], [4, 5]).reshape(FC * T, H, D)
    k_old = turn(x["old"][:, :, 1], x["wk"], [0, 1, 2, 3])
    # rows of `old` are history frames 0..2, then the sink; keys are current, sink, history
    order = [3, 0, 1, 2]
    k = torch.cat([turn(x["cur"][:, :, 1], x["wk"], [4, 5]).reshape(FC * T, H, D),
                   k_old[order].reshape(-1, H, D)])
    v = torch.cat([x["cur"][:, :, 2].reshape(FC * T, H, D), x["old"][:, :, 2][order].reshape(-1, H, D)])
    outs = []
    for h in range(H):
        see = R.visible(sh, bidx, cidx, h, q.device)
        s = (q[:, h] @ k[:, h].T * sh.scale).masked_fill(~see, float("-inf"))
        outs.append(torch.softmax(s, 1) @ v[:, h])
    return torch.stack(outs, 1)


def test_layer_gradient(gpu_lib):
    inp, sh = _inputs(), _shape()
    got, out, bidx, cidx = _layer(inp, sh)
    torch.cuda.synchronize()
    assert lf.lf_device_status(True) == 0
    x = {n: inp[n].double().requires_grad_(True) for n in ("cur", "old", "wq", "wk")}
    ref = _layer64(x, sh, bidx, cidx)
    assert float((out.double() - ref.detach()).norm() / ref.detach().norm()) < LIMIT
    (ref * inp["grad"].double()).sum().backward()
    for n, leaf in x.items():
        off = float((got[n].double() - leaf.grad).norm() / leaf.grad.norm())
        assert off < LIMIT, f"{n}: {off:.4f}"
    # the old queries and nothing else of `old` is unused
    assert bool((got["old"][:, :, 0] == 0).all()) and bool((got["old"][:, :, 1:] != 0).any())


def test_layer_gradient_equals_differences(gpu_lib):
    """The float64 gradient that the test above compares with, along random directions; and the
    library's, whose error along a direction is at most that of its norm."""
    inp, sh = _inputs(), _shape()
    got, _, bidx, cidx = _layer(inp, sh)
    x = {n: inp[n].double() for n in ("cur", "old", "wq", "wk")}
    loss = lambda y: float((_layer64(y, sh, bidx, cidx) * inp["grad"].double()).sum())
    g = torch.Generator(device="cuda").manual_seed(9)
    for n in x:
        u = torch.rand(x[n].shape, generator=g, device="cuda", dtype=torch.float64)
        u *= got[n].double()                                   # uphill, the larger entries more
        u /= u.norm()
        diff = (loss(dict(x, **{n: x[n] + 1e-4 * u})) - loss(dict(x, **{n: x[n] - 1e-4 * u}))) / 2e-4
        lib = float((got[n].double() * u).sum())
        assert abs(lib - diff) <= LIMIT * float(got[n].double().norm()) + 1e-4 * abs(diff), n
