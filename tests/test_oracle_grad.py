"""Pins of oracle/grad64.py (CPU): none uses the oracle to check itself."""
import math

import numpy as np
import pytest
import torch
import torch.nn.functional as F

import lf_workloads as W
from oracle import grad64 as G
from oracle import hsa64 as O

CASES = [dict(H=2, d=64, T=100, block=64, n_cur_frames=2, n_hist=3, n_sink=1, k_f=2, k_b=1),
         dict(H=1, d=64, T=130, block=128, n_cur_frames=1, n_hist=2, n_sink=0, k_f=1, k_b=2),
         dict(H=1, d=64, T=70, block=64, n_cur_frames=3, n_hist=0, n_sink=0, k_f=1, k_b=1, k_c=2)]


def _case(i):
    ci = W.random_small(i, **CASES[i])
    sh = ci.shape
    nqb = sh.n_cur_frames * -(-sh.T // sh.block)
    rng = np.random.default_rng(i)
    pick = lambda n, k: np.stack([np.stack([np.sort(rng.choice(n, k, replace=False))
                                            for _ in range(nqb)]) for _ in range(sh.H)])
    nb = -(-sh.T // sh.block)
    bidx = pick(sh.n_hist * nb, sh.k_f * sh.k_b) if sh.n_hist else None
    cidx = pick(nqb, sh.k_c) if sh.k_c else None
    g = torch.from_numpy(rng.standard_normal(tuple(ci.q.shape)))
    return ci, bidx, cidx, g


def _forward(ci, bidx, cidx, t):
    """Attention output as a function of the float64 leaves t, by SDPA under a token mask that
    comes from Python loops over tokens."""
    sh = ci.shape
    nb, ncur = -(-sh.T // sh.block), sh.n_cur_frames * sh.T
    fr = list(ci.sink_slots) + list(ci.hist_slots)
    outs = []
    for h in range(sh.H):
        keep = torch.zeros(ncur, ncur + len(fr) * sh.T, dtype=torch.bool)
        for i in range(ncur):
            qb = (i // sh.T) * nb + (i % sh.T) // sh.block
            for j in range(ncur):
                keep[i, j] = cidx is None or ((j // sh.T) * nb + (j % sh.T) // sh.block) in cidx[h, qb]
            keep[i, ncur:ncur + sh.n_sink * sh.T] = True
            for j in range(sh.n_hist * sh.T):
                keep[i, ncur + sh.n_sink * sh.T + j] = \
                    ((j // sh.T) * nb + (j % sh.T) // sh.block) in bidx[h, qb]
        k = torch.cat([t["k_cur"][:, h]] + [t["k_cache"][s, :, h] for s in fr])
        v = torch.cat([t["v_cur"][:, h]] + [t["v_cache"][s, :, h] for s in fr])
        outs.append(F.scaled_dot_product_attention(t["q"][None, :, h], k[None], v[None], keep,
                                                   scale=sh.scale)[0])
    return torch.stack(outs, 1)


NAMES = dict(dq="q", dk_cur="k_cur", dv_cur="v_cur", dk_cache="k_cache", dv_cache="v_cache")


def _leaves(ci):
    return {n: getattr(ci, n).double().requires_grad_(True) for n in NAMES.values()}


@pytest.mark.parametrize("i", range(len(CASES)))
def test_attention_gradient_equals_autograd(i):
    ci, bidx, cidx, g = _case(i)
    t = _leaves(ci)
    (_forward(ci, bidx, cidx, t) * g).sum().backward()
    with torch.no_grad():
        r = G.attention_backward(ci.shape, *[t[n] for n in ("q", "k_cur", "v_cur", "k_cache", "v_cache")],
                                 ci.hist_slots, ci.sink_slots, bidx, cidx, g)
    for name, leaf in NAMES.items():
        want = t[leaf].grad if t[leaf].grad is not None else torch.zeros_like(t[leaf])
        assert (r[name]["ref"] - want).abs().max() < 1e-12, name


@pytest.mark.parametrize("i", [0, 2])
def test_attention_gradient_equals_differences(i):
    """Central differences of the oracle of the forward pass along random directions."""
    ci, bidx, cidx, g = _case(i)
    t = {n: getattr(ci, n).double() for n in NAMES.values()}
    r = G.attention_backward(ci.shape, *[t[n] for n in ("q", "k_cur", "v_cur", "k_cache", "v_cache")],
                             ci.hist_slots, ci.sink_slots, bidx, cidx, g)
    rng = np.random.default_rng(7)
    for name, leaf in NAMES.items():
        if not t[leaf].numel():
            continue
        u = torch.from_numpy(rng.standard_normal(tuple(t[leaf].shape)))
        vals = []
        for s in (1e-4, -1e-4):
            p = dict(t, **{leaf: t[leaf] + s * u})
            vals.append(float((_forward(ci, bidx, cidx, p) * g).sum()))
        diff = (vals[0] - vals[1]) / 2e-4
        want = float((r[name]["ref"] * u).sum())
        # third derivatives times h^2 / 6 and the cancellation of values of a few hundred
        assert abs(diff - want) < 1e-5 * (1 + abs(want)), name


def test_forward_oracles_agree():
    ci, bidx, cidx, _ = _case(0)
    o, _ = O.attention(ci.shape, ci.q, ci.k_cur, ci.v_cur, ci.k_cache, ci.v_cache, ci.hist_slots,
                       ci.sink_slots, bidx)
    with torch.no_grad():
        assert np.abs(_forward(ci, bidx, cidx, _leaves(ci)).numpy() - o).max() < 1e-12


def test_rope_by_hand():
    """A head of two pairs turned by the row, one frame of two rows: 2 x 2 rotation matrices."""
    x = torch.randn(1, 2, 1, 4, dtype=torch.float64)
    y = G.rope(x, None, 2, 1, (0, 2, 0), base=100.0)
    for p, f in enumerate((1.0, 0.1)):
        c, s = math.cos(f), math.sin(f)
        a, b = x[0, 1, 0, 2 * p], x[0, 1, 0, 2 * p + 1]
        assert abs(y[0, 1, 0, 2 * p] - (a * c - b * s)) < 1e-15
        assert abs(y[0, 1, 0, 2 * p + 1] - (a * s + b * c)) < 1e-15
    assert torch.equal(y[0, 0], x[0, 0])


@pytest.mark.parametrize("halves", [False, True])
def test_rope_products_depend_on_offsets_only(halves):
    """q.k of turned vectors depends on the difference of their positions on each axis."""
    q = torch.randn(1, 1, 1, 64, dtype=torch.float64).expand(3, 12, 1, 64)
    k = torch.randn(1, 1, 1, 64, dtype=torch.float64).expand(3, 12, 1, 64)
    turn = lambda x, pos: G.rope(x, None, 3, 4, (12, 10, 10), halves=halves, frame_pos=pos)
    a = (turn(q, [5, 6, 7])[:, :, 0] @ turn(k, [5, 6, 7])[0, 0, 0])
    b = (turn(q, [105, 106, 107])[:, :, 0] @ turn(k, [105, 106, 107])[0, 0, 0])
    assert (a - b).abs().max() < 1e-10
    assert (a[0, 0] - a[1, 0]).abs() > 1e-3 and (a[0, 0] - a[0, 1]).abs() > 1e-3


@pytest.mark.parametrize("norm", [None, "head", "row"])
def test_rope_gradient_equals_differences(norm):
    x = torch.randn(2, 6, 3, 64, dtype=torch.float64)
    w = None if norm is None else 1 + 0.1 * torch.randn(64 if norm == "head" else 192, dtype=torch.float64)
    g = torch.randn_like(x)
    args = (2, 3, (12, 10, 9))
    dx, dw = G.rope_backward(x, w, g, *args, norm=norm, halves=True)
    f = lambda x, w: float((G.rope(x, w, *args, norm=norm, halves=True) * g).sum())
    u = torch.randn_like(x)
    assert abs((f(x + 1e-5 * u, w) - f(x - 1e-5 * u, w)) / 2e-5 - float((dx * u).sum())) < 1e-6
    if w is not None:
        u = torch.randn_like(w)
        assert abs((f(x, w + 1e-5 * u) - f(x, w - 1e-5 * u)) / 2e-5 - float((dw * u).sum())) < 1e-6


def test_rope_norm_without_turning_is_rms_norm():
    x = torch.randn(1, 4, 2, 64, dtype=torch.float64)
    w = torch.randn(128, dtype=torch.float64)
    y = G.rope(x, w, 2, 2, (0, 0, 0), norm="row", eps=1e-5)
    assert (y.view(4, 128) - F.rms_norm(x.view(4, 128), (128,), w, 1e-5)).abs().max() < 1e-12
