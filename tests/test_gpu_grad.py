"""lf_block_sparse_attn_backward against oracle/grad64.py on the same bf16 inputs.

Tolerances, from the arithmetic of the operator.  An element is a sum of terms t (over keys or
queries), P and dS enter the products rounded to bf16 (half a step: 2^-8 of the term) and the
sum is rounded to bf16 once (2^-8 of the value); scores, dP and sums are fp32, whose errors
stay below 2^-14 of the sizes involved (d + a few hundred additions of half a step, 2^-24
each, times scores of a few tens in the exponent).  So for every element
    |err| <= 2^-8 |ref| + (2^-8 + 2^-14) sum |t|,
and, the roundings being independent with zero mean, over a tensor
    ||err|| <= 2^-8 sqrt(||ref||^2 + ||rand||^2) + 2^-14 ||sum |t|||,  rand = sqrt(sum t^2),
where a uniform rounding error would reach 1 / sqrt(3) of the first term.
An exponential below fp32's normal numbers is zero (2^-126, off by less than itself), and so
is a product: at most 2^13 such terms here, times |dP - D| < 2^11 (128 products of values under
4 and 4), |q| < 2^8 and scale < 1/4 in a term of dk, the largest, so FLUSH = 2^-96.
"""
from dataclasses import replace

import numpy as np
import pytest
import torch

import block_sparse_attention_46_b200 as lf
import lf_workloads as W
from oracle import grad64 as R
from tests import gpu_helpers as G

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -8
FP32 = 2.0 ** -14
FLUSH = 2.0 ** -96
LF_ERR_BAD_INDEX = 6


def check(name, got, r):
    err = got.to(torch.float64) - r["ref"]
    assert torch.isfinite(err).all(), f"{name}: not finite"
    over = err.abs() - (STEP * r["ref"].abs() + (STEP + FP32) * r["abs"] + FLUSH)
    assert float(over.max()) <= 0, f"{name}: an element is off by {float(over.max()):.3e} too much"
    lim = STEP * (r["ref"].norm() ** 2 + r["rand"].norm() ** 2).sqrt() + FP32 * r["abs"].norm()
    assert float(err.norm()) <= float(lim), f"{name}: norm {float(err.norm()):.3e} > {float(lim):.3e}"


def lists(sh, seed, spread=1.0):
    """Random ascending block lists; spread < 1 draws from the first blocks only, so that some
    key blocks are in every list and others in none."""
    rng = np.random.default_rng(seed)
    nb, nqb, kf, kb = lf.derived(sh)
    def pick(n, k):
        m = max(k, int(round(n * spread)))
        return torch.from_numpy(np.stack([np.stack([np.sort(rng.choice(m, k, replace=False))
                                                    for _ in range(nqb)])
                                          for _ in range(sh.H)]).astype(np.int32)).cuda()
    kc = lf.current_blocks(sh)
    return (pick(sh.n_hist * nb, kf * kb) if sh.n_hist else None,
            pick(nqb, kc) if kc else None)


def forward(ci, t, bidx, cidx):
    sh = ci.shape
    out, lse = torch.empty_like(t["q"]), torch.empty(sh.H, t["q"].shape[0], device="cuda")
    lf.lf_block_sparse_attn(sh, t["q"], t["k_cur"], t["v_cur"], t["k_cache"], t["v_cache"],
                            ci.hist_slots, ci.sink_slots, bidx, out, lse, cur_idx=cidx)
    return out, lse


def dout_for(ci, seed=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(ci.q.shape, generator=g, device="cuda").to(torch.bfloat16)


def backward(ci, t, bidx, cidx, out, dout, lse, cache=True, workspace=None, stream=None):
    """All gradients; outputs start as NaN (current chunk) and 7 (cache: slots that no list
    names must keep it)."""
    g = {n: torch.full_like(t["q"], float("nan")) for n in ("dq", "dk_cur", "dv_cur")}
    for n in ("dk_cache", "dv_cache"):
        g[n] = torch.full_like(t["k_cache"], 7.0) if cache else None
    lf.lf_block_sparse_attn_backward(
        ci.shape, t["q"], t["k_cur"], t["v_cur"], t["k_cache"], t["v_cache"], ci.hist_slots,
        ci.sink_slots, bidx, out, dout, lse, g["dq"], g["dk_cur"], g["dv_cur"], g["dk_cache"],
        g["dv_cache"], workspace=workspace, stream=stream, cur_idx=cidx)
    return g


def run_case(ci, seed=0, cache=True, spread=1.0):
    t = G.to_dev(ci)
    bidx, cidx = lists(ci.shape, seed, spread)
    out, lse = forward(ci, t, bidx, cidx)
    dout = dout_for(ci)
    g = backward(ci, t, bidx, cidx, out, dout, lse, cache)
    torch.cuda.synchronize()
    assert lf.lf_device_status(True) == 0
    r = R.attention_backward(ci.shape, t["q"], t["k_cur"], t["v_cur"], t["k_cache"], t["v_cache"],
                             ci.hist_slots, ci.sink_slots, bidx, cidx, dout, out, lse)
    for n in ("dq", "dk_cur", "dv_cur"):
        check(n, g[n], r[n])
    if cache:
        listed = list(ci.sink_slots) + list(ci.hist_slots)
        others = [s for s in range(ci.shape.n_slots) if s not in listed]
        for n in ("dk_cache", "dv_cache"):
            if listed:
                check(n, g[n][listed], {w: x[listed] for w, x in r[n].items()})
            assert bool((g[n][others] == 7).all()), f"{n}: a slot outside the lists changed"
    return ci, t, bidx, cidx, out, dout, lse, g


def small(seed, **kw):
    base = dict(H=2, d=64, T=100, block=64, n_cur_frames=2, n_hist=3, n_sink=1, k_f=2, k_b=1)
    base.update(kw)
    return W.random_small(seed, **base)


CASES = {
    "ragged": dict(),
    "d128": dict(d=128),
    "one_token": dict(T=1, n_cur_frames=1, n_hist=0, n_sink=0),
    "one_token_frames": dict(T=1, n_cur_frames=3, n_hist=4, n_sink=2, k_f=3),
    "below_block": dict(T=40, n_cur_frames=3, k_f=1),
    "whole_blocks": dict(T=256, n_cur_frames=1, n_sink=0, k_f=2, k_b=2),
    "block_minus_one": dict(T=127, d=128, k_f=3, k_b=2),
    "block_plus_one": dict(T=129, d=128, k_f=3, k_b=2),
    "b128": dict(block=128, T=300, d=128, k_f=2, k_b=2),
    "b128_ragged": dict(block=128, T=130, k_f=3, k_b=2),
    "b128_short": dict(block=128, T=50, d=128),
    "odd_blocks": dict(T=300, H=5, n_cur_frames=3, k_f=2, k_b=3),
    "no_history": dict(T=300, n_hist=0, d=128),
    "current_alone": dict(T=500, n_hist=0, n_sink=0),
    "sinks_many": dict(T=200, n_sink=4, n_hist=2, d=128),
    "long": dict(T=1000, H=1, n_cur_frames=2, n_hist=6, k_f=4, k_b=7, d=128),
    "one_head_many_frames": dict(T=64, H=1, n_hist=40, k_f=20, k_b=1, n_sink=9),
    "sparse_current": dict(T=200, n_cur_frames=3, k_c=4),
    "sparse_current_alone": dict(T=300, n_cur_frames=3, n_hist=0, n_sink=0, k_c=5, d=128),
    "sparse_current_one": dict(T=40, n_cur_frames=4, n_hist=0, n_sink=0, k_c=1),
    "sparse_current_b128": dict(T=300, block=128, n_cur_frames=3, k_c=3, d=128),
}


@pytest.mark.parametrize("name", list(CASES))
def test_gradient_matches_definition(gpu_lib, name):
    run_case(small(100 + list(CASES).index(name), **CASES[name]))


@pytest.mark.parametrize("name", ["ragged", "b128", "sparse_current", "long"])
def test_gradient_without_cache(gpu_lib, name):
    """A detached cache: the same current-chunk gradients, bit for bit."""
    ci, t, bidx, cidx, out, dout, lse, g = run_case(small(7, **CASES[name]), 7)
    h = backward(ci, t, bidx, cidx, out, dout, lse, cache=False)
    for n in ("dq", "dk_cur", "dv_cur"):
        assert torch.equal(g[n], h[n]), n


@pytest.mark.parametrize("block", [64, 128])
def test_blocks_in_every_list_and_in_none(gpu_lib, block):
    """Lists from the first blocks only: key tiles that all queries attend to, and tiles whose
    gradient is zero."""
    ci = small(31, T=400, H=2, block=block, n_hist=6, n_sink=0, k_f=2, k_b=2, d=128)
    *_, g = run_case(ci, 3, spread=0.3)
    last = ci.hist_slots[-1]
    for n in ("dk_cache", "dv_cache"):
        assert bool((g[n][last] == 0).all()), f"{n}: a frame that no query attends to"


def test_gradient_through_the_layer(gpu_lib):
    """lf_forward_chunk's own lists, output and log-normaliser into the gradient."""
    ci = small(8, T=300, H=3, d=128, n_cur_frames=2, n_hist=5, n_sink=1, k_f=3, k_b=2, k_c=4)
    t = G.to_dev(ci)
    out, lse, bidx, cidx = G.gpu_forward(ci, t, with_cur=True)
    dout = dout_for(ci)
    g = backward(ci, t, bidx, cidx, out, dout, lse)
    r = R.attention_backward(ci.shape, t["q"], t["k_cur"], t["v_cur"], t["k_cache"], t["v_cache"],
                             ci.hist_slots, ci.sink_slots, bidx, cidx, dout, out, lse)
    for n in ("dq", "dk_cur", "dv_cur"):
        check(n, g[n], r[n])


@pytest.mark.parametrize("name", ["p480", "large_b128"])
def test_full_size_one_head(gpu_lib, name):
    """The 480p chunk and a 128-token-block chunk of the large model, checked on two heads."""
    base = W.p480(0) if name == "p480" else None
    if base is None:
        sh = replace(W.large_shape(), H=4, n_hist=12, n_slots=12)
        base = W.random_small(5, H=4, d=128, T=sh.T, block=128, n_cur_frames=3, n_hist=12,
                              n_sink=1, k_f=8, k_b=5)
    ci = base
    t = G.to_dev(ci)
    bidx, cidx = lists(ci.shape, 2)
    out, lse = forward(ci, t, bidx, cidx)
    dout = dout_for(ci)
    g = backward(ci, t, bidx, cidx, out, dout, lse)
    heads = [0, ci.shape.H - 1]
    r = R.attention_backward(ci.shape, t["q"], t["k_cur"], t["v_cur"], t["k_cache"], t["v_cache"],
                             ci.hist_slots, ci.sink_slots, bidx, cidx, dout, out, lse, heads)
    fr = list(ci.sink_slots) + list(ci.hist_slots)
    for n in ("dq", "dk_cur", "dv_cur"):
        check(n, g[n][:, heads], {w: x[:, heads] for w, x in r[n].items()})
    for n in ("dk_cache", "dv_cache"):
        check(n, g[n][fr][:, :, heads], {w: x[fr][:, :, heads] for w, x in r[n].items()})
    assert lf.lf_device_status(True) == 0


def test_repeatable(gpu_lib):
    """The same bits on every call, also with other work on the GPU and a used workspace."""
    ci = small(9, T=700, H=3, d=128, n_hist=6, k_f=4, k_b=5, n_cur_frames=3)
    t = G.to_dev(ci)
    bidx, cidx = lists(ci.shape, 4)
    out, lse = forward(ci, t, bidx, cidx)
    dout = dout_for(ci)
    ws = torch.full((lf.lf_attn_backward_workspace_size(ci.shape),), 255, dtype=torch.uint8,
                    device="cuda")
    first = backward(ci, t, bidx, cidx, out, dout, lse, workspace=ws)
    for _ in range(4):
        again = backward(ci, t, bidx, cidx, out, dout, lse, workspace=ws)
        for n, x in first.items():
            assert torch.equal(x, again[n]), n


def test_invalid_lists_are_dropped(gpu_lib):
    """A list with a bad id is dropped for its tile, as in the forward pass, and reported; rows
    left without any key get zero gradients and give none."""
    ci = small(10, T=64, H=2, n_cur_frames=4, n_hist=0, n_sink=0, k_c=2, d=128)
    t = G.to_dev(ci)
    _, cidx = lists(ci.shape, 4)
    cidx[1, 2, 0] = 99                                    # query blocks 2, 3 of head 1
    out, lse = forward(ci, t, None, cidx)
    assert lf.lf_device_status(True) == LF_ERR_BAD_INDEX
    assert bool((lse[1, 128:] == float("-inf")).all())
    dout = dout_for(ci)
    g = backward(ci, t, None, cidx, out, dout, lse)
    assert lf.lf_device_status(True) == LF_ERR_BAD_INDEX
    assert bool((g["dq"][128:, 1] == 0).all())
    cidx[1, 2] = cidx[1, 3] = torch.tensor([0, 1])        # any list: those rows' P is zero
    r = R.attention_backward(ci.shape, t["q"], t["k_cur"], t["v_cur"], t["k_cache"], t["v_cache"],
                             [], [], None, cidx, dout, out, lse)
    for n in ("dq", "dk_cur", "dv_cur"):
        check(n, g[n], r[n])


def test_far_scores(gpu_lib):
    """Scores of hundreds: one key per row carries all probability, the others underflow."""
    ci = small(11, T=200, H=2, d=128, n_hist=3, k_f=2, k_b=2)
    ci.q.mul_(24)
    run_case(ci)


def test_captured_and_replayed(gpu_lib):
    """Captured on a side stream with its own workspace, replayed with other inputs, beside an
    eager call on the current stream."""
    ci = small(12, T=300, H=2, d=128, n_hist=4, k_f=2, k_b=3)
    t = G.to_dev(ci)
    bidx, cidx = lists(ci.shape, 1)
    out, lse = forward(ci, t, bidx, cidx)
    dout = dout_for(ci)
    want = backward(ci, t, bidx, cidx, out, dout, lse)
    static = dout.clone()
    size = lf.lf_attn_backward_workspace_size(ci.shape)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    backward(ci, t, bidx, cidx, out, static, lse, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = backward(ci, t, bidx, cidx, out, static, lse, workspace=ws)
    static.copy_(dout_for(ci, 77))
    graph.replay()
    eager = backward(ci, t, bidx, cidx, out, static, lse)
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(g[n], eager[n]), n
        assert n.endswith("cache") or not torch.equal(g[n], want[n])
    static.copy_(dout)
    graph.replay()
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(g[n], want[n]), n


def test_two_streams_at_once(gpu_lib):
    """Two calls on two streams, each with the workspace that the binding takes from the
    stream's own memory."""
    cis = [small(13 + i, T=500, H=4, d=128, n_hist=4, k_f=3, k_b=4) for i in range(2)]
    jobs = []
    for ci in cis:
        t = G.to_dev(ci)
        bidx, cidx = lists(ci.shape, 1)
        out, lse = forward(ci, t, bidx, cidx)
        dout = dout_for(ci)
        jobs.append((ci, t, bidx, cidx, out, dout, lse, backward(ci, t, bidx, cidx, out, dout, lse)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cis]
    got = []
    for s, (ci, t, bidx, cidx, out, dout, lse, _) in zip(streams, jobs):
        with torch.cuda.stream(s):
            got.append(backward(ci, t, bidx, cidx, out, dout, lse, stream=s))
    torch.cuda.synchronize()
    for g, job in zip(got, jobs):
        for n, x in job[-1].items():
            assert torch.equal(g[n], x), n


def test_refusals(gpu_lib):
    ci = small(15, T=100)
    t = G.to_dev(ci)
    bidx, cidx = lists(ci.shape, 0)
    out, lse = forward(ci, t, bidx, cidx)
    dout = dout_for(ci)
    with pytest.raises(ValueError):
        backward(ci, t, bidx, cidx, out, dout.float(), lse)
    with pytest.raises(ValueError):
        backward(ci, t, bidx, cidx, out, dout[:-1], lse)
    with pytest.raises(ValueError):
        backward(ci, t, bidx, cidx, out, dout.cpu(), lse)
    with pytest.raises(ValueError):
        backward(ci, t, bidx[:, :-1], cidx, out, dout, lse)
    with pytest.raises(ValueError):
        backward(ci, t, bidx, cidx, out, dout, lse[:, :-1])
    with pytest.raises(lf.LfError):
        backward(ci, t, bidx, cidx, out, dout, lse,
                 workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    twice = replace(ci, hist_slots=[ci.hist_slots[0]] * len(ci.hist_slots))
    with pytest.raises(lf.LfError):                       # two gradients into one slot
        backward(twice, t, bidx, cidx, out, dout, lse)
    g = backward(twice, t, bidx, cidx, out, dout, lse, cache=False)
    assert torch.isfinite(g["dq"].float()).all()


def test_stalled_wait_times_out_and_context_recovers(gpu_lib):
    """The bounded waits, made to run out without a GPU fault: the first CTA's own tiles never
    arrive, it gives up after 20 ms, and the next call is right."""
    ci = small(16, T=200, H=2, d=128)
    t = G.to_dev(ci)
    bidx, cidx = lists(ci.shape, 0)
    out, lse = forward(ci, t, bidx, cidx)
    dout = dout_for(ci)
    assert lf.lf_device_status(True) == 0
    try:
        lf.lf_debug_configure(wait_limit_ns=20_000_000, stall=True)
        backward(ci, t, bidx, cidx, out, dout, lse)
        torch.cuda.synchronize()
    finally:
        lf.lf_debug_configure()
    assert lf.lf_device_status(True) == 4                 # LF_ERR_TIMEOUT
    run_case(ci)


def test_detached_dense_chunk_makes_no_block_boxes(gpu_lib):
    """Without lists of query blocks (a dense chunk, no gradient into the cache) the preparation
    writes the rows in token order only: 512 bytes per 64 of them, beside the key plans."""
    ci = small(17, T=300, H=4)
    t = G.to_dev(ci)
    bidx, _ = lists(ci.shape, 0)
    out, lse = forward(ci, t, bidx, None)
    ws = torch.full((lf.lf_attn_backward_workspace_size(ci.shape),), 255, dtype=torch.uint8,
                    device="cuda")
    backward(ci, t, bidx, None, out, dout_for(ci), lse, cache=False, workspace=ws)
    sh = ci.shape
    nb, nqb, kf, kb = lf.derived(sh)
    tiles = -(-nqb // 2)
    plans = 4 * sh.H * tiles * (1 + sh.n_sink * nb + 2 * kf * kb) + 4
    dense = sh.H * 2 * -(-sh.n_cur_frames * sh.T // 128) * 512
    assert int((ws != 255).sum()) <= plans + dense


@pytest.mark.parametrize("kind", ["dense", "sink", "history", "current"])
def test_stalled_key_tiles_time_out(gpu_lib, kind):
    """The waits of the dk, dv pass made to run out: a key tile's own rows never arrive.  CTAs
    are the query tiles, then the key tiles: dense current chunk, sinks, those with lists."""
    ci = small(18, T=200, H=2, d=128, k_c=3 if kind == "current" else 0)
    sh = ci.shape
    t = G.to_dev(ci)
    bidx, cidx = lists(sh, 0)
    out, lse = forward(ci, t, bidx, cidx)
    dout = dout_for(ci)
    nb, nqb, _, _ = lf.derived(sh)
    per_frame = -(-sh.T // 128)
    dense = 0 if kind == "current" else -(-sh.n_cur_frames * sh.T // 128) * sh.H
    first = -(-nqb // 2) * sh.H
    lists_at = first + dense + sh.n_sink * per_frame * sh.H
    if kind == "history":                                 # the first tile that a list names
        block = int(bidx[0].min())
        cta = lists_at + block // nb * per_frame + block % nb // 2
    elif kind == "current":
        block = int(cidx[0].min())
        cta = lists_at + block // nb * per_frame + block % nb // 2
    else:
        cta = first + (dense if kind == "sink" else 0)
    assert lf.lf_device_status(True) == 0
    try:
        lf.lf_debug_configure(wait_limit_ns=20_000_000, stall=cta + 1)
        backward(ci, t, bidx, cidx, out, dout, lse)
        torch.cuda.synchronize()
    finally:
        lf.lf_debug_configure()
    assert lf.lf_device_status(True) == 4                 # LF_ERR_TIMEOUT
    run_case(ci)


def test_dropped_history_beside_a_valid_current_list(gpu_lib, monkeypatch):
    """A bad history id drops the history of its query tile (two blocks of 64) and nothing else:
    the current-chunk lists stay, and the cache's gradient leaves those queries out."""
    ci = small(19, T=100, H=2, d=128, n_hist=4, n_sink=1, k_f=2, k_b=2, k_c=2)
    sh = ci.shape
    t = G.to_dev(ci)
    bidx, cidx = lists(sh, 5)
    good = bidx.clone()
    bidx[1, 2, -1] = 4 * 2                                # one past the last block: blocks 2, 3
    out, lse = forward(ci, t, bidx, cidx)
    assert lf.lf_device_status(True) == LF_ERR_BAD_INDEX
    dout = dout_for(ci)
    g = backward(ci, t, bidx, cidx, out, dout, lse)
    assert lf.lf_device_status(True) == LF_ERR_BAD_INDEX
    visible = R.visible

    def without(shape, block_idx, cur_idx, h, device):
        see = visible(shape, block_idx, cur_idx, h, device)
        if h == 1:
            see[100:, 200 + 100:] = False                 # frame 1: query blocks 2 and 3
        return see

    monkeypatch.setattr(R, "visible", without)
    r = R.attention_backward(sh, t["q"], t["k_cur"], t["v_cur"], t["k_cache"], t["v_cache"],
                             ci.hist_slots, ci.sink_slots, good, cidx, dout, out, lse)
    listed = list(ci.sink_slots) + list(ci.hist_slots)
    for n in ("dq", "dk_cur", "dv_cur"):
        check(n, g[n], r[n])
    for n in ("dk_cache", "dv_cache"):
        check(n, g[n][listed], {w: x[listed] for w, x in r[n].items()})


def test_cache_gradient_through_the_layer(gpu_lib):
    """The cache's gradient under the lists that lf_forward_chunk chose, and its status."""
    ci = small(20, T=300, H=3, d=128, n_cur_frames=2, n_hist=5, n_sink=1, k_f=3, k_b=2, k_c=4)
    t = G.to_dev(ci)
    out, lse, bidx, cidx = G.gpu_forward(ci, t, with_cur=True)
    dout = dout_for(ci)
    g = backward(ci, t, bidx, cidx, out, dout, lse)
    torch.cuda.synchronize()
    assert lf.lf_device_status(True) == 0
    r = R.attention_backward(ci.shape, t["q"], t["k_cur"], t["v_cur"], t["k_cache"], t["v_cache"],
                             ci.hist_slots, ci.sink_slots, bidx, cidx, dout, out, lse)
    listed = list(ci.sink_slots) + list(ci.hist_slots)
    for n in ("dk_cache", "dv_cache"):
        check(n, g[n][listed], {w: x[listed] for w, x in r[n].items()})


def _same_bits(a, b):
    return (a.view(torch.int16) == b.view(torch.int16)).all(-1)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_reach_of_a_bad_gradient_row(gpu_lib, value):
    """An infinity or NaN in one row of dout reaches that query's tile (two blocks of 64) in dq and
    the key tiles (128 rows of a frame) that its block attends to, and nothing further: every
    other gradient keeps its bits."""
    ci = small(21, T=300, H=2, d=128, n_cur_frames=2, n_hist=6, n_sink=0, k_f=1, k_b=2, k_c=2)
    sh = ci.shape
    t = G.to_dev(ci)
    bidx, cidx = lists(sh, 6)
    out, lse = forward(ci, t, bidx, cidx)
    dout = dout_for(ci)
    want = backward(ci, t, bidx, cidx, out, dout, lse)
    nb = lf.derived(sh)[0]
    qb, row = nb + 1, sh.T + 64 + 10                      # second block of the second frame
    dout[row, 1, 3] = value
    got = backward(ci, t, bidx, cidx, out, dout, lse)
    assert bool(got["dq"][row, 1].isnan().any())
    frame, blk = torch.arange(2 * sh.T) // sh.T, torch.arange(2 * sh.T) % sh.T // 64
    tile = (frame * nb + blk) // 2 == qb // 2
    clean = torch.ones(2 * sh.T, sh.H, dtype=torch.bool)
    clean[tile, 1] = False
    assert bool(_same_bits(got["dq"], want["dq"]).cpu()[clean].all())

    def check_keys(names, chosen, n_frames, rows):
        """chosen: block ids of the row's list; rows: gradient rows in frame order."""
        bad = torch.zeros(n_frames * sh.T, dtype=torch.bool)
        for g in chosen:
            f, b = g // nb, g % nb
            bad[f * sh.T + b // 2 * 128:f * sh.T + min(sh.T, b // 2 * 128 + 128)] = True
        assert not bool(bad.all())
        for n in names:
            x, y = rows(got[n]), rows(want[n])
            assert bool(_same_bits(x, y).cpu()[~bad, 1].all()) and bool(_same_bits(x, y)[:, 0].all()), n
            assert bool(x[:, 1].isfinite().logical_not().any()), n

    check_keys(("dk_cur", "dv_cur"), cidx[1, qb].tolist(), 2, lambda x: x)
    check_keys(("dk_cache", "dv_cache"), bidx[1, qb].tolist(), 6,
               lambda x: x[list(ci.hist_slots)].reshape(-1, sh.H, sh.d))


@pytest.mark.parametrize("name", ["k_cache", "v_cache"])
def test_reach_of_a_bad_key_row(gpu_lib, name):
    """A NaN in one cached key or value row reaches the query tiles whose plan holds its block and
    the gradients of its own key tile, and nothing further (out and lse of the clean pass)."""
    ci = small(22, T=300, H=2, d=128, n_cur_frames=2, n_hist=6, n_sink=0, k_f=1, k_b=2, k_c=2)
    sh = ci.shape
    t = G.to_dev(ci)
    bidx, cidx = lists(sh, 7)
    out, lse = forward(ci, t, bidx, cidx)
    dout = dout_for(ci)
    want = backward(ci, t, bidx, cidx, out, dout, lse)
    nb, nqb, _, _ = lf.derived(sh)
    bad = int(bidx[1, 4, 0])
    slot, at = ci.hist_slots[bad // nb], bad % nb * 64 + 5
    t[name][slot, at, 1, 2] = float("nan")
    got = backward(ci, t, bidx, cidx, out, dout, lse)
    holds = (bidx[1] == bad).any(-1).cpu()
    tiles = {q // 2 for q in range(nqb) if holds[q]}
    assert len(tiles) < -(-nqb // 2)
    tok = torch.arange(2 * sh.T)
    qb = tok // sh.T * nb + tok % sh.T // 64
    clean = torch.ones(2 * sh.T, sh.H, dtype=torch.bool)
    clean[torch.tensor([int(x) // 2 in tiles for x in qb]), 1] = False
    assert bool(_same_bits(got["dq"], want["dq"]).cpu()[clean].all())
    assert bool(got["dq"][:, 1].isnan().any())
    for n in ("dk_cur", "dv_cur"):
        assert bool(_same_bits(got[n], want[n]).all()), n
    clean = torch.ones(sh.n_slots, sh.T, sh.H, dtype=torch.bool)
    clean[slot, at // 128 * 128:at // 128 * 128 + 128, 1] = False
    for n in ("dk_cache", "dv_cache"):
        assert bool(_same_bits(got[n], want[n]).cpu()[clean].all()), n


@pytest.mark.parametrize("bad", [dict(d=0), dict(d=96), dict(block=0), dict(block=32), dict(H=0)])
def test_unsupported_shapes_are_library_errors(gpu_lib, bad):
    """Shapes that the library refuses are its errors (or the binding's, for tensors that do not
    fit them), with d or block zero too."""
    ci = small(15, T=100)
    t = G.to_dev(ci)
    bidx, cidx = lists(ci.shape, 0)
    out, lse = forward(ci, t, bidx, cidx)
    with pytest.raises(lf.LfError if 0 in (bad.get("d"), bad.get("block")) else ValueError):
        backward(replace(ci, shape=replace(ci.shape, **bad)), t, bidx, cidx, out, dout_for(ci), lse)


def test_slots_past_32_bits(gpu_lib):
    """Frames in slots whose elements lie past 2^31 (and 2^32 bytes) give the bits of the same
    frames in the first slots: rotation into and out of them, the attention, its gradient."""
    T, H, d, grid = 1560, 12, 128, (30, 52)
    far, n_far = [899, 897, 898], 900
    assert far[1] * T * H * d > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(2)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    old, cur, grad = rand(3, T, 3, H, d), rand(T, 3, H, d), rand(T, H, d)
    weight = 1 + 0.1 * torch.randn(H * d, generator=g, device="cuda")
    rope = lf.make_rope(H, d, 3, *grid, (24, 20, 20), norm="row")
    bidx = None

    def run(slots, n_slots):
        nonlocal bidx
        k_cache, v_cache, dkc, dvc = (torch.zeros(n_slots, T, H, d, dtype=torch.bfloat16, device="cuda")
                                      for _ in range(4))
        lf.lf_rope_frames(rope, old[:, :, 1], k_cache, weight=weight, out_slots=slots)
        v_cache[slots] = old[:, :, 2]
        sh = W.Shape(H=H, d=d, T=T, block=64, n_cur_frames=1, n_hist=2, n_sink=1, n_slots=n_slots,
                     k_f=2, k_b=5, scale=d ** -0.5)
        if bidx is None:
            bidx = lists(sh, 3)[0]
        q, k, v = (cur[:, i].contiguous() for i in range(3))
        out, lse = torch.empty_like(q), torch.empty(H, T, device="cuda")
        lf.lf_block_sparse_attn(sh, q, k, v, k_cache, v_cache, slots[:2], slots[2:], bidx, out, lse)
        res = [torch.empty_like(q) for _ in range(3)]
        lf.lf_block_sparse_attn_backward(sh, q, k, v, k_cache, v_cache, slots[:2], slots[2:], bidx,
                                         out, grad, lse, *res, dkc, dvc)
        dx, dw = torch.zeros_like(old)[:, :, 1], torch.empty_like(weight)
        lf.lf_rope_frames_backward(rope, old[:, :, 1], dkc, dx, weight=weight, dweight=dw,
                                   out_slots=slots)
        moved = torch.empty(3, T, H, d, dtype=torch.bfloat16, device="cuda")
        lf.lf_rope_frames(lf.make_rope(H, d, 3, *grid, (24, 20, 20)), k_cache, moved, in_slots=slots)
        return [out, lse, *res, k_cache[slots], dkc[slots], dvc[slots], dx, dw, moved]

    near = run([0, 1, 2], 3)
    for i, (a, b) in enumerate(zip(near, run(far, n_far))):
        assert torch.equal(a, b), i
    assert lf.lf_device_status(True) == 0
    assert all(bool(x.isfinite().all()) and bool((x != 0).any()) for x in near)
