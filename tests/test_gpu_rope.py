"""lf_rope_frames and lf_rope_frames_backward against oracle/grad64.py.

Tolerances.  Values are computed in fp32 from bf16 inputs and rounded to bf16 once: 2^-8 of
the value.  Before that: an angle in turns is reduced in 64 bits and rounded to 32 (2^-25 of
a turn, so under 2^-22 rad) with a sine and cosine good to a few 2^-24; a mean square of up to
12288 channels adds at most 80 terms in a row per thread and tree (80 * 2^-24 < 2^-17 of it,
half of that in its root).  Together under 2^-16 of the sizes that enter an element: a pair's
two channels (`amp`: the largest of the head times sqrt 2).  A weight's gradient stays in
fp32: its terms carry the same 2^-16, and its additions (a few hundred in a row) less.
"""
import pytest
import torch

import block_sparse_attention_46_b200 as lf
from oracle import grad64 as R

pytestmark = pytest.mark.gpu

STEP, FP32 = 2.0 ** -8, 2.0 ** -16


def case(H, d, frames, height, width, norm=None, halves=False, strided=False, pairs=None,
         slots=0, out_slots=0, pos=None, base=10000.0, eps=1e-6, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    T, parts = height * width, 3 if strided else 1
    third = d // 6
    n_in, n_out = slots or frames, out_slots or frames
    perm = lambda n: torch.randperm(n, generator=torch.Generator().manual_seed(seed + n))[:frames].tolist()
    c = dict(pairs=pairs if pairs is not None else (d // 2 - 2 * third, third, third),
             x=(rand(n_in, T, parts, H, d) * (0.25 + torch.rand(H, d, generator=g, device="cuda"))
                ).to(torch.bfloat16)[:, :, parts // 2],
             dout=rand(n_out, T, H, d).to(torch.bfloat16),
             ins=perm(n_in) if slots else None, outs=perm(n_out) if out_slots else None,
             pos=pos, weight=None, args=(height, width), n_out=n_out, frames=frames, T=T,
             kw=dict(halves=halves, norm=norm, base=base, eps=eps))
    if norm is not None:
        c["weight"] = 1.0 + 0.3 * rand(d if norm == "head" else H * d)
    c["rope"] = lf.make_rope(H, d, frames, height, width, c["pairs"], halves=halves, norm=norm,
                             base=base, eps=eps)
    return c


def take(c, t, which):
    return t[c[which]] if c[which] is not None else t[:c["frames"]]


def amp(v):
    return v.abs().amax(-1, keepdim=True) * 2 ** 0.5


def forward(c, out=None, **kw):
    out = torch.full((c["n_out"],) + tuple(c["x"].shape[1:]), 7.0, dtype=torch.bfloat16,
                     device="cuda") if out is None else out
    lf.lf_rope_frames(c["rope"], c["x"], out, frame_pos=c["pos"], weight=c["weight"],
                      in_slots=c["ins"], out_slots=c["outs"], **kw)
    return out


def backward(c, wide=False, **kw):
    """dx starts as 7; with `wide` it lies inside a wider projection."""
    n, T, H, d = c["x"].shape
    dx = torch.full((n, T, 2, H, d) if wide else (n, T, H, d), 7.0, dtype=torch.bfloat16,
                    device="cuda")
    view = dx[:, :, 1] if wide else dx
    dw = torch.full_like(c["weight"], float("nan")) if c["weight"] is not None else None
    lf.lf_rope_frames_backward(c["rope"], c["x"], c["dout"], view, frame_pos=c["pos"],
                               weight=c["weight"], dweight=dw, in_slots=c["ins"],
                               out_slots=c["outs"], **kw)
    return dx, view, dw


def check_forward(c):
    out = forward(c)
    x = take(c, c["x"], "ins").double()
    w = None if c["weight"] is None else c["weight"].double()
    ref = R.rope(x, w, *c["args"], c["pairs"], frame_pos=c["pos"], **c["kw"])
    got = take(c, out, "outs").double()
    over = (got - ref).abs() - (STEP * ref.abs() + FP32 * amp(ref))
    assert float(over.max()) <= 0, float(over.max())
    rest = [s for s in range(c["n_out"]) if s not in (c["outs"] or range(c["frames"]))]
    assert bool((out[rest] == 7).all()), "a slot outside the call changed"
    return out


def check_backward(c, wide=False):
    dx, view, dw = backward(c, wide)
    x = take(c, c["x"], "ins").double()
    g = take(c, c["dout"], "outs").double()
    w = None if c["weight"] is None else c["weight"].double()
    ref, dref = R.rope_backward(x, w, g, *c["args"], c["pairs"], frame_pos=c["pos"], **c["kw"])
    size = amp(g)
    H, d = x.shape[2:]
    if w is not None:
        over_ = (3,) if c["kw"]["norm"] == "head" else (2, 3)
        wv = w.abs() if c["kw"]["norm"] == "head" else w.abs().view(H, d)
        r = 1 / torch.sqrt(x.square().mean(over_, keepdim=True) + c["kw"]["eps"])
        xn, gw = (x * r).abs(), amp(g) * wv
        size = r * (gw + xn * (gw * xn).mean(over_, keepdim=True))
        terms = amp(g) * xn
        terms = terms.sum((0, 1, 2)) if c["kw"]["norm"] == "head" else terms.sum((0, 1)).flatten()
        over = (dw.double() - dref).abs() - FP32 * terms
        assert float(over.max()) <= 0, f"dweight {float(over.max()):.3e}"
    got = take(c, view, "ins").double()
    over = (got - ref).abs() - (STEP * ref.abs() + FP32 * size)
    assert float(over.max()) <= 0, f"dx {float(over.max()):.3e}"
    rest = [s for s in range(view.shape[0]) if s not in (c["ins"] or range(c["frames"]))]
    assert bool((view[rest] == 7).all()), "a slot outside the call changed"
    if wide:
        assert bool((dx[:, :, 0] == 7).all()), "the projection's other part changed"


SIZES = [
    dict(H=1, d=64, frames=1, height=1, width=1),
    dict(H=2, d=64, frames=1, height=1, width=1, strided=True),
    dict(H=3, d=64, frames=2, height=3, width=5),
    dict(H=5, d=64, frames=4, height=17, width=23, slots=6, out_slots=7),
    dict(H=7, d=128, frames=3, height=5, width=2, strided=True, slots=9),
    dict(H=12, d=128, frames=3, height=30, width=52, strided=True),
    dict(H=40, d=128, frames=2, height=9, width=7, out_slots=5),
    dict(H=33, d=64, frames=1, height=4, width=31),
    dict(H=96, d=128, frames=1, height=2, width=3),
    dict(H=1, d=128, frames=48, height=1, width=104, slots=50),
    dict(H=4, d=64, frames=9, height=60, width=1),
]


@pytest.mark.parametrize("norm", [None, "head", "row"])
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_values(gpu_lib, i, norm):
    c = case(norm=norm, halves=bool(i & 1), seed=i, **SIZES[i])
    check_forward(c)
    check_backward(c, wide=i % 3 == 0)


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("pairs", [(0, 0, 0), (64, 0, 0), (0, 33, 31), (1, 2, 3)])
def test_axes(gpu_lib, pairs, halves):
    c = case(3, 128, 2, 4, 6, norm="head", halves=halves, pairs=pairs, pos=[5, -9])
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("pos", [[0, 0], [2 ** 31 - 1, -2 ** 31], [123456789, 10 ** 6]])
def test_far_positions(gpu_lib, pos):
    """The first pair turns by the position itself in radians; in 32 bits it would be lost.
    In 64 bits the position's product with the frequency is off by half a step of up to 2^31
    rad, 2^-22 rad, on both sides: within the 2^-16 of the tolerance."""
    c = case(2, 64, 2, 3, 3, pos=pos)
    check_forward(c)
    check_backward(c)


def test_moves_frames_exactly(gpu_lib):
    c = case(6, 128, 3, 5, 9, pairs=(0, 0, 0), slots=5, out_slots=8, strided=True)
    out = check_forward(c)
    assert torch.equal(out[c["outs"]], c["x"][c["ins"]])


def test_frame_read_twice_and_in_place(gpu_lib):
    c = case(2, 64, 3, 4, 4, slots=4, out_slots=6, pos=[1, 2, 3])
    c["ins"] = [2, 2, 0]
    check_forward(c)
    with pytest.raises(lf.LfError):                       # its gradient would meet in one place
        backward(c)
    c = case(2, 64, 3, 4, 4, norm="row", slots=5)
    c["outs"] = c["ins"]
    c["n_out"] = 5
    want = forward(c)
    same = c["x"].clone()
    c["x"] = same
    got = forward(c, out=same)
    assert torch.equal(got[c["ins"]], want[c["ins"]])


def test_zero_and_huge_rows(gpu_lib):
    """A row of zeros has norm 1 / sqrt(eps); large values stay finite in fp32."""
    c = case(2, 64, 1, 2, 2, norm="row")
    c["x"][0, 0] = 0
    c["x"][0, 1] *= 2.0 ** 40
    check_forward(c)
    check_backward(c)


def test_rows_do_not_mix(gpu_lib):
    """A NaN in one token leaves every other token's result as it was (dweight sums all)."""
    c = case(5, 64, 2, 3, 7, norm="row")
    want, wdx = forward(c), backward(c)[1]
    c["x"][1, 4, 2, 3] = float("nan")
    got, dx = forward(c), backward(c)[1]
    keep = torch.ones(2, 21, dtype=torch.bool, device="cuda")
    keep[1, 4] = False
    assert torch.equal(got[keep], want[keep]) and torch.equal(dx[keep], wdx[keep])
    assert bool(got[1, 4].isnan().all()) and bool(dx[1, 4].isnan().all())


def test_repeatable_and_captured(gpu_lib):
    c = case(12, 128, 3, 30, 52, norm="row", strided=True)
    ws = torch.empty(lf.lf_rope_backward_workspace_size(c["rope"]), dtype=torch.uint8, device="cuda")
    out, (dx, _, dw) = forward(c), backward(c, workspace=ws)
    for _ in range(3):
        _, view, dw2 = backward(c, workspace=ws)
        assert torch.equal(dx, view) and torch.equal(dw, dw2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out2 = forward(c)
        dx2, _, dw2 = backward(c, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_refusals(gpu_lib):
    c = case(2, 64, 3, 4, 4, norm="row", slots=5)
    bad = lambda **kw: dict(c, **kw)
    with pytest.raises(ValueError):
        forward(bad(x=c["x"].float()))
    with pytest.raises(ValueError):
        forward(bad(x=c["x"].cpu()))
    with pytest.raises(ValueError):
        forward(bad(x=c["x"].transpose(2, 3)))
    with pytest.raises(ValueError):
        forward(bad(x=c["x"][:, ::2]))                    # not whole frames
    with pytest.raises(ValueError):
        forward(bad(weight=c["weight"][:64]))
    with pytest.raises(ValueError):
        forward(bad(ins=[0, 1]))
    with pytest.raises(lf.LfError):
        forward(bad(ins=[0, 1, 5]))                       # slot out of range
    with pytest.raises(lf.LfError):
        forward(bad(weight=None))
    with pytest.raises(lf.LfError):
        forward(bad(outs=[0, 1, 1]))
    with pytest.raises(lf.LfError):
        backward(c, workspace=torch.empty(256, dtype=torch.uint8, device="cuda")[:128])


@pytest.mark.parametrize("norm", ["head", "row"])
@pytest.mark.parametrize("power", [-57, -50, -43, 43, 50, 57])
def test_gradient_of_very_small_and_large_rows(gpu_lib, norm, power):
    """Rows of root mean square near 2^power, with a gradient along the normed row, so that the
    projection dx = r (w g - xn mean(w g xn)) takes away about as much as it leaves.  Every term
    is a product of r and values of the size of g, so fp32 keeps its relative error; the
    tolerances are those of ordinary rows.  Small rows have eps = 0."""
    c = case(3, 128, 1, 3, 5, norm=norm, eps=0.0 if power < 0 else 1e-6, seed=power + 100,
             strided=True)
    c["x"].mul_(2.0 ** power)                              # exact
    c["dout"] = (check_forward(c).float() + 0.5 * c["dout"].float()).to(torch.bfloat16)
    check_backward(c, wide=True)


# Calls of several waves, with last groups that are not full, up to those whose threads take four
# tokens each (16000 CTAs of one token per thread and more): both warp layouts (a token in part
# of a warp, in several warps), both head dimensions, few and many frames.
MANY = [
    dict(H=12, d=128, frames=3, height=29, width=53),
    dict(H=12, d=64, frames=5, height=41, width=43, slots=6),
    dict(H=12, d=128, frames=3, height=101, width=107, slots=5, out_slots=7, strided=True),
    dict(H=9, d=64, frames=3, height=101, width=217, slots=4),
    dict(H=12, d=128, frames=40, height=7, width=117, slots=44, out_slots=45, strided=True),
    dict(H=2, d=128, frames=20, height=113, width=115, out_slots=21),
]


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("norm", [None, "head", "row"])
@pytest.mark.parametrize("i", range(len(MANY)))
def test_values_of_many_tokens(gpu_lib, i, norm, halves):
    c = case(norm=norm, halves=halves, seed=40 + i, pos=[3 * f - 7 for f in range(MANY[i]["frames"])],
             **MANY[i])
    check_forward(c)
    check_backward(c, wide=bool(i & 1))


@pytest.mark.parametrize("norm", [None, "head", "row"])
@pytest.mark.parametrize("H, d, frames, height, width", [(5, 64, 3, 4, 7), (40, 128, 3, 5, 9),
                                                         (12, 128, 3, 30, 52)])
def test_gradient_in_place(gpu_lib, norm, H, d, frames, height, width):
    """dx may be dout, where strides and slots agree: the same bits, other slots untouched."""
    c = case(H, d, frames, height, width, norm=norm, slots=5, out_slots=5, seed=50)
    c["outs"] = c["ins"]
    _, want, dw = backward(c)
    same, dw2 = c["dout"].clone(), None if dw is None else torch.empty_like(dw)
    lf.lf_rope_frames_backward(c["rope"], c["x"], same, same, weight=c["weight"], dweight=dw2,
                               in_slots=c["ins"], out_slots=c["outs"])
    assert torch.equal(same[c["ins"]], want[c["ins"]])
    rest = [s for s in range(5) if s not in c["ins"]]
    assert torch.equal(same[rest], c["dout"][rest])
    assert dw is None or torch.equal(dw, dw2)
