"""Argument checks of the gradient and rotary entry points, without a GPU."""
import ctypes

import pytest

import block_sparse_attention_46_b200 as lf
from tests.test_abi import FAKE, _i32, _shape, lib  # noqa: F401 (lib: fixture)


def _attn_bwd(lib, shape, hist=(0, 1, 2, 3), sinks=(), ws=1 << 30, cache=FAKE, bidx=FAKE, q=FAKE,
              lse=FAKE, dvc=None):
    sh = lf.make_shape(shape)
    hp, _k = _i32(hist)
    sp, _k2 = _i32(sinks)
    return lib.lf_block_sparse_attn_backward(
        ctypes.byref(sh), q, FAKE, FAKE, FAKE, FAKE, hp, sp, bidx, None, FAKE, FAKE, lse, FAKE,
        FAKE, FAKE, cache, cache if dvc is None else dvc, FAKE, ws, None)


def test_attn_backward_validation(lib):
    assert _attn_bwd(lib, _shape(d=96)) == 2
    assert _attn_bwd(lib, _shape(n_cur_frames=0)) == 1
    assert _attn_bwd(lib, _shape(), hist=(0, 1, 2, 4)) == 1            # slot >= n_slots
    assert _attn_bwd(lib, _shape(), ws=16) == 5
    assert _attn_bwd(lib, _shape(), bidx=None) == 1
    assert _attn_bwd(lib, _shape(), q=None) == 1
    assert _attn_bwd(lib, _shape(), q=ctypes.c_void_p((1 << 20) + 8)) == 1
    assert _attn_bwd(lib, _shape(), lse=None) == 1
    assert _attn_bwd(lib, _shape(), cache=None, dvc=FAKE) == 1         # one of the two
    assert _attn_bwd(lib, _shape(), hist=(0, 1, 1, 3)) == 1            # a slot twice
    assert _attn_bwd(lib, _shape(n_sink=1), sinks=(2,)) == 1
    assert _attn_bwd(lib, _shape(k_c=2)) == 1                          # needs cur_idx
    assert lf.lf_attn_backward_workspace_size(_shape(d=96)) == 0
    assert lf.lf_attn_backward_workspace_size(_shape()) > lf.lf_attn_workspace_size(_shape())


def _rope(lib, x=FAKE, stride=128, n_in=4, ins=None, weight=FAKE, out=FAKE, n_out=4, outs=None,
          **kw):
    base = dict(H=2, d=64, n_frames=3, height=4, width=5, pairs=(12, 10, 10), norm="head")
    base.update(kw)
    r = lf.make_rope(**base)
    ip, _k = _i32(ins) if ins is not None else (None, None)
    op, _k2 = _i32(outs) if outs is not None else (None, None)
    return lib.lf_rope_frames(ctypes.byref(r), x, stride, n_in, ip, None, weight, out, n_out, op,
                              None)


def test_rope_validation(lib):
    assert _rope(lib, d=96) == 2
    assert _rope(lib, H=200) == 2                                      # 12800 channels
    assert _rope(lib, n_frames=300, n_in=300, n_out=300) == 2
    for kw in (dict(H=0), dict(height=0), dict(width=-1), dict(n_frames=0), dict(pairs=(33, 0, 0)),
               dict(pairs=(-1, 0, 0)), dict(pairs=(2 ** 31 - 1, 2 ** 31 - 1, 0)),
               dict(base=0.0), dict(base=float("inf")), dict(base=float("nan")), dict(eps=-1.0),
               dict(n_in=2), dict(n_out=2), dict(n_in=0), dict(ins=(0, 1, 4)), dict(outs=(0, 1, 4)),
               dict(outs=(0, 1, 1)), dict(stride=64), dict(stride=132), dict(x=None),
               dict(out=None), dict(weight=None), dict(norm=None),
               dict(x=ctypes.c_void_p((1 << 20) + 8))):
        assert _rope(lib, **kw) == 1, kw
    with pytest.raises(ValueError):
        lf.make_rope(2, 64, 1, 1, 1, (0, 0, 0), norm="channel")
    r = lf.make_rope(2, 64, 3, 4, 5, (12, 10, 10), norm="row")
    size = lf.lf_rope_backward_workspace_size(r)
    assert size >= 128 * 4
    assert lf.lf_rope_backward_workspace_size(lf.make_rope(2, 64, 3, 4, 5, (12, 10, 10))) == 0
    bwd = lambda **kw: lib.lf_rope_frames_backward(
        ctypes.byref(r), kw.get("x", FAKE), 128, 4, kw.get("ins"), None, kw.get("w", FAKE), FAKE, 4,
        None, FAKE, kw.get("dxs", 128), kw.get("dw", FAKE), FAKE, kw.get("ws", size), None)
    twice, _k = _i32([1, 2, 1])
    assert bwd(x=None) == 1 and bwd(w=None) == 1 and bwd(dw=None) == 1 and bwd(dxs=64) == 1
    assert bwd(ins=twice) == 1 and bwd(ws=size - 1) == 5


def test_rope_tokens_stay_in_their_storage():
    """Token strides that the kernels cannot follow are refused: broadcast tokens (stride 0, also
    under an outer dimension that has a stride) and tokens that overlap.  CPU tensors only."""
    import torch
    H, d, T, F = 2, 64, 6, 3

    def zeros(*size):
        return torch.zeros(*size, dtype=torch.bfloat16)

    def look(x):
        return lf._rope_tokens(H, d, T, x, "x", torch.device("cpu"), False)

    for x in (zeros(F, 1, H, d).expand(F, T, H, d), zeros(1, 1, H, d).expand(F, T, H, d),
              zeros(1, T, H, d).expand(F, T, H, d), zeros(1, H, d).expand(F * T, H, d),
              zeros(4000).as_strided((F, T, H, d), (T * 64, 64, 64, 1))):
        with pytest.raises(ValueError):
            look(x)
    for x, stride in ((zeros(F, T, H, d), H * d), (zeros(F * T, H, d), H * d),
                      (zeros(F, T, 3 * H, d)[:, :, H:2 * H], 3 * H * d),
                      (zeros(F, T, 3, H, d)[:, :, 1], 3 * H * d),
                      (zeros(F * T, 2 * H, d)[:, :H], 2 * H * d)):
        address, step, n = look(x)
        assert (step, n) == (stride, F)
        last = x.storage_offset() + (n * T - 1) * step + H * d
        assert last <= x.untyped_storage().nbytes() // 2


@pytest.mark.parametrize("far", [2 ** 31, -2 ** 31 - 1, 2 ** 32, 2 ** 63, 0.5])
def test_integers_are_not_wrapped(lib, far):
    """Positions and slots that are no 32-bit integers, and sizes that would wrap into valid ones
    (2^32 + 2 heads), are refused by the binding: the C side sees the wrapped value only."""
    for name in ("frame_pos", "in_slots", "out_slots"):
        with pytest.raises(ValueError, match="32-bit"):
            lf._frames(2, [0, far], name)
    with pytest.raises(ValueError, match="32-bit"):
        lf.lf_pool_frames(_shape(), None, [far], None)
    if far == int(far):
        with pytest.raises(ValueError, match="32-bit"):
            lf.make_rope(far + 2 if far > 0 else far, 64, 1, 1, 1, (0, 0, 0))
        with pytest.raises(ValueError, match="32-bit"):
            lf.make_rope(2, 64, 1, 1, 1, (far, 0, 0))


def test_32_bit_lists_pass_unchanged():
    import numpy as np
    import torch
    ends = [-2 ** 31, -1, 0, 2 ** 31 - 1]
    for v in (ends, tuple(ends), np.array(ends), torch.tensor(ends), [float(x) for x in ends]):
        pointer, keep = lf._slots(v)
        assert list(keep) == ends and pointer[3] == ends[3]
    assert len(lf._slots([])[1]) == 1


def test_rope_frequencies_are_finite(lib):
    """A base so small that base^(-i / n) overflows would turn by NaN, at position zero too."""
    assert _rope(lib, base=5e-324, pairs=(32, 0, 0)) == 1
    assert _rope(lib, base=5e-324, pairs=(0, 0, 32)) == 1
    assert lf.lf_rope_backward_workspace_size(
        lf.make_rope(2, 64, 3, 4, 5, (32, 0, 0), norm="row", base=5e-324)) == 0
