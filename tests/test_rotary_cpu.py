"""What the rotary calls refuse before any device work, through the C ABI on host-only pools, and the binding's own
checks.  Only refused calls are made where a GPU is visible."""
import ctypes
import gc
import weakref

import numpy as np
import pytest
import torch

from linear_attention_state_lsc_gb300 import lsc as L

from _util import gpu_present
from test_kv_step_cpu import BATCHES, DEV, batch, pool_of

FREQ = 10000.0 ** (-np.arange(0, 32, 2) / 32)
INV, MIS = L.LSC_ERR_INVALID_ARG, L.LSC_ERR_MISALIGNED


def rotary(**k):
    return L.rotary(**{**dict(rotary_dim=32, positions=DEV, inv_freq=FREQ, axes=2), **k})


def broken():
    """(rotary, what it is refused with) for head_dim 64 and 5 tokens"""
    out = [(rotary(rotary_dim=d, inv_freq=np.ones(d // 2)), INV) for d in (0, 66, 1024)]
    out += [(rotary(positions=None), INV), (rotary(positions=DEV + 2), MIS), (rotary(axes=0), INV), (rotary(axes=9), INV),
            (rotary(axes=-1), INV), (rotary(interleaved=2), INV), (rotary(scale=float("nan")), INV),
            (rotary(scale=float("inf")), INV), (rotary(axis_stride=4), INV), (rotary(axis_stride=-5), INV),
            (rotary(pair_axis=np.full(16, 2)), INV), (rotary(pair_axis=np.r_[[0] * 15, 255]), INV)]
    for bad in (float("nan"), float("inf"), 65537.0, -1e300):
        f = FREQ.copy()
        f[7] = bad
        out.append((rotary(inv_freq=f), INV))
    for field, value in (("rotary_dim", 31), ("rotary_dim", -2), ("inv_freq", None)):
        r = rotary()
        setattr(r, field, value)
        out.append((r, INV))
    return out


def test_rotate_refusals(lsc):
    base = dict(total_tokens=5, num_heads=3, head_dim=64, dtype=L.LSC_BF16, x=DEV, out=DEV + 4096, rotary=rotary())
    bad = [(dict(rotary=r), rc) for r, rc in broken()]
    bad += [(k, INV) for k in (dict(total_tokens=-1), dict(num_heads=0), dict(num_heads=-1), dict(head_dim=0), dict(head_dim=30),
                               dict(dtype=L.LSC_E4M3), dict(dtype=L.LSC_E2M1), dict(dtype=9), dict(x=None), dict(out=None),
                               dict(x_stride=191), dict(out_stride=191), dict(x_stride=-192), dict(out=DEV, x_stride=200))]
    bad += [(dict(x=DEV + 1), MIS), (dict(out=DEV + 1), MIS), (dict(dtype=L.LSC_F32, x=DEV + 2), MIS),
            (dict(num_heads=(1 << 24) + 1), L.LSC_ERR_UNSUPPORTED)]
    for k, want in bad:
        assert L.lsc_rotate(L.rotate_args(**{**base, **k})) == want, k
    assert L.load().lsc_rotate(None, None) == INV
    if not gpu_present():
        assert L.lsc_rotate(L.rotate_args(**base)) == L.LSC_ERR_CUDA


def test_append_rotated_refusals(lsc):
    pool = pool_of()
    app = lambda **k: L.kv_append_args(**{**dict(batch=batch(), k=DEV, v=DEV, dtype=L.LSC_BF16), **k})
    base = dict(append=app(), rotary=rotary(), num_q_heads=4, q=DEV, q_out=DEV + 65536)
    bad = [(dict(rotary=r), rc) for r, rc in broken()] + [(dict(append=app(batch=b)), rc) for b, rc in BATCHES]
    bad += [(dict(append=app(**k)), rc) for k, rc in (
        (dict(k=None), INV), (dict(v=None), INV), (dict(dtype=L.LSC_E2M1), INV), (dict(k_stride=127), INV),
        (dict(v_stride=-1), INV), (dict(k=DEV + 1), MIS), (dict(v=DEV + 1), MIS))]
    bad += [(k, INV) for k in (dict(num_q_heads=-1), dict(q=None), dict(q_out=None), dict(q_stride=255),
                               dict(q_out_stride=255), dict(q_out=DEV, q_out_stride=300))]
    bad += [(dict(q=DEV + 1), MIS), (dict(q_out=DEV + 1), MIS), (dict(num_q_heads=1 << 24), L.LSC_ERR_UNSUPPORTED)]
    for k, want in bad:
        assert L.lsc_kv_append_rotated(pool, 1, L.kv_append_rotated_args(**{**base, **k})) == want, k
    good = L.kv_append_rotated_args(**base)
    assert L.lsc_kv_append_rotated(pool, 2, good) == L.LSC_ERR_OUT_OF_RANGE
    assert L.lsc_kv_append_rotated(None, 0, good) == INV
    assert L.load().lsc_kv_append_rotated(pool, 0, None, None) == INV
    for field in ("reserved", "append.reserved", "append.batch.reserved"):
        a = L.kv_append_rotated_args(**base)
        o = a
        for part in field.split(".")[:-1]:
            o = getattr(o, part)
        o.reserved = 1
        assert L.lsc_kv_append_rotated(pool, 0, a) == INV
    if not gpu_present():
        assert L.lsc_kv_append_rotated(pool, 1, good) == L.LSC_ERR_CUDA
        assert L.lsc_kv_append_rotated(pool, 1, L.kv_append_rotated_args(app(), rotary())) == L.LSC_ERR_CUDA  # k alone
    L.lsc_kv_pool_destroy(pool)


def test_the_binding_reads_positions():
    p = torch.zeros(3, 9, dtype=torch.int32)
    r = L.rotary(32, p[:, :5], FREQ, pair_axis=[0, 1] * 8)
    assert (r.axes, r.axis_stride, r.positions) == (3, 9, p.data_ptr())
    assert (L.rotary(32, p[0], FREQ).axes, L.rotary(32, p[0], FREQ).axis_stride) == (1, 0)
    r = rotary()
    np.testing.assert_array_equal(np.ctypeslib.as_array(ctypes.cast(r.inv_freq, ctypes.POINTER(ctypes.c_double)), (16,)), FREQ)
    for bad in (dict(positions=p.long()), dict(positions=p.T), dict(positions=p[:, ::2]), dict(positions=p[None]),
                dict(inv_freq=FREQ[1:]), dict(pair_axis=[0])):
        with pytest.raises(ValueError):
            L.rotary(**{**dict(rotary_dim=32, positions=p, inv_freq=FREQ), **bad})


def test_a_row_expanded_to_every_axis():
    """Text: every axis takes the same position.  The library reads axis a at positions + a * (axis_stride or
    total_tokens), so no pair may be given an axis behind the one row that there is."""
    T = 9
    p = torch.arange(T, dtype=torch.int32)
    for pos in (p.expand(3, T), p[None].expand(3, T), p[:1].expand(3, 1), p.expand(8, T)):
        for axis in (None, [0, 1, 2, 1] * 4):
            r = L.rotary(32, pos, FREQ, pair_axis=axis)
            most = 0 if not r.pair_axis else max(ctypes.string_at(r.pair_axis, 16))
            last = most * (r.axis_stride or pos.shape[1]) + pos.shape[1]  # entries from `positions` on that may be read
            assert r.positions == p.data_ptr() and last <= pos.shape[1]
    # what is refused stays refused
    base = dict(total_tokens=T, num_heads=3, head_dim=64, dtype=L.LSC_BF16, x=DEV, out=DEV + 4096)
    for r in (L.rotary(32, p.expand(3, T), FREQ, pair_axis=np.full(16, 3)), L.rotary(32, p.expand(9, T), FREQ)):
        assert L.lsc_rotate(L.rotate_args(**base, rotary=r)) == INV


def test_pair_axis_is_held_as_it_is():
    """Axes that a byte does not hold are refused, not taken modulo 256 or cut to a whole number; those that it holds and
    that are not there are the library's to refuse."""
    p = torch.zeros(3, 9, dtype=torch.int32)
    for bad in (256, 257, -1, -256, 1 << 32, 0.5, 1.75, float("nan")):
        with pytest.raises(ValueError):
            L.rotary(32, p, FREQ, pair_axis=np.array([0, 1] * 7 + [2, bad]))
    for good in ([2] * 16, np.full(16, 2, np.int64), np.full(16, 2.0), [True] * 16, torch.full((16,), 1)):
        r = L.rotary(32, p, FREQ, pair_axis=good)
        assert list(ctypes.string_at(r.pair_axis, 16)) == [int(a) for a in good]


def test_positions_of_every_token():
    """A tensor of positions shorter than the call's tokens would be read past its end: refused when the call's arguments
    are made.  A longer one is fine (what lies behind is another call's)."""
    p = torch.zeros(3, 9, dtype=torch.int32)
    for pos, held in ((p[0], 9), (p[0, :4], 4), (p, 9), (p[:, :4], 4), (p[0, :4].expand(3, 4), 4), (p[0, :0], 0)):
        r = L.rotary(32, pos, FREQ)
        rotate = lambda t: L.rotate_args(t, 3, 64, L.LSC_BF16, DEV, DEV + 4096, r)
        append = lambda t: L.kv_append_rotated_args(L.kv_append_args(batch(total=t), DEV, DEV, L.LSC_BF16), r)
        for make in (rotate, append):
            for t in range(held + 1):
                make(t)
            for t in (held + 1, 10, 1 << 30):
                with pytest.raises(ValueError):
                    make(t)
    L.rotate_args(1 << 30, 3, 64, L.LSC_BF16, DEV, DEV, rotary())  # an address: the caller knows


def test_positions_live_as_long_as_the_arguments():
    """positions made in place of an argument (a cast, a slice moved to the device) are not given back before the call."""
    p = torch.zeros(9, dtype=torch.int64)
    made = p.to(torch.int32)
    alive = weakref.ref(made)
    args = L.rotate_args(9, 3, 64, L.LSC_BF16, DEV, DEV, L.rotary(32, made, FREQ))
    del made
    gc.collect()
    assert alive() is not None
    del args
    gc.collect()
    assert alive() is None
