"""GPU: lsc_rotate and lsc_kv_append_rotated against the plain 64-bit form (tests/_rotary.py): every type, pattern of
pairs and axes, odd head sizes, strides, in place, far and negative positions, rows that belong to no sequence, graphs,
and the step's calls together: rotated append, attend and gather over every type of pool.

Tolerance.  A cosine or sine is off by 2^-22 (include/lsc_kv.h), an element of the result is two products of it and an
element, each rounded in 32 bits (2^-24 of it) and added (2^-24 of the sum), so off by 2^-21.5 times the sum of the
products' magnitudes with the factor; then it is rounded once to its type: half a step of the result.  The reference's
own angle, position times frequency in 64 bits, is off by 2^-53 of itself: 2^-22 more at positions of 2^31.
"""
import decimal

import numpy as np
import pytest
import torch

from linear_attention_state_lsc_gb300 import lsc as L

import _kv
import _kv4
from _kv import NAME, TORCH, Batch, DevKv, HostKv
from _kv4 import Host4
from _rotary import angles, turn
from test_gpu_kv4 import check4
from test_gpu_kv_step import FLOATS, HALF, check_attend, cur, dense, run_attend, step_lengths

pytestmark = pytest.mark.gpu

BF, F16, F32 = L.LSC_BF16, L.LSC_F16, L.LSC_F32


def freqs(rotary_dim):
    return 10000.0 ** (-np.arange(0, rotary_dim, 2) / rotary_dim)


def plan(rng, T, rotary_dim, axes, far=0):
    """(positions on the device, a wider array behind them, their angles, the pairs' axes)"""
    pos = (rng.integers(-5, 3000, (axes, T)) + far).astype(np.int64)
    pos = np.clip(pos, -2 ** 31, 2 ** 31 - 1).astype(np.int32)
    axis = rng.integers(0, axes, rotary_dim // 2).astype(np.uint8) if axes > 1 else None
    dev = torch.full((axes, T + 5), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    dev[:, :T] = torch.from_numpy(pos)
    return dev[:, :T], angles(pos, freqs(rotary_dim), axis), axis


def check(got, want, size, dtype, extra=0.0):
    """got, want, size: [..., D]"""
    err = (2.0 ** -21.5 + extra) * size
    bound = err + HALF[dtype] * (np.abs(want) + err) + 1e-40
    if dtype == F16:
        bound = np.maximum(bound, err + 2.0 ** -25)  # subnormal results
    over = np.abs(got - want) / bound
    assert over.max(initial=0) <= 1, (over.max(), np.unravel_index(over.argmax(), over.shape))


SHAPES = [  # heads, head_dim, rotary_dim
    (4, 128, 128), (18, 256, 64), (3, 64, 64), (16, 80, 80), (5, 80, 20), (2, 96, 48), (1, 33, 32), (7, 64, 2), (2, 512, 512),
    (3, 272, 48), (1, 2, 2)]


@pytest.mark.parametrize("dtype", FLOATS, ids=NAME.get)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
def test_rotate(lsc, dtype, shape, interleaved):
    H, D, R = shape
    rng = np.random.default_rng(H * D + R)
    for T, axes, stride, far, scale in ((1, 1, 0, 0, 1.0), (37, 3, H * D + 8, 0, 1.25), (700, 2, H * D + 1, 10 ** 6, 1.0),
                                        (5001 if H * D < 2000 else 300, 4, 0, 0, 1.0), (9, 1, 0, -10 ** 6, -0.5)):
        pos, angle, axis = plan(rng, T, R, axes, far)
        x = rng.standard_normal((T, H, D)) * np.exp(2 * rng.standard_normal((T, H, 1)))
        x, xx = dense(x, dtype, stride or None)
        want, size = turn(xx, R, angle, interleaved, scale)
        r = L.rotary(R, pos, freqs(R), pair_axis=axis, interleaved=interleaved, scale=scale)
        w = stride or H * D
        out = torch.full((T, w), 7.0, dtype=TORCH[dtype], device="cuda")
        assert L.lsc_rotate(L.rotate_args(T, H, D, dtype, x, out, r, stride, stride), cur()) == L.LSC_OK
        got = out[:, :H * D].double().cpu().numpy().reshape(T, H, D)
        check(got, want, size, dtype)
        assert torch.equal(out[:, :H * D].view(T, H, D)[..., R:], x[:, :H * D].view(T, H, D)[..., R:])
        assert (out[:, H * D:] == 7).all()
        # in place: the same bits, and nothing between the rows
        between = x[:, H * D:].clone()
        assert L.lsc_rotate(L.rotate_args(T, H, D, dtype, x, x, r, stride, stride), cur()) == L.LSC_OK
        assert torch.equal(x[:, :H * D], out[:, :H * D])
        assert torch.equal(x[:, H * D:].isnan(), between.isnan())


@pytest.mark.parametrize("H,D,R,T,stride", [
    (2, 64, 64, 5, 2 ** 30 + 8), (2, 64, 64, 5, 2 ** 30 + 1),  # rows whose bytes pass 33 bits, both kernels
    (70001, 16, 16, 2, 0), (33000, 10, 6, 2, 0),               # more heads than a grid has rows
    (2, 4096, 512, 3, 0), (1, 100000, 2, 2, 0)], ids=str)      # heads wider than the vector kernel takes
def test_extreme_sizes(lsc, H, D, R, T, stride):
    rng = np.random.default_rng(H + D)
    pos, angle, axis = plan(rng, T, R, 3)
    x, xx = dense(rng.standard_normal((T, H, D)), BF)
    x = x.view(T, H * D)
    rows = x if not stride else torch.empty(T * stride, dtype=TORCH[BF], device="cuda").view(T, stride)
    if stride:
        rows[:, :H * D] = x
        rows[:, H * D:H * D + 64] = 7
    r = L.rotary(R, pos, freqs(R), pair_axis=axis)
    assert L.lsc_rotate(L.rotate_args(T, H, D, BF, rows, rows, r, stride, stride), cur()) == L.LSC_OK
    want, size = turn(xx, R, angle, False)
    check(rows[:, :H * D].double().cpu().numpy().reshape(T, H, D), want, size, BF)
    assert (rows[:, H * D:H * D + 64] == 7).all()


@pytest.mark.parametrize("D,R", [(128, 64), (80, 20)])
def test_rotate_in_a_graph_of_another_stream(lsc, D, R):
    """Captured in place and out of place behind each other, replayed with other positions and rows; frequencies are read
    when the call is made."""
    rng = np.random.default_rng(D)
    H, T = 6, 50
    pos, _, axis = plan(rng, T, R, 2)
    x, _ = dense(rng.standard_normal((T, H, D)), BF)
    y = torch.zeros_like(x)
    freq = freqs(R).copy()
    r = L.rotary(R, pos, freq, pair_axis=axis)
    there, back = L.rotate_args(T, H, D, BF, x, y, r), L.rotate_args(T, H, D, BF, x, x, r)
    s = torch.cuda.Stream()
    s.wait_stream(cur())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        assert L.lsc_rotate(there, s) == L.LSC_OK
        assert L.lsc_rotate(back, s) == L.LSC_OK
        assert L.lsc_rotate(L.rotate_args(0, H, D, BF, None, None, r), s) == L.LSC_OK
    freq[:] = 0
    r._host[0][:] = 0
    for _ in range(3):
        p = rng.integers(-9, 9999, (2, T)).astype(np.int32)
        pos.copy_(torch.from_numpy(p))
        rows, xx = dense(rng.standard_normal((T, H, D)), BF)
        x.copy_(rows)
        g.replay()
        torch.cuda.synchronize()
        want, size = turn(xx, R, angles(p, freqs(R), axis), False)
        check(y.double().cpu().numpy().reshape(T, H, D), want, size, BF)
        assert torch.equal(x, y)


def test_what_is_not_turned_keeps_its_bits(lsc):
    """NaN payloads, infinities and zeros behind rotary_dim, out of place and in place, both kernels."""
    for dtype, word in ((BF, torch.int16), (F16, torch.int16), (F32, torch.int32)):
        for stride in (64, 65):
            bits = torch.randint(-2 ** 15, 2 ** 15, (40, stride), dtype=torch.int32).to(word)
            if word == torch.int32:
                bits = bits * 65537 + 12345
            x = bits.cuda().view(TORCH[dtype])
            x[:, :16] = 1.0
            out = torch.zeros_like(x)
            pos = torch.arange(40, dtype=torch.int32, device="cuda")
            r = L.rotary(16, pos, freqs(16))
            for o in (out, x):
                assert L.lsc_rotate(L.rotate_args(40, 1, 64, dtype, x, o, r, stride, stride), cur()) == L.LSC_OK
            assert torch.equal(out[:, 16:64].view(word), x[:, 16:64].view(word))
            assert torch.equal(out[:, 16:64].view(word).cpu(), bits[:, 16:64])


def test_far_positions(lsc):
    """Every position of 32 bits: angles from 80-digit arithmetic."""
    decimal.getcontext().prec = 80
    tau = 2 * decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
    pos = [0, 1, -1, 4097, 10 ** 6 + 3, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, -2 ** 31 + 1, 123456789]
    freq = np.concatenate([freqs(32), [0.0, -1.0, 3.5, -0.37, 1e-9, 65536.0, -65535.7, 6.283185307179586]])
    angle = np.array([[float((decimal.Decimal(p) * decimal.Decimal(float(f)) % tau)) for f in freq] for p in pos])
    R, T = 2 * len(freq), len(pos)
    x = torch.zeros(T, R, device="cuda")
    x[:, :R // 2] = 1
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    for turned in (1, -1):
        out = torch.zeros_like(x)
        assert L.lsc_rotate(L.rotate_args(T, 1, R, F32, x, out, L.rotary(R, p, turned * freq)), cur()) == L.LSC_OK
        got = out.double().cpu().numpy()
        assert np.abs(got[:, :R // 2] - np.cos(angle)).max() <= 2.0 ** -22
        assert np.abs(got[:, R // 2:] - turned * np.sin(angle)).max() <= 2.0 ** -22


@pytest.mark.parametrize("interleaved", [False, True])
def test_the_turn_back_is_its_gradient(lsc, interleaved):
    """With negated frequencies the turn is transposed: the formula's gradient, and differences of the turn itself."""
    rng = np.random.default_rng(3)
    T, H, D, R = 9, 2, 64, 32
    pos, angle, axis = plan(rng, T, R, 3)
    x, xx = dense(rng.standard_normal((T, H, D)), F32)
    g, gx = dense(rng.standard_normal((T, H, D)), F32)
    back = torch.empty_like(g)
    r = L.rotary(R, pos, -freqs(R), pair_axis=axis, interleaved=interleaved, scale=1.5)
    assert L.lsc_rotate(L.rotate_args(T, H, D, F32, g, back, r), cur()) == L.LSC_OK
    dx = back.double().cpu().numpy().reshape(T, H, D)
    xt = torch.from_numpy(xx).requires_grad_()
    half = R // 2
    c, s = 1.5 * torch.from_numpy(np.cos(angle))[:, None], 1.5 * torch.from_numpy(np.sin(angle))[:, None]
    a, b = (xt[..., 0:R:2], xt[..., 1:R:2]) if interleaved else (xt[..., :half], xt[..., half:R])
    y = a * c - b * s, b * c + a * s
    gt = torch.from_numpy(gx)
    ga, gb = (gt[..., 0:R:2], gt[..., 1:R:2]) if interleaved else (gt[..., :half], gt[..., half:R])
    ((y[0] * ga).sum() + (y[1] * gb).sum() + (xt[..., R:] * gt[..., R:]).sum()).backward()
    _, size = turn(gx, R, angle, interleaved, 1.5)
    check(dx, xt.grad.numpy(), size, F32)
    d = rng.standard_normal(xx.shape)
    step = 2.0 ** -20
    up, down = (turn(xx + e * d, R, angle, interleaved, 1.5)[0] for e in (step, -step))
    slope = ((up - down) / (2 * step) * gx).sum()  # linear in x: the difference is off by roundings of 2^-53 / step alone
    assert abs(slope - (dx * d).sum()) <= 2.0 ** -20 * (size * np.abs(d)).sum()


def host_pool(kind, blocks, bt, H, D, **k):
    return Host4(blocks, bt, H, D, **k) if kind == L.LSC_E2M1 else HostKv(blocks, bt, H, D, kind, **k)


POOLS = FLOATS + [L.LSC_E4M3, L.LSC_E2M1]


@pytest.mark.parametrize("pool", POOLS, ids=lambda p: NAME.get(p, "e2m1"))
@pytest.mark.parametrize("dtype", FLOATS, ids=NAME.get)
@pytest.mark.parametrize("shape", [(16, 2, 64, 64, 4), (7, 3, 48, 32, 0), (64, 2, 256, 64, 16), (5, 1, 80, 80, 5),
                                   (3, 1, 272, 16, 2)], ids=str)
def test_append_rotated(lsc, pool, dtype, shape):
    """q and the pool's K rows against the turn in 64 bits, V rows and everything else bit by bit."""
    bt, H, D, R, Hq = shape
    rng = np.random.default_rng(bt * D + pool)
    for (name, stride, interleaved, axes) in (("ragged", 0, False, 3), ("ahead", 8, True, 1), ("decode", 3, False, 2)):
        n, kv = step_lengths(name)
        host = host_pool(pool, 50, bt, H, D)
        b = Batch(rng, n, kv, bt, 50, spare=3, wide=2)
        x = rng.standard_normal((2, b.T, H, D)) * np.exp(2 * rng.standard_normal((2, b.T, H, 1)))
        x[:, -3:] = np.nan
        ks = H * D + stride if stride else 0
        (k, kx), (v, vx) = (dense(y, dtype, ks or None) for y in x)
        qs = Hq * D + stride if stride else 0
        q, qx = dense(rng.standard_normal((b.T, Hq, D)), dtype, qs or None) if Hq else (None, None)
        pos, angle, axis = plan(rng, b.T, R, axes)
        r = L.rotary(R, pos, freqs(R), pair_axis=axis, interleaved=interleaved, scale=1.125)
        out = torch.full_like(q, 7.0) if Hq else None
        with DevKv(host) as dev:
            append = L.kv_append_args(b.device(), k, v, dtype, ks, ks)
            args = L.kv_append_rotated_args(append, r, Hq, q, out, qs, qs)
            assert L.lsc_kv_append_rotated(dev.pool, 1, args, cur()) == L.LSC_OK
            got = dev.download()
            assert dev.status() == L.LSC_OK
        T = int(b.cu[-1])
        if Hq:
            want, size = turn(qx, R, angle, interleaved, 1.125)
            check(out[:T, :Hq * D].double().cpu().numpy().reshape(T, Hq, D), want[:T], size[:T], dtype)
            assert (out[T:] == 7).all() and (out[:, Hq * D:] == 7).all()
            if R < D:
                assert torch.equal(out[:T, :Hq * D].view(T, Hq, D)[..., R:], q[:T, :Hq * D].view(T, Hq, D)[..., R:])
        want, size = turn(kx, R, angle, interleaved, 1.125)
        held = host_pool(pool, 50, bt, H, D)
        held.bytes[:] = got
        for i in range(len(n)):
            first = max(0, n[i] - kv[i])
            bl, rr = b.places(i, max(0, kv[i] - n[i]), kv[i])
            at = slice(b.cu[i] + first, b.cu[i + 1])
            host.write(1, 1, bl, rr, vx[at])
            if len(bl) == 0:
                continue
            back, w, z = held.read(1, 0, bl, rr), want[at], size[at]
            err = 2.0 ** -21.5 * z
            if pool in FLOATS:
                check(back, w, z, pool)
            elif pool == L.LSC_E4M3:  # 2^-4 of the element, or 2^-10 of the scale, which is above 2^-9 of the largest
                top = np.abs(w).max(-1, keepdims=True)
                assert (np.abs(back - w) <= err + 2.0 ** -4 * (np.abs(w) + err) + 2.0 ** -18 * top).all()
            else:  # 3/16 of its group's largest magnitude (plus what the turn was off by), the scale below 2^-14
                w16, e16 = w.reshape(*w.shape[:-1], -1, 16), err.reshape(*w.shape[:-1], -1, 16)
                top = (np.abs(w16) + e16).max(-1, keepdims=True)
                assert (np.abs(back.reshape(w16.shape) - w16) <= e16 + np.maximum(top * 3 / 16, 2.0 ** -14)).all()
            # the rows that K was written to, and nothing else
            es = host.rows(1, 0).shape[-1]
            host.rows(1, 0)[bl, rr] = held.rows(1, 0)[bl, rr]
            if pool not in FLOATS:
                host.scales(1, 0)[bl, rr] = held.scales(1, 0)[bl, rr]
        np.testing.assert_array_equal(got, host.bytes)


@pytest.mark.parametrize("pool", [BF, L.LSC_E4M3, L.LSC_E2M1], ids=lambda p: NAME.get(p, "e2m1"))
def test_at_position_zero_it_is_append(lsc, pool):
    """Angles of zero: the pool's bytes are those of lsc_kv_append, q its own bits; in place."""
    rng = np.random.default_rng(8)
    for D, R, stride in ((128, 128, 0), (64, 32, 0), (64, 32, 3)):
        n, kv = [5, 0, 1, 17], [5, 9, 64, 40]
        b = Batch(rng, n, kv, 16, 30, spare=2)
        T, H, Hq = b.T, 2, 6
        s = [h * D + stride if stride else 0 for h in (H, Hq)]
        (k, _), (v, _) = (dense(rng.standard_normal((T, H, D)), BF, s[0] or None) for _ in "kv")
        q, _ = dense(rng.standard_normal((T, Hq, D)), BF, s[1] or None)
        was = q.clone()
        host = host_pool(pool, 30, 16, H, D)
        got = []
        pos = torch.zeros(T, dtype=torch.int32, device="cuda")
        for rotated in (False, True):
            with DevKv(host) as dev:
                append = L.kv_append_args(b.device(), k, v, BF, s[0], s[0])
                if rotated:
                    args = L.kv_append_rotated_args(append, L.rotary(R, pos, freqs(R)), Hq, q, q, s[1], s[1])
                    assert L.lsc_kv_append_rotated(dev.pool, 0, args, cur()) == L.LSC_OK
                else:
                    assert L.lsc_kv_append(dev.pool, 0, append, cur()) == L.LSC_OK
                got.append(dev.download())
        np.testing.assert_array_equal(got[0], got[1])
        assert torch.equal(torch.nan_to_num(q), torch.nan_to_num(was))


def test_bad_batches_stay_inside(lsc):
    """Blocks, lengths and cu_seqlens that do not fit are recorded; the other sequences' rows are right."""
    rng = np.random.default_rng(6)
    H, Hq, D, bt, blocks = 2, 4, 64, 16, 30
    b = Batch(rng, [1, 3, 2, 1], [40, 50, 60, 33], bt, blocks, wide=1)
    k, kx = dense(rng.standard_normal((b.T, H, D)), BF)
    q, qx = dense(rng.standard_normal((b.T, Hq, D)), BF)
    pos, angle, axis = plan(rng, b.T, D, 1)
    want, size = turn(qx, D, angle, False)
    kw, ksize = turn(kx, D, angle, False)
    b.device()
    for what, bad, code in (("table", blocks, L.LSC_ERR_OUT_OF_RANGE), ("table", -1, L.LSC_ERR_OUT_OF_RANGE),
                            ("kv", -1, L.LSC_ERR_INVALID_ARG), ("kv", 2 ** 31 - 1, L.LSC_ERR_INVALID_ARG),
                            ("cu", [0, 5, 4, 6, 7], L.LSC_ERR_INVALID_ARG), ("cu", [3, 4, 5, 6, 99], L.LSC_ERR_INVALID_ARG)):
        host = host_pool(BF, blocks, bt, H, D)
        table, cu, kv = b.table.copy(), b.cu.copy(), b.kv.astype(np.int32)
        if what == "table":
            table[1, 49 // bt] = bad
        elif what == "kv":
            kv[1] = bad
        else:
            cu = np.array(bad, np.int32)
        dev_arrays = [torch.from_numpy(a).cuda() for a in (table, cu, kv)]
        batch = L.kv_batch(4, b.T, *dev_arrays, max_blocks=table.shape[1])
        out = torch.full_like(q, 7.0)
        with DevKv(host) as dev:
            args = L.kv_append_rotated_args(L.kv_append_args(batch, k, k, BF), L.rotary(D, pos, freqs(D)), Hq, q, out)
            assert L.lsc_kv_append_rotated(dev.pool, 1, args, cur()) == L.LSC_OK
            got = dev.download()
            assert dev.status() == code
        assert (got[0] == 0xFF).all()
        if what == "cu":
            continue
        check(out.double().cpu().numpy().reshape(b.T, Hq, D), want, size, BF)  # q is turned whatever the cache holds
        host.bytes[:] = got
        for i in (0, 2, 3):
            bl, r = b.places(i, int(b.kv[i] - b.n[i]), int(b.kv[i]))
            at = slice(b.cu[i], b.cu[i + 1])
            check(host.read(1, 0, bl, r), kw[at], ksize[at], BF)


@pytest.mark.parametrize("pool,dtype,D", [(BF, BF, 256), (L.LSC_E4M3, BF, 128), (L.LSC_E2M1, BF, 128), (L.LSC_E2M1, F16, 256),
                                          (F32, F32, 48)], ids=str)
def test_a_step_in_a_graph(lsc, pool, dtype, D):
    """Rotated append, attend and gather as a layer's step uses them: captured once on a side stream, replayed with
    other lengths, positions and values.  attend is held against the rows that gather reads back (bit for bit the
    pool's) and the turned q."""
    rng = np.random.default_rng(9)
    H, G, bt, S, R = 2, 4, 16, 4, 32
    mixes = [([1, 1, 2, 1], [1, 300, 64, 65]), ([40, 2, 1, 0], [200, 3, 128, 100])]
    blocks = 60
    batches = [Batch(rng, n, kv, bt, blocks) for n, kv in mixes]
    T, wide = max(b.T for b in batches), max(b.table.shape[1] for b in batches)
    table = torch.zeros(S, wide, dtype=torch.int32, device="cuda")
    cu, kvl = torch.zeros(S + 1, dtype=torch.int32, device="cuda"), torch.zeros(S, dtype=torch.int32, device="cuda")
    q, k, v = (torch.zeros(T, h * D, dtype=TORCH[dtype], device="cuda") for h in (H * G, H, H))
    pos = torch.zeros(3, T, dtype=torch.int32, device="cuda")
    turned, out = torch.zeros_like(q), torch.zeros_like(q)
    axis = np.arange(R // 2) % 3
    r = L.rotary(R, pos, freqs(R), pair_axis=axis)
    host = host_pool(pool, blocks, bt, H, D, layers=1, fill=0)
    side = torch.cuda.Stream()
    with DevKv(host) as dev:
        batch = L.kv_batch(S, T, table, cu, kvl, max_blocks=wide)
        a = L.kv_attend_args(batch, H * G, turned, out, dtype, D ** -0.5, max_seq_tokens=40, max_kv_tokens=300)
        rc, need = L.lsc_kv_attend_workspace_bytes(dev.pool, a)
        ws = torch.zeros(max(need, 1), dtype=torch.uint8, device="cuda")
        a.workspace, a.workspace_bytes = ws.data_ptr(), need
        step_args = L.kv_append_rotated_args(L.kv_append_args(batch, k, v, dtype), r, H * G, q, turned)

        def step(stream):
            assert L.lsc_kv_append_rotated(dev.pool, 0, step_args, stream) == L.LSC_OK
            assert L.lsc_kv_attend(dev.pool, 0, a, stream) == L.LSC_OK

        side.wait_stream(cur())
        with torch.cuda.stream(side):
            step(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(torch.cuda.current_stream())
        for b in batches:
            for lane in (0, 1):
                for i in range(S):
                    bl, rr = b.places(i, 0, int(b.kv[i]))
                    host.write(0, lane, bl, rr, rng.standard_normal((len(bl), H, D)))
            dev.buf.copy_(torch.from_numpy(host.bytes.reshape(-1)))
            t = np.zeros((S, wide), np.int32)
            t[:, :b.table.shape[1]] = b.table
            for d, s in ((table, t), (cu, b.cu), (kvl, b.kv.astype(np.int32))):
                d.copy_(torch.from_numpy(s))
            p = rng.integers(0, 5000, (3, T)).astype(np.int32)
            pos.copy_(torch.from_numpy(p))
            (kd, kx), (vd, vx), (qd, qx) = (dense(rng.standard_normal((T, h, D)), dtype) for h in (H, H, H * G))
            for d, s in ((k, kd), (v, vd), (q, qd)):
                d.copy_(s)
            graph.replay()
            got = dev.download()
            assert dev.status() == L.LSC_OK
            n = int(b.cu[-1])
            want, size = turn(qx, R, angles(p, freqs(R), axis), False)
            tq = turned.double().cpu().numpy().reshape(T, H * G, D)
            check(tq[:n], want[:n], size[:n], dtype)
            held = host_pool(pool, blocks, bt, H, D, layers=1)
            held.bytes[:] = got
            o = out[:n].clone()
            short = Batch.__new__(Batch)
            short.__dict__.update(b.__dict__)
            short.T = n
            (check4 if pool == L.LSC_E2M1 else check_attend)(held, 0, short, tq[:n], dtype, D ** -0.5, True, o, None)


@pytest.mark.parametrize("D,R", [(128, 64), (80, 20)])
def test_a_row_expanded_to_every_axis(lsc, D, R):
    """positions.expand(axes, T), each axis the same row: as the row alone, out of place and with the append."""
    rng = np.random.default_rng(R)
    T, H, Hq = 37, 2, 3
    p = rng.integers(0, 5000, T).astype(np.int32)
    pos = torch.from_numpy(p).cuda()
    axis = (np.arange(R // 2) % 3).astype(np.uint8)
    x, xx = dense(rng.standard_normal((T, Hq, D)), BF)
    k, kx = dense(rng.standard_normal((T, H, D)), BF)
    want, size = turn(xx, R, angles(p[None], freqs(R), None), False)
    kw, ksize = turn(kx, R, angles(p[None], freqs(R), None), False)
    host = host_pool(BF, 10, 16, H, D)
    b = Batch(rng, [T], [T + 9], 16, 10)
    for rows in (pos.expand(3, T), pos[None].expand(3, T)):
        r = L.rotary(R, rows, freqs(R), pair_axis=axis)
        out = torch.full_like(x, 7.0)
        assert L.lsc_rotate(L.rotate_args(T, Hq, D, BF, x, out, r), cur()) == L.LSC_OK
        check(out.double().cpu().numpy().reshape(T, Hq, D), want, size, BF)
        out.fill_(7.0)
        with DevKv(host) as dev:
            args = L.kv_append_rotated_args(L.kv_append_args(b.device(), k, k, BF), r, Hq, x, out)
            assert L.lsc_kv_append_rotated(dev.pool, 1, args, cur()) == L.LSC_OK
            assert dev.status() == L.LSC_OK
            host.bytes[:] = dev.download()
        check(out.double().cpu().numpy().reshape(T, Hq, D), want, size, BF)
        check(host.read(1, 0, *b.places(0, 9, T + 9)), kw, ksize, BF)
