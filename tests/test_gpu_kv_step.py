"""GPU: append, gather and attend over a layer of the K/V block pool against
their plain 64-bit forms (tests/_kv.py): every type, odd sizes and blocks,
strides, lengths of zero and one, rows behind the last sequence, rows that see
nothing, NaN wherever nothing may be read, bad blocks and lengths, other
streams, captured graphs, and a run of the calls as a step uses them.

Tolerances.  append and gather move or round once: equal bits.  attend: a score
is a sum of D products in 32 bits, off by at most D 2^-23 times the sum of their
magnitudes (`reach`; 2^-23 and not 2^-24 because the tensor cores cut off what
they align), which changes a weight by that share, above and below the bar: 2
D 2^-23 reach.  The weights of the 16-bit forms are rounded to 16 bits (half a
step: 2^-8 bf16, 2^-11 f16) before they meet v; f16 weights below 2^-14 are off
by 2^-25 at most, each times |v|.  E4M3 pools round them to f16 times v's
scale (chunks with bf16 q: to nine significant bits or more, which is within bf16's share).  The sums of N terms in 32 bits add N 2^-23.  All of that times the sum of
weight times |v| (`mass`), and the output is rounded once, half a step of the
result.  exp2 and log2 are good to 2^-21.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from linear_attention_state_lsc_gb300 import lsc as L

import _kv
from _kv import ES, NAME, TORCH, Batch, DevKv, HostKv

pytestmark = pytest.mark.gpu

FLOATS = [L.LSC_F32, L.LSC_BF16, L.LSC_F16]
POOLS = FLOATS + [L.LSC_E4M3]
HALF = {L.LSC_F32: 2.0 ** -24, L.LSC_BF16: 2.0 ** -8, L.LSC_F16: 2.0 ** -11}


def cur():
    return torch.cuda.current_stream()


def dense(x, dtype, stride=None):
    """float64 [T, H, D] -> (device buffer, its values as float64); a row every `stride` elements, NaN between."""
    T, H, D = x.shape
    t = torch.full((T, stride or H * D), float("nan"), dtype=TORCH[dtype])
    t[:, :H * D] = torch.from_numpy(x).float().reshape(T, -1).to(TORCH[dtype])
    return t.cuda(), t[:, :H * D].double().numpy().reshape(T, H, D)


def step_lengths(name):
    """(new tokens, cached tokens)"""
    return {"decode": ([1, 1, 1], [1, 70, 33]),
            "ragged": ([5, 0, 1, 17, 3], [5, 9, 64, 40, 0]),  # a whole prompt, nothing new, a block border, an empty cache
            "ahead": ([9, 4], [6, 4])}[name]                  # more new tokens than the cache holds


# ---- append ---------------------------------------------------------------------

@pytest.mark.parametrize("pool", POOLS, ids=NAME.get)
@pytest.mark.parametrize("dtype", FLOATS, ids=NAME.get)
@pytest.mark.parametrize("shape", [(16, 2, 64), (7, 3, 24), (5, 1, 33), (64, 2, 256)], ids=str)
def test_append(lsc, pool, dtype, shape):
    """Vector and element kernels; whole pool compared, so nothing else changed."""
    bt, H, D = shape
    rng = np.random.default_rng(bt * D)
    for name, stride in (("ragged", 0), ("ahead", H * D + 8), ("decode", H * D + 3)):
        n, kv = step_lengths(name)
        host = HostKv(30, bt, H, D, pool)
        b = Batch(rng, n, kv, bt, 30, spare=3, wide=2)
        x = rng.standard_normal((2, b.T, H, D)) * np.exp(2 * rng.standard_normal((2, b.T, H, 1)))
        x[0, 0] = 0
        x[:, -3:] = np.nan  # rows of no sequence: not read into the pool
        (k, kx), (v, vx) = (dense(y, dtype, stride or None) for y in x)
        with DevKv(host) as dev:
            args = L.kv_append_args(b.device(), k, v, dtype, stride, stride)
            assert L.lsc_kv_append(dev.pool, 1, args, cur()) == L.LSC_OK
            got = dev.download()
            assert dev.status() == L.LSC_OK
        for i in range(len(n)):
            first = max(0, n[i] - kv[i])  # tokens of negative positions have no row
            bl, r = b.places(i, max(0, kv[i] - n[i]), kv[i])
            for lane, y in enumerate((kx, vx)):
                host.write(1, lane, bl, r, y[b.cu[i] + first:b.cu[i + 1]])
        np.testing.assert_array_equal(got, host.bytes)


def test_append_quantises_border_values(lsc):
    """Rows whose largest magnitude sits at, just below and just above 448 times a power of two, ties between codes,
    tiny and huge rows, zeros of both signs, infinities and NaN: codes and scale bytes as the definition says."""
    H, D = 1, 16
    rows = []
    for e in (-140, -133, -127, -20, 0, 7, 30, 119):
        for top in (448.0, np.nextafter(np.float32(448), np.float32(0)), np.nextafter(np.float32(448), np.float32(500)),
                    256.0, 449.0, 1.0):
            r = np.linspace(-1, 1, D) * top * 0.9
            r[3] = top
            r[4:8] = np.array([17.0, 19.0, -21.0, 23.0]) / 32 * top / 448  # ties of small steps among them
            rows.append(np.float32(r) * np.float64(2.0) ** e)
    x = np.stack(rows)
    ties = np.concatenate([(_kv._POS[:-1] + _kv._POS[1:]) / 2, -_kv._POS])
    ties = np.pad(ties, (0, -len(ties) % (D - 1))).reshape(-1, D - 1)
    x = np.concatenate([x, np.concatenate([np.full((len(ties), 1), 448.0), ties], 1)])
    special = np.zeros((4, D))
    special[0] = -0.0
    special[1, 5], special[2, 6], special[3, 7] = np.inf, np.nan, -np.inf
    x = np.float64(np.float32(np.concatenate([x, special])))[:, None]
    T = len(x)
    host = HostKv(T // 8 + 1, 8, H, D, L.LSC_E4M3)
    b = Batch(np.random.default_rng(0), [T], [T], 8, T // 8 + 1)
    k, kx = dense(x, L.LSC_F32)
    with DevKv(host) as dev:
        assert L.lsc_kv_append(dev.pool, 0, L.kv_append_args(b.device(), k, k, L.LSC_F32), cur()) == L.LSC_OK
        got = dev.download()
    bl, r = b.places(0, 0, T)
    for lane in (0, 1):
        host.write(0, lane, bl, r, kx)
    np.testing.assert_array_equal(got, host.bytes)
    up = host.scales(0, 0)[bl, r][:, 0]
    assert (up[-3:] == 255).all() and up[-4] == 0


# ---- gather ---------------------------------------------------------------------

@pytest.mark.parametrize("pool", POOLS, ids=NAME.get)
@pytest.mark.parametrize("dtype", FLOATS, ids=NAME.get)
@pytest.mark.parametrize("shape", [(16, 2, 64), (7, 3, 24), (5, 1, 33), (64, 2, 256)], ids=str)
def test_gather(lsc, pool, dtype, shape):
    bt, H, D = shape
    rng = np.random.default_rng(bt + D)
    for name, stride in (("ragged", 0), ("ahead", H * D + 8), ("decode", H * D + 3)):
        n, kv = step_lengths(name)
        host = HostKv(30, bt, H, D, pool)
        b = Batch(rng, n, kv, bt, 30, spare=2, wide=1)
        for i in range(len(n)):
            bl, r = b.places(i, 0, kv[i])
            for lane in (0, 1):
                host.write(1, lane, bl, r, rng.standard_normal((kv[i], H, D)) * 3)
        w = stride or H * D
        k, v = (torch.full((b.T, w), 7.0, dtype=TORCH[dtype], device="cuda") for _ in "kv")
        with DevKv(host) as dev:
            args = L.kv_gather_args(b.device(), k, v, dtype, stride, stride)
            assert L.lsc_kv_gather(dev.pool, 1, args, cur()) == L.LSC_OK
            assert dev.status() == L.LSC_OK
        for lane, y in enumerate((k, v)):
            want = torch.full((b.T, w), 7.0, dtype=TORCH[dtype])
            for i in range(len(n)):
                first = max(0, n[i] - kv[i])
                bl, r = b.places(i, max(0, kv[i] - n[i]), kv[i])
                x = torch.from_numpy(host.read(1, lane, bl, r)).float().reshape(-1, H * D).to(TORCH[dtype])
                want[b.cu[i]:b.cu[i] + first, :H * D] = 0
                want[b.cu[i] + first:b.cu[i + 1], :H * D] = x
            assert torch.equal(y.cpu().view(torch.uint8), want.view(torch.uint8))


def test_gather_of_every_code_and_scale(lsc):
    """All 256 codes under scale bytes from one end to the other, to each float type: code times scale, rounded once
    (f16: to infinity beyond its range)."""
    host = HostKv(40, 8, 1, 256, L.LSC_E4M3)
    b = Batch(np.random.default_rng(1), [300], [300], 8, 40)
    bl, r = b.places(0, 0, 300)
    up = np.concatenate([np.arange(256), np.arange(100, 144)]).astype(np.uint8)
    for lane in (0, 1):
        host.rows(0, lane)[bl, r, 0] = np.arange(256, dtype=np.uint8)
        host.scales(0, lane)[bl, r, 0] = up
    want = host.read(0, 0, bl, r).reshape(300, 256)
    with DevKv(host) as dev:
        for dtype in FLOATS:
            k, v = (torch.zeros(300, 256, dtype=TORCH[dtype], device="cuda") for _ in "kv")
            assert L.lsc_kv_gather(dev.pool, 0, L.kv_gather_args(b.device(), k, v, dtype), cur()) == L.LSC_OK
            w = torch.from_numpy(want).float().to(TORCH[dtype])  # 4 significant bits: exact in fp32 down to 2^-136
            for got in (k.cpu(), v.cpu()):
                assert torch.equal(torch.isnan(got), torch.isnan(w))
                assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(w))


# ---- attend ---------------------------------------------------------------------

def filled(rng, b, blocks, bt, H, D, pool, layers=2, layer=1):
    host = HostKv(blocks, bt, H, D, pool, layers=layers)
    gain = np.exp(0.5 * rng.standard_normal((1, H, D)))
    for i in range(len(b.n)):
        bl, r = b.places(i, 0, int(b.kv[i]))
        host.write(layer, 0, bl, r, rng.standard_normal((len(r), H, D)) * gain)
        host.write(layer, 1, bl, r, rng.standard_normal((len(r), H, D)) * np.exp(rng.standard_normal((len(r), H, 1))))
    return host


def run_attend(dev, layer, b, q, dtype, Hq, scale, causal, stride=0, lse=True, **bounds):
    T, D = b.T, dev.host.D
    w = stride or Hq * D
    out = torch.full((T, w), 7.0, dtype=TORCH[dtype], device="cuda")
    ls = torch.full((T, Hq), 7.0, device="cuda") if lse else None
    args = L.kv_attend_args(b.device(), Hq, q, out, dtype, scale, lse=ls, causal=causal, q_stride=stride,
                            out_stride=stride, **bounds)
    rc, need = L.lsc_kv_attend_workspace_bytes(dev.pool, args)
    assert rc == L.LSC_OK
    ws = torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    args.workspace, args.workspace_bytes = ws.data_ptr(), need
    assert L.lsc_kv_attend(dev.pool, layer, args, cur()) == L.LSC_OK
    torch.cuda.synchronize()
    return out, ls


def check_attend(host, layer, b, qx, dtype, scale, causal, out, ls, rows=None):
    T, Hq, D = qx.shape
    want, lse, mass, reach, vmax = _kv.attend(host, layer, b, qx, scale, causal)
    got = out[:, :Hq * D].double().cpu().numpy().reshape(T, Hq, D)
    N = float(b.kv.max(initial=1))
    es = D * 2.0 ** -23 * reach
    weight = {L.LSC_F32: 0.0, L.LSC_BF16: HALF[L.LSC_BF16], L.LSC_F16: HALF[L.LSC_F16]}[dtype]
    rel = weight + 2 * es + (N + 8) * 2.0 ** -23 + 2.0 ** -20
    tail = N * 2.0 ** -25 * vmax if dtype != L.LSC_F32 else 0 * vmax
    bound = rel[..., None] * mass + tail[..., None] + HALF[dtype] * (np.abs(want) + rel[..., None] * mass) + 1e-30
    keep = slice(0, int(b.cu[-1])) if rows is None else rows
    over = np.abs(got - want)[keep] / bound[keep]
    assert np.isfinite(got[keep]).all()
    assert over.max(initial=0) <= 1, (over.max(), np.unravel_index(over.argmax(), over.shape))
    if ls is not None:
        l = ls.double().cpu().numpy()[keep]
        np.testing.assert_array_equal(np.isinf(l), np.isinf(lse[keep]))
        f = np.isfinite(lse[keep])
        lim = es[keep] + (N + 8) * 2.0 ** -23 + 2.0 ** -20 * (1 + np.abs(np.where(f, lse[keep], 0)))
        assert (np.abs(np.where(f, l - np.where(f, lse[keep], 0), 0)) <= lim).all()
    assert (out[int(b.cu[-1]):] == 7).all() and (ls is None or (ls[int(b.cu[-1]):] == 7).all())
    if out.shape[1] > Hq * D:
        assert (out[:, Hq * D:] == 7).all()


MIXES = [(L.LSC_BF16, L.LSC_BF16), (L.LSC_F16, L.LSC_F16), (L.LSC_E4M3, L.LSC_BF16), (L.LSC_E4M3, L.LSC_F16),
         (L.LSC_F32, L.LSC_F32), (L.LSC_BF16, L.LSC_F32), (L.LSC_E4M3, L.LSC_F32)]
# (new, cached) per sequence
LENGTHS = {
    "one": ([1], [1]),
    "decode": ([1] * 6, [1, 63, 64, 65, 200, 0]),                     # an empty cache among them
    "few": ([2, 3, 1, 4], [2, 130, 257, 64]),
    "chunk": ([40, 1, 0, 129], [40, 300, 17, 200]),
    "ahead": ([20, 70], [12, 66]),                                     # rows that see nothing
    "long": ([3, 1], [1500, 2049]),
    "whole": ([300, 2, 77], [300, 500, 770]),                          # a first prompt, a decode, a resumed prompt
}


@pytest.mark.parametrize("mix", MIXES, ids=lambda m: NAME[m[0]] + "-" + NAME[m[1]])
@pytest.mark.parametrize("name", list(LENGTHS))
@pytest.mark.parametrize("shape", [(16, 2, 4, 64), (64, 1, 8, 128), (24, 2, 5, 128), (64, 2, 8, 256), (5, 1, 3, 33)], ids=str)
def test_attend(lsc, mix, name, shape):
    pool, dtype = mix
    bt, H, G, D = shape
    rng = np.random.default_rng(abs(hash((pool, dtype, len(name), bt, D))) % 2 ** 31)
    n, kv = LENGTHS[name]
    blocks = int(sum(-(-k // bt) for k in kv)) + 3
    b = Batch(rng, n, kv, bt, blocks, spare=2, wide=1)
    host = filled(rng, b, blocks, bt, H, D, pool)
    q, qx = dense(2 * rng.standard_normal((b.T, H * G, D)), dtype)
    scale = D ** -0.5
    with DevKv(host) as dev:
        for causal in (True, False):
            out, ls = run_attend(dev, 1, b, q, dtype, H * G, scale, causal, max_seq_tokens=max(n), max_kv_tokens=max(max(kv), 1))
            check_attend(host, 1, b, qx, dtype, scale, causal, out, ls)
            again, _ = run_attend(dev, 1, b, q, dtype, H * G, scale, causal, lse=False)  # without bounds
            check_attend(host, 1, b, qx, dtype, scale, causal, again, None)
        assert dev.status() == L.LSC_OK
        np.testing.assert_array_equal(dev.download(), host.bytes)


@pytest.mark.parametrize("mix", MIXES, ids=lambda m: NAME[m[0]] + "-" + NAME[m[1]])
@pytest.mark.parametrize("shape", [(16, 2, 4, 64), (64, 1, 8, 128), (64, 1, 3, 256)], ids=str)
@pytest.mark.parametrize("n", [3, 90])
def test_what_a_row_does_not_see_does_not_enter(lsc, mix, shape, n):
    """K and V of some new tokens are NaN and infinite: earlier rows of the causal chunk are as if they were not there,
    the rows that see them get what the sum gives (an infinity, or NaN)."""
    pool, dtype = mix
    bt, H, G, D = shape
    rng = np.random.default_rng(n + D)
    kv = 150
    b = Batch(rng, [n, 1], [kv, 20], bt, 30)
    host = filled(rng, b, 30, bt, H, D, pool)
    bl, r = b.places(0, 0, kv)
    x = host.read(1, 1, bl, r)
    first = kv - n + 1 + (n - 2) // 2  # the first position whose v is not finite: the row before it does not see it
    x[first, :, 3] = np.inf
    x[first, :, 7] = -np.inf
    x[-1, :, 3] = -np.inf
    x[-1, :, 11] = np.nan
    host.write(1, 1, bl, r, x)
    k = host.read(1, 0, bl, r)
    k[-1] = np.nan  # the last token's scores: seen by the last row alone
    host.write(1, 0, bl, r, k)
    q, qx = dense(rng.standard_normal((b.T, H * G, D)), dtype)
    scale = D ** -0.5
    sees = first - (kv - n)  # new tokens below this one see finite values alone
    with DevKv(host) as dev:
        out, ls = run_attend(dev, 1, b, q, dtype, H * G, scale, True, max_seq_tokens=n)
    clean = np.r_[0:sees, n]
    k[-1] = 0  # scores that no clean row sees
    host.write(1, 0, bl, r, np.nan_to_num(k))
    host.write(1, 1, bl, r, np.nan_to_num(x, nan=0, posinf=0, neginf=0))
    check_attend(host, 1, b, qx, dtype, scale, True, out, ls, rows=clean)
    got = out.float().cpu().numpy().reshape(b.T, H * G, D)
    if pool == L.LSC_E4M3:  # a row that held one is NaN throughout
        assert np.isnan(got[sees:n]).all()
    else:
        assert np.isnan(got[n - 1]).all()
        assert (got[sees:n - 1, :, 3] == np.inf).all() and (got[sees:n - 1, :, 7] == -np.inf).all()
        assert np.isfinite(np.delete(got[sees:n - 1], [3, 7], -1)).all()


@pytest.mark.parametrize("pool,D", [(L.LSC_BF16, 64), (L.LSC_BF16, 256), (L.LSC_E4M3, 128), (L.LSC_E4M3, 256)])
@pytest.mark.parametrize("S", [3, 31, 60])
def test_runs_that_begin_and_end_anywhere(lsc, pool, D, S):
    """Many short units beside long ones: runs end before, inside and behind a unit's tiles."""
    rng = np.random.default_rng(71 + S)
    n = rng.integers(0, 12, S)
    kv = np.where(rng.random(S) < 0.3, rng.integers(1100, 2500, S), rng.integers(1, 300, S)) + n
    blocks = int((-(-kv // 64)).sum())
    b = Batch(rng, n, kv, 64, blocks, spare=1)
    host = filled(rng, b, blocks, 64, 2, D, pool)
    q, qx = dense(2 * rng.standard_normal((b.T, 32, D)), L.LSC_BF16)
    with DevKv(host) as dev:
        out, ls = run_attend(dev, 1, b, q, L.LSC_BF16, 32, D ** -0.5, True)
        check_attend(host, 1, b, qx, L.LSC_BF16, D ** -0.5, True, out, ls)
        assert dev.status() == L.LSC_OK


def test_attend_strides_and_slices(lsc):
    """q and out as slices of wider arrays, aligned (tensor cores) and not (CUDA cores)."""
    rng = np.random.default_rng(5)
    H, G, D, bt = 2, 4, 128, 16
    b = Batch(rng, [2, 60], [100, 200], bt, 30, spare=1)
    host = filled(rng, b, 30, bt, H, D, L.LSC_BF16)
    x = rng.standard_normal((b.T, H * G, D))
    with DevKv(host) as dev:
        for stride in (H * G * D + 256, H * G * D + 8, H * G * D + 1):
            q, qx = dense(x, L.LSC_BF16, stride)
            out, ls = run_attend(dev, 1, b, q, L.LSC_BF16, H * G, D ** -0.5, True, stride=stride)
            check_attend(host, 1, b, qx, L.LSC_BF16, D ** -0.5, True, out, ls)


def test_bad_batches_are_recorded_and_stay_inside(lsc):
    """Block ids, lengths and cu_seqlens that do not fit: the status word says so, the other sequences are right, and
    nothing outside the named rows changes."""
    rng = np.random.default_rng(6)
    H, G, D, bt, blocks = 2, 2, 64, 16, 30
    b = Batch(rng, [1, 3, 2, 1], [40, 50, 60, 33], bt, blocks, wide=1)
    host = filled(rng, b, blocks, bt, H, D, L.LSC_BF16)
    q, qx = dense(rng.standard_normal((b.T, H * G, D)), L.LSC_BF16)
    k, _ = dense(rng.standard_normal((b.T, H, D)), L.LSC_BF16)
    good = np.r_[0:1, 4:7]  # sequence 1 is the one that breaks

    def calls(dev, batch):
        out = torch.full((b.T, H * G * D), 7.0, dtype=torch.bfloat16, device="cuda")
        ls = torch.full((b.T, H * G), 7.0, device="cuda")
        g = [torch.full((b.T, H * D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        codes = []
        for call, args in ((L.lsc_kv_attend, L.kv_attend_args(batch, H * G, q, out, L.LSC_BF16, 0.125, lse=ls)),
                           (L.lsc_kv_gather, L.kv_gather_args(batch, *g, L.LSC_BF16)),
                           (L.lsc_kv_append, L.kv_append_args(batch, k, k, L.LSC_BF16))):
            assert call(dev.pool, 1, args, cur()) == L.LSC_OK
            codes.append(dev.status())
        return codes, out, ls, g

    for bad in (blocks, -1, 2 ** 31 - 1):
        b.device()
        with DevKv(host) as dev:
            table = b.table.copy()
            table[1, 50 // bt] = bad  # holds position 49, and 48: the last two of sequence 1's three
            t = torch.from_numpy(table).cuda()
            batch = L.kv_batch(4, b.T, t, b.dev[1], b.dev[2], max_blocks=table.shape[1])
            codes, out, ls, g = calls(dev, batch)
            assert codes == [L.LSC_ERR_OUT_OF_RANGE] * 3
            check_attend(host, 1, b, qx, L.LSC_BF16, 0.125, True, out, ls, rows=good)
            assert (g[0][2:4] == 0).all() and (g[0][1] != 0).any()
            assert dev.status() == L.LSC_OK  # cleared
    for kv1 in (-1, 1 << 20, 2 ** 31 - 1):
        with DevKv(host) as dev:
            kv = b.kv.astype(np.int32).copy()
            kv[1] = kv1
            t = torch.from_numpy(kv).cuda()
            batch = L.kv_batch(4, b.T, b.dev[0], b.dev[1], t, max_blocks=b.table.shape[1])
            codes, out, ls, g = calls(dev, batch)
            assert codes == [L.LSC_ERR_INVALID_ARG] * 3
            check_attend(host, 1, b, qx, L.LSC_BF16, 0.125, True, out, ls, rows=good)
            assert (out[1:4] == 0).all() and torch.isinf(ls[1:4]).all() and (g[0][1:4] == 0).all()
    for cu in ([0, 5, 4, 6, 7], [0, 1, 4, 6, 9], [3, 4, 5, 6, 7], [0, -4, 4, 6, 7], [-2 ** 31, 1, 4, 6, 2 ** 31 - 1]):
        with DevKv(host) as dev:
            t = torch.tensor(cu, dtype=torch.int32, device="cuda")
            batch = L.kv_batch(4, b.T, b.dev[0], t, b.dev[2], max_blocks=b.table.shape[1])
            codes, out, ls, g = calls(dev, batch)
            assert codes == [L.LSC_ERR_INVALID_ARG] * 3


def test_bounds_that_do_not_hold_are_recorded(lsc):
    rng = np.random.default_rng(7)
    b = Batch(rng, [1, 1], [40, 400], 16, 40)
    host = filled(rng, b, 40, 16, 2, 64, L.LSC_BF16)
    q, qx = dense(rng.standard_normal((b.T, 4, 64)), L.LSC_BF16)
    with DevKv(host) as dev:
        out, ls = run_attend(dev, 1, b, q, L.LSC_BF16, 4, 0.125, True, max_seq_tokens=1, max_kv_tokens=100)
        assert dev.status() == L.LSC_ERR_INVALID_ARG
        check_attend(host, 1, b, qx, L.LSC_BF16, 0.125, True, out, ls, rows=np.r_[0:1])
        assert (out[1] == 0).all() and torch.isinf(ls[1]).all()


def test_overlapping_sequences_that_count_past_31_bits_stay_inside(lsc):
    """cu_seqlens goes up and down, so that one set of rows counts 130056 times: 32 units of 1024 tiles and 8 more counts
    each are 2^32 + 2048.  It is recorded and nothing is written."""
    S, T, G, D, bt = 2 * 130056, 64, 64, 256, 65536
    assert (S // 2 * 32 * (1024 + 8)) % 2 ** 32 == 2048
    for kv in (bt, bt - 3 * 64):
        with DevKv(HostKv(1, bt, 1, D, L.LSC_BF16, pad=0, layers=1)) as dev:
            cu = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
            cu[1::2] = T
            table = torch.zeros((S, 1), dtype=torch.int32, device="cuda")
            lens = torch.full((S,), kv, dtype=torch.int32, device="cuda")
            q = torch.zeros((T, G * D), dtype=torch.bfloat16, device="cuda")
            out = torch.full_like(q, 7)
            args = L.kv_attend_args(L.kv_batch(S, T, table, cu, lens, max_blocks=1), G, q, out, L.LSC_BF16, 0.125,
                                    causal=False)
            assert L.lsc_kv_attend(dev.pool, 0, args, cur()) == L.LSC_OK
            assert dev.status() == L.LSC_ERR_INVALID_ARG and (out == 7).all()


@pytest.mark.parametrize("pool,dtype,G,bound", [(L.LSC_F32, L.LSC_F32, 2, 1), (L.LSC_BF16, L.LSC_BF16, 4, 2),
                                                (L.LSC_E4M3, L.LSC_F16, 8, 2), (L.LSC_F16, L.LSC_F16, 32, 2),
                                                (L.LSC_BF16, L.LSC_BF16, 64, 2), (L.LSC_E4M3, L.LSC_BF16, 64, 2)])
def test_a_sequence_of_too_many_new_tokens_stays_as_it_was(lsc, pool, dtype, G, bound):
    """Every form of the kernel; the sequence's table row is the last one and full, so reading on would leave it."""
    rng = np.random.default_rng(70)
    b = Batch(rng, [bound, 9], [40, 16 * 12], 16, 40)
    assert b.table.shape[1] == 12
    host = filled(rng, b, 40, 16, 1, 64, pool)
    q, qx = dense(rng.standard_normal((b.T, G, 64)), dtype)
    with DevKv(host) as dev:
        out, ls = run_attend(dev, 1, b, q, dtype, G, 0.125, True, max_seq_tokens=bound)
        assert dev.status() == L.LSC_ERR_INVALID_ARG
        check_attend(host, 1, b, qx, dtype, 0.125, True, out, ls, rows=np.r_[0:bound])
        assert (out[bound:] == 7).all() and (ls[bound:] == 7).all()


@pytest.mark.parametrize("pool", [L.LSC_BF16, L.LSC_E4M3], ids=NAME.get)
def test_a_step_on_its_own_stream_in_a_graph(lsc, pool):
    """append, attend and gather of each layer, captured once on a side stream and replayed with other lengths, tables
    and values: two graphs with workspaces of their own, replayed in turn; two calls give the same bits."""
    rng = np.random.default_rng(8)
    H, G, D, bt, blocks, S = 2, 8, 256, 64, 200, 5
    mixes = [([1, 1, 2, 1, 1], [1, 700, 64, 1300, 65]), ([1, 2, 1, 1, 1], [2000, 3, 128, 100, 1])]
    batches = [Batch(rng, n, kv, bt, blocks) for n, kv in mixes]
    wide = max(b.table.shape[1] for b in batches)
    table = torch.zeros(S, wide, dtype=torch.int32, device="cuda")
    cu, kvl = torch.zeros(S + 1, dtype=torch.int32, device="cuda"), torch.zeros(S, dtype=torch.int32, device="cuda")
    T = max(b.T for b in batches)
    q, k, v = (torch.zeros(T, h * D, dtype=torch.bfloat16, device="cuda") for h in (H * G, H, H))
    host = HostKv(blocks, bt, H, D, pool, layers=2, fill=0)
    side = torch.cuda.Stream()
    with DevKv(host) as dev:
        runs = []
        for _ in range(2):
            out = [torch.zeros(T, H * G * D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            gk = [torch.zeros(T, H * D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            batch = L.kv_batch(S, T, table, cu, kvl, max_blocks=wide)
            a = L.kv_attend_args(batch, H * G, q, out[0], L.LSC_BF16, D ** -0.5, max_seq_tokens=2, max_kv_tokens=2000)
            rc, need = L.lsc_kv_attend_workspace_bytes(dev.pool, a)
            ws = torch.zeros(need, dtype=torch.uint8, device="cuda")

            def step(stream):
                for l in range(2):
                    ar = L.kv_attend_args(batch, H * G, q, out[l], L.LSC_BF16, D ** -0.5, max_seq_tokens=2,
                                          max_kv_tokens=2000, workspace=ws, workspace_bytes=need)
                    assert L.lsc_kv_append(dev.pool, l, L.kv_append_args(batch, k, v, L.LSC_BF16), stream) == L.LSC_OK
                    assert L.lsc_kv_attend(dev.pool, l, ar, stream) == L.LSC_OK
                    assert L.lsc_kv_gather(dev.pool, l, L.kv_gather_args(batch, gk[l], gk[l], L.LSC_BF16), stream) == L.LSC_OK

            side.wait_stream(cur())
            with torch.cuda.stream(side):
                step(side)  # kernels loaded before the capture
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                step(torch.cuda.current_stream())
            runs.append((graph, out, gk, ws))
        for b in batches:
            x = rng.standard_normal((2, blocks, bt, H, D)) * 2
            for l in range(2):
                for lane in (0, 1):
                    for i in range(S):
                        bl, r = b.places(i, 0, int(b.kv[i]))
                        host.write(l, lane, bl, r, x[lane][bl, r] * (l + 1))
            dev.buf.copy_(torch.from_numpy(host.bytes.reshape(-1)))
            t = np.zeros((S, wide), np.int32)
            t[:, :b.table.shape[1]] = b.table
            table.copy_(torch.from_numpy(t))
            cu.copy_(torch.from_numpy(b.cu))
            kvl.copy_(torch.from_numpy(b.kv.astype(np.int32)))
            (kd, kx), (vd, vx), (qd, qx) = (dense(rng.standard_normal((b.T, h, D)), L.LSC_BF16) for h in (H, H, H * G))
            for a, s in ((k, kd), (v, vd), (q, qd)):
                a[:b.T].copy_(s)
            for graph, out, gk, ws in runs:
                ws.fill_(255)
                graph.replay()
            torch.cuda.synchronize()
            assert dev.status() == L.LSC_OK
            for i in range(S):
                bl, r = b.places(i, int(b.kv[i] - b.n[i]), int(b.kv[i]))
                for l in range(2):
                    host.write(l, 0, bl, r, kx[b.cu[i]:b.cu[i + 1]])
                    host.write(l, 1, bl, r, vx[b.cu[i]:b.cu[i + 1]])
            np.testing.assert_array_equal(dev.download(), host.bytes)
            for l in range(2):
                assert torch.equal(runs[0][1][l], runs[1][1][l])
                check_attend(host, l, b, qx, L.LSC_BF16, D ** -0.5, True, runs[0][1][l][:b.T], None)


def test_waits_that_run_out_are_reported(tmp_path):
    """With the injected fault every bounded wait gives up at once: the chunk kernel returns, the status word says so,
    and the next call in a clean process is right."""
    code = """
import sys
sys.path[:0] = [%r, %r]
import numpy as np, torch
import test_gpu_kv_step as T
from _kv import Batch, DevKv
from linear_attention_state_lsc_gb300 import lsc as L
rng = np.random.default_rng(3)
for D in (64, 128, 256):
    b = Batch(rng, [70], [300], 64, 10)
    host = T.filled(rng, b, 10, 64, 1, D, L.LSC_BF16)
    q, _ = T.dense(rng.standard_normal((70, 4, D)), L.LSC_BF16)
    with DevKv(host) as dev:
        T.run_attend(dev, 1, b, q, L.LSC_BF16, 4, 0.1, True)
        assert dev.status() == L.LSC_ERR_DEV_TIMEOUT
print("reported")
"""
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", code % (os.path.dirname(here), here)], capture_output=True, text=True,
                       env=dict(os.environ, LSC_FAULT="timeout0"), timeout=300)
    assert "reported" in r.stdout, r.stderr[-2000:]


def test_workspace_rules(lsc):
    """Too small a workspace is refused; without one the library finds its own; both give the same bits."""
    rng = np.random.default_rng(9)
    b = Batch(rng, [1, 1], [300, 900], 64, 30)
    host = filled(rng, b, 30, 64, 2, 128, L.LSC_BF16)
    q, qx = dense(rng.standard_normal((b.T, 8, 128)), L.LSC_BF16)
    with DevKv(host) as dev:
        out, ls = run_attend(dev, 1, b, q, L.LSC_BF16, 8, 0.1, True)
        own = torch.zeros_like(out)
        args = L.kv_attend_args(b.device(), 8, q, own, L.LSC_BF16, 0.1)
        rc, need = L.lsc_kv_attend_workspace_bytes(dev.pool, args)
        assert rc == L.LSC_OK and need > 0
        assert L.lsc_kv_attend(dev.pool, 1, args, cur()) == L.LSC_OK
        torch.cuda.synchronize()
        assert torch.equal(own, out)
        ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
        args.workspace, args.workspace_bytes = ws.data_ptr(), need - 1
        assert L.lsc_kv_attend(dev.pool, 1, args, cur()) == L.LSC_ERR_INVALID_ARG


def test_many_sequences_and_a_block_far_into_the_pool(lsc):
    """More sequences than a CTA has threads, empty ones among them; and pages whose byte offset passes 32 bits."""
    rng = np.random.default_rng(10)
    S = 700
    kv = rng.integers(0, 40, S)
    b = Batch(rng, np.minimum(1, kv), kv, 16, int((-(-kv // 16)).sum()))
    host = filled(rng, b, int((-(-kv // 16)).sum()), 16, 1, 64, L.LSC_BF16)
    q, qx = dense(rng.standard_normal((b.T, 2, 64)), L.LSC_BF16)
    with DevKv(host) as dev:
        for seen in (True, False):
            out, ls = run_attend(dev, 1, b, q, L.LSC_BF16, 2, 0.125, seen, max_seq_tokens=1)
            check_attend(host, 1, b, qx, L.LSC_BF16, 0.125, seen, out, ls)
    far = HostKv(6, 16, 1, 64, L.LSC_BF16, pad=0, layers=1)
    page = 1 << 30  # six pages of 1 GiB: lanes of 6 GiB
    desc = L.lsc_kv_pool_desc(1, 6, 16, 1, 64, L.LSC_BF16, page)
    buf = torch.empty(12 * page, dtype=torch.uint8, device="cuda")
    rc, pool = L.lsc_kv_pool_create(desc, buf, buf.numel())
    assert rc == L.LSC_OK
    b = Batch(rng, [80], [80], 16, 6)
    kx, vx = (dense(rng.standard_normal((80, 1, 64)), L.LSC_BF16) for _ in "kv")
    bl, r = b.places(0, 0, 80)
    far.write(0, 0, bl, r, kx[1])
    far.write(0, 1, bl, r, vx[1])
    q, qx = dense(rng.standard_normal((80, 2, 64)), L.LSC_BF16)
    batch = b.device()
    out, ls = torch.zeros(80, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(80, 2, device="cuda")
    assert L.lsc_kv_append(pool, 0, L.kv_append_args(batch, kx[0], vx[0], L.LSC_BF16), cur()) == L.LSC_OK
    assert L.lsc_kv_attend(pool, 0, L.kv_attend_args(batch, 2, q, out, L.LSC_BF16, 0.125, lse=ls), cur()) == L.LSC_OK
    torch.cuda.synchronize()
    check_attend(far, 0, b, qx, L.LSC_BF16, 0.125, True, out, ls)
    assert L.lsc_kv_pool_destroy(pool) == L.LSC_OK
