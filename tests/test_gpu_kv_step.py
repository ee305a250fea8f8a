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
scale.  The sums of N terms in 32 bits add N 2^-23.  All of that times the sum of
weight times |v| (`mass`), and the output is rounded once, half a step of the
result.  exp2 and log2 are good to 2^-21.
"""
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
