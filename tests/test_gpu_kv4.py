"""GPU: E2M1 pools (4 bits an element, a scale byte per 16) through append, gather, copy_prefix and attend, against
plain 64-bit forms (tests/_kv4.py, tests/_kv.py).

Tolerances.  append, gather and copy_prefix: equal bits (an element has 6 significant bits, so every float type holds
it).  attend: test_gpu_kv_step.py's bound.  Its weights are rounded to q's type at worst: f16 with f16 q, and with bf16
q f16 (half a step, 2^-11) or, where many rows of q read the rows at 16 bits, bf16 (half a step of 8 bits, 2^-8).  Where
they are f16, bf16 rows of q are brought to f16 by a power of two: elements keep their bits down to 2^-14 of their row's
largest and are off by 2^-25 of it below, so a score is off by D 2^-25 of largest q times largest k at most (`q_tail`).
"""
import numpy as np
import pytest
import torch

from linear_attention_state_lsc_gb300 import lsc as L

import _kv
from _kv import NAME, TORCH, Batch, DevKv
from _kv4 import LADDER, MAG, Host4, halves, quantise4, value4
from test_gpu_kv_step import FLOATS, HALF, LENGTHS, cur, dense, run_attend, step_lengths

pytestmark = pytest.mark.gpu

BF, F16, F32 = L.LSC_BF16, L.LSC_F16, L.LSC_F32


# ---- append ---------------------------------------------------------------------

@pytest.mark.parametrize("dtype", FLOATS, ids=NAME.get)
@pytest.mark.parametrize("shape", [(16, 2, 64), (7, 3, 48), (5, 1, 16), (64, 2, 256), (3, 1, 272)], ids=str)
def test_append(lsc, dtype, shape):
    """Vector and element kernels; the whole pool compared, so nothing else changed."""
    bt, H, D = shape
    rng = np.random.default_rng(bt * D)
    for name, stride in (("ragged", 0), ("ahead", H * D + 8), ("decode", H * D + 3)):
        n, kv = step_lengths(name)
        host = Host4(50, bt, H, D)
        b = Batch(rng, n, kv, bt, 50, spare=3, wide=2)
        x = rng.standard_normal((2, b.T, H, D)) * np.exp(2 * rng.standard_normal((2, b.T, H, 1)))
        x[0, 0] = 0
        x[:, -3:] = np.nan
        (k, kx), (v, vx) = (dense(y, dtype, stride or None) for y in x)
        with DevKv(host) as dev:
            args = L.kv_append_args(b.device(), k, v, dtype, stride, stride)
            assert L.lsc_kv_append(dev.pool, 1, args, cur()) == L.LSC_OK
            got = dev.download()
            assert dev.status() == L.LSC_OK
        for i in range(len(n)):
            first = max(0, n[i] - kv[i])
            bl, r = b.places(i, max(0, kv[i] - n[i]), kv[i])
            for lane, y in enumerate((kx, vx)):
                host.write(1, lane, bl, r, y[b.cu[i] + first:b.cu[i + 1]])
        np.testing.assert_array_equal(got, host.bytes)


def border_rows(dtype):
    """Groups whose largest magnitude is six times each scale or beside it, with ties between codes and their
    neighbours in the type; zeros, subnormals, magnitudes beyond the largest scale, infinities and NaN."""
    t = TORCH[dtype]

    def beside(x):
        x = torch.tensor(x, dtype=torch.float64).to(t)
        i = {2: torch.int16, 4: torch.int32}[x.element_size()]
        return torch.stack([x, (x.view(i) - 1).view(t), (x.view(i) + 1).view(t)], -1)

    tops = beside(6 * LADDER[1:])                                             # [226, 3]
    ties = beside((MAG[:-1] + MAG[1:]) / 2 * LADDER[1:, None]).flatten(1)     # [226, 21]
    groups = []
    for part in range(3):                                                     # 7 ties and their neighbours, 15 places
        for lo in (0, 7, 14):
            g = torch.cat([tops[:, part:part + 1], ties[:, lo:lo + 7], -ties[:, lo:lo + 7], ties[:, :1]], 1)
            groups.append(g)
    x = torch.cat(groups).double()
    special = torch.zeros(10, 16, dtype=torch.float64)
    special[0] = -0.0
    special[1, 3], special[2, 4], special[3, 5] = float("inf"), float("-inf"), float("nan")
    special[4] = torch.finfo(t).tiny * torch.linspace(-1, 1, 16)
    special[5, 7] = torch.finfo(t).smallest_normal * torch.finfo(t).eps
    special[6] = torch.linspace(-65504, 65504, 16)
    special[7, 0], special[7, 1] = torch.finfo(t).max, -61440
    special[8, 2], special[8, 3] = 61440, 2.0 ** -18
    special[9, 15] = 2.0 ** -18
    x = torch.cat([x, special.to(t).double()])
    return torch.nn.functional.pad(x, (0, 0, 0, -len(x) % 4)).reshape(-1, 1, 64).numpy()


@pytest.mark.parametrize("dtype", FLOATS, ids=NAME.get)
@pytest.mark.parametrize("stride", [64, 65])
def test_append_quantises_border_values(lsc, dtype, stride):
    x = border_rows(dtype)
    T = len(x)
    host = Host4(T // 8 + 1, 8, 1, 64)
    b = Batch(np.random.default_rng(0), [T], [T], 8, T // 8 + 1)
    k, kx = dense(x, dtype, stride)
    with DevKv(host) as dev:
        args = L.kv_append_args(b.device(), k, k, dtype, stride, stride)
        assert L.lsc_kv_append(dev.pool, 0, args, cur()) == L.LSC_OK
        got = dev.download()
    bl, r = b.places(0, 0, T)
    for lane in (0, 1):
        host.write(0, lane, bl, r, kx)
    np.testing.assert_array_equal(got, host.bytes)
    used = np.unique(host.scales(0, 0)[bl, r])
    assert 255 in used and 0 in used and 226 in used and len(used) > 200


def test_append_of_random_bits(lsc):
    """fp32 rows of every bit pattern's kind, and rows of random f16 and bf16 bits."""
    rng = np.random.default_rng(4)
    for dtype in FLOATS:
        D, T = 256, 600
        bits = torch.from_numpy(rng.integers(0, 2 ** 16, (T, D * TORCH[dtype].itemsize // 2)).astype(np.uint16).view(np.int16))
        x = bits.view(TORCH[dtype]).reshape(T, D)
        k, kx = x.contiguous().cuda(), x.double().numpy().reshape(T, 1, D)
        host = Host4(T // 8, 8, 1, D)
        b = Batch(rng, [T], [T], 8, T // 8)
        with DevKv(host) as dev:
            assert L.lsc_kv_append(dev.pool, 1, L.kv_append_args(b.device(), k, k, dtype), cur()) == L.LSC_OK
            got = dev.download()
        bl, r = b.places(0, 0, T)
        for lane in (0, 1):
            host.write(1, lane, bl, r, kx)
        np.testing.assert_array_equal(got, host.bytes)


# ---- gather and copy_prefix -----------------------------------------------------

@pytest.mark.parametrize("dtype", FLOATS, ids=NAME.get)
@pytest.mark.parametrize("shape", [(16, 2, 64), (7, 3, 48), (64, 2, 256), (3, 1, 272)], ids=str)
def test_gather(lsc, dtype, shape):
    bt, H, D = shape
    rng = np.random.default_rng(bt + D)
    for name, stride in (("ragged", 0), ("ahead", H * D + 8), ("decode", H * D + 3)):
        n, kv = step_lengths(name)
        host = Host4(50, bt, H, D)
        b = Batch(rng, n, kv, bt, 50, spare=2, wide=1)
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
                x = torch.from_numpy(host.read(1, lane, bl, r)).reshape(-1, H * D).to(TORCH[dtype])
                want[b.cu[i]:b.cu[i] + first, :H * D] = 0
                want[b.cu[i] + first:b.cu[i + 1], :H * D] = x
            assert torch.equal(y.cpu(), want)


def test_gather_of_every_code_and_scale(lsc):
    """The 16 codes under scale bytes 0 to 226 and 255, to each float type, aligned and not."""
    T = 228
    host = Host4(T // 4, 4, 1, 16)
    b = Batch(np.random.default_rng(1), [T], [T], 4, T // 4)
    bl, r = b.places(0, 0, T)
    code = np.arange(16, dtype=np.uint8)
    byte = np.r_[0:227, 255].astype(np.uint8)
    for lane in (0, 1):
        host.rows(0, lane)[bl, r, 0] = halves(code)
        host.scales(0, lane)[bl, r, 0, 0] = byte
    want = value4(np.tile(code, (T, 1)), byte[:, None])
    with DevKv(host) as dev:
        for dtype in FLOATS:
            for stride in (16, 17):
                k, v = (torch.zeros(T, stride, dtype=TORCH[dtype], device="cuda") for _ in "kv")
                args = L.kv_gather_args(b.device(), k, v, dtype, stride, stride)
                assert L.lsc_kv_gather(dev.pool, 0, args, cur()) == L.LSC_OK
                for got in (k, v):
                    np.testing.assert_array_equal(got[:, :16].cpu().double().numpy(), want)


@pytest.mark.parametrize("shape", [(16, 2, 64), (5, 3, 48), (64, 1, 256)], ids=str)
def test_copy_prefix_moves_codes_and_scales(lsc, shape):
    """Rows [0, n) of blocks, codes and scale bytes, in every layer and lane, and nothing else."""
    bt, H, D = shape
    rng = np.random.default_rng(2)
    host = Host4(9, bt, H, D, layers=3)
    host.bytes[:] = rng.integers(0, 256, host.bytes.shape)
    ops = L.kv_ops([0, 1, 2, 3], [5, 6, 7, 8], [bt, 1, bt - 1, 0])
    with DevKv(host) as dev:
        rc, copied = L.lsc_copy_prefix(dev.pool, ops, cur())
        assert rc == L.LSC_OK and copied == 2 * bt * H * (D // 2 + D // 16) * 2 * 3
        got = dev.download()
    for s, d, n in ((0, 5, bt), (1, 6, 1), (2, 7, bt - 1)):
        for w, at in ((H * D // 2, 0), (H * D // 16, host.scale_off)):
            host.bytes[:, :, d, at:at + n * w] = host.bytes[:, :, s, at:at + n * w]
    np.testing.assert_array_equal(got, host.bytes)


# ---- attend ---------------------------------------------------------------------

def filled4(rng, b, blocks, bt, H, D, layers=2, layer=1):
    host = Host4(blocks, bt, H, D, layers=layers)
    gain = np.exp(0.5 * rng.standard_normal((1, H, D)))
    for i in range(len(b.n)):
        bl, r = b.places(i, 0, int(b.kv[i]))
        host.write(layer, 0, bl, r, rng.standard_normal((len(r), H, D)) * gain)
        host.write(layer, 1, bl, r, rng.standard_normal((len(r), H, D)) * np.exp(rng.standard_normal((len(r), H, 1))))
    return host


def check4(host, layer, b, qx, dtype, scale, causal, out, ls, rows=None):
    T, Hq, D = qx.shape
    want, lse, mass, reach, vmax = _kv.attend(host, layer, b, qx, scale, causal)
    got = out[:, :Hq * D].double().cpu().numpy().reshape(T, Hq, D)
    N = float(b.kv.max(initial=1))
    kmax = np.nanmax(np.abs(np.concatenate([host.read(layer, 0, *b.places(i, 0, int(b.kv[i]))).reshape(-1)
                                            for i in range(len(b.n))])), initial=0)
    q_tail = 0 if dtype == F32 else D * 2.0 ** -25 * np.abs(qx).max(-1) * kmax * scale
    es = D * 2.0 ** -23 * reach + q_tail
    weight = 0.0 if dtype == F32 else HALF[dtype]
    rel = weight + 2 * es + (N + 8) * 2.0 ** -23 + 2.0 ** -20
    tail = N * 2.0 ** -32 * vmax if dtype != F32 else 0 * vmax  # f16 weights: multiples of 2^-24 beside 2^7 or more
    bound = rel[..., None] * mass + tail[..., None] + HALF[dtype] * (np.abs(want) + rel[..., None] * mass) + 1e-30
    keep = slice(0, int(b.cu[-1])) if rows is None else rows
    assert np.isfinite(got[keep]).all()
    over = np.abs(got - want)[keep] / bound[keep]
    assert over.max(initial=0) <= 1, (over.max(), np.unravel_index(over.argmax(), over.shape))
    if ls is not None:
        l = ls.double().cpu().numpy()[keep]
        np.testing.assert_array_equal(np.isinf(l), np.isinf(lse[keep]))
        f = np.isfinite(lse[keep])
        lim = es[keep] + (N + 8) * 2.0 ** -23 + 2.0 ** -20 * (1 + np.abs(np.where(f, lse[keep], 0)))
        assert (np.abs(np.where(f, l - np.where(f, lse[keep], 0), 0)) <= lim).all()
    assert (out[int(b.cu[-1]):] == 7).all() and (ls is None or (ls[int(b.cu[-1]):] == 7).all())


@pytest.mark.parametrize("dtype", [BF, F16, F32], ids=NAME.get)
@pytest.mark.parametrize("name", list(LENGTHS))
@pytest.mark.parametrize("shape", [(16, 2, 4, 64), (64, 1, 8, 128), (24, 2, 5, 128), (64, 2, 8, 256), (5, 1, 3, 48),
                                   (12, 2, 2, 128), (1, 1, 2, 64)], ids=str)
def test_attend(lsc, dtype, name, shape):
    bt, H, G, D = shape
    rng = np.random.default_rng(bt * 1000 + D + len(name))
    n, kv = LENGTHS[name]
    blocks = int(sum(-(-k // bt) for k in kv)) + 3
    b = Batch(rng, n, kv, bt, blocks, spare=2, wide=1)
    host = filled4(rng, b, blocks, bt, H, D)
    q, qx = dense(2 * rng.standard_normal((b.T, H * G, D)), dtype)
    scale = D ** -0.5
    with DevKv(host) as dev:
        for causal in (True, False):
            out, ls = run_attend(dev, 1, b, q, dtype, H * G, scale, causal, max_seq_tokens=max(n), max_kv_tokens=max(max(kv), 1))
            check4(host, 1, b, qx, dtype, scale, causal, out, ls)
            again, _ = run_attend(dev, 1, b, q, dtype, H * G, scale, causal, lse=False)  # without bounds
            check4(host, 1, b, qx, dtype, scale, causal, again, None)
        assert dev.status() == L.LSC_OK
        np.testing.assert_array_equal(dev.download(), host.bytes)
