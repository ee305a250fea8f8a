"""GPU: attention over E2M1 pools where it is easiest to get wrong, in every form it takes: the decode kernel, the chunk
kernel that converts tiles as it meets them, the chunk kernels over expanded rows, and the CUDA cores.  K and V that are
not finite, bytes of any kind where nothing may be read, queries that are not finite or far from 1, flat tails, blocks
that fit no TMA box and every box, runs cut anywhere, heads side by side, bad batches, one workspace for many steps,
streams and graphs, and waits that run out.  Plain 64-bit forms and tolerances are test_gpu_kv4.py's."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from linear_attention_state_lsc_gb300 import lsc as L

import _kv
from _kv import NAME, TORCH, Batch, DevKv
from _kv4 import Host4
from test_gpu_kv4 import check4, filled4
from test_gpu_kv_edges import shared
from test_gpu_kv_step import HALF, cur, dense, run_attend

pytestmark = pytest.mark.gpu

BF, F16, F32 = L.LSC_BF16, L.LSC_F16, L.LSC_F32
HERE = os.path.dirname(os.path.abspath(__file__))

# (dtype, new tokens, block, head_dim, q heads a kv head)
FORMS = {"decode-bf16": (BF, 2, 64, 128, 4), "decode-f16": (F16, 2, 16, 256, 8), "decode-64": (BF, 1, 8, 64, 3),
         "decode-4-rows": (F16, 2, 32, 128, 2), "decode-4-rows-256": (BF, 4, 64, 256, 1),
         "chunk-bf16": (BF, 20, 64, 128, 4), "chunk-f16": (F16, 20, 12, 64, 4), "chunk-256": (BF, 12, 5, 256, 8),
         "few-rows-no-box": (BF, 2, 12, 128, 2),
         "expanded-bf16": (BF, 300, 64, 128, 4), "expanded-f16": (F16, 300, 12, 64, 4), "expanded-256": (BF, 100, 16, 256, 8),
         "cuda-cores": (F32, 5, 16, 64, 2), "cuda-cores-48": (F16, 5, 16, 48, 2)}
every_form = pytest.mark.parametrize("form", list(FORMS))


def expands(form):
    """The row blocks a sequence from which rows are expanded: 4 of 256 rows, 6 of 128 at head_dim 256."""
    dtype, n, _, D, G = FORMS[form]
    return n * G >= (6 * 128 if D == 256 else 4 * 256)


def test_the_forms_are_what_they_are_called():
    assert [f for f in FORMS if expands(f)] == [f for f in FORMS if f.startswith("expanded")]
    for f, (dtype, n, bt, D, G) in FORMS.items():
        assert f.startswith("decode") == (dtype != F32 and n * G <= 16 and bt % 8 == 0 and D in (64, 128, 256))


@every_form
def test_what_a_row_does_not_see_does_not_enter(lsc, form):
    """K and V of some new tokens are NaN: earlier rows of the causal chunk are as if they were not there, rows that see
    them get NaN in the 16 columns of a V group, or throughout from K."""
    dtype, n, bt, D, G = FORMS[form]
    n = max(n, 3)
    H, kv = 2, n + 61
    rng = np.random.default_rng(n + D)
    b = Batch(rng, [n, 1], [kv, 20], bt, 120)
    host = filled4(rng, b, 120, bt, H, D)
    bl, r = b.places(0, 0, kv)
    v, k = host.read(1, 1, bl, r), host.read(1, 0, bl, r)
    first = kv - n + 1 + (n - 2) // 2  # the first position whose v is not finite: the row before it does not see it
    x = v.copy()
    x[first, :, 3], x[first, :, 40] = np.inf, np.nan
    host.write(1, 1, bl, r, x)
    y = k.copy()
    y[-1, :, 7] = np.nan  # the last token's scores: seen by the last row alone
    host.write(1, 0, bl, r, y)
    q, qx = dense(rng.standard_normal((b.T, H * G, D)), dtype)
    scale = D ** -0.5
    sees = first - (kv - n)  # new tokens below this one see finite values alone
    with DevKv(host) as dev:
        out, ls = run_attend(dev, 1, b, q, dtype, H * G, scale, True, max_seq_tokens=n)
        assert dev.status() == L.LSC_OK
    sick = np.r_[0:16, 32:48]
    v[first, :, sick] = 0  # what no clean row sees
    k[-1] = 0
    host.write(1, 0, bl, r, k)
    host.write(1, 1, bl, r, v)
    check4(host, 1, b, qx, dtype, scale, True, out, ls, rows=np.r_[0:sees, n])
    got = out.float().cpu().numpy().reshape(b.T, H * G, D)
    assert np.isnan(got[n - 1]).all()
    assert np.isnan(got[sees:n - 1][..., sick]).all()
    assert np.isfinite(np.delete(got[sees:n - 1], sick, -1)).all()


@every_form
@pytest.mark.parametrize("byte", [0x00, 0x7F, 0xF8, 0xFF])
def test_bytes_of_any_kind_behind_the_last_position(lsc, form, byte):
    """What a fresh pool holds: zeros, codes of 6 under scales of 6 10^-5 and of infinity, NaN."""
    dtype, n, bt, D, G = FORMS[form]
    rng = np.random.default_rng(byte + n)
    b = Batch(rng, [n, 1, n], [n, 0, n + 33], bt, 120, spare=1)
    host = Host4(120, bt, 2, D, fill=byte)
    for i in range(3):
        bl, r = b.places(i, 0, int(b.kv[i]))
        for lane in (0, 1):
            host.write(1, lane, bl, r, rng.standard_normal((len(r), 2, D)))
    q, qx = dense(rng.standard_normal((b.T, 2 * G, D)), dtype)
    with DevKv(host) as dev:
        for causal in (True, False):
            out, ls = run_attend(dev, 1, b, q, dtype, 2 * G, D ** -0.5, causal, max_seq_tokens=n)
            check4(host, 1, b, qx, dtype, D ** -0.5, causal, out, ls)


@every_form
def test_a_query_that_is_not_finite_is_nan_alone(lsc, form):
    dtype, n, bt, D, G = FORMS[form]
    H = 2
    rng = np.random.default_rng(n + 3 * D)
    b = Batch(rng, [n] * 3 + [1], [n + 60, n, n + 7, 0], bt, 300, spare=1)
    host = filled4(rng, b, 300, bt, H, D)
    x = 2 * rng.standard_normal((b.T, H * G, D))
    x[3 * n] = np.inf  # the last sequence sees nothing: zeros all the same
    sick = [(0, 1, np.inf), (n, 0, -np.inf), (2 * n + n - 1, G, np.nan)]  # (row, head, what)
    for t, h, what in sick:
        x[t, h, 2:20] *= 300  # the finite elements of such a row may be large too
        x[t, h, 5] = what
    q, qx = dense(x, dtype)
    with DevKv(host) as dev:
        out, ls = run_attend(dev, 1, b, q, dtype, H * G, D ** -0.5, True, max_seq_tokens=n)
        assert dev.status() == L.LSC_OK
    got = out.view(b.T, H * G, D)
    assert (got[3 * n] == 0).all() and torch.isinf(ls[3 * n]).all()
    for t, h, _ in sick:
        assert torch.isnan(got[t, h]).all(), (t, h)
        assert not torch.isfinite(ls[t, h])
        qx[t, h] = 0  # the plain form of a row of zeros in its place, so that all the others are compared
    qx[3 * n] = 0
    want, lse = _kv.attend(host, 1, b, qx, D ** -0.5, True)[:2]
    for t, h, _ in sick:
        got[t, h] = torch.from_numpy(want[t, h]).to(got)
        ls[t, h] = float(lse[t, h])
    check4(host, 1, b, qx, dtype, D ** -0.5, True, out, ls)


@every_form
@pytest.mark.parametrize("power", [-126, -60, -14, 14])
def test_queries_far_from_one(lsc, form, power):
    """Rows of q of any size a power of two brings them to, and elements 2^-12 of the largest beside it; the scale takes
    the size back where it can."""
    dtype, n, bt, D, G = FORMS[form]
    if dtype == F16 and power < -14:
        pytest.skip("f16 has no such elements")
    rng = np.random.default_rng(power + 200 + n)
    b = Batch(rng, [n] * 2, [n + 50, n + 3], bt, 120)
    host = filled4(rng, b, 120, bt, 2, D)
    x = rng.standard_normal((b.T, 2 * G, D)) * np.where(rng.random((b.T, 2 * G, D)) < 0.3, 2.0 ** -12, 1)
    x = x * 2.0 ** power
    if dtype == F16:
        x = np.clip(x, -65504, 65504)  # an element beyond would be an infinity: another test's
    q, qx = dense(x, dtype)
    scale = float(np.float32(2.0 ** np.clip(-power - 3, -20, 100)))
    with DevKv(host) as dev:
        out, ls = run_attend(dev, 1, b, q, dtype, 2 * G, scale, True, max_seq_tokens=n)
        assert dev.status() == L.LSC_OK
    check4(host, 1, b, qx, dtype, scale, True, out, ls)


def test_queries_too_small_to_count(lsc):
    """Rows of q below 2^-111 and scales that make every score 0: the mean of v, and hidden positions stay hidden."""
    rng = np.random.default_rng(3)
    for n, D, G in ((2, 128, 4), (40, 128, 4), (12, 256, 8)):
        b = Batch(rng, [n, n], [n, n + 70], 16, 40)
        host = filled4(rng, b, 40, 16, 2, D)
        q, qx = dense(rng.standard_normal((b.T, 2 * G, D)) * 2.0 ** -120, BF)
        with DevKv(host) as dev:
            for scale in (1.0, 2.0 ** -100):
                out, ls = run_attend(dev, 1, b, q, BF, 2 * G, scale, True, max_seq_tokens=n)
                check4(host, 1, b, qx, BF, scale, True, out, ls)


@every_form
def test_weights_have_eleven_bits(lsc, form):
    """V is zero but for two positions, +x and -x, whose weights differ little: what is left of them shows how many bits
    they had.  f16's half step (2^-11) in every form, BF16 q among them; beside it what 32-bit sums are off by."""
    dtype, n, bt, D, G = FORMS[form]
    kv, H = n + 61, 2
    rng = np.random.default_rng(n + 5 * D)
    b = Batch(rng, [n], [kv], bt, 120)
    host = Host4(120, bt, H, D)
    bl, r = b.places(0, 0, kv)
    host.write(1, 0, bl, r, 0.3 * rng.standard_normal((kv, H, D)))
    v = np.zeros((kv, H, D))
    v[7] = rng.standard_normal((H, D))
    v[40] = -v[7]
    host.write(1, 1, bl, r, v)
    q, qx = dense(rng.standard_normal((b.T, H * G, D)), dtype)
    scale = 0.5 * D ** -0.5
    want, _, mass, reach, vmax = _kv.attend(host, 1, b, qx, scale, False)
    kmax = np.abs(host.read(1, 0, bl, r)).max()
    es = D * 2.0 ** -23 * reach + (0 if dtype == F32 else D * 2.0 ** -25 * np.abs(qx).max(-1) * kmax * scale)
    rel = (2.0 ** -11 + 2 * es + (kv + 8) * 2.0 ** -23 + 2.0 ** -20)[..., None]
    err = rel * mass + kv * 2.0 ** -32 * vmax[..., None]
    bound = err + HALF[dtype] * (np.abs(want) + err) + 1e-30
    with DevKv(host) as dev:
        out, _ = run_attend(dev, 1, b, q, dtype, H * G, scale, False, max_seq_tokens=n)
        assert dev.status() == L.LSC_OK
    over = np.abs(out.double().cpu().numpy().reshape(want.shape) - want) / bound
    assert over.max() <= 1, (over.max(), np.unravel_index(over.argmax(), over.shape))


@every_form
@pytest.mark.parametrize("scale", [1.0, 4.0, 64.0])
def test_the_largest_queries_meet_zeros(lsc, form, scale):
    """Rows of q whose one element is the largest power of two of their type, and K zero there: every score is 0, however
    much the scale and that element come to together (2^133 at most, less than 2^14 beyond 32 bits)."""
    dtype, n, bt, D, G = FORMS[form]
    if dtype == F32:
        pytest.skip("32-bit rows are scaled in 32 bits")
    rng = np.random.default_rng(n + D)
    b = Batch(rng, [n, 1], [n + 61, 20], bt, 120)
    host = filled4(rng, b, 120, bt, 2, D)
    for i in range(2):
        bl, r = b.places(i, 0, int(b.kv[i]))
        k = host.read(1, 0, bl, r)
        k[:, :, 5] = 0
        host.write(1, 0, bl, r, k)
    x = np.zeros((b.T, 2 * G, D))
    x[:, :, 5] = 2.0 ** 15 if dtype == F16 else 2.0 ** 127
    q, qx = dense(x, dtype)
    with DevKv(host) as dev:
        out, ls = run_attend(dev, 1, b, q, dtype, 2 * G, scale, True, max_seq_tokens=n)
        assert dev.status() == L.LSC_OK
    check4(host, 1, b, qx, dtype, scale, True, out, ls)


@pytest.mark.parametrize("gap", [3.0, 16.9, 24.9, 25.1])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype,n", [(BF, 1), (F16, 2), (BF, 20), (F16, 20)])
def test_a_flat_tail_counts(lsc, dtype, n, D, gap):
    """One position with a score `gap` (in powers of two) above all others, which are equal.  v is 1 everywhere but in the
    large one's odd columns, where it is 0: even columns give 1, odd ones the share of the others' weights.  f16 weights
    are multiples of 2^-24 beside a largest one of 2^7 or more: off by 2^-32 of it at most, or by half a step of 11 bits."""
    kv, bt, G, S = 32768, 64, 4, 40
    b = shared(S, n, kv, bt)
    host = Host4(kv // bt, bt, 1, D, layers=1)
    k, v = np.zeros((1, 1, D)), np.ones((1, 1, D))
    at = np.arange(kv)
    for lane, one in ((0, k), (1, v)):
        host.write(0, lane, at // bt, at % bt, np.repeat(one, kv, 0))
    k[0, 0, 0] = 1
    v[0, 0, 1::2] = 0
    host.write(0, 0, [0], [0], k)
    host.write(0, 1, [0], [0], v)
    k0 = float(host.read(0, 0, np.array([0]), np.array([0]))[0, 0, 0])
    x = np.zeros((b.T, G, D))
    x[:, :, 0] = gap * np.log(2) * 8
    q, qx = dense(x, dtype)
    s = float(qx[0, 0, 0]) / 8 * k0
    with DevKv(host) as dev:
        out, ls = run_attend(dev, 0, b, q, dtype, G, 0.125, False, max_seq_tokens=n)
        assert dev.status() == L.LSC_OK
    one = float(host.read(0, 1, np.array([0]), np.array([1]))[0, 0, 0])  # v's 1 as the pool holds it
    rest = (kv - 1) * np.exp(-s)
    want = np.where(np.arange(D) % 2, rest, 1 + rest) / (1 + rest) * one
    err = (2.0 ** -11 + (kv + 8) * 2.0 ** -23 + 2.0 ** -20) * want + kv * 2.0 ** -32 * one
    bound = err + HALF[dtype] * (want + err)
    over = np.abs(out.double().cpu().numpy().reshape(-1, D) - want) / bound
    assert over.max() <= 1, over.max()
    assert (np.abs(ls.double().cpu().numpy() - s - np.log1p(rest)) <= (1 + s) * 2.0 ** -20 + (kv + 8) * 2.0 ** -23).all()


@pytest.mark.parametrize("lengths", [([1, 1, 1, 1], [1, 13, 300, 0]), ([2, 1], [900, 61]), ([70, 0, 130, 3], [70, 5, 400, 1]),
                                     ([9, 30], [4, 700]), ([300, 2], [300, 700])], ids=["decode", "few", "chunk", "ahead", "expanded"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bt", [1, 5, 8, 12, 16, 32, 48, 64, 128, 200])
def test_every_block_size(lsc, bt, D, lengths):
    """Blocks that fit no box, and boxes of 8 rows to a whole sub-tile."""
    n, kv = lengths
    rng = np.random.default_rng(bt * D + len(n))
    blocks = int(sum(-(-k // bt) for k in kv)) + 3
    b = Batch(rng, n, kv, bt, blocks, spare=2, wide=1)
    host = filled4(rng, b, blocks, bt, 2, D)
    dtype = F16 if bt % 3 == 0 else BF
    q, qx = dense(2 * rng.standard_normal((b.T, 8, D)), dtype)
    with DevKv(host) as dev:
        out, ls = run_attend(dev, 1, b, q, dtype, 8, D ** -0.5, True, max_seq_tokens=max(n))
        check4(host, 1, b, qx, dtype, D ** -0.5, True, out, ls)
        assert dev.status() == L.LSC_OK
        np.testing.assert_array_equal(dev.download(), host.bytes)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("S", [3, 31, 60])
@pytest.mark.parametrize("most", [2, 12])
def test_runs_that_begin_and_end_anywhere(lsc, D, S, most):
    rng = np.random.default_rng(71 + S + most)
    n = rng.integers(0, most, S)
    kv = np.where(rng.random(S) < 0.3, rng.integers(1100, 2500, S), rng.integers(1, 300, S)) + n
    bt = 64 if S != 31 else 12
    blocks = int((-(-kv // bt)).sum())
    b = Batch(rng, n, kv, bt, blocks, spare=1)
    host = filled4(rng, b, blocks, bt, 2, D)
    q, qx = dense(2 * rng.standard_normal((b.T, 32, D)), BF)
    with DevKv(host) as dev:
        out, ls = run_attend(dev, 1, b, q, BF, 32, D ** -0.5, True, max_seq_tokens=max(1, int(n.max())))
        check4(host, 1, b, qx, BF, D ** -0.5, True, out, ls)
        again, _ = run_attend(dev, 1, b, q, BF, 32, D ** -0.5, True, max_seq_tokens=max(1, int(n.max())))
        assert torch.equal(out, again)
        assert dev.status() == L.LSC_OK


@pytest.mark.parametrize("dtype,H,G,D,n,kv", [
    (BF, 8, 4, 128, [1], [31000]), (F16, 8, 1, 64, [1], [20011]), (BF, 2, 8, 256, [1, 1], [9000, 16001]),
    (F16, 4, 4, 64, [4, 1], [5003, 12345]), (BF, 2, 2, 256, [8], [8001]), (BF, 1, 16, 128, [1, 1, 1], [7000, 0, 40])], ids=str)
def test_few_long_sequences(lsc, dtype, H, G, D, n, kv):
    """Units of dozens of parts: rows that see less than others, an empty cache, V that is NaN in a group, twice the same
    bits."""
    rng = np.random.default_rng(sum(kv) + D)
    bt = 64
    blocks = sum(-(-x // bt) for x in kv)
    b = Batch(rng, n, kv, bt, blocks, spare=1)
    host = filled4(rng, b, blocks, bt, H, D)
    bl, r = b.places(0, kv[0] - 1, kv[0])  # the last token's v, seen by its own row alone
    keep = host.read(1, 1, bl, r)
    x = keep.copy()
    x[0, H - 1, 21] = np.nan
    host.write(1, 1, bl, r, x)
    q, qx = dense(2 * rng.standard_normal((b.T, H * G, D)), dtype)
    with DevKv(host) as dev:
        out, ls = run_attend(dev, 1, b, q, dtype, H * G, D ** -0.5, True, max_seq_tokens=max(n), max_kv_tokens=max(kv))
        again, ls2 = run_attend(dev, 1, b, q, dtype, H * G, D ** -0.5, True, max_seq_tokens=max(n), max_kv_tokens=max(kv))
        assert dev.status() == L.LSC_OK
    assert torch.equal(out.view(torch.uint8), again.view(torch.uint8)) and torch.equal(ls, ls2)
    got, heads, t = out.view(b.T, H * G, D), slice((H - 1) * G, H * G), int(b.cu[1]) - 1
    assert torch.isnan(got[t, heads, 16:32]).all()
    host.write(1, 1, bl, r, keep)
    want = _kv.attend(host, 1, b, qx, D ** -0.5, True)[0][t, heads]
    got[t, heads, 16:32] = torch.from_numpy(want[:, 16:32]).to(got)
    check4(host, 1, b, qx, dtype, D ** -0.5, True, out, ls)


@pytest.mark.parametrize("n", [1, 2])
@pytest.mark.parametrize("dtype,H,G,D", [(BF, 2, 2, 256), (BF, 4, 5, 128), (BF, 8, 1, 64), (BF, 2, 8, 128), (F16, 4, 3, 256),
                                         (F16, 4, 2, 64), (BF, 3, 4, 128)])
def test_decode_batches_with_heads_side_by_side(lsc, dtype, H, G, D, n):
    """Batches large enough for it, whole and cut units, V that is NaN in one head's group of some sequences."""
    rng = np.random.default_rng(H * D + n)
    S, bt, most = 48, 32, 1700
    kv = rng.integers(1, 300, S) + n
    kv[[3, 17, 40]] = [most, 1100, 900]
    new = np.where(rng.random(S) < 0.2, 0, n)
    new[[3, 17]] = n
    blocks = int((-(-kv // bt)).sum())
    b = Batch(rng, new, kv, bt, blocks, spare=1)
    host = filled4(rng, b, blocks, bt, H, D)
    sick, keep = H - 1, {}
    for i in (3, 17):  # the last token's v, seen by its own row alone
        bl, r = b.places(i, kv[i] - 1, kv[i])
        keep[i] = host.read(1, 1, bl, r)
        x = keep[i].copy()
        x[0, sick, 21] = np.nan
        host.write(1, 1, bl, r, x)
    q, qx = dense(2 * rng.standard_normal((b.T, H * G, D)), dtype)
    with DevKv(host) as dev:
        out, ls = run_attend(dev, 1, b, q, dtype, H * G, D ** -0.5, True, max_seq_tokens=n, max_kv_tokens=most)
        again, _ = run_attend(dev, 1, b, q, dtype, H * G, D ** -0.5, True, max_seq_tokens=n, max_kv_tokens=most)
        assert dev.status() == L.LSC_OK
    assert torch.equal(out.view(torch.uint8), again.view(torch.uint8))
    got = out.view(b.T, H * G, D)
    heads = slice(sick * G, (sick + 1) * G)
    for i in (3, 17):
        t, (bl, r) = int(b.cu[i + 1]) - 1, b.places(i, kv[i] - 1, kv[i])
        assert torch.isnan(got[t, heads, 16:32]).all()
        host.write(1, 1, bl, r, keep[i])
        want = _kv.attend(host, 1, b, qx, D ** -0.5, True)[0][t, heads]
        got[t, heads, 16:32] = torch.from_numpy(want[:, 16:32]).to(got)
    check4(host, 1, b, qx, dtype, D ** -0.5, True, out, ls)


@every_form
def test_bad_batches_are_recorded_and_stay_inside(lsc, form):
    """Block ids, lengths and cu_seqlens that do not fit: the status word says so and the other sequences are right."""
    dtype, n, bt, D, G = FORMS[form]
    rng = np.random.default_rng(6)
    H = 2
    b = Batch(rng, [n, n, 1], [n + 40, n + 50, 33], bt, 200, wide=1)
    host = filled4(rng, b, 200, bt, H, D)
    q, qx = dense(rng.standard_normal((b.T, H * G, D)), dtype)
    good = np.r_[0:n, 2 * n]  # sequence 1 is the one that breaks
    b.device()

    def call(dev, table, cu, kv):
        out = torch.full((b.T, H * G * D), 7.0, dtype=TORCH[dtype], device="cuda")
        ls = torch.full((b.T, H * G), 7.0, device="cuda")
        batch = L.kv_batch(3, b.T, *[torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (table, cu, kv)],
                           max_blocks=table.shape[1])
        a = L.kv_attend_args(batch, H * G, q, out, dtype, 0.125, lse=ls, max_seq_tokens=n)
        assert L.lsc_kv_attend(dev.pool, 1, a, cur()) == L.LSC_OK
        return dev.status(), out, ls

    table, cu, kv = b.table, b.cu, b.kv.astype(np.int32)
    with DevKv(host) as dev:
        for bad in (200, -1, 2 ** 31 - 1):
            t = table.copy()
            t[1, (n + 49) // bt] = bad
            code, out, ls = call(dev, t, cu, kv)
            assert code == L.LSC_ERR_OUT_OF_RANGE
            check4(host, 1, b, qx, dtype, 0.125, True, out, ls, rows=good)
        for bad in (-1, 1 << 20, 2 ** 31 - 1):
            k = kv.copy()
            k[1] = bad
            code, out, ls = call(dev, table, cu, k)
            assert code == L.LSC_ERR_INVALID_ARG
            check4(host, 1, b, qx, dtype, 0.125, True, out, ls, rows=good)
            assert (out[n:2 * n] == 0).all() and torch.isinf(ls[n:2 * n]).all()
        for bad in ([0, n + 1, n, 2 * n + 1], [0, n, 2 * n, 2 * n + 9], [3, n, 2 * n, 2 * n + 1], [0, -4, 2 * n, 2 * n + 1],
                    [-2 ** 31, 1, 4, 2 ** 31 - 1]):
            code, _, _ = call(dev, table, np.array(bad, np.int32), kv)
            assert code == L.LSC_ERR_INVALID_ARG
        k = kv.copy()
        t = b.cu.copy()
        t[2:] += 1  # a sequence of one token more than the bound: its rows stay as they were
        if n > 1:
            code, out, ls = call(dev, table, np.minimum(t, b.T).astype(np.int32), k)
            assert code == L.LSC_ERR_INVALID_ARG and (out[n:2 * n + 1] == 7).all()
        code, out, ls = call(dev, table, cu, kv)
        assert code == L.LSC_OK
        check4(host, 1, b, qx, dtype, 0.125, True, out, ls)


@pytest.mark.parametrize("H,G,D,bt", [(8, 4, 128, 16), (2, 8, 256, 64), (4, 2, 64, 12), (2, 16, 64, 5)])
def test_one_workspace_serves_every_smaller_step(lsc, H, G, D, bt):
    """Also where a smaller step expands its rows and the largest does not (its rows would pass what is allowed, or fill
    too few row blocks)."""
    rng = np.random.default_rng(13)
    pad = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    dev_ints = torch.zeros(1 << 12, dtype=torch.int32, device="cuda")
    host = Host4(20, bt, H, D, layers=1)

    def need(dev, n_seq, total, max_seq, max_kv, blocks, off=0):
        b = L.kv_batch(n_seq, total, dev_ints, dev_ints, dev_ints, max_blocks=blocks)
        at = pad.data_ptr() + off
        a = L.kv_attend_args(b, H * G, at, at, BF, 0.125, max_seq_tokens=max_seq, max_kv_tokens=max_kv)
        rc, bytes_ = L.lsc_kv_attend_workspace_bytes(dev.pool, a)
        assert rc == L.LSC_OK
        return bytes_

    with DevKv(host) as dev:
        for S, most, kv in ((64, 40, 1024), (8, 2000, 5000), (500, 3000, 40000), (3, 1, 900)):
            wide = -(-kv // bt)
            top = need(dev, S, S * most, most, kv, wide)
            assert top == need(dev, S, S * most, most, kv, wide, off=2)  # the pointers do not matter
            for _ in range(300):
                s = int(rng.integers(1, S + 1))
                m = int(rng.integers(1, most + 1)) if rng.random() < 0.7 else 1
                t = int(rng.integers(1, s * m + 1))
                assert need(dev, s, t, m, int(rng.integers(1, kv + 1)), wide, off=2 * int(rng.integers(0, 2))) <= top
        assert need(dev, 500, 10 ** 6, 3000, 40000, -(-40000 // bt)) < 5 << 30  # what is allowed
        top = need(dev, 4, 2000, 600, 1024, -(-1024 // bt))
    ws = torch.full((top,), 0xFF, dtype=torch.uint8, device="cuda")
    for n, kvs in (([600, 1, 9], [700, 900, 9]), ([1] * 4, [1, 600, 64, 0]), ([40, 3], [500, 77]), ([300, 290], [300, 1000])):
        blocks = int(sum(-(-x // bt) for x in kvs)) + 1
        b = Batch(rng, n, kvs, bt, blocks)
        host = filled4(rng, b, blocks, bt, H, D, layers=1, layer=0)
        q, qx = dense(rng.standard_normal((b.T, H * G, D)), BF)
        out = torch.full_like(q, 7.0)
        ls = torch.full((b.T, H * G), 7.0, device="cuda")
        with DevKv(host) as dev:
            a = L.kv_attend_args(b.device(), H * G, q, out, BF, D ** -0.5, lse=ls, max_seq_tokens=max(n),
                                 workspace=ws, workspace_bytes=top)
            assert L.lsc_kv_attend(dev.pool, 0, a, cur()) == L.LSC_OK
            torch.cuda.synchronize()
            assert dev.status() == L.LSC_OK
        check4(host, 0, b, qx, BF, D ** -0.5, True, out, ls)


@every_form
def test_workspace_rules(lsc, form):
    """Too small a workspace is refused; without one the library finds its own; both give the same bits."""
    dtype, n, bt, D, G = FORMS[form]
    rng = np.random.default_rng(9)
    b = Batch(rng, [n, n], [n + 900, n + 1200], bt, (2 * n + 2100) // bt + 3)
    host = filled4(rng, b, (2 * n + 2100) // bt + 3, bt, 2, D)
    q, qx = dense(rng.standard_normal((b.T, 2 * G, D)), dtype)
    with DevKv(host) as dev:
        out, _ = run_attend(dev, 1, b, q, dtype, 2 * G, 0.1, True, max_seq_tokens=n)
        own = torch.zeros_like(out)
        args = L.kv_attend_args(b.device(), 2 * G, q, own, dtype, 0.1, max_seq_tokens=n)
        rc, need = L.lsc_kv_attend_workspace_bytes(dev.pool, args)
        assert rc == L.LSC_OK and (need > 0) == (not form.startswith("cuda"))
        assert L.lsc_kv_attend(dev.pool, 1, args, cur()) == L.LSC_OK
        torch.cuda.synchronize()
        assert torch.equal(own, out)
        if need:
            if expands(form):
                assert need > 2 * (b.kv.sum()) * 2 * D * 2
            ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
            args.workspace, args.workspace_bytes = ws.data_ptr(), need - 1
            assert L.lsc_kv_attend(dev.pool, 1, args, cur()) == L.LSC_ERR_INVALID_ARG


@pytest.mark.parametrize("form", [f for f in FORMS if f.startswith("expanded")])
@pytest.mark.parametrize("kv", [900, 5000])
def test_without_memory_for_its_rows_a_step_goes_on(lsc, form, kv, monkeypatch):
    """Without a workspace, where the device has no room for the expanded rows (injected): converted by tile, the same
    bits, whole units and cut ones."""
    dtype, n, bt, D, G = FORMS[form]
    rng = np.random.default_rng(n + kv)
    blocks = (n + kv) // bt + 40
    b = Batch(rng, [n, n], [n + kv, n + 9], bt, blocks + n // bt)
    host = filled4(rng, b, blocks + n // bt, bt, 2, D)
    q, qx = dense(rng.standard_normal((b.T, 2 * G, D)), dtype)
    with DevKv(host) as dev:
        def call():
            out, ls = torch.zeros(b.T, 2 * G * D, dtype=TORCH[dtype], device="cuda"), torch.zeros(b.T, 2 * G, device="cuda")
            args = L.kv_attend_args(b.device(), 2 * G, q, out, dtype, 0.1, lse=ls, max_seq_tokens=n)
            assert L.lsc_kv_attend(dev.pool, 1, args, cur()) == L.LSC_OK
            assert dev.status() == L.LSC_OK
            return out, ls
        want = call()
        monkeypatch.setenv("LSC_FAULT", "no_rows")
        got = call()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    if kv < 1000:
        check4(host, 1, b, qx, dtype, 0.1, True, *got)


@pytest.mark.parametrize("form", ["decode-bf16", "chunk-bf16", "expanded-bf16", "expanded-256"])
def test_graphs_with_workspaces_of_their_own(lsc, form):
    """Append and attend captured twice on a side stream, replayed in turn with other lengths and tables: the status word
    stays clean and both give the same bits."""
    dtype, n, bt, D, G = FORMS[form]
    rng = np.random.default_rng(8)
    H, S, blocks = 2, 3, 300
    batches = [Batch(rng, [n, 1, n], [n + 400, 70, n + 5], bt, blocks), Batch(rng, [n - 1, n, 1], [n + 80, n, 1000], bt, blocks)]
    wide, T = max(b.table.shape[1] for b in batches), max(b.T for b in batches)
    table = torch.zeros(S, wide, dtype=torch.int32, device="cuda")
    cu, kvl = torch.zeros(S + 1, dtype=torch.int32, device="cuda"), torch.zeros(S, dtype=torch.int32, device="cuda")
    q, k, v = (torch.zeros(T, h * D, dtype=TORCH[dtype], device="cuda") for h in (H * G, H, H))
    host = Host4(blocks, bt, H, D, layers=1, fill=0)
    side = torch.cuda.Stream()
    with DevKv(host) as dev:
        batch = L.kv_batch(S, T, table, cu, kvl, max_blocks=wide)
        runs = []
        for _ in range(2):
            out = torch.zeros(T, H * G * D, dtype=TORCH[dtype], device="cuda")
            a = L.kv_attend_args(batch, H * G, q, out, dtype, D ** -0.5, max_seq_tokens=n, max_kv_tokens=n + 1000)
            rc, need = L.lsc_kv_attend_workspace_bytes(dev.pool, a)
            ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
            a.workspace, a.workspace_bytes = ws.data_ptr(), need
            ap = L.kv_append_args(batch, k, v, dtype)

            def step(stream):
                assert L.lsc_kv_append(dev.pool, 0, ap, stream) == L.LSC_OK
                assert L.lsc_kv_attend(dev.pool, 0, a, stream) == L.LSC_OK

            side.wait_stream(cur())
            with torch.cuda.stream(side):
                step(side)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                step(torch.cuda.current_stream())
            runs.append((graph, out, ws))
        for b in batches:
            for i in range(S):
                bl, r = b.places(i, 0, int(b.kv[i]))
                for lane in (0, 1):
                    host.write(0, lane, bl, r, rng.standard_normal((len(bl), H, D)))
            dev.buf.copy_(torch.from_numpy(host.bytes.reshape(-1)))
            t = np.zeros((S, wide), np.int32)
            t[:, :b.table.shape[1]] = b.table
            for d, s in ((table, t), (cu, b.cu), (kvl, b.kv.astype(np.int32))):
                d.copy_(torch.from_numpy(s))
            (kd, kx), (vd, vx), (qd, qx) = (dense(rng.standard_normal((b.T, h, D)), dtype) for h in (H, H, H * G))
            for a_, s in ((k, kd), (v, vd), (q, qd)):
                a_[:b.T].copy_(s)
            for graph, out, ws in runs:
                ws.fill_(255)
                graph.replay()
            assert dev.status() == L.LSC_OK
            for i in range(S):
                bl, r = b.places(i, int(b.kv[i] - b.n[i]), int(b.kv[i]))
                host.write(0, 0, bl, r, kx[b.cu[i]:b.cu[i + 1]])
                host.write(0, 1, bl, r, vx[b.cu[i]:b.cu[i + 1]])
            np.testing.assert_array_equal(dev.download(), host.bytes)
            assert torch.equal(runs[0][1][:b.T], runs[1][1][:b.T])
            check4(host, 0, b, qx, dtype, D ** -0.5, True, runs[0][1][:b.T].clone(), None)


def test_a_step_on_another_stream_and_pools_side_by_side(lsc):
    """Two pools' steps on two streams at once, with arrays made on the current one."""
    rng = np.random.default_rng(21)
    H, G, D, bt = 2, 4, 128, 16
    streams = [torch.cuda.Stream() for _ in range(2)]
    jobs = []
    for i, n in enumerate((300, 2)):
        b = Batch(rng, [n, 1], [n + 200, 900], bt, 100)
        host = filled4(rng, b, 100, bt, H, D)
        q, qx = dense(rng.standard_normal((b.T, H * G, D)), BF)
        jobs.append((b, host, q, qx, n, torch.full((b.T, H * G * D), 7.0, dtype=torch.bfloat16, device="cuda")))
    devs = [DevKv(j[1]) for j in jobs]
    batches = [j[0].device() for j in jobs]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, dev, batch, (b, host, q, qx, n, out) in zip(streams, devs, batches, jobs):
            a = L.kv_attend_args(batch, H * G, q, out, BF, 0.1, max_seq_tokens=n)
            assert L.lsc_kv_attend(dev.pool, 1, a, s) == L.LSC_OK
    torch.cuda.synchronize()
    for dev, (b, host, q, qx, n, out) in zip(devs, jobs):
        assert dev.status() == L.LSC_OK
        check4(host, 1, b, qx, BF, 0.1, True, out, None)
        assert L.lsc_kv_pool_destroy(dev.pool) == L.LSC_OK


def test_many_sequences_and_a_block_far_into_the_pool(lsc):
    """More sequences than a CTA has threads, empty ones among them; and pages whose byte offset passes 32 bits, through
    append, attend in every form and gather."""
    rng = np.random.default_rng(10)
    S = 700
    kv = rng.integers(0, 40, S)
    n = np.minimum(1, kv)
    b = Batch(rng, n, kv, 16, int((-(-kv // 16)).sum()))
    host = filled4(rng, b, int((-(-kv // 16)).sum()), 16, 1, 64)
    q, qx = dense(rng.standard_normal((b.T, 2, 64)), BF)
    x, _ = dense(host.read(1, 0, *[np.concatenate(a) for a in zip(*[b.places(i, kv[i] - n[i], kv[i]) for i in range(S)])]), BF)
    with DevKv(host) as dev:
        out, ls = run_attend(dev, 1, b, q, BF, 2, 0.125, True, max_seq_tokens=1)
        check4(host, 1, b, qx, BF, 0.125, True, out, ls)
        k, v = torch.zeros_like(x), torch.zeros_like(x)
        assert L.lsc_kv_gather(dev.pool, 1, L.kv_gather_args(b.device(), k, v, BF), cur()) == L.LSC_OK
        assert torch.equal(k, x)
        assert L.lsc_kv_append(dev.pool, 1, L.kv_append_args(b.device(), x, v, BF), cur()) == L.LSC_OK
        np.testing.assert_array_equal(dev.download(), host.bytes)  # what was read back is stored as it was
    page, bt, D = 1 << 30, 16, 64  # six pages of 1 GiB: lanes of 6 GiB
    desc = L.lsc_kv_pool_desc(1, 6, bt, 1, D, L.LSC_E2M1, page)
    buf = torch.empty(12 * page, dtype=torch.uint8, device="cuda")
    rc, pool = L.lsc_kv_pool_create(desc, buf, buf.numel())
    assert rc == L.LSC_OK
    for G, m in ((2, 80), (16, 80), (2, 3)):
        far = Host4(6, bt, 1, D, pad=0, layers=1)
        b = Batch(rng, [m], [80], bt, 6)
        (kd, kx), (vd, vx) = (dense(rng.standard_normal((80, 1, D)), BF) for _ in "kv")
        bl, r = b.places(0, 0, 80)
        far.write(0, 0, bl, r, kx)
        far.write(0, 1, bl, r, vx)
        whole = Batch(rng, [80], [80], bt, 6)
        whole.table = b.table
        wb, batch = whole.device(), b.device()
        q, qx = dense(rng.standard_normal((m, G, D)), BF)
        out, ls = torch.zeros(m, G * D, dtype=torch.bfloat16, device="cuda"), torch.zeros(m, G, device="cuda")
        assert L.lsc_kv_append(pool, 0, L.kv_append_args(wb, kd, vd, BF), cur()) == L.LSC_OK
        assert L.lsc_kv_attend(pool, 0, L.kv_attend_args(batch, G, q, out, BF, 0.125, lse=ls), cur()) == L.LSC_OK
        back = torch.zeros_like(kd)
        assert L.lsc_kv_gather(pool, 0, L.kv_gather_args(wb, back, torch.zeros_like(kd), BF), cur()) == L.LSC_OK
        torch.cuda.synchronize()
        check4(far, 0, b, qx, BF, 0.125, True, out, ls)
        np.testing.assert_array_equal(back.double().cpu().numpy().reshape(80, 1, D), far.read(0, 0, bl, r))
    assert L.lsc_kv_pool_destroy(pool) == L.LSC_OK


EXPIRING = ["decode-bf16", "decode-f16", "chunk-bf16", "chunk-256", "expanded-bf16", "few-rows-no-box"]


def expiring_call(form, expired):
    dtype, n, bt, D, G = FORMS[form]
    rng = np.random.default_rng(D + n)
    blocks = (3 * n + 2000) // bt + 4
    b = Batch(rng, [n] * 3, [n + 100, n + 1800, n], bt, blocks)
    host = filled4(rng, b, blocks, bt, 2, D)
    q, qx = dense(rng.standard_normal((b.T, 2 * G, D)), dtype)
    with DevKv(host) as dev:
        out, ls = run_attend(dev, 1, b, q, dtype, 2 * G, 0.1, True, max_seq_tokens=n)
        assert dev.status() == (L.LSC_ERR_DEV_TIMEOUT if expired else L.LSC_OK)
        np.testing.assert_array_equal(dev.download(), host.bytes)
    if not expired:
        check4(host, 1, b, qx, dtype, 0.1, True, out, ls)


def test_waits_that_run_out_in_every_form(lsc):
    """With the injected fault every bounded wait gives up at once: the kernels return, the status word says so; the same
    calls without it are right."""
    code = """
import sys
sys.path[:0] = [%r, %r]
import test_gpu_kv4_edges as E
for form in E.EXPIRING:
    E.expiring_call(form, expired=True)
print("reported")
"""
    r = subprocess.run([sys.executable, "-c", code % (os.path.dirname(HERE), HERE)], capture_output=True, text=True,
                       env=dict(os.environ, LSC_FAULT="timeout0"), timeout=300)
    assert "reported" in r.stdout, r.stderr[-2000:]
    for form in EXPIRING:
        expiring_call(form, expired=False)
