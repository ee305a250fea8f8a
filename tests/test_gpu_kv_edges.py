"""GPU: append, attend and copy_prefix over the K/V block pool where they are easiest to get wrong: flat tails behind
one large score, queries and scores that are not finite, V far from 1, blocks that fit no TMA box, decode batches
large enough to read several kv heads side by side, one workspace for many steps, pools made while a graph is being
captured, and waits that run out.  Plain 64-bit forms and tolerances are those of test_gpu_kv_step.py (where a test
needs another bound, its own comment derives it)."""
import functools
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from linear_attention_state_lsc_gb300 import lsc as L

import _kv
from _kv import NAME, TORCH, Batch, DevKv, HostKv
from test_gpu_kv_step import HALF, check_attend, cur, dense, filled, run_attend

pytestmark = pytest.mark.gpu

BF, F16, E4 = L.LSC_BF16, L.LSC_F16, L.LSC_E4M3
HERE = os.path.dirname(os.path.abspath(__file__))


def fill(host, layer, lane, block, row, x):
    """HostKv.write, all rows at once."""
    if host.dtype == E4:
        code, up = _kv.quantise(x)
        host.rows(layer, lane)[block, row] = code
        host.scales(layer, lane)[block, row] = up
    else:
        host.rows(layer, lane)[block, row] = _kv.to_bytes(x, host.dtype)


def shared(S, n, kv, bt):
    """S sequences of n new tokens that all read the same kv cached ones, in blocks 0, 1, 2 ..."""
    b = Batch(np.random.default_rng(0), [n] * S, [0] * S, bt, 0)
    b.kv = np.full(S, kv)
    b.table = np.tile(np.arange(-(-kv // bt), dtype=np.int32), (S, 1))
    return b


@functools.lru_cache(4)
def one_and_flat(pool, bt, D, kv):
    """Rows whose key is zero and whose v is 1, behind one whose key is e_0 and whose v is 1 in even columns and 0 in odd."""
    host = HostKv(-(-kv // bt), bt, 1, D, pool, layers=1)
    k, v = np.zeros((2, 1, 1, D)), np.ones((2, 1, 1, D))
    k[0, 0, 0, 0] = 1
    v[0, 0, 0, 1::2] = 0
    at = np.arange(kv)
    for lane, x in enumerate((k, v)):
        fill(host, 0, lane, at[1:] // bt, at[1:] % bt, x[1])
        fill(host, 0, lane, [0], [0], x[0])
    return host


def flat_tail(pool, dtype, n, bt, D, gap, floor, kv=32768, G=4, S=160):
    """One position with a score `gap` (in powers of two) above all others, which are equal.  v is 1 everywhere but in
    the large one's odd columns, where it is 0: even columns give 1, odd ones the share of the others' weights.  A
    weight is off by half a step of its bits (E4M3 chunks: nine significant ones) or by `floor` times the largest."""
    b, host = shared(S, n, kv, bt), one_and_flat(pool, bt, D, kv)
    x = np.zeros((b.T, G, D))
    x[:, :, 0] = gap * np.log(2) * 8
    q, qx = dense(x, dtype)
    s = float(qx[0, 0, 0]) / 8
    with DevKv(host) as dev:
        out, ls = run_attend(dev, 0, b, q, dtype, G, 0.125, False, max_seq_tokens=n)
        assert dev.status() == L.LSC_OK
    rest = (kv - 1) * np.exp(-s)
    want = np.where(np.arange(D) % 2, rest, 1 + rest) / (1 + rest)
    weight = HALF[dtype] if pool != E4 else 2.0 ** -9 if n * G > 64 else 2.0 ** -11
    err = (weight + (kv + 8) * 2.0 ** -23 + 2.0 ** -20) * want + kv * floor
    bound = err + HALF[dtype] * (want + err)
    got = out.double().cpu().numpy().reshape(-1, D)
    over = np.abs(got - want) / bound
    assert over.max() <= 1, (over.max(), got[over.argmax() // D, :2], want[:2])
    # a score is off by less than 2^-20 of itself here, the sum of kv terms by kv 2^-23 of itself
    assert (np.abs(ls.double().cpu().numpy() - s - np.log1p(rest)) <= (1 + s) * 2.0 ** -20 + (kv + 8) * 2.0 ** -23).all()


@pytest.mark.parametrize("gap", [3.0, 16.9, 17.1, 20.3, 25.1])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_flat_tail_counts_in_e4m3_chunks(lsc, D, gap):
    """Weights go to the products as e5m2 numbers, multiples of 2^-16, beside a largest one of 2^9 or more: 2^-26 of it
    is the most that one is off."""
    flat_tail(E4, BF, 40, 64, D, gap, 2.0 ** -26)


@pytest.mark.parametrize("gap", [3.0, 17.1, 24.9, 25.1])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("pool,dtype,n,bt", [(F16, F16, 40, 64), (F16, F16, 1, 64), (F16, F16, 1, 12), (E4, F16, 1, 64),
                                             (E4, BF, 1, 64), (E4, F16, 1, 12), (E4, F16, 8, 64), (BF, BF, 1, 64)],
                         ids=["chunk", "decode", "rows", "decode8", "decode8-bf16", "rows8", "rows8-32", "bf16"])
def test_a_flat_tail_counts_in_f16_weights(lsc, pool, dtype, n, bt, D, gap):
    """f16 weights are multiples of 2^-24 beside a largest one of 2^7 or more: off by 2^-32 of it at most."""
    flat_tail(pool, dtype, n, bt, D, gap, 0 if dtype == pool == BF else 2.0 ** -32)


FORMS = [(BF, BF, 40, 64), (F16, F16, 40, 64), (E4, BF, 40, 64), (BF, BF, 40, 12), (BF, BF, 2, 64), (F16, F16, 2, 12),
         (E4, BF, 2, 64), (E4, F16, 2, 64), (E4, BF, 2, 12), (E4, BF, 12, 64), (L.LSC_F32, L.LSC_F32, 5, 64)]
FORM_IDS = ["chunk-bf16", "chunk-f16", "chunk-e4m3", "chunk-bf16-12", "decode-bf16", "rows-f16", "decode-e4m3", "decode-e4m3-f16",
            "rows-e4m3", "rows-e4m3-48", "f32"]


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("pool,dtype,n,bt", FORMS, ids=FORM_IDS)
def test_a_query_that_is_not_finite_is_nan_alone(lsc, pool, dtype, n, bt, D):
    """An infinity or NaN in a row of q: that row is NaN (a score is infinite or NaN), the rows beside it are as if it
    were not there."""
    rng = np.random.default_rng(n + D)
    S, G = 4, 4
    b = Batch(rng, [n] * (S + 1), [n + 60, 150, 300, 77, 0], bt, 60, spare=1)
    host = filled(rng, b, 60, bt, 2, D, pool)
    x = 2 * rng.standard_normal((b.T, 2 * G, D))
    x[S * n:S * n + n, :, 3] = np.inf  # the last sequence sees nothing: zeros all the same
    sick = [(0, 1, np.inf), (n, 0, -np.inf), (2 * n + 1, 5, np.nan), (3 * n, 7, np.inf)]  # (row, head, what)
    for t, h, what in sick:
        x[t, h, 2:20] *= 300  # the finite elements of such a row may be large too
        x[t, h, 5] = what
    q, qx = dense(x, dtype)
    with DevKv(host) as dev:
        out, ls = run_attend(dev, 1, b, q, dtype, 2 * G, D ** -0.5, True, max_seq_tokens=n)
        assert dev.status() == L.LSC_OK
    got = out.view(b.T, 2 * G, D)
    for t, h, _ in sick:
        assert torch.isnan(got[t, h]).all(), (t, h)
        assert not torch.isfinite(ls[t, h])
        # the plain form of a row of zeros in its place, so that all the others are compared
        qx[t, h] = 0
        want, lse = (a[t, h] for a in _kv.attend(host, 1, b, qx, D ** -0.5, True)[:2])
        got[t, h] = torch.from_numpy(want).to(got)
        ls[t, h] = float(lse)
    check_attend(host, 1, b, qx, dtype, D ** -0.5, True, out, ls)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("pool,dtype,n,bt", [f for f in FORMS if f[0] != E4],
                         ids=[i for f, i in zip(FORMS, FORM_IDS) if f[0] != E4])
def test_a_row_whose_scores_are_all_minus_infinity_is_nan(lsc, pool, dtype, n, bt, D):
    """exp(-inf) / 0: not the zeros of a row that sees nothing.  One sequence whose parts are joined, one that is not,
    one that sees finite scores beside the infinite ones, and one that sees nothing."""
    rng = np.random.default_rng(n * D)
    b = Batch(rng, [n] * 4, [n, 2600, 90, 0], bt, 300, spare=1)
    host = filled(rng, b, 300, bt, 1, D, pool)
    for i, finite in ((0, 0), (1, 0), (2, 30)):
        bl, r = b.places(i, 0, int(b.kv[i]) - finite)
        k = host.read(1, 0, bl, r)
        k[:, 0, 3] = -np.inf
        fill(host, 1, 0, bl, r, k)
    x = rng.standard_normal((b.T, 4, D))
    x[:, :, 3] = 1
    q, qx = dense(x, dtype)
    with DevKv(host) as dev:
        out, ls = run_attend(dev, 1, b, q, dtype, 4, D ** -0.5, False, max_seq_tokens=n)
        assert dev.status() == L.LSC_OK
    assert torch.isnan(out[:2 * n]).all() and (ls[:2 * n] == -np.inf).all()
    assert (out[3 * n:4 * n] == 0).all() and (ls[3 * n:4 * n] == -np.inf).all()
    # the third: the positions of -infinity have weight 0; as if they held the largest negative scores
    bl, r = b.places(2, 0, 60)
    k = host.read(1, 0, bl, r)
    k[:, 0, 3] = -30000.0
    fill(host, 1, 0, bl, r, k)
    want = _kv.attend(host, 1, b, qx, D ** -0.5, False)[0]
    got = out.double().cpu().numpy().reshape(b.T, 4, D)
    assert np.isfinite(got[2 * n:3 * n]).all()
    assert np.abs(got - want)[2 * n:3 * n].max() <= 2.0 ** -6 * np.abs(want[2 * n:3 * n]).max()


@pytest.mark.parametrize("power", [-70, -50, 60, 100, 124])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,bt", [(40, 64), (2, 64), (2, 12), (12, 64)], ids=["chunk", "decode", "rows", "rows-48"])
def test_v_far_from_one(lsc, n, bt, D, power):
    """E4M3 pools whose V rows are all tiny or all huge: the bounds of test_attend, relative to V's size."""
    rng = np.random.default_rng(power + 2 * D)
    b = Batch(rng, [n] * 2, [300, 1400], bt, 160)
    host = HostKv(160, bt, 1, D, E4)
    for i in range(2):
        bl, r = b.places(i, 0, int(b.kv[i]))
        for lane, up in ((0, 0), (1, power)):
            fill(host, 1, lane, bl, r, rng.standard_normal((len(r), 1, D)) * 2.0 ** up)
    q, qx = dense(rng.standard_normal((b.T, 4, D)), BF)
    with DevKv(host) as dev:
        out, ls = run_attend(dev, 1, b, q, BF, 4, D ** -0.5, True, max_seq_tokens=n)
        assert dev.status() == L.LSC_OK
    check_attend(host, 1, b, qx, BF, D ** -0.5, True, out, ls)


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("n,bt", [(40, 64), (2, 64), (2, 12), (12, 64)], ids=["chunk", "decode", "rows", "rows-48"])
def test_the_sum_does_not_depend_on_a_v_row_of_nan(lsc, n, bt, D):
    """E4M3 pools: out is NaN where a row's scale byte says so, lse is what the scores give; scores from -80 to 80 (powers
    of two), the NaN row's among the smallest."""
    rng = np.random.default_rng(D + n)
    b = Batch(rng, [n] * 2, [200, 1400], bt, 160)
    host = HostKv(160, bt, 1, D, E4)
    for i in range(2):
        bl, r = b.places(i, 0, int(b.kv[i]))
        k, v = np.zeros((2, len(r), 1, D))
        k[:, 0, 0] = rng.integers(-10, 11, len(r))
        k[60, 0, 0] = -10
        v[:] = 1
        v[60, 0, 3] = np.nan
        fill(host, 1, 0, bl, r, k)
        fill(host, 1, 1, bl, r, v)
    x = np.zeros((b.T, 4, D))
    x[:, :, 0] = 8
    q, qx = dense(x, BF)
    with DevKv(host) as dev:
        out, ls = run_attend(dev, 1, b, q, BF, 4, np.log(2), True, max_seq_tokens=n)
        assert dev.status() == L.LSC_OK
    assert torch.isnan(out).all()
    with np.errstate(invalid="ignore"):
        want = _kv.attend(host, 1, b, qx, float(np.float32(np.log(2))), True)[1]
    # scores up to 56 and sums of up to 1400 terms in 32 bits
    assert (np.abs(ls.double().cpu().numpy() - want) <= 56 * 2.0 ** -20 + 1408 * 2.0 ** -23).all()


def test_lengths_at_the_end_of_31_bits_are_recorded(lsc):
    """Positions are counted in 31 bits with room for a tile: a longer sequence is recorded and has no cached tokens, in
    every form, though its table would hold it.  One block stands in all entries of the table."""
    bt = 1 << 16
    for pool, dtype, D, G, n in ((L.LSC_F32, L.LSC_F32, 8, 2, 1), (BF, BF, 64, 4, 1), (BF, BF, 64, 4, 40), (E4, BF, 64, 4, 12)):
        host = HostKv(1, bt, 1, D, pool, pad=0, layers=1, fill=0)
        for kv in (2 ** 31 - 1, 2 ** 31 - 1024):
            with DevKv(host) as dev:
                table = torch.zeros((1, 1 << 15), dtype=torch.int32, device="cuda")
                cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
                lens = torch.tensor([kv], dtype=torch.int32, device="cuda")
                q, out = (torch.full((n, G * D), 7.0, dtype=TORCH[dtype], device="cuda") for _ in "qo")
                ls = torch.full((n, G), 7.0, device="cuda")
                batch = L.kv_batch(1, n, table, cu, lens, max_blocks=1 << 15)
                args = L.kv_attend_args(batch, G, q, out, dtype, 0.125, lse=ls)
                assert L.lsc_kv_attend(dev.pool, 0, args, cur()) == L.LSC_OK
                assert dev.status() == L.LSC_ERR_INVALID_ARG
                assert (out == 0).all() and torch.isinf(ls).all()


def test_a_pool_is_made_and_used_while_a_graph_is_captured(lsc):
    """A pool on a borrowed buffer, made and one destroyed on the thread that is capturing a stream (the default, strict
    mode), as before the pool had a status word."""
    rng = np.random.default_rng(12)
    b = Batch(rng, [3, 1], [70, 20], 16, 10)
    host = HostKv(10, 16, 2, 64, BF, layers=1)
    buf = torch.from_numpy(host.bytes.reshape(-1).copy()).cuda()
    (k, kx), (v, vx) = (dense(rng.standard_normal((b.T, 2, 64)), BF) for _ in "kv")
    args = L.kv_append_args(b.device(), k, v, BF)
    rc, warm = L.lsc_kv_pool_create(host.desc, buf, buf.numel())  # the kernel is loaded before the capture
    assert rc == L.LSC_OK and L.lsc_kv_append(warm, 0, args, cur()) == L.LSC_OK
    torch.cuda.synchronize()
    buf.copy_(torch.from_numpy(host.bytes.reshape(-1)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rc, pool = L.lsc_kv_pool_create(host.desc, buf, buf.numel())
        made = rc
        gone = L.lsc_kv_pool_destroy(warm)
        call = L.lsc_kv_append(pool, 0, args, cur()) if rc == L.LSC_OK else rc
    assert (made, gone, call) == (L.LSC_OK,) * 3
    graph.replay()
    torch.cuda.synchronize()
    assert L.lsc_kv_pool_status(pool, cur()) == L.LSC_OK
    for i in range(2):
        bl, r = b.places(i, int(b.kv[i] - b.n[i]), int(b.kv[i]))
        host.write(0, 0, bl, r, kx[b.cu[i]:b.cu[i + 1]])
        host.write(0, 1, bl, r, vx[b.cu[i]:b.cu[i + 1]])
    np.testing.assert_array_equal(buf.cpu().numpy().reshape(host.bytes.shape), host.bytes)
    del graph
    assert L.lsc_kv_pool_destroy(pool) == L.LSC_OK


@pytest.mark.parametrize("pool,H,G,D,bt", [(BF, 8, 4, 128, 16), (BF, 2, 8, 256, 64), (E4, 8, 4, 128, 64), (F16, 4, 2, 64, 12),
                                           (E4, 2, 16, 64, 5)])
def test_one_workspace_serves_every_smaller_step(lsc, pool, H, G, D, bt):
    """What the query answers for the largest sizes is enough for any step within them, whichever kernel it takes and
    however q and out are aligned; a small one of each kind is run in it."""
    rng = np.random.default_rng(13)
    dtype = F16 if pool == F16 else BF
    S, most, kv = 64, 40, 1024
    host = HostKv(20, bt, H, D, pool, layers=1)
    pad = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    dev_ints = torch.zeros(1 << 12, dtype=torch.int32, device="cuda")

    def need(dev, n_seq, total, max_seq, max_kv, off=0):
        b = L.kv_batch(n_seq, total, dev_ints, dev_ints, dev_ints, max_blocks=-(-kv // bt))
        at = pad.data_ptr() + off
        a = L.kv_attend_args(b, H * G, at, at, dtype, 0.125, max_seq_tokens=max_seq, max_kv_tokens=max_kv)
        rc, bytes_ = L.lsc_kv_attend_workspace_bytes(dev.pool, a)
        assert rc == L.LSC_OK
        return bytes_

    with DevKv(host) as dev:
        top = need(dev, S, S * most, most, kv)
        assert top == need(dev, S, S * most, most, kv, off=2)  # the pointers do not matter
        for _ in range(300):
            s = int(rng.integers(1, S + 1))
            m = int(rng.integers(1, most + 1)) if rng.random() < 0.7 else 1
            t = int(rng.integers(1, s * m + 1))
            assert need(dev, s, t, m, int(rng.integers(1, kv + 1)), off=2 * int(rng.integers(0, 2))) <= top
    ws = torch.full((top,), 0xFF, dtype=torch.uint8, device="cuda")
    for n, kvs in (([40, 1, 9], [40, 900, 9]), ([1] * 6, [1, 600, 64, 65, 200, 0]), ([3, 1], [500, 77]), ([1], [1000])):
        blocks = int(sum(-(-x // bt) for x in kvs)) + 1
        b = Batch(rng, n, kvs, bt, blocks)
        host = filled(rng, b, blocks, bt, H, D, pool, layers=1, layer=0)
        q, qx = dense(rng.standard_normal((b.T, H * G, D)), dtype)
        out = torch.full_like(q, 7.0)
        ls = torch.full((b.T, H * G), 7.0, device="cuda")
        with DevKv(host) as dev:
            a = L.kv_attend_args(b.device(), H * G, q, out, dtype, D ** -0.5, lse=ls, max_seq_tokens=max(n),
                                 workspace=ws, workspace_bytes=top)
            assert L.lsc_kv_attend(dev.pool, 0, a, cur()) == L.LSC_OK
            torch.cuda.synchronize()
            assert dev.status() == L.LSC_OK
        check_attend(host, 0, b, qx, dtype, D ** -0.5, True, out, ls)


def test_a_large_bound_stays_on_the_tensor_cores(lsc):
    """131072 rows of 16 q heads over 2 kv heads and a bound of 2^20 positions count 67 million tiles: far from 31 bits.
    With the injected fault every bounded wait gives up at once, so the status word tells the tensor-core kernel (which
    waits) from the CUDA-core one (which does not).  One sequence of 100 tokens is all that is there."""
    code = """
import sys
sys.path[:0] = [%r, %r]
import torch
from _kv import DevKv, HostKv
from linear_attention_state_lsc_gb300 import lsc as L
T, H, G, D, bt = 131072, 2, 8, 128, 64
with DevKv(HostKv(4, bt, H, D, L.LSC_BF16, layers=1, fill=0)) as dev:
    table = torch.zeros((1, 16384), dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 100], dtype=torch.int32, device="cuda")
    kv = torch.tensor([200], dtype=torch.int32, device="cuda")
    q = torch.zeros((T, H * G * D), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    a = L.kv_attend_args(L.kv_batch(1, T, table, cu, kv, max_blocks=16384), H * G, q, out, L.LSC_BF16, 0.1)
    assert L.lsc_kv_attend(dev.pool, 0, a, torch.cuda.current_stream()) == L.LSC_OK
    assert dev.status() == L.LSC_ERR_DEV_TIMEOUT, dev.status()
print("reported")
"""
    r = subprocess.run([sys.executable, "-c", code % (os.path.dirname(HERE), HERE)], capture_output=True, text=True,
                       env=dict(os.environ, LSC_FAULT="timeout0"), timeout=300)
    assert "reported" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("bt", [64, 12])
@pytest.mark.parametrize("pool,dtype", [(BF, BF), (F16, F16), (E4, BF)], ids=["bf16", "f16", "e4m3"])
def test_a_bound_above_the_step_s_tokens(lsc, pool, dtype, bt):
    """max_seq_tokens as a constant of the program, above what this step brings: the same bits as with the step's own."""
    rng = np.random.default_rng(14)
    b = Batch(rng, [1], [700], bt, 70)
    host = filled(rng, b, 70, bt, 2, 128, pool)
    q, qx = dense(rng.standard_normal((1, 16, 128)), dtype)
    with DevKv(host) as dev:
        own = run_attend(dev, 1, b, q, dtype, 16, 0.1, True, max_seq_tokens=1)
        for bound in (16, 1 << 30):
            out, ls = run_attend(dev, 1, b, q, dtype, 16, 0.1, True, max_seq_tokens=bound)
            check_attend(host, 1, b, qx, dtype, 0.1, True, out, ls)
            assert torch.equal(out, own[0]) and torch.equal(ls, own[1])
        assert dev.status() == L.LSC_OK
        need = [L.lsc_kv_attend_workspace_bytes(dev.pool, L.kv_attend_args(b.device(), 16, q, out, dtype, 0.1, max_seq_tokens=m))[1]
                for m in (1, 16, 1 << 30)]
    assert need[0] == need[1] == need[2]  # the same rows a tile


@pytest.mark.parametrize("lengths", [([1, 1, 1, 1], [1, 13, 300, 0]), ([2, 1], [900, 61]), ([70, 0, 130, 3], [70, 5, 400, 1]),
                                     ([9, 30], [4, 700])], ids=["decode", "few", "chunk", "ahead"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bt", [12, 5, 1])
@pytest.mark.parametrize("pool,dtype", [(BF, BF), (F16, F16), (E4, BF), (E4, F16)], ids=["bf16", "f16", "e4m3", "e4m3-f16"])
def test_blocks_that_fit_no_box(lsc, pool, dtype, bt, D, lengths):
    """Block sizes that are no multiple of 8 tokens: rows come one by one; below 8 the table is looked up directly."""
    n, kv = lengths
    rng = np.random.default_rng(bt * D + len(n))
    blocks = int(sum(-(-k // bt) for k in kv)) + 3
    b = Batch(rng, n, kv, bt, blocks, spare=2, wide=1)
    host = filled(rng, b, blocks, bt, 2, D, pool)
    q, qx = dense(2 * rng.standard_normal((b.T, 8, D)), dtype)
    with DevKv(host) as dev:
        for causal in (True, False):
            out, ls = run_attend(dev, 1, b, q, dtype, 8, D ** -0.5, causal, max_seq_tokens=max(n))
            check_attend(host, 1, b, qx, dtype, D ** -0.5, causal, out, ls)
        assert dev.status() == L.LSC_OK
        np.testing.assert_array_equal(dev.download(), host.bytes)


@pytest.mark.parametrize("pool,D", [(BF, 64), (BF, 256), (E4, 64), (E4, 128)])
@pytest.mark.parametrize("bt", [12, 5])
@pytest.mark.parametrize("few", [False, True])
def test_runs_that_begin_and_end_anywhere_without_boxes(lsc, pool, D, bt, few):
    """Many short units beside long ones, cut between, inside and behind a unit's tiles."""
    rng = np.random.default_rng(bt + D)
    S = 31
    n = rng.integers(0, 3 if few else 12, S)
    kv = np.where(rng.random(S) < 0.3, rng.integers(1100, 2500, S), rng.integers(1, 300, S)) + n
    blocks = int((-(-kv // bt)).sum())
    b = Batch(rng, n, kv, bt, blocks, spare=1)
    host = filled(rng, b, blocks, bt, 2, D, pool)
    q, qx = dense(2 * rng.standard_normal((b.T, 16, D)), BF)
    with DevKv(host) as dev:
        out, ls = run_attend(dev, 1, b, q, BF, 16, D ** -0.5, True, max_seq_tokens=int(n.max()))
        check_attend(host, 1, b, qx, BF, D ** -0.5, True, out, ls)
        assert dev.status() == L.LSC_OK


@pytest.mark.parametrize("pool,dtype", [(BF, BF), (F16, F16), (E4, BF)], ids=["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("D,bt", [(256, 8), (256, 16), (256, 32), (256, 48), (256, 128), (64, 8), (64, 32), (64, 128), (64, 200),
                                  (128, 8), (128, 48), (128, 128), (128, 256)])
def test_every_shape_of_box(lsc, pool, dtype, D, bt):
    """Boxes of 8 rows to a whole tile, of one 128-byte column and of all, for single tokens and for chunks."""
    rng = np.random.default_rng(bt + D)
    for n, kv in (([1, 2, 1], [1, 333, 700]), ([70, 3], [150, 530])):
        blocks = int(sum(-(-k // bt) for k in kv)) + 2
        b = Batch(rng, n, kv, bt, blocks, spare=1)
        host = filled(rng, b, blocks, bt, 2, D, pool)
        q, qx = dense(2 * rng.standard_normal((b.T, 8, D)), dtype)
        with DevKv(host) as dev:
            out, ls = run_attend(dev, 1, b, q, dtype, 8, D ** -0.5, True, max_seq_tokens=max(n))
            check_attend(host, 1, b, qx, dtype, D ** -0.5, True, out, ls)
            assert dev.status() == L.LSC_OK


def together(H, row):
    """Heads that the decode kernel reads side by side in a large batch: up to 1 KB of a position's row."""
    return 4 if H % 4 == 0 and row <= 256 else 2 if H % 2 == 0 and row <= 512 else 1


@pytest.mark.parametrize("n", [1, 2])
@pytest.mark.parametrize("pool,dtype,H,G,D", [(BF, BF, 2, 2, 256), (BF, BF, 4, 5, 128), (BF, BF, 8, 1, 64), (BF, BF, 2, 8, 128),
                                              (F16, F16, 2, 4, 128), (F16, F16, 4, 2, 64), (E4, BF, 8, 2, 128),
                                              (E4, BF, 4, 4, 256), (E4, BF, 2, 4, 256), (E4, F16, 4, 3, 64), (E4, F16, 2, 7, 128)])
def test_decode_batches_with_heads_side_by_side(lsc, pool, dtype, H, G, D, n):
    """Batches large enough for it (the rule's condition is checked), whole and cut units, and V that is not finite in one
    head of some sequences: neither the other heads nor the rows that do not see it change."""
    rng = np.random.default_rng(H * D + n)
    side = together(H, D * _kv.ES[pool])
    assert side > 1
    S, bt, most = 48, 32, 1700
    kv = rng.integers(1, 300, S) + n
    kv[[3, 17, 40]] = [most, 1100, 900]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert S * (H // side) * most >= sms * 4 * 64
    new = np.where(rng.random(S) < 0.2, 0, n)
    new[[3, 17]] = n
    blocks = int((-(-kv // bt)).sum())
    b = Batch(rng, new, kv, bt, blocks, spare=1)
    host = filled(rng, b, blocks, bt, H, D, pool)
    sick = H - 1
    for i in (3, 17):  # the last token's v, seen by its own row alone
        bl, r = b.places(i, kv[i] - 1, kv[i])
        x = host.read(1, 1, bl, r)
        x[0, sick, 5], x[0, sick, 9], x[0, sick, 12] = np.inf, -np.inf, np.nan
        fill(host, 1, 1, bl, r, x)
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
        if pool == E4:  # a row that held one is NaN throughout
            assert torch.isnan(got[t, heads]).all()
        else:
            assert (got[t, heads, 5] == np.inf).all() and (got[t, heads, 9] == -np.inf).all()
            assert torch.isnan(got[t, heads, 12]).all()
            keep = np.delete(np.arange(D), [5, 9, 12])
            assert torch.isfinite(got[t, heads][:, keep]).all()
        x = np.nan_to_num(host.read(1, 1, bl, r), nan=0, posinf=0, neginf=0)
        fill(host, 1, 1, bl, r, x)
        want = _kv.attend(host, 1, b, qx, D ** -0.5, True)[0][t, heads]
        cols = np.arange(D) if pool == E4 else np.array([5, 9, 12])
        got[t, heads][:, cols] = torch.from_numpy(want[:, cols]).to(got)
    check_attend(host, 1, b, qx, dtype, D ** -0.5, True, out, ls)


def test_waits_that_run_out_in_every_form(lsc):
    """As the test of the chunk kernel's waits: a decode batch with cut units, E4M3 chunks, and blocks without boxes give
    up, report it and return; the same call without the fault is right."""
    code = """
import sys
sys.path[:0] = [%r, %r]
import test_gpu_kv_edges as E
for case in E.EXPIRING:
    E.expiring_call(*case, expired=True)
print("reported")
"""
    r = subprocess.run([sys.executable, "-c", code % (os.path.dirname(HERE), HERE)], capture_output=True, text=True,
                       env=dict(os.environ, LSC_FAULT="timeout0"), timeout=300)
    assert "reported" in r.stdout, r.stderr[-2000:]
    for case in EXPIRING:
        expiring_call(*case, expired=False)


EXPIRING = [(BF, 64, 1, 64), (BF, 256, 1, 64), (E4, 128, 1, 64), (E4, 64, 70, 64), (E4, 128, 70, 64), (E4, 256, 70, 64),
            (BF, 128, 70, 12), (E4, 256, 70, 12)]


def expiring_call(pool, D, n, bt, expired):
    rng = np.random.default_rng(D + n)
    b = Batch(rng, [n] * 3, [300, 2600, n], bt, 300)
    host = filled(rng, b, 300, bt, 2, D, pool)
    q, qx = dense(rng.standard_normal((b.T, 8, D)), BF)
    with DevKv(host) as dev:
        out, ls = run_attend(dev, 1, b, q, BF, 8, 0.1, True, max_seq_tokens=n)
        assert dev.status() == (L.LSC_ERR_DEV_TIMEOUT if expired else L.LSC_OK)
        np.testing.assert_array_equal(dev.download(), host.bytes)
    if not expired:
        check_attend(host, 1, b, qx, BF, 0.1, True, out, ls)


@pytest.mark.parametrize("shape", [(2, 24, 16, 2, 64, 48), (3, 20, 5, 3, 7, 16), (1, 12, 64, 8, 128, 512), (2, 9, 7, 1, 33, 0)],
                         ids=str)
def test_copy_prefix_moves_the_scale_bytes(lsc, shape):
    """E4M3 pools: the codes and the scale bytes of rows [0, n) and nothing else of the destination pages."""
    layers, blocks, bt, H, D, pad = shape
    rng = np.random.default_rng(D)
    host = HostKv(blocks, bt, H, D, E4, pad=pad, layers=layers)
    host.bytes[:] = rng.integers(0, 256, host.bytes.shape, dtype=np.uint8)
    perm = rng.permutation(blocks)
    dst, src = perm[:6], rng.choice(perm[6:], 6)
    count = np.array([0, 1, bt, bt - 1, max(1, bt // 2), bt])
    with DevKv(host) as dev:
        rc, moved = L.lsc_copy_prefix(dev.pool, L.kv_ops(src, dst, count), cur())
        assert rc == L.LSC_OK
        got = dev.download()
    assert moved == int(count.sum()) * (H * D + H) * 2 * layers
    for s, d, n in zip(src, dst, count):
        for at, w in ((0, n * H * D), (host.scale_off, n * H)):
            host.bytes[:, :, d, at:at + w] = host.bytes[:, :, s, at:at + w]
    np.testing.assert_array_equal(got, host.bytes)
