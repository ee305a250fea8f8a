"""GPU: the row calls over E2M1 pools (append, rotated append, gather) with batches that do not fit, in their vector and
their element kernels; which kernels the calls of test_gpu_kv4_edges.py's forms take, as the device saw them; and the
layers of a step behind one another with one workspace."""
import numpy as np
import pytest
import torch

from linear_attention_state_lsc_gb300 import lsc as L

from _kv import TORCH, Batch, DevKv
from _kv4 import Host4
from test_gpu_kv4 import filled4
from test_gpu_kv4_edges import FORMS, every_form
from test_gpu_kv_step import cur, dense, run_attend
from test_gpu_rotary import freqs

pytestmark = pytest.mark.gpu

BF, F32 = L.LSC_BF16, L.LSC_F32
INV, OUT = L.LSC_ERR_INVALID_ARG, L.LSC_ERR_OUT_OF_RANGE
BAD = [("table", 40, OUT), ("table", -1, OUT), ("table", 2 ** 31 - 1, OUT), ("table", -2 ** 31, OUT), ("kv", -1, INV),
       ("kv", 1 << 20, INV), ("kv", 2 ** 31 - 1, INV), ("cu", [0, 5, 4, 6, 7], INV), ("cu", [3, 4, 5, 6, 99], INV),
       ("cu", [0, -4, 2, 3, 7], INV), ("cu", [-2 ** 31, 1, 4, 5, 2 ** 31 - 1], INV), ("cu", [0, 7, 7, 7, 10], INV)]


@pytest.mark.parametrize("call", ["append", "rotated", "gather"])
@pytest.mark.parametrize("dtype,H,D,stride", [(BF, 2, 64, 0), (BF, 4, 256, 0), (F32, 3, 64, 0), (BF, 2, 64, 131), (BF, 1, 48, 0)],
                         ids=str)
def test_bad_batches_are_recorded_and_stay_inside(lsc, call, dtype, H, D, stride):
    """Block ids, lengths and cu_seqlens that do not fit: the status word says so, the other sequences' rows are right,
    a token without a row is skipped or reads as zeros, and blocks of no sequence keep their bytes."""
    rng = np.random.default_rng(D + stride)
    bt, blocks = 16, 40
    b = Batch(rng, [1, 3, 2, 1], [40, 50, 60, 33], bt, blocks, spare=2, wide=1)
    w = stride or H * D
    (k, kx), (v, vx) = (dense(rng.standard_normal((b.T, H, D)), dtype, w) for _ in "kv")
    pos = torch.zeros(b.T, dtype=torch.int32, device="cuda")  # at position 0: the rows themselves
    r = L.rotary(32, pos, freqs(32))
    start = Host4(blocks, bt, H, D)
    for i in range(4):
        bl, row = b.places(i, 0, int(b.kv[i]))
        for lane in (0, 1):
            start.write(1, lane, bl, row, rng.standard_normal((len(bl), H, D)))
    for what, bad, code in BAD:
        host = Host4(blocks, bt, H, D)
        host.bytes[:] = start.bytes
        table, cu, kv = b.table.copy(), b.cu.copy(), b.kv.astype(np.int32)
        if what == "table":
            table[1, 49 // bt] = bad
        elif what == "kv":
            kv[1] = bad
        else:
            cu = np.array(bad, np.int32)
        arrays = [torch.from_numpy(a).cuda() for a in (table, cu, kv)]
        batch = L.kv_batch(4, b.T, *arrays, max_blocks=table.shape[1])
        out = [torch.full((b.T, w), 7.0, dtype=TORCH[dtype], device="cuda") for _ in "kv"]
        with DevKv(host) as dev:
            append = L.kv_append_args(batch, k, v, dtype, stride, stride)
            if call == "append":
                rc = L.lsc_kv_append(dev.pool, 1, append, cur())
            elif call == "rotated":
                rc = L.lsc_kv_append_rotated(dev.pool, 1, L.kv_append_rotated_args(append, r), cur())
            else:
                rc = L.lsc_kv_gather(dev.pool, 1, L.kv_gather_args(batch, *out, dtype, stride, stride), cur())
            assert rc == L.LSC_OK
            got = dev.download()
            assert dev.status() == code, (what, bad)
        used = np.unique(b.table[b.table >= 0])
        if call == "gather":
            np.testing.assert_array_equal(got, start.bytes)
            for y, lane in zip(out, (0, 1)):
                assert (y[:, H * D:] == 7).all()
                if what == "cu":
                    continue
                y = y[:, :H * D].double().cpu().numpy().reshape(b.T, H, D)
                assert (y[b.cu[1]:b.cu[2]][-1 if what == "table" else slice(None)] == 0).all()
                assert (y[b.cu[4]:] == 7).all()
                for i in (0, 2, 3):
                    want = start.read(1, lane, *b.places(i, int(b.kv[i] - b.n[i]), int(b.kv[i])))
                    np.testing.assert_array_equal(y[b.cu[i]:b.cu[i + 1]],
                                                  torch.from_numpy(want).to(TORCH[dtype]).double().numpy())
            continue
        np.testing.assert_array_equal(got[0], start.bytes[0])
        rest = np.setdiff1d(np.arange(blocks), used)
        np.testing.assert_array_equal(got[1][:, rest], start.bytes[1][:, rest])
        np.testing.assert_array_equal(got[1][:, :, start.payload:], start.bytes[1][:, :, start.payload:])
        if what == "cu":
            continue
        for i in (0, 2, 3):
            bl, row = b.places(i, int(b.kv[i] - b.n[i]), int(b.kv[i]))
            for lane, x in ((0, kx), (1, vx)):
                host.write(1, lane, bl, row, x[b.cu[i]:b.cu[i + 1]])
        if what == "table":  # its tokens in front of the bad block, if any, have their rows
            for t, p in enumerate(range(47, 50)):
                if p // bt != 49 // bt:
                    bl, row = b.places(1, p, p + 1)
                    for lane, x in ((0, kx), (1, vx)):
                        host.write(1, lane, bl, row, x[b.cu[1] + t:b.cu[1] + t + 1])
        np.testing.assert_array_equal(got, host.bytes, err_msg=f"{what} {bad}")


def kernels_of(call):
    """The names of the kernels that a call ran on the device."""
    from torch.profiler import ProfilerActivity, profile

    call()
    torch.cuda.synchronize()
    for _ in range(3):  # a process's first profile may come back empty
        with profile(activities=[ProfilerActivity.CUDA]) as prof:
            call()
            torch.cuda.synchronize()
        names = [e.name for e in prof.events() if e.device_type == torch.autograd.DeviceType.CUDA]
        if names:
            return " ".join(names)
    pytest.skip("no profiler on this machine")


@every_form
def test_forms_of_attend_as_the_device_sees_them(lsc, form):
    dtype, n, bt, D, G = FORMS[form]
    rng = np.random.default_rng(3)
    b = Batch(rng, [n, n], [n + 20, n + 33], bt, 2 * (n + 40) // bt + 4)
    host = filled4(rng, b, 2 * (n + 40) // bt + 4, bt, 2, D)
    q, _ = dense(rng.standard_normal((b.T, 2 * G, D)), dtype)
    with DevKv(host) as dev:
        names = kernels_of(lambda: run_attend(dev, 1, b, q, dtype, 2 * G, 0.1, True, max_seq_tokens=n))
    what = form.split("-")[0]
    want = {"decode": "decode4_attend_kernel", "chunk": "chunk_attend_kernel", "few": "chunk_attend_kernel",
            "expanded": "chunk_attend_kernel", "cuda": "attend_any_kernel"}[what]
    kinds = ("decode4_attend_kernel", "chunk_attend_kernel", "attend_any_kernel", "attend_rows_kernel")
    assert [k for k in kinds if k in names] == [want], names
    assert ("expand_kernel" in names) == (what == "expanded"), names


@pytest.mark.parametrize("dtype,D,stride,rotary_dim", [(BF, 64, 0, 32), (BF, 128, 0, 128), (F32, 256, 0, 64), (BF, 64, 131, 32),
                                                       (BF, 80, 0, 80), (BF, 48, 0, 16)], ids=str)
def test_row_kernels_as_the_device_sees_them(lsc, dtype, D, stride, rotary_dim):
    """Aligned rows of any head size take the E2M1 row kernels; a rotated append takes the vector kernel where groups of
    16 are pairs of its lanes."""
    rng = np.random.default_rng(4)
    H, bt = 2, 16
    w = stride or H * D
    b = Batch(rng, [5, 1], [5, 30], bt, 9)
    host = Host4(9, bt, H, D)
    k, _ = dense(rng.standard_normal((b.T, H, D)), dtype, w)
    out = torch.zeros_like(k)
    pos = torch.zeros(b.T, dtype=torch.int32, device="cuda")
    r = L.rotary(rotary_dim, pos, freqs(rotary_dim))
    aligned = w * (4 if dtype == F32 else 2) % 16 == 0
    with DevKv(host) as dev:
        append = L.kv_append_args(b.device(), k, k, dtype, stride, stride)
        calls = (("append", lambda: L.lsc_kv_append(dev.pool, 1, append, cur())),
                 ("gather", lambda: L.lsc_kv_gather(dev.pool, 1, L.kv_gather_args(append.batch, out, out, dtype, stride, stride), cur())),
                 ("rotated", lambda: L.lsc_kv_append_rotated(dev.pool, 1, L.kv_append_rotated_args(append, r), cur())))
        got = {name: kernels_of(f) for name, f in calls}
    assert ("append4_kernel" if aligned else "rows_any_kernel") in got["append"]
    assert ("gather4_kernel" if aligned else "rows_any_kernel") in got["gather"]
    vec = aligned and D % 32 == 0 and rotary_dim % 32 == 0
    assert ("rotary_kernel" in got["rotated"], "rotary_any_kernel" in got["rotated"]) == (vec, not vec), got["rotated"]


@pytest.mark.parametrize("n,D,G", [(1, 128, 4), (2, 256, 8), (20, 128, 4), (300, 128, 4), (100, 256, 8)], ids=str)
def test_layers_behind_one_another_share_a_workspace(lsc, n, D, G):
    """A step of twelve layers, rotated append, attend and the rows read back of each, with one workspace and the next
    layer's q made from this one's result: enqueued without a pause the bits are those of waiting after every call."""
    rng = np.random.default_rng(n + D)
    H, bt, layers, S, R = 2, 64, 12, 3, 32
    kv = [n + 400, n, n + 900]
    blocks = sum(-(-x // bt) for x in kv)
    b = Batch(rng, [n] * S, kv, bt, blocks)
    host = Host4(blocks, bt, H, D, layers=layers, fill=0)
    for i in range(S):
        bl, row = b.places(i, 0, kv[i])
        x = rng.standard_normal((len(bl), H, D))
        for layer in range(layers):
            for lane in (0, 1):
                host.write(layer, lane, bl, row, np.roll(x, layer + 7 * lane, 0))
    (first, _), (k, _), (v, _) = (dense(rng.standard_normal((b.T, h, D)), BF) for h in (H * G, H, H))
    pos = torch.arange(b.T, dtype=torch.int32, device="cuda").expand(3, b.T)
    r = L.rotary(R, pos, freqs(R), pair_axis=np.arange(R // 2) % 3)
    results, batch = [], b.device()
    with DevKv(host) as dev:
        for wait in (True, False, False):
            dev.buf.copy_(torch.from_numpy(host.bytes.reshape(-1)))
            q, out, ws, seen = first.clone(), torch.empty_like(first), None, []
            backs = [[torch.empty_like(k) for _ in "kv"] for _ in range(layers)]
            for layer in range(layers):
                append = L.kv_append_args(batch, k, v, BF)
                steps = [lambda: L.lsc_kv_append_rotated(dev.pool, layer, L.kv_append_rotated_args(append, r, H * G, q, q), cur())]
                a = L.kv_attend_args(batch, H * G, q, out, BF, D ** -0.5, max_seq_tokens=n, max_kv_tokens=max(kv))
                if ws is None:
                    rc, need = L.lsc_kv_attend_workspace_bytes(dev.pool, a)
                    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
                a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel()
                steps.append(lambda: L.lsc_kv_attend(dev.pool, layer, a, cur()))
                steps.append(lambda: L.lsc_kv_gather(dev.pool, layer, L.kv_gather_args(batch, *backs[layer], BF), cur()))
                for step in steps:
                    assert step() == L.LSC_OK
                    if wait:
                        torch.cuda.synchronize()
                q.copy_(out)
                seen.append(out.clone())
            results.append((seen, backs, dev.download()))
            assert dev.status() == L.LSC_OK
    for seen, backs, held in results[1:]:
        for layer in range(layers):
            assert torch.isfinite(seen[layer]).all()
            assert torch.equal(seen[layer], results[0][0][layer]), layer
            assert all(torch.equal(x, y) for x, y in zip(backs[layer], results[0][1][layer]))
        np.testing.assert_array_equal(held, results[0][2])
