"""What append, gather and attend refuse before any device work, and the E4M3
pool's layout, through the C ABI on host-only pools (a borrowed base that is
never dereferenced); and the plain quantiser of the GPU tests against torch's
cast.  Only refused calls are made where a GPU is visible."""
import ctypes

import numpy as np
import pytest
import torch

from linear_attention_state_lsc_gb300 import lsc as L

import _kv
from _util import gpu_present

FAKE_BASE = 1 << 40
DEV = 1 << 41  # a stand-in device address


def pool_of(dtype=L.LSC_BF16, bt=16, heads=2, hd=64, page=1 << 16, layers=2):
    rc, pool = L.lsc_kv_pool_create(L.lsc_kv_pool_desc(layers, 8, bt, heads, hd, dtype, page), FAKE_BASE, 1 << 44)
    assert rc == L.LSC_OK
    return pool


def batch(n_seq=2, total=5, max_blocks=4, table=DEV, cu=DEV, kv=DEV):
    return L.kv_batch(n_seq, total, table, cu, kv, max_blocks)


def test_e4m3_pool_layout(lsc):
    d = L.lsc_kv_pool_desc(2, 8, 5, 3, 7, L.LSC_E4M3, 160)  # 105 codes, scales at 112, 15 of them
    pool = L.lsc_kv_pool_create(d, FAKE_BASE, 1 << 44)[1]
    rc, v = L.lsc_kv_pool_layer_view(pool, 1)
    assert rc == L.LSC_OK
    assert (v.scale_offset, v.payload_bytes, v.row_bytes) == (112, 127, 21)
    assert list(v.strides) == [160, 21, 7, 1] and v.region_bytes == 2 * 8 * 160
    L.lsc_kv_pool_destroy(pool)
    d.page_bytes = 112  # the codes fit, the scales do not
    assert L.lsc_kv_pool_create(d, FAKE_BASE, 1 << 44)[0] == L.LSC_ERR_LAYOUT
    for dt in (L.LSC_F32, L.LSC_BF16, L.LSC_F16):
        pool = pool_of(dt)
        assert L.lsc_kv_pool_layer_view(pool, 0)[1].scale_offset == 0
        L.lsc_kv_pool_destroy(pool)


def test_e4m3_is_no_state_type(lsc):
    d = L.make_pool_desc([L.LSC_LAYER_GDN], 4, 16, 4, L.LSC_BF16, 1, 16, 16, L.LSC_E4M3, 4096)
    assert L.lsc_pool_create(d, FAKE_BASE, 1 << 30)[0] == L.LSC_ERR_INVALID_ARG


BATCHES = [(batch(n_seq=-1), L.LSC_ERR_INVALID_ARG), (batch(total=-1), L.LSC_ERR_INVALID_ARG),
           (batch(max_blocks=-1), L.LSC_ERR_INVALID_ARG), (batch(table=None), L.LSC_ERR_INVALID_ARG),
           (batch(cu=None), L.LSC_ERR_INVALID_ARG), (batch(kv=None), L.LSC_ERR_INVALID_ARG),
           (batch(table=DEV + 2), L.LSC_ERR_MISALIGNED), (batch(cu=DEV + 1), L.LSC_ERR_MISALIGNED),
           (batch(kv=DEV + 2), L.LSC_ERR_MISALIGNED)]


@pytest.mark.parametrize("call,make", [(L.lsc_kv_append, L.kv_append_args), (L.lsc_kv_gather, L.kv_gather_args)],
                         ids=["append", "gather"])
def test_rows_refusals(lsc, call, make):
    pool = pool_of()
    ok = batch()
    cases = [(1, make(b, DEV, DEV, L.LSC_BF16), rc) for b, rc in BATCHES]
    for k, rc in [(dict(k=None), L.LSC_ERR_INVALID_ARG), (dict(v=None), L.LSC_ERR_INVALID_ARG),
                  (dict(dtype=L.LSC_E4M3), L.LSC_ERR_INVALID_ARG), (dict(dtype=9), L.LSC_ERR_INVALID_ARG),
                  (dict(k_stride=127), L.LSC_ERR_INVALID_ARG), (dict(v_stride=-1), L.LSC_ERR_INVALID_ARG),
                  (dict(k=DEV + 1), L.LSC_ERR_MISALIGNED), (dict(v=DEV + 2, dtype=L.LSC_F32), L.LSC_ERR_MISALIGNED)]:
        cases.append((1, make(ok, **{**dict(k=DEV, v=DEV, dtype=L.LSC_BF16), **k}), rc))
    cases += [(2, make(ok, DEV, DEV, L.LSC_BF16), L.LSC_ERR_OUT_OF_RANGE),
              (-1, make(ok, DEV, DEV, L.LSC_BF16), L.LSC_ERR_OUT_OF_RANGE)]
    for field in ("reserved", "batch.reserved"):
        a = make(ok, DEV, DEV, L.LSC_BF16)
        setattr(a.batch if "." in field else a, "reserved", 1)
        cases.append((0, a, L.LSC_ERR_INVALID_ARG))
    for layer, a, want in cases:
        assert call(pool, layer, a) == want
    assert call(None, 0, make(ok, DEV, DEV, L.LSC_BF16)) == L.LSC_ERR_INVALID_ARG
    if not gpu_present():  # a good call on a host-only pool has nothing to run on
        assert call(pool, 1, make(ok, DEV, DEV, L.LSC_BF16)) == L.LSC_ERR_CUDA
    L.lsc_kv_pool_destroy(pool)


def test_attend_refusals(lsc):
    pool = pool_of()
    base = dict(batch=batch(), num_q_heads=4, q=DEV, out=DEV, dtype=L.LSC_BF16, scale=0.125, lse=DEV)
    bad = [(dict(batch=b), rc) for b, rc in BATCHES]
    bad += [(k, L.LSC_ERR_INVALID_ARG) for k in
            (dict(num_q_heads=0), dict(num_q_heads=3), dict(num_q_heads=-2), dict(dtype=L.LSC_E4M3), dict(dtype=-1),
             dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3.4e38),
             dict(causal=2), dict(causal=-1), dict(max_seq_tokens=-1), dict(max_kv_tokens=-1), dict(q=None),
             dict(out=None), dict(q_stride=255), dict(out_stride=255), dict(q_stride=-256))]
    bad += [(k, L.LSC_ERR_MISALIGNED) for k in
            (dict(q=DEV + 1), dict(out=DEV + 1), dict(lse=DEV + 2), dict(workspace=DEV + 8, workspace_bytes=1 << 40))]
    for k, want in bad:
        a = L.kv_attend_args(**{**base, **k})
        assert L.lsc_kv_attend(pool, 1, a) == want, k
        assert L.lsc_kv_attend_workspace_bytes(pool, a)[0] == want, k
    assert L.lsc_kv_attend(pool, 2, L.kv_attend_args(**base)) == L.LSC_ERR_OUT_OF_RANGE
    assert L.lsc_kv_attend(None, 0, L.kv_attend_args(**base)) == L.LSC_ERR_INVALID_ARG
    if not gpu_present():
        assert L.lsc_kv_attend(pool, 1, L.kv_attend_args(**base)) == L.LSC_ERR_CUDA
    L.lsc_kv_pool_destroy(pool)
    pool = pool_of(hd=520)
    assert L.lsc_kv_attend(pool, 0, L.kv_attend_args(**base)) == L.LSC_ERR_UNSUPPORTED
    L.lsc_kv_pool_destroy(pool)


def test_status_needs_a_device_pool(lsc):
    if gpu_present():
        pytest.skip("a pool made here is a device pool")
    pool = pool_of()
    with pytest.raises(L.LscError):
        L.lsc_kv_pool_status(pool)
    n = ctypes.c_int32(5)
    assert L.load().lsc_kv_pool_status(None, None, ctypes.byref(n)) == L.LSC_ERR_INVALID_ARG
    L.lsc_kv_pool_destroy(pool)


def test_plain_quantiser_against_torch():
    """The GPU tests' own quantiser: each code is torch's cast of the scaled element, and no smaller power of two
    would do."""
    rng = np.random.default_rng(0)
    x = np.float64(np.float32(rng.standard_normal((500, 24)) * np.exp(8 * rng.standard_normal((500, 1)))))
    x[0] = 0
    code, up = _kv.quantise(x)
    y = x * 2.0 ** (127.0 - up)[:, None]
    want = torch.from_numpy(y).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(code, want)
    top = np.abs(y).max(-1)
    assert (top <= 448).all() and (top[1:] > 224).all() and up[0] == 0
    table = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(np.nan_to_num(table), np.nan_to_num(_kv.E4M3))
