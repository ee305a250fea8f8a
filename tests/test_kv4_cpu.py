"""E2M1 pools without a GPU: their layout, what is refused, and the tests' plain quantiser against the definition."""
import numpy as np
import torch

from linear_attention_state_lsc_gb300 import lsc as L

from _kv4 import LADDER, MAG, quantise4, value4
from test_kv_step_cpu import DEV, FAKE_BASE, batch, pool_of


def test_layout(lsc):
    d = L.lsc_kv_pool_desc(2, 8, 5, 3, 48, L.LSC_E2M1, 416)  # 360 bytes of codes, scales at 368, 45 of them
    pool = L.lsc_kv_pool_create(d, FAKE_BASE, 1 << 44)[1]
    rc, v = L.lsc_kv_pool_layer_view(pool, 1)
    assert rc == L.LSC_OK
    assert (v.scale_offset, v.payload_bytes, v.row_bytes, v.dtype) == (368, 413, 72, L.LSC_E2M1)
    assert list(v.strides) == [832, 144, 48, 1] and v.lane_stride == 8 * 832 and v.region_bytes == 2 * 8 * 416
    assert v.v - v.k == 8 * 416
    L.lsc_kv_pool_destroy(pool)
    assert L.lsc_kv_pool_required_bytes(d) == 2 * 2 * 8 * 416


def test_refusals(lsc):
    def made(**k):
        a = {**dict(layers=1, blocks=4, bt=16, heads=2, hd=64, page=1 << 16), **k}
        d = L.lsc_kv_pool_desc(a["layers"], a["blocks"], a["bt"], a["heads"], a["hd"], L.LSC_E2M1, a["page"])
        rc, pool = L.lsc_kv_pool_create(d, FAKE_BASE, 1 << 50)
        if rc == L.LSC_OK:
            L.lsc_kv_pool_destroy(pool)
        return rc
    assert made() == L.LSC_OK
    for hd in (8, 24, 33, 65, 100):
        assert made(hd=hd) == L.LSC_ERR_LAYOUT
    assert made(page=16 * 2 * 36) == L.LSC_OK           # codes and scales just fit
    assert made(page=16 * 2 * 36 - 16) == L.LSC_ERR_LAYOUT
    assert made(page=(1 << 16) + 8) == L.LSC_ERR_MISALIGNED
    assert made(bt=1 << 21, heads=64, hd=64, page=1 << 40) == L.LSC_ERR_LAYOUT       # a block of more than 2 GiB
    assert made(bt=1 << 20, heads=56, hd=64, page=1 << 40, blocks=1) == L.LSC_OK     # 2016 MiB of both
    assert made(bt=1 << 20, heads=60, hd=64, page=1 << 40, blocks=1) == L.LSC_ERR_LAYOUT  # the codes fit, the scales do not
    d = L.make_pool_desc([L.LSC_LAYER_GDN], 4, 16, 4, L.LSC_BF16, 1, 16, 16, L.LSC_E2M1, 4096)
    assert L.lsc_pool_create(d, FAKE_BASE, 1 << 30)[0] == L.LSC_ERR_INVALID_ARG  # no state type
    pool = pool_of()
    for call, args in ((L.lsc_kv_append, L.kv_append_args(batch(), DEV, DEV, L.LSC_E2M1)),  # nor a dense one
                       (L.lsc_kv_gather, L.kv_gather_args(batch(), DEV, DEV, L.LSC_E2M1)),
                       (L.lsc_kv_attend, L.kv_attend_args(batch(), 2, DEV, DEV, L.LSC_E2M1, 0.1))):
        assert call(pool, 0, args) == L.LSC_ERR_INVALID_ARG
    L.lsc_kv_pool_destroy(pool)


def test_plain_quantiser():
    """Scales are f16 values; no smaller scale would do; every code is a nearest one; stored values come back as they
    are."""
    f16 = (torch.arange(227, dtype=torch.int16) << 7).view(torch.float16).double().numpy()
    np.testing.assert_array_equal(LADDER, f16)
    rng = np.random.default_rng(0)
    x = np.float64(np.float32(rng.standard_normal((300, 64)) * np.exp(4 * rng.standard_normal((300, 1)))))
    code, byte = quantise4(x)
    top = np.abs(x.reshape(300, 4, 16)).max(-1)
    held = np.minimum(top, 6 * LADDER[226])  # larger magnitudes become the largest one
    assert (6 * LADDER[byte] >= held).all() and (6 * LADDER[byte - 1] < held)[byte > 0].all() and (top[byte == 0] == 0).all()
    y = value4(code, byte)
    s = LADDER[byte].repeat(16, -1)
    best = np.abs(x[..., None] - np.concatenate([MAG, -MAG]) * s[..., None]).min(-1)
    np.testing.assert_array_equal(np.abs(x - y), best)
    full = ((byte >= 8) & (top <= held)).repeat(16, -1)  # scales with all their bits
    assert (best <= top.repeat(16, -1) * 3 / 16)[full].all() and full.any()
    np.testing.assert_array_equal(value4(*quantise4(y))[full], y[full])


def test_rows_near_two_to_the_31_elements(lsc):
    """The row kernels round a row up to whole stretches of 1024 elements and count them in 32 bits."""
    for short, want in ((1024, L.LSC_OK), (1008, L.LSC_ERR_LAYOUT), (512, L.LSC_ERR_LAYOUT), (16, L.LSC_ERR_LAYOUT)):
        d = L.lsc_kv_pool_desc(1, 2, 1, (2 ** 31 - short) // 16, 16, L.LSC_E2M1, 1 << 31)
        rc, pool = L.lsc_kv_pool_create(d, FAKE_BASE, 1 << 50)
        assert rc == want
        if rc == L.LSC_OK:
            L.lsc_kv_pool_destroy(pool)
