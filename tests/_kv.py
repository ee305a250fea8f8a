"""Plain 64-bit forms of the K/V step calls (append, gather, attend) and a pool
with host bytes to hold them against.  Every byte of a fresh pool is 0xFF (NaN in
each float type, NaN scale bytes), so that a row nobody wrote shows when read."""
import numpy as np
import torch

from linear_attention_state_lsc_gb300 import lsc as L

ES = {L.LSC_F32: 4, L.LSC_BF16: 2, L.LSC_F16: 2, L.LSC_E4M3: 1}
TORCH = {L.LSC_F32: torch.float32, L.LSC_BF16: torch.bfloat16, L.LSC_F16: torch.float16}
NAME = {L.LSC_F32: "f32", L.LSC_BF16: "bf16", L.LSC_F16: "f16", L.LSC_E4M3: "e4m3"}

# the values of the 256 e4m3 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits; no infinity
_c = np.arange(256)
_e, _m = (_c >> 3) & 15, _c & 7
E4M3 = np.where(_e == 0, _m * 2.0 ** -9, (8 + _m) * 2.0 ** (_e - 10.0)) * np.where(_c & 128, -1.0, 1.0)
E4M3[[127, 255]] = np.nan
_POS = E4M3[:127]


def quantise(x):
    """float64 rows [..., D] -> (codes, scale bytes): the smallest power of two in [2^-127, 2^127] that brings the
    row's largest magnitude to 448 or less, codes to nearest with ties to the even code."""
    x = np.asarray(x, np.float64)
    top = np.abs(x).max(-1)
    bad = ~np.isfinite(top)
    m, e = np.frexp(np.where(bad, 1.0, top))          # top = m 2^e, m in [0.5, 1)
    p = np.where(top == 0, -127, np.clip(e - 9 + (m > 0.875), -127, 127))
    y = np.where(bad[..., None], 0.0, x) * (2.0 ** -p.astype(np.float64))[..., None]
    a = np.abs(y)
    hi = np.clip(np.searchsorted(_POS, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    code = (code | np.where(np.signbit(y), 128, 0)).astype(np.uint8)
    code[bad] = 127
    return code, np.where(bad, 255, p + 127).astype(np.uint8)


def to_bytes(x, dtype):
    """float64 -> values of a 16- or 32-bit type, as raw bytes on a new last axis."""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(torch.float32).to(TORCH[dtype]).contiguous()
    return t.view(torch.uint8).numpy().reshape(*x.shape[:-1], -1)


class HostKv:
    """A pool's description and its bytes on the host."""

    def __init__(self, blocks, bt, heads, hd, dtype, pad=32, layers=2, fill=0xFF):
        self.blocks, self.bt, self.H, self.D, self.dtype, self.layers = blocks, bt, heads, hd, dtype, layers
        self.codes = bt * heads * hd * ES[dtype]
        self.scale_off = (self.codes + 15) // 16 * 16
        self.payload = self.scale_off + bt * heads if dtype == L.LSC_E4M3 else self.codes
        self.page = (self.payload + 15) // 16 * 16 + pad
        self.desc = L.lsc_kv_pool_desc(layers, blocks, bt, heads, hd, dtype, self.page)
        self.bytes = np.full((layers, 2, blocks, self.page), fill, np.uint8)

    def rows(self, layer, lane):
        return self.bytes[layer, lane, :, :self.codes].reshape(self.blocks, self.bt, self.H, -1)

    def scales(self, layer, lane):
        at = self.scale_off
        return self.bytes[layer, lane, :, at:at + self.bt * self.H].reshape(self.blocks, self.bt, self.H)

    def write(self, layer, lane, block, row, x):
        """float64 rows [n, H, D] into (block, row) places."""
        b = self.bytes[layer, lane]
        for (bl, r, v) in zip(block, row, x):
            if self.dtype == L.LSC_E4M3:
                code, up = quantise(v)
                b[bl, r * self.H * self.D:(r + 1) * self.H * self.D] = code.reshape(-1)
                b[bl, self.scale_off + r * self.H:self.scale_off + (r + 1) * self.H] = up
            else:
                w = self.H * self.D * ES[self.dtype]
                b[bl, r * w:(r + 1) * w] = to_bytes(v, self.dtype).reshape(-1)

    def read(self, layer, lane, block, row):
        """Values at (block, row) places: float64 [n, H, D]."""
        if len(block) == 0:
            return np.zeros((0, self.H, self.D))
        raw = np.ascontiguousarray(self.rows(layer, lane)[block, row])
        if self.dtype == L.LSC_E4M3:
            up = self.scales(layer, lane)[block, row].astype(np.float64)
            return E4M3[raw] * np.where(up == 255, np.nan, 2.0 ** (up - 127))[..., None]
        return torch.from_numpy(raw).view(TORCH[self.dtype]).double().numpy()


class DevKv:
    """The same pool on the GPU."""

    def __init__(self, host):
        self.host = host
        self.buf = torch.from_numpy(host.bytes.reshape(-1).copy()).cuda()
        rc, self.pool = L.lsc_kv_pool_create(host.desc, self.buf, self.buf.numel())
        assert rc == L.LSC_OK, L.lsc_error_string(rc)

    def download(self):
        torch.cuda.synchronize()
        return self.buf.cpu().numpy().reshape(self.host.bytes.shape)

    def status(self):
        return L.lsc_kv_pool_status(self.pool, torch.cuda.current_stream())

    def __enter__(self):
        return self

    def __exit__(self, *a):
        assert L.lsc_kv_pool_destroy(self.pool) == L.LSC_OK


class Batch:
    """New and cached tokens of each sequence on random blocks.  spare: rows of the dense arrays behind the last
    sequence."""

    def __init__(self, rng, n, kv, bt, blocks, spare=0, wide=0):
        self.n, self.kv, self.bt = np.asarray(n, np.int64), np.asarray(kv, np.int64), bt
        self.cu = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)
        self.T = int(self.cu[-1]) + spare
        per = -(-self.kv // bt)
        assert per.sum() <= blocks
        self.table = np.full((len(self.n), int(per.max(initial=0)) + wide), -7, np.int32)
        order, at = rng.permutation(blocks).astype(np.int32), 0
        for i, k in enumerate(per):
            self.table[i, :k] = order[at:at + k]
            at += k

    def places(self, i, lo, hi):
        p = np.arange(lo, hi)
        return self.table[i, p // self.bt], p % self.bt

    def device(self):
        self.dev = [torch.from_numpy(np.ascontiguousarray(a)).cuda()
                    for a in (self.table, self.cu, self.kv.astype(np.int32))]
        return L.kv_batch(len(self.n), self.T, *self.dev, max_blocks=self.table.shape[1])


def attend(host, layer, batch, q, scale, causal):
    """float64: out [T, Hq, D], lse [T, Hq], the sum of weight times |v| [T, Hq, D], the largest sum of |q k| times
    scale of a row's scores [T, Hq] and the largest |v| of a row; rows without a visible position: 0 and -inf."""
    T, Hq, D = q.shape
    G = Hq // host.H
    out, mass, lse = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    reach, vmax = np.zeros((T, Hq)), np.zeros((T, Hq))
    for i in range(len(batch.n)):
        kv, n = int(batch.kv[i]), int(batch.n[i])
        bl, r = batch.places(i, 0, kv)
        k, v = host.read(layer, 0, bl, r), host.read(layer, 1, bl, r)
        for j in range(n):
            t = int(batch.cu[i]) + j
            vis = min(kv, max(0, kv - n + j + 1)) if causal else kv
            if vis == 0:
                continue
            for h in range(Hq):
                kk, vv = k[:vis, h // G], v[:vis, h // G]
                s = kk @ q[t, h] * scale
                w = np.exp(s - s.max())
                lse[t, h] = s.max() + np.log(w.sum())
                w /= w.sum()
                out[t, h], mass[t, h] = w @ vv, w @ np.abs(vv)
                reach[t, h] = (np.abs(kk) @ np.abs(q[t, h])).max() * scale
                vmax[t, h] = np.abs(vv).max()
    return out, lse, mass, reach, vmax
