"""E2M1 pools for the K/V step's tests: the plain 64-bit quantiser and a host pool to hold results against (the pool,
batch and attention forms of _kv.py take it as they take the others)."""
import numpy as np

from linear_attention_state_lsc_gb300 import lsc as L

from _kv import HostKv

MAG = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
VALUE = np.concatenate([MAG, -MAG])  # of the 16 codes
_b = np.arange(227)
LADDER = np.where(_b < 8, _b * 2.0 ** -17, (8 + _b % 8) * 2.0 ** (_b // 8 - 18.0))  # of the scale bytes that append writes


def quantise4(x):
    """float64 rows [..., D] -> (codes [..., D] one a byte, scale bytes [..., D / 16]): the smallest scale with six times
    it at least the group's largest magnitude, codes to nearest with ties to the even code."""
    x = np.asarray(x, np.float64)
    x = x.reshape(*x.shape[:-1], -1, 16)
    top = np.abs(x).max(-1)
    bad = ~np.isfinite(top)
    byte = np.minimum(np.searchsorted(6 * LADDER, np.where(bad, 0, top)), 226)
    zero = (byte == 0) | bad
    s = np.where(zero, 1.0, LADDER[byte])[..., None]
    a = np.abs(np.where(bad[..., None], 0, x))
    # between codes c and c + 1 the sum of both over two is the tie (times the scale: 7 bits, exact)
    code = np.zeros(a.shape, np.int64)
    for c in range(7):
        tie = (MAG[c] + MAG[c + 1]) / 2 * s
        code += (a > tie) | ((a == tie) & (c % 2 == 1))
    code = np.where(zero[..., None], 0, code + 8 * np.signbit(x))
    return code.reshape(*code.shape[:-2], -1).astype(np.uint8), np.where(bad, 255, byte).astype(np.uint8)


def value4(code, byte):
    """Codes one a byte and their scale bytes -> float64; 255 is NaN."""
    s = np.where(byte == 255, np.nan, LADDER[np.minimum(byte, 226)])
    return (VALUE[code].reshape(*code.shape[:-1], -1, 16) * s[..., None]).reshape(code.shape)


def halves(code):
    """Codes one a byte -> two a byte, the first in the low nibble."""
    return code[..., 0::2] | code[..., 1::2] << 4


class Host4(HostKv):
    """An E2M1 pool's description and its bytes on the host.  A fresh pool's bytes are 0xFF: codes of -6, scales of NaN."""

    def __init__(self, blocks, bt, heads, hd, pad=32, layers=2, fill=0xFF, dtype=L.LSC_E2M1):
        assert dtype == L.LSC_E2M1
        self.blocks, self.bt, self.H, self.D, self.dtype, self.layers = blocks, bt, heads, hd, dtype, layers
        self.codes = bt * heads * hd // 2
        self.scale_off = (self.codes + 15) // 16 * 16
        self.payload = self.scale_off + bt * heads * hd // 16
        self.page = (self.payload + 15) // 16 * 16 + pad
        self.desc = L.lsc_kv_pool_desc(layers, blocks, bt, heads, hd, dtype, self.page)
        self.bytes = np.full((layers, 2, blocks, self.page), fill, np.uint8)

    def scales(self, layer, lane):
        at = self.scale_off
        return self.bytes[layer, lane, :, at:at + self.bt * self.H * self.D // 16].reshape(self.blocks, self.bt, self.H, -1)

    def write(self, layer, lane, block, row, x):
        if len(block) == 0:
            return
        code, byte = quantise4(x)
        self.rows(layer, lane)[block, row] = halves(code)
        self.scales(layer, lane)[block, row] = byte

    def read(self, layer, lane, block, row):
        if len(block) == 0:
            return np.zeros((0, self.H, self.D))
        raw = self.rows(layer, lane)[block, row]
        return value4(np.stack([raw & 15, raw >> 4], -1).reshape(*raw.shape[:-1], -1), self.scales(layer, lane)[block, row])
