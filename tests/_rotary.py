"""Plain 64-bit form of rotary positions."""
import numpy as np


def turn(x, rotary_dim, angle, interleaved, scale=1.0):
    """float64 rows [T, heads, D] turned by angle [T, rotary_dim / 2]; and the sum of the two products' magnitudes."""
    half = rotary_dim // 2
    c, s = scale * np.cos(angle)[:, None], scale * np.sin(angle)[:, None]
    one, two = ((slice(0, rotary_dim, 2), slice(1, rotary_dim, 2)) if interleaved else
                (slice(0, half), slice(half, rotary_dim)))
    out, size = x.copy(), np.abs(x)
    out[..., one], out[..., two] = x[..., one] * c - x[..., two] * s, x[..., two] * c + x[..., one] * s
    size[..., one] = size[..., two] = abs(scale) * (np.abs(x[..., one]) + np.abs(x[..., two]))
    return out, size


def angles(positions, inv_freq, pair_axis):
    """[T, pairs] of float64; positions [axes, T]."""
    axis = np.zeros(len(inv_freq), int) if pair_axis is None else np.asarray(pair_axis)
    return positions[axis].T.astype(np.float64) * np.asarray(inv_freq)
