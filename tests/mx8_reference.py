"""8-bit matrices in 64 bits, from the format's definition."""
import numpy as np

MOST = 448.0   # of e4m3


def scale_bytes(w):
    """Bytes [.., N, ceil(K/32)] of w [.., N, K]: the smallest power of two with |w| <= 448 scale, at least 2^-126."""
    w = np.asarray(w, np.float64)
    K = w.shape[-1]
    p = np.concatenate([w, np.zeros((*w.shape[:-1], -K % 32))], -1)
    big = np.abs(p.reshape(*w.shape[:-1], -1, 32)).max(-1)
    m, e = np.frexp(np.where(np.isfinite(big), big, 1))     # m 2^e, m in [.5, 1); 448 = .875 2^9
    e = np.maximum(e - 9 + (m > 0.875), -126)
    return np.where(~np.isfinite(big), 255, np.where(big == 0, 127, e + 127)).astype(np.int64)


def spread(groups, K):
    return np.repeat(groups, 32, -1)[..., :K]


def two(byte):
    return np.where(byte == 255, np.nan, 2.0 ** (np.asarray(byte, np.float64) - 127))


def half_step(r):
    """Half the distance between the e4m3 numbers around |r| <= 448."""
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(r), 2.0 ** -6))) - 4)


def values(w):
    """What w [.., N, K] becomes in 8 bits."""
    w = np.asarray(w, np.float64)
    s = two(spread(scale_bytes(w), w.shape[-1]))
    with np.errstate(all="ignore"):
        r = w / s
        step = 2 * half_step(r)
        return np.round(r / step) * step * s   # numpy rounds ties to even


def pack_scale(groups, K):
    """Bytes [.., N, ceil(K/32)] in the layout [.., ceil(K/128), N, 4], padding 127."""
    pad = -groups.shape[-1] % 4
    g = np.concatenate([groups, np.full((*groups.shape[:-1], pad), 127)], -1)
    return np.ascontiguousarray(np.swapaxes(g.reshape(*groups.shape[:-1], -1, 4), -3, -2), np.uint8)


def unpack_scale(scale, K):
    s = np.swapaxes(scale, -3, -2)
    return s.reshape(*s.shape[:-2], -1)[..., :-(-K // 32)].astype(np.int64)


def decode(byte):
    """e4m3 bytes as numbers."""
    b = np.asarray(byte).astype(np.int64)
    e, m = b >> 3 & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7))
    return np.where((b & 127) == 127, np.nan, np.where(b > 127, -v, v))
