"""Plain MXFP4 arithmetic in 64 bits (numpy), written from the format's definition: the reference
of the MXFP4 tests."""
import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def scale_bytes(x, rule):
    """E8M0 bytes [rows, cols / 32] of a float64 matrix. floor: floor(log2 m) - 2; ceil: the
    smallest s with m <= 6 * 2^s. frexp gives m = f * 2^e with 0.5 <= f < 1."""
    v = x.reshape(x.shape[0], -1, 32)
    bad = ~np.isfinite(v).all(-1)
    m = np.abs(np.where(np.isfinite(v), v, 0.0)).max(-1)
    if rule == "floor":
        s = np.frexp(m)[1] - 3
    else:
        f, e = np.frexp(m)  # m <= 6 * 2^s  <=>  f * 2^e <= 0.75 * 2^(s + 3)
        s = np.where(f <= 0.75, e - 3, e - 2)
    s = np.where(m > 0.0, np.maximum(s, -127), -127)
    return np.where(bad, 255, s + 127).astype(np.uint8)


def codes(x, sb):
    """E2M1 codes [rows, cols] of a float64 matrix with its scale bytes."""
    q = np.where(np.repeat(sb, 32, 1) == 255, 0.0,
                 x * np.exp2(127.0 - np.repeat(sb, 32, 1).astype(np.float64)))
    a = np.minimum(np.abs(q), 6.0)
    d = np.abs(a[..., None] - MAGNITUDES)
    best = d.min(-1, keepdims=True)
    n = np.zeros(a.shape, np.int64)
    for c in range(7, -1, -1):  # among the nearest: the even code of a tie
        near = d[..., c] == best[..., 0]
        n = np.where(near & ((c % 2 == 0) | (d == best).sum(-1).__eq__(1)), c, n)
    n = n + 8 * np.signbit(q)
    return np.where(np.repeat(sb, 32, 1) == 255, 0, n).astype(np.uint8)


def quantize(x, rule="floor"):
    """(packed codes [rows, cols / 2], scale bytes [rows, cols / 32]) of a matrix."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        sb = scale_bytes(x, rule)
        c = codes(x, sb)
    return c[:, 0::2] | (c[:, 1::2] << 4), sb


def values(packed, sb):
    """float64 values of packed codes with their scale bytes."""
    c = np.empty((packed.shape[0], packed.shape[1] * 2), np.int64)
    c[:, 0::2], c[:, 1::2] = packed & 15, packed >> 4
    v = np.where(c >= 8, -1.0, 1.0) * MAGNITUDES[c & 7]
    s = np.repeat(sb, 32, 1).astype(np.float64)
    return np.where(s == 255, np.nan, v * np.exp2(s - 127.0))


def swizzle(sb):
    """Scale bytes in the operand layout, byte by byte from its definition."""
    rows, nb = sb.shape
    atoms = (nb + 3) // 4
    out = np.zeros((rows + 127) // 128 * atoms * 512, np.uint8)
    for r in range(rows):
        for b in range(nb):
            out[((r // 128) * atoms + b // 4) * 512 + 16 * (r % 32) + 4 * ((r % 128) // 32)
                + b % 4] = sb[r, b]
    return out


def transposed(x):
    """x^T with its columns padded with zeros to whole blocks of 32."""
    return np.pad(np.asarray(x).T, ((0, 0), (0, -x.shape[0] % 32)))
