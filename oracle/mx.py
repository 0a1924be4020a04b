"""Oracle of the MXFP4 calls and of dropout: plain numpy, fp64.

OCP Microscaling Formats v1.0: blocks of 32 elements along a row share an E8M0
scale 2^(b - 127); an element is an E2M1 code.  Dropout: Philox4x32-10
(Salmon et al., SC 2011), 16 bits an element.
"""

from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 32


def mx_quantize(x):
    """(codes uint8 [R, C], scale bytes uint8 [R, C / 32]) of x [R, C] (exact
    in fp64), one code a byte."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[0], -1, BLOCK)
    with np.errstate(invalid="ignore"):
        m = np.abs(b).max(axis=2)
    bad = ~np.isfinite(b).all(axis=2)
    m = np.where(bad, 1.0, m)
    e = np.where(m > 0, np.frexp(m)[1] - 1, -200)          # floor(log2 m)
    s = np.where(bad, 255, np.maximum(e - 2 + 127, 0)).astype(np.uint8)
    scale = np.ldexp(1.0, np.where(bad, 0, s.astype(int) - 127))[:, :, None]
    v = np.where(bad[:, :, None], 0.0, b) / scale
    a = np.abs(v)
    d = np.abs(a[..., None] - E2M1)
    best = d.min(axis=-1, keepdims=True)
    hit = d == best                                         # one level, or the two around a tie
    first = hit.argmax(axis=-1)
    last = 7 - hit[..., ::-1].argmax(axis=-1)
    code = np.where(first % 2 == 0, first, last)            # a tie goes to the even code
    code = code + 8 * np.signbit(v)
    return code.reshape(x.shape).astype(np.uint8), s


def mx_values(codes, s):
    """What (codes, scale bytes) stand for, fp64; a scale of 255 is NaN."""
    v = np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]
    scale = np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(int) - 127))
    return (v.reshape(s.shape + (BLOCK,)) * scale[:, :, None]).reshape(codes.shape)


def mx_pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).reshape(-1)


def mx_tile_scales(s):
    """Scale bytes [rows, blocks] in the tiled storage, byte by byte."""
    r, b = s.shape
    kt = -(-b // 4)
    out = np.zeros(-(-r // 128) * kt * 512, np.uint8)
    i, j = np.meshgrid(np.arange(r), np.arange(b), indexing="ij")
    out[((i // 128) * kt + j // 4) * 512 + (i % 32) * 16 + (i % 128) // 32 * 4 + j % 4] = s
    return out


def mx_rounded(x):
    return mx_values(*mx_quantize(x))


def philox4x32(ctr, key, rounds=10):
    """ctr: 4 uint64 arrays below 2^32, key: 2 ints; the 4 output words."""
    c = [np.asarray(v, np.uint64) for v in ctr]
    k = list(key)
    mask = np.uint64(0xFFFFFFFF)
    for _ in range(rounds):
        p0, p1 = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & mask,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p0 & mask]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def dropout_threshold(p):
    return int(np.rint(65536 * p))


def dropout_keep(n, p, seed, offset):
    """bool [n]: which elements are kept."""
    q = np.arange(-(-n // 8), dtype=np.uint64)
    lo = np.uint64(0xFFFFFFFF)
    one = np.ones_like(q)
    w = philox4x32([q & lo, q >> np.uint64(32), one * np.uint64(offset & 0xFFFFFFFF), one * np.uint64(offset >> 32)],
                   (seed & 0xFFFFFFFF, seed >> 32))
    halves = np.stack([h for x in w for h in (x & np.uint64(0xFFFF), x >> np.uint64(16))], 1).reshape(-1)[:n]
    return halves >= np.uint64(dropout_threshold(p))


def dropout_scale(p):
    return 65536.0 / (65536 - dropout_threshold(p))


def mx_linear_fwd(X, What, L1, L2, s, mask=None):
    """X, L1, L2 fp64; What the weight's values; mask = keep * scale or None."""
    T = (X if mask is None else X * mask) @ L1
    return mx_rounded(X) @ What.T + s * T @ L2, T


def mx_linear_bwd(dY, X, T, WTval, L1, L2, s, mask=None):
    """WTval [K, N]: the values of the weight's backward form."""
    dT = s * dY @ L2.T
    lora = dT @ L1.T
    Xm = X if mask is None else X * mask
    return mx_rounded(dY) @ WTval.T + (lora if mask is None else lora * mask), Xm.T @ dT, s * T.T @ dY
