"""Plain 64-bit references of the 4-bit latent cache, on the CPU."""
import numpy as np
import torch

ENTRY = 400
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
VALUES = np.concatenate([GRID, -GRID])


def bf16(x):
    with np.errstate(over="ignore"):
        return torch.as_tensor(np.asarray(x, dtype=np.float32)).bfloat16()


def quantise(x):
    """Codes [.., 512] (0 .. 15) and exponent bytes [.., 16] of latents [.., 512] (finite unless a group says otherwise)."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(*x.shape[:-1], 16, 32)
    bad = ~np.isfinite(g).all(-1)
    y = np.where(bad[..., None], 0.0, g)
    amax = np.abs(y).max(-1)
    k = np.full(amax.shape, -1000)
    nz = amax >= 2.0 ** -126          # smaller ones end at -126 in any case
    m, ex = np.frexp(np.where(nz, amax, 1.0))
    k[nz] = np.where(m <= 0.75, ex - 3, ex - 2)[nz]
    k = np.maximum(np.maximum(k, k.max(-1, keepdims=True) - 14), -126)
    a = np.abs(y) / 2.0 ** k[..., None]
    up = np.searchsorted(GRID, a)                       # GRID[up - 1] < a <= GRID[up]
    up = np.minimum(up, 7)
    lo = np.maximum(up - 1, 0)
    dl, dh = a - GRID[lo], GRID[up] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, up)
    code = np.where(a == 0, 0, code)
    code = np.where(bad[..., None], 0, code | (np.signbit(y).astype(np.int64) << 3))
    return code.reshape(x.shape), np.where(bad, 255, k + 127)


def records(lat, rope):
    """uint8 [.., 400] of latents [.., 512] and rope values [.., 64] (bf16 tensor)."""
    code, ex = quantise(lat)
    packed = (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)
    r = rope.contiguous().view(torch.uint8).numpy()
    return np.concatenate([packed, ex.astype(np.uint8), r], -1)


def values(rec):
    """Latents [.., 512] and rope [.., 64] in 64 bits."""
    rec = np.asarray(rec)
    b = rec[..., :256].astype(np.int64)
    code = np.stack([b & 15, b >> 4], -1).reshape(*rec.shape[:-1], 512)
    ex = rec[..., 256:272].astype(np.int64)
    sc = np.where(ex == 255, np.nan, 2.0 ** (ex - 127.0))
    pair = rec[..., 272:400].astype(np.uint32)
    rope = ((pair[..., 0::2] | (pair[..., 1::2] << 8)) << 16).view(np.float32).astype(np.float64)
    return VALUES[code] * np.repeat(sc, 32, -1), rope


def attend(q, lat, rope, scale, eps=0.0):
    """Row [H, 576] over keys: out [H, 512], lse [H], and the bounds of an output's and an lse's error.

    The kernel's weights carry two E4M3 terms: half a step of the second is 2^-4 of the first's rest, 2^-8 of the weight,
    and 2^-14 of the unit where they end; the largest weight of a column, in the same units, is at least 2^1.  The
    key's power of two joins the weight, so that in values the floor is 2^-15 max|code| 2^(K_max' - 6) a key, at most
    2^-15 times 384 / 256 of the largest value of the key with the largest weight times scale.  The output is
    rounded to bf16 (2^-8).  Logits are sums of 576 exact products in fp32; the query's second term ends 2^-23 below the
    row's largest value.  eps: relative error of the scale, where fp32 does not hold it whole."""
    if lat.shape[0] == 0:
        z = np.zeros((q.shape[0], 512))
        return z, np.full(q.shape[0], -np.inf), z, np.zeros(q.shape[0])
    x = (q[:, :512] @ lat.T + q[:, 512:] @ rope.T) * scale
    m = x.max(-1, keepdims=True)
    lse = np.log(np.exp(x - m).sum(-1)) + m[:, 0]
    p = np.exp(x - lse[:, None])
    out = p @ lat
    mag = np.abs(q[:, :512]) @ np.abs(lat).T + np.abs(q[:, 512:]) @ np.abs(rope).T
    dx = abs(scale) * ((576 * 2.0 ** -24) * mag + 2.0 ** -22 * np.abs(q[:, :512]).max(-1, keepdims=True) * np.abs(lat).sum(-1)) + 2.0 ** -20 * (1 + np.abs(x)) + eps * np.abs(x)
    top = np.abs(lat).max(-1)                          # largest value of a key: at least 3 * 2^K
    w = p * top                                        # weights with the key's power of two, up to a factor of two
    floor = 2.0 ** -14 * w.max(-1, keepdims=True) * lat.shape[0] * 2
    tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + dx.max(-1, keepdims=True)) * (p @ np.abs(lat)) + floor + 1e-30
    return out, lse, tol, dx.max(-1) + 1e-6


def keys_of(cache, table, n, bs):
    """Records of one request's first n positions, in order: [n, 400]."""
    pos = np.arange(n)
    return cache[table[pos // bs], pos % bs]


def decode(q, cache, table, lens, bs, q_len, scale, eps=0.0):
    """q [B * q_len, H, 576]; returns out, lse, and their bounds, each stacked over the rows."""
    rows = []
    for b, L in enumerate(lens):
        for i in range(q_len):
            n = max(0, L - q_len + 1 + i)
            lat, rope = values(keys_of(cache, table[b], n, bs))
            rows.append(attend(q[b * q_len + i], lat, rope, scale, eps))
    return [np.stack(z) for z in zip(*rows)]
