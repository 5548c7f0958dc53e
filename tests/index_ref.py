"""Plain 64-bit forms of the selector's operators (index cache, scores, selection, selected pages)
for the tests: numpy on the host, from the definitions, row by row."""
import numpy as np

E4M3 = np.array([(-1.0) ** (c >> 7) * ((c & 7) / 8 * 2.0 ** -6 if (c >> 3) & 15 == 0 else
                                       np.nan if c & 127 == 127 else (1 + (c & 7) / 8) * 2.0 ** (((c >> 3) & 15) - 7))
                 for c in range(256)])


def bf16_to_f64(bits):
    return (np.asarray(bits, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def to_bf16_bits(x):
    """Round to nearest even of finite values."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def to_e4m3(x):
    """Nearest code, ties to the even one, saturating (|x| <= 448 here)."""
    x = np.asarray(x, dtype=np.float64)
    vals = E4M3[:127]
    a = np.abs(x)
    hi = np.clip(np.searchsorted(vals, a), 1, 126)
    lo = hi - 1
    dl, dh = a - vals[lo], vals[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a >= vals[126], 126, code)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def rotate(x, cs):
    """x [..., 128] fp64 holding bf16 values, cs [..., 64] fp32: fp32 results of the GPT-J rotation of
    the last 64 values, the product with the sine rounded to fp32 first."""
    y = x.astype(np.float32)
    if cs is None:
        return y
    c, s = cs[..., :32], cs[..., 32:]
    a, b = y[..., 64::2].copy(), y[..., 65::2].copy()
    y[..., 64::2] = (a.astype(np.float64) * c - (b * s).astype(np.float32).astype(np.float64)).astype(np.float32)
    y[..., 65::2] = (b.astype(np.float64) * c + (a * s).astype(np.float32).astype(np.float64)).astype(np.float32)
    return y


def pow2_scale(amax):
    k = np.zeros(amax.shape, dtype=np.int64)
    for i in np.ndindex(amax.shape):
        a = float(amax[i])
        if a > 0:
            kk = -126
            while 448.0 * 2.0 ** kk < a:
                kk += 1
            k[i] = kk
    return 2.0 ** k.astype(np.float64)


def quantise(y):
    s = pow2_scale(np.abs(y.astype(np.float64)).max(-1))
    return to_e4m3(y.astype(np.float64) / s[..., None]), s


def visible(seq_lens, cu_q, T):
    """(request, visible keys) of every row; request -1 for rows of none."""
    out = []
    for t in range(T):
        b = -1
        for r in range(len(seq_lens)):
            if cu_q[r] <= t < cu_q[r + 1]:
                b = r
        out.append((b, 0 if b < 0 else max(0, int(seq_lens[b]) - int(cu_q[b + 1] - cu_q[b]) + (t - int(cu_q[b])) + 1)))
    return out


def scores(q, w, keys, key_scale, table, seq_lens, cu_q, width, bt, num_blocks):
    """(scores, magnitudes): fp64 [T, width]; NaN marks columns that stay unwritten.  q [T, Hi, 128] and
    keys [num_blocks, page, 128] are values; the magnitude is the sum of absolute terms of the largest
    token of a block."""
    T, ps = q.shape[0], keys.shape[1]
    out, mag = np.full((T, width), np.nan), np.zeros((T, width))
    written = np.zeros((T, width), dtype=bool)
    for t, (b, vis) in enumerate(visible(seq_lens, cu_q, T)):
        vis = min(vis, width * bt)
        if b < 0 or vis == 0:
            continue
        s, m = np.empty(vis), np.empty(vis)
        for j0 in range(0, vis, ps):
            n = min(ps, vis - j0)
            blk = int(table[b, j0 // ps]) if j0 // ps < table.shape[1] else -1
            if not 0 <= blk < num_blocks:
                s[j0:j0 + n], m[j0:j0 + n] = -np.inf, 0
                continue
            k, ks = keys[blk, :n], key_scale[blk, :n]
            with np.errstate(invalid="ignore"):
                dot = q[t] @ k.T
                s[j0:j0 + n] = (w[t][:, None] * np.where(np.isnan(dot), np.nan, np.maximum(dot, 0))).sum(0) * ks
                m[j0:j0 + n] = (np.abs(w[t])[:, None] * (np.abs(q[t]) @ np.abs(k.T))).sum(0) * ks
        for c in range(-(-vis // bt)):
            part = s[c * bt:min(vis, (c + 1) * bt)]
            out[t, c] = np.nan if np.isnan(part).any() else part.max()
            mag[t, c] = m[c * bt:min(vis, (c + 1) * bt)].max()
            written[t, c] = True
    return out, mag, written


def select(scores_, seq_lens, cu_q, bt, k, first, last, table=None, page=0, num_blocks=0):
    T, W = scores_.shape
    blocks = np.full((T, k), -1, dtype=np.int64)
    slots = np.full((T, k * bt), -1, dtype=np.int64)
    rows = visible(seq_lens, cu_q, T)
    for t, (b, vis) in enumerate(rows):
        n = min(-(-vis // bt), W)
        order = []
        for c in range(n):
            if c < first or c >= n - last:
                order.append((0, 0.0, c))
            elif scores_[t, c] > -np.inf:
                order.append((1, -float(scores_[t, c]), c))
        got = sorted(c for _, _, c in sorted(order)[:k])
        blocks[t, :len(got)] = got
        if table is not None and b >= 0:
            for j, c in enumerate(got):
                for u in range(bt):
                    pos = c * bt + u
                    if pos < vis and pos // page < table.shape[1] and 0 <= table[b, pos // page] < num_blocks:
                        slots[t, j * bt + u] = table[b, pos // page] * page + pos % page
    return blocks, slots, [b for b, _ in rows]


def attend(q, entries, scale):
    """Softmax attention of q [H, 576] over entries [n, 576]: (out [H, 512], lse [H])."""
    if len(entries) == 0:
        return np.zeros((q.shape[0], 512)), np.full(q.shape[0], -np.inf)
    x = q @ entries.T * scale
    m = x.max(1, keepdims=True)
    p = np.exp(x - m)
    l = p.sum(1, keepdims=True)
    return p @ entries[:, :512] / l, (m + np.log(l))[:, 0]
