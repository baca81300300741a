"""The attention operators in 64 bits, element by element from the documented
formulas and the documented cache layout (include/qk.h); numpy only."""
import numpy as np


def places(D):
    """(key byte, key shift, value byte, value shift) [16][D] of a block and (key, value) scale bytes [16][G]."""
    G = D // 32
    Gp = 4 if G % 4 == 0 else G
    kb, ks, vb, vs = (np.zeros((16, D), np.int64) for _ in range(4))
    sk, sv = np.zeros((16, G), np.int64), np.zeros((16, G), np.int64)
    for a in range(4):
        for h in range(2):
            for b in range(2):
                t = 4 * a + 2 * h + b
                for ch in range(D):
                    g, i = divmod(ch, 32)
                    c, n = divmod(i, 8)
                    word = ((g // Gp * 16 + 8 * h + 2 * a + b) * 4 + c) * Gp + g % Gp
                    kb[t, ch], ks[t, ch] = 4 * word + n // 2, 4 * (n % 2)
                    # values: token 4c + 2u + b has c = a, u = h
                    r, j = divmod(i, 4)
                    word = ((g // Gp * 2 + h) * 8 + r) * 4 * Gp + a * Gp + g % Gp
                    n = 4 * b + j
                    vb[t, ch], vs[t, ch] = 8 * D + 4 * word + n // 2, 4 * (n % 2)
                for g in range(G):
                    sk[t, g] = 16 * D + 2 * (t * G + g)
                    sv[t, g] = 17 * D + 2 * (t * G + g)
    return kb, ks, vb, vs, sk, sv


def quantise(x):
    """x [..., D] -> (nibbles, fp16 scales [..., D/32]), from the definition in 64 bits."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    hi, lo = g.max(-1), g.min(-1)
    m = np.where(hi >= -lo, hi, lo)
    d = np.clip(m / -8, -65504, 65504).astype(np.float16)
    with np.errstate(divide="ignore", invalid="ignore"):
        n = np.clip(np.floor(g / d.astype(np.float64)[..., None] + 8.5), 0, 15)
    n = np.where(d[..., None] == 0, 8, n)
    return n.reshape(x.shape).astype(np.uint8), d


def pack(kn, kd, vn, vd):
    """Nibbles [..., page, D] and scales of keys and values -> [..., page/16, 18 D] bytes."""
    *lead, page, D = kn.shape
    kb, ks, vb, vs, sk, sv = places(D)
    out = np.zeros((int(np.prod(lead, dtype=np.int64)) * (page // 16), 18 * D), np.uint8)
    for n, byte, shift in ((kn, kb, ks), (vn, vb, vs)):
        n = n.reshape(-1, 16, D)
        for half in (0, 4):
            sel = shift == half
            out[:, byte[sel]] |= (n[:, sel] << half).astype(np.uint8)
    for d, at in ((kd, sk), (vd, sv)):
        b = np.ascontiguousarray(d.reshape(-1, 16, D // 32)).view(np.uint8).reshape(-1, 16, D // 32, 2)
        out[:, at] = b[..., 0]
        out[:, at + 1] = b[..., 1]
    return out.reshape(*lead, page // 16, 18 * D)


def unpack(blocks):
    """[..., 18 D] bytes -> keys, values [..., 16, D] in 64 bits."""
    *lead, size = blocks.shape
    D = size // 18
    kb, ks, vb, vs, sk, sv = places(D)
    b = blocks.reshape(-1, size)
    got = []
    for byte, shift, at in ((kb, ks, sk), (vb, vs, sv)):
        n = ((b[:, byte] >> shift) & 15).astype(np.float64) - 8
        d = (b[:, at].astype(np.uint16) | (b[:, at + 1].astype(np.uint16) << 8)).view(np.float16).astype(np.float64)
        with np.errstate(invalid="ignore"):
            got.append((n * np.repeat(d, 32, -1)).reshape(*lead, 16, D))
    return got


def norm_rope(x, weight, eps, table, positions, rot, interleaved):
    """x [T][heads][D] -> (result, sum of the magnitudes each result is made of), 64 bits."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    y, mag = x.copy(), np.abs(x)
    if rot:
        t = np.asarray(table, np.float64)[np.asarray(positions)]
        for i in range(rot // 2):
            p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            c, s = t[:, None, i, 0], t[:, None, i, 1]
            y[..., p] = x[..., p] * c - x[..., q] * s
            y[..., q] = x[..., p] * s + x[..., q] * c
            mag[..., p] = np.abs(x[..., p] * c) + np.abs(x[..., q] * s)
            mag[..., q] = np.abs(x[..., p] * s) + np.abs(x[..., q] * c)
    return y, mag


def attention(q, k, v, pos, scale, window):
    """One sequence: q [n][nq][D], k, v [L][nkv][D], pos [n] -> (out, A, S) with A [n][nq] the largest sum of the
    magnitudes of a score's terms and S [n][nq][D] the sum of p |v|."""
    n, nq, D = q.shape
    L, nkv = k.shape[:2]
    rep = nq // nkv
    out, S, A = np.zeros((n, nq, D)), np.zeros((n, nq, D)), np.zeros((n, nq))
    j = np.arange(L)
    for i in range(n):
        see = j <= pos[i]
        if window:
            see &= j > pos[i] - window
        if not see.any():
            continue
        for h in range(nq):
            kk, vv = k[see, h // rep], v[see, h // rep]
            s = scale * (kk @ q[i, h])
            A[i, h] = abs(scale) * (np.abs(kk) @ np.abs(q[i, h])).max()
            p = np.exp(s - s.max())
            p /= p.sum()
            out[i, h] = p @ vv
            S[i, h] = p @ np.abs(vv)
    return out, A, S
