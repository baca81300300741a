"""The operators of experts and adapters in 64 bits, from their formulas, on the CPU; with bounds of what 32-bit sums and the
operands' pieces may change."""
import numpy as np
import torch

from oracle import oracle as orc

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}       # relative, of a rounding to the type
SUBNORMAL = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}                     # and absolute, below its normal numbers


def silu(z):
    return z / (1 + np.exp(-np.clip(z, -700, 700)))


def route(z, top_k, score, bias, groups, top_groups, group_top, renorm, scale):
    """ids and weights of rows z, in 64 bits; the lower index wins a tie."""
    z = np.asarray(z, np.float64)
    T, E = z.shape
    if score == "softmax":
        top = z.max(1, keepdims=True)
        e = np.where(np.isneginf(z), 0.0, np.exp(z - np.where(np.isneginf(top), 0.0, top)))
        s = e.sum(1, keepdims=True)
        p = np.divide(e, s, out=np.zeros_like(e), where=s > 0)
    else:
        p = np.where(z < 0, np.exp(np.minimum(z, 0)) / (1 + np.exp(np.minimum(z, 0))), 1 / (1 + np.exp(-np.maximum(z, 0))))
    c = p if bias is None else p + np.asarray(bias, np.float64)
    if bias is None and (groups == 1 or group_top == 1):
        c = z                 # scores rise strictly with their logits, also where 64 bits hold them as equal
    each = E // groups
    ids, weights = np.zeros((T, top_k), np.int32), np.zeros((T, top_k))
    for t in range(T):
        allowed = range(E)
        if groups > 1:
            total = [sum(sorted(c[t, i * each:(i + 1) * each], reverse=True)[:group_top]) for i in range(groups)]
            best = sorted(range(groups), key=lambda i: (-total[i], i))[:top_groups]
            allowed = [e for e in range(E) if e // each in best]
        ids[t] = sorted(allowed, key=lambda e: (-c[t, e], e))[:top_k]
        w = p[t, ids[t]]
        if renorm:
            if score == "sigmoid" and w.max() == 0 and np.isfinite(z[t, ids[t]]).any():     # below the exponents' range
                w = np.exp(z[t, ids[t]] - z[t, ids[t]].max())
            w = w / w.sum() if w.sum() > 0 else np.zeros_like(w)
        weights[t] = w * scale
    return ids, weights


def ffn(x, ids, weights, gate, up, down, x_type, y_type, dw=None):
    """y and its bound for decoded weights gate, up [E][F][K], down [E][N][F] (f64) and rows x as the call has them.

    Bound: a sum of products in 32 bits is within 1e-5 of the products' magnitudes (as the GEMVs' bound), silu's slope is
    below 1.1 and its evaluation within 2e-6; h is held to 2^-22 (2^-11 with 16-bit x and y) of itself, or to 2^-39
    (2^-26) of its row's largest; the output is rounded once.  dw: what the weights themselves may be off by, arrays like
    gate, up and down (rounded_weights)."""
    T, k = ids.shape
    N = down.shape[1]
    exact = x_type == "f32" or y_type == "f32"
    rel, low = (2.0 ** -22, 2.0 ** -39) if exact else (2.0 ** -11, 2.0 ** -26)
    y, bound = np.zeros((T, N)), np.zeros((T, N))
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if e < 0:
                continue
            g, u = gate[e] @ x[t], up[e] @ x[t]
            # x in pieces, too
            dx = rel * np.abs(x[t]) + low * np.abs(x[t]).max() if exact else low * np.abs(x[t]).max() * np.ones_like(x[t])
            dg = 1e-5 * np.abs(gate[e]) @ np.abs(x[t]) + np.abs(gate[e]) @ dx
            du = 1e-5 * np.abs(up[e]) @ np.abs(x[t]) + np.abs(up[e]) @ dx
            if dw is not None:
                dg, du = dg + dw[0][e] @ (np.abs(x[t]) + dx), du + dw[1][e] @ (np.abs(x[t]) + dx)
            h = silu(g) * u
            dh = 1.1 * dg * np.abs(u) + (np.abs(silu(g)) + 1.1 * dg) * du + 2e-6 * np.abs(h)
            dh += rel * (np.abs(h) + dh) + low * np.abs(h).max()
            w = float(weights[t, j])
            y[t] += w * (down[e] @ h)
            bound[t] += abs(w) * (np.abs(down[e]) @ (dh + 1e-5 * np.abs(h)))
            if dw is not None:
                bound[t] += abs(w) * (dw[2][e] @ (np.abs(h) + dh))
    bound += 1e-6 * np.abs(y)
    return y, bound + HALF_STEP[y_type] * (np.abs(y) + bound) + SUBNORMAL[y_type] + 1e-30


def lora(x, y, A, B, ids, scales, y_type):
    """out and its bound.  Operands are exact in 16 bits and held to 2^-22 in fp32, A x too; a 32-bit sum of n products is
    within 1e-5 of their magnitudes."""
    out, bound = y.copy(), np.zeros_like(y)
    for t, a in enumerate(ids):
        if a < 0:
            continue
        s = 1.0 if scales is None else float(scales[a])
        v = A[a] @ x[t]
        out[t] += s * (B[a] @ v)
        bound[t] = abs(s) * (np.abs(B[a]) @ (1.2e-5 * np.abs(A[a]) @ np.abs(x[t]) + 1.2e-5 * np.abs(v)))
    bound += 2.0 ** -23 * np.abs(out)
    return out, np.where(bound > 0, bound + HALF_STEP[y_type] * (np.abs(out) + bound) + SUBNORMAL[y_type], 0)


def expert_weights(fmt, E, rows, K, seed):
    """Block bytes [E * rows][row bytes] and the decoded [E][rows][K]."""
    from quantised_gguf_weight_gb300 import synth
    b = synth.weights(fmt, E * rows, K, seed=seed)
    return b, orc.decode(fmt, b, K, n_rows_total=E * rows).reshape(E, rows, K)


def rounded_weights(fmt, b, w):
    """What weights of bytes b, decoded w [E][rows][K], may be off by where they are rounded to fp16 after a power of two
    that puts the largest that a row's scales allow into [2^14, 2^15), as bf16 rows and outputs let them.

    A rounding is 2^-11 of the value at most, or 2^-25 (half the smallest fp16), 2^-39 of the row's largest.  Q8_0: d is
    exact, d q rounded once.  Q6_K: d sc is rounded, and its product with q: twice.  Q4_K: d and sc q are exact, the minimum
    is rounded, and the sum: 2^-11 of |w| and of |dmin| 63.  The second order is below a 2^-10th of these."""
    E, rows, K = w.shape
    most = {"q8_0": 128, "q6_k": 4096, "q4_k": 945}[fmt]
    if fmt == "q8_0":
        d = np.abs(b.reshape(E, rows, -1, 34)[..., :2].copy().view(np.float16)[..., 0].astype(np.float64))
        dw, largest = 2.0 ** -11 * np.abs(w), most * d.max(2)
    elif fmt == "q6_k":
        d = np.abs(b.reshape(E, rows, -1, 210)[..., 208:].copy().view(np.float16)[..., 0].astype(np.float64))
        dw, largest = 2.0 ** -10 * np.abs(w), most * d.max(2)
    else:
        d = np.abs(b.reshape(E, rows, -1, 144)[..., :4].copy().view(np.float16).astype(np.float64))
        m = np.repeat(63 * d[..., 1], 256, axis=2)[..., :K]
        dw, largest = 2.0 ** -11 * (np.abs(w) + m), (most * d[..., 0] + 63 * d[..., 1]).max(2)
    return (1 + 2.0 ** -10) * dw + 2.0 ** -38 * largest[..., None]


def as_rows(x, dtype):
    """fp64 rows rounded to a type: the tensor and the values it holds."""
    t = torch.from_numpy(x).to(torch.float32).to(TORCH[dtype])
    return t, t.double().numpy()
