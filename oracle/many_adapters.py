"""Plain float64 definitions of the operators for many adapters on one base, and the
float32 definition of the AdamW step with 8-bit states.  Test infrastructure only:
imports nothing from the product.

Page citations: "What is LoRA?" (IBM): one frozen base, small LoRA modules swapped per
task; "Grokking QLoRA" (vnread), "Paged Optimizers": Adam's two states per parameter.
"""

import numpy as np


def groups(idx, n):
    """(order, offsets): tokens of adapter 0, 1, ... in token order, then those without one."""
    idx = np.asarray(idx)
    key = np.where((idx >= 0) & (idx < n), idx, n)
    order = [t for a in range(n + 1) for t in np.flatnonzero(key == a)]
    offsets = [0]
    for a in range(n):
        offsets.append(offsets[-1] + int((key == a).sum()))
    return np.array(order, dtype=np.int32), np.array(offsets, dtype=np.int32)


def _parts(A, B, ranks, a):
    rk = A.shape[1] if ranks is None else ranks[a]
    return A[a, :rk].astype(np.float64), B[a, :, :rk].astype(np.float64)


def fwd(A, B, scales, idx, X, Y, ranks=None):
    """(Y + term, |term| bound inputs): returns Y', term, T_abs, where bounds[t] uses the sums of magnitudes:
    mag1 = |s| sum_j |B||T|, mag2 = |s| sum_j |B| sum_k |a||x| (same shape as Y)."""
    Y, X = Y.astype(np.float64), X.astype(np.float64)
    term, mag1, mag2 = np.zeros_like(Y), np.zeros_like(Y), np.zeros_like(Y)
    for t, a in enumerate(idx):
        if a < 0:
            continue
        Aa, Ba = _parts(A, B, ranks, a)
        T = Aa @ X[t]
        s = float(scales[a])
        term[t] = s * (Ba @ T)
        mag1[t] = abs(s) * (np.abs(Ba) @ np.abs(T))
        mag2[t] = abs(s) * (np.abs(Ba) @ (np.abs(Aa) @ np.abs(X[t])))
    return Y + term, term, mag1, mag2


def bwd(A, B, scales, idx, X, dY, dX, ranks=None):
    """dict of dX, dA, dB and their magnitude sums (as fwd's mag1, mag2)."""
    X, dY, dX = (v.astype(np.float64) for v in (X, dY, dX))
    n, r, K = A.shape
    N = B.shape[1]
    out = {"dX": dX.copy(), "dX1": np.zeros_like(dX), "dX2": np.zeros_like(dX)}
    for k, shape in (("dA", (n, r, K)), ("dB", (n, N, r))):
        for suffix in ("", "1", "2"):
            out[k + suffix] = np.zeros(shape)
    for a in range(n):
        rows = np.flatnonzero(np.asarray(idx) == a)
        if not len(rows):
            continue
        Aa, Ba = _parts(A, B, ranks, a)
        rk = Aa.shape[0]
        s = float(scales[a])
        x, dy = X[rows], dY[rows]
        U, T = dy @ Ba, x @ Aa.T
        Uabs, Tabs = np.abs(dy) @ np.abs(Ba), np.abs(x) @ np.abs(Aa).T
        out["dX"][rows] += s * (U @ Aa)
        out["dX1"][rows] = abs(s) * (np.abs(U) @ np.abs(Aa))
        out["dX2"][rows] = abs(s) * (Uabs @ np.abs(Aa))
        out["dA"][a, :rk] = s * (U.T @ x)
        out["dA1"][a, :rk] = abs(s) * (np.abs(U).T @ np.abs(x))
        out["dA2"][a, :rk] = abs(s) * (Uabs.T @ np.abs(x))
        out["dB"][a, :, :rk] = s * (dy.T @ T)
        out["dB1"][a, :, :rk] = abs(s) * (np.abs(dy).T @ np.abs(T))
        out["dB2"][a, :, :rk] = abs(s) * (np.abs(dy).T @ Tabs)
    return out


# ---------------------------------------------------------------------------
# 8-bit states
# ---------------------------------------------------------------------------
def state_hash(element, tensor, seed):
    """The 32 random bits of an element of the tensor-th tensor of a list."""
    mask = (1 << 32) - 1
    x = [((int(e) + seed * 0xB7E15163 + tensor * 0x3504F333) * 0x9E3779B9) & mask for e in element]
    x = [((v ^ (v >> 16)) * 0x6A09E667) & mask for v in x]
    x = [((v ^ (v >> 15)) * 0xBB67AE85) & mask for v in x]
    return np.array([v ^ (v >> 16) for v in x], dtype=np.uint32)


def float8_values(mantissa, lowest):
    """The non-negative finite values of a float8 format, in code order."""
    exps = {3: 16, 2: 31}[mantissa]
    vals = []
    for e in range(exps):
        for f in range(1 << mantissa):
            v = f / (1 << mantissa) * 2.0 ** lowest if e == 0 else (1 + f / (1 << mantissa)) * 2.0 ** (lowest + e - 1)
            vals.append(v)
    return np.array(vals[:127] if mantissa == 3 else vals)  # E4M3: the last code is NaN


def stochastic_round(x, u, values):
    """x >= 0 (float32) to the grid `values`: the lower neighbour, or the upper one where the
    position between them plus u (in [0, 1)) reaches 1; the largest value above the grid."""
    x = np.asarray(x, dtype=np.float64)
    i = np.clip(np.searchsorted(values, x, side="right") - 1, 0, len(values) - 1)
    up = np.minimum(i + 1, len(values) - 1)
    step = np.where(up > i, values[up] - values[i], 1.0)
    return np.where((x - values[i]) / step + u >= 1.0, values[up], values[i])


E4M3, E5M2 = float8_values(3, -6), float8_values(2, -14)


def adamw8(p, g, m, v, ms, vs, step, tensor, seed, lr, beta1, beta2, eps, weight_decay, clip=1.0, lr_scale=1.0):
    """One step on one tensor, float32 operation by operation: p, g float32 [n]; m, v code
    values [n]; ms, vs float32 scales per 256.  Returns (p, m, v, ms, vs)."""
    f = np.float32
    n = len(p)
    b1, b2, lr64 = f(beta1), f(beta2), float(f(lr)) * float(f(lr_scale))
    bc1, bc2 = 1.0 - float(b1) ** step, 1.0 - float(b2) ** step
    decay, step_size = f(1.0 - lr64 * float(f(weight_decay))), f(lr64 / bc1)
    g = g.astype(f) * f(clip)
    block = np.arange(n) // 256
    mm = b1 * (m.astype(f) * ms[block]) + (f(1) - b1) * g
    vv = b2 * (v.astype(f) * vs[block]) + (f(1) - b2) * (g * g)
    denom = np.sqrt(vv) / f(np.sqrt(bc2)) + f(eps)
    p = p * decay - (step_size * mm) / denom
    h = state_hash(np.arange(n), tensor, seed)
    um, uv = (h & 0xFFFFF) / 2.0 ** 20, (h >> 11) / 2.0 ** 21
    nm, nv, nms, nvs = np.zeros(n, f), np.zeros(n, f), np.zeros_like(ms), np.zeros_like(vs)
    for b in range(len(ms)):
        at = block == b
        top_m, top_v = f(np.abs(mm[at]).max()), f(vv[at].max())
        if top_m >= 2.0 ** -100:
            nms[b] = top_m / f(448)
            nm[at] = np.copysign(stochastic_round(np.abs(mm[at]) * (f(448) * (f(1) / top_m)), um[at], E4M3), mm[at])
        if top_v >= 2.0 ** -100:
            nvs[b] = top_v / f(57344)
            q = stochastic_round(vv[at] * (f(57344) * (f(1) / top_v)), uv[at], E5M2)
            nv[at] = np.where(vv[at] > 0, np.maximum(q, 2.0 ** -16), q)
    return p.astype(f), nm, nv, nms, nvs
