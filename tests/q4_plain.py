"""The 4-bit expert products evaluated plainly in 64 bits, with a bound of
the kernels' rounding errors for every element.

Bounds count roundings (u = 2^-24, half a step of fp32; a rounding to bf16 is
off by at most 2^-8 of the value, to fp16 by 2^-11): an fp32 sum of K terms is
within K u of the sum of the terms' magnitudes.  INT4 codes enter the matrix
pipe as 128 + code <= 143 and 136 times the operand's sum is taken off again,
so the sums of a group run over terms of at most 143 + 136 = 279 times the
operand's magnitude."""
import numpy as np

U = 2.0 ** -24
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6])
NIBBLE = {"int4": [(i >> 1) + 4 * (i & 1) for i in range(8)], "e2m1": list(range(8))}


def tile_rows(N, gate_up):
    """Matrix rows in the order of the stored tiles."""
    r = np.arange(N)
    if not gate_up:
        return r
    q, i = r // 16, r % 16
    return np.where(i < 8, 8 * q + i, N // 2 + 8 * q + i - 8)


def stride(K, group):
    return 4 * (-(-(-(-K // 128)) // 4)) * (128 // group)


def pack(codes, scales, fmt, group, gate_up):
    """codes [M, N, K] (0..15), scales [M, N, K/group] -> stored bytes [M, N/16, KB, 1024] and scales [M, N, S],
    written element by element from the description of the storage."""
    M, N, K = codes.shape
    KB = -(-K // 128)
    zero = 8 if fmt == "int4" else 0
    order = tile_rows(N, gate_up)
    full = np.full((M, N, KB * 128), zero, np.uint8)
    full[:, :, :K] = codes[:, order]
    out = np.zeros((M, N // 16, KB, 1024), np.uint8)
    for lane in range(64):
        for j in range(4):
            for i in range(8):
                nib = NIBBLE[fmt][i]
                v = full[:, lane % 16::16].reshape(M, N // 16, KB, 128)[:, :, :, 32 * j + 8 * (lane // 16) + i]
                out[:, :, :, 16 * lane + 4 * j + nib // 2] |= v << (4 * (nib % 2))
    s = np.zeros((M, N, stride(K, group)), scales.dtype)
    s[:, :, :K // group] = scales[:, order]
    return out, s


def values(codes, scales, fmt, group):
    v = codes.astype(np.float64) - 8 if fmt == "int4" else E2M1[codes]
    return v * np.repeat(scales.astype(np.float64), group, axis=-1)


def product(a, da, codes, scales, fmt, group, offset_trick):
    """rows a [n, K] (error da) times W^T: values, and the bound of their error."""
    w = values(codes, scales, fmt, group)
    K = w.shape[-1]
    y = a @ w.T
    err = da @ np.abs(w).T + K * U * (np.abs(a) @ np.abs(w).T)
    if offset_trick and fmt == "int4":
        sums = np.abs(a).reshape(len(a), -1, group).sum(-1)
        err += group * U * 279 * (sums @ np.abs(scales.astype(np.float64)).T)
    return y, err


def silu(z):
    return z / (1 + np.exp(-z))


def layer(x, ids, w, w1, w2, fmt, group, bf16, round_y=True):
    """x [T, H] fp64, ids and w [T, k]; w1 = (codes [mu, E, 2Im, H], scales), w2 = (codes [mu, E, H, Im], scales).
    Returns h [R, mu*Im], y [R, H], out [T, H] (routes r = t*k + j in order) and the error bound of each."""
    T, k = ids.shape
    mu, E, N, H = w1[0].shape
    Im = N // 2
    R = T * k
    eps = 2.0 ** -8 if bf16 else U
    h, dh = np.zeros((R, mu * Im)), np.zeros((R, mu * Im))
    y, dy = np.zeros((R, H)), np.zeros((R, H))
    for e in range(E):
        r = np.nonzero(ids.reshape(-1) == e)[0]
        if not len(r):
            continue
        a = x[r // k]
        for m in range(mu):
            gu, d = product(a, np.zeros_like(a), w1[0][m, e], w1[1][m, e], fmt, group, bf16)
            g, u, dg, du = gu[:, :Im], gu[:, Im:], d[:, :Im], d[:, Im:]
            v = silu(g) * u
            dv = 1.1 * np.abs(u) * dg + np.abs(silu(g)) * du + 1.1 * dg * du + 16 * U * np.abs(v)
            sl = slice(m * Im, (m + 1) * Im)
            h[r, sl], dh[r, sl] = v, dv + eps * (np.abs(v) + dv)
        for m in range(mu):
            sl = slice(m * Im, (m + 1) * Im)
            p, dp = product(h[r, sl], dh[r, sl], w2[0][m, e], w2[1][m, e], fmt, group, bf16)
            y[r] += p
            dy[r] += dp + mu * U * np.abs(p)
    if bf16 and round_y:  # block-scaled half: 11 bits, below the block's largest value's 2^-24 a fixed step
        nb = -(-H // 256)
        M = np.stack([np.abs(y[:, 256 * b:256 * b + 256]).max(1) for b in range(nb)], 1)
        dy = dy + 2.0 ** -11 * (np.abs(y) + dy) + 2.0 ** -24 * np.repeat(M, 256, 1)[:, :H]
    wt = w.astype(np.float64)
    out = (wt[:, :, None] * y.reshape(T, k, H)).sum(1)
    dout = (wt[:, :, None] * (dy + (k + 4) * U * np.abs(y)).reshape(T, k, H)).sum(1)
    dout += eps * (np.abs(out) + dout)
    return h, dh, y, dy, out, dout
