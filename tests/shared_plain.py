"""Plain evaluations in 64 bits, with error bounds, of the shared expert's
training step, of dropout and of the request adapters (CPU, torch.float64).

Bounds.  A value that is stored in a type is off by at most half a step,
U(type) = finfo.eps / 2 relative to it.  A sum of n products in fp32 is off by at
most (n + 4) 2^-24 times the sum of the products' magnitudes (n additions, each
rounded; the products of bf16 are exact in fp32, those of fp32 rounded once).
SiLU and the logistic function are taken with the device's exponential and
reciprocal: 16 2^-24 relative.  Errors of inputs go through a function by the
largest slope: SiLU 1.1, its derivative 0.5.  Second-order terms: a factor 1.02."""
import numpy as np
import torch

F32 = 2.0 ** -24
EXP = 16 * F32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def philox_blocks(n, seed, offset):
    """Philox 4x32, ten rounds, of the counters (i, offset), i < n, as four uint64 arrays of 32-bit words."""
    m = np.uint64(0xFFFFFFFF)
    i = np.arange(n, dtype=np.uint64)
    return philox([i & m, i >> np.uint64(32), np.full(n, offset & 0xFFFFFFFF, np.uint64), np.full(n, offset >> 32, np.uint64)],
                  [seed & 0xFFFFFFFF, seed >> 32])


def philox(c, key):
    m = np.uint64(0xFFFFFFFF)
    k = list(key)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & m, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & m]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def drop_factors(rows, cols, p, seed, offset):
    """0 or the scale, [rows, cols] float64."""
    cut = int(p * 65536 + 0.5)
    if cut == 0:
        return torch.ones(rows, cols, dtype=torch.float64)
    words = philox_blocks(rows * cols // 8, seed, offset)
    bits = np.stack([(words[e // 2] >> np.uint64(16 * (e % 2))) & np.uint64(0xFFFF) for e in range(8)], 1)
    return torch.from_numpy(np.where(bits.reshape(rows, cols) < cut, 0.0, 65536.0 / (65536 - cut)))


def _mm(a, b):
    """a @ b and the bound of its fp32 evaluation."""
    return a @ b, (a.shape[1] + 4) * F32 * (a.abs() @ b.abs())


def _stored(v, e, dtype):
    return e + half_step(dtype) * (v.abs() + e)


def ffn(x, w1, w2, residual, d_out, factors, dtype):
    """{name: (value, bound)} of the training step; inputs float64 holding values of dtype, factors [T, Is]."""
    Is = w2.shape[1]
    z, ez = _mm(x, w1.T)
    g, u, eg, eu = z[:, :Is], z[:, Is:], ez[:, :Is], ez[:, Is:]
    s = torch.sigmoid(g)
    silu = g * s
    h = factors * silu * u
    eh = _stored(h, factors * (1.02 * (1.1 * eg * u.abs() + silu.abs() * eu) + (EXP + 2 * F32) * (silu * u).abs()), dtype)
    out, eo = _mm(h, w2.T)
    eo = eo + 1.02 * (eh @ w2.abs().T)
    if residual is not None:
        out = out + residual
        eo = eo + F32 * out.abs()
    r = dict(gu=(z, ez), hs=(h, eh), out=(out, _stored(out, eo, dtype)))
    dh, ed = _mm(d_out, w2)
    dh, ed = factors * dh, factors * (ed + F32 * dh.abs())
    slope = s * (1 + g * (1 - s))
    dg, du = dh * u * slope, dh * silu
    e_dg = 1.02 * (ed * (u * slope).abs() + dh.abs() * (eu * slope.abs() + 0.5 * eg * u.abs())) + (3 * EXP) * (dh * u).abs()
    e_du = 1.02 * (ed * silu.abs() + dh.abs() * 1.1 * eg) + 2 * EXP * du.abs()
    d, e = torch.cat([dg, du], 1), torch.cat([_stored(dg, e_dg, dtype), _stored(du, e_du, dtype)], 1)
    for name, (a, ea, b, eb) in dict(d_x=(d, e, w1, None), d_w1s=(d.T, e.T, x, None), d_w2s=(d_out.T, None, h, eh)).items():
        v, ev = _mm(a, b)
        if ea is not None:
            ev = ev + 1.02 * (ea @ b.abs())
        if eb is not None:
            ev = ev + 1.02 * (a.abs() @ eb)
        r[name] = (v, _stored(v, ev, dtype))
    return r


def projection(x, w, a, b, scale, ids, dtype, rounded):
    """(value, bound) of x w^T plus each token's adapter; rounded: the low-rank values pass through two operands of
    dtype, their rounding and the rounding of the rest (off by a half step of a half step)."""
    z, ez = _mm(x, w.T)
    for l in torch.unique(ids).tolist():
        if not 0 <= l < a.shape[0]:
            continue
        rows = torch.nonzero(ids == l)[:, 0]
        v, ev = _mm(x[rows], a[l].T)
        v, ev = v * scale[l], (ev + 9 * F32 * v.abs()) * abs(scale[l])  # up to eight parts of K, then the scale
        if rounded:
            ev = ev + half_step(dtype) ** 2 * (v.abs() + ev)
        y, ey = _mm(v, b[l].T)
        z[rows] += y
        ez[rows] += ey + 1.02 * (ev @ b[l].abs().T) + F32 * (y.abs() + z[rows].abs())
    return z, ez


def swiglu(z, ez, dtype):
    Is = z.shape[1] // 2
    g, u, eg, eu = z[:, :Is], z[:, Is:], ez[:, :Is], ez[:, Is:]
    silu = g * torch.sigmoid(g)
    h = silu * u
    return h, _stored(h, 1.02 * (1.1 * eg * u.abs() + silu.abs() * eu) + (EXP + 2 * F32) * h.abs(), dtype)


def add_residual(z, ez, residual, dtype):
    if residual is not None:
        z = z + residual
        ez = ez + F32 * z.abs()
    return z, _stored(z, ez, dtype)


def check(name, got, value, bound, dtype):
    """Element by element within the bound, and in the norm within a few roundings."""
    got = got.double().cpu().reshape(value.shape)
    bad = ~((got - value).abs() <= bound + 1e-37)
    assert not bad.any(), (name, int(bad.sum()), torch.nonzero(bad)[:4].tolist(), float((got - value).abs().max()))
    # at most five roundings to dtype lie between the inputs and any output, each at most a half step in
    # the norm; fp32 sums add their own, which for random signs stay far below n half steps
    n = value.norm()
    if n > 0 and value.numel() >= 64:
        assert float((got - value).norm() / n) <= 5 * half_step(dtype) + 64 * F32, (name, float((got - value).norm() / n))
