"""The small-token path of the 4-bit layer where its kernels take every branch,
the benchmark's decode layer among the shapes (test_q4.py's are smaller).

Two things decide the branches, both mirrored on the host here and asserted for
every case (test_cases_reach_every_branch, no GPU):
* the gate|up kernel hands (active expert, 8 columns) units to 256 workgroups;
  of a workgroup's units, sixteen at a time go whole to its 16 waves ("whole"),
  the rest are cut along H ("cut");
* the down kernel stages as many experts' rows of h as 128 KB hold, in rounds.

Everything is compared with a 64-bit evaluation on the same inputs; tolerances
as in q4_plain.py, whose functions the torch ones here are checked against."""
import numpy as np
import pytest

import q4_plain as qp

torch = pytest.importorskip("torch")
U = qp.U
E2M1 = torch.tensor(qp.E2M1)


@pytest.fixture(scope="module")
def m():
    import mixture_experts_ffn_moe_amd as m
    return m


@pytest.fixture
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield "cuda"
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- storage and the plain layer, in torch

def pack(codes, scales, fmt, group, gate_up):
    """qp.pack for tensors [M, N, K] and [M, N, K / group] (large ones, on their device)."""
    M, N, K = codes.shape
    if gate_up:
        codes = codes.view(M, 2, N // 16, 8, K).transpose(1, 2).reshape(M, N, K)
        scales = scales.view(M, 2, N // 16, 8, -1).transpose(1, 2).reshape(M, N, -1)
    KB = -(-K // 128)
    full = torch.nn.functional.pad(codes, (0, KB * 128 - K), value=8 if fmt == "int4" else 0)
    t = full.view(M, N // 16, 16, KB, 4, 4, 8).permute(0, 1, 3, 5, 2, 4, 6)  # .., kb, lane / 16, lane % 16, word, element
    at = [qp.NIBBLE[fmt].index(i) for i in range(8)]                         # element of a nibble
    b = torch.stack([t[..., at[2 * i]] | (t[..., at[2 * i + 1]] << 4) for i in range(4)], -1)
    return b.reshape(M, N // 16, KB, 1024), torch.nn.functional.pad(scales, (0, qp.stride(K, group) - K // group)).contiguous()


def product(a, da, codes, scales, fmt, group, offset_trick=True):
    """qp.product, and the sum of the terms' magnitudes."""
    v = codes.double() - 8 if fmt == "int4" else E2M1.to(codes.device)[codes.long()]
    s = scales.double()
    w = v * s.repeat_interleave(group, -1)
    K = w.shape[-1]
    size = a.abs() @ w.abs().T
    err = da @ w.abs().T + K * U * size
    if offset_trick and fmt == "int4":
        err += group * U * 279 * (a.abs().view(len(a), -1, group).sum(-1) @ s.abs().T)
    return a @ w.T, err, size


def layer(x, ids, w, w1, w2, fmt, group):
    """qp.layer of a bf16 layer: h, y (before its rounding) and out in 64 bits with their bounds, dy with y's rounding
    too, and the bound of an out whose y was never rounded."""
    T, k = ids.shape
    mu, E, N, H = w1[0].shape
    Im, R, dev, eps = N // 2, T * k, x.device, 2.0 ** -8
    z = lambda *s: torch.zeros(*s, dtype=torch.float64, device=dev)  # noqa: E731
    h, dh, y, dy, size = z(R, mu * Im), z(R, mu * Im), z(R, H), z(R, H), z(R, H)
    for e in range(E):
        r = (ids.reshape(-1) == e).nonzero()[:, 0]
        if not len(r):
            continue
        a = x[r // k]
        for i in range(mu):
            gu, d, _ = product(a, torch.zeros_like(a), w1[0][i, e], w1[1][i, e], fmt, group)
            g, u, dg, du = gu[:, :Im], gu[:, Im:], d[:, :Im], d[:, Im:]
            sg = g / (1 + torch.exp(-g))
            v = sg * u
            dv = 1.1 * u.abs() * dg + sg.abs() * du + 1.1 * dg * du + 16 * U * v.abs()
            h[r, i * Im:(i + 1) * Im], dh[r, i * Im:(i + 1) * Im] = v, dv + eps * (v.abs() + dv)
        for i in range(mu):
            sl = slice(i * Im, (i + 1) * Im)
            p, dp, sz = product(h[r, sl], dh[r, sl], w2[0][i, e], w2[1][i, e], fmt, group)
            y[r] += p
            dy[r] += dp + mu * U * p.abs()
            size[r] += sz
    nb = -(-H // 256)
    M = torch.stack([y[:, 256 * b:256 * b + 256].abs().amax(1) for b in range(nb)], 1)
    dyr = dy + 2.0 ** -11 * (y.abs() + dy) + 2.0 ** -24 * M.repeat_interleave(256, 1)[:, :H]
    wt = w.double()[:, :, None]
    out = (wt * y.view(T, k, H)).sum(1)
    # a term's way after its product: times the weight, over the experts of a wave, over 16 waves
    free = (wt * (dy + (k + 20) * U * (size + dy)).view(T, k, H)).sum(1)
    dout = (wt * (dyr + (k + 4) * U * y.abs()).view(T, k, H)).sum(1)
    return h, dh, y, dyr, out, dout + eps * (out.abs() + dout), free + eps * (out.abs() + free)


# ---------------------------------------------------------------- cases

class Case:
    def __init__(self, T, H, E, k, Im, mu, fmt, group, renorm=True):
        self.T, self.H, self.E, self.k, self.Im, self.mu, self.fmt, self.group, self.renorm = T, H, E, k, Im, mu, fmt, group, renorm
        g = torch.Generator().manual_seed(T + H + E)
        self.x = torch.randn(T, H, generator=g).bfloat16()
        self.wg = torch.randn(E, H, generator=g) * 2 / H ** 0.5

    def weights(self, dev):
        g = torch.Generator(device=dev).manual_seed(self.T)
        def one(rows, K):
            codes = torch.randint(0, 16, (self.mu, self.E, rows, K), generator=g, device=dev, dtype=torch.uint8)
            s = torch.rand(self.mu, self.E, rows, K // self.group, generator=g, device=dev) * 0.004 + 0.002
            s *= torch.where(torch.rand(s.shape, generator=g, device=dev) < 0.1, -1.0, 1.0)
            return codes, s.bfloat16()
        return one(2 * self.Im, self.H), one(self.H, self.Im)


def case_id(c):
    return f"{c.T}x{c.H}x{c.E}x{c.k}x{c.Im}x{c.mu}-{c.fmt}-g{c.group}"


BENCH = (4096, 64, 8, 768, 1)  # the benchmark's decode layer
CASES = [Case(16, *BENCH, f, g, g != 64) for f in ("int4", "e2m1") for g in (32, 64, 128)]
CASES += [Case(8, *BENCH, "int4", 128), Case(8, *BENCH, "e2m1", 32), Case(1, *BENCH, "int4", 128), Case(1, *BENCH, "e2m1", 64)]
CASES += [
    Case(16, 2048, 32, 32, 1024, 1, "int4", 128),   # whole units only
    Case(16, 2048, 40, 40, 1024, 1, "e2m1", 128),
    Case(3, 4096, 64, 64, 1056, 1, "int4", 32),     # two whole units a wave and a cut one; K ends inside a tile
    Case(2, 8192, 64, 64, 640, 1, "e2m1", 64, False),
    Case(13, 2048, 64, 64, 96, 2, "int4", 32),      # every expert for every token, two narrow micro-shards
    Case(16, 2048, 64, 64, 128, 1, "e2m1", 128),    # 1024 routes
    Case(16, 2048, 1, 1, 4096, 1, "int4", 64),      # a round that fills the rows' memory to the last byte
    Case(4, 16384, 16, 8, 128, 1, "int4", 128),     # the longest hidden size of four tokens
    Case(1, 16384, 16, 4, 256, 2, "e2m1", 32),
]


def branches(counts, c):
    """Whole and cut units of the workgroups, and the rounds, from the tokens of each expert."""
    act = [int(n) for n in counts if n]
    units = len(act) * c.mu * c.Im // 8
    mine = {(b + 1) * units // 256 - b * units // 256 for b in range(256)}
    fit = 16 * 4096 * 2 // (c.mu * -(-c.Im // 128) * 256)
    rounds, at = 0, 0
    while at < len(act):
        rows, n = act[at], 1
        while at + n < len(act) and rows + act[at + n] <= fit:
            rows += act[at + n]
            n += 1
        at += n
        rounds += 1
    return {n // 16 for n in mine}, {n % 16 for n in mine}, rounds


def test_cases_reach_every_branch():
    seen = {}
    for c in CASES:
        lg = (c.x.double() @ c.wg.double().T).float()
        counts = torch.bincount(lg.topk(c.k, 1)[1].reshape(-1), minlength=c.E)
        seen[case_id(c)] = branches(counts, c)
    bench16 = [v for n, v in seen.items() if n.startswith("16x4096")]
    assert len(bench16) == 6
    for whole, cut, rounds in bench16:
        assert whole == {1} and min(cut) > 0 and rounds == 2
    assert seen["8x4096x64x8x768x1-int4-g128"][2] == 1 and seen["1x4096x64x8x768x1-int4-g128"] == ({0}, {3}, 1)
    assert seen["16x2048x32x32x1024x1-int4-g128"] == ({1}, {0}, 8)
    assert seen["3x4096x64x64x1056x1-int4-g32"][:2] == ({2}, {1})
    assert any(w == {0, 1} for w, _, _ in seen.values())  # workgroups with and without whole units in one launch
    assert max(r for _, _, r in seen.values()) >= 4


@pytest.mark.parametrize("fmt,group", [("int4", 32), ("e2m1", 64), ("int4", 128)])
def test_plain_forms_agree(fmt, group):
    """The torch evaluation and storage against q4_plain.py's numpy ones."""
    rng = np.random.default_rng(group)
    T, k, mu, E, Im, H = 5, 2, 2, 3, 128, 384
    x = rng.standard_normal((T, H))
    ids = np.argsort(rng.random((T, E)), 1)[:, :k]
    w = rng.random((T, k)).astype(np.float32)
    w1 = (rng.integers(0, 16, (mu, E, 2 * Im, H), dtype=np.uint8), rng.random((mu, E, 2 * Im, H // group)).astype(np.float32))
    w2 = (rng.integers(0, 16, (mu, E, H, Im), dtype=np.uint8), rng.random((mu, E, H, Im // group)).astype(np.float32))
    f = lambda p: tuple(torch.from_numpy(a) for a in p)  # noqa: E731
    got = layer(torch.from_numpy(x), torch.from_numpy(ids), torch.from_numpy(w), f(w1), f(w2), fmt, group)
    for a, b in zip(got[:6], qp.layer(x, ids, w, w1, w2, fmt, group, True)):
        np.testing.assert_allclose(a.numpy(), b, rtol=1e-9, atol=0)
    for (c, s), gate_up in ((w1, True), (w2, False)):
        c, s = c.reshape((-1,) + c.shape[2:]), s.reshape((-1,) + s.shape[2:])
        ref = qp.pack(c, s, fmt, group, gate_up)
        got = pack(torch.from_numpy(c), torch.from_numpy(s), fmt, group, gate_up)
        assert np.array_equal(got[0].numpy(), ref[0]) and np.array_equal(got[1].numpy(), ref[1])


def y_values(y, R, H):
    e = y[R * H * 2:].view(torch.int8).view(R, -1).double().repeat_interleave(256, 1)[:, :H]
    return torch.ldexp(y[:R * H * 2].view(torch.float16).view(R, H).double(), e)


def within(name, got, ref, tol):
    d = (got.double() - ref).abs()
    assert (d <= tol + 1e-30).all(), (name, float((d - tol).max()), int((d > tol).sum()))


@pytest.mark.gpu
@pytest.mark.parametrize("c", CASES, ids=case_id)
def test_decode_layer(m, dev, c):
    print(f"decode layer {case_id(c)}", flush=True)
    R = c.T * c.k
    s, q4 = m.make_shape(c.T, c.H, c.E, c.k, c.Im, c.mu, "bf16", c.renorm), m.make_q4(c.fmt, c.group)
    x, wg = c.x.to(dev), c.wg.to(dev)
    w1, w2 = c.weights(dev)
    flat = lambda p, up: pack(p[0].flatten(0, 1), p[1].flatten(0, 1), c.fmt, c.group, up)  # noqa: E731
    stored = (*flat(w1, True), *flat(w2, False))
    buf = m.MoELayerBuffers(s)
    buf.workspace.fill_(0xA5)
    buf.out.fill_(float("nan"))
    out = buf.forward_q4(q4, x, wg, None, *stored).clone()
    v = buf.views()
    # routing: the bits of the steps
    e = lambda *sh, dt=torch.int32: torch.empty(*sh, dtype=dt, device=dev)  # noqa: E731
    st = dict(logits=e(c.T, c.E, dt=torch.float32), ids=e(c.T, c.k), w=e(c.T, c.k, dt=torch.float32), counts=e(c.E),
              offsets=e(c.E + 1), perm=e(R), inv=e(R))
    m.moe_route(s, x, wg, None, st["logits"], st["ids"], st["w"])
    m.moe_permute(s, st["ids"], st["counts"], st["offsets"], st["perm"], st["inv"])
    for n, t in st.items():
        assert torch.equal(v[n].view(-1), t.view(-1)), n
    h, dh, y, dy, ref, _, dout = layer(x.double(), st["ids"], st["w"], w1, w2, c.fmt, c.group)
    inv = st["inv"].long()
    within("out", out, ref, dout)
    # what the path leaves for the backward pass: h and offsets, from which the down product writes y
    within("h", v["h"][inv], h, dh)
    yb = torch.full((m.y_nbytes(s, R),), 0xFF, dtype=torch.uint8, device=dev)
    m.moe_q4_down(s, q4, v["h"], v["offsets"], stored[2], stored[3], yb)
    within("y", y_values(yb, R, c.H)[inv], y, dy)
    # again, in a workspace that holds other data
    buf.workspace.fill_(0x3C)
    assert torch.equal(buf.forward_q4(q4, x, wg, None, *stored), out)
