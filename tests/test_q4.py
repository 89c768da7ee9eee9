"""The layer over 4-bit expert weights (moe_q4.h) against a plain evaluation
in 64 bits (q4_plain.py, which derives the tolerances)."""
import ctypes

import numpy as np
import pytest

import moe_inputs as mi
import q4_plain as qp
from helpers import decode_y, to_dev, to_host_f32

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def m():
    import mixture_experts_ffn_moe_amd as m
    return m


@pytest.fixture
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return "cuda"


def gpu(fn):
    return pytest.mark.gpu(fn)


def layer_scales(rng, shape, bf16):
    s = (rng.random(shape) * 0.02 + 0.01).astype(np.float32)
    s[rng.random(shape) < 0.05] = 0.0           # a group of zeros
    s[rng.random(shape) < 0.1] *= -1.0          # a scale may have any sign
    return mi.bf16_bits_to_f32(mi.f32_to_bf16_bits(s)) if bf16 else s


class Case:
    """One layer: dense description, stored weights, device tensors."""

    def __init__(self, m, T, H, E, k, Im, mu, dtype, fmt, group, seed=0, renorm=True, bias=None, dev="cuda"):
        rng = np.random.default_rng(seed)
        self.bf16 = dtype == "bf16"
        self.T, self.H, self.E, self.k, self.Im, self.mu, self.fmt, self.group = T, H, E, k, Im, mu, fmt, group
        x = rng.standard_normal((T, H), dtype=np.float32)
        self.xbits = mi.f32_to_bf16_bits(x) if self.bf16 else x
        self.x = (mi.bf16_bits_to_f32(self.xbits) if self.bf16 else x).astype(np.float64)
        self.wg = (rng.standard_normal((E, H)) * 2 / np.sqrt(H)).astype(np.float32)
        self.bias = None if bias is None else (rng.standard_normal(E) * bias).astype(np.float32)
        c1 = rng.integers(0, 16, (mu, E, 2 * Im, H), dtype=np.uint8)
        c2 = rng.integers(0, 16, (mu, E, H, Im), dtype=np.uint8)
        s1 = layer_scales(rng, (mu, E, 2 * Im, H // group), self.bf16)
        s2 = layer_scales(rng, (mu, E, H, Im // group), self.bf16)
        self.w1, self.w2 = (c1, s1), (c2, s2)
        self.shape = m.make_shape(T, H, E, k, Im, mu, dtype, renorm)
        self.q4 = m.make_q4(fmt, group)
        f = lambda a: a.reshape((-1,) + a.shape[2:])  # noqa: E731
        p1, t1 = qp.pack(f(c1), f(s1), fmt, group, True)
        p2, t2 = qp.pack(f(c2), f(s2), fmt, group, False)
        sc = lambda t: to_dev(mi.f32_to_bf16_bits(t) if self.bf16 else t, mi.BF16 if self.bf16 else mi.F32, dev)  # noqa: E731
        self.d = dict(x=to_dev(self.xbits, mi.BF16 if self.bf16 else mi.F32, dev), wg=torch.from_numpy(self.wg).to(dev),
                      bias=None if bias is None else torch.from_numpy(self.bias).to(dev),
                      w=(torch.from_numpy(p1).to(dev), sc(t1), torch.from_numpy(p2).to(dev), sc(t2)))

    def forward(self, m):
        buf = m.MoELayerBuffers(self.shape)
        buf.workspace.fill_(0xA5)
        buf.out.fill_(float("nan"))
        d = self.d
        out = buf.forward_q4(self.q4, d["x"], d["wg"], d["bias"], *d["w"])
        torch.cuda.synchronize()
        return out, buf

    def dense_steps(self, m):
        """The step-wise path: route, permute, the two 4-bit products, finalize."""
        s, d, T, k, R = self.shape, self.d, self.T, self.k, self.T * self.k
        e = lambda *sh, dt=torch.float32: torch.empty(*sh, dtype=dt, device=d["x"].device)  # noqa: E731
        i32 = torch.int32
        r = dict(logits=e(T, self.E), ids=e(T, k, dt=i32), w=e(T, k), counts=e(self.E, dt=i32), offsets=e(self.E + 1, dt=i32),
                 perm=e(R, dt=i32), inv=e(R, dt=i32), h=e(R, self.mu * self.Im, dt=d["x"].dtype).fill_(float("nan")),
                 y=e(m.y_nbytes(s, R), dt=torch.uint8).fill_(0xFF), out=e(T, self.H, dt=d["x"].dtype).fill_(float("nan")))
        m.moe_route(s, d["x"], d["wg"], d["bias"], r["logits"], r["ids"], r["w"])
        m.moe_permute(s, r["ids"], r["counts"], r["offsets"], r["perm"], r["inv"])
        m.moe_q4_w13_swiglu(s, self.q4, d["x"], r["perm"], r["offsets"], d["w"][0], d["w"][1], r["h"])
        m.moe_q4_down(s, self.q4, r["h"], r["offsets"], d["w"][2], d["w"][3], r["y"])
        m.moe_finalize(s, r["y"], r["inv"], r["w"], r["out"])
        torch.cuda.synchronize()
        return r


class Rows:
    def __init__(self, c):
        self.T, self.H, self.dtype = c.T, c.H, mi.BF16 if c.bf16 else mi.F32


def check_steps(c, r):
    ids, w = r["ids"].cpu().numpy(), r["w"].cpu().numpy()
    h, dh, y, dy, out, dout = qp.layer(c.x, ids, w, c.w1, c.w2, c.fmt, c.group, c.bf16)
    inv = r["inv"].cpu().numpy()
    got_h = to_host_f32(r["h"]).astype(np.float64)[inv]
    got_y = decode_y(Rows(c), r["y"], c.T * c.k)[inv]
    for name, got, ref, tol in (("h", got_h, h, dh), ("y", got_y, y, dy), ("out", to_host_f32(r["out"]), out, dout)):
        bad = ~(np.abs(got - ref) <= tol + 1e-30)
        assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.abs(got - ref).max()))
    return out, dout


FORMATS = [("int4", 32), ("int4", 64), ("int4", 128), ("e2m1", 32), ("e2m1", 64), ("e2m1", 128)]

# T, H, E, k, Im, mu, dtype: rows that end inside a tile, K that ends inside a 128-column tile, one token,
# experts without rows, more output tiles than a workgroup takes, all three row-block heights
SHAPES = [
    (1, 128, 1, 1, 128, 1, "bf16"), (1, 256, 64, 8, 128, 2, "bf16"), (5, 384, 8, 3, 128, 1, "bf16"),
    (17, 640, 3, 2, 256, 2, "bf16"), (40, 128, 2, 2, 384, 1, "bf16"), (150, 256, 5, 3, 128, 3, "bf16"),
    (129, 128, 1, 1, 128, 1, "bf16"), (70, 512, 33, 4, 128, 1, "bf16"),
    (1, 128, 4, 2, 128, 1, "f32"), (37, 384, 7, 3, 256, 2, "f32"), (100, 256, 2, 2, 128, 1, "f32"),
]
# sizes only the finer groups divide
NARROW = [
    (3, 64, 4, 2, 32, 1, "bf16", 32), (50, 320, 5, 2, 96, 2, "bf16", 32), (90, 448, 2, 1, 160, 1, "bf16", 32),
    (33, 192, 6, 2, 64, 2, "bf16", 64), (20, 448, 7, 3, 160, 2, "f32", 32), (9, 64, 3, 3, 192, 1, "f32", 64),
]


def run_steps(m, shape, fmt, group, seed):
    print(f"q4 steps {shape} {fmt} g{group}", flush=True)
    c = Case(m, *shape, fmt, group, seed=seed, renorm=seed % 2 == 0, bias=None if seed % 3 else 1.0)
    out, dout = check_steps(c, c.dense_steps(m))
    got, buf = c.forward(m)
    # the one call: same routing; its output within the bound (twice: its sums may run in another order)
    got = to_host_f32(got)
    assert (np.abs(got - out) <= 2 * dout + 1e-30).all(), float(np.abs(got - out).max())


@gpu
@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_steps(m, dev, shape, fmt, group):
    run_steps(m, shape, fmt, group, seed=shape[0])


@gpu
@pytest.mark.parametrize("fmt", ["int4", "e2m1"])
@pytest.mark.parametrize("shape", NARROW, ids=lambda s: "x".join(map(str, s)))
def test_narrow_steps(m, dev, shape, fmt):
    run_steps(m, shape[:-1], fmt, shape[-1], seed=shape[0])


# the small-token path: one unit per wave and fewer, more, cut ones; K tails of the down product; every token on
# every expert; all tokens on the same experts
DECODE = [(1, 2048, 64, 8, 128, 1), (1, 2048, 1, 1, 128, 1), (3, 4096, 16, 4, 128, 2), (8, 2048, 64, 8, 256, 1),
          (16, 2048, 6, 6, 128, 2), (16, 4096, 64, 2, 128, 1), (5, 2048, 40, 8, 384, 1), (16, 2048, 16, 16, 128, 1)]


@gpu
@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("shape", DECODE, ids=lambda s: "x".join(map(str, s)))
def test_decode(m, dev, shape, fmt, group):
    print(f"q4 decode {shape} {fmt} g{group}", flush=True)
    c = Case(m, *shape, "bf16", fmt, group, seed=shape[0] + group, renorm=group != 64, bias=4.0 if shape[0] == 5 else None)
    r = c.dense_steps(m)
    out, dout = check_steps(c, r)
    got, buf = c.forward(m)
    v = buf.views()
    for n in ("logits", "ids", "w", "counts", "offsets", "perm", "inv"):
        assert torch.equal(v[n], r[n]), n
    got = to_host_f32(got)
    assert (np.abs(got - out) <= 2 * dout + 1e-30).all(), float(np.abs(got - out).max())
    again, _ = c.forward(m)
    assert np.array_equal(to_host_f32(again), got)


@gpu
@pytest.mark.parametrize("shape", [(2, 2048, 8, 3, 32, 2), (7, 2048, 24, 5, 96, 1), (16, 2048, 5, 2, 224, 1)])
@pytest.mark.parametrize("fmt", ["int4", "e2m1"])
def test_decode_narrow(m, dev, shape, fmt):
    """Intermediate widths that end inside a 128-column tile on the small-token path."""
    print(f"q4 decode {shape} {fmt}", flush=True)
    c = Case(m, *shape, "bf16", fmt, 32, seed=shape[0])
    out, dout = check_steps(c, c.dense_steps(m))
    got = to_host_f32(c.forward(m)[0])
    assert (np.abs(got - out) <= 2 * dout + 1e-30).all()


@gpu
@pytest.mark.parametrize("T,H,E,k", [(17, 2048, 64, 8), (40, 4096, 5, 2), (257, 2048, 33, 3), (1024, 2048, 64, 4),
                                     (1025, 2048, 8, 2), (30, 2048, 4, 1)])
def test_routing_of_batches(m, dev, T, H, E, k):
    """The one call's routing of medium batches: the step-wise path's bits."""
    print(f"q4 routing T={T} H={H} E={E} k={k}", flush=True)
    c = Case(m, T, H, E, k, 128, 1, "bf16", "int4", 128, seed=T, bias=2.0 if T == 40 else None, renorm=T != 257)
    r = c.dense_steps(m)
    got, buf = c.forward(m)
    v = buf.views()
    for n in ("logits", "ids", "w", "counts", "offsets", "perm", "inv", "h"):
        assert torch.equal(v[n], r[n]), n
    assert torch.equal(got, r["out"])


@gpu
def test_graph_replay_and_streams(m, dev):
    """Captured and replayed with new tokens in the same buffers, eager calls between; another stream; both paths."""
    for T in (6, 30):
        c = Case(m, T, 2048, 12, 3, 128, 1, "bf16", "int4", 128, seed=T)
        d = c.d
        graphed, eager = m.MoELayerBuffers(c.shape), m.MoELayerBuffers(c.shape)
        eager.forward_q4(c.q4, d["x"], d["wg"], d["bias"], *d["w"])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphed.forward_q4(c.q4, d["x"], d["wg"], d["bias"], *d["w"])
        for i in range(4):
            d["x"].copy_(torch.randn(T, 2048, generator=torch.Generator().manual_seed(i)))
            graphed.out.fill_(float("nan"))
            graph.replay()
            eager.forward_q4(c.q4, d["x"], d["wg"], d["bias"], *d["w"])
            torch.cuda.synchronize()
            assert torch.equal(graphed.out, eager.out), (T, i)
        st = torch.cuda.Stream()
        eager.out.fill_(float("nan"))
        torch.cuda.synchronize()
        eager.forward_q4(c.q4, d["x"], d["wg"], d["bias"], *d["w"], stream=st)
        torch.cuda.synchronize()
        assert torch.equal(graphed.out, eager.out)


@gpu
def test_quantized_layer_near_the_dense_one(m, dev):
    """Quantise a dense bf16 layer and run both: the 4-bit layer equals the dense layer on the dequantised weights
    (rounded to bf16, 2^-8 of each weight)."""
    T, H, E, k, Im, mu = 24, 256, 6, 2, 128, 2
    g = torch.Generator().manual_seed(2)
    r = lambda *sh: torch.randn(*sh, generator=g)  # noqa: E731
    x, wg = r(T, H).bfloat16().to(dev), (r(E, H) * 0.1).to(dev)
    w1, w2 = (r(mu, E, 2 * Im, H) * 0.05).bfloat16().to(dev), (r(mu, E, H, Im) * 0.05).bfloat16().to(dev)
    s, q4 = m.make_shape(T, H, E, k, Im, mu, "bf16"), m.make_q4("e2m1", 32)
    z = m.moe_q4_get_sizes(s, q4)
    st = {n: torch.empty(b, dtype=torch.uint8, device=dev) for n, b in z.items()}
    m.moe_q4_quantize_w13(s, q4, w1, st["w1_codes"], st["w1_scales"])
    m.moe_q4_quantize_down(s, q4, w2, st["w2_codes"], st["w2_scales"])
    buf = m.MoELayerBuffers(s)
    got = buf.forward_q4(q4, x, wg, None, st["w1_codes"], st["w1_scales"], st["w2_codes"], st["w2_scales"]).float().clone()

    def dequantised(codes, scales, N, K, gate_up):
        KB, S = -(-K // 128), qp.stride(K, 32)
        b = codes.cpu().numpy().reshape(mu * E, N // 16, KB, 4, 16, 4, 4)
        nib = np.stack([b & 15, b >> 4], -1).reshape(mu * E, N // 16, KB, 4, 16, 4, 8)   # lane / 16, lane % 16, word, nibble
        c = nib.transpose(0, 1, 4, 2, 5, 3, 6).reshape(mu * E, N, KB * 128)[:, :, :K]
        sc = scales.view(torch.bfloat16).float().cpu().numpy().reshape(mu * E, N, S)[:, :, :K // 32]
        w = np.empty((mu * E, N, K))
        w[:, qp.tile_rows(N, gate_up)] = qp.values(c, sc, "e2m1", 32)
        return torch.from_numpy(w.astype(np.float32)).bfloat16().to(dev)

    d1 = dequantised(st["w1_codes"], st["w1_scales"], 2 * Im, H, True).view(mu, E, 2 * Im, H)
    d2 = dequantised(st["w2_codes"], st["w2_scales"], H, Im, False).view(mu, E, H, Im)
    assert (d1.float() - w1.float()).norm() < 0.15 * w1.float().norm()  # 4 bits: a step of at most 1/3 of a value
    ref = m.MoELayerBuffers(s).forward(x, wg, None, d1, d2).float()
    # six roundings to bf16 apart (weights twice, h twice, out twice): 2^-8 each of independent terms
    assert (got - ref).norm() <= 6 * 2.0 ** -8 * ref.norm()


@gpu
@pytest.mark.parametrize("fmt,group", [("int4", 32), ("int4", 128), ("e2m1", 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Im", [(128, 128), (384, 256), (2176, 128)])
def test_quantize(m, dev, H, Im, dtype, fmt, group):
    """Stored codes and scales, bit for bit: scale = M / 7 (6) rounded to the
    layer's type, the nearest code, ties to even; constructed ties and zero
    groups."""
    E, mu = 2, 2
    rng = np.random.default_rng(H + Im + group)
    bf16 = dtype == "bf16"
    low = lambda a: mi.bf16_bits_to_f32(mi.f32_to_bf16_bits(a)) if bf16 else a.astype(np.float32)  # noqa: E731
    s = m.make_shape(4, H, E, 1, Im, mu, dtype)
    q4 = m.make_q4(fmt, group)
    z = m.moe_q4_get_sizes(s, q4)
    top = 7.0 if fmt == "int4" else 6.0
    for gate_up, N, K, call, names in ((True, 2 * Im, H, m.moe_q4_quantize_w13, ("w1_codes", "w1_scales")),
                                       (False, H, Im, m.moe_q4_quantize_down, ("w2_codes", "w2_scales"))):
        w = low((rng.standard_normal((mu * E, N, K)) * 0.02).astype(np.float32))
        w[:, 3, :group] = 0.0
        # ties: a group whose scale is exactly 1/4
        w[:, 5, :group] = low(((np.arange(group) % 29 - 14) / 8 * (top / 7)).astype(np.float32))
        w[:, 5, 0] = top / 4
        g = w.reshape(mu * E, N, K // group, group)
        scales = low((np.abs(g).max(-1).astype(np.float32) / np.float32(top)).astype(np.float32))
        with np.errstate(divide="ignore", invalid="ignore"):
            quot = np.where(scales[..., None] > 0, g.astype(np.float64) / scales[..., None].astype(np.float64), 0.0)
        if fmt == "int4":
            codes = np.clip(np.rint(quot), -7, 7).astype(np.int64) + 8
        else:
            a = np.abs(quot)
            dist = np.abs(a[..., None] - qp.E2M1[:8])
            near = dist == dist.min(-1, keepdims=True)
            # of two equally near magnitudes the one with the even code
            mag = np.where(near[..., ::2].any(-1) & (near.sum(-1) > 1), 2 * near[..., ::2].argmax(-1), near.argmax(-1))
            codes = np.where((mag > 0) & (quot < 0), mag + 8, mag)
        codes = codes.reshape(mu * E, N, K).astype(np.uint8)
        ref_c, ref_s = qp.pack(codes, scales, fmt, group, gate_up)
        dc = torch.full((z[names[0]],), 0xEE, dtype=torch.uint8, device=dev)
        ds = torch.full((z[names[1]] // (2 if bf16 else 4),), 7.0, dtype=torch.bfloat16 if bf16 else torch.float32, device=dev)
        call(s, q4, to_dev(mi.f32_to_bf16_bits(w) if bf16 else w, mi.BF16 if bf16 else mi.F32, dev), dc, ds)
        assert np.array_equal(to_host_f32(ds).reshape(ref_s.shape), ref_s)
        assert np.array_equal(dc.cpu().numpy().reshape(ref_c.shape), ref_c)


# ---------------------------------------------------------------- refusals (no GPU: nothing is enqueued)

def test_refusals(m):
    lib = m._lib.lib
    P, mis = ctypes.c_void_p(4096), ctypes.c_void_p(4096 + 8)
    INV, UNS, WS = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED, m.MOE_ERR_WORKSPACE
    ok = m.make_shape(8, 256, 8, 2, 128, 1, "bf16")
    q = m.make_q4("int4", 128)
    big = ctypes.c_size_t(1 << 40)
    ref = lambda v: None if v is None else ctypes.byref(v)  # noqa: E731

    def calls(s, q4):
        s, q4 = ref(s), ref(q4)
        return [lib.moe_q4_quantize_w13(s, q4, P, P, P, None), lib.moe_q4_quantize_down(s, q4, P, P, P, None),
                lib.moe_q4_w13_swiglu(s, q4, P, P, P, P, P, P, None), lib.moe_q4_down(s, q4, P, P, P, P, P, None),
                lib.moe_forward_q4(s, q4, P, P, None, P, P, P, P, P, P, big, None),
                lib.moe_q4_get_sizes(s, q4, ctypes.byref(m._lib.MoeQ4Sizes()))]

    cases = [(None, q, INV), (ok, None, INV), (ok, m.MoeQ4Spec(2, 128), INV), (ok, m.MoeQ4Spec(-1, 128), INV),
             (ok, m.MoeQ4Spec(0, 16), INV), (ok, m.MoeQ4Spec(0, 256), INV), (ok, m.MoeQ4Spec(0, 0), INV),
             (m.make_shape(8, 200, 8, 2, 128, 1, "bf16"), q, UNS), (m.make_shape(8, 256, 65, 2, 128, 1, "bf16"), q, UNS),
             (m.make_shape(8, 256, 8, 2, 160, 1, "bf16"), q, UNS),    # 128 does not divide Im
             (m.make_shape(8, 320, 8, 2, 128, 1, "bf16"), q, UNS),    # nor H
             (m.make_shape(8, 256, 8, 9, 128, 1, "bf16"), q, INV)]
    for s, q4, want in cases:
        assert calls(s, q4) == [want] * 6, (s, q4)
    assert lib.moe_q4_get_sizes(ref(ok), ref(q), None) == INV
    s, qq = ref(ok), ref(q)
    need = m.moe_workspace_size(ok)
    f = lambda *a: lib.moe_forward_q4(s, qq, *a, None)  # noqa: E731
    assert f(None, P, None, P, P, P, P, P, P, big) == INV
    assert f(P, P, None, P, None, P, P, P, P, big) == INV
    assert f(P, P, mis, P, P, P, P, P, P, big) == UNS
    assert f(P, P, None, P, mis, P, P, P, P, big) == UNS
    assert f(P, P, None, P, P, P, P, P, None, big) == WS
    assert f(P, P, None, P, P, P, P, P, P, ctypes.c_size_t(need - 1)) == WS
    assert f(P, P, None, P, P, P, P, P, ctypes.c_void_p(4096 + 16), big) == UNS
    assert lib.moe_q4_w13_swiglu(s, qq, P, None, P, P, P, P, None) == INV
    assert lib.moe_q4_down(s, qq, P, P, mis, P, P, None) == UNS
    assert lib.moe_q4_quantize_w13(s, qq, None, P, P, None) == INV
    # no tokens: nothing to do
    zero = ref(m.make_shape(0, 256, 8, 2, 128, 1, "bf16"))
    assert lib.moe_forward_q4(zero, qq, P, P, None, P, P, P, P, P, P, ctypes.c_size_t(0), None) == m.MOE_OK
    assert lib.moe_q4_w13_swiglu(zero, qq, None, None, None, None, None, None, None) == m.MOE_OK


@pytest.mark.parametrize("H,Im,group", [(4096, 768, 128), (4096, 768, 32), (448, 160, 32), (64, 32, 32), (192, 64, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sizes(m, H, Im, group, dtype):
    s = m.make_shape(4, H, 6, 2, Im, 2, dtype)
    z = m.moe_q4_get_sizes(s, m.make_q4("e2m1", group))
    es = 2 if dtype == "bf16" else 4
    assert z["w1_codes"] == 2 * 6 * 2 * Im * -(-H // 128) * 64
    assert z["w2_codes"] == 2 * 6 * H * -(-Im // 128) * 64
    assert z["w1_scales"] == 2 * 6 * 2 * Im * qp.stride(H, group) * es
    assert z["w2_scales"] == 2 * 6 * H * qp.stride(Im, group) * es


def test_binding_checks(m):
    s, q = m.make_shape(4, 128, 4, 2, 128, 1, "bf16"), m.make_q4("int4", 64)
    z = torch.zeros
    with pytest.raises(KeyError):
        m.make_q4("int8", 64)
    with pytest.raises(m.MoeError):
        m.moe_q4_get_sizes(s, m.make_q4("int4", 48))
    with pytest.raises(ValueError, match="GPU tensor"):
        m.moe_q4_quantize_w13(s, q, z(4 * 256 * 128, dtype=torch.bfloat16), z(1), z(1))
    with pytest.raises(ValueError, match="GPU tensor"):
        m.moe_forward_q4(s, q, z(4, 128, dtype=torch.bfloat16), z(4, 128), None, z(1), z(1), z(1), z(1), z(1), z(1))
