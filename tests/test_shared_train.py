"""The shared expert's training step and dropout (moe_shared_train.h) against
plain evaluations in 64 bits (shared_plain.py, which derives the tolerances)."""
import ctypes

import numpy as np
import pytest

import shared_plain as sp

torch = pytest.importorskip("torch")

SEED, OFFSET = 0x9A3C5B7D12E4F608, (7 << 32) + 11


@pytest.fixture(scope="module")
def m():
    import mixture_experts_ffn_moe_amd as m
    return m


@pytest.fixture
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return "cuda"


def dtype_of(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def rng_tensor(seed=SEED, offset=OFFSET):
    signed = lambda v: v - 2 ** 64 if v >= 2 ** 63 else v  # noqa: E731
    return torch.tensor([signed(seed), signed(offset)], dtype=torch.int64, device="cuda")


def shape_of(m, T, H, dtype):
    return m.make_shape(T, H, 1, 1, 32, 1, dtype)


class Step:
    """One training step: inputs on the device, their values in float64, outputs full of NaN between guards."""

    def __init__(self, m, T, H, Is, dtype, p, residual, seed=0):
        g = torch.Generator().manual_seed(seed + 1000 * T + H + Is)
        dt = self.dt = dtype_of(dtype)
        self.T, self.H, self.Is, self.p = T, H, Is, p
        r = lambda *d, s=1.0: (torch.randn(*d, generator=g) * s).to(dt)  # noqa: E731
        self.host = dict(x=r(T, H), w1=r(2 * Is, H, s=1.5 * H ** -0.5), w2=r(H, Is, s=Is ** -0.5),
                         residual=r(T, H) if residual else None, d_out=r(T, H, s=0.1))
        self.d = {k: None if v is None else v.cuda() for k, v in self.host.items()}
        self.rng = rng_tensor()
        self.shape = shape_of(m, T, H, dtype)
        self.ws = torch.empty(m.moe_shared_backward_workspace_size(self.shape, Is), dtype=torch.uint8, device="cuda")
        self.o = {}
        self.all = {}
        for n, dims in dict(gu=(T, 2 * Is), hs=(T, Is), out=(T, H), d_x=(T, H), d_w1s=(2 * Is, H), d_w2s=(H, Is)).items():
            k = int(np.prod(dims))
            buf = torch.full((k + 512,), float("nan"), dtype=torch.float32 if n == "gu" else dt, device="cuda")
            self.all[n] = buf
            self.o[n] = buf[256:256 + k].view(*dims)

    def forward(self, m, stream=None):
        d, o = self.d, self.o
        m.moe_shared_ffn_train(self.shape, self.Is, self.p, self.rng, d["x"], d["w1"], d["w2"], d["residual"], o["gu"],
                               o["hs"], o["out"], stream)

    def backward(self, m, x=True, w=True, stream=None):
        d, o = self.d, self.o
        m.moe_shared_ffn_backward(self.shape, self.Is, self.p, self.rng, d["x"] if w else None, d["w1"] if x else None,
                                  d["w2"], o["gu"], o["hs"] if w else None, d["d_out"], o["d_x"] if x else None,
                                  o["d_w1s"] if w else None, o["d_w2s"] if w else None, self.ws, stream)

    def reference(self):
        h = {k: None if v is None else v.double() for k, v in self.host.items()}
        f = sp.drop_factors(self.T, self.Is, self.p, SEED, OFFSET)
        return sp.ffn(h["x"], h["w1"], h["w2"], h["residual"], h["d_out"], f, self.dt)

    def check(self):
        torch.cuda.synchronize()
        for n, (v, e) in self.reference().items():
            sp.check(n, self.o[n], v, e, self.o[n].dtype)
        for n, b in self.all.items():
            assert torch.isnan(b[:256]).all() and torch.isnan(b[-256:]).all(), n


# (T, H, Is): one token, rows and columns short of a tile, T around the k-tiles of the weights' gradients, and larger
# ones (every launch at every tile size: test_tile_sizes.py)
SIZES = [(1, 64, 32), (2, 192, 96), (15, 64, 64), (63, 128, 32), (64, 256, 128), (65, 64, 160), (127, 320, 96),
         (129, 448, 224), (333, 1024, 352), (700, 1280, 1056), (6200, 64, 1056), (6200, 2048, 96), (33, 3008, 2080)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,Is", SIZES)
def test_training_step(m, dev, T, H, Is, dtype):
    p, residual = (0.0, False) if (T + Is) % 3 == 0 else (0.15, True)
    s = Step(m, T, H, Is, dtype, p, residual)
    s.forward(m)
    s.backward(m)
    s.check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_half_the_outputs(m, dev, dtype):
    """d_x alone and the weights' gradients alone are the bits of the whole call; the others stay untouched."""
    s = Step(m, 130, 256, 96, dtype, 0.1, True)
    s.forward(m)
    s.backward(m)
    whole = {n: s.o[n].clone() for n in ("d_x", "d_w1s", "d_w2s")}
    for n in whole:
        s.o[n].fill_(float("nan"))
    s.backward(m, w=False)
    assert torch.equal(s.o["d_x"], whole["d_x"]) and torch.isnan(s.o["d_w1s"]).all() and torch.isnan(s.o["d_w2s"]).all()
    s.o["d_x"].fill_(float("nan"))
    s.backward(m, x=False)
    assert torch.isnan(s.o["d_x"]).all()
    assert torch.equal(s.o["d_w1s"], whole["d_w1s"]) and torch.equal(s.o["d_w2s"], whole["d_w2s"])


@pytest.mark.gpu
def test_no_tokens(m, dev):
    s = Step(m, 0, 128, 96, "bf16", 0.1, True)
    s.forward(m)
    s.backward(m)
    torch.cuda.synchronize()
    assert (s.o["d_w1s"] == 0).all() and (s.o["d_w2s"] == 0).all()


@pytest.mark.gpu
def test_padding_rows_leave_the_weights_alone(m, dev):
    """Rows with d_out of zero: the weights' gradients are the bits of the batch without their x."""
    s = Step(m, 200, 128, 64, "bf16", 0.0, False)
    s.d["d_out"][77:120] = 0
    s.forward(m)
    s.backward(m)
    first = s.o["d_w1s"].clone(), s.o["d_w2s"].clone()
    assert (s.o["d_x"][77:120] == 0).all()
    s.d["x"][77:120] = 3.0
    s.forward(m)
    s.backward(m)
    assert torch.equal(first[0], s.o["d_w1s"]) and torch.equal(first[1], s.o["d_w2s"])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_bits_on_any_stream_and_in_place(m, dev, dtype):
    s = Step(m, 300, 512, 160, dtype, 0.2, True)
    s.forward(m)
    s.backward(m)
    torch.cuda.synchronize()
    first = {n: t.clone() for n, t in s.o.items()}
    for t in s.o.values():
        t.fill_(float("nan"))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    s.forward(m, st)
    s.backward(m, stream=st)
    st.synchronize()
    for n, t in s.o.items():
        assert torch.equal(t, first[n]), n
    # out in the residual's place
    s.o["out"].copy_(s.d["residual"])
    d = s.d
    m.moe_shared_ffn_train(s.shape, s.Is, s.p, s.rng, d["x"], d["w1"], d["w2"], s.o["out"], s.o["gu"], s.o["hs"], s.o["out"])
    assert torch.equal(s.o["out"], first["out"])


@pytest.mark.gpu
def test_captured_steps_take_the_stream_state_of_their_replay(m, dev):
    """Two steps' graphs in turn, each with its own workspace, the random stream moved between replays."""
    steps = [Step(m, 90, 256, 96, "bf16", 0.3, True, seed=i) for i in range(2)]
    graphs = []
    for s in steps:
        s.forward(m)
        s.backward(m)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.forward(m)
            s.backward(m)
        graphs.append(g)
    for r in range(3):
        for s, g in zip(steps, graphs):
            s.rng.copy_(rng_tensor(SEED, OFFSET + r))
            for t in s.o.values():
                t.fill_(float("nan"))
            g.replay()
        torch.cuda.synchronize()
        for s in steps:
            got = {n: t.clone() for n, t in s.o.items()}
            s.forward(m)
            s.backward(m)
            torch.cuda.synchronize()
            for n, t in s.o.items():
                assert torch.equal(got[n], t), (r, n)


@pytest.mark.gpu
def test_gradients_against_differences(m, dev):
    """d loss / d step along a direction, loss = sum(d_out * out): central differences of the 64-bit forward pass.
    Their own error is of order step^2 = 1e-10; the gradients' bounds add up along the direction."""
    s = Step(m, 21, 128, 96, "f32", 0.25, True)
    s.forward(m)
    s.backward(m)
    torch.cuda.synchronize()
    h = {k: v.double() for k, v in s.host.items()}
    f = sp.drop_factors(s.T, s.Is, s.p, SEED, OFFSET)

    def loss(x, w1, w2):
        z = x @ w1.T
        return float((((torch.nn.functional.silu(z[:, :96]) * z[:, 96:] * f) @ w2.T + h["residual"]) * h["d_out"]).sum())

    ref = s.reference()
    g = torch.Generator().manual_seed(5)
    for name, arg in (("d_x", 0), ("d_w1s", 1), ("d_w2s", 2)):
        args = [h["x"], h["w1"], h["w2"]]
        v = torch.randn(args[arg].shape, generator=g, dtype=torch.float64)
        step = 1e-5
        ends = []
        for sign in (1, -1):
            moved = list(args)
            moved[arg] = args[arg] + sign * step * v
            ends.append(loss(*moved))
        diff = (ends[0] - ends[1]) / (2 * step)
        got = float((s.o[name].double().cpu() * v).sum())
        bound = float((ref[name][1] * v.abs()).sum()) + 1e-6 * max(1.0, abs(diff))
        assert abs(got - diff) <= bound, (name, got, diff, bound)


# ---------------------------------------------------------------- dropout

def test_plain_generator_gives_the_published_blocks():
    """The known answers that the generator's authors publish."""
    one = lambda *v: [np.array([x], np.uint64) for x in v]  # noqa: E731
    for counter, key, want in (
            ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        assert [int(w[0]) for w in sp.philox(one(*counter), list(key))] == list(want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,p,residual", [(1, 64, 0.5, False), (5, 320, 0.3, True), (1000, 448, 0.1, True),
                                            (77, 4096, 0.999, True), (300, 64, 0.0, True), (3, 64, 2e-6, False)])
def test_dropout(m, dev, T, H, p, residual, dtype):
    dt = dtype_of(dtype)
    g = torch.Generator().manual_seed(T)
    y, r, d = (torch.randn(T, H, generator=g).to(dt) for _ in range(3))
    f = sp.drop_factors(T, H, p, SEED, OFFSET)
    y[f == 0] = float("nan")  # a dropped element counts for nothing, whatever it was
    d[f == 0] = float("inf")
    sh, rng = shape_of(m, T, H, dtype), rng_tensor()
    out, dy = (torch.full((T, H), float("nan"), dtype=dt, device="cuda") for _ in range(2))
    m.moe_dropout_add(sh, p, rng, y.cuda(), r.cuda() if residual else None, out)
    m.moe_dropout_backward(sh, p, rng, d.cuda(), dy)
    # the factor is fp32 (one rounding), the product and the sum one each
    for got, v, res in ((out, y, r if residual else None), (dy, d, None)):
        v = torch.where(f == 0, 0.0, v.double()) * f
        e = 2 * sp.F32 * v.abs()
        if res is not None:
            v = v + res.double()
            e = e + sp.F32 * v.abs()
        sp.check("dropout", got, v, e + sp.half_step(dt) * (v.abs() + e), dt)
    # in place, both ways
    a, b = y.cuda(), r.cuda()
    m.moe_dropout_add(sh, p, rng, a, b, a)
    m.moe_dropout_add(sh, p, rng, y.cuda(), b, b)
    assert torch.equal(a, b)


@pytest.mark.gpu
def test_dropout_past_32_bits(m, dev):
    """The counter of the last elements of 2^31 - 2^17 of them; rows near the end against the plain generator."""
    T, H = 32766, 65536
    sh, rng = shape_of(m, T, H, "bf16"), rng_tensor()
    y = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    m.moe_dropout_add(sh, 0.25, rng, y, None, y)
    mask = np.uint64(0xFFFFFFFF)
    for row in (0, 16384, T - 1):
        i = np.arange(row * H // 8, (row + 1) * H // 8, dtype=np.uint64)
        w = sp.philox([i & mask, i >> np.uint64(32), np.full_like(i, OFFSET & 0xFFFFFFFF), np.full_like(i, OFFSET >> 32)],
                      [SEED & 0xFFFFFFFF, SEED >> 32])
        bits = np.stack([(w[e // 2] >> np.uint64(16 * (e % 2))) & np.uint64(0xFFFF) for e in range(8)], 1).reshape(-1)
        assert np.array_equal((y[row] != 0).cpu().numpy(), bits >= 16384)
    share = float((y != 0).float().mean())
    assert abs(share - 0.75) < 1e-4  # standard deviation 1e-5


@pytest.mark.gpu
def test_dropout_in_a_graph(m, dev):
    sh, rng = shape_of(m, 64, 256, "bf16"), rng_tensor()
    y = torch.randn(64, 256, device="cuda").to(torch.bfloat16)
    out, want = torch.empty_like(y), torch.empty_like(y)
    m.moe_dropout_add(sh, 0.5, rng, y, None, out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.moe_dropout_add(sh, 0.5, rng, y, None, out)
    seen = []
    for r in range(3):
        rng.copy_(rng_tensor(SEED + r, OFFSET))
        g.replay()
        m.moe_dropout_add(sh, 0.5, rng, y, None, want)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        seen.append(out.clone())
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


# ---------------------------------------------------------------- refusals (host only: nothing is enqueued)

P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4096 + 8)
BIG = ctypes.c_size_t(1 << 40)


def test_refused_dropouts(m):
    lib, s = m._lib.lib, shape_of(m, 8, 64, "bf16")
    ref = ctypes.byref(s)
    call = lambda p, rng=P, y=P, r=P, out=P: lib.moe_dropout_add(ref, p, rng, y, r, out, None)  # noqa: E731
    for p in (-0.1, 1.0, 1.5, float("nan"), float("inf"), 0.999999):
        assert call(p) == m.MOE_ERR_INVALID_ARG
        assert lib.moe_dropout_backward(ref, p, P, P, P, None) == m.MOE_ERR_INVALID_ARG
    assert call(0.5, rng=None) == m.MOE_ERR_INVALID_ARG
    assert call(0.5, rng=ODD) == m.MOE_ERR_UNSUPPORTED
    assert call(0.5, y=None) == m.MOE_ERR_INVALID_ARG and call(0.5, out=None) == m.MOE_ERR_INVALID_ARG
    assert call(0.5, r=ODD) == m.MOE_ERR_UNSUPPORTED
    assert lib.moe_dropout_add(None, 0.5, P, P, P, P, None) == m.MOE_ERR_INVALID_ARG
    none = shape_of(m, 0, 64, "bf16")
    assert lib.moe_dropout_add(ctypes.byref(none), 0.5, P, P, P, P, None) == m.MOE_OK


def test_refused_training_calls(m):
    lib, s = m._lib.lib, shape_of(m, 8, 64, "bf16")
    ref = ctypes.byref(s)

    def fwd(s=ref, Is=64, p=0.1, rng=P, x=P, w1=P, w2=P, r=P, gu=P, hs=P, out=P):
        return lib.moe_shared_ffn_train(s, Is, p, rng, x, w1, w2, r, gu, hs, out, None)

    def bwd(s=ref, Is=64, p=0.1, rng=P, x=P, w1=P, w2=P, gu=P, hs=P, d=P, dx=P, d1=P, d2=P, ws=P, n=BIG):
        return lib.moe_shared_ffn_backward(s, Is, p, rng, x, w1, w2, gu, hs, d, dx, d1, d2, ws, n, None)

    for call in (fwd, bwd):
        assert call(Is=0) == call(Is=-32) == call(s=None) == call(p=1.0) == call(rng=None) == m.MOE_ERR_INVALID_ARG
        assert call(Is=48) == call(Is=1 << 20) == call(rng=ODD) == m.MOE_ERR_UNSUPPORTED
        wide = shape_of(m, 1, (1 << 20) + 64, "bf16")
        assert call(s=ctypes.byref(wide)) == m.MOE_ERR_UNSUPPORTED
        long = shape_of(m, 1 << 24, 64, "bf16")
        assert call(s=ctypes.byref(long)) == m.MOE_ERR_UNSUPPORTED  # 2 T Is = 2^31
        heavy = shape_of(m, 1, 65536, "f32")
        assert call(s=ctypes.byref(heavy), Is=8192) == m.MOE_ERR_UNSUPPORTED  # fp32 w1s of 4 GiB
    for n in ("x", "w1", "w2", "gu", "hs", "out"):
        assert fwd(**{n: None}) == m.MOE_ERR_INVALID_ARG and fwd(**{n: ODD}) == m.MOE_ERR_UNSUPPORTED
    assert fwd(r=ODD) == m.MOE_ERR_UNSUPPORTED
    for n in ("x", "w1", "w2", "gu", "hs", "d"):
        assert bwd(**{n: None}) == m.MOE_ERR_INVALID_ARG and bwd(**{n: ODD}) == m.MOE_ERR_UNSUPPORTED
    assert bwd(d1=None) == bwd(d2=None) == bwd(dx=None, d1=None, d2=None) == m.MOE_ERR_INVALID_ARG
    assert bwd(dx=ODD) == bwd(d1=ODD) == bwd(d2=ODD) == m.MOE_ERR_UNSUPPORTED
    need = m.moe_shared_backward_workspace_size(s, 64)
    assert need >= 8 * 128 * 2
    assert bwd(n=ctypes.c_size_t(need - 1)) == bwd(ws=None) == m.MOE_ERR_WORKSPACE
    assert bwd(ws=ctypes.c_void_p(4096 + 16)) == m.MOE_ERR_UNSUPPORTED
    assert m.moe_shared_backward_workspace_size(s, 48) == 0


def test_binding_refuses_wrong_tensors(m):
    s = shape_of(m, 8, 64, "bf16")
    host = torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="rng"):
        m.moe_dropout_add(s, 0.5, None, host, None, host)
    with pytest.raises(ValueError, match="GPU tensor"):
        m.moe_dropout_add(s, 0.0, None, host, None, host)
    with pytest.raises(TypeError, match="x"):
        m.moe_shared_ffn_train(s, 64, 0.0, None, 3, host, host, None, host, host, host)
