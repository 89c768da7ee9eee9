"""The request adapters (moe_lora.h) against plain evaluations in 64 bits
(shared_plain.py, which derives the tolerances)."""
import ctypes

import pytest

import shared_plain as sp

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


def ids_of(kind, T, L, g):
    if kind == "none":
        return torch.full((T,), -1, dtype=torch.int32)
    if kind == "one":
        return torch.full((T,), L - 1, dtype=torch.int32)
    if kind == "outside":  # any id without an adapter
        return torch.tensor([-1, L, -2 ** 31, 2 ** 31 - 1, 0], dtype=torch.int64)[torch.randint(0, 5, (T,), generator=g)].to(torch.int32)
    if kind == "runs":
        starts = torch.sort(torch.randint(0, T, (min(T, 5),), generator=g))[0]
        which = torch.randint(-1, L, (min(T, 5) + 1,), generator=g)
        return which[torch.searchsorted(starts, torch.arange(T), right=True)].to(torch.int32)
    ids = torch.randint(0, L, (T,), generator=g)
    ids[torch.rand(T, generator=g) < 0.1] = -1
    return ids.to(torch.int32)


class Call:
    def __init__(self, m, T, H, Is, L, r, dtype, kind, residual=True, seed=0):
        g = torch.Generator().manual_seed(seed + T + 7 * L + r)
        dt = self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.T, self.H, self.Is, self.L, self.r = T, H, Is, L, r
        n = lambda *d, s=1.0: (torch.randn(*d, generator=g) * s).to(dt)  # noqa: E731
        self.host = dict(x=n(T, H), w1=n(2 * Is, H, s=H ** -0.5), w2=n(H, Is, s=Is ** -0.5), a1=n(L, r, H, s=H ** -0.5),
                         b1=n(L, 2 * Is, r, s=r ** -0.5), a2=n(L, r, Is, s=Is ** -0.5), b2=n(L, H, r, s=r ** -0.5),
                         scale=torch.rand(L, generator=g) * 3 - 1, ids=ids_of(kind, T, L, g),
                         residual=n(T, H) if residual else None)
        # adapters that no token names hold NaN
        unused = torch.ones(L, dtype=torch.bool)
        named = self.host["ids"].long()
        unused[named[(named >= 0) & (named < L)]] = False
        for k in ("a1", "b1", "a2", "b2", "scale"):
            self.host[k][unused] = float("nan")
        self.d = {k: None if v is None else v.cuda() for k, v in self.host.items()}
        self.shape, self.lora = m.make_shape(T, H, 1, 1, 32, 1, dtype), m.make_lora(L, r)
        self.ws = torch.full((m.moe_lora_workspace_size(self.shape, Is, self.lora),), 0xFF, dtype=torch.uint8, device="cuda")
        self.guarded = {k: torch.full((T * w + 512,), float("nan"), dtype=dt, device="cuda") for k, w in (("hs", Is), ("out", H))}
        self.hs, self.out = (self.guarded[k][256:256 + T * w].view(T, w) for k, w in (("hs", Is), ("out", H)))

    def w13(self, m, stream=None):
        d = self.d
        m.moe_lora_w13_swiglu(self.shape, self.Is, self.lora, d["x"], d["w1"], d["a1"], d["b1"], d["scale"], d["ids"], self.hs,
                              self.ws, stream)

    def down(self, m, stream=None):
        d = self.d
        m.moe_lora_down(self.shape, self.Is, self.lora, self.hs, d["w2"], d["a2"], d["b2"], d["scale"], d["ids"], d["residual"],
                        self.out, self.ws, stream)

    def both(self, m, stream=None):
        d = self.d
        m.moe_shared_ffn_lora(self.shape, self.Is, self.lora, d["x"], d["w1"], d["w2"], d["a1"], d["b1"], d["a2"], d["b2"],
                              d["scale"], d["ids"], d["residual"], self.hs, self.out, self.ws, stream)

    def check(self):
        torch.cuda.synchronize()
        h = {k: None if v is None else v.double() if v.is_floating_point() else v for k, v in self.host.items()}
        rounded = self.dt == torch.bfloat16
        z = sp.projection(h["x"], h["w1"], h["a1"], h["b1"], h["scale"], h["ids"], self.dt, rounded)
        sp.check("hs", self.hs, *sp.swiglu(*z, self.dt), self.dt)
        hs = self.hs.double().cpu()  # the down projection from the activations as stored
        z = sp.projection(hs, h["w2"], h["a2"], h["b2"], h["scale"], h["ids"], self.dt, rounded)
        sp.check("out", self.out, *sp.add_residual(*z, h["residual"], self.dt), self.dt)
        for k, b in self.guarded.items():
            assert torch.isnan(b[:256]).all() and torch.isnan(b[-256:]).all(), k


# (T, H, Is, L, r): both sides of the small path's last token count, ranks within and past a matrix step, adapters
# that share a row fragment, tokens enough for larger tiles (every tile size: test_tile_sizes.py)
SIZES = [(1, 64, 32, 1, 8), (2, 192, 96, 3, 24), (8, 4096, 768, 64, 16), (15, 320, 160, 4, 128), (16, 2048, 544, 70, 40),
         (17, 64, 32, 5, 8), (31, 192, 96, 7, 16), (33, 448, 160, 40, 24), (77, 256, 128, 3, 64), (130, 1280, 352, 9, 40),
         (300, 512, 288, 64, 16), (257, 64, 64, 2, 128), (1100, 2048, 1056, 12, 32), (6200, 64, 1056, 30, 72),
         (6200, 2048, 96, 1000, 8)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,Is,L,r", SIZES)
def test_both_projections(m, dev, T, H, Is, L, r, dtype):
    c = Call(m, T, H, Is, L, r, dtype, "tokens", residual=T % 2 == 0)
    c.both(m)
    c.check()
    first = c.hs.clone(), c.out.clone()
    c.hs.fill_(float("nan"))
    c.out.fill_(float("nan"))
    c.w13(m)
    c.down(m)
    assert torch.equal(c.hs, first[0]) and torch.equal(c.out, first[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 9, 16, 45, 200])
@pytest.mark.parametrize("kind", ["none", "one", "outside", "runs"])
def test_who_has_which_adapter(m, dev, kind, T, dtype):
    c = Call(m, T, 128, 96, 6, 16, dtype, kind)
    c.both(m)
    c.check()


# 8192 low-rank values (T * r) of adapters of 65536 elements (r * K) are the most that are computed one by one
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,Is,r", [(64, 192, 96, 128), (65, 192, 96, 128), (341, 192, 96, 24), (342, 192, 96, 24),
                                      (1024, 192, 96, 8), (1025, 192, 96, 8), (33, 512, 544, 128), (40, 576, 512, 128)])
@pytest.mark.parametrize("kind", ["tokens", "runs"])
def test_few_and_many_low_rank_values(m, dev, kind, T, H, Is, r, dtype):
    c = Call(m, T, H, Is, 7, r, dtype, kind)
    c.both(m)
    c.check()
    first = c.hs.clone(), c.out.clone()
    c.out.fill_(float("nan"))
    c.down(m)
    assert torch.equal(c.out, first[1])
    mine = c.d["ids"] != 2
    for k in ("a1", "b1", "a2", "b2"):
        c.d[k][2] = float("nan")
    c.d["x"][~mine] = float("inf")
    c.both(m)
    assert torch.equal(c.hs[mine], first[0][mine]) and torch.equal(c.out[mine], first[1][mine])


# about every row of a tile another adapter, in tiles of 64 rows and (fp32) 128, ranks of one matrix step and past it
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,Is,r", [(1000, 64, 800, 16), (1000, 64, 800, 32), (1000, 64, 800, 40), (500, 1024, 1056, 24),
                                      (1000, 1024, 544, 8), (1200, 64, 1312, 16)])
def test_many_adapters_in_a_tile(m, dev, T, H, Is, r, dtype):
    c = Call(m, T, H, Is, 400, r, dtype, "tokens")
    c.both(m)
    c.check()


# the token counts at which the kernels change, K short of a copied row, sixteen rows of W a workgroup
@pytest.mark.gpu
@pytest.mark.parametrize("T", [16, 17, 32, 33])
@pytest.mark.parametrize("H,Is,r", [(320, 160, 8), (192, 96, 128), (4096, 32, 40), (64, 2080, 24)])
def test_few_tokens(m, dev, T, H, Is, r):
    c = Call(m, T, H, Is, 9, r, "bf16", "tokens")
    c.both(m)
    c.check()
    first = c.hs.clone(), c.out.clone()
    mine = c.d["ids"] != 2
    for k in ("a1", "b1", "a2", "b2"):
        c.d[k][2] = float("nan")
    c.d["x"][~mine] = float("inf")
    c.both(m)
    assert torch.equal(c.hs[mine], first[0][mine]) and torch.equal(c.out[mine], first[1][mine])


@pytest.mark.gpu
def test_many_tokens_in_the_plan(m, dev):
    """More tokens than one workgroup sorts."""
    for kind in ("tokens", "runs"):
        c = Call(m, 20011, 64, 32, 100, 8, "bf16", kind)
        c.both(m)
        c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [12, 64, 200])
def test_a_row_is_its_own(m, dev, T):
    """Another request's NaN, its order in the batch and the adapters around it change no bit of a row."""
    c = Call(m, T, 192, 96, 5, 16, "bf16", "tokens")
    c.both(m)
    torch.cuda.synchronize()
    hs, out = c.hs.clone(), c.out.clone()
    mine = c.d["ids"] != 2
    for k in ("a1", "b1", "a2", "b2"):
        c.d[k][2] = float("nan")
    c.d["x"][~mine] = float("inf")
    c.both(m)
    assert torch.equal(c.hs[mine], hs[mine]) and torch.equal(c.out[mine], out[mine])
    order = torch.randperm(T, generator=torch.Generator().manual_seed(3)).cuda()
    o = Call(m, T, 192, 96, 5, 16, "bf16", "tokens")
    for k in ("x", "ids", "residual"):
        o.d[k] = o.d[k][order].contiguous()
    o.both(m)
    assert torch.equal(o.hs, hs[order]) and torch.equal(o.out, out[order])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 150])
def test_stream_graph_and_place(m, dev, T):
    """A call on another stream, replays of two captured calls with workspaces of their own, out in residual's place."""
    calls = [Call(m, T, 256, 96, 8, 16, "bf16", "tokens", seed=s) for s in range(2)]
    want, graphs = [], []
    for c in calls:
        c.both(m)
        torch.cuda.synchronize()
        want.append((c.hs.clone(), c.out.clone()))
        st = torch.cuda.Stream()
        c.out.fill_(float("nan"))
        torch.cuda.synchronize()
        c.both(m, st)
        st.synchronize()
        assert torch.equal(c.out, want[-1][1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.both(m)
        graphs.append(g)
    for r in range(3):
        for c, g in zip(calls, graphs):
            c.hs.fill_(float("nan"))
            c.out.fill_(float("nan"))
            g.replay()
        torch.cuda.synchronize()
        for c, w in zip(calls, want):
            assert torch.equal(c.hs, w[0]) and torch.equal(c.out, w[1]), r
    # a replay takes the ids that the tensor holds then
    c, g = calls[0], graphs[0]
    c.d["ids"].copy_(torch.roll(c.d["ids"], 1))
    g.replay()
    got = c.out.clone()
    c.both(m)
    assert torch.equal(got, c.out)
    d = c.d
    place = d["residual"].clone()
    m.moe_lora_down(c.shape, c.Is, c.lora, c.hs, d["w2"], d["a2"], d["b2"], d["scale"], d["ids"], place, place, c.ws)
    assert torch.equal(place, c.out)


# ---------------------------------------------------------------- refusals (host only: nothing is enqueued)

P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4096 + 8)
BIG = ctypes.c_size_t(1 << 40)


def test_refusals(m):
    lib = m._lib.lib
    s, spec = m.make_shape(8, 64, 1, 1, 32, 1, "bf16"), m.make_lora(4, 16)

    def w13(s=s, Is=64, spec=spec, x=P, w1=P, a1=P, b1=P, scale=P, ids=P, hs=P, ws=P, n=BIG):
        ref = None if spec is None else ctypes.byref(spec)
        return lib.moe_lora_w13_swiglu(ctypes.byref(s), Is, ref, x, w1, a1, b1, scale, ids, hs, ws, n, None)

    def down(s=s, Is=64, spec=spec, hs=P, w2=P, a2=P, b2=P, scale=P, ids=P, r=P, out=P, ws=P, n=BIG):
        ref = None if spec is None else ctypes.byref(spec)
        return lib.moe_lora_down(ctypes.byref(s), Is, ref, hs, w2, a2, b2, scale, ids, r, out, ws, n, None)

    def both(s=s, Is=64, spec=spec, x=P, w1=P, w2=P, a1=P, b1=P, a2=P, b2=P, scale=P, ids=P, r=P, hs=P, out=P, ws=P, n=BIG):
        ref = None if spec is None else ctypes.byref(spec)
        return lib.moe_shared_ffn_lora(ctypes.byref(s), Is, ref, x, w1, w2, a1, b1, a2, b2, scale, ids, r, hs, out, ws, n, None)

    pointers = dict(w13="x w1 a1 b1 scale ids hs", down="hs w2 a2 b2 scale ids out",
                    both="x w1 w2 a1 b1 a2 b2 scale ids hs out")
    for name, call in (("w13", w13), ("down", down), ("both", both)):
        for k in pointers[name].split():
            assert call(**{k: None}) == m.MOE_ERR_INVALID_ARG, k
            assert call(**{k: ODD}) == m.MOE_ERR_UNSUPPORTED, k
        assert call(Is=0) == call(spec=None) == m.MOE_ERR_INVALID_ARG
        for adapters, rank, want in ((0, 16, m.MOE_ERR_INVALID_ARG), (-1, 16, m.MOE_ERR_INVALID_ARG), (4, 0, m.MOE_ERR_INVALID_ARG),
                                     (4, -8, m.MOE_ERR_INVALID_ARG), (1025, 16, m.MOE_ERR_UNSUPPORTED), (4, 12, m.MOE_ERR_UNSUPPORTED),
                                     (4, 136, m.MOE_ERR_UNSUPPORTED)):
            assert call(spec=m.make_lora(adapters, rank)) == want
            assert m.moe_lora_workspace_size(s, 64, m.make_lora(adapters, rank)) == 0
        assert call(Is=40) == m.MOE_ERR_UNSUPPORTED
        wide = m.make_shape(1 << 22, 256, 1, 1, 32, 1, "f32")
        assert call(s=wide) == m.MOE_ERR_UNSUPPORTED  # T * H of 4 GiB
        need = m.moe_lora_workspace_size(s, 64, spec)
        assert call(n=ctypes.c_size_t(need - 1)) == call(ws=None) == m.MOE_ERR_WORKSPACE
        assert call(ws=ctypes.c_void_p(4096 + 16)) == m.MOE_ERR_UNSUPPORTED
        assert call(s=m.make_shape(0, 64, 1, 1, 32, 1, "bf16"), ws=None) == m.MOE_OK
    assert down(r=ODD) == both(r=ODD) == m.MOE_ERR_UNSUPPORTED
    assert m.moe_lora_workspace_size(m.make_shape(0, 64, 1, 1, 32, 1, "bf16"), 64, spec) > 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_workspace_grows_with_the_tokens(m, dtype):
    for H, Is, L, r in ((4096, 768, 64, 16), (64, 32, 3, 128), (2048, 2048, 1000, 8)):
        sizes = [m.moe_lora_workspace_size(m.make_shape(T, H, 1, 1, 32, 1, dtype), Is, m.make_lora(L, r))
                 for T in [*range(1, 1200), *range(1200, 40000, 321)]]
        assert all(0 < a <= b for a, b in zip(sizes, sizes[1:]))


def test_binding_refuses_wrong_tensors(m):
    s, spec = m.make_shape(8, 64, 1, 1, 32, 1, "bf16"), m.make_lora(4, 16)
    t = torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensor"):
        m.moe_lora_w13_swiglu(s, 64, spec, t, t, t, t, t, t, t, t)
    with pytest.raises(ValueError, match="required"):
        m.moe_lora_down(s, 64, spec, None, t, t, t, t, t, None, t, t)
