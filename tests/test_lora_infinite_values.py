"""Low-rank values at the end of fp32's range and past it.  Whatever the number
of tokens and the kernels that serve them, an infinite value gives the infinity
(or, against a zero of B, the NaN) that B_a v has, and a finite one that bf16
would round to infinity is itself (shared_plain.py derives the tolerances)."""
import pytest

import shared_plain as sp

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# (T, H, Is, r): few tokens; low-rank values by waves and by tiles; ranks of one matrix step and past it; B read
# straight from memory and through LDS, in small and in large tiles
SIZES = [(3, 64, 32, 8), (32, 128, 96, 40), (33, 64, 32, 8), (33, 192, 96, 128), (300, 64, 32, 16), (300, 64, 32, 40),
         (600, 1024, 1056, 24), (1500, 2048, 1056, 16)]


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mixture_experts_ffn_moe_amd as m
    return m


def call(m, T, H, Is, r, dtype, infinite):
    """Both projections; rank 2 of adapter 1 is the large one.  (host values, hs, out)"""
    L, dt = 3, torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(T + r)
    n = lambda *d, s=1.0: (torch.randn(*d, generator=g) * s).to(dt)  # noqa: E731
    h = dict(x=n(T, H), hs=n(T, Is), w1=n(2 * Is, H, s=H ** -0.5), w2=n(H, Is, s=Is ** -0.5), a1=n(L, r, H, s=H ** -0.5),
             b1=n(L, 2 * Is, r, s=r ** -0.5), a2=n(L, r, Is, s=Is ** -0.5), b2=n(L, H, r, s=r ** -0.5),
             scale=torch.tensor([0.5, 1.003, -2.0]), ids=torch.randint(-1, L, (T,), generator=g).to(torch.int32))
    h["ids"][0] = 1
    top = torch.finfo(torch.bfloat16).max
    for x, a, b in (("x", "a1", "b1"), ("hs", "a2", "b2")):
        h[x][:, :2] = 1.0
        h[a][1, 2] = 0.0
        h[a][1, 2, :2] = top if infinite else 0.0  # 1.003 * 2 * top is past fp32's range,
        if not infinite:
            h[a][1, 2, 0] = top  # 1.003 * top is not, but rounds to bf16's infinity
            h[b][1, :, 2] = (h[b][1, :, 2].float() * 2.0 ** -124).to(dt)
    if infinite:  # gate: SiLU(inf) = inf
        h["b1"][1, :Is, 2] = h["b1"][1, :Is, 2].abs() + 0.25
        for b in ("b1", "b2"):
            col = h[b][1, :, 2]
            col[col == 0] = 1.0
        h["b2"][1, 5, 2] = 0.0
    d = {k: v.cuda() for k, v in h.items()}
    shape, lora = m.make_shape(T, H, 1, 1, 32, 1, dtype), m.make_lora(L, r)
    ws = torch.empty(m.moe_lora_workspace_size(shape, Is, lora), dtype=torch.uint8, device="cuda")
    hs, out = torch.empty(T, Is, dtype=dt, device="cuda"), torch.empty(T, H, dtype=dt, device="cuda")
    m.moe_lora_w13_swiglu(shape, Is, lora, d["x"], d["w1"], d["a1"], d["b1"], d["scale"], d["ids"], hs, ws)
    m.moe_lora_down(shape, Is, lora, d["hs"], d["w2"], d["a2"], d["b2"], d["scale"], d["ids"], None, out, ws)
    torch.cuda.synchronize()
    return h, hs, out, dt


def reference(h, dt):
    v = {k: t.double() if t.is_floating_point() else t for k, t in h.items()}
    z = sp.projection(v["x"], v["w1"], v["a1"], v["b1"], v["scale"], v["ids"], dt, dt == torch.bfloat16)
    y = sp.projection(v["hs"], v["w2"], v["a2"], v["b2"], v["scale"], v["ids"], dt, dt == torch.bfloat16)
    return sp.swiglu(*z, dt), sp.add_residual(*y, None, dt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,Is,r", SIZES)
def test_infinite_values_stay_infinite(m, T, H, Is, r, dtype):
    h, hs, out, dt = call(m, T, H, Is, r, dtype, True)
    own = h["ids"] == 1
    inf = torch.tensor(float("inf"))
    up = (inf * h["b1"][1, Is:, 2].float().sign()).expand(int(own.sum()), Is)
    assert torch.equal(hs.cpu()[own].float(), up)
    down = (inf * h["b2"][1, :, 2].float().sign()).expand(int(own.sum()), H)
    got = out.cpu()[own].float()
    assert torch.isnan(down[:, 5]).all() and torch.isnan(got[:, 5]).all()  # infinity times zero
    rest = torch.arange(H) != 5
    assert torch.equal(got[:, rest], down[:, rest])
    # the other tokens' rows
    (v, e), (w, f) = reference({k: t[~own] if k in ("x", "hs", "ids") else t for k, t in h.items()}, dt)
    sp.check("hs", hs.cpu()[~own], v, e, dt)
    sp.check("out", out.cpu()[~own], w, f, dt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,Is,r", SIZES)
def test_finite_values_past_the_type(m, T, H, Is, r, dtype):
    h, hs, out, dt = call(m, T, H, Is, r, dtype, False)
    (v, e), (w, f) = reference(h, dt)
    assert torch.isfinite(hs).all() and torch.isfinite(out).all()
    sp.check("hs", hs, v, e, dt)
    sp.check("out", out, w, f, dt)
