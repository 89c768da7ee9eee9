"""Every launch of the shared expert's tiled products at every tile size that
it may take: the training step's four launches and the adapters' two, against
plain evaluations in 64 bits (shared_plain.py, which derives the tolerances; on
the GPU here, in float64).  T, H and Is end inside tiles and k-tiles.  Which
tile a launch takes is asked of the library's own estimate on the CPU."""
import shutil

import pytest

import shared_plain as sp
import tile_choice

torch = pytest.importorskip("torch")

# (T, H, Is): tiles of w13, down, d_gu with d_w2, d_x with d_w1, by their place in the order of sizes
TRAIN = {
    "bf16": {(33, 64, 32): (0, 0, 0, 0), (8201, 320, 32): (1, 3, 1, 2), (8197, 64, 288): (4, 1, 2, 1),
             (785, 1344, 992): (2, 2, 3, 3), (2663, 2816, 736): (3, 4, 4, 4), (3909, 3456, 1696): (5, 5, 5, 5)},
    "f32": {(33, 64, 32): (0, 0, 0, 0), (914, 576, 416): (1, 1, 1, 1), (1873, 1728, 928): (2, 2, 2, 2)},
}
# (T, H, Is): tiles of w13 and down
LORA = {
    "bf16": {(33, 64, 32): (0, 0), (8227, 320, 32): (1, 3), (4101, 128, 288): (3, 1), (6553, 640, 96): (2, 4),
             (5510, 192, 608): (4, 2), (8873, 1024, 672): (5, 5), (3666, 1984, 96): (1, 4)},
    "f32": {(33, 64, 32): (0, 0), (8249, 448, 32): (1, 1), (7126, 448, 224): (2, 2)},
}
# (adapters, rank): within and past a matrix step and a row of B in LDS, a few adapters a tile and about one a row
ADAPTERS = [(11, 24), (5, 72), (900, 40), (600, 8)]


@pytest.fixture(scope="module")
def m():
    import mixture_experts_ffn_moe_amd as m
    return m


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_sizes_reach_every_tile(tmp_path, dtype):
    if shutil.which("g++") is None:
        pytest.skip("g++ not installed")
    tiles = tile_choice.Tiles(tmp_path)
    sizes = tiles.sizes(dtype)
    for table, names in ((TRAIN[dtype], ("w13", "down", "d_gu", "d_x")), (LORA[dtype], ("w13", "down"))):
        for dims, places in table.items():
            q = tile_choice.launches(dtype, *dims)
            assert tuple(sizes.index(t) for t in tiles.ask([q[n] for n in names])) == places, dims
        for launch in zip(*table.values()):
            assert set(launch) == set(range(len(sizes)))


def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def maker(seed, dt):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *d, s=1.0: (torch.randn(*d, generator=g, device="cuda") * s).to(dt)


def check(name, got, value, bound, dt):
    sp.check(name, got, value.cpu(), bound.cpu(), dt)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,T,H,Is", [(d, *s) for d in TRAIN for s in TRAIN[d]])
def test_training_step(m, dtype, T, H, Is):
    gpu()
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    n = maker(T + H + Is, dt)
    x, d_out, residual = n(T, H), n(T, H, s=0.1), n(T, H)
    w1, w2 = n(2 * Is, H, s=1.5 * H ** -0.5), n(H, Is, s=Is ** -0.5)
    p, seed, offset = 0.15, 77, 5
    rng = torch.tensor([seed, offset], device="cuda")
    b = m.SharedTrainBuffers(m.make_shape(T, H, 1, 1, 32, 1, dtype), Is, p)
    names = ("gu", "hs", "out", "d_x", "d_w1s", "d_w2s")
    for k in names:
        getattr(b, k).fill_(float("nan"))
    b.forward(x, w1, w2, residual, rng)
    b.backward(x, w1, w2, d_out, rng)
    torch.cuda.synchronize()
    f = sp.drop_factors(T, Is, p, seed, offset).cuda()
    ref = sp.ffn(x.double(), w1.double(), w2.double(), residual.double(), d_out.double(), f, dt)
    for k in names:
        check(k, getattr(b, k), *ref[k], getattr(b, k).dtype)
    # either half of the gradients alone (other tiles may serve it)
    for k in names[3:]:
        getattr(b, k).fill_(float("nan"))
    m.moe_shared_ffn_backward(b.shape, Is, p, rng, None, w1, w2, b.gu, None, d_out, b.d_x, None, None, b.workspace)
    m.moe_shared_ffn_backward(b.shape, Is, p, rng, x, None, w2, b.gu, b.hs, d_out, None, b.d_w1s, b.d_w2s, b.workspace)
    torch.cuda.synchronize()
    for k in names[3:]:
        check(k, getattr(b, k), *ref[k], dt)


@pytest.mark.gpu
@pytest.mark.parametrize("L,r", ADAPTERS)
@pytest.mark.parametrize("dtype,T,H,Is", [(d, *s) for d in LORA for s in LORA[d]])
def test_adapters(m, dtype, T, H, Is, L, r):
    gpu()
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    n = maker(T + H + Is + r, dt)
    x, residual, w1, w2 = n(T, H), n(T, H), n(2 * Is, H, s=H ** -0.5), n(H, Is, s=Is ** -0.5)
    a1, b1, a2, b2 = n(L, r, H, s=H ** -0.5), n(L, 2 * Is, r, s=r ** -0.5), n(L, r, Is, s=Is ** -0.5), n(L, H, r, s=r ** -0.5)
    scale = torch.linspace(-1.0, 2.0, L, device="cuda")
    ids = torch.randint(-1, L, (T,), generator=torch.Generator().manual_seed(r)).to(torch.int32)
    if L == 5:  # runs of a request's tokens, whole tiles of one adapter among them
        ids = torch.sort(ids)[0]
    ids = ids.cuda()
    shape, lora = m.make_shape(T, H, 1, 1, 32, 1, dtype), m.make_lora(L, r)
    ws = torch.empty(m.moe_lora_workspace_size(shape, Is, lora), dtype=torch.uint8, device="cuda")
    hs, out = (torch.full((T, w), float("nan"), dtype=dt, device="cuda") for w in (Is, H))
    m.moe_shared_ffn_lora(shape, Is, lora, x, w1, w2, a1, b1, a2, b2, scale, ids, residual, hs, out, ws)
    torch.cuda.synchronize()
    rounded = dt == torch.bfloat16
    z = sp.projection(x.double(), w1.double(), a1.double(), b1.double(), scale.double(), ids, dt, rounded)
    check("hs", hs, *sp.swiglu(*z, dt), dt)
    z = sp.projection(hs.double(), w2.double(), a2.double(), b2.double(), scale.double(), ids, dt, rounded)
    check("out", out, *sp.add_residual(*z, residual.double(), dt), dt)
