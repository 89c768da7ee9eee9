"""Sums over a million tokens that are exact, and a sort of millions of tokens
by a thousand adapters, every element checked.

The training step's inputs are small integers and every gate is 64, whose
logistic function is 1 in fp32: SiLU(g) = 64 and its derivative 1.  Each
element of u and of d_out w2 has four terms of at most 2, so |u| <= 8,
|d_out w2| <= 4, h = 64 u and dg|du = (dh u | 64 dh) are exact in bf16.  A product
of a weight's gradient is then a whole number of at most 64 (times 64 in d_w2
and for up rows) with mean zero: a sum over T of them deviates by at most
64 sqrt(T) = 65500, and a partial sum would have to lie 250 deviations out to
pass 2^24, below which fp32 adds whole numbers exactly, in any order.  So the
results have to be equal, rounded once: no row or k-tile may be missing."""
import pytest

torch = pytest.importorskip("torch")


def integers(T, H, Is, dt, device, seed=0):
    g = torch.Generator(device=device).manual_seed(seed)
    draw = lambda lo, hi, *d: torch.randint(lo, hi + 1, d, generator=g, device=device, dtype=torch.int8).to(dt)  # noqa: E731
    x, d_out, residual = draw(-2, 2, T, H), draw(-1, 1, T, H), draw(-2, 2, T, H)
    x[:, 0] = 1
    i = torch.arange(Is, device=device)
    w1 = torch.zeros(2 * Is, H, dtype=dt, device=device)
    w2 = torch.zeros(H, Is, dtype=dt, device=device)
    w1[:Is, 0] = 64
    for q in range(4):  # four terms a column, another pattern for either weight
        w1[Is + i, (5 * i + 17 * q) % H] = (1 - 2 * ((i + q) % 2)).to(dt)
        w2[(3 * i + 13 * q) % H, i] = (1 - 2 * ((i // 2 + q) % 2)).to(dt)
    return x, d_out, residual, w1, w2


def exact_rows(x, d_out, residual, w1, w2):
    """(h, dg|du, out, d_x) of some rows, float64."""
    Is = w2.shape[1]
    x, d_out, residual, w1, w2 = (t.double() for t in (x, d_out, residual, w1, w2))
    u, dh = x @ w1[Is:].T, d_out @ w2
    h, d = 64 * u, torch.cat([dh * u, 64 * dh], 1)
    return h, d, h @ w2.T + residual, d @ w1


def rounded(t, dt):
    return t.float().to(dt)


def test_a_missing_k_tile_shows():
    """On the CPU, for 16 columns: without any 64 of the tokens the rounded gradients differ, in bf16 too."""
    T, H, Is = 1048511, 64, 16
    x, d_out, residual, w1, w2 = integers(T, H, Is, torch.float32, "cpu")
    u = x @ w1[Is:].T
    dh = d_out @ w2
    assert float(u.abs().max()) <= 8 and float(dh.abs().max()) <= 4
    h, d = 64 * u, torch.cat([dh * u, 64 * dh], 1)
    for a, b in ((d, x), (d_out, h)):
        whole = a.double().T @ b.double()
        for dt in (torch.bfloat16, torch.float32):
            for start, n in ((0, 64), (T // 2, 64), (T - 63, 63), (T - 1, 1)):
                if dt == torch.bfloat16 and n == 1:
                    continue
                part = whole - a[start:start + n].double().T @ b[start:start + n].double()
                changed = (rounded(whole, dt) != rounded(part, dt)).double().mean()
                assert changed > (0.2 if n > 1 else 0.0), (dt, start, n, float(changed))


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mixture_experts_ffn_moe_amd as m
    return m


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,Is", [(1048511, 64, 1024), (262147, 512, 2080), (70001, 64, 96)])
def test_training_step(m, T, H, Is, dtype):
    """d_w1 and d_w2 over every token, and every row of out and d_x.  At 1048511 tokens 2 T Is is short of 2^31."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x, d_out, residual, w1, w2 = integers(T, H, Is, dt, "cuda")
    b = m.SharedTrainBuffers(m.make_shape(T, H, 1, 1, 32, 1, dtype), Is)
    for t in (b.out, b.d_x, b.d_w1s, b.d_w2s):
        t.fill_(float("nan"))
    b.forward(x, w1, w2, residual)
    b.backward(x, w1, w2, d_out)
    torch.cuda.synchronize()
    d_w1 = torch.zeros(2 * Is, H, dtype=torch.float64, device="cuda")
    d_w2 = torch.zeros(H, Is, dtype=torch.float64, device="cuda")
    for i in range(0, T, 65536):
        rows = slice(i, min(T, i + 65536))
        h, d, out, d_x = exact_rows(x[rows], d_out[rows], residual[rows], w1, w2)
        assert torch.equal(b.hs[rows].double(), h)
        assert torch.equal(b.out[rows], rounded(out, dt)) and torch.equal(b.d_x[rows], rounded(d_x, dt)), i
        d_w1 += d.T.contiguous() @ x[rows].double()
        d_w2 += d_out[rows].double().T.contiguous() @ h
    assert float(d_w1[:Is].abs().max()) < 2 ** 24 and float(torch.maximum(d_w1[Is:].abs().max(), d_w2.abs().max())) < 2 ** 30
    assert torch.equal(b.d_w1s, rounded(d_w1, dt))
    assert torch.equal(b.d_w2s, rounded(d_w2, dt))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [8192, 8193, 100003, 4000037])
def test_every_token_has_its_adapter(m, T, dtype):
    """1024 adapters and ids without one: the first columns of a token's output spell its adapter and its place."""
    H, Is, L, r = 64, 32, 1024, 8
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(T)
    ids = torch.randint(-1, L + 1, (T,), generator=g, device="cuda", dtype=torch.int32)
    ids[T // 3:T // 3 + 3000] = 511  # a request's tokens in a row
    place = torch.arange(T, device="cuda")
    hs = torch.zeros(T, Is, dtype=dt, device="cuda")
    hs[:, 0], hs[:, 1] = 1, (place % 251).to(dt)
    a2, b2 = torch.zeros(L, r, Is, dtype=dt, device="cuda"), torch.zeros(L, H, r, dtype=dt, device="cuda")
    a2[:, 0, 0], a2[:, r - 1, 1] = 1, 1
    number = torch.arange(L, device="cuda")
    b2[:, 0, 0], b2[:, 1, 0], b2[:, 2, r - 1] = (number % 32).to(dt), (number // 32 + 1).to(dt), 1
    w2 = torch.zeros(H, Is, dtype=dt, device="cuda")
    shape, lora = m.make_shape(T, H, 1, 1, 32, 1, dtype), m.make_lora(L, r)
    ws = torch.empty(m.moe_lora_workspace_size(shape, Is, lora), dtype=torch.uint8, device="cuda")
    out = torch.full((T, H), float("nan"), dtype=dt, device="cuda")
    m.moe_lora_down(shape, Is, lora, hs, w2, a2, b2, torch.ones(L, device="cuda"), ids, None, out, ws)
    torch.cuda.synchronize()
    has = (ids >= 0) & (ids < L)
    zero = torch.zeros_like(ids)
    for column, want in ((0, torch.where(has, ids % 32, zero)), (1, torch.where(has, ids // 32 + 1, zero)),
                         (2, torch.where(has, (place % 251).to(torch.int32), zero))):
        assert torch.equal(out[:, column].float(), want.float()), column
    assert (out[:, 3:] == 0).all()
