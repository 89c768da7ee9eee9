"""The shared expert's training step and its adapters at the ends of their
range: buffers whose offsets pass 32 bits, tens of millions of tokens.  Rows
drawn from both ends and between are checked against the 64-bit plain forms
(shared_plain.py), sums over all rows against chunked 64-bit sums on the GPU."""
import pytest

import shared_plain as sp

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import mixture_experts_ffn_moe_amd as m
    return m


@pytest.fixture
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return "cuda"


def rows_of(T):
    return torch.tensor(sorted({0, 1, 31, 255, 8191, 8192, T // 3, T // 2 + 7, T - 300, T - 33, T - 2, T - 1}))


def randn(shape, seed, dt, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(shape, dtype=dt, device="cuda")
    flat = t.view(-1, shape[-1])
    for i in range(0, flat.shape[0], 1 << 20):
        n = min(1 << 20, flat.shape[0] - i)
        flat[i:i + n] = (torch.randn(n, shape[-1], generator=g, device="cuda") * scale).to(dt)
    return t


def test_training_step_past_32_bits(m, dev):
    """gu of 8.6 GB, d_gu of 4.3 GB: 2 T Is = 2^31 - 2^19."""
    T, H, Is, dt = 1048320, 64, 1024, torch.bfloat16
    shape = m.make_shape(T, H, 1, 1, 32, 1, "bf16")
    x, d_out, res = randn((T, H), 1, dt), randn((T, H), 2, dt, 0.1), randn((T, H), 3, dt)
    w1, w2 = randn((2 * Is, H), 4, dt, 0.2), randn((H, Is), 5, dt, 0.05)
    b = m.SharedTrainBuffers(shape, Is, 0.0)
    b.forward(x, w1, w2, res)
    b.backward(x, w1, w2, d_out)
    torch.cuda.synchronize()
    rows = rows_of(T).cuda()
    h = lambda t: t[rows].double().cpu()  # noqa: E731
    ref = sp.ffn(h(x), w1.double().cpu(), w2.double().cpu(), h(res), h(d_out), torch.ones(len(rows), Is, dtype=torch.float64), dt)
    for name, got in (("gu", b.gu), ("hs", b.hs), ("out", b.out), ("d_x", b.d_x)):
        sp.check(name, got[rows], *ref[name], got.dtype)
    # the weights' gradients: every row's part, operands as the step stored them
    d_w2 = torch.zeros(H, Is, dtype=torch.float64, device="cuda")
    d_w1 = torch.zeros(2 * Is, H, dtype=torch.float64, device="cuda")
    mag1, mag2 = torch.zeros_like(d_w1), torch.zeros_like(d_w2)
    w2d = w2.double()
    for i in range(0, T, 65520):
        xs, ds, hs, gu = (t[i:i + 65520].double() for t in (x, d_out, b.hs, b.gu))
        d_w2 += ds.T.contiguous() @ hs
        mag2 += ds.abs().T.contiguous() @ hs.abs()
        s = torch.sigmoid(gu[:, :Is])
        dh = ds @ w2d
        d = torch.cat([dh * gu[:, Is:] * s * (1 + gu[:, :Is] * (1 - s)), dh * gu[:, :Is] * s], 1)
        d_w1 += d.T.contiguous() @ xs
        mag1 += d.abs().T.contiguous() @ xs.abs()
    # T products in fp32 sums: at most (T + 4) 2^-24 of their magnitudes if every addition rounds the same way;
    # rounded either way their errors add like a walk of T steps, 8 sqrt(T) 2^-24 is eight deviations.  d_gu's own
    # rounding is a half step of each product, and adds up likewise; the result is rounded once.
    u = sp.half_step(dt)
    walk = 8 * T ** 0.5 * sp.F32
    for got, want, mag, operand in ((b.d_w2s, d_w2, mag2, 0.0), (b.d_w1s, d_w1, mag1, 8 * u / T ** 0.5 + 64 * sp.F32)):
        err = (got.double() - want).abs()
        assert (err <= u * want.abs() + (walk + operand) * mag).all(), float((err / mag).max())


def test_adapters_of_tens_of_millions_of_tokens(m, dev):
    """x of 4.2 GB, rows gathered with offsets up to 2^32; thousands of workgroups in the sort."""
    T, H, Is, L, r, dt = 33_000_001, 64, 32, 5, 8, torch.bfloat16
    shape, lora = m.make_shape(T, H, 1, 1, 32, 1, "bf16"), m.make_lora(L, r)
    x = randn((T, H), 1, dt)
    w1, w2 = randn((2 * Is, H), 4, dt, 0.1), randn((H, Is), 5, dt, 0.2)
    a1, b1 = randn((L, r, H), 6, dt, 0.1), randn((L, 2 * Is, r), 7, dt, 0.3)
    a2, b2 = randn((L, r, Is), 8, dt, 0.2), randn((L, H, r), 9, dt, 0.3)
    scale = torch.rand(L, device="cuda") + 0.5
    g = torch.Generator(device="cuda").manual_seed(10)
    ids = torch.randint(-1, L, (T,), generator=g, device="cuda", dtype=torch.int32)
    hs, out = torch.empty(T, Is, dtype=dt, device="cuda"), torch.empty(T, H, dtype=dt, device="cuda")
    ws = torch.empty(m.moe_lora_workspace_size(shape, Is, lora), dtype=torch.uint8, device="cuda")
    m.moe_shared_ffn_lora(shape, Is, lora, x, w1, w2, a1, b1, a2, b2, scale, ids, None, hs, out, ws)
    torch.cuda.synchronize()
    rows = rows_of(T).cuda()
    h = lambda t: t.double().cpu()  # noqa: E731
    z = sp.projection(h(x[rows]), h(w1), h(a1), h(b1), h(scale), ids[rows].cpu(), dt, True)
    sp.check("hs", hs[rows], *sp.swiglu(*z, dt), dt)
    z = sp.projection(h(hs[rows]), h(w2), h(a2), h(b2), h(scale), ids[rows].cpu(), dt, True)
    sp.check("out", out[rows], *sp.add_residual(*z, None, dt), dt)
    # every token was written, and written once: the same call of the second half alone gives the same rows
    half = T // 2
    shape2 = m.make_shape(T - half, H, 1, 1, 32, 1, "bf16")
    ws2 = torch.empty(m.moe_lora_workspace_size(shape2, Is, lora), dtype=torch.uint8, device="cuda")
    hs2 = torch.empty(T - half, Is, dtype=dt, device="cuda")
    # (rows from `half` on start at a multiple of 16 bytes: 64 columns of 2 bytes; ids are copied)
    m.moe_lora_w13_swiglu(shape2, Is, lora, x[half:], w1, a1, b1, scale, ids[half:].clone(), hs2, ws2)
    assert torch.equal(hs2, hs[half:])
