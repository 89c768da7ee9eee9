"""The 4-bit products and the router's gradients at the ends of their range
(buffers whose byte offsets pass 32 bits, long batches), and outputs that lie
between other data."""
import numpy as np
import pytest

import q4_plain as qp
from helpers import decode_y, to_host_f32
from test_q4 import Case, Rows

torch = pytest.importorskip("torch")
U = 2.0 ** -24
pytestmark = pytest.mark.gpu


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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_products_past_32_bit_offsets(m, dev, dtype):
    """h of just under 2^31 elements: 4.3 GB in bf16, 8.6 GB in fp32."""
    print(f"4-bit products, large h, {dtype}", flush=True)
    c = Case(m, 131071, 64, 64, 8, 2048, 1, dtype, "int4", 64, seed=3, bias=1.0)
    r = c.dense_steps(m)
    R, I, size = c.T * c.k, c.Im, 2 if c.bf16 else 4
    rows = [*range(4), *range(R - 40, R)]
    for at in (2 ** 31, 2 ** 32, 2 ** 33):
        mid = at // (I * size)
        rows += [p for p in range(mid - 2, mid + 3) if p < R]
    rows = np.array(rows)
    offsets, perm = r["offsets"].cpu().numpy(), r["perm"].cpu().numpy()
    assert (np.bincount(r["ids"].cpu().numpy().reshape(-1), minlength=64) == np.diff(offsets)).all()
    ids = (np.searchsorted(offsets, rows, side="right") - 1)[:, None]
    h, dh, y, dy, _, _ = qp.layer(c.x[perm[rows] // c.k], ids, np.ones(ids.shape), c.w1, c.w2, "int4", 64, c.bf16)
    got = to_host_f32(r["h"][torch.from_numpy(rows).to(dev)]).astype(np.float64)
    assert (np.abs(got - h) <= dh + 1e-30).all(), float(np.abs(got - h).max())
    got = decode_y(Rows(c), r["y"], R)[rows].astype(np.float64)
    assert (np.abs(got - y) <= dy + 1e-30).all(), float(np.abs(got - y).max())


def test_weights_gradient_past_32_bit_offsets(m, dev):
    """y of just under 2^31 elements: 4.3 GB and its exponents."""
    print("weights gradient, large y", flush=True)
    T, H, k = 65535, 4096, 8
    R = T * k
    s = m.make_shape(T, H, 64, k, 32, 1, "bf16")
    y = torch.zeros(m.y_nbytes(s, R), dtype=torch.uint8, device=dev)
    half, ye = y[:R * H * 2].view(torch.float16).view(R, H), y[R * H * 2:].view(torch.int8).view(R, H // 256)
    inv = torch.arange(R - 1, -1, -1, dtype=torch.int32, device=dev)  # the first token's rows are the last ones
    g = torch.Generator(device=dev).manual_seed(1)
    d_out = torch.randn(T, H, generator=g, device=dev).bfloat16()
    tokens = torch.tensor([0, T // 2, T - 1], device=dev)
    rows = inv.view(T, k)[tokens].long()
    half[rows] = torch.randn(3, k, H, generator=g, device=dev).half()
    ye[rows] = torch.randint(-20, 20, (3, k, H // 256), generator=g, device=dev, dtype=torch.int8)
    d_w = torch.full((T, k), np.nan, device=dev)
    m.moe_finalize_backward(s, y, inv, d_out, d_w)
    v = torch.ldexp(half[rows].double(), ye[rows].repeat_interleave(256, -1).double()) * d_out[tokens].double()[:, None]
    tol = (9 * 2 + 12) * U * v.abs().sum(-1)  # a lane's terms, 6 steps over the wave, 4 waves
    assert ((d_w[tokens].double() - v.sum(-1)).abs() <= tol).all()
    d_w[tokens] = 0
    assert (d_w == 0).all()


def test_weight_gradient_past_32_bit_offsets(m, dev):
    """x of just under 2^31 elements: 4.3 GB, zero but for a few rows."""
    print("weight gradient, large x", flush=True)
    T, H, E = 524287, 4096, 64
    s = m.make_shape(T, H, E, 1, 32, 1, "bf16")
    g = torch.Generator(device=dev).manual_seed(2)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=dev)
    rows = torch.tensor([0, 262143, 262144, T - 2, T - 1], device=dev)
    x[rows] = torch.randn(5, H, generator=g, device=dev).bfloat16()
    d = torch.randn(T, E, generator=g, device=dev)
    d_wg, d_bias = torch.full((E, H), np.nan, device=dev), torch.full((E,), np.nan, device=dev)
    ws = torch.empty(m.moe_router_grad_workspace_size(s), dtype=torch.uint8, device=dev)
    m.moe_router_weight_grad(s, x, d, None, d_wg, d_bias, ws)
    a, b = d[rows].double(), x[rows].double()
    # five products of three parts each that are not zero; sums of zeros are exact
    assert ((d_wg.double() - a.T @ b).abs() <= 16 * U * (a.abs().T @ b.abs())).all()
    # a thread sums its tokens in turn (16 runs, an eighth of each), then 8 waves and 16 runs
    tb = (T / 16 / 8 + 64 + 8 + 16) * U * d.double().abs().sum(0)
    assert ((d_bias.double() - d.double().sum(0)).abs() <= tb).all()


@pytest.mark.parametrize("mask", ["none", "some"])
@pytest.mark.parametrize("T,H,E", [(16384, 64, 64), (16391, 320, 33), (20000, 192, 7)])
def test_weight_gradient_of_long_batches(m, dev, T, H, E, mask):
    print(f"weight gradient T={T} H={H} E={E} mask={mask}", flush=True)
    g = torch.Generator().manual_seed(T + H)
    x, d = torch.randn(T, H, generator=g).bfloat16(), torch.randn(T, E, generator=g) * 1e-3
    keep = torch.ones(T, dtype=torch.uint8)
    if mask == "some":
        keep = (torch.rand(T, generator=g) < 0.7).to(torch.uint8)
        x[keep == 0], d[keep == 0] = float("nan"), float("-inf")
    s = m.make_shape(T, H, E, 1, 32, 1, "bf16")
    d_wg, d_bias = torch.full((E, H), np.nan, device=dev), torch.full((E,), np.nan, device=dev)
    ws = torch.empty(m.moe_router_grad_workspace_size(s), dtype=torch.uint8, device=dev)
    m.moe_router_weight_grad(s, x.to(dev), d.to(dev), None if mask == "none" else keep.to(dev), d_wg, d_bias, ws)
    a, b = d[keep != 0].double(), x[keep != 0].double()
    # at most 256 runs, each of at least 128 tokens or T / 64 of them; a wave adds three parts of a run's
    # tokens in turn, then 4 waves, then the runs; the parts' magnitudes sum to less than 1.01 times the value's
    run = max(160, T // 64 + 32)
    tol = 1.01 * (3 * run + 4 + 256) * U
    assert ((d_wg.cpu().double() - a.T @ b).abs() <= tol * (a.abs().T @ b.abs())).all()
    assert ((d_bias.cpu().double() - a.sum(0)).abs() <= tol * a.abs().sum(0)).all()


class Between:
    """Tensors in the middle of larger buffers whose rest must stay."""

    def __init__(self, dev):
        self.dev, self.held = dev, []

    def __call__(self, *dims, dtype=torch.float32):
        n = int(np.prod(dims)) * torch.empty(0, dtype=dtype).element_size()
        buf = torch.full((256 + n + 256,), 0x5A, dtype=torch.uint8, device=self.dev)
        self.held.append((buf, n))
        return buf[256:256 + n].view(dtype).view(*dims)

    def check(self):
        torch.cuda.synchronize()
        for i, (buf, n) in enumerate(self.held):
            assert (buf[:256] == 0x5A).all() and (buf[256 + n:] == 0x5A).all(), i


@pytest.mark.parametrize("shape", [(1, 2048, 8, 3, 96, 2, "bf16"), (13, 2048, 9, 8, 32, 1, "bf16"), (53, 192, 5, 3, 96, 2, "bf16"),
                                   (37, 448, 7, 3, 160, 2, "f32"), (200, 320, 64, 8, 32, 1, "bf16")])
def test_q4_writes_its_outputs_only(m, dev, shape):
    print(f"4-bit outputs {shape}", flush=True)
    c = Case(m, *shape, "int4", 32, seed=5)
    T, H, E, k, Im, mu = shape[:6]
    R, b, dt = T * k, Between(dev), c.d["x"].dtype
    ws, out = b(m.moe_workspace_size(c.shape), dtype=torch.uint8), b(T, H, dtype=dt)
    m.moe_forward_q4(c.shape, c.q4, c.d["x"], c.d["wg"], None, *c.d["w"], out, ws)
    b.check()
    steps = c.dense_steps(m)
    h, y = b(R, mu * Im, dtype=dt), b(m.y_nbytes(c.shape, R), dtype=torch.uint8)
    m.moe_q4_w13_swiglu(c.shape, c.q4, c.d["x"], steps["perm"], steps["offsets"], c.d["w"][0], c.d["w"][1], h)
    m.moe_q4_down(c.shape, c.q4, h, steps["offsets"], c.d["w"][2], c.d["w"][3], y)
    z = m.moe_q4_get_sizes(c.shape, c.q4)
    dense = torch.randn(mu, E, 2 * Im, H, device=dev).to(dt), torch.randn(mu, E, H, Im, device=dev).to(dt)
    m.moe_q4_quantize_w13(c.shape, c.q4, dense[0], b(z["w1_codes"], dtype=torch.uint8), b(z["w1_scales"], dtype=torch.uint8))
    m.moe_q4_quantize_down(c.shape, c.q4, dense[1], b(z["w2_codes"], dtype=torch.uint8), b(z["w2_scales"], dtype=torch.uint8))
    b.check()
    assert torch.equal(h, steps["h"]) and torch.equal(y, steps["y"])


@pytest.mark.parametrize("T,H,E,k,dtype", [(1, 64, 1, 1, "bf16"), (77, 448, 33, 5, "bf16"), (333, 320, 64, 8, "f32"),
                                           (4097, 192, 7, 3, "bf16")])
def test_router_gradients_write_their_outputs_only(m, dev, T, H, E, k, dtype):
    print(f"router gradient outputs T={T} H={H} E={E} k={k} {dtype}", flush=True)
    g = torch.Generator(device=dev).manual_seed(T)
    s, b, R = m.make_shape(T, H, E, k, 32, 1, dtype, renormalize=False), Between(dev), T * k
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    logits = torch.randn(T, E, generator=g, device=dev)
    w, ids = torch.softmax(logits, 1).topk(k)
    ids = ids.to(torch.int32).contiguous()
    mask = (torch.rand(T, generator=g, device=dev) < 0.8).to(torch.uint8)
    counts, mean, loss, d = b(E, dtype=torch.int32), b(E), b(1), b(T, E)
    m.moe_balance_loss(s, logits, ids, mask, counts, mean, loss, b(m.moe_balance_workspace_size(s), dtype=torch.uint8))
    y = torch.zeros(m.y_nbytes(s, R), dtype=torch.uint8, device=dev)
    inv = torch.randperm(R, generator=g, device=dev).to(torch.int32)
    d_w, d_wg, d_bias = b(T, k), b(E, H), b(E)
    m.moe_finalize_backward(s, y, inv, torch.randn(T, H, generator=g, device=dev).to(dt), d_w)
    m.moe_route_backward(s, logits, ids, w.contiguous(), mask, counts, d_w, torch.ones(1, device=dev), d)
    m.moe_router_weight_grad(s, torch.randn(T, H, generator=g, device=dev).to(dt), d, mask, d_wg, d_bias,
                             b(m.moe_router_grad_workspace_size(s), dtype=torch.uint8))
    b.check()
    assert (d_w == 0).all() and (d[mask == 0] == 0).all() and torch.isfinite(d_wg).all() and torch.isfinite(d_bias).all()
    assert int(counts.sum()) == k * int(mask.sum())
