"""The balance loss with its counts, and the router's gradients
(moe_router_grad.h), against plain evaluations in 64 bits.

Tolerances, from the arithmetic of the kernels (u = 2^-24, half a step of
fp32): a probability is expf of an argument rounded once (at most 16 in size:
16 u absolute, so relative in the result), expf itself within 2 u, a sum of
at most 64 positive terms in at most 10 additions, a reciprocal and a
product: below 32 u = 2e-6 relative.  Everything else is a sum of known
terms: its error is bounded by the number of roundings on a term's way times
u times the sum of the terms' magnitudes."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

U = 2.0 ** -24
P_TOL = 32 * U


@pytest.fixture(scope="module")
def m():
    import mixture_experts_ffn_moe_amd as m
    return m


def gpu(fn):
    return pytest.mark.gpu(fn)


@pytest.fixture
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return "cuda"


# ---------------------------------------------------------------- inputs and the plain evaluation

def make(T, E, k, renorm, mask, seed, garbage=True):
    """Router outputs of T tokens, in numpy; masked rows hold garbage."""
    rng = np.random.default_rng(seed)
    logits = (rng.standard_normal((T, E)) * 1.5 + rng.standard_normal(E)).astype(np.float32)
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    sel = np.take_along_axis(logits, ids, 1).astype(np.float64)
    den = np.exp(sel - sel[:, :1]).sum(1) if renorm else np.exp(logits.astype(np.float64) - sel[:, :1]).sum(1)
    w = (np.exp(sel - sel[:, :1]) / den[:, None]).astype(np.float32)
    d_w = (rng.standard_normal((T, k)) * 1e-2).astype(np.float32)
    keep = {"none": np.ones(T), "some": rng.random(T) < 0.7, "all": np.zeros(T)}[mask].astype(np.uint8)
    pad = keep == 0
    if garbage:
        logits[pad], d_w[pad], w[pad], ids[pad] = np.nan, np.inf, np.nan, 1 << 30
    return dict(logits=logits, ids=ids, w=w, d_w=d_w, keep=keep, mask=None if mask == "none" else keep)


def plain_loss(c, E, k):
    ok = c["keep"] != 0
    n = int(ok.sum())
    if n == 0:
        return np.zeros(E, np.int64), np.zeros(E), 0.0, np.zeros((len(ok), E))
    L = c["logits"][ok].astype(np.float64)
    mx = L.max(1, keepdims=True)
    mx[np.isinf(mx)] = 0.0
    ex = np.exp(L - mx)
    s = ex.sum(1, keepdims=True)
    p = ex / np.where(s > 0, s, 1.0)
    counts = np.bincount(c["ids"][ok].ravel(), minlength=E)
    full = np.zeros((len(ok), E))
    full[ok] = p
    return counts, p.sum(0) / n, E * float((counts / (n * k) * p.sum(0) / n).sum()), full


def plain_backward(c, E, k, renorm, d_loss, use_w):
    """d_logits and, element by element, the sum of the magnitudes of its terms."""
    counts, _, _, p = plain_loss(c, E, k)
    T = len(p)
    ok = c["keep"] != 0
    g, size = np.zeros((T, E)), np.zeros((T, E))
    if d_loss is not None and ok.any():
        f = counts / counts.sum()
        co = d_loss * E / ok.sum()
        fp = (p * f).sum(1, keepdims=True)
        g += co * p * (f - fp)
        size += abs(co) * p * (f + fp)
    if use_w:
        for t in np.nonzero(ok)[0]:
            w, dw = c["w"][t].astype(np.float64), c["d_w"][t].astype(np.float64)
            dot, adot = (w * dw).sum(), (w * np.abs(dw)).sum()
            if renorm:
                g[t, c["ids"][t]] += w * (dw - dot)
                size[t, c["ids"][t]] += w * (np.abs(dw) + adot)
            else:
                one = np.zeros(E)
                one[c["ids"][t]] = dw
                g[t] += p[t] * (one - dot)
                size[t] += p[t] * (np.abs(one) + adot)
    return g, size


def to(a, dev):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def run_loss(m, s, c, dev, stream=None):
    T, E = s.T, s.E
    counts = torch.full((E,), -7, dtype=torch.int32, device=dev)
    mean, loss = torch.full((E,), np.nan, device=dev), torch.full((1,), np.nan, device=dev)
    ws = torch.empty(m.moe_balance_workspace_size(s), dtype=torch.uint8, device=dev)
    m.moe_balance_loss(s, to(c["logits"], dev), to(c["ids"], dev), to(c["mask"], dev), counts, mean, loss, ws, stream)
    torch.cuda.synchronize()
    return counts, mean, loss


SHAPES = [(1, 1, 1), (1, 64, 8), (2, 2, 1), (3, 7, 7), (63, 16, 3), (64, 17, 4), (65, 33, 8), (300, 64, 64),
          (1000, 48, 6), (4096, 64, 8), (20000, 64, 20)]


@gpu
@pytest.mark.parametrize("mask", ["none", "some", "all"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_loss_and_gradient(m, dev, T, E, k, renorm, mask):
    print(f"balance T={T} E={E} k={k} renorm={renorm} mask={mask}", flush=True)
    c = make(T, E, k, renorm, mask, seed=T + E)
    s = m.make_shape(T, 64, E, k, 32, 1, "bf16", renorm)
    counts, mean, loss = run_loss(m, s, c, dev)
    rc, rm, rl, _ = plain_loss(c, E, k)
    assert np.array_equal(counts.cpu().numpy(), rc)
    assert (np.abs(mean.cpu().numpy() - rm) <= P_TOL * rm).all()
    assert abs(float(loss) - rl) <= P_TOL * rl
    for d_loss, use_w in ((0.3, True), (0.3, False), (None, True)):
        d = torch.full((T, E), np.nan, device=dev)
        m.moe_route_backward(s, to(c["logits"], dev), to(c["ids"], dev), to(c["w"], dev), to(c["mask"], dev), counts,
                             to(c["d_w"], dev) if use_w else None,
                             None if d_loss is None else torch.tensor([d_loss], device=dev), d)
        g, size = plain_backward(c, E, k, renorm, np.float32(d_loss) if d_loss else None, use_w)
        got = d.cpu().numpy()
        # two probabilities (the factor and the sum over f p), a dot of k terms, a handful of products
        tol = (2 * P_TOL + (k / 16 + 12) * U) * size
        assert (np.abs(got - g) <= tol + 1e-38).all(), float((np.abs(got - g) - tol).max())
        assert (got[c["keep"] == 0] == 0).all()


@gpu
def test_large_and_infinite_logits(m, dev):
    """Logits near the type's largest value, switched-off experts (-inf), a row of nothing but -inf."""
    T, E, k = 40, 10, 3
    c = make(T, E, k, False, "some", 3)
    c["keep"][:4] = 1
    for t in range(4):  # rows that were padding get values
        c["logits"][t] = np.arange(E)
        c["ids"][t], c["w"][t], c["d_w"][t] = [9, 8, 7], [0.5, 0.2, 0.1], [1e-2, 2e-2, -1e-2]
    c["logits"][0, 2:7] = -np.inf
    c["logits"][1] = np.linspace(-3.0e38, 3.3e38, E).astype(np.float32)
    c["logits"][2] = -np.inf
    c["logits"][3] = np.finfo(np.float32).min
    s = m.make_shape(T, 64, E, k, 32, 1, "bf16", False)
    counts, mean, loss = run_loss(m, s, c, dev)
    with np.errstate(invalid="ignore", over="ignore"):
        rc, rm, rl, _ = plain_loss(c, E, k)
        g, size = plain_backward(c, E, k, False, 0.5, True)
    assert np.array_equal(counts.cpu().numpy(), rc)
    assert (np.abs(mean.cpu().numpy() - rm) <= P_TOL * rm).all() and abs(float(loss) - rl) <= P_TOL * rl
    d = torch.empty(T, E, device=dev)
    m.moe_route_backward(s, to(c["logits"], dev), to(c["ids"], dev), to(c["w"], dev), to(c["mask"], dev), counts,
                         to(c["d_w"], dev), torch.tensor([0.5], device=dev), d)
    assert (np.abs(d.cpu().numpy() - g) <= (2 * P_TOL + 13 * U) * size + 1e-38).all()
    assert (d[2] == 0).all()


@gpu
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(m, dev, renorm):
    """The gradient of the plain objective by central differences in 64 bits, counts and selection fixed."""
    T, E, k = 9, 11, 3
    c = make(T, E, k, renorm, "some", 8, garbage=False)
    ok = c["keep"] != 0
    s = m.make_shape(T, 64, E, k, 32, 1, "bf16", renorm)
    counts, _, _ = run_loss(m, s, c, dev)
    d_loss = 0.25
    f = counts.cpu().numpy() / counts.cpu().numpy().sum()

    def objective(L):
        ex = np.exp(L - L.max(1, keepdims=True))
        p = ex / ex.sum(1, keepdims=True)
        q = np.take_along_axis(p, c["ids"].astype(np.int64), 1)
        w = q / q.sum(1, keepdims=True) if renorm else q
        return (w * c["d_w"])[ok].sum() + d_loss * E * (f * p[ok].mean(0)).sum()

    L = c["logits"].astype(np.float64)
    h = 1e-5
    num = np.zeros((T, E))
    for t in range(T):
        for e in range(E):
            a, b = L.copy(), L.copy()
            a[t, e] += h
            b[t, e] -= h
            num[t, e] = (objective(a) - objective(b)) / (2 * h)
    d = torch.empty(T, E, device=dev)
    m.moe_route_backward(s, to(c["logits"], dev), to(c["ids"], dev), to(c["w"], dev), to(c["mask"], dev), counts,
                         to(c["d_w"], dev), torch.tensor([d_loss], device=dev), d)
    # differences: h^2 / 6 times a third derivative below 1, and 1e-16 / h of cancellation; topk_w was rounded to fp32
    assert np.abs(d.cpu().numpy() - num).max() <= 1e-9 + 1e-6 * np.abs(num).max()


@gpu
@pytest.mark.parametrize("T", [0])
def test_no_tokens(m, dev, T):
    s = m.make_shape(0, 128, 6, 2, 32, 1, "bf16")
    e = lambda *sh, dt=torch.float32: torch.empty(*sh, dtype=dt, device=dev)  # noqa: E731
    counts, mean, loss = e(6, dt=torch.int32).fill_(5), e(6).fill_(5), e(1).fill_(5)
    ws = e(m.moe_balance_workspace_size(s), dt=torch.uint8)
    m.moe_balance_loss(s, e(0, 6), e(0, 2, dt=torch.int32), None, counts, mean, loss, ws)
    d_wg, d_bias = e(6, 128).fill_(5), e(6).fill_(5)
    m.moe_router_weight_grad(s, e(0, 128, dt=torch.bfloat16), e(0, 6), None, d_wg, d_bias,
                             e(m.moe_router_grad_workspace_size(s), dt=torch.uint8))
    m.moe_route_backward(s, e(0, 6), e(0, 2, dt=torch.int32), e(0, 2), None, counts, e(0, 2), None, e(0, 6))
    m.moe_finalize_backward(s, e(0, dt=torch.uint8), e(0, dt=torch.int32), e(0, 128, dt=torch.bfloat16), e(0, 2))
    torch.cuda.synchronize()
    for t in (counts, mean, loss, d_wg, d_bias):
        assert (t == 0).all()


# ---------------------------------------------------------------- the weight's gradient

def wgrad_inputs(T, H, E, dtype, mask, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g).to(dtype)
    d = torch.randn(T, E, generator=g) * torch.exp(torch.randn(T, 1, generator=g) * 3) * 1e-3
    keep = torch.ones(T, dtype=torch.uint8) if mask == "none" else (torch.rand(T, generator=g) < 0.7).to(torch.uint8)
    if mask == "all":
        keep.zero_()
    x[keep == 0], d[keep == 0] = float("nan"), float("inf")
    return x, d, keep


@gpu
@pytest.mark.parametrize("mask", ["none", "some", "all"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,E", [(1, 64, 1), (3, 64, 64), (31, 192, 5), (64, 128, 16), (65, 448, 17), (500, 320, 40),
                                   (1025, 4096, 64), (3000, 64, 33)])
def test_router_weight_grad(m, dev, T, H, E, dtype, mask):
    print(f"weight gradient T={T} H={H} E={E} {dtype} mask={mask}", flush=True)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x, d, keep = wgrad_inputs(T, H, E, dt, mask, T + H + E)
    s = m.make_shape(T, H, E, 1, 32, 1, dtype)
    ws = torch.empty(m.moe_router_grad_workspace_size(s), dtype=torch.uint8, device=dev)
    d_wg, d_bias = torch.full((E, H), np.nan, device=dev), torch.full((E,), np.nan, device=dev)
    mk = None if mask == "none" else keep.to(dev)
    m.moe_router_weight_grad(s, x.to(dev), d.to(dev), mk, d_wg, d_bias, ws)
    ok = keep != 0
    a, b = d[ok].double(), x[ok].double()
    ref, size = a.T @ b, a.T.abs() @ b.abs()
    # a product within u, a wave's sum of at most T/16 + 32 terms, then 16 waves and at most 256 runs in
    # sequences of at most 4 and 256 additions; half of the additions' bound is never reached, none is assumed
    tol = (T / 16 + 32 + 4 + min(256, T // 64 + 1) + 2) * U * size
    assert ((d_wg.cpu().double() - ref).abs() <= tol).all()
    tb = (T / 16 + 32 + 18 + min(256, T // 64 + 1)) * U * a.abs().sum(0)
    assert ((d_bias.cpu().double() - a.sum(0)).abs() <= tb).all()
    again = torch.empty_like(d_wg)
    m.moe_router_weight_grad(s, x.to(dev), d.to(dev), mk, again, None, ws)  # no bias wanted
    assert torch.equal(again, d_wg)


# ---------------------------------------------------------------- the routing weights' gradient

def y_of(y, H):
    """A y buffer of the bf16 layers (block-scaled half) holding y rounded, and the values it stands for."""
    R = y.shape[0]
    B = -(-H // 256)
    pad = torch.nn.functional.pad(y, (0, B * 256 - H)).view(R, B, 256).abs().amax(-1)
    e = torch.where(pad > 0, torch.frexp(pad)[1] - 15, torch.zeros((), dtype=torch.int32)).clamp(-128, 127)
    full = e.repeat_interleave(256, 1)[:, :H]
    half = torch.ldexp(y.double(), -full).to(torch.float16)
    buf = torch.cat([half.view(torch.uint8).reshape(-1), e.to(torch.int8).view(torch.uint8).reshape(-1)])
    return buf, torch.ldexp(half.double(), full)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,k", [(1, 64, 1), (1, 4096, 8), (5, 192, 2), (7, 320, 3), (33, 448, 5), (64, 2048, 15),
                                   (200, 2112, 8), (40, 256, 64)])
def test_finalize_backward(m, dev, T, H, k, dtype):
    print(f"finalize backward T={T} H={H} k={k} {dtype}", flush=True)
    g = torch.Generator().manual_seed(T + H + k)
    R = T * k
    # rows of very different size, one of them all zero
    y = torch.randn(R, H, generator=g) * torch.exp(torch.randn(R, 1, generator=g) * 4)
    y[R // 2] = 0
    inv = torch.randperm(R, generator=g).to(torch.int32)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    d_out = torch.randn(T, H, generator=g).to(dt)
    buf, val = y_of(y, H) if dtype == "bf16" else (y, y.double())
    s = m.make_shape(T, H, 64, k, 32, 1, dtype)
    d_w = torch.full((T, k), np.nan, device=dev)
    m.moe_finalize_backward(s, buf.to(dev), inv.to(dev), d_out.to(dev), d_w)
    rows = val[inv.long()].view(T, k, H)
    ref, size = (rows * d_out.double()[:, None]).sum(-1), (rows.abs() * d_out.double().abs()[:, None]).sum(-1)
    tol = (9 * (-(-H // 2048)) + 12) * U * size  # a lane's terms, 6 steps over the wave, 4 waves
    assert ((d_w.cpu().double() - ref).abs() <= tol).all()


# ---------------------------------------------------------------- together, streams, graphs

@gpu
def test_backward_of_a_routed_layer(m, dev):
    """The three calls from the output's gradient to the router's parameters,
    after a step-wise layer, against differences of that layer in 64 bits
    with the routing held fixed."""
    T, H, E, k, Im = 24, 128, 6, 2, 64
    g = torch.Generator().manual_seed(4)
    x, wg, bias = torch.randn(T, H, generator=g), torch.randn(E, H, generator=g) * 0.1, torch.randn(E, generator=g) * 0.2
    w1, w2 = torch.randn(1, E, 2 * Im, H, generator=g) * 0.1, torch.randn(1, E, H, Im, generator=g) * 0.1
    d_out = torch.randn(T, H, generator=g)
    s = m.make_shape(T, H, E, k, Im, 1, "f32")
    buf = m.MoELayerBuffers(s)
    buf.forward(x.to(dev), wg.to(dev), bias.to(dev), w1.to(dev), w2.to(dev))
    v = buf.views()
    ids = v["ids"].cpu().long()
    e = lambda *sh: torch.empty(*sh, device=dev)  # noqa: E731
    counts, mean, loss, alpha = torch.empty(E, dtype=torch.int32, device=dev), e(E), e(1), torch.tensor([0.1], device=dev)
    m.moe_balance_loss(s, v["logits"], v["ids"], None, counts, mean, loss,
                       torch.empty(m.moe_balance_workspace_size(s), dtype=torch.uint8, device=dev))
    assert torch.equal(counts, v["counts"])
    d_w, d_logits, d_wg, d_bias = e(T, k), e(T, E), e(E, H), e(E)
    m.moe_finalize_backward(s, v["y"], v["inv"], d_out.to(dev), d_w)
    m.moe_route_backward(s, v["logits"], v["ids"], v["w"], None, counts, d_w, alpha, d_logits)
    m.moe_router_weight_grad(s, x.to(dev), d_logits, None, d_wg, d_bias,
                             torch.empty(m.moe_router_grad_workspace_size(s), dtype=torch.uint8, device=dev))
    X, W1, W2 = x.double(), w1[0].double(), w2[0].double()
    a = torch.einsum("th,eih->tei", X, W1)
    y = torch.einsum("tei,ehi->teh", torch.nn.functional.silu(a[..., :Im]) * a[..., Im:], W2)
    yt = torch.gather(y, 1, ids[:, :, None].expand(T, k, H))
    f = counts.cpu().double() / (T * k)

    def objective(G, b):
        p = torch.softmax(X @ G.T + b, 1)
        q = torch.gather(p, 1, ids)
        return ((q / q.sum(1, keepdim=True))[:, :, None] * yt * d_out.double()[:, None]).sum() + 0.1 * E * (f * p.mean(0)).sum()

    h = 1e-5
    num_b = torch.stack([(objective(wg.double(), bias.double() + h * o) - objective(wg.double(), bias.double() - h * o)) / (2 * h)
                         for o in torch.eye(E, dtype=torch.float64)])
    G = wg.double().requires_grad_()
    B = bias.double().requires_grad_()
    objective(G, B).backward()
    assert (num_b - B.grad).abs().max() <= 1e-7 * B.grad.abs().max() + 1e-8  # the objective's own gradient by differences
    # y is within the fp32 layer's 1e-5 of the plain one, everything after it within a few u
    assert (d_bias.cpu() - B.grad).abs().max() <= 2e-5 * B.grad.abs().max()
    assert (d_wg.cpu() - G.grad).abs().max() <= 2e-5 * G.grad.abs().max()


@gpu
def test_streams_and_graph_replay(m, dev):
    """The same bits on another stream and from a captured graph, replayed
    several times with new inputs in the same buffers and eager work between."""
    T, H, E, k = 700, 192, 20, 4
    s = m.make_shape(T, H, E, k, 32, 1, "bf16")
    R = T * k
    e = lambda *sh, dt=torch.float32: torch.empty(*sh, dtype=dt, device=dev)  # noqa: E731
    b = dict(logits=e(T, E), ids=e(T, k, dt=torch.int32), w=e(T, k), mask=e(T, dt=torch.uint8), x=e(T, H, dt=torch.bfloat16),
             y=e(m.y_nbytes(s, R), dt=torch.uint8), inv=e(R, dt=torch.int32), d_out=e(T, H, dt=torch.bfloat16),
             d_loss=torch.tensor([0.2], device=dev))

    def fill(seed):
        c = make(T, E, k, True, "some", seed, garbage=False)
        g = torch.Generator().manual_seed(seed)
        y, _ = y_of(torch.randn(R, H, generator=g), H)
        for n, v in (("logits", c["logits"]), ("ids", c["ids"]), ("w", c["w"]), ("mask", c["keep"])):
            b[n].copy_(torch.from_numpy(v))
        b["x"].copy_(torch.randn(T, H, generator=g))
        b["y"].copy_(y)
        b["inv"].copy_(torch.randperm(R, generator=g))
        b["d_out"].copy_(torch.randn(T, H, generator=g))

    def outputs():
        return [e(E, dt=torch.int32), e(E), e(1), e(T, k), e(T, E), e(E, H), e(E),
                e(m.moe_balance_workspace_size(s), dt=torch.uint8), e(m.moe_router_grad_workspace_size(s), dt=torch.uint8)]

    def calls(o, stream=None):
        m.moe_balance_loss(s, b["logits"], b["ids"], b["mask"], o[0], o[1], o[2], o[7], stream)
        m.moe_finalize_backward(s, b["y"], b["inv"], b["d_out"], o[3], stream)
        m.moe_route_backward(s, b["logits"], b["ids"], b["w"], b["mask"], o[0], o[3], b["d_loss"], o[4], stream)
        m.moe_router_weight_grad(s, b["x"], o[4], b["mask"], o[5], o[6], o[8], stream)

    fill(1)
    eager, other, graphed = outputs(), outputs(), outputs()
    calls(eager)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    calls(other, st)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(eager[:7], other[:7]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(graphed)
    for seed in (1, 2, 3, 4):
        fill(seed)
        for t in graphed:
            t.zero_()
        graph.replay()
        calls(eager)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(eager[:7], graphed[:7])), seed


# ---------------------------------------------------------------- refusals (no GPU: nothing is enqueued)

def test_refusals(m):
    lib = m._lib.lib
    P, mis = ctypes.c_void_p(4096), ctypes.c_void_p(4096 + 4)
    s = ctypes.byref(m.make_shape(64, 256, 8, 2, 32, 1, "bf16"))
    bad = ctypes.byref(m.make_shape(64, 200, 8, 2, 32, 1, "bf16"))
    wide = ctypes.byref(m.make_shape(64, 256, 65, 2, 32, 1, "bf16"))
    big = ctypes.c_size_t(1 << 40)
    sz = ctypes.c_size_t
    INV, UNS, WS = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED, m.MOE_ERR_WORKSPACE
    for sh, want in ((None, INV), (bad, UNS), (wide, UNS)):
        assert lib.moe_balance_loss(sh, P, P, None, P, P, P, P, big, None) == want
        assert lib.moe_route_backward(sh, P, P, P, None, P, P, P, P, None) == want
        assert lib.moe_router_weight_grad(sh, P, P, None, P, P, P, big, None) == want
        assert lib.moe_finalize_backward(sh, P, P, P, P, None) == want
        assert lib.moe_balance_workspace_size(sh) == 0 and lib.moe_router_grad_workspace_size(sh) == 0
    need = lib.moe_balance_workspace_size(s)
    assert need > 0 and need % 256 == 0
    bal = lambda *a: lib.moe_balance_loss(s, *a, None)  # noqa: E731
    assert bal(None, P, None, P, P, P, P, big) == INV
    assert bal(P, P, None, P, P, None, P, big) == INV
    assert bal(P, P, mis, P, P, P, P, big) == UNS
    assert bal(P, P, None, P, P, P, None, big) == WS
    assert bal(P, P, None, P, P, P, P, sz(need - 1)) == WS
    assert bal(P, P, None, P, P, P, ctypes.c_void_p(4096 + 16), big) == UNS
    rb = lambda *a: lib.moe_route_backward(s, *a, None)  # noqa: E731
    assert rb(P, P, P, None, P, None, None, P) == INV          # neither gradient
    assert rb(P, P, P, None, None, P, P, P) == INV             # the loss's gradient needs the counts
    assert rb(P, P, mis, None, P, P, P, P) == UNS
    assert rb(P, P, P, None, P, P, P, None) == INV
    need = lib.moe_router_grad_workspace_size(s)
    wg = lambda *a: lib.moe_router_weight_grad(s, *a, None)  # noqa: E731
    assert need > 0
    assert wg(P, None, None, P, P, P, big) == INV
    assert wg(P, P, None, None, P, P, big) == INV
    assert wg(P, P, None, P, mis, P, big) == UNS
    assert wg(P, P, None, P, None, None, big) == WS
    assert wg(P, P, None, P, None, P, sz(need - 1)) == WS
    assert lib.moe_finalize_backward(s, P, P, None, P, None) == INV
    assert lib.moe_finalize_backward(s, mis, P, P, P, None) == UNS


def test_workspaces_stay_small(m):
    """At most 256 workgroups' sums whatever the shape: 768 bytes + padding each for the loss, 64 experts x 256
    columns for the weight."""
    for T in (1, 64, 65, 4096, 60000):
        for H in (64, 448, 4096):
            s = m.make_shape(T, H, 64, 8, 32, 1, "bf16")
            assert 0 < m.moe_balance_workspace_size(s) <= 256 * 1024
            assert 0 < m.moe_router_grad_workspace_size(s) <= 17 << 20


def test_binding_checks(m):
    s = m.make_shape(4, 64, 8, 2, 32, 1, "bf16")
    z = torch.zeros
    with pytest.raises(ValueError, match="GPU tensor"):
        m.moe_balance_loss(s, z(4, 8), z(4, 2, dtype=torch.int32), None, z(8, dtype=torch.int32), z(8), z(1), z(1))
    with pytest.raises(ValueError, match="required"):
        m.moe_route_backward(s, None, None, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="GPU tensor"):
        m.moe_router_weight_grad(s, z(4, 64), z(4, 8), None, z(8, 64), None, z(1))
    with pytest.raises(ValueError, match="GPU tensor"):
        m.moe_finalize_backward(s, z(1, dtype=torch.uint8), z(8, dtype=torch.int32), z(4, 64), z(4, 2))
