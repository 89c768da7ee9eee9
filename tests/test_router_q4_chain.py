"""Router tuning over 4-bit experts, the calls in a row as a program makes
them: the layer (on the small-token path also the down product that writes y
from the workspace's h and offsets), the balance loss, and the three gradient
calls down to the router's weight and bias.  Padded tokens hold infinities
and NaN where the calls allow it.

y is compared with the plain layer's (test_q4_decode_layer.py); from it the
reference is the 64-bit objective's gradient by autograd, the selection held
fixed.  Tolerances follow the calls: each one's own roundings as in
test_router_grad.py, through the sums behind it.  Logits are off by half a step of fp32,
which moves a probability by twice that, relatively: both sides of every
product, 4 U max|logit| in all."""
import pytest

from test_q4_decode_layer import Case, layer, pack, y_values

torch = pytest.importorskip("torch")
U = 2.0 ** -24
P_TOL = 32 * U


@pytest.fixture
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return "cuda"


# T, H, E, k, Im, mu, format, group, renormalised: the small-token path, the split router, the plain one, one token
CASES = [Case(12, 2048, 16, 4, 128, 2, "int4", 128, True), Case(16, 2048, 8, 3, 96, 1, "e2m1", 32, False),
         Case(40, 2048, 12, 4, 128, 1, "e2m1", 64, True), Case(150, 192, 9, 3, 96, 2, "int4", 32, False),
         Case(1, 2048, 8, 2, 128, 1, "int4", 64, True)]


@pytest.mark.gpu
@pytest.mark.parametrize("c", CASES, ids=lambda c: f"{c.T}x{c.H}x{c.E}x{c.k}-{c.fmt}-renorm{int(c.renorm)}")
def test_router_tuning(dev, c):
    import mixture_experts_ffn_moe_amd as m
    T, H, E, k, R = c.T, c.H, c.E, c.k, c.T * c.k
    print(f"router tuning T={T} H={H} E={E} k={k} {c.fmt}", flush=True)
    g = torch.Generator().manual_seed(T)
    d_out = torch.randn(T, H, generator=g).bfloat16().to(dev)
    bias = torch.randn(E, generator=g).to(dev) * 0.2
    mask = (torch.rand(T, generator=g) < 0.8).to(torch.uint8).to(dev)
    mask[0] = 1
    pad = mask == 0
    d_out[pad] = float("inf")
    x, wg = c.x.to(dev), c.wg.to(dev)
    w1, w2 = c.weights(dev)
    flat = lambda p, up: pack(p[0].flatten(0, 1), p[1].flatten(0, 1), c.fmt, c.group, up)  # noqa: E731
    stored = (*flat(w1, True), *flat(w2, False))

    # the program's calls
    s, q4 = m.make_shape(T, H, E, k, c.Im, c.mu, "bf16", c.renorm), m.make_q4(c.fmt, c.group)
    buf = m.MoELayerBuffers(s)
    buf.workspace.fill_(0xFF)
    buf.forward_q4(q4, x, wg, bias, *stored)
    v = buf.views()
    if T <= 16:
        m.moe_q4_down(s, q4, v["h"], v["offsets"], stored[2], stored[3], v["y"])
    e = lambda *sh, dt=torch.float32: torch.empty(*sh, dtype=dt, device=dev)  # noqa: E731
    counts, mean, loss, alpha = e(E, dt=torch.int32), e(E), e(1), torch.tensor([0.5], device=dev)
    d_w, d_l, d_wg, d_bias = e(T, k), e(T, E), e(E, H), e(E)
    m.moe_balance_loss(s, v["logits"], v["ids"], mask, counts, mean, loss, e(m.moe_balance_workspace_size(s), dt=torch.uint8))
    m.moe_finalize_backward(s, v["y"], v["inv"], d_out, d_w)
    m.moe_route_backward(s, v["logits"], v["ids"], v["w"], mask, counts, d_w, alpha, d_l)
    xp = x.clone()
    xp[pad] = float("nan")
    m.moe_router_weight_grad(s, xp, d_l, mask, d_wg, d_bias, e(m.moe_router_grad_workspace_size(s), dt=torch.uint8))
    torch.cuda.synchronize()

    # the objective in 64 bits, on the CPU (fp64 products and their backward are elementary there)
    ids = v["ids"].cpu().long()
    ok = (mask != 0).cpu()
    n = int(ok.sum())
    _, _, y, dy, _, _, _ = layer(x.double(), v["ids"], v["w"], w1, w2, c.fmt, c.group)
    got = y_values(v["y"], R, H)[v["inv"].view(-1).long()]
    assert ((got - y).abs() <= dy + 1e-30).all()
    y = got.cpu().view(T, k, H)
    X, do = x.double().cpu(), torch.where(ok[:, None], d_out.double().cpu(), 0.0)
    assert torch.equal(counts.cpu().long(), torch.bincount(ids[ok].reshape(-1), minlength=E))
    f = counts.double().cpu() / (n * k)
    G, B = wg.double().cpu().requires_grad_(), bias.double().cpu().requires_grad_()
    L = X @ G.T + B
    L.retain_grad()
    p = torch.softmax(L, 1)
    w = torch.gather(p, 1, ids)
    w = w / w.sum(1, keepdim=True) if c.renorm else w
    bal = E * (f * p[ok].mean(0)).sum()
    ((w[:, :, None] * y * do[:, None]).sum() + 0.5 * bal).backward()
    bal, p, w = bal.detach(), p.detach(), w.detach()
    eL = 4 * U * float(L.detach().abs().max())

    dw = (y * do[:, None]).sum(-1)
    size = (y * do[:, None]).abs().sum(-1)
    e_dw = (9 * -(-H // 2048) + 12) * U * size
    assert ((d_w.cpu().double() - dw).abs() <= e_dw)[ok].all()
    assert abs(float(loss) - float(bal)) <= (P_TOL + eL) * float(bal)

    # the logits' gradient: a bound of its terms, and of their errors
    fp = (p * f).sum(1, keepdim=True)
    terms = 0.5 * E / n * p * (f + fp)
    dot, e_dot = (w * dw.abs()).sum(1, keepdim=True), (w * e_dw).sum(1, keepdim=True)
    if c.renorm:
        terms = terms.scatter_add(1, ids, w * (dw.abs() + dot))
        e_l = torch.zeros(T, E, dtype=torch.float64).scatter_add(1, ids, w * (e_dw + e_dot))
    else:
        put = lambda a: torch.zeros(T, E, dtype=torch.float64).scatter_add(1, ids, a)  # noqa: E731
        terms = terms + p * (put(dw.abs()) + dot)
        e_l = p * (put(e_dw) + e_dot)
    e_l = e_l + (2 * P_TOL + (k / 16 + 12) * U + 2 * eL) * (terms + e_l)
    e_l[~ok] = 0
    terms[~ok] = 0
    ref = torch.where(ok[:, None], L.grad, 0.0)
    got = d_l.cpu().double()
    assert (got[~ok] == 0).all()
    assert ((got - ref).abs() <= e_l + 1e-38).all(), float(((got - ref).abs() - e_l).max())

    # the parameters' gradients
    size = terms + e_l
    tol = (T / 16 + 32 + 4 + T // 64 + 1 + 2) * U
    assert ((d_wg.cpu().double() - G.grad).abs() <= e_l.T @ X.abs() + tol * (size.T @ X.abs())).all()
    assert ((d_bias.cpu().double() - B.grad).abs() <= e_l.sum(0) + tol * size.sum(0)).all()
