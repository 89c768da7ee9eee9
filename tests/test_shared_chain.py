"""The shared expert's operators as a program runs them: the layer served with
adapters, and a training step of the shared expert and the router over frozen
routed experts, each in a row, captured and replayed."""
import ctypes

import numpy as np
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


def layer_inputs(T, H, E, k, Im, Is, dt, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *d, s=1.0, t=dt: (torch.randn(*d, generator=g) * s).to(t)  # noqa: E731
    return dict(x=n(T, H), wg=n(E, H, s=0.1, t=torch.float32), w1=n(1, E, 2 * Im, H, s=H ** -0.5), w2=n(1, E, H, Im, s=Im ** -0.5),
                w1s=n(2 * Is, H, s=H ** -0.5), w2s=n(H, Is, s=Is ** -0.5)), n, g


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 8, 150])
def test_layer_with_adapters(m, dev, T, dtype):
    H, E, k, Im, Is, L, r = 256, 8, 2, 128, 96, 5, 16
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    h, n, g = layer_inputs(T, H, E, k, Im, Is, dt)
    h.update(a1=n(L, r, H, s=H ** -0.5), b1=n(L, 2 * Is, r, s=r ** -0.5), a2=n(L, r, Is, s=Is ** -0.5), b2=n(L, H, r, s=r ** -0.5),
             scale=torch.rand(L, generator=g) + 0.5, ids=torch.randint(-1, L, (T,), generator=g).to(torch.int32))
    d = {key: v.cuda() for key, v in h.items()}
    shape = m.make_shape(T, H, E, k, Im, 1, dtype)
    routed = m.MoELayerBuffers(shape).forward(d["x"], d["wg"], None, d["w1"], d["w2"])
    buf = m.MoELayerBuffers(shape, shared_Im=Is, lora=m.make_lora(L, r))
    args = [d[key] for key in ("x", "wg")] + [None] + [d[key] for key in ("w1", "w2", "w1s", "w2s", "a1", "b1", "a2", "b2", "scale", "ids")]
    out = buf.forward_shared_lora(*args)
    torch.cuda.synchronize()
    want = out.clone()
    v = {key: t.double() if t.is_floating_point() else t for key, t in h.items()}
    z = sp.projection(v["x"], v["w1s"], v["a1"], v["b1"], v["scale"], v["ids"], dt, dt == torch.bfloat16)
    hs = buf._hs()
    sp.check("hs", hs, *sp.swiglu(*z, dt), dt)
    z = sp.projection(hs.double().cpu(), v["w2s"], v["a2"], v["b2"], v["scale"], v["ids"], dt, dt == torch.bfloat16)
    sp.check("out", out, *sp.add_residual(*z, routed.double().cpu(), dt), dt)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        buf.forward_shared_lora(*args)
    for _ in range(3):
        buf.out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf.out, want)
    # without any adapter: the layer as moe_forward_shared has it.  Its h may be a step off (another order of
    # the fp32 sums, so up to two half steps a value), the routed output is rounded here and y (to 11 bits) there,
    # and either output once; fp32 sums besides.
    d["ids"].fill_(-1)
    plain = m.MoELayerBuffers(shape, shared_Im=Is).forward_shared(*args[:7])
    got = buf.forward_shared_lora(*args)
    u = sp.half_step(dt)
    mags = hs.double().abs() @ d["w2s"].double().abs().T
    bound = (2 * u + 2.0 ** -11 + (H + Is + 64) * 4 * sp.F32) * (mags + routed.double().abs()) + 3 * u * plain.double().abs()
    assert ((got.double() - plain.double()).abs() <= bound).all()


def test_buffers_without_adapters_refuse(m):
    shape = m.make_shape(4, 64, 4, 2, 32, 1, "bf16")
    with pytest.raises(ValueError, match="shared_Im"):
        m.MoELayerBuffers(shape, device="cpu", lora=m.make_lora(2, 8))
    with pytest.raises(ValueError, match="envelope"):
        m.MoELayerBuffers(shape, device="cpu", shared_Im=32, lora=m.make_lora(2, 12))
    with pytest.raises(ValueError, match="without lora"):
        m.MoELayerBuffers(shape, device="cpu", shared_Im=32).forward_shared_lora(*[None] * 13)
    with pytest.raises(ValueError, match="envelope"):
        m.SharedTrainBuffers(shape, 40, device="cpu")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_training_step_over_frozen_experts(m, dev, dtype):
    """Routed layer, shared expert added with dropout inside, dropout of the sum onto x, and back: the gradients of
    the shared expert's weights, of the router's and of x's shared part, eager and replayed."""
    T, H, E, k, Im, Is, p = 200, 256, 8, 2, 64, 96, 0.2
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    h, n, _ = layer_inputs(T, H, E, k, Im, Is, dt, seed=3)
    d = {key: v.cuda() for key, v in h.items()}
    d_final = n(T, H, s=0.1).cuda()
    shape = m.make_shape(T, H, E, k, Im, 1, dtype)
    R = T * k
    layer, tune = m.MoELayerBuffers(shape), m.SharedTrainBuffers(shape, Is, p)
    rng = [torch.tensor([91, o], dtype=torch.int64, device="cuda") for o in (4, 5)]
    e = lambda *dims: torch.empty(*dims, device="cuda")  # noqa: E731
    final, d_sum = torch.empty(T, H, dtype=dt, device="cuda"), torch.empty(T, H, dtype=dt, device="cuda")
    d_w, d_logits, d_wg = e(T, k), e(T, E), e(E, H)
    ws = torch.empty(m.moe_router_grad_workspace_size(shape), dtype=torch.uint8, device="cuda")

    def step():
        routed = layer.forward(d["x"], d["wg"], None, d["w1"], d["w2"])
        v = layer.views()
        out = tune.forward(d["x"], d["w1s"], d["w2s"], routed, rng[0])
        m.moe_dropout_add(shape, p, rng[1], out, d["x"], final)
        m.moe_dropout_backward(shape, p, rng[1], d_final, d_sum)
        tune.backward(d["x"], d["w1s"], d["w2s"], d_sum, rng[0])
        m.moe_finalize_backward(shape, v["y"], v["inv"], d_sum, d_w)
        m.moe_route_backward(shape, v["logits"], v["ids"], v["w"], None, None, d_w, None, d_logits)
        m.moe_router_weight_grad(shape, d["x"], d_logits, None, d_wg, None, ws)

    outputs = [tune.out, final, d_sum, tune.d_x, tune.d_w1s, tune.d_w2s, d_w, d_logits, d_wg]
    step()
    torch.cuda.synchronize()
    first = [t.clone() for t in outputs]
    routed = layer.out.double().cpu()
    f_in, f_out = sp.drop_factors(T, Is, p, 91, 4), sp.drop_factors(T, H, p, 91, 5)
    d_s = f_out * d_final.double().cpu()
    sp.check("d_sum", d_sum, d_s, 2 * sp.F32 * d_s.abs() + 1.01 * sp.half_step(dt) * d_s.abs(), dt)
    v = {key: t.double() for key, t in h.items()}
    ref = sp.ffn(v["x"], v["w1s"], v["w2s"], routed, d_sum.double().cpu(), f_in, dt)
    for name, got in (("out", tune.out), ("d_x", tune.d_x), ("d_w1s", tune.d_w1s), ("d_w2s", tune.d_w2s)):
        sp.check(name, got, *ref[name], dt)
    value = f_out * tune.out.double().cpu() + v["x"]
    bound = 3 * sp.F32 * value.abs() + 2 * sp.F32 * (f_out * tune.out.double().cpu()).abs()
    sp.check("final", final, value, bound + 1.01 * sp.half_step(dt) * value.abs(), dt)
    # the router's gradient from the same d_sum: d_w[t, j] . y of route j
    views = layer.views()
    assert views["ids"].shape == (T, k) and R == views["inv"].numel()
    w = views["w"].double()
    dw = d_w.double()
    by_hand = torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_(
        1, views["ids"].long(), w * (dw - (w * dw).sum(1, keepdim=True)))
    assert torch.allclose(d_logits.double(), by_hand, rtol=1e-5, atol=1e-6 * float(by_hand.abs().max()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in outputs:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outputs, first):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_refused_calls_leave_everything(m, dev):
    lib, B, sz = m._lib.lib, ctypes.byref, ctypes.c_size_t
    T, H, Is, L, r = 24, 128, 64, 4, 16
    shape, spec = m.make_shape(T, H, 1, 1, 32, 1, "bf16"), m.make_lora(L, r)
    held = [torch.full((1 << 17,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(6)]
    a, b, c, d, e, ws = (t.data_ptr() for t in held)
    src = torch.zeros(1 << 18, dtype=torch.uint8, device="cuda").data_ptr()
    n, nl = m.moe_shared_backward_workspace_size(shape, Is), m.moe_lora_workspace_size(shape, Is, spec)
    assert max(n, nl) <= 1 << 17
    codes = [
        lib.moe_dropout_add(B(shape), 2.0, src, src, src, a, None),
        lib.moe_dropout_backward(B(shape), 0.5, None, src, a, None),
        lib.moe_shared_ffn_train(B(shape), Is, 0.5, src, src, src, src, src, a, b, c + 8, None),
        lib.moe_shared_ffn_train(B(shape), 40, 0.5, src, src, src, src, src, a, b, c, None),
        lib.moe_shared_ffn_backward(B(shape), Is, 0.0, None, src, src, src, src, src, src, a, b, None, ws, sz(n), None),
        lib.moe_shared_ffn_backward(B(shape), Is, 0.0, None, src, src, src, src, src, src, a, b, c, ws, sz(n - 1), None),
        lib.moe_lora_w13_swiglu(B(shape), Is, B(spec), src, src, src, src, src, None, a, ws, sz(nl), None),
        lib.moe_lora_down(B(shape), Is, B(m.make_lora(L, 12)), src, src, src, src, src, src, src, a, ws, sz(nl), None),
        lib.moe_shared_ffn_lora(B(shape), Is, B(spec), src, src, src, src, src, src, src, src, src, src, d, e, ws, sz(nl - 1), None)]
    assert all(code != m.MOE_OK for code in codes), codes
    torch.cuda.synchronize()
    for t in held:
        assert (t == 0x5A).all()


def test_plain_factors_agree_with_a_small_case():
    """The first elements of a stream by hand: words of block 0, low half first."""
    words = sp.philox([np.array([0], np.uint64)] * 2 + [np.array([5], np.uint64), np.array([0], np.uint64)], [91, 0])
    bits = [int(words[i // 2][0]) >> (16 * (i % 2)) & 0xFFFF for i in range(8)]
    f = sp.drop_factors(1, 8, 0.2, 91, 5)[0]
    assert [float(x) for x in f] == [0.0 if b < 13107 else 65536 / (65536 - 13107) for b in bits]
