"""An empty batch through the shared expert's backward pass, whichever outputs
are wanted: the pointer of a tensor without elements is null, which must not
be taken for an output that is not wanted."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

P = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def m():
    import mixture_experts_ffn_moe_amd as m
    return m


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_empty_batch_with_frozen_weights(m, dtype):
    """d_x alone, of no tokens: nothing is enqueued (no GPU is needed), with and without the other pointers."""
    none, one = (m.make_shape(T, 64, 1, 1, 32, 1, dtype) for T in (0, 1))

    def call(s, d_x, d_w1, d_w2, other, p=0.0, rng=None):
        return m._lib.lib.moe_shared_ffn_backward(ctypes.byref(s), 64, p, rng, other, other, other, other, other, other, d_x, d_w1,
                                                  d_w2, None, ctypes.c_size_t(0), None)

    for d_x in (None, P):
        for other in (None, P):
            assert call(none, d_x, None, None, other) == m.MOE_OK
            # half of the weights' gradients stays an error, and so does a bad argument of any other kind
            assert call(none, d_x, P, None, other) == call(none, d_x, None, P, other) == m.MOE_ERR_INVALID_ARG
            assert call(none, d_x, None, None, other, p=1.0) == call(none, d_x, None, None, other, p=0.5) == m.MOE_ERR_INVALID_ARG
    assert call(none, ctypes.c_void_p(4096 + 8), None, None, P) == m.MOE_ERR_UNSUPPORTED
    assert call(one, None, None, None, P) == m.MOE_ERR_INVALID_ARG  # with a token, an output is required


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_empty_tensors(m, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    H, Is, p = 128, 96, 0.2
    shape = m.make_shape(0, H, 1, 1, 32, 1, dtype)
    b = m.SharedTrainBuffers(shape, Is, p)
    e = lambda *d: torch.ones(*d, dtype=b.out.dtype, device="cuda")  # noqa: E731
    x, w1, w2 = e(0, H), e(2 * Is, H), e(H, Is)
    rng = torch.tensor([3, 4], device="cuda")
    assert b.forward(x, w1, w2, x, rng).shape == (0, H)
    m.moe_shared_ffn_backward(shape, Is, p, rng, None, w1, w2, b.gu, None, x, b.d_x, None, None, b.workspace)
    b.d_w1s.fill_(float("nan"))
    b.d_w2s.fill_(float("nan"))
    d_x, d_w1, d_w2 = b.backward(x, w1, w2, x, rng)
    torch.cuda.synchronize()
    assert d_x.shape == (0, H) and (d_w1 == 0).all() and (d_w2 == 0).all()
    b.d_w1s.fill_(float("nan"))
    b.d_w2s.fill_(float("nan"))
    m.moe_shared_ffn_backward(shape, Is, p, rng, x, None, w2, b.gu, b.hs, x, None, b.d_w1s, b.d_w2s, b.workspace)
    torch.cuda.synchronize()
    assert (b.d_w1s == 0).all() and (b.d_w2s == 0).all()
