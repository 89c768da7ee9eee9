"""moe_route_backward without the routing weights' gradient needs neither the
ids nor the weights."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


def test_ids_and_weights_are_needed_with_their_gradient_only():
    """No GPU: a later argument is misaligned, so nothing is enqueued and its error tells that the earlier ones passed."""
    import mixture_experts_ffn_moe_amd as m
    P, mis = ctypes.c_void_p(4096), ctypes.c_void_p(4096 + 4)
    s = ctypes.byref(m.make_shape(64, 256, 8, 2, 32, 1, "bf16"))
    rb = lambda *a: m._lib.lib.moe_route_backward(s, *a, None)  # noqa: E731
    assert rb(P, None, None, None, mis, None, P, P) == m.MOE_ERR_UNSUPPORTED  # the counts are the first fault
    assert rb(P, None, P, None, P, P, P, P) == m.MOE_ERR_INVALID_ARG
    assert rb(P, P, None, None, P, P, P, P) == m.MOE_ERR_INVALID_ARG
    assert rb(P, P, mis, None, P, P, P, P) == m.MOE_ERR_UNSUPPORTED


@pytest.mark.gpu
@pytest.mark.parametrize("renorm", [True, False])
def test_loss_gradient_alone(renorm):
    import mixture_experts_ffn_moe_amd as m
    T, E, k, dev = 333, 20, 4, "cuda"
    s = m.make_shape(T, 64, E, k, 32, 1, "bf16", renorm)
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(1)).to(dev)
    w, ids = torch.softmax(logits, 1).topk(k)
    w, ids = w.contiguous(), ids.to(torch.int32).contiguous()
    counts = torch.bincount(ids.view(-1), minlength=E).to(torch.int32)
    d_loss = torch.tensor([0.3], device=dev)
    a, b = torch.empty(T, E, device=dev), torch.empty(T, E, device=dev)
    m.moe_route_backward(s, logits, ids, w, None, counts, None, d_loss, a)
    m.moe_route_backward(s, logits, None, None, None, counts, None, d_loss, b)
    assert torch.equal(a, b)
    with pytest.raises(ValueError, match="topk_ids"):
        m.moe_route_backward(s, logits, None, w, None, counts, torch.zeros(T, k, device=dev), d_loss, b)
