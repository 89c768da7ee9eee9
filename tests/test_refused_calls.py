"""A refused call of the 4-bit layer or the router's gradients leaves its
outputs and workspace as they were (real buffers; the refusal comes from the
host's checks, so no kernel runs)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_outputs_stay():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mixture_experts_ffn_moe_amd as m
    lib, dev = m._lib.lib, "cuda"
    T, H, E, k, Im = 24, 256, 8, 2, 128
    R = T * k
    ok, bad_shape = m.make_shape(T, H, E, k, Im, 1, "bf16"), m.make_shape(T, H, 65, k, Im, 1, "bf16")
    q, odd = m.make_q4("int4", 128), m.MoeQ4Spec(0, 48)
    z = m.moe_q4_get_sizes(ok, q)
    held = []

    def buffer(n):
        t = torch.full((n + 64,), 0x5A, dtype=torch.uint8, device=dev)
        held.append(t)
        return t.data_ptr()

    src = torch.zeros(max(T * H * 4, E * 2 * Im * H * 2, R * H * 2 + R, z["w1_codes"]) + 64, dtype=torch.uint8, device=dev).data_ptr()
    ws_n, bal_n, wg_n = m.moe_workspace_size(ok), m.moe_balance_workspace_size(ok), m.moe_router_grad_workspace_size(ok)
    ws, bal, wgw = buffer(ws_n), buffer(bal_n), buffer(wg_n)
    out, h, y, codes, scales = buffer(T * H * 2), buffer(R * Im * 2), buffer(m.y_nbytes(ok, R)), buffer(z["w1_codes"]), buffer(z["w1_scales"])
    counts, mean, loss, d_l, d_w, d_wg, d_b = (buffer(n * 4) for n in (E, E, 1, T * E, R, E * H, E))
    B, sz = ctypes.byref, ctypes.c_size_t
    INV, UNS, WS = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED, m.MOE_ERR_WORKSPACE
    mis = src + 8
    calls = []
    for s, spec, want in ((bad_shape, q, UNS), (ok, odd, INV)):
        calls += [(want, lib.moe_q4_quantize_w13(B(s), B(spec), src, codes, scales, None)),
                  (want, lib.moe_q4_quantize_down(B(s), B(spec), src, codes, scales, None)),
                  (want, lib.moe_q4_w13_swiglu(B(s), B(spec), src, src, src, src, src, h, None)),
                  (want, lib.moe_q4_down(B(s), B(spec), src, src, src, src, y, None)),
                  (want, lib.moe_forward_q4(B(s), B(spec), src, src, None, src, src, src, src, out, ws, sz(ws_n), None))]
    S, Q = B(ok), B(q)
    calls += [
        (UNS, lib.moe_q4_quantize_w13(S, Q, mis, codes, scales, None)), (INV, lib.moe_q4_quantize_down(S, Q, None, codes, scales, None)),
        (UNS, lib.moe_q4_quantize_w13(S, Q, src, codes, scales + 8, None)),
        (UNS, lib.moe_q4_w13_swiglu(S, Q, mis, src, src, src, src, h, None)), (UNS, lib.moe_q4_w13_swiglu(S, Q, src, src, src, src, src, h + 8, None)),
        (INV, lib.moe_q4_down(S, Q, src, None, src, src, y, None)),
        (WS, lib.moe_forward_q4(S, Q, src, src, None, src, src, src, src, out, ws, sz(ws_n - 1), None)),
        (UNS, lib.moe_forward_q4(S, Q, src, src, None, src, src, src, src, out, ws + 16, sz(ws_n), None)),
        (UNS, lib.moe_forward_q4(S, Q, src, src, mis, src, src, src, src, out, ws, sz(ws_n), None)),
        (WS, lib.moe_balance_loss(S, src, src, None, counts, mean, loss, bal, sz(bal_n - 1), None)),
        (UNS, lib.moe_balance_loss(S, src, src, mis, counts, mean, loss, bal, sz(bal_n), None)),
        (INV, lib.moe_balance_loss(S, src, None, None, counts, mean, loss, bal, sz(bal_n), None)),
        (INV, lib.moe_route_backward(S, src, src, src, None, src, None, None, d_l, None)),
        (INV, lib.moe_route_backward(S, src, src, src, None, None, src, src, d_l, None)),
        (UNS, lib.moe_route_backward(S, mis, src, src, None, src, src, src, d_l, None)),
        (WS, lib.moe_router_weight_grad(S, src, src, None, d_wg, d_b, wgw, sz(wg_n - 1), None)),
        (UNS, lib.moe_router_weight_grad(S, src, mis, None, d_wg, d_b, wgw, sz(wg_n), None)),
        (INV, lib.moe_router_weight_grad(S, None, src, None, d_wg, d_b, wgw, sz(wg_n), None)),
        (INV, lib.moe_finalize_backward(S, src, None, src, d_w, None)), (UNS, lib.moe_finalize_backward(S, src, src, mis, d_w, None)),
    ]
    torch.cuda.synchronize()
    assert [got for _, got in calls] == [want for want, _ in calls]
    for i, t in enumerate(held):
        assert (t == 0x5A).all(), i
