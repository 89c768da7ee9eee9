"""The bf16 weight gradient on both sides of the rule that picks its column
groups (H >= 512 and T * H >= 3 * 2^25: four of them, otherwise two)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
U = 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("mask", ["none", "some"])
@pytest.mark.parametrize("T,H,E", [(196607, 512, 5), (196608, 512, 64), (174763, 576, 33), (24577, 4160, 64), (24575, 4096, 7)])
def test_column_groups(T, H, E, mask):
    import mixture_experts_ffn_moe_amd as m
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print(f"weight gradient T={T} H={H} E={E} mask={mask}", flush=True)
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(T + E)
    x = torch.randn(T, H, generator=g, device=dev).bfloat16()
    d = torch.randn(T, E, generator=g, device=dev) * 1e-3
    keep = torch.ones(T, dtype=torch.uint8, device=dev)
    if mask == "some":
        keep = (torch.rand(T, generator=g, device=dev) < 0.7).to(torch.uint8)
        x[keep == 0], d[keep == 0] = float("nan"), float("inf")
    s = m.make_shape(T, H, E, 1, 32, 1, "bf16")
    d_wg, d_bias = torch.full((E, H), np.nan, device=dev), torch.full((E,), np.nan, device=dev)
    ws = torch.empty(m.moe_router_grad_workspace_size(s), dtype=torch.uint8, device=dev)
    m.moe_router_weight_grad(s, x, d, None if mask == "none" else keep, d_wg, d_bias, ws)
    a, b = d[keep != 0].double(), x[keep != 0].double()
    # runs of T / splits tokens, splits at least 256 / ceil(H / 128) - 1 (two groups take the most columns' workgroups);
    # a wave adds three parts of its tokens in turn, then 4 waves, then at most 256 runs; the parts' magnitudes sum to
    # less than 1.01 times the value's
    run = T // (256 // -(-H // 128)) + 256
    tol = 1.01 * (3 * run + 4 + 256) * U
    assert ((d_wg.double() - a.T @ b).abs() <= tol * (a.abs().T @ b.abs())).all()
    assert ((d_bias.double() - a.sum(0)).abs() <= tol * a.abs().sum(0)).all()
    again = torch.empty_like(d_wg)
    m.moe_router_weight_grad(s, x, d, None if mask == "none" else keep, again, None, ws)
    assert torch.equal(again, d_wg)
    torch.cuda.empty_cache()
