"""Launches of one workgroup per token or route at the envelope's largest
numbers of them: 2^24 workgroups of 256 are 2^32 work-items, more than a
dimension of a launch holds."""
import glob
import os
import re

import pytest

torch = pytest.importorskip("torch")

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_ffn_moe_amd", "csrc")


def test_no_launch_has_all_rows_along_x():
    for path in glob.glob(os.path.join(CSRC, "*")):
        if path.endswith((".hip", ".h")):
            found = re.findall(r"hipLaunchKernelGGL\([^;]*?\bdim3\((?:s\.T|R|s\.R\(\))\)", open(path).read())
            assert not found, (os.path.basename(path), found)


@pytest.mark.gpu
def test_more_than_2_24_tokens():
    """T just past 2^24 (the smallest H, one route a token): the tokens repeat a short batch, whose outputs are the
    reference.  The steps and the 4-bit layer in one call, the permuted copy of x, and the router's gradients."""
    import mixture_experts_ffn_moe_amd as m
    P, H, E, Im, dev = 4096, 64, 2, 32, "cuda"
    T = 4096 * P + 5
    g = torch.Generator(device=dev).manual_seed(6)
    r = lambda *sh: torch.randn(*sh, generator=g, device=dev)  # noqa: E731
    tile = lambda a: torch.cat([a.repeat(4096, *([1] * (a.dim() - 1))), a[:5]])  # noqa: E731
    x, d_out, wg = r(P, H).bfloat16(), r(P, H).bfloat16(), r(E, H) * 0.2
    q4 = m.make_q4("int4", 32)
    shapes = [m.make_shape(n, H, E, 1, Im, 1, "bf16", renormalize=False) for n in (P, T)]
    z = m.moe_q4_get_sizes(shapes[0], q4)
    st = {n: torch.empty(b, dtype=torch.uint8, device=dev) for n, b in z.items()}
    m.moe_q4_quantize_w13(shapes[0], q4, r(1, E, 2 * Im, H).bfloat16(), st["w1_codes"], st["w1_scales"])
    m.moe_q4_quantize_down(shapes[0], q4, r(1, E, H, Im).bfloat16(), st["w2_codes"], st["w2_scales"])
    res = []
    for s, xs, ds in zip(shapes, (x, tile(x)), (d_out, tile(d_out))):
        n = s.T
        print(f"T={n}: layer", flush=True)
        e = lambda *sh, dt=torch.float32: torch.empty(*sh, dtype=dt, device=dev)  # noqa: E731
        buf = m.MoELayerBuffers(s)
        out = buf.forward_q4(q4, xs, wg, None, st["w1_codes"], st["w1_scales"], st["w2_codes"], st["w2_scales"])
        v = buf.views()
        print(f"T={n}: gradients", flush=True)
        d_w, d_l, counts, mean, loss = e(n, 1), e(n, E), e(E, dt=torch.int32), e(E), e(1)
        m.moe_finalize_backward(s, v["y"], v["inv"], ds, d_w)
        m.moe_route_backward(s, v["logits"], v["ids"], v["w"], None, None, d_w, None, d_l)
        m.moe_balance_loss(s, v["logits"], v["ids"], None, counts, mean, loss,
                           e(m.moe_balance_workspace_size(s), dt=torch.uint8))
        d_wg, d_bias = e(E, H), e(E)
        m.moe_router_weight_grad(s, xs, d_l, None, d_wg, d_bias, e(m.moe_router_grad_workspace_size(s), dt=torch.uint8))
        print(f"T={n}: permuted x", flush=True)
        xp, c2, off, perm, inv = e(n, H, dt=torch.bfloat16), e(E, dt=torch.int32), e(E + 1, dt=torch.int32), e(n, dt=torch.int32), e(n, dt=torch.int32)
        m.moe_permute(s, v["ids"], c2, off, perm, inv, xs, xp)
        torch.cuda.synchronize()
        assert torch.equal(xp, xs[perm.long()])
        for a, b in ((c2, v["counts"]), (off, v["offsets"]), (perm, v["perm"].view(-1)), (inv, v["inv"].view(-1)), (counts, c2)):
            assert torch.equal(a, b)
        res.append(dict(out=out, d_w=d_w, d_l=d_l, d_wg=d_wg, d_bias=d_bias, counts=counts, mean=mean, ids=v["ids"], x=xs))
        del xp, perm, inv
    a, b = res
    for n in ("out", "d_w", "d_l"):  # a token's outputs do not depend on the others
        assert torch.equal(b[n][:-5].view(4096, *a[n].shape), a[n].expand(4096, *a[n].shape)), n
        assert torch.equal(b[n][-5:], a[n][:5]), n
    assert torch.equal(b["counts"].long(), a["counts"].long() * 4096 + torch.bincount(a["ids"][:5, 0].long(), minlength=E))
    d, xx = a["d_l"].double(), a["x"].double()
    # 256 runs of 2^16 tokens: a wave adds three parts of its tokens in turn, then 8 waves, then the runs
    tol = 1.01 * (3 * 65536 + 8 + 256) * 2.0 ** -24
    ref = 4096 * (d.T @ xx) + d[:5].T @ xx[:5]
    assert ((b["d_wg"].double() - ref).abs() <= tol * 4097 * (d.abs().T @ xx.abs())).all()
    assert ((b["d_bias"].double() - 4096 * d.sum(0) - d[:5].sum(0)).abs() <= tol * 4097 * d.abs().sum(0)).all()
    # the mean of 4096 equal means and five tokens: these weigh 5 / T, then one rounding each
    assert ((b["mean"] - a["mean"]).abs() <= 5 / T + 2 * 2.0 ** -24).all()
    torch.cuda.empty_cache()
