"""A run of the operators together: one decoder block made of LRB projections, its norms, residual
and per-request adapters, forward and backward, each step against 64 bits on the inputs that the
step had."""
import numpy as np
import pytest
import torch

import oracle
from rank_binary_factorized_b200 import synth
from tests.gpu_util import check_tolerance, download_bf16_bits, need_gpu, nq, upload_projection
from tests.operator_util import adapter_grad_reference, adapter_reference, check, norm_grad_reference, norm_reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 6, 70])
def test_block(M):
    need_gpu()
    D, F, r, n = 256, 384, 128, 3
    P = {k: synth.make_projection(k, o, i, r, seed=77, key=j)
         for j, (k, o, i) in enumerate((("qkv", D, D), ("gate", F, D), ("up", F, D), ("down", D, F)))}
    L = {k: upload_projection(p) for k, p in P.items()}
    g = torch.Generator(device="cuda").manual_seed(3)

    def rnd(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).bfloat16()

    ids = torch.randint(-1, n, (M,), generator=g, device="cuda", dtype=torch.int32)
    groups = nq().adapter_rows(ids, n)
    AB = {k: (rnd(n, 8, L[k].d_in, std=L[k].d_in ** -0.5), rnd(n, L[k].d_out, 8, std=0.3)) for k in ("qkv", "down")}
    ad = {k: nq().Adapters(*v) for k, v in AB.items()}
    w = [rnd(D, std=0.1, mean=1.0) for _ in range(4)]
    N1 = nq().BlockNorm(D, w_pre=w[0])
    N2 = nq().BlockNorm(D, w_pre=w[1], w_post=w[2], post_norm=True)
    gate = rnd(D, std=0.2, mean=0.7)

    def norm(N, y, h, gate=None):
        out = nq().block_norm(N, y, h, gate=gate)
        refs, tols = norm_reference(y, h, gate, N.w_post, N.w_pre, N.post_norm, 1.0, 1e-5, 0.0)
        for o, a, b in zip(out, refs, tols):
            check(o, a, b, "norm")
        return out

    def project(k, x):
        base = nq().layer_forward(L[k], x)
        ref, S = oracle.dense_packed(P[k].U, P[k].V, P[k].s1, P[k].s2, r, download_bf16_bits(x))
        check_tolerance(download_bf16_bits(base), ref, S, "projection " + k)
        if k not in ad:
            return base, None
        t = torch.empty((M, 8), device="cuda")
        y = nq().layer_forward(L[k], x, adapters=ad[k], groups=groups, t=t)
        want, _, tol, _ = adapter_reference(*AB[k], None, ids, x, base)
        check(y, want, tol, "adapted " + k)
        return y, t

    h0 = rnd(M, D)
    h, x0 = norm(N1, None, h0)
    a, ta = project("qkv", x0)
    h1, x1 = norm(N2, a, h, gate)
    m = nq().mlp_gate_up(L["gate"], L["up"], x1)
    y, ty = project("down", m)
    h2, x2 = norm(N2, y, h1, gate)
    nq().sync_status()

    # back through the last norm, the adapted down projection and its norm
    gx, gh = rnd(M, D, std=0.1), rnd(M, D, std=0.1)
    back = nq().block_norm_backward(N2, y, h2, gx, gh, gate=gate)
    res, tol = norm_grad_reference(y, h2, gate, w[2], w[1], True, 1.0, 1e-5, 0.0, gx, gh)
    for v, a_, b_ in zip(back, res, tol):
        check(v, a_, b_, "norm gradients")
    xbar = nq().lrb_transposed(L["down"], back[1])
    got = nq().adapter_backward(ad["down"], groups, m, back[1], ty, xbar)
    refs, tols = adapter_grad_reference(*AB["down"], None, ids, m, back[1], ty, xbar)
    for v, a_, b_ in zip(got, refs, tols):
        check(v, a_, b_, "adapter gradients")
    nq().sync_status()
    assert all(torch.isfinite(v).all() for v in got)
    assert np.isfinite(x2.float().cpu().numpy()).all()
