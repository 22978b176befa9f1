"""The norms, gate and residual between two blocks (nq_block_norm_*) against 64 bits."""
import itertools

import pytest
import torch

from tests.gpu_util import need_gpu, nq
from tests.operator_util import check, norm_grad_reference, norm_reference

pytestmark = pytest.mark.gpu
EPS = 1e-5


def _make(M, d, f32, gate, seed, with_y=True):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)

    hd = torch.float32 if f32 else torch.bfloat16
    return dict(y=rnd(M, d, std=2.0) if with_y else None, h=rnd(M, d, std=1.5, dtype=hd),
                gate={None: None, "channel": rnd(d, std=0.5), "row": rnd(M, d, std=0.5)}[gate],
                w_pre=rnd(d, std=0.2, mean=1.0), w_post=rnd(d, std=0.2, mean=0.5), gx=rnd(M, d, std=0.3),
                gh=rnd(M, d, std=0.3, dtype=hd))


def _both(c, post, alpha=0.875, eps=EPS, offset=0.0, what=""):
    """Forward and backward against the references."""
    d = c["h"].shape[1]
    N = nq().BlockNorm(d, c["w_pre"], c["w_post"], post_norm=post, alpha=alpha, eps=eps, w_offset=offset)
    h_out, x = nq().block_norm(N, c["y"], c["h"], gate=c["gate"])
    (rh, rx), (th, tx) = norm_reference(c["y"], c["h"], c["gate"], c["w_post"], c["w_pre"], post, alpha, eps, offset)
    nq().sync_status()
    check(h_out, rh, th, what + " h_out")
    check(x, rx, tx, what + " x")
    got = nq().block_norm_backward(N, c["y"], c["h"], c["gx"], c["gh"], gate=c["gate"])
    nq().sync_status()
    res, tol = norm_grad_reference(c["y"], c["h"], c["gate"], c["w_post"], c["w_pre"], post, alpha, eps, offset,
                                   c["gx"], c["gh"])
    for name, g, r, t in zip(("gh", "gy", "g_w_pre", "g_w_post", "g_gate"), got, res, tol):
        assert (g is None) == (r is None), what + " " + name
        if g is not None:
            check(g, r, t, what + " " + name)


@pytest.mark.parametrize("f32,gate,post", list(itertools.product([False, True], [None, "channel", "row"], [False, True])))
@pytest.mark.parametrize("M,d", [(1, 1), (1, 8192), (3, 7), (5, 264), (37, 1001), (311, 4096), (2, 4095), (20, 8200)])
def test_norm(M, d, f32, gate, post):
    need_gpu()
    _both(_make(M, d, f32, gate, 7 * M + d), post, what="M=%d d=%d" % (M, d))


@pytest.mark.parametrize("M,d,f32", [(1, 16384, False), (3, 20000, True), (2, 28672, False), (2, 50001, True),
                                     (2, 131072, False), (700, 2048, True), (1200, 129, False), (601, 11008, False)])
def test_norm_wide_and_long(M, d, f32):
    need_gpu()
    _both(_make(M, d, f32, "channel", 11 + M), True, what="M=%d d=%d" % (M, d))


@pytest.mark.parametrize("f32,gate", [(False, "row"), (True, "channel")])
@pytest.mark.parametrize("M,d", [(5000, 1), (3001, 3), (1500, 9), (2000, 31), (400, 255), (1000, 513), (297, 8191)])
def test_norm_many_narrow_rows(M, d, f32, gate):
    need_gpu()
    _both(_make(M, d, f32, gate, M + d), True, what="M=%d d=%d" % (M, d))


def test_norm_without_a_block():
    need_gpu()
    c = _make(9, 1024, False, None, 5, with_y=False)
    _both(c, False, alpha=1.0, what="no block")
    _both(c, False, alpha=1.0, offset=1.0, eps=1e-6, what="weights stored less one")


def test_norm_unit_weights_and_zero_rows():
    need_gpu()
    c = _make(6, 512, True, None, 6)
    c["w_pre"] = c["w_post"] = None
    c["h"][2] = 0
    c["y"][2] = 0
    c["y"][4] = 0
    N = nq().BlockNorm(512, post_norm=True, alpha=0.5, eps=EPS)
    h_out, x = nq().block_norm(N, c["y"], c["h"])
    (rh, rx), (th, tx) = norm_reference(c["y"], c["h"], None, None, None, True, 0.5, EPS, 0.0)
    check(h_out, rh, th, "h_out")
    check(x, rx, tx, "x")
    assert not h_out[2].any() and not x[2].any()
    got = nq().block_norm_backward(N, c["y"], c["h"], c["gx"], c["gh"])
    assert got[2] is None and got[3] is None and got[4] is None
    res, tol = norm_grad_reference(c["y"], c["h"], None, None, None, True, 0.5, EPS, 0.0, c["gx"], c["gh"])
    for g, r, t in zip(got[:2], res[:2], tol[:2]):
        check(g, r, t, "unit weights")


@pytest.mark.parametrize("d", [1000, 1003])
def test_norm_absent_gradients_and_outputs_in_place(d):
    need_gpu()
    c = _make(33, d, False, "row", 8)
    N = nq().BlockNorm(d, c["w_pre"], c["w_post"], post_norm=True, eps=EPS)
    for gx, gh in ((None, c["gh"]), (c["gx"], None), (None, None)):
        got = nq().block_norm_backward(N, c["y"], c["h"], gx, gh, gate=c["gate"])
        res, tol = norm_grad_reference(c["y"], c["h"], c["gate"], c["w_post"], c["w_pre"], True, 1.0, EPS, 0.0, gx, gh)
        for i in (0, 1, 3, 4):
            check(got[i], res[i], tol[i], "absent gradient, output %d" % i)
        if gx is None:
            assert not got[2].any()
    apart = nq().block_norm_backward(N, c["y"], c["h"], c["gx"], c["gh"], gate=c["gate"])
    gx, gh = c["gx"].clone(), c["gh"].clone()
    got = nq().block_norm_backward(N, c["y"], c["h"], gx, gh, gate=c["gate"], gh=gh, gy=gx)
    assert got[0].data_ptr() == gh.data_ptr() and got[1].data_ptr() == gx.data_ptr()
    assert all(torch.equal(p, q) for p, q in zip(apart, got))
    h_out, x = nq().block_norm(N, c["y"], c["h"], gate=c["gate"])
    y, h = c["y"].clone(), c["h"].clone()
    h2, x2 = nq().block_norm(N, y, h, gate=c["gate"], h_out=h, x=y)
    assert h2 is h and x2 is y and torch.equal(h, h_out) and torch.equal(y, x)


def test_norm_strided_gate_rows_and_one_row():
    need_gpu()
    wide = torch.randn(40, 1024, device="cuda").bfloat16()
    for rows, cols in ((40, 512), (40, 513), (1, 512)):
        c = _make(rows, cols, True, None, 3)
        c["gate"] = wide[:rows, :cols]
        _both(c, False, what="strided gate")


def test_norm_nan_and_infinity_stay_in_their_rows():
    need_gpu()
    for d in (256, 257):
        c = _make(8, d, True, "channel", 4)
        N = nq().BlockNorm(d, c["w_pre"], c["w_post"], post_norm=True, eps=EPS)
        clean = nq().block_norm(N, c["y"], c["h"], gate=c["gate"])
        back = nq().block_norm_backward(N, c["y"], c["h"], c["gx"], c["gh"], gate=c["gate"])
        c["y"][1, 5], c["h"][3, 7], c["h"][6, 0] = float("nan"), float("inf"), float("-inf")
        got = nq().block_norm(N, c["y"], c["h"], gate=c["gate"])
        gback = nq().block_norm_backward(N, c["y"], c["h"], c["gx"], c["gh"], gate=c["gate"])
        keep = [0, 2, 4, 5, 7]
        for p, q in zip(clean + back[:2], got + gback[:2]):
            assert torch.equal(p[keep], q[keep])
        assert got[1][1].isnan().all() and got[1][3].isnan().any()


def test_norm_repeats_on_other_streams_and_in_graphs():
    need_gpu()
    c = _make(700, 2048, True, "channel", 9)
    N = nq().BlockNorm(2048, c["w_pre"], c["w_post"], post_norm=True, eps=EPS)
    want = nq().block_norm_backward(N, c["y"], c["h"], c["gx"], c["gh"], gate=c["gate"])
    fwd = nq().block_norm(N, c["y"], c["h"], gate=c["gate"])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for s in streams:
        ws = torch.empty(N.workspace_bytes(700), dtype=torch.uint8, device="cuda")
        outs.append((nq().block_norm(N, c["y"], c["h"], gate=c["gate"], stream=s),
                     nq().block_norm_backward(N, c["y"], c["h"], c["gx"], c["gh"], gate=c["gate"], ws=ws, stream=s), ws))
    torch.cuda.synchronize()
    for f, b, _ in outs:
        assert all(torch.equal(p, q) for p, q in zip(fwd + want, f + b))
    h_out, x, ws = torch.empty_like(c["h"]), torch.empty_like(c["y"]), N.workspace(700)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nq().block_norm(N, c["y"], c["h"], gate=c["gate"], h_out=h_out, x=x)
        got = nq().block_norm_backward(N, c["y"], c["h"], c["gx"], c["gh"], gate=c["gate"], ws=ws)
    for _ in range(2):
        h_out.zero_(), x.zero_(), [v.zero_() for v in got]
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(h_out, fwd[0]) and torch.equal(x, fwd[1])
        assert all(torch.equal(p, q) for p, q in zip(want, got))


def test_norm_beyond_31_bit_offsets():
    need_gpu()
    M, d = 270001, 8192  # 2.2e9 elements
    g = torch.Generator(device="cuda").manual_seed(1)
    y = torch.empty((M, d), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    h = torch.empty_like(y).normal_(generator=g)
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    N = nq().BlockNorm(d, w, w, post_norm=True, eps=EPS)
    h_out, x = nq().block_norm(N, y, h)
    part = slice(M - 3, M)
    (rh, rx), (th, tx) = norm_reference(y[part], h[part], None, w, w, True, 1.0, EPS, 0.0)
    check(h_out[part], rh, th, "far h_out")
    check(x[part], rx, tx, "far x")
    gh, gy = nq().block_norm_backward(N, y, h, x, h_out, need_weights=False)[:2]
    res, tol = norm_grad_reference(y[part], h[part], None, w, w, True, 1.0, EPS, 0.0, x[part], h_out[part])
    check(gh[part], res[0], tol[0], "far gh")
    check(gy[part], res[1], tol[1], "far gy")


def test_norm_gradients_against_differences():
    """The backward kernel against central differences of the forward reference in 64 bits: the
    differences' own error is O(step^2) of third derivatives, far below the bound used."""
    need_gpu()
    M, d = 3, 24
    c = _make(M, d, True, "channel", 12)
    N = nq().BlockNorm(d, c["w_pre"], c["w_post"], post_norm=True, alpha=0.875, eps=EPS)

    def loss(y, h, gate, w_post, w_pre):
        (ho, x), _ = norm_reference(y, h, gate, w_post, w_pre, True, 0.875, EPS, 0.0)
        return (x * c["gx"].double()).sum() + (ho * c["gh"].double()).sum()

    base = [c[k].double() for k in ("y", "h", "gate", "w_post", "w_pre")]
    (h_out, _), _ = norm_reference(*base, True, 0.875, EPS, 0.0)
    gh, gy, gwp, gwo, gg = nq().block_norm_backward(N, c["y"], h_out.float(), c["gx"], c["gh"], gate=c["gate"])
    for which, grad, step in ((1, gh, 2.0 ** -20), (0, gy, 2.0 ** -8), (2, gg, 2.0 ** -20), (3, gwo, 2.0 ** -20),
                              (4, gwp, 2.0 ** -20)):
        num = torch.zeros_like(base[which])
        flat = num.view(-1)
        for i in range(flat.numel()):
            v = [b.clone() for b in base]
            v[which].view(-1)[i] += 1e-5
            up = loss(*v)
            v[which].view(-1)[i] -= 2e-5
            flat[i] = (up - loss(*v)) / 2e-5
        err = (grad.double() - num).abs().max()
        assert err <= step * num.abs().max() + 1e-6, (which, float(err))
