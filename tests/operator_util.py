"""64-bit references and derived tolerances of the adapter and block-norm operators.

Bounds count roundings: an output held in bf16 is off by half a unit (2^-8 of its value at most),
an fp32 sum of k terms by k 2^-23 of the sum of the terms' magnitudes (2^-23 a term: the tensor
cores' accumulator may cut instead of rounding), a value handed on as two bf16 parts by 2^-16.
"""
import torch

BF16 = 2.0 ** -8
F32 = 2.0 ** -24
SUM = 2.0 ** -23
PARTS = 2.0 ** -16
TINY = 1e-30


def check(got, ref, tol, what):
    got, ref = got.double().cpu(), ref.cpu()
    bad = ~((got - ref).abs() <= tol.cpu() + TINY)  # NaN counts as bad
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError("%s: %d of %d outside tolerance, first %s: got %r, expected %r +- %r" %
                             (what, int(bad.sum()), bad.numel(), i, float(got[i]), float(ref[i]), float(tol.cpu()[i])))


def adapter_reference(A, B, scale, ids, x, y):
    """(out, t, tolerances of both) in 64 bits; ids outside 0..n-1: none."""
    n, R, K = A.shape
    out, t = y.double().clone(), torch.zeros((len(ids), R), dtype=torch.float64, device=y.device)
    tol, tol_t = torch.zeros_like(out), torch.zeros_like(t)
    for a in range(n):
        m = (ids == a).nonzero()[:, 0]
        if not len(m):
            continue
        s = scale[a].double() if scale is not None else torch.ones((), dtype=torch.float64, device=y.device)
        Ad, Bd, xd = A[a].double(), B[a].double(), x[m].double()
        t[m] = s * (xd @ Ad.T)
        tol_t[m] = (K + 2) * SUM * s.abs() * (xd.abs() @ Ad.abs().T)
        out[m] += t[m] @ Bd.T
        tol[m] = ((tol_t[m] + (PARTS + (R + 2) * SUM) * t[m].abs()) @ Bd.abs().T) * (1 + BF16) + BF16 * out[m].abs()
    return out, t, tol, tol_t


def adapter_grad_reference(A, B, scale, ids, x, ybar, t, xbar):
    """(xbar_out, gA, gB) and their tolerances."""
    n, R, _ = A.shape
    K = ybar.shape[1]
    f = dict(dtype=torch.float64, device=ybar.device)
    out, gA, gB = xbar.double().clone(), torch.zeros(A.shape, **f), torch.zeros(B.shape, **f)
    tols = [torch.zeros_like(v) for v in (out, gA, gB)]
    for a in range(n):
        m = (ids == a).nonzero()[:, 0]
        if not len(m):
            continue
        s = scale[a].double() if scale is not None else torch.ones((), **f)
        Ad, Bd, yb, xd, td = A[a].double(), B[a].double(), ybar[m].double(), x[m].double(), t[m].double()
        u = s * (yb @ Bd)
        tol_u = (K + 2) * SUM * s.abs() * (yb.abs() @ Bd.abs())
        out[m] += u @ Ad
        tols[0][m] = ((tol_u + (PARTS + (R + 2) * SUM) * u.abs()) @ Ad.abs()) * (1 + BF16) + BF16 * out[m].abs()
        gA[a], gB[a] = u.T @ xd, yb.T @ td
        k = PARTS + (len(m) + 2) * SUM
        tols[1][a] = ((tol_u + k * u.abs()).T @ xd.abs()) * (1 + BF16) + BF16 * gA[a].abs()
        tols[2][a] = k * (yb.abs().T @ td.abs()) * (1 + BF16) + BF16 * gB[a].abs()
    return (out, gA, gB), tols


def _weight(w, offset, like):
    return torch.ones(like.shape[1], dtype=torch.float64, device=like.device) if w is None else w.double() + offset


def _step(dtype):
    return BF16 if dtype == torch.bfloat16 else F32


def norm_reference(y, h, gate, w_post, w_pre, post, alpha, eps, offset):
    """(h_out, x) in 64 bits and their tolerances."""
    d = h.shape[1]
    k = (64 + d / 128) * F32  # a sum of squares in fp32 by 256 threads or more, and the operations after it
    hd = alpha * h.double()
    size = hd.abs()
    if y is not None:
        z = y.double()
        if post:
            z = z / (z.square().mean(1, keepdim=True) + eps).sqrt() * _weight(w_post, offset, z)
        z = z * (1.0 if gate is None else gate.double())
        hd, size = hd + z, size + z.abs()
    q = (hd.square().mean(1, keepdim=True) + eps).sqrt()
    w = _weight(w_pre, offset, hd)
    x = hd / q * w
    # x's norm also carries the elements' errors: at most their rms over q
    rel = (size.square().mean(1, keepdim=True)).sqrt() / q
    tol_x = k * w.abs() * (size / q + (hd / q).abs() * (1 + rel)) * (1 + BF16) + BF16 * x.abs()
    return (hd, x), (k * size * 1.01 + _step(h.dtype) * hd.abs(), tol_x)


def norm_grad_reference(y, h_out, gate, w_post, w_pre, post, alpha, eps, offset, gx, gh_out):
    """[gh, gy, g_w_pre, g_w_post, g_gate] in 64 bits (None where there is none) and tolerances."""
    M, d = h_out.shape
    k = 2 * (64 + d / 128) * F32

    def back(v, tv, vn, q):  # through vn = v / q, with tv the magnitude of v's parts
        out = (v - vn * (v * vn).mean(1, keepdim=True)) / q
        return out, (tv + vn.abs() * (tv * vn.abs()).mean(1, keepdim=True)) / q

    def total(v, tv):
        return v.sum(0), ((k + (M + 2) * F32) * tv).sum(0) + F32 * v.sum(0).abs()

    h = h_out.double()
    q = (h.square().mean(1, keepdim=True) + eps).sqrt()
    hn = h / q
    dh = torch.zeros_like(h) if gh_out is None else gh_out.double()
    size = dh.abs()
    res, tol = [None] * 5, [None] * 5
    if gx is not None:
        v = gx.double() * _weight(w_pre, offset, h)
        b, t = back(v, v.abs(), hn, q)
        dh, size = dh + b, size + t
        res[2], tol[2] = total(gx.double() * hn, (gx.double() * hn).abs())
    res[0], tol[0] = alpha * dh, k * abs(alpha) * size * 1.01 + _step(h_out.dtype) * (alpha * dh).abs()
    if y is not None:
        g = torch.ones(d, dtype=torch.float64, device=h.device) if gate is None else gate.double()
        yd = y.double()
        dz, tz = dh * g, size * g.abs()
        z = yd
        res[1], tz1 = dz, tz
        if post:
            yq = (yd.square().mean(1, keepdim=True) + eps).sqrt()
            yn, w = yd / yq, _weight(w_post, offset, h)
            z = yn * w
            res[1], tz1 = back(dz * w, tz * w.abs(), yn, yq)
            res[3], tol[3] = total(dz * yn, tz * yn.abs())
        tol[1] = 2 * k * tz1 * 1.01 + BF16 * res[1].abs()
        if gate is not None:
            if gate.dim() == 1:
                res[4], tol[4] = total(dh * z, size * z.abs())
            else:
                res[4], tol[4] = dh * z, k * size * z.abs() * 1.01 + BF16 * (dh * z).abs()
    return res, tol
