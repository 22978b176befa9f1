"""Edges of the low-rank adapters (nq_adapter_*): infinities, several tiles of the largest ranks in one cluster,
workspaces of captured calls, arguments refused before anything runs."""
import pytest
import torch

from tests.gpu_util import need_gpu, nq
from tests.operator_util import adapter_grad_reference, adapter_reference, check

pytestmark = pytest.mark.gpu

INF = float("inf")


def _make(M, d_in, d_out, rank, n, whole=False, seed=0):
    """whole: x, A and ybar are small whole numbers and B halves, so that t and u are exact in bf16."""
    g = torch.Generator(device="cuda").manual_seed(seed + M + 3 * rank)

    def rnd(*shape, std=1.0):
        v = torch.randn(shape, generator=g, device="cuda")
        return (v.clamp(-1, 1).round() if whole else v * std).bfloat16()

    ids = (torch.arange(M, device="cuda") % (n + 1) - 1).to(torch.int32)
    return dict(ids=ids, A=rnd(n, rank, d_in, std=d_in ** -0.5), B=rnd(n, d_out, rank, std=rank ** -0.5) / 2, x=rnd(M, d_in),
                y=rnd(M, d_out), ybar=rnd(M, d_out, std=0.1), xbar=rnd(M, d_in, std=0.1))


def _same_kind(got, ref, tol, what):
    """NaN where the definition has NaN, each infinity where it has that one, and within tolerance elsewhere."""
    got = got.double()
    for kind in (torch.isnan, torch.isposinf, torch.isneginf):
        wrong = kind(got) != kind(ref)
        assert not wrong.any(), "%s: %d wrong by %s" % (what, int(wrong.sum()), kind.__name__)
    f = ref.isfinite()
    check(got[f], ref[f], tol[f], what)


# the CUDA cores; products on the CUDA cores with gradients on the tensor cores; the tensor cores
@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("M,rank,n", [(6, 8, 2), (40, 16, 1), (300, 16, 2), (300, 120, 3)])
def test_adapter_infinities_as_the_definition_has_them(M, rank, n, whole):
    """An infinite weight or activation gives the infinity of the exact product, whichever kernel a batch gets:
    t and u enter the tensor cores' second products in parts, none of which may turn it into NaN."""
    need_gpu()
    clean = _make(M, 72, 136, rank, n, whole)
    groups = nq().adapter_rows(clean["ids"], n)
    t = torch.empty((M, rank), device="cuda")
    nq().adapter_forward(nq().Adapters(clean["A"], clean["B"]), groups, clean["x"], clean["y"], t=t)
    rows = (clean["ids"] == n - 1).nonzero()[:, 0]
    for where, at, value in (("B", (n - 1, 3, 2), INF), ("B", (0, 100, rank - 1), -INF), ("A", (n - 1, 1, 6), INF),
                             ("A", (0, rank - 1, 70), -INF), ("x", (int(rows[0]), 4), -INF), ("x", (int(rows[-1]), 71), INF),
                             ("ybar", (int(rows[0]), 7), INF), ("ybar", (int(rows[-1]), 135), -INF)):
        c = {k: v.clone() for k, v in clean.items()}
        c[where][at] = value
        ad = nq().Adapters(c["A"], c["B"])
        out = nq().adapter_forward(ad, groups, c["x"], c["y"])
        back = nq().adapter_backward(ad, groups, c["x"], c["ybar"], t, c["xbar"])
        nq().sync_status()
        ref, _, tol, _ = adapter_reference(c["A"], c["B"], None, c["ids"], c["x"], c["y"])
        _same_kind(out, ref, tol, "%s %s out" % (where, at))
        refs, tols = adapter_grad_reference(c["A"], c["B"], None, c["ids"], c["x"], c["ybar"], t, c["xbar"])
        for name, v, r, e in zip(("xbar", "gA", "gB"), back, refs, tols):
            _same_kind(v, r, e, "%s %s %s" % (where, at, name))
