"""Edges of the low-rank adapters (nq_adapter_*): infinities, several tiles of the largest ranks in one cluster,
workspaces of captured calls, arguments refused before anything runs."""
import pytest
import torch

from tests.gpu_util import need_gpu, nq
from tests.operator_util import adapter_grad_reference, adapter_reference, check
from tests.test_gpu_adapter import _make as make_batch
from tests.test_gpu_adapter import _run as run_and_check

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


def _again(c, ad, groups, t, out, back, times):
    """The same calls give the same bits."""
    for _ in range(times):
        t2 = torch.empty_like(t)
        assert torch.equal(nq().adapter_forward(ad, groups, c["x"], c["y"], t=t2), out) and torch.equal(t2, t)
        got = nq().adapter_backward(ad, groups, c["x"], c["ybar"], t, c["xbar"])
        assert all(torch.equal(p, q) for p, q in zip(got, back))
    nq().sync_status()


# Groups of 129 rows make two tiles each, more than the launch reckons with, so that a cluster of 8, 6, 4, 2 or 1
# blocks takes a second tile (the hand-over of the inbox, the staging tiles, t's rows and the slots between tiles).
@pytest.mark.parametrize("groups_of_129", [10, 14, 21, 46, 160])
@pytest.mark.parametrize("rank", [128, 72, 40])
@pytest.mark.parametrize("in_order", [True, False])
def test_adapter_clusters_that_take_several_tiles(groups_of_129, rank, in_order):
    """rows side by side (TMA boxes and stores) and in any order (row gathers, stores by threads)."""
    need_gpu()
    n = groups_of_129
    ids = torch.arange(n, device="cuda", dtype=torch.int32).repeat_interleave(129)
    if not in_order:
        ids = ids[torch.randperm(len(ids), generator=torch.Generator(device="cuda").manual_seed(n), device="cuda")]
    c = make_batch(len(ids), 264, 328, rank, n, ids=ids)
    _again(c, *run_and_check(c, "%d groups, rank %d" % (n, rank)), 5)


# more tiles than clusters by rows alone, and by ragged groups; more units of the gradients than multiprocessors
@pytest.mark.parametrize("shape", [(40000, 136, 72, 128, 2), (700, 136, 72, 104, 300), (600, 2056, 4104, 128, 8),
                                   (600, 2056, 4104, 64, 8)])
def test_adapter_large_ranks_over_many_tiles(shape):
    need_gpu()
    c = make_batch(*shape)
    _again(c, *run_and_check(c, "%r" % (shape,)), 5)


def test_captured_calls_do_not_depend_on_a_cached_workspace_that_grows():
    """A captured call that passes no workspace keeps none that a later, larger call would replace: what is then
    allocated in its place stays as it is when the graph is replayed."""
    need_gpu()
    c, large = make_batch(300, 264, 328, 16, 2), make_batch(1200, 264, 328, 16, 2)
    ad, groups, t, out, back = run_and_check(c)
    N = nq().BlockNorm(264, w_pre=c["x"][0].clone())
    want = nq().block_norm_backward(N, None, c["x"], c["xbar"], None)
    ws, wn = ad.workspace(300), N.workspace(300)
    sizes = [ws.numel(), wn.numel()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = nq().adapter_backward(ad, groups, c["x"], c["ybar"], t, c["xbar"])
        gn = nq().block_norm_backward(N, None, c["x"], c["xbar"], None)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, back)) and torch.equal(gn[0], want[0]) and torch.equal(gn[2], want[2])
    del ws, wn
    assert ad.workspace(1200).numel() > sizes[0]
    ad.workspace(1200), N.workspace(12000)  # grown: the old ones are given back
    theirs = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    for v in got + (gn[0], gn[2]):
        v.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all((v == 0x5A).all() for v in theirs)
    assert all(torch.equal(p, q) for p, q in zip(got, back)) and torch.equal(gn[0], want[0]) and torch.equal(gn[2], want[2])


def test_two_graphs_without_workspaces_run_at_the_same_time():
    need_gpu()
    c = make_batch(2000, 264, 328, 64, 3)
    ad, groups, t, _, _ = run_and_check(c)
    N = nq().BlockNorm(264, w_pre=c["x"][0].clone())
    inputs = [(c["x"], c["ybar"], c["xbar"]), tuple(-2 * c[k].flip(0) for k in ("x", "ybar", "xbar"))]
    want = [nq().adapter_backward(ad, groups, x, yb, t, xb) + nq().block_norm_backward(N, None, x, xb, None)
            for x, yb, xb in inputs]
    graphs, results, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for x, yb, xb in inputs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            results.append([nq().adapter_backward(ad, groups, x, yb, t, xb) + nq().block_norm_backward(N, None, x, xb, None)
                            for _ in range(8)])
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for one, w in zip(results, want):
            assert all(torch.equal(p, q) for r in one for p, q in zip(r, w) if q is not None)


def test_captured_call_on_a_forked_stream():
    """A capture that forks to another stream: the workspace is not reused on the first one meanwhile."""
    need_gpu()
    c = make_batch(300, 264, 328, 16, 2)
    ad, groups, t, out, back = run_and_check(c)
    side, g, M = torch.cuda.Stream(), torch.cuda.CUDAGraph(), 300
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        got = nq().adapter_backward(ad, groups, c["x"], c["ybar"], t, c["xbar"], stream=side)
        other = [torch.zeros(ad.workspace_bytes(M), dtype=torch.uint8, device="cuda") for _ in range(4)]
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, back)) and not any(v.any() for v in other)
