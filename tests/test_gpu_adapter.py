"""Low-rank adapters of many requests beside a shared projection (nq_adapter_*) against 64 bits."""
import pytest
import torch

from tests.gpu_util import need_gpu, nq
from tests.operator_util import adapter_grad_reference, adapter_reference, check

pytestmark = pytest.mark.gpu


def _make(M, d_in, d_out, rank, n, ids=None, seed=0, pad=0, pad_b=None, scale=True):
    g = torch.Generator(device="cuda").manual_seed(seed + 31 * M + d_in)

    def rnd(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()

    if ids is None:
        ids = torch.randint(-1, n, (M,), generator=g, device="cuda", dtype=torch.int32)
    pad_b = pad if pad_b is None else pad_b
    A = rnd(n, rank, d_in + pad, std=d_in ** -0.5)[..., :d_in]
    B = rnd(n, d_out, rank + pad_b, std=rank ** -0.5)[..., :rank]
    s = torch.rand(n, generator=g, device="cuda") + 0.5 if scale else None
    return dict(ids=ids, A=A, B=B, scale=s, x=rnd(M, d_in), y=rnd(M, d_out), ybar=rnd(M, d_out, std=0.1),
                xbar=rnd(M, d_in, std=0.1))


def _run(c, what=""):
    ad = nq().Adapters(c["A"], c["B"], c["scale"])
    groups = nq().adapter_rows(c["ids"], ad.n)
    M = len(c["ids"])
    t = torch.full((M, ad.rank), -7.0, device="cuda")
    out = nq().adapter_forward(ad, groups, c["x"], c["y"], t=t)
    back = nq().adapter_backward(ad, groups, c["x"], c["ybar"], t, c["xbar"])
    nq().sync_status()
    ref, rt, tol, tol_t = adapter_reference(c["A"], c["B"], c["scale"], c["ids"], c["x"], c["y"])
    check(out, ref, tol, what + " out")
    check(t, rt, tol_t, what + " t")
    refs, tols = adapter_grad_reference(c["A"], c["B"], c["scale"], c["ids"], c["x"], c["ybar"], t, c["xbar"])
    for name, g, r, e in zip(("xbar", "gA", "gB"), back, refs, tols):
        check(g, r, e, what + " " + name)
    return ad, groups, t, out, back


# M, d_in, d_out, rank, n: single rows, widths and ranks that are no multiples of anything, tiles that
# end inside a group, the largest rank, more adapters than rows
SHAPES = [(1, 64, 96, 8, 1), (1, 5, 3, 1, 1), (7, 17, 33, 3, 4), (9, 256, 264, 16, 2), (64, 512, 1000, 16, 64),
          (130, 264, 136, 24, 3), (300, 1024, 72, 128, 5), (257, 2056, 520, 40, 2), (40, 1001, 515, 20, 7),
          (3, 128, 128, 104, 300), (700, 328, 4104, 64, 3), (65, 4096, 4096, 8, 1), (200, 72, 64, 127, 2),
          (129, 8, 8, 8, 1),
          # 17 to 150 tiles: every number of blocks that share one
          (2100, 640, 712, 16, 1), (3000, 576, 136, 24, 2), (4100, 136, 520, 64, 2), (5000, 584, 600, 8, 1),
          (9000, 72, 136, 40, 3), (700, 64, 72, 8, 1200), (700, 136, 72, 16, 100), (19000, 136, 72, 16, 2), (2100, 640, 520, 128, 1)]


@pytest.mark.parametrize("shape", SHAPES)
def test_adapter(shape):
    need_gpu()
    _run(_make(*shape), "%r" % (shape,))


@pytest.mark.parametrize("M,d_in,d_out,rank", [(100, 512, 384, 16), (33, 75, 39, 5)])
def test_adapter_groupings(M, d_in, d_out, rank):
    need_gpu()
    dev = "cuda"
    none = torch.full((M,), -1, dtype=torch.int32, device=dev)
    last = torch.full((M,), 4, dtype=torch.int32, device=dev)
    above = torch.full((M,), 1 << 30, dtype=torch.int32, device=dev)
    split = torch.where(torch.arange(M, device=dev) < M // 2 + 1, 3, 0).to(torch.int32)
    for ids, what in ((none, "none"), (last, "all the last"), (above, "none, by large ids"), (split, "two runs")):
        _run(_make(M, d_in, d_out, rank, 5, ids=ids), what)


@pytest.mark.parametrize("M", [50, 300])
@pytest.mark.parametrize("pad,scale", [(8, True), (3, False)])
def test_adapter_strides_and_unit_scale(M, pad, scale):
    need_gpu()
    _run(_make(M, 256, 320, 16, 3, pad=pad, scale=scale), "pad %d" % pad)


@pytest.mark.parametrize("M", [3, 40, 300])
@pytest.mark.parametrize("rank,pad_b", [(13, 3), (3, 5), (121, 7), (65, 7)])
def test_adapter_odd_ranks_with_rows_on_16_bytes(M, rank, pad_b):
    need_gpu()
    _run(_make(M, 200, 328, rank, 2, pad=8, pad_b=pad_b), "rank %d" % rank)


def test_adapter_rows_in_any_order():
    """A caller's own lists: the rows of a group need not be in order or side by side."""
    need_gpu()
    for M, n, d in ((20, 2, 64), (700, 3, 136), (700, 3, 139)):
        c = _make(M, d, d, 16, n)
        ad, groups, t, out, back = _run(c)
        order = torch.randperm(M, device="cuda")
        key = torch.where(c["ids"] < 0, n, c["ids"]).long()[order]
        rows = order[torch.sort(key, stable=True).indices].int()
        mine = nq().AdapterRows(rows, groups.offsets)
        t2 = torch.empty_like(t)
        assert torch.equal(nq().adapter_forward(ad, mine, c["x"], c["y"], t=t2), out) and torch.equal(t, t2)
        got = nq().adapter_backward(ad, mine, c["x"], c["ybar"], t, c["xbar"])
        assert torch.equal(got[0], back[0])
        refs, tols = adapter_grad_reference(c["A"], c["B"], c["scale"], c["ids"], c["x"], c["ybar"], t, c["xbar"])
        for g, r, e in zip(got, refs, tols):
            check(g, r, e, "rows in any order")
        nq().sync_status()


def test_adapter_first_call_of_a_process_inside_a_capture():
    """Nothing that a call sets up on its first use needs a call outside a capture before it."""
    need_gpu()
    code = """
import torch
from rank_binary_factorized_b200 import nq
torch.manual_seed(0)
for M in (3, 300):
    A, B = torch.randn(2, 16, 256, device="cuda").bfloat16(), torch.randn(2, 264, 16, device="cuda").bfloat16()
    x, y = torch.randn(M, 256, device="cuda").bfloat16(), torch.randn(M, 264, device="cuda").bfloat16()
    ids = torch.arange(M, device="cuda", dtype=torch.int32) % 2
    ad, t = nq.Adapters(A, B), torch.empty(M, 16, device="cuda")
    N = nq.BlockNorm(256, w_pre=x[0].clone())
    ws, wn = ad.workspace(M), N.workspace(M)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gr = nq.adapter_rows(ids, 2)
        out = nq.adapter_forward(ad, gr, x, y, t=t)
        back = nq.adapter_backward(ad, gr, x, y, t, x, ws=ws)
        norm = nq.block_norm(N, None, x)
        nback = nq.block_norm_backward(N, None, x, x, None, ws=wn)
    g.replay()
    torch.cuda.synchronize()
    kept = [v.clone() for v in (out, t) + back + norm + (nback[0], nback[2])]
    gr = nq.adapter_rows(ids, 2)
    t2 = torch.empty_like(t)
    want = [nq.adapter_forward(ad, gr, x, y, t=t2), t2] + list(nq.adapter_backward(ad, gr, x, y, t2, x))
    want += list(nq.block_norm(N, None, x))
    nb = nq.block_norm_backward(N, None, x, x, None)
    want += [nb[0], nb[2]]
    nq.sync_status()
    assert all(torch.equal(a, b) for a, b in zip(kept, want))
print("same")
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr


def test_adapter_rows_are_grouped_in_order():
    need_gpu()
    for M, n in ((1, 1), (5, 3), (1000, 7), (4097, 300), (64, 5000)):
        ids = torch.randint(-3, n + 2, (M,), dtype=torch.int32, device="cuda")
        g = nq().adapter_rows(ids, n)
        key = torch.where((ids < 0) | (ids >= n), n, ids).long()
        assert torch.equal(g.rows.long(), torch.sort(key, stable=True).indices)
        want = torch.bucketize(torch.arange(n + 1, device="cuda"), key.sort().values)
        assert torch.equal(g.offsets.long(), want)


@pytest.mark.parametrize("M,rank", [(12, 8), (400, 32), (30, 7)])
def test_adapter_nan_and_infinity_stay_where_they_are(M, rank):
    """Rows without an adapter do not read x, and an adapter or a row that holds NaN or infinity
    changes only its own rows, and only its own adapter's gradients."""
    need_gpu()
    c = _make(M, 264, 200, rank, 4, ids=torch.arange(M, device="cuda", dtype=torch.int32) % 5 - 1)
    ad, groups, t, out, back = _run(c)
    bad = {k: v.clone() for k, v in c.items()}
    bad["A"][2], bad["B"][2, 3] = float("nan"), float("inf")
    none = (c["ids"] < 0)
    bad["x"][none] = float("nan")
    bad["ybar"][none] = float("inf")
    bad["x"][1] = float("inf")  # row 1 has adapter 0
    ad2 = nq().Adapters(bad["A"], bad["B"], bad["scale"])
    t2 = torch.empty_like(t)
    out2 = nq().adapter_forward(ad2, groups, bad["x"], bad["y"], t=t2)
    keep = (c["ids"] != 2)
    keep[1] = False
    assert torch.equal(out2[keep], out[keep]) and torch.equal(t2[keep], t[keep])
    assert not t2[none].any() and torch.equal(out2[none], c["y"][none])
    back2 = nq().adapter_backward(ad2, groups, bad["x"], bad["ybar"], t2, bad["xbar"])
    assert torch.equal(back2[0][c["ids"] != 2], back[0][c["ids"] != 2])
    for a in (1, 3):
        assert torch.equal(back2[1][a], back[1][a]) and torch.equal(back2[2][a], back[2][a])


@pytest.mark.parametrize("M", [20, 500])
def test_adapter_in_place_and_parts_of_the_backward(M):
    need_gpu()
    c = _make(M, 512, 256, 16, 3)
    ad, groups, t, out, back = _run(c)
    y, xbar = c["y"].clone(), c["xbar"].clone()
    assert nq().adapter_forward(ad, groups, c["x"], y, out=y) is y and torch.equal(y, out)
    got = nq().adapter_backward(ad, groups, None, c["ybar"], None, xbar, out=xbar, need_weights=False)
    assert got[1] is None and got[2] is None and torch.equal(xbar, back[0])
    got = nq().adapter_backward(ad, groups, c["x"], c["ybar"], t, None, need_x=False)
    assert got[0] is None and torch.equal(got[1], back[1]) and torch.equal(got[2], back[2])


@pytest.mark.parametrize("M,width", [(6, 64), (6, 63), (300, 64)])
def test_adapter_bad_lists_are_reported(M, width):
    """A list entry that is no row is skipped, offsets out of order leave their adapters out, rows
    that are not listed stay as they were; the next status call says so once."""
    need_gpu()
    c = _make(M, width, width, 8, 2, ids=torch.zeros(M, dtype=torch.int32, device="cuda"))
    ad, groups, t, out, _ = _run(c)
    rows = groups.rows.clone()
    rows[1], rows[4] = M + 5, -2147483648
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[1] = keep[4] = False
    got = torch.full_like(out, 3.0)
    nq().adapter_forward(ad, nq().AdapterRows(rows, groups.offsets), c["x"], c["y"], out=got)
    with pytest.raises(nq().NQError) as e:
        nq().sync_status()
    assert e.value.status == 10
    nq().sync_status()
    assert torch.equal(got[keep], out[keep]) and (got[~keep] == 3.0).all()
    for offsets in ([0, M + 9, M], [0, -5, M], [3, 2, M], [0, 2147483647, 2147483647]):
        off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        groups2 = nq().AdapterRows(groups.rows, off)
        nq().adapter_forward(ad, groups2, c["x"], c["y"])
        nq().adapter_backward(ad, groups2, c["x"], c["ybar"], t, c["xbar"])
        with pytest.raises(nq().NQError) as e:
            nq().sync_status()
        assert e.value.status == 10
    nq().sync_status()


@pytest.mark.parametrize("M,n", [(60, 5), (300, 5), (300, 40), (300, 700), (300, 1500)])
def test_adapter_offsets_whose_groups_overlap(M, n):
    """Offsets that are each within 0..M but not in order (0, M, 0, M, ...): the first group counts, what
    follows is empty, and nothing is written behind the workspace."""
    need_gpu()
    c = _make(M, 64, 72, 16, n, ids=torch.zeros(M, dtype=torch.int32, device="cuda"))
    ad, groups, t, out, back = _run(c)
    off = torch.tensor([M * (i % 2) for i in range(n + 1)], dtype=torch.int32, device="cuda")
    bad = nq().AdapterRows(groups.rows, off)
    need = ad.workspace_bytes(M)
    ws = torch.full((need + 4096 * n,), 0x5A, dtype=torch.uint8, device="cuda")
    t2 = torch.zeros_like(t)
    got = nq().adapter_forward(ad, bad, c["x"], c["y"], t=t2)
    grads = nq().adapter_backward(ad, bad, c["x"], c["ybar"], t, c["xbar"], ws=ws)
    with pytest.raises(nq().NQError) as e:
        nq().sync_status()
    assert e.value.status == 10
    assert (ws[need:] == 0x5A).all()
    assert torch.equal(got, out) and torch.equal(t2, t)
    assert torch.equal(grads[0], back[0]) and torch.equal(grads[1][0], back[1][0]) and torch.equal(grads[2][0], back[2][0])


def test_adapter_repeats_on_other_streams_and_in_graphs():
    need_gpu()
    for M in (24, 600):
        c = _make(M, 1024, 512, 16, 4)
        ad, groups, t, out, back = _run(c)
        torch.cuda.synchronize()
        outs = []
        for s in [torch.cuda.Stream() for _ in range(3)]:
            ws = torch.empty(ad.workspace_bytes(M), dtype=torch.uint8, device="cuda")
            outs.append((nq().adapter_forward(ad, groups, c["x"], c["y"], stream=s),) +
                        nq().adapter_backward(ad, groups, c["x"], c["ybar"], t, c["xbar"], ws=ws, stream=s) + (ws,))
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(p, q) for p, q in zip((out,) + back, o))
        ids, got = c["ids"].clone(), torch.empty_like(out)
        ad.workspace(M)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):  # the grouping too: a replay follows the ids
            gr = nq().adapter_rows(ids, ad.n)
            nq().adapter_forward(ad, gr, c["x"], c["y"], out=got)
            gb = nq().adapter_backward(ad, gr, c["x"], c["ybar"], t, c["xbar"])
        ids.fill_(-1)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, c["y"]) and torch.equal(gb[0], c["xbar"]) and not gb[1].any() and not gb[2].any()
        ids.copy_(c["ids"])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, out) and all(torch.equal(p, q) for p, q in zip(gb, back))


def test_adapter_beyond_31_bit_offsets():
    need_gpu()
    M, d_in, d_out = 270001, 64, 8192  # 2.2e9 elements of y
    g = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    ids[M - 5:] = torch.tensor([1, 0, -1, 1, 0], device="cuda")
    x = torch.empty((M, d_in), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    y = torch.empty((M, d_out), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    A = torch.empty((2, 8, d_in), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    B = torch.empty((2, d_out, 8), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    ad = nq().Adapters(A, B)
    groups = nq().adapter_rows(ids, 2)
    part = slice(M - 5, M)
    ref, _, tol, _ = adapter_reference(A, B, None, ids[part], x[part], y[part])
    base = y[part].clone()
    nq().adapter_forward(ad, groups, x, y, out=y)
    nq().sync_status()
    check(y[part], ref, tol, "far rows")
    xb = nq().adapter_backward(ad, groups, None, y, None, x, need_weights=False)[0]
    nq().sync_status()
    refs, tols = adapter_grad_reference(A, B, None, ids[part], x[part], y[part], x[part, :8].float(), x[part])
    check(xb[part], refs[0], tols[0], "far gradients")
    assert torch.equal(y[M - 3], base[2])


def test_adapter_gradients_against_differences():
    """A loss linear in the output: differences of the 64-bit forward in each operand are exact up to
    rounding, as the output is linear in each."""
    need_gpu()
    c = _make(6, 24, 16, 8, 2, ids=torch.tensor([0, 1, 1, -1, 0, 1], dtype=torch.int32, device="cuda"))
    ad = nq().Adapters(c["A"], c["B"], c["scale"])
    groups = nq().adapter_rows(c["ids"], 2)
    t = torch.empty((6, 8), device="cuda")
    nq().adapter_forward(ad, groups, c["x"], c["y"], t=t)
    got = nq().adapter_backward(ad, groups, c["x"], c["ybar"], t, torch.zeros_like(c["xbar"]))

    def loss(x, A, B):
        return (adapter_reference(A, B, c["scale"], c["ids"], x, c["y"])[0] * c["ybar"].double()).sum()

    base = [c[k].double() for k in ("x", "A", "B")]
    for which, grad in enumerate(got):
        num = torch.zeros_like(base[which])
        flat = num.view(-1)
        for i in range(flat.numel()):
            v = [b.clone() for b in base]
            v[which].view(-1)[i] += 0.5
            up = loss(*v)
            v[which].view(-1)[i] -= 1.0
            flat[i] = up - loss(*v)
        # half a bf16 unit, and what t and u carry: 2^-16 and their fp32 sums
        assert (grad.double() - num).abs().max() <= 2.0 ** -8 * num.abs().max() + 2.0 ** -14 * num.abs().max()
