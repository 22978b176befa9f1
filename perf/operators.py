"""Cases of the operators around a low-rank binary projection: the low-rank adapters of many requests
beside it (forward, backward) and the norms, gate and residual between blocks (forward, backward).

`run` computes them from elementary torch operations in 32 bits, or, where `own` is true, calls the
package.  Sizes are those of the layers this repository is built for: 7B (4096, 11008) and 70B (8192,
28672) projections, decode batches and prefills up to 8192 tokens, adapter ranks 8 to 128.
"""
import math

import torch

own = False

EPS = 1e-5


def _adapter(name, op, M, d_in, d_out, rank, n, used, none, mixed):
    """M rows; n adapters are loaded, `used` of them occur in the batch, `none` rows have no adapter; mixed: every
    row is a request of its own (decode), otherwise requests are runs of rows (prefill, training)."""
    return {"name": name, "op": op, "M": M, "d_in": d_in, "d_out": d_out, "rank": rank, "n": n, "used": used, "none": none, "mixed": mixed}


def _norm(name, op, M, d, f32, post, gate):
    """M rows of d; f32: the residual stream is kept in 32 bits; post: the block's output is normed too; gate: "none",
    "channel" (one vector) or "row" (a vector a row)."""
    return {"name": name, "op": op, "M": M, "d": d, "f32": f32, "post": post, "gate": gate}


def listed():
    return [
        # one request with an adapter, a 7B attention projection: latency
        _adapter("adapter 1 token", "adapter", 1, 4096, 4096, 16, 8, 1, 0, True),
        # a decode batch of 64 requests, most with an adapter of their own, a 70B attention projection
        _adapter("adapter 64 requests", "adapter", 64, 8192, 8192, 16, 64, 40, 6, True),
        # a prefill of a few requests with ragged lengths, a 7B gate projection, an uneven rank
        _adapter("adapter ragged prefill", "adapter", 1777, 4096, 11008, 24, 6, 5, 100, False),
        # the largest prefill beside a 70B gate projection
        _adapter("adapter long prefill", "adapter", 8192, 8192, 28672, 64, 4, 4, 0, False),
        # a small tuning batch of two tenants
        _adapter("adapter grad small", "adapter_grad", 96, 4096, 4096, 8, 2, 2, 0, False),
        # three tenants tuned together at the largest rank, ragged, a 7B gate projection
        _adapter("adapter grad ragged", "adapter_grad", 2500, 4096, 11008, 128, 3, 3, 60, False),
        # one adapter tuned beside a 70B gate projection
        _adapter("adapter grad large", "adapter_grad", 4096, 8192, 28672, 64, 1, 1, 0, False),
        # between two blocks while decoding one token of a 70B model: latency
        _norm("norm 1 token", "norm", 1, 8192, False, False, "none"),
        # a middling batch, norms on both sides of the block, a gate per channel
        _norm("norm both sides", "norm", 300, 4096, False, True, "channel"),
        # a long prefill, residual stream in 32 bits, a gate per row
        _norm("norm long prefill", "norm", 16384, 8192, True, True, "row"),
        # gradients of a small batch, odd width
        _norm("norm grad odd", "norm_grad", 77, 4095, False, True, "channel"),
        # gradients of a long batch
        _norm("norm grad long", "norm_grad", 8192, 8192, False, True, "channel"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adapter", "adapter_grad", "norm", "norm_grad"])
    if op in ("adapter", "adapter_grad"):
        M = _log(rng, 1, 8192 if op == "adapter" else 4096)
        rank = 8 * _log(rng, 1, min(16, (65536 if op == "adapter" else 32768) // M))
        d_in, d_out = 8 * _log(rng, 32, 1024), 8 * _log(rng, 32, 3584)
        mixed = M <= 256 and rng.random() < 0.7
        used = min(M, _log(rng, 1, 64 if mixed else 8))
        none = rng.randint(0, M - used) // 4
        n = used + rng.randint(0, 3)
        c = _adapter("", op, M, d_in, d_out, rank, n, used, none, mixed)
    else:
        M, d = _log(rng, 1, 16384 if op == "norm" else 8192), _log(rng, 100, 8192)
        c = _norm("", op, M, d, rng.random() < 0.5, rng.random() < 0.6, rng.choice(["none", "channel", "row"]))
    del c["name"]
    return c


def _rows_of(case, gen):
    """The adapter of each row (-1: none), the rows grouped by adapter and where each adapter's rows begin."""
    M, n, used, none = case["M"], case["n"], case["used"], case["none"]
    dev = "cuda"
    which = torch.randperm(n, generator=gen, device=dev)[:used]
    with_one = M - none
    if case["mixed"]:
        ids = torch.full((M,), -1, dtype=torch.int64, device=dev)
        ids[:with_one] = which[torch.arange(with_one, device=dev) % used]
        ids = ids[torch.randperm(M, generator=gen, device=dev)]
    else:  # runs of rows with ragged lengths, one for each adapter used, rows without one last
        cuts = torch.randperm(with_one - 1, generator=gen, device=dev)[:used - 1].sort().values + 1
        ids = torch.full((M,), -1, dtype=torch.int64, device=dev)
        ids[:with_one] = which[torch.bucketize(torch.arange(with_one, device=dev), cuts, right=True)]
    key = torch.where(ids < 0, n, ids)
    order = torch.sort(key, stable=True).indices
    offsets = torch.bucketize(torch.arange(n + 1, device=dev), key[order], right=False)
    return ids, order.to(torch.int32), offsets.to(torch.int32)


def _spread(ids, n, rank):
    """[M][n * rank]: whether the column belongs to the row's adapter."""
    return ids[:, None] == torch.arange(n, device=ids.device).repeat_interleave(rank)[None, :]


def _flat(A, B):
    n, rank, d_in = A.shape
    return A.float().reshape(n * rank, d_in), B.float().permute(0, 2, 1).reshape(n * rank, -1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dev = "cuda"

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device=dev).mul_(std).add_(mean).to(dtype)

    M = case["M"]
    if case["op"] in ("adapter", "adapter_grad"):
        d_in, d_out, rank, n = case["d_in"], case["d_out"], case["rank"], case["n"]
        ids, rows, offsets = _rows_of(case, gen)
        A = normal(n, rank, d_in, std=d_in ** -0.5)
        B = normal(n, d_out, rank, std=0.3 * rank ** -0.5)
        scale = torch.rand(n, generator=gen, device=dev) + 0.5
        s = {"op": case["op"], "ids": ids, "rows": rows, "offsets": offsets, "A": A, "B": B, "scale": scale, "x": normal(M, d_in)}
        if case["op"] == "adapter":
            s["y"] = normal(M, d_out)
            s["out"] = torch.empty_like(s["y"])
        else:
            s["ybar"], s["xbar"] = normal(M, d_out, std=0.1), normal(M, d_in, std=0.1)
            t = s["x"].float() @ _flat(A, B)[0].T  # what the forward pass kept: scale * A x of the row's adapter
            t = torch.where(_spread(ids, n, rank), t * scale.repeat_interleave(rank), 0.0)
            s["t"] = t.reshape(M, n, rank).sum(1)
            s["out"], s["gA"], s["gB"] = torch.empty_like(s["xbar"]), torch.empty_like(A), torch.empty_like(B)
        if own:  # the handle that a program keeps with its adapters: addresses and sizes, nothing computed
            from rank_binary_factorized_b200 import nq
            s["adapters"] = nq.Adapters(A, B, scale)
            s["groups"] = nq.AdapterRows(rows, offsets)
            if case["op"] == "adapter_grad":
                s["ws"] = s["adapters"].workspace(M)
        return s
    d = case["d"]
    htype = torch.float32 if case["f32"] else torch.bfloat16
    s = {"op": case["op"], "alpha": 0.875, "post": case["post"], "per_row": case["gate"] == "row"}
    s["w_pre"] = normal(d, std=0.1, mean=1.0)
    s["w_post"] = normal(d, std=0.1, mean=0.5) if case["post"] else None
    s["gate"] = {"none": None, "channel": (d,), "row": (M, d)}[case["gate"]]
    s["gate"] = None if s["gate"] is None else normal(*s["gate"], std=0.3, mean=0.8)
    s["y"] = normal(M, d, std=2.0)
    s["h"] = normal(M, d, std=1.5, dtype=htype)
    f32 = {"device": dev, "dtype": torch.float32}
    if case["op"] == "norm":
        s["h_out"], s["x"] = torch.empty_like(s["h"]), torch.empty_like(s["y"])
    else:  # h is then the residual stream after the block, as the forward pass kept it
        s["gx"], s["gh_out"] = normal(M, d, std=0.1), normal(M, d, std=0.1, dtype=htype)
        s["gh"], s["gy"], s["g_w_pre"] = torch.empty_like(s["h"]), torch.empty_like(s["y"]), torch.empty(d, **f32)
        s["g_w_post"] = torch.empty(d, **f32) if case["post"] else None
        s["g_gate"] = {"none": None, "channel": torch.empty(d, **f32), "row": torch.empty_like(s["y"])}[case["gate"]]
    if own:  # likewise
        from rank_binary_factorized_b200 import nq
        s["norm"] = nq.BlockNorm(d, w_pre=s["w_pre"], w_post=s["w_post"], post_norm=case["post"], alpha=s["alpha"], eps=EPS)
        if case["op"] == "norm_grad":
            s["ws"] = s["norm"].workspace(M)
    return s


def _own(s):
    from rank_binary_factorized_b200 import nq
    if s["op"] == "adapter":
        return nq.adapter_forward(s["adapters"], s["groups"], s["x"], s["y"], out=s["out"])
    if s["op"] == "adapter_grad":
        return nq.adapter_backward(s["adapters"], s["groups"], s["x"], s["ybar"], s["t"], s["xbar"], out=s["out"], gA=s["gA"], gB=s["gB"],
                                   ws=s["ws"])
    if s["op"] == "norm":
        return nq.block_norm(s["norm"], s["y"], s["h"], gate=s["gate"], h_out=s["h_out"], x=s["x"])
    return nq.block_norm_backward(s["norm"], s["y"], s["h"], s["gx"], s["gh_out"], gate=s["gate"], gh=s["gh"], gy=s["gy"],
                                  g_w_pre=s["g_w_pre"], g_w_post=s["g_w_post"], g_gate=s["g_gate"], ws=s["ws"])


def run(s):
    if own:
        return _own(s)
    if s["op"] in ("adapter", "adapter_grad"):
        n, rank = s["A"].shape[:2]
        A, B = _flat(s["A"], s["B"])
        mine, scale = _spread(s["ids"], n, rank), s["scale"].repeat_interleave(rank)
        x = s["x"].float()
        if s["op"] == "adapter":
            t = torch.where(mine, (x @ A.T) * scale, 0.0)
            return (s["y"].float() + t @ B).bfloat16()
        ybar = s["ybar"].float()
        u = torch.where(mine, (ybar @ B.T) * scale, 0.0)
        t = torch.where(mine, s["t"].repeat(1, n), 0.0)
        out = (s["xbar"].float() + u @ A).bfloat16()
        gA = (u.T @ x).reshape(s["A"].shape).bfloat16()
        gB = (t.T @ ybar).reshape(n, rank, -1).permute(0, 2, 1).contiguous().bfloat16()
        return out, gA, gB
    y, h, d = s["y"].float(), s["h"].float(), s["y"].shape[1]
    w_pre = s["w_pre"].float()
    gate = 1.0 if s["gate"] is None else s["gate"].float()
    r_post = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
    z = y * r_post * s["w_post"].float() if s["post"] else y
    if s["op"] == "norm":
        h = s["alpha"] * h + gate * z
        x = w_pre * h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
        return h.to(s["h"].dtype), x.bfloat16()
    gx = s["gx"].float()
    r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    v = w_pre * gx
    dh = s["gh_out"].float() + r * v - h * r.pow(3) * ((v * h).sum(1, keepdim=True) / d)
    dz = gate * dh
    out = [(s["alpha"] * dh).to(s["h"].dtype), dz.bfloat16(), (gx * h * r).sum(0), None, None]
    if s["post"]:
        v = dz * s["w_post"].float()
        out[1] = (r_post * v - y * r_post.pow(3) * ((v * y).sum(1, keepdim=True) / d)).bfloat16()
        out[3] = (dz * y * r_post).sum(0)
    if s["gate"] is not None:
        out[4] = (dh * z).bfloat16() if s["per_row"] else (dh * z).sum(0)
    return tuple(out)


def exact(case, seed):
    """The definitions in 64 bits: adapters one after the other over their own rows, norms through each row's unit vector."""
    s = prepare(case, seed)
    if s["op"] in ("adapter", "adapter_grad"):
        pick = [(a, (s["ids"] == a).nonzero()[:, 0]) for a in range(case["n"])]
        if s["op"] == "adapter":
            y = s["y"].double()
            for a, m in pick:
                y[m] += s["scale"][a].double() * ((s["x"][m].double() @ s["A"][a].double().T) @ s["B"][a].double().T)
            return y
        xbar, gA, gB = s["xbar"].double(), torch.zeros_like(s["A"], dtype=torch.float64), torch.zeros_like(s["B"], dtype=torch.float64)
        for a, m in pick:
            yb = s["ybar"][m].double()
            u = s["scale"][a].double() * (yb @ s["B"][a].double())
            xbar[m] += u @ s["A"][a].double()
            gA[a] = u.T @ s["x"][m].double()
            gB[a] = yb.T @ s["t"][m].double()
        return xbar, gA, gB

    def unit(v):  # v over its root mean square, and that
        q = (v.square().mean(1, keepdim=True) + EPS).sqrt()
        return v / q, q

    y, h = s["y"].double(), s["h"].double()
    w, wp = s["w_pre"].double(), s["w_post"].double() if s["post"] else None
    g = torch.ones((), dtype=torch.float64, device=y.device) if s["gate"] is None else s["gate"].double()
    yn, yq = unit(y)
    z = yn * wp if s["post"] else y
    if s["op"] == "norm":
        h = s["alpha"] * h + g * z
        return h, unit(h)[0] * w

    def back(v, vn, q):  # through vn = v / q
        return (v - vn * (v * vn).mean(1, keepdim=True)) / q

    hn, hq = unit(h)
    gx = s["gx"].double()
    dh = s["gh_out"].double() + back(gx * w, hn, hq)
    dz = dh * g
    gy = back(dz * wp, yn, yq) if s["post"] else dz
    g_gate = None if s["gate"] is None else dh * z if s["per_row"] else (dh * z).sum(0)
    return s["alpha"] * dh, gy, (gx * hn).sum(0), (dz * yn).sum(0) if s["post"] else None, g_gate


def work(case):
    M = case["M"]
    if case["op"] in ("adapter", "adapter_grad"):
        d_in, d_out, rank = case["d_in"], case["d_out"], case["rank"]
        rows = M - case["none"]  # rows with an adapter: the others' x and ybar are not needed
        weights = 2 * case["used"] * rank * (d_in + d_out) + 4 * case["used"]
        lists = 4 * (M + case["n"] + 1)
        if case["op"] == "adapter":
            return {"bytes": 2 * (rows * d_in + 2 * M * d_out) + weights + lists, "flops": 2 * rows * rank * (d_in + d_out)}
        grads = 2 * case["n"] * rank * (d_in + d_out)
        return {"bytes": 2 * (rows * (d_in + d_out) + 2 * M * d_in) + 4 * rows * rank + weights + grads + lists,
                "flops": 4 * rows * rank * (d_in + d_out)}
    d, e = case["d"], 4 if case["f32"] else 2
    gate = {"none": 0, "channel": 2 * d, "row": 2 * M * d}[case["gate"]]
    vectors = 2 * d * (2 if case["post"] else 1)
    if case["op"] == "norm":
        return {"bytes": M * d * (2 + e + e + 2) + gate + vectors, "flops": M * d * (11 if case["post"] else 7)}
    sums = 4 * d * (1 + case["post"] + (case["gate"] == "channel")) + (2 * M * d if case["gate"] == "row" else 0)
    reads_y = case["post"] or case["gate"] != "none"
    return {"bytes": M * d * (2 * reads_y + e + 2 + e + e + 2) + gate + vectors + sums, "flops": M * d * (30 if case["post"] else 16)}
