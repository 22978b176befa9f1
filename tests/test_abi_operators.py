"""Refusals of the adapter and block-norm entry points, on the host, before anything is launched.
No pointer below is ever dereferenced."""
import ctypes

import pytest
import torch

NULL, SHAPE, ALIGN, WORKSPACE, DEVICE, VALUE = 1, 2, 3, 4, 5, 9


@pytest.fixture(scope="module")
def nq():
    from rank_binary_factorized_b200 import nq as mod
    return mod


def _set(nq, n=2, rank=8, d_in=64, d_out=96, A=0x10000, lda=None, B=0x20000, ldb=None, scale=0x30000):
    return nq.nq_adapters(n, rank, d_in, d_out, A, d_in if lda is None else lda, B, rank if ldb is None else ldb, scale)


BAD_SETS = [(dict(A=0), NULL), (dict(B=0), NULL), (dict(n=0), SHAPE), (dict(n=16385), SHAPE), (dict(rank=0), SHAPE),
            (dict(rank=129), SHAPE), (dict(d_in=0), SHAPE), (dict(d_out=-1), SHAPE), (dict(lda=63), SHAPE),
            (dict(ldb=7), SHAPE), (dict(d_in=1 << 31), SHAPE), (dict(A=0x10008), ALIGN), (dict(scale=0x30004), ALIGN)]


def _forward(nq, S, rows=0x40000, offsets=0x50000, x=0x60000, y=0x70000, out=0x80000, t=0, M=4):
    return nq.raw_lib().nq_adapter_forward(ctypes.byref(S) if S is not None else None, rows, offsets, x, y, out, t, M, None)


def _backward(nq, S, rows=0x40000, offsets=0x50000, x=0x60000, ybar=0x70000, t=0x80000, xbar=0x90000, out=0xA0000,
              gA=0xB0000, gB=0xC0000, M=4, ws=0xD0000, ws_bytes=1 << 30):
    return nq.raw_lib().nq_adapter_backward(ctypes.byref(S) if S is not None else None, rows, offsets, x, ybar, t, xbar,
                                            out, gA, gB, M, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", BAD_SETS)
def test_adapter_sets(nq, kw, status):
    S = _set(nq, **kw)
    assert _forward(nq, S) == status and _backward(nq, S) == status
    assert nq.raw_lib().nq_adapter_workspace_bytes(ctypes.byref(S), 4) == 0


def test_adapter_arguments(nq):
    S = _set(nq)
    assert _forward(nq, None) == NULL and _backward(nq, None) == NULL
    for M in (0, -1, 1 << 31):
        assert _forward(nq, S, M=M) == SHAPE and _backward(nq, S, M=M) == SHAPE
        assert nq.raw_lib().nq_adapter_workspace_bytes(ctypes.byref(S), M) == 0
    for k in ("rows", "offsets", "x", "y", "out"):
        assert _forward(nq, S, **{k: 0}) == NULL
        assert _forward(nq, S, **{k: 0x60008}) == ALIGN
    assert _forward(nq, S, t=0x60004) == ALIGN
    for k in ("rows", "offsets", "x", "ybar", "t", "xbar", "ws"):
        assert _backward(nq, S, **{k: 0}) == NULL
    for k in ("rows", "offsets", "x", "ybar", "t", "xbar", "out", "gA", "gB", "ws"):
        assert _backward(nq, S, **{k: 0x60008}) == ALIGN
    assert _backward(nq, S, ws_bytes=16) == WORKSPACE
    assert nq.raw_lib().nq_adapter_workspace_bytes(ctypes.byref(S), 4) > 4 * 8 * 4
    if not torch.cuda.is_available():
        assert _forward(nq, S) == DEVICE and _backward(nq, S) == DEVICE
        assert _backward(nq, S, x=0, t=0, gA=0, gB=0) == DEVICE  # only xbar: x and t are not needed
        assert _backward(nq, S, xbar=0, out=0) == DEVICE


def test_adapter_rows_arguments(nq):
    f = nq.raw_lib().nq_adapter_rows
    assert f(0x1000, 0, 2, 0x2000, 0x3000, None) == SHAPE
    assert f(0x1000, 4, 0, 0x2000, 0x3000, None) == SHAPE
    assert f(0x1000, 4, 16385, 0x2000, 0x3000, None) == SHAPE
    assert f(0, 4, 2, 0x2000, 0x3000, None) == NULL
    assert f(0x1000, 4, 2, 0, 0x3000, None) == NULL
    assert f(0x1000, 4, 2, 0x2000, 0, None) == NULL
    assert f(0x1004, 4, 2, 0x2000, 0x3000, None) == ALIGN


def _norm(nq, d=64, w_pre=0x1000, w_post=0x2000, off=0.0, alpha=1.0, eps=1e-5, post=1, f32=0):
    return nq.nq_block_norm(d, w_pre, w_post, off, alpha, eps, post, f32)


def _nf(nq, N, y=0x10000, h=0x20000, gate=0x30000, ld=0, h_out=0x40000, x=0x50000, M=3):
    return nq.raw_lib().nq_block_norm_forward(ctypes.byref(N) if N is not None else None, y, h, gate, ld, h_out, x, M, None)


def _nb(nq, N, y=0x10000, h_out=0x20000, gate=0x30000, ld=0, gx=0x40000, gh_out=0x50000, gh=0x60000, gy=0x70000,
        gwp=0x80000, gwo=0x90000, gg=0xA0000, M=3, ws=0xB0000, ws_bytes=1 << 30):
    return nq.raw_lib().nq_block_norm_backward(ctypes.byref(N) if N is not None else None, y, h_out, gate, ld, gx, gh_out,
                                               gh, gy, gwp, gwo, gg, M, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=0), SHAPE), (dict(d=(1 << 20) + 1), SHAPE), (dict(eps=0.0), VALUE), (dict(eps=-1.0), VALUE),
    (dict(eps=float("nan")), VALUE), (dict(eps=float("inf")), VALUE), (dict(alpha=float("nan")), VALUE),
    (dict(off=float("inf")), VALUE), (dict(post=2), VALUE), (dict(f32=-1), VALUE), (dict(w_pre=0x1004), ALIGN),
    (dict(w_post=0x2002), ALIGN)])
def test_norm_parameters(nq, kw, status):
    N = _norm(nq, **kw)
    assert _nf(nq, N) == status and _nb(nq, N) == status
    assert nq.raw_lib().nq_block_norm_workspace_bytes(ctypes.byref(N), 3) == 0


def test_norm_arguments(nq):
    N = _norm(nq)
    assert _nf(nq, None) == NULL and _nb(nq, None) == NULL
    for M in (0, -2, 1 << 31):
        assert _nf(nq, N, M=M) == SHAPE and _nb(nq, N, M=M) == SHAPE
    assert _nf(nq, N, h=0) == NULL and _nf(nq, N, h_out=0, x=0) == NULL
    assert _nf(nq, N, ld=63) == SHAPE and _nb(nq, N, ld=-64) == SHAPE
    for k in ("y", "h", "gate", "h_out", "x"):
        assert _nf(nq, N, **{k: 0x10002}) == ALIGN
    for k in ("y", "h_out", "gate", "gx", "gh_out", "gh", "gy", "gwp", "gwo", "gg", "ws"):
        assert _nb(nq, N, **{k: 0x10002}) == ALIGN
    assert _nb(nq, N, h_out=0) == NULL and _nb(nq, N, ws=0) == NULL
    assert _nb(nq, N, y=0) == NULL  # gy needs y
    assert _nb(nq, N, gate=0) == NULL  # g_gate needs the gate
    assert _nb(nq, _norm(nq, post=0)) == VALUE  # g_w_post needs the norm
    assert _nb(nq, N, ws_bytes=16) == WORKSPACE
    if not torch.cuda.is_available():
        assert _nf(nq, N) == DEVICE and _nb(nq, N) == DEVICE
        assert _nf(nq, N, y=0, gate=0, h_out=0) == DEVICE


def test_binding_refuses_host_tensors(nq):
    z = torch.zeros
    with pytest.raises(ValueError, match="CUDA"):
        nq.Adapters(z((2, 8, 64), dtype=torch.bfloat16), z((2, 96, 8), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA"):
        nq.adapter_rows(z(4, dtype=torch.int32), 2)
    with pytest.raises(ValueError, match="CUDA"):
        nq.AdapterRows(z(4, dtype=torch.int32), z(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        nq.BlockNorm(64, w_pre=z(64, dtype=torch.bfloat16))
    N = nq.BlockNorm(64)
    with pytest.raises(ValueError, match="CUDA"):
        nq.block_norm(N, None, z((2, 64)))
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        nq.block_norm(N, None, z((2, 64), dtype=torch.float16))
    with pytest.raises(ValueError, match="expected \\[M\\]"):
        nq.block_norm(N, None, z((2, 63)))
