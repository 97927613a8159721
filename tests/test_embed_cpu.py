"""Embedding lookup and gradient: argument checks. Nothing is launched: every call here is refused, or needs no GPU."""
import ctypes

import pytest
import torch

import adamw_hybrid_optimizer_muon_b200 as ma

IDS, TAB, OUT, DY, GRAD, WS = (0x6000_0000_0000 + k * (1 << 36) for k in range(6))  # made up, never followed
BIG = ctypes.c_size_t(1 << 40)


def lookup(n=10, ids=IDS, idt=3, rows=100, dim=64, table=TAB, tdt=0, ldt=64, scale=1.0, padding=ma.NO_PADDING, out=OUT,
           odt=0, ldo=64):
    return ma.lib().ma_embed_lookup(n, ids, idt, rows, dim, table, tdt, ldt, scale, padding, out, odt, ldo, None)


def grad(n=10, ids=IDS, idt=3, rows=100, dim=64, dy=DY, ydt=0, ldy=64, scale=1.0, padding=ma.NO_PADDING, accumulate=0,
         grad=GRAD, gdt=0, ldg=64, ws=WS, ws_bytes=1 << 40):
    return ma.lib().ma_embed_grad(n, ids, idt, rows, dim, dy, ydt, ldy, scale, padding, accumulate, grad, gdt, ldg, ws,
                                  ws_bytes, None)


COMMON = [
    (dict(n=-1), ma.MA_ERR_SHAPE), (dict(rows=-1), ma.MA_ERR_SHAPE), (dict(dim=-1), ma.MA_ERR_SHAPE),
    (dict(idt=0), ma.MA_ERR_DTYPE), (dict(idt=4), ma.MA_ERR_DTYPE), (dict(ids=None), ma.MA_ERR_NULL),
    (dict(ids=IDS + 4), ma.MA_ERR_ALIGN), (dict(ids=IDS + 2, idt=2), ma.MA_ERR_ALIGN),
    (dict(n=1 << 31), ma.MA_ERR_UNSUPPORTED), (dict(rows=(1 << 30) + 1), ma.MA_ERR_UNSUPPORTED),
    (dict(scale=float("nan")), ma.MA_ERR_ARG), (dict(scale=float("inf")), ma.MA_ERR_ARG),
]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(table=None), ma.MA_ERR_NULL), (dict(out=None), ma.MA_ERR_NULL), (dict(tdt=2), ma.MA_ERR_DTYPE),
    (dict(odt=3), ma.MA_ERR_DTYPE), (dict(ldt=63), ma.MA_ERR_SHAPE), (dict(ldo=63), ma.MA_ERR_SHAPE),
    (dict(ldt=(1 << 31) + 1), ma.MA_ERR_UNSUPPORTED), (dict(table=TAB + 2), ma.MA_ERR_ALIGN),
    (dict(out=OUT + 1, odt=1), ma.MA_ERR_ALIGN), (dict(out=TAB), ma.MA_ERR_ARG),
    (dict(out=TAB + 4 * (99 * 64 + 63)), ma.MA_ERR_ARG), (dict(out=IDS), ma.MA_ERR_ARG)])
def test_lookup_refuses(kw, code):
    assert lookup(**kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(dy=None), ma.MA_ERR_NULL), (dict(grad=None), ma.MA_ERR_NULL), (dict(ydt=2), ma.MA_ERR_DTYPE),
    (dict(gdt=5), ma.MA_ERR_DTYPE), (dict(ldy=0), ma.MA_ERR_SHAPE), (dict(ldg=10), ma.MA_ERR_SHAPE),
    (dict(dy=DY + 2), ma.MA_ERR_ALIGN), (dict(grad=GRAD + 1, gdt=1), ma.MA_ERR_ALIGN),
    (dict(accumulate=2), ma.MA_ERR_ARG), (dict(ws=None), ma.MA_ERR_WORKSPACE), (dict(ws=WS + 64), ma.MA_ERR_WORKSPACE),
    (dict(ws_bytes=1000), ma.MA_ERR_WORKSPACE), (dict(grad=DY + 4), ma.MA_ERR_ARG), (dict(ws=DY), ma.MA_ERR_ARG),
    (dict(ws=GRAD), ma.MA_ERR_ARG), (dict(ws=IDS), ma.MA_ERR_ARG), (dict(grad=IDS), ma.MA_ERR_ARG)])
def test_grad_refuses(kw, code):
    assert grad(**kw) == code


def test_workspace_sizes():
    f = ma.embed_grad_workspace_bytes
    assert f(0, 100, 64) == 0
    assert f(1, 1, 1) > 0
    last = 0
    for n in (1, 100, 8192, 8193, 100_000, 1 << 20, (1 << 31) - 1):
        assert f(n, 32000, 4096) > last
        last = f(n, 32000, 4096)
    for bad in ((-1, 1, 1), (1, -1, 1), (1, 1, -1), (1 << 31, 1, 1), (1, (1 << 30) + 1, 1)):
        with pytest.raises(ma.MAError):
            f(*bad)


def test_host_tensors_and_shapes_are_refused():
    ids, tab = torch.zeros(4, dtype=torch.int64), torch.zeros(5, 8)
    for call in (lambda: ma.embedding_lookup(ids, tab), lambda: ma.embedding_grad(ids, torch.zeros(4, 8), tab),
                 lambda: ma.embedding(ids, tab), lambda: ma.embedding(ids, tab, grad=torch.zeros(4, 8))):
        with pytest.raises(ma.MAError):
            call()
