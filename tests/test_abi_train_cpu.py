"""The calls of include/usaf_train.h on the host: exports, prototypes, workspace queries, and the
refusals that come before anything is enqueued."""
import ctypes
import os
import re

import pytest
import torch

from sparse_moe_fine_gb300 import binding as B

fake_addresses = pytest.mark.skipif(torch.cuda.is_available(),
                                    reason="fake device addresses; run where no GPU is visible")
FAKE = ctypes.c_void_p(4096)  # never dereferenced: the calls below fail on the host


def _arity():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "usaf_train.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return {n: p.count(",") + 1
            for n, p in re.findall(r"\b(usaf_[a-z0-9_]+)\s*\(([^)]*)\)\s*;", text)}


def test_exports_and_prototypes_match_the_header():
    arity = _arity()
    assert set(arity) == set(B._TRAIN_SIGS)
    for name, (_, args) in B._TRAIN_SIGS.items():
        assert len(args) == arity[name], name
        assert hasattr(B.lib(), name)


def test_workspace_queries():
    assert B.router_aux_workspace_size(4096, 128, 8) >= 4096 // 32 * 128 * 8
    assert B.router_aux_workspace_size(4096, 128, 8, 4096) > B.router_aux_workspace_size(4096, 128, 8)
    for bad in ((0, 8, 2, 1), (8, 0, 1, 1), (8, 1025, 2, 1), (8, 8, 9, 1), (8, 64, 33, 1),
                (8, 8, 2, 0), (8, 8, 2, (1 << 20) + 1), (1 << 30, 8, 2, 1)):
        assert B.router_aux_workspace_size(*bad) == 0
    assert B.router_grad_workspace_size(4096, 128, 2048, torch.bfloat16) > 0
    assert B.router_grad_workspace_size(100, 7, 33, torch.float32) > 0
    for bad in ((0, 8, 64), (8, 0, 64), (8, 1025, 64), (8, 8, 0), (1 << 31, 8, 64)):
        assert B.router_grad_workspace_size(*bad, torch.bfloat16) == 0
    assert B.router_grad_workspace_size(8, 8, 96, torch.bfloat16) == 0  # H not a multiple of 64


@fake_addresses
def test_aux_refusals():
    L = B.lib()

    def fwd(T=8, E=4, k=2, logits=FAKE, ld=4, idx=FAKE, off=None, G=1, cb=1e-2, cz=1e-3, count=FAKE,
            loss=FAKE, ws=FAKE, n=1 << 30):
        return L.usaf_router_aux_fwd(T, E, k, logits, ld, idx, None, off, G, cb, cz, count, FAKE,
                                     FAKE, loss, None, ws, n, None)

    for bad in (dict(T=0), dict(E=0), dict(E=1025, ld=1025), dict(k=5), dict(k=0), dict(ld=3),
                dict(logits=None), dict(idx=None), dict(count=None), dict(loss=None), dict(G=2),
                dict(G=0), dict(cb=float("nan")), dict(cz=float("inf")), dict(cb=1e39)):
        assert fwd(**bad) == 1, bad
    assert fwd(ws=None) == 3 and fwd(n=16) == 3

    def bwd(T=8, E=4, k=2, logits=FAKE, ld=4, off=None, G=1, count=FAKE, out=ctypes.c_void_p(8192),
            ld_out=4, acc=0):
        return L.usaf_router_aux_bwd(T, E, k, logits, ld, None, off, G, 1e-2, 1e-3, count, FAKE,
                                     None, out, ld_out, acc, None, None)

    for bad in (dict(T=-1), dict(logits=None), dict(count=None), dict(out=None), dict(ld_out=3),
                dict(acc=2), dict(G=3), dict(out=FAKE, acc=1), dict(out=FAKE, ld_out=5)):
        assert bwd(**bad) == 1, bad


@fake_addresses
def test_router_grad_refusals():
    L = B.lib()

    def call(T=8, E=4, H=64, dt=1, dl=FAKE, ld=4, x=FAKE, w=FAKE, g=FAKE,
             dx=ctypes.c_void_p(1 << 20), ws=FAKE, n=1 << 30):
        return L.usaf_router_grad(T, E, H, dt, dl, ld, x, w, None, g, None, dx, None, ws, n, None)

    for bad in (dict(T=0), dict(E=0), dict(H=0), dict(dt=2), dict(dl=None), dict(ld=3),
                dict(g=None, dx=None), dict(x=None), dict(w=None), dict(x=ctypes.c_void_p(4104)),
                dict(dx=ctypes.c_void_p(4098)), dict(x=FAKE, dx=FAKE)):
        assert call(**bad) == 1, bad
    assert call(H=96) == 2           # bf16 needs a multiple of 64
    assert call(ws=None) == 3 and call(n=0) == 3


@fake_addresses
def test_act8_refusals():
    L = B.lib()
    s = B.shape(8, 64, 4, 2, 64)
    full = B._Routing(*[4096] * 7)
    none = B._Routing()
    odd = ctypes.c_void_p(4100)

    def save(sh=s, dt=1, x=FAKE, h=FAKE, rt=full, store=(FAKE,) * 4):
        return L.usaf_act8_save(ctypes.byref(sh) if sh else None, dt, x, h, ctypes.byref(rt),
                                *store, None, None)

    def restore(sh=s, dt=1, rt=full, xp=FAKE, h=FAKE, wa=FAKE, x=None, store=(FAKE,) * 4):
        return L.usaf_act8_restore(ctypes.byref(sh) if sh else None, dt, *store, ctypes.byref(rt),
                                   x, xp, h, wa, None)

    bad_shape = B.shape(8, 64, 4, 5, 64)
    for bad in (dict(sh=None), dict(sh=bad_shape), dict(dt=7), dict(x=None), dict(h=None),
                dict(rt=none), dict(store=(FAKE, None, FAKE, FAKE)), dict(h=odd),
                dict(store=(odd, FAKE, FAKE, FAKE))):
        assert save(**bad) == 1, bad
    for bad in (dict(sh=bad_shape), dict(dt=-1), dict(rt=none), dict(xp=None), dict(h=None),
                dict(wa=None), dict(x=odd), dict(store=(FAKE, FAKE, FAKE, None)), dict(wa=odd)):
        assert restore(**bad) == 1, bad


def test_binding_refuses_wrong_tensors():
    """Shapes, dtypes and devices are refused before the library is called."""
    l = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        B.router_aux_fwd(l, torch.zeros(8, dtype=torch.int32), 2,
                         torch.zeros(1, 8, dtype=torch.int32), torch.zeros(1, 8),
                         torch.zeros(1, dtype=torch.int32), torch.zeros(3), 1.0, 1.0)
    with pytest.raises(ValueError):
        B.router_grad(l, torch.zeros(4, 64), torch.zeros(8, 64), g_router=torch.zeros(8, 64))
    with pytest.raises(ValueError):
        B.router_grad(l, None, torch.zeros(8, 64))
    s = B.shape(4, 64, 4, 2, 64)
    with pytest.raises(ValueError):
        B.act8_save(s, torch.zeros(4, 64), torch.zeros(3, 3), None, None)
