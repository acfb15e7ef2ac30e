"""Pins of the fp64 restatements of the router's auxiliary losses, its dense gradient products and
the 8-bit activation store: closed forms, autograd, central differences and hand cases."""
import numpy as np
import pytest
import torch

from oracle import train_oracle as TO


def _case(T, E, k, G, seed, masked):
    rng = np.random.default_rng(seed)
    l = rng.standard_normal((T, E)) * 1.5
    idx = np.argsort(-l, axis=1, kind="stable")[:, :k]
    off = None if G == 1 else np.concatenate([[0], np.sort(rng.integers(0, T + 1, G - 1)), [T]])
    mask = (rng.random(T) < 0.8).astype(np.uint8) if masked else None
    return l, idx, mask, off


def test_even_router_has_balance_one():
    T, E, k = 12, 4, 2
    idx = np.array([[t % E, (t + 1) % E] for t in range(T)])
    r = TO.router_aux(np.zeros((T, E)), idx, k, 0.5, 0.25)
    assert r["loss"][1] == pytest.approx(1.0)
    assert r["loss"][2] == pytest.approx(np.log(E) ** 2)
    assert r["loss"][0] == pytest.approx(0.5 + 0.25 * np.log(E) ** 2)
    assert (r["count"] == T * k // E).all() and r["n_tok"].tolist() == [T]
    # an even router is a stationary point of the balance term
    assert np.abs(TO.router_aux(np.zeros((T, E)), idx, k, 0.5, 0.0)["dlogit"]).max() < 1e-15


@pytest.mark.parametrize("T,E,k,G,masked", [(9, 5, 2, 1, False), (14, 6, 3, 3, True)])
def test_aux_gradient_against_differences_and_autograd(T, E, k, G, masked):
    l, idx, mask, off = _case(T, E, k, G, 3, masked)
    l[1, 0] = -np.inf
    a, b = 0.7, 0.3
    r = TO.router_aux(l, idx, k, a, b, mask, off)
    eps = 1e-6
    for t in range(T):
        for e in range(E):
            if np.isinf(l[t, e]):
                assert r["dlogit"][t, e] == 0
                continue
            up, dn = l.copy(), l.copy()
            up[t, e] += eps
            dn[t, e] -= eps
            num = (TO.router_aux(up, idx, k, a, b, mask, off)["loss"][0]
                   - TO.router_aux(dn, idx, k, a, b, mask, off)["loss"][0]) / (2 * eps)
            assert num == pytest.approx(r["dlogit"][t, e], rel=1e-5, abs=1e-8)
    lt = torch.tensor(l, requires_grad=True)
    live = torch.ones(T, dtype=torch.bool) if mask is None else torch.tensor(mask != 0)
    p, s = torch.softmax(lt, 1), torch.logsumexp(lt, 1)
    loss = 0
    n = int(live.sum())
    bounds = [0, T] if off is None else off
    for g in range(len(bounds) - 1):
        tt = [t for t in range(bounds[g], bounds[g + 1]) if live[t]]
        if not tt:
            continue
        c = torch.tensor(r["count"][g].astype(np.float64))
        loss = loss + a * E / (k * n * len(tt)) * (c * p[tt].sum(0)).sum() + b / n * (s[tt] ** 2).sum()
    loss.backward()
    np.testing.assert_allclose(loss.item(), r["loss"][0], rtol=1e-12)
    np.testing.assert_allclose(np.nan_to_num(lt.grad.numpy()), r["dlogit"], rtol=1e-9, atol=1e-15)


def test_aux_of_nothing_is_zero():
    l, idx, _, _ = _case(6, 4, 2, 1, 5, False)
    r = TO.router_aux(l, idx, 2, 1.0, 1.0, np.zeros(6, np.uint8))
    assert not r["loss"].any() and not r["count"].any() and not r["dlogit"].any()
    l[2] = -np.inf  # a row without any expert takes no part
    r = TO.router_aux(l, idx, 2, 1.0, 1.0)
    assert r["n_tok"].tolist() == [5] and not r["dlogit"][2].any()
    assert np.isfinite(r["loss"]).all()


def test_router_grad_against_differences():
    rng = np.random.default_rng(7)
    T, E, H = 6, 3, 5
    x, w, r = rng.standard_normal((T, H)), rng.standard_normal((E, H)), rng.standard_normal((T, E))
    loss = lambda xx, ww: float((r * (xx @ ww.T)).sum())  # dL/dlogits = r
    g, dx = TO.router_grad(r, x, w)
    eps = 1e-6
    for a, d, f in ((x, dx, lambda v: loss(v, w)), (w, g, lambda v: loss(x, v))):
        for i in np.ndindex(a.shape):
            up, dn = a.copy(), a.copy()
            up[i] += eps
            dn[i] -= eps
            assert (f(up) - f(dn)) / (2 * eps) == pytest.approx(d[i], rel=1e-6, abs=1e-8)


def test_act8_hand_cases():
    v = np.zeros((1, 40))
    v[0, 0], v[0, 1], v[0, 2] = 127.0, -63.5, 0.5     # exponent 0: ties to even
    v[0, 16] = 127.5                                  # just above: exponent 1
    v[0, 17], v[0, 18] = 3.0, -5.0                    # 1.5 -> 2, -2.5 -> -2
    v[0, 32], v[0, 33] = 2.0 ** -140, 1e-40           # below the smallest exponent
    code, byte = TO.act8_encode(v)
    assert byte.tolist() == [[127, 128, 1]]
    assert code[0, :3].tolist() == [127, -64, 0]
    assert code[0, 16:19].tolist() == [64, 2, -2]
    assert not code[0, 32:].any()
    assert TO.act8_encode(np.full((1, 16), 3.3e38))[1][0, 0] == 248
    assert (TO.act8_encode(np.full((1, 16), np.float64(np.finfo(np.float32).max)))[0] == 127).all()
    bad = np.ones((1, 16))
    bad[0, 5] = np.inf
    code, byte = TO.act8_encode(bad)
    assert byte[0, 0] == 255 and not code.any() and np.isnan(TO.act8_decode(code, byte)).all()
    assert TO.act8_encode(np.zeros((2, 3)))[1].tolist() == [[0], [0]]


def test_act8_error_is_half_a_step_and_a_second_pass_changes_nothing():
    rng = np.random.default_rng(11)
    v = rng.standard_normal((50, 70)) * np.exp(rng.standard_normal((50, 70)) * 3)
    code, byte = TO.act8_encode(v)
    out = TO.act8_decode(code, byte)
    amax = np.stack([np.abs(v[:, 16 * b:16 * b + 16]).max(1) for b in range(byte.shape[1])], 1)
    assert (amax <= 127 * np.exp2(byte - 127.0)).all()
    assert (amax > 127 * np.exp2(byte - 128.0)).all()   # the least exponent
    step = np.repeat(np.exp2(byte - 127.0), 16, axis=1)[:, :70]
    assert (np.abs(out - v) <= step / 2).all()
    # every value is a bf16 number
    f = out.astype(np.float32)
    assert (f == out).all() and (f.view(np.uint32) & 0xFFFF == 0).all()
    np.testing.assert_array_equal(TO.act8_decode(*TO.act8_encode(out)), out)
