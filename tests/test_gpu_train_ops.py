"""The calls of include/usaf_train.h on the GPU against their fp64 restatements.

Bounds, from the arithmetic. u = 2^-24, the rounding of fp32.
- A probability: exponent differences of up to 25 rounded once (25 u), exp and the sum a few u each:
  below 64 u of itself. A sum of them in chains of at most 512: below 600 u. So prob_sum and the
  loss are held to 2^-14, each entry to itself.
- A gradient's bracket: errors of its terms, below 256 u of each: 2^-16 of the terms' sizes.
- A product: n terms summed in fp32, each addition rounded (tensor cores may truncate, twice that):
  2 (n + 32) u of the sum of the terms' magnitudes, and in norm 1e-5, this library's bound of fp32
  results. dx of a bf16 layer: dlogit and w_router carried to 2^-16 each, so 2^-14 of the terms'
  sum, and one rounding of the result to bf16, 2^-8 with the margin of a double rounding.
- Codes, exponents and decoded values: bit-equal. wa: one rounding, 2^-8 of itself.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import train_oracle as TO
from sparse_moe_fine_gb300 import binding as B
from sparse_moe_fine_gb300 import synth

from _gpu import device, rel_l2, to_dev

pytestmark = pytest.mark.gpu

F32_LOW = float(np.finfo(np.float32).min)


# ---------------------------------------------------------------------------------- aux losses
def _aux_inputs(T, E, k, G, seed, mask="none", dead=0):
    rng = np.random.default_rng(seed)
    l = (rng.standard_normal((T, E)) * 1.5 + rng.standard_normal(E)).astype(np.float32)
    if dead:
        l[:, rng.permutation(E)[:dead]] = -np.inf
    idx = np.argsort(-l, axis=1, kind="stable")[:, :k].astype(np.int32)
    off = None
    if G > 1:
        off = np.concatenate([[0], np.sort(rng.integers(0, T + 1, G - 1)), [T]]).astype(np.int32)
    m = None
    if mask != "none":
        m = (rng.random(T) < 0.8).astype(np.uint8) * 3
        if mask == "all":
            m[:] = 0
        elif off is not None:
            m[off[0]:off[1]] = 0  # a group that its mask leaves empty
    return l, idx, m, off


def _aux_run(dev, l, idx, k, G, cb, cz, m=None, off=None, ld=None, d_loss=None, base=None,
             status=None, stream=None):
    T, E = l.shape
    buf = torch.full((T, ld or E), 7.0, device=dev)
    lg = buf[:, :E]
    lg.copy_(torch.from_numpy(l))
    out = dict(count=torch.full((G, E), -1, dtype=torch.int32, device=dev),
               prob_sum=torch.full((G, E), -1.0, device=dev),
               n_tok=torch.full((G,), -1, dtype=torch.int32, device=dev),
               loss=torch.full((3,), -1.0, device=dev))
    obuf = torch.full((T, (ld or E) + 1), 5.0, device=dev)
    dl = obuf[:, :E]
    if base is not None:
        dl.copy_(torch.from_numpy(base))
    td = lambda a: None if a is None else torch.from_numpy(a).to(dev)
    mm, oo = td(m), td(off)
    ii = td(idx.reshape(-1))
    B.router_aux_fwd(lg, ii, k, out["count"], out["prob_sum"], out["n_tok"], out["loss"], cb, cz,
                     token_mask=mm, group_offset=oo, dev_status=status, stream=stream)
    B.router_aux_bwd(lg, k, out["count"], out["n_tok"], dl, cb, cz, token_mask=mm, group_offset=oo,
                     d_loss=None if d_loss is None else torch.tensor([d_loss], device=dev),
                     accumulate=0 if base is None else 1, dev_status=status, stream=stream)
    torch.cuda.synchronize()
    assert (obuf[:, E:] == 5.0).all() and (buf[:, E:] == 7.0).all()  # the gaps between rows
    res = {n: v.cpu().numpy() for n, v in out.items()}
    res["dlogit"] = dl.cpu().numpy()
    return res


def _aux_check(got, ref, base=None):
    np.testing.assert_array_equal(got["count"], ref["count"])
    np.testing.assert_array_equal(got["n_tok"], ref["n_tok"])
    np.testing.assert_allclose(got["prob_sum"], ref["prob_sum"], rtol=2.0 ** -14, atol=1e-30)
    np.testing.assert_allclose(got["loss"], ref["loss"], rtol=2.0 ** -14, atol=1e-30)
    want, tol = ref["dlogit"], 2.0 ** -16 * ref["scale"]
    if base is not None:
        want = want + base
        tol = tol + 2.0 ** -23 * np.abs(base)
    assert (np.abs(got["dlogit"] - want) <= tol + 1e-37).all()


@pytest.mark.parametrize("T,E,k,G", [
    (1, 1, 1, 1), (1, 8, 2, 1), (3, 5, 5, 1), (128, 8, 2, 1), (31, 16, 3, 2), (65, 24, 4, 9),
    (300, 60, 4, 5), (257, 128, 8, 3), (1000, 129, 8, 1), (511, 256, 6, 7), (70, 500, 3, 4),
    (65, 1024, 32, 2), (4096, 128, 8, 1), (4099, 8, 2, 64), (9731, 128, 8, 37), (200, 16, 4, 200),
    (24, 9, 6, 13), (2000, 128, 8, 1500), (135, 300, 8, 51), (20, 1024, 4, 90),
    (20011, 96, 6, 3)])
@pytest.mark.parametrize("mask", ["none", "some", "all"])
def test_aux_matches_fp64(T, E, k, G, mask):
    dev = device()
    l, idx, m, off = _aux_inputs(T, E, k, G, T + E, mask, dead=(E - k) // 3)
    got = _aux_run(dev, l, idx, k, G, 1e-2, 1e-3, m, off)
    _aux_check(got, TO.router_aux(l, idx, k, 1e-2, 1e-3, m, off))


@pytest.mark.parametrize("cb,cz", [(0.0, 1e-3), (1e-2, 0.0), (0.0, 0.0)])
def test_aux_strides_upstream_accumulation_and_zero_coefficients(cb, cz):
    dev = device()
    l, idx, m, off = _aux_inputs(333, 40, 4, 3, 8, "some")
    base = np.random.default_rng(1).standard_normal(l.shape).astype(np.float32) * 1e-5
    got = _aux_run(dev, l, idx, 4, 3, cb, cz, m, off, ld=47, d_loss=-2.5, base=base)
    ref = TO.router_aux(l, idx, 4, cb, cz, m, off, d_loss=-2.5)
    _aux_check(got, ref, base)


def test_aux_group_offsets_that_leave_tokens_out_and_empty_groups():
    dev = device()
    l, idx, _, _ = _aux_inputs(100, 8, 2, 1, 9)
    off = np.array([7, 20, 20, 20, 64, 90], np.int32)  # tokens 0..6 and 90.. are in no group
    got = _aux_run(dev, l, idx, 2, 5, 1e-2, 1e-3, None, off)
    inside = np.zeros(100, np.uint8)
    inside[7:90] = 1
    whole = off.copy()
    whole[0], whole[-1] = 0, 100
    _aux_check(got, TO.router_aux(l, idx, 2, 1e-2, 1e-3, inside, whole))


def test_aux_rows_without_experts_and_the_types_lowest_value():
    dev = device()
    l, idx, _, _ = _aux_inputs(50, 12, 2, 1, 10)
    l[3] = -np.inf
    l[4, 1:] = -np.inf          # one expert left: probability 1
    l[5, 2:] = F32_LOW          # masked with the lowest value, not -inf
    idx[4] = 0
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    got = _aux_run(dev, l, idx, 2, 1, 1e-2, 1e-3, status=st)
    _aux_check(got, TO.router_aux(l, idx, 2, 1e-2, 1e-3))
    assert not got["dlogit"][3].any() and int(st.item()) == 0
    # whole rows at the lowest value: an even softmax; its square is past fp32, so z is infinite
    l[6] = F32_LOW
    got = _aux_run(dev, l, idx, 2, 1, 1e-2, 0.0, status=st)
    ref = TO.router_aux(l, idx, 2, 1e-2, 0.0)
    assert np.isinf(got["loss"][2]) and int(st.item()) & B.DEV_NONFINITE
    np.testing.assert_allclose(got["loss"][:2], ref["loss"][:2], rtol=2.0 ** -14)
    assert (np.abs(got["dlogit"] - ref["dlogit"]) <= 2.0 ** -16 * ref["scale"] + 1e-37).all()


@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_aux_nonfinite_logits_are_reported_and_masked_ones_are_not_read(bad):
    dev = device()
    l, idx, _, _ = _aux_inputs(90, 16, 2, 1, 11)
    clean = TO.router_aux(l, idx, 2, 1e-2, 1e-3, np.array([t != 33 for t in range(90)], np.uint8))
    l[33, 5] = bad
    m = np.ones(90, np.uint8)
    m[33] = 0
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    _aux_check(_aux_run(dev, l, idx, 2, 1, 1e-2, 1e-3, m, status=st), clean)
    assert int(st.item()) == 0
    got = _aux_run(dev, l, idx, 2, 1, 1e-2, 1e-3, status=st)
    assert int(st.item()) & B.DEV_NONFINITE and np.isnan(got["loss"][0])
    assert np.isnan(got["dlogit"][33]).all()


def test_aux_bad_indices_and_offsets_set_the_status_and_stay_in_bounds():
    dev = device()
    l, idx, _, _ = _aux_inputs(64, 8, 2, 1, 12)
    idx2 = idx.copy()
    idx2[5, 0], idx2[6, 1] = 8, -1
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    got = _aux_run(dev, l, idx2, 2, 1, 1e-2, 1e-3, status=st)
    assert int(st.item()) == B.DEV_BAD_INDEX and got["count"].sum() == 64 * 2 - 2
    for off in ([0, 40, 20, 64], [0, 10, 20, 70], [-3, 10, 20, 64]):
        st.zero_()
        _aux_run(dev, l, idx, 2, 3, 1e-2, 1e-3, None, np.array(off, np.int32), status=st)
        assert int(st.item()) & B.DEV_BAD_INDEX


def test_aux_gradient_may_overwrite_the_logits_and_is_reproducible():
    dev = device()
    l, idx, m, off = _aux_inputs(5000, 128, 8, 11, 13, "some")
    a = _aux_run(dev, l, idx, 8, 11, 1e-2, 1e-3, m, off)
    b = _aux_run(dev, l, idx, 8, 11, 1e-2, 1e-3, m, off)
    for n in a:
        np.testing.assert_array_equal(a[n], b[n])
    lg = torch.from_numpy(l).to(dev)
    td = lambda v: torch.from_numpy(v).to(dev)
    B.router_aux_bwd(lg, 8, td(a["count"]), td(a["n_tok"]), lg, 1e-2, 1e-3, token_mask=td(m),
                     group_offset=td(off))
    np.testing.assert_array_equal(lg.cpu().numpy(), a["dlogit"])


def test_aux_counts_summed_over_two_halves_give_the_whole_batchs_gradient():
    """Data parallel: each half's forward, counts added, each half's backward."""
    dev = device()
    l, idx, _, _ = _aux_inputs(600, 32, 4, 1, 14)
    ref = TO.router_aux(l, idx, 4, 1e-2, 1e-3)
    half = [_aux_run(dev, l[s], idx[s], 4, 1, 1e-2, 1e-3) for s in (slice(0, 350), slice(350, 600))]
    td = lambda v: torch.from_numpy(v).to(dev)
    cnt, n = (td(half[0][q] + half[1][q]) for q in ("count", "n_tok"))
    for s in (slice(0, 350), slice(350, 600)):
        lg = td(l[s])
        dl = torch.empty_like(lg)
        B.router_aux_bwd(lg, 4, cnt, n, dl, 1e-2, 1e-3)
        err = np.abs(dl.cpu().numpy() - ref["dlogit"][s])
        assert (err <= 2.0 ** -16 * ref["scale"][s] + 1e-37).all()


# ---------------------------------------------------------------------------------- products
def _grad_inputs(T, E, H, bf16, seed):
    rng = np.random.default_rng(seed)
    dl = (rng.standard_normal((T, E)) * np.exp(2 * rng.standard_normal((T, E)))).astype(np.float32)
    r = oracle.bf16_round if bf16 else (lambda a: a)
    x = r(rng.standard_normal((T, H)).astype(np.float32))
    w = (rng.standard_normal((E, H)) * 0.02).astype(np.float32)
    g_in = rng.standard_normal((E, H)).astype(np.float32)
    dx_in = r((rng.standard_normal((T, H)) * 0.1).astype(np.float32))
    return dl, x, w, g_in, dx_in


def _grad_check(g, dx, dl, x, w, g_in, dx_in, bf16):
    T, E = dl.shape
    ad = np.abs(dl.astype(np.float64))
    rg, rx = TO.router_grad(dl, x, w, g_in, dx_in)
    u = 2.0 ** -24
    if g is not None:
        terms = ad.T @ np.abs(x) + (0 if g_in is None else np.abs(g_in))
        assert (np.abs(g - rg) <= 2 * (T + 32) * u * terms).all()
        assert rel_l2(g, rg) <= 1e-5
    if dx is not None:
        terms = ad @ np.abs(w) + (0 if dx_in is None else np.abs(dx_in))
        tol = 2 * (E + 32) * u * terms
        if bf16:
            tol = tol + 2.0 ** -14 * (ad @ np.abs(w)) + 2.0 ** -8 * np.abs(rx)
        assert (np.abs(dx - rx) <= tol).all()
        assert rel_l2(dx, rx) <= (4e-3 if bf16 else 1e-5)


@pytest.mark.parametrize("T,E,H,bf16", [
    (1, 1, 64, True), (1, 128, 2048, True), (5, 7, 64, True), (64, 8, 128, True),
    (129, 128, 192, True), (200, 3, 4096, True), (333, 60, 320, True), (1000, 129, 256, True),
    (700, 256, 448, True), (2600, 8, 4160, True), (2600, 128, 4160, True),
    (2600, 200, 4160, True), (2600, 300, 4160, True), (130, 300, 64, True), (90, 1024, 128, True), (4097, 128, 512, True),
    (1, 1, 1, False), (128, 8, 64, False), (77, 13, 33, False), (300, 130, 65, False),
    (2100, 16, 100, False), (3, 1024, 7, False),
    (2000, 70, 1283, False)])
def test_router_grad_matches_fp64(T, E, H, bf16):
    dev = device()
    dl, x, w, g_in, dx_in = _grad_inputs(T, E, H, bf16, T + H)
    d_dl, d_w, d_gi = (to_dev(a, dev) for a in (dl, w, g_in))
    d_x, d_xi = to_dev(x, dev, bf16), to_dev(dx_in, dev, bf16)
    g = torch.empty(E, H, device=dev)
    dx = torch.empty_like(d_x)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    B.router_grad(d_dl, d_x, d_w, g_router=g, g_in=d_gi, dx=dx, dx_in=d_xi, dev_status=st)
    _grad_check(g.cpu().numpy(), dx.float().cpu().numpy(), dl, x, w, g_in, dx_in, bf16)
    # without the addends, one product at a time
    g2, dx2 = torch.empty_like(g), torch.empty_like(dx)
    B.router_grad(d_dl, d_x, None, g_router=g2, dev_status=st)
    B.router_grad(d_dl, None, d_w, dx=dx2, dev_status=st)
    _grad_check(g2.cpu().numpy(), dx2.float().cpu().numpy(), dl, x, w, None, None, bf16)
    # in place, and the same bits again
    gi, xi = d_gi.clone(), d_xi.clone()
    B.router_grad(d_dl, d_x, d_w, g_router=gi, g_in=gi, dx=xi, dx_in=xi, dev_status=st)
    assert torch.equal(gi, g) and torch.equal(xi, dx) and int(st.item()) == 0


def test_router_grad_strided_dlogit_and_another_stream():
    dev = device()
    dl, x, w, g_in, dx_in = _grad_inputs(517, 40, 256, True, 3)
    buf = torch.full((517, 43), float("nan"), device=dev)
    buf[:, :40] = torch.from_numpy(dl).to(dev)
    d_x, d_w = to_dev(x, dev, True), to_dev(w, dev)
    g, dx = torch.empty(40, 256, device=dev), torch.empty_like(d_x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    B.router_grad(buf[:, :40], d_x, d_w, g_router=g, dx=dx, stream=s)
    s.synchronize()
    _grad_check(g.cpu().numpy(), dx.float().cpu().numpy(), dl, x, w, None, None, True)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("where", ["dlogit", "x"])
def test_router_grad_reports_nonfinite(bf16, where):
    dev = device()
    dl, x, w, _, _ = _grad_inputs(150, 16, 128, bf16, 4)
    (dl if where == "dlogit" else x)[77, 5] = np.nan
    d_dl, d_x, d_w = to_dev(dl, dev), to_dev(x, dev, bf16), to_dev(w, dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    g, dx = torch.empty(16, 128, device=dev), torch.empty_like(d_x)
    B.router_grad(d_dl, d_x, d_w, g_router=g, dx=dx, dev_status=st)
    assert int(st.item()) & B.DEV_NONFINITE
    bad_g = np.isnan(g.cpu().numpy())
    if where == "dlogit":   # expert 5's row of g_router, token 77's row of dx
        assert bad_g[5].all() and not np.delete(bad_g, 5, 0).any()
        bad_x = np.isnan(dx.float().cpu().numpy())
        assert bad_x[77].all() and not np.delete(bad_x, 77, 0).any()
    else:                   # feature 5's column of g_router
        assert bad_g[:, 5].all() and not np.delete(bad_g, 5, 1).any()
        assert torch.isfinite(dx.float()).all()


# ---------------------------------------------------------------------------------- 8-bit store
def _layer(T, H, E, k, I, bf16, seed, spread=1.0):
    """Routing of random logits by the library, x, and an h as a forward leaves it."""
    dev = device()
    rng = np.random.default_rng(seed)
    s = B.shape(T, H, E, k, I)
    cap = B.routed_rows_capacity(s)
    rt = B.Routing.empty(s, dev)
    l = rng.standard_normal((T, E)).astype(np.float32) + spread * rng.standard_normal(E)
    B.route_topk(s, None, None, rt, logits_in=to_dev(l.astype(np.float32), dev))
    dt = torch.bfloat16 if bf16 else torch.float32
    mag = lambda *sh: np.exp(2 * rng.standard_normal(sh))
    x = to_dev((rng.standard_normal((T, H)) * mag(1, H)).astype(np.float32), dev).to(dt)
    h = to_dev((rng.standard_normal((2 * I, cap)) * mag(2 * I, 1)).astype(np.float32), dev).to(dt)
    rows = int(rt.expert_offset[E].item())
    h *= (rt.perm_slot >= 0).to(dt)
    h[:, rows:] = float("nan")  # rows that no expert owns are not read
    return s, cap, rt, x, h, rows


def _trip(s, cap, rt, x, h, rows, stream=None):
    dev, dt = x.device, x.dtype
    store = B.ActStore8.empty(s, dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    B.act8_save(s, x, h, rt, store, dev_status=st, stream=stream)
    new = lambda *sh: torch.full(sh, 9.0, dtype=dt, device=dev)
    out = new(s.T, s.H), new(s.H, cap), new(2 * s.I, cap), new(s.I, cap)
    B.act8_restore(s, store, rt, out[1], out[2], out[3], x=out[0], stream=stream)
    torch.cuda.synchronize()
    return store, int(st.item()), out


@pytest.mark.parametrize("T,H,E,k,I,bf16", [
    (1, 64, 1, 1, 64, True), (1, 128, 8, 2, 64, True), (200, 128, 8, 2, 128, True),
    (517, 320, 60, 4, 192, True), (1000, 64, 128, 8, 64, True), (33, 2048, 16, 3, 768, True),
    (700, 100, 5, 3, 36, True),                       # sizes no bf16 layer takes, the store does
    (128, 64, 8, 2, 32, False), (77, 33, 6, 2, 5, False), (300, 250, 16, 4, 48, False),
    (1, 1, 1, 1, 1, False)])
def test_act8_matches_fp64_bit_for_bit(T, H, E, k, I, bf16):
    s, cap, rt, x, h, rows = _layer(T, H, E, k, I, bf16, T + H + I, spread=2.0)
    store, st, (xo, xp, ho, wa) = _trip(s, cap, rt, x, h, rows)
    xs, hs = x.float().cpu().numpy(), h.float().cpu().numpy()[:, :rows]
    xc, xe = TO.act8_encode(xs)
    hc, he = TO.act8_encode(hs)
    assert st == 0
    np.testing.assert_array_equal(store.x_code.cpu().numpy(), xc)
    np.testing.assert_array_equal(store.x_exp.cpu().numpy(), xe)
    np.testing.assert_array_equal(store.h_code.cpu().numpy()[:, :rows], hc)
    np.testing.assert_array_equal(store.h_exp.cpu().numpy()[:, :rows // 16], he)
    rx, rxp, rh, rwa = TO.act8_restore(xc, xe, hc, he, rt.topk_w.cpu().numpy(),
                                       rt.perm_tok.cpu().numpy(), rt.perm_slot.cpu().numpy(), rows)
    f = lambda t: t.float().cpu().numpy()
    np.testing.assert_array_equal(f(xo), rx)
    np.testing.assert_array_equal(f(xp)[:, :rows], rxp)
    assert not f(xp)[:, rows:].any()
    np.testing.assert_array_equal(f(ho)[:, :rows], rh)
    tol = 2.0 ** -8 if bf16 else 2.0 ** -18
    assert (np.abs(f(wa)[:, :rows] - rwa) <= tol * np.abs(rwa) + 1e-37).all()


def test_act8_without_x_and_on_another_stream():
    s, cap, rt, x, h, rows = _layer(300, 192, 8, 2, 64, True, 21)
    _, _, ref = _trip(s, cap, rt, x, h, rows)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    store, _, got = _trip(s, cap, rt, x, h, rows, stream=side)
    for a, b in zip(ref, got):
        assert torch.equal(a, b)
    xp, ho, wa = (torch.full_like(t, 9.0) for t in ref[1:])
    B.act8_restore(s, store, rt, xp, ho, wa)
    for a, b in zip(ref[1:], (xp, ho, wa)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bf16", [True, False])
def test_act8_zeros_extremes_and_nonfinite_blocks(bf16):
    s, cap, rt, x, h, rows = _layer(64, 128, 4, 2, 64, bf16, 22)
    big = torch.finfo(x.dtype).max
    x[0] = 0
    x[1, :16] = big
    x[2, :16] = 1e-39
    x[2, 16:32] = 2.0 ** -120
    h[5, :16] = 0
    _, st, (xo, xp, ho, wa) = _trip(s, cap, rt, x, h, rows)
    rx = TO.act8_decode(*TO.act8_encode(x.float().cpu().numpy()))
    np.testing.assert_array_equal(xo.float().cpu().numpy(), rx)
    assert st == 0 and torch.isfinite(xo.float()).all()
    for bad in (float("nan"), float("inf"), -float("inf")):
        y = x.clone()
        y[7, 37] = bad
        _, st, (xo, xp, ho, wa) = _trip(s, cap, rt, y, h, rows)
        assert st == B.DEV_NONFINITE
        nan = torch.isnan(xo.float()).cpu().numpy()
        assert nan[7, 32:48].all() and nan.sum() == 16
        g = h.clone()
        g[9, 3] = bad
        _, st, (xo, xp, ho, wa) = _trip(s, cap, rt, x, g, rows)
        assert st == B.DEV_NONFINITE
        nan = torch.isnan(ho[:, :rows].float()).cpu().numpy()
        assert nan[9, :16].all() and nan.sum() == 16
        assert torch.isnan(wa[9, :16].float()).all()


def test_backward_from_the_store_is_close_to_the_backward_from_bf16():
    """One layer: forward, 8-bit store, restore into other buffers, sparse backward. The store's
    rounding is at most 1/127 of a block's largest value per entry and half that in the mean, so
    the gradients agree within 2e-2 in norm (each is linear in x or a smooth function of h)."""
    dev = device()
    cfg = synth.small_config("act8", T=400, H=256, E=8, k=2, I=128, bf16=True, frac=0.05)
    inp = synth.moe_inputs(cfg, seed=5)
    s = B.shape(cfg.T, cfg.H, cfg.E, cfg.k, cfg.I)
    cap = B.routed_rows_capacity(s)
    x, wgu, wd, dy = (to_dev(inp[n], dev, True) for n in ("x", "w_gate_up", "w_down", "dy"))
    wr = to_dev(inp["w_router"], dev)
    rt = B.Routing.empty(s, dev)
    B.route_topk(s, x, wr, rt, logits_out=torch.empty(cfg.T, cfg.E, device=dev))
    new = lambda *sh: torch.zeros(*sh, dtype=torch.bfloat16, device=dev)
    xp, h, wa, y = new(cfg.H, cap), new(2 * cfg.I, cap), new(cfg.I, cap), new(cfg.T, cfg.H)
    B.moe_fwd(s, x, wgu, wd, rt, xp, h, wa, y)
    store = B.ActStore8.empty(s, dev)
    B.act8_save(s, x, h, rt, store)
    x2, xp2, h2, wa2 = new(cfg.T, cfg.H), new(cfg.H, cap), new(2 * cfg.I, cap), new(cfg.I, cap)
    B.act8_restore(s, store, rt, xp2, h2, wa2, x=x2)
    act = to_dev(synth.uniform_mask(cfg.N, cfg.K, seed=5), dev)
    res = []
    for a, b, c, d in ((x, xp, h, wa), (x2, xp2, h2, wa2)):
        g, gr, dx = torch.empty(cfg.K, device=dev), torch.empty(cfg.E, cfg.H, device=dev), new(cfg.T, cfg.H)
        B.moe_bwd_sparse(s, a, wr, wgu, wd, rt, b, c, d, dy, act, g, gr, dx=dx)
        res.append([t.float().cpu().numpy() for t in (g, gr, dx)])
    for full, kept in zip(*res):
        err = rel_l2(kept, full)
        assert 0 < err <= 2e-2, err
