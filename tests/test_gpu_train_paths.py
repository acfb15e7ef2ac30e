"""Launch paths of the calls of include/usaf_train.h that take larger sizes, their order among one
another, and their behaviour in the layer and the stack.

Bounds are those of the fp32 arithmetic, u = 2^-24: see each test. Restatements in fp64 are
oracle/train_oracle.py's.
"""
import numpy as np
import pytest
import torch

from oracle import train_oracle as TO
from sparse_moe_fine_gb300 import binding as B
from sparse_moe_fine_gb300 import synth
from sparse_moe_fine_gb300.layer import MoELayer
from sparse_moe_fine_gb300.trainer import StackTrainer

import test_gpu_train_ops as ops
from _gpu import device, rel_l2, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,H", [(4096, 128, 2048), (1500, 8, 512), (900, 300, 256)])
def test_router_grad_calls_in_a_row_on_one_workspace(T, E, H):
    """Calls that follow one another at once, on other inputs and one workspace, give the bits that
    each gives alone: no kernel of a call reads parts or sums before they are written."""
    dev = device()
    g = torch.Generator(device=dev)
    g.manual_seed(T)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)
    n = 4
    dl, w = [rand(T, E) * 10.0 ** i for i in range(n)], [rand(E, H) for _ in range(n)]
    x, xi = ([rand(T, H).bfloat16() for _ in range(n)] for _ in range(2))
    ws = torch.empty(B.router_grad_workspace_size(T, E, H, torch.bfloat16), dtype=torch.uint8,
                     device=dev)

    def call(i):
        gr, dx = torch.empty(E, H, device=dev), torch.empty_like(x[i])
        B.router_grad(dl[i], x[i], w[i], g_router=gr, dx=dx, dx_in=xi[i], ws=ws)
        return gr, dx

    alone = []
    for i in range(n):
        torch.cuda.synchronize()
        ws.fill_(255)  # NaN, so that a read of what is not yet written shows
        torch.cuda.synchronize()
        alone.append(call(i))
        torch.cuda.synchronize()
    for _ in range(5):
        row = [call(i) for i in range(n)]
        torch.cuda.synchronize()
        for a, b in zip(alone, row):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.isfinite(alone[0][0]).all() and torch.isfinite(alone[0][1].float()).all()


@pytest.mark.parametrize("E,apart", [(8, 2.0 ** -14), (40, 2.0 ** -13), (64, 2.0 ** -12),
                                     (128, 2.0 ** -12), (160, 2.0 ** -12), (250, 2.0 ** -12)])
def test_dx_of_router_rows_that_share_a_component(E, apart):
    """Rows of w_router that differ by little from what they share, under a softmax's gradient, whose
    rows sum to zero: the shared part cancels, and what is left has to be as good as an fp32 sum.
    With terms = sum |dlogit| |w|: products left out 3 u of them; the sums, at most 6 E / 16
    additions, each within 2 u of an accumulator that wanders about terms / sqrt(E), below 13 u.
    So 16 u of terms in norm, and the rounding of the result to bf16, 2^-9."""
    dev = device()
    T, H = 300, 256
    rng = np.random.default_rng(E)
    l = rng.standard_normal((T, E))
    p = np.exp(l) / np.exp(l).sum(1, keepdims=True)
    a = rng.standard_normal((T, E))
    dl = (p * (a - (p * a).sum(1, keepdims=True))).astype(np.float32)
    w = (1.0 + apart * rng.standard_normal((E, H))).astype(np.float32)
    dx = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    B.router_grad(to_dev(dl, dev), None, to_dev(w, dev), dx=dx)
    _, ref = TO.router_grad(dl, np.zeros((T, 1)), w)
    terms = np.abs(dl.astype(np.float64)) @ np.abs(w)
    bound = 2.0 ** -9 + 16 * 2.0 ** -24 * np.linalg.norm(terms) / np.linalg.norm(ref)
    err = rel_l2(dx.float().cpu().numpy(), ref)
    assert err <= bound, (err, bound)


def _layers(dev, cfg, T, n, seed=60, **kw):
    """n layers for T tokens with the weights of `cfg`'s inputs, whatever T is."""
    out = []
    for i in range(n):
        inp = synth.moe_inputs(cfg, seed=seed + i)
        t = lambda a: torch.from_numpy(a).to(dev).to(torch.bfloat16 if cfg.bf16 else torch.float32)
        act = torch.from_numpy(synth.uniform_mask(cfg.N, cfg.K, seed=seed + i)).to(dev)
        out.append(MoELayer(T, cfg.H, cfg.E, cfg.k, cfg.I, t(inp["w_gate_up"]), t(inp["w_down"]),
                            torch.from_numpy(inp["w_router"]).to(dev), act, device=dev, **kw))
    return out


CFG = synth.small_config("aux_paths", T=256, H=128, E=8, k=2, I=128, bf16=True, frac=0.05)


@pytest.mark.parametrize("M", [2, 4])
def test_a_batch_cut_into_micro_batches_has_the_whole_batchs_loss_gradient(M):
    """No upstream gradient, so the router's gradient is the losses' alone. The cut batch's sequences
    are the micro-batches. fp32 results of the same terms: 1e-5 in norm each way, with the logits'."""
    dev = device()
    T = CFG.T
    x = to_dev(synth.moe_inputs(CFG, seed=3)["x"], dev, True)
    zero = torch.zeros_like(x)
    whole, = _layers(dev, CFG, T, 1, balance_coef=2.0, z_coef=0.5)
    whole.set_sequences(torch.arange(0, T + 1, T // M, dtype=torch.int32, device=dev))
    StackTrainer([whole], total_steps=10, reselect_every=0).step([x], [zero])
    cut, = _layers(dev, CFG, T // M, 1, balance_coef=2.0, z_coef=0.5)
    StackTrainer([cut], total_steps=10, reselect_every=0).step(list(x.split(T // M)),
                                                               list(zero.split(T // M)))
    torch.cuda.synchronize()
    a, b = whole.g_router.cpu().numpy(), cut.g_router.cpu().numpy()
    assert np.linalg.norm(a) > 0 and rel_l2(b, a) <= 4e-5


def test_micro_batches_of_their_own_sequences():
    """A packed, masked batch in one call, and cut in two with a packing and a mask for each half: the
    same gradient, 4e-5 in norm as above. The halves differ in sequences and in tokens."""
    dev = device()
    T, h = CFG.T, CFG.T // 2
    x = to_dev(synth.moe_inputs(CFG, seed=4)["x"], dev, True)
    zero = torch.zeros_like(x)
    mask = (torch.arange(T, device=dev) % 5 != 0).to(torch.uint8)
    mask[h:h + 90] = 0
    offs = [[0, 11, 50, h], [0, 100, h]]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    whole, = _layers(dev, CFG, T, 1, balance_coef=2.0, z_coef=0.5)
    whole.set_sequences(i32(offs[0] + [h + o for o in offs[1][1:]]), mask)
    StackTrainer([whole], total_steps=10, reselect_every=0).step([x], [zero])
    cut, = _layers(dev, CFG, h, 1, balance_coef=2.0, z_coef=0.5)
    tr = StackTrainer([cut], total_steps=10, reselect_every=0)
    tr.step(list(x.split(h)), list(zero.split(h)),
            sequences=[(i32(o), m.contiguous()) for o, m in zip(offs, mask.split(h))])
    torch.cuda.synchronize()
    a, b = whole.g_router.cpu().numpy(), cut.g_router.cpu().numpy()
    assert np.linalg.norm(a) > 0 and rel_l2(b, a) <= 4e-5
    assert cut.aux_count.shape[0] == 2 and int(cut.status.item()) == 0


@pytest.mark.parametrize("up", [float("inf"), float("nan")])
@pytest.mark.parametrize("E", [8, 100])
def test_tokens_without_a_part_have_no_gradient_under_a_nonfinite_upstream(up, E):
    """A scaled loss that overflowed: masked tokens, rows without experts, tokens outside the sequences
    and experts no token may take stay 0 (and what an accumulation held stays there), the rest says so."""
    dev = device()
    T, k = 60, 2
    rng = np.random.default_rng(E)
    l = to_dev(rng.standard_normal((T, E)).astype(np.float32), dev)
    l[:, 3] = float("-inf")
    l[7] = float("-inf")
    idx = l.topk(k, dim=1).indices.to(torch.int32).reshape(-1)
    mask = torch.ones(T, dtype=torch.uint8, device=dev)
    mask[20:30] = 0
    off = torch.tensor([5, 40, 55], dtype=torch.int32, device=dev)
    new = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device=dev)
    cnt, n = new(2, E, dt=torch.int32), new(2, dt=torch.int32)
    B.router_aux_fwd(l, idx, k, cnt, new(2, E), n, new(3), 1.0, 1.0, token_mask=mask,
                     group_offset=off)
    none = torch.zeros(T, E, dtype=torch.bool, device=dev)
    none[:, 3] = none[7] = none[20:30] = none[:5] = none[55:] = True
    for acc in (0, 1):
        st, d = new(1, dt=torch.int32), torch.full((T, E), 0.5, device=dev)
        B.router_aux_bwd(l, k, cnt, n, d, 1.0, 1.0, d_loss=torch.tensor([up], device=dev),
                         token_mask=mask, group_offset=off, accumulate=acc, dev_status=st)
        assert (d[none] == 0.5 * acc).all()
        assert not torch.isfinite(d[~none]).any() and int(st.item()) == B.DEV_NONFINITE


def test_dx_that_rounding_makes_infinite_is_reported():
    """bf16 ends at (2 - 2^-7) 2^127; a finite fp32 sum from half a step above it on rounds to infinity."""
    dev = device()
    top = (2 - 2.0 ** -8) * 2.0 ** 127
    for E in (8, 130):
        for value, odd in ((np.nextafter(np.float32(top), np.float32(0)), 0),
                           (np.float32(top), B.DEV_NONFINITE), (-np.float32(top), B.DEV_NONFINITE)):
            dl = torch.zeros(3, E, device=dev)
            dl[1, 2] = float(value)
            w = torch.zeros(E, 64, device=dev)
            w[2, 9] = 1.0
            dx = torch.empty(3, 64, dtype=torch.bfloat16, device=dev)
            st = torch.zeros(1, dtype=torch.int32, device=dev)
            B.router_grad(dl, None, w, dx=dx, dev_status=st)
            assert bool(torch.isinf(dx[1, 9])) == bool(odd) and int(st.item()) == odd
            dx[1, 9] = 0
            assert not dx.float().any()


@pytest.mark.parametrize("bf16", [True, False])
def test_act8_of_very_wide_tokens(bf16):
    """More feature tiles than a grid's second axis has places: 65,537 of 64."""
    dev = device()
    H = 64 * 65536 + 1
    dt = torch.bfloat16 if bf16 else torch.float32
    s = B.shape(1, H, 1, 1, 1)
    cap = B.routed_rows_capacity(s)
    rt = B.Routing.empty(s, dev)
    B.route_topk(s, None, None, rt, logits_in=torch.zeros(1, 1, device=dev))
    x = (torch.arange(H, device=dev) % 127 + 1)[None].to(dt)
    h = torch.zeros(2, cap, dtype=dt, device=dev)
    store = B.ActStore8.empty(s, dev)
    B.act8_save(s, x, h, rt, store)
    xo, xp = torch.empty_like(x), torch.empty(H, cap, dtype=dt, device=dev)
    ho, wa = torch.empty_like(h), torch.empty(1, cap, dtype=dt, device=dev)
    B.act8_restore(s, store, rt, xp, ho, wa, x=xo)
    torch.cuda.synchronize()
    row = int((rt.perm_slot[:16] == 0).nonzero()[0, 0])
    assert torch.equal(xo, x) and torch.equal(xp[:, row], x[0])
    xp[:, row] = 0
    assert not xp.any()


def test_a_stack_of_8_bit_activations_never_holds_all_layers_buffers():
    """Eight layers, built, stacked and stepped: at no time more than a layer's weights, state, routing
    tables and store each (10 MB of store, below 8 MB of the rest), and three layers' activations
    and workspaces (75 MB a layer); eight layers' own would be 600 MB."""
    dev = device()
    cfg = synth.small_config("act8_peak", T=4096, H=256, E=4, k=4, I=256, bf16=True, frac=0.05)
    x = to_dev(synth.moe_inputs(cfg, seed=1)["x"], dev, True)
    torch.cuda.synchronize()
    base = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    layers = _layers(dev, cfg, cfg.T, 8, balance_coef=1.0)
    tr = StackTrainer(layers, total_steps=10, reselect_every=0, act8=True)
    tr.step([x], [x])
    torch.cuda.synchronize()
    peak = torch.cuda.max_memory_allocated() - base
    own = sum(getattr(layers[0], n).nbytes for n in (
        "x_perm", "h", "wa", "y", "dx", "ws_route", "ws_fwd", "ws_bwd", "ws_rgrad", "dlogit_aux"))
    assert own > 70e6 and peak < 8 * 18e6 + 3 * own, (peak, own)
    assert len({L.ws_bwd.data_ptr() for L in layers}) == 1
    assert not any(tr.metrics()[0]["skipped"])


def test_layers_allocate_when_they_first_run_and_in_a_capture():
    """A layer holds no buffers before its first step; a step captured before any has run works too."""
    dev = device()
    cfg = synth.small_config("lazy", T=256, H=128, E=8, k=2, I=128, bf16=True, frac=0.05)
    inp = synth.moe_inputs(cfg, seed=2)
    x, dy = (to_dev(inp[n], dev, True) for n in ("x", "dy"))
    a, = _layers(dev, cfg, cfg.T, 1)
    b, = _layers(dev, cfg, cfg.T, 1)
    assert not a._held and not b._held
    a.status.zero_()
    a.route(x)
    a.forward(x)
    a.backward(x, dy)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        b.route(x, s)
        b.forward(x, s)
        b.backward(x, dy, stream=s)
    g.replay()
    torch.cuda.synchronize()
    # y and dx are added in any order, the compact gradient is not; rows past the last expert's are
    # nobody's
    rows = int(a.rt.expert_offset[-1].item())
    assert torch.equal(a.g_act, b.g_act) and torch.equal(a.h[:, :rows], b.h[:, :rows])
    assert rel_l2(b.y.float().cpu().numpy(), a.y.float().cpu().numpy()) <= 1e-2


def test_the_bottom_layer_of_an_8_bit_stack_reads_its_own_input():
    """The bottom layer's input is still the caller's at its backward. With no gradient from above (the
    layers there have no losses), its router's gradient is dlogit^T x with the exact x, bit for bit
    that of a stack that keeps everything."""
    dev = device()
    x = to_dev(synth.moe_inputs(CFG, seed=5)["x"], dev, True)
    got = []
    for act8 in (False, True):
        layers = _layers(dev, CFG, CFG.T, 1, balance_coef=2.0, z_coef=0.5)
        layers += _layers(dev, CFG, CFG.T, 2, seed=61)
        StackTrainer(layers, total_steps=10, reselect_every=0, act8=act8).step(
            [x], [torch.zeros_like(x)])
        torch.cuda.synchronize()
        got.append(layers[0].g_router.clone())
    assert torch.equal(*got) and got[0].any()


# Sizes at which the calls take paths of their own, at the bounds of test_gpu_train_ops.py.
@pytest.mark.parametrize("T,E,k,G", [
    (8192, 128, 8, 1),        # more chunks than one final block takes: blocks of 32 experts
    (40000, 128, 8, 50), (40000, 100, 4, 1),    # several rows of a lane in the gradient, groups change
    (20000, 200, 4, 9), (10000, 500, 3, 7),     # the same with 16 and 32 lanes a row
    (2600001, 8, 2, 1), (2600001, 8, 2, 5)])    # chunks at their largest
@pytest.mark.parametrize("mask", ["none", "some"])
def test_aux_of_long_batches(T, E, k, G, mask):
    dev = device()
    l, idx, m, off = ops._aux_inputs(T, E, k, G, T + E, mask, dead=(E - k) // 3)
    got = ops._aux_run(dev, l, idx, k, G, 1e-2, 1e-3, m, off)
    ops._aux_check(got, TO.router_aux(l, idx, k, 1e-2, 1e-3, m, off))


@pytest.mark.parametrize("T,E,H,bf16", [
    # g_router's two accumulators of few experts used again and again, the leading one emptied often
    (8192, 8, 4096, True), (8192, 40, 4096, True), (16383, 128, 2048, True),
    # dx: several tiles a CTA with each count of boxes and ring slots; one box of features left over
    (2600, 16, 4160, True), (2600, 17, 4160, True), (2600, 64, 4160, True), (2600, 100, 4160, True),
    (2600, 150, 4160, True), (2600, 161, 4160, True), (2600, 600, 4160, True),
    (4000, 200, 1000, False)])
def test_router_grad_of_long_batches(T, E, H, bf16):
    dev = device()
    dl, x, w, g_in, dx_in = ops._grad_inputs(T, E, H, bf16, T + E)
    d_dl, d_w, d_gi = (to_dev(a, dev) for a in (dl, w, g_in))
    d_x, d_xi = to_dev(x, dev, bf16), to_dev(dx_in, dev, bf16)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    g, dx = torch.empty(E, H, device=dev), torch.empty_like(d_x)
    B.router_grad(d_dl, d_x, d_w, g_router=g, g_in=d_gi, dx=dx, dx_in=d_xi, dev_status=st)
    host = lambda t: t.float().cpu().numpy()
    ops._grad_check(host(g), host(dx), dl, x, w, g_in, dx_in, bf16)
    g2, dx2 = torch.empty_like(g), torch.empty_like(dx)  # one product at a time
    B.router_grad(d_dl, d_x, None, g_router=g2, g_in=d_gi, dev_status=st)
    B.router_grad(d_dl, None, d_w, dx=dx2, dx_in=d_xi, dev_status=st)
    assert torch.equal(g2, g) and torch.equal(dx2, dx) and int(st.item()) == 0


@pytest.mark.parametrize("T,H,E,k,I,bf16", [
    (3000, 1000, 16, 3, 40, True), (1500, 256, 16, 4, 64, False), (2000, 2048, 32, 4, 128, True)])
def test_act8_of_larger_layers(T, H, E, k, I, bf16):
    ops.test_act8_matches_fp64_bit_for_bit(T, H, E, k, I, bf16)


def test_tokens_without_a_part_have_no_gradient_under_a_huge_upstream():
    """A finite upstream gradient whose product with the counts is past fp32: 0 stays 0."""
    dev = device()
    T, E, k = 200, 64, 4
    l = torch.randn(T, E, device=dev)
    l[:, 5] = float("-inf")
    mask = (torch.arange(T, device=dev) % 3 != 0).to(torch.uint8)
    idx = l.topk(k, dim=1).indices.to(torch.int32).reshape(-1)
    new = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device=dev)
    cnt, n, d = new(1, E, dt=torch.int32), new(1, dt=torch.int32), torch.ones(T, E, device=dev)
    B.router_aux_fwd(l, idx, k, cnt, new(1, E), n, new(3), 1e4, 1e4, token_mask=mask)
    B.router_aux_bwd(l, k, cnt, n, d, 1e4, 1e4, d_loss=torch.tensor([3e38], device=dev),
                     token_mask=mask)
    assert not d[mask == 0].any() and not d[:, 5].any() and not torch.isfinite(d[mask != 0]).all()


def test_a_store_made_for_another_stream_is_that_streams_memory():
    """A store that save_act8 allocates may be memory that was just freed; it has to have been freed on
    the stream that writes it, or work pending on the freeing stream would see it overwritten."""
    dev = device()
    L, = _layers(dev, CFG, CFG.T, 1)
    x = to_dev(synth.moe_inputs(CFG, seed=6)["x"], dev, True)
    L.route(x)
    L.forward(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    store = L.save_act8(x, stream=side)
    torch.cuda.synchronize()
    for t in (store.x_code, store.x_exp, store.h_code, store.h_exp):
        seg, = [s for s in torch.cuda.memory_snapshot()
                if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]]
        assert seg["stream"] == side.cuda_stream
