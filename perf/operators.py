"""What is timed of the router's auxiliary losses, its dense gradient products and the 8-bit
activation store: inputs of the sizes a train step meets, each operator's plain form in elementary
torch operations, its definition in 64 bits, and the calls a user makes of the library.

Kinds of case:
  aux      forward and backward of the balance loss and the z-loss over router logits
  rgrad    the products of a dense router gradient with the tokens and with the router weight
  trip     a layer's x and h into the 8-bit store and back into what the backward reads
  restore  the second half alone: the backward's inputs from a store kept since the forward
"""
import torch

own = False

DEV = "cuda"
BLOCK = 16        # elements that share an exponent in the 8-bit store
ROW_ALIGN = 16    # an expert's rows start at a multiple of this
COEF_BALANCE, COEF_Z = 1e-2, 1e-3


# ------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # the framework's tiny fp32 layer: one small micro-batch, where launches are the time
        dict(name="aux_tiny", kind="aux", T=128, E=8, k=2, G=1, masked=False, dead=0),
        # a Qwen3-30B-A3B-shaped layer's routing of one batch
        dict(name="aux_qwen3", kind="aux", T=4096, E=128, k=8, G=1, masked=False, dead=0),
        # the same router over a long packed batch: ragged sequences, padding tokens, ten experts
        # that no token may take
        dict(name="aux_packed", kind="aux", T=16383, E=128, k=8, G=37, masked=True, dead=10),
        # router gradients of the tiny fp32 layer, the Qwen3 layer, the Mixtral layer (few experts,
        # wide tokens) and a long odd batch of the Qwen3 layer
        dict(name="rgrad_tiny_f32", kind="rgrad", T=128, E=8, H=64, dtype="f32"),
        dict(name="rgrad_qwen3", kind="rgrad", T=4096, E=128, H=2048, dtype="bf16"),
        dict(name="rgrad_mixtral", kind="rgrad", T=8192, E=8, H=4096, dtype="bf16"),
        dict(name="rgrad_qwen3_long", kind="rgrad", T=16383, E=128, H=2048, dtype="bf16"),
        # a small layer, a Qwen3 layer and a Mixtral layer checkpointed and brought back
        dict(name="trip_small", kind="trip", T=200, E=8, k=2, H=128, I=128, dtype="bf16",
             zipf=0.0),
        dict(name="trip_qwen3", kind="trip", T=4096, E=128, k=8, H=2048, I=768, dtype="bf16",
             zipf=0.0),
        dict(name="trip_mixtral", kind="trip", T=8192, E=8, k=2, H=4096, I=14336, dtype="bf16",
             zipf=0.0),
        # the backward's half: a Qwen3 layer, and a long odd batch with Zipf-skewed experts
        dict(name="restore_qwen3", kind="restore", T=4096, E=128, k=8, H=2048, I=768,
             dtype="bf16", zipf=0.0),
        dict(name="restore_skewed", kind="restore", T=16383, E=128, k=8, H=2048, I=768,
             dtype="bf16", zipf=1.2),
    ]


def _log_int(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    import math
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {}
    for c in listed():
        for q, v in work(c).items():
            most[c["kind"], q] = max(v, most.get((c["kind"], q), 0))
    kind = rng.choice(["aux", "rgrad", "trip", "restore"])
    while True:
        E = _log_int(rng, 2, 256)
        k = rng.randint(1, min(8, E))
        if kind == "aux":
            T = _log_int(rng, 1, 32768)
            c = dict(kind=kind, T=T, E=E, k=k, G=_log_int(rng, 1, min(64, T)),
                     masked=rng.random() < 0.5, dead=rng.randint(0, (E - k) // 2))
        elif kind == "rgrad":
            f32 = rng.random() < 0.25
            H = _log_int(rng, 3, 1025) if f32 else 64 * _log_int(rng, 1, 64)
            T = _log_int(rng, 1, 2048 if f32 else 32768)
            c = dict(kind=kind, T=T, E=E, H=H, dtype="f32" if f32 else "bf16")
        else:
            f32 = rng.random() < 0.25
            H = _log_int(rng, 3, 1025) if f32 else 64 * _log_int(rng, 1, 64)
            I = _log_int(rng, 3, 1025) if f32 else 64 * _log_int(rng, 1, 224)
            c = dict(kind=kind, T=_log_int(rng, 1, 2048 if f32 else 16384), E=E, k=k, H=H, I=I,
                     dtype="f32" if f32 else "bf16", zipf=rng.choice([0.0, 0.0, 1.2]))
        if 3072 not in c.values() and all(v <= most[kind, q] for q, v in work(c).items()):
            return c


def work(case):
    """What a pass cannot do without: each input read once, each output written once."""
    T, E = case["T"], case["E"]
    if case["kind"] == "aux":
        k, G = case["k"], case["G"]
        read = 4 * T * E + 4 * T * k + (T if case["masked"] else 0) + 4 * (G + 1)
        write = 8 * G * E + 4 * G + 12 + 4 * T * E
        return {"bytes": read + write, "flops": 12 * T * E + 2 * T * k}
    b = 4 if case["dtype"] == "f32" else 2
    H = case["H"]
    if case["kind"] == "rgrad":
        read = 4 * T * E + 4 * E * H + 2 * b * T * H
        return {"bytes": read + 4 * E * H + b * T * H, "flops": 4 * T * E * H + T * H}
    k, I = case["k"], case["I"]
    R = T * k
    n = T * H + 2 * I * R                      # values that go into the store
    store = n + (T * -(-H // BLOCK) + 2 * I * -(-R // BLOCK))
    out = b * (T * H + H * R + 3 * I * R)
    tables = 4 * (3 * R + E + 1)
    if case["kind"] == "restore":
        return {"bytes": store + out + tables, "flops": n + H * R + 6 * I * R}
    return {"bytes": b * n + store + store + out + tables, "flops": 4 * n + H * R + 6 * I * R}


# ------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _router_logits(case, g):
    """Logits of a trained router: a token part and an expert bias (Zipf-like where skewed)."""
    T, E = case["T"], case["E"]
    l = torch.randn(T, E, generator=g, device=DEV)
    l += 0.7 * torch.randn(E, generator=g, device=DEV)
    if case.get("zipf"):
        rank = torch.randperm(E, generator=g, device=DEV).float() + 1
        l -= case["zipf"] * torch.log(rank)
    return l


def _routing_tables(topk, w, E):
    """The tables of a routing call: experts' slots in token order, each expert's rows starting at
    a multiple of ROW_ALIGN. The row capacity is the library's."""
    T, k = topk.shape
    R = T * k
    cap = -(-(R + E * (ROW_ALIGN - 1)) // 256) * 256 + 256
    flat = topk.reshape(-1).long()
    count = torch.bincount(flat, minlength=E)
    padded = (count + ROW_ALIGN - 1) // ROW_ALIGN * ROW_ALIGN
    off = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    off[1:] = padded.cumsum(0)
    order = torch.sort(flat, stable=True).indices
    first = torch.zeros(E, dtype=torch.int64, device=DEV)
    first[1:] = count.cumsum(0)[:-1]
    e_sorted = flat[order]
    row = off[e_sorted] + torch.arange(R, device=DEV) - first[e_sorted]
    slot_row = torch.empty(R, dtype=torch.int64, device=DEV)
    slot_row[order] = row
    perm_slot = torch.full((cap,), -1, dtype=torch.int64, device=DEV)
    perm_slot[row] = order
    perm_tok = torch.where(perm_slot >= 0, perm_slot // k, torch.zeros_like(perm_slot))
    i32 = torch.int32
    return dict(topk_idx=flat.to(i32), topk_w=w.reshape(-1).contiguous(),
                expert_count=count.to(i32), expert_offset=off.to(i32), perm_tok=perm_tok.to(i32),
                perm_slot=perm_slot.to(i32), slot_row=slot_row.to(i32)), cap


def _torch_dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _inputs(case, seed):
    g = _gen(seed)
    T, E = case["T"], case["E"]
    if case["kind"] == "aux":
        k, G = case["k"], case["G"]
        l = _router_logits(case, g)
        if case["dead"]:  # experts no token may take: their logits are -inf
            l[:, torch.randperm(E, generator=g, device=DEV)[:case["dead"]]] = float("-inf")
        idx = torch.topk(l, k, dim=1).indices.to(torch.int32).contiguous()
        cuts = torch.randint(0, T + 1, (G - 1,), generator=g, device=DEV).sort().values
        ends = torch.tensor([T], device=DEV)
        off = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), cuts, ends])
        mask = None
        if case["masked"]:
            mask = (torch.rand(T, generator=g, device=DEV) < 0.9).to(torch.uint8)
        return dict(logits=l, topk_idx=idx.reshape(-1), mask=mask,
                    group_offset=off.to(torch.int32) if G > 1 else None)
    H, dt = case["H"], _torch_dtype(case)
    if case["kind"] == "rgrad":
        p = torch.softmax(_router_logits(dict(T=T, E=E), g), dim=1)
        a = torch.randn(T, E, generator=g, device=DEV)
        dl = p * (a - (p * a).sum(1, keepdim=True))  # a softmax's gradient: rows sum to zero
        return dict(dlogit=dl, x=torch.randn(T, H, generator=g, device=DEV).to(dt),
                    w_router=0.02 * torch.randn(E, H, generator=g, device=DEV),
                    dx_in=(0.01 * torch.randn(T, H, generator=g, device=DEV)).to(dt))
    k, I = case["k"], case["I"]
    l = _router_logits(case, g)
    top = torch.topk(l, k, dim=1)
    rt, cap = _routing_tables(top.indices, torch.softmax(top.values, dim=1), E)
    # hidden states: features of uneven size, a few of them large
    scale = torch.exp(0.5 * torch.randn(H, generator=g, device=DEV))
    scale[torch.rand(H, generator=g, device=DEV) < 0.005] *= 20
    x = (torch.randn(T, H, generator=g, device=DEV) * scale).to(dt)
    h = torch.randn(2 * I, cap, generator=g, device=DEV, dtype=dt)
    h *= (rt["perm_slot"] >= 0).to(dt)  # padding rows hold zeros
    return dict(x=x, h=h, rt=rt, cap=cap)


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    T, E = case["T"], case["E"]
    if own:
        from sparse_moe_fine_gb300 import binding as B
        st["B"] = B
    if case["kind"] == "aux":
        if own:
            G = case["G"]
            st["out"] = dict(loss=torch.zeros(3, device=DEV),
                             count=torch.zeros(G, E, dtype=torch.int32, device=DEV),
                             prob_sum=torch.zeros(G, E, device=DEV),
                             n_tok=torch.zeros(G, dtype=torch.int32, device=DEV),
                             dlogit=torch.zeros(T, E, device=DEV))
            st["ws"] = torch.empty(st["B"].router_aux_workspace_size(T, E, case["k"], G),
                                   dtype=torch.uint8, device=DEV)
        return st
    H, dt = case["H"], _torch_dtype(case)
    if case["kind"] == "rgrad":
        if own:
            B = st["B"]
            st["g_router"] = torch.zeros(E, H, device=DEV)
            st["dx"] = torch.zeros(T, H, dtype=dt, device=DEV)
            st["ws"] = torch.empty(B.router_grad_workspace_size(T, E, H, st["x"].dtype),
                                   dtype=torch.uint8, device=DEV)
        return st
    I, cap = case["I"], st["cap"]
    if case["kind"] == "restore":  # the store, as the forward left it
        x, h = st.pop("x"), st.pop("h")
        st["store"] = _encode_f32(x, True) + _encode_f32(h, False)
        del x, h
    if own:
        B = st["B"]
        st["shape"] = B.shape(T, H, E, case["k"], I)
        st["routing"] = B.Routing(**st["rt"])
        if case["kind"] == "restore":
            st["act"] = B.ActStore8(*st["store"])
        else:
            st["act"] = B.ActStore8.empty(st["shape"], DEV)
        new = lambda *s: torch.zeros(*s, dtype=dt, device=DEV)
        st["out"] = dict(x=new(T, H), x_perm=new(H, cap), h=new(2 * I, cap), wa=new(I, cap))
    return st


# ------------------------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    if own:
        return _RUN_OWN[case["kind"]](state)
    return _RUN_PLAIN[case["kind"]](state)


def _own_aux(st):
    B, o, case = st["B"], st["out"], st["case"]
    B.router_aux_fwd(st["logits"], st["topk_idx"], case["k"], o["count"], o["prob_sum"],
                     o["n_tok"], o["loss"], COEF_BALANCE, COEF_Z, token_mask=st["mask"],
                     group_offset=st["group_offset"], ws=st["ws"])
    B.router_aux_bwd(st["logits"], case["k"], o["count"], o["n_tok"], o["dlogit"], COEF_BALANCE,
                     COEF_Z, token_mask=st["mask"], group_offset=st["group_offset"])
    return o


def _own_rgrad(st):
    st["B"].router_grad(st["dlogit"], st["x"], st["w_router"], g_router=st["g_router"],
                        dx=st["dx"], dx_in=st["dx_in"], ws=st["ws"])
    return {"g_router": st["g_router"], "dx": st["dx"]}


def _own_restore(st):
    o = st["out"]
    st["B"].act8_restore(st["shape"], st["act"], st["routing"], o["x_perm"], o["h"], o["wa"],
                         x=o["x"])
    return o


def _own_trip(st):
    st["B"].act8_save(st["shape"], st["x"], st["h"], st["routing"], st["act"])
    return _own_restore(st)


def _plain_aux(st):
    case, l, mask, off = st["case"], st["logits"], st["mask"], st["group_offset"]
    T, E, k = case["T"], case["E"], case["k"]
    top = l.max(1, keepdim=True).values
    live = top[:, 0] != float("-inf")
    if mask is not None:
        live = live & (mask != 0)
    ex = torch.exp(l - torch.where(live[:, None], top, torch.zeros_like(top)))
    total = ex.sum(1, keepdim=True)
    one = torch.ones_like(total)
    p = torch.where(live[:, None], ex / torch.where(live[:, None], total, one), 0.0)
    lse = torch.where(live, (top + torch.log(torch.where(live[:, None], total, one)))[:, 0], 0.0)
    tok = torch.arange(T, device=DEV)
    if off is None:
        member = live[None, :].float()
    else:
        member = ((tok >= off[:-1, None]) & (tok < off[1:, None]) & live).float()
    n_g = member.sum(1)
    n = n_g.sum()
    chosen = torch.zeros(T, E, device=DEV)
    chosen.scatter_add_(1, st["topk_idx"].view(T, k).long(), torch.ones(T, k, device=DEV))
    count = member @ chosen
    prob = member @ p
    inv_g = torch.where(n_g > 0, 1 / n_g.clamp(min=1), 0.0)
    inv_n = torch.where(n > 0, 1 / n.clamp(min=1), 0.0)
    balance = E / k * inv_n * ((count * prob).sum(1) * inv_g).sum()
    z = inv_n * (lse * lse).sum()
    loss = torch.stack([COEF_BALANCE * balance + COEF_Z * z, balance, z])
    c_t = member.t() @ (count * inv_g[:, None])       # each token's group counts over n_g
    d = COEF_BALANCE * E / k * inv_n * (c_t - (p * c_t).sum(1, keepdim=True))
    dlogit = p * (d + COEF_Z * 2 * inv_n * lse[:, None])
    return dict(loss=loss, count=count.to(torch.int32), prob_sum=prob,
                n_tok=n_g.to(torch.int32), dlogit=dlogit)


def _plain_rgrad(st):
    dl, x = st["dlogit"], st["x"]
    g = dl.t() @ x.float()
    dx = st["dx_in"].float() + dl @ st["w_router"]
    return {"g_router": g, "dx": dx.to(x.dtype)}


def _encode_f32(v, ragged):
    """(codes, exponent bytes) of blocks of 16 along the last axis: the least power of two whose
    127-fold covers the block's largest magnitude. `ragged`: the last block may be short."""
    rows, n = v.shape
    nb = -(-n // BLOCK)
    f = v.float()
    if ragged and nb * BLOCK != n:
        f = torch.nn.functional.pad(f, (0, nb * BLOCK - n))
    f = f.view(rows, nb, BLOCK)
    amax = f.abs().amax(2)
    bits = amax.contiguous().view(torch.int32)
    # amax = m 2^q, 1 <= m < 2: 127 2^(q - 6) covers it while m <= 127 / 64
    byte = (bits >> 23) - 6 + ((bits & 0x7FFFFF) > 0x7E0000).int()
    byte = torch.where(amax == 0, 0, byte.clamp(1, 248))
    inv = ((254 - byte) << 23).view(torch.float32)
    inv = torch.where(byte == 0, 0.0, inv)
    code = torch.round(f * inv[..., None]).clamp(-127, 127)
    code = code.to(torch.int8).view(rows, nb * BLOCK)[:, :n].contiguous()
    return code, byte.to(torch.uint8)


def _decode_f32(code, byte):
    rows, n = code.shape
    scale = (byte.int() << 23).view(torch.float32)
    scale = scale.repeat_interleave(BLOCK, dim=1)[:, :n]
    return code.float() * scale


def _plain_restore(st, store=None):
    case, rt = st["case"], st["rt"]
    dt, I = _torch_dtype(case), case["I"]
    xc, xe, hc, he = st["store"] if store is None else store
    live = rt["perm_slot"] >= 0
    x = _decode_f32(xc, xe)
    x_perm = (x[rt["perm_tok"].long()] * live[:, None].float()).to(dt).t().contiguous()
    h = _decode_f32(hc, he)
    w = torch.where(live, rt["topk_w"][rt["perm_slot"].long().clamp(min=0)], 0.0)
    gate = h[:I]
    wa = w * (gate / (1 + torch.exp(-gate))) * h[I:]
    return dict(x=x.to(dt), x_perm=x_perm, h=h.to(dt), wa=wa.to(dt))


def _plain_trip(st):
    return _plain_restore(st, _encode_f32(st["x"], True) + _encode_f32(st["h"], False))


_RUN_OWN = dict(aux=_own_aux, rgrad=_own_rgrad, trip=_own_trip, restore=_own_restore)
_RUN_PLAIN = dict(aux=_plain_aux, rgrad=_plain_rgrad, trip=_plain_trip, restore=_plain_restore)


# ------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    inp = _inputs(case, seed)
    f64 = torch.float64
    T, E = case["T"], case["E"]
    if case["kind"] == "aux":
        return _exact_aux(case, inp)
    if case["kind"] == "rgrad":
        dl, x, w = inp["dlogit"].to(f64), inp["x"].to(f64), inp["w_router"].to(f64)
        return {"g_router": torch.einsum("te,th->eh", dl, x),
                "dx": inp["dx_in"].to(f64) + torch.einsum("te,eh->th", dl, w)}
    I, rt = case["I"], inp["rt"]
    x = _round_trip64(inp.pop("x").to(f64))
    h = _round_trip64(inp.pop("h").to(f64))
    slot = rt["perm_slot"].long()
    x_perm = torch.zeros(x.shape[1], slot.numel(), dtype=f64, device=DEV)
    routed = torch.nonzero(slot >= 0)[:, 0]
    x_perm[:, routed] = x[slot[routed] // case["k"]].t()
    wa = torch.zeros(I, slot.numel(), dtype=f64, device=DEV)
    gate, up = h[:I][:, routed], h[I:][:, routed]
    wa[:, routed] = rt["topk_w"].to(f64)[slot[routed]] * gate * torch.sigmoid(gate) * up
    return dict(x=x, x_perm=x_perm, h=h, wa=wa)


def _round_trip64(v):
    """What the 8-bit store keeps of v, block by block, by exponents from frexp."""
    out = torch.empty_like(v)
    n = v.shape[1]
    whole = n - n % BLOCK
    parts = [(0, whole, BLOCK)] if whole else []
    if n > whole:
        parts.append((whole, n, n - whole))
    for lo, hi, width in parts:
        b = v[:, lo:hi].unflatten(1, (-1, width))
        amax = b.abs().amax(2, keepdim=True)
        m, q = torch.frexp(amax)                     # amax = m 2^q, 1/2 <= m < 1
        e = torch.where(m <= 127 / 128, q - 7, q - 6).clamp(-126, 121)
        step = ((e.long() + 1023) << 52).view(torch.float64)  # 2^e from its bits: exact
        out[:, lo:hi] = (torch.round(b / step).clamp(-127, 127) * step).flatten(1)
    return out


def _exact_aux(case, inp):
    f64 = torch.float64
    T, E, k, G = case["T"], case["E"], case["k"], case["G"]
    l = inp["logits"].to(f64)
    live = ~torch.isinf(l).all(1)
    if inp["mask"] is not None:
        live &= inp["mask"].bool()
    p = torch.softmax(l, dim=1)
    lse = torch.logsumexp(l, dim=1)
    off = [0, T] if inp["group_offset"] is None else inp["group_offset"].tolist()
    idx = inp["topk_idx"].view(T, k).long()
    count = torch.zeros(G, E, dtype=torch.int32, device=DEV)
    prob = torch.zeros(G, E, dtype=f64, device=DEV)
    n_tok = torch.zeros(G, dtype=torch.int32, device=DEV)
    for g in range(G):
        sel = torch.nonzero(live[off[g]:off[g + 1]])[:, 0] + off[g]
        n_tok[g] = sel.numel()
        count[g] = torch.bincount(idx[sel].reshape(-1), minlength=E).to(torch.int32)
        prob[g] = p[sel].sum(0)
    n = int(n_tok.sum())
    dlogit = torch.zeros(T, E, dtype=f64, device=DEV)
    balance = torch.zeros((), dtype=f64, device=DEV)
    z = torch.zeros((), dtype=f64, device=DEV)
    for g in range(G):
        sel = torch.nonzero(live[off[g]:off[g + 1]])[:, 0] + off[g]
        if not sel.numel():
            continue
        c = count[g].to(f64)
        share = E / (k * n * sel.numel())
        balance += share * (c * prob[g]).sum()
        z += (lse[sel] ** 2).sum() / n
        ps = p[sel]
        pull = COEF_BALANCE * share * (c - (ps * c).sum(1, keepdim=True))
        dlogit[sel] = ps * (pull + COEF_Z * 2 / n * lse[sel, None])
    loss = torch.stack([COEF_BALANCE * balance + COEF_Z * z, balance, z])
    return dict(loss=loss, count=count, prob_sum=prob, n_tok=n_tok, dlogit=dlogit)
