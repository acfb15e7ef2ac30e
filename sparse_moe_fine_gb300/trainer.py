"""Training loop around the layer calls: a stack of USAF MoE layers, several micro-batches per
step, a cosine learning-rate schedule, and reselection of the active sets every few steps.

The schedule and cadence follow the USAF README: learning rate peaking at LR_PEAK with cosine
decay, MICROBATCH micro-batches accumulated per optimizer step, the active set reselected every
RESELECT_EVERY steps from an accumulated dense gradient (RigL drop/grow, or a full re-rank), and
steps with a non-finite gradient skipped and counted. Every tensor operation on the path is one of
the library's calls; this module sequences them and keeps the counters.
"""
from __future__ import annotations

import math

import torch

from . import binding as B
from . import dist_select as DS
from .layer import allreduce_dense_grad
from .optim import AdamW


def cosine_lr(step: int, total_steps: int, peak: float, warmup_steps: int = 0,
              floor: float = 0.0) -> float:
    """Learning rate of optimizer step `step` (counted from 1): linear warm-up to `peak` over
    `warmup_steps`, then cosine decay from `peak` to `floor` at `total_steps`."""
    if warmup_steps > 0 and step <= warmup_steps:
        return peak * step / warmup_steps
    span = max(1, total_steps - warmup_steps)
    prog = min(max((step - warmup_steps) / span, 0.0), 1.0)
    return floor + 0.5 * (peak - floor) * (1.0 + math.cos(math.pi * prog))


def reselect_due(step: int, every: int) -> bool:
    """Whether optimizer step `step` (from 1) ends with a reselection of the active sets."""
    return every > 0 and step % every == 0


class StackTrainer:
    """Steps a stack of MoELayer objects: the output y of layer i is the input x of layer i+1, and
    the input gradient dx of layer i+1 is the upstream gradient dy of layer i."""

    def __init__(self, layers, total_steps, lr_peak=2e-4, warmup_steps=0, reselect_every=50,
                 reselect="rigl", drop_frac=0.3, skip_nonfinite=True, dense_exchange="allreduce",
                 act8=False, router_adamw=None):
        """router_adamw: options of optim.AdamW (a dict: weight_decay, state_bits, max_norm, ...) that
        trains the routers of all layers together in one step at the trainer's learning rate, instead of
        each layer's SparseAdam on its own: with weight decay, clipped by the norm of all their gradients,
        or with states in 8 bits. A non-finite gradient in one layer then keeps all routers as they are.
        The optimizer is self.router_opt; its state is in its own state_dict.

        act8: keep each layer's activations in 8 bits between its forward and its backward
        (usaf_act8_save / _restore). Layers of the same shape then share x_perm, h, wa and their
        workspaces, and all layers two output and two input-gradient buffers per shape, so a layer
        below the top costs 17/16 bytes a value of x and h instead of its own bf16 buffers (layers
        allocate those when they first use them: layers that have not run hold none). The top layer's backward
        follows its forward and reads its activations as they are. Layers' y and dx are then only
        what the last call left there.

        dense_exchange (data parallel only): how the replicas agree on the importance phase's
        gradient. "allreduce": every rank sums the whole dense gradient and selects alone;
        "reduce_scatter": every rank sums one part and the selection runs over the parts
        (dist_select), moving half the bytes and ranking 1/world of the entries per rank."""
        if reselect not in ("rigl", "full"):
            raise ValueError("reselect must be 'rigl' or 'full'")
        if dense_exchange not in ("allreduce", "reduce_scatter"):
            raise ValueError("dense_exchange must be 'allreduce' or 'reduce_scatter'")
        self.dense_exchange = dense_exchange
        self.layers = list(layers)
        self.total_steps = total_steps
        self.lr_peak, self.warmup_steps = lr_peak, warmup_steps
        self.reselect_every, self.reselect = reselect_every, reselect
        self.drop_frac = drop_frac
        self.skip_nonfinite = skip_nonfinite
        self.step_no = 0
        self.history = []  # per step: lr, status words, turnover (device tensors until read)
        self._g_dense = [None] * len(self.layers)
        self.act8 = bool(act8)
        if self.act8:
            self._share_buffers()
        self.router_opt = None
        if router_adamw is not None:
            flat = lambda t: t.view(-1)
            self.router_opt = AdamW([L.r_p for L in self.layers],
                                    [flat(L.g_router) for L in self.layers],
                                    copies=[flat(L.w_router) for L in self.layers],
                                    **{"eps": self.layers[0].eps, "betas": self.layers[0].betas,
                                       **router_adamw})
            self._router_status = torch.zeros(1, dtype=torch.int32, device=self.layers[0].dev)

    def _share_buffers(self):
        """One x_perm, h, wa, set of workspaces and restored input per layer shape, two y and two dx; a
        store per layer below the top."""
        first, self._x8, flow = {}, {}, {}
        self._key = [(L.dev, L.dtype, L.T, L.H, L.I, B.routed_rows_capacity(L.s))
                     for L in self.layers]
        for i, (L, key) in enumerate(zip(self.layers, self._key)):
            if 0 < i < len(self.layers) - 1 and key not in self._x8:
                self._x8[key] = torch.empty(L.T, L.H, dtype=L.dtype, device=L.dev)
            if key not in first:
                first[key] = L
            else:
                L.share_activations(first[key])
                L.share_scratch(first[key])
            side = (L.dev, L.dtype, L.T, L.H), i % 2
            if side not in flow:
                flow[side] = L.y, L.dx
            L.y, L.dx = flow[side]
            L._graphs = {}
        self._stores = [B.ActStore8.empty(L.s, L.dev) for L in self.layers[:-1]]

    # ------------------------------------------------------------------ one micro-batch
    def _forward(self, x):
        inputs = []
        for L in self.layers:
            inputs.append(x)
            L.route(x)
            y = L.forward(x)
            if self.act8 and L is not self.layers[-1]:
                L.save_act8(x, self._stores[len(inputs) - 1])
            x = y
        return inputs

    def _backward(self, inputs, dy, first, dense, share):
        for i in reversed(range(len(self.layers))):
            L = self.layers[i]
            x = inputs[i]
            if self.act8 and i < len(self.layers) - 1:
                # the bottom layer's input is the caller's, as it was; the others' went with the next
                # layer but one
                x8 = self._x8[self._key[i]] if i > 0 else None
                restored = L.restore_act8(self._stores[i], x8)
                x = x if x8 is None else restored
            dx = L.dx if i > 0 else None  # the bottom layer's input needs no gradient
            L.backward_into(x, dy, accumulate=0 if first else 1, dx=dx,
                            aux_share=share(L) if L.aux else None)
            if dense:
                # the importance phase's dense gradient of this micro-batch, accumulated, from
                # the dh and permuted dy the sparse call just left in the layer's workspace
                if self._g_dense[i] is None:
                    self._g_dense[i] = torch.zeros(L.N, device=L.dev)
                B.moe_wgrad_dense(L.s, L.rt, L.x_perm, L.wa, self._g_dense[i], L.ws_bwd,
                                  accumulate=1, dev_status=L.status)
            dy = L.dx

    def _router_step(self, lr, status):
        """All layers' routers in one AdamW step, or none of them where a layer's step was skipped."""
        bad = (torch.cat(status) & B.DEV_SKIP_MASK).ne(0).any()
        self._router_status.copy_(bad.to(torch.int32) * B.DEV_NONFINITE)
        self.router_opt.step(lr=lr, dev_status=self._router_status,
                             skip_if_nonfinite=1 if self.skip_nonfinite else 0)

    # ------------------------------------------------------------------ one optimizer step
    def _shares(self, sequences):
        """Each micro-batch's share of the step's auxiliary losses: its tokens' share of the tokens of
        all of them, on all ranks."""
        L = next(L for L in self.layers if L.aux)
        n = torch.stack([L.live_tokens(*s) for s in sequences]).float()
        total = n.sum()
        if L.group is not None:
            torch.distributed.all_reduce(total, group=L.group)
        return (n / total.clamp(min=1.0)).split(1)

    def step(self, x_micro, dy_micro, sequences=None):
        """One optimizer step over the micro-batches: x_micro[j] [T,H] is micro-batch j's input
        to the bottom layer, dy_micro[j] [T,H] the gradient at the top layer's output. The
        layers' gradients are summed over the micro-batches, their auxiliary losses averaged.
        sequences[j]: micro-batch j's (group_offset, token_mask) as MoELayer.set_sequences takes them,
        for every layer with auxiliary losses or a gate's bias (the last one's stay set); a micro-batch
        then counts by its tokens (data parallel: on every rank or on none). Without it the layers' own
        sequences hold for every micro-batch, and micro-batches and ranks count alike."""
        if len(x_micro) != len(dy_micro) or not x_micro:
            raise ValueError("need the same number (>= 1) of inputs and upstream gradients")
        if sequences is not None:
            if len(sequences) != len(x_micro):
                raise ValueError("need one (group_offset, token_mask) per micro-batch")
            counting = [L for L in self.layers if L.aux or getattr(L, "gate_bias", None) is not None]
            if not counting:
                raise ValueError("sequences are only for the auxiliary losses and a gate's bias, which are off")
            for L in counting:
                for s in sequences:
                    L._check_sequences(*s)
            # (shares are of the losses' gradients)
            shares = self._shares(sequences) if any(L.aux for L in counting) else [None] * len(sequences)
        self.step_no += 1
        n = self.step_no
        lr = cosine_lr(n, self.total_steps, self.lr_peak, self.warmup_steps)
        dense = reselect_due(n, self.reselect_every)
        for i, L in enumerate(self.layers):
            L.status = L.status2[L.step_count % 2:L.step_count % 2 + 1]
            L.status.zero_()
        for j, (x, dy) in enumerate(zip(x_micro, dy_micro)):
            share = lambda L: L.aux_share(len(x_micro))
            if sequences is not None:
                share = lambda L, s=shares[j]: s
                for L in counting:
                    L.set_sequences(*sequences[j])
            inputs = self._forward(x)
            self._backward(inputs, dy, first=(j == 0), dense=dense, share=share)
        status = []
        for L in self.layers:
            L.lr = lr
            L.optimizer_step(skip_if_nonfinite=1 if self.skip_nonfinite else 0,
                             router=self.router_opt is None)
            L.wait_optimizer()  # the expert update's status bits are in before they are kept
            status.append(L.status.clone())
        if self.router_opt is not None:
            self._router_step(lr, status)
        rec = {"step": n, "lr": lr, "status": status, "turnover": None,
               "router_status": None if self.router_opt is None else self._router_status.clone(),
               "expert_count": [L.rt.expert_count.clone() for L in self.layers],
               "aux_loss": [L.aux_loss.clone() if L.aux else None for L in self.layers]}
        if dense:
            rec["turnover"] = self._reselect()
        self.history.append(rec)
        return rec

    def _reselect(self):
        """New active sets from the accumulated dense gradients; state carried by the library."""
        turn = []
        for i, L in enumerate(self.layers):
            L.wait_optimizer()
            g = self._g_dense[i]
            K = L.K
            new = torch.empty(K, dtype=torch.int64, device=L.dev)
            p, m, v = (torch.empty(K, device=L.dev) for _ in range(3))
            cnt = torch.zeros(1, dtype=torch.int64, device=L.dev)
            if L.group is not None and self.dense_exchange == "reduce_scatter":
                turn.append(self._reselect_parts(L, g, new, p, m, v, cnt))
                L.set_active(new, p, m, v)
                g.zero_()
                continue
            if L.group is not None:
                # data parallel: rank the whole batch's gradient, so the replicas' sets agree
                allreduce_dense_grad(g, L.group)
            if self.reselect == "rigl":
                D = int(self.drop_frac * K)
                B.rigl_swap(g, L.act, D, L.p, L.m, L.v, L.w_gate_up, L.N_gu, L.w_down, new, p, m,
                            v, cnt)
                turn.append(cnt)  # entries swapped
            else:
                B.reselect_full(g, K, L.act, L.p, L.m, L.v, L.w_gate_up, L.N_gu, L.w_down, new,
                                p, m, v, cnt)
                turn.append(K - cnt)  # entries not kept
            L.set_active(new, p, m, v)
            g.zero_()
        return turn

    def _reselect_parts(self, L, g, new, p, m, v, cnt):
        """Reselection with the dense gradient reduce-scattered: each rank holds the batch's sum
        over one part of the entries; the new set (or RigL's grow set) is selected over the parts
        of all ranks, and every rank carries its state with the library as on one GPU."""
        part, lo = DS.reduce_scatter_part(g, L.group)
        comm, ops = DS.TorchComm(L.group), DS.LibShardOps()
        if self.reselect == "rigl":
            D = int(self.drop_frac * L.K)
            excl = DS.part_bitmap(L.act, lo, part.numel())
            grown = DS.topk_over_parts([(part, lo, excl)], D, ops, comm)
            B.rigl_apply(L.act, D, grown, L.p, L.m, L.v, L.w_gate_up, L.N_gu, L.w_down, new, p,
                         m, v, cnt)
            return cnt
        new.copy_(DS.topk_over_parts([(part, lo, None)], L.K, ops, comm))
        B.reselect_carry(new, L.act, L.p, L.m, L.v, L.w_gate_up, L.N_gu, L.w_down, p, m, v, cnt)
        return L.K - cnt

    # ------------------------------------------------------------------ metrics
    def metrics(self):
        """Host view of the recorded steps (synchronises): learning rate, whether the step was
        skipped for a non-finite gradient, turnover fraction at reselections, and the load
        balance (largest expert count over the mean) and, where they are on, the auxiliary losses
        (total, balance, z) of the last micro-batch per layer. router_skipped: whether the step of all
        routers together (router_adamw; else None) was skipped, for one layer's skip or because the norm
        of their gradients is not finite, which is known only after the layers' own updates."""
        torch.cuda.synchronize()
        out = []
        for r in self.history:
            skipped = [bool(int(s.item()) & 1) for s in r["status"]]
            turnover = None
            if r["turnover"] is not None:
                turnover = [int(t.item()) / L.K for t, L in zip(r["turnover"], self.layers)]
            balance = [float(c.max().item()) / max(1e-9, float(c.float().mean().item()))
                       for c in r["expert_count"]]
            rs = r["router_status"]
            out.append({"step": r["step"], "lr": r["lr"], "skipped": skipped,
                        "router_skipped": None if rs is None else bool(int(rs.item()) & 1),
                        "turnover": turnover, "load_balance": balance,
                        "aux_loss": [None if a is None else a.tolist() for a in r["aux_loss"]]})
        return out
