"""Per-view training step over the libgs C ABI (the BoundedGS schedule).

BoundedGS project page, section 01: for one view the parameters stay fixed,
each Leaf runs forward, loss and backward, its gradient is merged and its
buffers are released before the next Leaf; after the whole view one update
is applied.  Section 02: A -> B (raster backward collects the projected
gradients, the raster buffers are released, then projection backward runs),
B -> C (load-budgeted Leaves, re-planned from the current view's counts),
C -> D -> E (candidate-only projected state and compact gradients).

This module only sequences library calls and carves device buffers out of
torch allocations; every stage runs in libgs kernels.
"""
from __future__ import annotations

import dataclasses
import math

import numpy as np
import torch

from . import binding as B
from .codebook import SH_PLANE

DEFAULT_BUDGET = 384 << 20

STAGES = ("project", "sort_depth", "bin", "sort_tiles", "expand", "raster_fwd", "ssim",
          "raster_bwd", "project_bwd")


def _carve(arena: torch.Tensor, sizes):
    """Split a uint8 arena into 256-byte aligned byte views."""
    out, off = [], 0
    for s in sizes:
        off = (off + 255) // 256 * 256
        out.append(arena[off:off + s])
        off += s
    return out, off


def _carved_bytes(sizes):
    off = 0
    for s in sizes:
        off = (off + 255) // 256 * 256 + s
    return off


@dataclasses.dataclass
class ViewStats:
    n_cand: int
    n_isect: int          # entries of the (tight) tile lists
    n_isect_square: int   # tiles of the candidates' plain 3-sigma squares
    n_block_entries: int  # entries of the per-block lists (two-level binning)
    n_block_reads: int    # block-list entries the Leaves' expansions read (summed)
    n_leaves: int
    leaves: np.ndarray
    leaf_isect: np.ndarray
    leaf_bytes: np.ndarray
    over_budget: np.ndarray
    peak_ws_bytes: int
    arena_bytes: int
    launches: int


def _merge_stats(stats):
    """Statistics of a view run as several regions."""
    return ViewStats(
        n_cand=sum(x.n_cand for x in stats), n_isect=sum(x.n_isect for x in stats),
        n_isect_square=sum(x.n_isect_square for x in stats),
        n_block_entries=sum(x.n_block_entries for x in stats),
        n_block_reads=sum(x.n_block_reads for x in stats),
        n_leaves=sum(x.n_leaves for x in stats),
        leaves=np.concatenate([x.leaves for x in stats]),
        leaf_isect=np.concatenate([x.leaf_isect for x in stats]),
        leaf_bytes=np.concatenate([x.leaf_bytes for x in stats]),
        over_budget=np.concatenate([x.over_budget for x in stats]),
        peak_ws_bytes=max(x.peak_ws_bytes for x in stats),
        arena_bytes=max(x.arena_bytes for x in stats),
        launches=sum(x.launches for x in stats))


class GaussianModel:
    """Parameters and Adam moments, planar [P][n_pad] fp32 on the device."""

    def __init__(self, params, n: int, sh_degree: int, device="cuda"):
        p = torch.as_tensor(params, dtype=torch.float32)
        self.params = p.to(device).contiguous()
        self.m = torch.zeros_like(self.params)
        self.v = torch.zeros_like(self.params)
        self.n = int(n)
        self.sh_degree = int(sh_degree)
        self.step = 0

    @property
    def P(self):
        return self.params.shape[0]

    @property
    def n_pad(self):
        return self.params.shape[1]

    def struct(self) -> B.gs_model:
        return B.gs_model(self.n, self.n_pad, self.sh_degree, 0, self.params.data_ptr())


class TargetPrefetcher:
    """Supplies views' targets to the device one view ahead.  While the step
    of view k runs, the target of the next view in the order is copied from
    pinned host memory on a copy stream into the other of two device buffers,
    so its upload overlaps the step instead of the Leaves' compute.  Holds
    two device targets (2 x 3 x H x W fp32); the per-Leaf crop supply of
    `Stepper.run_view` with a host target holds two Leaf crops instead.

    Given the Stepper that consumes the targets, the next upload is issued
    once the current view's projection tables have reached the host: a
    device-to-host copy queued behind a 200 MB upload would hold back the
    host's Leaf planning (0.12 ms per step on the 5000x3300 views).

        feeder = TargetPrefetcher(host_targets, stepper=stepper)
        for v, target in feeder.iterate(order):
            stepper.run_view(cams[v], target)
    """

    def __init__(self, host_targets, device="cuda", stepper=None):
        self.host = host_targets          # indexable: view -> pinned [3][H][W] fp32
        self.device = torch.device(device)
        self.stream = torch.cuda.Stream(device=self.device)
        self.stepper = stepper
        # the two device buffers are allocated here, not in the first step
        # of an iteration (where a new device allocation would stall it)
        self._bufs = None
        if len(host_targets):
            self._alloc(tuple(host_targets[0].shape))

    def _alloc(self, shape):
        self._bufs = [torch.empty(shape, dtype=torch.float32, device=self.device)
                      for _ in range(2)]

    def iterate(self, order):
        order = list(order)
        if not order:
            return
        shape = tuple(self.host[order[0]].shape)
        if self._bufs is None or tuple(self._bufs[0].shape) != shape:
            self._alloc(shape)
        main = torch.cuda.current_stream(self.device)
        ready, free = [None, None], [None, None]

        def upload(slot, v):
            # after the work issued on the main stream so far (with a Stepper:
            # the current view's projection and its tables' read-back), and
            # after the buffer's previous reader (two views back)
            self.stream.wait_stream(main)
            if free[slot] is not None:
                self.stream.wait_event(free[slot])
            with torch.cuda.stream(self.stream):
                self._bufs[slot].copy_(self.host[v], non_blocking=True)
            ev = torch.cuda.Event()
            ev.record(self.stream)
            ready[slot] = ev

        upload(0, order[0])
        for i, v in enumerate(order):
            slot = i & 1
            if i + 1 < len(order):
                nxt = (1 - slot, order[i + 1])
                if self.stepper is not None:
                    self.stepper._after_tables.append(lambda nxt=nxt: upload(*nxt))
                else:
                    upload(*nxt)
            main.wait_event(ready[slot])
            yield v, self._bufs[slot]
            if self.stepper is not None and self.stepper._after_tables:
                # the view was not stepped through this Stepper: upload now
                calls, self.stepper._after_tables = self.stepper._after_tables, []
                for f in calls:
                    f()
            ev = torch.cuda.Event()
            ev.record(main)   # after the step's work on this buffer
            free[slot] = ev


class _Timer:
    def __init__(self, timing):
        self.timing = timing

    def tic(self, name):
        if self.timing is None:
            return None
        e0 = torch.cuda.Event(enable_timing=True)
        e0.record()
        return name, e0

    def toc(self, tk):
        if tk is None:
            return
        e1 = torch.cuda.Event(enable_timing=True)
        e1.record()
        self.timing.setdefault(tk[0], []).append((tk[1], e1))


class Stepper:
    """Runs the per-view step.  `hooks` (optional) is an object whose methods
    `on_project(ctx)`, `on_leaf(ctx, leaf_ctx)`, `on_bwd(ctx)` see
    intermediate buffers (used by the parity tests).

    Options: budget (bytes per Leaf), Adam's lr / betas / eps, raster_flags
    (pixels per thread of the raster kernels, 0 = their defaults), fuse_adam
    (True: projection backward fused with Adam, geometric chain as its own
    pass; "in_stream": the chain inside the Adam stream; False: compact 3D
    gradients and a separate Adam), binning ("fused", "expand", "sort": the
    three list builders), mode ("bounded" or the whole-image "original"),
    loss ("l1" or "l1_ssim" with weight ssim_lambda), leaf_streams (1: one
    Leaf at a time; k = 2..4: consecutive Leaves on k streams with k raster
    arenas), max_grad_norm (the view's whole gradient is scaled to at most
    this L2 norm before Adam; `last_grad_norm` gives the norm before that),
    codebook (codebook.ColorCodebook: the SH planes are decoded from its
    table, and the update trains the table instead of them).  Both take the
    view's gradient as compact 3D gradients (fuse_adam's fused pass never
    holds the whole gradient): 4 P bytes per candidate, and a codebook about
    4 (P - 6) more for its workspace, beyond the Leaf budget and sized by the
    view's candidates, not by `reserve`."""

    def __init__(self, model: GaussianModel, budget: int = DEFAULT_BUDGET, lr=1e-3,
                 betas=(0.9, 0.999), eps=1e-8, raster_flags=0, fuse_adam=True,
                 binning="fused", mode="bounded", loss="l1", ssim_lambda=B.SSIM_LAMBDA,
                 leaf_streams=1, device="cuda", max_grad_norm=None, codebook=None):
        if binning not in ("fused", "expand", "sort"):
            raise ValueError(f"binning must be 'fused', 'expand' or 'sort', not {binning!r}")
        if mode not in ("bounded", "original"):
            raise ValueError(f"mode must be 'bounded' or 'original', not {mode!r}")
        # bounded: two-stage backward, Leaves under the budget, candidate-index
        # projection and compact gradients (BoundedGS page, section 02, A -> E);
        # original: the whole-image configuration A of the same page (dense
        # projection state, one whole-image Leaf whose raster buffers stay
        # alive through the projection backward, dense gradients)
        if loss not in ("l1", "l1_ssim"):
            raise ValueError(f"loss must be 'l1' or 'l1_ssim', not {loss!r}")
        # leaf_streams = k > 1: consecutive Leaves rotate over k streams and
        # k raster arenas, so one Leaf's kernels fill the SMs that another's
        # last CTAs leave idle (k Leaves' raster buffers in flight,
        # each within the budget)
        if leaf_streams not in (1, 2, 3, 4):
            raise ValueError(f"leaf_streams must be 1 to 4, not {leaf_streams!r}")
        if max_grad_norm is not None and not 0.0 <= float(max_grad_norm) < math.inf:
            raise ValueError(f"max_grad_norm must be finite and not negative, not {max_grad_norm!r}")
        if codebook is not None:
            codebook.check(model)
        self.max_grad_norm = None if max_grad_norm is None else float(max_grad_norm)
        self.codebook = codebook
        self._clip = None     # device {norm, coefficient}
        self._clip_ws = None
        # l1: the L1 photometric loss; l1_ssim: the composite
        # (1 - lambda) L1 + lambda (1 - SSIM) of 3DGS training (SkipGS notes,
        # "loss function / training strategy"), SSIM windows local to each Leaf
        self.loss = loss
        self.ssim_lambda = float(ssim_lambda)
        self.mode = mode
        self.model = model
        self.binning = binning
        self.budget = int(budget)
        self.lr, self.betas, self.eps = lr, betas, eps
        self.raster_flags = raster_flags
        self.fuse_adam = fuse_adam
        self.device = torch.device(device)
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._last_loss = None
        self._copy_stream = None
        self.leaf_streams = leaf_streams
        self._side_streams = []
        self._fill_stream = None
        # one-shot callables run once the view's projection tables are on the
        # host, before its Leaves are issued (TargetPrefetcher starts the next
        # view's target upload there, after the tables' device-to-host copies)
        self._after_tables = []
        self._arena_hint = 0  # bytes per Leaf arena (bounded runs), see run_view
        self._cap_hint = {}  # region -> candidate capacity for the next view
        if codebook is not None:
            codebook.decode(model, self.dev_status)

    def reserve(self, cams, region=None):
        """Sizes the Leaf arenas for the views a run will step through: each
        view is projected and its Leaves planned (no raster, no update), and
        later steps' arenas take the largest Leaf over these views plus 1/16
        (at most the Leaf budget), so that no step needs a new device
        allocation for them.  Also seeds the candidate-capacity hint."""
        for cam in cams:
            self.run_view(cam, None, region=region, plan_only=True)

    def _zeroed_g2d(self, rows):
        """The compact 2D gradient [rows][12], zeroed on a side stream; the
        event marks the end of the fill."""
        dev = self.device
        g2d = torch.empty(rows * 12, dtype=torch.float32, device=dev)
        if self._fill_stream is None:
            self._fill_stream = torch.cuda.Stream(device=dev)
        self._fill_stream.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(self._fill_stream):
            g2d.zero_()
        ready = torch.cuda.Event()
        ready.record(self._fill_stream)
        return g2d, ready

    def _depth_order(self, proj, count, cap, clk):
        """Candidates in depth order and their rects (gs_depth_order), for
        `count` candidates (or GS_COUNT_ON_DEVICE) in buffers of `cap`."""
        dev = self.device
        order = torch.empty(cap, dtype=torch.int32, device=dev)
        drect = torch.empty(cap * 4, dtype=torch.int16, device=dev)
        ows = torch.empty(B.gs_depth_order_workspace_size(cap), dtype=torch.uint8, device=dev)
        tk = clk.tic("sort_depth")
        B.gs_depth_order(proj, count, order, drect, ows, self.dev_status)
        clk.toc(tk)
        return order, drect

    def check(self):
        st = B.gs_check(self.dev_status)
        if st < 0:
            raise B.GsError("device status", st)

    def adam_args(self, step):
        return B.gs_adam_args(self.lr, self.betas[0], self.betas[1], self.eps, step, 0)

    def last_loss(self) -> float:
        return float(self._last_loss.item())

    def last_grad_norm(self) -> float:
        """The norm of the last update's gradient, before clipping.  An infinite
        norm gives an update of zero gradients (infinite elements count as 0
        too), a NaN norm one of NaN; check() raises after either."""
        if self._clip is None:
            raise ValueError("no update with max_grad_norm was taken")
        return float(self._clip[0].item())

    def _update(self, g, stride, slot, cols, cand_idx):
        """One Adam update from the view's gradient g [P][stride] (`cols`
        columns, of the candidates cand_idx with their slots, or of all
        Gaussians), through the codebook and clipped as the options say."""
        m, cb = self.model, self.codebook
        m.step += 1
        args = self.adam_args(m.step)
        planes = m.P if cb is None else SH_PLANE
        g2 = g.view(m.P, -1)[:, :cols]
        if cb is not None:
            cb.gradient(g2[SH_PLANE:], cand_idx, self.dev_status)
        if self.max_grad_norm is None:
            B.gs_adam(m.params, m.m, m.v, g, stride, slot, m.n, m.n_pad, planes, args)
            if cb is not None:
                size = cb.grad.numel()
                B.gs_adam(cb.table, cb.m, cb.v, cb.grad, size, None, size, size, 1, args)
        else:
            grads = B.tensor_list([g2[:planes]] + ([cb.grad] if cb is not None else []))
            if self._clip is None:
                self._clip = torch.empty(2, dtype=torch.float32, device=self.device)
                self._clip_ws = torch.empty(B.gs_grad_norm_workspace_size(grads),
                                            dtype=torch.uint8, device=self.device)
            B.gs_grad_norm(grads, self.max_grad_norm, self._clip, self._clip_ws,
                           dev_status=self.dev_status)
            B.gs_adam_clipped(m.params, m.m, m.v, g, stride, slot, m.n, m.n_pad, planes, args,
                              self._clip)
            if cb is not None:
                size = cb.grad.numel()
                B.gs_adam_clipped(cb.table, cb.m, cb.v, cb.grad, size, None, size, size, 1, args,
                                  self._clip)
        if cb is not None:
            cb.decode(m, self.dev_status)

    # ------------------------------------------------------------------
    def run_view(self, cam, target, leaves=None, hooks=None, update=True, backward=True,
                 timing=None, counters=None, region=None, grad_out=None,
                 gate=None, plan_only=False) -> ViewStats:
        """One view.  target: [3][H][W] fp32, a device tensor (the whole view
        resident, read in place) or a pinned host tensor (each Leaf's crop is
        uploaded before its forward); None renders only (no loss, backward or
        update).  leaves: tile rects overriding the planner.  timing: dict
        that receives (start, end) CUDA event pairs per stage (STAGES).
        counters: device int64[6] work counters ([0:4] forward, [4:6]
        backward).  region: tile rect (x0, y0, x1, y1) the step is restricted
        to (its Gaussians projected, its Leaves planned; default the whole
        grid).  grad_out: dense [P][n_pad] gradient the view's gradient is
        added to instead of taking the Adam step.  gate: callable(loss) ->
        bool asked with the view's forward loss (skipgs.BackwardGate); False
        skips the backward and the update.  plan_only: project and plan the
        Leaves, size later arenas by them, and return None (`reserve`)."""
        dev = self.device
        if target is None:
            backward = update = False
        clk = _Timer(timing)
        cnt_f = counters[0:4] if counters is not None else None
        cnt_b = counters[4:6] if counters is not None else None
        m = self.model
        W, H = cam.width, cam.height
        TW, TH = (W + 15) // 16, (H + 15) // 16
        T = TW * TH
        tile_bits = max(1, math.ceil(math.log2(T))) if T > 1 else 1
        camS = B.camera_struct(cam)
        mod = m.struct()
        st = self.dev_status
        base_alloc = torch.cuda.memory_allocated(dev)
        torch.cuda.reset_peak_memory_stats(dev)
        launch0 = B.gs_launch_counter()

        # ---- projection (+ counts, SAT) ---------------------------------
        # Candidate state is sized for the candidates, not the model: from
        # the last count of this region plus 5 %; a view with more candidates
        # than that is projected again with the exact count.
        n = m.n
        original = self.mode == "original"
        pflags = B.GS_PROJ_DENSE if original else 0
        hint_key = tuple(region) if region is not None else None
        hint = self._cap_hint.get(hint_key)
        cap = max(n, 1) if (original or hint is None) else max(min(n, hint), 1)
        slot = torch.empty(max(n, 1), dtype=torch.int32, device=dev)
        sat = torch.empty((TH + 1) * (TW + 1), dtype=torch.int64, device=dev)
        ws = torch.empty(B.gs_project_workspace_size(n, W, H), dtype=torch.uint8, device=dev)
        tk = clk.tic("project")
        # fused: per-block lists, each tile's list built inside the forward;
        # expand: per-block lists expanded into full tile lists per Leaf;
        # sort: per-Leaf (tile, candidate) entries sorted by tile
        fused = self.binning == "fused"
        expand = self.binning in ("expand", "fused")
        if expand:
            BW, BH = (TW + B.TILE_BLOCK - 1) // B.TILE_BLOCK, (TH + B.TILE_BLOCK - 1) // B.TILE_BLOCK
            bsat = torch.empty((BH + 1) * (BW + 1), dtype=torch.int64, device=dev)
            bws = torch.empty(B.gs_block_sat_workspace_size(TW, TH), dtype=torch.uint8, device=dev)
            bsat_h = torch.empty(bsat.shape, dtype=torch.int64, pin_memory=True)
        sat_h = torch.empty(sat.shape, dtype=torch.int64, pin_memory=True)
        nc_h = torch.empty(1, dtype=torch.int32, pin_memory=True)
        sq_h = torch.empty(1, dtype=torch.int64, pin_memory=True)
        while True:
            n_cand_d = torch.empty(1, dtype=torch.int32, device=dev)   # written by gs_project
            cand_idx = torch.empty(cap, dtype=torch.int32, device=dev)
            rec = torch.empty(cap * 12, dtype=torch.float32, device=dev)
            rect = torch.empty(cap * 4, dtype=torch.int16, device=dev)
            dkey = torch.empty(cap, dtype=torch.int32, device=dev)
            sq_d = torch.empty(1, dtype=torch.int64, device=dev)       # cleared by gs_project
            proj = B.gs_proj(cap, n_cand_d.data_ptr(), cand_idx.data_ptr(), slot.data_ptr(),
                             rec.data_ptr(), rect.data_ptr(), dkey.data_ptr(), sq_d.data_ptr())
            if region is None:
                B.gs_project(mod, camS, proj, sat, ws, st, flags=pflags)
            else:
                B.gs_project_region(mod, camS, region, proj, sat, ws, st, flags=pflags)
            if expand:
                B.gs_block_sat(proj, TW, TH, bsat, bws, st)
                bsat_h.copy_(bsat, non_blocking=True)
            sat_h.copy_(sat, non_blocking=True)
            nc_h.copy_(n_cand_d, non_blocking=True)
            sq_h.copy_(sq_d, non_blocking=True)
            clk.toc(tk)
            tables_ready = torch.cuda.Event()
            tables_ready.record()
            # what needs no host decision is issued before the host waits, so
            # the GPU works while the host reads the tables and plans: the
            # compact 2D gradient, zeroed on a side stream (the raster
            # backward, its first user, waits for it), and the depth presort
            # on the candidate count the projection left on the device.  Both
            # are sized by the capacity; without a capacity hint (a region's
            # first view, whose capacity is every Gaussian) they wait for the
            # count instead, so that they are sized by it.
            early = hint is not None or original
            g2d = g2d_ready = order = drect = None
            if early:
                if not plan_only:
                    g2d, g2d_ready = self._zeroed_g2d(cap)
                order, drect = self._depth_order(proj, B.GS_COUNT_ON_DEVICE, cap, clk)
            tables_ready.synchronize()   # the one host wait per view
            if int(nc_h[0]) <= cap:
                break
            # more candidates than the capacity hint: the kernel skipped (and
            # flagged) those beyond it; clear the flag and project again
            B.gs_check(st)
            cap = int(nc_h[0])
            tk = clk.tic("project")
        del ws
        if expand:
            del bws
        C = int(nc_h[0])
        if not early:
            if not plan_only:
                g2d, g2d_ready = self._zeroed_g2d(max(C, 1))
            order, drect = self._depth_order(proj, C, max(C, 1), clk)
        if not original:
            self._cap_hint[hint_key] = C + C // 20 + 1024
        n_square = int(sq_h[0])
        sat_np = sat_h.numpy().reshape(TH + 1, TW + 1)
        ctx = dict(proj=proj, cand_idx=cand_idx, slot=slot, rec=rec, rect=rect, depth_key=dkey,
                   sat=sat, sat_host=sat_np, n_cand=C, TW=TW, TH=TH, cam=cam)
        if hooks is not None and hasattr(hooks, "on_project"):
            hooks.on_project(ctx)
        if not plan_only:
            calls, self._after_tables = self._after_tables, []
            for f in calls:
                f()

        ctx["depth_order"] = order
        ctx["depth_rect"] = drect

        # ---- per-block candidate lists (two-level binning) ------------------
        if expand:
            bsat_np = bsat_h.numpy().reshape(BH + 1, BW + 1)
            n_blk = int(bsat_np[BH, BW])
            bvals = torch.empty(max(n_blk, 1), dtype=torch.int32, device=dev)
            branges = torch.empty(2 * BW * BH, dtype=torch.int64, device=dev)
            ws = torch.empty(max(B.gs_bin_blocks_workspace_size(C, n_blk, TW, TH), 256),
                             dtype=torch.uint8, device=dev)
            tk = clk.tic("bin")
            B.gs_bin_blocks(proj, C, order, drect, TW, TH, bsat, n_blk, bvals, max(n_blk, 1),
                            branges, ws, st)
            clk.toc(tk)
            del ws
            ctx.update(block_sat=bsat, block_sat_host=bsat_np, block_vals=bvals,
                       block_ranges=branges, n_block_entries=n_blk)

        # ---- Leaf plan ------------------------------------------------------
        ssim = self.loss == "l1_ssim" and (target is not None or plan_only)
        lm = B.gs_leaf_load_model(tile_bits, (B.GS_BIN_EXPAND if expand else B.GS_BIN_SORT) |
                                  (B.GS_LOAD_SSIM if ssim else 0))
        if leaves is None and original:
            leaves = [tuple(region) if region is not None else (0, 0, TW, TH)]
        if leaves is None and region is not None:
            # plan inside the region: its own SAT (zero first row and column)
            rx0, ry0, rx1, ry1 = (int(v) for v in region)
            sub = (sat_np[ry0:ry1 + 1, rx0:rx1 + 1] - sat_np[ry0:ry1 + 1, rx0:rx0 + 1]
                   - sat_np[ry0:ry0 + 1, rx0:rx1 + 1] + sat_np[ry0, rx0])
            rw = min(16 * rx1, W) - 16 * rx0
            rh = min(16 * ry1, H) - 16 * ry0
            _, lv, li, lb, ov = B.gs_leaf_partition(sub, rx1 - rx0, ry1 - ry0, rw, rh, lm,
                                                    self.budget)
            lv = lv + np.array([rx0, ry0, rx0, ry0], np.int32)
        elif leaves is None:
            _, lv, li, lb, ov = B.gs_leaf_partition(sat_np, TW, TH, W, H, lm, self.budget)
        else:
            lv = np.asarray(leaves, np.int32).reshape(-1, 4)
            li = np.array([sat_np[y1, x1] - sat_np[y0, x1] - sat_np[y1, x0] + sat_np[y0, x0]
                           for x0, y0, x1, y1 in lv], np.int64)
            lb = np.zeros(len(lv), np.int64)
            ov = np.zeros(len(lv), bool)

        # ---- per-Leaf raster: forward + L1 + backward into compact g2d ------
        # every tile's loss partial is written by its Leaf's forward when the
        # planned Leaves cover the grid; a region or caller-given Leaves may
        # leave tiles out, which must then count zero
        zero_tiles = region is not None or leaves is not None
        loss_tiles = (torch.zeros if zero_tiles else torch.empty)(T, dtype=torch.float32,
                                                                    device=dev)
        if fused:
            bin_ws = torch.empty(256, dtype=torch.uint8, device=dev)
        elif expand:
            bin_ws = torch.empty(max(max((B.gs_expand_workspace_size(L, B.block_entries(bsat_np, L))
                                          for L in lv), default=0), 256),
                                 dtype=torch.uint8, device=dev)
        else:
            bin_ws = torch.empty(max(B.gs_bin_workspace_size(C), 256), dtype=torch.uint8,
                                 device=dev)
        resident_target = target is not None and target.is_cuda

        def leaf_sizes(L, I):
            x0, y0, x1, y1 = (int(v) for v in L)
            pw = min(16 * x1, W) - 16 * x0
            ph = min(16 * y1, H) - 16 * y0
            npx = pw * ph
            nt = (x1 - x0) * (y1 - y0)
            if expand:
                sizes = [0, 4 * I, 16 * nt, 0, 12 * npx, 4 * npx, 4 * npx, 12 * npx]
            else:
                lb_bits = B.local_tile_bits(L)
                sizes = [4 * I, 4 * I, 16 * nt, B.gs_sort_workspace_size(I, 4, 0, lb_bits),
                         12 * npx, 4 * npx, 4 * npx, 12 * npx]
            sizes.append(36 * npx if ssim else 0)  # the SSIM term's partials
            return sizes, (16 * x0, 16 * y0, pw, ph)

        arena_bytes = max((_carved_bytes(leaf_sizes(L, int(I))[0]) for L, I in zip(lv, li)),
                          default=0)
        # a bounded run's arenas keep 1/16 headroom over the largest Leaf seen
        # (up to the Leaf budget; more only for an over-budget Leaf), so that
        # later views reuse the same cached blocks: an arena sized to each
        # view's largest Leaf needs a new device allocation (a host stall of
        # up to tens of milliseconds) on the first view whose largest Leaf
        # beats every earlier one.  `reserve` plans a set of views up front.
        if not original:
            self._arena_hint = max(self._arena_hint,
                                   min(self.budget, arena_bytes + arena_bytes // 16))
        if plan_only:
            return None
        alloc_bytes = arena_bytes if original else max(arena_bytes, self._arena_hint)
        arena = torch.empty(max(alloc_bytes, 256), dtype=torch.uint8, device=dev)
        n_ls = 1 if original else max(1, min(self.leaf_streams, len(lv)))
        main = torch.cuda.current_stream(dev)
        arenas, lstreams = [arena], [main]
        bin_wss = [bin_ws]
        while len(self._side_streams) < n_ls - 1:
            self._side_streams.append(torch.cuda.Stream(device=dev))
        for k in range(n_ls - 1):
            arenas.append(torch.empty(max(alloc_bytes, 256), dtype=torch.uint8, device=dev))
            bin_wss.append(torch.empty_like(bin_ws))  # the list builders' scratch, per stream
            lstreams.append(self._side_streams[k])
        norm = 1.0 / (3.0 * W * H)
        # with the SSIM term the forward's L1 part carries (1 - lambda)
        norm_l1 = (1.0 - self.ssim_lambda) * norm if ssim else norm
        # bounded supply of a host target: each Leaf's crop is uploaded on a
        # copy stream into one of two buffers, Leaf k + 2's upload waiting
        # until Leaf k's forward (the only reader) is done
        host_target = target is not None and not resident_target
        if host_target:
            rects = [leaf_sizes(L, 0)[1] for L in lv]
            crop_n = max((3 * w * h for _, _, w, h in rects), default=1)
            crops = [torch.empty(max(crop_n, 1), dtype=torch.float32, device=dev) for _ in range(2)]
            if self._copy_stream is None:
                self._copy_stream = torch.cuda.Stream(device=dev)
            cs = self._copy_stream

        hstate = {}  # the host target's upload state, shared by leaf_pass and leaf_one

        main.wait_event(g2d_ready)

        def leaf_pass(with_bwd):
            """Every Leaf: lists, forward (+ L1) and, if with_bwd, backward."""
            for side in lstreams[1:]:
                side.wait_stream(main)  # g2d, lists and tables are ready
            if host_target:
                up = [torch.cuda.Event() for _ in lv]
                freed = [None, None]

                def upload(k):
                    x_, y_, w_, h_ = rects[k]
                    if freed[k % 2] is not None:
                        cs.wait_event(freed[k % 2])
                    else:
                        cs.wait_stream(main)  # the buffers were allocated on the main stream
                    B.gs_upload_crop(target, x_, y_, w_, h_, crops[k % 2], stream=cs)
                    up[k].record(cs)

                for k in range(min(2, len(lv))):
                    upload(k)
                hstate.update(up=up, freed=freed, upload=upload)
            for li_k, (L, I) in enumerate(zip(lv, li)):
                with torch.cuda.stream(lstreams[li_k % len(lstreams)]):
                    leaf_one(li_k, L, I, with_bwd)
            for side in lstreams[1:]:
                main.wait_stream(side)

        def leaf_one(li_k, L, I, with_bwd):
            """One Leaf on the current stream, with its arena."""
            ls = torch.cuda.current_stream(dev)
            up, freed, upload = hstate.get("up"), hstate.get("freed"), hstate.get("upload")
            I = int(I)
            sizes, (px0, py0, pw, ph) = leaf_sizes(L, I)
            bufs, _ = _carve(arenas[li_k % len(arenas)], sizes)
            lws = bin_wss[li_k % len(bin_wss)]
            keys = bufs[0].view(torch.int32)
            vals = bufs[1].view(torch.int32)
            ranges = bufs[2].view(torch.int64)
            sort_ws = bufs[3]
            img = bufs[4].view(torch.float32)
            Tf = bufs[5].view(torch.float32)
            last = bufs[6].view(torch.int32)
            dL = bufs[7].view(torch.float32)
            if resident_target:
                # the whole view's target is read in place with its own pitch
                px = B.pixels(px0, py0, pw, ph, img, Tf, last, dL, target=target,
                              target_origin=(0, 0), target_pitch=W, target_plane=W * H,
                              loss_tiles=loss_tiles, norm=norm_l1, counters=cnt_f)
            elif host_target:
                crop = crops[li_k % 2][:3 * pw * ph].view(3, ph, pw)
                ls.wait_event(up[li_k])
                px = B.pixels(px0, py0, pw, ph, img, Tf, last, dL, target=crop,
                              target_origin=(px0, py0), loss_tiles=loss_tiles,
                              norm=norm_l1, counters=cnt_f)
            else:
                px = B.pixels(px0, py0, pw, ph, img, Tf, last, dL, counters=cnt_f)
            if fused:
                B.gs_tile_ranges(sat, TW, TH, L, ranges)
            elif expand:
                tk = clk.tic("expand")
                B.gs_expand_tiles(proj, bvals, branges, B.block_entries(bsat_np, L), L, TW, TH,
                                  sat, I, vals, max(I, 1), ranges, lws, st)
                clk.toc(tk)
            else:
                tk = clk.tic("bin")
                B.gs_bin_tiles(proj, C, order, drect, L, TW, TH, sat, I, keys, vals, max(I, 1),
                               ranges, lws, st)
                clk.toc(tk)
            lb_bits = B.local_tile_bits(L)
            if not expand and I > 0 and lb_bits > 0:
                tk = clk.tic("sort_tiles")
                B.gs_sort_tiles(keys, vals, I, ranges, (L[2] - L[0]) * (L[3] - L[1]), sort_ws, st)
                clk.toc(tk)
            tk = clk.tic("raster_fwd")
            if fused:
                B.gs_raster_fwd_blocks(proj, bvals, branges, L, camS, px, vals, max(I, 1), I,
                                       ranges, st, self.raster_flags)
            else:
                B.gs_raster_fwd(proj, vals, ranges, L, camS, px, st, self.raster_flags)
            clk.toc(tk)
            if ssim:
                # the Leaf's SSIM term: loss, and with the backward its
                # gradient added to the L1 part of dL
                tk = clk.tic("ssim")
                B.gs_loss_ssim(px, L, camS, self.ssim_lambda * norm,
                               bufs[8] if with_bwd else None)
                clk.toc(tk)
            if host_target:
                ev = torch.cuda.Event()
                ev.record(ls)
                freed[li_k % 2] = ev
                if li_k + 2 < len(lv):
                    upload(li_k + 2)
            if hooks is not None and hasattr(hooks, "on_leaf"):
                hooks.on_leaf(ctx, dict(leaf=tuple(int(v) for v in L), keys=keys, vals=vals,
                                        ranges=ranges, img=img, T_final=Tf, last=last, dL=dL,
                                        n_isect=I, px_rect=(px0, py0, pw, ph)))
            if with_bwd:
                if cnt_b is not None:
                    px.counters = cnt_b.data_ptr()
                tk = clk.tic("raster_bwd")
                B.gs_raster_bwd(proj, vals, ranges, L, camS, px, g2d, st, self.raster_flags)
                clk.toc(tk)

        # SkipGS gate: the view's loss from a forward pass decides whether the
        # backward and the update run (then the Leaves are rendered again
        # with their backward; the projection and lists are reused)
        if gate is not None and backward:
            leaf_pass(False)
            pre = torch.empty(1, dtype=torch.float64, device=dev)  # written by gs_loss_total
            B.gs_loss_total(loss_tiles, T, pre)
            if gate(float(pre.item())):
                if zero_tiles:
                    loss_tiles.zero_()
                leaf_pass(True)
            else:
                backward = update = False
        else:
            leaf_pass(backward)
        if not original:
            # raster buffers released before projection backward (the main
            # stream has waited for the Leaf stream, so the memory is free)
            arenas.clear()
            bin_wss.clear()
            del arena, bin_ws
            if host_target:
                del crops

        loss_d = torch.zeros(1, dtype=torch.float64, device=dev) if target is None else \
            torch.empty(1, dtype=torch.float64, device=dev)
        if target is not None:
            B.gs_loss_total(loss_tiles, T, loss_d)
        self._last_loss = loss_d
        ctx["g2d"] = g2d
        if hooks is not None and hasattr(hooks, "on_bwd"):
            hooks.on_bwd(ctx)

        # ---- projection backward fused with ONE Adam update -----------------
        if update and grad_out is not None:
            # the view's gradient goes to the caller's dense sum
            g3d = torch.empty(m.P * max(C, 1), dtype=torch.float32, device=dev)
            tk = clk.tic("project_bwd")
            B.gs_project_bwd(mod, camS, proj, C, g2d, g3d=g3d, g3d_stride=max(C, 1),
                             dev_status=st)
            B.gs_grad_accumulate(g3d, max(C, 1), cand_idx, C, m.P, grad_out, m.n_pad)
            clk.toc(tk)
            del g3d
        elif update and (self.max_grad_norm is not None or self.codebook is not None):
            g3d = torch.empty(m.P * max(C, 1), dtype=torch.float32, device=dev)
            tk = clk.tic("project_bwd")
            B.gs_project_bwd(mod, camS, proj, C, g2d, g3d=g3d, g3d_stride=max(C, 1),
                             dev_status=st)
            self._update(g3d, max(C, 1), slot, C, cand_idx[:C])
            clk.toc(tk)
            del g3d
        elif update:
            m.step += 1
            if self.fuse_adam and not original:
                # default: a separate geometric chain pass into a 14-float
                # scratch per candidate, then the Adam stream (faster);
                # "in_stream": the chain inside the stream, no scratch
                # (56 bytes per candidate less working set, ~3% slower)
                two = self.fuse_adam != "in_stream"
                geo = torch.empty(14 * max(C, 1), dtype=torch.float32, device=dev) if two else None
                tk = clk.tic("project_bwd")
                B.gs_project_bwd(mod, camS, proj, C, g2d, g3d=geo,
                                 g3d_stride=geo.numel() if two else 0,
                                 adam_m=m.m, adam_v=m.v, fused=self.adam_args(m.step),
                                 dev_status=st)
                clk.toc(tk)
                del geo
            else:
                g3d = torch.empty(m.P * max(C, 1), dtype=torch.float32, device=dev)
                tk = clk.tic("project_bwd")
                B.gs_project_bwd(mod, camS, proj, C, g2d, g3d=g3d, g3d_stride=max(C, 1),
                                 dev_status=st)
                B.gs_adam(m.params, m.m, m.v, g3d, max(C, 1), slot, m.n, m.n_pad, m.P,
                          self.adam_args(m.step))
                clk.toc(tk)
                del g3d
        peak = torch.cuda.max_memory_allocated(dev) - base_alloc
        if resident_target:
            peak += target.numel() * target.element_size()
        return ViewStats(n_cand=C, n_isect=int(li.sum()), n_isect_square=n_square,
                         n_block_entries=n_blk if expand else 0,
                         n_block_reads=sum(B.block_entries(bsat_np, L) for L in lv) if expand else 0,
                         n_leaves=len(lv), leaves=lv,
                         leaf_isect=li, leaf_bytes=lb, over_budget=ov, peak_ws_bytes=int(peak),
                         arena_bytes=int(arena_bytes),
                         launches=B.gs_launch_counter() - launch0)

    @staticmethod
    def split_regions(TW, TH, gx, gy):
        """gx x gy tile-aligned regions covering the grid, row by row."""
        xs = [round(k * TW / gx) for k in range(gx + 1)]
        ys = [round(k * TH / gy) for k in range(gy + 1)]
        return [(xs[i], ys[j], xs[i + 1], ys[j + 1]) for j in range(gy) for i in range(gx)
                if xs[i + 1] > xs[i] and ys[j + 1] > ys[j]]

    def run_view_grouped(self, cam, target, groups=(3, 3), timing=None, hooks=None):
        """One view in gx x gy groups (BoundedGS page, section 02, "finer
        grouping", ablation F): each group projects only the Gaussians that
        can touch it and plans its own Leaves; their gradients are summed into
        one dense gradient (kept, like the Adam moments, for the model's
        lifetime), then ONE Adam update.  Same image, loss and update as
        run_view (the sums reorder)."""
        m = self.model
        TW, TH = (cam.width + 15) // 16, (cam.height + 15) // 16
        if getattr(self, "_G", None) is None or self._G.shape != m.params.shape:
            self._G = torch.zeros_like(m.params)
        else:
            self._G.zero_()
        stats, loss = [], None
        for r in self.split_regions(TW, TH, *groups):
            st = self.run_view(cam, target, region=r, grad_out=self._G, timing=timing,
                               hooks=hooks)
            stats.append(st)
            loss = self._last_loss if loss is None else loss + self._last_loss
        base_alloc = torch.cuda.memory_allocated(self.device)
        torch.cuda.reset_peak_memory_stats(self.device)
        tk = _Timer(timing).tic("project_bwd")
        self._update(self._G, m.n_pad, None, m.n, None)
        _Timer(timing).toc(tk)
        peak = torch.cuda.max_memory_allocated(self.device) - base_alloc
        if target is not None and target.is_cuda:
            peak += target.numel() * target.element_size()
        self._last_loss = loss
        merged = _merge_stats(stats)
        # a codebook's workspace for the whole model's gradient
        merged.peak_ws_bytes = max(merged.peak_ws_bytes, int(peak))
        return merged

    def run_view_blocks(self, cam, target, blocks=(8, 8), timing=None, hooks=None):
        """The fixed-block schedule of the BoundedGS page (Figs. 5-6): the
        view cut into a fixed bx x by grid, each block a step of its own with
        its own Adam update.  Returns the merged statistics; the loss is the
        sum of the blocks' losses.  A codebook is decoded into the whole model
        after each block's update, as the next block may need any Gaussian
        (0.25 ms a block at 6M Gaussians)."""
        TW, TH = (cam.width + 15) // 16, (cam.height + 15) // 16
        stats, loss = [], None
        for r in self.split_regions(TW, TH, *blocks):
            st = self.run_view(cam, target, region=r, timing=timing, hooks=hooks)
            stats.append(st)
            loss = self._last_loss if loss is None else loss + self._last_loss
        self._last_loss = loss
        return _merge_stats(stats)

    def render(self, cam) -> torch.Tensor:
        """Forward-only render of the whole view: [3][H][W] fp32 on the device."""
        img = torch.zeros((3, cam.height, cam.width), dtype=torch.float32, device=self.device)

        class _Copy:
            def on_leaf(self, ctx, lc):
                x0, y0, w, h = lc["px_rect"]
                img[:, y0:y0 + h, x0:x0 + w] = lc["img"][:3 * w * h].view(3, h, w)

        self.run_view(cam, None, hooks=_Copy())
        return img
