"""One optimizer step of the LoGRA path over many matrices, scheduled over
several HIP streams.

The sketched set is every attention and MLP projection of a model ("NVIDIA's
LoGRA fits RL post-training of a 27B model onto a single eight-GPU node",
section "Why it matters"), so a step is many independent matrices, most of
them too small to fill the chip alone. This module only schedules the C-ABI
calls: it holds no arithmetic of the method, and every number is produced by
the library's kernels.

A step, in the order the host drives it:
  1. sketch: for every microbatch (in order, as a backward pass produces
     them) and every matrix, logra_sketch_project then the fold: for a
     matrix that keeps its sketch in parts during the step (the `parts`
     policy), logra_sketch_fold_parts with LOGRA_FOLD_FIRST on the first
     microbatch and LOGRA_FOLD_LAST on the last, so that the workgroups
     sharing a tile of S never wait for each other; otherwise
     logra_sketch_fold (accumulate = 0 for the first microbatch). Matrix i
     runs on sketch lane i mod n_sketch; each lane is a stream with its own
     workspace. An expert group (one projection of every expert of a layer)
     is one call per microbatch, logra_sketch_experts, on a lane of its own
     turn; its experts are matrices like the others from there on.
  2. clipping, if the caller asks for it (`clip`): the global norm over every
     sketch and the caller's dense gradients, and all of them scaled in place
     (logra_grad_clip).
  3. pass 1: logra_update_sqnorm for every matrix (v -> v'), in batches of
     up to 16 matrices per apply lane (logra_update_sqnorm_batch: two
     launches per batch), matrix i on apply lane i mod n_apply.
  4. one device-to-host read of every sqnorm (the host step controller's
     input).
  5. pass 2: logra_rowadam_apply for every matrix given a scale; a matrix
     that is given none (or whose sqnorm is not finite, when the caller asks
     to skip those) keeps W and v. Each applied matrix then swaps v and v'.
  6. the dense parameters that are not sketched (embeddings, norm gains, router
     weights), if the step was given any: one AdamW step over all of them
     (`dense_update`, logra_adamw), at any time after clipping.
Every lane forks from the caller's current stream at the start of a phase
and joins it at the end, so the caller can time phases with events on its
own stream. Callbacks that make the sketch's inputs when they are called run on
a stream of their own, so that a lane which waits for what they enqueue waits
for no other lane (the caller's stream is itself a lane). The calls carry launch options that declare the lane counts to
the kernels (the projection and pass 2 size their grids for a 1/n share of
the chip) and a device counter of fold time-outs.
"""
from __future__ import annotations

import contextlib
import dataclasses
import math
from typing import Callable, Dict, List, Optional, Sequence, Tuple

import torch

from . import binding as B
from . import hip_timing

MAX_SKETCH_LANES = 4   # HIP gives a process four hardware queues by default
DEFAULT_APPLY_LANES = 3


@dataclasses.dataclass
class Matrix:
    """One sketched projection W (d x k). W and v are the caller's state
    (updated in place by the step: W by pass 2, v by the swap with v')."""
    d: int
    k: int
    matrix_id: int
    W: torch.Tensor
    v: torch.Tensor
    name: str = ""
    # allocated by Step
    S: Optional[torch.Tensor] = None
    v_new: Optional[torch.Tensor] = None
    sq: Optional[torch.Tensor] = None
    rowsq: Optional[torch.Tensor] = None
    desc: Optional[B.MatrixDesc] = None
    parts: Optional[torch.Tensor] = None
    lane: int = 0
    alane: int = 0


@dataclasses.dataclass
class ExpertGroup:
    """One projection of every expert of a layer: expert e's W[e] is d x k and
    its matrix id matrix_id + e (matrices of one id share their signs, so give
    every group its own n_experts ids). W (experts x d x k) and v (experts x d) are
    the caller's state: W is updated in place, v is read by the first pass
    that needs it, then members[e].v is expert e's (as for a Matrix, and for
    every step that the group is given to). members[e].W and .S are W[e] and
    S[e]. Another tensor, or other memory, in the place of W, v or S is what
    the next phase uses. topk choices of an expert per token make tokens topk
    rows of dY per microbatch."""
    n_experts: int
    d: int
    k: int
    matrix_id: int
    topk: int
    W: torch.Tensor
    v: torch.Tensor
    name: str = ""
    # allocated by Step
    S: Optional[torch.Tensor] = None
    ws: Optional[torch.Tensor] = None
    members: Optional[List[Matrix]] = None
    lane: int = 0
    # what the members' W, v and S were last taken from, and its address
    taken: Dict[str, Tuple[torch.Tensor, int]] = dataclasses.field(default_factory=dict, repr=False)

    def bind(self, r: int):
        """The members, and what they hold taken from the group's W, v and S
        where that is not what it was."""
        if self.members is None:
            self.members = [Matrix(self.d, self.k, self.matrix_id + e, None, None, "%s.%d" % (self.name, e))
                            for e in range(self.n_experts)]
        shapes = {"W": (self.n_experts, self.d, self.k), "v": (self.n_experts, self.d), "S": (self.n_experts, self.d, r)}
        for what, shape in shapes.items():
            t = getattr(self, what)
            if t is None:
                continue
            had, at = self.taken.get(what, (None, 0))
            if had is t and at == t.data_ptr() and tuple(t.shape) == shape:
                if what == "S" and any(m.S.data_ptr() != at + 4 * e * self.d * r for e, m in enumerate(self.members)):
                    raise ValueError("expert group %s: its members' S are views of the group's" % self.name)
                continue
            if tuple(t.shape) != shape:
                raise ValueError("expert group %s: W experts x d x k, v experts x d and S experts x d x r expected"
                                 % self.name)
            if what == "S" and (t.dtype is not torch.float32 or not t.is_contiguous() or t.device != self.W.device):
                raise ValueError("expert group %s: contiguous float32 S expected" % self.name)
            for m, x in zip(self.members, t):
                setattr(m, what, x)
            self.taken[what] = (t, t.data_ptr())


def _event(stream):
    # timing only: no system-scope fence, which would add its cost to the
    # probed kernel's time and to the step
    return hip_timing.record(stream)


class Step:
    """Streams, workspaces and per-phase calls for a fixed set of matrices.

    matrices  the Matrix records (W, v on the device).
    groups    the ExpertGroup records; their experts follow the matrices in
              `mats`, group by group (sqnorms, scales).
    grads     dense gradients that `clip` takes along with the sketches
              (device tensors written in place every step).
    adamw     the B.AdamWList of the dense parameters that `dense_update` takes
              a step with; `clip` takes its gradients along too.
    r, tokens the sketch rank and the tokens of every microbatch.
    act_dtype B.LOGRA_BF16 or B.LOGRA_F32 (X, dY and the compute dtype).
    sketch_lanes / apply_lanes  stream counts (0: min(4, n) for the sketch;
              1 for a single matrix, else 3, for the apply).
    batch_pass1  pass 1 in batches of up to 16 matrices per apply lane.
    seed      the library seed of the sign matrices.
    rowsq     also keep every matrix's per-row sums of squares from pass 1
              (Matrix.rowsq), for callers that inspect them.
    parts     which matrices hold their sketch in parts during the step:
              "pair" (those whose fold tiles are shared by two workgroups:
              one extra d x r array each), "all" (every matrix whose fold
              splits its tiles: up to 31 arrays for small d), or "none".
    """

    def __init__(self, matrices: Sequence[Matrix], r: int, tokens: int, act_dtype: int,
                 device=None, sketch_lanes: int = 0, apply_lanes: int = 0,
                 batch_pass1: bool = True, seed: int = 0, rowsq: bool = False, parts: str = "pair",
                 groups: Sequence[ExpertGroup] = (), grads: Sequence[torch.Tensor] = (),
                 adamw: Optional[B.AdamWList] = None):
        if not matrices and not groups:
            raise ValueError("a step needs at least one matrix")
        self.dense: List[Matrix] = list(matrices)
        self.groups: List[ExpertGroup] = list(groups)
        self.grads = list(grads)
        self.adamw = adamw
        if adamw is not None:
            self.grads += [g for g in adamw.grads if not any(g is x for x in self.grads)]
        self._clipped = False       # whether the host called `clip` since the last `sketch`
        self._clip_captured = False     # whether a graph may write `norm` without the host's knowing
        self.mats: List[Matrix] = list(matrices)
        for g in self.groups:
            g.S = None
            g.bind(int(r))
            self.mats.extend(g.members)
        self.r, self.tokens, self.code, self.seed = int(r), int(tokens), int(act_dtype), int(seed)
        dev = torch.device(device) if device is not None else self.mats[0].W.device
        self.device = dev
        n = len(self.mats)
        n_calls = len(self.dense) + len(self.groups)
        self.n_sketch = max(1, min(sketch_lanes or min(MAX_SKETCH_LANES, n_calls), n_calls))
        self.n_apply = max(1, min(apply_lanes or (1 if n == 1 else DEFAULT_APPLY_LANES), n))
        self.timeouts = torch.zeros(1, dtype=torch.int32, device=dev)
        self.sketch_opts = B.LaunchOpts(sketch_concurrency=self.n_sketch, fold_timeouts=self.timeouts)
        self.apply_opts = B.LaunchOpts(apply_concurrency=self.n_apply)
        ws_bytes = max([0] + [B.logra_sketch_workspace_bytes(B.MatrixDesc(m.d, m.k, r), tokens, act_dtype)
                              for m in self.dense])
        sq_ws_bytes = max(B.logra_sqnorm_workspace_bytes(B.MatrixDesc(m.d, m.k, r), act_dtype)
                          for m in self.mats)
        self.main = torch.cuda.current_stream(dev)
        n_lanes = max(self.n_sketch, self.n_apply)
        self.lanes = []
        for i in range(n_lanes):
            self.lanes.append({
                "stream": self.main if i == 0 else torch.cuda.Stream(device=dev),
                "ws": torch.empty(max(16, ws_bytes), dtype=torch.uint8, device=dev),
                "sq_ws": torch.empty(max(16, sq_ws_bytes), dtype=torch.uint8, device=dev),
            })
        self.callbacks = None       # the callbacks' stream, made when first needed
        if parts not in ("pair", "all", "none"):
            raise ValueError("parts must be 'pair', 'all' or 'none'")
        self.parts_bytes = 0
        self.expert_ws_bytes = 0
        for i, g in enumerate(self.groups):
            g.lane = (len(self.dense) + i) % self.n_sketch
            g.S = torch.empty(g.n_experts, g.d, r, dtype=torch.float32, device=dev)
            nb = max(16, B.logra_sketch_experts_workspace_bytes(B.MatrixDesc(g.d, g.k, r), g.n_experts,
                                                                tokens * g.topk, act_dtype))
            g.ws = torch.empty(nb, dtype=torch.uint8, device=dev)
            self.expert_ws_bytes += nb
            g.bind(int(r))
        for i, m in enumerate(self.mats):
            if m.S is None or i < len(self.dense):
                m.S = torch.empty(m.d, r, dtype=torch.float32, device=dev)
            pb = 0 if i >= len(self.dense) else B.logra_sketch_parts_bytes(B.MatrixDesc(m.d, m.k, r), tokens, act_dtype)
            use = pb > 0 and (parts == "all" or (parts == "pair" and pb == 4 * m.d * r))
            m.parts = torch.empty(pb // 4, dtype=torch.float32, device=dev) if use else None
            self.parts_bytes += pb if use else 0
            m.v_new = torch.empty(m.d, dtype=torch.float32, device=dev)
            m.sq = torch.empty(1, dtype=torch.float32, device=dev)
            m.rowsq = torch.empty(m.d, dtype=torch.float32, device=dev) if rowsq else None
            m.lane = i % self.n_sketch
            m.alane = i % self.n_apply
        # Pass-1 batches: each apply lane's matrices in as few chunks of at
        # most MAX_BATCH as hold them, of equal size (65 matrices: 5 x 13,
        # not 4 x 16 + 1); a chunk of one matrix uses the single-matrix call.
        # A batched matrix's sqnorm is a view of its chunk's output.
        self.batches = []
        self.batch_ws_bytes = 0
        for li in range(self.n_apply):
            own = [m for m in self.mats if m.alane == li]
            if not batch_pass1:
                self.batches.extend((li, [m], None, None) for m in own)
                continue
            n_chunks = -(-len(own) // B.MAX_BATCH)
            bounds = [len(own) * c // max(1, n_chunks) for c in range(n_chunks + 1)]
            for c0, c1 in zip(bounds[:-1], bounds[1:]):
                chunk = own[c0:c1]
                if len(chunk) == 1:
                    self.batches.append((li, chunk, None, None))
                    continue
                sq = torch.empty(len(chunk), dtype=torch.float32, device=dev)
                for j, m in enumerate(chunk):
                    m.sq = sq[j:j + 1]
                wsb = B.logra_sqnorm_batch_workspace_bytes([B.MatrixDesc(m.d, m.k, r) for m in chunk],
                                                           act_dtype)
                self.batch_ws_bytes += wsb
                self.batches.append((li, chunk, sq, torch.empty(max(16, wsb), dtype=torch.uint8, device=dev)))
        self.workspace_bytes = (n_lanes * (max(16, ws_bytes) + max(16, sq_ws_bytes)) + self.batch_ws_bytes
                                + self.expert_ws_bytes)
        self.norm = torch.zeros(1, dtype=torch.float32, device=dev)
        self.coef = torch.ones(1, dtype=torch.float32, device=dev)
        self._captured = []         # (list, workspace) that graphs captured from `clip` read
        self._list_gradients()      # copies a table to the device, which a captured `clip` could not

    # ---- streams ---------------------------------------------------------
    def _fork(self):
        if len(self.lanes) > 1:
            e = torch.cuda.Event()
            e.record(self.main)
            for ln in self.lanes[1:]:
                ln["stream"].wait_event(e)

    def _join(self):
        for ln in self.lanes[1:]:
            e = torch.cuda.Event()
            e.record(ln["stream"])
            self.main.wait_event(e)

    def _members(self):
        """The experts' W, v and S are their groups'."""
        for g in self.groups:
            g.bind(self.r)

    @contextlib.contextmanager
    def _late_inputs(self):
        """The callbacks' stream made current, after the fork; joins the
        step's stream. One lane alone has no other to wait for: its callbacks
        stay on the caller's stream."""
        if self.n_sketch == 1:
            yield
            return
        if self.callbacks is None:
            self.callbacks = torch.cuda.Stream(device=self.device)
        self.callbacks.wait_stream(torch.cuda.current_stream(self.device))
        self.callbacks.wait_stream(self.main)
        try:
            with torch.cuda.stream(self.callbacks):
                yield
        finally:
            self.main.wait_stream(self.callbacks)

    def _take(self, lane, tensors):
        """What a callback has just made, for a lane to read: the lane waits
        for the work that the callback enqueued, and the memory goes to no
        other use before the lane is done with it."""
        cur = torch.cuda.current_stream(self.device)
        if cur == lane:
            return
        # no event if the callbacks' stream has no work left: one delays the
        # lane's next kernel by some microseconds
        if torch.cuda.is_current_stream_capturing() or not cur.query():
            e = torch.cuda.Event()
            e.record(cur)
            lane.wait_event(e)
        for t in tensors:
            if t is not None:
                t.record_stream(lane)

    # ---- phases ----------------------------------------------------------
    def set_step(self, step: int):
        """The optimizer step whose sign matrices the calls use."""
        for m in self.mats:
            m.desc = B.MatrixDesc(m.d, m.k, self.r, seed=self.seed, step=step, matrix_id=m.matrix_id)

    def sketch(self, step: int, microbatches: int,
               inputs: Optional[Callable[[int, int], Tuple[torch.Tensor, torch.Tensor]]] = None,
               probe: Optional[Tuple[int, int]] = None,
               expert_inputs: Optional[Callable[[int, int], Tuple]] = None,
               late: Optional[bool] = None):
        """Fold `microbatches` microbatches into every matrix's S, microbatch
        by microbatch; inputs(i, mb) returns (X, dY) of matrix i, and
        expert_inputs(g, mb) returns (X, dY, offsets, order) of group g: dY
        (tokens topk rows) sorted by expert, offsets and order as
        logra_expert_sort gives them, X the tokens' activations (or their
        sorted copy, with order None).

        late     whether the callbacks make their tensors when they are
                 called (run the microbatch's router, sort and backward pass);
                 default: with expert groups. They do so on the stream that is
                 current in them, one of the step's own if it has several
                 lanes; the calls that read the tensors wait for that work,
                 and nobody need keep the tensors. As on any such stream, what
                 a callback enqueues on others it joins to the current one,
                 and memory of others that it reads and drops it records there
                 (Tensor.record_stream). Not late: every tensor is made on the
                 caller's stream before this call, and stays until the work of
                 this call is over; no stream waits for another then. (Late
                 callbacks of inputs that are there already: 56 calls of a
                 seven-matrix set 1.07 -> 1.42 ms, the 28-layer 7B stack 68.2
                 -> 70.4.)

        probe = (i, mb), mb >= 1: time matrix i's projection and fold
        without an event between the two (an event record delays the next
        kernel by a few microseconds): one event pair on its stream around
        the projection of microbatch mb - 1 alone, one around the projection
        and fold of microbatch mb; returns those two pairs,
        ((project_start, project_end), (both_start, both_end)), else None.
        The fold's time is the second pair's less the first's: each holds
        one event record's delay."""
        if probe is not None and probe[1] < 1:
            raise ValueError("probe: the microbatch must have one before it")
        if late is None:
            late = bool(self.groups)
        self._clipped = False
        self._members()
        self.set_step(step)
        if self.adamw is not None:
            with torch.cuda.stream(self.main):
                # a norm that `dense_update` reads also in a step that is not clipped
                if self._clip_captured or torch.cuda.is_current_stream_capturing():
                    self.norm.zero_()
        self._fork()
        try:                # a callback may fail: what is enqueued by then is joined all the same
            with self._late_inputs() if late else contextlib.nullcontext():
                return self._sketch(microbatches, inputs, probe, expert_inputs, self._take if late else None)
        finally:
            self._join()

    def _sketch(self, microbatches, inputs, probe, expert_inputs, take):
        events = None
        for mb in range(microbatches):
            for i, m in enumerate(self.dense):
                X, dY = inputs(i, mb)
                ln = self.lanes[m.lane]
                st = ln["stream"]
                if take:
                    take(st, (X, dY))
                alone = probe == (i, mb + 1)     # the projection before the probed one
                both = probe == (i, mb)
                if alone or both:
                    start = _event(st)
                B.logra_sketch_project(m.desc, X, ln["ws"], st, opts=self.sketch_opts)
                if alone:
                    proj_pair = (start, _event(st))
                if m.parts is not None:
                    phase = ((B.LOGRA_FOLD_FIRST if mb == 0 else 0)
                             | (B.LOGRA_FOLD_LAST if mb == microbatches - 1 else 0))
                    B.logra_sketch_fold_parts(m.desc, dY, m.S, m.parts, phase, ln["ws"], st,
                                              opts=self.sketch_opts)
                else:
                    B.logra_sketch_fold(m.desc, dY, m.S, mb > 0, ln["ws"], st, opts=self.sketch_opts)
                if both:
                    events = (proj_pair, (start, _event(st)))
            for i, g in enumerate(self.groups):
                X, dY, offsets, order = expert_inputs(i, mb)
                st = self.lanes[g.lane]["stream"]
                if take:
                    take(st, (X, dY, offsets, order))
                if dY.shape[0] != self.tokens * g.topk:
                    raise ValueError("expert group %s: %d rows of dY expected" % (g.name, self.tokens * g.topk))
                B.logra_sketch_experts(g.members[0].desc, offsets, X, dY, g.S, mb > 0, order=order, topk=g.topk,
                                       ws=g.ws, stream=st)
        return events

    def _gradients(self):
        return [m.S for m in self.dense] + [g.S for g in self.groups] + self.grads

    def _list_gradients(self):
        with torch.cuda.stream(self.main):      # where `clip` reads the table and the workspace
            self._grad_list = B.GradList(self._gradients())
            self._grad_ws = torch.empty(self._grad_list.workspace_bytes, dtype=torch.uint8, device=self.device)

    def clip(self, max_norm: float):
        """Clip the step's gradients by their global norm: every S (which
        holds the whole step after `sketch`) and the dense gradients given to
        Step, in place, before pass 1. Returns the device tensors (norm, coef)
        without waiting for them; a norm that is not finite clips nothing.

        Captured in a graph, it clips the gradients of the capture at every
        replay, also after another one (or another storage of the same one)
        has taken a gradient's place; the step keeps what such a graph reads. After a replacement the first clip
        lists the gradients anew, which a capture cannot: ValueError there."""
        self._members()
        with torch.cuda.stream(self.main):
            capturing = torch.cuda.is_current_stream_capturing()
        if not self._grad_list.describes(self._gradients()):    # a sketch or gradient was replaced since
            if capturing:
                raise ValueError("a gradient was replaced: clip once before the capture")
            self._list_gradients()
        self._clip_captured |= capturing
        if capturing and not any(kept[0] is self._grad_list for kept in self._captured):
            self._captured.append((self._grad_list, self._grad_ws))
        B.logra_grad_clip(self._grad_list, max_norm, self.norm, self.coef, ws=self._grad_ws, stream=self.main)
        self._clipped = True
        return self.norm, self.coef

    def dense_update(self, lr: float, beta1: float, beta2: float, eps: float, weight_decay: float, step: int):
        """One AdamW step (its `step`-th, from 1) over the dense parameters
        given to Step, on the caller's stream. After `clip` (or a replay of a
        graph that holds one), a norm that is not finite leaves parameters and
        moments as they are: the host that reads the norm does not count that
        step. Called eagerly, also between the replays of a captured step: in a
        graph it would repeat one step's number and learning rate. The step's
        seed keys the rounding of 8-bit moments. After a gradient in `grads` was
        replaced, give `adamw` a list that has the new one (with the old list's
        state): ValueError until then."""
        if self.adamw is None:
            raise ValueError("the step was given no dense parameters")
        a = self.adamw
        if not a.describes(a.params, a.grads, a.copies):
            raise ValueError("a dense parameter or gradient has other memory than its list was made with")
        clipped = self._clipped or self._clip_captured
        if clipped and not {id(g) for g in a.grads} <= {id(g) for g in self.grads}:
            raise ValueError("a dense parameter's gradient is not among those that clip takes: give the step a list of what it has now")
        B.logra_adamw(a, lr, beta1, beta2, eps, weight_decay, step, norm=self.norm if clipped else None,
                      seed=self.seed, stream=self.main)

    def pass1(self, beta2: float, eps: float):
        """v' and sqnorm of every matrix (v unchanged)."""
        self._members()
        self._fork()
        for li, chunk, sq, bws in self.batches:
            ln = self.lanes[li]
            if sq is None:
                m = chunk[0]
                B.logra_update_sqnorm(m.desc, self.code, m.S, m.v, beta2, eps, m.v_new, m.sq, m.rowsq,
                                      ln["sq_ws"], ln["stream"])
            else:
                rq = [m.rowsq for m in chunk] if chunk[0].rowsq is not None else None
                B.logra_update_sqnorm_batch([m.desc for m in chunk], self.code, [m.S for m in chunk],
                                            [m.v for m in chunk], beta2, eps, [m.v_new for m in chunk], sq,
                                            rq, bws, ln["stream"])
        self._join()

    def sqnorms(self) -> List[float]:
        """Every matrix's sqnorm on the host (one device-to-host copy)."""
        return torch.cat([m.sq for m in self.mats]).cpu().tolist()

    def pass2(self, lr: float, scales: Sequence[Optional[float]], eps: float) -> int:
        """W -= lr * scale * Ghat / (sqrt(v') + eps) for every matrix whose
        scale is not None, then v' becomes its v (buffer swap); the others
        keep W and v. Returns the number of matrices updated."""
        if len(scales) != len(self.mats):
            raise ValueError("one scale (or None) per matrix")
        self._members()
        self._fork()
        done = 0
        for m, sc in zip(self.mats, scales):
            if sc is None:
                continue
            B.logra_rowadam_apply(m.desc, self.code, m.S, m.v_new, m.W, lr, sc, eps,
                                  self.lanes[m.alane]["stream"], opts=self.apply_opts)
            m.v, m.v_new = m.v_new, m.v
            done += 1
        self._join()
        return done

    @staticmethod
    def finite_scales(sqnorms: Sequence[float], scales: Sequence[float]) -> List[Optional[float]]:
        """The scales with None where a matrix's sqnorm is not finite (its
        update is skipped)."""
        return [sc if math.isfinite(q) else None for q, sc in zip(sqnorms, scales)]

    def fold_timeouts(self) -> int:
        """Fold workgroups that gave up waiting for their partner since the
        counter was last cleared (0 in a healthy run)."""
        return int(self.timeouts.item())

    def clear_fold_timeouts(self):
        self.timeouts.zero_()
