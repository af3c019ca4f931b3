"""GradClip: the norms of many tensors and their clipping, in place or into other buffers.

``clip_grad_norm_`` of the pages' loops for grads that this library's AdamW does not
read (it folds one clip over everything into its own pass): tensors of mixed
types, the norm of each tensor and of groups of tensors beside the norm of all,
p = 1, 2 or infinity, a limit for each group, unscaling in the same pass, and the
same for one rank's flat shard, joined with the other ranks' sums.  Nothing
waits for the host, so a whole step can be captured in a graph.
"""
from __future__ import annotations

import math
from typing import List, NamedTuple, Optional, Sequence, Union

import numpy as np
import torch

from . import zero_shard as zs
from .optimizer import GradTable, GradTables, gather_sqnorms, torch_stream


class ClipResult(NamedTuple):
    """A clip read on the host: the norm over all tensors, whether it is finite (if not, no
    grad was written), each group's norm (float64) and coefficient (float32)."""
    norm: float
    finite: bool
    group_norms: np.ndarray
    coefs: np.ndarray
    whole: zs.NormResult


class GradEntries(NamedTuple):
    """A list of grads prepared for launches: the list, its table's stream, whether its grads may be
    written; for a registered one the tensors that launches read and write, which it keeps alive,
    and the streams besides the table's that their memory was recorded on."""
    list: zs.GradList
    table: GradTable
    write: bool
    tensors: tuple
    streams: set


class GradClip(GradTables):
    """The clip over tensors of the sizes `numels`.  max_norm: the limit, or one per group (inf:
    not clipped); group_of: each tensor's group (with one limit by default 0 for all; several
    limits need it), with range(len(numels)) each tensor is clipped by its own norm; norm_type: 1, 2 or inf.

    After a launch, on the device: ``tensor_norms``, ``group_norms`` (float32), ``norm`` (0-d),
    ``tensor_sums`` (float64, this rank's; ``joined_sums``: of gathered ones, all ranks'),
    ``results`` (a zero_norm_result per group) and ``result``, the one over all with a
    coefficient of 1: what launch_step(norm_result=...) of the optimizers takes after the grads have been clipped here.  The buffers are rewritten by
    each launch: launches of one object that overlap on the GPU race, and the object has to
    outlive the graphs that captured it.

    Making a GradClip and registering grads copies tables to the device and waits for the current
    stream.  A launch waits for nothing, but for one with grads of its own on a stream that is
    not the current one (its table is copied first).  wait=False: nothing is waited for, and the
    clip is for the current stream alone."""

    def __init__(self, numels: Sequence[int], *, max_norm: Union[float, Sequence[float]] = math.inf,
                 norm_type: float = 2.0, group_of: Optional[Sequence[int]] = None, device="cuda", wait: bool = True):
        self._init_tables(numels, device)
        if one_limit(max_norm):
            n_groups = 1 if group_of is None or len(group_of) == 0 else int(max(group_of)) + 1
        else:
            n_groups = len(max_norm)
            need_groups(max_norm, group_of)
        self.norm_type, self.n_groups = float(norm_type), n_groups
        if not self.numels:
            raise ValueError("an empty tensor list")
        dev = self.device
        limits = self._limits(max_norm)
        not_in_capture(self._index)
        self.plan = zs.zero_grad_plan(self.numels, group_of, n_groups, norm_type, dev, wait)
        n, g = len(self.numels), n_groups
        self.max_norms = zs._to_device(limits.numpy(), dev, wait)
        self.buffers = zs.norm_buffers(self.plan, self.max_norms, wait)
        self.tensor_sums, self.joined_sums = self.buffers.sums, self.buffers.joined
        norms, self.results = self.buffers.norms, self.buffers.results
        self.tensor_norms, self.group_norms, self.norm = norms[:n], norms[n:n + g], norms[n + g]
        self.result = self.results[g * zs.NORM_RESULT_BYTES:]
        self.found_nonfinite = self.buffers.found
        self._home = self._current()  # the stream whose order the buffers' memory follows
        self._last: Optional[int] = None  # the stream of the last launch that was not captured
        self.shard: Optional[torch.Tensor] = None
        self._replayed: List[GradEntries] = []  # what captured graphs read and write

    @classmethod
    def of_shard(cls, numels: Sequence[int], grad: torch.Tensor, start: int, **kw) -> "GradClip":
        """The clip over one rank's flat grad: elements start .. start + grad.numel() of the
        FlatParameter of the tensors `numels`.  tensor_sums are those of the pieces that lie in it
        (0 for a tensor elsewhere); launch(process_group=...) or launch_sums() and
        launch(gathered_sums=...) join them with the other ranks'."""
        if grad.dim() != 1 or not grad.is_contiguous():
            raise ValueError("the shard's grad must be 1-D and contiguous")
        sizes = np.asarray(numels, dtype=np.int64)
        ends = np.cumsum(sizes)
        end, total = start + grad.numel(), int(ends[-1]) if len(ends) else 0
        if start < 0 or end > total:
            raise ValueError(f"[{start}, {end}) is not a shard of {total} elements")
        lo, hi = np.maximum(ends - sizes, start), np.minimum(ends, end)
        local = np.maximum(0, hi - lo)
        clip = cls(local.tolist(), **{"device": grad.device, **kw})
        gl = zs.flat_grad_list(clip.plan, grad, lo - start)
        clip._registered, clip.shard = clip._prepared(gl, True, (grad,)), grad
        return clip

    # ------------------------------------------------------------ limits
    def _limits(self, max_norm) -> torch.Tensor:
        values = [max_norm] * self.n_groups if one_limit(max_norm) else list(max_norm)
        if len(values) != self.n_groups:
            raise ValueError(f"{len(values)} limits for {self.n_groups} groups")
        if any(math.isnan(v) or v < 0 for v in values):
            raise ValueError("max_norm must be >= 0")
        return torch.tensor([float(v) for v in values], dtype=torch.float64)

    def set_max_norm(self, max_norm: Union[float, Sequence[float]], stream=None) -> None:
        """Change the limits for every later launch (also for the next replay of a captured graph),
        and for none before.  They are written on `stream` (default: the current one), behind what
        was enqueued there and behind the last launch, whichever its stream; this waits for that.
        Replays that may still run on another stream have to be waited for, or that stream given."""
        limits = self._limits(max_norm)
        if self._index is None:
            self.max_norms.copy_(limits)
            return
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("change the limits outside the capture: the graph's replays follow them")
        raw = self._handle(stream)
        st = torch_stream(raw, self.device)
        if self._last is not None and self._last != raw:
            st.wait_stream(torch_stream(self._last, self.device))
        with torch.cuda.stream(st):
            self.max_norms.copy_(limits)  # waits, as the limits are not in pinned memory: any stream may launch then

    # ------------------------------------------------------------- grads
    def register_grads(self, grads: Sequence[Optional[torch.Tensor]],
                       out: Optional[Sequence[Optional[torch.Tensor]]] = None, *, write: bool = True) -> None:
        """Fix the grads once: per tensor an f32, bf16 or f16 tensor, or None (reads as zeros).
        out: other buffers for the clipped grads (None for a tensor: it is not written; a
        tensor without a grad gets zeros); without it they are clipped in place.  A launch
        without grads then does no work per tensor on the host, and can be captured.  The
        tensors are kept alive until others are registered, and as long as this object where a
        launch of them was captured.
        write=False: for norms only; a tensor may then be listed twice."""
        tensors = tuple(t for t in (*grads, *(out or ())) if t is not None)
        self._registered = self._entries(grads, out, write, tensors)
        self.shard = None  # no longer the clip over a flat buffer, which that buffer's step takes

    def device_table(self, grads: Sequence[Optional[torch.Tensor]]):
        """The FlatParameter table of a grads list (see GradTables).  A clip's launches read tables of
        their own kind, so the registered grads have none."""
        if grads is None:
            raise ValueError("device_table() of a GradClip needs the grads: its registered ones have no FlatParameter table")
        return super().device_table(grads)

    def _entries(self, grads, out, write, tensors=(), wait=True) -> GradEntries:
        not_in_capture(self._index)
        return self._prepared(zs.grad_list(self.plan, grads, out, write, wait), write, tensors)

    def _prepared(self, gl, write, tensors) -> GradEntries:
        return GradEntries(gl, GradTable(gl.entries, self._current()), write, tensors, set())

    def _current(self) -> int:
        return 0 if self._index is None else self._handle(None)  # host: only to be refused at a launch

    def _list(self, grads, out, write, stream) -> GradEntries:
        if grads is not None:
            here = self._index is not None and self._handle(stream) == self._current()
            return self._entries(grads, out, write, wait=not here)
        if out is not None:
            raise ValueError("out needs grads")
        if self._registered is None:
            raise ValueError("no grads given and none registered")
        if write and not self._registered.write:
            raise ValueError("the registered grads are for norms only (write=False)")
        return self._registered

    def _on(self, stream, of: GradEntries) -> int:
        """The handle of the stream to launch on, its use of the memory of this object and of the
        registered tensors noted."""
        if self._index is None:
            return 0
        raw = self._handle(stream)
        capturing = torch.cuda.is_current_stream_capturing()
        if not capturing:
            self._last = raw
        if raw == self._home == of.table.stream and not capturing:
            return raw
        self._read_on(of.table, raw)
        if capturing:
            if not any(r is of for r in self._replayed):
                self._replayed.append(of)
            return raw
        if raw != self._home:
            st = torch_stream(raw, self.device)
            for t in (self.plan.ints, *self.buffers[1:8]):
                t.record_stream(st)
        if raw != of.table.stream and raw not in of.streams:
            # once: whatever was launched there until their memory is freed is waited for
            st = torch_stream(raw, self.device)
            for t in of.tensors:
                t.record_stream(st)
            of.streams.add(raw)
        return raw

    def _used_on(self, raw: int, *lists) -> None:
        """Tensors of this launch that are read or written on a stream other than the current one:
        their memory is not given out again before that is done."""
        if self._index is None or raw == self._current():
            return
        st = torch_stream(raw, self.device)
        for t in (t for ts in lists if ts is not None for t in ts):
            if t is not None:
                t.record_stream(st)

    # ------------------------------------------------------------ launch
    def launch_sums(self, grads: Optional[Sequence[Optional[torch.Tensor]]] = None, *, scale: float = 1.0,
                    loss_scale=None, stream=None) -> None:
        """Enqueue each tensor's sum into ``tensor_sums``: what ranks exchange."""
        if self._elsewhere():
            with torch.cuda.device(self._index):
                return self.launch_sums(grads, scale=scale, loss_scale=loss_scale, stream=stream)
        sc, dsc, _ = self._scale_args(scale, loss_scale)
        of = self._list(grads, None, False, stream)
        gl, raw = of.list, self._on(stream, of)
        self._used_on(raw, grads)
        zs.zero_list_sums(gl, sc, self.buffers, raw, d_scale=dsc)

    def _elsewhere(self) -> bool:
        """Whether another device than the clip's is the current one."""
        return self._index is not None and torch.cuda.current_device() != self._index

    def launch_norms(self, grads: Optional[Sequence[Optional[torch.Tensor]]] = None, *, scale: float = 1.0,
                     loss_scale=None, gathered_sums: Optional[torch.Tensor] = None, process_group=None,
                     stream=None) -> None:
        """launch() without writing any grad."""
        self._launch(False, grads, None, scale, loss_scale, gathered_sums, process_group, stream)

    def launch(self, grads: Optional[Sequence[Optional[torch.Tensor]]] = None, *,
               out: Optional[Sequence[Optional[torch.Tensor]]] = None, scale: float = 1.0, loss_scale=None,
               gathered_sums: Optional[torch.Tensor] = None, process_group=None, stream=None) -> None:
        """Enqueue the norms and the clipping without waiting.  grads, out: as register_grads takes
        them, for this launch (default: the registered ones).  scale: multiplies every grad before
        the norm (unscaling, averaging); loss_scale: a DeviceLossScale, whose unscale factor
        replaces `scale` and whose flag a norm that is not finite raises.  gathered_sums: the
        ranks' tensor_sums in rank order, [ranks, tensors] (launch_sums() has run, its row is this
        rank's); process_group: the sums are gathered here, ordered on `stream`.

        y = scale * coefficient * x, written where the norm over all tensors is finite.  Autograd
        counts that as a change in place of tensors given here (so that a graph that has saved one
        refuses to use it), not of registered ones."""
        self._launch(True, grads, out, scale, loss_scale, gathered_sums, process_group, stream)

    def _launch(self, clip, grads, out, scale, loss_scale, gathered, process_group, stream) -> None:
        if self._elsewhere():
            with torch.cuda.device(self._index):
                return self._launch(clip, grads, out, scale, loss_scale, gathered, process_group, stream)
        self._enqueue(clip, grads, out, scale, loss_scale, gathered, process_group, stream)
        if clip and grads is not None:  # 55 ns a tensor, which a registered list is spared
            torch.autograd.graph.increment_version([t for t in (grads if out is None else out) if t is not None])

    def _enqueue(self, clip, grads, out, scale, loss_scale, gathered, process_group, stream) -> None:
        n, dev = len(self.numels), self.plan.ints.device
        if gathered is not None and (gathered.numel() == 0 or gathered.numel() % n or gathered.device != dev
                                     or (gathered.dim() > 1 and gathered.shape[-1] != n)):
            raise ValueError(f"gathered_sums must be [ranks, {n}] on {dev}")
        of = self._list(grads, out, clip, stream)
        gl, raw = of.list, self._on(stream, of)
        if grads is not None or gathered is not None:
            self._used_on(raw, grads, out, None if gathered is None else [gathered])
        sc, dsc, flag = self._scale_args(scale, loss_scale)
        if loss_scale is None:
            flag = None  # the buffers' own
        if gathered is None and process_group is not None and _world(process_group) > 1:
            zs.zero_list_sums(gl, sc, self.buffers, raw, d_scale=dsc)
            with torch.cuda.stream(torch_stream(raw, self.device)):
                gathered = gather_sqnorms(self.tensor_sums, process_group)
        if gathered is None:
            zs.zero_list_norms(gl, sc, clip, self.buffers, flag, raw, d_scale=dsc)
            return
        zs.zero_sums_norms(gl, gathered, gathered.numel() // n, self.buffers, flag, raw)
        if clip:
            zs.zero_list_clip(gl, sc, self.buffers, raw, d_scale=dsc)

    def finish(self, stream=None) -> ClipResult:
        """Read the last launch's result (a device-to-host copy on `stream`, where it was enqueued)."""
        with torch.cuda.stream(torch_stream(stream, self.device)):
            raw = self.results.cpu()
        r = np.frombuffer(raw.numpy().tobytes(), dtype=_RESULT)
        whole = zs.decode_norm_result(raw[self.n_groups * zs.NORM_RESULT_BYTES:])
        return ClipResult(whole.norm, whole.finite, r["norm"][:-1].copy(), r["clip_coef"][:-1].copy(), whole)

    def clip_(self, grads: Optional[Sequence[Optional[torch.Tensor]]] = None, **kw) -> ClipResult:
        """launch() and finish(): one clip, read on the host."""
        self.launch(grads, **kw)
        return self.finish(kw.get("stream"))


_RESULT = np.dtype([("sqnorm", np.float64), ("norm", np.float64), ("clip_coef", np.float32), ("finite", np.int32)])


def clip_grad_norm_(grads: Sequence[Optional[torch.Tensor]], max_norm: float, norm_type: float = 2.0, *,
                    scale: float = 1.0, stream=None) -> torch.Tensor:
    """Clip `grads` in place by the norm of all of them and return that norm (a 0-d float32
    device tensor) without waiting, on the current stream or on `stream`.  Where it is not finite
    nothing is written.  For a loop, a GradClip with registered grads spares the tables."""
    grads = list(grads)
    some = [g for g in grads if g is not None]
    if not some:
        raise ValueError("no grads")
    clip = GradClip([0 if g is None else g.numel() for g in grads], max_norm=max_norm, norm_type=norm_type,
                    device=some[0].device, wait=stream is not None)
    clip.launch(grads, scale=scale, stream=stream)
    return clip.norm


def one_limit(max_norm) -> bool:
    """Whether max_norm is a number and not one for each group."""
    return not hasattr(max_norm, "__len__") or getattr(max_norm, "ndim", 1) == 0


def need_groups(max_norm, group_of) -> None:
    """Several limits without groups would all but the first belong to no tensor."""
    if len(max_norm) > 1 and group_of is None:
        raise ValueError(f"max_norm has {len(max_norm)} limits: group_of has to say which tensors each is for")


def not_in_capture(index) -> None:
    """Tables are copied to the device when a clip is made or grads are registered: not in a capture."""
    if index is not None and torch.cuda.is_current_stream_capturing():
        raise RuntimeError("make the GradClip and register its grads before the capture")


def _world(group) -> int:
    import torch.distributed as dist
    return dist.get_world_size(group)
