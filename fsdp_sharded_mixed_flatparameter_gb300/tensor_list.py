"""TensorListAdamW: one AdamW step over many separate tensors at once.

For parameters that are not flattened into a FlatParameter: each tensor keeps
its own fp32 master, grad and low-precision copy, and belongs to a parameter
group with hyper-parameters of its own (decayed matrices, undecayed norms and
biases).  The moments are fp32 or 8 bits (``state_bits``); whichever, the
whole list is one kernel launch after the grad norm, with the clipping, skip
policy, step counter, loss scale and graph capture of FlatShardAdamW.  With
fp32 moments the result is FlatShardAdamW's bit for bit, tensor by tensor.
"""
from __future__ import annotations

import math
from typing import List, Optional, Sequence, Tuple, Union

import numpy as np
import torch

from . import zero_shard as zs
from .grad_clip import GradClip, need_groups, not_in_capture, one_limit
from .optimizer import GradTables, torch_stream

_DEFAULTS = ("lr", "betas", "eps", "weight_decay")


class TensorListAdamW(GradTables):
    """masters: contiguous fp32 CUDA tensors of any shape, updated in place.  lowp: None,
    or per tensor None or its bf16 / f16 copy.  groups: a dict per parameter group with any
    of lr, betas, eps, weight_decay (the rest from the keyword arguments); group_of: each
    tensor's group (default: all in group 0).  rounding_seed (8 bits only): an integer seeds
    stochastic rounding of the moments (default 0); None rounds them to nearest, by which they
    do not follow their recurrences over a run (optimizer.py).  Lists that share a seed take
    rounding_streams that are further apart than they have tensors.

    max_norm: the limit of the norm over all grads, or a limit for each group (inf: not clipped;
    several need group_of): then every group's grads are clipped by the group's own norm (``clip``, a GradClip, has the
    norms, and its set_max_norm() changes the limits; the grads themselves stay as they are), the
    step is skipped where the norm over all is not finite, and step() gives that norm with a
    coefficient of 1.  Those norms are finite for any finite grads, where the one norm's squares
    end at 2^64: a group without a limit takes grads of that size, whose squares exp_avg_sq cannot
    hold, and so does any group of grads whose scaled values leave binary32.

    The moments live in storages of this object, tensor i's at elements offsets[i] ..
    offsets[i] + numels[i]: ``exp_avg`` and ``exp_avg_sq`` (fp32), or ``state8`` (8 bits:
    codes at offsets[i], scales at offsets[i] / 256).  Offsets are multiples of 256."""

    def __init__(self, masters: Sequence[torch.Tensor], *, lowp: Optional[Sequence[Optional[torch.Tensor]]] = None,
                 groups: Optional[Sequence[dict]] = None, group_of: Optional[Sequence[int]] = None, lr: float = 1e-4,
                 betas: Tuple[float, float] = (0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.0,
                 max_norm: Union[float, Sequence[float]] = math.inf, state_bits: int = 32,
                 rounding_seed: Union[int, None, str] = zs.DEFAULT_SEED,
                 rounding_stream: int = 0, capturable: bool = False):
        rounding_seed = zs.rounding_choice(state_bits, rounding_seed)
        self.masters = list(masters)
        if not self.masters:
            raise ValueError("an empty tensor list")
        self.lowp = None if lowp is None else list(lowp)
        self.device = self.masters[0].device
        self.state_bits, self.rounding_seed, self.capturable = state_bits, rounding_seed, capturable
        self.max_norm, self.rounding_stream = max_norm, rounding_stream
        defaults = dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay)
        self._groups: List[list] = []
        for g in ([{}] if groups is None else groups):
            if set(g) - set(_DEFAULTS):
                raise ValueError(f"a group takes {', '.join(_DEFAULTS)}: got {sorted(g)}")
            h = {**defaults, **g}
            self._groups.append([float(h["lr"]), float(h["betas"][0]), float(h["betas"][1]), float(h["eps"]),
                                 float(h["weight_decay"])])
        if not 1 <= len(self._groups) <= zs.LIST_MAX_GROUPS:
            raise ValueError(f"1 to {zs.LIST_MAX_GROUPS} groups")
        self._hp = zs.list_groups(self._groups)
        per_group = not one_limit(max_norm)
        if per_group and len(max_norm) != len(self._groups):
            raise ValueError(f"{len(max_norm)} limits for {len(self._groups)} groups")
        if per_group:
            need_groups(max_norm, group_of)
        columns, numels, lowp_dtype = zs.list_masters(self.masters, self.lowp, group_of)
        self._init_tables(numels, self.device)
        blocks = np.cumsum([0] + [zs.state8_blocks(n) for n in numels])  # each tensor starts on a block's border
        self.offsets, total = (blocks[:-1] * zs.STATE8_BLOCK).tolist(), int(blocks[-1]) * zs.STATE8_BLOCK
        if state_bits == 8:
            self.state8, self.exp_avg, self.exp_avg_sq = zs.new_state8(total, self.device), None, None
        else:
            self.state8 = None
            self.exp_avg = torch.zeros(total, dtype=torch.float32, device=self.device)
            self.exp_avg_sq = torch.zeros(total, dtype=torch.float32, device=self.device)
        # every tensor's moments by their address in the storages; none where there are no elements
        at, some = blocks[:-1].astype(np.uint64), np.asarray(numels) > 0
        fields = {"exp_avg": (self.exp_avg, 1024), "exp_avg_sq": (self.exp_avg_sq, 1024)} if state_bits == 32 else {
            "exp_avg": (self.state8.exp_avg, 256), "exp_avg_sq": (self.state8.root, 256),
            "exp_avg_scale": (self.state8.exp_avg_scale, 4), "root_scale": (self.state8.root_scale, 4)}
        for nm, (t, block_bytes) in fields.items():
            columns[nm] = np.where(some, np.uint64(t.data_ptr()) + at * np.uint64(block_bytes), np.uint64(0))
        self._list = zs.make_tensor_list(columns, numels, group_of, len(self._groups), state_bits, lowp_dtype, self.device)
        self.ws = torch.empty(max(zs.zero_grad_sqnorm_workspace_bytes(self.total), 8), dtype=torch.uint8,
                              device=self.device)
        self.clip: Optional[GradClip] = None
        if per_group:
            of = [0] * len(numels) if group_of is None else group_of
            self.clip = GradClip(numels, max_norm=max_norm, group_of=of, device=self.device)
            self.norm_buf, self.found_nonfinite = self.clip.result, self.clip.found_nonfinite
        else:
            self.norm_buf = zs.new_norm_result(self.device)
            self.found_nonfinite = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._t = 0
        if capturable:
            self._dev_hp = torch.cat([zs.device_hparams(*g, self.device) for g in self._groups])
            self._dev_states = zs.new_adamw_device_state(self.device).repeat(len(self._groups))

    # ------------------------------------------------------------- state
    def state_of(self, i: int):
        """Tensor i's moments: views of the storages, (exp_avg, exp_avg_sq) or a State8."""
        a, n = self.offsets[i], self.numels[i]
        if self.state_bits == 32:
            return self.exp_avg[a:a + n], self.exp_avg_sq[a:a + n]
        q, b, k = self.state8, a // zs.STATE8_BLOCK, zs.state8_blocks(n)
        return zs.State8(q.exp_avg[a:a + n], q.exp_avg_scale[b:b + k], q.root[a:a + n], q.root_scale[b:b + k])

    @property
    def t(self) -> int:
        """Steps applied so far (with capturable=True read from the device: a sync)."""
        if self.capturable:
            return zs.decode_adamw_device_state(self._dev_states).step
        return self._t

    @t.setter
    def t(self, value: int) -> None:
        if self.capturable:
            self._dev_states.copy_(zs.new_adamw_device_state(self.device, int(value)).repeat(len(self._groups)))
        else:
            self._t = int(value)

    def group(self, i: int) -> dict:
        """Group i's hyper-parameters."""
        lr, b1, b2, eps, wd = self._groups[i]
        return dict(lr=lr, betas=(b1, b2), eps=eps, weight_decay=wd)

    def set_group(self, i: int, **hp) -> None:
        """Change hyper-parameters of group i, e.g. lr from a schedule (with capturable=True also
        for the next replay of a captured graph)."""
        if set(hp) - set(_DEFAULTS):
            raise ValueError(f"a group takes {', '.join(_DEFAULTS)}: got {sorted(hp)}")
        h = {**self.group(i), **hp}
        self._groups[i] = [float(h["lr"]), float(h["betas"][0]), float(h["betas"][1]), float(h["eps"]),
                           float(h["weight_decay"])]
        self._hp = zs.list_groups(self._groups)
        if self.capturable:
            i %= len(self._groups)
            zs.device_hparams(*self._groups[i], self.device,
                              out=self._dev_hp[i * zs.HPARAMS_BYTES:(i + 1) * zs.HPARAMS_BYTES])

    # -------------------------------------------------------------- step
    def register_grads(self, grads: Sequence[Optional[torch.Tensor]]) -> None:
        """Fix the grads once (see GradTables); with a limit for each group needed before a capture,
        and on this list's device."""
        before = self._registered
        super().register_grads(grads)
        if self.clip is not None:
            try:
                self.clip.register_grads(grads, write=False)
            except Exception:  # the step's grads and those of its norms are the same ones
                self._registered = before
                raise

    def launch_step(self, grads: Optional[Sequence[Optional[torch.Tensor]]] = None, *, scale: float = 1.0, stream=None,
                    loss_scale=None, norm_result: Optional[torch.Tensor] = None) -> None:
        """Enqueue the grad norm over the whole list and the update for step t + 1 without
        waiting.  grads: a grad or None (reads as zeros) per tensor, any alignment, one dtype (in
        pinned host memory only with one limit); None: the registered ones.  loss_scale: a DeviceLossScale, whose unscale factor
        replaces `scale`.  norm_result: a zero_norm_result computed elsewhere (one clip over
        several optimizers): used as is, no norm is computed."""
        if grads is not None and norm_result is None and self.clip is not None:
            not_in_capture(self._index)
        table, count, dt, stream = self._launch_tables(grads, stream)
        sc, dsc, flag = self._scale_args(scale, loss_scale)
        clip, clips = norm_result, norm_result is None and self.clip is not None
        if clips:
            self.clip.launch_norms(grads, scale=scale, loss_scale=loss_scale, stream=stream)
            clip = self.clip.results
        elif clip is None:
            clip = self.norm_buf
            zs.zero_flatten_cast(table, count, self.total, dt, 0, self.total, sc, False, None, flag, self.ws, stream,
                                 d_scale=dsc)
            zs.zero_grad_sqnorm_finalize(self.ws, self.total, 0.0, self.max_norm, clip, stream)
        if self.capturable:
            zs.zero_adamw_prepare_list_device(self._dev_hp, len(self._groups), self.clip.result if clips else clip,
                                              self._dev_states, stream)
            zs.zero_adamw_list_device(self._list, table, dt, sc, self._dev_states, clip, stream, d_scale=dsc,
                                      rounding_seed=self.rounding_seed, rounding_stream=self.rounding_stream,
                                      clips=clips)
        else:
            zs.zero_adamw_list(self._list, table, dt, sc, self._hp, self._t + 1, clip, stream, d_scale=dsc,
                               rounding_seed=self.rounding_seed, rounding_stream=self.rounding_stream, clips=clips)

    def finish_step(self, stream=None, norm_result: Optional[torch.Tensor] = None) -> zs.NormResult:
        """Read the step's norm (a device-to-host copy on `stream`, the stream the step was
        enqueued on) and count the step unless it was skipped.  norm_result: the buffer given
        to launch_step, if any."""
        with torch.cuda.stream(torch_stream(stream, self.device)):
            r = zs.decode_norm_result(self.norm_buf if norm_result is None else norm_result)
        if r.finite and not self.capturable:
            self._t += 1
        return r

    def step(self, grads: Optional[Sequence[Optional[torch.Tensor]]] = None, *, scale: float = 1.0, stream=None,
             loss_scale=None) -> zs.NormResult:
        """One step: norm, clip, AdamW; nothing changes (and t stays) when the norm is not finite."""
        self.launch_step(grads, scale=scale, stream=stream, loss_scale=loss_scale)
        return self.finish_step(stream)

    # -------------------------------------------------------- checkpoint
    def state_dict(self) -> dict:
        """Step count, masters and moments on the host, in the moments' own form."""
        sd = {"t": self.t, "numels": list(self.numels), "state_bits": self.state_bits,
              "masters": [p.detach().cpu().clone() for p in self.masters]}
        if self.state_bits == 8:
            sd["state8"] = tuple(x.cpu() for x in self.state8)
        else:
            sd["exp_avg"], sd["exp_avg_sq"] = self.exp_avg.cpu(), self.exp_avg_sq.cpu()
        return sd

    def load_state_dict(self, sd: dict, stream=None) -> None:
        """Restore a checkpoint of the same tensors.  One with moments of the other width is
        converted: 32-bit moments are packed to nearest, 8-bit ones unpacked.  The low-precision
        copies are rewritten from the masters.  Masters and copies may require grad.  Everything
        is written on `stream` (default: the current one), in order with the steps there.  A
        checkpoint that does not fit is refused before anything is written."""
        if list(sd["numels"]) != list(self.numels) or [x.numel() for x in sd["masters"]] != list(self.numels):
            raise ValueError("state belongs to another tensor list")
        zs.check_moments(sd, (self.exp_avg if self.state_bits == 32 else self.state8.exp_avg).numel())
        with torch.no_grad(), torch.cuda.stream(torch_stream(stream, self.device)):
            self.t = int(sd["t"])  # on the device with capturable=True: in the stream's order too
            for p, x in zip(self.masters, sd["masters"]):
                p.copy_(x.view(p.shape))
            for p, c in zip(self.masters, self.lowp or ()):
                if c is not None:
                    c.copy_(p.view(c.shape))
            zs.load_moments(sd, self.state8, self.exp_avg, self.exp_avg_sq, self.device)

    def resident_bytes(self) -> int:
        """Device bytes of the masters, copies and moments."""
        own = [self.exp_avg, self.exp_avg_sq] if self.state_bits == 32 else list(self.state8)
        return sum(t.numel() * t.element_size() for t in [*self.masters, *(c for c in self.lowp or () if c is not None),
                                                          *own])
