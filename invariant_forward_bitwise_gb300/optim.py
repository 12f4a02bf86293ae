"""AdamW over a model's tensors, as libbiv calls: a launch per combination of
types (usually one) updates every weight in place, with the global gradient-norm clip before it.

The trainer keeps BF16 weights that the inference forward reads ("Finish RL
Training Faster", section "让训练前向使用推理的数值"); the step writes them where
they are, so captured rollout graphs replay with the new weights.  Learning
rate, step count and clip coefficient live in device memory: a captured
``step()`` can be replayed too.
"""
from __future__ import annotations

from typing import Optional, Sequence, Union

import torch

from . import biv

BLOCK = 128   # elements per scale of an 8-bit state

_DT = {torch.float32: biv.F32, torch.bfloat16: biv.BF16}
_STATE = {torch.float32: biv.F32, torch.uint8: biv.E4M3, torch.float8_e4m3fn: biv.E4M3}


def _blocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


class AdamW:
    """params: bf16 or float32 tensors; grads: float32 or bf16 tensors of the
    same sizes, read at every step (their memory must stay).  master: float32
    copies of bf16 params (None, or None entries: the bf16 weight itself is
    updated).  State tensors may be passed in (a resumed run); those missing
    are created as zeros: float32, or 8-bit e4m3 codes with a float32 scale
    per 128 elements where ``bits`` is 8.  lr: a float, or a float32 device
    tensor of one value that the caller keeps; weight_decay and lr_scale: one
    value, or one per tensor; max_norm: 0 takes no norm.  rounding "nearest"
    or "stochastic" (8-bit states and bf16 weights without a master; the bits
    come from a hash of seed, step and element).

    ``step()`` runs on the current stream.  Attributes: ``norm`` float32 [4]
    (gradient norm and clip coefficient of the last step; the rest is the kernel's), ``steps`` int32 [2]
    (steps taken; the second value is the kernel's own).  With a max_norm, a step
    whose gradient norm is not finite changes nothing; without one nothing looks for
    NaN and infinite gradients, and their weights become NaN.

    The norm is that of the gradients given here, on this process.  Where ranks
    hold different weights besides replicated ones (experts spread over ranks),
    ``step()`` with a max_norm would scale the replicated ones differently on each:
    take ``biv.biv_grad_norm`` on ``table``, reduce ``norm`` over the ranks (the root
    of the sum of squares, a replicated weight's counted once) and its coefficient
    with it, then ``biv.biv_adamw(desc)``.
    """

    def __init__(self, params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], master=None,
                 exp_avg=None, exp_avg_sq=None, exp_avg_scale=None, exp_avg_sq_scale=None,
                 lr: Union[float, torch.Tensor] = 1e-6, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay=0.0, lr_scale=1.0, max_norm: float = 0.0, bits: int = 32,
                 rounding: str = "nearest", seed: int = 0, step: Optional[torch.Tensor] = None):
        biv.load()
        n = len(params)
        if n == 0:
            raise ValueError("AdamW needs at least one tensor")
        if bits not in (8, 32):
            raise ValueError("bits must be 8 or 32")
        if rounding not in ("nearest", "stochastic"):
            raise ValueError('rounding must be "nearest" or "stochastic"')
        self.device = params[0].device
        if not params[0].is_cuda or self.device.index != torch.cuda.current_device():
            raise ValueError("the tensors must be on the current CUDA device")

        def per_tensor(x, what):
            x = [x] * n if x is None or isinstance(x, (int, float)) else list(x)
            if len(x) != n:
                raise ValueError(f"{what}: {len(x)} entries for {n} tensors")
            return x

        self.params, self.grads = list(params), per_tensor(grads, "grads")
        self.master = per_tensor(master, "master")
        wd, ls = per_tensor(weight_decay, "weight_decay"), per_tensor(lr_scale, "lr_scale")
        state = torch.float32 if bits == 32 else torch.uint8
        self.exp_avg, self.exp_avg_sq = [], []
        self.exp_avg_scale, self.exp_avg_sq_scale = [], []
        given = [per_tensor(x, w) for x, w in
                 ((exp_avg, "exp_avg"), (exp_avg_sq, "exp_avg_sq"), (exp_avg_scale, "exp_avg_scale"),
                  (exp_avg_sq_scale, "exp_avg_sq_scale"))]
        arr = (biv.OptTensor * n)()
        for i, (p, g, w) in enumerate(zip(self.params, self.grads, self.master)):
            m, v, ms, vs = (x[i] for x in given)
            size = p.numel()
            if m is None:
                m = torch.zeros(size, dtype=state, device=self.device)
            if v is None:
                v = torch.zeros(size, dtype=m.dtype, device=self.device)
            if _STATE.get(m.dtype) == biv.E4M3:
                ms = torch.zeros(_blocks(size), device=self.device) if ms is None else ms
                vs = torch.zeros(_blocks(size), device=self.device) if vs is None else vs
            for what, t, types, cnt in (("param", p, _DT, size), ("grad", g, _DT, size),
                                        ("master", w, (torch.float32,), size), ("exp_avg", m, _STATE, size),
                                        ("exp_avg_sq", v, _STATE, size),
                                        ("exp_avg_scale", ms, (torch.float32,), _blocks(size)),
                                        ("exp_avg_sq_scale", vs, (torch.float32,), _blocks(size))):
                if t is None and what in ("master", "exp_avg_scale", "exp_avg_sq_scale"):
                    continue
                if t is None or t.dtype not in types:
                    raise ValueError(f"tensor {i}: {what} is missing or of an unsupported type")
                if t.device != self.device or not t.is_contiguous() or t.numel() != cnt:
                    raise ValueError(f"tensor {i}: {what} must be contiguous, of {cnt} values, on {self.device}")
            if _STATE[m.dtype] != _STATE[v.dtype]:
                raise ValueError(f"tensor {i}: exp_avg and exp_avg_sq differ in type")
            self.exp_avg.append(m)
            self.exp_avg_sq.append(v)
            self.exp_avg_scale.append(ms)
            self.exp_avg_sq_scale.append(vs)
            a = arr[i]
            a.param, a.grad, a.m, a.v = p.data_ptr(), g.data_ptr(), m.data_ptr(), v.data_ptr()
            a.master = None if w is None else w.data_ptr()
            a.m_scale = None if ms is None else ms.data_ptr()
            a.v_scale = None if vs is None else vs.data_ptr()
            a.numel, a.lr_scale, a.weight_decay = size, float(ls[i]), float(wd[i])
            a.param_dtype, a.grad_dtype, a.state_dtype = _DT[p.dtype], _DT[g.dtype], _STATE[m.dtype]
        self.chunks, kinds = biv.biv_opt_plan(arr)
        self.n = n
        self.table = torch.frombuffer(bytearray(bytes(arr)), dtype=torch.uint8).to(self.device)
        self.lr = lr if isinstance(lr, torch.Tensor) else torch.tensor([float(lr)], device=self.device)
        self.steps = torch.zeros(2, dtype=torch.int32, device=self.device) if step is None else step
        for what, t, dt, cnt in (("lr", self.lr, torch.float32, 1), ("step", self.steps, torch.int32, 2)):
            if t.device != self.device or t.dtype != dt or t.numel() != cnt or not t.is_contiguous():
                raise ValueError(f"{what} must be a {dt} tensor of {cnt} on {self.device}")
        if not max_norm >= 0.0:
            raise ValueError("max_norm must not be negative")
        self.max_norm = float(max_norm)
        self.norm = torch.zeros(4, device=self.device)
        self.ws = torch.empty(biv.biv_grad_norm_workspace(self.chunks), dtype=torch.uint8, device=self.device)
        d = biv.AdamWDesc()
        d.tensors, d.n, d.chunks, d.kinds = self.table.data_ptr(), n, self.chunks, kinds
        d.lr, d.step = self.lr.data_ptr(), self.steps.data_ptr()
        d.clip = self.norm.data_ptr() if self.max_norm > 0 else None
        d.beta1, d.beta2, d.eps = float(betas[0]), float(betas[1]), float(eps)
        d.rounding = biv.ROUND_STOCHASTIC if rounding == "stochastic" else biv.ROUND_NEAREST
        d.seed = int(seed) & 0xFFFFFFFFFFFFFFFF
        self.desc = d
        # what was made here is ready for a step on any stream
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream().synchronize()

    def set_lr(self, lr: float):
        """A new learning rate for the steps (and graph replays) issued after this."""
        self.lr.fill_(float(lr))

    def step(self, stream=None):
        """One update of every tensor from its gradient."""
        if biv._device() != self.device.index:
            raise ValueError(f"step() runs on the optimizer's device, {self.device}")
        if self.max_norm > 0:
            biv.biv_grad_norm(self.table, self.n, self.chunks, self.max_norm, self.norm, self.ws, stream=stream)
        biv.biv_adamw(self.desc, stream=stream)
