"""AdamW over the tensors of a quantisation-aware training run, on ``bcjr_adamw_step``.

``AdamW(params, state_bits=8)`` keeps the moments in 2.06 bytes a weight in place of 8: e4m3 codes in
blocks of 32 with a power of two each, rounded by a dither that a hash of the weight's place, the step
and ``seed`` gives, so runs repeat bit for bit. All tensors go through one launch (of up to 96).
Latent weights belong in fp32: bf16 and fp16 params are rounded to nearest at each step.
"""
from __future__ import annotations

import torch

from . import bcjr


class AdamW:
    """Decoupled weight decay: p -= lr (weight_decay p + m_hat / (sqrt(v_hat) + eps)).

    ``params`` are contiguous CUDA tensors of one type on one device, updated in place by ``step``.
    They stay this object's for good: it reads their addresses anew at each step, but their number
    and sizes are fixed. ``lr``, ``betas``, ``eps`` and ``weight_decay`` may be changed between steps.
    """

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 1e-2, state_bits: int = 32, seed: int = 0):
        self.params = list(params)
        if not self.params:
            raise ValueError("no params")
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32, got {state_bits}")
        for i, p in enumerate(self.params):
            bcjr._spec(p, f"params[{i}]", self.params[0].dtype, None)
            bcjr._dtype_code(p, f"params[{i}]")
        dev = bcjr._device(*self.params)
        self.lr, self.betas, self.eps, self.weight_decay = lr, tuple(betas), eps, weight_decay
        self.state_bits, self.seed, self.steps = state_bits, int(seed), 0
        self._first = [0]
        for p in self.params:
            self._first.append(self._first[-1] + bcjr.bcjr_adamw_state_numel([p.numel()]))
        total = self._first[-1]
        if state_bits == 32:
            self.exp_avg, self.exp_avg_sq = (torch.zeros(total, dtype=torch.float32, device=dev) for _ in range(2))
            self.avg_scale = self.avg_sq_scale = None
        else:
            self.exp_avg, self.exp_avg_sq = (torch.zeros(total, dtype=torch.uint8, device=dev).view(bcjr.E4M3) for _ in range(2))
            self.avg_scale, self.avg_sq_scale = (
                torch.zeros(total // bcjr.MOMENT_BLOCK, dtype=torch.uint8, device=dev) for _ in range(2))

    def step(self, grads=None):
        """One step with these gradients, or with the params' own ``.grad``. The step's number is part of
        the formula, so a step cannot be captured into a graph, whose replays would repeat it."""
        grads = [p.grad for p in self.params] if grads is None else list(grads)
        for i, g in enumerate(grads):
            if g is None:
                raise ValueError(f"params[{i}] has no gradient")
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("AdamW.step counts its steps on the host and cannot be captured")
        bcjr.bcjr_adamw_step(self.params, grads, self.exp_avg, self.exp_avg_sq, self.avg_scale, self.avg_sq_scale,
                             step=self.steps + 1, lr=self.lr, beta1=self.betas[0], beta2=self.betas[1], eps=self.eps,
                             weight_decay=self.weight_decay, seed=self.seed)
        self.steps += 1

    def moments(self, i: int):
        """The first and second moments of params[i] as fp32 tensors of its shape."""
        p = self.params[i]
        o, end = self._first[i], self._first[i + 1]
        if self.state_bits == 32:
            m, v = self.exp_avg[o:end].clone(), self.exp_avg_sq[o:end].clone()
        else:
            block = slice(o // bcjr.MOMENT_BLOCK, end // bcjr.MOMENT_BLOCK)
            m, r = (torch.ldexp(t[o:end].float().view(-1, bcjr.MOMENT_BLOCK), s[block].int()[:, None] - 127).view(-1)
                    for t, s in ((self.exp_avg, self.avg_scale), (self.exp_avg_sq, self.avg_sq_scale)))
            v = r.square()
        return m[:p.numel()].view(p.shape), v[:p.numel()].view(p.shape)

    def state_dict(self) -> dict:
        """Everything a run needs to go on bit for bit, as tensors of its own and plain numbers."""
        keep = {k: getattr(self, k).clone() for k in ("exp_avg", "exp_avg_sq", "avg_scale", "avg_sq_scale")
                if getattr(self, k) is not None}
        return {"steps": self.steps, "state_bits": self.state_bits, "seed": self.seed, "lr": self.lr, "betas": self.betas,
                "eps": self.eps, "weight_decay": self.weight_decay, "numels": [p.numel() for p in self.params], **keep}

    def load_state_dict(self, state: dict) -> None:
        if state["state_bits"] != self.state_bits or list(state["numels"]) != [p.numel() for p in self.params]:
            raise ValueError("the state is of other tensors or another number of bits")
        for k in ("exp_avg", "exp_avg_sq", "avg_scale", "avg_sq_scale"):
            if getattr(self, k) is not None:
                if state[k].shape != getattr(self, k).shape or state[k].dtype != getattr(self, k).dtype:
                    raise ValueError(f"{k} of the state has another shape or type")
        for k in ("exp_avg", "exp_avg_sq", "avg_scale", "avg_sq_scale"):
            if getattr(self, k) is not None:
                getattr(self, k).view(torch.uint8).copy_(state[k].view(torch.uint8))
        self.steps, self.seed, self.lr, self.betas = int(state["steps"]), int(state["seed"]), state["lr"], tuple(state["betas"])
        self.eps, self.weight_decay = state["eps"], state["weight_decay"]
