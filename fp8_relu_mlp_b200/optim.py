"""AdamW over a model's tensors: buffers and the two library calls of a step.

One step is the norm of all gradients with the clip coefficient
(``fp8mlp_grad_norm``, when ``max_norm`` is given) and one pass over all
tensors (``fp8mlp_adamw_step``): every weight, its BF16 copy, gradient and
moments are read and written once.  Moments are fp32 or, with
``state_bits=8``, e4m3 codes with a scale for each block of 128 (2.06 bytes
per element in place of 8).  Nothing is read back to the host, so a step can
be captured into a CUDA graph; lr, the step count and the seed live on the
device.
"""
from __future__ import annotations

import math
from bisect import bisect

import torch

from . import _abi as A
from ._order import after_current, as_stream, used_on


class AdamW:
    """With a ``stream`` of its own, what the optimizer launches waits for the
    current stream's work so far; nothing waits for the optimizer but
    ``set_lr`` and ``read_state``, and a capture is made on that stream.
    Parameters may be added between steps; a
    step captured before goes on with the parameters that it had."""

    def __init__(self, state_bits: int = 32, lr: float = 1e-3, betas=(0.9, 0.95), eps: float = 1e-8, seed: int = 0,
                 max_norm: float | None = None, step_count: int = 0, device="cuda", stream=None):
        if state_bits not in (32, 8):
            raise ValueError("state_bits must be 32 or 8")
        if max_norm is not None and not max_norm > 0:
            raise ValueError("max_norm must be > 0")
        if not (0 <= betas[0] < 1 and 0 <= betas[1] < 1 and eps > 0):
            raise ValueError("betas must be in [0, 1) and eps > 0")
        self.state_bits, self.betas, self.eps, self.max_norm = state_bits, tuple(betas), eps, max_norm
        self.device, self.stream = torch.device(device), stream
        self._moments = (torch.float32,) if state_bits == 32 else (torch.float8_e4m3fn, torch.uint8)  # codes as bytes too
        self.entries = []  # the tensors of each parameter: the descriptors hold their addresses
        self._descriptors = []
        self._plan = self._workspace = None
        self._outgrown = []  # workspaces that steps under way or captured ones may still use
        self._first, self._behind = [], []  # addresses of every tensor's first byte, in order, and behind its last
        self.state = torch.empty(8, dtype=torch.int32, device=self.device)  # fp8mlp_adamw_state (32 bytes)
        self.norm = torch.zeros(2, dtype=torch.float32, device=self.device)  # gradient norm, clip coefficient
        self._coef = self.norm[1:]
        self._settle()
        A.fp8mlp_adamw_state_init(self.state, lr, seed & 0xFFFFFFFF, step_count, stream)

    def add(self, grad, master=None, weight=None, weight_decay: float = 0.0, lr_mult: float = 1.0, state=None) -> dict:
        """One parameter: ``grad`` fp32; ``master`` fp32 weights and / or
        ``weight`` the BF16 weights (a copy where there is a master, else the
        weights themselves, rounded stochastically).  ``state`` may bring the
        moments (``m``, ``v`` and with 8 bits ``m_scale``, ``v_scale``); else
        they are allocated and start at zero.  Returns the entry."""
        n = grad.numel()
        if grad.dtype != torch.float32:
            raise ValueError("grad must be fp32")
        if master is None and weight is None:
            raise ValueError("master or weight is needed")
        if master is not None and (master.dtype != torch.float32 or master.numel() != n):
            raise ValueError("master must be fp32 of the gradient's size")
        if weight is not None and (weight.dtype != torch.bfloat16 or weight.numel() != n):
            raise ValueError("weight must be bf16 of the gradient's size")
        if state is None:
            if self.state_bits == 32:
                state = {k: torch.zeros(n, dtype=torch.float32, device=grad.device) for k in ("m", "v")}
            else:
                state = {k: torch.zeros(n, dtype=torch.float8_e4m3fn, device=grad.device) for k in ("m", "v")}
                state.update({k: torch.ones(-(-n // 128), dtype=torch.float32, device=grad.device)
                              for k in ("m_scale", "v_scale")})
        if state["m"].dtype not in self._moments or state["v"].dtype not in self._moments:
            raise ValueError(f"the moments must have {self.state_bits} bits: {' or '.join(map(str, self._moments))}")
        if self.state_bits == 8:
            if state.get("m_scale") is None or state.get("v_scale") is None:
                raise ValueError("8-bit moments need m_scale and v_scale")
            if state["m_scale"].dtype != torch.float32 or state["v_scale"].dtype != torch.float32:
                raise ValueError("m_scale and v_scale must be fp32")
        e = dict(grad=grad, master=master, weight=weight, **state)
        firsts, behinds = self._first, self._behind
        added = []  # this parameter's, taken back where it is refused
        try:
            for t in e.values():
                if t is None:
                    continue
                first = t.data_ptr()
                behind = first + t.nbytes
                if first == behind:
                    continue
                i = bisect(firsts, first)
                if (i and behinds[i - 1] > first) or (i < len(firsts) and firsts[i] < behind):
                    raise ValueError("a tensor is given twice, or overlaps another: one step updates each weight once")
                firsts.insert(i, first)
                behinds.insert(i, behind)
                added.append(first)
            self._descriptors.append(A.adamw_tensor(
                n, master, weight, grad, state["m"], state["v"], state.get("m_scale"), state.get("v_scale"), lr_mult,
                weight_decay, self.state_bits))
        except Exception:
            for first in added:
                i = bisect(firsts, first) - 1
                del firsts[i], behinds[i]
            raise
        self.entries.append(e)
        self._plan = None
        return e

    def _settle(self):
        """Buffers are filled on the current stream; a step on a stream of its
        own must not overtake that."""
        if self.stream is not None:
            after_current(self.stream, self.device)

    def _finish(self):
        """Steps on a stream of its own come to their end."""
        if self.stream is not None:
            as_stream(self.stream, self.device).synchronize()

    def set_lr(self, lr: float):
        """For the steps from here on (a device write on the current stream;
        also between replays of a captured step).  Waits for the steps before
        where the optimizer has a stream of its own."""
        if not isinstance(lr, torch.Tensor) and not math.isfinite(lr):
            raise ValueError("lr must be finite")
        self._finish()
        self.state[:1].view(torch.float32).fill_(lr)
        self._settle()

    def _replan(self):
        self._plan = A.adamw_tensors(self._descriptors)
        if self.max_norm is not None:
            need = A.fp8mlp_grad_norm_workspace_size(self._plan)
            if self._workspace is None or self._workspace.numel() < need:
                if self._workspace is not None:
                    self._outgrown.append(self._workspace)
                    need = max(need, 2 * self._workspace.numel())
                self._workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
        if self.stream is not None:
            # freed while a step is under way, their memory waits for it
            used_on(self.stream, self.device, [self.state, self.norm, self._workspace],
                    *(e.values() for e in self.entries))

    def step(self):
        if self._plan is None:
            self._replan()
        self._settle()
        coef = None
        if self.max_norm is not None:
            A.fp8mlp_grad_norm(self._plan, self.max_norm, self.norm, self._workspace, self.stream)
            coef = self._coef
        A.fp8mlp_adamw_step(self._plan, self.state, self.state_bits, *self.betas, self.eps, coef, self.stream)

    def read_state(self) -> dict:
        self._finish()
        s = self.state.cpu()
        return dict(lr=float(s.view(torch.float32)[0]), step=int(s[1]), seed=int(s[2]) & 0xFFFFFFFF,
                    skipped=int(s[4]))
