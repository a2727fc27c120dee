"""AdamW over many tensors at once, over the C ABI of ``include/basp_optim.h``: one
launch for a few hundred tensors, states in 32 bits or in 8.

    optimizer = optim.AdamW(layer.parameters(), lr=3e-4, weight_decay=0.1, state_bits=8)
    loss.backward()
    optimizer.step()

8-bit states hold m and the root of v in e4m3 with a power-of-two scale for each 128
elements, rounded at random (2 bytes and a 64th an element instead of 8).
"""
from __future__ import annotations

import torch

from . import fp8


@torch.no_grad()
def adamw(params, grads, m, v, step, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, seed=0,
          numbers=None):
    """One step over lists of tensors, in place: params (bfloat16, float16 or
    float32), grads (their type or float32), and the states m and v: float32 tensors,
    or :class:`fp8.Quantized` of one row ([1, n]), v then the root of v.

    ``step`` counts from 1; as an int32 tensor of one element on the GPU it is read
    when the kernel runs, so that a captured step can be replayed; a list of those has
    one for each parameter.  The random rounding of 8-bit states depends on ``seed``,
    the step, the tensor's number (its place in the list, or ``numbers``) and each
    element's place alone.  Every tensor is dense, and none overlaps
    another: the same parameter twice is refused."""
    m, v = list(m), list(v)
    m_scales = v_scales = None
    if m and isinstance(m[0], fp8.Quantized):
        m, m_scales = _parts(m)
        v, v_scales = _parts(v)
    (fp8._ops or fp8._load()).adamw(list(params), list(grads), m, v, m_scales, v_scales, step, lr, betas[0], betas[1],
                                    eps, weight_decay, seed, numbers)


def _parts(states):
    if not all(isinstance(s, fp8.Quantized) and s.block_rows == 1 for s in states):
        raise ValueError("adamw: states must all be float32 tensors, or all fp8.Quantized with a scale for each row's 128")
    return [s.data for s in states], [s.scales for s in states]


class AdamW(torch.optim.Optimizer):
    """Adam with decoupled weight decay; parameters on the current GPU, dense.

    ``state_bits`` 32 or 8.  ``seed`` is that of the 8-bit states' rounding.  With
    ``capturable`` the numbers of the steps live on the GPU, so ``step()`` can be captured
    in a CUDA graph and replayed (with the lr and the other options of the capture),
    once a step has been taken; otherwise a capture is refused."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, state_bits=32, seed=0,
                 capturable=False):
        defaults = dict(lr=lr, betas=tuple(betas), eps=eps, weight_decay=weight_decay, state_bits=state_bits, seed=seed,
                        capturable=capturable)
        self._check(defaults)
        super().__init__(params, defaults)

    @staticmethod
    def _check(options):
        if options["state_bits"] not in (8, 32):
            raise ValueError("AdamW: state_bits must be 8 or 32, got %r" % (options["state_bits"],))
        if not (options["lr"] >= 0 and options["eps"] >= 0 and options["weight_decay"] >= 0 and
                len(options["betas"]) == 2 and all(0 <= b < 1 for b in options["betas"])):
            raise ValueError("AdamW: lr, eps and weight_decay must not be negative, betas two in [0, 1)")

    def add_param_group(self, param_group):
        """As torch's; a group's own options are checked as the constructor's are."""
        if isinstance(param_group, dict):
            self._check({**self.defaults, **param_group})
        super().add_param_group(param_group)

    def _init(self, p, group):
        state = self.state[p]
        state["step"] = torch.zeros(1, dtype=torch.int32, device=p.device) if group["capturable"] else 0
        for name in ("exp_avg", "exp_avg_sq" if group["state_bits"] == 32 else "exp_avg_sq_root"):
            if group["state_bits"] == 32:
                state[name] = torch.zeros(p.shape, dtype=torch.float32, device=p.device)
                continue
            state[name] = torch.zeros(1, p.numel(), dtype=torch.uint8, device=p.device).view(torch.float8_e4m3fn)
            state[name + "_scales"] = torch.full((1, -(-p.numel() // fp8.BLOCK)), 127, dtype=torch.uint8,
                                                 device=p.device).view(torch.float8_e8m0fnu)
        return state

    @torch.no_grad()
    def step(self, closure=None):
        """One step over every parameter that has a gradient.  Each parameter counts the
        steps that it takes itself, with or without ``capturable``."""
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        before = 0                                    # parameters of the groups before
        for group in self.param_groups:
            if not group["capturable"] and torch.cuda.is_current_stream_capturing():
                raise RuntimeError("AdamW: a captured step would keep its number: pass capturable=True")
            capturable = group["capturable"]
            together = {}                             # of each step's number, where it is known: (parameters, gradients, states, their numbers)
            for i, p in enumerate(group["params"]):
                g = p.grad
                if g is None:
                    continue
                s = self.state[p]
                if not s:
                    if torch.cuda.is_current_stream_capturing():
                        raise RuntimeError("AdamW: every replay of a captured first step would begin with new states: "
                                           "take a step before the capture")
                    s = self._init(p, group)
                number = None if capturable else s["step"]
                lists = together.get(number)
                if lists is None:
                    lists = together[number] = [], [], [], []
                lists[0].append(p)
                lists[1].append(g if g.is_contiguous() else g.contiguous())
                lists[2].append(s)
                lists[3].append(before + i)
            for lists in together.values():
                self._take(*lists, group)
            before += len(group["params"])
        return loss

    def _take(self, params, grads, states, numbers, group):
        if group["capturable"]:
            step = [s["step"] for s in states]
            torch._foreach_add_(step, 1)
        else:
            step = states[0]["step"] + 1
        if group["state_bits"] == 32:
            m, v, numbers = [s["exp_avg"] for s in states], [s["exp_avg_sq"] for s in states], None
        else:
            m, v = ([fp8.Quantized(s[n], s[n + "_scales"]) for s in states] for n in ("exp_avg", "exp_avg_sq_root"))
        adamw(params, grads, m, v, step, group["lr"], group["betas"], group["eps"], group["weight_decay"], group["seed"],
              numbers)
        if not group["capturable"]:
            for s in states:
                s["step"] = step

    def load_state_dict(self, state_dict):
        """As torch's, but states keep the types they were saved in."""
        super().load_state_dict(state_dict)
        numbers = [i for g in state_dict["param_groups"] for i in g["params"]]
        places = [(p, g) for g in self.param_groups for p in g["params"]]
        for i, (p, group) in zip(numbers, places):
            if i not in state_dict["state"]:
                continue
            state = {n: x.detach().to(p.device, copy=True) if torch.is_tensor(x) else x
                     for n, x in state_dict["state"][i].items()}
            count = int(state["step"])
            state["step"] = torch.full((1,), count, dtype=torch.int32, device=p.device) if group["capturable"] else count
            self.state[p] = state
