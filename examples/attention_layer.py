"""A sequence-parallel attention layer with 8-bit projections, trained for a few
steps: residual + norm + packed QKV projection, seq -> head re-layout,
attention, head -> seq re-layout, output projection, and a step of AdamW.  After the
training the weights are rounded to 8 bits once, and the layer runs without gradients.

    python examples/attention_layer.py [--workload qwen1.5-1.8b_B2_S16384] [--seq 2048] [--steps 3]
                                       [--norm layer] [--window 512 --sinks 4] [--state-bits 8]

The tokens of all virtual ranks lie back to back (the seq-sharded buffer of
include/basp.h), and norm and projections work on each token by itself, so
they take the buffer as it is.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sequence_re_layout_gb300 as basp                      # noqa: E402
from sequence_re_layout_gb300 import autograd, fp8, optim      # noqa: E402
from sequence_re_layout_gb300.workloads import WORKLOADS     # noqa: E402


class AttentionLayer(torch.nn.Module):
    """``forward(x, residual) -> (out, h)`` for x, residual [B * S, hidden] in
    seq-sharded order; h is the residual stream after the layer's addition.  ``norm``
    is "rms" or "layer"; ``window`` and ``sinks`` are those of the causal attention."""

    def __init__(self, layout, hidden, dtype=torch.bfloat16, causal=True, norm="rms", window=None, sinks=0):
        super().__init__()
        i = layout.info
        self.layout, self.causal, self.frozen = layout, causal, None
        self.mask = {"window": window, "sinks": sinks}
        q, packed = i["Hq"] * i["d"], (i["Hq"] + 2 * i["Hkv"]) * i["d"]
        self.norm = torch.nn.Parameter(torch.ones(hidden, dtype=dtype, device="cuda"))
        self.norm_bias = torch.nn.Parameter(torch.zeros_like(self.norm)) if norm == "layer" else None
        self.wqkv = torch.nn.Parameter(torch.randn(packed, hidden, device="cuda") * hidden ** -0.5)
        self.bqkv = torch.nn.Parameter(torch.zeros(packed, dtype=dtype, device="cuda"))
        self.wo = torch.nn.Parameter(torch.randn(hidden, q, device="cuda") * q ** -0.5)

    def forward(self, x, residual):
        i = self.layout.info
        wqkv, wo = self.frozen or (self.wqkv, self.wo)
        if self.norm_bias is None:
            qkv, h = autograd.rmsnorm_linear_fp8(x, self.norm, wqkv, self.bqkv, residual=residual)
        else:
            qkv, h = autograd.layernorm_linear_fp8(x, self.norm, self.norm_bias, wqkv, self.bqkv, residual=residual)
        # [N ranks x Bg sequences, S, heads of one rank, d]: attention is local to a rank
        heads = [t.view(i["N"] * i["seqs_per_group"], i["S"], -1, i["d"])
                 for t in autograd.seq2head_qkv(self.layout, qkv)]
        if self.causal:
            o = autograd.attention(*heads, **self.mask)
        else:
            o = torch.nn.functional.scaled_dot_product_attention(*(t.transpose(1, 2) for t in heads),
                                                                 enable_gqa=i["Hq"] != i["Hkv"]).transpose(1, 2)
        o = autograd.head2seq(self.layout, o.reshape(-1))
        return autograd.linear_fp8(o.view(-1, i["Hq"] * i["d"]), wo), h

    @torch.no_grad()
    def freeze(self):
        """The weights in 8 bits, once, for calls under no_grad."""
        self.frozen = tuple(fp8.quantize(w, block_rows=fp8.BLOCK) for w in (self.wqkv, self.wo))


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--workload", default="qwen1.5-1.8b_B2_S16384", choices=sorted(WORKLOADS))
    p.add_argument("--seq", type=int, default=2048, help="tokens of a sequence (the workload's heads are kept)")
    p.add_argument("--steps", type=int, default=3)
    p.add_argument("--norm", choices=("rms", "layer"), default="rms")
    p.add_argument("--window", type=int, help="keys that a query sees (all if not given)")
    p.add_argument("--sinks", type=int, default=0, help="first keys that stay visible")
    p.add_argument("--state-bits", type=int, choices=(8, 32), default=32, help="of the optimiser")
    a = p.parse_args()
    w = WORKLOADS[a.workload]
    torch.manual_seed(0)
    with basp.Layout(w.B, a.seq, w.Hq, w.Hkv, w.d, w.N, w.K_basp, "bf16") as layout:
        hidden = w.Hq * w.d
        layer = AttentionLayer(layout, hidden, norm=a.norm, window=a.window, sinks=a.sinks)
        optimizer = optim.AdamW(layer.parameters(), lr=0.002, weight_decay=0.0, state_bits=a.state_bits)
        x, residual, target = (torch.randn(w.B * a.seq, hidden, device="cuda").bfloat16() for _ in range(3))
        for step in range(a.steps):
            out, h = layer(x, residual)
            loss = (out + h - target).float().square().mean()
            optimizer.zero_grad(set_to_none=True)
            loss.backward()
            optimizer.step()
            print("step %d: loss %.5f" % (step, loss.item()))
        layer.freeze()
        with torch.no_grad():
            out, h = layer(x, residual)
        print("without gradients: loss %.5f" % (out + h - target).float().square().mean().item())


if __name__ == "__main__":
    main()
