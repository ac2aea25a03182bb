"""The feed-forward half of a decoder's step on one GPU: two layers, one with a
dense MLP and one with a mixture of experts, boundaries between the sublayers,
and the output head.

    attention partials -> boundary -> quantize -> matmul -> swiglu -> matmul -> MLP output
            MLP output -> boundary -> moe ----------v
            MLP output -> boundary (the head's) -> add_rms_norm -> matmul -> logits

The MLP's output is the (only) partial of the next boundary, which adds it to
the residual streams and hands the next sublayer its normalised input.  The
last sublayer has no boundary behind it: its output is not spread over the
streams once more, but added, in the final norm, to what the head reads of them,
which the head's boundary takes from the streams as the MoE layer found them.  All
buffers are made once; a step is launches only, so it can be captured in a
CUDA graph.  The weights and the attention's partials are random.

    python examples/decoder_step.py [--tokens 8] [--hidden 5120] ...
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mhc_residual_boundary_gb300 import Boundary, Sublayer, synth  # noqa: E402

F8, BF16, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32


def blocks(n: int) -> int:
    return (n + 127) // 128


class DecoderStep:
    """One step of m tokens (m up to 32, as many as the MoE layer takes)."""

    def __init__(self, m: int, *, hidden: int, tp: int, mlp: int, intermediate: int, experts: int,
                 shared_experts: int, top_k: int, vocab: int, seed: int = 0):
        self.m, self.hidden, self.mlp, self.vocab = m, hidden, mlp, vocab
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        # the attention's output comes in `tp` partials, the MLPs' in one
        self.after_attention = Boundary(hidden=hidden, tp=tp, max_num_tokens=m, static_weight=True)
        self.after_mlp = Boundary(hidden=hidden, tp=1, max_num_tokens=m, static_weight=True)
        self.sub = Sublayer(hidden=hidden, intermediate=intermediate, experts=experts, shared_experts=shared_experts,
                            top_k=top_k, max_moe_tokens=m, score="sigmoid")

        # ---- weights
        every = experts + shared_experts
        self.gate_up, self.down = self.weight(2 * mlp, hidden), self.weight(hidden, mlp)
        self.head = self.weight(vocab, hidden)
        self.norm_weight = torch.ones(hidden, dtype=BF16, device="cuda")
        self.router = (self.randn(experts, hidden) / hidden ** 0.5).to(BF16)
        self.bias = 0.01 * self.randn(experts)
        experts_gu, scales_gu = zip(*(self.weight(2 * intermediate, hidden, halves=2) for _ in range(every)))
        experts_d, scales_d = zip(*(self.weight(hidden, intermediate) for _ in range(every)))
        self.experts = {"gate_up": torch.stack(experts_gu), "gate_up_scales": torch.stack(scales_gu),
                        "down": torch.stack(experts_d), "down_scales": torch.stack(scales_d)}

        # ---- the state a step starts from, and each boundary's parameters
        names = ("partials", "residual", "post", "comb", "hc_fn", "scale", "base", "norm_weight")
        drawn = [self.to_device(synth.make_inputs(hidden, tp if k == 0 else 1, m, seed=seed + k)) for k in range(3)]
        self.start = {n: drawn[0][n] for n in names}
        self.parameters = [{n: d[n] for n in ("hc_fn", "scale", "base", "norm_weight")} for d in drawn]

        # ---- buffers
        sub = self.sub
        self.at = [self.after_attention.empty_outputs(m), self.after_mlp.empty_outputs(m),
                   self.after_mlp.empty_outputs(m)]
        self.x8 = sub.empty_outputs("quantize", m, hidden)
        self.gate_up_out = sub.empty_outputs("matmul", m, 2 * mlp)
        self.h8 = sub.empty_outputs("swiglu", m, mlp)
        del self.h8["output"]   # only the 8-bit form is needed
        self.mlp_out = sub.empty_outputs("matmul", m, hidden)
        self.moe_out = sub.empty_outputs("moe", m)
        self.final = sub.empty_outputs("add_rms_norm", m, hidden)
        self.logits = sub.empty_outputs("matmul", m, vocab, dtype=F32)

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda")

    def weight(self, n: int, k: int, halves: int = 1):
        """A random 8-bit weight [n][k] of size 1 / sqrt(k) and its block scales; `halves`: gate and up
        each begin a new row of blocks."""
        w = (100 * self.randn(n, k)).clamp(-448, 448).to(F8)
        shape = (blocks(n), blocks(k)) if halves == 1 else (halves, blocks(n // halves), blocks(k))
        return w, torch.full(shape, 0.01 / k ** 0.5, device="cuda")

    @staticmethod
    def to_device(inputs: dict) -> dict:
        # 16-bit arrays hold BF16 bit patterns
        return {"norm_weight" if n == "gamma" else n: torch.from_numpy(a.view("int16")).view(BF16).cuda()
                if a.dtype == "uint16" else torch.from_numpy(a).cuda() for n, a in inputs.items()}

    def matmul(self, a: dict, weight: tuple, out: dict) -> None:
        self.sub.matmul({"values": a["values"], "scales": a["scales"], "weight": weight[0],
                         "weight_scales": weight[1]}, out)

    def boundary(self, k: int, partials: torch.Tensor) -> torch.Tensor:
        """Boundary k: the streams' state and a sublayer's partials in, the next sublayer's input out.  The first
        one begins from `start`, the others from the first."""
        state = self.start if k == 0 else {"residual": self.at[0]["residual_out"], "post": self.at[0]["post_out"],
                                           "comb": self.at[0]["comb_out"]}
        b = self.after_attention if k == 0 else self.after_mlp
        b.run({**state, **self.parameters[k], "partials": partials}, self.at[k])
        b.join()
        return self.at[k]["layer_input"]

    def step(self) -> torch.Tensor:
        sub = self.sub
        # a dense MLP
        x = self.boundary(0, self.start["partials"])
        sub.quantize({"x": x}, self.x8)
        self.matmul(self.x8, self.gate_up, self.gate_up_out)
        sub.swiglu({"gate_up": self.gate_up_out["output"]}, self.h8)
        self.matmul(self.h8, self.down, self.mlp_out)
        # a mixture of experts
        x = self.boundary(1, self.mlp_out["output"][None])
        sub.moe({"x": x, "router": self.router, "bias": self.bias, **self.experts}, self.moe_out)
        # the head: the streams that the MoE layer found, collapsed for the head, and its output, normalised
        x = self.boundary(2, self.mlp_out["output"][None])
        sub.add_rms_norm({"x": self.moe_out["output"], "residual": x, "norm_weight": self.norm_weight}, self.final)
        self.matmul(self.final, self.head, self.logits)
        return self.logits["output"]

    def capture(self) -> torch.cuda.CUDAGraph:
        self.step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        return graph

    def check_errors(self) -> None:
        for handle in (self.after_attention, self.after_mlp, self.sub):
            handle.check_errors()


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, default in (("tokens", 8), ("hidden", 5120), ("tp", 4), ("mlp", 10240), ("intermediate", 2048),
                          ("experts", 64), ("shared-experts", 1), ("top-k", 8), ("vocab", 32768), ("steps", 50)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args()
    model = DecoderStep(a.tokens, hidden=a.hidden, tp=a.tp, mlp=a.mlp, intermediate=a.intermediate,
                        experts=a.experts, shared_experts=a.shared_experts, top_k=a.top_k, vocab=a.vocab)
    graph = model.capture()
    for run, name in ((model.step, "calls"), (graph.replay, "graph")):
        for _ in range(3):
            run()
        torch.cuda.synchronize()
        begin = time.perf_counter()
        for _ in range(a.steps):
            run()
        torch.cuda.synchronize()
        print(f"{name}: {(time.perf_counter() - begin) / a.steps * 1e6:.1f} us a step of {a.tokens} tokens")
    model.check_errors()
    print("next tokens:", model.logits["output"].argmax(1).tolist())


if __name__ == "__main__":
    main()
