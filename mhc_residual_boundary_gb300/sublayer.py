"""PyTorch-facing wrapper of the operators between two boundaries
(include/mhc_sublayer.h): norm with the residual's addition, 8-bit
quantisers, block-scaled 8-bit products, and a whole MoE layer for a few
tokens.

Like Boundary: the wrapper checks shapes, dtypes and devices and passes raw
pointers; all arithmetic runs in the CUDA kernels.  Calls take a dict of
input tensors and a dict of output tensors (see empty_outputs) and return
the latter; an optional output that the dict lacks is not computed.
"""
from __future__ import annotations

import torch

from . import capi

QBLOCK = 128
F8, BF16, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32


def scale_blocks(n: int) -> int:
    """Scales of a row of n 8-bit values."""
    return (n + QBLOCK - 1) // QBLOCK


class Sublayer:
    """The operators between two boundaries on one GPU.

    With experts > 0 the handle also serves moe() for layers of that shape:
    hidden H, intermediate I, `experts` routed and `shared_experts` shared
    experts, top_k routes a token, up to max_moe_tokens tokens a call; fp8:
    8-bit expert weights with block scales (else BF16); score: "softmax" or
    "sigmoid"; renormalize: divide the chosen scores by their sum;
    router_f32: the router weight is FP32.

    The handle owns scratch that moe uses, so its calls run one after another:
    on one stream, or on streams that the caller orders."""

    def __init__(self, *, hidden: int = 0, intermediate: int = 0, experts: int = 0, shared_experts: int = 0,
                 top_k: int = 0, max_moe_tokens: int = 0, fp8: bool = True, score: str = "softmax",
                 renormalize: bool = True, routed_scale: float = 1.0, router_f32: bool = False, device=None):
        if device is None:
            device = torch.cuda.current_device()
        self.device = torch.device("cuda", int(torch.device("cuda", device).index
                                               if not isinstance(device, int) else device))
        scores = {"softmax": capi.MHC_SCORE_SOFTMAX, "sigmoid": capi.MHC_SCORE_SIGMOID}
        if score not in scores:
            raise ValueError(f"score: expected one of {sorted(scores)}, got {score!r}")
        flags = ((capi.MHC_SUBLAYER_FP8 if fp8 else 0) | (capi.MHC_SUBLAYER_RENORMALIZE if renormalize else 0)
                 | (capi.MHC_SUBLAYER_ROUTER_F32 if router_f32 else 0))
        self.config = capi.mhc_sublayer_config_t(hidden, intermediate, experts, shared_experts, top_k,
                                                 max_moe_tokens, scores[score], routed_scale, flags)
        self.hidden, self.intermediate, self.experts, self.shared = hidden, intermediate, experts, shared_experts
        self.top_k, self.fp8, self.router_f32 = top_k, fp8, router_f32
        self.handle = capi.mhc_sublayer_create(self.config, self.device.index)

    # ------------------------------------------------------------ lifecycle
    def close(self) -> None:
        if getattr(self, "handle", None):
            capi.mhc_sublayer_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    # -------------------------------------------------------------- helpers
    def empty_outputs(self, op: str, m: int, n: int = 0, *, dtype=BF16) -> dict:
        """Output tensors of an m-row call: n is the output's width (the
        handle's hidden size for "moe"), dtype the matmul's output type."""
        def new(shape, dt):
            return torch.empty(shape, dtype=dt, device=self.device)

        if op == "matmul":
            return {"output": new((m, n), dtype)}
        if op == "moe":
            return {"output": new((m, self.hidden), BF16), "idx": new((m, self.top_k), torch.int32),
                    "weights": new((m, self.top_k), F32)}
        out = {"values": new((m, n), F8), "scales": new((m, scale_blocks(n)), F32)}
        if op == "add_rms_norm":
            out["residual_out"] = new((m, n), BF16)
        if op in ("add_rms_norm", "swiglu"):
            out["output"] = new((m, n), BF16)
        elif op != "quantize":
            raise ValueError(f"unknown operator {op!r}")
        return out

    def _ptr(self, name: str, t: torch.Tensor, dtype, shape: tuple) -> int:
        """Pointer of a dense tensor."""
        if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name}: expected contiguous {dtype} {shape}, got {t.dtype} {tuple(t.shape)}")
        if t.device != self.device:
            raise ValueError(f"{name} must be a tensor on {self.device}, got {t.device}")
        return t.data_ptr()

    def _rows(self, name: str, t: torch.Tensor, dtype, shape: tuple) -> tuple:
        """(pointer, row stride) of a matrix with contiguous rows."""
        if t.dtype != dtype or t.shape != shape or (shape[1] > 1 and t.stride(1) != 1):
            raise ValueError(f"{name}: expected {dtype} {shape} with contiguous rows, got {t.dtype} {tuple(t.shape)} "
                             f"strides {t.stride()}")
        if t.device != self.device:
            raise ValueError(f"{name} must be a tensor on {self.device}, got {t.device}")
        # a single row's stride is never used: give the dense one
        return t.data_ptr(), t.stride(0) if shape[0] > 1 else -(-shape[1] // 16) * 16

    @staticmethod
    def _names(outputs: dict, allowed: tuple) -> None:
        for name in outputs:
            if name not in allowed:
                raise ValueError(f"unknown output {name!r}: expected some of {allowed}")

    # ---------------------------------------------------------------- calls
    def add_rms_norm(self, inputs: dict, outputs: dict, *, eps: float = 1e-6, stream=None) -> dict:
        """r = x + residual; y = r * rsqrt(mean(r^2) + eps) * norm_weight.
        inputs: x [m][h], norm_weight [h] and optionally residual [m][h];
        outputs: some of residual_out (r), output (y), values with scales (y
        in 8 bits)."""
        x = inputs["x"]
        m, h = x.shape
        a = capi.mhc_sublayer_norm_args_t()
        a.m, a.h, a.eps = m, h, eps
        a.x, a.x_stride = self._rows("x", x, BF16, (m, h))
        residual = inputs.get("residual")
        if residual is not None:
            a.residual, a.residual_stride = self._rows("residual", residual, BF16, (m, h))
        a.norm_weight = self._ptr("norm_weight", inputs["norm_weight"], BF16, (h,))
        self._names(outputs, ("residual_out", "output", "values", "scales"))
        self._quantized(a, outputs, m, h)
        for name in ("residual_out", "output"):
            if name in outputs:
                setattr(a, name, self._ptr(name, outputs[name], BF16, (m, h)))
        capi.mhc_sublayer_add_rms_norm(self.handle, a, stream)
        return outputs

    def _quantized(self, a, outputs: dict, m: int, h: int) -> None:
        if "values" in outputs:
            a.values = self._ptr("values", outputs["values"], F8, (m, h))
        if "scales" in outputs:
            a.scales = self._ptr("scales", outputs["scales"], F32, (m, scale_blocks(h)))

    def quantize(self, inputs: dict, outputs: dict, *, stream=None) -> dict:
        """x [m][h] BF16 to 8 bits: values, scales."""
        x = inputs["x"]
        m, h = x.shape
        a = capi.mhc_sublayer_quantize_args_t()
        a.m, a.h = m, h
        a.x, a.x_stride = self._rows("x", x, BF16, (m, h))
        self._names(outputs, ("values", "scales"))
        self._quantized(a, outputs, m, h)
        capi.mhc_sublayer_quantize(self.handle, a, stream)
        return outputs

    def swiglu(self, inputs: dict, outputs: dict, *, stream=None) -> dict:
        """silu(gate) * up of gate_up [m][2h] (gate, then up) to 8 bits:
        values, scales and optionally output (BF16)."""
        x = inputs["gate_up"]
        m, h = x.shape[0], x.shape[1] // 2
        a = capi.mhc_sublayer_quantize_args_t()
        a.m, a.h = m, h
        a.x, a.x_stride = self._rows("gate_up", x, BF16, (m, 2 * h))
        self._names(outputs, ("output", "values", "scales"))
        self._quantized(a, outputs, m, h)
        if "output" in outputs:
            a.output = self._ptr("output", outputs["output"], BF16, (m, h))
        capi.mhc_sublayer_swiglu(self.handle, a, stream)
        return outputs

    def matmul(self, inputs: dict, outputs: dict, *, stream=None) -> dict:
        """output [m][n] (BF16 or FP32, by its dtype) = (values * scales)
        (weight * weight_scales)^T: values [m][k] and weight [n][k] in 8 bits,
        scales [m][ceil(k/128)], weight_scales [ceil(n/128)][ceil(k/128)]."""
        values, weight, out = inputs["values"], inputs["weight"], outputs["output"]
        m, k = values.shape
        n = weight.shape[0]
        a = capi.mhc_sublayer_matmul_args_t()
        a.m, a.n, a.k = m, n, k
        a.values, a.values_stride = self._rows("values", values, F8, (m, k))
        a.scales, a.scales_stride = self._rows("scales", inputs["scales"], F32, (m, scale_blocks(k)))
        a.weight, a.weight_stride = self._rows("weight", weight, F8, (n, k))
        a.weight_scales = self._ptr("weight_scales", inputs["weight_scales"], F32, (scale_blocks(n), scale_blocks(k)))
        self._names(outputs, ("output",))
        if out.dtype not in (BF16, F32):
            raise ValueError(f"output: expected {BF16} or {F32}, got {out.dtype}")
        a.output_f32 = out.dtype == F32
        a.output, a.output_stride = self._rows("output", out, out.dtype, (m, n))
        capi.mhc_sublayer_matmul(self.handle, a, stream)
        return outputs

    def moe(self, inputs: dict, outputs: dict, *, stream=None) -> dict:
        """One MoE layer over x [m][H] BF16, m up to max_moe_tokens.  inputs:
        x, router [E][H], optionally bias [E] (added for the selection only),
        gate_up [E+S][2I][H], down [E+S][H][I] and, with fp8, gate_up_scales
        [E+S][2][ceil(I/128)][ceil(H/128)] and down_scales
        [E+S][ceil(H/128)][ceil(I/128)]; outputs: output [m][H] BF16 and
        optionally idx [m][top_k] int32 and weights [m][top_k] FP32."""
        x = inputs["x"]
        m, H, I, E, S = x.shape[0], self.hidden, self.intermediate, self.experts, self.shared
        a = capi.mhc_sublayer_moe_args_t()
        a.m = m
        a.x = self._ptr("x", x, BF16, (m, H))
        a.router = self._ptr("router", inputs["router"], F32 if self.router_f32 else BF16, (E, H))
        if inputs.get("bias") is not None:
            a.bias = self._ptr("bias", inputs["bias"], F32, (E,))
        wt = F8 if self.fp8 else BF16
        a.gate_up = self._ptr("gate_up", inputs["gate_up"], wt, (E + S, 2 * I, H))
        a.down = self._ptr("down", inputs["down"], wt, (E + S, H, I))
        if self.fp8:
            hb, ib = scale_blocks(H), scale_blocks(I)
            a.gate_up_scales = self._ptr("gate_up_scales", inputs["gate_up_scales"], F32, (E + S, 2, ib, hb))
            a.down_scales = self._ptr("down_scales", inputs["down_scales"], F32, (E + S, hb, ib))
        self._names(outputs, ("output", "idx", "weights"))
        a.output = self._ptr("output", outputs["output"], BF16, (m, H))
        if "idx" in outputs:
            a.idx = self._ptr("idx", outputs["idx"], torch.int32, (m, self.top_k))
        if "weights" in outputs:
            a.weights = self._ptr("weights", outputs["weights"], F32, (m, self.top_k))
        capi.mhc_sublayer_moe(self.handle, a, stream)
        return outputs

    def check_errors(self) -> None:
        capi.mhc_sublayer_check_errors(self.handle)
