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

import struct

import torch

from . import capi
from .boundary import cuda_device

QBLOCK = 128
F8, BF16, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32

# the argument structs of include/mhc_sublayer.h (native sizes and alignment)
NORM_ARGS = struct.Struct("@iiPqPqPfPPPP")
QUANTIZE_ARGS = struct.Struct("@iiPqPPP")
MATMUL_ARGS = struct.Struct("@iiiPqPqPqPPqi")
MOE_ARGS = struct.Struct("@iPPPPPPPPPP")


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
        self.device = cuda_device(device)
        scores = {"softmax": capi.MHC_SCORE_SOFTMAX, "sigmoid": capi.MHC_SCORE_SIGMOID}
        if score not in scores:
            raise ValueError(f"score: expected one of {sorted(scores)}, got {score!r}")
        flags = ((capi.MHC_SUBLAYER_FP8 if fp8 else 0) | (capi.MHC_SUBLAYER_RENORMALIZE if renormalize else 0)
                 | (capi.MHC_SUBLAYER_ROUTER_F32 if router_f32 else 0))
        self.config = capi.mhc_sublayer_config_t(hidden, intermediate, experts, shared_experts, top_k,
                                                 max_moe_tokens, scores[score], routed_scale, flags)
        self.hidden, self.intermediate, self.experts, self.shared = hidden, intermediate, experts, shared_experts
        self.top_k, self.fp8, self.router_f32 = top_k, fp8, router_f32
        self._index = self.device.index
        lib = capi.sublayer_calls()
        self._norm, self._quantize, self._swiglu = lib["add_rms_norm"], lib["quantize"], lib["swiglu"]
        self._matmul, self._moe = lib["matmul"], lib["moe"]
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

    # A call's checks run on every call, beside kernels of a few microseconds, so
    # they are written for their own time: one test a tensor for the usual case,
    # the message in a function that only a refusal reaches, the arguments packed
    # in one step.
    def _ptr(self, name: str, t: torch.Tensor, dtype, shape: tuple) -> int:
        """Pointer of a dense tensor."""
        if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != self._index:
            self._refuse(name, t, dtype, shape, "contiguous ")
        return t.data_ptr()

    def _stride(self, name: str, t: torch.Tensor, dtype, shape: tuple) -> int:
        """Row stride of a matrix with contiguous rows."""
        if t.dtype is not dtype or t.shape != shape or t.get_device() != self._index:
            self._refuse(name, t, dtype, shape, "")
        if t.is_contiguous() and shape[0] > 1:
            return shape[1]
        if shape[1] > 1 and t.stride(1) != 1:
            self._refuse(name, t, dtype, shape, "contiguous rows, ")
        # a single row's stride is never used: give one that suits every type
        return t.stride(0) if shape[0] > 1 else -(-shape[1] // 16) * 16

    def _refuse(self, name: str, t: torch.Tensor, dtype, shape: tuple, what: str) -> None:
        if t.device != self.device:
            raise ValueError(f"{name} must be a tensor on {self.device}, got {t.device}")
        raise ValueError(f"{name}: expected {what}{dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)} "
                         f"strides {t.stride()}")

    def _call(self, fn, args: bytes, stream) -> None:
        """One library call: `args` is its argument struct, laid out as in C."""
        if stream is None:
            stream = torch._C._cuda_getCurrentRawStream(self._index)
        elif isinstance(stream, torch.cuda.Stream):
            stream = stream.cuda_stream
        status = fn(self.handle, args, stream)
        if status:
            capi._check_sublayer(status, self.handle)

    @staticmethod
    def _unknown(outputs: dict, allowed: tuple) -> None:
        for name in outputs:
            if name not in allowed:
                raise ValueError(f"unknown output {name!r}: expected some of {allowed}")

    # ---------------------------------------------------------------- calls
    def add_rms_norm(self, inputs: dict, outputs: dict, *, eps: float = 1e-6, stream=None) -> dict:
        """r = x + residual; y = r * rsqrt(mean(r^2) + eps) * norm_weight.
        inputs: x [m][h], norm_weight [h] and optionally residual [m][h];
        outputs: some of residual_out (r), output (y), values with scales (y
        in 8 bits)."""
        x, weight, residual = inputs["x"], inputs["norm_weight"], inputs.get("residual")
        shape = x.shape
        m, h = shape
        x_stride = self._stride("x", x, BF16, shape)
        res = res_stride = 0
        if residual is not None:
            res_stride = self._stride("residual", residual, BF16, shape)
            res = residual.data_ptr()
        gamma = self._ptr("norm_weight", weight, BF16, (h,))
        get, ptr, blocks = outputs.get, self._ptr, (m, (h + 127) // 128)
        r, y, v, s = get("residual_out"), get("output"), get("values"), get("scales")
        rp = 0 if r is None else ptr("residual_out", r, BF16, shape)
        yp = 0 if y is None else ptr("output", y, BF16, shape)
        vp = 0 if v is None else ptr("values", v, F8, shape)
        sp = 0 if s is None else ptr("scales", s, F32, blocks)
        if len(outputs) != (r is not None) + (y is not None) + (v is not None) + (s is not None):
            self._unknown(outputs, ("residual_out", "output", "values", "scales"))
        self._call(self._norm, NORM_ARGS.pack(m, h, x.data_ptr(), x_stride, res, res_stride, gamma, eps, rp, yp, vp, sp),
                   stream)
        return outputs

    def quantize(self, inputs: dict, outputs: dict, *, stream=None) -> dict:
        """x [m][h] BF16 to 8 bits: values, scales."""
        x, values, scales = inputs["x"], outputs["values"], outputs["scales"]
        shape = x.shape
        m, h = shape
        stride = self._stride("x", x, BF16, shape)
        v = self._ptr("values", values, F8, shape)
        s = self._ptr("scales", scales, F32, (m, (h + 127) // 128))
        if len(outputs) != 2:
            self._unknown(outputs, ("values", "scales"))
        self._call(self._quantize, QUANTIZE_ARGS.pack(m, h, x.data_ptr(), stride, 0, v, s), stream)
        return outputs

    def swiglu(self, inputs: dict, outputs: dict, *, stream=None) -> dict:
        """silu(gate) * up of gate_up [m][2h] (gate, then up) to 8 bits:
        values, scales and optionally output (BF16)."""
        x, values, scales, out = inputs["gate_up"], outputs["values"], outputs["scales"], outputs.get("output")
        m, h2 = x.shape
        h = h2 // 2
        stride = self._stride("gate_up", x, BF16, (m, 2 * h))
        v = self._ptr("values", values, F8, (m, h))
        s = self._ptr("scales", scales, F32, (m, (h + 127) // 128))
        o = 0 if out is None else self._ptr("output", out, BF16, (m, h))
        if len(outputs) != (2 if out is None else 3):
            self._unknown(outputs, ("output", "values", "scales"))
        self._call(self._swiglu, QUANTIZE_ARGS.pack(m, h, x.data_ptr(), stride, o, v, s), stream)
        return outputs

    def matmul(self, inputs: dict, outputs: dict, *, stream=None) -> dict:
        """output [m][n] (BF16 or FP32, by its dtype) = (values * scales)
        (weight * weight_scales)^T: values [m][k] and weight [n][k] in 8 bits,
        scales [m][ceil(k/128)], weight_scales [ceil(n/128)][ceil(k/128)]."""
        values, weight, out = inputs["values"], inputs["weight"], outputs["output"]
        scales, weight_scales = inputs["scales"], inputs["weight_scales"]
        m, k = values.shape
        n, kb = weight.shape[0], (k + 127) // 128
        v_stride = self._stride("values", values, F8, (m, k))
        s_stride = self._stride("scales", scales, F32, (m, kb))
        w_stride = self._stride("weight", weight, F8, (n, k))
        ws = self._ptr("weight_scales", weight_scales, F32, ((n + 127) // 128, kb))
        dtype = out.dtype
        if dtype is not BF16 and dtype is not F32:
            raise ValueError(f"output: expected {BF16} or {F32}, got {dtype}")
        o_stride = self._stride("output", out, dtype, (m, n))
        if len(outputs) != 1:
            self._unknown(outputs, ("output",))
        self._call(self._matmul, MATMUL_ARGS.pack(m, n, k, values.data_ptr(), v_stride, scales.data_ptr(), s_stride,
                                                  weight.data_ptr(), w_stride, ws, out.data_ptr(), o_stride,
                                                  dtype is F32), stream)
        return outputs

    def moe(self, inputs: dict, outputs: dict, *, stream=None) -> dict:
        """One MoE layer over x [m][H] BF16, m up to max_moe_tokens.  inputs:
        x, router [E][H], optionally bias [E] (added for the selection only),
        gate_up [E+S][2I][H], down [E+S][H][I] and, with fp8, gate_up_scales
        [E+S][2][ceil(I/128)][ceil(H/128)] and down_scales
        [E+S][ceil(H/128)][ceil(I/128)]; outputs: output [m][H] BF16 and
        optionally idx [m][top_k] int32 and weights [m][top_k] FP32."""
        x, bias = inputs["x"], inputs.get("bias")
        m, H, I, E, every = x.shape[0], self.hidden, self.intermediate, self.experts, self.experts + self.shared
        xp = self._ptr("x", x, BF16, (m, H))
        router = self._ptr("router", inputs["router"], F32 if self.router_f32 else BF16, (E, H))
        bp = 0 if bias is None else self._ptr("bias", bias, F32, (E,))
        wt = F8 if self.fp8 else BF16
        gate_up = self._ptr("gate_up", inputs["gate_up"], wt, (every, 2 * I, H))
        down = self._ptr("down", inputs["down"], wt, (every, H, I))
        gs = ds = 0
        if self.fp8:
            hb, ib = (H + 127) // 128, (I + 127) // 128
            gs = self._ptr("gate_up_scales", inputs["gate_up_scales"], F32, (every, 2, ib, hb))
            ds = self._ptr("down_scales", inputs["down_scales"], F32, (every, hb, ib))
        out, idx, weights = outputs["output"], outputs.get("idx"), outputs.get("weights")
        op = self._ptr("output", out, BF16, (m, H))
        ip = 0 if idx is None else self._ptr("idx", idx, torch.int32, (m, self.top_k))
        wp = 0 if weights is None else self._ptr("weights", weights, F32, (m, self.top_k))
        if len(outputs) != 1 + (idx is not None) + (weights is not None):
            self._unknown(outputs, ("output", "idx", "weights"))
        self._call(self._moe, MOE_ARGS.pack(m, xp, router, bp, gate_up, gs, down, ds, op, ip, wp), stream)
        return outputs

    def check_errors(self) -> None:
        capi.mhc_sublayer_check_errors(self.handle)
