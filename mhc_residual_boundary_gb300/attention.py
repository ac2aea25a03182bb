"""PyTorch-facing wrapper of attention over a paged key-value cache
(include/mhc_attention.h): append (rotation by position, keys and values into
the cache) and attend (one new token of each sequence, or prompts and chunks
of them, causal, with an optional window and first positions that stay
visible).

Like Sublayer: the wrapper checks shapes, dtypes and devices and passes raw
pointers; all arithmetic runs in the CUDA kernels.  Calls take a dict of
input tensors and a dict of output tensors and return the latter.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import capi
from .boundary import cuda_device

F8, BF16, F32, I32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int32

# the argument structs of include/mhc_attention.h (native sizes and alignment)
APPEND_ARGS = struct.Struct("@iiPqPqPqPPPqPqPqPP")
ATTEND_ARGS = struct.Struct("@iiiiPqPPPqPqPqPPfiiPqP")


class Attention:
    """Attention of one layer shape on one GPU: `heads` query heads that share
    `kv_heads` key and value heads of head_dim 64 or 128, a cache of pages of
    page_size positions (16, 32, 64 or 128), BF16 or with fp8 in 8 bits.

    append rotates the first rotary_dim elements of a head: pair i by position *
    frequencies[i] (radians; default theta ** (-2 i / rotary_dim)), neighbouring
    elements with interleaved, else i and i + rotary_dim / 2.

    The handle owns scratch that attend uses, so its attend calls run one after
    another: on one stream, or on streams that the caller orders."""

    def __init__(self, *, heads: int, kv_heads: int, head_dim: int = 128, page_size: int = 64, fp8: bool = False,
                 rotary_dim: int = 0, theta: float = 10000.0, frequencies=None, interleaved: bool = False, device=None):
        self.device = cuda_device(device)
        flags = (capi.MHC_ATTENTION_FP8 if fp8 else 0) | (capi.MHC_ATTENTION_INTERLEAVED if interleaved else 0)
        values = None
        if frequencies is not None:
            values = [float(f) for f in frequencies]
            if len(values) != rotary_dim // 2:
                raise ValueError(f"frequencies: expected {rotary_dim // 2} values, got {len(values)}")
            values = (ctypes.c_double * len(values))(*values)
        self.config = capi.mhc_attention_config_t(heads, kv_heads, head_dim, page_size, rotary_dim, flags, theta, values)
        self.heads, self.kv_heads, self.head_dim, self.page_size, self.fp8 = heads, kv_heads, head_dim, page_size, fp8
        self._index = self.device.index
        self._page = kv_heads * page_size * head_dim
        self._cache_dtype, self._scale = F8 if fp8 else BF16, head_dim ** -0.5
        lib = capi.attention_calls()
        self._append, self._attend = lib["append"], lib["attend"]
        self.handle = capi.mhc_attention_create(self.config, self.device.index)

    # ------------------------------------------------------------ lifecycle
    def close(self) -> None:
        if getattr(self, "handle", None):
            capi.mhc_attention_destroy(self.handle)
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
    def empty_cache(self, pages: int) -> dict:
        """A cache of that many pages: k_cache, v_cache [pages][kv_heads]
        [page_size][head_dim] and, with fp8, k_scales, v_scales [pages]
        [kv_heads][page_size]."""
        shape = (pages, self.kv_heads, self.page_size)
        out = {name: torch.empty(*shape, self.head_dim, dtype=F8 if self.fp8 else BF16, device=self.device)
               for name in ("k_cache", "v_cache")}
        if self.fp8:
            out.update({name: torch.empty(shape, dtype=F32, device=self.device) for name in ("k_scales", "v_scales")})
        return out

    def empty_outputs(self, tokens: int) -> dict:
        """attend's outputs: output [tokens][heads][head_dim] BF16, lse [tokens][heads] FP32."""
        return {"output": torch.empty(tokens, self.heads, self.head_dim, dtype=BF16, device=self.device),
                "lse": torch.empty(tokens, self.heads, dtype=F32, device=self.device)}

    # The checks run on every call, beside kernels of a few microseconds: the usual
    # layout (dense caches, tokens whose heads are dense) passes one condition within the
    # call, everything else goes through the functions below, tensor by tensor, to an
    # argument or a refusal.
    def _ptr(self, name: str, t: torch.Tensor, dtype, shape: tuple) -> int:
        """Pointer of a dense tensor."""
        if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != self._index:
            self._refuse(name, t, dtype, shape, "contiguous ")
        return t.data_ptr()

    def _token_stride(self, name: str, t: torch.Tensor, tokens: int, heads: int) -> int:
        """Distance of two tokens of a [tokens][heads][head_dim] BF16 tensor whose tokens are dense."""
        d = self.head_dim
        if t.dtype is not BF16 or t.shape != (tokens, heads, d) or t.get_device() != self._index:
            self._refuse(name, t, BF16, (tokens, heads, d), "")
        stride, head, one = t.stride()
        if one != 1 or (heads > 1 and head != d):
            self._refuse(name, t, BF16, (tokens, heads, d), "dense tokens, ")
        return stride if tokens > 1 else heads * d   # a single token's stride is never used

    def _cache(self, name: str, t: torch.Tensor, pages: int) -> int:
        """Distance of two pages of a cache whose pages are dense."""
        shape, dtype = (pages, self.kv_heads, self.page_size, self.head_dim), F8 if self.fp8 else BF16
        if t.dtype is not dtype or t.shape != shape or t.get_device() != self._index:
            self._refuse(name, t, dtype, shape, "")
        if t.is_contiguous():
            return self._page
        if pages and not t[0].is_contiguous():
            self._refuse(name, t, dtype, shape, "dense pages, ")
        return t.stride(0) if pages > 1 else self._page

    def _scales(self, tensors: dict, pages: int) -> tuple:
        if not self.fp8:
            if "k_scales" in tensors or "v_scales" in tensors:
                raise ValueError("a BF16 cache has no scales")
            return 0, 0
        shape = (pages, self.kv_heads, self.page_size)
        return (self._ptr("k_scales", tensors["k_scales"], F32, shape),
                self._ptr("v_scales", tensors["v_scales"], F32, shape))

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
            capi._check_attention(status, self.handle)

    @staticmethod
    def _unknown(tensors: dict, allowed: tuple, what: str) -> None:
        for name in tensors:
            if name not in allowed:
                raise ValueError(f"unknown {what} {name!r}: expected some of {allowed}")

    # ---------------------------------------------------------------- calls
    def append(self, inputs: dict, outputs: dict, *, stream=None) -> dict:
        """New tokens' keys and values into the cache, their queries rotated.
        inputs: k, v [t][kv_heads][head_dim] BF16, positions [t] int32, slots
        [t] int32 (page * page_size + offset, each at most once; -1: a padding
        token, which is not written) and optionally q [t][heads][head_dim];
        outputs: k_cache, v_cache (with fp8 k_scales, v_scales) and, with q,
        q_out, which may be q itself.  q, k and v may be slices of one packed
        projection."""
        k, v, positions, slots = inputs["k"], inputs["v"], inputs["positions"], inputs["slots"]
        k_cache, v_cache, q, q_out = outputs["k_cache"], outputs["v_cache"], inputs.get("q"), outputs.get("q_out")
        t, pages, kv, d, index = k.shape[0], k_cache.shape[0], self.kv_heads, self.head_dim, self._index
        kv_shape, cache_shape, t_shape = (t, kv, d), (pages, kv, self.page_size, d), (t,)
        dtype = self._cache_dtype
        if (q is not None and q_out is not None and len(outputs) == (5 if self.fp8 else 3)
                and k.dtype is BF16 and v.dtype is BF16 and q.dtype is BF16 and q_out.dtype is BF16
                and k_cache.dtype is dtype and v_cache.dtype is dtype and positions.dtype is I32 and slots.dtype is I32
                and k.shape == kv_shape and v.shape == kv_shape and q.shape == (q_shape := (t, self.heads, d))
                and q_out.shape == q_shape and k_cache.shape == cache_shape and v_cache.shape == cache_shape
                and positions.shape == t_shape and slots.shape == t_shape
                and k_cache.is_contiguous() and v_cache.is_contiguous() and positions.is_contiguous()
                and slots.is_contiguous()
                and (ks := k.stride())[1] == d == (vs := v.stride())[1] and (qs := q.stride())[1] == d
                and (os := q_out.stride())[1] == d and ks[2] == vs[2] == qs[2] == os[2] == 1
                and k.get_device() == index and v.get_device() == index and q.get_device() == index
                and q_out.get_device() == index and k_cache.get_device() == index and v_cache.get_device() == index
                and positions.get_device() == index and slots.get_device() == index):
            k_scales = v_scales = 0
            if self.fp8:
                k_scales, v_scales, shape = outputs["k_scales"], outputs["v_scales"], cache_shape[:3]
                if (k_scales.dtype is F32 and v_scales.dtype is F32 and k_scales.shape == shape and v_scales.shape == shape
                        and k_scales.is_contiguous() and v_scales.is_contiguous() and k_scales.get_device() == index
                        and v_scales.get_device() == index):
                    k_scales, v_scales = k_scales.data_ptr(), v_scales.data_ptr()
                else:
                    k_scales, v_scales = self._scales(outputs, pages)
            if t > 1:
                qs, ks, vs, os = qs[0], ks[0], vs[0], os[0]
            else:   # a single token's stride is never used
                qs = os = self.heads * d
                ks = vs = kv * d
            args = APPEND_ARGS.pack(t, pages, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, positions.data_ptr(),
                                    slots.data_ptr(), q_out.data_ptr(), os, k_cache.data_ptr(), self._page,
                                    v_cache.data_ptr(), self._page, k_scales, v_scales)
        else:
            args = self._append_args(inputs, outputs)
        self._call(self._append, args, stream)
        return outputs

    def _append_args(self, inputs: dict, outputs: dict) -> bytes:
        k, v, q, q_out = inputs["k"], inputs["v"], inputs.get("q"), outputs.get("q_out")
        k_cache, v_cache = outputs["k_cache"], outputs["v_cache"]
        t, kv, pages = k.shape[0], self.kv_heads, k_cache.shape[0]
        ks, vs = self._token_stride("k", k, t, kv), self._token_stride("v", v, t, kv)
        qp = qs = op = os = 0
        if q is not None or q_out is not None:
            if q is None or q_out is None:
                raise ValueError("q and q_out go together")
            qs, os = self._token_stride("q", q, t, self.heads), self._token_stride("q_out", q_out, t, self.heads)
            qp, op = q.data_ptr(), q_out.data_ptr()
        positions, slots = (self._ptr(n, inputs[n], I32, (t,)) for n in ("positions", "slots"))
        kcs, vcs = self._cache("k_cache", k_cache, pages), self._cache("v_cache", v_cache, pages)
        k_scales, v_scales = self._scales(outputs, pages)
        if len(outputs) != 2 + 2 * self.fp8 + (q is not None):
            self._unknown(outputs, ("q_out", "k_cache", "v_cache", "k_scales", "v_scales"), "output")
        return APPEND_ARGS.pack(t, pages, qp, qs, k.data_ptr(), ks, v.data_ptr(), vs, positions, slots, op, os,
                                k_cache.data_ptr(), kcs, v_cache.data_ptr(), vcs, k_scales, v_scales)

    def attend(self, inputs: dict, outputs: dict, *, window: int = 0, sinks: int = 0, scale: float | None = None,
               stream=None) -> dict:
        """Attention of each sequence's newest tokens over its cache.  inputs: q
        [t][heads][head_dim] BF16, k_cache, v_cache (with fp8 k_scales,
        v_scales), pages [s][w] int32 (a sequence's pages in order), lengths [s]
        int32 (positions in the cache, the new ones among them) and, unless
        each sequence has one query, q_starts [s + 1] int32 (sequence i has
        the queries q_starts[i] .. q_starts[i + 1] - 1, its newest); outputs:
        output [t][heads][head_dim] BF16 and optionally lse [t][heads] FP32.

        A query sees the positions up to its own; with a window the last `window`
        of them and the first `sinks` of the sequence.  scale: factor of the
        scores, head_dim ** -0.5 by default."""
        q, k_cache, v_cache, table = inputs["q"], inputs["k_cache"], inputs["v_cache"], inputs["pages"]
        lengths, starts, out, lse = inputs["lengths"], inputs.get("q_starts"), outputs["output"], outputs.get("lse")
        t, s, pages, heads, d, index = q.shape[0], lengths.shape[0], k_cache.shape[0], self.heads, self.head_dim, self._index
        q_shape, cache_shape, dtype = (t, heads, d), (pages, self.kv_heads, self.page_size, d), self._cache_dtype
        if (q.dtype is BF16 and out.dtype is BF16 and k_cache.dtype is dtype and v_cache.dtype is dtype
                and table.dtype is I32 and lengths.dtype is I32 and q.shape == q_shape and out.shape == q_shape
                and k_cache.shape == cache_shape and v_cache.shape == cache_shape and lengths.shape == (s,)
                and (shape := table.shape)[0] == s and len(shape) == 2
                and k_cache.is_contiguous() and v_cache.is_contiguous() and q.is_contiguous() and out.is_contiguous()
                and table.is_contiguous() and lengths.is_contiguous()
                and q.get_device() == index and out.get_device() == index and k_cache.get_device() == index
                and v_cache.get_device() == index and table.get_device() == index and lengths.get_device() == index
                and len(outputs) == (1 if lse is None else 2) and (self.fp8 or "k_scales" not in inputs)):
            k_scales, v_scales = self._scales(inputs, pages) if self.fp8 or "v_scales" in inputs else (0, 0)
            width, row = shape[1], heads * d
            args = ATTEND_ARGS.pack(
                t, s, pages, width, q.data_ptr(), row, 0 if starts is None else self._ptr("q_starts", starts, I32, (s + 1,)),
                lengths.data_ptr(), table.data_ptr(), width, k_cache.data_ptr(), self._page, v_cache.data_ptr(), self._page,
                k_scales, v_scales, self._scale if scale is None else scale, window, sinks, out.data_ptr(), row,
                0 if lse is None else self._ptr("lse", lse, F32, (t, heads)))
        else:
            args = self._attend_args(inputs, outputs, window, sinks, scale)
        self._call(self._attend, args, stream)
        return outputs

    def _attend_args(self, inputs: dict, outputs: dict, window: int, sinks: int, scale: float | None) -> bytes:
        q, k_cache, v_cache, table = inputs["q"], inputs["k_cache"], inputs["v_cache"], inputs["pages"]
        lengths, starts, out, lse = inputs["lengths"], inputs.get("q_starts"), outputs["output"], outputs.get("lse")
        t, s, pages, width = q.shape[0], lengths.shape[0], k_cache.shape[0], table.shape[1]
        qs, os = self._token_stride("q", q, t, self.heads), self._token_stride("output", out, t, self.heads)
        lengths_p = self._ptr("lengths", lengths, I32, (s,))
        starts_p = 0 if starts is None else self._ptr("q_starts", starts, I32, (s + 1,))
        if table.dtype is not I32 or table.shape[0] != s or table.get_device() != self._index or (
                width > 1 and table.stride(1) != 1):
            self._refuse("pages", table, I32, (s, width), "contiguous rows, ")
        ts = table.stride(0) if s > 1 else width
        kcs, vcs = self._cache("k_cache", k_cache, pages), self._cache("v_cache", v_cache, pages)
        k_scales, v_scales = self._scales(inputs, pages)
        lp = 0 if lse is None else self._ptr("lse", lse, F32, (t, self.heads))
        if len(outputs) != 1 + (lse is not None):
            self._unknown(outputs, ("output", "lse"), "output")
        return ATTEND_ARGS.pack(t, s, pages, width, q.data_ptr(), qs, starts_p, lengths_p, table.data_ptr(), ts,
                                k_cache.data_ptr(), kcs, v_cache.data_ptr(), vcs, k_scales, v_scales,
                                self._scale if scale is None else scale, window, sinks, out.data_ptr(), os, lp)

    def check_errors(self) -> None:
        capi.mhc_attention_check_errors(self.handle)
