"""The operators between two boundaries against their definitions in 64 bits:
norm with the residual's addition, the 8-bit quantisers, the block-scaled
product.

Tolerances, from the arithmetic:
* a BF16 output: half a BF16 ulp (8 significant bits, of the binade that the
  value lies in) and the FP32 steps before it (2^-20 of the value, a few dozen
  roundings);
* an 8-bit value: half an E4M3 ulp (2^-4 of the value, or half the smallest
  subnormal, 2^-10, below the normals) at its scale, and the same FP32 steps;
* a scale: 2^-20 of itself;
* a product: FP32 sums, 2^-20 of the sum of the terms' magnitudes (sums of
  128 exact products in the tensor core, then one fused multiply-add for each
  block), and half a BF16 ulp where the output is BF16.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

F8, BF16, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
STEPS = 2.0 ** -20


@pytest.fixture(scope="module")
def sub():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from mhc_residual_boundary_gb300 import Sublayer
    s = Sublayer()
    yield s
    s.check_errors()
    s.close()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def blocks(n):
    return (n + 127) // 128


def exact_scales(y):
    pad = torch.nn.functional.pad(y, (0, blocks(y.shape[1]) * 128 - y.shape[1]))
    return pad.view(y.shape[0], -1, 128).abs().amax(2).clamp(min=2.0 ** -100) / 448.0


def half_ulp_bf16(x):
    return torch.ldexp(torch.ones_like(x), torch.frexp(x)[1] - 9)


def check_bf16(got, want, what):
    bad = (got.double() - want).abs() > half_ulp_bf16(want) + STEPS * want.abs() + 1e-38
    assert not bad.any(), (what, bad.nonzero()[:4].tolist())


def check_quantized(out, y):
    scales = exact_scales(y)
    assert ((out["scales"].double() - scales).abs() <= STEPS * scales).all()
    spread = out["scales"].double().repeat_interleave(128, 1)[:, :y.shape[1]]
    off = (out["values"].double() * spread - y).abs()
    bound = (2.0 ** -4 + 2 * STEPS) * y.abs() + spread * 2.0 ** -10 * (1 + STEPS)
    assert (off <= bound).all(), (off / bound).max().item()


def silu_product(x):
    h = x.shape[1] // 2
    x = x.double()
    return x[:, :h] * torch.sigmoid(x[:, :h]) * x[:, h:]


# ------------------------------------------------------------------- norm
@pytest.mark.parametrize("m,h", [(1, 8), (1, 5120), (2, 128), (3, 136), (7, 264), (5, 2048), (4, 2056), (33, 1000),
                                 (2, 6144), (3, 8200), (2, 16384), (700, 520)])
@pytest.mark.parametrize("residual", [True, False])
def test_norm(sub, m, h, residual):
    g = gen(m * 31 + h)
    inp = {"x": randn(g, m, h).bfloat16(), "norm_weight": (1 + 0.1 * randn(g, h)).bfloat16()}
    r = inp["x"].double()
    out = sub.empty_outputs("add_rms_norm", m, h)
    if residual:
        inp["residual"] = (3 * randn(g, m, h)).bfloat16()
        r = r + inp["residual"].double()
    else:
        del out["residual_out"]
    sub.add_rms_norm(inp, out, eps=1e-5)
    y = r / (r.square().mean(1, keepdim=True) + 1e-5).sqrt() * inp["norm_weight"].double()
    if residual:
        check_bf16(out["residual_out"], r, "residual_out")
    check_bf16(out["output"], y, "output")
    check_quantized(out, y)


def test_norm_strides_and_in_place(sub):
    g = gen(5)
    wide = torch.full((9, 1024), float("nan"), device="cuda").bfloat16()
    wide[:, 256:776] = randn(g, 9, 520).bfloat16()
    x, res = wide[:, 256:776], randn(g, 9, 520).bfloat16()
    w = randn(g, 520).bfloat16()
    r = x.double() + res.double()
    y = r / (r.square().mean(1, keepdim=True) + 1e-6).sqrt() * w.double()
    out = {"residual_out": res, "output": torch.empty(9, 520, dtype=BF16, device="cuda")}
    sub.add_rms_norm({"x": x, "residual": res, "norm_weight": w}, out)
    check_bf16(res, r, "residual in place")
    check_bf16(out["output"], y, "output")


def test_norm_single_outputs_and_no_rows(sub):
    g = gen(6)
    x, w = randn(g, 3, 256).bfloat16(), randn(g, 256).bfloat16()
    both = sub.empty_outputs("add_rms_norm", 3, 256)
    del both["residual_out"]
    sub.add_rms_norm({"x": x, "norm_weight": w}, both)
    for names in (("output",), ("values", "scales")):
        out = {n: torch.zeros_like(both[n]) for n in names}
        sub.add_rms_norm({"x": x, "norm_weight": w}, out)
        for n in names:
            assert torch.equal(out[n].view(torch.uint8), both[n].view(torch.uint8))
    empty = sub.empty_outputs("quantize", 0, 256)
    sub.add_rms_norm({"x": x[:0], "norm_weight": w}, empty)


def test_norm_of_zeros_and_non_finite_rows(sub):
    x = torch.zeros(4, 256, dtype=BF16, device="cuda")
    x[1, 5] = float("inf")
    x[2, 7] = float("nan")
    x[3] = 1.0
    w = torch.ones(256, dtype=BF16, device="cuda")
    out = sub.empty_outputs("add_rms_norm", 4, 256)
    del out["residual_out"]
    sub.add_rms_norm({"x": x, "norm_weight": w}, out)
    assert (out["output"][0] == 0).all() and (out["values"][0].float() == 0).all()
    assert torch.isnan(out["output"][1, 5]) and torch.isnan(out["output"][2]).all()
    assert (out["output"][3] == 1).all() and (out["values"][3].float() == 448).all()


# -------------------------------------------------------------- quantisers
@pytest.mark.parametrize("m,h", [(1, 8), (1, 128), (2, 120), (3, 136), (5, 384), (17, 1000), (64, 5120), (1, 16392),
                                 (999, 264)])
@pytest.mark.parametrize("op", ["quantize", "swiglu"])
def test_quantisers(sub, op, m, h):
    g = gen(m + h)
    # blocks of very different magnitude
    size = torch.exp(6 * torch.rand(m, 1, generator=g, device="cuda") - 3)
    out = sub.empty_outputs(op, m, h)
    if op == "quantize":
        x = (size * randn(g, m, h)).bfloat16()
        sub.quantize({"x": x}, out)
        y = x.double()
    else:
        x = (size * randn(g, m, 2 * h)).bfloat16()
        sub.swiglu({"gate_up": x}, out)
        y = silu_product(x)
        check_bf16(out["output"], y, "output")
    check_quantized(out, y)


# enough blocks for the wide form: rows of whole and of half 32-byte pieces, of
# one block, of less than one
@pytest.mark.parametrize("m,h", [(600, 5120), (700, 4088), (2500, 1000), (20000, 8), (20000, 16), (5000, 520)])
@pytest.mark.parametrize("op", ["quantize", "swiglu"])
@pytest.mark.parametrize("offset", [0, 8])
def test_quantisers_many_blocks(sub, op, m, h, offset):
    g = gen(m + h)
    width = 2 * h if op == "swiglu" else h
    wide = torch.full((m, offset + width), float("nan"), device="cuda").bfloat16()
    x = wide[:, offset:]
    x.copy_(2 * randn(g, m, width))
    out = sub.empty_outputs(op, m, h)
    out["values"].view(torch.uint8).fill_(0x7f)
    out["scales"].fill_(float("nan"))
    getattr(sub, op)({"gate_up" if op == "swiglu" else "x": x}, out)
    y = silu_product(x) if op == "swiglu" else x.double()
    check_quantized(out, y)
    if op == "swiglu":
        check_bf16(out["output"], y, "output")


def test_quantize_strided_rows(sub):
    g = gen(9)
    wide = randn(g, 6, 640).bfloat16()
    out = sub.empty_outputs("quantize", 6, 264)
    sub.quantize({"x": wide[:, 128:392]}, out)
    check_quantized(out, wide[:, 128:392].double())


def test_quantize_edges(sub):
    x = torch.zeros(5, 256, dtype=BF16, device="cuda")
    x[1, 130] = 2.0 ** -120                      # below the floor of the block's maximum
    x[2, 3] = float("inf")
    x[3, 200] = float("nan")
    x[4] = torch.finfo(BF16).max
    out = sub.empty_outputs("quantize", 5, 256)
    sub.quantize({"x": x}, out)
    v, s = out["values"].float(), out["scales"]
    floor = torch.tensor(2.0 ** -100, device="cuda") / 448
    assert (v[0] == 0).all() and (s[0] == floor).all()
    assert (v[1] == 0).all() and (s[1] == floor).all()
    assert s[2, 0] == float("inf") and s[2, 1] == floor
    assert torch.isnan(s[3, 1]) and s[3, 0] == floor
    assert (v[4] == 448).all() and torch.isfinite(s[4]).all()


def test_swiglu_extremes(sub):
    h = 128
    x = torch.zeros(3, 2 * h, dtype=BF16, device="cuda")
    x[0, :h], x[0, h:] = -1e4, 3.0               # silu underflows to zero
    x[1, :h], x[1, h:] = 1e4, -2.0
    x[2, :h], x[2, h:] = 0.0, 5.0
    out = sub.empty_outputs("swiglu", 3, h)
    sub.swiglu({"gate_up": x}, out)
    assert (out["output"][0] == 0).all() and (out["output"][2] == 0).all()
    check_bf16(out["output"], silu_product(x), "output")


# ----------------------------------------------------------------- product
def matmul_inputs(g, m, n, k):
    return {"values": (60 * randn(g, m, k)).clamp(-448, 448).to(F8),
            "scales": torch.rand(m, blocks(k), generator=g, device="cuda") + 0.1,
            "weight": (60 * randn(g, n, k)).clamp(-448, 448).to(F8),
            "weight_scales": torch.rand(blocks(n), blocks(k), generator=g, device="cuda") + 0.1}


def exact_product(inp):
    """(product, sum of the terms' magnitudes) in 64 bits."""
    m, k = inp["values"].shape
    n = inp["weight"].shape[0]
    a = inp["values"].double() * inp["scales"].double().repeat_interleave(128, 1)[:, :k]
    ws = inp["weight_scales"].double().repeat_interleave(128, 1)[:, :k].repeat_interleave(128, 0)[:n]
    w = inp["weight"].double() * ws
    return a @ w.t(), a.abs() @ w.abs().t()


def check_product(got, inp):
    want, size = exact_product(inp)
    bound = STEPS * size
    if got.dtype == BF16:
        bound = bound + half_ulp_bf16(want.abs() + bound)
    off = (got.double() - want).abs()
    assert (off <= bound).all(), ((off / bound.clamp(min=1e-30)).max().item(), (off > bound).nonzero()[:4].tolist())


@pytest.mark.parametrize("m", [1, 2, 7, 8, 33, 64, 127, 128, 129, 300])
@pytest.mark.parametrize("n,k", [(8, 16), (1, 128), (100, 112), (128, 144), (200, 1024), (1000, 2064)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_matmul(sub, m, n, k, dtype):
    inp = matmul_inputs(gen(m * 7 + n + k), m, n, k)
    out = sub.empty_outputs("matmul", m, n, dtype=dtype)
    out["output"].fill_(float("nan"))
    sub.matmul(inp, out)
    check_product(out["output"], inp)


# from few to many tiles a GPU: split tiles, one tile an SM, several tiles an SM
@pytest.mark.parametrize("m,n,k", [(1, 6144, 5120), (16, 5120, 2048), (200, 2120, 1040), (640, 4096, 512),
                                   (1030, 4000, 784), (2048, 6144, 512), (4096, 2000, 256)])
def test_matmul_sizes(sub, m, n, k):
    inp = matmul_inputs(gen(m + n + k), m, n, k)
    out = sub.empty_outputs("matmul", m, n)
    out["output"].fill_(float("nan"))
    sub.matmul(inp, out)
    check_product(out["output"], inp)


def test_matmul_strides(sub):
    g = gen(3)
    m, n, k = 37, 72, 272
    inp = matmul_inputs(g, m, n, k)
    nan8 = torch.full((max(m, n) + 4, 400), 0x7f, dtype=torch.uint8, device="cuda")
    wide_a, wide_w = nan8.clone().view(F8), nan8.clone().view(F8)
    wide_a[2:2 + m, 16:16 + k] = inp["values"]
    wide_w[2:2 + n, 32:32 + k] = inp["weight"]
    wide_s = torch.full((m, 7), float("nan"), device="cuda")
    wide_s[:, 2:5] = inp["scales"]
    view = dict(inp, values=wide_a[2:2 + m, 16:16 + k], weight=wide_w[2:2 + n, 32:32 + k], scales=wide_s[:, 2:5])
    for dtype, width, at in ((BF16, 90, 5), (BF16, 96, 8), (F32, 77, 1), (F32, 80, 4)):
        wide_o = torch.full((m, width), 7.0, dtype=dtype, device="cuda")
        sub.matmul(view, {"output": wide_o[:, at:at + n]})
        check_product(wide_o[:, at:at + n], inp)
        assert (wide_o[:, :at] == 7).all() and (wide_o[:, at + n:] == 7).all()


def test_matmul_nan_and_infinite_scale_stay_in_their_row(sub):
    inp = matmul_inputs(gen(4), 40, 136, 512)
    inp["values"].view(torch.uint8)[3, 100] = 0x7f
    inp["scales"][5, 2] = float("inf")
    out = sub.empty_outputs("matmul", 40, 136)
    sub.matmul(inp, out)
    keep = [i for i in range(40) if i not in (3, 5)]
    assert torch.isnan(out["output"][3]).all() and not torch.isfinite(out["output"][5]).any()
    part = dict(inp, values=inp["values"][keep], scales=inp["scales"][keep])
    check_product(out["output"][keep], part)


def test_matmul_repeats_its_bits_on_another_stream_and_in_a_graph(sub):
    inp = matmul_inputs(gen(8), 3, 640, 4096)
    first = sub.empty_outputs("matmul", 3, 640, dtype=F32)
    sub.matmul(inp, first)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    second = sub.empty_outputs("matmul", 3, 640, dtype=F32)
    with torch.cuda.stream(stream):
        for _ in range(20):
            sub.matmul(inp, second)
    stream.synchronize()
    assert torch.equal(first["output"], second["output"])
    third = sub.empty_outputs("matmul", 3, 640, dtype=F32)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sub.matmul(inp, third)
        sub.matmul(inp, third)
    third["output"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first["output"], third["output"])


def test_chain_of_a_dense_mlp(sub):
    """norm -> gate and up -> swiglu -> down, each call's outputs the next one's inputs."""
    g = gen(12)
    m, h, i = 19, 1024, 640
    x, res = randn(g, m, h).bfloat16(), randn(g, m, h).bfloat16()
    w = (1 + 0.1 * randn(g, h)).bfloat16()
    up = matmul_inputs(g, 1, 2 * i, h)
    down = matmul_inputs(g, 1, h, i)
    a = sub.empty_outputs("add_rms_norm", m, h)
    sub.add_rms_norm({"x": x, "residual": res, "norm_weight": w}, a)
    first = {"values": a["values"], "scales": a["scales"], "weight": up["weight"],
             "weight_scales": up["weight_scales"] * 1e-4}
    b = sub.matmul(first, sub.empty_outputs("matmul", m, 2 * i))
    c = sub.swiglu({"gate_up": b["output"]}, sub.empty_outputs("swiglu", m, i))
    second = {"values": c["values"], "scales": c["scales"], "weight": down["weight"],
              "weight_scales": down["weight_scales"]}
    d = sub.matmul(second, sub.empty_outputs("matmul", m, h))
    check_product(b["output"], first)
    check_quantized(c, silu_product(b["output"]))
    check_product(d["output"], second)


# --------------------------------------------------------------- refusals
def test_refusals(sub):
    from mhc_residual_boundary_gb300 import capi
    x = torch.zeros(4, 256, dtype=BF16, device="cuda")
    w = torch.zeros(256, dtype=BF16, device="cuda")
    q = sub.empty_outputs("quantize", 4, 256)
    with pytest.raises(capi.MhcError, match="residual_out needs residual"):
        sub.add_rms_norm({"x": x, "norm_weight": w}, {"residual_out": x})
    with pytest.raises(capi.MhcError, match="no output"):
        sub.add_rms_norm({"x": x, "norm_weight": w}, {})
    with pytest.raises(capi.MhcError, match="go together"):
        sub.add_rms_norm({"x": x, "norm_weight": w}, {"values": q["values"]})
    with pytest.raises(capi.MhcError, match="multiple of 8"):
        sub.quantize({"x": x[:, :100].contiguous()}, sub.empty_outputs("quantize", 4, 100))
    with pytest.raises(capi.MhcError, match="16-byte aligned"):
        sub.quantize({"x": x[:, 4:132]}, sub.empty_outputs("quantize", 4, 128))
    with pytest.raises(capi.MhcError, match="x_stride"):
        sub.quantize({"x": torch.zeros(4, 260, dtype=BF16, device="cuda")[:, :128]},
                     sub.empty_outputs("quantize", 4, 128))
    with pytest.raises(ValueError, match="expected"):
        sub.quantize({"x": x.half()}, q)
    with pytest.raises(ValueError, match="must be a tensor on"):
        sub.quantize({"x": x.cpu()}, q)
    with pytest.raises(ValueError, match="unknown output"):
        sub.quantize({"x": x}, dict(q, output=x))
    with pytest.raises(ValueError, match="contiguous rows"):
        sub.quantize({"x": torch.zeros(256, 4, dtype=BF16, device="cuda").t()}, q)
    inp = matmul_inputs(gen(1), 4, 64, 256)
    out = sub.empty_outputs("matmul", 4, 64)
    with pytest.raises(capi.MhcError, match="k must be a positive multiple of 16"):
        sub.matmul(dict(inp, values=inp["values"][:, :200], weight=inp["weight"][:, :200]), out)
    with pytest.raises(capi.MhcError, match="16-byte aligned"):
        sub.matmul(dict(inp, values=inp["values"][:, 8:136], weight=inp["weight"][:, :128],
                        scales=inp["scales"][:, :1], weight_scales=inp["weight_scales"][:, :1].contiguous()), out)
    with pytest.raises(ValueError, match="weight_scales"):
        sub.matmul(dict(inp, weight_scales=inp["weight_scales"].repeat(2, 1)), out)
    with pytest.raises(ValueError, match="output"):
        sub.matmul(inp, {"output": out["output"].half()})
    sub.matmul(dict(inp, values=inp["values"][:0], scales=inp["scales"][:0]), sub.empty_outputs("matmul", 0, 64))
    a = capi.mhc_sublayer_matmul_args_t()
    with pytest.raises(capi.MhcError, match="n must be positive"):
        capi.mhc_sublayer_matmul(sub.handle, a)
    a.m, a.n, a.k = 1, 8, 16
    with pytest.raises(capi.MhcError, match="values is NULL"):
        capi.mhc_sublayer_matmul(sub.handle, a)


def test_stalled_copies_report_a_timeout_and_the_handle_recovers(sub):
    from mhc_residual_boundary_gb300 import capi
    inp = matmul_inputs(gen(2), 5, 256, 2048)
    out = sub.empty_outputs("matmul", 5, 256)
    torch.cuda.synchronize()
    capi.mhc_test_stall_sublayer_copies(True)
    try:
        sub.matmul(inp, out)
        torch.cuda.synchronize()
    finally:
        capi.mhc_test_stall_sublayer_copies(False)
    with pytest.raises(capi.MhcError, match="MHC_ERR_TIMEOUT"):
        sub.check_errors()
    sub.check_errors()
    sub.matmul(inp, out)
    check_product(out["output"], inp)


# tiles whose k blocks' scales come in more than one chunk of 32: whole chunks,
# ragged ones, several tiles a CTA, and split tiles with more than 32 blocks a CTA
@pytest.mark.parametrize("m,n,k", [(2048, 2500, 4096), (2048, 2500, 4240), (1100, 4000, 8336), (1300, 2100, 8192),
                                   (4096, 4096, 6144), (3, 100, 40976), (64, 136, 65536), (128, 200, 49168),
                                   (300, 1500, 33008)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_matmul_long_rows(sub, m, n, k, dtype):
    inp = matmul_inputs(gen(m + n + k), m, n, k)
    out = sub.empty_outputs("matmul", m, n, dtype=dtype)
    out["output"].fill_(float("nan"))
    sub.matmul(inp, out)
    check_product(out["output"], inp)


def test_norm_in_place_of_dense_inputs(sub):
    """Each BF16 output in the place of each input, alone and both at once."""
    g = gen(21)
    for m, h in ((9, 520), (1, 264), (300, 5120), (5, 16384)):
        x, res = randn(g, m, h).bfloat16(), randn(g, m, h).bfloat16()
        w = randn(g, h).bfloat16()
        want = sub.empty_outputs("add_rms_norm", m, h)
        sub.add_rms_norm({"x": x, "residual": res, "norm_weight": w}, want)
        for places in (("x", None), ("residual", None), (None, "x"), (None, "residual"), ("x", "residual"),
                       ("residual", "x")):
            inp = {"x": x.clone(), "residual": res.clone(), "norm_weight": w}
            out = sub.empty_outputs("add_rms_norm", m, h)
            for name, place in zip(("residual_out", "output"), places):
                if place:
                    out[name] = inp[place]
            sub.add_rms_norm(inp, out)
            for name in want:
                assert torch.equal(out[name].view(torch.uint8), want[name].view(torch.uint8)), (m, h, places, name)


def test_norm_overlap_refusals(sub):
    """Outputs that overlap an input but in the allowed way are refused; those
    that only lie between its rows are not."""
    from mhc_residual_boundary_gb300 import capi
    g = gen(22)
    h, w = 256, torch.ones(256, dtype=BF16, device="cuda")
    buffer = torch.zeros(64 * 1024, dtype=BF16, device="cuda")

    def dense(at, m, dtype=BF16, width=h):
        size = torch.tensor([], dtype=dtype).element_size()
        return buffer.view(torch.uint8)[2 * at:2 * at + m * width * size].view(dtype).view(m, width)

    def strided(at, m, stride):
        return buffer[at:].as_strided((m, h), (stride, 1))

    def norm(x, residual, out):
        sub.add_rms_norm({"x": x, "norm_weight": w, **({} if residual is None else {"residual": residual})}, out)

    other = torch.zeros(8, h, dtype=BF16, device="cuda")
    values, scales = torch.zeros(8, h, device="cuda").to(F8), torch.zeros(8, 2, device="cuda")
    refused = [
        (strided(0, 8, 512), None, {"output": dense(0, 8)}),                       # the same start, another stride
        (other, strided(0, 8, 264), {"residual_out": dense(0, 8)}),
        (dense(0, 8), None, {"output": dense(8, 8)}),                              # shifted by a fragment
        (dense(2048, 8), None, {"output": dense(8, 8)}),                           # ends inside the first row
        (strided(4096, 4, 1024), None, {"output": dense(4096 + 3 * 1024 + 248, 4)}),   # only the last row's end
        (dense(0, 8), None, {"values": dense(0, 8, F8), "scales": scales}),
        (dense(0, 8), None, {"values": values, "scales": dense(2040, 8, F32, 2)}),
        (other, dense(0, 8), {"residual_out": torch.zeros_like(other), "output": dense(1024, 8)}),
    ]
    for x, residual, out in refused:
        with pytest.raises(capi.MhcError, match="overlaps"):
            norm(x, residual, out)
    with pytest.raises(capi.MhcError, match="output overlaps norm_weight"):
        sub.add_rms_norm({"x": other, "norm_weight": dense(0, 1)[0]}, {"output": dense(0, 8)})
    rows = randn(g, 8, h).bfloat16()
    want = torch.zeros(8, h, dtype=BF16, device="cuda")
    norm(rows, None, {"output": want})
    for x, out in ((strided(0, 2, 8192), dense(256, 2)),                           # between two rows
                   (strided(4096, 2, 8192), dense(4096 + 8192 + 256, 2)),          # right after the last
                   (dense(4096, 8), dense(2048, 8)), (dense(2048, 8), dense(4096, 8)),   # side by side
                   (strided(0, 1, 8192), dense(0, 1))):                            # one row
        m = x.shape[0]
        x.copy_(rows[:m])
        norm(x, None, {"output": out})
        assert torch.equal(out, want[:m])


def test_device_argument(sub):
    from mhc_residual_boundary_gb300 import Sublayer
    x = torch.zeros(2, 128, dtype=BF16, device="cuda")
    for device in (None, 0, "cuda", "cuda:0", x.device, torch.device("cuda")):
        with Sublayer(device=device) as s:
            assert s.device == x.device
            s.quantize({"x": x}, s.empty_outputs("quantize", 2, 128))


def test_the_c_entry_points_by_struct(sub):
    """The binding's functions of the C names, with argument structs: the same
    bits as the wrapper's calls, which pack the structs themselves."""
    from mhc_residual_boundary_gb300 import capi
    g = gen(31)
    m, h = 11, 264
    x, res, w = randn(g, m, h).bfloat16(), randn(g, m, h).bfloat16(), randn(g, h).bfloat16()
    gate_up = randn(g, m, 2 * h).bfloat16()
    stream = torch.cuda.current_stream().cuda_stream

    def fields(a, **kw):
        for name, v in kw.items():
            setattr(a, name, v.data_ptr() if isinstance(v, torch.Tensor) else v)
        return a

    def same(got, want):
        for name in want:
            assert torch.equal(got[name].view(torch.uint8), want[name].view(torch.uint8)), name

    want = sub.add_rms_norm({"x": x, "residual": res, "norm_weight": w}, sub.empty_outputs("add_rms_norm", m, h), eps=1e-5)
    got = sub.empty_outputs("add_rms_norm", m, h)
    capi.mhc_sublayer_add_rms_norm(sub.handle, fields(
        capi.mhc_sublayer_norm_args_t(), m=m, h=h, x=x, x_stride=h, residual=res, residual_stride=h, norm_weight=w,
        eps=1e-5, **got), stream)
    same(got, want)
    want = sub.quantize({"x": x}, sub.empty_outputs("quantize", m, h))
    got = sub.empty_outputs("quantize", m, h)
    capi.mhc_sublayer_quantize(sub.handle, fields(capi.mhc_sublayer_quantize_args_t(), m=m, h=h, x=x, x_stride=h, **got),
                               stream)
    same(got, want)
    a = fields(capi.mhc_sublayer_quantize_args_t(), m=m, h=h, x=x, x_stride=h, output=x.clone(), **got)
    with pytest.raises(capi.MhcError, match="no BF16 output"):
        capi.mhc_sublayer_quantize(sub.handle, a, stream)
    want = sub.swiglu({"gate_up": gate_up}, sub.empty_outputs("swiglu", m, h))
    got = sub.empty_outputs("swiglu", m, h)
    capi.mhc_sublayer_swiglu(sub.handle, fields(capi.mhc_sublayer_quantize_args_t(), m=m, h=h, x=gate_up, x_stride=2 * h,
                                                **got), stream)
    same(got, want)
    inp = matmul_inputs(g, m, 72, h - 8)
    want = sub.matmul(inp, sub.empty_outputs("matmul", m, 72, dtype=F32))
    got = sub.empty_outputs("matmul", m, 72, dtype=F32)
    capi.mhc_sublayer_matmul(sub.handle, fields(
        capi.mhc_sublayer_matmul_args_t(), m=m, n=72, k=h - 8, values_stride=h - 8, scales_stride=2, weight_stride=h - 8,
        output_stride=72, output_f32=1, **inp, **got), stream)
    same(got, want)
