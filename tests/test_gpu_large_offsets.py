"""The sublayer operators over tensors of more than 2^31 elements: rows on both
sides of each 32-bit limit against the same rows in a call by themselves (norm,
quantisers), or against the definition in 64 bits (products)."""
import pytest
import torch

from test_gpu_sublayer import BF16, F32, F8, blocks, check_product, gen, matmul_inputs, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sub():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    from mhc_residual_boundary_gb300 import Sublayer
    s = Sublayer()
    yield s
    s.check_errors()
    s.close()
    torch.cuda.empty_cache()


def sampled(m, width):
    """Rows at the ends and around the offsets of 2^31 and 2^32 elements and bytes."""
    rows = {0, 1, m - 2, m - 1}
    for limit in (2 ** 30, 2 ** 31, 2 ** 32):
        for r in range(limit // width - 1, limit // width + 2):
            rows.add(r)
    return [r for r in sorted(rows) if 0 <= r < m]


def same(got, want, rows):
    for name in want:
        assert torch.equal(got[name][rows].view(torch.uint8), want[name].view(torch.uint8)), name


def filled(m, h, seed):
    x = torch.empty(m, h, dtype=BF16, device="cuda")
    part = randn(gen(seed), 4099, h).bfloat16()
    for r in range(0, m, 4099):
        x[r:r + 4099] = part[:min(4099, m - r)]
    return x


@pytest.mark.parametrize("m,h", [(530000, 8200), (33000000, 136)])
def test_rows(sub, m, h):
    x = filled(m, h, 1)
    rows = sampled(m, h)
    few = x[rows].contiguous()
    out = sub.empty_outputs("quantize", m, h)
    sub.quantize({"x": x}, out)
    same(out, sub.quantize({"x": few}, sub.empty_outputs("quantize", len(rows), h)), rows)
    w = randn(gen(2), h).bfloat16()
    out = dict(out, output=torch.empty_like(x))
    sub.add_rms_norm({"x": x, "norm_weight": w}, out)
    want = sub.empty_outputs("add_rms_norm", len(rows), h)
    del want["residual_out"]
    same(out, sub.add_rms_norm({"x": few, "norm_weight": w}, want), rows)


@pytest.mark.parametrize("m,h", [(530000, 4104), (18000000, 136)])
def test_swiglu(sub, m, h):
    x = filled(m, 2 * h, 3)
    rows = sorted(set(sampled(m, h) + sampled(m, 2 * h)))
    out = sub.empty_outputs("swiglu", m, h)
    sub.swiglu({"gate_up": x}, out)
    same(out, sub.swiglu({"gate_up": x[rows].contiguous()}, sub.empty_outputs("swiglu", len(rows), h)), rows)


@pytest.mark.parametrize("m,n,k,dtype", [(70000, 62000, 128, BF16), (40000, 60008, 64, F32), (1500000, 24, 2880, BF16),
                                         (40, 1500000, 2880, F32)])
def test_products(sub, m, n, k, dtype):
    g = gen(m + n)
    inp = matmul_inputs(g, 1, 1, k)
    for name, rows in (("values", m), ("weight", n)):
        inp[name] = torch.randint(0, 0x7e, (rows, k), generator=g, device="cuda", dtype=torch.uint8).view(F8)
    inp["scales"] = torch.rand(m, blocks(k), generator=g, device="cuda") + 0.1
    inp["weight_scales"] = torch.rand(blocks(n), blocks(k), generator=g, device="cuda") + 0.1
    out = torch.empty(m, n, dtype=dtype, device="cuda")
    sub.matmul(inp, {"output": out})
    rows = sorted(set(sampled(m, n) + sampled(m, k)))
    # whole blocks of the columns that lie at the ends and around the limits
    cols = sorted({0, (n - 1) // 128} | {c // 128 for c in sampled(n, k)})
    for c in cols:
        at = slice(c * 128, min(n, c * 128 + 128))
        part = {"values": inp["values"].view(torch.uint8)[rows].view(F8), "scales": inp["scales"][rows],
                "weight": inp["weight"][at], "weight_scales": inp["weight_scales"][c:c + 1]}
        check_product(out[rows, at], part)
