"""The 8-bit values and the scales of the quantisers, bit for bit: scale = amax *
(1 / 448) and value = x * ((1 / amax) * 448), every step rounded to nearest in
FP32, the value then to E4M3; and the same bits from the short form in PyTorch,
amax / 448 and x * (448 / amax).

The inputs make every step before the quantisation exact: the norm's rows have
a mean square of one and are multiplied by BF16 weights, and a SiLU's gate is
large enough for its sigmoid to be one.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

F8, BF16, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sub():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from mhc_residual_boundary_gb300 import Sublayer
    s = Sublayer()
    yield s
    s.check_errors()
    s.close()


def every_magnitude(largest_bits=0x7f80):
    """Rows of 128 BF16 values: row i's largest is the positive value of bit
    pattern i, the others spread over the 128 patterns before it and the
    binades below."""
    top = torch.arange(largest_bits, device="cuda")
    back = torch.arange(128, device="cuda")
    steps = torch.where(back < 64, back, back * 23)
    bits = (top[:, None] - steps[None]).clamp(min=0)
    sign = ((bits * 7 + back) % 3 == 0).int() << 15
    bits = bits | sign
    return torch.where(bits >= 1 << 15, bits - (1 << 16), bits).to(torch.int16).view(BF16)


def plain(y):
    """The definition on exact FP32 values [m][128 n]."""
    b = y.float().view(y.shape[0], -1, 128)
    amax = b.abs().amax(2).clamp(min=2.0 ** -100)
    one, top = torch.ones_like(amax), torch.full_like(amax, 448.0)
    inv, scales = (one / amax) * top, amax * (one / top)
    assert torch.equal(448.0 / amax, inv) and torch.equal(amax / 448.0, scales)
    return (b * inv[:, :, None]).to(F8).view(y.shape), scales


def check(out, y):
    values, scales = plain(y)
    assert torch.equal(out["scales"].view(torch.int32), scales.view(torch.int32)), \
        (out["scales"] != scales).sum().item()
    assert torch.equal(out["values"].view(torch.uint8), values.view(torch.uint8)), \
        (out["values"].float() != values.float()).sum().item()


# rows of one block, of two, and of few rows: the forms that take one and two
# fragments a lane
@pytest.mark.parametrize("blocks", [1, 2, 17])
def test_quantize(sub, blocks):
    x = every_magnitude()
    x = torch.cat([x.roll(37 * k, 0) for k in range(blocks)], 1).contiguous()
    check(sub.quantize({"x": x}, sub.empty_outputs("quantize", *x.shape)), x)
    few = x[16000:16300].contiguous()
    check(sub.quantize({"x": few}, sub.empty_outputs("quantize", *few.shape)), few)


def test_quantize_of_eighths(sub):
    """Values at and beside the ties of E4M3, in blocks of every mantissa."""
    k = torch.arange(128, device="cuda").float()
    largest = 1 + k[:, None] / 128
    x = torch.cat([largest, (largest * (k[None, 1:] + 0.5) / 128)], 1).bfloat16()
    check(sub.quantize({"x": x}, sub.empty_outputs("quantize", 128, 128)), x)


@pytest.mark.parametrize("scale", [2.0 ** -4, 2.0 ** 6])
def test_swiglu(sub, scale):
    up = every_magnitude(0x7b00)[0x400:]
    gate = torch.full_like(up, 64.0)
    x = torch.cat([gate, (up.float() * scale).bfloat16()], 1)
    out = sub.swiglu({"gate_up": x}, sub.empty_outputs("swiglu", *up.shape))
    y = 64.0 * x[:, 128:].float()
    check(out, y)
    few = sub.swiglu({"gate_up": x[:99].contiguous()}, sub.empty_outputs("swiglu", 99, 128))
    check(few, y[:99])


@pytest.mark.parametrize("rows", [1, 3])
def test_norm(sub, rows):
    w = every_magnitude()
    for at in range(0, w.shape[0], 128):
        part = w[at:at + 128].reshape(-1).contiguous()
        h = part.shape[0]
        x = torch.ones(rows, h, dtype=BF16, device="cuda")
        x[:, ::3] = -1.0
        out = sub.empty_outputs("add_rms_norm", rows, h)
        del out["residual_out"], out["output"]
        sub.add_rms_norm({"x": x, "norm_weight": part}, out, eps=0.0)
        check(out, x.float() * part.float())
