"""append against its definition in 64 bits.

Tolerances, from the arithmetic: an angle is exact to 2^-24 of a half turn (its
FP32 form) and sine and cosine to 2^-22 of 1, so a rotated element is off by at most
2^-20 of |a| + |b| before it is rounded, to BF16 (half an ulp) or, over the
block's scale (2^-20 of itself), to E4M3 (half an ulp: 2^-4 of the value, or 2^-10
below the normals).  Values are not rotated: BF16 ones are copied.
"""
import math

import pytest
import torch

from attention_cases import BF16, F8, F32, I32, gen, half_ulp_bf16, randn

pytestmark = pytest.mark.gpu
STEPS = 2.0 ** -20


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def rotate(x, positions, frequencies, rotary, interleaved):
    """(rotated, |a| + |b|) in 64 bits."""
    x = x.double()
    y, mag = x.clone(), x.abs()
    for i in range(rotary // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
        w = positions.double() * frequencies[i]
        c, s = torch.cos(w)[:, None], torch.sin(w)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        mag[..., a] = mag[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, mag


def check_bf16(got, want, mag):
    bad = ~((got.double() - want).abs() <= half_ulp_bf16(want) + STEPS * mag + 1e-38)
    assert not bad.any(), (bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist())


def check_fp8(values, scales, want, mag):
    amax = want.abs().amax(-1)
    want_scales = amax.clamp(min=2.0 ** -100) / 448
    assert ((scales.double() - want_scales).abs() <= 2 * STEPS * (want_scales + mag.amax(-1) / 448)).all()
    v = want / scales.double()[..., None]
    half = torch.ldexp(torch.ones_like(v), torch.frexp(v)[1].clamp(min=-5) - 5)
    bad = ~((values.double() - v).abs() <= half + STEPS * (v.abs() + mag / scales.double()[..., None]))
    assert not bad.any(), (bad.nonzero()[:4].tolist(), values[bad][:4].tolist(), v[bad][:4].tolist())


CASES = [
    # tokens, heads, kv, d, page, rotary, interleaved
    (1, 1, 1, 64, 16, 64, False),
    (1, 40, 8, 128, 16, 128, False),
    (7, 6, 2, 128, 32, 64, False),
    (33, 16, 2, 64, 64, 32, True),
    (100, 12, 4, 128, 128, 128, True),
    (50, 5, 1, 64, 16, 16, False),
    (20, 128, 1, 128, 32, 0, False),
    (301, 24, 3, 128, 16, 112, False),
    (64, 9, 9, 64, 16, 48, True),
    # two and four tokens a CTA, and a last one with fewer
    (903, 35, 5, 128, 64, 128, False),
    (1001, 120, 8, 128, 16, 96, True),
    (6003, 34, 2, 64, 32, 32, False),
]


def draw(case, fp8, seed=0):
    t, heads, kv, d, page, rotary, interleaved = CASES[case]
    from mhc_residual_boundary_gb300 import Attention
    g = gen(seed + case)
    a = Attention(heads=heads, kv_heads=kv, head_dim=d, page_size=page, fp8=fp8, rotary_dim=rotary, theta=10000.0,
                  interleaved=interleaved)
    pages = t // page + 2
    packed = (3 * randn(g, t, heads + 2 * kv, d)).to(BF16)
    q, k, v = packed.split([heads, kv, kv], 1)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:t].int()
    positions = torch.randint(0, 2 ** 31 - 1, (t,), generator=g, device="cuda").int()
    positions[: t // 2] %= 5000
    positions[0] = 0
    if t > 6:
        positions[5] = -17
    cache = a.empty_cache(pages)
    for x in cache.values():
        x.view(torch.uint8).fill_(0x11)
    frequencies = [10000.0 ** (-2.0 * i / rotary) for i in range(rotary // 2)]
    return a, {"q": q, "k": k, "v": v, "slots": slots, "positions": positions}, cache, frequencies


def check_append(case, fp8, inputs, cache, frequencies, q_out, q):
    t, heads, kv, d, page, rotary, interleaved = CASES[case]
    if q_out is not None:
        check_bf16(q_out, *rotate(q, inputs["positions"], frequencies, rotary, interleaved))
    slots = inputs["slots"].long()
    live = (slots >= 0).nonzero()[:, 0]
    where, offset = slots[live] // page, slots[live] % page
    for name in ("k", "v"):
        x = inputs[name][live]
        want, mag = rotate(x, inputs["positions"][live], frequencies, rotary, interleaved) if name == "k" else (
            x.double(), x.double().abs())
        stored = cache[name + "_cache"]
        if fp8:
            got = stored.view(torch.uint8)[where, :, offset].view(F8).float()
            check_fp8(got, cache[name + "_scales"][where, :, offset], want, mag)
        elif name == "v":
            assert torch.equal(stored[where, :, offset], x)
        else:
            check_bf16(stored[where, :, offset], want, mag)
    # nothing else is written
    other = torch.ones(cache["k_cache"].shape[0], page, dtype=torch.bool, device="cuda")
    other[where, offset] = False
    for x in cache.values():
        raw = x.view(torch.uint8).view(*x.shape[:3], -1)
        assert (raw.transpose(1, 2)[other] == 0x11).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_append(case, fp8):
    a, inputs, cache, frequencies = draw(case, fp8)
    inputs["slots"][3::5] = -1
    q_out = torch.empty(*inputs["q"].shape, dtype=BF16, device="cuda")
    a.append(inputs, {"q_out": q_out, **cache})
    a.check_errors()
    check_append(case, fp8, inputs, cache, frequencies, q_out, inputs["q"])
    # the queries in place, the same bits; then without queries
    before = inputs["q"].clone()
    a.append(inputs, {"q_out": inputs["q"], **cache})
    assert torch.equal(inputs["q"], q_out)
    del inputs["q"]
    a.append(inputs, cache)
    a.check_errors()
    check_append(case, fp8, inputs, cache, frequencies, q_out, before)


def test_far_positions():
    """Angles of positions up to 2^31 lose nothing: the product is reduced exactly."""
    from mhc_residual_boundary_gb300 import Attention
    d, t = 128, 64
    f = [1.0, math.pi, 6.5, 0.1, 1e-9, 2 * math.pi] + [0.5 ** i for i in range(58)]
    a = Attention(heads=1, kv_heads=1, head_dim=d, page_size=64, rotary_dim=d, frequencies=f)
    x = torch.zeros(t, 1, d, dtype=BF16, device="cuda")
    x[..., :64] = 1.0
    positions = (2 ** 31 - 1 - torch.arange(t, device="cuda") * 33333333).int()
    cache, q_out = a.empty_cache(1), torch.empty_like(x)
    a.append({"q": x, "k": x, "v": x, "positions": positions, "slots": torch.arange(t, device="cuda").int()},
             {"q_out": q_out, **cache})
    # the angle in exact integers: turns = position * f / 2 pi, f / 2 pi to 2^-120
    from fractions import Fraction
    two_pi = Fraction(2 * 314159265358979323846264338327950288419716939937510, 10 ** 50)
    for i in (0, 1, 2, 3, 4, 5, 20):
        turns = Fraction(f[i]) / two_pi
        want = torch.tensor([math.cos(2 * math.pi * float(Fraction(int(p)) * turns % 1)) for p in positions.tolist()],
                            dtype=torch.float64, device="cuda")
        # f / 2 pi is the quotient of two doubles: off by 2^-52 of itself (at most 1.04 here), times 2^31 and 2 pi
        assert ((q_out[:, 0, i].double() - want).abs() <= half_ulp_bf16(want) + 2.0 ** -18).all(), i
    a.check_errors()


def test_zeros_infinities_and_nan():
    """A row of zeros has the floor's scale; a row with an infinity or a NaN has a non-finite one."""
    from mhc_residual_boundary_gb300 import Attention
    a = Attention(heads=1, kv_heads=1, head_dim=64, page_size=16, fp8=True)
    x = torch.ones(4, 1, 64, dtype=BF16, device="cuda")
    x[0] = 0
    x[1, 0, 5], x[2, 0, 63] = math.inf, math.nan
    cache = a.empty_cache(1)
    t = torch.arange(4, dtype=I32, device="cuda")
    a.append({"k": x, "v": x, "positions": t, "slots": t}, cache)
    for name in ("k", "v"):
        s = cache[name + "_scales"][0, 0]
        assert s[0] == torch.tensor(2.0 ** -100, dtype=F32) / 448 and not torch.isfinite(s[1:3]).any()
        assert (cache[name + "_cache"][0, 0, 0].float() == 0).all() and s[3] == torch.tensor(1.0) / 448
    a.check_errors()


def test_bad_slots_are_not_followed():
    from mhc_residual_boundary_gb300 import capi
    for fp8 in (False, True):
        a, inputs, cache, frequencies = draw(2, fp8)
        rows = cache["k_cache"].shape[0] * CASES[2][4]
        inputs["slots"][1], inputs["slots"][2], inputs["slots"][4], inputs["slots"][5] = rows, -2, 2 ** 31 - 1, -2 ** 31
        q_out = torch.empty(*inputs["q"].shape, dtype=BF16, device="cuda")
        a.append(inputs, {"q_out": q_out, **cache})
        with pytest.raises(capi.MhcError, match="INVALID_ARG"):
            a.check_errors()
        inputs["slots"][[1, 2, 4, 5]] = -1
        check_append(2, fp8, inputs, cache, frequencies, q_out, inputs["q"])
        a.check_errors()


def test_page_strides_and_far_slots():
    """Pages more than 2^31 elements into a buffer that holds keys and values side by side."""
    from mhc_residual_boundary_gb300 import Attention
    kv, d, page = 8, 128, 128
    pages = 2 ** 31 // (kv * d * page) // 2 + 3
    a = Attention(heads=kv, kv_heads=kv, head_dim=d, page_size=page)
    both = torch.zeros(pages, 2, kv, page, d, dtype=BF16, device="cuda")
    x = randn(gen(1), 3, kv, d).to(BF16)
    slots = torch.tensor([pages * page - 1, 5, (pages - 2) * page], dtype=I32, device="cuda")
    a.append({"k": x, "v": -x, "positions": slots, "slots": slots}, {"k_cache": both[:, 0], "v_cache": both[:, 1]})
    for i, s in enumerate(slots.tolist()):
        assert torch.equal(both[s // page, 0, :, s % page], x[i]) and torch.equal(both[s // page, 1, :, s % page], -x[i])
    assert int((both != 0).sum()) == 2 * int((x != 0).sum())
    a.check_errors()


def test_refusals():
    from mhc_residual_boundary_gb300 import capi
    a, inputs, cache, _ = draw(2, False)
    q_out = torch.empty(*inputs["q"].shape, dtype=BF16, device="cuda")

    def refuse(error, match, changed=None, outputs=None):
        with pytest.raises(error, match=match):
            a.append({**inputs, **(changed or {})}, outputs or {"q_out": q_out, **cache})

    refuse(ValueError, "k: expected", {"k": inputs["k"].float()})
    refuse(ValueError, "v must be a tensor on", {"v": inputs["v"].cpu()})
    refuse(ValueError, "positions", {"positions": inputs["positions"].long()})
    refuse(ValueError, "slots", {"slots": inputs["slots"][:-1]})
    refuse(ValueError, "go together", outputs=dict(cache))
    refuse(ValueError, "unknown output", outputs={"q_out": q_out, "x": q_out, **cache})
    refuse(ValueError, "no scales", outputs={"q_out": q_out, "k_scales": q_out, **cache})
    moved = torch.as_strided(inputs["q"], inputs["q"].shape, inputs["q"].stride(), inputs["q"].storage_offset() + 128)
    refuse(capi.MhcError, "q_out reaches over", outputs={**cache, "q_out": moved})
    a.append({n: x[:0] for n, x in inputs.items()}, {"q_out": q_out[:0], **cache})   # nothing to do
    a.check_errors()
