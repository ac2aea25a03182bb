"""The wrapper's two forms of a call's checks, without a GPU: what passes the one condition of the usual layout has the
arguments that the checks tensor by tensor give, and what these refuse does not pass it."""
import itertools

import pytest
import torch

from mhc_residual_boundary_gb300 import attention

BF16, F8, F32, I32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.int32
HEADS, KV, D, PAGE, PAGES = 6, 2, 64, 16, 5


@pytest.fixture
def make(monkeypatch):
    def made(fp8):
        a = object.__new__(attention.Attention)
        a.device, a._index, a.handle = torch.device("cpu"), -1, None   # a tensor's get_device() on the CPU
        a.heads, a.kv_heads, a.head_dim, a.page_size, a.fp8 = HEADS, KV, D, PAGE, fp8
        a._page, a._cache_dtype, a._scale = KV * PAGE * D, F8 if fp8 else BF16, D ** -0.5
        a._append, a._attend, a.args = "append", "attend", []
        a._call = lambda fn, args, stream: a.args.append((fn, args))
        return a
    return made


def cache(fp8):
    out = {n: torch.zeros(PAGES, KV, PAGE, D, dtype=F8 if fp8 else BF16) for n in ("k_cache", "v_cache")}
    if fp8:
        out.update({n: torch.ones(PAGES, KV, PAGE, dtype=F32) for n in ("k_scales", "v_scales")})
    return out


def append_call(fp8, t, queries=True):
    packed = torch.zeros(t, HEADS + 2 * KV, D, dtype=BF16)
    q, k, v = packed.split([HEADS, KV, KV], 1)
    inputs = {"k": k, "v": v, "positions": torch.zeros(t, dtype=I32), "slots": torch.zeros(t, dtype=I32)}
    outputs = cache(fp8)
    if queries:
        inputs["q"], outputs["q_out"] = q, torch.zeros(t, HEADS, D, dtype=BF16)
    return inputs, outputs


def attend_call(fp8, t, s, starts, lse):
    inputs = {"q": torch.zeros(t, HEADS, D, dtype=BF16), **cache(fp8), "pages": torch.zeros(s, 3, dtype=I32),
              "lengths": torch.zeros(s, dtype=I32)}
    if starts:
        inputs["q_starts"] = torch.zeros(s + 1, dtype=I32)
    outputs = {"output": torch.zeros(t, HEADS, D, dtype=BF16)}
    if lse:
        outputs["lse"] = torch.zeros(t, HEADS, dtype=F32)
    return inputs, outputs


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("t", [1, 2, 7])
def test_append_arguments(make, monkeypatch, fp8, t):
    a = make(fp8)
    inputs, outputs = append_call(fp8, t)
    with monkeypatch.context() as m:   # the usual layout does not need the other form
        m.setattr(a, "_append_args", lambda *x: pytest.fail("the usual layout"), raising=False)
        assert a.append(inputs, outputs) is outputs
        a.append(inputs, {**outputs, "q_out": inputs["q"]})
    assert a.args == [("append", a._append_args(inputs, outputs)),
                      ("append", a._append_args(inputs, {**outputs, "q_out": inputs["q"]}))]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("t, s, starts, lse, kw", [
    (4, 4, False, True, {}), (4, 4, False, False, {"window": 5, "sinks": 2}), (9, 3, True, True, {"scale": 0.25}),
    (1, 1, False, True, {}), (9, 1, True, False, {})])
def test_attend_arguments(make, monkeypatch, fp8, t, s, starts, lse, kw):
    a = make(fp8)
    inputs, outputs = attend_call(fp8, t, s, starts, lse)
    with monkeypatch.context() as m:
        m.setattr(a, "_attend_args", lambda *x: pytest.fail("the usual layout"), raising=False)
        assert a.attend(inputs, outputs, **kw) is outputs
    want = a._attend_args(inputs, outputs, kw.get("window", 0), kw.get("sinks", 0), kw.get("scale"))
    assert a.args == [("attend", want)]


def spoiled(x):
    """Tensors that are not what x was, each in one way."""
    yield x.to(torch.float64) if x.dtype != F8 else x.view(torch.uint8)
    yield x[:-1] if x.shape[0] > 1 else x.repeat(2, *[1] * (x.dim() - 1))
    if x.dim() > 1:
        yield x[..., :-1]
        yield x.repeat(*[1] * (x.dim() - 1), 2)[..., ::2]
        if x.dim() == 3:
            yield x.transpose(0, 2).contiguous().transpose(0, 2)
    else:
        yield x.repeat_interleave(2)[::2]


def calls(make, fp8):
    a = make(fp8)
    inputs, outputs = append_call(fp8, 4)
    yield a, a.append, inputs, outputs
    for starts, lse in itertools.product((False, True), repeat=2):
        inputs, outputs = attend_call(fp8, 4, 4, starts, lse)
        yield a, a.attend, inputs, outputs


@pytest.mark.parametrize("fp8", [False, True])
def test_what_one_form_refuses_the_call_refuses(make, fp8):
    """One tensor at a time: another type or shape, elements that are not dense.  Of these only a page table with wider
    rows than its pages passes, through the checks tensor by tensor."""
    refused = passed = 0
    for a, call, inputs, outputs in calls(make, fp8):
        for which, name in [(0, n) for n in inputs] + [(1, n) for n in outputs]:
            for x in spoiled((inputs, outputs)[which][name]):
                given = [dict(inputs), dict(outputs)]
                given[which][name] = x
                form = a._append_args if call == a.append else lambda i, o: a._attend_args(i, o, 0, 0, None)
                try:
                    want = form(*given)
                except (ValueError, IndexError):
                    want = None
                a.args.clear()
                if want is None:
                    with pytest.raises((ValueError, IndexError)):
                        call(*given)
                    assert not a.args
                    refused += 1
                else:
                    call(*given)
                    assert a.args[0][1] == want
                    passed += 1
    assert refused > 100 and passed == 4, (refused, passed)


@pytest.mark.parametrize("fp8", [False, True])
def test_names_and_scales(make, fp8):
    for a, call, inputs, outputs in calls(make, fp8):
        with pytest.raises(ValueError, match="unknown output"):
            call(inputs, {**outputs, "weights": torch.zeros(1)})
        if not fp8:
            for name in ("k_scales", "v_scales"):
                with pytest.raises(ValueError, match="no scales"):
                    where = {name: torch.ones(PAGES, KV, PAGE)}
                    if call == a.append:
                        call(inputs, {**outputs, **where})
                    else:
                        call({**inputs, **where}, outputs)
    a = make(fp8)
    inputs, outputs = append_call(fp8, 4)
    for name, given in (("q", inputs), ("q_out", outputs)):
        kept = given.pop(name)
        with pytest.raises(ValueError, match="go together"):
            a.append(inputs, outputs)
        given[name] = kept
    assert not a.args
