"""attend against its definition in 64 bits (tests/attention_cases.py derives the
tolerances): one query a sequence and several, BF16 and 8-bit caches, all head and
page sizes, windows and first positions, lengths of zero and one, odd ones, ones
that end inside pages and tiles."""
import math

import pytest
import torch

from attention_cases import BF16, F32, I32, check, define, gen, make_inputs, randn, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handles():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from mhc_residual_boundary_gb300 import Attention
    made = {}

    def get(heads, kv, d, page, fp8):
        key = (heads, kv, d, page, fp8)
        if key not in made:
            made[key] = Attention(heads=heads, kv_heads=kv, head_dim=d, page_size=page, fp8=fp8)
        return made[key]

    yield get
    for a in made.values():
        a.check_errors()
        a.close()


def attend(handles, inputs, page, **kw):
    q, cache = inputs["q"], inputs["k_cache"]
    a = handles(q.shape[1], cache.shape[1], q.shape[2], page, "k_scales" in inputs)
    return a, a.attend(inputs, a.empty_outputs(q.shape[0]), **kw)


# lengths, heads, kv heads, head_dim, page, window, sinks
ONE = [
    ([1], 1, 1, 128, 16, 0, 0),
    ([17], 8, 1, 128, 16, 0, 0),
    ([0, 1, 2, 15, 16, 17, 127, 128, 129], 10, 2, 128, 32, 0, 0),
    ([700], 40, 8, 128, 16, 0, 0),
    ([1000, 3, 0, 513, 64], 16, 1, 128, 64, 0, 0),
    ([255, 256, 257, 31, 33, 1], 12, 4, 64, 16, 0, 0),
    ([5000, 1, 77], 14, 2, 64, 128, 0, 0),
    ([333, 12, 40, 100, 99], 8, 2, 128, 16, 40, 0),
    ([333, 12, 40, 47, 100, 99], 8, 2, 128, 64, 40, 7),
    ([2000, 300, 301, 302], 9, 3, 64, 32, 300, 4),
    ([900, 20], 4, 2, 128, 128, 1, 0),
    ([900, 20], 4, 2, 128, 32, 16, 1000),
    ([0, 0, 0], 6, 3, 64, 64, 0, 0),
    ([20011], 3, 1, 128, 64, 0, 0),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(ONE)))
def test_one_query(handles, case, fp8):
    lengths, heads, kv, d, page, window, sinks = ONE[case]
    inputs = make_inputs(case, lengths=lengths, heads=heads, kv=kv, d=d, page=page, fp8=fp8)
    a, out = attend(handles, inputs, page, window=window, sinks=sinks)
    check(out, inputs, page=page, window=window, sinks=sinks)
    a.check_errors()


@pytest.mark.parametrize("fp8", [False, True])
def test_one_query_many_sequences(handles, fp8):
    g = torch.Generator().manual_seed(5)
    lengths = torch.randint(0, 200, (700,), generator=g).tolist()
    inputs = make_inputs(3, lengths=lengths, heads=4, kv=2, d=64, page=16, fp8=fp8)
    a, out = attend(handles, inputs, 16)
    check(out, inputs, page=16)
    a.check_errors()


# (length, queries) of the sequences, heads, kv heads, head_dim, page, window, sinks
SEVERAL = [
    ([(1, 1)], 1, 1, 128, 16, 0, 0),
    ([(17, 17)], 40, 8, 128, 16, 0, 0),
    ([(129, 129), (128, 128), (127, 127), (1, 1), (64, 3)], 4, 2, 128, 32, 0, 0),
    ([(300, 300)], 6, 1, 128, 64, 0, 0),
    ([(200, 40), (0, 0), (77, 77), (50, 0), (513, 130)], 10, 2, 128, 16, 0, 0),
    ([(900, 4), (1200, 4), (3, 3), (128, 4)], 16, 2, 128, 64, 0, 0),
    ([(400, 400)], 8, 2, 64, 16, 0, 0),
    ([(700, 260), (129, 100)], 7, 1, 64, 128, 0, 0),
    ([(500, 500), (90, 30)], 8, 2, 128, 64, 100, 0),
    ([(500, 500), (390, 130)], 8, 2, 128, 32, 100, 5),
    ([(640, 300)], 12, 4, 64, 16, 64, 200),
    ([(350, 350)], 3, 3, 64, 64, 1, 1),
    ([(5, 9), (0, 4), (300, 300)], 4, 1, 128, 32, 0, 0),      # more queries than positions
    ([(5, 9), (40, 44)], 4, 1, 64, 32, 8, 2),
    ([(2500, 70)], 4, 1, 128, 64, 0, 0),
    ([(150, 9)], 128, 1, 128, 64, 0, 0),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(SEVERAL)))
def test_several_queries(handles, case, fp8):
    sequences, heads, kv, d, page, window, sinks = SEVERAL[case]
    inputs = make_inputs(100 + case, lengths=[n for n, _ in sequences], queries=[q for _, q in sequences], heads=heads,
                         kv=kv, d=d, page=page, fp8=fp8)
    a, out = attend(handles, inputs, page, window=window, sinks=sinks)
    check(out, inputs, page=page, window=window, sinks=sinks)
    a.check_errors()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,kv", [(17, 1), (64, 2), (128, 1)])
def test_one_query_of_many_heads(handles, heads, kv, fp8):
    inputs = make_inputs(7, lengths=[600, 1, 0, 129], heads=heads, kv=kv, d=128, page=32, fp8=fp8)
    a, out = attend(handles, inputs, 32, window=200, sinks=3)
    check(out, inputs, page=32, window=200, sinks=3)
    a.check_errors()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("several", [False, True])
def test_scale_and_large_scores(handles, several, fp8):
    """Scores of several hundred: all but the largest vanish, and the largest may come last."""
    inputs = make_inputs(11, lengths=[300, 40], queries=[20, 3] if several else None, heads=8, kv=2, d=128, page=16,
                         fp8=fp8, size=20.0)
    for scale in (None, 0.5, 1e-3):
        a, out = attend(handles, inputs, 16, scale=scale)
        check(out, inputs, page=16, scale=scale)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("several", [False, True])
def test_one_row_set_in_many_parts(handles, several, fp8):
    """A long sequence of one kv head: every CTA has a part of it, and the parts are joined in two steps."""
    lengths, queries = ([40000, 7], [3, 2]) if several else ([40000], None)
    inputs = make_inputs(71, lengths=lengths, queries=queries, heads=8, kv=1, d=128, page=128, fp8=fp8)
    a, out = attend(handles, inputs, 128)
    check(out, inputs, page=128)
    again = attend(handles, inputs, 128)[1]
    assert all(torch.equal(out[n], again[n]) for n in out)
    inputs = make_inputs(72, lengths=[90000], queries=[130] if several else None, heads=16, kv=1, d=64, page=64, fp8=fp8)
    a, out = attend(handles, inputs, 64)
    check(out, inputs, page=64)
    a.check_errors()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("several", [False, True])
def test_hidden_places_hold_anything(handles, several, fp8):
    """NaN and infinities behind a sequence's end, before its window, in pages of nobody and in rows of q_starts'
    other sequences change nothing."""
    page, window, sinks = 32, 50, 3
    lengths, queries = [205, 17, 100], [60, 5, 1] if several else None
    inputs = make_inputs(13, lengths=lengths, queries=queries, heads=8, kv=2, d=128, page=page, fp8=fp8)
    want = define(inputs, window=window, sinks=sinks, page=page)
    if several:
        inputs["q"] = torch.cat([inputs["q"], torch.full_like(inputs["q"][:4], math.nan)])
    used = torch.zeros(inputs["k_cache"].shape[0], page, dtype=torch.bool, device="cuda")
    for s, n in enumerate(lengths):
        first = n - (queries[s] if several else 1)   # the first query's position
        for j in range(n):
            if j > first - window or j < sinks:
                used[inputs["pages"][s, j // page], j % page] = True
    for k, name in enumerate(("k_cache", "v_cache", "k_scales", "v_scales")):
        if name not in inputs:
            continue
        x = inputs[name]
        poison = torch.tensor([math.nan, math.inf, -math.inf], device="cuda")[torch.arange(page, device="cuda") % 3]
        mask = ~used[:, None, :].expand(x.shape[:3])
        if x.dim() == 3:
            x[mask] = poison.expand(x.shape)[mask]
        elif fp8:
            x.view(torch.uint8)[mask] = 0x7f   # NaN
        else:
            x[mask] = poison[:, None].expand(x.shape)[mask].to(x.dtype)
    a, out = attend(handles, inputs, page, window=window, sinks=sinks)
    check(out, inputs, page=page, want=want)
    a.check_errors()


@pytest.mark.parametrize("d,window,sinks,heads", [(128, 0, 0, 8), (128, 70, 2, 8), (64, 0, 0, 8), (64, 33, 5, 8),
                                                  (128, 0, 0, 2), (128, 150, 2, 2), (64, 0, 0, 2)])
@pytest.mark.parametrize("fp8", [False, True])
def test_values_that_some_rows_do_not_see(handles, fp8, d, window, sinks, heads):
    """Infinities and NaN among the values reach the rows that see them, in their columns, and no others: neither
    earlier queries nor later ones that a window keeps from them, in one tile with those that do."""
    page, lengths, queries = 16, [300, 260, 40], [300, 90, 40]
    inputs = make_inputs(59, lengths=lengths, queries=queries, heads=heads, kv=2, d=d, page=page, fp8=fp8)
    values = inputs["v_cache"]
    spots = [(0, 100, 3, math.inf), (0, 101, 7, math.nan), (0, 40, d - 1, -math.inf), (0, 1, 5, math.inf),
             (0, 2, 5, -math.inf), (1, 200, 0, math.nan), (1, 259, 33, -math.inf), (2, 39, 1, math.inf)]
    for s, position, column, value in spots:
        at = int(inputs["pages"][s, position // page]), 1, position % page, column
        if fp8:
            values.view(torch.uint8)[at] = 0x7f   # NaN: E4M3 has no infinities
        else:
            values[at] = value
    out, lse, mag, size = define(inputs, window=window, sinks=sinks, page=page)
    a, got = attend(handles, inputs, page, window=window, sinks=sinks)
    assert torch.equal(torch.isfinite(got["output"]), torch.isfinite(out))
    assert torch.equal(torch.isnan(got["output"]), torch.isnan(out)) and torch.isnan(out).any()
    infinite = torch.isinf(out)
    assert torch.equal(got["output"][infinite].double(), out[infinite])
    fine = torch.isfinite(out)
    got["output"] = torch.where(fine, got["output"], 0.0)
    check(got, inputs, page=page, want=(torch.where(fine, out, 0.0), lse, torch.where(fine, mag, 0.0), size))
    a.check_errors()


@pytest.mark.parametrize("several", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_queries_and_keys_that_are_not_finite(handles, several, fp8):
    """A NaN among the queries, or in a key that a query sees, makes that query and head NaN and no other."""
    inputs = make_inputs(61, lengths=[200, 150], queries=[150, 9] if several else None, heads=8, kv=2, d=128, page=32,
                         fp8=fp8)
    want = define(inputs, page=32)
    inputs["q"][1, 3, 77] = math.nan
    # the last position's key of sequence 0: seen by its last query only
    at = int(inputs["pages"][0, 199 // 32]), 1, 199 % 32, 5
    if fp8:
        inputs["k_cache"].view(torch.uint8)[at] = 0x7f
    else:
        inputs["k_cache"][at] = math.nan
    a, got = attend(handles, inputs, 32)
    nan = torch.zeros(got["lse"].shape, dtype=torch.bool, device="cuda")
    nan[1, 3] = True
    nan[149 if several else 0, 4:] = True
    assert torch.equal(torch.isnan(got["lse"]), nan) and torch.isnan(got["output"][nan]).all()
    got = {"output": torch.where(nan[..., None], want[0].to(BF16), got["output"]),
           "lse": torch.where(nan, want[1].float(), got["lse"])}
    check(got, inputs, page=32, want=want)
    a.check_errors()


@pytest.mark.parametrize("d,fp8", [(128, False), (128, True), (64, False), (64, True)])
def test_a_wait_that_gives_up(d, fp8):
    """Without its copies the kernel gives up, check_errors says so once, and the next call is right."""
    from mhc_residual_boundary_gb300 import Attention, capi
    a = Attention(heads=8, kv_heads=2, head_dim=d, page_size=16, fp8=fp8)
    inputs = make_inputs(67, lengths=[300, 5000], queries=[300, 4], heads=8, kv=2, d=d, page=16, fp8=fp8)
    out = a.empty_outputs(304)
    capi.mhc_test_stall_attention_copies(True)
    try:
        a.attend(inputs, out)
        with pytest.raises(capi.MhcError, match="TIMEOUT"):
            a.check_errors()
    finally:
        capi.mhc_test_stall_attention_copies(False)
    a.check_errors()
    a.attend(inputs, out)
    a.check_errors()
    check(out, inputs, page=16)
    a.close()


def test_strides(handles):
    """Queries inside a packed projection, output inside wider rows, a table of wider rows, a cache whose pages hold
    keys and values side by side."""
    heads, kv, d, page = 6, 2, 128, 16
    for queries in (None, [30, 7]):
        inputs = make_inputs(17, lengths=[100, 50], queries=queries, heads=heads, kv=kv, d=d, page=page, fp8=False)
        t = inputs["q"].shape[0]
        want = define(inputs, page=page)
        packed = randn(gen(1), t, heads + 2 * kv, d).to(BF16)
        packed[:, :heads] = inputs["q"]
        both = torch.stack([inputs["k_cache"], inputs["v_cache"]], 1)
        table = torch.full((2, inputs["pages"].shape[1] + 3), -7, dtype=I32, device="cuda")
        table[:, :-3] = inputs["pages"]
        moved = {**inputs, "q": packed[:, :heads], "k_cache": both[:, 0], "v_cache": both[:, 1], "pages": table[:, :-3]}
        wide = torch.full((t, heads + 1, d), 5.0, dtype=BF16, device="cuda")
        a = handles(heads, kv, d, page, False)
        out = a.attend(moved, {"output": wide[:, :heads]})
        check(out, inputs, page=page, want=want)
        assert (wide[:, heads] == 5.0).all()


@pytest.mark.parametrize("first, row", [(8, 256), (0, 264), (8, 264)])
def test_output_rows_at_odd_multiples_of_16_bytes(handles, first, row):
    heads, kv, d, page = 2, 1, 128, 16
    for queries in (None, [200, 9]):
        inputs = make_inputs(43, lengths=[333, 50], queries=queries, heads=heads, kv=kv, d=d, page=page, fp8=False)
        t = inputs["q"].shape[0]
        flat = torch.full((t * row + 16,), 5.0, dtype=BF16, device="cuda")
        assert flat.data_ptr() % 32 == 0
        output = flat[first:first + t * row].view(t, row)[:, :heads * d].unflatten(1, (heads, d))
        out = handles(heads, kv, d, page, False).attend(inputs, {"output": output})
        check(out, inputs, page=page)
        untouched = torch.ones_like(flat, dtype=torch.bool)
        untouched[first:first + t * row].view(t, row)[:, :heads * d] = False
        assert (flat[untouched] == 5.0).all()


def test_rows_behind_the_last_sequence_stay(handles):
    inputs = make_inputs(19, lengths=[100, 50], queries=[30, 7], heads=4, kv=2, d=64, page=16, fp8=False)
    want = define(inputs, page=16)
    inputs["q"] = torch.cat([inputs["q"], torch.randn_like(inputs["q"][:20])])
    a = handles(4, 2, 64, 16, False)
    out = a.empty_outputs(57)
    for x in out.values():
        x.fill_(3.0)
    a.attend(inputs, out)
    check(out, inputs, page=16, want=want)
    assert (out["output"][37:] == 3.0).all() and (out["lse"][37:] == 3.0).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_same_bits_each_time(handles, fp8):
    for queries in (None, [700, 4, 33]):
        inputs = make_inputs(23, lengths=[3000, 4, 100], queries=queries, heads=8, kv=1, d=128, page=64, fp8=fp8)
        a, first = attend(handles, inputs, 64)
        for _ in range(5):
            _, again = attend(handles, inputs, 64)
            assert all(torch.equal(first[n], again[n]) for n in first)


def test_sequences_share_pages(handles):
    """Two sequences with a common prefix name the same pages."""
    inputs = make_inputs(29, lengths=[200, 230], heads=8, kv=2, d=128, page=16, fp8=False)
    inputs["pages"][1, :10] = inputs["pages"][0, :10]
    a, out = attend(handles, inputs, 16)
    check(out, inputs, page=16)


def test_one_query_by_either_form(handles):
    """A q_starts of single queries names the same rows as none."""
    inputs = make_inputs(31, lengths=[500, 0, 65, 1], heads=8, kv=2, d=128, page=16, fp8=False)
    a, out = attend(handles, inputs, 16)
    inputs["q_starts"] = torch.arange(5, dtype=I32, device="cuda")
    _, out = attend(handles, inputs, 16)
    check(out, inputs, page=16)


@pytest.mark.parametrize("several", [False, True])
def test_graph_and_streams(handles, several):
    """A captured call, replayed on new inputs, between calls on another stream."""
    inputs = make_inputs(37, lengths=[900, 31], queries=[9, 2] if several else None, heads=8, kv=2, d=128, page=16,
                         fp8=False)
    a, out = attend(handles, inputs, 16)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.attend(inputs, out)
        a.attend(inputs, out)
    other = make_inputs(38, lengths=[900, 31], queries=[9, 2] if several else None, heads=8, kv=2, d=128, page=16,
                        fp8=False)
    for name in ("q", "k_cache", "v_cache", "pages"):
        inputs[name].copy_(other[name])
    inputs["lengths"].copy_(torch.tensor([555, 30], dtype=I32))
    stream = torch.cuda.Stream()
    for _ in range(3):
        out["output"].zero_()
        graph.replay()
        check(out, inputs, page=16)
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            _, again = attend(handles, inputs, 16)
        torch.cuda.current_stream().wait_stream(stream)
        assert torch.equal(again["output"], out["output"])
    a.check_errors()


def test_bad_indices_are_not_followed(handles):
    """Pages, lengths and starts out of range: their positions are taken as not there, and check_errors says so."""
    from mhc_residual_boundary_gb300 import capi
    for queries in (None, [40, 3]):
        inputs = make_inputs(41, lengths=[100, 60], queries=queries, heads=4, kv=2, d=128, page=16, fp8=False)
        a = handles(4, 2, 128, 16, False)
        pages = inputs["k_cache"].shape[0]
        for bad in (-1, pages, 2 ** 31 - 1, -2 ** 31):
            broken = {**inputs, "pages": inputs["pages"].clone()}
            broken["pages"][1, 1] = bad
            out = a.attend(broken, a.empty_outputs(inputs["q"].shape[0]))
            with pytest.raises(capi.MhcError, match="INVALID_ARG"):
                a.check_errors()
            check(out, inputs, page=16, want=define(inputs, page=16, gone=[(1, 1)]))
        for bad in (-5, 10 ** 6):
            broken = {**inputs, "lengths": torch.tensor([100, bad], dtype=I32, device="cuda")}
            broken["pages"] = inputs["pages"].clamp(min=0)
            out = a.attend(broken, a.empty_outputs(inputs["q"].shape[0]))
            with pytest.raises(capi.MhcError, match="INVALID_ARG"):
                a.check_errors()
            assert torch.isfinite(out["output"].float()).all()
        if queries:
            for starts in ([0, -3, 43], [0, 40, 10 ** 6], [0, 43, 20], [-9, 40, 43], [5, 2, 43]):
                broken = {**inputs, "q_starts": torch.tensor(starts, dtype=I32, device="cuda")}
                a.attend(broken, a.empty_outputs(43))
                with pytest.raises(capi.MhcError, match="INVALID_ARG"):
                    a.check_errors()
        _, out = attend(handles, inputs, 16)
        check(out, inputs, page=16)
        a.check_errors()


def test_far_offsets(handles):
    """Pages more than 2^31 elements into a cache."""
    from mhc_residual_boundary_gb300 import Attention
    page, kv, d = 128, 8, 128
    pages = 2 ** 31 // (page * kv * d) + 40
    a = Attention(heads=8, kv_heads=kv, head_dim=d, page_size=page)
    small = make_inputs(43, lengths=[1000, 4000], heads=8, kv=kv, d=d, page=page, fp8=False)
    count = small["k_cache"].shape[0]
    far = {n: torch.zeros(pages, kv, page, d, dtype=BF16, device="cuda") for n in ("k_cache", "v_cache")}
    for n in far:
        far[n][pages - count:] = small[n]
    table = torch.where(small["pages"] >= 0, small["pages"] + (pages - count), -1).int()
    for queries in (None, [37, 6]):
        inputs = dict(small) if queries is None else {**small, "q": randn(gen(2), 43, 8, d).to(BF16),
                                                      "q_starts": torch.tensor([0, 37, 43], dtype=I32, device="cuda")}
        out = a.attend({**inputs, **far, "pages": table}, a.empty_outputs(inputs["q"].shape[0]))
        check(out, inputs, page=page)
    a.check_errors()
    a.close()


def test_nothing_to_do(handles):
    a = handles(4, 2, 64, 16, False)
    inputs = make_inputs(47, lengths=[5], heads=4, kv=2, d=64, page=16, fp8=False)
    none = {**inputs, "q": inputs["q"][:0], "lengths": inputs["lengths"][:0], "pages": inputs["pages"][:0]}
    a.attend(none, a.empty_outputs(0))
    a.check_errors()


def test_refusals(handles):
    a = handles(4, 2, 64, 16, False)
    from mhc_residual_boundary_gb300 import capi
    inputs = make_inputs(53, lengths=[50, 20], heads=4, kv=2, d=64, page=16, fp8=False)
    out = a.empty_outputs(2)

    def refuse(error, match, changed=None, outputs=None, **kw):
        with pytest.raises(error, match=match):
            a.attend({**inputs, **(changed or {})}, outputs or out, **kw)

    refuse(ValueError, "q: expected", {"q": inputs["q"].float()})
    refuse(ValueError, "q: expected", {"q": inputs["q"].transpose(1, 2).contiguous().transpose(1, 2)})
    refuse(ValueError, "q must be a tensor on", {"q": inputs["q"].cpu()})
    refuse(ValueError, "lengths", {"lengths": inputs["lengths"].long()})
    refuse(ValueError, "pages", {"pages": inputs["pages"].t()})
    refuse(ValueError, "k_cache", {"k_cache": inputs["k_cache"][:, :, :8]})
    refuse(ValueError, "v_cache", {"v_cache": inputs["v_cache"][:-1]})
    refuse(ValueError, "q_starts", {"q_starts": torch.zeros(2, dtype=I32, device="cuda")})
    refuse(ValueError, "no scales", {"k_scales": torch.zeros(1, device="cuda")})
    refuse(ValueError, "unknown output", outputs={**out, "weights": out["lse"]})
    refuse(capi.MhcError, "one token", {"lengths": inputs["lengths"][:1], "pages": inputs["pages"][:1]})
    refuse(capi.MhcError, "window", window=-1)
    refuse(capi.MhcError, "sinks", sinks=-1)
    for scale in (0.0, -1.0, math.inf, math.nan):
        refuse(capi.MhcError, "scale", scale=scale)
    refuse(capi.MhcError, "reaches over q", outputs={"output": inputs["q"]})
    odd = torch.zeros(2 * 4 * 64 + 8, dtype=BF16, device="cuda")[1:513].view(2, 4, 64)
    refuse(capi.MhcError, "aligned", {"q": odd})
    a.check_errors()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("several", [False, True])
def test_windows_of_any_size(handles, several, fp8):
    """A window of at least the length hides nothing, up to the largest integer; also beside queries that lie before
    their sequence."""
    inputs = make_inputs(47, lengths=[5, 300, 41], queries=[9, 40, 41] if several else None, heads=8, kv=2, d=64, page=16,
                         fp8=fp8)
    want = define(inputs, page=16)
    for window, sinks in ((301, 0), (2 ** 30, 2), (2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1)):
        _, out = attend(handles, inputs, 16, window=window, sinks=sinks)
        check(out, inputs, page=16, want=want)
    want = define(inputs, page=16, window=3, sinks=10 ** 6)
    _, out = attend(handles, inputs, 16, window=3, sinks=2 ** 31 - 1)
    check(out, inputs, page=16, want=want)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("several", [False, True])
def test_small_scales_and_queries(handles, several, fp8):
    """Scales down to FP32's least and queries of zero: the weights are equal, lse is the logarithm of their number."""
    inputs = make_inputs(53, lengths=[200, 37], queries=[9, 37] if several else None, heads=4, kv=2, d=128, page=16,
                         fp8=fp8)
    inputs["q"][0] = 0
    for scale in (1.0, 1e-3, 1e-30, 1e-38, 2.0 ** -149):
        _, out = attend(handles, inputs, 16, scale=scale)
        check(out, inputs, page=16, scale=scale)



def test_scales_that_are_not_finite_in_the_exponent_are_refused(handles):
    from mhc_residual_boundary_gb300 import capi
    inputs = make_inputs(59, lengths=[50], heads=4, kv=2, d=64, page=16, fp8=False)
    with pytest.raises(capi.MhcError, match="scale"):
        attend(handles, inputs, 16, scale=3e38)


def test_two_handles_at_once():
    """Calls of two handles on two streams, side by side: the bits that each has alone."""
    from mhc_residual_boundary_gb300 import Attention
    calls = []
    for seed, queries, fp8 in ((61, [300, 40], False), (62, [200, 90], True), (63, None, False)):
        inputs = make_inputs(seed, lengths=[3000, 700], queries=queries, heads=8, kv=2, d=64, page=16, fp8=fp8)
        a = Attention(heads=8, kv_heads=2, head_dim=64, page_size=16, fp8=fp8)
        alone = a.attend(inputs, a.empty_outputs(inputs["q"].shape[0]))
        calls.append((a, inputs, alone, a.empty_outputs(inputs["q"].shape[0]), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for a, inputs, _, out, stream in calls:
            a.attend(inputs, out, stream=stream)
    torch.cuda.synchronize()
    for a, _, alone, out, _ in calls:
        a.check_errors()
        assert all(torch.equal(alone[n], out[n]) for n in alone)
        a.close()
