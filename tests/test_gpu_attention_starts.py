"""q_starts that are out of range or decrease: the sequences before them have their outputs, they and all behind them
have no queries, whose rows stay as they are, and check_errors reports it."""
import pytest
import torch

from attention_cases import BF16, F32, I32, check, make_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def run(a, inputs, starts, good, page, guard=3):
    """`good` sequences have their outputs, all else is untouched."""
    from mhc_residual_boundary_gb300 import capi
    t, heads, d = inputs["q"].shape
    whole = {"output": torch.full((t + 2 * guard, heads, d), 3.0, dtype=BF16, device="cuda"),
             "lse": torch.full((t + 2 * guard, heads), 3.0, dtype=F32, device="cuda")}
    out = {name: x[guard:guard + t] for name, x in whole.items()}
    a.attend({**inputs, "q_starts": torch.tensor(starts, dtype=I32, device="cuda")}, out)
    with pytest.raises(capi.MhcError, match="INVALID_ARG"):
        a.check_errors()
    a.check_errors()
    rows = starts[good] if good else 0
    for x in whole.values():
        assert (x[:guard] == 3.0).all() and (x[guard + rows:] == 3.0).all()
    if rows:
        well = {**inputs, "lengths": inputs["lengths"][:good], "pages": inputs["pages"][:good],
                "q_starts": torch.tensor(starts[:good + 1], dtype=I32, device="cuda")}
        check({name: x.contiguous() for name, x in out.items()}, well, page=page)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("starts, good", [
    ([0, 40, 30, 50], 1), ([0, 40, 43, 20], 2), ([0, 40, 43, 51], 2), ([0, 40, 10 ** 6, 50], 1), ([0, 40, -1, 50], 1),
    ([0, -3, 43, 50], 0), ([5, 2, 43, 50], 0), ([-9, 40, 43, 50], 0), ([2 ** 31 - 1, -2 ** 31, 0, 50], 0),
    ([0, 50, 0, 50], 1), ([0, 0, 50, 0], 2), ([0, 12, 12, 11], 2)])
def test_few_sequences(starts, good, fp8):
    from mhc_residual_boundary_gb300 import Attention
    page = 16
    inputs = make_inputs(3, lengths=[100, 60, 33], queries=[40, 3, 7], heads=8, kv=2, d=128, page=page, fp8=fp8)
    with Attention(heads=8, kv_heads=2, head_dim=128, page_size=page, fp8=fp8) as a:
        run(a, inputs, starts, good, page)


@pytest.mark.parametrize("at", [0, 1, 2, 3, 383, 384, 767, 1037, 1099])
def test_many_sequences(at):
    """More sequences than a CTA has threads; sequence `at` ends before it begins."""
    from mhc_residual_boundary_gb300 import Attention
    page, g = 16, torch.Generator().manual_seed(at)
    lengths = torch.randint(0, 60, (1100,), generator=g).tolist()
    queries = torch.randint(1, 4, (1100,), generator=g).tolist()   # some before their sequence's first position
    inputs = make_inputs(5, lengths=lengths, queries=queries, heads=4, kv=2, d=64, page=page, fp8=False)
    starts = inputs["q_starts"].tolist()
    starts[at + 1] = starts[at] - 1
    with Attention(heads=4, kv_heads=2, head_dim=64, page_size=page) as a:
        run(a, inputs, starts, at, page)


def test_places_of_overlapping_sequences_are_not_counted():
    """Starts that go up and down: taken as they are, the sequences' work would be more than 2^31 units."""
    from mhc_residual_boundary_gb300 import Attention
    page, n, pairs, heads, d = 128, 2 ** 17, 1050, 8, 64
    blocks = n // (2 * (128 // 1))
    assert pairs * heads * blocks * (n // 128 // 2) > 2 ** 31
    inputs = make_inputs(7, lengths=[n], queries=[1], heads=heads, kv=heads, d=d, page=page, fp8=False)
    inputs["q"] = torch.randn(n, heads, d, dtype=BF16, device="cuda")
    inputs["pages"] = inputs["pages"].expand(2 * pairs + 1, -1).contiguous()
    inputs["lengths"] = inputs["lengths"].expand(2 * pairs + 1).contiguous()
    with Attention(heads=heads, kv_heads=heads, head_dim=d, page_size=page) as a:
        run(a, inputs, [0, 1] + [0, n] * pairs, 1, page)
