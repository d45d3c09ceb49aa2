"""What the runner of packed attention holds without a GPU."""
import pytest
import torch

from rank_bottleneck_block_gb300 import inputs as I
from rank_bottleneck_block_gb300 import runner as R


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from rank_bottleneck_block_gb300 import build

    build.build()


def test_rows_of_no_sequence_begin_as_zeros():
    """No call writes them, and what sums over all rows (a projection's weight gradient, the norm's gains) reads them."""
    shape = I.PackedShape(T=300, nseq=2, Hq=4, Hk=2, dh=64)
    case = I.make_packed_case(shape, [200, 77], first=3)
    was = torch.are_deterministic_algorithms_enabled()
    torch.use_deterministic_algorithms(True)  # new memory holds NaN
    try:
        run = R.PackedAttention(shape, case, device="cpu")
    finally:
        torch.use_deterministic_algorithms(was)
    for n in ("o", "lse", "dq", "dk", "dv"):
        assert (getattr(run, n) == 0).all(), n
