"""What the binding of the norm, rotation, append and attention refuses before it calls the library."""
import pytest

torch = pytest.importorskip("torch")

from paged_top_sparse_gb300 import binding as B
from paged_top_sparse_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def test_page_table_rows_are_the_plans():
    """The kernels step max_pages_per_req entries from request to request: a table with wider rows
    would give request 1 the entries of request 0."""
    plan = B.Plan([1, 1, 1], [10, 300, 0], 4, 2, 64, 1, 3, 9)
    table = torch.zeros((8, 3), dtype=torch.int32)
    flat = torch.zeros(9, dtype=torch.int32)
    for good in (table[:3], table, flat, torch.zeros(20, dtype=torch.int32)):
        assert B._table(good, plan) == good.data_ptr()
    wide = torch.zeros((3, 4), dtype=torch.int32)
    for bad in (wide, torch.zeros((9, 2), dtype=torch.int32), wide[:, :3], table[:2], flat[:8],
                table.long(), torch.zeros((3, 1, 9), dtype=torch.int32)):
        with pytest.raises(ValueError, match="page_table"):
            B._table(bad, plan)
