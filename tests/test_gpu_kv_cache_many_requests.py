"""Block tables of more requests than the GPU has threads for at once."""
import numpy as np
import pytest

from oracle import kv_cache as oracle
from test_gpu_kv_cache import run_tables, same_plan, tables_problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,page,hi_ctx,hi_new", [(5000, 16, 60, 3), (20011, 64, 100, 1)])
def test_block_tables_of_thousands_of_requests(n, page, hi_ctx, hi_new):
    """Ten and forty requests a thread: the walks inside a thread's share."""
    ctx, new, table, free, nb = tables_problem(n, page, hi_ctx, hi_new, n)
    T = int(new.sum()) + 7
    ref = oracle.block_tables(ctx, new, table, free, page, nb, T)
    assert ref[5][2] == 0
    same_plan(run_tables(ctx, new, table, free, page, nb, T), ref)
    short = free[:len(free) // 3]  # the later requests lack pages
    ref = oracle.block_tables(ctx, new, table, short, page, nb, T)
    assert ref[5][2] > 0
    same_plan(run_tables(ctx, new, table, short, page, nb, T), ref)
    assert np.array_equal(ref[1], np.minimum(np.concatenate([[0], np.cumsum(np.maximum(new, 0))]), T))
