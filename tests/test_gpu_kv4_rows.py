"""Requests on both sides of the bounds between the attention kernels: 24, 25, 32 and 33 query rows per kv head, in batches
that fill the GPU and in small ones."""
import numpy as np
import pytest

from test_gpu_kv4 import _batch, _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("batch,q_heads,heads", [(70, 1, 1), (9, 8, 8), (3, 2, 2)])
@pytest.mark.parametrize("rows", [24, 25, 28, 32, 33])
def test_rows_around_the_bounds(rows, batch, q_heads, heads, dim):
    """All requests with the same number of rows, and one each of 1, 24, 25, 32, 33 and 70 in their places."""
    lens = np.random.default_rng(rows).integers(70, 300, batch).tolist()
    nqs = [rows] * batch
    _check(*_batch(lens, nqs, 32, heads, dim, q_heads, seed=rows + dim))
    for i, n in enumerate((1, 24, 25, 32, 33, 70)[:batch]):
        nqs[-1 - i] = n
    _check(*_batch(lens, nqs, 32, heads, dim, q_heads, seed=rows + dim + 1), window=100)
