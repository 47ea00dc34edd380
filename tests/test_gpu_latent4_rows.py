"""The 4-bit latent cache at shapes of their own: many rows of one tile, rows that share one sequence's pages, appends
and reads over many blocks (needs a B200).  Tolerances: those of test_gpu_latent4.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import long_context_sparse_11_b200 as dsa  # noqa: E402
from test_gpu_kernels import i32_dev  # noqa: E402
from test_gpu_latent4 import SCALE, check_attention, lib, run_attention, selection  # noqa: E402,F401


@pytest.mark.parametrize("lens,rows,k", [([200] * 1000, 2, 96), ([130] * 1500, 1, 128), ([9] * 900, 3, 1)])
def test_rows_of_one_tile_over_and_over(lens, rows, k):
    """13 rows of one tile and more per SM, every row with data of its own: the same bits each time."""
    rng = np.random.default_rng(k)
    idx = selection(rng, lens, k)
    idx[7] = -1
    qd, view, kv, out, lse = run_attention(rng, lens, rows, k, idx)
    idxd = i32_dev(idx)
    for _ in range(30):
        o, e = dsa.sparse_mla_attn(qd, view, idxd, k, SCALE, rows)
        assert torch.equal(o, out) and torch.equal(e, lse)
    dsa.sync_status()
    some = sorted({0, 7, len(lens) - 1} | {int(b) for b in rng.integers(0, len(lens), 12)})
    take = [r for b in some for r in range(b * rows, (b + 1) * rows)]
    check_attention(qd[take], [kv[b] for b in some], idx[some], rows, out[take], lse[take])
