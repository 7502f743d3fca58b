"""Evictions of pools whose rows are no multiple of 16 bytes, on both sides of the
2,124 bytes (531 units of 4) from which splitting a lane's unit into row and
column by a reciprocal needs more than 32 bits."""

import numpy as np
import pytest
import torch

from oracle import l4_oracle as l4
from tests.l4_testutil import Paged
from tests.test_gpu_evict import _evict

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("units", [(4, 1023, 1024, 533), (1, 531, 767, 6), (530, 534, 535, 1021)])
@pytest.mark.parametrize("lens,budget", [([300, 90], 128), ([9000] * 5, 4000)],
                         ids=["two rows a warp", "four rows a warp"])
def test_evict_moves_rows_of_odd_widths(units, lens, budget):
    """units: row widths in 4-byte units (2,124 bytes are 531)."""
    rng = np.random.default_rng(units[0])
    pg = Paged(lens, seed=6)
    mass = rng.exponential(1.0, (len(lens), max(lens))).astype(np.float32)
    pools = [torch.randint(-2 ** 31, 2 ** 31 - 1, (pg.num_pages, 64, w), dtype=torch.int32, device="cuda")
             for w in units]
    dst, table, _, new_lens, _, st = _evict(pg, mass, budget, 2, 30, pools, rng)
    assert st == (0, 0)
    for b, n in enumerate(lens):
        keep = l4.evict_keep(mass[b, :n], budget, 2, 30)
        assert int(new_lens[b]) == len(keep)
        i = np.arange(len(keep))
        to = torch.from_numpy(table[b][i // 64].astype(np.int64) * 64 + i % 64).cuda()
        src = torch.from_numpy(pg.rows(b, keep)).cuda()
        for p, d in zip(pools, dst):
            assert torch.equal(d.flatten(0, 1)[to], p.flatten(0, 1)[src])
