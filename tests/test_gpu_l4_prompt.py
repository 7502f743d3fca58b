"""The whole step over a 4-bit cache on prompt chunks of middling length, where the
key scan of one call spreads over many key tiles and row groups."""

import numpy as np
import pytest
import torch

import sparse_attention_scores_b200 as dsa
from oracle import dsa_oracle as orc
from oracle import l4_oracle as l4
from tests.l4_testutil import Paged, attention_bounds, bf16_cuda, random_l4, to_bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,pos0,k", [(803, 0, 256), (517, 1100, 300), (1000, 37, 64)])
def test_forward_of_a_prompt_chunk(n, pos0, k):
    rng = np.random.default_rng(n)
    H, R, P, HI, DI = 16, 256, 64, 32, 128
    pg = Paged([pos0 + n], seed=n)
    pool, values = random_l4(rng, pg.num_pages, R + P)
    keys = rng.integers(-3, 4, (pg.num_pages * 64, DI)).astype(np.float64)
    q_idx = rng.integers(-3, 4, (n, HI, DI)).astype(np.float64)
    w = rng.integers(0, 4, (n, HI)).astype(np.float64)
    q = to_bf16(rng.standard_normal((n, H, R + P)))
    cache = pg.cache()
    dims = dsa.Dims(n, HI, DI, k, H, R, P, 1, pos0, 0.0625)
    idx = torch.full((n, k), -7, dtype=torch.int32, device="cuda")
    out, lse = torch.zeros(n, H, R, device="cuda"), torch.zeros(n, H, device="cuda")
    ws = dsa.l4_workspace(dsa.L4_OP_ATTENTION_FORWARD, dims, cache)
    dsa.dsa_attention_forward_l4(bf16_cuda(q_idx), torch.from_numpy(w).float().cuda(),
                                 bf16_cuda(keys).view(pg.num_pages, 64, DI), bf16_cuda(q),
                                 torch.from_numpy(pool).cuda(), cache, dims, idx, out, lse, ws)
    assert dsa.workspace_check(ws) == (0, 0)
    mine = keys[pg.rows(0, np.arange(pos0 + n))]
    got = idx.cpu().numpy()
    for r in range(n):
        keep = np.asarray(orc.topk_select(orc.indexer_scores(q_idx[r], w[r], mine[:pos0 + r + 1]), k))
        keep = keep[keep >= 0]
        assert np.array_equal(got[r, :len(keep)], keep) and (got[r, len(keep):] == -1).all(), r
        if r % 50 == 0 or r == n - 1:
            L = values[pg.rows(0, keep)]
            ref, ref_lse, p = l4.attention(q[r], L, R, 0.0625)
            tol, ltol = attention_bounds(q[r], L, R, 0.0625, p)
            assert (np.abs(out[r].double().cpu().numpy() - ref) <= tol).all(), r
            assert (np.abs(lse[r].double().cpu().numpy() - ref_lse) <= ltol).all(), r
