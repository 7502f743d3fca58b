"""Attention mass of values at the ends of their types."""

import numpy as np
import pytest
import torch

import sparse_attention_scores_b200 as dsa
from tests.l4_testutil import Paged, bf16_cuda, select, to_bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [0, 1])
def test_a_token_of_infinite_scale_shows_in_the_mass(causal):
    """An E4M3 token whose scale is infinite has a weight that is not finite (the
    logits are infinite, of either sign), and no other token's changes."""
    rng = np.random.default_rng(causal)
    n, H, R, P, k, tok = 40, 64, 64, 16, 24, 5
    lens = [n] if causal else [30] * n
    pg = Paged(lens, seed=3)
    codes = torch.from_numpy(to_bf16(rng.standard_normal((pg.num_pages * 64, R + P)))).float().to(torch.float8_e4m3fn)
    codes = codes.view(torch.uint8).view(pg.num_pages, 64, R + P).cuda()
    scale = torch.ones(pg.num_pages * 64, device="cuda")
    q = bf16_cuda(to_bf16(rng.standard_normal((n, H, R + P))))
    idx = select(rng, [t + 1 for t in range(n)] if causal else lens, k)
    cache, dims = pg.cache(), dsa.Dims(n, 1, 32, k, H, R, P, causal, 0, 0.125)
    dev_idx = torch.from_numpy(idx).cuda()
    attend = dsa.dsa_sparse_mla_prefill_l8 if causal else dsa.dsa_sparse_mla_decode_l8
    ws_a = dsa.workspace(dsa.OP_SPARSE_MLA_PREFILL if causal else dsa.OP_SPARSE_MLA_DECODE, dims, cache)
    ws = dsa.l4_workspace(dsa.L4_OP_ATTENTION_MASS, dims, cache)
    out, lse = torch.zeros(n, H, R, device="cuda"), torch.zeros(n, H, device="cuda")
    ld = max(lens)

    def mass(l):
        got = torch.zeros(1 if causal else n, ld, device="cuda")
        dsa.dsa_attention_mass_l8(q, codes, scale, cache, dev_idx, l, dims, 1.0, None, got, ws)
        return got.cpu().numpy()

    attend(q, codes, scale, cache, dev_idx, dims, out, lse, ws_a)
    plain = mass(lse)
    for b in range(1 if causal else n):
        scale[int(pg.rows(b, [tok])[0])] = float("inf")
    held = [tok in row for row in idx]
    assert any(held) and not all(held)
    now = mass(lse)
    for r in range(n):
        b = 0 if causal else r
        assert np.isfinite(plain[b, tok])
        if held[r]:
            assert not np.isfinite(now[b, tok]), r
    rest = np.arange(ld) != tok
    assert np.array_equal(now[:, rest], plain[:, rest])
    assert dsa.workspace_check(ws) == (0, 0)
