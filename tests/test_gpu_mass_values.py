"""Attention mass of values at the ends of their types."""

import numpy as np
import pytest
import torch

import sparse_attention_scores_b200 as dsa
from oracle import l4_oracle as l4
from tests.l4_testutil import Paged, U, bf16_cuda, logit_bound, random_l4, select, to_bf16

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


@pytest.mark.parametrize("n,log2_w", [(1, -53), (4, -48), (512, -44), (700, -43)])
def test_small_weights_of_a_chunk_are_not_lost(n, log2_w):
    """lse far above the logits: weights of about 2^log2_w, which a chunk of n rows
    adds in steps of 2^-56 times n (rounded up to a power of two)."""
    rng = np.random.default_rng(n)
    H, R, P, k, pos0 = 2, 64, 16, 8, 20
    pg = Paged([pos0 + n], seed=2)
    pool, values = random_l4(rng, pg.num_pages, R + P)
    q = to_bf16(rng.standard_normal((n, H, R + P)))
    idx = select(rng, [pos0 + t + 1 for t in range(n)], k)
    lse = np.zeros((n, H), np.float32)
    ref, tol = np.zeros(pos0 + n), np.zeros(pos0 + n)
    for t in range(n):
        L = values[pg.rows(0, idx[t])]
        z = 0.125 * (q[t] @ L.T)
        lse[t] = z.max(1) - log2_w * np.log(2)
        w = np.exp(z - lse[t].astype(np.float64)[:, None])
        # a head's weight: its logit's error, the exponential's 2^-19, the rounding of
        # an argument below 128; then half a step for the row
        rel = logit_bound(q[t], L, 0.125) + 2.0 ** -19 + 144 * U
        np.add.at(ref, idx[t], w.sum(0))
        np.add.at(tol, idx[t], (w * rel).sum(0) + 2.0 ** (np.ceil(np.log2(n)) - 57))
    cache, dims = pg.cache(), dsa.Dims(n, 1, 32, k, H, R, P, 1, pos0, 0.125)
    got = torch.zeros(1, pos0 + n, device="cuda")
    ws = dsa.l4_workspace(dsa.L4_OP_ATTENTION_MASS, dims, cache)
    dsa.dsa_attention_mass_l4(bf16_cuda(q), torch.from_numpy(pool).cuda(), cache, torch.from_numpy(idx).cuda(),
                              torch.from_numpy(lse).cuda(), dims, 1.0, None, got, ws)
    assert dsa.workspace_check(ws) == (0, 0)
    g = got[0].double().cpu().numpy()
    assert (np.abs(g - ref) <= tol + 4 * U * ref).all(), (np.abs(g - ref) - tol).max()
    assert ref.max() > 8 * tol[ref.argmax()]  # a sum that lost its weights would show


def test_the_largest_chunk_does_not_overflow():
    """65,535 rows that give one token the most weight lse of the step's can leave."""
    n, H, R, P = 65535, 64, 64, 0
    pg = Paged([n], seed=1)
    pool = torch.zeros(pg.num_pages, 64, 48, dtype=torch.uint8, device="cuda")
    q = torch.zeros(n, H, R, dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros(n, 1, dtype=torch.int32, device="cuda")  # every row keeps the first token only
    lse = torch.zeros(n, H, device="cuda")
    cache, dims = pg.cache(), dsa.Dims(n, 1, 32, 1, H, R, P, 1, 0, 0.125)
    got = torch.zeros(1, n, device="cuda")
    ws = dsa.l4_workspace(dsa.L4_OP_ATTENTION_MASS, dims, cache)
    dsa.dsa_attention_mass_l4(q, pool, cache, idx, lse, dims, 1.0, None, got, ws)
    assert dsa.workspace_check(ws) == (0, 0)
    assert float(got[0, 0]) == float(np.float32(n * H)) and float(got[0, 1:].abs().max()) == 0


def test_sums_over_evictions_in_two_swapped_buffers():
    """Decode steps and evictions in turn, the masses moving between two buffers that
    hold other sums before: with a new token's entry set to 0 the sums are those of
    the tokens that are there."""
    rng = np.random.default_rng(4)
    H, R, P, k, budget, pages = 16, 64, 16, 40, 96, 12
    W, scale = R + P, 0.125
    pool = torch.zeros(pages, 64, l4.row_bytes(W), dtype=torch.uint8, device="cuda")
    keys = torch.zeros(pages, 64, 32, dtype=torch.bfloat16, device="cuda")
    tables = torch.tensor([[3, 1, 8], [5, 2, 9]], dtype=torch.int32, device="cuda")
    sums = [torch.full((1, 192), 1000.0 + i, device="cuda") for i in range(2)]
    seq = torch.zeros(1, dtype=torch.int32, device="cuda")
    new_lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept = torch.zeros(1, budget, dtype=torch.int32, device="cuda")
    one = dsa.Dims(1, 1, 32, k, H, R, P, 0, 0, scale)
    values, ref, tol = np.zeros((0, W)), np.zeros(0), np.zeros(0)
    at = 0
    for length in (130, 110, 140):  # up to so many tokens, then an eviction
        cache = dsa.PagedCache(seq, tables[at:at + 1], pages, 192)
        ws = dsa.l4_workspace(dsa.L4_OP_ATTENTION_MASS, one, cache)
        while len(values) < length:
            seq += 1
            row = to_bf16(rng.standard_normal((1, W)))
            dsa.dsa_cache_append_l4(torch.zeros(1, 32, dtype=torch.bfloat16, device="cuda"), bf16_cuda(row), keys, pool,
                                    cache, one, ws)
            sums[at][0, len(values)] = 0
            values = np.concatenate([values, l4.quantise(row)[1]])
            ref, tol = np.append(ref, 0.0), np.append(tol, 0.0)
            q = to_bf16(rng.standard_normal((1, H, W)))
            idx = select(rng, [len(values)], k)
            pos = idx[0][idx[0] >= 0]
            L = values[pos]
            lse = l4.attention(q[0], L, R, scale)[1].astype(np.float32)
            dsa.dsa_attention_mass_l4(bf16_cuda(q), pool, cache, torch.from_numpy(idx).cuda(),
                                      torch.from_numpy(lse[None]).cuda(), one, 0.875, sums[at], sums[at], ws)
            ref, tol = 0.875 * ref, 0.875 * tol + U * ref
            l4.add_mass(ref, pos, q[0], L, lse, scale)
            w = np.exp(scale * (q[0] @ L.T) - lse.astype(np.float64)[:, None])
            np.add.at(tol, pos, (w * (logit_bound(q[0], L, scale) + 2.0 ** -19 + 144 * U)).sum(0))
            tol = tol + 2 * U * ref
        assert dsa.workspace_check(ws) == (0, 0)
        assert (np.abs(sums[at][0, :length].double().cpu().numpy() - ref) <= tol).all()
        ws = dsa.l4_workspace(dsa.L4_OP_CACHE_EVICT, None, cache)
        dsa.dsa_cache_evict([(pool, pool), (keys, keys)], cache, dsa.Eviction(budget, 2, 10), sums[at],
                            tables[1 - at:2 - at], sums[1 - at], new_lens, kept, ws)
        assert dsa.workspace_check(ws) == (0, 0)
        left = kept[0].cpu().numpy()
        assert np.array_equal(left, l4.evict_keep(sums[at][0, :length].cpu().numpy(), budget, 2, 10))
        values, ref, tol = values[left], ref[left], tol[left]
        at, seq = 1 - at, new_lens.clone()
