"""How near the attention over 4-bit rows and the attention mass come to float64 at
W = 576, on fixed inputs: bounds of what their accumulations lose on average,
far below the worst cases of l4_testutil, so that a term that went missing shows.

Sums on the tensor cores lose at most one unit in the last place, 2^-23 of the
partial sum, per accumulation, half of it on average and always towards zero.
Every row here has at most 1,024 keys per CTA: 64 accumulations of 16 keys for
each of the weights' two terms, 128 in all, so an element of out loses about
128 * 2^-24 = 7.6e-6 of itself at most, and another 2^-21 for the weights' 22
bits.  A logit loses 36 * 2^-24 = 2.1e-6 of its partial sums, which random
signs keep at about two thirds of it: 1.4e-6 |z|.  That shortens all logits alike; in out
it is their covariance with one latent column, below 1e-6 of the largest
element; in lse it is 1.4e-6 times the mean logit, about 4: 6e-6, with 2^-20
for the logarithm.  The mass has two partial sums, 0.7e-6 |z| for |z| up to 8, and
an argument of exp below 2^5 rounded to 2^-20.  All four stay below 1e-5 of the
largest element (lse: absolute)."""

import functools

import numpy as np
import pytest

import sparse_attention_scores_b200 as dsa
from oracle import l4_oracle as l4
from tests.l4_testutil import Paged, bf16_cuda, random_l4, select, to_bf16

BOUND = 1e-5
R, P, H = 512, 64, 64
W = R + P
SCALE = float(np.float32(1 / np.sqrt(192.0)))
# rows, keys kept, first position of a causal chunk (-1: decode rows)
CASES = [(1, 2048, -1), (5, 2048, -1), (32, 2048, -1), (150, 320, -1), (160, 1024, 1500)]
IDS = ["one row", "five rows", "32 rows", "whole rows", "prompt rows"]


@functools.lru_cache(maxsize=1)
def _inputs(n, k, pos0):
    rng = np.random.default_rng([n, k])
    lens = [pos0 + n] if pos0 >= 0 else [k + 100 + int(x) for x in rng.integers(0, 50, n)]
    pg = Paged(lens, seed=n)
    pool, values = random_l4(rng, pg.num_pages, W, spread=0.5)
    q = to_bf16(rng.standard_normal((n, H, W)))
    idx = select(rng, [pos0 + t + 1 for t in range(n)] if pos0 >= 0 else lens, k)
    return pg, pool, values, q, idx, sorted({0, n // 2, n - 1})


def _row(pg, values, idx, r, pos0):
    pos = idx[r][idx[r] >= 0]
    return pos, values[pg.rows(0 if pos0 >= 0 else r, pos)]


@pytest.mark.parametrize("n,k,pos0", CASES, ids=IDS)
def test_weights_of_one_term_would_miss_the_bound(n, k, pos0):
    """The definition with the weights rounded once to fp16, at the scale they
    enter the tensor cores with."""
    pg, _, values, q, idx, rows = _inputs(n, k, pos0)
    for r in rows:
        _, L = _row(pg, values, idx, r, pos0)
        out, lse, p = l4.attention(q[r], L, R, SCALE)
        e = l4.row_exponent(np.abs(L).max(1))
        w = p * 2.0 ** e
        w = w / w.max(1, keepdims=True) * 64
        hi = w.astype(np.float16).astype(np.float64)
        one = (hi * 2.0 ** -e[None]) @ L[:, :R] / (w * 2.0 ** -e[None]).sum(1, keepdims=True)
        assert np.abs(one - out).max() > 3 * BOUND * np.abs(out).max()


@pytest.mark.gpu
@pytest.mark.parametrize("n,k,pos0", CASES, ids=IDS)
def test_attention_is_near_float64(n, k, pos0):
    import torch
    pg, pool, values, q, idx, rows = _inputs(n, k, pos0)
    causal = int(pos0 >= 0)
    cache, dims = pg.cache(), dsa.Dims(n, 1, 32, k, H, R, P, causal, max(0, pos0), SCALE)
    out, lse = torch.zeros(n, H, R, device="cuda"), torch.zeros(n, H, device="cuda")
    ws = dsa.l4_workspace(dsa.L4_OP_SPARSE_MLA, dims, cache)
    call = dsa.dsa_sparse_mla_prefill_l4 if causal else dsa.dsa_sparse_mla_decode_l4
    call(bf16_cuda(q), torch.from_numpy(pool).cuda(), cache, torch.from_numpy(idx).cuda(), dims, out, lse, ws)
    assert dsa.workspace_check(ws) == (0, 0)
    for r in rows:
        _, L = _row(pg, values, idx, r, pos0)
        ref, ref_lse, _ = l4.attention(q[r], L, R, SCALE)
        err = np.abs(out[r].double().cpu().numpy() - ref)
        top = np.abs(ref).max()
        print(f"row {r}: out {err[:, :256].max() / top:.2e} {err[:, 256:].max() / top:.2e}, "
              f"lse {np.abs(lse[r].double().cpu().numpy() - ref_lse).max():.2e}")
        assert err.max() <= BOUND * top
        assert np.abs(lse[r].double().cpu().numpy() - ref_lse).max() <= BOUND


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["l4", "l8", "bf16"])
@pytest.mark.parametrize("n,k,pos0", CASES, ids=IDS)
def test_mass_is_near_float64(n, k, pos0, fmt):
    import torch
    pg, pool, values, q, idx, _ = _inputs(n, k, pos0)
    if fmt == "l4":
        call, lat = dsa.dsa_attention_mass_l4, (torch.from_numpy(pool).cuda(),)
    elif fmt == "bf16":  # the same rows: their values are exact in bf16
        call, lat = dsa.dsa_attention_mass, (bf16_cuda(values).view(pg.num_pages, 64, W),)
    else:
        codes = torch.from_numpy(values / 4).float().to(torch.float8_e4m3fn)
        values = codes.double().numpy() * 4.0
        call = dsa.dsa_attention_mass_l8
        lat = (codes.view(torch.uint8).view(pg.num_pages, 64, W).cuda(),
               torch.full((pg.num_pages * 64,), 4.0, device="cuda"))
    causal = int(pos0 >= 0)
    cache, dims = pg.cache(), dsa.Dims(n, 1, 32, k, H, R, P, causal, max(0, pos0), SCALE)
    ld = max(pg.lens)
    ref = np.zeros((len(pg.lens), ld))
    lse = np.zeros((n, H), np.float32)
    for r in range(n):
        pos, L = _row(pg, values, idx, r, pos0)
        z = SCALE * (q[r] @ L.T)
        m = z.max(1)
        lse[r] = m + np.log(np.exp(z - m[:, None]).sum(1))
        l4.add_mass(ref[0 if causal else r], pos, q[r], L, lse[r], SCALE)
    got = torch.zeros(len(pg.lens), ld, device="cuda")
    ws = dsa.l4_workspace(dsa.L4_OP_ATTENTION_MASS, dims, cache)
    call(bf16_cuda(q), *lat, cache, torch.from_numpy(idx).cuda(), torch.from_numpy(lse).cuda(), dims, 1.0,
         None, got, ws)
    assert dsa.workspace_check(ws) == (0, 0)
    err = np.abs(got.double().cpu().numpy() - ref).max() / ref.max()
    print(f"mass {err:.2e}")
    assert err <= BOUND
