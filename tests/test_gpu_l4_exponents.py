"""Attention over 4-bit rows whose powers of two lie as far apart as the format
allows: the weight sum counts tokens by their weight, the output by weight times
size, and neither may be lost under the other."""

import numpy as np
import pytest
import torch

import sparse_attention_scores_b200 as dsa
from oracle import l4_oracle as l4
from tests.l4_testutil import Paged, attention_bounds, bf16_cuda, to_bf16

pytestmark = pytest.mark.gpu

WIDE = (64, 512, 64)  # heads, value columns, key-only columns


def _rows(rng, e, W):
    """Rows whose exponents are e: bf16 values of up to 2688 * 2^e, the last key-only
    column at the row's largest magnitude for the lowest exponent and 0 for the others
    (a query in that column alone then reaches the lowest tokens only)."""
    e = np.asarray(e)
    x = rng.standard_normal((len(e), W))
    x = x / np.abs(x[:, :W - 1]).max(1, keepdims=True) * 2600.0
    x[:, W - 1] = np.where(e == e.min(), 2600.0, 0.0)
    packed, values = l4.quantise(to_bf16(np.ldexp(x, e[:, None])))
    assert np.array_equal(packed[:, W // 2 + W // 16].astype(int) - 127, e)
    return packed, values


def _check(lens, exps, k, rng, shape=WIDE, causal=0):
    """exps: each sequence's exponents.  Head h's logits (base 2) are 0 for the tokens
    above the lowest exponent and between -40 and 40 for those."""
    H, R, P = shape
    W = R + P
    pg = Paged(lens, seed=len(lens))
    packed = np.zeros((pg.num_pages * 64, l4.row_bytes(W)), np.uint8)
    values = np.zeros((pg.num_pages * 64, W))
    n = lens[0] if causal else len(lens)
    q = np.zeros((n, H, W))
    for b, e in enumerate(exps):
        at = pg.rows(b, np.arange(lens[b]))
        packed[at], values[at] = _rows(rng, e, W)
        top = values[at][:, W - 1].max()
        q[slice(None) if causal else b, :, W - 1] = np.linspace(-40, 40, H) * np.log(2) / (0.0625 * top)
    q = to_bf16(q)
    idx = np.full((n, k), -1, np.int32)
    for b in range(n):
        m = min(k, b + 1 if causal else lens[b])
        idx[b, :m] = np.arange(m)
    cache = pg.cache()
    dims = dsa.Dims(n, 1, 32, k, H, R, P, causal, 0, 0.0625)
    out, lse = torch.zeros(n, H, R, device="cuda"), torch.zeros(n, H, device="cuda")
    ws = dsa.l4_workspace(dsa.L4_OP_SPARSE_MLA, dims, cache)
    call = dsa.dsa_sparse_mla_prefill_l4 if causal else dsa.dsa_sparse_mla_decode_l4
    call(bf16_cuda(q), torch.from_numpy(packed).view(pg.num_pages, 64, -1).cuda(), cache,
         torch.from_numpy(idx).cuda(), dims, out, lse, ws)
    assert dsa.workspace_check(ws) == (0, 0)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(n):
        L = values[pg.rows(0 if causal else b, idx[b][idx[b] >= 0])]
        ref, ref_lse, p = l4.attention(q[b], L, R, 0.0625)
        tol, ltol = attention_bounds(q[b], L, R, 0.0625, p)
        assert (np.abs(lse[b] - ref_lse) <= ltol).all(), (b, np.abs(lse[b] - ref_lse).max())
        assert (np.abs(out[b] - ref) <= tol).all(), (b, (np.abs(out[b] - ref) / np.abs(ref).max(1, keepdims=True)).max())


# one high token among low ones: the first, one inside, the last; then blocks
ORDERS = ["first", "inside", "last", "halves", "halves back", "three"]


def _exponents(order, n, low, high):
    e = np.full(n, low)
    if order in ("first", "inside", "last"):
        e[{"first": 0, "inside": n // 2, "last": n - 1}[order]] = high
    elif order == "halves":
        e[n // 2:] = high
    elif order == "halves back":
        e[:n // 2] = high
    else:  # ordinary tokens before and between the far ones
        e[:] = 0
        e[n // 3:n // 2] = high
        e[2 * n // 3:] = low
    return e


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("low,high", [(-60, 60), (-60, 0), (-31, 30), (-45, 50)])
@pytest.mark.parametrize("split", [False, True], ids=["whole rows", "split rows"])
def test_exponents_at_both_ends_of_a_row(order, low, high, split):
    rng = np.random.default_rng([ORDERS.index(order), high, split])
    if split:
        lens, k = [2048], 2048                       # a slot or two per CTA, joined by the merge
    else:
        lens, k = [330] + [60] * 148, 330            # one CTA a row
    exps = [_exponents(order, n, low, high) for n in lens]
    _check(lens, exps, k, rng)


@pytest.mark.parametrize("e", [-60, 60, 31, -31])
def test_rows_of_one_far_exponent(e):
    rng = np.random.default_rng(e + 100)
    _check([200], [np.full(200, e)], 200, rng)


@pytest.mark.parametrize("shape", [(5, 64, 16), (33, 448, 48), (16, 64, 512), (64, 192, 0), (1, 320, 16)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("form", ["whole rows", "split rows", "prompt rows"])
def test_far_exponents_at_other_shapes(shape, form):
    """Random exponents over the whole range, the first far one in any slot."""
    rng = np.random.default_rng([shape[1], len(form)])
    if form == "whole rows":
        lens, k = [400] + [30] * 149, 400
    elif form == "split rows":
        lens, k = [900, 70, 1], 900
    else:
        lens, k = [260], 200
    exps = []
    for n in lens:
        e = rng.integers(-24, 25, n)
        at = rng.integers(0, n)
        e[at:] = rng.integers(-60, 61, n - at)
        exps.append(e)
    _check(lens, exps, k, rng, shape, int(form == "prompt rows"))
