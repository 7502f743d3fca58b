"""4-bit latent cache on the GPU: quantising append and exact read-back byte for
byte against the float64 definition, sparse MLA over it (decode, prefill, the
whole step) within bounds derived from its roundings."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import sparse_attention_scores_b200 as dsa
from oracle import dsa_oracle as orc
from oracle import l4_oracle as l4
from tests.l4_testutil import Paged, attention_bounds, bf16_cuda, random_l4, select, to_bf16

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _dims(n_q, W, P, *, topk=1, H=1, D_I=32, causal=0, q_pos0=0, scale=1.0, H_I=1):
    return dsa.Dims(n_q, H_I, D_I, topk, H, W - P, P, causal, q_pos0, scale)


def _hard_rows(rng, n, W):
    """Rows that meet the format's edges: zeros, single values, boundaries
    between codes, tiny blocks beside large ones, the ends of the exponent
    range, bf16 subnormals."""
    x = rng.standard_normal((n, W)) * np.exp2(rng.uniform(-20, 20, (n, 1)))
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.5, 4.0])
    x[0] = 0
    x[1] = 0
    x[1, W - 1] = -3.0
    x[2] = rng.choice(ties, W) * rng.choice([-1, 1], W)
    x[3] = rng.choice(ties, W) * 2.0 ** 30
    x[4] = np.where(np.arange(W) // 16 % 2 == 0, 2688.0, 1e-3)
    x[5] = 2688.0 * 2.0 ** 60
    x[6] = 3.0e38 * rng.choice([-1, 1], W)
    x[7] = rng.standard_normal(W) * 2.0 ** -75
    x[8] = 2.0 ** -130
    x[9] = 5.25
    x[10] = np.nextafter(np.float32(5.25), np.float32(6))
    x[11] = np.exp2(rng.uniform(-24, 0, W))
    return to_bf16(x)


@pytest.mark.parametrize("W,P,D_I", [(576, 64, 128), (512, 0, 64), (80, 16, 32), (224, 32, 128),
                                     (64, 0, 32)])
@pytest.mark.parametrize("causal", [0, 1])
def test_append_stores_the_defined_bytes(W, P, D_I, causal):
    rng = np.random.default_rng(W + causal)
    n = 45
    pg = Paged([37 + n] if causal else rng.integers(1, 300, n).tolist(), seed=W)
    x = _hard_rows(rng, n, W)
    k_new = to_bf16(rng.standard_normal((n, D_I)))
    rb = l4.row_bytes(W)
    assert dsa.l4_row_bytes(W - P, P) == rb
    keys = torch.full((pg.num_pages, 64, D_I), 7.0, dtype=torch.bfloat16, device="cuda")
    pool = torch.full((pg.num_pages, 64, rb), 0xAB, dtype=torch.uint8, device="cuda")
    cache, dims = pg.cache(), _dims(n, W, P, D_I=D_I, causal=causal, q_pos0=37 if causal else 0)
    ws = dsa.l4_workspace(dsa.L4_OP_STATUS, dims, cache)
    dsa.dsa_cache_append_l4(bf16_cuda(k_new), bf16_cuda(x), keys, pool, cache, dims, ws)
    assert dsa.workspace_check(ws) == (0, 0)
    rows = pg.rows(0, 37 + np.arange(n)) if causal else \
        np.array([pg.rows(b, [m - 1])[0] for b, m in enumerate(pg.lens)])
    ref_pool = np.full((pg.num_pages * 64, rb), 0xAB, np.uint8)
    packed, values = l4.quantise(x)
    ref_pool[rows] = packed
    got = pool.cpu().numpy().reshape(-1, rb)
    # a value that rounds to zero may keep its sign: codes 0 and 8 are the same value
    assert np.array_equal(l4.dequantise(got[rows], W), values)
    assert np.array_equal(got[rows][:, W // 2:], packed[:, W // 2:])
    ref_pool[rows] = got[rows]
    assert np.array_equal(got, ref_pool), "rows of other tokens changed"
    ref_keys = np.full((pg.num_pages * 64, D_I), 7.0)
    ref_keys[rows] = k_new
    assert np.array_equal(keys.float().cpu().numpy().reshape(-1, D_I), ref_keys)


def test_append_saturates_infinities_and_stores_finite_rows():
    x = torch.zeros(3, 80, dtype=torch.bfloat16, device="cuda")
    x[0, 5], x[1, 0], x[2, 7] = float("inf"), float("-inf"), float("nan")
    x[:, 40:] = 1.0
    pg = Paged([10, 20, 30])
    pool = torch.zeros(pg.num_pages, 64, 48, dtype=torch.uint8, device="cuda")
    keys = torch.zeros(pg.num_pages, 64, 32, dtype=torch.bfloat16, device="cuda")
    cache, dims = pg.cache(), _dims(3, 80, 16)
    ws = dsa.l4_workspace(dsa.L4_OP_STATUS, dims, cache)
    dsa.dsa_cache_append_l4(torch.zeros(3, 32, dtype=torch.bfloat16, device="cuda"), x, keys, pool,
                            cache, dims, ws)
    v = l4.dequantise(pool.cpu().numpy().reshape(-1, 48), 80)
    assert np.isfinite(v).all()
    assert v[pg.rows(0, [9])[0], 5] == 2688.0 * 2.0 ** 60
    assert v[pg.rows(1, [19])[0], 0] == -2688.0 * 2.0 ** 60


@pytest.mark.parametrize("W,P,k", [(576, 64, 300), (80, 16, 7), (448, 0, 1)])
def test_read_gives_the_stored_values(W, P, k):
    rng = np.random.default_rng(W + k)
    pg = Paged([400, 1, 129, 333], seed=3)
    # any bytes: random codes, all finite scales, exponents out of range too
    pool = rng.integers(0, 256, (pg.num_pages, 64, l4.row_bytes(W))).astype(np.uint8)
    sc = pool[..., W // 2:W // 2 + W // 16]
    sc[:] = np.minimum(sc & 0x7F, 0x7E)
    idx = np.stack([rng.integers(0, n, k) for n in pg.lens]).astype(np.int32)  # any order, repeats
    idx[1, 0] = -1
    cache, dims = pg.cache(), _dims(4, W, P, topk=k)
    out = torch.full((4, k, W), 9.0, dtype=torch.bfloat16, device="cuda")
    ws = dsa.l4_workspace(dsa.L4_OP_STATUS, dims, cache)
    dsa.dsa_cache_read_l4(torch.from_numpy(pool).cuda(), cache, torch.from_numpy(idx).cuda(), dims,
                          out, ws)
    assert dsa.workspace_check(ws) == (0, 0)
    values = l4.dequantise(pool.reshape(-1, pool.shape[2]), W)
    ref = np.stack([values[pg.rows(b, np.maximum(idx[b], 0))] for b in range(4)])
    ref[1, 0] = 0
    assert np.array_equal(out.double().cpu().numpy(), ref)


def test_append_and_read_report_what_is_out_of_range():
    pg = Paged([200, 300], seed=5)
    cache, dims = pg.cache(), _dims(2, 80, 16, topk=2)
    bad = pg.table.copy()
    bad[1, 299 // 64] = pg.num_pages
    cache.block_table = torch.from_numpy(bad).cuda()
    keys = torch.zeros(pg.num_pages, 64, 32, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(pg.num_pages, 64, 48, dtype=torch.uint8, device="cuda")
    ws = dsa.l4_workspace(dsa.L4_OP_STATUS, dims, cache)
    one = torch.ones(2, 80, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_cache_append_l4(torch.ones(2, 32, dtype=torch.bfloat16, device="cuda"), one, keys, pool,
                            cache, dims, ws)
    st, info = dsa.workspace_check(ws)
    assert st == 6 and info >> 24 == 5
    changed = (pool.view(-1, 48) != 0).any(1).nonzero().flatten().tolist()
    assert changed == pg.rows(0, [199]).tolist()
    ws = dsa.l4_workspace(dsa.L4_OP_STATUS, dims, cache)
    out = torch.full((2, 2, 80), 9.0, dtype=torch.bfloat16, device="cuda")
    idx = torch.tensor([[199, 200], [299, 0]], dtype=torch.int32, device="cuda")
    dsa.dsa_cache_read_l4(pool, cache, idx, dims, out, ws)
    st, info = dsa.workspace_check(ws)
    assert st == 6 and info >> 24 == 7
    stored = l4.quantise(np.ones((1, 80)))[1][0]   # 1 / 6 is no E4M3 scale: 1 is stored as 1.03125
    assert np.array_equal(out[0, 0].double().cpu().numpy(), stored)
    assert (out[0, 1] == 0).all() and (out[1] == 0).all()


# ---------------------------------------------------------------- attention
def _check_attention(q, values, pg, idx, out, lse, R, scale, causal, rows=None):
    for r in range(len(idx)) if rows is None else rows:
        pos = idx[r][idx[r] >= 0]
        L = values[pg.rows(0 if causal else r, pos)]
        ref, ref_lse, p = l4.attention(q[r], L, R, scale)
        if len(pos) == 0:
            assert (out[r] == 0).all() and np.isneginf(lse[r]).all()
            continue
        tol, ltol = attention_bounds(q[r], L, R, scale, p)
        bad = np.abs(out[r] - ref) - tol
        assert (bad <= 0).all(), (r, bad.max(), np.abs(out[r] - ref).max())
        assert (np.abs(lse[r] - ref_lse) <= ltol).all(), (r, np.abs(lse[r] - ref_lse).max())


def _run_mla(pg, pool, q, idx, dims, cache=None, ws=None):
    cache = pg.cache() if cache is None else cache
    out = torch.full((dims.n_q, dims.H, dims.R), float("nan"), device="cuda")
    lse = torch.full((dims.n_q, dims.H), float("nan"), device="cuda")
    ws = dsa.l4_workspace(dsa.L4_OP_SPARSE_MLA, dims, cache) if ws is None else ws
    call = dsa.dsa_sparse_mla_prefill_l4 if dims.causal else dsa.dsa_sparse_mla_decode_l4
    call(bf16_cuda(q), torch.from_numpy(pool).cuda(), cache, torch.from_numpy(idx).cuda(), dims,
         out, lse, ws)
    st = dsa.workspace_check(ws)
    return out.double().cpu().numpy(), lse.double().cpu().numpy(), st


SHAPES = [
    # batch, H, R, P, topk, longest context: every way a row's keys are split
    (1, 64, 512, 64, 2048, 3000), (3, 64, 512, 64, 2048, 2500), (9, 64, 512, 64, 1024, 1500),
    (32, 64, 512, 64, 512, 900), (150, 64, 512, 64, 130, 300), (7, 4, 64, 16, 256, 500),
    (5, 33, 448, 48, 300, 700), (4, 17, 192, 0, 65, 200), (2, 1, 128, 0, 64, 100),
    (1, 64, 512, 0, 4097, 6000), (6, 64, 320, 16, 1, 50), (2, 16, 512, 48, 63, 64),
    (1, 64, 512, 64, 20000, 21000), (3, 8, 64, 0, 70, 100), (2, 64, 256, 64, 1024, 2000),
    (40, 64, 384, 32, 200, 400),
    # more columns that only the logits read than the latent rows' own blocks leave
    (3, 64, 64, 512, 300, 400), (2, 5, 128, 96, 100, 150), (160, 64, 256, 320, 70, 100),
    (1, 64, 192, 384, 2048, 2100), (2, 32, 64, 144, 130, 200),
]


@pytest.mark.parametrize("B,H,R,P,k,longest", SHAPES)
def test_decode_matches_definition(B, H, R, P, k, longest):
    rng = np.random.default_rng([B, H, R, P, k])
    lens = rng.integers(1, longest + 1, B).tolist()
    lens[0] = longest
    if B > 2:
        lens[1] = 1
    pg = Paged(lens, seed=B)
    pool, values = random_l4(rng, pg.num_pages, R + P)
    q = to_bf16(rng.standard_normal((B, H, R + P)))
    idx = select(rng, lens, k)
    if B > 3:
        idx[2] = -1                                   # a row that keeps nothing
        idx[3, rng.random(k) < 0.5] = -1              # unused slots between used ones
    scale = 1 / np.sqrt(R + P)
    dims = _dims(B, R + P, P, topk=k, H=H, scale=float(np.float32(scale)))
    out, lse, st = _run_mla(pg, pool, q, idx, dims)
    assert st == (0, 0)
    _check_attention(q, values, pg, idx, out, lse, R, float(np.float32(scale)), False)


@pytest.mark.parametrize("T,pos0,H,R,P,k", [(150, 0, 64, 512, 64, 96), (70, 1000, 64, 512, 64, 700),
                                            (5, 3, 4, 64, 16, 256), (1, 0, 64, 512, 64, 64)])
def test_prefill_matches_definition(T, pos0, H, R, P, k):
    rng = np.random.default_rng([T, k])
    pg = Paged([pos0 + T], seed=T)
    pool, values = random_l4(rng, pg.num_pages, R + P)
    q = to_bf16(rng.standard_normal((T, H, R + P)))
    idx = select(rng, [pos0 + t + 1 for t in range(T)], k)
    if T > 2:
        idx[1] = -1
    dims = _dims(T, R + P, P, topk=k, H=H, causal=1, q_pos0=pos0, scale=0.0625)
    out, lse, st = _run_mla(pg, pool, q, idx, dims)
    assert st == (0, 0)
    _check_attention(q, values, pg, idx, out, lse, R, 0.0625, True)


@pytest.mark.parametrize("power", [115, -110])
def test_queries_of_any_size_carry_over(power):
    """q times a power of two and scale divided by it: the same products, bit for
    bit, up to the ends of bf16."""
    rng = np.random.default_rng(3)
    pg = Paged([300, 200], seed=3)
    pool, _ = random_l4(rng, pg.num_pages, 576)
    q, idx = to_bf16(rng.standard_normal((2, 64, 576))), select(rng, [300, 200], 130)
    runs = [_run_mla(pg, pool, q * 2.0 ** p, idx, _dims(2, 576, 64, topk=130, H=64, scale=0.0625 * 2.0 ** -p))
            for p in (0, power)]
    assert runs[0][2] == runs[1][2] == (0, 0)
    assert np.array_equal(runs[0][0], runs[1][0]) and np.array_equal(runs[0][1], runs[1][1])


def test_logits_far_apart_and_rows_of_unequal_size():
    """Weights from 1 to 0, token exponents far apart, heads of tiny and large
    queries in one row, a token of zeros."""
    rng = np.random.default_rng(8)
    pg = Paged([700, 64, 300], seed=1)
    W, R, P, H, k = 576, 512, 64, 64, 640
    x = rng.standard_normal((pg.num_pages * 64, W)) * np.exp2(rng.integers(-12, 5, (pg.num_pages * 64, 1)))
    x[pg.rows(0, [5])] = 0
    packed, values = l4.quantise(to_bf16(x))
    q = rng.standard_normal((3, H, W)) * np.exp2(rng.integers(-18, 3, (3, H, 1)))
    q[2, 5] = 0
    q = to_bf16(q)
    idx = select(rng, pg.lens, k)
    dims = _dims(3, W, P, topk=k, H=H, scale=0.0625)
    out, lse, st = _run_mla(pg, packed.reshape(pg.num_pages, 64, -1), q, idx, dims)
    assert st == (0, 0)
    for r in range(3):
        pos = idx[r][idx[r] >= 0]
        L = values[pg.rows(r, pos)]
        ref, ref_lse, p = l4.attention(q[r], L, R, 0.0625)
        tol, _ = attention_bounds(q[r], L, R, 0.0625, p)
        assert (np.abs(out[r] - ref) <= tol).all(), r
        # |lse| reaches past 64 here: its own rounding counts relative to it
        d = (p * 0.0625 * (np.abs(q[r]) @ np.abs(L).T)).sum(1) * 2 * (W / 16 + 28) * 2.0 ** -23
        assert (np.abs(lse[r] - ref_lse) <= d + 2e-4 + np.abs(ref_lse) * 2.0 ** -20).all()


def test_running_maximum_moves_late():
    """The largest logits come last, far above the first ones: every earlier
    partial sum has to be rescaled."""
    W, R, P, H, k = 576, 512, 64, 64, 512
    pg = Paged([k], seed=2)
    rng = np.random.default_rng(3)
    x = rng.standard_normal((pg.num_pages * 64, W))
    q = to_bf16(rng.standard_normal((1, H, W)))
    rows = pg.rows(0, np.arange(k))
    ramp = np.linspace(-1, 1, k)[:, None] ** 3
    x[rows] = x[rows] * 0.3 + ramp * 1.2 * np.sign(q[0].sum(0))[None]
    packed, values = l4.quantise(to_bf16(x))
    idx = np.arange(k, dtype=np.int32)[None]
    dims = _dims(1, W, P, topk=k, H=H, scale=0.5)
    out, lse, st = _run_mla(pg, packed.reshape(pg.num_pages, 64, -1), q, idx, dims)
    assert st == (0, 0)
    L = values[rows]
    ref, ref_lse, p = l4.attention(q[0], L, R, 0.5)
    tol, _ = attention_bounds(q[0], L, R, 0.5, p)
    assert (np.abs(out[0] - ref) <= tol).all()
    assert np.isfinite(lse).all()


def test_same_position_twice_counts_twice():
    rng = np.random.default_rng(4)
    pg = Paged([100], seed=2)
    pool, values = random_l4(rng, pg.num_pages, 80)
    q = to_bf16(rng.standard_normal((1, 4, 80)))
    idx = np.array([[3, 3, 9, 64, 64, 64, 99, -1]], np.int32)
    dims = _dims(1, 80, 16, topk=8, H=4, scale=0.125)
    out, lse, st = _run_mla(pg, pool, q, idx, dims)
    assert st == (0, 0)
    _check_attention(q, values, pg, idx, out, lse, 64, 0.125, False)


def test_out_of_range_positions_and_pages_are_skipped_and_reported():
    rng = np.random.default_rng(6)
    pg = Paged([300, 200], seed=4)
    pool, values = random_l4(rng, pg.num_pages, 576)
    q = to_bf16(rng.standard_normal((2, 64, 576)))
    idx = select(rng, pg.lens, 128)
    dims = _dims(2, 576, 64, topk=128, H=64, scale=0.0625)
    bad = idx.copy()
    bad[0, 100] = 300                       # one past the context
    out, lse, st = _run_mla(pg, pool, q, bad, dims)
    assert st[0] == 6 and st[1] >> 24 == 8
    ref = idx.copy()
    ref[0, 100] = -1
    _check_attention(q, values, pg, ref, out, lse, 512, 0.0625, False)
    cache = pg.cache()
    table = pg.table.copy()
    table[1, 1] = -5
    cache.block_table = torch.from_numpy(table).cuda()
    out, lse, st = _run_mla(pg, pool, q, idx, dims, cache)
    assert st[0] == 6 and st[1] >> 24 == 8
    ref = idx.copy()
    ref[1, (idx[1] >= 64) & (idx[1] < 128)] = -1
    _check_attention(q, values, pg, ref, out, lse, 512, 0.0625, False)


def test_rows_of_masked_slots_may_hold_anything():
    """NaN scales in rows that no slot selects do not reach the result."""
    rng = np.random.default_rng(7)
    pg = Paged([500], seed=4)
    pool, values = random_l4(rng, pg.num_pages, 576)
    idx = select(rng, [500], 200)
    used = np.zeros(pg.num_pages * 64, bool)
    used[pg.rows(0, idx[0])] = True
    flat = pool.reshape(-1, pool.shape[2])
    flat[~used, 288:324] = 0x7F
    q = to_bf16(rng.standard_normal((1, 64, 576)))
    idx = np.concatenate([idx, np.full((1, 30), -1, np.int32)], 1)
    dims = _dims(1, 576, 64, topk=230, H=64, scale=0.0625)
    out, lse, st = _run_mla(pg, pool, q, idx, dims)
    assert st == (0, 0)
    _check_attention(q, values, pg, idx, out, lse, 512, 0.0625, False)


def test_repeated_and_captured_calls_agree():
    """The same call again, on another stream, and as a replayed graph beside
    a second graph with its own workspace: bit-identical."""
    rng = np.random.default_rng(9)
    pg = Paged([2300, 1111], seed=4)
    pool, _ = random_l4(rng, pg.num_pages, 576)
    pool = torch.from_numpy(pool).cuda()
    q = bf16_cuda(to_bf16(rng.standard_normal((2, 64, 576))))
    idx = torch.from_numpy(select(rng, pg.lens, 1024)).cuda()
    cache, dims = pg.cache(), _dims(2, 576, 64, topk=1024, H=64, scale=0.0625)

    def buffers():
        return (torch.zeros(2, 64, 512, device="cuda"), torch.zeros(2, 64, device="cuda"),
                dsa.l4_workspace(dsa.L4_OP_SPARSE_MLA, dims, cache))

    def call(b):
        dsa.dsa_sparse_mla_decode_l4(q, pool, cache, idx, dims, b[0], b[1], b[2])

    first = buffers()
    call(first)
    second = buffers()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(second)
    torch.cuda.synchronize()
    assert torch.equal(first[0], second[0]) and torch.equal(first[1], second[1])
    graphs, bufs = [], [buffers(), buffers()]
    torch.cuda.synchronize()
    for b in bufs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(b)
        graphs.append(g)
    for b in bufs:
        b[0].zero_()
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for b in bufs:
        assert torch.equal(first[0], b[0]) and torch.equal(first[1], b[1])


@pytest.mark.parametrize("causal", [0, 1])
def test_forward_matches_definition(causal):
    rng = np.random.default_rng(21 + causal)
    n, k, H, R, P, HI, DI = 5, 200, 64, 512, 64, 32, 128
    pos0 = 250 if causal else 0
    lens = [pos0 + n] if causal else [700, 1, 200, 513, 201]
    pg = Paged(lens, seed=9)
    pool, values = random_l4(rng, pg.num_pages, R + P)
    keys = rng.integers(-3, 4, (pg.num_pages * 64, DI)).astype(np.float64)
    q_idx = rng.integers(-3, 4, (n, HI, DI)).astype(np.float64)
    w = rng.integers(0, 4, (n, HI)).astype(np.float64)
    q = to_bf16(rng.standard_normal((n, H, R + P)))
    cache = pg.cache()
    dims = _dims(n, R + P, P, topk=k, H=H, D_I=DI, H_I=HI, causal=causal, q_pos0=pos0, scale=0.0625)
    idx = torch.full((n, k), -7, dtype=torch.int32, device="cuda")
    out, lse = torch.zeros(n, H, R, device="cuda"), torch.zeros(n, H, device="cuda")
    ws = dsa.l4_workspace(dsa.L4_OP_ATTENTION_FORWARD, dims, cache)
    args = (bf16_cuda(q_idx), torch.from_numpy(w).float().cuda(),
            bf16_cuda(keys).view(pg.num_pages, 64, DI), bf16_cuda(q), torch.from_numpy(pool).cuda(),
            cache, dims)
    dsa.dsa_attention_forward_l4(*args, idx, out, lse, ws)
    assert dsa.workspace_check(ws) == (0, 0)
    ref = np.full((n, k), -1, np.int32)
    for r in range(n):
        seen = pos0 + r + 1 if causal else lens[r]
        kr = keys[pg.rows(0 if causal else r, np.arange(seen))]
        keep = orc.topk_select(orc.indexer_scores(q_idx[r], w[r], kr), k)
        ref[r, :len(keep)] = keep
    assert np.array_equal(idx.cpu().numpy(), ref)
    _check_attention(q, values, pg, ref, out.double().cpu().numpy(), lse.double().cpu().numpy(), R,
                     0.0625, causal)
    # without idx_out the selection stays in the workspace
    out2, lse2 = torch.zeros_like(out), torch.zeros_like(lse)
    dsa.dsa_attention_forward_l4(*args, None, out2, lse2, ws)
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_rows_without_context_and_a_4_byte_aligned_output():
    """A sequence of length 0 in the batch, and results at addresses that are
    only 4-byte aligned, with guard values around them."""
    rng = np.random.default_rng(12)
    for k, B in ((512, 3), (64, 160)):  # split rows and their merge; whole rows
        lens = rng.integers(1, 600, B).tolist()
        lens[1] = 0
        pg = Paged(lens, seed=5)
        pool, values = random_l4(rng, pg.num_pages, 576)
        q = to_bf16(rng.standard_normal((B, 64, 576)))
        idx = select(rng, lens, k)
        cache, dims = pg.cache(), _dims(B, 576, 64, topk=k, H=64, scale=0.0625)
        flat = torch.full((B * 64 * 512 + 2,), 5.0, device="cuda")
        flat_lse = torch.full((B * 64 + 2,), 5.0, device="cuda")
        out, lse = flat[1:-1].view(B, 64, 512), flat_lse[1:-1].view(B, 64)
        assert out.data_ptr() % 16 == 4
        ws = dsa.l4_workspace(dsa.L4_OP_SPARSE_MLA, dims, cache)
        dsa.dsa_sparse_mla_decode_l4(bf16_cuda(q), torch.from_numpy(pool).cuda(), cache,
                                     torch.from_numpy(idx).cuda(), dims, out, lse, ws)
        assert dsa.workspace_check(ws) == (0, 0)
        assert flat[0] == 5 and flat[-1] == 5 and flat_lse[0] == 5 and flat_lse[-1] == 5
        rows = range(B) if B < 10 else (0, 1, 2, 77, 159)
        _check_attention(q, values, pg, idx, out.double().cpu().numpy(), lse.double().cpu().numpy(),
                         512, 0.0625, False, rows)


def test_offsets_past_32_bits():
    """A pool of more than 2^31 bytes: rows at its end are written, read and attended."""
    W, rb = 576, 336
    pages = 2 ** 31 // (64 * rb) + 40
    pool = torch.zeros(pages, 64, rb, dtype=torch.uint8, device="cuda")
    keys = torch.zeros(pages, 64, 32, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(2)
    n = 128
    x = to_bf16(rng.standard_normal((n, W)))
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device="cuda")
    cache = dsa.PagedCache(torch.tensor([n], dtype=torch.int32, device="cuda"), table, pages, n)
    dims = _dims(n, W, 64, causal=1)
    ws = dsa.l4_workspace(dsa.L4_OP_STATUS, dims, cache)
    dsa.dsa_cache_append_l4(torch.zeros(n, 32, dtype=torch.bfloat16, device="cuda"), bf16_cuda(x), keys,
                            pool, cache, dims, ws)
    values = l4.quantise(x)[1]
    one = _dims(1, W, 64, topk=n, H=64, scale=0.0625)
    idx = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    rows = torch.zeros(1, n, W, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_cache_read_l4(pool, cache, idx, one, rows, ws)
    assert np.array_equal(rows[0].double().cpu().numpy(), values)
    q = to_bf16(rng.standard_normal((1, 64, W)))
    out, lse = torch.zeros(1, 64, 512, device="cuda"), torch.zeros(1, 64, device="cuda")
    ws = dsa.l4_workspace(dsa.L4_OP_SPARSE_MLA, one, cache)
    dsa.dsa_sparse_mla_decode_l4(bf16_cuda(q), pool, cache, idx, one, out, lse, ws)
    assert dsa.workspace_check(ws) == (0, 0)
    ref, ref_lse, p = l4.attention(q[0], values, 512, 0.0625)
    tol, ltol = attention_bounds(q[0], values, 512, 0.0625, p)
    assert (np.abs(out[0].double().cpu().numpy() - ref) <= tol).all()
    assert (np.abs(lse[0].double().cpu().numpy() - ref_lse) <= ltol).all()


def test_two_calls_at_once_on_two_streams():
    """Calls with workspaces of their own overlap without touching each other."""
    rng = np.random.default_rng(15)
    pg = Paged([1500] * 8, seed=4)
    pool, _ = random_l4(rng, pg.num_pages, 576)
    pool = torch.from_numpy(pool).cuda()
    cache, dims = pg.cache(), _dims(8, 576, 64, topk=1024, H=64, scale=0.0625)
    calls = []
    for i in range(2):
        q = bf16_cuda(to_bf16(rng.standard_normal((8, 64, 576))))
        idx = torch.from_numpy(select(rng, pg.lens, 1024)).cuda()
        calls.append((q, idx, torch.zeros(8, 64, 512, device="cuda"), torch.zeros(8, 64, device="cuda"),
                      dsa.l4_workspace(dsa.L4_OP_SPARSE_MLA, dims, cache)))
    alone = []
    for q, idx, out, lse, ws in calls:
        dsa.dsa_sparse_mla_decode_l4(q, pool, cache, idx, dims, out, lse, ws)
        torch.cuda.synchronize()
        alone.append((out.clone(), lse.clone()))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for (q, idx, out, lse, ws), s in zip(calls, streams):
            with torch.cuda.stream(s):
                out.zero_()
                dsa.dsa_sparse_mla_decode_l4(q, pool, cache, idx, dims, out, lse, ws)
        torch.cuda.synchronize()
        for (_, _, out, lse, _), (ref, ref_lse) in zip(calls, alone):
            assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


@pytest.mark.parametrize("kernel", [8, 9], ids=["attention", "mass"])
def test_bounded_wait_times_out(kernel):
    """DSA_DEBUG_STALL makes the kernel wait once on a barrier that nothing
    arrives at: with a 50 ms limit it reports a time-out, drains what is in
    flight and returns, and the context stays usable (in a child process: the
    library reads both variables once)."""
    code = r"""
import sys, numpy as np, torch
sys.path.insert(0, %r)
import sparse_attention_scores_b200 as dsa
from tests.l4_testutil import Paged, bf16_cuda, random_l4, select
rng = np.random.default_rng(0)
pg = Paged([3000, 1500], seed=1)
pool, _ = random_l4(rng, pg.num_pages, 576)
cache = pg.cache()
dims = dsa.Dims(2, 1, 32, 2048, 64, 512, 64, 0, 0, 0.0625)
pool, q = torch.from_numpy(pool).cuda(), bf16_cuda(rng.standard_normal((2, 64, 576)))
idx = torch.from_numpy(select(rng, pg.lens, 2048)).cuda()
out, lse = torch.zeros(2, 64, 512, device="cuda"), torch.zeros(2, 64, device="cuda")
if %d == 8:
    ws = dsa.l4_workspace(dsa.L4_OP_SPARSE_MLA, dims, cache)
    dsa.dsa_sparse_mla_decode_l4(q, pool, cache, idx, dims, out, lse, ws)
else:
    ws = dsa.l4_workspace(dsa.L4_OP_ATTENTION_MASS, dims, cache)
    mass = torch.zeros(2, 3000, device="cuda")
    dsa.dsa_attention_mass_l4(q, pool, cache, idx, lse, dims, 1.0, mass, mass, ws)
st, info = dsa.workspace_check(ws)
x = torch.ones(1000, device="cuda").sum().item()
print("STATUS", st, hex(info), x)
""" % (ROOT, kernel)
    env = dict(os.environ, DSA_WAIT_LIMIT_NS="50000000", DSA_DEBUG_STALL=str(kernel))
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env,
                         timeout=300, cwd=ROOT)
    assert res.returncode == 0, res.stderr[-2000:]
    line = [ln for ln in res.stdout.splitlines() if ln.startswith("STATUS")][0].split()
    assert int(line[1]) == 5 and int(line[2], 16) >> 24 == kernel and line[3] == "1000.0", line


def test_binding_checks_types_and_layouts():
    pg = Paged([100], seed=1)
    cache, dims = pg.cache(), _dims(1, 80, 16, topk=8, H=4)
    pool = torch.zeros(pg.num_pages, 64, 48, dtype=torch.uint8, device="cuda")
    q = torch.zeros(1, 4, 80, dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros(1, 8, dtype=torch.int32, device="cuda")
    out, lse = torch.zeros(1, 4, 64, device="cuda"), torch.zeros(1, 4, device="cuda")
    ws = dsa.l4_workspace(dsa.L4_OP_SPARSE_MLA, dims, cache)
    good = dict(q=q, latent4_pages=pool, idx=idx, out=out, lse=lse)
    for name, bad in (("q", q.float()), ("q", q.cpu()), ("q", q[:, :3]), ("idx", idx.long()),
                      ("latent4_pages", pool[:, :, :40]), ("latent4_pages", pool[:-1]),
                      ("out", torch.zeros(1, 64, 4, device="cuda").transpose(1, 2)),
                      ("lse", lse.double())):
        a = dict(good, **{name: bad})
        with pytest.raises(ValueError, match=name):
            dsa.dsa_sparse_mla_decode_l4(a["q"], a["latent4_pages"], cache, a["idx"], dims, a["out"],
                                         a["lse"], ws)
    with pytest.raises(dsa.DsaError):
        dsa.dsa_sparse_mla_prefill_l4(q, pool, cache, idx, dims, out, lse, ws)  # decode dims
    dsa.dsa_sparse_mla_decode_l4(q, pool, cache, idx, dims, out, lse, ws)
    assert dsa.workspace_check(ws) == (0, 0)
