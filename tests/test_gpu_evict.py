"""Attention mass and eviction on the GPU against their float64 definitions:
masses within bounds derived from their roundings, kept positions and moved
rows exactly; and a request's life over the 4-bit cache."""

import numpy as np
import pytest
import torch

import sparse_attention_scores_b200 as dsa
from oracle import l4_oracle as l4
from tests.l4_testutil import Paged, U, bf16_cuda, logit_bound, random_l4, select, to_bf16

pytestmark = pytest.mark.gpu


def _dims(n_q, R, P, H, k, *, causal=0, q_pos0=0, scale=0.0625, D_I=32, H_I=1):
    return dsa.Dims(n_q, H_I, D_I, k, H, R, P, causal, q_pos0, scale)


def _latents(fmt, rng, pg, W):
    """(call, its latent arguments, the rows' values) for one cache format."""
    if fmt == "l4":
        pool, values = random_l4(rng, pg.num_pages, W)
        return dsa.dsa_attention_mass_l4, (torch.from_numpy(pool).cuda(),), values
    x = to_bf16(rng.standard_normal((pg.num_pages * 64, W)))
    if fmt == "bf16":
        return dsa.dsa_attention_mass, (bf16_cuda(x).view(pg.num_pages, 64, W),), x
    codes = torch.from_numpy(x).float().to(torch.float8_e4m3fn)
    s = rng.uniform(0.5, 1.5, pg.num_pages * 64).astype(np.float32)
    return (dsa.dsa_attention_mass_l8,
            (codes.view(torch.uint8).view(pg.num_pages, 64, W).cuda(), torch.from_numpy(s).cuda()),
            codes.double().numpy() * s.astype(np.float64)[:, None])


def _reference(pg, values, q, idx, lse, decay, mass_in, causal, scale, n_q):
    """(mass, bound) over the live positions of every sequence."""
    ref = decay * mass_in.astype(np.float64)
    tol = 2 * U * np.abs(ref)
    for r in range(len(idx)):
        b = 0 if causal else r
        pos = idx[r][idx[r] >= 0]
        if len(pos) == 0:
            continue
        L = values[pg.rows(b, pos)]
        l4.add_mass(ref[b], pos, q[r], L, lse[r], scale)
        # each head's weight: its logit's error, the exponential's 2^-19, the
        # argument's rounding (|z - lse| < 128); then the head sum's roundings
        live = np.isfinite(lse[r])
        z = scale * (q[r] @ L.T)
        w = np.exp(np.minimum(z[live] - lse[r][live][:, None], 80))
        rel = logit_bound(q[r], L, scale)[live] + 2.0 ** -19 + 128 * U + 16 * U
        np.add.at(tol[b], pos, (w * rel).sum(0) + 2.0 ** -39)
    return ref, tol + 4 * U * np.abs(ref)


def _true_lse(pg, values, q, idx, causal, scale):
    out = np.full((len(idx), q.shape[1]), -np.inf)
    for r in range(len(idx)):
        pos = idx[r][idx[r] >= 0]
        if len(pos):
            out[r] = l4.attention(q[r], values[pg.rows(0 if causal else r, pos)], 64, scale)[1]
    return out.astype(np.float32)


@pytest.mark.parametrize("fmt", ["l4", "l8", "bf16"])
@pytest.mark.parametrize("B,H,R,P,k,longest", [
    (5, 64, 512, 64, 300, 700), (1, 64, 512, 64, 2048, 5000), (40, 16, 192, 32, 64, 200),
    (3, 4, 64, 16, 256, 300), (2, 33, 448, 0, 65, 100), (160, 64, 512, 0, 5, 40),
    (3, 64, 64, 512, 100, 150), (150, 64, 512, 64, 1000, 1100)])
def test_decode_mass(fmt, B, H, R, P, k, longest):
    rng = np.random.default_rng([B, H, R, k])
    lens = rng.integers(1, longest + 1, B).tolist()
    lens[0] = longest
    pg = Paged(lens, seed=B)
    call, lat, values = _latents(fmt, rng, pg, R + P)
    q = to_bf16(rng.standard_normal((B, H, R + P)))
    idx = select(rng, lens, k)
    if B > 2:
        idx[1] = -1
        idx[2, rng.random(k) < 0.3] = -1
    scale = float(np.float32(1 / np.sqrt(R + P)))
    lse = _true_lse(pg, values, q, idx, False, scale)
    ld = longest + 5
    mass_in = rng.exponential(1.0, (B, ld)).astype(np.float32)
    cache, dims = pg.cache(), _dims(B, R, P, H, k, scale=scale)
    got = torch.full((B, ld), -7.0, device="cuda")
    ws = dsa.l4_workspace(dsa.L4_OP_ATTENTION_MASS, dims, cache)
    args = (bf16_cuda(q), *lat, cache, torch.from_numpy(idx).cuda(), torch.from_numpy(lse).cuda(),
            dims, 0.875)
    call(*args, torch.from_numpy(mass_in).cuda(), got, ws)
    assert dsa.workspace_check(ws) == (0, 0)
    ref, tol = _reference(pg, values, q, idx, lse, 0.875, mass_in, False, scale, B)
    g = got.double().cpu().numpy()
    for b, n in enumerate(lens):
        assert (np.abs(g[b, :n] - ref[b, :n]) <= tol[b, :n]).all(), (b, np.abs(g[b, :n] - ref[b, :n]).max())
        assert (g[b, n:] == -7.0).all(), "positions past the sequence changed"
    # the weights of a row that kept something sum to the heads
    add = g[0, :lens[0]] - 0.875 * mass_in[0, :lens[0]].astype(np.float64)
    assert abs(add.sum() - H) <= tol[0, :lens[0]].sum()
    # in place, and without an earlier sum
    again = torch.from_numpy(mass_in).cuda()
    call(*args, again, again, ws)
    fresh = torch.full((B, ld), 3.0, device="cuda")
    call(*args, None, fresh, ws)
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        assert torch.equal(again[b, :n], got[b, :n])
        assert np.array_equal(again[b, n:].cpu().numpy(), mass_in[b, n:])
        f = fresh[b, :n].double().cpu().numpy()
        assert (np.abs(f - (ref[b, :n] - 0.875 * mass_in[b, :n].astype(np.float64))) <= tol[b, :n]).all()


@pytest.mark.parametrize("fmt", ["l4", "l8", "bf16"])
@pytest.mark.parametrize("T,pos0,H,R,P,k", [(100, 0, 64, 512, 64, 64), (33, 500, 16, 192, 32, 300),
                                            (1, 0, 4, 64, 16, 8), (600, 10, 64, 512, 0, 40),
                                            (200, 900, 64, 512, 64, 1000)])
def test_causal_mass_does_not_depend_on_order(fmt, T, pos0, H, R, P, k):
    rng = np.random.default_rng([T, H])
    pg = Paged([pos0 + T], seed=T)
    call, lat, values = _latents(fmt, rng, pg, R + P)
    q = to_bf16(rng.standard_normal((T, H, R + P)))
    idx = select(rng, [pos0 + t + 1 for t in range(T)], k)
    if T > 2:
        idx[2] = -1
    lse = _true_lse(pg, values, q, idx, True, 0.0625)
    cache, dims = pg.cache(), _dims(T, R, P, H, k, causal=1, q_pos0=pos0)
    mass_in = rng.exponential(1.0, (1, pos0 + T + 3)).astype(np.float32)
    ws = dsa.l4_workspace(dsa.L4_OP_ATTENTION_MASS, dims, cache)
    runs = []
    for _ in range(3):
        got = torch.full((1, pos0 + T + 3), -7.0, device="cuda")
        call(bf16_cuda(q), *lat, cache, torch.from_numpy(idx).cuda(), torch.from_numpy(lse).cuda(),
             dims, 0.5, torch.from_numpy(mass_in).cuda(), got, ws)
        runs.append(got)
    assert dsa.workspace_check(ws) == (0, 0)
    assert torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2])
    ref, tol = _reference(pg, values, q, idx, lse, 0.5, mass_in, True, 0.0625, T)
    g, n = runs[0].double().cpu().numpy(), pos0 + T
    assert (np.abs(g[0, :n] - ref[0, :n]) <= tol[0, :n]).all(), np.abs(g[0, :n] - ref[0, :n]).max()
    assert (g[0, n:] == -7.0).all()


@pytest.mark.parametrize("fmt", ["l4", "l8", "bf16"])
@pytest.mark.parametrize("T,pos0,H,R,P,k", [(200, 800, 4, 256, 64, 1000), (300, 2000, 64, 64, 16, 2048)])
def test_mass_of_long_rows_repeats_bit_for_bit(fmt, T, pos0, H, R, P, k):
    """Rows of many slots, narrow or with few heads, so that the filling, the
    products and the sums run at different paces: no wait gives up, and every
    run adds the same weights."""
    rng = np.random.default_rng([T, k])
    pg = Paged([pos0 + T], seed=T)
    call, lat, values = _latents(fmt, rng, pg, R + P)
    q = bf16_cuda(to_bf16(0.3 * rng.standard_normal((T, H, R + P))))
    idx = torch.from_numpy(select(rng, [pos0 + t + 1 for t in range(T)], k)).cuda()
    lse = torch.full((T, H), 8.0, device="cuda")
    cache, dims = pg.cache(), _dims(T, R, P, H, k, causal=1, q_pos0=pos0)
    ws = dsa.l4_workspace(dsa.L4_OP_ATTENTION_MASS, dims, cache)
    runs = [torch.zeros(1, pos0 + T, device="cuda") for _ in range(40)]
    for got in runs:
        call(q, *lat, cache, idx, lse, dims, 1.0, None, got, ws)
    assert dsa.workspace_check(ws) == (0, 0)
    assert all(torch.equal(runs[0], got) for got in runs) and float(runs[0].sum()) > 0


def test_mass_counts_repeats_and_reports_what_is_out_of_range():
    rng = np.random.default_rng(5)
    pg = Paged([100, 64], seed=1)
    call, lat, values = _latents("l4", rng, pg, 80)
    q = to_bf16(rng.standard_normal((2, 4, 80)))
    idx = np.array([[3, 3, 99, -1], [1, 2, 64, 5]], np.int32)  # 64: past the context of row 1
    good = idx.copy()
    good[1, 2] = -1
    lse = _true_lse(pg, values, q, good, False, 0.125)
    cache, dims = pg.cache(), _dims(2, 64, 16, 4, 4, scale=0.125)
    got = torch.zeros(2, 100, device="cuda")
    ws = dsa.l4_workspace(dsa.L4_OP_ATTENTION_MASS, dims, cache)
    call(bf16_cuda(q), *lat, cache, torch.from_numpy(idx).cuda(), torch.from_numpy(lse).cuda(),
         dims, 1.0, None, got, ws)
    st, info = dsa.workspace_check(ws)
    assert st == 6 and info >> 24 == 9
    ref, tol = _reference(pg, values, q, good, lse, 0.0, np.zeros((2, 100), np.float32), False, 0.125, 2)
    g = got.double().cpu().numpy()
    assert (np.abs(g[0] - ref[0]) <= tol[0]).all() and (np.abs(g[1, :64] - ref[1, :64]) <= tol[1, :64]).all()


def test_a_nan_in_the_cache_shows_in_the_mass():
    """A NaN latent row gives NaN masses to the tokens of the rows that kept it
    (their lse is NaN), in a chunk as in a decode step, and to no others."""
    rng = np.random.default_rng(12)
    T, k, H = 70, 8, 16
    pg = Paged([T], seed=4)
    call, (pool,), values = _latents("bf16", rng, pg, 80)
    q = to_bf16(rng.standard_normal((T, H, 80)))
    idx = select(rng, [t + 1 for t in range(T)], k)
    bad = [t for t in range(T) if 40 in idx[t]]
    assert bad
    lse = _true_lse(pg, values, q, idx, True, 0.125)
    pool.view(-1, 80)[int(pg.rows(0, [40])[0]), 3] = float("nan")
    lse[bad] = np.nan
    cache, dims = pg.cache(), _dims(T, 64, 16, H, k, causal=1, scale=0.125)
    ws = dsa.l4_workspace(dsa.L4_OP_ATTENTION_MASS, dims, cache)
    got = torch.zeros(1, T, device="cuda")
    call(bf16_cuda(q), pool, cache, torch.from_numpy(idx).cuda(), torch.from_numpy(lse).cuda(), dims, 1.0,
         None, got, ws)
    touched = np.zeros(T, bool)
    for t in bad:
        touched[idx[t][idx[t] >= 0]] = True
    assert touched.any() and not touched.all()
    assert np.array_equal(np.isnan(got[0].cpu().numpy()), touched)
    g = got[0].double().cpu().numpy()
    clean = np.where(np.isin(np.arange(T), bad)[:, None], -1, idx).astype(np.int32)
    ref, tol = _reference(pg, values, q, clean, lse, 0.0, np.zeros((1, T), np.float32), True, 0.125, T)
    assert (np.abs(g - ref[0])[~touched] <= tol[0][~touched]).all()


def test_lengths_past_max_seq_len_and_views_too_narrow():
    """A length above max_seq_len counts as max_seq_len, and a view of a wider
    tensor that is too narrow for it is refused: nothing outside the view is written."""
    rng = np.random.default_rng(8)
    pg = Paged([150, 100], seed=2, max_seq_len=120)
    call, lat, values = _latents("bf16", rng, pg, 80)
    q = to_bf16(rng.standard_normal((2, 4, 80)))
    idx = np.array([[3, 119, 120, 7], [1, 2, 99, -1]], np.int32)  # 120: past max_seq_len
    good = np.where(idx == 120, -1, idx).astype(np.int32)
    lse = _true_lse(pg, values, q, good, False, 0.125)
    cache, dims = pg.cache(), _dims(2, 64, 16, 4, 4, scale=0.125)
    ws = dsa.l4_workspace(dsa.L4_OP_ATTENTION_MASS, dims, cache)
    whole = torch.full((2, 200), -7.0, device="cuda")
    args = (bf16_cuda(q), *lat, cache, torch.from_numpy(idx).cuda(), torch.from_numpy(lse).cuda(), dims, 1.0)
    call(*args, None, whole[:, :120], ws)
    st, info = dsa.workspace_check(ws)
    assert st == 6 and info >> 24 == 9
    ref, tol = _reference(pg, values, q, good, lse, 0.0, np.zeros((2, 200), np.float32), False, 0.125, 2)
    g = whole.double().cpu().numpy()
    for b, n in enumerate((120, 100)):
        assert (np.abs(g[b, :n] - ref[b, :n]) <= tol[b, :n]).all() and (g[b, n:] == -7.0).all()
    with pytest.raises(dsa.DsaError):
        call(*args, None, whole[:, :119], ws)
    new_lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    ws = dsa.l4_workspace(dsa.L4_OP_CACHE_EVICT, None, cache)
    for m, md in ((whole[:, :119], None), (whole[:, :120], torch.zeros(2, 300, device="cuda")[:, :99])):
        with pytest.raises(dsa.DsaError):
            dsa.dsa_cache_evict([], cache, dsa.Eviction(100), m, table, md, new_lens, None, ws)
    wide = torch.full((2, 300), -7.0, device="cuda")
    dsa.dsa_cache_evict([], cache, dsa.Eviction(100), whole[:, :120], table, wide[:, :100], new_lens, None, ws)
    assert dsa.workspace_check(ws) == (0, 0) and new_lens.tolist() == [100, 100]
    assert (wide[:, 100:] == -7.0).all() and (wide[:, :100] != -7.0).all()


# ------------------------------------------------------------------ eviction
def _evict(pg, mass, budget, sinks, recent, pools, rng, ld=None, with_kept=True, max_seq_len=None):
    B = len(pg.lens)
    most = min(budget, pg.max_seq_len)
    dpg = -(-most // 64)
    table = rng.permutation(dpg * B + 1)[:dpg * B].reshape(B, dpg).astype(np.int32)
    dst = [torch.full((dpg * B + 1, *p.shape[1:]), 77, dtype=torch.uint8, device="cuda").view(p.dtype)
           if p.dtype == torch.uint8 else torch.full((dpg * B + 1, *p.shape[1:]), 77, dtype=p.dtype, device="cuda")
           for p in pools]
    mass_dst = torch.full((B, most + 3), -7.0, device="cuda")
    new_lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    kept = torch.full((B, budget), -9, dtype=torch.int32, device="cuda") if with_kept else None
    cache = pg.cache()
    ws = dsa.l4_workspace(dsa.L4_OP_CACHE_EVICT, None, cache)
    dsa.dsa_cache_evict(list(zip(pools, dst)), cache, dsa.Eviction(budget, sinks, recent),
                        torch.from_numpy(mass).cuda(), torch.from_numpy(table).cuda(), mass_dst,
                        new_lens, kept, ws)
    return dst, table, mass_dst, new_lens, kept, dsa.workspace_check(ws)


def _masses(rng, B, ld, kind):
    if kind == "ties":
        return rng.integers(0, 3, (B, ld)).astype(np.float32)
    if kind == "zeros":
        return np.zeros((B, ld), np.float32)
    m = np.where(rng.random((B, ld)) < 0.5, 0, rng.exponential(1.0, (B, ld))).astype(np.float32)
    if kind == "odd":
        m[rng.random((B, ld)) < 0.05] = np.nan
        m[rng.random((B, ld)) < 0.02] = np.inf
        m[rng.random((B, ld)) < 0.02] = -np.inf
        m[rng.random((B, ld)) < 0.05] *= -1
    return m


@pytest.mark.parametrize("kind", ["plain", "ties", "zeros", "odd"])
@pytest.mark.parametrize("lens,budget,sinks,recent", [
    ([300, 1, 64, 65, 1000], 64, 4, 16), ([5000], 2500, 0, 0), ([200, 100], 300, 5, 5),
    ([129, 4097, 0], 1, 0, 1), ([9000, 20000], 8192, 8192, 0), ([40000], 33000, 7, 32993),
    ([100, 90], 100, 50, 50), ([777] * 20, 400, 10, 100)])
def test_evict_keeps_and_moves_exactly(kind, lens, budget, sinks, recent):
    rng = np.random.default_rng([budget, sinks, len(lens)])
    pg = Paged(lens, seed=budget)
    mass = _masses(rng, len(lens), max(lens) + 2, kind)
    pools = [torch.from_numpy(rng.integers(0, 256, (pg.num_pages, 64, 336)).astype(np.uint8)).cuda(),
             torch.from_numpy(rng.standard_normal((pg.num_pages, 64, 128)).astype(np.float32)).bfloat16().cuda(),
             torch.from_numpy(rng.standard_normal((pg.num_pages, 64)).astype(np.float32)).cuda()]
    dst, table, mass_dst, new_lens, kept, st = _evict(pg, mass, budget, sinks, recent, pools, rng)
    assert st == (0, 0)
    got_mass, got_kept = mass_dst.cpu().numpy(), kept.cpu().numpy()
    touched = np.zeros(dst[0].shape[0] * 64, bool)
    for b, n in enumerate(lens):
        keep = l4.evict_keep(mass[b, :n], budget, sinks, recent)
        assert new_lens[b] == len(keep) == min(n, budget)
        assert np.array_equal(got_kept[b, :len(keep)], keep) and (got_kept[b, len(keep):] == -1).all()
        i = np.arange(len(keep))
        to = table[b][i // 64].astype(np.int64) * 64 + i % 64
        touched[to] = True
        for p, d in zip(pools, dst):
            flat, dflat = p.reshape(pg.num_pages * 64, -1), d.reshape(len(touched), -1)
            assert torch.equal(dflat[torch.from_numpy(to).cuda()], flat[torch.from_numpy(pg.rows(b, keep)).cuda()])
        assert np.array_equal(got_mass[b, :len(keep)], mass[b][keep], equal_nan=True)
        assert (got_mass[b, len(keep):] == -7.0).all()
    for d in dst:
        rest = d.reshape(len(touched), -1)[torch.from_numpy(~touched).cuda()]
        assert (rest == 77).all(), "a row that nothing was moved to changed"
    # without kept, and without a mass to move, the rows are the same
    again = _evict(pg, mass, budget, sinks, recent, pools, np.random.default_rng(0), with_kept=False)
    assert torch.equal(again[3], new_lens)


@pytest.mark.parametrize("widths", [(4, 4092, 4096, 2128), (1, 1023, 532, 6), (84,), ()])
def test_evict_moves_rows_of_any_width(widths):
    """Row widths (in 4-byte units) from the smallest to the largest, odd ones among them."""
    rng = np.random.default_rng(len(widths))
    for lens, budget in (([300, 90], 128), ([9000] * 5, 4000)):
        pg = Paged(lens, seed=6)
        mass = rng.exponential(1.0, (len(lens), max(lens))).astype(np.float32)
        pools = [torch.randint(-2 ** 31, 2 ** 31 - 1, (pg.num_pages, 64, min(w, 1024)), dtype=torch.int32,
                               device="cuda") for w in widths]
        dst, table, _, new_lens, kept, st = _evict(pg, mass, budget, 2, 30, pools, rng)
        assert st == (0, 0)
        for b, n in enumerate(lens):
            keep = l4.evict_keep(mass[b, :n], budget, 2, 30)
            i = np.arange(len(keep))
            to = torch.from_numpy(table[b][i // 64].astype(np.int64) * 64 + i % 64).cuda()
            src = torch.from_numpy(pg.rows(b, keep)).cuda()
            for p, d in zip(pools, dst):
                assert torch.equal(d.flatten(0, 1)[to], p.flatten(0, 1)[src])


def test_evict_reports_pages_out_of_range():
    rng = np.random.default_rng(2)
    pg = Paged([200, 200], seed=3)
    mass = rng.exponential(1.0, (2, 200)).astype(np.float32)
    pools = [torch.zeros(pg.num_pages, 64, 48, dtype=torch.uint8, device="cuda")]
    pg.table[1, 2] = pg.num_pages + 7
    *_, st = _evict(pg, mass, 200, 0, 0, pools, rng)
    assert st[0] == 6 and st[1] >> 24 == 10


def test_evict_updates_the_lengths_in_place():
    """new_lens may be the cache's own seq_lens, which every part of the ranking
    reads; a call that moves neither masses nor positions out gives the same rows."""
    rng = np.random.default_rng(23)
    lens = [30000, 50, 9000, 30001]
    pg = Paged(lens, seed=9)
    mass = torch.from_numpy(_masses(rng, 4, max(lens), "plain")).cuda()
    pool = torch.from_numpy(rng.integers(0, 256, (pg.num_pages, 64, 336)).astype(np.uint8)).cuda()
    table = torch.arange(32, dtype=torch.int32, device="cuda").view(4, 8)
    out = []
    for in_place in (False, True):
        cache, dst = pg.cache(), torch.zeros(32, 64, 336, dtype=torch.uint8, device="cuda")
        lens_out = cache.seq_lens if in_place else torch.zeros(4, dtype=torch.int32, device="cuda")
        ws = dsa.l4_workspace(dsa.L4_OP_CACHE_EVICT, None, cache)
        kept = None if in_place else torch.zeros(4, 500, dtype=torch.int32, device="cuda")
        mass_dst = None if in_place else torch.zeros(4, 500, device="cuda")
        dsa.dsa_cache_evict([(pool, dst)], cache, dsa.Eviction(500, 4, 100), mass, table, mass_dst,
                            lens_out, kept, ws)
        assert dsa.workspace_check(ws) == (0, 0)
        out.append((dst, lens_out.tolist()))
    assert out[0][1] == out[1][1] == [500, 50, 500, 500]
    assert torch.equal(out[0][0], out[1][0])


def test_captured_calls_replay():
    """Append, mass and eviction in one captured graph give what eager calls
    give, replay after replay, beside a second graph with its own workspaces."""
    rng = np.random.default_rng(17)
    lens, H, k = [900, 300], 16, 128
    pg = Paged(lens, seed=3)
    _, (pool,), values = _latents("l4", rng, pg, 576)
    q = bf16_cuda(to_bf16(rng.standard_normal((2, H, 576))))
    sel = select(rng, lens, k)
    idx = torch.from_numpy(sel).cuda()
    cache, dims = pg.cache(), _dims(2, 512, 64, H, k)
    keys = torch.zeros(pg.num_pages, 64, 32, dtype=torch.bfloat16, device="cuda")
    new = bf16_cuda(to_bf16(rng.standard_normal((2, 576))))
    key = bf16_cuda(to_bf16(rng.standard_normal((2, 32))))
    lse = torch.full((2, H), 3.0, device="cuda")
    start = torch.rand(2, 900, device="cuda")
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)

    def buffers():
        return dict(mass=torch.zeros(2, 900, device="cuda"), dst=torch.zeros(8, 64, 336, dtype=torch.uint8, device="cuda"),
                    mass_dst=torch.zeros(2, 256, device="cuda"), lens=torch.zeros(2, dtype=torch.int32, device="cuda"),
                    kept=torch.zeros(2, 200, dtype=torch.int32, device="cuda"),
                    ws=[dsa.l4_workspace(op, dims, cache) for op in
                        (dsa.L4_OP_STATUS, dsa.L4_OP_ATTENTION_MASS, dsa.L4_OP_CACHE_EVICT)])

    def call(b):
        dsa.dsa_cache_append_l4(key, new, keys, pool, cache, dims, b["ws"][0])
        dsa.dsa_attention_mass_l4(q, pool, cache, idx, lse, dims, 0.5, start, b["mass"], b["ws"][1])
        dsa.dsa_cache_evict([(pool, b["dst"])], cache, dsa.Eviction(200, 4, 32), b["mass"], table,
                            b["mass_dst"], b["lens"], b["kept"], b["ws"][2])

    eager = buffers()
    call(eager)
    torch.cuda.synchronize()
    graphs, bufs = [], [buffers(), buffers()]
    torch.cuda.synchronize()
    for b in bufs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(b)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for b in bufs:
        for name in ("dst", "mass_dst", "lens", "kept"):
            assert torch.equal(b[name], eager[name]), name
        for r, n in enumerate(lens):
            assert torch.equal(b["mass"][r, :n], eager["mass"][r, :n])


def test_a_requests_life_over_the_4_bit_cache():
    """Prompt rows appended, attended, weighed; the cache evicted into fresh
    pages of the same pools; then decode steps on what is left: every stage
    against the float64 definition over the rows that the cache must hold."""
    rng = np.random.default_rng(31)
    T, H, R, P, HI, DI, k = 200, 64, 512, 64, 4, 64, 96
    W, scale, budget = R + P, 0.0625, 120
    pages = 8
    table = np.array([[2, 0, 5, 1]], np.int32)            # 256 tokens of room
    fresh = np.array([[7, 3, 6, 4]], np.int32)
    keys = torch.zeros(pages, 64, DI, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(pages, 64, l4.row_bytes(W), dtype=torch.uint8, device="cuda")
    lat_new, k_new = to_bf16(rng.standard_normal((T, W))), rng.integers(-3, 4, (T, DI)).astype(np.float64)
    values = l4.quantise(lat_new)[1]
    seq = torch.tensor([T], dtype=torch.int32, device="cuda")
    cache = dsa.PagedCache(seq, torch.from_numpy(table).cuda(), pages, 256)

    def forward(dims, cache, n, q, q_idx, w):
        idx = torch.zeros(n, k, dtype=torch.int32, device="cuda")
        out, lse = torch.zeros(n, H, R, device="cuda"), torch.zeros(n, H, device="cuda")
        ws = dsa.l4_workspace(dsa.L4_OP_ATTENTION_FORWARD, dims, cache)
        dsa.dsa_attention_forward_l4(bf16_cuda(q_idx), torch.from_numpy(w).float().cuda(), keys,
                                     bf16_cuda(q), pool, cache, dims, idx, out, lse, ws)
        assert dsa.workspace_check(ws) == (0, 0)
        return idx, out, lse

    def draw(n):
        return (to_bf16(rng.standard_normal((n, H, W))), rng.integers(-3, 4, (n, HI, DI)).astype(np.float64),
                rng.integers(0, 4, (n, HI)).astype(np.float64))

    def keep_of(q_idx, w, rows):
        s = (w[:, None] * np.maximum(q_idx @ rows.T, 0)).sum(0)
        return np.sort(np.argsort(-s, kind="stable")[:k])

    # the prompt
    dims = _dims(T, R, P, H, k, causal=1, D_I=DI, H_I=HI, scale=scale)
    ws = dsa.l4_workspace(dsa.L4_OP_STATUS, dims, cache)
    dsa.dsa_cache_append_l4(bf16_cuda(k_new), bf16_cuda(lat_new), keys, pool, cache, dims, ws)
    q, q_idx, w = draw(T)
    idx, out, lse = forward(dims, cache, T, q, q_idx, w)
    mass = torch.zeros(1, 256, device="cuda")
    ws = dsa.l4_workspace(dsa.L4_OP_ATTENTION_MASS, dims, cache)
    dsa.dsa_attention_mass_l4(bf16_cuda(q), pool, cache, idx, lse, dims, 1.0, mass, mass, ws)
    ref = np.zeros(256)
    for t in range(T):
        keep = keep_of(q_idx[t], w[t], k_new[:t + 1])
        assert np.array_equal(idx[t].cpu().numpy()[:len(keep)], keep)
        o, ls, p = l4.attention(q[t], values[keep], R, scale)
        assert np.abs(out[t].double().cpu().numpy() - o).max() <= 2e-3 * np.abs(o).max()
        np.add.at(ref, keep, p.sum(0))
    m = mass[0].double().cpu().numpy()
    assert np.abs(m - ref).max() <= 2e-3 * ref.max() and abs(m.sum() - T * H) <= 1e-3 * T * H
    # the eviction, into other pages of the same pools
    new_lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept = torch.zeros(1, budget, dtype=torch.int32, device="cuda")
    mass2 = torch.zeros(1, 256, device="cuda")
    ws = dsa.l4_workspace(dsa.L4_OP_CACHE_EVICT, None, cache)
    dsa.dsa_cache_evict([(pool, pool), (keys, keys)], cache, dsa.Eviction(budget, 4, 16), mass,
                        torch.from_numpy(fresh).cuda(), mass2, new_lens, kept, ws)
    assert dsa.workspace_check(ws) == (0, 0)
    left = l4.evict_keep(mass[0, :T].cpu().numpy(), budget, 4, 16)
    assert np.array_equal(kept[0].cpu().numpy(), left) and int(new_lens[0]) == budget
    assert torch.equal(mass2[0, :budget], mass[0][torch.from_numpy(left).cuda()])
    values, k_new = values[left], k_new[left]
    # two decode steps on what is left
    seq = new_lens.clone()
    cache = dsa.PagedCache(seq, torch.from_numpy(fresh).cuda(), pages, 256)
    dims = _dims(1, R, P, H, k, D_I=DI, H_I=HI, scale=scale)
    for _ in range(2):
        seq += 1
        row, key = to_bf16(rng.standard_normal((1, W))), rng.integers(-3, 4, (1, DI)).astype(np.float64)
        values, k_new = np.concatenate([values, l4.quantise(row)[1]]), np.concatenate([k_new, key])
        ws = dsa.l4_workspace(dsa.L4_OP_STATUS, dims, cache)
        dsa.dsa_cache_append_l4(bf16_cuda(key), bf16_cuda(row), keys, pool, cache, dims, ws)
        q, q_idx, w = draw(1)
        idx, out, lse = forward(dims, cache, 1, q, q_idx, w)
        keep = keep_of(q_idx[0], w[0], k_new)
        assert np.array_equal(idx[0].cpu().numpy()[:len(keep)], keep)
        o, ls, p = l4.attention(q[0], values[keep], R, scale)
        assert np.abs(out[0].double().cpu().numpy() - o).max() <= 2e-3 * np.abs(o).max()
        assert np.abs(lse[0].double().cpu().numpy() - ls).max() <= 2e-3
