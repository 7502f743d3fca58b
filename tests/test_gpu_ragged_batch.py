"""Indexer scores, exactly, of batches whose longest row promises many more
key tiles than there are: ragged decode batches and causal chunks of middling
length, for which the work counter is prepared and then not used."""

import numpy as np
import pytest
import torch

import sparse_attention_scores_b200 as dsa

pytestmark = pytest.mark.gpu


def _inputs(rng, lens, n_q, H, D):
    npg = [-(-n // 64) for n in lens]
    pages = sum(npg)
    table = np.full((len(lens), max(npg)), -1, np.int32)
    order, at = rng.permutation(pages), 0
    for b, k in enumerate(npg):
        table[b, :k] = order[at:at + k]
        at += k
    keys = torch.from_numpy(rng.integers(-3, 4, (pages, 64, D)).astype(np.float32)).cuda()
    q = torch.from_numpy(rng.integers(-3, 4, (n_q, H, D)).astype(np.float32)).cuda()
    w = torch.from_numpy(rng.integers(0, 4, (n_q, H)).astype(np.float32)).cuda()
    cache = dsa.PagedCache(torch.tensor(lens, dtype=torch.int32, device="cuda"),
                           torch.from_numpy(table).cuda(), pages, max(lens))
    return cache, torch.from_numpy(table).cuda().long(), keys, q, w


def _scores(keys, rows, q, w):
    """Exact: small integers, whose sums stay far below 2^24."""
    k = keys[rows].flatten(0, 1)
    return (torch.relu(q @ k.T) * w[:, None]).sum(0)


@pytest.mark.parametrize("lens,H,D", [
    ([2820, 11145, 14962, 15418, 3707, 15204, 10378, 9004, 5451, 16056, 4022, 12538, 13277, 15435,
      3573, 11603, 5364, 10459, 4403, 2816], 16, 64),
    ([1] * 31 + [20000], 32, 128), ([64, 128, 129] * 20 + [30000], 4, 32)])
def test_ragged_decode_scores_every_key(lens, H, D):
    rng = np.random.default_rng(len(lens))
    n = len(lens)
    cache, table, keys, q, w = _inputs(rng, lens, n, H, D)
    dims = dsa.Dims(n, H, D, 8, 1, 64, 0, 0, 0, 1.0)
    ws = dsa.workspace(dsa.OP_INDEXER_SCORES, dims, cache)
    scores = torch.full((n, (max(lens) + 3) // 4 * 4), -7.0, device="cuda")
    dsa.dsa_indexer_scores(q.bfloat16(), w, keys.bfloat16(), cache, dims, scores, ws)
    assert dsa.workspace_check(ws) == (0, 0)
    for b, m in enumerate(lens):
        ref = _scores(keys, table[b, :-(-m // 64)], q[b], w[b])[:m]
        assert torch.equal(scores[b, :m], ref), b


@pytest.mark.parametrize("T,pos0,H,D", [(800, 0, 32, 128), (700, 100, 32, 64), (1000, 0, 64, 128)])
def test_causal_chunk_scores_every_key(T, pos0, H, D):
    rng = np.random.default_rng(T)
    cache, table, keys, q, w = _inputs(rng, [pos0 + T], T, H, D)
    dims = dsa.Dims(T, H, D, 8, 1, 64, 0, 1, pos0, 1.0)
    ws = dsa.workspace(dsa.OP_INDEXER_SCORES, dims, cache)
    scores = torch.full((T, (pos0 + T + 3) // 4 * 4), -7.0, device="cuda")
    dsa.dsa_indexer_scores(q.bfloat16(), w, keys.bfloat16(), cache, dims, scores, ws)
    assert dsa.workspace_check(ws) == (0, 0)
    for t in range(T):
        ref = _scores(keys, table[0], q[t], w[t])[:pos0 + t + 1]
        assert torch.equal(scores[t, :pos0 + t + 1], ref), t
