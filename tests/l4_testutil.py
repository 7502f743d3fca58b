"""Helpers of the 4-bit cache, attention-mass and eviction tests: seeded paged
inputs, and the error bounds their comparisons use."""

from __future__ import annotations

import numpy as np
import torch

import dsa_inputs as di
import sparse_attention_scores_b200 as dsa
from oracle import dsa_oracle as orc
from oracle import l4_oracle as l4

U = 2.0 ** -23  # one fp32 rounding or truncation, relative


def to_bf16(x: np.ndarray) -> np.ndarray:
    """float64 values of x rounded to bf16."""
    return orc.bf16_to_f64(di.f32_to_bf16_bits(np.asarray(x, np.float32)))


def bf16_cuda(x: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).cuda()


class Paged:
    """A paged cache of `lens` tokens (shuffled pages, one spare page)."""

    def __init__(self, lens, seed=0, max_seq_len=None):
        rng = np.random.default_rng([seed, 77])
        self.lens = [int(n) for n in lens]
        npg = [max(1, -(-n // 64)) for n in self.lens]
        self.num_pages = sum(npg) + 1
        order = rng.permutation(self.num_pages)
        self.table = np.full((len(lens), max(npg)), -1, np.int32)
        at = 0
        for b, k in enumerate(npg):
            self.table[b, :k] = order[at:at + k]
            at += k
        self.max_seq_len = max(self.lens) if max_seq_len is None else max_seq_len

    def rows(self, b, pos):
        pos = np.asarray(pos, np.int64)
        return self.table[b][pos // 64].astype(np.int64) * 64 + pos % 64

    def cache(self):
        return dsa.PagedCache(torch.tensor(self.lens, dtype=torch.int32).cuda(),
                              torch.from_numpy(self.table).cuda(), self.num_pages,
                              self.max_seq_len)


def random_l4(rng, num_pages, W, spread=2.0):
    """(pool [num_pages, 64, row bytes], values [num_pages * 64, W]) of quantised rows whose sizes differ."""
    n = num_pages * 64
    x = rng.standard_normal((n, W)) * np.exp2(rng.uniform(-spread, spread, (n, 1)))
    packed, values = l4.quantise(to_bf16(x))
    return packed.reshape(num_pages, 64, -1), values


def select(rng, seen, k):
    """[rows, k] ascending distinct positions of what each row sees, -1 padded."""
    idx = np.full((len(seen), k), -1, np.int32)
    for r, n in enumerate(seen):
        m = min(n, k)
        if m > 0:
            idx[r, :m] = np.sort(rng.choice(n, size=m, replace=False))
    return idx


def logit_bound(q, L, scale):
    """Bound on |z - exact| [H, m]: the products are exact and the tensor cores
    add 16 of them per fp32 accumulation (a CUDA-core form adds fewer than 24
    per lane), so W / 16 + 24 roundings of partial sums of at most sum |q L|;
    the scales and the change to base 2 add four more of |z|."""
    W = q.shape[1]
    mag = scale * (np.abs(q) @ np.abs(L).T)
    return (W / 16 + 28) * U * mag


def attention_bounds(q, L, R, scale, p):
    """(bound on out [H, R], bound on lse [H]) of one row.  A logit error d and
    the exponential's own (2^-21 with its argument's rounding) change a weight
    by at most d + 2^-21 relative, which counts twice (weight and sum); the
    weights are carried to 2^-21; K / 8 + 64 accumulations of the weighted sum
    (16 keys each, two terms) and of the weight sum round once each."""
    K = len(L)
    if K == 0:
        return np.zeros((len(q), R)), np.zeros(len(q))
    d = logit_bound(q, L, scale)
    rel = 2 * d + 2.0 ** -19
    acc = (K / 8 + 64) * U
    mag = np.abs(L[:, :R])
    out = (p * rel) @ mag + (p * rel).sum(1, keepdims=True) * (p @ mag) + 2 * acc * (p @ mag)
    # The weights w_j = p_j 2^e_j (up to a factor) reach the tensor cores as
    # fp16 pairs scaled so that the largest is at least 2^6: fp16 ends in steps
    # of 2^-24, so no w_j is off by less than 2^-25 / 2^6 = 2^-31 of the largest
    # (a column that the large weights multiply by zero shows it).  Token j's
    # row enters as L_j 2^-e_j, and a row's largest magnitude lies in
    # (1250, 2688] 2^e: above half of 2688 2^e, less the scale's and the code's
    # rounding of at most 1/16 of it.
    big = np.abs(L).max(1)
    live = big > 0
    if live.any():
        top = (p[:, live] * big[live]).max(1, keepdims=True) / 1250
        out = out + 2.0 ** -31 * top * ((mag[live] * (2688 / big[live])[:, None]).sum(0))
    lse = (p * d).sum(1) * 2 + acc + 2.0 ** -20 + 64 * U  # |lse| below 64 in these tests
    return out + 1e-30, lse
