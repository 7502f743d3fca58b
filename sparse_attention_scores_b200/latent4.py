"""Binding of include/dsa_l4.h: the 4-bit latent cache, the attention weight its
tokens receive, and eviction by it.

Argument marshalling, as in the package's other functions, plus the checks a
raw pointer cannot carry: every tensor must be contiguous (a row-strided score
or mass tensor may have a row stride above its width), of the stated type, and
on the current CUDA device, whose current stream the call takes by default.  A
tensor of another kind raises ValueError before anything is launched; a refusal
by the library raises DsaError.
"""

from __future__ import annotations

import ctypes
import struct
from dataclasses import dataclass

import sparse_attention_scores_b200 as _dsa

L4_OP_STATUS = 0
L4_OP_SPARSE_MLA = 1
L4_OP_ATTENTION_FORWARD = 2
L4_OP_ATTENTION_MASS = 3
L4_OP_CACHE_EVICT = 4
EVICT_MAX_POOLS = 4  # DSA_EVICT_MAX_POOLS

L4_EXPORTED = ["dsa_l4_row_bytes", "dsa_l4_workspace_bytes", "dsa_cache_append_l4",
               "dsa_cache_read_l4", "dsa_sparse_mla_decode_l4", "dsa_sparse_mla_prefill_l4",
               "dsa_attention_forward_l4", "dsa_attention_mass", "dsa_attention_mass_l8",
               "dsa_attention_mass_l4", "dsa_cache_evict"]


class PoolStruct(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("row_bytes", ctypes.c_int32)]


class EvictStruct(ctypes.Structure):
    _fields_ = [("budget", ctypes.c_int32), ("sinks", ctypes.c_int32), ("recent", ctypes.c_int32),
                ("dst_block_table", ctypes.c_void_p), ("dst_max_pages", ctypes.c_int32),
                ("dst_num_pages", ctypes.c_int32)]


_ready = _torch = _bf16 = _f32 = _i32 = _u8 = None
# dsa_cache_t and dsa_dims_t as packed bytes: half the time of a ctypes structure,
# which counts in calls whose kernels run a few microseconds
_pack_cache = struct.Struct("@iPPiiii").pack
_pack_dims = struct.Struct("@9if").pack
assert struct.calcsize("@iPPiiii") == ctypes.sizeof(_dsa.CacheStruct)
assert struct.calcsize("@9if") == ctypes.sizeof(_dsa.DimsStruct)


def l4_lib() -> ctypes.CDLL:
    """The loaded library with the signatures of include/dsa_l4.h."""
    global _ready, _torch, _bf16, _f32, _i32, _u8
    if _ready is None:
        import torch
        _torch = torch
        _bf16, _f32, _i32, _u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
        L = _dsa.lib()
        vp, sz, i32, i64, f32 = (ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64,
                                 ctypes.c_float)
        pc = pd = vp  # structures by reference, or their bytes
        pp, pe = ctypes.POINTER(PoolStruct), ctypes.POINTER(EvictStruct)
        end = [vp, sz, vp]  # workspace, its size, stream
        mass_end = [pc, vp, vp, pd, f32, vp, vp, i64] + end
        sigs = {
            "dsa_l4_row_bytes": ([i32, i32], sz),
            "dsa_l4_workspace_bytes": ([ctypes.c_int, pd, pc], sz),
            "dsa_cache_append_l4": ([vp, vp, vp, vp, pc, pd] + end, ctypes.c_int),
            "dsa_cache_read_l4": ([vp, pc, vp, pd, vp] + end, ctypes.c_int),
            "dsa_sparse_mla_decode_l4": ([vp, vp, pc, vp, pd, vp, vp] + end, ctypes.c_int),
            "dsa_sparse_mla_prefill_l4": ([vp, vp, pc, vp, pd, vp, vp] + end, ctypes.c_int),
            "dsa_attention_forward_l4": ([vp, vp, vp, vp, vp, pc, pd, vp, vp, vp] + end,
                                         ctypes.c_int),
            "dsa_attention_mass": ([vp, vp] + mass_end, ctypes.c_int),
            "dsa_attention_mass_l8": ([vp, vp, vp] + mass_end, ctypes.c_int),
            "dsa_attention_mass_l4": ([vp, vp] + mass_end, ctypes.c_int),
            "dsa_cache_evict": ([pp, i32, pc, pe, vp, i64, vp, i64, vp, vp] + end, ctypes.c_int),
        }
        for name, (args, res) in sigs.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _ready = L
    return _ready


def _device():
    """The current CUDA device's index."""
    return _torch._C._cuda_getDevice()


def _arg(t, name, dtype, device, shape=None, rows=False):
    """The pointer of a tensor argument after its checks (None stays None).
    rows: a 2-d tensor whose rows are contiguous, at any row stride."""
    if t is None:
        return None
    if t.get_device() != device:
        raise ValueError(f"{name}: on {t.device}, the call runs on cuda:{device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: {t.dtype}, expected {dtype}")
    if not t.is_contiguous() and not (rows and t.dim() == 2 and t.stride(1) == 1 and
                                      t.stride(0) >= t.shape[1]):
        raise ValueError(f"{name}: not contiguous (strides {tuple(t.stride())})")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
    return t.data_ptr()


def _common(cache, dims, ws, device):
    """(cache and dims structures, workspace pointer, its size) of a call."""
    lens, table = cache.seq_lens, cache.block_table
    lens_ptr, table_ptr = _arg(lens, "seq_lens", _i32, device), _arg(table, "block_table", _i32, device)
    shape = table.shape
    if len(shape) != 2 or lens.shape != shape[:1]:
        raise ValueError("block_table: not [sequences, pages]")
    try:
        return (_pack_cache(shape[0], lens_ptr, table_ptr, shape[1], cache.page_size, cache.num_pages,
                            cache.max_seq_len),
                None if dims is None else
                _pack_dims(dims.n_q, dims.H_I, dims.D_I, dims.topk, dims.H, dims.R, dims.P,
                           dims.causal, dims.q_pos0, dims.scale),
                _arg(ws, "ws", _u8, device), ws.numel())
    except struct.error as e:
        raise ValueError(f"cache or dims: {e}") from None


def _on(stream, device):
    """The raw stream of a call: the given one, or the device's current one."""
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(device) or None
    return _dsa._stream(stream)


def _row_stride(t, seqs, need):
    """Elements between the rows of a [sequences, positions] tensor.  The library
    checks it against the `need` positions it may touch, so a tensor that is
    narrower than that states its width."""
    return t.stride(0) if seqs > 1 and t.shape[1] >= need else t.shape[1]


def _pool4(t, device, cache, dims):
    """A pool of 4-bit rows.  For an unsupported R or P any row width passes, so
    that the library's refusal is the one that is raised."""
    R, P = dims.R, dims.P
    W = R + P
    ok = 64 <= R <= 512 and R % 64 == 0 and P >= 0 and P % 16 == 0 and W <= 576
    width = (W // 2 + W // 16 + 16) // 16 * 16 if ok else t.shape[-1]
    return _arg(t, "latent4_pages", _u8, device, (cache.num_pages, cache.page_size, width))


def l4_row_bytes(R: int, P: int) -> int:
    """Bytes of one stored row of R + P columns."""
    n = int(l4_lib().dsa_l4_row_bytes(R, P))
    if n == 0:
        raise _dsa.DsaError(2, "dsa_l4_row_bytes")
    return n


def l4_workspace_bytes(op: int, dims, cache) -> int:
    return int(l4_lib().dsa_l4_workspace_bytes(
        op, ctypes.byref(dims.struct()) if dims is not None else None,
        ctypes.byref(cache.struct()) if cache is not None else None))


def l4_workspace(op: int, dims, cache, device="cuda", stream=None):
    """Allocate (with torch) and initialise a workspace for an L4_OP_* operation."""
    n = l4_workspace_bytes(op, dims, cache)
    if n == 0:
        raise _dsa.DsaError(1, "dsa_l4_workspace_bytes")
    ws = _torch.empty(n, dtype=_torch.uint8, device=device)
    _dsa._check(_dsa.lib().dsa_workspace_init(ws.data_ptr(), n, _dsa._stream(stream)),
                "dsa_workspace_init")
    return ws


def dsa_cache_append_l4(k_idx_new, latent_new, k_idx_pages, latent4_pages, cache, dims, ws,
                        stream=None) -> None:
    """Write the new tokens' index keys [n_q, D_I] (bf16) and latent rows
    [n_q, R + P] (bf16, quantised to 4 bits) into the page pools at the
    positions of the step's query rows."""
    L, dev = _ready or l4_lib(), _device()
    c, d, w, n = _common(cache, dims, ws, dev)
    status = L.dsa_cache_append_l4(
        _arg(k_idx_new, "k_idx_new", _bf16, dev, (dims.n_q, dims.D_I)),
        _arg(latent_new, "latent_new", _bf16, dev, (dims.n_q, dims.R + dims.P)),
        _arg(k_idx_pages, "k_idx_pages", _bf16, dev, (cache.num_pages, cache.page_size, dims.D_I)),
        _pool4(latent4_pages, dev, cache, dims), c, d, w, n, _on(stream, dev))
    if status:
        raise _dsa.DsaError(status, "dsa_cache_append_l4")


def dsa_cache_read_l4(latent4_pages, cache, idx, dims, rows, ws, stream=None) -> None:
    """The values of the stored rows at positions idx [n_q, topk], exactly, as
    bf16 rows [n_q, topk, R + P] (-1: a row of zeros)."""
    L, dev = _ready or l4_lib(), _device()
    c, d, w, n = _common(cache, dims, ws, dev)
    status = L.dsa_cache_read_l4(
        _pool4(latent4_pages, dev, cache, dims), c, _arg(idx, "idx", _i32, dev, (dims.n_q, dims.topk)),
        d, _arg(rows, "rows", _bf16, dev, (dims.n_q, dims.topk, dims.R + dims.P)), w, n,
        _on(stream, dev))
    if status:
        raise _dsa.DsaError(status, "dsa_cache_read_l4")


def _sparse_mla(where, q, latent4_pages, cache, idx, dims, out, lse, ws, stream):
    L, dev = _ready or l4_lib(), _device()
    c, d, w, n = _common(cache, dims, ws, dev)
    nq, H = dims.n_q, dims.H
    status = getattr(L, where)(
        _arg(q, "q", _bf16, dev, (nq, H, dims.R + dims.P)), _pool4(latent4_pages, dev, cache, dims), c,
        _arg(idx, "idx", _i32, dev, (nq, dims.topk)), d, _arg(out, "out", _f32, dev, (nq, H, dims.R)),
        _arg(lse, "lse", _f32, dev, (nq, H)), w, n, _on(stream, dev))
    if status:
        raise _dsa.DsaError(status, where)


def dsa_sparse_mla_decode_l4(q, latent4_pages, cache, idx, dims, out, lse, ws, stream=None) -> None:
    """Sparse MLA decode over a 4-bit latent cache."""
    _sparse_mla("dsa_sparse_mla_decode_l4", q, latent4_pages, cache, idx, dims, out, lse, ws, stream)


def dsa_sparse_mla_prefill_l4(q, latent4_pages, cache, idx, dims, out, lse, ws,
                              stream=None) -> None:
    """Sparse MLA of causal prefill rows over a 4-bit latent cache."""
    _sparse_mla("dsa_sparse_mla_prefill_l4", q, latent4_pages, cache, idx, dims, out, lse, ws, stream)


def dsa_attention_forward_l4(q_idx, w, k_idx_pages, q, latent4_pages, cache, dims, idx_out, out,
                             lse, ws, stream=None) -> None:
    """The whole step over bf16 index keys and a 4-bit latent cache (idx_out may be None)."""
    L, dev = _ready or l4_lib(), _device()
    c, d, wsp, n = _common(cache, dims, ws, dev)
    nq, H = dims.n_q, dims.H
    status = L.dsa_attention_forward_l4(
        _arg(q_idx, "q_idx", _bf16, dev, (nq, dims.H_I, dims.D_I)),
        _arg(w, "w", _f32, dev, (nq, dims.H_I)),
        _arg(k_idx_pages, "k_idx_pages", _bf16, dev, (cache.num_pages, cache.page_size, dims.D_I)),
        _arg(q, "q", _bf16, dev, (nq, H, dims.R + dims.P)), _pool4(latent4_pages, dev, cache, dims), c,
        d, _arg(idx_out, "idx_out", _i32, dev, (nq, dims.topk)),
        _arg(out, "out", _f32, dev, (nq, H, dims.R)), _arg(lse, "lse", _f32, dev, (nq, H)), wsp, n,
        _on(stream, dev))
    if status:
        raise _dsa.DsaError(status, "dsa_attention_forward_l4")


def _mass(where, q, latent, cache, idx, lse, dims, decay, mass_in, mass_out, ws, stream, dev):
    c, d, w, n = _common(cache, dims, ws, dev)
    seqs = cache.seq_lens.shape[0]
    if mass_out.dim() != 2 or mass_out.shape[0] != seqs:
        raise ValueError("mass_out: not [sequences, positions]")
    ld = _row_stride(mass_out, seqs, dims.q_pos0 + dims.n_q if dims.causal else cache.max_seq_len)
    if mass_in is not None and (mass_in.shape != mass_out.shape or
                                (seqs > 1 and mass_in.stride(0) != mass_out.stride(0))):
        raise ValueError("mass_in: not laid out as mass_out")
    status = getattr(_ready, where)(
        _arg(q, "q", _bf16, dev, (dims.n_q, dims.H, dims.R + dims.P)), *latent, c,
        _arg(idx, "idx", _i32, dev, (dims.n_q, dims.topk)),
        _arg(lse, "lse", _f32, dev, (dims.n_q, dims.H)), d, float(decay),
        _arg(mass_in, "mass_in", _f32, dev, rows=True),
        _arg(mass_out, "mass_out", _f32, dev, rows=True), ld, w, n, _on(stream, dev))
    if status:
        raise _dsa.DsaError(status, where)


def dsa_attention_mass(q, latent_pages, cache, idx, lse, dims, decay, mass_in, mass_out, ws,
                       stream=None) -> None:
    """Add the attention weight each kept token received to a running sum per
    token: mass_out = decay * mass_in + sum over heads of exp(z - lse), mass_*
    [sequences, positions] fp32 (mass_in None: zeros; mass_out may be mass_in).
    A token appended since has to hold 0 in mass_in: nothing else clears it."""
    _ready or l4_lib()
    dev = _device()
    lat = (_arg(latent_pages, "latent_pages", _bf16, dev,
                (cache.num_pages, cache.page_size, dims.R + dims.P)),)
    _mass("dsa_attention_mass", q, lat, cache, idx, lse, dims, decay, mass_in, mass_out, ws, stream, dev)


def dsa_attention_mass_l8(q, latent8_pages, latent_scale, cache, idx, lse, dims, decay, mass_in,
                          mass_out, ws, stream=None) -> None:
    """dsa_attention_mass over E4M3 latent rows with one fp32 scale per token."""
    _ready or l4_lib()
    dev = _device()
    lat = (_arg(latent8_pages, "latent8_pages", _u8, dev,
                (cache.num_pages, cache.page_size, dims.R + dims.P)),
           _arg(latent_scale, "latent_scale", _f32, dev, (cache.num_pages * cache.page_size,)))
    _mass("dsa_attention_mass_l8", q, lat, cache, idx, lse, dims, decay, mass_in, mass_out, ws, stream, dev)


def dsa_attention_mass_l4(q, latent4_pages, cache, idx, lse, dims, decay, mass_in, mass_out, ws,
                          stream=None) -> None:
    """dsa_attention_mass over a 4-bit latent cache."""
    _ready or l4_lib()
    dev = _device()
    _mass("dsa_attention_mass_l4", q, (_pool4(latent4_pages, dev, cache, dims),), cache, idx, lse,
          dims, decay, mass_in, mass_out, ws, stream, dev)


@dataclass
class Eviction:
    """Which tokens an eviction keeps: `budget` per sequence, the first `sinks`
    and the last `recent` among them whatever their mass."""
    budget: int
    sinks: int = 0
    recent: int = 0


def dsa_cache_evict(pools, cache, evict: Eviction, mass, dst_block_table, mass_dst, new_lens, kept,
                    ws, stream=None) -> None:
    """Keep min(budget, len) tokens of every sequence and compact their rows.

    pools: up to four (source, destination) pairs of page pools [pages, 64, ...]
    (any type; a per-token scale is a pool [pages, 64]); mass [sequences,
    positions] fp32; dst_block_table [sequences, pages] int32; mass_dst
    [sequences, positions] fp32 or None, left as it was past new_lens (zero an
    entry before the mass of a new token is added to it); new_lens [sequences]
    int32; kept [sequences, budget] int32 or None.
    """
    L, dev = _ready or l4_lib(), _device()
    c, _, w, n = _common(cache, None, ws, dev)
    seqs, size = cache.seq_lens.shape[0], cache.page_size
    if len(pools) > EVICT_MAX_POOLS:
        raise ValueError(f"pools: {len(pools)}, at most {EVICT_MAX_POOLS}")
    arr = (PoolStruct * max(1, len(pools)))()
    dst_pages = None
    for i, (src, dst) in enumerate(pools):
        sh, dh = src.shape, dst.shape
        if src.dtype is not dst.dtype or sh[1:] != dh[1:] or len(sh) < 2 or sh[0] != cache.num_pages \
                or sh[1] != size:
            raise ValueError(f"pools[{i}]: source {tuple(sh)} {src.dtype}, destination {tuple(dh)} {dst.dtype}")
        if dst_pages is not None and dst_pages != dh[0]:
            raise ValueError(f"pools[{i}]: destination pools of different sizes")
        dst_pages = dh[0]
        arr[i] = (_arg(src, "pool source", src.dtype, dev), _arg(dst, "pool destination", dst.dtype, dev),
                  src.element_size() * (src.numel() // (sh[0] * size)))
    if dst_block_table.dim() != 2 or dst_block_table.shape[0] != seqs:
        raise ValueError("dst_block_table: not [sequences, pages]")
    for name, t in (("mass", mass), ("mass_dst", mass_dst)):
        if t is not None and (t.dim() != 2 or t.shape[0] != seqs):
            raise ValueError(f"{name}: not [sequences, positions]")
    e = EvictStruct(evict.budget, evict.sinks, evict.recent,
                    _arg(dst_block_table, "dst_block_table", _i32, dev), dst_block_table.shape[1],
                    dst_pages if dst_pages is not None else 1 << 24)
    status = L.dsa_cache_evict(
        arr, len(pools), c, ctypes.byref(e), _arg(mass, "mass", _f32, dev, rows=True),
        _row_stride(mass, seqs, cache.max_seq_len), _arg(mass_dst, "mass_dst", _f32, dev, rows=True),
        0 if mass_dst is None else _row_stride(mass_dst, seqs, min(evict.budget, cache.max_seq_len)),
        _arg(new_lens, "new_lens", _i32, dev, (seqs,)), _arg(kept, "kept", _i32, dev, (seqs, evict.budget)),
        w, n, _on(stream, dev))
    if status:
        raise _dsa.DsaError(status, "dsa_cache_evict")
