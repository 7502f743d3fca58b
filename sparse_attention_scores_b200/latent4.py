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


_ready = _torch = None
_CacheStruct, _byref = _dsa.CacheStruct, ctypes.byref


def l4_lib() -> ctypes.CDLL:
    """The loaded library with the signatures of include/dsa_l4.h."""
    global _ready, _torch
    if _ready is None:
        import torch
        _torch = torch
        L = _dsa.lib()
        vp, sz, i32, i64, f32 = (ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64,
                                 ctypes.c_float)
        pc, pd = ctypes.POINTER(_dsa.CacheStruct), ctypes.POINTER(_dsa.DimsStruct)
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


_lib_of = l4_lib


def _types():
    """(bfloat16, float32, int32, uint8, the current device's index)"""
    if _ready is None:
        l4_lib()
    t = _torch
    return t.bfloat16, t.float32, t.int32, t.uint8, t.cuda.current_device()


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


def _pool(t, name, dtype, device, cache, width):
    """A page pool [num_pages, 64, width]."""
    return _arg(t, name, dtype, device, (cache.num_pages, cache.page_size, width))


def _common(cache, dims, ws, device, int32, uint8):
    """(cache struct, dims struct, workspace pointer, its size) of a call."""
    lens, table = cache.seq_lens, cache.block_table
    lens_ptr, table_ptr = _arg(lens, "seq_lens", int32, device), _arg(table, "block_table", int32, device)
    if table.dim() != 2 or lens.dim() != 1 or table.shape[0] != lens.shape[0]:
        raise ValueError("block_table: not [sequences, pages]")
    seqs, pages = table.shape
    return (_byref(_CacheStruct(seqs, lens_ptr, table_ptr, pages, cache.page_size, cache.num_pages,
                                cache.max_seq_len)),
            _byref(dims.struct()) if dims is not None else None, _arg(ws, "ws", uint8, device),
            ws.numel())


def _on(stream, device):
    """The raw stream of a call: the given one, or the device's current one."""
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(device) or None
    return _dsa._stream(stream)


def _row_bytes(dims, pool):
    """The stored row's width; for an unsupported R or P the pool's own, so that
    the library's refusal is the one that is raised."""
    return _lib_of().dsa_l4_row_bytes(dims.R, dims.P) or pool.shape[2]


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
    bf16, _, i32, u8, dev = _types()
    L = l4_lib()
    c, d, w, n = _common(cache, dims, ws, dev, i32, u8)
    row = _row_bytes(dims, latent4_pages)
    _dsa._check(L.dsa_cache_append_l4(
        _arg(k_idx_new, "k_idx_new", bf16, dev, (dims.n_q, dims.D_I)),
        _arg(latent_new, "latent_new", bf16, dev, (dims.n_q, dims.R + dims.P)),
        _pool(k_idx_pages, "k_idx_pages", bf16, dev, cache, dims.D_I),
        _pool(latent4_pages, "latent4_pages", u8, dev, cache, row),
        c, d, w, n, _on(stream, dev)), "dsa_cache_append_l4")


def dsa_cache_read_l4(latent4_pages, cache, idx, dims, rows, ws, stream=None) -> None:
    """The values of the stored rows at positions idx [n_q, topk], exactly, as
    bf16 rows [n_q, topk, R + P] (-1: a row of zeros)."""
    bf16, _, i32, u8, dev = _types()
    L = l4_lib()
    c, d, w, n = _common(cache, dims, ws, dev, i32, u8)
    row = _row_bytes(dims, latent4_pages)
    _dsa._check(L.dsa_cache_read_l4(
        _pool(latent4_pages, "latent4_pages", u8, dev, cache, row), c,
        _arg(idx, "idx", i32, dev, (dims.n_q, dims.topk)), d,
        _arg(rows, "rows", bf16, dev, (dims.n_q, dims.topk, dims.R + dims.P)),
        w, n, _on(stream, dev)), "dsa_cache_read_l4")


def _sparse_mla(fn, where, q, latent4_pages, cache, idx, dims, out, lse, ws, stream):
    bf16, f32, i32, u8, dev = _types()
    L = l4_lib()
    c, d, w, n = _common(cache, dims, ws, dev, i32, u8)
    row = _row_bytes(dims, latent4_pages)
    _dsa._check(fn(_arg(q, "q", bf16, dev, (dims.n_q, dims.H, dims.R + dims.P)),
                   _pool(latent4_pages, "latent4_pages", u8, dev, cache, row), c,
                   _arg(idx, "idx", i32, dev, (dims.n_q, dims.topk)), d,
                   _arg(out, "out", f32, dev, (dims.n_q, dims.H, dims.R)),
                   _arg(lse, "lse", f32, dev, (dims.n_q, dims.H)), w, n, _on(stream, dev)),
                where)


def dsa_sparse_mla_decode_l4(q, latent4_pages, cache, idx, dims, out, lse, ws, stream=None) -> None:
    """Sparse MLA decode over a 4-bit latent cache."""
    _sparse_mla(l4_lib().dsa_sparse_mla_decode_l4, "dsa_sparse_mla_decode_l4", q, latent4_pages,
                cache, idx, dims, out, lse, ws, stream)


def dsa_sparse_mla_prefill_l4(q, latent4_pages, cache, idx, dims, out, lse, ws,
                              stream=None) -> None:
    """Sparse MLA of causal prefill rows over a 4-bit latent cache."""
    _sparse_mla(l4_lib().dsa_sparse_mla_prefill_l4, "dsa_sparse_mla_prefill_l4", q, latent4_pages,
                cache, idx, dims, out, lse, ws, stream)


def dsa_attention_forward_l4(q_idx, w, k_idx_pages, q, latent4_pages, cache, dims, idx_out, out,
                             lse, ws, stream=None) -> None:
    """The whole step over bf16 index keys and a 4-bit latent cache (idx_out may be None)."""
    bf16, f32, i32, u8, dev = _types()
    L = l4_lib()
    c, d, wsp, n = _common(cache, dims, ws, dev, i32, u8)
    row = _row_bytes(dims, latent4_pages)
    _dsa._check(L.dsa_attention_forward_l4(
        _arg(q_idx, "q_idx", bf16, dev, (dims.n_q, dims.H_I, dims.D_I)),
        _arg(w, "w", f32, dev, (dims.n_q, dims.H_I)),
        _pool(k_idx_pages, "k_idx_pages", bf16, dev, cache, dims.D_I),
        _arg(q, "q", bf16, dev, (dims.n_q, dims.H, dims.R + dims.P)),
        _pool(latent4_pages, "latent4_pages", u8, dev, cache, row), c, d,
        _arg(idx_out, "idx_out", i32, dev, (dims.n_q, dims.topk)),
        _arg(out, "out", f32, dev, (dims.n_q, dims.H, dims.R)),
        _arg(lse, "lse", f32, dev, (dims.n_q, dims.H)), wsp, n, _on(stream, dev)),
        "dsa_attention_forward_l4")


def _mass(fn, where, q, latent, cache, idx, lse, dims, decay, mass_in, mass_out, ws, stream, types):
    bf16, f32, i32, u8, dev = types
    c, d, w, n = _common(cache, dims, ws, dev, i32, u8)
    seqs = int(cache.seq_lens.shape[0])
    ld = int(mass_out.stride(0)) if mass_out.dim() == 2 and seqs > 1 else int(mass_out.shape[-1])
    if mass_out.dim() != 2 or mass_out.shape[0] != seqs:
        raise ValueError("mass_out: not [sequences, positions]")
    if mass_in is not None and (mass_in.shape != mass_out.shape or
                                (seqs > 1 and mass_in.stride(0) != mass_out.stride(0))):
        raise ValueError("mass_in: not laid out as mass_out")
    _dsa._check(fn(_arg(q, "q", bf16, dev, (dims.n_q, dims.H, dims.R + dims.P)), *latent, c,
                   _arg(idx, "idx", i32, dev, (dims.n_q, dims.topk)),
                   _arg(lse, "lse", f32, dev, (dims.n_q, dims.H)), d, float(decay),
                   _arg(mass_in, "mass_in", f32, dev, rows=True),
                   _arg(mass_out, "mass_out", f32, dev, rows=True), ld, w, n,
                   _on(stream, dev)), where)


def dsa_attention_mass(q, latent_pages, cache, idx, lse, dims, decay, mass_in, mass_out, ws,
                       stream=None) -> None:
    """Add the attention weight each kept token received to a running sum per
    token: mass_out = decay * mass_in + sum over heads of exp(z - lse), mass_*
    [sequences, positions] fp32 (mass_in None: zeros; mass_out may be mass_in)."""
    t = _types()
    lat = (_pool(latent_pages, "latent_pages", t[0], t[4], cache, dims.R + dims.P),)
    _mass(l4_lib().dsa_attention_mass, "dsa_attention_mass", q, lat, cache, idx, lse, dims, decay,
          mass_in, mass_out, ws, stream, t)


def dsa_attention_mass_l8(q, latent8_pages, latent_scale, cache, idx, lse, dims, decay, mass_in,
                          mass_out, ws, stream=None) -> None:
    """dsa_attention_mass over E4M3 latent rows with one fp32 scale per token."""
    t = _types()
    lat = (_pool(latent8_pages, "latent8_pages", t[3], t[4], cache, dims.R + dims.P),
           _arg(latent_scale, "latent_scale", t[1], t[4], (cache.num_pages * cache.page_size,)))
    _mass(l4_lib().dsa_attention_mass_l8, "dsa_attention_mass_l8", q, lat, cache, idx, lse, dims,
          decay, mass_in, mass_out, ws, stream, t)


def dsa_attention_mass_l4(q, latent4_pages, cache, idx, lse, dims, decay, mass_in, mass_out, ws,
                          stream=None) -> None:
    """dsa_attention_mass over a 4-bit latent cache."""
    t = _types()
    row = _row_bytes(dims, latent4_pages)
    lat = (_pool(latent4_pages, "latent4_pages", t[3], t[4], cache, row),)
    _mass(l4_lib().dsa_attention_mass_l4, "dsa_attention_mass_l4", q, lat, cache, idx, lse, dims,
          decay, mass_in, mass_out, ws, stream, t)


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
    [sequences, positions] fp32 or None; new_lens [sequences] int32; kept
    [sequences, budget] int32 or None.
    """
    _, f32, i32, u8, dev = _types()
    L = l4_lib()
    c, _, w, n = _common(cache, None, ws, dev, i32, u8)
    seqs = int(cache.seq_lens.shape[0])
    if len(pools) > EVICT_MAX_POOLS:
        raise ValueError(f"pools: {len(pools)}, at most {EVICT_MAX_POOLS}")
    arr = (PoolStruct * max(1, len(pools)))()
    dst_pages = None
    for i, (src, dst) in enumerate(pools):
        if src.dtype is not dst.dtype or src.shape[1:] != dst.shape[1:] or \
                src.shape[0] != cache.num_pages or src.dim() < 2 or src.shape[1] != cache.page_size:
            raise ValueError(f"pools[{i}]: source {tuple(src.shape)} {src.dtype}, "
                             f"destination {tuple(dst.shape)} {dst.dtype}")
        if dst_pages not in (None, int(dst.shape[0])):
            raise ValueError(f"pools[{i}]: destination pools of different sizes")
        dst_pages = int(dst.shape[0])
        arr[i].src = _arg(src, f"pools[{i}] source", src.dtype, dev)
        arr[i].dst = _arg(dst, f"pools[{i}] destination", dst.dtype, dev)
        arr[i].row_bytes = src.element_size() * (src.numel() // (src.shape[0] * src.shape[1]))
    if dst_block_table.dim() != 2 or dst_block_table.shape[0] != seqs:
        raise ValueError("dst_block_table: not [sequences, pages]")
    for name, t in (("mass", mass), ("mass_dst", mass_dst)):
        if t is not None and (t.dim() != 2 or t.shape[0] != seqs):
            raise ValueError(f"{name}: not [sequences, positions]")
    ld = lambda t: int(t.stride(0)) if seqs > 1 else int(t.shape[1])  # noqa: E731
    e = EvictStruct(evict.budget, evict.sinks, evict.recent,
                    _arg(dst_block_table, "dst_block_table", i32, dev),
                    int(dst_block_table.shape[1]), dst_pages if dst_pages is not None else 1 << 24)
    _dsa._check(L.dsa_cache_evict(
        arr, len(pools), c, ctypes.byref(e), _arg(mass, "mass", f32, dev, rows=True), ld(mass),
        _arg(mass_dst, "mass_dst", f32, dev, rows=True), ld(mass_dst) if mass_dst is not None else 0,
        _arg(new_lens, "new_lens", i32, dev, (seqs,)),
        _arg(kept, "kept", i32, dev, (seqs, evict.budget)), w, n, _on(stream, dev)),
        "dsa_cache_evict")
