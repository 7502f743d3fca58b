"""include/dsa_l4.h without a GPU: exported symbols, sizes, refusals made on the
host, and the float64 definitions' own pins."""

import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

import sparse_attention_scores_b200 as dsa
from oracle import l4_oracle as l4
from sparse_attention_scores_b200 import build as dsa_build
from sparse_attention_scores_b200 import latent4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    dsa_build.build()
    return latent4.l4_lib()


def _dims(**kw):
    base = dict(n_q=2, H_I=32, D_I=128, topk=64, H=64, R=512, P=64, causal=0, q_pos0=0, scale=1.0)
    base.update(kw)
    return ctypes.byref(dsa.Dims(**base).struct())


def _cache(num_seqs=2, max_pages=4, num_pages=16, max_seq_len=256, page_size=64, lens=0x100000):
    # addresses that are never dereferenced: the host checks come first
    return ctypes.byref(dsa.CacheStruct(num_seqs, lens, 0x200000, max_pages, page_size, num_pages,
                                        max_seq_len))


A, WS = ctypes.c_void_p(0x300000), ctypes.c_void_p(0x400000)
MD = ctypes.c_void_p(0x380000)
OFF8, OFF2 = ctypes.c_void_p(0x300008), ctypes.c_void_p(0x300002)


def _host_only():
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake device addresses: host-only check")


def test_every_declared_symbol_is_exported(L):
    text = open(os.path.join(ROOT, "include", "dsa_l4.h")).read()
    declared = set(re.findall(r"^DSA_API[^(]*?\b(dsa_\w+)\s*\(", text, flags=re.M))
    assert declared == set(dsa.L4_EXPORTED)
    out = subprocess.run(["nm", "-D", "--defined-only", dsa.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    assert declared <= set(re.findall(r" T (dsa_\w+)$", out, flags=re.M))


def test_headers_compile_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "dsa_l4.h"\nint main(void) { return (int)DSA_L4_OP_STATUS; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I",
                    os.path.join(ROOT, "include"), str(src)], check=True)


def test_row_bytes(L):
    assert L.dsa_l4_row_bytes(512, 64) == 336 and L.dsa_l4_row_bytes(64, 16) == 48
    for R in range(64, 513, 64):
        for P in range(0, 577 - R, 16):
            n = L.dsa_l4_row_bytes(R, P)
            assert n == l4.row_bytes(R + P) and n % 16 == 0 and n > (R + P) // 2 + (R + P) // 16
    for R, P in ((0, 0), (32, 0), (100, 16), (576, 0), (512, 80), (512, 8), (64, -16)):
        assert L.dsa_l4_row_bytes(R, P) == 0


def test_workspace_bytes(L):
    d, c = _dims(), _cache()
    assert L.dsa_l4_workspace_bytes(dsa.L4_OP_STATUS, d, None) == 256
    mla = L.dsa_l4_workspace_bytes(dsa.L4_OP_SPARSE_MLA, d, None)
    fwd = L.dsa_l4_workspace_bytes(dsa.L4_OP_ATTENTION_FORWARD, d, c)
    assert mla >= 256 and fwd == mla + 2 * 256 * 4 + 2 * 64 * 4
    assert L.dsa_l4_workspace_bytes(dsa.L4_OP_ATTENTION_FORWARD, d, None) == 0
    assert L.dsa_l4_workspace_bytes(dsa.L4_OP_SPARSE_MLA, _dims(R=100), None) == 0
    assert L.dsa_l4_workspace_bytes(dsa.L4_OP_ATTENTION_MASS, _dims(), None) == 256
    assert L.dsa_l4_workspace_bytes(dsa.L4_OP_ATTENTION_MASS, _dims(causal=1, q_pos0=100), None) == 256 + 1024
    assert L.dsa_l4_workspace_bytes(dsa.L4_OP_CACHE_EVICT, None, c) == 256 + 256 + 2 * 2 * 256 * 4
    assert L.dsa_l4_workspace_bytes(dsa.L4_OP_CACHE_EVICT, None, None) == 0
    assert L.dsa_l4_workspace_bytes(9, d, c) == 0


def test_append_and_read_refuse(L):
    _host_only()
    ap = lambda k=A, x=A, kp=A, lp=A, c=None, d=None, ws=WS, n=256: L.dsa_cache_append_l4(  # noqa: E731
        k, x, kp, lp, c or _cache(), d or _dims(), ws, n, None)
    for bad in (dict(k=None), dict(x=None), dict(kp=None), dict(lp=None), dict(x=OFF8),
                dict(lp=OFF8), dict(c=_cache(num_seqs=3)), dict(c=_cache(lens=None)),
                dict(d=_dims(n_q=-1))):
        assert ap(**bad) == 1, bad
    for bad in (dict(d=_dims(D_I=48)), dict(d=_dims(P=8)), dict(d=_dims(R=100)),
                dict(c=_cache(page_size=32))):
        assert ap(**bad) == 2, bad
    assert ap(n=16) == 4 and ap(ws=OFF8) == 4 and ap(ws=None) == 4
    rd = lambda lp=A, i=A, o=A, c=None, d=None, n=256: L.dsa_cache_read_l4(  # noqa: E731
        lp, c or _cache(), i, d or _dims(), o, WS, n, None)
    for bad in (dict(lp=None), dict(i=None), dict(o=None), dict(o=OFF8), dict(i=OFF2),
                dict(d=_dims(topk=0))):
        assert rd(**bad) == 1, bad
    assert rd(d=_dims(R=96)) == 2 and rd(n=0) == 4


def test_attention_refuses(L):
    _host_only()
    for fn, causal in ((L.dsa_sparse_mla_decode_l4, 0), (L.dsa_sparse_mla_prefill_l4, 1)):
        call = lambda q=A, lp=A, i=A, o=A, l=A, c=None, n=1 << 30, **kw: fn(  # noqa: E731
            q, lp, c or _cache(), i, _dims(**dict(dict(causal=causal), **kw)), o, l, WS, n, None)
        for bad in (dict(q=None), dict(lp=None), dict(i=None), dict(o=None), dict(l=None),
                    dict(q=OFF8), dict(lp=OFF8), dict(i=OFF2), dict(causal=1 - causal),
                    dict(scale=float("nan"))):
            assert call(**bad) == 1, bad
        for bad in (dict(H=65), dict(H=0), dict(topk=0), dict(topk=65537), dict(R=80), dict(P=24)):
            assert call(**bad) == 2, bad
        assert call(n=100) == 4
    fw = lambda qi=A, w=A, k=A, q=A, lp=A, o=A, c=None, n=1 << 30, idx=None, **kw: (  # noqa: E731
        L.dsa_attention_forward_l4(qi, w, k, q, lp, c or _cache(), _dims(**kw), idx, o, A, WS, n, None))
    for bad in (dict(qi=None), dict(w=None), dict(k=None), dict(q=None), dict(lp=None), dict(o=None),
                dict(lp=OFF8), dict(k=OFF8), dict(idx=OFF2), dict(c=_cache(num_seqs=1))):
        assert fw(**bad) == 1, bad
    assert fw(H_I=65) == 2 and fw(D_I=16) == 2 and fw(n=2000) == 4


def test_mass_refuses(L):
    _host_only()
    mass = lambda q=A, lp=A, i=A, l=A, mi=A, mo=A, ld=256, decay=1.0, c=None, n=1 << 20, **kw: (  # noqa: E731
        L.dsa_attention_mass_l4(q, lp, c or _cache(), i, l, _dims(**kw), decay, mi, mo, ld, WS, n, None))
    for bad in (dict(q=None), dict(lp=None), dict(i=None), dict(l=None), dict(mo=None),
                dict(decay=-0.5), dict(decay=float("inf")), dict(decay=float("nan")), dict(ld=255),
                dict(ld=0), dict(mi=OFF2), dict(causal=1, q_pos0=100, ld=101)):
        assert mass(**bad) == 1, bad
    assert mass(H=65) == 2 and mass(n=255) == 4
    assert mass(causal=1, q_pos0=100, n=256 + 100) == 4  # no room for the chunk's sums
    assert L.dsa_attention_mass_l8(A, A, None, _cache(), A, A, _dims(), 1.0, A, A, 256, WS, 1 << 20, None) == 1
    assert L.dsa_attention_mass(A, None, _cache(), A, A, _dims(), 1.0, A, A, 256, WS, 1 << 20, None) == 1


def test_evict_refuses(L):
    _host_only()

    def call(pools=((0x300000, 0x500000, 336),), n=None, c=None, budget=128, sinks=0, recent=0,
             table=0x600000, mp=2, pages=8, mass=A, ld=256, md=MD, mld=128, lens=A, ws=1 << 20):
        arr = (latent4.PoolStruct * max(1, len(pools)))(*[latent4.PoolStruct(*p) for p in pools])
        e = latent4.EvictStruct(budget, sinks, recent, table, mp, pages)
        return L.dsa_cache_evict(arr, len(pools) if n is None else n, c or _cache(), ctypes.byref(e),
                                 mass, ld, md, mld, lens, None, WS, ws, None)

    for bad in (dict(mass=None), dict(lens=None), dict(budget=0), dict(sinks=-1), dict(recent=-1),
                dict(sinks=100, recent=29), dict(table=None), dict(mp=1), dict(pages=0), dict(ld=255),
                dict(mld=127), dict(md=A, mass=A), dict(n=5), dict(n=-1), dict(pools=((0, 0x500000, 336),)),
                dict(pools=((0x300000, 0x500000, 6),)), dict(pools=((0x300000, 0x500000, 0),)),
                dict(pools=((0x300008, 0x500000, 336),)), dict(pools=((0x300002, 0x500000, 4),)),
                dict(c=_cache(num_seqs=0)), dict(mass=OFF2)):
        assert call(**bad) == 1, bad
    assert call(pools=((0x300000, 0x500000, 8192),)) == 2
    assert call(c=_cache(num_seqs=70000)) == 2
    assert call(ws=1024) == 4


def test_block_tables_past_32_bit_positions_are_refused(L):
    _host_only()
    for pages, st in ((2 ** 25, 2), (2 ** 25 - 1, 4)):  # the second passes on to the workspace check
        c = _cache(max_pages=pages)
        d, p = _dims(), _dims(causal=1)
        assert L.dsa_cache_append_l4(A, A, A, A, c, d, WS, 16, None) == st
        assert L.dsa_cache_read_l4(A, c, A, d, A, WS, 16, None) == st
        assert L.dsa_sparse_mla_decode_l4(A, A, c, A, d, A, A, WS, 16, None) == st
        assert L.dsa_sparse_mla_prefill_l4(A, A, c, A, p, A, A, WS, 16, None) == st
        assert L.dsa_attention_forward_l4(A, A, A, A, A, c, d, A, A, A, WS, 16, None) == st
        assert L.dsa_attention_mass_l4(A, A, c, A, A, d, 1.0, A, A, 256, WS, 16, None) == st
        e = latent4.EvictStruct(128, 0, 0, 0x600000, 2, 8)
        assert L.dsa_cache_evict(None, 0, c, ctypes.byref(e), A, 256, MD, 128, A, None, WS, 16, None) == st


def test_binding_refuses_what_a_pointer_cannot_carry():
    """Strides, types and devices are checked before the library is called."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("CPU tensors stand in for a wrong device")
    t = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="runs on cuda"):
        latent4._arg(t, "t", torch.float32, 0)

    class Fake:  # a CUDA tensor's face
        device, dtype = torch.device("cuda", 0), torch.float32

        def get_device(self):
            return 0

        def __init__(self, t):
            self.t = t

        def __getattr__(self, name):
            return getattr(self.t, name)

    assert latent4._arg(Fake(t), "t", torch.float32, 0, (4, 8)) == t.data_ptr()
    for args, kw in (((Fake(t), "t", torch.bfloat16, 0), {}), ((Fake(t), "t", torch.float32, 1), {}),
                     ((Fake(t.T), "t", torch.float32, 0), {}),
                     ((Fake(t[:, :4]), "t", torch.float32, 0), {}),
                     ((Fake(t), "t", torch.float32, 0, (8, 4)), {}),
                     ((Fake(t.T), "t", torch.float32, 0), dict(rows=True))):
        with pytest.raises(ValueError):
            latent4._arg(*args, **kw)
    assert latent4._arg(Fake(t[:, :4]), "t", torch.float32, 0, rows=True) == t.data_ptr()
    assert latent4._arg(None, "t", torch.float32, 0) is None


# ------------------------------------------------- the definitions themselves
def test_every_code_and_scale_decodes_to_its_value():
    rows = np.zeros((16, 48), np.uint8)
    rows[:, :40] = (np.arange(16) * 17)[:, None]      # both nibbles the same code
    rows[:, 40:45] = 0x38                              # E4M3 1.0
    rows[:, 45] = 127 + 3
    v = l4.dequantise(rows, 80)
    want = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]) * 8
    assert np.array_equal(v, np.repeat(want[:, None], 80, 1))
    rows[:, :40] = 0x2                                 # value 1 in even columns, 0 in odd ones
    assert (l4.dequantise(rows, 80)[:, 0::2] == 8).all() and (l4.dequantise(rows, 80)[:, 1::2] == 0).all()


def test_quantise_is_exact_on_its_own_values_and_within_half_a_step():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 80)) * np.exp2(rng.uniform(-30, 30, (200, 1)))
    packed, v = l4.quantise(x)
    assert np.array_equal(l4.dequantise(packed, 80), v)
    e = packed[:, 45].astype(int) - 127
    amax = np.abs(x).max(1)
    assert (amax <= 2688.0 * 2.0 ** e).all() and (amax > 2688.0 * 2.0 ** (e - 1)).all()
    # a block's largest value is off by the scale's half step and the code's half step at most
    s = l4.E4M3[packed[:, 40:45]] * 2.0 ** e[:, None]
    err = np.abs(x - v).reshape(200, 5, 16)
    assert (err <= s[:, :, None] * (1.0 + 6.0 / 16) + 1e-300).all()
    # the values of a row whose blocks reach 6 in full scale store as themselves
    y = v.copy().reshape(200, 5, 16)
    y[:, :, 0] = 6 * s
    y[:, 0, 1] = 0
    packed2, v2 = l4.quantise(y.reshape(200, 80))
    keep = l4.row_exponent(np.abs(y).max((1, 2))) == e
    assert keep.any() and np.array_equal(v2[keep], y.reshape(200, 80)[keep])


def test_evict_keep_by_hand():
    m = np.array([0.0, 5.0, 1.0, 1.0, np.nan, 1.0, 0.0, 0.0], np.float32)
    assert l4.evict_keep(m, 4, 1, 1).tolist() == [0, 1, 2, 7]      # ties: the lower position
    assert l4.evict_keep(m, 7, 0, 0).tolist() == [0, 1, 2, 3, 5, 6, 7]  # NaN goes first
    assert l4.evict_keep(m, 100, 3, 3).tolist() == list(range(8))
    m[1] = np.inf
    assert l4.evict_keep(m, 2, 0, 2).tolist() == [6, 7]            # a protected token beats infinity


def test_masses_sum_to_heads():
    rng = np.random.default_rng(1)
    q, L = rng.standard_normal((3, 8)), rng.standard_normal((5, 8))
    _, lse, p = l4.attention(q, L, 4, 0.3)
    m = np.zeros(9)
    l4.add_mass(m, np.array([1, 3, 3, 5, 8]), q, L, lse, 0.3)
    assert np.isclose(m.sum(), 3) and np.isclose(m[3], p[:, 1:3].sum()) and (m[[0, 2, 4, 6, 7]] == 0).all()
