"""Workloads of the 4-bit latent cache and of cache eviction: the operators'
plain forms in elementary torch operations, and the framework's own calls.

A latent row of W = R + P columns is held in 4 bits per column:
    L[c] = 2^e * s[c // 16] * v[c]
with v an e2m1 value, s an e4m3 block scale and 2^e one power of two per token.
Row layout in bytes: W / 2 codes (even column in the low nibble), W / 16 block
scales, the exponent e + 127, zeros up to a multiple of 16.
"""

import math

import torch

own = False

PAGE = 64
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _case(name, op, **kw):
    base = dict(op=op, n=1, lo=1, hi=1, causal=False, pos0=0, heads=64, R=512, P=64, topk=2048,
                HI=32, DI=128, budget=0, sinks=0, recent=0, fmt="l4", shuffle=True)
    base.update(kw)
    return dict(name=name, **base) if name else base


def listed():
    return [
        # a decode step's new tokens of 32 sequences go into the cache: one row each, latency
        _case("append_decode_b32", "append", n=32, lo=100, hi=2048),
        # a long prompt's rows go into the cache in one call
        _case("append_prompt_16k", "append", n=16384, causal=True),
        # the smallest attention call: a few heads, a narrow row
        _case("mla_tiny_4k", "mla", lo=4096, hi=4096, heads=4, R=64, P=16, topk=256),
        # one user decoding at context 8,192
        _case("mla_decode_8k", "mla", lo=8192, hi=8192),
        # a serving batch of ragged contexts
        _case("mla_decode_b32_ragged", "mla", n=32, lo=2048, hi=65536),
        # a prompt chunk with causal selections, rows past 2,048 keep 2,048
        _case("mla_prefill_2300", "mla", n=2300, causal=True),
        # the whole step at long context: key scan, selection, attention
        _case("forward_4x128k", "forward", n=4, lo=131072, hi=131072),
        # one decode step of a batch as it is served: append, step, accumulated weight
        _case("step_b16", "step", n=16, lo=300, hi=16384),
        # the weight a decode step gave each kept token, added to the running sums
        _case("mass_decode_b32", "mass", n=32, lo=2048, hi=65536),
        # the last rows of a prompt over bf16 latent rows, 512 queries adding to the same tokens
        _case("mass_chunk_512_bf16", "mass", n=512, causal=True, pos0=3585, fmt="bf16"),
        # one sequence cut to half
        _case("evict_8k", "evict", lo=8191, hi=8191, budget=4096, sinks=4, recent=256),
        # long contexts cut to an eighth
        _case("evict_4x128k", "evict", n=4, lo=131072, hi=131072, budget=16384, sinks=64, recent=2048),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "mla", "mla", "forward", "step", "mass", "evict"])
    R, P = rng.choice([(512, 64), (512, 64), (512, 0), (448, 48), (256, 64), (192, 32), (64, 16)])
    heads = rng.choice([64, 64, 32, 16, rng.randint(1, 64)])
    if op == "append":
        causal = rng.random() < 0.5
        n = _log(rng, 1, 16384 if causal else 256)
        return _case(None, op, n=n, lo=1, hi=_log(rng, 64, 2048), causal=causal, R=R, P=P,
                     DI=rng.choice([32, 64, 128]), pos0=rng.randint(0, 1000) if causal else 0)
    if op == "evict":
        n = _log(rng, 1, 16)
        hi = _log(rng, 200, 32768)
        budget = _log(rng, 16, hi)
        recent = rng.randint(0, budget // 2)
        return _case(None, op, n=n, lo=rng.randint(1, hi), hi=hi, R=R, P=P, DI=rng.choice([32, 64, 128]),
                     budget=budget, recent=recent, sinks=rng.randint(0, budget // 4))
    causal = op in ("mla", "mass") and rng.random() < 0.3
    if causal:
        n, pos0 = _log(rng, 2, 700), rng.choice([0, rng.randint(1, 3000)])
        return _case(None, op, n=n, causal=True, pos0=pos0, heads=heads, R=R, P=P,
                     topk=_log(rng, 16, 2048), fmt=rng.choice(["l4", "l8", "bf16"]) if op == "mass" else "l4")
    n = _log(rng, 1, 64)
    hi = _log(rng, 64, 32768)
    return _case(None, op, n=n, lo=rng.randint(1, hi), hi=hi, heads=heads, R=R, P=P,
                 topk=_log(rng, 16, 4096 if op in ("mla", "mass") else 2048), HI=rng.choice([4, 16, 32]),
                 DI=rng.choice([32, 64, 128]), fmt=rng.choice(["l4", "l8", "bf16"]) if op == "mass" else "l4")


# --------------------------------------------------------------------------
# the row format
# --------------------------------------------------------------------------
def _row_bytes(W):
    return (W // 2 + W // 16 + 1 + 15) // 16 * 16


def _quantise(x):
    """x [n, W] -> (signed e2m1 values [n, W], codes [n, W], block scales [n, W / 16], exponents [n])."""
    x = x.float()
    n, W = x.shape
    amax = x.abs().amax(1)
    m, ex = torch.frexp(amax.double() / 2688.0)            # amax / 2688 = m 2^ex, m in [0.5, 1)
    e = torch.where(m == 0.5, ex - 1, ex).clamp(-60, 60)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    y = torch.ldexp(x, -e[:, None]).view(n, W // 16, 16)
    s = (y.abs().amax(2) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    a = torch.where(s[:, :, None] > 0, y.abs() / s[:, :, None], torch.zeros_like(y))
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    val = torch.tensor(E2M1, device=x.device)[code.long()]
    neg = (y < 0) & (s[:, :, None] > 0)
    return (torch.where(neg, -val, val).view(n, W), (code + 8 * neg).view(n, W).to(torch.uint8), s, e.int())


def _pack(x):
    """Rows x [n, W] as the cache holds them, [n, row bytes] uint8."""
    n, W = x.shape
    _, code, s, e = _quantise(x)
    row = torch.zeros(n, _row_bytes(W), dtype=torch.uint8, device=x.device)
    row[:, : W // 2] = code[:, 0::2] | (code[:, 1::2] << 4)
    row[:, W // 2 : W // 2 + W // 16] = s.to(torch.float8_e4m3fn).view(torch.uint8)
    row[:, W // 2 + W // 16] = (e + 127).to(torch.uint8)
    return row


def _unpack(row, W, dtype=torch.float32):
    """The values of packed rows [..., row bytes]."""
    b = row[..., : W // 2]
    code = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    v = torch.tensor(E2M1, device=row.device, dtype=dtype)[(code & 7).long()]
    v = torch.where(code >= 8, -v, v)
    s = row[..., W // 2 : W // 2 + W // 16].contiguous().view(torch.float8_e4m3fn).to(dtype)
    e = row[..., W // 2 + W // 16].to(torch.int32) - 127
    v = v.unflatten(-1, (W // 16, 16)) * s[..., None]
    return torch.ldexp(v.flatten(-2), e[..., None])


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _lens(c):
    """The sequences' lengths: a case's own, so that its sizes are the same for every seed."""
    if c["causal"]:
        return [c["pos0"] + c["n"]]
    g = torch.Generator().manual_seed(7 * c["n"] + 13 * c["lo"] + c["hi"])
    return [int(v) for v in torch.randint(c["lo"], c["hi"] + 1, (c["n"],), generator=g)]


def _select(lens, k, gen, causal, n, pos0):
    """[rows, k] ascending positions, -1 padded: what a top-k leaves of scattered scores."""
    dev = "cuda"
    if causal:
        lens = [pos0 + t + 1 for t in range(n)]
    out = torch.full((len(lens), k), -1, dtype=torch.int32, device=dev)
    longest = max(lens)
    step = max(1, (1 << 26) // longest)
    for r0 in range(0, len(lens), step):
        ln = torch.tensor(lens[r0 : r0 + step], device=dev)[:, None]
        score = torch.rand(len(ln), longest, device=dev, generator=gen)
        score = score.masked_fill(torch.arange(longest, device=dev)[None] >= ln, -1.0)
        m = min(k, longest)
        v, i = score.topk(m, dim=1)
        i = torch.where(v >= 0, i, longest).sort(1).values
        out[r0 : r0 + step, :m] = torch.where(i < longest, i, -1).int()
    return out


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    W, op = c["R"] + c["P"], c["op"]
    lens = _lens(c)
    npg = [(n + PAGE - 1) // PAGE for n in lens]
    total, maxp = sum(npg), max(npg)
    order = torch.randperm(total, device=dev, generator=gen) if c["shuffle"] else torch.arange(total, device=dev)
    table = torch.full((len(lens), maxp), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, k in enumerate(npg):
        table[b, :k] = order[at : at + k].int()
        at += k
    st = dict(case=c, W=W, lens=lens, seq_lens=torch.tensor(lens, dtype=torch.int32, device=dev), table=table,
              pages=total, scale=1.0 / math.sqrt(192.0 if W == 576 else W))

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=gen)

    # latent rows: a normalised part and a rotary part of about unit size
    fmt = c["fmt"]
    width = {"l4": _row_bytes(W), "l8": W, "bf16": W}[fmt]
    lat = torch.empty(total * PAGE, width, device=dev, dtype=torch.bfloat16 if fmt == "bf16" else torch.uint8)
    if fmt == "l8":
        st["lat_scale"] = torch.rand(total * PAGE, device=dev, generator=gen) * 0.02 + 0.005
    for r0 in range(0, total * PAGE, 1 << 16):
        r1 = min(total * PAGE, r0 + (1 << 16))
        x = normal(r1 - r0, W).bfloat16()
        if fmt == "l4":
            lat[r0:r1] = _pack(x)
        elif fmt == "l8":
            lat[r0:r1] = (x.float() / st["lat_scale"][r0:r1, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            lat[r0:r1] = x
    st["latent"] = lat.view(total, PAGE, width)
    if op in ("append", "forward", "step", "evict"):
        st["keys"] = torch.randint(-3, 4, (total, PAGE, c["DI"]), device=dev, generator=gen).bfloat16()
    n = c["n"]
    if op in ("append", "step"):
        st["k_new"] = torch.randint(-3, 4, (n, c["DI"]), device=dev, generator=gen).bfloat16()
        st["lat_new"] = (normal(n, W) * torch.exp(normal(n, 1))).bfloat16()
    if op == "append":
        pos = torch.tensor([c["pos0"] + t for t in range(n)] if c["causal"] else [v - 1 for v in lens], device=dev)
        st["pos"] = pos.int().view((1, n) if c["causal"] else (n, 1)).contiguous()
    if op in ("mla", "forward", "step", "mass"):
        st["q"] = normal(n, c["heads"], W).bfloat16()
    if op in ("forward", "step"):
        st["q_idx"] = torch.randint(-3, 4, (n, c["HI"], c["DI"]), device=dev, generator=gen).bfloat16()
        st["w"] = torch.randint(0, 4, (n, c["HI"]), device=dev, generator=gen).float()
    if op in ("mla", "mass"):
        st["idx"] = _select(lens, c["topk"], gen, c["causal"], n, c["pos0"])
    if op in ("mass", "step"):
        # sums of earlier steps: many tokens were never selected
        ld = (max(lens) + 3) // 4 * 4
        u = torch.rand(len(lens), ld, device=dev, generator=gen)
        st["mass_in"] = torch.where(u < 0.5, torch.zeros_like(u), torch.exp(8 * u - 6))
        st["mass_out"] = torch.zeros_like(st["mass_in"])
        st["decay"] = 0.984375
    if op == "mass":
        st["lse"] = _attend(st, st["idx"], torch.float64, want_out=False)[1].float()
    if op == "evict":
        ld = (max(lens) + 3) // 4 * 4
        u = torch.rand(len(lens), ld, device=dev, generator=gen)
        st["mass"] = torch.where(u < 0.6, torch.zeros_like(u), torch.exp(10 * u - 8))
        keep = min(c["budget"], max(lens))
        dpg = (keep + PAGE - 1) // PAGE
        dtotal = dpg * len(lens)
        st["dst_table"] = torch.randperm(dtotal, device=dev, generator=gen).int().view(len(lens), dpg).contiguous()
        st["dst_latent"] = torch.zeros(dtotal, PAGE, width, device=dev, dtype=torch.uint8)
        st["dst_keys"] = torch.zeros(dtotal, PAGE, c["DI"], device=dev, dtype=torch.bfloat16)
        st["dst_mass"] = torch.zeros(len(lens), (keep + 3) // 4 * 4, device=dev)
        st["new_lens"] = torch.zeros(len(lens), dtype=torch.int32, device=dev)
        st["kept"] = torch.zeros(len(lens), c["budget"], dtype=torch.int32, device=dev)
    return st


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _rows_of(st, seq, pos):
    """Physical rows of positions pos of sequences seq (tensors of one shape)."""
    return st["table"][seq, pos // PAGE].long() * PAGE + pos % PAGE


def _latents(st, rows, dtype):
    c, W = st["case"], st["W"]
    got = st["latent"].view(-1, st["latent"].shape[2])[rows]
    if c["fmt"] == "l4":
        return _unpack(got, W, dtype)
    if c["fmt"] == "l8":
        return got.view(torch.float8_e4m3fn).to(dtype) * st["lat_scale"][rows].to(dtype)[..., None]
    return got.to(dtype)


def _logits(st, idx, r0, r1, dtype):
    """(z [rows, H, k], L [rows, k, W]) of query rows r0 .. r1 over their selections; -inf at unused slots."""
    c = st["case"]
    sel = idx[r0:r1].long()
    seq = torch.zeros_like(sel) if c["causal"] else torch.arange(r0, r1, device=sel.device)[:, None].expand_as(sel)
    L = _latents(st, _rows_of(st, seq, sel.clamp(min=0)), dtype)
    z = torch.matmul(st["q"][r0:r1].to(dtype), L.transpose(1, 2)) * st["scale"]
    return z.masked_fill((sel < 0)[:, None, :], -math.inf), L


def _row_step(st, idx, dtype):
    return max(1, (1 << (31 if dtype == torch.float32 else 30)) // (idx.shape[1] * st["W"] * 4))


def _attend(st, idx, dtype, want_out=True):
    c = st["case"]
    n, step = idx.shape[0], _row_step(st, idx, dtype)
    outs, lses = [], []
    for r0 in range(0, n, step):
        z, L = _logits(st, idx, r0, min(n, r0 + step), dtype)
        m = z.amax(2, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        p = torch.exp(z - m)
        l = p.sum(2, keepdim=True)
        if want_out:
            outs.append(torch.matmul(p, L[..., : c["R"]]) / torch.where(l == 0, torch.ones_like(l), l))
        lses.append((m + torch.log(l))[..., 0])
    return (torch.cat(outs) if want_out else None), torch.cat(lses)


def _mass(st, idx, lse, dtype):
    c = st["case"]
    n, step = idx.shape[0], _row_step(st, idx, dtype)
    add = torch.zeros_like(st["mass_in"], dtype=torch.float64)
    for r0 in range(0, n, step):
        r1 = min(n, r0 + step)
        z, _ = _logits(st, idx, r0, r1, dtype)
        ref = lse[r0:r1].to(dtype)[..., None]
        w = torch.exp(z - torch.where(ref == -math.inf, torch.zeros_like(ref), ref)).sum(1)
        sel = idx[r0:r1].long()
        seq = torch.zeros_like(sel) if c["causal"] else torch.arange(r0, r1, device=sel.device)[:, None].expand_as(sel)
        add.index_put_((seq, sel.clamp(min=0)), torch.where(sel < 0, torch.zeros_like(w), w).double(), accumulate=True)
    lens = torch.tensor(st["lens"], device=add.device)[:, None]
    live = torch.arange(add.shape[1], device=add.device)[None] < lens
    return torch.where(live, st["decay"] * st["mass_in"].double() + add, st["mass_out"].double()).to(dtype)


def _append(st):
    """Writes the new rows into the pools; the rows' physical places."""
    c = st["case"]
    if c["causal"]:
        pos = torch.arange(c["pos0"], c["pos0"] + c["n"], device="cuda")
        rows = _rows_of(st, torch.zeros_like(pos), pos)
    else:
        rows = _rows_of(st, torch.arange(c["n"], device="cuda"), st["seq_lens"].long() - 1)
    st["keys"].view(-1, c["DI"])[rows] = st["k_new"]
    st["latent"].view(-1, st["latent"].shape[2])[rows] = _pack(st["lat_new"])
    return rows


def _scores(st, b, dtype):
    """Index scores of every token of sequence b."""
    pos = torch.arange(st["lens"][b], device="cuda")
    k = st["keys"].view(-1, st["case"]["DI"])[_rows_of(st, torch.full_like(pos, b), pos)].to(dtype)
    s = torch.matmul(st["q_idx"][b].to(dtype), k.T).clamp(min=0)
    return (s * st["w"][b].to(dtype)[:, None]).sum(0)


def _topk(score, k):
    """Positions of the k best, lower position first among equals, ascending, -1 padded."""
    best = torch.sort(score, descending=True, stable=True).indices[:k].sort().values
    return torch.cat([best, best.new_full((k - best.numel(),), -1)]).int()


def _evict_idx(st, b):
    c, n = st["case"], st["lens"][b]
    m = st["mass"][b, :n].clone()
    m[: c["sinks"]] = math.inf
    m[max(0, n - c["recent"]) :] = math.inf
    return _topk(m, c["budget"])


def _plain(st):
    c, op, W = st["case"], st["case"]["op"], st["W"]
    if op == "append":
        rows = _append(st)
        back = _unpack(st["latent"].view(-1, st["latent"].shape[2])[rows], W).bfloat16()
        return {"keys": st["keys"], "rows": back.view(*st["pos"].shape, W)}
    if op == "mla":
        out, lse = _attend(st, st["idx"], torch.float32)
        return {"out": out, "lse": lse}
    if op in ("forward", "step"):
        if op == "step":
            _append(st)
        idx = torch.stack([_topk(_scores(st, b, torch.float32), c["topk"]) for b in range(c["n"])])
        out, lse = _attend(st, idx, torch.float32)
        got = {"idx": idx, "out": out, "lse": lse}
        if op == "step":
            st["mass_out"].copy_(_mass(st, idx, lse, torch.float32))
            got["mass"] = st["mass_out"]
        return got
    if op == "mass":
        st["mass_out"].copy_(_mass(st, st["idx"], st["lse"], torch.float32))
        return {"mass": st["mass_out"]}
    for b, n in enumerate(st["lens"]):
        kept = _evict_idx(st, b)
        st["kept"][b] = kept
        new = min(n, c["budget"])
        st["new_lens"][b] = new
        src = kept[:new].long()
        pos = torch.arange(new, device="cuda")
        rows = _rows_of(st, torch.full_like(src, b), src)
        dst = st["dst_table"][b, pos // PAGE].long() * PAGE + pos % PAGE
        for s, d in (("latent", "dst_latent"), ("keys", "dst_keys")):
            st[d].view(-1, st[d].shape[2])[dst] = st[s].view(-1, st[s].shape[2])[rows]
        st["dst_mass"][b, :new] = st["mass"][b][src]
    return {k: st[k] for k in ("kept", "new_lens", "dst_latent", "dst_keys", "dst_mass")}


# --------------------------------------------------------------------------
# the framework's calls
# --------------------------------------------------------------------------
def _own(st):
    import sparse_attention_scores_b200 as dsa
    c, op, W = st["case"], st["case"]["op"], st["W"]
    n, H, R = c["n"], c["heads"], c["R"]
    if "ws" not in st:  # a user's program keeps the plan, the workspaces and the result buffers
        st["cache"] = dsa.PagedCache(st["seq_lens"], st["table"], num_pages=st["pages"], max_seq_len=max(st["lens"]))
        st["dims"] = dsa.Dims(n_q=n, H_I=c["HI"], D_I=c["DI"], topk=c["topk"], H=H, R=R, P=c["P"],
                              causal=int(c["causal"]), q_pos0=c["pos0"], scale=st["scale"])
        which = {"append": dsa.L4_OP_STATUS, "mla": dsa.L4_OP_SPARSE_MLA, "forward": dsa.L4_OP_ATTENTION_FORWARD,
                 "step": dsa.L4_OP_ATTENTION_FORWARD, "mass": dsa.L4_OP_ATTENTION_MASS, "evict": dsa.L4_OP_CACHE_EVICT}[op]
        if op == "append":
            k = st["pos"].shape[1]
            st["read_dims"] = dsa.Dims(n_q=st["pos"].shape[0], H_I=1, D_I=32, topk=k, H=1, R=R, P=c["P"])
            st["rows"] = torch.empty(*st["pos"].shape, W, dtype=torch.bfloat16, device="cuda")
        if op in ("mla", "forward", "step"):
            st["out"] = torch.empty(n, H, R, device="cuda")
            st["lse_out"] = torch.empty(n, H, device="cuda")
        if op in ("forward", "step"):
            st["idx_out"] = torch.empty(n, c["topk"], dtype=torch.int32, device="cuda")
        if op == "evict":
            st["evict"] = dsa.Eviction(c["budget"], c["sinks"], c["recent"])
            st["pools"] = [(st["latent"], st["dst_latent"]), (st["keys"], st["dst_keys"])]
        if op == "step":
            st["mass_ws"] = dsa.l4_workspace(dsa.L4_OP_ATTENTION_MASS, st["dims"], st["cache"])
        st["ws"] = dsa.l4_workspace(which, st["dims"], st["cache"])
    cache, dims, ws = st["cache"], st["dims"], st["ws"]
    if op in ("append", "step"):
        dsa.dsa_cache_append_l4(st["k_new"], st["lat_new"], st["keys"], st["latent"], cache, dims, ws)
    if op == "append":
        dsa.dsa_cache_read_l4(st["latent"], cache, st["pos"], st["read_dims"], st["rows"], ws)
        return {"keys": st["keys"], "rows": st["rows"]}
    if op == "mla":
        call = dsa.dsa_sparse_mla_prefill_l4 if c["causal"] else dsa.dsa_sparse_mla_decode_l4
        call(st["q"], st["latent"], cache, st["idx"], dims, st["out"], st["lse_out"], ws)
        return {"out": st["out"], "lse": st["lse_out"]}
    if op in ("forward", "step"):
        dsa.dsa_attention_forward_l4(st["q_idx"], st["w"], st["keys"], st["q"], st["latent"], cache, dims,
                                     st["idx_out"], st["out"], st["lse_out"], ws)
        got = {"idx": st["idx_out"], "out": st["out"], "lse": st["lse_out"]}
        if op == "step":
            dsa.dsa_attention_mass_l4(st["q"], st["latent"], cache, st["idx_out"], st["lse_out"], dims, st["decay"],
                                      st["mass_in"], st["mass_out"], st["mass_ws"])
            got["mass"] = st["mass_out"]
        return got
    if op == "mass":
        rest = (cache, st["idx"], st["lse"], dims, st["decay"], st["mass_in"], st["mass_out"], ws)
        if c["fmt"] == "l4":
            dsa.dsa_attention_mass_l4(st["q"], st["latent"], *rest)
        elif c["fmt"] == "l8":
            dsa.dsa_attention_mass_l8(st["q"], st["latent"], st["lat_scale"], *rest)
        else:
            dsa.dsa_attention_mass(st["q"], st["latent"], *rest)
        return {"mass": st["mass_out"]}
    dsa.dsa_cache_evict(st["pools"], cache, st["evict"], st["mass"], st["dst_table"], st["dst_mass"], st["new_lens"],
                        st["kept"], ws)
    return {k: st[k] for k in ("kept", "new_lens", "dst_latent", "dst_keys", "dst_mass")}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    c = case
    W, H, R, n = c["R"] + c["P"], c["heads"], c["R"], c["n"]
    row = {"l4": W // 2 + W // 16 + 1, "l8": W + 4, "bf16": 2 * W}[c["fmt"]]
    # contexts: the mean of the drawn range
    length = (c["lo"] + c["hi"]) / 2
    if c["causal"]:
        kept = sum(min(c["topk"], c["pos0"] + t + 1) for t in range(n))
        distinct = c["pos0"] + n
        tokens = distinct
    else:
        kept = distinct = n * min(c["topk"], length)
        tokens = n * length
    bytes_, flops = 0.0, 0.0
    if c["op"] in ("append", "step"):
        bytes_ += n * (2 * W + row + 4 * c["DI"])
        flops += 4.0 * n * W
    if c["op"] == "append":
        bytes_ += n * (row + 2 * W)
    if c["op"] in ("mla", "forward", "step"):
        bytes_ += distinct * row + 4 * kept + n * H * (2 * W + 4 * R + 4)
        flops += 2.0 * kept * H * (W + R)
    if c["op"] in ("forward", "step"):
        bytes_ += tokens * 2 * c["DI"] + n * c["HI"] * (2 * c["DI"] + 4)
        flops += 2.0 * tokens * c["HI"] * c["DI"]
    if c["op"] in ("mass", "step"):
        again = 0 if c["op"] == "step" else 1
        bytes_ += again * (distinct * row + 4 * kept + n * H * (2 * W + 4)) + 8 * tokens
        flops += again * 2.0 * kept * H * W
    if c["op"] == "evict":
        left = n * min(c["budget"], length)
        bytes_ += 4 * tokens + left * (2 * (row + 2 * c["DI"] + 4) + 4)
        flops += 1.0 * tokens
    return {"bytes": float(bytes_), "flops": float(flops)}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _exact_code_rows(raw, W):
    """Packed rows -> float64 values, one column at a time from the format's definition."""
    n = raw.shape[0]
    v = torch.zeros(n, W, dtype=torch.float64, device=raw.device)
    nib = torch.zeros(n, W, dtype=torch.int64, device=raw.device)
    nib[:, 0::2] = raw[:, : W // 2].long() % 16
    nib[:, 1::2] = raw[:, : W // 2].long() // 16
    mag = nib % 8
    exp, man = mag // 2, mag % 2
    v = torch.where(exp == 0, man * 0.5, (1 + 0.5 * man) * torch.pow(2.0, (exp - 1).double()))
    v = torch.where(nib >= 8, -v, v)
    sb = raw[:, W // 2 : W // 2 + W // 16].long()
    se, sm = (sb // 8) % 16, sb % 8
    s = torch.where(se == 0, sm * 2.0 ** -9, (1 + sm / 8.0) * torch.pow(2.0, (se - 7).double()))
    t = torch.pow(2.0, (raw[:, W // 2 + W // 16].long() - 127).double())
    return v * s.repeat_interleave(16, 1) * t[:, None]


def _exact_latents(st, rows):
    raw = st["latent"].view(-1, st["latent"].shape[2])[rows]
    if st["case"]["fmt"] == "l4":
        return _exact_code_rows(raw, st["W"])
    if st["case"]["fmt"] == "l8":
        return raw.view(torch.float8_e4m3fn).double() * st["lat_scale"][rows].double()[:, None]
    return raw.double()


def _exact_round(x, grid):
    """The nearest of the ascending grid's values to |x| (ties to the entry of even number), saturating."""
    g = torch.tensor(grid, dtype=torch.float64, device=x.device)
    a = x.abs().clamp(max=g[-1])
    hi = torch.searchsorted(g, a.contiguous()).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = g[hi] - a, a - g[lo]
    i = torch.where(up < down, hi, torch.where(down < up, lo, torch.where(hi % 2 == 0, hi, lo)))
    return g[i]


def _exact_rows(x):
    """bf16 rows -> the values the cache stands for."""
    x = x.double()
    top = x.abs().amax(1)
    bounds = 2688.0 * torch.pow(2.0, torch.arange(-60, 60, device=x.device).double())
    e = -60.0 + (top[:, None] > bounds).sum(1)
    e = torch.where(top == 0, torch.zeros_like(e), e)
    y = (x / torch.pow(2.0, e)[:, None]).view(x.shape[0], -1, 16)
    grid8 = [m * 2.0 ** -9 for m in range(8)] + [(1 + m / 8.0) * 2.0 ** (k - 7) for k in range(1, 16) for m in range(8)]
    s = _exact_round(y.abs().amax(2) / 6.0, grid8[:-1])
    v = _exact_round(y / torch.where(s == 0, torch.ones_like(s), s)[..., None], list(E2M1))
    v = torch.where(s[..., None] == 0, torch.zeros_like(v), torch.copysign(v, y))
    return (v * s[..., None]).view(x.shape) * torch.pow(2.0, e)[:, None]


def _exact_row(st, r, sel):
    """(z [H, m], L [m, W]) of query row r over the positions sel."""
    b = 0 if st["case"]["causal"] else r
    rows = st["table"][b].long()[sel // PAGE] * PAGE + sel % PAGE
    L = _exact_latents(st, rows)
    return st["q"][r].double() @ L.T * st["scale"], L


def exact(case, seed):
    c, st = case, prepare(case, seed)
    op, W, n, H, R = c["op"], st["W"], c["n"], c["heads"], c["R"]
    if op == "evict":
        return None  # whole numbers and copies
    if op == "append":
        return {"keys": None, "rows": _exact_rows(st["lat_new"]).view(*st["pos"].shape, W)}
    mass = st["mass_in"].double().clone() if "mass_in" in st else None
    if mass is not None:
        for b, ln in enumerate(st["lens"]):
            mass[b, :ln] *= st["decay"]
            mass[b, ln:] = 0.0
    if op == "step":
        for b in range(n):
            p = st["lens"][b] - 1
            at = int(st["table"][b, p // PAGE]) * PAGE + p % PAGE
            st["keys"].view(-1, c["DI"])[at] = st["k_new"][b]
    out = torch.zeros(n, H, R, dtype=torch.float64, device="cuda")
    lse = torch.full((n, H), -math.inf, dtype=torch.float64, device="cuda")
    for r in range(n):
        if op in ("forward", "step"):
            pos = torch.arange(st["lens"][r], device="cuda")
            k = st["keys"].view(-1, c["DI"])[st["table"][r].long()[pos // PAGE] * PAGE + pos % PAGE].double()
            score = torch.relu(st["q_idx"][r].double() @ k.T).mul(st["w"][r].double()[:, None]).sum(0)
            sel = torch.argsort(-score, stable=True)[: c["topk"]].sort().values
        else:
            sel = st["idx"][r].long()
            sel = sel[sel >= 0]
        if sel.numel() == 0:
            continue
        z, L = _exact_row(st, r, sel)
        if op == "step":  # the newest token's row is the one just written
            here = sel == st["lens"][r] - 1
            L = torch.where(here[:, None], _exact_rows(st["lat_new"][r : r + 1]), L)
            z = st["q"][r].double() @ L.T * st["scale"]
        if op == "mass":
            mass[0 if c["causal"] else r].index_add_(0, sel, torch.exp(z - st["lse"][r].double()[:, None]).sum(0))
            continue
        lse[r] = torch.logsumexp(z, 1)
        p = torch.exp(z - lse[r][:, None])
        out[r] = p @ L[:, :R]
        if op == "step":
            mass[r].index_add_(0, sel, p.sum(0))
    if op == "mass":
        return {"mass": mass}
    got = {"out": out, "lse": lse}
    if op != "mla":
        got["idx"] = None
    if op == "step":
        got["mass"] = mass
    return got
