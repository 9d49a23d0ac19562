"""Workloads of the sliding-window attention and of the paged 8-bit KV cache.

Every case names one operator (``op``) and its sizes; ``run`` makes one pass
through it, either as plain torch operations in fp32 (``own`` false) or with
the library's calls (``own`` true).

  window_fwd   sliding-window attention with sinks, forward: out and LSE
  window_train the same, forward and backward: out, dq, dk, dv
  kv8_attn     attention over the paged 8-bit cache (newest Nq positions)
  kv8_append   quantises new keys and values into the paged cache
  pages_fork   beams / n-best: slots become children of others, tails copied
  pages_compact live pages moved to the front of the pool
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # Prefill of one prompt through a grouped-query model whose layers keep a 4K window and the
        # first four tokens (the 14:2 heads of the GQA prefill workload).
        {"name": "window_prefill_gqa", "op": "window_fwd", "B": 1, "Hq": 14, "Hkv": 2, "Nq": 16384,
         "Nk": 16384, "D": 64, "W": 4096, "S": 4, "dtype": "fp16"},
        # Evaluation forward at the training shape, window of 1K, no sinks.
        {"name": "window_forward_mha", "op": "window_fwd", "B": 2, "Hq": 16, "Hkv": 16, "Nq": 8192,
         "Nk": 8192, "D": 128, "W": 1024, "S": 0, "dtype": "bf16"},
        # One ragged chunk of a chunked prefill against a dense cache of odd length.
        {"name": "window_chunk", "op": "window_fwd", "B": 1, "Hq": 16, "Hkv": 4, "Nq": 501, "Nk": 20011,
         "D": 128, "W": 2000, "S": 17, "dtype": "bf16"},
        # A training step of the attention at the training shape.
        {"name": "window_train_mha", "op": "window_train", "B": 2, "Hq": 16, "Hkv": 16, "Nq": 8192,
         "Nk": 8192, "D": 128, "W": 1024, "S": 4, "dtype": "bf16"},
        # A training step with grouped heads and an odd length.
        {"name": "window_train_gqa", "op": "window_train", "B": 1, "Hq": 14, "Hkv": 2, "Nq": 4099, "Nk": 4099,
         "D": 64, "W": 1000, "S": 3, "dtype": "fp16"},
        # Decode of eight long conversations (the decode workload's 64K), one token each.
        {"name": "kv8_decode_long", "op": "kv8_attn", "B": 8, "Hq": 14, "Hkv": 2, "Nq": 1, "D": 64, "P": 64,
         "min_len": 65000, "max_len": 65536, "W": 0, "S": 0, "dtype": "fp16"},
        # A serving batch of very different lengths.
        {"name": "kv8_decode_mixed", "op": "kv8_attn", "B": 32, "Hq": 32, "Hkv": 8, "Nq": 1, "D": 128, "P": 64,
         "min_len": 200, "max_len": 32768, "W": 0, "S": 0, "dtype": "bf16"},
        # Four drafted tokens of one user in a windowed layer, small pages: latency counts.
        {"name": "kv8_decode_small", "op": "kv8_attn", "B": 1, "Hq": 14, "Hkv": 2, "Nq": 4, "D": 64, "P": 16,
         "min_len": 1500, "max_len": 1500, "W": 512, "S": 4, "dtype": "fp16"},
        # A prompt's keys and values of one layer go into the cache.
        {"name": "kv8_append_prompt", "op": "kv8_append", "B": 2, "Hkv": 8, "T": 8190, "D": 128, "P": 64,
         "min_old": 0, "max_old": 100, "dtype": "bf16"},
        # One decoding step of a batch of 64.
        {"name": "kv8_append_step", "op": "kv8_append", "B": 64, "Hkv": 8, "T": 1, "D": 128, "P": 64,
         "min_old": 1, "max_old": 4000, "dtype": "bf16"},
        # A quarter of the slots survive, the others become their children, over eight layers.
        {"name": "pages_fork_beams", "op": "pages_fork", "n": 64, "L": 8, "Hkv": 2, "D": 128, "P": 64,
         "max_pages": 32, "keep": 16},
        # The pool of a finished batch is compacted: two pages in three are free.
        {"name": "pages_compact", "op": "pages_compact", "n": 48, "L": 4, "Hkv": 4, "D": 128, "P": 64,
         "max_pages": 48, "live": 0.33},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["window_fwd", "window_train", "kv8_attn", "kv8_attn", "kv8_append", "pages_fork",
                         "pages_compact"])
        dt = rng.choice(["fp16", "bf16"])
        D = rng.choice([64, 128])
        if op in ("window_fwd", "window_train"):
            G = rng.choice([1, 2, 4, 7, 8])
            Hkv = rng.choice([1, 2, 4, 8])
            nq = _log(rng, 64, 8192)
            nk = nq + (rng.choice([0, _log(rng, 1, 8192)]) if op == "window_fwd" else 0)
            c = {"op": op, "B": rng.choice([1, 2, 3]), "Hq": G * Hkv, "Hkv": Hkv, "Nq": nq, "Nk": nk, "D": D,
                 "W": _log(rng, 16, 4096), "S": rng.choice([0, 1, 4, 130]), "dtype": dt}
            if c["B"] * c["Hq"] * nk > 32 * 8192:
                continue
        elif op == "kv8_attn":
            G = rng.choice([1, 2, 4, 7, 8])
            Hkv = rng.choice([1, 2, 4, 8])
            m = _log(rng, 30, 40000)
            c = {"op": op, "B": _log(rng, 1, 40), "Hq": G * Hkv, "Hkv": Hkv, "Nq": rng.choice([1, 1, 2, 5]),
                 "D": D, "P": rng.choice([16, 32, 64, 128]), "min_len": rng.randint(8, m), "max_len": m,
                 "W": rng.choice([0, 0, _log(rng, 16, 4096)]), "S": rng.choice([0, 4, 70]), "dtype": dt}
            if c["B"] * c["Hkv"] * m * D > 32 * 8 * 16384 * 128:
                continue
        elif op == "kv8_append":
            c = {"op": op, "B": _log(rng, 1, 100), "Hkv": rng.choice([1, 2, 4, 8]),
                 "T": rng.choice([1, 3, _log(rng, 10, 10000)]), "D": D, "P": rng.choice([16, 32, 64, 128]),
                 "min_old": 0, "max_old": _log(rng, 1, 4000), "dtype": dt}
            if c["B"] * (c["T"] + c["max_old"]) * c["Hkv"] * D > 64 * 4000 * 8 * 128:
                continue
        else:
            n = _log(rng, 4, 96)
            c = {"op": op, "n": n, "L": rng.randint(1, 8), "Hkv": rng.choice([1, 2, 4, 8]), "D": D,
                 "P": rng.choice([16, 32, 64]), "max_pages": _log(rng, 4, 80)}
            if op == "pages_fork":
                c["keep"] = rng.randint(1, n)
            else:
                c["live"] = round(rng.uniform(0.1, 0.9), 2)
            if n * c["max_pages"] * c["L"] * c["Hkv"] * D * c["P"] > 48 * 48 * 4 * 4 * 128 * 64:
                continue
        return c


# ------------------------------------------------------------------ inputs

def _pow2(e):
    """2^e in fp32, for whole e of -126 to 127 (the exponent's bits: a power function rounds)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """x [pages, H, P, D] fp32 -> e4m3 values and the power-of-two scale of each (page, head)."""
    amax = x.abs().amax(dim=(2, 3))
    m, e = torch.frexp(amax / 448.0)
    e = torch.where(m > 0.5, e, e - 1)
    e = torch.where(amax > 0, e, torch.full_like(e, -126)).clamp_min(-126)
    s = _pow2(e)
    return (x / s[:, :, None, None]).to(F8), s


def _pool(g, n_pages, c):
    """Keys and values as a model leaves them: some channels larger than the others."""
    H, P, D = c["Hkv"], c["P"], c["D"]
    dev = "cuda"
    chan = torch.exp(0.7 * torch.randn((H, 1, D), generator=g, device=dev))
    out = []
    for amp in (0.6, 1.0):
        q = torch.empty((n_pages, H, P, D), device=dev, dtype=F8)
        s = torch.empty((n_pages, H), device=dev)
        step = max(1, (1 << 26) // (H * P * D))
        for a in range(0, n_pages, step):
            b = min(n_pages, a + step)
            x = torch.randn((b - a, H, P, D), generator=g, device=dev) * chan * amp
            q[a:b], s[a:b] = _quantise(x)
        out += [q, s]
    return out


def _lens(g, n, lo, hi):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    st = {"c": c}
    if c["op"] in ("window_fwd", "window_train"):
        dt = TYPES[c["dtype"]]
        shape_q, shape_k = (c["B"], c["Hq"], c["Nq"], c["D"]), (c["B"], c["Hkv"], c["Nk"], c["D"])
        st["q"] = torch.randn(shape_q, generator=g, device="cuda").to(dt)
        st["k"] = torch.randn(shape_k, generator=g, device="cuda").to(dt)
        st["v"] = torch.randn(shape_k, generator=g, device="cuda").to(dt)
        if c["op"] == "window_train":
            st["dout"] = torch.randn(shape_q, generator=g, device="cuda").to(dt)
            if own:
                for n in "qkv":
                    st[n].requires_grad_(True)
        return st
    if c["op"] == "kv8_attn":
        B, P = c["B"], c["P"]
        mp = -(-c["max_len"] // P)
        n_pages = B * mp + 3
        st["kp"], st["ks"], st["vp"], st["vs"] = _pool(g, n_pages, c)
        st["table"] = torch.randperm(n_pages, generator=g, device="cuda")[: B * mp].to(torch.int32).reshape(B, mp)
        st["lens"] = _lens(g, B, c["min_len"], c["max_len"])
        st["q"] = torch.randn((B, c["Hq"], c["Nq"], c["D"]), generator=g, device="cuda").to(TYPES[c["dtype"]])
        return st
    if c["op"] == "kv8_append":
        B, P, T = c["B"], c["P"], c["T"]
        dt = TYPES[c["dtype"]]
        mp = -(-(c["max_old"] + T) // P)
        n_pages = B * mp + 1
        st["kp"], st["ks"], st["vp"], st["vs"] = _pool(g, n_pages, c)
        st["table"] = torch.randperm(n_pages, generator=g, device="cuda")[: B * mp].to(torch.int32).reshape(B, mp)
        old = _lens(g, B, c["min_old"], c["max_old"])
        # most sequences take all T new tokens, some fewer (a ragged batch), none of them more
        st["n_new"] = torch.where(torch.rand((B,), generator=g, device="cuda") < 0.7, torch.full_like(old, T),
                                  _lens(g, B, min(1, T - 1), T))
        st["lens"] = old + st["n_new"]
        for n, amp in (("k", 0.8), ("v", 1.3)):
            st[n] = (amp * torch.randn((B, c["Hkv"], T, c["D"]), generator=g, device="cuda")).to(dt)
        return st
    # page bookkeeping: n slots with random lengths over one pool
    n, mp, P, L = c["n"], c["max_pages"], c["P"], c["L"]
    n_pages = n * mp + 1
    page = (L, n_pages, c["Hkv"], P, c["D"])
    for a in "kv":
        st[a + "p"] = torch.randint(0, 120, page, generator=g, device="cuda", dtype=torch.uint8).view(F8)
        st[a + "s"] = _pow2(torch.randint(-9, 3, page[:3], generator=g, device="cuda"))
    if c["op"] == "pages_fork":
        lens = _lens(g, n, 1, mp * P)
        st["parents"] = torch.arange(n, device="cuda", dtype=torch.int32)
        perm = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
        kept, rest = perm[: c["keep"]], perm[c["keep"]:]
        pick = torch.randint(0, c["keep"], (n - c["keep"],), generator=g, device="cuda")
        st["parents"][rest.long()] = kept[pick]
    else:
        lens = _lens(g, n, 1, mp * P)
        gone = torch.rand((n,), generator=g, device="cuda") > c["live"]
        lens = torch.where(gone, torch.zeros_like(lens), lens)
    ids = torch.randperm(n_pages, generator=g, device="cuda")[: n * mp].to(torch.int32).reshape(n, mp)
    used = torch.arange(mp, device="cuda")[None] * P < lens[:, None]
    st["table"] = torch.where(used, ids, torch.full_like(ids, -1))
    st["lens"] = lens
    st["refs"] = torch.zeros(n_pages, device="cuda", dtype=torch.int32)
    st["refs"][st["table"][used].long()] = 1
    if own:
        from tiled_memory_efficient_gb300 import _lib
        st["src"] = torch.empty(n_pages, device="cuda", dtype=torch.int32)
        st["dst"] = torch.empty(n_pages, device="cuda", dtype=torch.int32)
        st["info"] = torch.zeros(4, device="cuda", dtype=torch.int32)
        st["ws"] = torch.empty(_lib.kvp_workspace_size(n, mp, n_pages), device="cuda", dtype=torch.uint8)
        st["table_out"] = torch.empty_like(st["table"])
        st["refs_out"] = torch.empty_like(st["refs"])
    return st


# ------------------------------------------------------------------ plain forms

def _visible(pos, keys, W, S):
    """[queries, keys] truth values: key <= position, inside the window or one of the first S."""
    d = pos[:, None] - keys[None]
    ok = d >= 0
    return ok & ((d < W) | (keys[None] < S)) if W > 0 else ok


def _window_blocks(c):
    """Query blocks with the keys their windows reach: (first, last + 1, key indices)."""
    off, step = c["Nk"] - c["Nq"], 512
    for a in range(0, c["Nq"], step):
        b = min(c["Nq"], a + step)
        lo = max(0, a + off - c["W"] + 1)
        keys = torch.cat([torch.arange(0, min(c["S"], lo), device="cuda"),
                          torch.arange(lo, b + off, device="cuda")])
        yield a, b, keys, _visible(torch.arange(a, b, device="cuda") + off, keys, c["W"], c["S"])


def _window_fwd(c, q, k, v):
    B, Hq, Nq, D = q.shape
    Hkv = k.shape[1]
    scale = 1.0 / math.sqrt(D)
    qf, kf, vf = q.float().reshape(B, Hkv, Hq // Hkv, Nq, D), k.float(), v.float()
    out = torch.empty_like(qf)
    lse = torch.empty(qf.shape[:4], device=q.device)
    for a, b, keys, ok in _window_blocks(c):
        kb, vb = kf[:, :, None, keys], vf[:, :, None, keys]
        s = (qf[:, :, :, a:b] @ kb.transpose(-1, -2)) * scale
        s = s.masked_fill(~ok, float("-inf"))
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        z = p.sum(-1, keepdim=True)
        out[:, :, :, a:b] = (p @ vb) / z
        lse[:, :, :, a:b] = (m + torch.log(z)).squeeze(-1)
    return out.reshape(B, Hq, Nq, D), lse.reshape(B, Hq, Nq)


def _window_bwd(c, q, k, v, out, lse, dout):
    B, Hq, Nq, D = q.shape
    Hkv = k.shape[1]
    G, scale = Hq // Hkv, 1.0 / math.sqrt(D)
    split = lambda t: t.float().reshape(B, Hkv, G, Nq, -1)
    qf, of, gf, lf = split(q), split(out), split(dout), split(lse)
    kf, vf = k.float(), v.float()
    dq, dk, dv = torch.empty_like(qf), torch.zeros_like(kf), torch.zeros_like(vf)
    delta = (gf * of).sum(-1, keepdim=True)
    for a, b, keys, ok in _window_blocks(c):
        kb, vb = kf[:, :, None, keys], vf[:, :, None, keys]
        s = (qf[:, :, :, a:b] @ kb.transpose(-1, -2)) * scale
        p = torch.exp(s - lf[:, :, :, a:b]) * ok
        ds = p * (gf[:, :, :, a:b] @ vb.transpose(-1, -2) - delta[:, :, :, a:b])
        dq[:, :, :, a:b] = scale * (ds @ kb)
        dv[:, :, keys] += (p.transpose(-1, -2) @ gf[:, :, :, a:b]).sum(2)
        dk[:, :, keys] += scale * (ds.transpose(-1, -2) @ qf[:, :, :, a:b]).sum(2)
    return dq.reshape(q.shape), dk, dv


def _kv8_attn(st):
    c = st["c"]
    q = st["q"]
    B, Hq, Nq, D = q.shape
    Hkv, P = c["Hkv"], c["P"]
    scale = 1.0 / math.sqrt(D)
    outs, lses = [], []
    for b in range(B):
        ids = st["table"][b].long()
        deq = lambda pages, s: (pages[ids].float() * s[ids][:, :, None, None]).transpose(0, 1).reshape(Hkv, -1, D)
        k, v = deq(st["kp"], st["ks"]), deq(st["vp"], st["vs"])
        keys = torch.arange(k.shape[1], device="cuda")
        ok = _visible(st["lens"][b] - Nq + torch.arange(Nq, device="cuda"), keys, c["W"], c["S"])
        s = (q[b].float().reshape(Hkv, Hq // Hkv, Nq, D) @ k[:, None].transpose(-1, -2)) * scale
        s = s.masked_fill(~ok, float("-inf"))
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        z = p.sum(-1, keepdim=True)
        outs.append(((p @ v[:, None]) / z).reshape(Hq, Nq, D))
        lses.append((m + torch.log(z)).reshape(Hq, Nq))
    return torch.stack(outs).to(q.dtype), torch.stack(lses)


def _append_one(st, new, pages, scales):
    c = st["c"]
    B, P, T = c["B"], c["P"], c["T"]
    lens, start = st["lens"].long(), (st["lens"] - st["n_new"]).long()
    j = start[:, None] // P + torch.arange(T // P + 2, device="cuda")[None]          # pages touched
    live = (j * P < lens[:, None]) & (lens > start)[:, None]
    bi, ji = torch.nonzero(live, as_tuple=True)
    jj = j[bi, ji]
    pid = st["table"][bi, jj].long()
    pos = jj[:, None] * P + torch.arange(P, device="cuda")[None]
    is_new = (pos >= start[bi][:, None]) & (pos < lens[bi][:, None])
    is_old = pos < start[bi][:, None]
    tok = (pos - start[bi][:, None]).clamp(0, T - 1)
    x = new[bi[:, None], :, tok].float().transpose(1, 2)                              # [n, H, P, D]
    amax = torch.where(is_new[:, None, :, None], x.abs(), torch.zeros_like(x)).amax(dim=(2, 3))
    m, e = torch.frexp(amax / 448.0)
    e = torch.where(m > 0.5, e, e - 1)
    e = torch.where(amax > 0, e, torch.full_like(e, -126)).clamp_min(-126)
    s_new = _pow2(e)
    s_old = scales[pid]
    s = torch.where(is_old.any(1)[:, None], torch.maximum(s_old, s_new), s_new)
    held = pages[pid]
    kept = (held.float() * (s_old / s)[:, :, None, None]).to(F8)
    put = (x / s[:, :, None, None]).to(F8)
    r = torch.where(is_new[:, None, :, None], put.view(torch.uint8),
                    torch.where(is_old[:, None, :, None], kept.view(torch.uint8), held.view(torch.uint8)))
    pages[pid] = r.view(F8)
    scales[pid] = s


def _copy(st, src, dst):
    for n in ("kp", "ks", "vp", "vs"):
        t = st[n].view(torch.uint8) if st[n].dtype == F8 else st[n]
        t[:, dst] = t[:, src]


def _fork(st):
    c = st["c"]
    n, P = c["n"], c["P"]
    par = st["parents"].long()
    me = torch.arange(n, device="cuda")
    table, lens = st["table"][par], st["lens"][par]
    # who keeps a parent's partly filled last page: the parent itself, else its first child
    keeper = torch.full((n,), n, device="cuda", dtype=torch.long)
    keeper = keeper.scatter_reduce(0, par, torch.where(par == me, torch.full_like(me, -1), me), "amin")
    keeper = torch.where(keeper < 0, me, keeper)
    copies = torch.nonzero((lens % P != 0) & (keeper[par] != me)).flatten()
    refs = torch.zeros_like(st["refs"])
    ids = table.clone()
    last = (lens[copies] // P).long()
    src = ids[copies, last].long()
    ids[copies, last] = -1
    held = ids[ids >= 0].long()
    refs.index_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    dst = torch.nonzero(refs == 0).flatten()[: copies.numel()]
    table[copies, last] = dst.to(torch.int32)
    refs[dst] = 1
    st["table"].copy_(table)
    st["lens"].copy_(lens)
    st["refs"].copy_(refs)
    _copy(st, src, dst)
    return {k: st[k] for k in ("table", "lens", "refs", "kp", "ks", "vp", "vs")}


def _compact(st):
    refs, table = st["refs"], st["table"]
    live = refs > 0
    n_live = live.sum()
    ids = torch.arange(refs.numel(), device="cuda")
    dst = torch.nonzero(~live & (ids < n_live)).flatten()
    src = torch.nonzero(live & (ids >= n_live)).flatten()
    remap = ids.clone()
    remap[src] = dst
    new_table = torch.where(table >= 0, remap[table.clamp_min(0).long()].to(torch.int32), table)
    new_refs = refs.clone()
    new_refs[dst] = refs[src]
    new_refs[src] = 0
    _copy(st, src, dst)
    return {"table": new_table, "refs": new_refs, **{k: st[k] for k in ("kp", "ks", "vp", "vs")}}


def _plain(st):
    c = st["c"]
    if c["op"] == "window_fwd":
        out, lse = _window_fwd(c, st["q"], st["k"], st["v"])
        return {"out": out.to(st["q"].dtype), "lse": lse}
    if c["op"] == "window_train":
        q, k, v = st["q"], st["k"], st["v"]
        out, lse = _window_fwd(c, q, k, v)
        dq, dk, dv = _window_bwd(c, q, k, v, out, lse, st["dout"])
        dt = q.dtype
        return {"out": out.to(dt), "dq": dq.to(dt), "dk": dk.to(dt), "dv": dv.to(dt)}
    if c["op"] == "kv8_attn":
        out, lse = _kv8_attn(st)
        return {"out": out, "lse": lse}
    if c["op"] == "kv8_append":
        _append_one(st, st["k"], st["kp"], st["ks"])
        _append_one(st, st["v"], st["vp"], st["vs"])
        return {n: st[n] for n in ("kp", "ks", "vp", "vs")}
    return _fork(st) if c["op"] == "pages_fork" else _compact(st)


def _own(st):
    from tiled_memory_efficient_gb300 import _lib, sdpa
    c = st["c"]
    if c["op"] == "window_fwd":
        out, lse = _lib.attn_fwd_window(st["q"], st["k"], st["v"], window=c["W"], sinks=c["S"])
        return {"out": out, "lse": lse}
    if c["op"] == "window_train":
        out = sdpa.window_attention(st["q"], st["k"], st["v"], window=c["W"], sinks=c["S"])
        dq, dk, dv = torch.autograd.grad(out, (st["q"], st["k"], st["v"]), st["dout"])
        return {"out": out.detach(), "dq": dq, "dk": dk, "dv": dv}
    if c["op"] == "kv8_attn":
        out, lse = _lib.kv8_attn(st["q"], st["kp"], st["vp"], st["ks"], st["vs"], st["table"], st["lens"],
                                 window=c["W"], sinks=c["S"])
        return {"out": out, "lse": lse}
    if c["op"] == "kv8_append":
        _lib.kv8_append(st["k"], st["v"], st["kp"], st["vp"], st["ks"], st["vs"], st["table"], st["lens"],
                        n_new=st["n_new"])
        return {n: st[n] for n in ("kp", "ks", "vp", "vs")}
    pools = (st["kp"], st["vp"], st["ks"], st["vs"])
    if c["op"] == "pages_fork":
        _lib.kvp_reassign(st["table"], st["lens"], st["refs"], st["parents"], c["P"], st["src"], st["dst"],
                          st["info"], workspace=st["ws"])
        _lib.kv8_copy_pages(*pools, st["src"], st["dst"], st["info"][1:], max_count=c["n"])
        return {k: st[k] for k in ("table", "lens", "refs", "kp", "ks", "vp", "vs")}
    _lib.kvp_compact(st["table"], st["refs"], st["src"], st["dst"], st["info"], table_out=st["table_out"],
                     refs_out=st["refs_out"], workspace=st["ws"])
    _lib.kv8_copy_pages(*pools, st["src"], st["dst"], st["info"][1:], max_count=st["refs"].numel() // 2)
    return {"table": st["table_out"], "refs": st["refs_out"], "kp": st["kp"], "ks": st["ks"], "vp": st["vp"],
            "vs": st["vs"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work

def _pairs(nq, nk, W, S):
    """Visible (query, key) pairs of one head: queries at the last nq positions of nk."""
    total = 0
    for p in range(max(0, nk - nq), nk):
        total += p + 1 if W <= 0 or p < W else W + min(S, p + 1 - W)
    return total


def _seen(nq, nk, W, S):
    """Keys at least one of the queries sees."""
    if W <= 0:
        return nk
    lo = max(0, nk - nq - W + 1)
    return nk - lo + min(S, lo)


def work(case):
    c = case
    if c["op"] in ("window_fwd", "window_train"):
        pairs = c["B"] * c["Hq"] * _pairs(c["Nq"], c["Nk"], c["W"], c["S"])
        nq = c["B"] * c["Hq"] * c["Nq"]
        nk = c["B"] * c["Hkv"] * _seen(c["Nq"], c["Nk"], c["W"], c["S"])
        if c["op"] == "window_fwd":
            return {"bytes": 2 * c["D"] * (2 * nq + 2 * nk) + 4 * nq, "flops": 4 * c["D"] * pairs}
        return {"bytes": 2 * c["D"] * (4 * nq + 4 * nk), "flops": 14 * c["D"] * pairs}
    if c["op"] == "kv8_attn":
        mean = (c["min_len"] + c["max_len"]) // 2
        seen = c["B"] * _seen(c["Nq"], mean, c["W"], c["S"])
        q = c["B"] * c["Hq"] * c["Nq"]
        return {"bytes": seen * c["Hkv"] * (2 * c["D"] + 8 / c["P"]) + q * (4 * c["D"] + 4),
                "flops": 4 * c["D"] * c["B"] * c["Hq"] * _pairs(c["Nq"], mean, c["W"], c["S"])}
    if c["op"] == "kv8_append":
        n = c["B"] * c["Hkv"] * max(1, int(0.85 * c["T"]))
        return {"bytes": n * c["D"] * 2 * 3 + n / c["P"] * 8, "flops": 2 * n * c["D"]}
    page = c["L"] * c["Hkv"] * (2 * c["P"] * c["D"] + 8)
    table = 4 * c["n"] * c["max_pages"]
    if c["op"] == "pages_fork":
        return {"bytes": 2 * page * (c["n"] - c["keep"]) + 2 * table, "flops": 0}
    pages = c["n"] * c["max_pages"]
    moved = pages * 0.5 * c["live"] * (1 - 0.5 * c["live"])
    return {"bytes": 2 * page * moved + 2 * table + 8 * pages, "flops": 0}


# ------------------------------------------------------------------ exact

def _dense(q, k, v, W, S, dout=None):
    """One head in 64 bits, from the definition: every score, softmax, weighted sum; with dout the
    gradients of sum(out * dout) by differentiating it."""
    nq, nk = q.shape[0], k.shape[0]
    q, k, v = (t.double().requires_grad_(dout is not None) for t in (q, k, v))
    i = torch.arange(nk - nq, nk, device=q.device).view(-1, 1)
    j = torch.arange(nk, device=q.device).view(1, -1)
    hidden = j > i
    if W > 0:
        hidden = hidden | ((j <= i - W) & (j >= S))
    s = torch.where(hidden, -math.inf, (q @ k.t()) * q.shape[1] ** -0.5)
    out = torch.softmax(s, dim=1) @ v
    if dout is None:
        return out, torch.logsumexp(s, dim=1)
    return (out.detach(),) + torch.autograd.grad(out, (q, k, v), dout.double())


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    if c["op"] in ("window_fwd", "window_train"):
        q, k, v = (st[n].detach() for n in "qkv")
        G = c["Hq"] // c["Hkv"]
        train = c["op"] == "window_train"
        if c["B"] * c["Hq"] * c["Nq"] * c["Nk"] * c["D"] * (14 if train else 4) > 1.2e13:
            return None
        names = ("out", "dq", "dk", "dv") if train else ("out", "lse")
        shape = {"out": q.shape, "lse": q.shape[:3], "dq": q.shape, "dk": k.shape, "dv": k.shape}
        res = {n: torch.zeros(shape[n], device="cuda", dtype=torch.float64) for n in names}
        for b in range(c["B"]):
            for h in range(c["Hq"]):
                r = _dense(q[b, h], k[b, h // G], v[b, h // G], c["W"], c["S"], st["dout"][b, h] if train else None)
                for n, t in zip(names, r):
                    res[n][b, h // G if n in ("dk", "dv") else h] += t
        return res
    if c["op"] == "kv8_attn":
        q = st["q"]
        G = c["Hq"] // c["Hkv"]
        res = {"out": torch.zeros(q.shape, device="cuda", dtype=torch.float64),
               "lse": torch.zeros(q.shape[:3], device="cuda", dtype=torch.float64)}
        for b, n in enumerate(st["lens"].tolist()):
            ids = st["table"][b, : -(-n // c["P"])].long()
            for h in range(c["Hkv"]):
                k, v = ((st[p][ids, h].double() * st[s][ids, h].double()[:, None, None]).reshape(-1, c["D"])[:n]
                        for p, s in (("kp", "ks"), ("vp", "vs")))
                for e in range(h * G, (h + 1) * G):
                    res["out"][b, e], res["lse"][b, e] = _dense(q[b, e], k, v, c["W"], c["S"])
        return res
    if c["op"] == "kv8_append":
        return _exact_append(st)
    # whole numbers and moved bytes: compared for equality, nothing is computed in floating point
    return None


def _round_e4m3(x):
    """float64 -> the nearest e4m3 value, ties to even: 4 significant bits, spacing at least 2^-9."""
    _, e = torch.frexp(x)
    ulp = (((e.long() - 4).clamp_min(-9) + 1023) << 52).view(torch.float64)
    return (torch.round(x / ulp) * ulp).clamp(-448, 448)


def _exact_append(st):
    c = st["c"]
    P, res = c["P"], {}
    table, lens, n_new = st["table"].tolist(), st["lens"].tolist(), st["n_new"].tolist()
    if sum(-(-n // P) + 2 for n in n_new) * c["Hkv"] > 20000:
        return None
    for new, pages, scales in (("k", "kp", "ks"), ("v", "vp", "vs")):
        vals, sc = st[pages].double(), st[scales].double().clone()
        for b in range(c["B"]):
            start = lens[b] - n_new[b]
            if n_new[b] == 0:
                continue
            for j in range(start // P, (lens[b] - 1) // P + 1):
                pid, first, end = table[b][j], max(start, j * P), min(lens[b], (j + 1) * P)
                x = st[new][b, :, first - start: end - start].double()
                amax = x.abs().amax(dim=(1, 2))
                e = torch.ceil(torch.log2(amax.clamp_min(1e-300) / 448.0)).clamp_min(-126)
                s = ((e.long() + 1023) << 52).view(torch.float64)
                o = first - j * P
                if o > 0:
                    s = torch.maximum(s, sc[pid])
                    vals[pid, :, :o] = _round_e4m3(vals[pid, :, :o] * (sc[pid] / s)[:, None, None])
                vals[pid, :, o: end - j * P] = _round_e4m3(x / s[:, None, None])
                sc[pid] = s
        res[pages], res[scales] = vals, sc
    return res
