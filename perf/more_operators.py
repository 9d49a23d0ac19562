"""Workloads of rotary positions, of the cache's append that rotates on the way, and of
attention over a cache whose sequences share a long prefix.

Every case names one operator (``op``) and its sizes; ``run`` makes one pass
through it, either as plain torch operations (``own`` false) or with the
library's calls (``own`` true).

  rope         queries and keys rotated to their positions
  rope_train   the same, forward and backward
  append_rope  a step's keys rotated and quantised into the paged cache, its values
               quantised, its queries rotated
  shared_attn  attention of the newest positions over a paged cache whose sequences
               start with the same pages
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # A training step's queries and keys at the training shape, gradients included.
        {"name": "rope_train_mha", "op": "rope_train", "B": 2, "Hq": 16, "Hkv": 16, "N": 8192, "D": 128, "rot": 128,
         "inter": False, "scaling": "none", "far": 0, "heads_last": False, "dtype": "bf16"},
        # Grouped heads at an odd length, half of each head rotated, as views of a projection's rows.
        {"name": "rope_train_gqa", "op": "rope_train", "B": 1, "Hq": 14, "Hkv": 2, "N": 4099, "D": 64, "rot": 32,
         "inter": True, "scaling": "linear", "far": 0, "heads_last": True, "dtype": "fp16"},
        # A long prompt through the grouped-query model, frequencies scaled for its length.
        {"name": "rope_prefill_gqa", "op": "rope", "B": 1, "Hq": 14, "Hkv": 2, "N": 16384, "D": 64, "rot": 64,
         "inter": False, "scaling": "yarn", "far": 100000, "heads_last": True, "dtype": "fp16"},
        # One token each of a serving batch, far positions: latency counts.
        {"name": "rope_decode", "op": "rope", "B": 64, "Hq": 32, "Hkv": 8, "N": 1, "D": 128, "rot": 128,
         "inter": False, "scaling": "bands", "far": 120000, "heads_last": False, "dtype": "bf16"},
        # A prompt's queries, keys and values of one layer.
        {"name": "append_prompt", "op": "append_rope", "B": 2, "Hq": 32, "Hkv": 8, "T": 8190, "D": 128, "P": 64,
         "rot": 128, "inter": False, "scaling": "bands", "min_old": 0, "max_old": 100, "dtype": "bf16"},
        # One decoding step of a batch of 64.
        {"name": "append_step", "op": "append_rope", "B": 64, "Hq": 32, "Hkv": 8, "T": 1, "D": 128, "P": 64,
         "rot": 128, "inter": False, "scaling": "none", "min_old": 1, "max_old": 4000, "dtype": "bf16"},
        # Drafts of up to five tokens on small pages, a quarter of each head rotated in interleaved pairs.
        {"name": "append_drafts", "op": "append_rope", "B": 7, "Hq": 14, "Hkv": 2, "T": 5, "D": 64, "P": 16,
         "rot": 16, "inter": True, "scaling": "ntk", "min_old": 1000, "max_old": 70000, "dtype": "fp16"},
        # Sixty-four samples of one long prompt (the decode workload's heads).
        {"name": "shared_samples", "op": "shared_attn", "B": 64, "groups": 1, "Hq": 14, "Hkv": 2, "Nq": 1, "D": 64,
         "P": 64, "prefix": 32768, "max_tail": 600, "dtype": "fp16"},
        # A serving batch under one instruction text of 16K tokens.
        {"name": "shared_serving", "op": "shared_attn", "B": 128, "groups": 1, "Hq": 32, "Hkv": 8, "Nq": 1, "D": 128,
         "P": 64, "prefix": 16384, "max_tail": 1000, "dtype": "bf16"},
        # Four prompts of odd length, twelve samples each, three drafted tokens a step, small pages.
        {"name": "shared_drafts", "op": "shared_attn", "B": 48, "groups": 4, "Hq": 16, "Hkv": 4, "Nq": 3, "D": 128,
         "P": 16, "prefix": 5008, "max_tail": 333, "dtype": "fp16"},
        # A few beams of a middling prompt: latency counts.
        {"name": "shared_beams", "op": "shared_attn", "B": 8, "groups": 1, "Hq": 14, "Hkv": 2, "Nq": 1, "D": 64,
         "P": 32, "prefix": 4096, "max_tail": 100, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["rope", "rope_train", "append_rope", "append_rope", "shared_attn", "shared_attn"])
        D = rng.choice([64, 128])
        G, Hkv = rng.choice([1, 2, 4, 7, 8]), rng.choice([1, 2, 4, 8])
        c = {"op": op, "Hq": G * Hkv, "Hkv": Hkv, "D": D, "dtype": rng.choice(["fp16", "bf16"])}
        if op != "shared_attn":
            c |= {"rot": rng.choice([D, D, D // 2, D // 4, 2 * rng.randint(1, D // 2)]),
                  "inter": rng.random() < 0.4,
                  "scaling": rng.choice(["none", "linear", "ntk", "yarn", "bands"])}
        if op in ("rope", "rope_train"):
            c |= {"B": _log(rng, 1, 64), "N": _log(rng, 1, 20000), "far": rng.choice([0, _log(rng, 10, 500000)]),
                  "heads_last": rng.random() < 0.5}
            if c["B"] * c["N"] * (c["Hq"] + Hkv) * D > 2 * 8192 * 32 * 128:
                continue
        elif op == "append_rope":
            c |= {"B": _log(rng, 1, 100), "T": rng.choice([1, 1, rng.randint(2, 9), _log(rng, 10, 10000)]),
                  "P": rng.choice([16, 32, 64, 128]), "min_old": 0, "max_old": _log(rng, 1, 100000)}
            if c["B"] * c["T"] * (c["Hq"] + 2 * Hkv) * D > 2 * 8190 * 48 * 128 or \
                    c["B"] * (c["T"] + c["max_old"]) * Hkv * D > 64 * 8000 * 8 * 128:
                continue
        else:
            groups = rng.choice([1, 1, 2, rng.randint(2, 6)])
            P = rng.choice([16, 32, 64, 128])
            c |= {"B": max(groups, _log(rng, 2, 160)), "groups": groups, "Nq": rng.choice([1, 1, 1, 2, 5]), "P": P,
                  "prefix": max(1, _log(rng, 64, 40000) // P) * P, "max_tail": _log(rng, 5, 2000)}
            if c["B"] * c["Hq"] * c["Nq"] * (c["prefix"] + c["max_tail"]) * D > 128 * 32 * 17384 * 128 or \
                    c["B"] * Hkv * c["prefix"] * D > 128 * 8 * 16384 * 128:
                continue
        return c


# ------------------------------------------------------------------ inputs

def _pow2(e):
    """2^e in fp32, for whole e of -126 to 127 (the exponent's bits: a power function rounds)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(amax):
    """Smallest e of at least -126 with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax / 448.0)
    e = torch.where(m > 0.5, e, e - 1)
    return torch.where(amax > 0, e, torch.full_like(e, -126)).clamp_min(-126)


def _pool(g, n_pages, c):
    """Keys and values as a model leaves them: some channels larger than the others."""
    H, P, D = c["Hkv"], c["P"], c["D"]
    chan = torch.exp(0.7 * torch.randn((H, 1, D), generator=g, device="cuda"))
    out = []
    for amp in (0.6, 1.0):
        q = torch.empty((n_pages, H, P, D), device="cuda", dtype=F8)
        s = torch.empty((n_pages, H), device="cuda")
        step = max(1, (1 << 26) // (H * P * D))
        for a in range(0, n_pages, step):
            b = min(n_pages, a + step)
            x = torch.randn((b - a, H, P, D), generator=g, device="cuda") * chan * amp
            s[a:b] = _pow2(_exponent(x.abs().amax(dim=(2, 3))))
            q[a:b] = (x / s[a:b, :, None, None]).to(F8)
        out += [q, s]
    return out


def _lens(g, n, lo, hi):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


# What a model's configuration says of its positions: the scaling and its numbers.
SCALINGS = {
    "none": None,
    "linear": {"kind": "linear", "factor": 4.0},
    "ntk": {"kind": "ntk", "factor": 8.0},
    "yarn": {"kind": "yarn", "factor": 16.0, "original_len": 8192},
    "bands": {"kind": "bands", "factor": 8.0, "low": 1.0, "high": 4.0, "original_len": 8192},
}
BASES = {"none": 10000.0, "linear": 10000.0, "ntk": 10000.0, "yarn": 1000000.0, "bands": 500000.0}


def _rope(c):
    from tiled_memory_efficient_gb300.rope import Rope
    return Rope(c["D"], rotary_dim=c["rot"], base=BASES[c["scaling"]], interleaved=c["inter"],
                scaling=SCALINGS[c["scaling"]])


def _rows(g, c, H, N, amp=1.0):
    """[B, H, N, D] with outlying channels; heads_last: a view of [B, N, H, D] rows."""
    chan = torch.exp(0.7 * torch.randn((H, 1, c["D"]), generator=g, device="cuda"))
    x = (amp * chan * torch.randn((c["B"], H, N, c["D"]), generator=g, device="cuda")).to(TYPES[c["dtype"]])
    return x.transpose(1, 2).contiguous().transpose(1, 2) if c.get("heads_last") else x


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    st = {"c": c}
    if own and c["op"] != "shared_attn":
        st["rope"] = _rope(c)
    if c["op"] in ("rope", "rope_train"):
        for n, H in (("q", c["Hq"]), ("k", c["Hkv"])):
            st[n] = _rows(g, c, H, c["N"])
            if c["op"] == "rope_train":
                st["d" + n] = _rows(g, c, H, c["N"])
                if own:
                    st[n].requires_grad_(True)
        start = _lens(g, c["B"], 0, c["far"])
        st["positions"] = start[:, None] + torch.arange(c["N"], device="cuda", dtype=torch.int32)[None]
        return st
    B, P = c["B"], c["P"]
    if c["op"] == "append_rope":
        T = c["T"]
        old = _lens(g, B, c["min_old"], c["max_old"])
        # most sequences take all T new tokens, some fewer (a ragged batch), none of them more
        st["n_new"] = torch.where(torch.rand((B,), generator=g, device="cuda") < 0.7, torch.full_like(old, T),
                                  _lens(g, B, min(1, T - 1), T))
        st["lens"] = old + st["n_new"]
        # only the pages that the step touches need memory: earlier ones stand for others
        mp, touched = -(-(c["max_old"] + T) // P), T // P + 2
        n_pages = B * touched + 1
        st["kp"], st["ks"], st["vp"], st["vs"] = _pool(g, n_pages, c)
        ids = torch.randperm(n_pages, generator=g, device="cuda")[: B * touched].to(torch.int32).reshape(B, touched)
        st["table"] = ids[:, torch.arange(mp, device="cuda") % touched].contiguous()
        for n, H, amp in (("q", c["Hq"], 1.0), ("k", c["Hkv"], 0.8), ("v", c["Hkv"], 1.3)):
            st[n] = _rows(g, c, H, T, amp)
        return st
    # sequence b belongs to prompt b % groups, whose pages its table begins with
    head, tail = c["prefix"] // P, -(-c["max_tail"] // P)
    n_pages = c["groups"] * head + B * tail + 3
    st["kp"], st["ks"], st["vp"], st["vs"] = _pool(g, n_pages, c)
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    prompts = ids[: c["groups"] * head].reshape(c["groups"], head)
    rest = ids[c["groups"] * head: c["groups"] * head + B * tail].reshape(B, tail)
    st["table"] = torch.cat([prompts[torch.arange(B, device="cuda") % c["groups"]], rest], 1).contiguous()
    st["lens"] = c["prefix"] + _lens(g, B, min(c["Nq"], c["max_tail"]), c["max_tail"])
    st["q"] = torch.randn((B, c["Hq"], c["Nq"], c["D"]), generator=g, device="cuda").to(TYPES[c["dtype"]])
    if own:   # made after a fork, kept until the next one
        from tiled_memory_efficient_gb300 import _lib
        st["plan"] = _lib.kvp_find_shared(st["table"], st["lens"], P)
    return st


# ------------------------------------------------------------------ plain forms

def _frequencies(c):
    """(radians per position of each pair, the rotation's amplitude)."""
    r, base, s = c["rot"], BASES[c["scaling"]], SCALINGS[c["scaling"]]
    kind = s["kind"] if s else "none"
    if kind == "ntk" and r > 2:
        base = base * s["factor"] ** (r / (r - 2))
    i = torch.arange(r // 2, device="cuda", dtype=torch.float64)
    f = base ** (-2.0 * i / r)
    if kind == "linear":
        f = f / s["factor"]
    elif kind == "yarn":
        turns = lambda n: r * math.log(s["original_len"] / (2 * math.pi * n)) / (2 * math.log(base))
        lo, hi = max(math.floor(turns(32.0)), 0), min(math.ceil(turns(1.0)), r - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f * (1 - ramp) + f / s["factor"] * ramp
        return f, 0.1 * math.log(s["factor"]) + 1.0
    elif kind == "bands":
        blend = ((s["original_len"] * f / (2 * math.pi) - s["low"]) / (s["high"] - s["low"])).clamp(0, 1)
        f = f / s["factor"] * (1 - blend) + f * blend
    return f, 1.0


def _rotate(c, x, cos, sin):
    """x [..., D] in fp32, cos and sin [..., rot / 2]."""
    r = c["rot"]
    if c["inter"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., : r // 2], x[..., r // 2: r]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., r:]), -1)


def _cos_sin(c, positions):
    f, amp = _frequencies(c)
    t = positions.double()[..., None] * f    # far positions: 64 bits
    return (torch.cos(t) * amp).float(), (torch.sin(t) * amp).float()


def _plain_rope(st):
    c = st["c"]
    cos, sin = (t[:, None] for t in _cos_sin(c, st["positions"]))
    dt = TYPES[c["dtype"]]
    out = {n: _rotate(c, st[n].float(), cos, sin).to(dt) for n in "qk"}
    if c["op"] == "rope_train":
        out |= {n: _rotate(c, st[n].float(), cos, -sin).to(dt) for n in ("dq", "dk")}
    return out


def _append_one(st, new, pages, scales):
    """new [B, H, T, D] in fp32."""
    c = st["c"]
    P, T = c["P"], c["T"]
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
    x = new[bi[:, None], :, tok].transpose(1, 2)                                      # [n, H, P, D]
    s_new = _pow2(_exponent(torch.where(is_new[:, None, :, None], x.abs(), torch.zeros_like(x)).amax(dim=(2, 3))))
    s_old = scales[pid]
    s = torch.where(is_old.any(1)[:, None], torch.maximum(s_old, s_new), s_new)
    held = pages[pid]
    kept = (held.float() * (s_old / s)[:, :, None, None]).to(F8)
    put = (x / s[:, :, None, None]).to(F8)
    r = torch.where(is_new[:, None, :, None], put.view(torch.uint8),
                    torch.where(is_old[:, None, :, None], kept.view(torch.uint8), held.view(torch.uint8)))
    pages[pid] = r.view(F8)
    scales[pid] = s


def _plain_append(st):
    c = st["c"]
    t = torch.arange(c["T"], device="cuda")
    cos, sin = (x[:, None] for x in _cos_sin(c, (st["lens"] - st["n_new"])[:, None] + t[None]))
    live = (t[None] < st["n_new"][:, None])[:, None, :, None]
    q = torch.where(live, _rotate(c, st["q"].float(), cos, sin), 0.0).to(TYPES[c["dtype"]])
    _append_one(st, _rotate(c, st["k"].float(), cos, sin), st["kp"], st["ks"])
    _append_one(st, st["v"].float(), st["vp"], st["vs"])
    return {"q": q, **{n: st[n] for n in ("kp", "ks", "vp", "vs")}}


def _plain_shared(st):
    """Sequence by sequence: the keys and values of all of them at once would take tens of GB."""
    c, q = st["c"], st["q"]
    B, Hq, Nq, D = q.shape
    Hkv = c["Hkv"]
    outs, lses = [], []
    for b in range(B):
        ids = st["table"][b].long()
        deq = lambda pages, s: (pages[ids].float() * s[ids][:, :, None, None]).transpose(0, 1).reshape(Hkv, -1, D)
        k, v = deq(st["kp"], st["ks"]), deq(st["vp"], st["vs"])
        pos = st["lens"][b] - Nq + torch.arange(Nq, device="cuda")
        ok = torch.arange(k.shape[1], device="cuda")[None] <= pos[:, None]
        s = (q[b].float().reshape(Hkv, Hq // Hkv, Nq, D) @ k[:, None].transpose(-1, -2)) / math.sqrt(D)
        s = s.masked_fill(~ok, float("-inf"))
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        z = p.sum(-1, keepdim=True)
        outs.append(((p @ v[:, None]) / z).reshape(Hq, Nq, D))
        lses.append((m + torch.log(z)).reshape(Hq, Nq))
    return {"out": torch.stack(outs).to(q.dtype), "lse": torch.stack(lses)}


def _own(st):
    from tiled_memory_efficient_gb300 import _lib
    c = st["c"]
    if c["op"] in ("rope", "rope_train"):
        q, k = st["rope"](st["q"], st["k"], st["positions"])
        if c["op"] == "rope":
            return {"q": q, "k": k}
        dq, dk = torch.autograd.grad((q, k), (st["q"], st["k"]), (st["dq"], st["dk"]))
        return {"q": q.detach(), "k": k.detach(), "dq": dq, "dk": dk}
    if c["op"] == "append_rope":
        q = _lib.kv8_append(st["k"], st["v"], st["kp"], st["vp"], st["ks"], st["vs"], st["table"], st["lens"],
                            n_new=st["n_new"], rope=st["rope"], q=st["q"])
        return {"q": q, **{n: st[n] for n in ("kp", "ks", "vp", "vs")}}
    out, lse = _lib.kv8_attn_shared(st["q"], st["kp"], st["vp"], st["ks"], st["vs"], st["table"], st["lens"],
                                    st["plan"])
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _own(state)
    op = state["c"]["op"]
    return _plain_append(state) if op == "append_rope" else _plain_shared(state) if op == "shared_attn" else \
        _plain_rope(state)


# ------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] in ("rope", "rope_train"):
        n = c["B"] * (c["Hq"] + c["Hkv"]) * c["N"]
        times = 2 if c["op"] == "rope_train" else 1
        return {"bytes": times * 4 * n * c["D"] + 4 * c["B"] * c["N"], "flops": times * 3 * n * c["rot"]}
    if c["op"] == "append_rope":
        n = c["B"] * max(1, int(0.85 * c["T"]))
        return {"bytes": n * c["D"] * (6 * c["Hkv"] + 4 * c["Hq"]) + 8 * n * c["Hkv"] / c["P"],
                "flops": n * (3 * (c["Hq"] + c["Hkv"]) * c["rot"] + 2 * c["Hkv"] * c["D"])}
    tail = c["B"] * (c["max_tail"] + c["Nq"]) // 2
    rows = c["B"] * c["Hq"] * c["Nq"]
    return {"bytes": (c["groups"] * c["prefix"] + tail) * c["Hkv"] * (2 * c["D"] + 8 / c["P"]) + rows * (4 * c["D"] + 4),
            "flops": 4 * c["D"] * c["Hq"] * c["Nq"] * (c["B"] * c["prefix"] + tail)}


# ------------------------------------------------------------------ exact

def _turn(x, c, positions, back=False):
    """The rotation of rows x [B, H, N, D] in 64 bits, pair by pair as complex numbers."""
    r, s = c["rot"], SCALINGS[c["scaling"]] or {}
    kind, base, L, k = s.get("kind"), BASES[c["scaling"]], s.get("original_len", 0), s.get("factor", 1.0)
    amp = 1.0 + 0.1 * math.log(k) if kind == "yarn" else 1.0
    y = x.double().clone()
    for i in range(r // 2):
        w = math.exp(-math.log(base) * 2 * i / r)
        if kind == "linear":
            w /= k
        elif kind == "ntk":
            w *= 1.0 if i == 0 else k ** (-2 * i / (r - 2))
        elif kind == "yarn":
            # pairs turning more than 32 times over the original length stay, less than once are stretched
            at = lambda n: 0.5 * r * math.log(L / (2 * math.pi * n), base)
            lo, hi = max(math.floor(at(32)), 0), min(math.ceil(at(1)), r - 1)
            part = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            w = w - w * part * (1 - 1 / k)
        elif kind == "bands":
            wave = 2 * math.pi / w
            if wave > L / s["low"]:
                w /= k
            elif wave > L / s["high"]:
                part = (L / wave - s["low"]) / (s["high"] - s["low"])
                w = w * part + w / k * (1 - part)
        t = (-w if back else w) * positions.double()[:, None]
        j = (2 * i, 2 * i + 1) if c["inter"] else (i, i + r // 2)
        z = torch.complex(x[..., j[0]].double(), x[..., j[1]].double()) * torch.polar(torch.full_like(t, amp), t)
        y[..., j[0]], y[..., j[1]] = z.real, z.imag
    return y


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    if c["op"] in ("rope", "rope_train"):
        res = {n: _turn(st[n].detach(), c, st["positions"]) for n in "qk"}
        if c["op"] == "rope_train":
            res |= {n: _turn(st[n], c, st["positions"], back=True) for n in ("dq", "dk")}
        return res
    if c["op"] == "append_rope":
        return _exact_append(st)
    q, G, P = st["q"], c["Hq"] // c["Hkv"], c["P"]
    res = {"out": torch.zeros(q.shape, device="cuda", dtype=torch.float64),
           "lse": torch.zeros(q.shape[:3], device="cuda", dtype=torch.float64)}
    for b, n in enumerate(st["lens"].tolist()):
        ids = st["table"][b, : -(-n // P)].long()
        seen = torch.ones(c["Nq"], n, dtype=torch.bool, device="cuda").tril(n - c["Nq"])
        for h in range(c["Hkv"]):
            k, v = ((st[p][ids, h].double() * st[s][ids, h].double()[:, None, None]).reshape(-1, c["D"])[:n]
                    for p, s in (("kp", "ks"), ("vp", "vs")))
            s = torch.where(seen, (q[b, h * G:(h + 1) * G].double() @ k.t()) * c["D"] ** -0.5, -math.inf)
            res["out"][b, h * G:(h + 1) * G] = torch.softmax(s, -1) @ v
            res["lse"][b, h * G:(h + 1) * G] = torch.logsumexp(s, -1)
    return res


def _round_e4m3(x):
    """float64 -> the nearest e4m3 value, ties to even: 4 significant bits, spacing at least 2^-9."""
    _, e = torch.frexp(x)
    ulp = (((e.long() - 4).clamp_min(-9) + 1023) << 52).view(torch.float64)
    return (torch.round(x / ulp) * ulp).clamp(-448, 448)


def _exact_pow2(e):
    return ((e.long() + 1023).clamp_min(1) << 52).view(torch.float64)


def _exact_append(st):
    c = st["c"]
    P, res = c["P"], {}
    table, lens, n_new = st["table"].tolist(), st["lens"].tolist(), st["n_new"].tolist()
    if sum(-(-n // P) + 2 for n in n_new) > 2500:
        return None
    at = (st["lens"] - st["n_new"])[:, None] + torch.arange(c["T"], device="cuda")[None]
    res["q"] = _turn(st["q"], c, at)
    for b, n in enumerate(n_new):
        res["q"][b, :, n:] = 0.0
    new = {"kp": _turn(st["k"], c, at), "vp": st["v"].double()}
    for pages, scales in (("kp", "ks"), ("vp", "vs")):
        vals, sc = st[pages].double(), st[scales].double().clone()
        for b in range(c["B"]):
            start = lens[b] - n_new[b]
            if n_new[b] == 0:
                continue
            for j in range(start // P, (lens[b] - 1) // P + 1):
                pid, first, end = table[b][j], max(start, j * P), min(lens[b], (j + 1) * P)
                x = new[pages][b, :, first - start: end - start]
                amax = x.abs().amax(dim=(1, 2))
                e = torch.ceil(torch.log2(amax.clamp_min(1e-300) / 448.0)) + 1    # or one less, or two:
                for _ in range(2):                                                # a logarithm rounds
                    e = torch.where(amax <= 448.0 * _exact_pow2(e - 1), e - 1, e)
                s = _exact_pow2(e.clamp_min(-126))
                o = first - j * P
                if o > 0:
                    s = torch.maximum(s, sc[pid])
                    vals[pid, :, :o] = _round_e4m3(vals[pid, :, :o] * (sc[pid] / s)[:, None, None])
                vals[pid, :, o: end - j * P] = _round_e4m3(x / s[:, None, None])
                sc[pid] = s
        res[pages], res[scales] = vals, sc
    return res
