"""Measured cases of the draft-and-verify and cache-eviction operators.

Five operators around the shared K/V cache of a Hybrid Block:

  rope_append   rotary positions on the queries and keys of new tokens, whose K/V rows go into the cache
  tree_attn     attention of a tree of drafted tokens over the whole cache and their own ancestors
  tree_accept   the accepted path's rows move to the front of the draft
  accumulate    the full layer's attention, its weights added to a running sum per cached token
  evict         the tokens with the largest sums stay, in order, at the front of the cache

`own` chooses between the plain form (elementary torch operations in 32 bits) and the library's calls.
"""
import math

import numpy as np
import torch

own = False

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}


def listed():
    base = {"hkv": 4, "group": 8, "dim": 128, "dtype": "bf16", "page": 64}
    return [
        # one decoded token per sequence of a small batch: the smallest append, where latency counts
        dict(base, name="rope_decode_b4", op="rope_append", batch=4, tokens=1, lo=262144, hi=262144, rot=128,
             interleaved=False, scaling="none"),
        # a prefill chunk over a quantised cache: half of each head rotated, positions scaled for a long context
        dict(base, name="rope_prefill_e4m3", op="rope_append", dtype="e4m3", batch=3, tokens=4001, lo=4001, hi=131072,
             rot=64, interleaved=True, scaling="yarn"),
        # eight drafted tokens verified at the headline context
        dict(base, name="tree_256k_n8", op="tree_attn", batch=4, tokens=8, lo=262144, hi=262144),
        # a full tree of 64 drafts: as many rows as a small prefill, bound by the matrix products
        dict(base, name="tree_32k_n64", op="tree_attn", batch=8, tokens=64, lo=32768, hi=32768),
        # one long conversation over a quantised cache
        dict(base, name="tree_1m_e4m3_n16", op="tree_attn", dtype="e4m3", batch=1, tokens=16, lo=1048576, hi=1048576),
        # the small parity configuration in fp32, an odd draft
        dict(base, name="tree_2k_f32_n5", op="tree_attn", dtype="f32", hkv=1, group=4, dim=64, page=0, batch=1, tokens=5,
             lo=2048, hi=2048),
        # after a verification: a short path of a small batch, and long paths of a large one
        dict(base, name="accept_b4_n8", op="tree_accept", batch=4, tokens=8, lo=8192, hi=8192),
        dict(base, name="accept_b64_n64_e4m3", op="tree_accept", dtype="e4m3", batch=64, tokens=64, lo=1000, hi=8191),
        # the full layer's step with its running sums, at the headline context and for short ragged sequences
        dict(base, name="accumulate_256k", op="accumulate", batch=4, tokens=1, lo=262144, hi=262144),
        dict(base, name="accumulate_ragged_e4m3", op="accumulate", dtype="e4m3", batch=13, tokens=1, lo=777, hi=9001),
        # halving a 64K cache; a quantised, ragged batch trimmed to a small budget
        dict(base, name="evict_64k_to_32k", op="evict", batch=4, tokens=1, lo=65536, hi=65536, budget=32768, window=128),
        dict(base, name="evict_b24_e4m3", op="evict", dtype="e4m3", batch=24, tokens=1, lo=900, hi=12000, budget=2049,
             window=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rope_append", "tree_attn", "tree_attn", "tree_accept", "accumulate", "evict"])
    dtype = rng.choice(["bf16", "bf16", "e4m3", "f32"] if op != "evict" else ["bf16", "e4m3"])
    group = rng.choice([1, 2, 4, 8] if dtype == "f32" else [1, 2, 4, 8, 8, 16, 32])
    c = {"op": op, "dtype": dtype, "group": group, "hkv": rng.choice([1, 2, 4, 8] if group < 16 else [1, 2]),
         "dim": 128 if dtype == "e4m3" else rng.choice([64, 128, 128]), "page": rng.choice([0, 16, 32, 64, 128, 64]),
         "batch": _log(rng, 1, 32), "tokens": 1}
    hi = _log(rng, 64, 65536 if dtype == "f32" else 262144)  # fp32 caches serve short contexts
    if op == "rope_append":
        c["tokens"] = _log(rng, 1, 4096)
        c["batch"] = max(1, min(c["batch"], 12000 // c["tokens"] + 1))
        c["rot"] = rng.choice([c["dim"], c["dim"] // 2, 48])
        c["interleaved"] = rng.random() < 0.5
        c["scaling"] = rng.choice(["none", "linear", "ntk", "yarn", "bands"])
        hi = max(c["tokens"], min(hi, 2 ** 17))
    elif op in ("tree_attn", "tree_accept"):
        c["tokens"] = _log(rng, 1, 64)
    row = c["hkv"] * c["dim"] * SIZE[dtype] * 2
    while True:  # no more than the largest listed cases
        rows = c["batch"] * hi
        flops = 4.0 * c["tokens"] * group * c["hkv"] * c["dim"] * rows if op == "tree_attn" else 0.0
        if rows * row <= 1.5e9 and rows * c["hkv"] * 8 <= 1.2e9 and flops <= (2.0e10 if dtype == "f32" else 2.5e11):
            break
        hi = hi * 3 // 4
    c["hi"] = max(hi, c["tokens"], 2)
    c["lo"] = rng.choice([c["hi"], _log(rng, max(1, min(c["tokens"], c["hi"])), c["hi"])])
    if op == "evict":
        c["window"] = rng.choice([0, 1, 128, 77])
        c["budget"] = max(c["window"] + 1, _log(rng, 16, max(17, c["hi"] - 1)))
    return c


# ---------------------------------------------------------------- shapes
def lengths(c):
    """Tokens in the cache of each sequence, the new ones among them: spread from lo to hi."""
    b, lo, hi = c["batch"], c["lo"], c["hi"]
    return [hi if b == 1 else lo + (hi - lo) * i // (b - 1) for i in range(b)]


def new_tokens(c):
    """New tokens of each sequence: `tokens`, fewer for every third sequence of a larger batch."""
    return [min(t, max(1, c["tokens"] - (c["tokens"] // 3 if i % 3 == 2 else 0))) for i, t in enumerate(lengths(c))]


def capacity(c):
    """(page size, pages per sequence, slots): a page size of 0 is the contiguous layout."""
    hi = max(lengths(c)) + 1
    if not c["page"]:
        cap = -(-hi // 64) * 64
        return cap, 1, cap * c["batch"]
    pages = -(-hi // c["page"])
    return c["page"], pages, pages * c["page"] * c["batch"]


def work(c):
    es, d, hkv, g = SIZE[c["dtype"]], c["dim"], c["hkv"], c["group"]
    row = hkv * (d * es + (4 if es == 1 else 0)) * 2  # K and V of one token
    qrow = hkv * g * d * (4 if es == 4 else 2)
    T, n = lengths(c), new_tokens(c)
    if c["op"] == "rope_append":
        kv_in = 2 * hkv * d * (4 if es == 4 else 2)
        return {"bytes": sum(n) * (2 * qrow + kv_in + row + 4), "flops": sum(n) * hkv * (g + 1) * 3 * c["rot"]}
    if c["op"] == "tree_attn":
        return {"bytes": sum(T) * row + sum(n) * (2 * qrow + 8),
                "flops": sum(4.0 * t * k * hkv * g * d for t, k in zip(T, n))}
    if c["op"] == "tree_accept":
        a = [max(1, k // 2) for k in n]
        return {"bytes": sum(2 * k * row + 4 * k for k in a), "flops": 0}
    if c["op"] == "accumulate":
        return {"bytes": sum(T) * (row + 8 * hkv) + 2 * c["batch"] * qrow, "flops": sum(4.0 * t * hkv * g * d for t in T)}
    moved = [min(t, c["budget"]) if t > c["budget"] else 0 for t in T]
    return {"bytes": sum(2 * m * row + 8 * hkv * m for m in moved) + sum(4 * hkv * t for t in T) +
            4 * hkv * c["batch"] * c["budget"], "flops": 0}


# ---------------------------------------------------------------- inputs
def _quantise(x):
    s = x.abs().amax(-1) / 448.0
    s = torch.where(s > 0, s, torch.ones_like(s))
    return (x / s.unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn), s


def _rows(shape, dtype, gen):
    if dtype != "e4m3":
        return torch.randn(shape, device="cuda", generator=gen, dtype=TORCH[dtype]), None
    x = torch.empty(shape, device="cuda", dtype=torch.float8_e4m3fn)
    s = torch.empty(shape[:2], device="cuda")
    for i in range(0, shape[0], 1 << 18):
        x[i:i + (1 << 18)], s[i:i + (1 << 18)] = _quantise(
            torch.randn((min(1 << 18, shape[0] - i),) + shape[1:], device="cuda", generator=gen))
    return x, s


def _trees(c, seed):
    """Ancestor-or-self bits of a random tree per sequence: drafted token i continues an earlier one, or the context."""
    r = np.random.RandomState(seed % (1 << 31))
    m = np.zeros((c["batch"], c["tokens"]), np.uint64)
    for b in range(c["batch"]):
        for i in range(c["tokens"]):
            p = i - 1 if r.rand() < 0.5 else r.randint(-1, i) if i else -1
            m[b, i] = (m[b, p] if p >= 0 else np.uint64(0)) | np.uint64(1 << i)
    return m


def _paths(c, seed):
    """The accepted drafts of each sequence, ascending: half of its draft."""
    r = np.random.RandomState(seed % (1 << 31))
    p, a = np.zeros((c["batch"], c["tokens"]), np.int32), []
    for b, n in enumerate(new_tokens(c)):
        a.append(max(1, n // 2))
        p[b, :a[-1]] = np.sort(r.choice(n, a[-1], replace=False))
    return p, a


ROPE = {  # base, scaling and its numbers
    "none": dict(base=500000.0),
    "linear": dict(base=10000.0, scaling="linear", factor=8.0),
    "ntk": dict(base=10000.0, scaling="ntk", factor=4.0),
    "yarn": dict(base=10000.0, scaling="yarn", factor=32.0, original_context=4096, beta_fast=32.0, beta_slow=1.0),
    "bands": dict(base=500000.0, scaling="bands", factor=8.0, original_context=8192, low_freq_factor=1.0,
                  high_freq_factor=4.0),
}


def _inv_freq(c):
    """Radians per position of each rotated pair, in 64 bits, and the factor on the rotated values."""
    r, rot = ROPE[c["scaling"]], c["rot"]
    i = np.arange(rot // 2, dtype=np.float64)
    f = r["base"] ** (-2.0 * i / rot)
    if c["scaling"] == "linear":
        f = f / r["factor"]
    if c["scaling"] == "ntk":
        f = (r["base"] * r["factor"] ** (rot / (rot - 2.0))) ** (-2.0 * i / rot)
    if c["scaling"] == "yarn":
        at = [rot * math.log(r["original_context"] / (b * 2 * math.pi)) / (2 * math.log(r["base"]))
              for b in (r["beta_fast"], r["beta_slow"])]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        return f / r["factor"] * ramp + f * (1 - ramp), 0.1 * math.log(r["factor"]) + 1.0
    if c["scaling"] == "bands":
        turns = r["original_context"] * f / (2 * math.pi)
        s = np.clip((turns - r["low_freq_factor"]) / (r["high_freq_factor"] - r["low_freq_factor"]), 0, 1)
        f = (1 - s) * f / r["factor"] + s * f
    return f, 1.0


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    page, pages, slots = capacity(c)
    T, n = lengths(c), new_tokens(c)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    B, N, hkv, hq, d = c["batch"], c["tokens"], c["hkv"], c["hkv"] * c["group"], c["dim"]
    qt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    s = {"c": c, "page": page, "lens": i32(T), "new": i32(n), "table": None}
    s["k"], s["ks"] = _rows((slots, hkv, d), c["dtype"], gen)
    s["v"], s["vs"] = _rows((slots, hkv, d), c["dtype"], gen)
    if c["page"]:
        s["table"] = torch.randperm(B * pages, device="cuda", generator=gen).to(torch.int32).view(B, pages)
    randn = lambda *shape: torch.randn(shape, device="cuda", generator=gen).to(qt)  # noqa: E731
    if c["op"] == "rope_append":
        # one projection's output: the queries, keys and values of a token side by side
        s["qkv"] = randn(B, N, hq + 2 * hkv, d)
        s["q_out"] = torch.zeros(B, N, hq, d, dtype=qt, device="cuda")
        first = torch.tensor([t - k for t, k in zip(T, n)], device="cuda")
        s["pos"] = (first[:, None] + torch.arange(N, device="cuda")).to(torch.int32)
        f, s["mscale"] = _inv_freq(c)
        s["freq"] = torch.from_numpy(f).cuda()
        if own:
            from long_context_decode_full_b200 import hs2
            s["rope"] = hs2.rope_table(c["rot"], interleaved=c["interleaved"], **ROPE[c["scaling"]])
    elif c["op"] == "tree_attn":
        s["q"] = randn(B, N, hq, d)
        s["mask"] = torch.from_numpy(_trees(c, seed).view(np.int64)).cuda()
        s["out"] = torch.zeros(B, N, hq, d, dtype=qt, device="cuda")
        if own:
            from long_context_decode_full_b200 import hs2
            s["ws"] = hs2.alloc_tree_workspace(s["q"], s["k"])
    elif c["op"] == "tree_accept":
        p, a = _paths(c, seed)
        s["path"], s["path_len"] = torch.from_numpy(p).cuda(), i32(a)
    elif c["op"] == "accumulate":
        s["q"] = randn(B, hq, d)
        # sums of some hundred earlier steps
        s["acc"] = torch.rand(B, hkv, page * pages, device="cuda", generator=gen) * (300.0 * c["group"] / max(T))
        if own:
            from long_context_decode_full_b200 import hs2
            s["ws"] = hs2.alloc_workspace(B, hkv, c["group"], d, page * pages)
    else:
        # attention weight is heavy-tailed, and much of it underflows to zero: many equal sums
        x = torch.exp(3.0 * torch.randn(B, hkv, page * pages, device="cuda", generator=gen))
        s["acc"] = torch.where(x < 0.2, torch.zeros_like(x), x / max(T))
        s["kept"] = torch.full((B, hkv, c["budget"]), -1, dtype=torch.int32, device="cuda")
    s["lens_out"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return (_own if own else _plain)[s["c"]["op"]](s)


def _slots(s, t):
    """Cache rows of positions t [B, ...] of each sequence."""
    b = torch.arange(t.shape[0], device=t.device).view((-1,) + (1,) * (t.dim() - 1))
    if s["table"] is None:
        return b * s["page"] + t
    return s["table"][b, t // s["page"]].long() * s["page"] + t % s["page"]


def _f32(x, scale, rows):
    y = x[rows].float()
    return y if scale is None else y * scale[rows].unsqueeze(-1)


def _caches(s):
    return [s["k"], s["v"]] + ([] if s["ks"] is None else [s["ks"], s["vs"]])


def _rope_plain(s):
    c, x = s["c"], s["qkv"].float()
    hq, hkv, rot = c["hkv"] * c["group"], c["hkv"], c["rot"]
    angle = s["pos"].double().unsqueeze(-1) * s["freq"]  # far positions lose their angle in 32 bits
    cos, sin = ((f(angle) * s["mscale"]).float().unsqueeze(2) for f in (torch.cos, torch.sin))
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["interleaved"] else (x[..., :rot // 2], x[..., rot // 2:rot])
    y = (a * cos - b * sin, b * cos + a * sin)
    y = torch.stack(y, -1).flatten(-2) if c["interleaved"] else torch.cat(y, -1)
    y = torch.cat([y, x[..., rot:]], -1)
    i = torch.arange(c["tokens"], device=x.device)
    here = i < s["new"].unsqueeze(1)  # the tokens that there are
    s["q_out"] = torch.where(here[:, :, None, None], y[:, :, :hq].to(s["q_out"].dtype), s["q_out"])
    t = (s["lens"] - s["new"]).unsqueeze(1) + torch.where(here, i, 0)
    rows = _slots(s, t.long())[here]
    for name, new in (("k", y[:, :, hq:hq + hkv][here]), ("v", x[:, :, hq + hkv:][here])):
        if s["ks"] is None:
            s[name][rows] = new.to(s[name].dtype)
        else:
            code, scale = _quantise(new)
            s[name].view(torch.uint8)[rows] = code.view(torch.uint8)
            s[name + "s"][rows] = scale
    return [s["q_out"]] + _caches(s)


def _rope_own(s):
    from long_context_decode_full_b200 import hs2
    c = s["c"]
    hq = c["hkv"] * c["group"]
    x = s["qkv"]
    hs2.rope_append(x[:, :, :hq], x[:, :, hq:hq + c["hkv"]], x[:, :, hq + c["hkv"]:], s["pos"], s["rope"], s["k"], s["v"],
                    s["lens"], s["table"], s["page"], num_new=s["new"], k_scale=s["ks"], v_scale=s["vs"], q_out=s["q_out"])
    return [s["q_out"]] + _caches(s)


def _attend(q, k, v, seen, scale):
    """softmax(q k^T scale) v over what is seen, zeros where nothing is; q [B, h, rows, d], seen [B, 1, rows, T]."""
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    l = x.sum(-1, keepdim=True)
    x = x.div_(torch.where(l > 0, l, torch.ones_like(l)))
    return torch.matmul(x, v), x


def _tree_plain(s):
    c = s["c"]
    B, N, hkv, g, d = c["batch"], c["tokens"], c["hkv"], c["group"], c["dim"]
    t = torch.arange(max(lengths(c)), device="cuda")
    rows = _slots(s, t.expand(B, -1))
    k, v = (_f32(x, sc, rows).transpose(1, 2) for x, sc in ((s["k"], s["ks"]), (s["v"], s["vs"])))
    j = t - (s["lens"] - s["new"]).unsqueeze(1)  # place in the draft; the context's are below 0
    seen = (s["mask"].unsqueeze(2) >> j.clamp(0, 63).unsqueeze(1)) & 1 > 0
    seen = (j < 0).unsqueeze(1) | (seen & (j < s["new"].unsqueeze(1)).unsqueeze(1))
    q = s["q"].float().view(B, N, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, N * g, d)
    o, _ = _attend(q, k, v, seen.repeat_interleave(g, 1).unsqueeze(1), 1.0 / math.sqrt(d))
    o = o.view(B, hkv, N, g, d).permute(0, 2, 1, 3, 4).reshape(B, N, hkv * g, d).to(s["out"].dtype)
    here = torch.arange(N, device="cuda") < s["new"].unsqueeze(1)
    s["out"] = torch.where(here[:, :, None, None], o, s["out"])
    return s["out"]


def _tree_own(s):
    from long_context_decode_full_b200 import hs2
    return hs2.tree_attn(s["q"], s["k"], s["v"], s["lens"], s["table"], s["page"], tree_mask=s["mask"], num_draft=s["new"],
                         k_scale=s["ks"], v_scale=s["vs"], out=s["out"], workspace=s["ws"])


def _bytes(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _accept_plain(s):
    first = (s["lens"] - s["new"]).unsqueeze(1)
    i = torch.arange(s["path"].shape[1], device="cuda")
    here = i < s["path_len"].unsqueeze(1)
    src, dst = _slots(s, (first + s["path"]).long())[here], _slots(s, (first + torch.where(here, i, 0)).long())[here]
    for x in _caches(s):
        _bytes(x)[dst] = _bytes(x)[src]
    s["lens_out"] = (first.squeeze(1) + s["path_len"]).to(torch.int32)
    return [s["lens_out"]] + _caches(s)


def _accept_own(s):
    from long_context_decode_full_b200 import hs2
    hs2.tree_accept(s["k"], s["v"], s["lens"], s["path"], s["path_len"], s["table"], s["page"], num_draft=s["new"],
                    k_scale=s["ks"], v_scale=s["vs"], lens_out=s["lens_out"])
    return [s["lens_out"]] + _caches(s)


DECAY = 0.96875


def _accumulate_plain(s):
    c = s["c"]
    B, hkv, g, d = c["batch"], c["hkv"], c["group"], c["dim"]
    t = torch.arange(max(lengths(c)), device="cuda")
    rows = _slots(s, t.expand(B, -1))
    k, v = (_f32(x, sc, rows).transpose(1, 2) for x, sc in ((s["k"], s["ks"]), (s["v"], s["vs"])))
    seen = t < s["lens"].unsqueeze(1)
    o, p = _attend(s["q"].float().view(B, hkv, g, d), k, v, seen[:, None, None], 1.0 / math.sqrt(d))
    w = p.sum(2)
    old = s["acc"][:, :, :len(t)]
    new = torch.where((t == s["lens"].unsqueeze(1) - 1)[:, None], w, DECAY * old + w)  # the newest token's sum starts
    s["acc"][:, :, :len(t)] = torch.where(seen[:, None], new, old)
    return [o.reshape(B, hkv * g, d).to(s["q"].dtype), s["acc"]]


def _accumulate_own(s):
    from long_context_decode_full_b200 import hs2
    out, acc = hs2.full_attn_accumulate(s["q"], s["k"], s["v"], s["lens"], s["acc"], s["table"], s["page"], decay=DECAY,
                                        k_scale=s["ks"], v_scale=s["vs"], workspace=s["ws"])
    return [out, acc]


def _evict_plain(s):
    c = s["c"]
    B, hkv, W, K = c["batch"], c["hkv"], c["window"], c["budget"]
    T = s["lens"].long().view(B, 1, 1)
    over = T > K
    t = torch.arange(max(lengths(c)), device="cuda")
    a = s["acc"][:, :, :len(t)]
    # the window first, then the largest sums, ties to the lower position; everything where there is room
    key = torch.where(t >= T, -math.inf, torch.where(t >= T - W, math.inf, a))
    best = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :, :K]
    none = torch.full_like(best, 1 << 40)
    i = torch.arange(best.shape[2], device="cuda")
    pos = torch.sort(torch.where(over | (i < T), torch.where(over, best, i), none), dim=-1).values
    here = pos < (1 << 40)
    s["kept"] = torch.full((B, hkv, K), -1, dtype=torch.int32, device="cuda")
    s["kept"][:, :, :pos.shape[2]] = torch.where(here, pos, -1).to(torch.int32)
    b, h, i = torch.nonzero(here & over, as_tuple=True)
    p = pos[b, h, i]
    slot = lambda q: b * s["page"] + q if s["table"] is None else s["table"][b, q // s["page"]].long() * s["page"] + q % s["page"]  # noqa: E731
    src, dst = slot(p), slot(i)
    for x in _caches(s):
        _bytes(x)[dst, h] = _bytes(x)[src, h]
    s["acc"][b, h, i] = s["acc"][b, h, p]
    s["lens_out"] = s["lens"].clamp(max=K)
    return [s["lens_out"], s["kept"], s["acc"]] + _caches(s)


def _evict_own(s):
    from long_context_decode_full_b200 import hs2
    hs2.cache_evict(s["k"], s["v"], s["lens"], s["acc"], s["c"]["budget"], s["c"]["window"], s["table"], s["page"],
                    k_scale=s["ks"], v_scale=s["vs"], kept=s["kept"], lens_out=s["lens_out"])
    return [s["lens_out"], s["kept"], s["acc"]] + _caches(s)


_plain = {"rope_append": _rope_plain, "tree_attn": _tree_plain, "tree_accept": _accept_plain,
          "accumulate": _accumulate_plain, "evict": _evict_plain}
_own = {"rope_append": _rope_own, "tree_attn": _tree_own, "tree_accept": _accept_own, "accumulate": _accumulate_own,
        "evict": _evict_own}


# ---------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c, T, n = s["c"], lengths(case), new_tokens(case)
    page = s["page"]
    at = lambda b, t: b * page + t if s["table"] is None else s["table"][b].long()[t // page] * page + t % page  # noqa: E731
    wide = lambda x, sc, r, h: x[r, h].double() * (1.0 if sc is None else sc[r, h].double().unsqueeze(-1))  # noqa: E731
    values = [x.double() for x in _caches(s)]
    d, g, hkv = c["dim"], c["group"], c["hkv"]
    if c["op"] == "rope_append":
        x, hq, rot = s["qkv"].double(), hkv * g, c["rot"]
        z = torch.polar(torch.full_like(s["freq"], s["mscale"]).expand(c["batch"], c["tokens"], -1).contiguous(),
                        s["pos"].double().unsqueeze(-1) * s["freq"]).unsqueeze(2)
        y = x[:, :, :hq + hkv]  # the values stay as they are
        part = y[..., :rot].unflatten(-1, (rot // 2, 2) if c["interleaved"] else (2, rot // 2))
        part = part if c["interleaved"] else part.transpose(-1, -2)
        part = torch.view_as_real(torch.view_as_complex(part.contiguous()) * z)
        y[..., :rot] = (part if c["interleaved"] else part.transpose(-1, -2)).flatten(-2)
        q_out = s["q_out"].double()
        for b in range(c["batch"]):
            q_out[b, :n[b]] = x[b, :n[b], :hq]
            r = at(b, torch.arange(T[b] - n[b], T[b], device="cuda"))
            for w, new in enumerate((x[b, :n[b], hq:hq + hkv], x[b, :n[b], hq + hkv:])):
                if c["dtype"] == "e4m3":
                    values[2 + w][r] = new.abs().amax(-1) / 448.0
                    new = new / values[2 + w][r].unsqueeze(-1)
                values[w][r] = new
        return [q_out] + values
    if c["op"] in ("tree_attn", "accumulate"):
        tree = c["op"] == "tree_attn"
        out = s["out"].double() if tree else torch.zeros(c["batch"], hkv * g, d, dtype=torch.float64, device="cuda")
        acc = None if tree else s["acc"].double()
        bits = _trees(case, seed) if tree else None
        for b in range(c["batch"]):
            r = at(b, torch.arange(T[b], device="cuda"))
            for h in range(hkv):
                k, v = wide(s["k"], s["ks"], r, h), wide(s["v"], s["vs"], r, h)
                if not tree:
                    p = torch.softmax(s["q"][b, h * g:(h + 1) * g].double() @ k.T / math.sqrt(d), -1)
                    out[b, h * g:(h + 1) * g] = p @ v
                    acc[b, h, :T[b] - 1] *= DECAY
                    acc[b, h, T[b] - 1] = 0
                    acc[b, h, :T[b]] += p.sum(0)
                    continue
                for i0 in range(0, n[b], 16):
                    i1 = min(n[b], i0 + 16)
                    x = torch.einsum("igd,td->igt", s["q"][b, i0:i1, h * g:(h + 1) * g].double(), k) / math.sqrt(d)
                    hide = torch.tensor([[not int(bits[b, i]) >> j & 1 for j in range(n[b])] for i in range(i0, i1)], device="cuda")
                    x[:, :, T[b] - n[b]:].masked_fill_(hide.unsqueeze(1), -math.inf)
                    out[b, i0:i1, h * g:(h + 1) * g] = torch.softmax(x, -1).nan_to_num() @ v
        return out if tree else [out, acc]
    if c["op"] == "tree_accept":
        p, a = _paths(case, seed)
        for b in range(c["batch"]):
            first = T[b] - n[b]
            src = at(b, torch.from_numpy(p[b, :a[b]]).long().cuda() + first)
            dst = at(b, torch.arange(first, first + a[b], device="cuda"))
            values = [x.index_copy(0, dst, x[src]) for x in values]
        return [None] + values
    acc, K, W = s["acc"].double(), c["budget"], c["window"]
    for b in range(c["batch"]):
        if T[b] <= K:
            continue
        for h in range(hkv):
            sums = s["acc"][b, h, :T[b] - W]
            least = torch.topk(sums, K - W).values.min() if K > W else math.inf
            take = sums > least
            equal = torch.nonzero(sums == least).flatten()[:K - W - int(take.sum())]
            take[equal] = True
            pos = torch.cat([torch.nonzero(take).flatten(), torch.arange(T[b] - W, T[b], device="cuda")])
            src, dst = at(b, pos), at(b, torch.arange(K, device="cuda"))
            for x in values:
                x[dst, h] = x[src, h].clone()
            acc[b, h, :K] = acc[b, h, pos]
    return [None, None, acc] + values
