"""Plain 64-bit forms of the drafted-token and bounded-cache calls, and the
small paged caches that their tests run on."""
from __future__ import annotations

import math

import torch

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}


def q_dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


class PagedCache:
    """K/V caches of random rows with shuffled pages; every row that belongs to no position below T, and every page
    that no such position needs, holds poison (NaN rows; page numbers outside the cache)."""

    def __init__(self, dtype, lens, hkv, d, page, seed=0, spare=40, device="cuda", poison=True):
        g = torch.Generator().manual_seed(seed)
        B, cap = len(lens), max(max(lens), 1) + spare
        self.lens = torch.tensor(lens, dtype=torch.int32, device=device)
        self.T, self.hkv, self.d, self.device = list(lens), hkv, d, device
        if page:
            pages = -(-cap // page)
            self.page, self.cap, slots = page, pages * page, B * pages * page + page
            perm = torch.randperm(B * pages + 1, generator=g)[:B * pages].view(B, pages)
            self.table = perm.to(torch.int32)
        else:
            self.page, self.cap, slots, self.table = cap, cap, B * cap, None
        live = torch.zeros(slots, dtype=torch.bool)
        for b, t in enumerate(lens):
            live[self._slots_cpu(b, torch.arange(t))] = True
        if self.table is not None and poison:  # pages behind the sequence: any number
            for b, t in enumerate(lens):
                for j in range(-(-t // page), self.table.shape[1]):
                    self.table[b, j] = [-1, 2 ** 31 - 1, -2 ** 31, slots][j % 4]
        rows = {}
        for name in ("k", "v"):
            x = torch.randn(slots, hkv, d, generator=g)
            if dtype == "e4m3":
                s = x.abs().amax(-1) / 448 * torch.exp(torch.rand(slots, hkv, generator=g) * 4 - 2)
                x = (x / s.unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn)
                s[~live] = math.nan if poison else 1.0
                rows[name + "_scale"] = s.to(device)
            else:
                x = x.to(DTYPES[dtype])
                rows[name + "_scale"] = None
            if poison:
                if dtype == "e4m3":
                    x.view(torch.uint8)[~live] = 0x7f
                else:
                    x[~live] = math.nan
            rows[name] = x.to(device)
        self.k, self.v, self.k_scale, self.v_scale = rows["k"], rows["v"], rows["k_scale"], rows["v_scale"]
        self.live = live
        if self.table is not None:
            self.table = self.table.to(device)

    def _slots_cpu(self, b, t):
        if self.table is None:
            return b * self.page + t
        return self.table[b, t // self.page].long() * self.page + t % self.page

    def slots(self, b, t):
        t = torch.as_tensor(t, dtype=torch.long, device=self.device)
        if self.table is None:
            return b * self.page + t
        return self.table[b, t // self.page].long() * self.page + t % self.page

    def kw(self):
        return dict(page_table=self.table, page_size=self.page, k_scale=self.k_scale, v_scale=self.v_scale)

    def wide(self, which, b, t):
        """Rows of positions t in 64 bits: [len(t), Hkv, d]."""
        x, s = getattr(self, which), getattr(self, which + "_scale")
        r = self.slots(b, t)
        y = x[r].double()
        return y if s is None else y * s[r].double().unsqueeze(-1)

    def snapshot(self):
        raw = lambda x: None if x is None else x.clone()  # noqa: E731
        return [raw(self.k), raw(self.v), raw(self.k_scale), raw(self.v_scale)]

    def tensors(self):
        return [x for x in (self.k, self.v, self.k_scale, self.v_scale) if x is not None]


def bits(x):
    """The bytes of a tensor, so that NaN equals NaN."""
    return x.contiguous().view(torch.uint8).clone()


def attend(q, k, v, seen, dtype):
    """softmax(q k^T / sqrt d) v over `seen`, zeros where nothing is, and a bound on the kernels' error.
    q [rows, d] (exact values), k, v [T, d] in 64 bits, seen [rows, T].

    The bound.  A logit is a sum of d products in fp32 (any order): off by (d + 2) 2^-24 sum|q k|; over an E4M3 cache
    the query is carried as a sum of two E4M3 numbers scaled to at most 448, off by at most 2^-10 of that scale, that is
    2^-17.8 max|q| (an element below 2^-6 of the scale meets E4M3's subnormal step 2^-9).  Scaling, the base-2 exponent
    (below 2^8 in size here) and the exponential add 2^-14.  A relative error e of every weight moves
    the softmax's output by at most 2 e sum p|v|.  Weights are rounded to bf16 before the product with v, and v's
    scale joins the weight before: 2^-8.  The sum over T in fp32 adds (T + 2) 2^-24, the output's rounding half a step."""
    d = q.shape[1]
    x = q @ k.T / math.sqrt(d)
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    p = torch.softmax(x, -1).nan_to_num(0.0)
    hide = ~seen.any(0)
    v = torch.where(hide.unsqueeze(1), torch.zeros_like(v), v)
    out = p @ v
    kz = torch.where(hide.unsqueeze(1), torch.zeros_like(k), k).abs()
    e = (d + 2) * 2.0 ** -24 * (q.abs() @ kz.T).amax(-1) / math.sqrt(d) if len(k) else torch.zeros(len(q)).to(q)
    if dtype == "e4m3" and len(k):
        e = e + 2.0 ** -17.8 * q.abs().amax(-1) * kz.sum(-1).max() / math.sqrt(d)
    e = e + 2.0 ** -14 + (len(k) + 2) * 2.0 ** -24
    rounding = 0.0 if dtype == "f32" else 2.0 ** -8
    bound = (2 * e.unsqueeze(1) + rounding) * (p @ v.abs()) + HALF_STEP[q_dtype(dtype)] * out.abs() * (1 + 2 ** -6) + 1e-30
    return out, bound, p


def tree_reference(c, q, n, masks, dtype):
    """tree_attn() of q [B, N, Hq, d] over PagedCache c: outputs and bounds [B, N, Hq, d] (NaN: not written)."""
    B, N, Hq, d = q.shape
    G = Hq // c.hkv
    out = torch.full((B, N, Hq, d), math.nan, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    for b in range(B):
        T = max(c.T[b], 0)
        nb = max(0, min(n[b], N, T))
        if nb == 0:
            continue
        first = T - nb
        seen = torch.ones(nb, T, dtype=torch.bool, device=q.device)
        for i in range(nb):
            for j in range(nb):
                seen[i, first + j] = bool(masks[b][i] >> j & 1)
        k, v = c.wide("k", b, torch.arange(T)), c.wide("v", b, torch.arange(T))
        for h in range(Hq):
            out[b, :nb, h], bound[b, :nb, h], _ = attend(q[b, :nb, h].double(), k[:, h // G], v[:, h // G], seen, dtype)
    return out, bound


def inv_freq(rot, base, scaling=None, factor=1.0, original_context=0.0, beta_fast=32.0, beta_slow=1.0,
             low_freq_factor=1.0, high_freq_factor=4.0):
    """Radians per position of each pair, in 64 bits, and the factor on the rotated values."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        lo, hi = (rot * math.log(original_context / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (beta_fast, beta_slow))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    if scaling == "bands":
        turns = original_context * f / (2 * math.pi)
        s = ((turns - low_freq_factor) / (high_freq_factor - low_freq_factor)).clamp(0, 1)
        return (1 - s) * f / factor + s * f, 1.0
    return f, 1.0


def rotate(x, positions, f, scale, interleaved):
    """x [B, N, H, d] in 64 bits, rotated on its first 2 len(f) elements."""
    rot = 2 * len(f)
    a = positions.double().unsqueeze(-1) * f.to(x.device)
    cos, sin = (torch.cos(a) * scale).unsqueeze(2), (torch.sin(a) * scale).unsqueeze(2)
    y = x.clone()
    if interleaved:
        u, w = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = u * cos - w * sin, w * cos + u * sin
    else:
        u, w = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = u * cos - w * sin, w * cos + u * sin
    return y


def kept_positions(sums, T, budget, window):
    """Positions kept of a unit whose sums are a list of floats: the window and the largest others, ties to the lower
    position, NaN below everything."""
    if T <= budget:
        return list(range(T))
    n = T - window
    order = sorted(range(n), key=lambda t: (math.isnan(sums[t]), 0.0 if math.isnan(sums[t]) else -sums[t], t))
    return sorted(order[:budget - window]) + list(range(n, T))
