"""The drafted-token and bounded-cache calls on the GPU against plain 64-bit forms (tests/draft_ref.py)."""
import math

import pytest
import torch

import draft_ref as R
from long_context_decode_full_b200 import hs2

pytestmark = pytest.mark.gpu
NAN = float("nan")


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def random_tree(n, seed):
    r = torch.Generator().manual_seed(seed)
    return [(i - 1 if torch.rand((), generator=r) < 0.5 else int(torch.randint(-1, i, (), generator=r))) if i else -1
            for i in range(n)]


def mask_words(parents):
    m = []
    for i, p in enumerate(parents):
        m.append((m[p] if p >= 0 else 0) | 1 << i)
    return m


def signed(words):
    return [[x - (1 << 64) if x >> 63 else x for x in row] for row in words]


def check(got, want, bound, written):
    """Within the bound where written, else still the sentinel."""
    got = got.double()
    err = (got - want).abs()
    ok = (err <= bound) | ~written
    assert bool(ok.all()), f"worst excess {float((err - bound)[written].max()):.3g} at {(~ok).nonzero()[0].tolist()}"
    assert bool((got[~written] == 77.0).all())


# ---------------------------------------------------------------- tree attention
TREES = [
    # dtype, hkv, G, d, page, N, lens, drafts
    ("bf16", 2, 8, 128, 64, 8, [513, 1, 0, 130], [8, 1, 8, 5]),
    ("bf16", 1, 8, 128, 16, 64, [64, 300, 127], [64, 64, 33]),
    ("bf16", 1, 32, 128, 0, 13, [1000, 14], [13, 13]),
    ("bf16", 2, 4, 64, 32, 64, [65, 1537, 128], [64, 63, 64]),
    ("bf16", 4, 1, 64, 128, 1, [1, 2, 129, 4097], [1, 1, 1, 0]),
    ("bf16", 1, 16, 64, 0, 31, [31, 255, 256, 257], [31, 31, 1, 30]),
    ("bf16", 1, 32, 128, 64, 64, [777, 70], [64, 50]),
    ("bf16", 3, 2, 128, 192, 5, [900, 385], [5, 5]),
    ("e4m3", 2, 8, 128, 64, 16, [700, 16, 0, 129], [16, 16, 3, 9]),
    ("e4m3", 1, 32, 128, 16, 40, [41, 333], [40, 40]),
    ("e4m3", 2, 1, 128, 0, 3, [5000, 3], [3, 1]),
    ("e4m3", 1, 16, 128, 32, 64, [2049, 64, 65], [64, 64, 1]),
    ("f32", 1, 4, 64, 0, 5, [2048, 5, 6], [5, 5, 0]),
    ("f32", 2, 8, 128, 48, 33, [100, 33, 511], [33, 33, 20]),
    ("f32", 2, 1, 64, 16, 64, [64, 1, 700], [64, 1, 64]),
    ("f32", 2, 4, 128, 64, 4, [3000, 4, 0, 65], [4, 4, 1, 3]),
    ("f32", 3, 1, 64, 16, 16, [129, 16, 20000], [16, 9, 16]),
    ("f32", 1, 8, 128, 0, 1, [5000, 1], [1, 1]),
    ("f32", 1, 4, 128, 128, 8, [900, 31], [8, 5]),
]


def tree_case(dtype, hkv, G, d, page, N, lens, drafts, seed=0, masks=None):
    c = R.PagedCache(dtype, lens, hkv, d, page, seed)
    q = torch.randn(len(lens), N, hkv * G, d, device="cuda", generator=gen(seed)).to(R.q_dtype(dtype))
    if masks is None:
        masks = [mask_words(random_tree(N, seed + b)) for b in range(len(lens))]
    return c, q, masks, torch.tensor(signed(masks), device="cuda")


@pytest.mark.parametrize("case", TREES, ids=lambda c: "-".join(str(x) for x in c[:6]))
def test_tree_attn(case):
    dtype, hkv, G, d, page, N, lens, drafts = case
    c, q, masks, words = tree_case(*case, seed=5)
    want, bound = R.tree_reference(c, q, drafts, masks, dtype)
    written = ~want.isnan()
    out = torch.full_like(q, 77.0)
    ws = hs2.alloc_tree_workspace(q, c.k)
    ws[256:].random_(0, 256)  # results do not depend on what the workspace holds
    before = [R.bits(x) for x in c.tensors()]
    hs2.tree_attn(q, c.k, c.v, c.lens, tree_mask=words, num_draft=i32(drafts), out=out, workspace=ws, **c.kw())
    check(out, want, bound, written)
    assert all(torch.equal(R.bits(x), y) for x, y in zip(c.tensors(), before))
    again = torch.full_like(q, 77.0)  # the same bits from a used workspace
    hs2.tree_attn(q, c.k, c.v, c.lens, tree_mask=words, num_draft=i32(drafts), out=again, workspace=ws, **c.kw())
    assert torch.equal(R.bits(again), R.bits(out))


@pytest.mark.parametrize("dtype,d,G", [("bf16", 128, 8), ("bf16", 64, 2), ("e4m3", 128, 8), ("f32", 64, 4)])
def test_tree_attn_rows_that_see_nothing_and_poisoned_drafts(dtype, d, G):
    """Masks that leave a row empty, lengths of the draft alone, and drafts whose rows hold infinities and NaN."""
    N, lens = 40, [40, 40, 200]
    masks = [[0] * N for _ in lens]
    for b in range(3):
        for i in range(N):
            masks[b][i] = (1 << i | 1 << 3) if i % 5 else 0
            if i == 3:
                masks[b][i] = 1 << 3
    masks[1] = [m | ~((1 << N) - 1) & (1 << 64) - 1 for m in masks[1]]  # bits behind the draft mean nothing
    c, q, masks, words = tree_case(dtype, 2, G, d, 16, N, lens, [N] * 3, seed=9, masks=masks)
    bad = [7, 8, 9, 21]  # seen by themselves alone
    for b in range(3):
        first = lens[b] - N
        s = c.slots(b, [first + j for j in bad])
        if dtype == "e4m3":
            c.v.view(torch.uint8)[s[0], :, 5] = 0x7f
            c.k.view(torch.uint8)[s[1], :, 100] = 0xff
            c.v_scale[s[2]] = math.inf
            c.k_scale[s[3]] = NAN
        else:
            c.v[s[0], :, 5] = NAN
            c.k[s[1], :, 60] = -math.inf
            c.v[s[2], :, :3] = math.inf
            c.k[s[3]] = NAN
    clean = R.PagedCache(dtype, lens, 2, d, 16, 9)
    want, bound = R.tree_reference(clean, q, [N] * 3, masks, dtype)
    out = torch.full_like(q, 77.0)
    hs2.tree_attn(q, c.k, c.v, c.lens, tree_mask=words, out=out, **c.kw())
    sees_bad = torch.tensor([[any(masks[b][i] >> j & 1 for j in bad) for i in range(N)] for b in range(3)], device="cuda")
    good = ~sees_bad[:, :, None, None].expand_as(out)
    err = (out.double() - want).abs()
    assert bool((err <= bound)[good].all())
    empty = torch.tensor([i % 5 == 0 for i in range(N)], device="cuda")
    assert bool((out[:2, empty] == 0).all())
    # a bad value that is seen is seen: NaN or infinity in its elements alone
    assert bool(out[:, 7, :, 5].isnan().all())
    if dtype == "e4m3":
        assert bool((~out[:, 9].isfinite() | (out[:, 9] == 0)).all())
    else:
        assert bool((out[:, 9, :, :3] == math.inf).all()) and bool(out[:, 9, :, 3:].isfinite().all())
        assert bool(out[:, 7, :, :5].isfinite().all())
    assert bool(out[:, 21].isnan().all())


def test_tree_attn_fused_projection_stream_and_default_mask():
    """q and out as slices of wider rows, another stream than the current one, the chain mask, default lengths."""
    dtype, hkv, G, d, N, lens = "bf16", 2, 8, 128, 6, [300, 7]
    c, q, _, _ = tree_case(dtype, hkv, G, d, 64, N, lens, [N, N], seed=2)
    wide_q = torch.full((2, N, hkv * G + 5, d), NAN, device="cuda", dtype=q.dtype)
    wide_q[:, :, 2:2 + hkv * G] = q
    wide_o = torch.full_like(wide_q, 77.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = hs2.tree_attn(wide_q[:, :, 2:2 + hkv * G], c.k, c.v, c.lens, out=wide_o[:, :, 3:3 + hkv * G], stream=s, **c.kw())
    s.synchronize()
    chain = [[(1 << i + 1) - 1 for i in range(N)]] * 2
    want, bound = R.tree_reference(c, q, [N, N], chain, dtype)
    check(out, want, bound, ~want.isnan())
    assert bool((wide_o[:, :, :3] == 77.0).all()) and bool((wide_o[:, :, 3 + hkv * G:] == 77.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
def test_tree_attn_two_streams_and_graph(dtype):
    """Two calls at once on workspaces of their own, and a captured call whose inputs change between replays."""
    case = (dtype, 2, 4, 128, 64, 9, [1000, 400], [9, 7])
    sides = [tree_case(*case, seed=s) for s in (1, 2)]
    outs, streams = [torch.full_like(x[1], 77.0) for x in sides], [torch.cuda.Stream() for _ in sides]
    ws = [hs2.alloc_tree_workspace(x[1], x[0].k) for x in sides]
    nd = i32([9, 7])
    torch.cuda.synchronize()

    def call(i, out, stream=None):
        c, q, _, words = sides[i]
        hs2.tree_attn(q, c.k, c.v, c.lens, tree_mask=words, num_draft=nd, out=out, workspace=ws[i], stream=stream, **c.kw())

    for _ in range(10):
        for i in (0, 1):
            call(i, outs[i], streams[i])
    torch.cuda.synchronize()
    refs = [R.tree_reference(c, q, [9, 7], masks, dtype) for c, q, masks, _ in sides]
    for out, (want, bound) in zip(outs, refs):
        check(out, want, bound, ~want.isnan())
    out = torch.full_like(outs[0], 77.0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(0, out)
    assert bool((out == 77.0).all())
    g.replay()
    check(out, *refs[0], ~refs[0][0].isnan())
    c, q, masks, _ = sides[0]
    q.copy_(sides[1][1])
    c.lens.copy_(i32([500, 9]))
    nd.copy_(i32([4, 9]))
    out.fill_(77.0)
    g.replay()
    c.T = [500, 9]
    want, bound = R.tree_reference(c, q, [4, 9], masks, dtype)
    check(out, want, bound, ~want.isnan())


def test_tree_attn_lengths_and_pages_out_of_range():
    """Lengths beyond the capacity and below zero are clamped; a page outside the cache reads as zeros."""
    c, q, masks, words = tree_case("bf16", 1, 4, 128, 16, 3, [200, 64], [3, 3], seed=4)
    out = torch.full_like(q, 77.0)
    hs2.tree_attn(q, c.k, c.v, i32([-5, -2 ** 31]), tree_mask=words, out=out, **c.kw())
    assert bool((out == 77.0).all())
    hs2.tree_attn(q, c.k, c.v, c.lens, tree_mask=words, num_draft=i32([-1, -2 ** 31]), out=out, **c.kw())
    assert bool((out == 77.0).all())
    table = torch.full_like(c.table, 2 ** 31 - 1)
    table[1, :] = -7
    hs2.tree_attn(q, c.k, c.v, i32([2 ** 31 - 1, 50]), page_table=table, page_size=16, tree_mask=words, out=out)
    assert bool((out == 0).all())


def test_tree_attn_long_context_splits():
    """One long sequence beside short ones: many shares of one unit joined, fp32 sums over 100,000 rows."""
    c, q, masks, words = tree_case("bf16", 1, 8, 128, 64, 8, [100003, 17, 9000], [8, 8, 8], seed=6)
    out = torch.full_like(q, 77.0)
    hs2.tree_attn(q, c.k, c.v, c.lens, tree_mask=words, out=out, **c.kw())
    want, bound = R.tree_reference(c, q, [8] * 3, masks, "bf16")
    check(out, want, bound, ~want.isnan())


@pytest.mark.parametrize("dtype,G,N", [("bf16", 8, 5), ("e4m3", 8, 16), ("bf16", 8, 33), ("e4m3", 16, 20)])
def test_tree_attn_many_units_per_share(dtype, G, N):
    """A large batch of short sequences: shares that hold several whole units of several tiles, and cut ones."""
    lens = [300 + 37 * i % 411 for i in range(60)] + [0, 20000]
    c, q, masks, words = tree_case(dtype, 4, G, 128, 32, N, lens, [N] * len(lens), seed=10)
    out = torch.full_like(q, 77.0)
    hs2.tree_attn(q, c.k, c.v, c.lens, tree_mask=words, out=out, **c.kw())
    want, bound = R.tree_reference(c, q, [N] * len(lens), masks, dtype)
    check(out, want, bound, ~want.isnan())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_tree_attn_growing_and_large_logits(dtype):
    """Logits that grow along the context by hundreds of nats (the running maximum moves at every tile), and shrink."""
    c, q, masks, words = tree_case(dtype, 1, 8, 128, 64, 20, [1500, 1500], [20, 20], seed=8)
    for b, sign in ((0, 1.0), (1, -1.0)):
        t = torch.arange(1500, device="cuda")
        amp = 0.02 * torch.exp(sign * (t.float() / 1500 - int(sign < 0)) * 6) * (1 if sign > 0 else math.exp(-6))
        if dtype == "e4m3":
            c.k_scale[c.slots(b, t)] *= amp.unsqueeze(1) * 4
        else:
            c.k[c.slots(b, t)] *= (amp * 4).to(c.k.dtype).view(-1, 1, 1)
    out = torch.full_like(q, 77.0)
    hs2.tree_attn(q, c.k, c.v, c.lens, tree_mask=words, out=out, **c.kw())
    want, bound = R.tree_reference(c, q, [20] * 2, masks, dtype)
    check(out, want, bound, ~want.isnan())


# ---------------------------------------------------------------- accept
@pytest.mark.parametrize("dtype,hkv,d,page", [("bf16", 4, 128, 64), ("e4m3", 9, 128, 16), ("f32", 1, 64, 0), ("bf16", 3, 64, 32)])
def test_tree_accept(dtype, hkv, d, page):
    N, lens = 64, [64, 500, 0, 129, 10, 77]
    drafts, plen = [64, 64, 64, 40, 64, -3], [32, 64, 5, 3, 70, 4]
    c = R.PagedCache(dtype, lens, hkv, d, page, seed=3)
    g = torch.Generator().manual_seed(1)
    path = torch.stack([torch.randperm(N, generator=g) for _ in lens]).to(torch.int32)  # any order
    path[0, :4] = torch.tensor([5, 5, -1, 64])  # the same row twice, and two that are no drafts
    path[3, :3] = torch.tensor([2, 39, 40])
    before = c.snapshot()
    got = hs2.tree_accept(c.k, c.v, c.lens, path.cuda(), i32(plen), num_draft=i32(drafts), **c.kw())
    want = [None if x is None else x.clone() for x in before]
    new = []
    for b, T in enumerate(lens):
        n = max(0, min(drafts[b], N, T))
        a = max(0, min(plen[b], n))
        new.append(T - n + a)
        for i in range(a):
            j = int(path[b, i])
            if 0 <= j < n:
                src, dst = int(c.slots(b, T - n + j)), int(c.slots(b, T - n + i))
                for x, y in zip(want, before):
                    if x is not None:
                        x[dst] = y[src]
    assert got.tolist() == new
    for x, y in zip((c.k, c.v, c.k_scale, c.v_scale), want):
        assert x is None or torch.equal(R.bits(x), R.bits(y))


# ---------------------------------------------------------------- accumulate
@pytest.mark.parametrize("dtype,hkv,G,d,page,decay,fresh", [
    ("bf16", 2, 8, 128, 64, 0.9, 1), ("e4m3", 1, 16, 128, 32, 1.0, 4), ("f32", 2, 1, 64, 0, 0.0, 0),
    ("bf16", 1, 32, 64, 16, 0.5, 2 ** 31 - 1), ("f32", 1, 8, 128, 16, 0.75, 3),
    ("f32", 3, 2, 128, 48, 0.25, 2), ("f32", 1, 4, 64, 64, 1.0, 1), ("f32", 2, 8, 64, 0, 0.5, 5), ("f32", 5, 1, 128, 16, 0.9, 1)])
def test_full_attn_accumulate(dtype, hkv, G, d, page, decay, fresh):
    lens = [1, 700, 0, 130, 4099]
    c = R.PagedCache(dtype, lens, hkv, d, page, seed=7)
    q = torch.randn(len(lens), hkv * G, d, device="cuda", generator=gen(3)).to(R.q_dtype(dtype))
    acc0 = torch.rand(len(lens), hkv, c.cap + 3, device="cuda", generator=gen(4)) * 5
    for b, T in enumerate(lens):
        acc0[b, :, max(0, T - min(fresh, T)):T] = NAN  # not read
    acc = acc0.clone()
    out, back = hs2.full_attn_accumulate(q, c.k, c.v, c.lens, acc, decay=decay, fresh=fresh, **c.kw())
    assert back is acc
    for b, T in enumerate(lens):
        k, v = c.wide("k", b, torch.arange(T)), c.wide("v", b, torch.arange(T))
        for h in range(hkv):
            rows = q[b, h * G:(h + 1) * G].double()
            o, bound, p = R.attend(rows, k[:, h], v[:, h], torch.ones(G, T, dtype=torch.bool, device="cuda"), dtype)
            tol = {"f32": 1e-3, "bf16": 2e-2, "e4m3": 6e-2}[dtype]  # the attention's own, as in its tests
            assert T == 0 or float((out[b, h * G:(h + 1) * G].double() - o).abs().max()) <= tol
            old = acc0[b, h, :T].double() * decay
            old[max(0, T - min(fresh, T)):] = 0
            w = p.sum(0)
            # logits as in attend()'s bound (fp32 sums; the E4M3 path's query in fp16 pieces or converted keys), the
            # exponent's rounding 2^-20 and the exponential 2^-21, G fp32 additions, and the update's own rounding
            e = (d + 2) * 2.0 ** -24 * (rows.abs() @ k[:, h].abs().T).amax() / math.sqrt(d) if T else 0.0
            slack = 2 * e + 2.0 ** -12 + (G + 2) * 2.0 ** -24
            err = (acc[b, h, :T].double() - (old + w)).abs()
            assert bool((err <= slack * w + 2.0 ** -22 * old + 1e-30).all()), float((err - slack * w).max())
            assert torch.equal(R.bits(acc[b, h, T:]), R.bits(acc0[b, h, T:]))


# ---------------------------------------------------------------- evict
@pytest.mark.parametrize("dtype,hkv,d,page,budget,window", [
    ("bf16", 2, 128, 64, 100, 16), ("e4m3", 3, 128, 16, 333, 128), ("f32", 1, 64, 0, 1, 0), ("bf16", 2, 64, 32, 64, 64),
    ("bf16", 1, 128, 64, 2000, 7), ("e4m3", 1, 128, 0, 1023, 0), ("bf16", 2, 64, 16, 690, 3)])
def test_cache_evict(dtype, hkv, d, page, budget, window):
    lens = [5000, 99, 0, budget, budget + 1, 2100, 700]
    c = R.PagedCache(dtype, lens, hkv, d, page, seed=11)
    acc = torch.exp(3 * torch.randn(len(lens), hkv, c.cap + 1, device="cuda", generator=gen(12)))
    acc[acc < 0.3] = 0.0  # many equal sums
    acc[0, 0, ::7] = -0.0
    acc[0, 0, 5:50:5] = NAN
    acc[0, -1, 100:120] = math.inf
    acc[0, -1, 200:220] = -math.inf
    acc[5] = 1.5  # all equal
    acc[6, 0] = NAN
    acc0, before = acc.clone(), c.snapshot()
    want = [None if x is None else x.clone() for x in before]
    want_acc = acc.clone()
    lens_out, kept = hs2.cache_evict(c.k, c.v, c.lens, acc, budget, window, **c.kw())
    for b, T in enumerate(lens):
        for h in range(hkv):
            keep = R.kept_positions(acc0[b, h, :T].tolist(), T, budget, window)
            assert kept[b, h].tolist() == keep + [-1] * (budget - len(keep)), (b, h)
            if T <= budget:
                continue
            src, dst = c.slots(b, keep), c.slots(b, list(range(budget)))
            for x, y in zip(want, before):
                if x is not None:
                    x[dst, h] = y[src, h]
            want_acc[b, h, :budget] = acc0[b, h, keep]
    assert lens_out.tolist() == [min(T, budget) for T in lens]
    for b, T in enumerate(lens):
        live = budget if T > budget else T
        s = c.slots(b, list(range(live)))
        for x, y in zip((c.k, c.v, c.k_scale, c.v_scale), want):
            assert x is None or torch.equal(R.bits(x[s]), R.bits(y[s]))
        assert torch.equal(R.bits(acc[b, :, :live]), R.bits(want_acc[b, :, :live]))
        assert torch.equal(R.bits(acc[b, :, T:]), R.bits(acc0[b, :, T:]))
    untouched = torch.ones(c.k.shape[0], dtype=torch.bool, device="cuda")  # rows of no sequence
    for b, T in enumerate(lens):
        if T:
            untouched[c.slots(b, list(range(T)))] = False
    for x, y in zip((c.k, c.v, c.k_scale, c.v_scale), before):
        assert x is None or torch.equal(R.bits(x[untouched]), R.bits(y[untouched]))


@pytest.mark.parametrize("T,budget,window,hkv", [(300000, 150001, 128, 1), (131072, 70000, 0, 1), (140000, 1000, 5, 2)])
def test_cache_evict_long(T, budget, window, hkv):
    """Shares of more positions than a CTA's registers hold, and many runs of rows; a short sequence beside."""
    c = R.PagedCache("e4m3", [T, budget // 2], hkv, 128, 64, seed=13, poison=False)
    acc = torch.exp(3 * torch.randn(2, hkv, c.cap, device="cuda", generator=gen(14)))
    acc[acc < 1.0] = 0.0  # more zeros than are dropped: the last ones taken are among equals
    acc0, before = acc.clone(), c.snapshot()
    lens_out, kept = hs2.cache_evict(c.k, c.v, c.lens, acc, budget, window, **c.kw())
    assert lens_out.tolist() == [budget, budget // 2]
    for h in range(hkv):
        keep = torch.tensor(R.kept_positions(acc0[0, h, :T].tolist(), T, budget, window), device="cuda")
        assert torch.equal(kept[0, h].long(), keep)
        src, dst = c.slots(0, keep), c.slots(0, torch.arange(budget))
        for x, y in zip((c.k, c.v, c.k_scale, c.v_scale), before):
            assert torch.equal(R.bits(x[dst, h]), R.bits(y[src, h]))
        assert torch.equal(acc[0, h, :budget], acc0[0, h, keep])
    short = c.slots(1, torch.arange(budget // 2))
    for x, y in zip((c.k, c.v, c.k_scale, c.v_scale), before):
        assert torch.equal(R.bits(x[short]), R.bits(y[short]))


# ---------------------------------------------------------------- rope
ROPES = [
    ("bf16", 2, 4, 128, 64, 128, False, {}),
    ("bf16", 1, 8, 64, 16, 48, False, dict(scaling="linear", factor=8.0)),
    ("bf16", 4, 1, 128, 0, 16, True, dict(scaling="ntk", factor=4.0)),
    ("e4m3", 2, 4, 128, 32, 64, True, dict(scaling="yarn", factor=32.0, original_context=4096)),
    ("e4m3", 3, 2, 128, 64, 128, False, dict(base=500000.0, scaling="bands", factor=8.0, original_context=8192)),
    ("f32", 1, 4, 64, 0, 64, True, dict(base=500000.0)),
    ("f32", 2, 2, 128, 16, 96, False, dict(scaling="yarn", factor=4.0, original_context=2048)),
]


def rope_check(got, exact, x, positions, f, scale, dtype):
    """The rotation's error: the angle is exact to 2^-23 rad here and to pos 2^-52 f in the 64-bit form, sine and cosine
    to 2^-22, two products and a sum 3 2^-24, all relative to the pair's size; then the output's rounding."""
    pair = x.abs().amax() * scale * 2
    angle = positions.abs().double().max() * float(f.max()) * 2.0 ** -51
    tol = pair * (2.0 ** -20 + angle) + exact.abs() * HALF[dtype] * (1 + 2 ** -6)
    assert bool(((got.double() - exact).abs() <= tol).all()), float(((got.double() - exact).abs() - tol).max())


HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -8}


@pytest.mark.parametrize("N", [1, 37])
@pytest.mark.parametrize("case", ROPES, ids=lambda c: f"{c[0]}-{c[5]}-{c[7].get('scaling', 'none')}")
def test_rope_append(case, N):
    dtype, hkv, G, d, page, rot, inter, kw = case
    lens = [200, N, 0, 129, 2 * N, 5]
    new = [N, N, N, max(N // 2, 1), 0, N]
    B, hq = len(lens), hkv * G
    c = R.PagedCache(dtype, lens, hkv, d, page, seed=21)
    qt = R.q_dtype(dtype)
    qkv = torch.randn(B, N, hq + 2 * hkv, d, device="cuda", generator=gen(22)).to(qt)
    qkv[0, 0, hq:] = 0  # an all-zero row: E4M3 scale 1
    positions = torch.randint(0, 2 ** 20, (B, N), device="cuda", generator=gen(23), dtype=torch.int32)
    positions[0, N - 1], positions[3, 0] = 2 ** 31 - 1, -12345
    table = hs2.rope_table(rot, interleaved=inter, **kw)
    f, scale = R.inv_freq(rot, **dict(dict(base=10000.0), **kw))
    before = c.snapshot()
    q_out = torch.full((B, N, hq, d), 77.0, device="cuda", dtype=qt)
    got = hs2.rope_append(qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:], positions, table, c.k, c.v, c.lens,
                          num_new=i32(new), q_out=q_out, **c.kw())
    assert got is q_out
    x = qkv.double()
    exact = R.rotate(x[:, :, :hq + hkv], positions, f, scale, inter)
    mine = torch.zeros(c.k.shape[0], dtype=torch.bool, device="cuda")
    for b, T in enumerate(lens):
        n = max(0, min(new[b], N, T))
        assert bool((q_out[b, n:] == 77.0).all())
        for i in range(n):
            p = positions[b:b + 1, i]
            rope_check(q_out[b, i], exact[b, i, :hq], x[b, i, :hq], p, f, scale, dtype)
            slot = int(c.slots(b, T - n + i))
            mine[slot] = True
            for cache, sc, want in ((c.k, c.k_scale, exact[b, i, hq:]), (c.v, c.v_scale, x[b, i, hq + hkv:])):
                if dtype != "e4m3":
                    rope_check(cache[slot], want, x[b, i], p, f, scale, dtype)
                    continue
                top = want.abs().amax(-1)
                s = sc[slot].double()
                slack = (2.0 ** -20 + float(p.abs()) * float(f.max()) * 2.0 ** -51) * 2 * scale * x[b, i].abs().amax()
                assert bool(((s - torch.where(top > 0, top / 448, torch.ones_like(top))).abs() <= slack / 448 + s * 2.0 ** -22).all())
                err = (cache[slot].double() * s.unsqueeze(-1) - want).abs()
                assert bool((err <= 2.0 ** -4 * want.abs() * (1 + 2 ** -6) + s.unsqueeze(-1) * 2.0 ** -10 + slack).all())
            if dtype != "e4m3" or N == 1:
                assert torch.equal(R.bits(c.v[slot]), R.bits(qkv[b, i, hq + hkv:])) or dtype == "e4m3"
    for y, z in zip((c.k, c.v, c.k_scale, c.v_scale), before):
        assert y is None or torch.equal(R.bits(y[~mine]), R.bits(z[~mine]))
    # keys and values alone; then the queries in place
    hs2.rope_append(None, qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:], positions, table, c.k, c.v, c.lens, num_new=i32(new), **c.kw())
    q2 = qkv[:, :, :hq].contiguous()
    hs2.rope_append(q2, qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:], positions, table, c.k, c.v, c.lens, num_new=i32(new), q_out=q2, **c.kw())
    for b, T in enumerate(lens):
        n = max(0, min(new[b], N, T))
        assert torch.equal(R.bits(q2[b, :n]), R.bits(q_out[b, :n])) and torch.equal(R.bits(q2[b, n:]), R.bits(qkv[b, n:, :hq]))


def test_rope_append_e4m3_rows_of_any_size():
    """Rows of subnormal, tiny and huge elements, and rows with one large element: scale and codes as for any other."""
    c = R.PagedCache("e4m3", [40], 2, 128, 16, seed=1)
    x = torch.randn(1, 8, 2, 128, device="cuda", generator=gen(7))
    x *= torch.tensor([1e-39, 1e-37, 1e-30, 1.0, 1e30, 1e37, 1.0, 1.0], device="cuda").view(1, 8, 1, 1)
    x[0, 6, :, 3] = 1e20
    x[0, 7, :, 1:] = 0
    x = x.bfloat16()
    pos = torch.zeros(1, 8, dtype=torch.int32, device="cuda")
    hs2.rope_append(None, x, x, pos, hs2.rope_table(128), c.k, c.v, c.lens, **c.kw())
    for i in range(8):
        slot, want = int(c.slots(0, 32 + i)), x[0, i].double()
        for cache, sc in ((c.k, c.k_scale), (c.v, c.v_scale)):
            s = sc[slot].double()
            top = want.abs().amax(-1)
            # one rounding of max / 448, which may be subnormal
            assert bool(((s - top / 448).abs() <= top / 448 * 2.0 ** -23 + 2.0 ** -149).all())
            err = (cache[slot].double() * s.unsqueeze(-1) - want).abs()
            # half a step of the code (a subnormal one: 2^-10 of the scale), the quotient's error of two roundings, and the
            # half unit by which a subnormal scale is off, taken 448 times
            tol = 2.0 ** -4 * want.abs() * (1 + 2.0 ** -6) + s.unsqueeze(-1) * 2.0 ** -10 + 448 * 2.0 ** -149
            assert bool((err <= tol).all()), (i, float((err - tol).max()))


def test_rope_append_page_outside_the_cache():
    c = R.PagedCache("bf16", [40, 40], 2, 128, 16, seed=1)
    c.table[1, 2] = 2 ** 31 - 1  # the page of positions 32 to 47
    before = c.snapshot()
    x = torch.randn(2, 3, 2, 128, device="cuda").bfloat16()
    pos = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    hs2.rope_append(None, x, x, pos, hs2.rope_table(128), c.k, c.v, c.lens, **c.kw())
    mine = torch.zeros(c.k.shape[0], dtype=torch.bool, device="cuda")
    mine[c.slots(0, [37, 38, 39])] = True
    assert torch.equal(R.bits(c.k[~mine]), R.bits(before[0][~mine])) and torch.equal(R.bits(c.k[c.slots(0, [37, 38, 39])]), R.bits(x[0]))


def test_rope_is_relative():
    """Rotated products depend on the distance of the positions alone."""
    t = hs2.rope_table(128, base=10000.0)
    q = torch.randn(1, 1, 1, 128, device="cuda", generator=gen(1))
    k = torch.randn(1, 1, 1, 128, device="cuda", generator=gen(2))
    dots = []
    for far in (0, 1, 12345, 2 ** 30):
        c = R.PagedCache("f32", [1], 1, 128, 0, seed=1)
        r = hs2.rope_append(q, k, k, i32([[far + 77]]), t, c.k, c.v, c.lens, **c.kw())
        rk = hs2.rope_append(k, k, k, i32([[far]]), t, c.k, c.v, c.lens, **c.kw())
        assert torch.equal(rk[0, 0], c.k[0])
        dots.append(float((r.double() * rk.double()).sum()))
    size = float((q.abs() * k.abs()).sum())
    assert max(dots) - min(dots) <= 4 * size * 2.0 ** -20  # twice two roundings of sine, cosine and products each


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
def test_calls_captured_and_replayed(dtype):
    """One graph of all five calls, replayed on other inputs, leaves what the calls leave one by one."""
    hkv, G, d, N, B = 2, 4, 128, 5, 3
    def state(seed):
        c = R.PagedCache(dtype, [400, 77, 150], hkv, d, 16, seed=seed, poison=False)
        g = gen(seed)
        return c, dict(
            qkv=torch.randn(B, N, hkv * (G + 2), d, device="cuda", generator=g).to(R.q_dtype(dtype)),
            pos=torch.randint(0, 5000, (B, N), device="cuda", generator=g, dtype=torch.int32), new=i32([5, 3, 1]),
            words=torch.tensor(signed([mask_words(random_tree(N, seed + b)) for b in range(B)]), device="cuda"),
            path=torch.randint(0, 5, (B, N), device="cuda", generator=g, dtype=torch.int32), plen=i32([3, 2, 1]),
            acc=torch.rand(B, hkv, c.cap, device="cuda", generator=g), out=torch.zeros(B, N, hkv * G, d, device="cuda", dtype=R.q_dtype(dtype)),
            q_out=torch.zeros(B, N, hkv * G, d, device="cuda", dtype=R.q_dtype(dtype)), lens1=torch.zeros_like(c.lens),
            lens2=torch.zeros_like(c.lens), kept=torch.zeros(B, hkv, 90, dtype=torch.int32, device="cuda"),
            o1=torch.zeros(B, hkv * G, d, device="cuda", dtype=R.q_dtype(dtype)))
    table = hs2.rope_table(64)

    def step(c, s, ws_tree, ws_full):
        x, hq = s["qkv"], hkv * G
        hs2.rope_append(x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:], s["pos"], table, c.k, c.v, c.lens,
                        num_new=s["new"], q_out=s["q_out"], **c.kw())
        hs2.tree_attn(s["q_out"], c.k, c.v, c.lens, tree_mask=s["words"], num_draft=s["new"], out=s["out"], workspace=ws_tree, **c.kw())
        hs2.tree_accept(c.k, c.v, c.lens, s["path"], s["plen"], num_draft=s["new"], lens_out=s["lens1"], **c.kw())
        hs2.full_attn_accumulate(s["o1"], c.k, c.v, s["lens1"], s["acc"], decay=0.5, out=s["o1"].clone(), workspace=ws_full, **c.kw())
        hs2.cache_evict(c.k, c.v, s["lens1"], s["acc"], 90, 10, kept=s["kept"], lens_out=s["lens2"], **c.kw())

    c, s = state(3)
    ws_tree = hs2.alloc_tree_workspace(s["q_out"], c.k)
    ws_full = hs2.alloc_workspace(B, hkv, G, d, c.cap)
    first = c.snapshot() + [x.clone() for x in s.values()]
    step(c, s, ws_tree, ws_full)  # the kernels are loaded before the capture
    live = [x for x in (c.k, c.v, c.k_scale, c.v_scale)] + list(s.values())
    for x, y in zip(live, first):
        if x is not None:
            x.copy_(y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(c, s, ws_tree, ws_full)
    for seed in (4, 5):
        other, t = state(seed)
        c.lens.copy_(other.lens)
        if c.table is not None:
            c.table.copy_(other.table)
        for x, y in zip(live, [other.k, other.v, other.k_scale, other.v_scale] + list(t.values())):
            if x is not None:
                x.copy_(y)
        g.replay()
        step(other, t, hs2.alloc_tree_workspace(t["q_out"], other.k), hs2.alloc_workspace(B, hkv, G, d, other.cap))
        torch.cuda.synchronize()
        for x, y in zip(live, [other.k, other.v, other.k_scale, other.v_scale] + list(t.values())):
            assert x is None or torch.equal(R.bits(x), R.bits(y))
    assert hs2.workspace_status(ws_tree) == hs2.OK and hs2.workspace_status(ws_full) == hs2.OK


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("dtype,page", [("bf16", 16), ("e4m3", 64), ("f32", 0)])
def test_draft_verify_accumulate_evict_together(dtype, page):
    """Steps of a user's loop: append a drafted tree, verify it, keep a path, append a token with its weights, trim.
    Every step's inputs are the state that the calls left; every step is held against the plain forms on that state."""
    hkv, G, d, N, B, budget, window = 2, 4, 128, 7, 3, 60, 12
    lens = [50, 9, 64]
    c = R.PagedCache(dtype, lens, hkv, d, page, seed=31, spare=80, poison=False)
    qt = R.q_dtype(dtype)
    table = hs2.rope_table(64, interleaved=True)
    f, scale = R.inv_freq(64, 10000.0)
    acc = torch.rand(B, hkv, c.cap, device="cuda", generator=gen(5))
    seen = list(lens)  # tokens so far: the next position
    T = list(lens)
    g = torch.Generator().manual_seed(77)
    for step in range(4):
        parents = [random_tree(N, 100 * step + b) for b in range(B)]
        depth = [[0] * N for _ in range(B)]
        for b in range(B):
            for i, p in enumerate(parents[b]):
                depth[b][i] = 0 if p < 0 else depth[b][p] + 1
        words = hs2.tree_mask(parents).cuda()
        masks = [mask_words(p) for p in parents]
        nd = [N, N - 2, 1 + step]
        qkv = torch.randn(B, N, hkv * (G + 2), d, device="cuda", generator=gen(40 + step)).to(qt)
        pos = i32([[seen[b] + depth[b][i] for i in range(N)] for b in range(B)])
        T = [t + n for t, n in zip(T, nd)]
        c.T, c.lens = T, i32(T)
        q = hs2.rope_append(qkv[:, :, :hkv * G], qkv[:, :, hkv * G:hkv * (G + 1)], qkv[:, :, hkv * (G + 1):], pos, table, c.k, c.v,
                            c.lens, num_new=i32(nd), **c.kw())
        exact = R.rotate(qkv[:, :, :hkv * (G + 1)].double(), pos, f, scale, True)
        for b in range(B):
            rope_check(q[b, :nd[b]], exact[b, :nd[b], :hkv * G], qkv[b].double(), pos[b], f, scale, dtype)
        want, bound = R.tree_reference(c, q, nd, masks, dtype)
        out = torch.full_like(q, 77.0)
        hs2.tree_attn(q, c.k, c.v, c.lens, tree_mask=words, num_draft=i32(nd), out=out, **c.kw())
        check(out, want, bound, ~want.isnan())
        # the path to a random accepted draft
        path, plen = [], []
        for b in range(B):
            i, p = int(torch.randint(0, nd[b], (), generator=g)), []
            while i >= 0:
                p.append(i)
                i = parents[b][i]
            path.append(p[::-1] + [0] * (N - len(p)))
            plen.append(len(p))
        rows = [c.wide("k", b, [T[b] - nd[b] + j for j in path[b][:plen[b]]]) for b in range(B)]
        c.lens = hs2.tree_accept(c.k, c.v, c.lens, i32(path), i32(plen), num_draft=i32(nd), **c.kw())
        T = [t - n + a for t, n, a in zip(T, nd, plen)]
        assert c.lens.tolist() == T
        for b in range(B):
            assert torch.equal(c.wide("k", b, torch.arange(T[b] - plen[b], T[b])), rows[b])
        seen = [s + a for s, a in zip(seen, plen)]
        # the next token, its weights, and the budget
        qkv = torch.randn(B, 1, hkv * (G + 2), d, device="cuda", generator=gen(80 + step)).to(qt)
        T = [t + 1 for t in T]
        c.T, c.lens = T, i32(T)
        q = hs2.rope_append(qkv[:, :, :hkv * G], qkv[:, :, hkv * G:hkv * (G + 1)], qkv[:, :, hkv * (G + 1):],
                            i32([[s] for s in seen]), table, c.k, c.v, c.lens, **c.kw())
        seen = [s + 1 for s in seen]
        acc0 = acc.clone()
        fresh = max(plen) + 1
        hs2.full_attn_accumulate(q[:, 0], c.k, c.v, c.lens, acc, decay=0.9, fresh=fresh, **c.kw())
        for b in range(B):
            k = c.wide("k", b, torch.arange(T[b]))
            old = acc0[b, :, :T[b]].double() * 0.9
            old[:, max(0, T[b] - fresh):] = 0
            for h in range(hkv):
                w = torch.softmax(q[b, 0, h * G:(h + 1) * G].double() @ k[:, h].T / math.sqrt(d), -1).sum(0)
                assert bool(((acc[b, h, :T[b]].double() - old[h] - w).abs() <= 2.0 ** -11 * (w + old[h])).all())
        sums = acc.clone()
        lens_out, kept = hs2.cache_evict(c.k, c.v, c.lens, acc, budget, window, **c.kw())
        for b in range(B):
            for h in range(hkv):
                keep = R.kept_positions(sums[b, h, :T[b]].tolist(), T[b], budget, window)
                assert kept[b, h, :len(keep)].tolist() == keep
                assert torch.equal(acc[b, h, :len(keep)], sums[b, h, keep])
        T = lens_out.tolist()
        c.T, c.lens = T, lens_out
    assert max(T) == budget
