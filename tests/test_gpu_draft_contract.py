"""What the drafted-token and bounded-cache calls promise beside their formulas: where results and workspaces are made,
counts of each sequence's own, paths narrower than the draft, codes that both appends write, rows and sums that nothing
may read.  Plain 64-bit forms in tests/draft_ref.py."""
import math

import pytest
import torch

import draft_ref as R
from test_gpu_draft import check, gen, i32, random_tree, tree_case
from long_context_decode_full_b200 import hs2

pytestmark = pytest.mark.gpu
NAN = float("nan")
BUSY = 100_000_000  # cycles, some 50 ms: longer than any call here


# ---------------------------------------------------------------- another stream
class StreamCase:
    """One cache and the arguments of every call on it; a call takes a stream and leaves out all that is optional."""

    def __init__(self):
        hkv, G, d, N, B = 2, 4, 128, 5, 2
        self.c = c = R.PagedCache("bf16", [700, 90], hkv, d, 16, seed=41, poison=False)
        qkv = torch.randn(B, N, hkv * (G + 2), d, device="cuda", generator=gen(42)).bfloat16()
        pos = torch.randint(0, 900, (B, N), device="cuda", generator=gen(43), dtype=torch.int32)
        table, q = hs2.rope_table(128), qkv[:, :, :hkv * G]
        kn, vn = qkv[:, :, hkv * G:hkv * (G + 1)], qkv[:, :, hkv * (G + 1):]
        self.acc = acc = torch.rand(B, hkv, c.cap, device="cuda", generator=gen(44))
        path, plen = i32([[1, 3, 4, 0, 0], [0, 2, 4, 0, 0]]), i32([3, 2])
        hidden = torch.randn(B, 256, device="cuda", generator=gen(45)).bfloat16()
        w = torch.randn(256, hkv * d, device="cuda", generator=gen(46)).bfloat16()
        q1 = q[:, 0].contiguous()
        idx = c.slots(0, torch.arange(40)).to(torch.int32).expand(B, hkv, 40).contiguous()
        pg = dict(page_table=c.table, page_size=c.page)
        self.calls = {
            "rope_append": lambda s: hs2.rope_append(q, kn, vn, pos, table, c.k, c.v, c.lens, stream=s, **pg),
            "tree_attn": lambda s: hs2.tree_attn(q, c.k, c.v, c.lens, stream=s, **pg),
            "tree_accept": lambda s: hs2.tree_accept(c.k, c.v, c.lens, path, plen, stream=s, **pg),
            "full_attn_accumulate": lambda s: hs2.full_attn_accumulate(q1, c.k, c.v, c.lens, acc, stream=s, **pg),
            "cache_evict": lambda s: hs2.cache_evict(c.k, c.v, c.lens, acc, 80, 10, stream=s, **pg),
            "kv_bridge_append": lambda s: hs2.kv_bridge_append(hidden, w, w, c.k, c.v, c.lens, stream=s, **pg),
            "full_attn_select": lambda s: hs2.full_attn_select(q1, c.k, c.v, c.lens, window=16, k_global=32, stream=s, **pg),
            "full_attn_select_blocks": lambda s: hs2.full_attn_select_blocks(q1, c.k, c.v, c.lens, window=16, k_global=32,
                                                                             stream=s, **pg),
            "full_attn_select_static": lambda s: hs2.full_attn_select_static(q1, c.k, c.v, c.lens, window=16, k_global=32,
                                                                             stream=s, **pg),
            "sparse_attn": lambda s: hs2.sparse_attn(q1, c.k, c.v, idx, stream=s),
        }
        self.state = [c.k, c.v, acc]
        self.start = [x.clone() for x in self.state]

    def reset(self):
        for x, y in zip(self.state, self.start):
            x.copy_(y)


def results(r):
    return [] if r is None else [r] if torch.is_tensor(r) else list(r)


STREAM_CALLS = ["rope_append", "tree_attn", "tree_accept", "full_attn_accumulate", "cache_evict", "kv_bridge_append",
                "full_attn_select", "full_attn_select_blocks", "full_attn_select_static", "sparse_attn"]


@pytest.mark.parametrize("busy", ["current", "given"])
@pytest.mark.parametrize("name", STREAM_CALLS)
def test_results_and_workspaces_belong_to_the_given_stream(name, busy):
    """A call on another stream makes what it is not given on that stream: nothing queued on the current one may reach
    its results, and no memory of the call may pass to the current stream while the call runs."""
    case = StreamCase()
    want = [x.clone() for x in results(case.calls[name](None)) + case.state]
    case.reset()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    if busy == "current":  # a fill of a result on the current stream would come after the call
        torch.cuda._sleep(BUSY)
        got = results(case.calls[name](s))
    else:  # the call waits; memory that it gave back would be taken and overwritten meanwhile
        with torch.cuda.stream(s):
            torch.cuda._sleep(BUSY)
        got = results(case.calls[name](s))
        taken = [torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") for n in [1 << 8, 1 << 12, 1 << 16, 1 << 20] * 20 + [1 << 26] * 4]
    torch.cuda.synchronize()
    for x, y in zip(got + case.state, want):
        assert torch.equal(R.bits(x), R.bits(y))


# ---------------------------------------------------------------- a workspace used twice at once
@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
def test_tree_attn_graphs_that_share_a_workspace(dtype):
    """One workspace for two captured calls of other lengths and batches: right one after the other.  At once their
    outputs are undefined, but nothing outside the workspace is touched, and a call after them is right."""
    sides = [tree_case(dtype, 2, 4, 128, 64, 9, lens, [9] * len(lens), seed=s)
             for s, lens in ((1, [3000, 400]), (2, [9, 70, 20000, 11, 12, 500, 64, 65]))]
    refs = [R.tree_reference(c, q, [9] * len(c.T), masks, dtype) for c, q, masks, _ in sides]
    ws = max((hs2.alloc_tree_workspace(q, c.k) for c, q, _, _ in sides), key=lambda w: w.numel())
    ws = torch.cat([ws, torch.full((1 << 16,), 0x5A, dtype=torch.uint8, device="cuda")])  # the end is not the calls'
    n, graphs, outs, streams = ws.numel() - (1 << 16), [], [], [torch.cuda.Stream() for _ in sides]
    for c, q, _, words in sides:
        out = torch.full_like(q, 77.0)
        call = lambda: hs2.tree_attn(q, c.k, c.v, c.lens, tree_mask=words, out=out, workspace=ws[:n], **c.kw())  # noqa: B023, E731
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
        outs.append(out)
    def each():
        for g, out, (want, bound) in zip(graphs, outs, refs):
            out.fill_(77.0)
            g.replay()
            torch.cuda.synchronize()
            check(out, want, bound, ~want.isnan())
    each()
    for _ in range(50):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert hs2.workspace_status(ws[:n]) == hs2.OK
    each()
    assert bool((ws[n:] == 0x5A).all())


# ---------------------------------------------------------------- one workspace for drafts of all lengths
@pytest.mark.parametrize("dtype,hkv,G,d,N", [("bf16", 1, 32, 128, 8), ("f32", 1, 8, 128, 4), ("f32", 4, 4, 64, 5), ("e4m3", 2, 8, 128, 3)])
def test_tree_attn_short_drafts_in_a_long_drafts_workspace(dtype, hkv, G, d, N):
    most = R.PagedCache(dtype, [64] * 40, hkv, d, 64, seed=1)
    ws = hs2.alloc_tree_workspace(torch.empty(40, 64, hkv * G, d, device="cuda", dtype=R.q_dtype(dtype)), most.k)
    for lens in ([3000], [700, N, 65]):
        case = (dtype, hkv, G, d, 64, N, lens, [N] * len(lens))
        c, q, masks, words = tree_case(*case, seed=15)
        out = torch.full_like(q, 77.0)
        hs2.tree_attn(q, c.k, c.v, c.lens, tree_mask=words, out=out, workspace=ws, **c.kw())
        want, bound = R.tree_reference(c, q, [N] * len(lens), masks, dtype)
        check(out, want, bound, ~want.isnan())


# ---------------------------------------------------------------- parts of the same rows
def test_tree_attn_queries_and_output_side_by_side():
    """q and out as parts of the same wider rows, in either order: between each other in memory, no element shared."""
    for at_q, at_o in ((0, 8), (9, 0)):
        c, q, masks, words = tree_case("bf16", 2, 4, 128, 64, 6, [300, 7], [6, 6], seed=2)
        wide = torch.full((2, 6, 17, 128), 77.0, device="cuda", dtype=q.dtype)
        wide[:, :, at_q:at_q + 8] = q
        before = wide.clone()
        out = hs2.tree_attn(wide[:, :, at_q:at_q + 8], c.k, c.v, c.lens, tree_mask=words, out=wide[:, :, at_o:at_o + 8], **c.kw())
        want, bound = R.tree_reference(c, q, [6, 6], masks, "bf16")
        check(out, want, bound, ~want.isnan())
        wide[:, :, at_o:at_o + 8] = before[:, :, at_o:at_o + 8]
        assert torch.equal(wide, before)


def test_rope_append_queries_in_place_beside_keys_and_values():
    """One token per sequence of a fused projection, its queries rotated where they are."""
    c = R.PagedCache("bf16", [40], 2, 128, 16, seed=1)
    qkv = torch.randn(1, 1, 12, 128, device="cuda", generator=gen(7)).bfloat16()
    pos, table, before = i32([[39]]), hs2.rope_table(128), c.snapshot()
    want = hs2.rope_append(qkv[:, :, :8].contiguous(), qkv[:, :, 8:10], qkv[:, :, 10:], pos, table, c.k, c.v, c.lens, **c.kw())
    rows = c.k[c.slots(0, 39)].clone()
    c.k.copy_(before[0])
    same = qkv.clone()
    got = hs2.rope_append(same[:, :, :8], same[:, :, 8:10], same[:, :, 10:], pos, table, c.k, c.v, c.lens, q_out=same[:, :, :8], **c.kw())
    assert torch.equal(got, want) and torch.equal(same[:, :, 8:], qkv[:, :, 8:]) and torch.equal(c.k[c.slots(0, 39)], rows)


def all_calls(c, N, lens, G, d, hkv, acc, dtype, seed):
    """Every call of a verification step on cache c; returns what they gave."""
    B = len(lens)
    qkv = torch.randn(B, N, hkv * (G + 2), d, device="cuda", generator=gen(seed)).to(R.q_dtype(dtype))
    pos = torch.arange(N, device="cuda", dtype=torch.int32).repeat(B, 1) + c.lens[:, None] - N
    q = hs2.rope_append(qkv[:, :, :hkv * G], qkv[:, :, hkv * G:hkv * (G + 1)], qkv[:, :, hkv * (G + 1):], pos, hs2.rope_table(64),
                        c.k, c.v, c.lens, **c.kw())
    out = hs2.tree_attn(q, c.k, c.v, c.lens, **c.kw())
    path = torch.tensor([[1, N - 1]] * B, dtype=torch.int32, device="cuda")
    two = torch.full((B,), 2, dtype=torch.int32, device="cuda")
    lens = hs2.tree_accept(c.k, c.v, c.lens, path, two, num_draft=two * 0 + N, **c.kw())
    o, _ = hs2.full_attn_accumulate(q[:, 1].contiguous(), c.k, c.v, lens, acc, fresh=two, **c.kw())
    lens2, kept = hs2.cache_evict(c.k, c.v, lens, acc, 100, **c.kw())
    return [q, out, lens, o, lens2, kept, acc]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
def test_calls_on_one_pool_of_alternating_k_and_v_pages(dtype):
    """Caches [pages, 2, page, heads, d]: K's pages the even ones, V's the odd ones of the same memory."""
    hkv, G, d, N, page, lens = 2, 2, 128, 4, 16, [300, 70, 129]
    apart = R.PagedCache(dtype, lens, hkv, d, page, seed=44, poison=False)
    pool = R.PagedCache(dtype, lens, hkv, d, page, seed=44, poison=False)
    for k, v in (("k", "v"), ("k_scale", "v_scale")):
        if getattr(pool, k) is not None:
            both = torch.stack([getattr(pool, x).unflatten(0, (-1, page)) for x in (k, v)], 1).flatten(0, 2)
            setattr(pool, k, both[:-page])
            setattr(pool, v, both[page:])
    pool.table = apart.table * 2
    acc = torch.rand(len(lens), hkv, apart.cap, device="cuda", generator=gen(45))
    got = all_calls(pool, N, lens, G, d, hkv, acc.clone(), dtype, 46)
    want = all_calls(apart, N, lens, G, d, hkv, acc.clone(), dtype, 46)
    for x, y in zip(got, want):
        assert torch.equal(R.bits(x), R.bits(y))
    for name in ("k", "v", "k_scale", "v_scale"):
        x, y = getattr(pool, name), getattr(apart, name)
        assert x is None or torch.equal(R.bits(x.unflatten(0, (-1, page))[::2]), R.bits(y.unflatten(0, (-1, page))))


# ---------------------------------------------------------------- rows that see nothing, drafts that nobody may see
@pytest.mark.parametrize("dtype,N,G,d,T", [
    ("f32", 4, 2, 128, 200), ("f32", 8, 1, 64, 3000),    # one block of 8 rows
    ("f32", 4, 4, 64, 200), ("f32", 8, 2, 128, 3000),    # two
    ("f32", 8, 4, 128, 300), ("f32", 8, 4, 64, 3000),    # 32 rows, in tiles of 32 and of 64 positions
    ("f32", 7, 8, 128, 300),                             # 64 rows
    ("bf16", 8, 8, 128, 300), ("bf16", 4, 4, 64, 300), ("e4m3", 8, 8, 128, 300), ("e4m3", 5, 2, 128, 3000)])
def test_tree_attn_small_trees_with_empty_rows_and_poisoned_drafts(dtype, N, G, d, T):
    """Every shape of the kernels: masks that leave rows empty, with and without a context, and drafts whose values or
    keys are infinite or NaN, seen by themselves alone."""
    lens = [N, N, T]
    mask = [0 if i % 5 == 0 else 1 << i if i in (2, 3) else 1 << i | 1 << 1 for i in range(N)]
    masks = [mask, [m | ~((1 << N) - 1) & (1 << 64) - 1 for m in mask], mask]  # bits behind the draft mean nothing
    c, q, masks, words = tree_case(dtype, 2, G, d, 16, N, lens, [N] * 3, seed=9, masks=masks)
    for b in range(3):
        values, keys = (int(s) for s in c.slots(b, [lens[b] - N + 2, lens[b] - N + 3]))
        if dtype == "e4m3":
            c.v.view(torch.uint8)[values, :, 5] = 0x7f
            c.k.view(torch.uint8)[keys, :, 100] = 0xff
        else:
            c.v[values, :, 5] = NAN
            c.v[values, :, 9] = -math.inf
            c.k[keys, :, 60] = NAN
    clean = R.PagedCache(dtype, lens, 2, d, 16, 9)
    want, bound = R.tree_reference(clean, q, [N] * 3, masks, dtype)
    out = torch.full_like(q, 77.0)
    hs2.tree_attn(q, c.k, c.v, c.lens, tree_mask=words, out=out, **c.kw())
    good = torch.tensor([i not in (2, 3) for i in range(N)], device="cuda")
    assert bool(((out.double() - want).abs() <= bound)[:, good].all())
    assert bool((out[:2, [i % 5 == 0 for i in range(N)]] == 0).all())
    assert bool(out[:, 2, :, 5].isnan().all()) and bool(out[:, 2, :, :5].isfinite().all()) and bool(out[:, 2, :, 10:].isfinite().all())
    assert dtype == "e4m3" or bool((out[:, 2, :, 9] == -math.inf).all())
    assert bool(out[:, 3].isnan().all())


# ---------------------------------------------------------------- weights far below a dominating one
@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("at", [3, 30000])
def test_tree_attn_weights_far_below_a_dominating_one(dtype, at):
    """One row takes all but 2^-20 of the weight and has no value, as the first row of a context often does: the output is
    what the 40,000 others add, with weights 2^-40 below the largest, and as exact as any."""
    T, N, hkv, G, d = 40000, 5, 1, 4, 128
    c, q, masks, words = tree_case(dtype, hkv, G, d, 64, N, [T], [N], seed=23)
    q[..., 0] = 8.0
    row = int(c.slots(0, at))
    if dtype == "e4m3":
        live = c.slots(0, torch.arange(T))
        c.k.view(torch.uint8)[live, :, 0] = 0
        c.k.view(torch.uint8)[row], c.v.view(torch.uint8)[row] = 0, 0
        c.k[row, :, 0] = 448.0
        c.k_scale[row] = 39.0 / 448.0
    else:
        c.k[c.slots(0, torch.arange(T)), :, 0] = 0.0
        c.k[row], c.v[row] = 0.0, 0.0
        c.k[row, :, 0] = 39.0
    out = torch.full_like(q, 77.0)
    hs2.tree_attn(q, c.k, c.v, c.lens, tree_mask=words, out=out, **c.kw())
    want, bound = R.tree_reference(c, q, [N], masks, dtype)
    assert float(want.abs().max()) < 2.0 ** -20
    check(out, want, bound, ~want.isnan())


# ---------------------------------------------------------------- accepted paths
@pytest.mark.parametrize("dtype,width", [("bf16", 5), ("e4m3", 1), ("f32", 17)])
def test_tree_accept_path_narrower_than_the_draft(dtype, width):
    """A path of a few drafts out of a tree of many: the draft's size is num_draft, not the path's width."""
    lens, drafts = [500, 64, 129, 30], [64, 64, 40, 30]
    plen = [width, min(3, width), width + 9, 0]
    c = R.PagedCache(dtype, lens, 2, 128, 16, seed=3)
    g = torch.Generator().manual_seed(2)
    path = torch.stack([torch.randperm(n, generator=g)[:width].sort().values for n in (64, 64, 40, 30)]).to(torch.int32)
    before = c.snapshot()
    got = hs2.tree_accept(c.k, c.v, c.lens, path.cuda(), i32(plen), num_draft=i32(drafts), **c.kw())
    want = [None if x is None else x.clone() for x in before]
    new = []
    for b, (T, n) in enumerate(zip(lens, drafts)):
        a = min(plen[b], width, n)
        new.append(T - n + a)
        for i in range(a):
            src, dst = int(c.slots(b, T - n + int(path[b, i]))), int(c.slots(b, T - n + i))
            for x, y in zip(want, before):
                if x is not None:
                    x[dst] = y[src]
    assert got.tolist() == new
    for x, y in zip((c.k, c.v, c.k_scale, c.v_scale), want):
        assert x is None or torch.equal(R.bits(x), R.bits(y))


# ---------------------------------------------------------------- running sums
def weights(c, q, b, h, G, d):
    """Summed softmax probabilities of a group, and their error's bound relative to them: logits in fp32 sums, the
    exponent's rounding 2^-20 and the exponential 2^-21, G additions (R.attend() and the update kernel)."""
    k = c.wide("k", b, torch.arange(c.T[b]))[:, h]
    rows = q[b, h * G:(h + 1) * G].double()
    e = (d + 2) * 2.0 ** -24 * float((rows.abs() @ k.abs().T).amax()) / math.sqrt(d)
    return torch.softmax(rows @ k.T / math.sqrt(d), -1).sum(0), 2 * e + 2.0 ** -12 + (G + 2) * 2.0 ** -24


@pytest.mark.parametrize("dtype,G,page", [("bf16", 8, 64), ("e4m3", 4, 16), ("f32", 2, 0), ("bf16", 16, 32), ("f32", 8, 16)])
def test_accumulate_starts_each_sequences_own_new_tokens(dtype, G, page):
    """Sequences that gained different counts: the sums of each one's newest tokens start, all others are kept."""
    hkv, d, decay = 2, 128, 0.75
    lens, gained = [700, 77, 150, 0, 4099, 33, 5], [5, 0, 150, 3, 2 ** 31 - 1, 1, -4]
    c = R.PagedCache(dtype, lens, hkv, d, page, seed=51)
    q = torch.randn(len(lens), hkv * G, d, device="cuda", generator=gen(52)).to(R.q_dtype(dtype))
    acc0 = torch.rand(len(lens), hkv, c.cap, device="cuda", generator=gen(53)) * 5
    fresh = [max(0, min(n, T)) for n, T in zip(gained, lens)]
    for b, T in enumerate(lens):
        acc0[b, :, T - fresh[b]:] = NAN  # not read
    acc = acc0.clone()
    hs2.full_attn_accumulate(q, c.k, c.v, c.lens, acc, decay=decay, fresh=i32(gained), **c.kw())
    for b, T in enumerate(lens):
        for h in range(hkv):
            if T:
                w, slack = weights(c, q, b, h, G, d)
                old = acc0[b, h, :T].double() * decay
                old[T - fresh[b]:] = 0
                err = (acc[b, h, :T].double() - old - w).abs()
                assert bool((err <= slack * w + 2.0 ** -22 * old + 1e-30).all()), (b, h)
            assert torch.equal(R.bits(acc[b, h, T:]), R.bits(acc0[b, h, T:]))


# ---------------------------------------------------------------- the full layer's output beside its sums
@pytest.mark.parametrize("dtype,hkv,G,d,page", [
    ("bf16", 2, 8, 128, 64), ("bf16", 1, 32, 64, 16), ("bf16", 1, 1, 128, 0), ("e4m3", 1, 16, 128, 32), ("e4m3", 2, 8, 128, 64),
    ("f32", 2, 1, 64, 0), ("f32", 1, 8, 128, 16), ("f32", 3, 2, 128, 48), ("f32", 1, 4, 64, 64)])
def test_full_attn_accumulate_output_within_its_bound(dtype, hkv, G, d, page):
    """Elementwise, so that a segment left out or weighted wrongly shows: the oracle without a sixteenth of the positions
    must not pass (a quarter of the longest: outputs shrink with the root of the length, bounds do not).

    R.attend()'s bound holds for the full layer's kernels, but that weights over E4M3 are rounded to fp16: 2^-11 instead
    of 2^-8, and, normalised by the largest V scale so far, below 2^-14 by up to 2^-25 of it, times the row's code, where
    the sum of weights is at least 1."""
    lens = [1, 700, 0, 130, 4099, 20011]
    c = R.PagedCache(dtype, lens, hkv, d, page, seed=17)
    q = torch.randn(len(lens), hkv * G, d, device="cuda", generator=gen(18)).to(R.q_dtype(dtype))
    acc = torch.zeros(len(lens), hkv, c.cap, device="cuda")
    out, _ = hs2.full_attn_accumulate(q, c.k, c.v, c.lens, acc, **c.kw())
    for b, T in enumerate(lens):
        k, v = c.wide("k", b, torch.arange(T)), c.wide("v", b, torch.arange(T))
        seen = torch.ones(G, T, dtype=torch.bool, device="cuda")
        for h in range(hkv):
            rows, got = q[b, h * G:(h + 1) * G].double(), out[b, h * G:(h + 1) * G].double()
            want, bound, p = R.attend(rows, k[:, h], v[:, h], seen, dtype)
            if dtype == "e4m3" and T:
                s = c.slots(b, torch.arange(T))
                bound = bound - (2.0 ** -8 - 2.0 ** -11) * (p @ v[:, h].abs()) + 2.0 ** -25 * c.v_scale[s, h].max().double() * c.v[s, h].double().abs().sum(0)
            assert bool(((got - want).abs() <= bound).all()), (b, h, float(((got - want).abs() - bound).max()))
            if T >= 130:
                cut = T // 16 if T < 5000 else T // 4
                short, _, _ = R.attend(rows, k[cut:, h], v[cut:, h], seen[:, cut:], dtype)
                assert bool(((short - want).abs() > bound).any())


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("dtype,page", [("bf16", 16), ("e4m3", 64), ("f32", 0)])
def test_verify_accumulate_evict_reads_no_undefined_sum(dtype, page):
    """The sequence of the documentation: a drafted tree, its accepted path, the full layer with running sums, eviction.
    Sums behind a sequence's length are NaN before every step; none may reach a sum that counts."""
    hkv, G, d, N, B, budget, window, decay = 2, 4, 128, 6, 3, 40, 8, 0.9
    T = [38, 9, 60]
    c = R.PagedCache(dtype, T, hkv, d, page, seed=61, spare=40, poison=False)
    acc = torch.rand(B, hkv, c.cap, device="cuda", generator=gen(62))
    table, seen = hs2.rope_table(128), list(T)
    g = torch.Generator().manual_seed(63)
    for step in range(4):
        for b in range(B):
            acc[b, :, T[b]:] = NAN
        parents = [random_tree(N, 7 * step + b) for b in range(B)]
        nd = [N, 1 + step, N - 1]
        qkv = torch.randn(B, N, hkv * (G + 2), d, device="cuda", generator=gen(70 + step)).to(R.q_dtype(dtype))
        T = [t + n for t, n in zip(T, nd)]
        c.T, c.lens = T, i32(T)
        pos = i32([[s + i for i in range(N)] for s in seen])
        q = hs2.rope_append(qkv[:, :, :hkv * G], qkv[:, :, hkv * G:hkv * (G + 1)], qkv[:, :, hkv * (G + 1):], pos, table,
                            c.k, c.v, c.lens, num_new=i32(nd), **c.kw())
        hs2.tree_attn(q, c.k, c.v, c.lens, tree_mask=hs2.tree_mask(parents).cuda(), num_draft=i32(nd), **c.kw())
        path = []
        for b in range(B):
            i, p = int(torch.randint(0, nd[b], (), generator=g)), []
            while i >= 0:
                p.append(i)
                i = parents[b][i]
            path.append(p[::-1])
        plen, width = [len(p) for p in path], max(len(p) for p in path)
        c.lens = hs2.tree_accept(c.k, c.v, c.lens, i32([p + [0] * (width - len(p)) for p in path]), i32(plen), num_draft=i32(nd), **c.kw())
        T = [t - n + a for t, n, a in zip(T, nd, plen)]
        assert c.lens.tolist() == T
        c.T, seen = T, [s + a for s, a in zip(seen, plen)]
        q1 = torch.stack([q[b, path[b][-1]] for b in range(B)])
        acc0 = acc.clone()
        hs2.full_attn_accumulate(q1, c.k, c.v, c.lens, acc, decay=decay, fresh=i32(plen), **c.kw())
        for b in range(B):
            for h in range(hkv):
                w, slack = weights(c, q1, b, h, G, d)
                old = acc0[b, h, :T[b]].double() * decay
                old[T[b] - plen[b]:] = 0
                err = (acc[b, h, :T[b]].double() - old - w).abs()
                assert bool((err <= slack * w + 2.0 ** -22 * old + 1e-30).all()), (step, b, h)
        sums = acc.clone()
        c.lens, kept = hs2.cache_evict(c.k, c.v, c.lens, acc, budget, window, **c.kw())
        for b in range(B):
            for h in range(hkv):
                keep = R.kept_positions(sums[b, h, :T[b]].tolist(), T[b], budget, window)
                assert kept[b, h, :len(keep)].tolist() == keep
        c.T = T = c.lens.tolist()
    assert max(T) == budget


# ---------------------------------------------------------------- eviction
@pytest.mark.parametrize("budget", [64, 128, 200])
def test_cache_evict_default_window(budget):
    """Without a window given: 128 tokens, or the whole of a smaller budget."""
    cases = [R.PagedCache("bf16", [500, 50], 2, 128, 16, seed=71) for _ in (0, 1)]
    acc = torch.rand(2, 2, cases[0].cap, device="cuda", generator=gen(72))
    got = hs2.cache_evict(cases[0].k, cases[0].v, cases[0].lens, acc.clone(), budget, **cases[0].kw())
    want = hs2.cache_evict(cases[1].k, cases[1].v, cases[1].lens, acc.clone(), budget, min(128, budget), **cases[1].kw())
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    assert torch.equal(R.bits(cases[0].k), R.bits(cases[1].k))


# ---------------------------------------------------------------- E4M3 rows
def test_rope_append_and_kv_bridge_append_write_the_same_e4m3_rows():
    """The same bf16 rows through both appends: codes and scales equal, where x / scale lies next to the middle of two
    codes (x = a maximum's 448th times such a middle), among random, tiny and huge rows."""
    hkv, d, dm = 1, 128, 384
    rows = torch.randn(dm, d, generator=torch.Generator().manual_seed(81)).to(torch.bfloat16).double()
    middles = [m * 2.0 ** k for k in range(-9, 5) for m in (17, 19, 21, 23, 25, 27, 29, 31)]
    for a in range(1, 256):  # the maximum a / 256; elements that are bf16 and exactly in the middle, up to the scale's rounding
        x = [a / 256 * m / 448 for m in middles]
        x = [v for v in x if float(torch.tensor(v).to(torch.bfloat16)) == v and v <= a / 256]
        rows[a, 0] = a / 256
        rows[a, 1:] *= a / 256 / rows[a, 1:].abs().max()
        rows[a] = rows[a].to(torch.bfloat16).double()
        rows[a, 1:1 + len(x)] = torch.tensor(x[:d - 1], dtype=torch.float64) * torch.where(torch.arange(len(x[:d - 1])) % 2 > 0, -1.0, 1.0)
    for i, size in enumerate([2.0 ** -120, 2.0 ** -100, 2.0 ** -70, 2.0 ** -60, 2.0 ** -59, 2.0 ** 60, 2.0 ** 120]):
        rows[300 + i] = rows[85] * size
    rows[310] = 0
    w = rows.to(torch.bfloat16).cuda()
    hidden = torch.eye(dm, device="cuda", dtype=torch.bfloat16)  # sequence b's row is row b of w
    caches = [R.PagedCache("e4m3", [1] * dm, hkv, d, 16, seed=82, spare=3) for _ in (0, 1)]
    a, b = caches
    hs2.kv_bridge_append(hidden, w, w, a.k, a.v, a.lens, **a.kw())
    x = w.view(dm, 1, hkv, d)
    hs2.rope_append(None, x, x, torch.zeros(dm, 1, dtype=torch.int32, device="cuda"), hs2.rope_table(128), b.k, b.v, b.lens, **b.kw())
    # an element of -0 is 0 in the product's sum, which starts from +0: zeros of either sign are equal
    code = lambda t: torch.where(R.bits(t) == 0x80, torch.zeros_like(R.bits(t)), R.bits(t))  # noqa: E731
    assert torch.equal(code(a.k), code(b.k)) and torch.equal(code(a.v), code(b.v))
    assert torch.equal(R.bits(a.k_scale), R.bits(b.k_scale)) and torch.equal(R.bits(a.v_scale), R.bits(b.v_scale))


def test_rope_append_e4m3_codes_are_the_quotients():
    """Codes of many rows of all sizes against fp32 divisions by the stored scale, bit for bit."""
    B, N, hkv, d = 4, 257, 8, 128
    x = torch.randn(B, N, hkv, d, device="cuda", generator=gen(91))
    x *= torch.exp2(torch.randint(-130, 120, (B, N, hkv, 1), device="cuda", generator=gen(92)).float())
    x = x.bfloat16()
    c = R.PagedCache("e4m3", [N] * B, hkv, d, 64, seed=93)
    hs2.rope_append(None, x, x, torch.zeros(B, N, dtype=torch.int32, device="cuda"), hs2.rope_table(64), c.k, c.v, c.lens, **c.kw())
    top = x.float().abs().amax(-1)
    scale = top / torch.full_like(top, 448.0)  # by a tensor: a number's reciprocal would be multiplied
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    codes = (x.float() / scale.unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn)
    for b in range(B):
        s = c.slots(b, torch.arange(N))
        assert torch.equal(c.v_scale[s], scale[b]) and torch.equal(R.bits(c.v[s]), R.bits(codes[b]))


# ---------------------------------------------------------------- sizes at both ends
@pytest.mark.parametrize("dtype,elements", [("bf16", 2 ** 32), ("e4m3", 2 ** 32), ("f32", 2 ** 31)])
def test_calls_at_the_end_of_a_large_cache(dtype, elements):
    """Rows whose elements lie beyond 32 bits: the same results as in a small cache."""
    hkv, G, d, N, page, lens = 8, 2, 128, 4, 64, [300, 70, 129]
    small = R.PagedCache(dtype, lens, hkv, d, page, seed=33, poison=False)
    acc = torch.rand(len(lens), hkv, small.cap, device="cuda", generator=gen(34))
    n = small.k.shape[0]
    slots = (elements // (hkv * d) // page + 1) * page + n
    big = R.PagedCache(dtype, lens, hkv, d, page, seed=33, poison=False)
    for name in ("k", "v", "k_scale", "v_scale"):
        x = getattr(small, name)
        if x is not None:
            y = torch.empty((slots,) + tuple(x.shape[1:]), dtype=x.dtype, device="cuda")
            y[-n:] = x
            setattr(big, name, y)
    big.table = small.table + (slots - n) // page
    got = all_calls(big, N, lens, G, d, hkv, acc.clone(), dtype, 35)
    want = all_calls(small, N, lens, G, d, hkv, acc.clone(), dtype, 35)
    for x, y in zip(got, want):
        assert torch.equal(R.bits(x), R.bits(y))
    for name in ("k", "v", "k_scale", "v_scale"):
        x = getattr(small, name)
        assert x is None or torch.equal(R.bits(getattr(big, name)[-n:]), R.bits(x))


@pytest.mark.parametrize("dtype,G,N", [("bf16", 2, 3), ("e4m3", 1, 2), ("f32", 2, 2), ("f32", 8, 5)])
def test_calls_of_a_thousand_sequences(dtype, G, N):
    """More sequences than a warp or a block walks at once, a few tokens each, some without any."""
    hkv, d, B = 1, 128, 1100
    lens = [(7 * i) % 23 for i in range(B)]
    c, q, masks, words = tree_case(dtype, hkv, G, d, 16, N, lens, [N] * B, seed=36)
    out = torch.full_like(q, 77.0)
    hs2.tree_attn(q, c.k, c.v, c.lens, tree_mask=words, out=out, **c.kw())
    want, bound = R.tree_reference(c, q, [N] * B, masks, dtype)
    check(out, want, bound, ~want.isnan())
    acc = torch.full((B, hkv, c.cap), NAN, device="cuda")
    hs2.full_attn_accumulate(q[:, 0].contiguous(), c.k, c.v, c.lens, acc, fresh=c.lens, **c.kw())
    sums = acc.clone()
    for b in range(0, B, 41):
        if lens[b]:
            w, slack = weights(c, q[:, 0], b, 0, G, d)
            assert bool(((acc[b, 0, :lens[b]].double() - w).abs() <= slack * w).all())
    before = c.snapshot()
    lens_out, kept = hs2.cache_evict(c.k, c.v, c.lens, acc, 9, 2, **c.kw())
    assert lens_out.tolist() == [min(t, 9) for t in lens]
    for b in range(B):
        keep = R.kept_positions(sums[b, 0, :lens[b]].tolist(), lens[b], 9, 2)
        assert kept[b, 0].tolist() == keep + [-1] * (9 - len(keep))
        assert torch.equal(R.bits(c.v[c.slots(b, list(range(len(keep))))]), R.bits(before[1][c.slots(b, keep)]))


def test_tree_attn_chain_of_64():
    """The default mask at its widest, in each type."""
    for dtype in ("bf16", "e4m3", "f32"):
        c, q, _, _ = tree_case(dtype, 1, 4, 128, 64, 64, [64, 500], [64, 64], seed=37)
        out = torch.full_like(q, 77.0)
        hs2.tree_attn(q, c.k, c.v, c.lens, out=out, **c.kw())
        want, bound = R.tree_reference(c, q, [64, 64], [[(1 << i + 1) - 1 for i in range(64)]] * 2, dtype)
        check(out, want, bound, ~want.isnan())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
def test_tree_attn_queries_of_zero_and_of_all_sizes(dtype):
    """Rows of zeros see the mean of the values; tiny and large rows beside them."""
    c, q, masks, words = tree_case(dtype, 2, 4, 128, 64, 8, [700, 20], [8, 8], seed=38)
    q *= torch.tensor([0.0, 1e-38, 1e-30, 1e-3, 1.0, 3.0, 10.0, 30.0], device="cuda", dtype=q.dtype).view(1, 8, 1, 1)
    out = torch.full_like(q, 77.0)
    hs2.tree_attn(q, c.k, c.v, c.lens, tree_mask=words, out=out, **c.kw())
    want, bound = R.tree_reference(c, q, [8, 8], masks, dtype)
    check(out, want, bound, ~want.isnan())


# ---------------------------------------------------------------- pages outside the cache
@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
def test_moves_between_pages_outside_the_cache_move_nothing(dtype):
    """accept and evict with page numbers that the cache does not have: rows whose two places exist move, no other row
    changes."""
    lens, hkv, page, n, budget = [100, 90], 2, 16, 40, 50
    for call in ("accept", "evict"):
        c = R.PagedCache(dtype, lens, hkv, 128, page, seed=39, poison=False)
        good = c.table.clone()
        bad = [(0, 1, 2 ** 31 - 1), (0, 4, -3), (1, 0, c.k.shape[0] // page), (1, 5, -2 ** 31)]
        table = good.clone()
        for b, j, number in bad:
            table[b, j] = number
        exists = lambda b, t: all((b, t // page) != x[:2] for x in bad)  # noqa: B023, E731
        before = c.snapshot()
        kw = dict(c.kw(), page_table=table)
        moves = []
        if call == "accept":
            path = torch.arange(n - 1, -1, -2).repeat(2, 1)
            hs2.tree_accept(c.k, c.v, c.lens, path.to(torch.int32).cuda(), i32([20, 20]), num_draft=i32([n, n]), **kw)
            moves = [(b, T - n + int(path[b, i]), T - n + i, range(hkv)) for b, T in enumerate(lens) for i in range(20)]
        else:
            acc = torch.rand(2, hkv, c.cap, device="cuda", generator=gen(40))
            _, kept = hs2.cache_evict(c.k, c.v, c.lens, acc, budget, 10, **kw)
            moves = [(b, t, i, [h]) for b in range(2) for h in range(hkv) for i, t in enumerate(kept[b, h].tolist())]
        want = [None if x is None else x.clone() for x in before]
        for b, src, dst, heads in moves:
            if exists(b, src) and exists(b, dst):
                s, t = int(c.slots(b, src)), int(c.slots(b, dst))
                for x, y in zip(want, before):
                    if x is not None:
                        for h in heads:
                            x[t, h] = y[s, h]
        for x, y in zip((c.k, c.v, c.k_scale, c.v_scale), want):
            assert x is None or torch.equal(R.bits(x), R.bits(y)), call


# ---------------------------------------------------------------- captured
@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
def test_counts_are_read_at_every_replay(dtype):
    """Path widths, drafts' sizes and each sequence's new positions in a graph: other counts at every replay."""
    hkv, G, d, N, B = 2, 4, 128, 16, 3
    lens = [300, 60, 129]
    q = torch.randn(B, hkv * G, d, device="cuda", generator=gen(41)).to(R.q_dtype(dtype))
    cases = [R.PagedCache(dtype, lens, hkv, d, 16, seed=42, poison=False) for _ in (0, 1)]
    acc0 = torch.rand(B, hkv, cases[0].cap, device="cuda", generator=gen(43))
    ws = hs2.alloc_workspace(B, hkv, G, d, cases[0].cap)
    args = [dict(path=i32([[2, 5, 9]] * B), plen=i32([3] * B), nd=i32([N] * B), acc=acc0.clone(), lens=torch.zeros_like(c.lens),
                 out=torch.zeros_like(q)) for c in cases]

    def step(c, a):
        hs2.tree_accept(c.k, c.v, c.lens, a["path"], a["plen"], num_draft=a["nd"], lens_out=a["lens"], **c.kw())
        hs2.full_attn_accumulate(q, c.k, c.v, a["lens"], a["acc"], fresh=a["plen"], out=a["out"], workspace=ws, **c.kw())

    start = cases[0].snapshot()
    step(cases[0], args[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(cases[0], args[0])
    for path, plen, nd in (([[0, 1, 2], [3, 1, 15], [4, 4, 4]], [1, 3, 0], [16, 16, 5]), ([[7, 8, 9]] * 3, [0, 2, 9], [10, 9, 16])):
        for c, a in zip(cases, args):
            for x, y in zip((c.k, c.v, c.k_scale, c.v_scale), start):
                if x is not None:
                    x.copy_(y)
            a["path"].copy_(i32(path))
            a["plen"].copy_(i32(plen))
            a["nd"].copy_(i32(nd))
            a["acc"].copy_(acc0)
        g.replay()
        step(cases[1], args[1])
        torch.cuda.synchronize()
        for x, y in zip(cases[0].tensors() + list(args[0].values()), cases[1].tensors() + list(args[1].values())):
            assert torch.equal(R.bits(x), R.bits(y))
        a = [max(0, min(p, 3, n)) for p, n in zip(plen, nd)]
        assert args[0]["lens"].tolist() == [t - n + p for t, n, p in zip(lens, nd, a)]
