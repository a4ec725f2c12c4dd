"""The drafted-token and bounded-cache calls without a GPU: refusals and sizes that a caller relies on (nothing
launches)."""
import pytest
import torch

import test_draft_abi as abi
from long_context_decode_full_b200 import hs2
from test_draft_abi import FAKE, cache, ref


# ---------------------------------------------------------------- running sums
def accumulate_each(fresh=FAKE, lens=FAKE, acc=FAKE, stride=4096, ws=FAKE * 16, n=1 << 40):
    q, k = hs2.Heads(FAKE, 1, 2, 16, 128), cache()
    return hs2.lib().hs2_full_attn_accumulate_each(ref(q), ref(k), ref(k), lens, FAKE, 64, 0.5, fresh, acc, stride, ref(q), ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(fresh=None), hs2.ERR_INVALID_ARG), (dict(lens=None), hs2.ERR_INVALID_ARG), (dict(acc=FAKE + 2), hs2.ERR_INVALID_ARG),
    (dict(stride=4095), hs2.ERR_INVALID_ARG), (dict(ws=None), hs2.ERR_WORKSPACE), (dict(n=1024), hs2.ERR_WORKSPACE)])
def test_full_attn_accumulate_each_refuses(libhs2, kw, code):
    assert accumulate_each(**kw) == code
    assert hs2.last_error()


def test_fresh_counts_are_checked(libhs2):
    k, q = torch.zeros(256, 2, 128, dtype=torch.bfloat16), torch.zeros(2, 16, 128, dtype=torch.bfloat16)
    lens, acc = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 2, 128)
    for fresh, word in ((lens.long(), "dtype"), (lens[:1], "shape"), (lens.view(2, 1), "shape")):
        with pytest.raises(hs2.HS2Error, match=f"fresh: {word}"):
            hs2.full_attn_accumulate(q, k, k.clone(), lens, acc, fresh=fresh)


# ---------------------------------------------------------------- workspaces
@pytest.mark.parametrize("dtype,groups,dims", [(0, (1, 2, 4, 8), (64, 128)), (1, (1, 2, 8, 16, 32), (64, 128)), (2, (1, 8, 32), (128,))])
def test_tree_workspace_serves_every_smaller_call(libhs2, dtype, groups, dims):
    """A server that sizes its workspace for the longest draft and the largest batch: no smaller call asks for more."""
    for group in groups:
        for dim in dims:
            for heads in (1, 4):
                size = lambda b, n: hs2.tree_workspace_bytes(b, n, heads, group, dim, dtype)  # noqa: B023, E731
                for tokens in (1, 2, 5, 8, 16, 33, 64):
                    for batch in (1, 8, 64, 500):
                        most = size(batch, tokens)
                        assert all(size(b, n) <= most for b in (1, 2, batch) for n in range(1, tokens + 1) if b <= batch)


# ---------------------------------------------------------------- memory that arguments share
A = [FAKE + (i << 28) for i in range(16)]  # far apart: the caches of test_draft_abi.cache() have 2^25 bytes


def two_caches(**kw):
    return dict(kc=cache(data=A[0], **kw), vc=cache(data=A[1], **kw))


def refused(code, word):
    assert code == hs2.ERR_INVALID_ARG and word in hs2.last_error(), (code, hs2.last_error())


def test_calls_that_write_refuse_k_and_v_in_the_same_memory(libhs2):
    """K and V rows written side by side in one memory would overwrite each other."""
    e4m3 = dict(dtype=2)
    for kc, vc in ((cache(data=A[0]), cache(data=A[0])), (cache(data=A[0]), cache(data=A[0] + (1 << 25) - 256)),
                   (cache(data=A[0], scale=A[2], **e4m3), cache(data=A[1], scale=A[2] + 4, **e4m3)),
                   (cache(data=A[0]), cache(data=A[0] + 32 * 512))):  # half a page further
        refused(abi.rope(q=None, out=None, k=abi.tokens(h=2, data=A[3]), v=abi.tokens(h=2, data=A[4]), kc=kc, vc=vc), "caches overlap")
        refused(abi.accept(kc=kc, vc=vc, lens=A[5], path=A[6], plen=A[7], out=A[8], pt=A[9]), "caches overlap")
        refused(abi.evict(kc=kc, vc=vc, lens=A[5], acc=A[6], kept=A[7], out=A[8], pt=A[9]), "caches overlap")


def test_calls_that_write_refuse_contiguous_caches_a_sequence_apart(libhs2):
    """Without a page table every sequence has its place in both: V's first would be K's second."""
    kw = dict(kc=cache(data=A[0], page=1 << 14), vc=cache(data=A[0] + (512 << 14), page=1 << 14), pt=None)
    refused(abi.accept(lens=A[5], path=A[6], plen=A[7], out=A[8], pages=1, **kw), "caches overlap")
    refused(abi.evict(lens=A[5], acc=A[6], kept=A[7], out=A[8], pages=1, stride=1 << 14, **kw), "caches overlap")


@pytest.mark.parametrize("kw,word", [
    (dict(out=A[3] + 256), "q_out overlaps"), (dict(out=A[4]), "q_out overlaps"),
    (dict(out=A[2] + 4096), "q_out overlaps"),  # the next token's queries
    (dict(out=A[2] - 16), "q_out overlaps"),
])
def test_rope_append_refuses_memory_that_it_would_write_and_read(libhs2, kw, word):
    at = dict(dict(q=A[2], k=A[3], v=A[4], out=A[5]), **kw)
    refused(abi.rope(q=abi.tokens(data=at["q"]), k=abi.tokens(h=2, data=at["k"]), v=abi.tokens(h=2, data=at["v"]), out=at["out"],
                     pos=A[6], table=A[7], lens=A[8], pt=A[9], **two_caches()), word)


@pytest.mark.parametrize("q,out", [
    (dict(), dict(data=A[2] + 256)), (dict(), dict(data=A[2] - 4096)),
    (dict(stride=5120), dict(data=A[2] + 2 * 4000, stride=5120)),    # the last columns reach the next row's queries
    (dict(stride=5120), dict(data=A[2] + 2 * 2000, stride=5120)),
    (dict(stride=5120), dict(data=A[2] + 2 * 2048, stride=6144)),    # rows of other widths
    (dict(stride=5120), dict(data=A[2] - 2 * 2048 + 16, stride=5120)),
])
def test_tree_attn_refuses_an_output_on_its_queries(libhs2, q, out):
    refused(abi.tree(q=abi.tokens(data=A[2], **q), out=abi.tokens(**out), lens=A[5], pt=A[6], ws=A[7], **two_caches()), "out overlaps q")


@pytest.mark.parametrize("out", [A[5] + 4, A[6], A[6] + 4 * 15, A[7] + 4, A[9] + 4 * 127, A[9] - 4])
def test_tree_accept_refuses_lengths_on_its_inputs(libhs2, out):
    refused(abi.accept(lens=A[5], path=A[6], plen=A[7], out=out, pt=A[9], **two_caches()), "lens_out overlaps")


@pytest.mark.parametrize("kw,word", [
    (dict(out=A[5] + 4), "lens_out overlaps"), (dict(out=A[9] + 4), "lens_out overlaps"),
    (dict(kept=A[5] + 4), "kept overlaps"), (dict(kept=A[9] - 4), "kept overlaps"), (dict(kept=A[8] - 4 * 3999), "kept overlaps"),
    (dict(kept=A[6] + 4 * (2 * 2 * 4096 - 1)), "kept overlaps"), (dict(kept=A[6] - 4 * 3999), "kept overlaps")])
def test_cache_evict_refuses_results_on_its_inputs(libhs2, kw, word):
    at = dict(dict(kept=A[7], out=A[8]), **kw)
    refused(abi.evict(lens=A[5], acc=A[6], pt=A[9], **at, **two_caches()), word)


# ---------------------------------------------------------------- masks
@pytest.mark.parametrize("shape", [(1, 65), (2, 200), (3,), (1, 2, 2)])
def test_tree_mask_refuses_drafts_that_its_words_cannot_hold(shape):
    with pytest.raises(hs2.HS2Error):
        hs2.tree_mask(torch.full(shape, -1))
