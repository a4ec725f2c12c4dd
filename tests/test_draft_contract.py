"""The drafted-token and bounded-cache calls without a GPU: refusals and sizes that a caller relies on (nothing
launches)."""
import pytest
import torch

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
