"""The drafted-token and bounded-cache calls without a GPU: refusals with the documented codes (nothing launches), the
frequency table against its formula, tree masks, and the binding's own checks."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

import draft_ref as R
from long_context_decode_full_b200 import hs2

FAKE = 0x10000  # aligned, never dereferenced on the host


def cache(dtype=1, heads=2, dim=128, page=64, slots=1 << 16, scale=None, data=FAKE):
    return hs2.Cache(data, scale, dtype, heads, dim, page, slots)


def tokens(dtype=1, b=2, n=8, h=16, dim=128, data=FAKE, stride=None):
    return hs2.Tokens(data, dtype, b, n, h, dim, h * dim if stride is None else stride)


def ref(x):
    return None if x is None else ctypes.byref(x)


def rope(q=tokens(), k=tokens(h=2), v=tokens(h=2), pos=FAKE, table=FAKE, rot=128, lens=FAKE, new=None, pt=FAKE, pages=64,
         kc=cache(), vc=cache(), out=FAKE):
    return hs2.lib().hs2_rope_append(ref(q), ref(k), ref(v), pos, table, rot, 0, 1.0, lens, new, pt, pages, ref(kc), ref(vc), out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), hs2.ERR_INVALID_ARG),
    (dict(k=tokens(h=2, data=FAKE + 8)), hs2.ERR_INVALID_ARG),
    (dict(k=tokens(h=4)), hs2.ERR_INVALID_ARG),
    (dict(v=tokens(h=2, n=7)), hs2.ERR_INVALID_ARG),
    (dict(v=tokens(h=2, b=3)), hs2.ERR_INVALID_ARG),
    (dict(q=tokens(n=7)), hs2.ERR_INVALID_ARG),
    (dict(q=tokens(dtype=0)), hs2.ERR_UNSUPPORTED),
    (dict(k=tokens(h=2, stride=255)), hs2.ERR_INVALID_ARG),
    (dict(k=tokens(h=2, stride=260)), hs2.ERR_INVALID_ARG),  # not whole 16 bytes
    (dict(k=tokens(h=2, n=0)), hs2.ERR_INVALID_ARG),
    (dict(out=None), hs2.ERR_INVALID_ARG),
    (dict(out=FAKE + 4), hs2.ERR_INVALID_ARG),
    (dict(q=None), hs2.ERR_INVALID_ARG),                      # q_out without q
    (dict(q=tokens(stride=4096)), hs2.ERR_INVALID_ARG),       # in place, not contiguous
    (dict(pos=None), hs2.ERR_INVALID_ARG),
    (dict(table=None), hs2.ERR_INVALID_ARG),
    (dict(lens=None), hs2.ERR_INVALID_ARG),
    (dict(rot=8), hs2.ERR_UNSUPPORTED),
    (dict(rot=40), hs2.ERR_UNSUPPORTED),
    (dict(rot=144), hs2.ERR_UNSUPPORTED),
    (dict(pages=0), hs2.ERR_INVALID_ARG),
    (dict(pt=None), hs2.ERR_INVALID_ARG),
    (dict(pages=1 << 20), hs2.ERR_UNSUPPORTED),
    (dict(kc=cache(dtype=2), vc=cache(dtype=2)), hs2.ERR_INVALID_ARG),
    (dict(vc=cache(page=32)), hs2.ERR_INVALID_ARG),
    (dict(kc=cache(dtype=2, scale=FAKE), vc=cache(dtype=2, scale=FAKE + 2)), hs2.ERR_INVALID_ARG),
])
def test_rope_append_refuses(libhs2, kw, code):
    assert rope(**kw) == code
    assert hs2.last_error()


def tree(q=tokens(), kc=cache(), vc=cache(), lens=FAKE, pt=FAKE, pages=64, out=tokens(data=FAKE * 2), ws=FAKE * 16, n=1 << 40):
    return hs2.lib().hs2_tree_attn(ref(q), ref(kc), ref(vc), lens, None, None, pt, pages, ref(out), ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), hs2.ERR_INVALID_ARG),
    (dict(out=None), hs2.ERR_INVALID_ARG),
    (dict(out=tokens(n=9)), hs2.ERR_INVALID_ARG),
    (dict(out=tokens()), hs2.ERR_INVALID_ARG),  # out is q
    (dict(out=tokens(h=8)), hs2.ERR_INVALID_ARG),
    (dict(q=tokens(n=65), out=tokens(n=65, data=FAKE * 2)), hs2.ERR_UNSUPPORTED),
    (dict(q=tokens(n=0), out=tokens(n=0, data=FAKE * 2)), hs2.ERR_INVALID_ARG),
    (dict(q=tokens(h=17), out=tokens(h=17, data=FAKE * 2)), hs2.ERR_INVALID_ARG),
    (dict(q=tokens(h=24), out=tokens(h=24, data=FAKE * 2)), hs2.ERR_UNSUPPORTED),  # group 12
    (dict(q=tokens(h=32, dtype=0), out=tokens(h=32, dtype=0, data=FAKE * 2), kc=cache(dtype=0), vc=cache(dtype=0)), hs2.ERR_UNSUPPORTED),
    (dict(q=tokens(dim=64), out=tokens(dim=64, data=FAKE * 2)), hs2.ERR_INVALID_ARG),
    (dict(kc=cache(page=48), vc=cache(page=48)), hs2.ERR_UNSUPPORTED),
    (dict(q=tokens(b=4097), out=tokens(b=4097, data=FAKE * 2)), hs2.ERR_UNSUPPORTED),
    (dict(lens=None), hs2.ERR_INVALID_ARG),
    (dict(ws=None), hs2.ERR_WORKSPACE),
    (dict(ws=FAKE + 16), hs2.ERR_WORKSPACE),
    (dict(n=255), hs2.ERR_WORKSPACE),
    (dict(kc=None), hs2.ERR_INVALID_ARG),
])
def test_tree_attn_refuses(libhs2, kw, code):
    assert tree(**kw) == code
    assert hs2.last_error()


def accept(kc=cache(), vc=cache(), lens=FAKE, path=FAKE, plen=FAKE, b=2, m=8, pt=FAKE, pages=64, out=FAKE * 2):
    return hs2.lib().hs2_tree_accept(ref(kc), ref(vc), lens, None, path, plen, b, m, pt, pages, out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(lens=None), hs2.ERR_INVALID_ARG), (dict(path=None), hs2.ERR_INVALID_ARG), (dict(plen=None), hs2.ERR_INVALID_ARG),
    (dict(out=None), hs2.ERR_INVALID_ARG), (dict(out=FAKE), hs2.ERR_INVALID_ARG), (dict(out=FAKE + 4), hs2.ERR_INVALID_ARG),
    (dict(m=0), hs2.ERR_UNSUPPORTED), (dict(m=65), hs2.ERR_UNSUPPORTED), (dict(b=0), hs2.ERR_INVALID_ARG),
    (dict(b=4097), hs2.ERR_UNSUPPORTED), (dict(pages=0), hs2.ERR_INVALID_ARG)])
def test_tree_accept_refuses(libhs2, kw, code):
    assert accept(**kw) == code
    assert hs2.last_error()


def accumulate(kc=cache(), vc=cache(), lens=FAKE, acc=FAKE, stride=4096, fresh=1, ws=FAKE * 16, n=1 << 40):
    q = hs2.Heads(FAKE, 1, 2, 16, 128)
    return hs2.lib().hs2_full_attn_accumulate(ref(q), ref(kc), ref(vc), lens, FAKE, 64, 0.5, fresh, acc, stride, ref(q), ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(lens=None), hs2.ERR_INVALID_ARG), (dict(acc=None), hs2.ERR_INVALID_ARG), (dict(acc=FAKE + 2), hs2.ERR_INVALID_ARG),
    (dict(stride=4095), hs2.ERR_INVALID_ARG), (dict(fresh=-1), hs2.ERR_INVALID_ARG), (dict(ws=None), hs2.ERR_WORKSPACE),
    (dict(n=1024), hs2.ERR_WORKSPACE)])
def test_full_attn_accumulate_refuses(libhs2, kw, code):
    assert accumulate(**kw) == code
    assert hs2.last_error()


def evict(kc=cache(), vc=cache(), lens=FAKE, b=2, pt=FAKE, pages=64, acc=FAKE, stride=4096, budget=1000, window=128, kept=FAKE,
          out=FAKE * 2):
    return hs2.lib().hs2_cache_evict(ref(kc), ref(vc), lens, b, pt, pages, acc, stride, budget, window, kept, out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(lens=None), hs2.ERR_INVALID_ARG), (dict(acc=None), hs2.ERR_INVALID_ARG), (dict(acc=FAKE + 1), hs2.ERR_INVALID_ARG),
    (dict(kept=None), hs2.ERR_INVALID_ARG), (dict(out=None), hs2.ERR_INVALID_ARG), (dict(out=FAKE), hs2.ERR_INVALID_ARG),
    (dict(out=FAKE + 4), hs2.ERR_INVALID_ARG),
    (dict(budget=0), hs2.ERR_INVALID_ARG), (dict(budget=2 ** 31 - 1), hs2.ERR_INVALID_ARG), (dict(window=-1), hs2.ERR_INVALID_ARG),
    (dict(window=1001), hs2.ERR_INVALID_ARG), (dict(stride=4095), hs2.ERR_INVALID_ARG), (dict(b=0), hs2.ERR_INVALID_ARG),
    (dict(pages=0), hs2.ERR_INVALID_ARG)])
def test_cache_evict_refuses(libhs2, kw, code):
    assert evict(**kw) == code
    assert hs2.last_error()


@pytest.mark.parametrize("rot,kw", [
    (128, {}), (16, dict(base=500000.0)), (48, dict(scaling="linear", factor=8.0)), (64, dict(scaling="ntk", factor=4.0)),
    (64, dict(scaling="yarn", factor=32.0, original_context=4096.0)),
    (128, dict(base=500000.0, scaling="bands", factor=8.0, original_context=8192.0))])
def test_rope_table_is_the_formula(libhs2, rot, kw):
    t = hs2.rope_table(rot, device="cpu", **kw)
    f, scale = R.inv_freq(rot, **dict(dict(base=10000.0), **kw))
    assert t.rot_dim == rot and t.turns.shape == (rot // 2,) and t.scale == pytest.approx(scale, rel=2.0 ** -23)
    for word, radians in zip(t.turns.tolist(), f.tolist()):
        turns = Fraction(word, 2 ** 64)  # below half a turn: no sign bit
        # pow, log and the division by 2 pi in 64 bits: a few units of 2^-53, and half a unit of the table
        assert abs(float(turns) - radians / (2 * math.pi)) <= 2.0 ** -48 * radians + 2.0 ** -65


@pytest.mark.parametrize("kw", [dict(rot_dim=8), dict(rot_dim=40), dict(rot_dim=144), dict(rot_dim=64, base=1.0),
                                dict(rot_dim=64, base=math.nan), dict(rot_dim=64, scaling="linear", factor=0.5),
                                dict(rot_dim=64, scaling="yarn", factor=2.0), dict(rot_dim=64, scaling="spiral"),
                                dict(rot_dim=64, scaling="yarn", factor=2.0, original_context=10.0, beta_fast=1.0, beta_slow=2.0),
                                dict(rot_dim=64, scaling="bands", factor=2.0, original_context=10.0, low_freq_factor=4.0),
                                dict(rot_dim=64, scaling="linear", factor=math.inf)])
def test_rope_table_refuses(libhs2, kw):
    with pytest.raises(hs2.HS2Error):
        hs2.rope_table(device="cpu", **kw)


def test_tree_mask_words():
    m = hs2.tree_mask([[-1, 0, 0, 1, -1], [-1, 0, 1, 2, 3]])
    assert m.tolist() == [[1, 3, 5, 11, 16], [1, 3, 7, 15, 31]]
    chain = hs2.tree_mask([[i - 1 for i in range(64)]])
    assert int(chain[0, 63]) == -1 and int(chain[0, 62]) == 2 ** 63 - 1
    for bad in ([[0]], [[-2]], [[-1, 1]]):
        with pytest.raises(hs2.HS2Error):
            hs2.tree_mask(bad)


def test_binding_checks_what_pointers_cannot_carry(libhs2):
    """Element types, ranks, shapes, strides and devices; on the CPU no call gets as far as a launch."""
    k = torch.zeros(256, 2, 128, dtype=torch.bfloat16)
    q = torch.zeros(2, 4, 16, 128, dtype=torch.bfloat16)
    kv = torch.zeros(2, 4, 2, 128, dtype=torch.bfloat16)
    lens, pos = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32)
    t = hs2.rope_table(64, device="cpu")
    acc = torch.zeros(2, 2, 128)
    calls = [
        lambda: hs2.tree_attn(q.float(), k, k, lens),
        lambda: hs2.tree_attn(q[0], k, k, lens),
        lambda: hs2.tree_attn(q.transpose(1, 2), k, k, lens),
        lambda: hs2.tree_attn(q[:, ::2], k, k, lens),
        lambda: hs2.tree_attn(q, k, k, lens.long()),
        lambda: hs2.tree_attn(q, k, k, lens[:1]),
        lambda: hs2.tree_attn(q, k, k, lens, tree_mask=torch.zeros(2, 4, dtype=torch.int32)),
        lambda: hs2.tree_attn(q, k, k, lens, tree_mask=torch.zeros(2, 5, dtype=torch.int64)),
        lambda: hs2.tree_attn(q, k, k, lens, page_table=torch.zeros(2, 2, dtype=torch.int32)),
        lambda: hs2.tree_attn(q, k, k, lens, out=q.clone(), workspace=torch.zeros(1 << 20, dtype=torch.uint8)),
        lambda: hs2.tree_attn(q, k.view(-1), k, lens),
        lambda: hs2.tree_attn(q, k.half(), k.half(), lens),
        lambda: hs2.rope_append(q, kv, kv, pos.long(), t, k, k, lens),
        lambda: hs2.rope_append(q, kv, kv, pos[:, :3], t, k, k, lens),
        lambda: hs2.rope_append(q, kv.float(), kv, pos, t, k, k, lens),
        lambda: hs2.rope_append(q, kv, kv, pos, t, k, k, lens, q_out=q.float()),
        lambda: hs2.rope_append(q, kv, kv, pos, t, k, k, lens),
        lambda: hs2.tree_accept(k, k, lens, pos.long(), lens),
        lambda: hs2.tree_accept(k, k, lens, pos, lens[:1]),
        lambda: hs2.tree_accept(k, k, lens, pos, lens),
        lambda: hs2.full_attn_accumulate(q[:, 0].contiguous(), k, k, lens, acc.double()),
        lambda: hs2.full_attn_accumulate(q[:, 0].contiguous(), k, k, lens, acc[:1]),
        lambda: hs2.full_attn_accumulate(q[:, 0].contiguous(), k, k, lens, acc),
        lambda: hs2.cache_evict(k, k, lens, acc, 16, kept=torch.zeros(2, 2, 15, dtype=torch.int32)),
        lambda: hs2.cache_evict(k, k, lens, acc[0], 16),
        lambda: hs2.cache_evict(k, k, lens, acc, 16),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(hs2.HS2Error):
            call()
            pytest.fail(f"call {i} was not refused")
