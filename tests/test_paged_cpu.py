"""CPU checks of the paged serving operators: what the C calls refuse before any launch, and the plain forms the GPU tests use."""
import copy
import ctypes
import os
import pickle

import numpy as np
import pytest
import torch

from llama_decoder_block_kv_b200 import binding as B
from tests import paged_reference as R

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="library not built")

P16 = ctypes.c_void_p(4096)  # an aligned address that no refused call reads
GOOD = dict(n_heads=8, n_kv_heads=2, head_dim=128, page_size=16, num_pages=64, max_pages=8, dtype="bf16")


def page_args(**kw):
    return B.PageArgs(**(GOOD | kw)).c()


BAD_SHAPES = [dict(page_size=8), dict(page_size=48), dict(page_size=256), dict(page_size=0), dict(num_pages=0),
              dict(max_pages=0), dict(max_pages=1 << 27), dict(num_pages=1 << 27)]
BAD_HEADS = [dict(n_heads=7), dict(n_heads=0), dict(n_kv_heads=0), dict(n_kv_heads=-2), dict(head_dim=96), dict(head_dim=256),
             dict(num_pages=1 << 26, n_kv_heads=4)]


def plan(a, n=4, T=8, **kw):
    names = ("cached", "new", "table", "free", "count", "count_out", "cu", "kv", "pos", "slot", "status")
    p = {k: kw.get(k, P16) for k in names}
    return B.lib().llama_page_plan(None if a is None else ctypes.byref(a), p["cached"], p["new"], n, T,
                                   *[p[k] for k in names[2:]], None)


def append(a, stride=12 * 128, dtype=B.LLAMA_FP32, n=4, n_pos=9, **kw):
    p = {k: kw.get(k, P16) for k in ("qkv", "pos", "slot", "rope", "q", "k", "v", "st")}
    return B.lib().llama_rope_append(None if a is None else ctypes.byref(a), p["qkv"], stride, dtype, p["pos"], p["slot"], n,
                                     p["rope"], n_pos, p["q"], p["k"], p["v"], p["st"], None)


def paged(a, stride=8 * 128, B_=3, n=5, max_new=2, ws_bytes=1 << 40, **kw):
    p = {k: kw.get(k, P16) for k in ("q", "k", "v", "table", "cu", "kv", "out", "ws", "st")}
    return B.lib().llama_attn_paged(None if a is None else ctypes.byref(a), p["q"], stride, p["k"], p["v"], p["table"], p["cu"],
                                    p["kv"], B_, n, max_new, p["out"], p["ws"], ws_bytes, p["st"], None)


def packed(dtype=B.LLAMA_BF16, H=8, Hkv=2, D=128, qs=1024, ks=256, vs=256, B_=3, n=5, max_len=2, ws_bytes=1 << 40, **kw):
    p = {k: kw.get(k, P16) for k in ("q", "k", "v", "cu", "out", "ws", "st")}
    return B.lib().llama_attn_packed(dtype, H, Hkv, D, p["q"], qs, p["k"], ks, p["v"], vs, p["cu"], B_, n, max_len, p["out"],
                                     p["ws"], ws_bytes, p["st"], None)


@pytest.mark.parametrize("bad", BAD_SHAPES)
def test_shapes_are_refused(bad):
    a = page_args(**bad)
    assert plan(a) == append(a) == paged(a) == B.LLAMA_ERR_INVALID_ARGS


@pytest.mark.parametrize("bad", BAD_HEADS)
def test_heads_are_refused(bad):
    a = page_args(**bad)
    assert append(a, stride=1 << 20) == paged(a, stride=1 << 20) == B.LLAMA_ERR_INVALID_ARGS
    if "num_pages" not in bad:
        assert packed(H=a.n_heads, Hkv=a.n_kv_heads, D=a.head_dim, qs=1 << 20, ks=1 << 20, vs=1 << 20) == B.LLAMA_ERR_INVALID_ARGS
        assert B.lib().llama_attn_workspace_bytes(B.LLAMA_BF16, a.n_heads, a.n_kv_heads, a.head_dim) == B.LLAMA_ERR_INVALID_ARGS


def test_types_are_refused():
    a = page_args()
    a.dtype = 2
    assert append(a) == paged(a) == packed(dtype=2) == B.LLAMA_ERR_INVALID_ARGS
    assert append(page_args(), dtype=5) == B.LLAMA_ERR_INVALID_ARGS
    assert append(page_args(dtype="fp32"), dtype=B.LLAMA_BF16) == B.LLAMA_ERR_INVALID_ARGS
    assert plan(None) == append(None) == paged(None) == B.LLAMA_ERR_INVALID_ARGS


def test_sizes_strides_and_pointers_are_refused():
    a, odd, bad = page_args(), ctypes.c_void_p(4098), B.LLAMA_ERR_INVALID_ARGS
    for kw in (dict(n=0), dict(n=-1), dict(n=B.LLAMA_MAX_SEQS + 1), dict(T=0), dict(pos=ctypes.c_void_p(4100))):
        assert plan(a, **kw) == bad
    for kw in (dict(n=0), dict(n_pos=0), dict(stride=12 * 128 - 4), dict(stride=12 * 128 + 2), dict(stride=1 << 31),
               dict(dtype=B.LLAMA_BF16, stride=12 * 128 + 4)):
        assert append(a, **kw) == bad
    for kw in (dict(B_=0), dict(B_=B.LLAMA_MAX_SEQS + 1), dict(n=0), dict(max_new=0), dict(stride=1024 - 8),
               dict(stride=1024 + 4), dict(stride=-1024), dict(ws_bytes=0), dict(ws=ctypes.c_void_p(4096 + 16))):
        assert paged(a, **kw) == bad
    for kw in (dict(B_=0), dict(n=0), dict(max_len=0), dict(qs=1016), dict(ks=248), dict(vs=260), dict(ws_bytes=8)):
        assert packed(**kw) == bad
    for f, names in ((plan, "cached new table free count count_out cu kv pos slot status"), (append, "qkv pos slot rope q k v st"),
                     (paged, "q k v table cu kv out ws st")):
        for k in names.split():
            assert f(a, **{k: None}) == bad and f(a, **{k: odd}) == bad, k
    for k in "q k v cu out ws st".split():
        assert packed(**{k: None}) == bad and packed(**{k: odd}) == bad, k
    assert B.lib().llama_paged_status(None, None) == bad


def test_workspace_is_the_same_for_equal_shapes():
    assert B.llama_attn_workspace_bytes(32, 8, 128) == B.llama_attn_workspace_bytes(32, 8, 128) > 0
    assert B.strerror(B.LLAMA_ERR_PAGE_RANGE).startswith("page") and "pages" in B.strerror(B.LLAMA_ERR_OUT_OF_PAGES)


def test_plain_plan_on_a_worked_example():
    table = np.full((3, 4), -1)
    table[0, :1], table[2, :2] = [7], [4, 5]
    out, refused = R.plan([3, 0, 17], [14, 2, -1], 16, 4, 9, 20, table, np.array([0, 1, 2, 3, 6, -9, -9, -9, -9]), 5)
    assert not refused
    assert out["table"][0].tolist() == [7, 6, -1, -1] and out["table"][1].tolist() == [3, -1, -1, -1]
    assert out["cu"].tolist() == [0, 14, 16, 16] and out["kv"].tolist() == [17, 2, 0] and out["count"] == 5
    assert out["free"][:5].tolist() == [0, 1, 2, 4, 5]
    assert out["slot"][:3].tolist() == [7 * 16 + 3, 7 * 16 + 4, 7 * 16 + 5] and out["slot"][13:17].tolist() == [96, 48, 49, -1]


def test_plain_attention_is_the_library_attention():
    q, k, v = torch.randn(5, 4, 64), torch.randn(9, 2, 64), torch.randn(9, 2, 64)
    out, _, _ = R.attention(q, k, v)
    mask = torch.ones(5, 9, dtype=torch.bool).tril(4)
    want = torch.nn.functional.scaled_dot_product_attention(
        q.double().transpose(0, 1), k.double().transpose(0, 1), v.double().transpose(0, 1), attn_mask=mask, enable_gqa=True)
    assert torch.allclose(out, want.transpose(0, 1), atol=1e-12)
    assert (R.attention(q, k[:2], v[:2])[0][:3] == 0).all()


@pytest.mark.parametrize("M", [1, 2, 31, 129, 700, B.LLAMA_MAX_SEQS])
@pytest.mark.parametrize("H,Hkv", [(4, 4), (32, 8), (64, 8), (12, 4), (20, 1)])
def test_attention_lists_cover_every_tile_once(M, H, Hkv):
    """The lists of key tiles of the three attention kernels, walked on the host inside llama_selfcheck_plans: single
    tokens, chunks, whole prompts and mixtures of M requests, some without new tokens."""
    for S in (1, 130, 8192):
        for sms in (148, 7):
            assert B.lib().llama_selfcheck_plans(M, H * 64, H, Hkv, 1024, S, sms) == B.LLAMA_OK, (M, H, Hkv, S, sms)


def test_page_args_are_copied_and_pickled_after_use():
    a = B.PageArgs(**GOOD)
    a.ref()
    for b in (copy.copy(a), copy.deepcopy(a), pickle.loads(pickle.dumps(a))):
        assert b == a and b.ref() is not a.ref()
        b.num_pages += 1  # each with a C structure of its own
        assert b.ref()._obj.num_pages == a.ref()._obj.num_pages + 1 == a.num_pages + 1


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [64, 128])
def test_one_workspace_serves_every_head_layout(D, dtype):
    """Its size follows from dtype and head_dim alone: layers and models of other head counts share it."""
    sizes = {B.llama_attn_workspace_bytes(H, Hkv, D, dtype) for H, Hkv in ((1, 1), (4, 2), (32, 8), (64, 8), (20, 1), (17, 1), (1 << 16, 1))}
    assert len(sizes) == 1 and min(sizes) > 0


def test_lengths_whose_tiles_would_pass_32_bits_are_refused():
    """A request's last key tile and a call's last unit of rows end up to 255 past its keys and tokens."""
    bad = B.LLAMA_ERR_INVALID_ARGS
    for page in (16, 128):
        most = (2 ** 31 - 256) // page
        for k in range(1, 256 // page):
            a = page_args(max_pages=most + k, page_size=page)
            assert plan(a) == append(a) == paged(a) == bad
    for n in (2 ** 31 - 255, 2 ** 31 - 1):
        assert paged(page_args(), n=n) == packed(n=n) == bad
