"""The serving operators over a paged cache where values are not finite, lengths are malformed and calls overlap."""
import threading
import time

import numpy as np
import pytest
import torch

from llama_decoder_block_kv_b200 import binding as B
from tests import paged_reference as R
from tests.test_gpu_paged import DT, LEFT, Paged, check_attention, ints, normal, status_word, workspace

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def put(p, which, at, value, cols=slice(None), request=0):
    """`value` in columns `cols` of key `at` of a request, in the pages and in the request's own copy."""
    t, q, k, v = p.seqs[request]
    b = [i for i, (n, _) in enumerate(p.lens) if n][request]
    page = p.a.page_size
    (p.kp if which == "k" else p.vp)[int(p.table[b, at // page]), :, at % page, cols] = value
    x = (k if which == "k" else v).clone()
    x[at, :, cols] = value
    p.seqs[request] = (t, q, x, v) if which == "k" else (t, q, k, x)


def same_kinds(p, what=""):
    """NaN, infinities and finite values stand where the 64-bit form has them, the finite ones within two roundings of
    the storage type and of P (the bound's weights would be infinite next to infinite values)."""
    assert B.llama_paged_status(p.st) == (B.LLAMA_OK, 0), what
    for t, q, k, v in p.seqs:
        want, _, _ = R.attention(q, k, v)
        got = p.out[t:t + q.shape[0]].double()
        for kind in (torch.isnan, torch.isposinf, torch.isneginf):
            wrong = int((kind(got) != kind(want)).sum())
            assert wrong == 0, (what, t, kind.__name__, wrong)
        fine = torch.isfinite(want)
        assert ((got - want)[fine].abs() <= 2.0 ** -6 * (want[fine].abs() + 1)).all(), (what, t)


# ------------------------------------------------------------------ NaN scores alone in a tile

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H,Hkv,D", [(4, 2, 64), (4, 4, 64), (8, 2, 128), (16, 1, 128)])
@pytest.mark.parametrize("n,kv", [(1, 321), (1, 577), (1, 641), (3, 321), (3, 641), (40, 1025)])
def test_a_nan_key_alone_in_its_tile_reaches_the_row(n, kv, H, Hkv, D, dtype):
    """The newest key has a key tile, and so a CTA, of its own, and its scores are NaN: the rows that see it are NaN,
    the others as they would be without it."""
    p = Paged([(n, kv)], H, Hkv, D, 16, dtype)
    put(p, "k", kv - 1, NAN)
    p.call()
    assert torch.isnan(p.out[n - 1].float()).all()
    same_kinds(p)


# ------------------------------------------------------------------ infinite values

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H,Hkv,D", [(8, 2, 128), (4, 4, 64), (16, 1, 128), (20, 1, 64)])
@pytest.mark.parametrize("kv,at", [(1, 0), (17, 16), (40, 3), (65, 64), (130, 0), (3000, 1), (3000, 2999)])
def test_single_tokens_see_infinite_values(kv, at, H, Hkv, D, dtype):
    """An infinite value of a key that a single token sees is infinite in its row, whatever the key's weight."""
    p = Paged([(1, kv), (1, 70)], H, Hkv, D, 32, dtype)
    put(p, "v", at, INF, slice(0, None, 2))
    put(p, "v", at, -INF, slice(1, None, 4))
    p.call()
    same_kinds(p, "one key")
    if kv > 1:
        put(p, "v", (at + kv // 2) % kv, INF, slice(0, None, 3))  # meets the first one's signs: NaN there
        p.call()
        same_kinds(p, "two keys")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H,Hkv,D", [(8, 2, 128), (4, 4, 64), (5, 1, 64), (3, 3, 128)])
@pytest.mark.parametrize("n,kv", [(2, 2), (40, 40), (130, 130), (300, 300), (300, 1000), (20, 3000), (257, 513)])
def test_values_that_are_not_finite_at_every_place(n, kv, H, Hkv, D, dtype):
    """Values that are not finite before the new tokens, among them, at the first and at the last: in whole units and in
    cut ones, each row has what the keys that it sees give."""
    places = sorted({0, max(kv - n - 1, 0), kv - n, kv - n + n // 3, kv - n // 2, kv - 2, kv - 1})
    for i, at in enumerate(places):
        p = Paged([(n, kv), (1, 65)], H, Hkv, D, 16, dtype, seed=i)
        put(p, "v", at, (INF, NAN, -INF)[i % 3], slice(i % 3, None, 3))
        p.call()
        same_kinds(p, at)
    p = Paged([(n, kv), (1, 65)], H, Hkv, D, 16, dtype, seed=9)
    for i, at in enumerate(places):
        put(p, "v", at, (INF, -INF, NAN)[i % 3], slice(i, None, 5))
    p.call()
    same_kinds(p, "all of them")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H,Hkv,D", [(8, 2, 128), (4, 4, 64), (16, 1, 128), (20, 1, 64)])
@pytest.mark.parametrize("n", [1, 5])
def test_huge_values_of_no_weight_count_nothing(n, H, Hkv, D, dtype):
    """Values near the type's largest under keys whose weight is zero in fp32 (scores 256 below the others)."""
    kv = 150
    p = Paged([(n, kv)], H, Hkv, D, 16, dtype)
    p.wide.fill_(8.0)
    p.kp.fill_(4.0 * (64 / D) ** 0.5)  # scores of 256
    p.vp.fill_(1.0)
    for at in (0, 3, 70, 129, kv - n - 1):
        page, off = int(p.table[0, at // 16]), at % 16
        p.kp[page, :, off], p.vp[page, :, off] = 0, 3e38
    p.call()
    assert B.llama_paged_status(p.st) == (B.LLAMA_OK, 0)
    # Weights of 1 and 0: whole numbers times their own reciprocals, two roundings of 2^-24, (1 + 2^-24)^2 - 1 < 2^-22;
    # in bf16 the nearest value is 1.
    assert ((p.out[:n].double() - 1).abs() <= (2.0 ** -22 if dtype == "fp32" else 0)).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,kv", [(1, 300), (5, 300), (140, 400), (3, 3000)])
def test_a_huge_value_under_a_score_somewhat_above_the_others(n, kv, dtype):
    """One key scores 5 (7.2 in powers of two) above the others, which come before and behind it, and holds values of 3e36: its
    weight times them stays finite, as the maximum of the scores so far is never more than the score itself."""
    p = Paged([(n, kv)], 8, 2, 128, 16, dtype)
    t, q, k, v = p.seqs[0]
    p.wide.fill_(1.0)
    k, v = torch.zeros_like(k), torch.ones_like(v)
    at = kv - n - 1
    k[at], v[at] = 5 / 128 ** 0.5, 3e36
    page = p.a.page_size
    for j in range(kv):
        p.kp[int(p.table[0, j // page]), :, j % page], p.vp[int(p.table[0, j // page]), :, j % page] = k[j], v[j]
    p.seqs = [(t, q, k, v)]
    p.call()
    check_attention(p.out[:n], [(0, q, k, v)], p.dt)
    assert B.llama_paged_status(p.st) == (B.LLAMA_OK, 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_packed_values_that_are_not_finite(dtype):
    """The same over packed rows, K and V slices of one matrix, in the middle of a batch."""
    H, Hkv, D, lens = 8, 2, 128, [33, 290, 5]
    N, c = sum(lens), np.concatenate([[0], np.cumsum(lens)]).tolist()
    x = normal((N, H + 2 * Hkv, D), DT[dtype], 7)
    q, k, v = x[:, :H], x[:, H: H + Hkv], x[:, H + Hkv:]
    for at, val, cols in ((33, INF, slice(0, None, 7)), (33 + 63, -INF, slice(1, None, 7)), (33 + 64, NAN, slice(2, None, 7)),
                          (33 + 200, INF, slice(3, None, 7)), (33 + 289, -INF, slice(0, None, 7))):
        v[at, :, cols] = val
    out = torch.full((N, H, D), LEFT, dtype=DT[dtype], device="cuda")
    st = status_word()
    B.llama_attn_packed(q, k, v, ints(c), max(lens), out, workspace(H, Hkv, D, dtype), st)
    assert B.llama_paged_status(st) == (B.LLAMA_OK, 0)
    for b in (0, 2):
        check_attention(out[c[b]:c[b + 1]], [(0, q[c[b]:c[b + 1]], k[c[b]:c[b + 1]], v[c[b]:c[b + 1]])], DT[dtype])
    want, _, _ = R.attention(q[33:323], k[33:323], v[33:323])
    got = out[33:323].double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.isinf(got), torch.isinf(want))
    fine = torch.isfinite(want)
    assert ((got - want)[fine].abs() <= 2.0 ** -6 * (want[fine].abs() + 1)).all()


def device_ms(f, n=5):
    f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    best = INF
    for _ in range(n):
        a.record()
        f()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_an_infinite_value_does_not_make_the_call_slow(dtype):
    """A value that is not finite at the start of a prompt is seen by every row; it costs no more than other values."""
    H, Hkv, D, n = 4, 1, 128, 8192
    q, k, v = (normal((n, h, D), DT[dtype], i) for i, h in enumerate((H, Hkv, Hkv)))
    out, ws, st = torch.empty((n, H, D), dtype=DT[dtype], device="cuda"), workspace(H, Hkv, D, dtype), status_word()

    def call():
        B.llama_attn_packed(q, k, v, ints([0, n]), n, out, ws, st)

    clean = device_ms(call)
    v[0, :, 5] = INF
    assert device_ms(call) < 2 * clean  # an order of magnitude lies between the two when rows are computed one by one
    assert (out[:, :, 5] == INF).all() and torch.isfinite(out[:, :, 6:].float()).all()
    assert B.llama_paged_status(st) == (B.LLAMA_OK, 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_values_that_are_not_finite_over_a_very_long_history(dtype):
    """A chunk over 600 thousand keys: an infinity at the first and NaN at the last of them leave the other columns as they
    are, bit by bit, and the call neither times out nor takes more than about twice as long."""
    n, kv, H, D = 140, 600_000, 4, 128
    p = Paged([(n, kv)], H, 1, D, 128, dtype)
    clean = device_ms(p.call, 3)
    want = p.call().clone()
    p.vp[int(p.table[0, 0]), :, 0, 5] = INF
    last = int(p.table[0, (kv - 1) // 128])
    p.vp[last, :, (kv - 1) % 128, 9] = NAN
    p.vp[last, :, (kv - 2) % 128, 11] = -INF
    p.out.fill_(LEFT)
    assert device_ms(p.call, 3) < 3 * clean
    assert B.llama_paged_status(p.st) == (B.LLAMA_OK, 0)
    assert (p.out[:n, :, 5] == INF).all()
    assert torch.isnan(p.out[n - 1, :, 9]).all() and (p.out[n - 2: n, :, 11] == -INF).all()
    want[:, :, 5], want[n - 1, :, 9], want[n - 2: n, :, 11] = p.out[:, :, 5], 0, -INF
    p.out[n - 1, :, 9] = 0
    want[n:], p.out[n:] = 0, 0
    assert torch.equal(p.out, want)


# ------------------------------------------------------------------ the status word

def test_a_flag_raised_right_after_a_status_call_is_kept():
    """Another thread keeps the default stream busy, so that whatever a status call leaves running there runs late: a flag
    that the next call raises on a stream of its own must still stand."""
    a = B.PageArgs(1, 1, 64, 16, 4, 2)
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, new, table, free = ints([0]), ints([1]), torch.zeros((1, 2), **i32), torch.zeros(4, **i32)
    none, c_out, cu, kv, pos, slot = ints([0]), ints([0]), torch.zeros(2, **i32), torch.zeros(1, **i32), torch.zeros(4, **i32), torch.zeros(4, **i32)
    st, side, done = status_word(), torch.cuda.Stream(), threading.Event()
    torch.cuda.synchronize()

    def busy():
        while not done.is_set():
            for _ in range(3):
                torch.cuda._sleep(150_000)
            time.sleep(2.4e-4)

    other = threading.Thread(target=busy)
    other.start()
    try:
        for i in range(4000):  # a clear that runs late lost about one flag in 80
            B.llama_paged_status(st)
            # no page is free: the plan is refused with a flag
            B.llama_page_plan(a, lens, new, table, free, none, c_out, cu, kv, pos, slot, st, stream=side)
            side.synchronize()
            assert B.llama_paged_status(st) == (B.LLAMA_ERR_OUT_OF_PAGES, 16), i
    finally:
        done.set()
        other.join()
        torch.cuda.synchronize()


def test_the_status_word_is_the_current_devices():
    for bad in (torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError):
            B.llama_paged_status(bad)
    host = torch.ones(1, dtype=torch.int32)
    assert B.lib().llama_paged_status(host.data_ptr(), None) == B.LLAMA_ERR_INVALID_ARGS and int(host) == 1
    st = status_word()
    st.fill_(2 + 8)
    assert B.llama_paged_status(st) == (B.LLAMA_ERR_PAGE_RANGE, 10) and int(st) == 0


# ------------------------------------------------------------------ malformed lengths

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 6])
def test_malformed_starts_leave_rows_alone(n, dtype):
    """Whatever cu holds, only the rows of requests with valid bounds are written, with their own values."""
    p = Paged([(n, 40), (n, 33), (n, 300)], 4, 2, 64, 16, dtype)
    N = 3 * n
    q_all, hist = p.q, [(k, v) for _, _, k, v in p.seqs]
    rows = p.out.shape[0]
    for cu in ([0, n, n - 1, N], [0, n, 10 ** 6, 10 ** 6], [-5, n, n, N], [2 ** 31 - 1, -2 ** 31, 0, 0], [0, N, n, 2 * n],
               [0, n, 2 * n, rows + 1], [0, 0, -1, N], [n, 0, n, 2 * n]):
        p.cu.copy_(ints(cu))
        p.out.fill_(LEFT)
        p.call(max_new=n)
        good = [0 <= a <= b <= rows and b - a <= n for a, b in zip(cu, cu[1:])]
        assert not all(good)
        assert B.llama_paged_status(p.st) == (B.LLAMA_ERR_POS_RANGE, 2), cu
        check_attention(p.out, [(a, q_all[a:b], *hist[i]) for i, (a, b) in enumerate(zip(cu, cu[1:])) if good[i] and b > a], p.dt, cu)


# ------------------------------------------------------------------ a block over a paged cache

def block_workload(act, **kw):
    import oracle as O
    from llama_decoder_block_kv_b200 import synth

    return synth.Workload(**(dict(name="paged block edges", dim=256, n_layers=1, n_heads=4, n_kv_heads=2, ffn_hidden=O.ffn_hidden_dim(256, 256),
                                  vocab_size=0, multiple_of=256, ffn_dim_multiplier=None, norm_eps=1e-5, rope_theta=10000.0,
                                  max_batch_size=1, max_seq_len=64, act=act, batch=1, seed=9, norm_weights="random") | kw))


class Block:
    """One request's tokens through a paged block: its pages, tables and a call."""

    def __init__(self, w, ctx, n):
        from llama_decoder_block_kv_b200 import synth

        self.ctx, self.a = ctx, B.PageArgs(w.n_heads, w.n_kv_heads, w.head_dim, 16, 8, 4, w.act)
        self.h = synth.hidden(w, (1, n, w.dim), call=1)[0].to("cuda").contiguous()
        self.kp, self.vp = (torch.zeros((8, w.n_kv_heads, 16, w.head_dim), dtype=DT[w.act], device="cuda") for _ in range(2))
        self.table, self.cu, self.kv = ints([[5, 2, 7, 0]]), ints([0, n]), ints([n])
        self.pos, self.slot = ints(list(range(n))), ints([(5, 2, 7, 0)[i // 16] * 16 + i % 16 for i in range(n)])
        self.ws = torch.zeros(B.llama_block_paged_workspace_bytes(ctx, n), dtype=torch.uint8, device="cuda")
        self.st, self.n = status_word(), n

    def call(self, **kw):
        x = dict(h=self.h, table=self.table) | kw
        B.llama_block_forward_paged(self.ctx, 0, x["h"], self.a, self.kp, self.vp, x["table"], self.cu, self.kv, self.pos, self.slot, self.n,
                                    self.ws, self.st)


def test_a_block_runs_on_its_contexts_device(monkeypatch):
    """The tensors' device counts, not the current one; tensors that are not on the context's device are refused."""
    import ctypes

    from tests.gpu_util import Pair

    w = block_workload("bf16")
    pair = Pair(w)
    try:
        want = Block(w, pair.ctx, 20)
        want.call()
        b = Block(w, pair.ctx, 20)
        with monkeypatch.context() as m:
            m.setattr(torch.cuda, "current_device", lambda: torch.cuda.device_count())
            b.call()
            for kw in (dict(h=b.h.cpu()), dict(table=b.table.cpu())):
                with pytest.raises(ValueError):
                    b.call(**kw)
        torch.cuda.synchronize()
        assert torch.equal(b.h, want.h) and torch.equal(b.kp, want.kp) and torch.equal(b.vp, want.vp)
        host = torch.zeros((20, w.dim))
        code = B.lib().llama_block_forward_paged(
            pair.ctx, 0, ctypes.c_void_p(host.data_ptr()), b.a.ref(), *[x.data_ptr() for x in (b.kp, b.vp, b.table, b.cu, b.kv, b.pos, b.slot)],
            1, 20, 20, b.ws.data_ptr(), b.ws.numel(), b.st.data_ptr(), None)
        assert code == B.LLAMA_ERR_INVALID_ARGS and (host == 0).all()
    finally:
        pair.close()


@pytest.mark.parametrize("act", ["fp32", "bf16"])
def test_pages_of_a_half_split_block_hold_interleaved_pairs(act):
    """The same weights given in the half-split order: the same hidden states and the same pages, bit by bit."""
    import dataclasses

    from llama_decoder_block_kv_b200 import synth
    from tests.gpu_util import Pair
    from tests.test_gpu_rope_half_split import _to_half_split

    w = block_workload(act)
    lw = synth.layer_weights(w, 0, device="cpu")
    lw["wq"], lw["wk"] = (_to_half_split(lw[k], n, w.head_dim) for k, n in (("wq", w.n_heads), ("wk", w.n_kv_heads)))
    pair, half = Pair(w), B.Llama(dataclasses.replace(B.ModelArgs.from_workload(w), rope_half_split=True))
    try:
        B.llama_set_layer(half.ctx, 0, {k: v.cuda().contiguous() for k, v in lw.items()})
        a, b = Block(w, pair.ctx, 40), Block(w, half.ctx, 40)
        for x in (a, b):
            x.call()
            assert B.llama_paged_status(x.st) == (B.LLAMA_OK, 0)
        assert torch.equal(a.h, b.h) and torch.equal(a.kp, b.kp) and torch.equal(a.vp, b.vp)
        assert (a.kp[[5, 2]] != 0).any(-1).all() and (a.kp[7, :, :8] != 0).any(-1).all() and not a.kp[[0, 1, 3, 4, 6]].any()
    finally:
        half.close()
        pair.close()
