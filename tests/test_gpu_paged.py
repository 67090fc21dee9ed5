"""The serving operators over a paged cache on the GPU, each against its plain 64-bit form (paged_reference.py)."""
import random

import numpy as np
import pytest
import torch

from llama_decoder_block_kv_b200 import binding as B
from tests import paged_reference as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
LEFT = 776.0  # what rows that a call leaves alone hold (a bf16 value)


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def normal(shape, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def workspace(H, Hkv, D, dtype):
    return torch.zeros(B.llama_attn_workspace_bytes(H, Hkv, D, dtype), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ page plan

def run_plan(cached, new, page, max_pages, num_pages, max_tokens, table, free, count, alias=False):
    a = B.PageArgs(1, 1, 64, page, num_pages, max_pages)
    t, f, c = ints(table), ints(free), ints([count])
    c_out = c if alias else ints([-5])
    lens = ints(cached)
    kv = lens if alias else torch.full_like(lens, -5)
    cu = torch.full((len(new) + 1,), -5, dtype=torch.int32, device="cuda")
    pos, slot = (torch.full((max_tokens,), -5, dtype=torch.int32, device="cuda") for _ in range(2))
    st = status_word()
    B.llama_page_plan(a, lens, ints(new), t, f, c, c_out, cu, kv, pos, slot, st)
    code, flags = B.llama_paged_status(st)
    n = lambda x: x.cpu().numpy()  # noqa: E731
    return {"table": n(t), "free": n(f), "count": int(c_out), "cu": n(cu), "kv": n(kv), "pos": n(pos), "slot": n(slot)}, code, flags


def same_plan(got, want):
    for k, w in want.items():
        assert np.array_equal(got[k], w), k


def plan_case(seed, n, page, hi, ended=0.1, spare=3):
    r = random.Random(seed)
    cached = [r.choice([0, 1, page - 1, page, page + 1, r.randint(0, hi)]) for _ in range(n)]
    new = [-1 if r.random() < ended else r.choice([0, 1, 1, page, r.randint(0, hi)]) for _ in range(n)]
    max_pages = -(-2 * hi // page) + 3
    held = [-(-c // page) for c in cached]
    need = sum(-(-(c + x) // page) - h for c, x, h in zip(cached, new, held) if x >= 0)
    num_pages = sum(held) + need + spare
    ids = list(range(num_pages))
    r.shuffle(ids)
    table = np.full((n, max_pages), -3, np.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = ids[at: at + h]
        at += h
    count = num_pages - at
    free = np.full(num_pages, -9, np.int32)
    free[:count] = ids[at:]
    return cached, new, page, max_pages, num_pages, sum(max(x, 0) for x in new) + r.choice([1, 2, 7]), table, free, count


@pytest.mark.parametrize("seed,n,page,hi,alias", [
    (0, 1, 16, 5, False), (1, 2, 128, 300, True), (2, 33, 16, 40, False), (3, 513, 32, 70, True), (4, 1000, 64, 200, False),
    (5, 4096, 16, 33, True), (6, 7, 16, 9000, False), (7, 511, 128, 900, False)])
def test_plan_equals_the_plain_form(seed, n, page, hi, alias):
    case = plan_case(seed, n, page, hi)
    got, code, flags = run_plan(*case, alias=alias)
    want, refused = R.plan(*case)
    assert not refused and (code, flags) == (B.LLAMA_OK, 0)
    same_plan(got, want)


@pytest.mark.parametrize("what,flag", [("pages", 16), ("tokens", 2), ("row", 2), ("negative", 2), ("count", 16), ("overflow", 2)])
def test_plan_that_cannot_be_met_changes_nothing(what, flag):
    cached, new, page, max_pages, num_pages, max_tokens, table, free, count = plan_case(11, 40, 16, 60, ended=0.0)
    if what == "pages":
        need = sum(-(-(c + x) // page) - -(-c // page) for c, x in zip(cached, new))
        count = need - 1
    elif what == "tokens":
        max_tokens = sum(new) - 1
    elif what == "row":
        new[3] = max_pages * page - cached[3] + 1
        max_tokens, count = 10 ** 6, num_pages
    elif what == "negative":
        cached[5] = -1
    elif what == "count":
        count = num_pages + 1
    else:
        new = [2 ** 31 - 1 - c for c in cached]  # sums far past 32 bits
    case = (cached, new, page, max_pages, num_pages, max_tokens, table, free, count)
    got, code, flags = run_plan(*case)
    want, refused = R.plan(*case)
    assert refused and flags & flag, flags
    assert code in (B.LLAMA_ERR_POS_RANGE, B.LLAMA_ERR_OUT_OF_PAGES)
    same_plan(got, want)


def test_plan_flags_page_numbers_outside_the_pool():
    case = plan_case(13, 20, 16, 50, ended=0.3)
    cached, new, page, max_pages, num_pages, max_tokens, table, free, count = case
    ended = next(b for b, (c, n) in enumerate(zip(cached, new)) if n < 0 and c > 0)
    part = next(b for b, (c, n) in enumerate(zip(cached, new)) if n > 0 and c % page)
    table[ended, 0] = num_pages
    table[part, cached[part] // page] = -2
    free[count - 1] = 1 << 30
    got, code, flags = run_plan(*case)
    want, refused = R.plan(*case)
    assert not refused and (code, flags) == (B.LLAMA_ERR_PAGE_RANGE, 8)
    same_plan(got, want)


def test_plan_pages_come_back_and_go_out_again():
    """Requests join, grow and end over many steps: no page is ever held twice, none is lost."""
    r, page, n, num_pages, max_pages = random.Random(3), 16, 12, 60, 20
    table, free, count, cached = np.full((n, max_pages), -1, np.int32), np.arange(num_pages, dtype=np.int32), num_pages, [0] * n
    for _ in range(25):
        new = [-1 if c > 150 or (c and r.random() < 0.1) else r.choice([0, 1, 1, r.randint(1, 40)]) for c in cached]
        got, code, _ = run_plan(cached, new, page, max_pages, num_pages, 600, table, free, count, alias=True)
        want, refused = R.plan(cached, new, page, max_pages, num_pages, 600, table, free, count)
        same_plan(got, want)
        assert refused == (code != B.LLAMA_OK)
        table, free, count, cached = got["table"], got["free"], got["count"], got["kv"].tolist()
        held = [p for b in range(n) for p in table[b, : -(-cached[b] // page)]]
        assert sorted(held + free[:count].tolist()) == list(range(num_pages))


# ------------------------------------------------------------------ RoPE + append

def rope_table(n_pos, D, theta=10000.0):
    ang = torch.arange(n_pos, dtype=torch.float64)[:, None] * theta ** -(torch.arange(0, D, 2, dtype=torch.float64) / D)
    return torch.stack([ang.cos(), ang.sin()], -1).float().cuda().contiguous()


@pytest.mark.parametrize("n,H,Hkv,D,page,dtype,in_dtype,pad", [
    (1, 4, 2, 64, 16, "fp32", "fp32", 0), (33, 4, 4, 64, 128, "fp32", "fp32", 8), (1, 32, 8, 128, 16, "bf16", "fp32", 0),
    (70, 6, 2, 128, 32, "bf16", "bf16", 24), (257, 5, 1, 64, 64, "bf16", "fp32", 4)])
def test_rope_append(n, H, Hkv, D, page, dtype, in_dtype, pad):
    P, n_pos = -(-n // page) + 3, 5000
    a = B.PageArgs(H, Hkv, D, page, P, 4, dtype)
    wide = normal((n, (H + 2 * Hkv) * D + pad), DT[in_dtype], 1)
    qkv = wide[:, : (H + 2 * Hkv) * D]
    r = random.Random(n)
    slots = r.sample(range(P * page), n)
    pos = [r.randrange(n_pos) for _ in range(n)]
    pos[-1] = n_pos - 1
    skip = n // 2 if n > 1 else None
    if skip is not None:
        slots[skip] = -1
    cs = rope_table(n_pos, D)
    q_out = torch.full((n, H, D), LEFT, dtype=DT[dtype], device="cuda")
    kp, vp = (torch.full((P, Hkv, page, D), LEFT, dtype=DT[dtype], device="cuda") for _ in range(2))
    st = status_word()
    B.llama_rope_append(a, qkv, ints(pos), ints(slots), cs, q_out, kp, vp, st)
    assert B.llama_paged_status(st) == (B.LLAMA_OK, 0)
    x = qkv.double().view(n, H + 2 * Hkv, D)
    t = cs[torch.tensor(pos, device="cuda")][:, None]
    turned = R.rope(x[:, : H + Hkv], t)
    # two products and a sum in fp32, then one rounding to the storage type
    mag = R.rope(x[:, : H + Hkv].abs(), torch.stack([t[..., 0].abs(), -t[..., 1].abs()], -1)).abs() + turned.abs()
    u = 2.0 ** -8 if dtype == "bf16" else 0.0
    tol = u * turned.abs() + 3 * 2.0 ** -24 * (1 + u) * (mag + x[:, : H + Hkv].abs())
    want_q = torch.full((n, H, D), LEFT, dtype=torch.float64, device="cuda")
    want_k, want_v = (torch.full((P, Hkv, page, D), LEFT, dtype=torch.float64, device="cuda") for _ in range(2))
    tol_q, tol_k = torch.zeros_like(want_q), torch.zeros_like(want_k)
    for i, s in enumerate(slots):
        if s < 0:
            continue
        want_q[i], tol_q[i] = turned[i, :H], tol[i, :H]
        want_k[s // page, :, s % page], tol_k[s // page, :, s % page] = turned[i, H:], tol[i, H:]
        want_v[s // page, :, s % page] = x[i, H + Hkv:].to(DT[dtype]).double()
    assert ((q_out.double() - want_q).abs() <= tol_q).all()
    assert ((kp.double() - want_k).abs() <= tol_k).all()
    assert torch.equal(vp.double(), want_v)


def test_rope_append_skips_and_flags_bad_positions_and_slots():
    a = B.PageArgs(2, 1, 64, 16, 3, 2, "bf16")
    qkv, cs = normal((6, 4 * 64), torch.bfloat16, 2), rope_table(10, 64)
    for pos, slots, code, good in (([0, 10, 2, 3, 4, 5], [0, 1, 2, 3, 4, 5], B.LLAMA_ERR_POS_RANGE, [0, 2, 3, 4, 5]),
                                   ([0, -1, 2, 3, 4, 5], [0, 1, 2, 3, 4, 5], B.LLAMA_ERR_POS_RANGE, [0, 2, 3, 4, 5]),
                                   ([0, 1, 2, 3, 4, 5], [0, 48, 2, 3, -2, 5], B.LLAMA_ERR_PAGE_RANGE, [0, 2, 3, 5])):
        q = torch.full((6, 2, 64), LEFT, dtype=torch.bfloat16, device="cuda")
        k, v = (torch.full((3, 1, 16, 64), LEFT, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        st = status_word()
        B.llama_rope_append(a, qkv, ints(pos), ints(slots), cs, q, k, v, st)
        assert B.llama_paged_status(st)[0] == code
        assert [i for i in range(6) if (q[i] != LEFT).any()] == good
        assert sorted(i for i in range(48) if (v.view(3, 16, 64)[i // 16, i % 16] != LEFT).any()) == sorted(slots[i] for i in good)


# ------------------------------------------------------------------ attention

def check_attention(got, seqs, dtype, what=""):
    """got [N][H][D]; seqs: (first row, q, k, v) of each request."""
    covered = torch.zeros(got.shape[0], dtype=torch.bool, device="cuda")
    for q0, q, k, v in seqs:
        n = q.shape[0]
        out, A, E = R.attention(q, k, v)
        tol = R.attention_bound(out, A, E, k.shape[0], dtype)
        x = got[q0: q0 + n].double()
        assert torch.isfinite(x).all(), (what, q0)
        bad = (x - out).abs() > tol
        assert not bad.any(), (what, q0, n, k.shape[0], int(bad.sum()), bad.nonzero()[:3].tolist(),
                               float((x - out).abs().max()), float((x - out).abs()[bad].max()))
        covered[q0: q0 + n] = True
    assert (got[~covered] == LEFT).all(), what


class Paged:
    """A paged batch: new tokens and keys per request; everything that no request owns holds NaN or rubbish."""

    def __init__(self, lens, H, Hkv, D, page, dtype, seed=0, q_pad=0, rows_after=3):
        r = random.Random(seed)
        self.lens, self.dt = lens, DT[dtype]
        B_, N = len(lens), sum(n for n, _ in lens)
        pages = [-(-kv // page) for _, kv in lens]
        P, cols = sum(pages) + 5, max(pages + [1]) + 2
        ids = list(range(P))
        r.shuffle(ids)
        self.a = B.PageArgs(H, Hkv, D, page, P, cols, dtype)
        self.kp, self.vp = (torch.full((P, Hkv, page, D), float("nan"), dtype=self.dt, device="cuda") for _ in range(2))
        table = np.array([[r.choice([-1, P, 2 ** 31 - 1, -2 ** 31]) for _ in range(cols)] for _ in range(B_)], np.int64)
        ks, vs = normal((sum(kv for _, kv in lens) + 1, Hkv, D), self.dt, seed + 1), normal((sum(kv for _, kv in lens) + 1, Hkv, D), self.dt, seed + 2)
        self.wide = normal((N + rows_after, H * D + q_pad), self.dt, seed + 3)
        self.q = self.wide[:, : H * D].unflatten(1, (H, D))
        self.seqs, at, t = [], 0, 0
        for b, (n, kv) in enumerate(lens):
            mine, ids = ids[: pages[b]], ids[pages[b]:]
            table[b, : pages[b]] = mine
            k, v = ks[at: at + kv], vs[at: at + kv]
            at += kv
            for j in range(pages[b]):
                m = min(page, kv - j * page)
                self.kp[mine[j], :, :m] = k[j * page: j * page + m].transpose(0, 1)
                self.vp[mine[j], :, :m] = v[j * page: j * page + m].transpose(0, 1)
            if n:
                self.seqs.append((t, self.q[t: t + n], k, v))
            t += n
        self.table = ints(table)
        self.cu = ints(np.concatenate([[0], np.cumsum([n for n, _ in lens])]))
        self.kv = ints([kv for _, kv in lens])
        self.max_new = max([n for n, _ in lens] + [1])
        self.ws, self.st = workspace(H, Hkv, D, dtype), status_word()
        self.out = torch.full((N + rows_after, H, D), LEFT, dtype=self.dt, device="cuda")

    def call(self, max_new=None, out=None, **kw):
        B.llama_attn_paged(self.a, self.q, self.kp, self.vp, self.table, self.cu, self.kv, max_new or self.max_new,
                           self.out if out is None else out, self.ws, self.st, **kw)
        return self.out if out is None else out

    def check(self, what=""):
        check_attention(self.out, self.seqs, self.dt, what)
        assert B.llama_paged_status(self.st) == (B.LLAMA_OK, 0)


HEADS = [(4, 4, 128), (8, 2, 128), (8, 1, 128), (12, 4, 64), (5, 1, 64), (16, 1, 128), (20, 1, 64)]
SINGLE = [[(1, 1)], [(1, 2), (0, 5), (1, 17)], [(1, 130), (1, 1), (1, 64), (1, 65), (0, 0)], [(1, 1000)], [(1, 3), (1, 700), (1, 129)],
          [(1, 5000), (0, 40)]]
CHUNKS = [[(2, 2)], [(3, 20), (1, 1), (0, 9)], [(17, 17), (1, 300), (5, 128)], [(64, 64), (65, 129)], [(130, 130), (1, 2), (3, 260)],
          [(257, 400)], [(33, 1500), (2, 1500)]]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", SINGLE)
def test_paged_single_tokens(lens, dtype, page):
    for i, (H, Hkv, D) in enumerate(HEADS):
        if (i + page // 16 + len(lens)) % 2:  # half of the head layouts with each page size
            continue
        p = Paged(lens, H, Hkv, D, page, dtype, seed=i)
        p.call()
        p.check((H, Hkv, D))


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", CHUNKS)
def test_paged_chunks(lens, dtype, page):
    for i, (H, Hkv, D) in enumerate(HEADS):
        if (i + page // 16 + len(lens)) % 3:  # a third of the head layouts with each page size
            continue
        p = Paged(lens, H, Hkv, D, page, dtype, seed=i, q_pad=8 * i)
        p.call()
        p.check((H, Hkv, D))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", [[(1, 0)], [(3, 1), (2, 0), (4, 4)], [(1, 0), (1, 33)], [(140, 7), (130, 0)]])
def test_paged_rows_that_see_no_key_are_zero(lens, dtype):
    p = Paged(lens, 4, 2, 128, 16, dtype)
    p.call()
    p.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("single", [True, False])
def test_paged_many_requests(single, dtype):
    """More requests than CTAs, most of them short; more units than one wave."""
    r = random.Random(5)
    lens = [(1 if single else r.choice([0, 1, 1, 2, 9]), 0) for _ in range(700)]
    lens = [(n, n + r.choice([0, 0, 3, 15, 16, 40])) for n, _ in lens]
    p = Paged(lens, 2, 1, 64, 16, dtype)
    p.call()
    p.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", [[(1, 40), (1, 3), (1, 300)], [(5, 40), (1, 3), (70, 300)]])
def test_paged_flags(lens, dtype):
    """Malformed lengths skip their request only; a page outside the pool counts as zeros."""
    p = Paged(lens, 4, 2, 64, 16, dtype)
    p.kv[1] = p.a.max_pages * 16 + 1
    p.call()
    assert B.llama_paged_status(p.st) == (B.LLAMA_ERR_POS_RANGE, 2)
    q1 = p.seqs.pop(1)
    check_attention(p.out, p.seqs, p.dt)
    p.kv[1] = -1
    p.call()
    assert B.llama_paged_status(p.st) == (B.LLAMA_ERR_POS_RANGE, 2)
    check_attention(p.out, p.seqs, p.dt)
    p.kv[1] = lens[1][1]
    for bad in (p.a.num_pages, -1, 2 ** 31 - 1, -2 ** 31):
        keep = int(p.table[2, 1])
        p.table[2, 1] = bad
        p.call()
        assert B.llama_paged_status(p.st) == (B.LLAMA_ERR_PAGE_RANGE, 8)
        t, q, k, v = p.seqs[-1]
        k, v = k.clone(), v.clone()
        k[16:32], v[16:32] = 0, 0
        check_attention(p.out, [p.seqs[0], q1, (t, q, k, v)], p.dt, bad)
        p.table[2, 1] = keep
    n = lens[0][0]
    if n > 1:
        p.out.fill_(LEFT)
        p.call(max_new=n - 1)  # requests 0 and 2 have more
        assert B.llama_paged_status(p.st) == (B.LLAMA_ERR_POS_RANGE, 2)
        check_attention(p.out, [q1], p.dt)
    for cu in ([0, n, n - 2, 2], [0, n, 10 ** 6, 10 ** 6], [-5, n, n + 1, n + 2], [2 ** 31 - 1, -2 ** 31, 0, 0]):
        p.cu.copy_(ints(cu))
        p.call()
        assert B.llama_paged_status(p.st) == (B.LLAMA_ERR_POS_RANGE, 2)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_later_keys_do_not_reach_earlier_rows(what, dtype):
    """NaN or infinities in the K and V rows of later tokens leave earlier tokens' rows as they are."""
    for n, kv, at in ((40, 40, 20), (200, 333, 300), (130, 700, 699)):
        p = Paged([(n, kv), (2, 150)], 8, 2, 128, 16, dtype)
        page, off = int(p.table[0, at // 16]), at % 16
        bad = float(what)
        p.kp[page, :, off] = bad
        p.vp[page, :, off] = bad
        p.call()
        assert B.llama_paged_status(p.st) == (B.LLAMA_OK, 0)
        t, q, k, v = p.seqs[0]
        before = at - (kv - n)  # rows that do not see the key
        out, A, E = R.attention(q[:before], k[: kv - n + before], v[: kv - n + before])
        tol = R.attention_bound(out, A, E, kv, p.dt)
        assert ((p.out[:before].double() - out).abs() <= tol).all()
        assert not torch.isfinite(p.out[before: n].float()).all(-1).any()
        t, q, k, v = p.seqs[1]
        check_attention(p.out[t:t + 2], [(0, q, k, v)], p.dt)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_large_and_lowest_scores(dtype):
    """Scores far apart (one key takes all), and all of them far below zero."""
    for scale in (30.0, 1e3):
        p = Paged([(3, 200), (70, 90), (1, 500)], 4, 1, 64, 32, dtype)
        p.wide *= scale
        p.call()
        p.check(scale)
    p = Paged([(3, 200), (70, 90)], 4, 1, 64, 32, dtype)
    p.wide.copy_(p.wide.abs() * 100)
    p.kp.copy_(-p.kp.abs())
    p.seqs = [(t, q, -k.abs(), v) for t, q, k, v in p.seqs]
    p.call()
    p.check("all scores negative")


def packed(lens, H, Hkv, D, dtype, seed=0, fused=False, rows_after=2):
    N = sum(lens) + rows_after
    if fused:
        x = normal((N, H + 2 * Hkv, D), DT[dtype], seed)
        q, k, v = x[:, :H], x[:, H: H + Hkv], x[:, H + Hkv:]
    else:
        q, k, v = (normal((N, h, D), DT[dtype], seed + i) for i, h in enumerate((H, Hkv, Hkv)))
    return q, k, v, ints(np.concatenate([[0], np.cumsum(lens)]))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", [[1], [2, 1, 0, 3], [127, 128, 129], [300, 1, 1, 50], [513], [0, 0, 40]])
def test_packed(lens, dtype):
    for i, (H, Hkv, D) in enumerate(HEADS):
        if (i + len(lens)) % 2:
            continue
        q, k, v, cu = packed(lens, H, Hkv, D, dtype, seed=i, fused=i % 4 < 2)
        if len(lens) > 1:
            k[sum(lens):] = float("nan")
            v[sum(lens):] = float("nan")
        out = torch.full((q.shape[0], H, D), LEFT, dtype=DT[dtype], device="cuda")
        st = status_word()
        B.llama_attn_packed(q, k, v, cu, max(lens), out, workspace(H, Hkv, D, dtype), st)
        assert B.llama_paged_status(st) == (B.LLAMA_OK, 0)
        c = cu.tolist()
        check_attention(out, [(c[b], q[c[b]:c[b + 1]], k[c[b]:c[b + 1]], v[c[b]:c[b + 1]]) for b in range(len(lens)) if lens[b]],
                        DT[dtype], (H, Hkv, D))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_packed_neighbours_do_not_reach_each_other(dtype):
    """A sequence of NaN and infinities between two others changes neither."""
    lens = [45, 30, 200]
    q, k, v, cu = packed(lens, 8, 2, 128, dtype)
    for x in (q, k, v):
        x[45:75] = float("nan")
        x[60:70] = float("inf")
    out = torch.full((q.shape[0], 8, 128), LEFT, dtype=DT[dtype], device="cuda")
    st = status_word()
    B.llama_attn_packed(q, k, v, cu, 200, out, workspace(8, 2, 128, dtype), st)
    assert B.llama_paged_status(st) == (B.LLAMA_OK, 0)
    out[45:75] = LEFT
    check_attention(out, [(c, q[c:c + n], k[c:c + n], v[c:c + n]) for c, n in ((0, 45), (75, 200))], DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", [SINGLE[4], CHUNKS[2], [(300, 2000), (1, 1800)]])
def test_equal_calls_give_equal_bits_and_leave_the_workspace_ready(lens, dtype):
    p = Paged(lens, 8, 2, 128, 16, dtype)
    first = p.call().clone()
    for _ in range(5):
        p.out.fill_(LEFT)
        assert torch.equal(p.call(), first)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 40])
def test_captured_calls_follow_the_lengths_and_share_nothing(n, dtype):
    """Two graphs with a workspace each, replayed on two streams; the lengths change between replays."""
    ps = [Paged([(n, 900), (n, 300), (1, 77)], 8, 2, 128, 32, dtype, seed=s) for s in (1, 2)]
    graphs = []
    for p in ps:
        p.call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.call()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in ps]
    for turn, kv0 in enumerate((900, 500, n, 899)):
        for p in ps:
            p.kv[0] = kv0
            t, q, k, v = p.seqs[0]
            p.full = getattr(p, "full", (k, v))
            p.seqs[0] = (t, q, p.full[0][:kv0], p.full[1][:kv0])
            p.out.fill_(LEFT)
        torch.cuda.synchronize()
        for _ in range(3):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for p in ps:
            p.check(turn)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_steps_of_a_server(dtype):
    """Plan, append and attention step by step with requests that join, grow by chunks and tokens, and end, against
    each request's own history; whole prompts also through the packed attention."""
    H, Hkv, D, page, P, cols, n_pos = 8, 2, 128, 16, 64, 24, 400
    a = B.PageArgs(H, Hkv, D, page, P, cols, dtype)
    dt, r = DT[dtype], random.Random(8)
    n_req, T = 6, 260
    table = torch.full((n_req, cols), -1, dtype=torch.int32, device="cuda")
    free, count = torch.arange(P, dtype=torch.int32, device="cuda"), ints([P])
    kv = torch.zeros(n_req, dtype=torch.int32, device="cuda")
    cu = torch.zeros(n_req + 1, dtype=torch.int32, device="cuda")
    pos, slot = (torch.zeros(T, dtype=torch.int32, device="cuda") for _ in range(2))
    kp, vp = (torch.full((P, Hkv, page, D), float("nan"), dtype=dt, device="cuda") for _ in range(2))
    cs, ws, st = rope_table(n_pos, D), workspace(H, Hkv, D, dtype), status_word()
    hist = [[None, None] for _ in range(n_req)]  # K and V rows as stored
    for step in range(14):
        have = [0 if h[0] is None else len(h[0]) for h in hist]
        new = [-1 if n > 180 else r.choice([1, 1, 1, 0]) if n else r.choice([0, 33, 64, r.randint(1, 70)]) for n in have]
        if step == 5:
            new = [1 if n else 0 for n in have]  # a step of single tokens
        B.llama_page_plan(a, kv, ints(new), table, free, count, count, cu, kv, pos, slot, st)
        qkv = normal((T, (H + 2 * Hkv) * D), torch.float32, 100 + step)
        q = torch.full((T, H, D), LEFT, dtype=dt, device="cuda")
        B.llama_rope_append(a, qkv, pos, slot, cs, q, kp, vp, st)
        out = torch.full((T, H, D), LEFT, dtype=dt, device="cuda")
        B.llama_attn_paged(a, q, kp, vp, table, cu, kv, max(max(new), 1), out, ws, st)
        assert B.llama_paged_status(st) == (B.LLAMA_OK, 0)
        seqs, t, fresh = [], 0, []
        for b, n in enumerate(new):
            if n < 0:
                hist[b] = [None, None]
                continue
            turned = R.rope(qkv[t:t + n].view(n, H + 2 * Hkv, D)[:, : H + Hkv],
                            cs[have[b]: have[b] + n][:, None]).to(dt)
            rows = [gather_new(kp, table[b], have[b], n), gather_new(vp, table[b], have[b], n)]
            # rounding of one fp32 value may fall to either side of a tie: a step of the storage type
            step_size = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -20
            assert ((rows[0].double() - turned[:, H:].double()).abs() <= step_size * turned[:, H:].double().abs() + 1e-6).all()
            assert torch.equal(rows[1], qkv[t:t + n].view(n, H + 2 * Hkv, D)[:, H + Hkv:].to(dt))
            hist[b] = rows if hist[b][0] is None else [torch.cat([o, x]) for o, x in zip(hist[b], rows)]
            if n:
                seqs.append((t, q[t:t + n], *hist[b]))
                if have[b] == 0:
                    fresh.append((t, n, *rows))
            t += n
        check_attention(out, seqs, dt, step)
        for t, n, k, v in fresh:
            one = torch.full((n, H, D), LEFT, dtype=dt, device="cuda")
            B.llama_attn_packed(q[t:t + n], k, v, ints([0, n]), n, one, ws, st)
            check_attention(one, [(0, q[t:t + n], k, v)], dt, step)


def gather_new(pages, row, start, n):
    P, Hkv, ps, D = pages.shape
    j = torch.arange(start, start + n, device="cuda")
    return pages[row.long()[j // ps], :, j % ps]


def test_binding_refuses_what_the_calls_cannot_take():
    p = Paged([(2, 40)], 4, 2, 64, 16, "bf16")
    ok = dict(q=p.q, kp=p.kp, vp=p.vp, table=p.table, cu=p.cu, kv=p.kv, out=p.out, ws=p.ws, st=p.st)

    def call(**kw):
        x = ok | kw
        B.llama_attn_paged(p.a, x["q"], x["kp"], x["vp"], x["table"], x["cu"], x["kv"], 2, x["out"], x["ws"], x["st"])

    call()
    for kw in (dict(q=p.q.float()), dict(q=p.q.transpose(0, 1)), dict(kp=p.kp[:-1]), dict(vp=p.vp.cpu()), dict(table=p.table.long()),
               dict(cu=p.cu[:-1]), dict(out=p.out[:-1]), dict(ws=p.ws.float()), dict(kv=torch.zeros(3, dtype=torch.int32, device="cuda")),
               dict(q=p.q[..., :32])):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(B.LlamaError):
        call(ws=p.ws[:-1])
    with pytest.raises(ValueError):
        B.PageArgs(4, 2, 64, 16, 8, 2, "fp16")


# ------------------------------------------------------------------ a block over a paged cache

@pytest.mark.parametrize("act,dim,H,Hkv,page", [("fp32", 256, 4, 2, 16), ("bf16", 512, 4, 2, 32), ("bf16", 1024, 8, 8, 16),
                                                ("bf16", 2048, 32, 4, 128)])
def test_block_over_a_paged_cache(act, dim, H, Hkv, page):
    """Requests of different lengths through one block: prompts, a chunk beside single tokens, then single tokens from
    a captured step (plan and block) that is replayed; each request against an oracle block with a cache of its own."""
    import oracle as O
    from llama_decoder_block_kv_b200 import synth
    from tests.gpu_util import BF16_HIDDEN_ABS, Pair, assert_abs_close, assert_fp32_close
    from tests.helpers import build_oracle, t2np

    D = dim // H
    w = synth.Workload(name=f"paged block dim {dim} H {H}/{Hkv}", dim=dim, n_layers=1, n_heads=H, n_kv_heads=Hkv,
                       ffn_hidden=O.ffn_hidden_dim(dim, 256), vocab_size=0, multiple_of=256, ffn_dim_multiplier=None, norm_eps=1e-5,
                       rope_theta=10000.0, max_batch_size=2, max_seq_len=256, act=act, batch=2, seed=9, norm_weights="random")
    pair = Pair(w)
    try:
        lw = [{k: v.cpu() for k, v in synth.layer_weights(w, 0, device="cpu").items()}]
        n_req, P, cols, T = 3, 3 * (256 // page), 256 // page, 130
        oracles = [build_oracle(w, lw, None) for _ in range(n_req)]
        a = B.PageArgs(H, Hkv, D, page, P, cols, act)
        kp, vp = (torch.full((P, Hkv, page, D), float("nan"), dtype=DT[act], device="cuda") for _ in range(2))
        table = torch.full((n_req, cols), -1, dtype=torch.int32, device="cuda")
        free, count = torch.arange(P, dtype=torch.int32, device="cuda"), ints([P])
        kv, cu = torch.zeros(n_req, dtype=torch.int32, device="cuda"), torch.zeros(n_req + 1, dtype=torch.int32, device="cuda")
        st = status_word()
        ws = torch.zeros(B.llama_block_paged_workspace_bytes(pair.ctx, T), dtype=torch.uint8, device="cuda")

        def step(new, h, pos, slot, max_new):
            B.llama_page_plan(a, kv, new, table, free, count, count, cu, kv, pos, slot, st)
            B.llama_block_forward_paged(pair.ctx, 0, h, a, kp, vp, table, cu, kv, pos, slot, max_new, ws, st)

        def check(h, rows, have, new, what):
            assert B.llama_paged_status(st) == (B.LLAMA_OK, 0)
            pair.check_error()
            t = 0
            for b, n in enumerate(new):
                if n:
                    ref = oracles[b].block(0, t2np(rows[t:t + n])[None], have[b])[0]
                    got = t2np(h[t:t + n])
                    if act == "fp32":
                        assert_fp32_close(got, ref, (what, b))
                    else:
                        assert_abs_close(got, ref, BF16_HIDDEN_ABS, (what, b))
                t += n

        have = [0] * n_req
        for i, new in enumerate(([77, 33, 0], [40, 1, 12], [1, 1, 100], [1, 5, 1])):
            n = sum(new)
            rows = synth.hidden(w, (1, n, dim), call=i)[0]
            h = rows.to("cuda").contiguous()
            pos, slot = (torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(2))
            step(ints(new), h, pos, slot, max(new))
            check(h, rows, have, new, i)
            have = [x + y for x, y in zip(have, new)]
        rows = synth.hidden(w, (1, 4 * n_req, dim), call=9)[0]
        h, one = torch.zeros((n_req, dim), device="cuda"), ints([1] * n_req)
        pos, slot = (torch.zeros(n_req, dtype=torch.int32, device="cuda") for _ in range(2))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(one, h, pos, slot, 1)
        for i in range(4):
            h.copy_(rows[i * n_req:(i + 1) * n_req])
            g.replay()
            check(h, rows[i * n_req:(i + 1) * n_req], have, [1] * n_req, ("replayed", i))
            have = [x + 1 for x in have]
    finally:
        pair.close()


def test_block_over_a_paged_cache_refuses():
    import oracle as O
    from llama_decoder_block_kv_b200 import synth
    from tests.gpu_util import Pair

    w = synth.Workload(name="paged block refusals", dim=256, n_layers=1, n_heads=4, n_kv_heads=2, ffn_hidden=O.ffn_hidden_dim(256, 256),
                       vocab_size=0, multiple_of=256, ffn_dim_multiplier=None, norm_eps=1e-5, rope_theta=10000.0, max_batch_size=1,
                       max_seq_len=64, act="bf16", batch=1, seed=9, norm_weights="random")
    pair = Pair(w)
    try:
        a = B.PageArgs(4, 2, 64, 16, 4, 4)
        x = dict(h=torch.zeros((2, 256), device="cuda"), kp=torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device="cuda"),
                 table=ints([[0, 1, 2, 3]]), cu=ints([0, 2]), kv=ints([2]), pos=ints([0, 1]), slot=ints([0, 1]),
                 ws=torch.zeros(B.llama_block_paged_workspace_bytes(pair.ctx, 2), dtype=torch.uint8, device="cuda"), st=status_word())

        def call(layer=0, a=a, max_new=2, **kw):
            y = x | kw
            B.llama_block_forward_paged(pair.ctx, layer, y["h"], a, y["kp"], y["kp"].clone(), y["table"], y["cu"], y["kv"], y["pos"],
                                        y["slot"], max_new, y["ws"], y["st"])

        call()
        for kw in (dict(layer=1), dict(layer=-1), dict(max_new=0), dict(ws=x["ws"][:-256])):
            with pytest.raises(B.LlamaError):
                call(**kw)
        for bad in (dict(n_heads=8), dict(n_kv_heads=4), dict(dtype="fp32")):
            y = dict(n_heads=4, n_kv_heads=2, head_dim=64, page_size=16, num_pages=4, max_pages=4, dtype="bf16") | bad
            b = B.PageArgs(**y)
            kp = torch.zeros((4, b.n_kv_heads, 16, 64), dtype=DT[b.dtype], device="cuda")
            with pytest.raises((B.LlamaError, ValueError)):
                call(a=b, kp=kp)
        with pytest.raises(ValueError):
            call(h=x["h"].double())
        # positions past the context's max_seq_len are flagged, not appended
        call(pos=ints([0, 64]))
        assert B.llama_paged_status(x["st"]) == (B.LLAMA_ERR_POS_RANGE, 2)
    finally:
        pair.close()


# ------------------------------------------------------------------ far pages, shared pages, the most requests

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 40])
def test_pages_far_into_a_large_pool(n, dtype):
    """Pools of more than 2^32 elements (and 2^33 bytes): rows past every 32-bit offset are appended to and read."""
    H, Hkv, D, page = 8, 4, 128, 128
    P = (2 ** 32 // (Hkv * page * D)) + 70
    a = B.PageArgs(H, Hkv, D, page, P, 4, dtype)
    kp, vp = (torch.empty((P, Hkv, page, D), dtype=DT[dtype], device="cuda") for _ in range(2))
    ids = [P - 1, 3, P - 2]
    kv = 300
    for x in (kp, vp):
        x[ids] = float("nan")
    slots = [ids[j // page] * page + j % page for j in range(kv)]
    qkv, cs = normal((kv, (H + 2 * Hkv) * D), torch.float32, 4), rope_table(kv, D)
    q = torch.empty((kv, H, D), dtype=DT[dtype], device="cuda")
    st = status_word()
    B.llama_rope_append(a, qkv, ints(list(range(kv))), ints(slots), cs, q, kp, vp, st)
    x = qkv.double().view(kv, H + 2 * Hkv, D)
    k, v = (R.gather(p, ids, kv) for p in (kp, vp))
    step = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -20  # either side of a tie
    turned = R.rope(x[:, H: H + Hkv], cs[:, None])
    assert ((k - turned).abs() <= step * turned.abs() + 1e-6).all()
    assert torch.equal(v, x[:, H + Hkv:].to(DT[dtype]).double())
    out = torch.empty((n, H, D), dtype=DT[dtype], device="cuda")
    B.llama_attn_paged(a, q[kv - n:], kp, vp, ints([ids + [-1]]), ints([0, n]), ints([kv]), n, out, workspace(H, Hkv, D, dtype), st)
    assert B.llama_paged_status(st) == (B.LLAMA_OK, 0)
    check_attention(out, [(0, q[kv - n:], k.to(DT[dtype]), v.to(DT[dtype]))], DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 20])
def test_requests_that_share_pages(n, dtype):
    """Requests with a common prefix list the same pages."""
    p = Paged([(n, 150), (n, 170), (n, 96)], 8, 2, 128, 32, dtype)
    t = p.table.tolist()
    for b in (1, 2):
        t[b][:2] = t[0][:2]
    p.table = ints(t)
    k0, v0 = p.seqs[0][2][:64], p.seqs[0][3][:64]
    p.seqs = [(s, q, torch.cat([k0, k[64:]]), torch.cat([v0, v[64:]])) for s, q, k, v in p.seqs]
    p.call()
    p.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("single", [True, False])
def test_the_most_requests(single, dtype):
    """LLAMA_MAX_SEQS requests, most of them without a new token, the last one with."""
    r = random.Random(6)
    lens = [((1 if single else r.choice([1, 2, 70])) if b % 41 == 0 or b == B.LLAMA_MAX_SEQS - 1 else 0, 0) for b in range(B.LLAMA_MAX_SEQS)]
    lens = [(n, n + r.choice([0, 1, 16, 130])) if n else (0, r.choice([0, 5])) for n, _ in lens]
    p = Paged(lens, 2, 1, 64, 16, dtype)
    p.call()
    p.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_call_on_another_stream(dtype):
    """The stream argument is the stream of the work: it waits there for what comes before it."""
    p = Paged([(1, 300), (30, 90)], 8, 2, 128, 16, dtype)
    want = p.call().clone()
    p.out.fill_(LEFT)
    q = p.wide.clone()
    p.wide.zero_()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        p.wide.copy_(q)
    p.call(stream=s)
    s.synchronize()
    assert torch.equal(p.out, want)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_infinite_values_give_what_the_formula_gives(dtype):
    """V rows with infinities and K rows that make every score -inf or NaN, seen by some rows of a tile and not by
    others, in whole units and in cut ones: finite, infinite and NaN values stand where the 64-bit form has them."""
    inf = float("inf")
    for n, kv, at, what in ((40, 40, 20, "v"), (260, 700, 500, "v"), (40, 300, 280, "k"), (30, 30, 0, "k"), (3, 3000, 2998, "v")):
        p = Paged([(n, kv), (1, 65)], 8, 2, 128, 16, dtype, seed=3)
        page, off = int(p.table[0, at // 16]), at % 16
        t, q, k, v = p.seqs[0]
        if what == "v":
            p.vp[page, :, off, ::2] = inf
            v = v.clone()
            v[at, :, ::2] = inf
        else:
            p.kp[page, :, off, 5] = inf
            k = k.clone()
            k[at, :, 5] = inf
        p.call()
        assert B.llama_paged_status(p.st) == (B.LLAMA_OK, 0)
        want, _, _ = R.attention(q, k, v)
        got = p.out[t:t + n].double()
        assert torch.equal(torch.isnan(got), torch.isnan(want)), (n, kv, what)
        assert torch.equal(torch.isinf(got), torch.isinf(want)), (n, kv, what)
        fine = torch.isfinite(want)
        # finite values next to infinite ones of the same row: two roundings of the storage type and of P, as the bound's
        # weights would be infinite too
        assert ((got - want)[fine].abs() <= 2.0 ** -6 * (want[fine].abs() + 1)).all(), (n, kv, what)
        check_attention(p.out[n:n + 1], [(0, *p.seqs[1][1:])], p.dt)
