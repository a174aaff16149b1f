"""The 4-bit cache's operators against plain float64 forms (kv4_util), with
tolerances that count roundings, at the sizes, masks and orders where they
could go wrong; and the operators run together."""
import numpy as np
import pytest
import torch

import attention_qk_norm_b200 as qkn
from tests import kv4_util as ku

pytestmark = pytest.mark.gpu
EPS = 1e-6


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def bits(t):
    return t.contiguous().view(torch.uint8)


def make_qkv(seed, T, Hq, Hk, D, dtype, pad=0):
    g = gen(seed)
    x = torch.randn((T, (Hq + 2 * Hk) * D + pad), generator=g, device="cuda")
    x *= torch.exp(torch.randn((T, 1), generator=g, device="cuda"))
    return x.clamp(-400, 400).to(ku.DTYPES[dtype])


# ------------------------------------------------------------ append, read --
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32", "fp8"])
@pytest.mark.parametrize("T,Hq,Hk,D,page,pad", [
    (1, 4, 1, 64, 16, 0), (5, 7, 3, 128, 64, 16), (131, 0, 2, 256, 32, 0), (77, 8, 8, 128, 256, 32),
    (1000, 2, 1, 64, 128, 0)])
def test_append_holds_rows_bit_for_bit(dtype, T, Hq, Hk, D, page, pad):
    x = make_qkv(11 * T + D, T, Hq, Hk, D, dtype, pad)
    if T > 4:
        x[3] = 0
    g = gen(5)
    gq = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    gk = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    pages = -(-T // page) + 1
    cache = qkn.KV4Cache.empty(pages, Hk, D, page, scores=True)
    cache.pool.fill_(0xA5)
    cache.scores.fill_(3.0)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].contiguous()
    if T > 4:
        slots[1] = -1  # a padded token
    want = x.clone()
    qkn.qknorm_per_head(want, Hq, Hk, D, gq if Hq else None, gk, EPS)
    got = x.clone()
    assert qkn.qknorm_kv4_append(cache, got, slots, Hq, gq if Hq else None, gk, EPS) is got
    # Its sums are added in another order, so a value may be rounded the other
    # way: one step of the type (fp32: the factor's and two products' roundings).
    qk, W = (Hq + Hk) * D, (Hq + 2 * Hk) * D
    step = 8 * 2.0 ** -24 if dtype == "fp32" else 2 * ku.HALF_STEP[dtype]
    d = (got[:, :qk].double() - want[:, :qk].double()).abs()
    assert torch.all(d <= step * 1.001 * want[:, :qk].double().abs() + 2 * ku.TINY[dtype])
    assert torch.equal(bits(got[:, qk:]), bits(x[:, qk:]))
    # And it is what elementary torch operations give, bit for bit.
    y = x[:, :qk].float().view(T, Hq + Hk, D).contiguous()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
    y = torch.cat([y[:, :Hq] * gq, y[:, Hq:] * gk], 1).flatten(1)
    y = (y.clamp(-448, 448) if dtype == "fp8" else y).to(x.dtype)
    assert torch.equal(bits(got[:, :qk]), bits(y))

    held, at, n = ku.Held(cache), slots.cpu().numpy(), x.float().cpu().numpy()
    live = at >= 0
    rows = n[:, :(Hq + 2 * Hk) * D].reshape(T, -1, D)[live]
    p, o = at[live] // page, at[live] % page
    keys = rows[:, Hq:Hq + Hk]
    factor = 1 / np.sqrt((keys.astype(np.float64) ** 2).mean(-1) + EPS)
    for kv, y, f in ((0, keys * gk.cpu().numpy(), factor), (1, rows[:, Hq + Hk:], 1.0)):
        codes, step, mid = ku.hold(y)
        assert np.array_equal(held.codes[kv][p, :, o], codes)
        for i, w in enumerate((step * f, mid * f)):
            g_ = held.params[kv][p, :, o, i]
            # One rounding to bf16, of a product whose factor carries up to
            # D + 4 roundings in fp32 (the norm) or none.
            tol = 2.0 ** -8 + (D + 4) * 2.0 ** -24 if kv == 0 else 2.0 ** -8
            assert np.all(np.abs(g_ - w) <= tol * np.abs(w) + 2.0 ** -134)
    scores = cache.scores.cpu().numpy()
    assert np.all(scores[p, :, o] == 0)
    untouched = np.ones((pages, page), bool)
    untouched[p, o] = False
    assert np.all(scores.transpose(0, 2, 1)[untouched] == 3.0)
    for kv in range(2):
        c = held.codes[kv].transpose(0, 2, 1, 3)[untouched]
        assert np.all(c[..., 0::2] == 5) and np.all(c[..., 1::2] == 10)

    # Read back: one rounding of mid + scale * (c - 8); a padded slot is zeros.
    for name, t in ku.DTYPES.items():
        k, v = qkn.qknorm_kv4_read(cache, slots, dtype=t)
        for kv, r in ((0, k), (1, v)):
            w = np.zeros((T, Hk, D))
            s = held.params[kv][p, :, o]
            w[live] = s[..., 1:] + s[..., :1] * (held.codes[kv][p, :, o].astype(np.float64) - 8)
            if name == "fp8":
                w = np.clip(w, -448, 448)
            err = np.abs(ku.f64(r).reshape(T, Hk, D) - w)
            assert np.all(err <= ku.HALF_STEP[name] * 1.001 * np.abs(w) + ku.TINY[name])
    # Without weights the buffer is read only, and holds its rows as they are.
    plain = got.clone()
    qkn.qknorm_kv4_append(cache, plain, slots, Hq)
    assert torch.equal(bits(plain), bits(got))
    y = got.float().cpu().numpy()[:, :(Hq + 2 * Hk) * D].reshape(T, -1, D)[live][:, Hq:Hq + Hk]
    codes, step, mid = ku.hold(y)
    held = ku.Held(cache)
    assert np.array_equal(held.codes[0][p, :, o], codes)
    assert np.array_equal(held.params[0][p, :, o, 0], ku.bf16(step).astype(np.float64))


def test_append_extreme_rows():
    D, page = 128, 16
    x = torch.zeros((9, 3 * D), dtype=torch.float32, device="cuda")
    # (linspace's own step overflows here: a row of infinities and NaN)
    x[1, 2 * D:] = torch.linspace(-3.4e38, 3.4e38, D, device="cuda")
    x[8, 2 * D:] = torch.linspace(-1.0, 1.0, D, device="cuda") * 3.4e38  # the whole range
    x[2, 2 * D:] = 5.0                                               # constant
    x[3, 2 * D + 7] = float("nan")
    x[4, 2 * D + 9] = float("inf")
    x[5, 2 * D + 1] = -float("inf")
    x[6, 2 * D:] = torch.linspace(-1e-39, 1e-39, D, device="cuda")   # below the smallest step
    x[7, 2 * D] = 1e4                                                # one outlier
    cache = qkn.KV4Cache.empty(1, 1, D, page)
    slots = torch.arange(9, device="cuda")
    qkn.qknorm_kv4_append(cache, x, slots, 1)
    _, v = qkn.qknorm_kv4_read(cache, slots, dtype=torch.float32)
    v = v.cpu().numpy()
    assert np.all(v[0] == 0) and np.all(v[2] == 5.0)
    assert np.all(np.isnan(v[[1, 3, 4, 5]]))
    assert np.all(np.abs(v[6]) <= 2e-39)
    step = 6.8e38 / 15
    assert np.all(np.abs(v[8] - x[8, 2 * D:].cpu().numpy()) <= 0.6 * step)
    assert abs(v[7, 0] - 1e4) <= 1e4 * 2.0 ** -7 and np.all(np.abs(v[7, 1:]) <= 1e4 / 15)


def test_slots_outside_the_pool_are_counted_and_skipped():
    D, page = 64, 16
    cache = qkn.KV4Cache.empty(2, 1, D, page)
    x = make_qkv(3, 4, 1, 1, D, "bf16")
    before = qkn.kv4_bad_pages()
    slots = torch.tensor([32, 2 ** 40, 31, -5], device="cuda")
    qkn.qknorm_kv4_append(cache, x, slots, 1)
    assert qkn.kv4_bad_pages() == before + 4  # K and V of two tokens
    k, v = qkn.qknorm_kv4_read(cache, slots)
    assert qkn.kv4_bad_pages() > before + 4
    assert torch.all(k[[0, 1, 3]] == 0) and torch.all(v[[0, 1, 3]] == 0) and torch.any(k[2] != 0)
    assert torch.all(cache.pool[0] == 0)


# --------------------------------------------------------------- attention --
def problem(seed, lens, nqs, Hq, Hk, D, page, dtype, scores=False, behind=0, poison=False):
    """A cache with shuffled pages, its table (-1 behind a sequence's pages), and
    queries; rows that no sequence has are poisoned with NaN parameters."""
    g = gen(seed)
    B = len(lens)
    need = [-(-n // page) for n in lens]
    total = sum(need) + 2
    cache = qkn.KV4Cache.empty(total, Hk, D, page, scores=scores)
    ku.fill(cache, seed)
    order = torch.randperm(total, generator=g, device="cuda").tolist()
    table = torch.full((B, max(max(need), 1) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    if poison:
        live = torch.zeros((total, page), dtype=torch.bool)
        for b, n in enumerate(lens):
            for j in range(n):
                live[table[b, j // page], j % page] = True
        par = cache.pool[..., 16 * D:].view(total, Hk, page // 16, 2, 16, 4)
        dead = ~live.view(total, 1, page // 16, 1, 16, 1).cuda()
        par.masked_fill_(dead, 0xFF)
    T = sum(nqs) + behind
    q = torch.randn((T, (Hq + 2 * Hk) * D), generator=g, device="cuda") * 1.5
    q = q.to(ku.DTYPES[dtype])
    starts = np.concatenate([[0], np.cumsum(nqs)]).astype(np.int32)
    return cache, q, table, starts


def check(cache, q, Hq, table, lens, starts, dtype, out, lse, scale=None, scores_before=None):
    D = cache.D
    scale = D ** -0.5 if scale is None else scale
    want, wlse, add, bound, lse_bound, add_bound = ku.attend(
        cache, q, Hq, table.numpy(), [max(0, n) for n in lens], starts, scale, dtype)
    n = starts[-1]
    err = np.abs(ku.f64(out) - want)[:n]
    assert np.all(err <= bound[:n]), (err - bound[:n]).max()
    empty = np.isneginf(wlse[:n])
    got = ku.f64(lse)[:n]
    assert np.array_equal(np.isneginf(got), empty)
    assert np.all(np.abs(got[~empty] - wlse[:n][~empty]) <= lse_bound[:n][~empty])
    if scores_before is not None:
        got = ku.f64(cache.scores)
        b = scores_before.astype(np.float64)
        err = np.abs(got - b - add)
        assert np.all(err <= add_bound + 2.0 ** -23 * (np.abs(b) + add) + 1e-30), err.max()
        assert np.array_equal(got[add == 0], b[add == 0])


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 64, 100, 257]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32", "fp8"])
@pytest.mark.parametrize("Hq,Hk,D,page", [
    (4, 1, 128, 16), (8, 8, 64, 64), (10, 2, 256, 32), (28, 4, 128, 128), (16, 1, 64, 256),
    (40, 1, 128, 64), (9, 3, 256, 16)])
@pytest.mark.parametrize("scores", [False, True])
def test_attention_ragged(dtype, Hq, Hk, D, page, scores):
    lens, nqs = LENS, [1] * len(LENS)
    cache, q, table, starts = problem(D + Hq, lens, nqs, Hq, Hk, D, page, dtype, scores, poison=True)
    before = None
    if scores:
        cache.scores.uniform_(0, 2)
        before = cache.scores.cpu().numpy()
    bad = qkn.kv4_bad_pages()
    out, lse = qkn.qknorm_kv4_attention(cache, q, Hq, table.cuda(),
                                        torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                        add_scores=scores)
    check(cache, q, Hq, table, lens, starts, dtype, out, lse, scores_before=before)
    assert qkn.kv4_bad_pages() == bad


@pytest.mark.parametrize("dtype,Hq,Hk,D,page,nq", [
    ("bf16", 4, 1, 128, 16, 5), ("fp16", 16, 16, 64, 16, 7), ("fp32", 6, 2, 256, 64, 3),
    ("fp8", 8, 1, 128, 32, 9), ("bf16", 8, 8, 64, 128, 70), ("bf16", 32, 2, 128, 64, 4)])
@pytest.mark.parametrize("scores", [False, True])
def test_attention_several_query_tokens(dtype, Hq, Hk, D, page, nq, scores):
    """Query counts of 0 to nq, more than the rows there are among them; rows of
    no sequence are left as they were."""
    lens = [0, 1, 3, 16, 40, 100, 130, 515]
    nqs = [2, nq, 0, 1, nq, min(nq, 4), nq, nq]
    cache, q, table, starts = problem(nq + D, lens, nqs, Hq, Hk, D, page, dtype, scores, behind=3,
                                      poison=True)
    before = None
    if scores:
        cache.scores.uniform_(0, 2)
        before = cache.scores.cpu().numpy()
    T = q.shape[0]
    out = torch.full((T, Hq * D + 64), 7.0, device="cuda").to(q.dtype)[:, :Hq * D]
    lse = torch.full((T, Hq), 7.0, device="cuda")
    qkn.qknorm_kv4_attention(cache, q, Hq, table.cuda(),
                             torch.tensor(lens, dtype=torch.int32, device="cuda"),
                             q_starts=torch.from_numpy(starts).cuda(), max_q=nq, scale=0.11,
                             add_scores=scores, out=out, lse=lse)
    check(cache, q, Hq, table, lens, starts, dtype, out, lse, 0.11, before)
    assert torch.all(out[-3:].float() == 7.0) and torch.all(lse[-3:] == 7.0)


@pytest.mark.parametrize("B,n,Hq,Hk,D,page", [(1, 5003, 4, 1, 128, 64), (3, 2049, 8, 2, 64, 16),
                                              (2, 9000, 2, 1, 256, 256)])
def test_attention_long(B, n, Hq, Hk, D, page):
    lens = [n - 7 * b for b in range(B)]
    cache, q, table, starts = problem(n, lens, [1] * B, Hq, Hk, D, page, "fp32", True)
    before = cache.scores.cpu().numpy()
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    first = qkn.qknorm_kv4_attention(cache, q, Hq, table.cuda(), dl, add_scores=True)
    check(cache, q, Hq, table, lens, starts, "fp32", *first, scores_before=before)
    sums = cache.scores.clone()
    cache.scores.zero_()
    again = qkn.qknorm_kv4_attention(cache, q, Hq, table.cuda(), dl, add_scores=True)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert torch.equal(sums, cache.scores)  # the same bits on every run


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", [[700], [33] * 70, [5, 4000, 900, 1] * 3])
def test_whole_items_and_split_items_agree(dtype, lens):
    """The same call with a table of its own width and with a wide one (which
    decides whether an item goes to one block), both against the plain form."""
    B = len(lens)
    for scores in (False, True):
        cache, q, table, starts = problem(B, lens, [1] * B, 8, 2, 128, 64, dtype, scores)
        if scores:
            cache.scores.uniform_(0, 2)
        first = None if not scores else cache.scores.clone()
        dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for pad in (0, 3000):
            wide = torch.cat([table, torch.full((B, pad), -1, dtype=torch.int32)], 1)
            if scores:
                cache.scores.copy_(first)
            out, lse = qkn.qknorm_kv4_attention(cache, q, 8, wide.cuda(), dl, add_scores=scores)
            check(cache, q, 8, table, lens, starts, dtype, out, lse,
                  scores_before=first.cpu().numpy() if scores else None)


def test_attention_without_lse_through_the_c_entry():
    lens = [300, 17]
    cache, q, table, starts = problem(2, lens, [1, 1], 4, 2, 64, 16, "fp16")
    dl, dt = torch.tensor(lens, dtype=torch.int32, device="cuda"), table.cuda()
    ws = qkn.kv4_attention_workspace(cache, q, 4, dt)
    out = torch.empty(2, 256, dtype=torch.float16, device="cuda")
    rc = qkn._kv4._lib().qknorm_kv4_attention(
        q.data_ptr(), 2, 2, 4, 2, 64, q.stride(0), cache.pool.data_ptr(), cache.num_pages, 16,
        dt.data_ptr(), dt.stride(0), dt.shape[1], dl.data_ptr(), 2, None, 1, 0.125, out.data_ptr(),
        256, None, None, ws.data_ptr(), ws.nbytes, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    want, lse = qkn.qknorm_kv4_attention(cache, q, 4, dt, dl)
    assert torch.equal(out, want)
    # Queries may be written over: the output in the query columns themselves.
    same, _ = qkn.qknorm_kv4_attention(cache, q, 4, dt, dl, out=q[:, :256])
    assert torch.equal(same, want)


def test_attention_sharp_and_large_logits():
    """One row takes all the weight; logits far from zero; V scales far apart."""
    lens = [300, 300]
    cache, q, table, starts = problem(9, lens, [1, 1], 4, 1, 128, 64, "bf16")
    ku.fill(cache, 10, spread=3.0)
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for scale in (0.0, 0.5, -0.5, 30.0):
        out, lse = qkn.qknorm_kv4_attention(cache, q, 4, table.cuda(), dl, scale=scale)
        check(cache, q, 4, table, lens, starts, "bf16", out, lse, scale)


def test_attention_nan_rows_reach_only_who_sees_them():
    lens = [40, 40]
    cache, q, table, starts = problem(4, lens, [4, 4], 2, 1, 64, 16, "bf16")
    page, row = int(table[0, 38 // 16]), 38 % 16
    par = cache.pool[..., 16 * 64:].view(-1, 1, 1, 2, 16, 4)
    par[page, :, 0, 1, row] = 0xFF  # V of sequence 0's row 38 is NaN
    out, lse = qkn.qknorm_kv4_attention(cache, q, 2, table.cuda(),
                                        torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                        q_starts=torch.from_numpy(starts).cuda(), max_q=4)
    nan = torch.isnan(out.float()).all(1).cpu().tolist()
    # Query i of 4 sees 37 + i rows: row 38 is seen by the last two.
    assert nan == [False, False, True, True, False, False, False, False]
    assert not torch.isnan(out[[0, 1, 4, 5, 6, 7]].float()).any()
    assert torch.isfinite(lse).all()


def test_attention_bad_pages_and_lengths():
    """Pages outside the pool give no rows, lengths and query ranges are taken
    into range; each bad page is counted."""
    Hq, D, page = 2, 64, 16
    lens = [48, 48, 1 << 30, -3]
    cache, q, table, _ = problem(8, [48, 48, 48, 48], [1] * 4, Hq, 1, D, page, "bf16", True)
    table = table[:, :3].contiguous()
    table[1, 1] = cache.num_pages
    before = qkn.kv4_bad_pages()
    out, lse = qkn.qknorm_kv4_attention(cache, q, Hq, table.cuda(),
                                        torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                        add_scores=True)
    assert qkn.kv4_bad_pages() > before
    # Sequence 1 without its middle page is a sequence of the other two.
    table[1] = torch.stack([table[1, 0], table[1, 2], table[1, 0]])
    starts = np.arange(5, dtype=np.int32)
    check(cache, q, Hq, table, [48, 32, 48, 0], starts, "bf16", out, lse)
    # Query ranges: the second one runs past T, the third goes back.
    starts = torch.tensor([0, 3, 9, 1, 2], dtype=torch.int32, device="cuda")
    out2, _ = qkn.qknorm_kv4_attention(cache, q, Hq, table.cuda(),
                                       torch.tensor([48, 32, 48, 0], dtype=torch.int32,
                                                    device="cuda"), q_starts=starts, max_q=3)
    torch.cuda.synchronize()
    assert out2.shape == out.shape


def test_offsets_beyond_32_bits():
    """A pool of over 4 GiB, its last pages used."""
    Hk, D, page = 1, 256, 256
    pages = (4 << 30) // (16 * (16 * D + 128)) + 70
    cache = qkn.KV4Cache.empty(pages, Hk, D, page, scores=True)
    small = qkn.KV4Cache.empty(4, Hk, D, page, scores=True)
    x = make_qkv(5, 600, 2, Hk, D, "bf16")
    j = torch.arange(600, device="cuda")
    for c, first in ((cache, pages - 4), (small, 0)):
        qkn.qknorm_kv4_append(c, x.clone(), first * page + j, 2)
        table = torch.arange(first, first + 3, dtype=torch.int32, device="cuda")[None]
        lens = torch.tensor([600], dtype=torch.int32, device="cuda")
        o = qkn.qknorm_kv4_attention(c, x[:1].contiguous(), 2, table, lens, add_scores=True)
        to = torch.tensor([[first + 3]], dtype=torch.int32, device="cuda")
        e = qkn.qknorm_kv4_evict(c, table, lens, to, 200, 50)
        r = qkn.qknorm_kv4_read(c, (first + 3) * page + j[:200])
        if first:
            big = (*o, *e, *r)
        else:
            assert all(torch.equal(a, b) for a, b in zip(big, (*o, *e, *r)))


# ---------------------------------------------------------------- eviction --
@pytest.mark.parametrize("Hk,D,page,budget,recent", [
    (1, 64, 16, 1, 0), (2, 128, 64, 100, 30), (3, 256, 32, 64, 64), (8, 128, 128, 257, 0),
    (2, 64, 256, 300, 299)])
@pytest.mark.parametrize("kind", ["spread", "ties", "special"])
@pytest.mark.parametrize("wide", [False, True])
def test_evict(Hk, D, page, budget, recent, kind, wide):
    lens = [0, 1, budget - 1, budget, budget + 1, 700, 1500]
    cache, _, table, _ = problem(budget, lens, [1] * len(lens), 1, Hk, D, page, "bf16", True)
    g = gen(budget + 1)
    s = torch.rand(cache.scores.shape, generator=g, device="cuda")
    if kind == "ties":
        s = torch.floor(s * 4) - 1
        s[s == 0] = -0.0
    if kind == "special":
        s[s < 0.2] = float("nan")
        s[(s > 0.2) & (s < 0.3)] = float("inf")
        s[(s > 0.3) & (s < 0.5)] = -float("inf")
        s[(s > 0.6) & (s < 0.62)] = 1e-42
    B, dp = len(lens), -(-budget // page)
    old = cache.num_pages
    both = qkn.KV4Cache(torch.cat([cache.pool, torch.full_like(cache.pool[:1], 0x5A).expand(
        B * dp, -1, -1, -1)]), Hk, D, page, torch.cat([s, torch.full_like(s[:1], 9.0).expand(
            B * dp, -1, -1)]))
    to = old + torch.randperm(B * dp, generator=g, device="cuda").to(torch.int32).view(B, dp)
    before = ku.Held(both)
    sb = both.scores.cpu().numpy()
    if wide:  # a table for sequences that no cluster holds
        table = torch.cat([table, torch.full((B, 400000 // page), -1, dtype=torch.int32)], 1)
    new_lens, kept = qkn.qknorm_kv4_evict(both, table.cuda(),
                                          torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                          to, budget, recent)
    want = ku.evict(sb, table.numpy(), lens, page, budget, recent)
    assert np.array_equal(kept.cpu().numpy(), want)
    assert new_lens.tolist() == [min(n, budget) for n in lens]
    after, sa, to = ku.Held(both), both.scores.cpu().numpy(), to.cpu().numpy()
    assert torch.equal(both.pool[:old], cache.pool)
    for b, n in enumerate(lens):
        for h in range(Hk):
            m = min(n, budget)
            src, d = want[b, h, :m], np.arange(m)
            p, t = table.numpy()[b][src // page], to[b][d // page]
            for kv in range(2):
                assert np.array_equal(after.codes[kv][t, h, d % page],
                                      before.codes[kv][p, h, src % page])
                assert np.array_equal(after.params[kv][t, h, d % page],
                                      before.params[kv][p, h, src % page])
            assert np.array_equal(sa[t, h, d % page], sb[p, h, src % page], equal_nan=True)
            rest = np.arange(m, dp * page)
            assert np.all(sa[to[b][rest // page], h, rest % page] == 9.0)
            assert np.all(after.codes[0][to[b][rest // page], h, rest % page, 0] == 0xA)


@pytest.mark.parametrize("n,budget,wide", [(40000, 5000, 0), (131072, 16384, 0), (20000, 19999, 0),
                                           (300001, 70000, 0), (30011, 300, 4000)])
def test_evict_long(n, budget, wide):
    page = 128
    cache, _, table, _ = problem(3, [n, 777], [1, 1], 1, 2, 64, page, "bf16", True)
    g = gen(4)
    s = torch.rand(cache.scores.shape, generator=g, device="cuda")
    s[s < 0.5] = 0.25  # most of the rows share one score
    dp = -(-budget // page)
    both = qkn.KV4Cache(torch.cat([cache.pool, cache.pool.new_zeros((2 * dp,) + cache.pool.shape[1:])]),
                        2, 64, page, torch.cat([s, s.new_zeros((2 * dp,) + s.shape[1:])]))
    to = torch.arange(cache.num_pages, cache.num_pages + 2 * dp, dtype=torch.int32,
                      device="cuda").view(2, dp)
    table = torch.cat([table, torch.full((2, wide), -1, dtype=torch.int32)], 1)
    lens, kept = qkn.qknorm_kv4_evict(both, table.cuda(),
                                      torch.tensor([n, 777], dtype=torch.int32, device="cuda"),
                                      to, budget, budget // 8)
    assert np.array_equal(kept.cpu().numpy(), ku.evict(s.cpu().numpy(), table.numpy(), [n, 777],
                                                       page, budget, budget // 8))
    slots = to[0].long().repeat_interleave(page) * page + torch.arange(page, device="cuda").repeat(dp)
    k, v = qkn.qknorm_kv4_read(both, slots[:budget])
    src = kept[0, 1].long()
    ks, vs = qkn.qknorm_kv4_read(both, table[0].cuda().long()[src // page] * page + src % page)
    assert torch.equal(k[:, 64:], ks[:, 64:]) and torch.equal(v[:, 64:], vs[:, 64:])


# ---------------------------------------------------------------- together --
class Server:
    """A small decode loop: store a token, attend, evict when over budget."""

    def __init__(self, seed, B=3, Hq=8, Hk=2, D=128, page=16, prompt=50, dtype=torch.bfloat16):
        self.g, self.B, self.Hq, self.Hk, self.D, self.page = gen(seed), B, Hq, Hk, D, page
        self.width = 8
        pages = 2 * B * self.width
        self.cache = qkn.KV4Cache.empty(pages, Hk, D, page, scores=True)
        self.tables = [torch.arange(i * B * self.width, (i + 1) * B * self.width, dtype=torch.int32,
                                    device="cuda").view(B, self.width) for i in range(2)]
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.gq = 1 + 0.1 * torch.randn(D, generator=self.g, device="cuda")
        self.gk = 1 + 0.1 * torch.randn(D, generator=self.g, device="cuda")
        self.dtype = dtype

    def rows(self, n):
        return torch.randn((self.B * n, (self.Hq + 2 * self.Hk) * self.D), generator=self.g,
                           device="cuda").to(self.dtype)

    def slots(self, n):
        j = self.lens.long()[:, None] + torch.arange(n, device="cuda")
        return (self.tables[0].long().gather(1, j // self.page) * self.page + j % self.page).view(-1)

    def step(self, x, n=1, stream=None):
        qkn.qknorm_kv4_append(self.cache, x, self.slots(n), self.Hq, self.gq, self.gk, EPS)
        self.lens += n
        starts = torch.arange(0, self.B * n + 1, n, dtype=torch.int32, device="cuda")
        return qkn.qknorm_kv4_attention(self.cache, x, self.Hq, self.tables[0], self.lens,
                                        q_starts=starts, max_q=n, add_scores=True)

    def evict(self, budget, recent):
        self.lens, kept = qkn.qknorm_kv4_evict(self.cache, self.tables[0], self.lens,
                                               self.tables[1], budget, recent)
        self.tables.reverse()
        return kept


def test_a_decode_loop_with_eviction():
    s = Server(1)
    prompt = s.rows(50)
    s.step(prompt, 50)
    for step in range(6):
        x = s.rows(1)
        before = s.cache.scores.cpu().numpy()
        out, lse = s.step(x)
        lens = s.lens.tolist()
        starts = np.arange(s.B + 1, dtype=np.int32)
        check(s.cache, x, s.Hq, s.tables[0].cpu(), lens, starts, "bf16", out, lse)
        assert lens == [51 + step if step < 3 else 41 + step - 3] * s.B
        # Each sequence's weights of a step add up to its query rows.
        added = s.cache.scores.cpu().numpy() - before
        if step == 2:
            scores = s.cache.scores.cpu().numpy()
            kept = s.evict(40, 10)
            want = ku.evict(scores, s.tables[1].cpu().numpy(), lens, s.page, 40, 10)
            assert np.array_equal(kept.cpu().numpy(), want)
        elif step < 2:
            total = added.sum((1, 2)).sum()
            assert abs(total - s.B * s.Hq) < 1e-3 * s.B * s.Hq


def test_captured_and_replayed():
    """One decode step captured in a graph, replayed on new inputs, gives the
    bits of eager calls; an eager call with the same workspace between replays
    changes nothing."""
    a, b = Server(7), Server(7)
    prompt = a.rows(50)
    b.rows(50)
    a.step(prompt.clone(), 50)
    b.step(prompt.clone(), 50)
    x = a.rows(1).clone()
    b.rows(1)
    out = torch.empty((a.B, a.Hq * a.D), dtype=x.dtype, device="cuda")
    lse = torch.empty((a.B, a.Hq), device="cuda")
    slots = torch.empty(a.B, dtype=torch.int64, device="cuda")
    ws = qkn.kv4_attention_workspace(a.cache, x, a.Hq, a.tables[0], add_scores=True)

    def step():
        qkn.qknorm_kv4_append(a.cache, x, slots, a.Hq, a.gq, a.gk, EPS)
        qkn.qknorm_kv4_attention(a.cache, x, a.Hq, a.tables[0], a.lens, add_scores=True, out=out,
                                 lse=lse, workspace=ws)

    def evict():
        return qkn.qknorm_kv4_evict(a.cache, a.tables[0], a.lens, a.tables[1], 40, 10)

    slots.fill_(-1)
    keep = a.cache.scores.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
        lens2, kept = evict()
    a.cache.scores.copy_(keep)
    for _ in range(3):
        new = b.rows(1)
        x.copy_(new)
        slots.copy_(a.slots(1))
        a.lens += 1
        graph.replay()
        want, wlse = b.step(new)
        assert torch.equal(out, want) and torch.equal(lse, wlse)
        assert torch.equal(a.cache.scores[:24], b.cache.scores[:24])
        wl, wk = qkn.qknorm_kv4_evict(b.cache, b.tables[0], b.lens, b.tables[1], 40, 10)
        assert torch.equal(lens2, wl) and torch.equal(kept, wk)
        # An eager call on the graph's workspace.
        other = b.rows(1)
        qkn.qknorm_kv4_attention(a.cache, other, a.Hq, a.tables[0], a.lens, workspace=ws)


def test_two_graphs_share_a_workspace():
    """Captured calls of different sizes on one workspace, replayed in turn."""
    a, b = Server(11), Server(12, prompt=50)
    pa, pb = a.rows(50), b.rows(20)
    a.step(pa, 50)
    b.step(pb, 20)
    xa, xb = a.rows(1), b.rows(1)
    wide = torch.cat([b.tables[0], torch.full((3, 4000), -1, dtype=torch.int32, device="cuda")], 1)
    ws = qkn.kv4_attention_workspace(b.cache, xb, b.Hq, wide, add_scores=True)
    want_a = qkn.qknorm_kv4_attention(a.cache, xa, a.Hq, a.tables[0], a.lens)
    want_b = qkn.qknorm_kv4_attention(b.cache, xb, b.Hq, wide, b.lens)
    graphs, outs = [], []
    for c, x, s, t in ((a.cache, xa, a, a.tables[0]), (b.cache, xb, b, wide)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(qkn.qknorm_kv4_attention(c, x, s.Hq, t, s.lens, add_scores=c is b.cache,
                                                 workspace=ws))
        graphs.append(g)
    for _ in range(2):
        for g, got, want in zip(graphs, outs, (want_a, want_b)):
            g.replay()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_on_another_stream():
    s = Server(5)
    s.step(s.rows(50), 50)
    x = s.rows(1)
    want, wlse = qkn.qknorm_kv4_attention(s.cache, x, s.Hq, s.tables[0], s.lens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        out, lse = qkn.qknorm_kv4_attention(s.cache, x, s.Hq, s.tables[0], s.lens, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, want) and torch.equal(lse, wlse)


def test_two_calls_at_once():
    """Split calls on two streams, each with a workspace of its own."""
    lens = [9000, 41, 7000]
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    calls = []
    for seed in (21, 22):
        cache, q, table, _ = problem(seed, lens, [1] * 3, 8, 2, 128, 64, "bf16", True)
        want = qkn.qknorm_kv4_attention(cache, q, 8, table.cuda(), dl, add_scores=True)
        calls.append((cache, q, table.cuda(), want, cache.scores.clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for cache, q, table, _, _, stream in calls:
            cache.scores.zero_()
            stream.wait_stream(torch.cuda.current_stream())
            got.append(qkn.qknorm_kv4_attention(cache, q, 8, table, dl, add_scores=True,
                                                stream=stream))
        torch.cuda.synchronize()
        for (o, l), (cache, _, _, (wo, wl), sums, _) in zip(got, calls):
            assert torch.equal(o, wo) and torch.equal(l, wl) and torch.equal(cache.scores, sums)


def test_binding_refusals():
    s = Server(6)
    x = s.rows(1)
    c, t, n = s.cache, s.tables[0], s.lens
    att = qkn.qknorm_kv4_attention
    bare = qkn.KV4Cache(c.pool, s.Hk, s.D, s.page)
    for call in (
            lambda: qkn.KV4Cache(c.pool[:, :1], 1, s.D, s.page),
            lambda: qkn.KV4Cache(c.pool, s.Hk, 64, s.page),
            lambda: qkn.KV4Cache(c.pool, s.Hk, s.D, s.page, scores=c.scores.double()),
            lambda: att(c, x, s.Hq, t.long(), n),
            lambda: att(c, x, s.Hq, t[:2], n),
            lambda: att(c, x, s.Hq, t, n.long()),
            lambda: att(c, x, s.Hq, t, n.cpu()),
            lambda: att(c, x.t(), s.Hq, t, n),
            lambda: att(c, x[:, :512], s.Hq, t, n),
            lambda: att(c, x.cpu(), s.Hq, t, n),
            lambda: att(c, x, s.Hq, t, n, out=torch.empty(2, 2, device="cuda")),
            lambda: att(c, x, s.Hq, t, n, lse=torch.empty(2, 2, device="cuda")),
            lambda: att(bare, x, s.Hq, t, n, add_scores=True),
            lambda: att(c, x, s.Hq, t, n, workspace=torch.empty(8, dtype=torch.uint8)),
            lambda: qkn.qknorm_kv4_evict(bare, t, n, s.tables[1], 10, 1),
            lambda: qkn.qknorm_kv4_evict(c, t, n, s.tables[1], 129, 1),
            lambda: qkn.qknorm_kv4_evict(c, t, n, s.tables[1], 10, 11),
            lambda: qkn.qknorm_kv4_append(c, x, torch.zeros(2, dtype=torch.int64, device="cuda"),
                                          s.Hq),
            lambda: qkn.qknorm_kv4_append(c, x, torch.zeros(3, dtype=torch.int32, device="cuda"),
                                          s.Hq),
            lambda: qkn.qknorm_kv4_append(c, x, torch.zeros(3, dtype=torch.int64, device="cuda"),
                                          s.Hq, s.gq[:64], s.gk),
            lambda: qkn.qknorm_kv4_append(c, x[:, :256], s.slots(1), s.Hq),
            lambda: qkn.qknorm_kv4_read(c, torch.zeros(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            call()
    for call in (lambda: att(c, x, 7, t, n), lambda: att(c, x, s.Hq, t, n, max_q=2),
                 lambda: att(c, x, s.Hq, t, n,
                             workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
                 lambda: qkn.qknorm_kv4_append(c, x, s.slots(1), s.Hq, s.gq, None)):
        with pytest.raises(qkn.QKNormError):
            call()
