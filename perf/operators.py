"""The 4-bit key/value cache operators as a measured workload: what each is
called with, its plain form in elementary torch operations, and the bytes and
operations that one pass cannot do without.

The cache is paged.  A pool is a uint8 tensor [num_pages, Hk, page/16, 16*D + 128]:
for each page and key/value head, blocks of 16 tokens, each block holding

    bytes [0, 8*D)              K codes, 16 rows of D/2 bytes
    bytes [8*D, 16*D)           V codes, 16 rows of D/2 bytes
    bytes [16*D, 16*D + 64)     K parameters, 16 pairs of bf16 {scale, mid}
    bytes [16*D + 64, ...+128)  V parameters, likewise

Element 2j of a row is the low nibble of byte j, element 2j+1 the high one, and
a code c in 0..15 stands for mid + scale * (c - 8).

Operators:
  store   per-head QK-Norm of a fused QKV buffer in place, its key and value
          rows written to cache slots, and rows read back as values (what a
          server does to reuse a cached prefix at full precision);
  attend  attention of each sequence's query tokens over its cached rows,
          optionally adding every cached row's attention weight to its score;
  evict   keep, per sequence and key/value head, the newest rows and the
          highest-scored others, moved to other pages in order.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
          "fp8": torch.float8_e4m3fn}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4, "fp8": 1}
EPS = 1e-6


# ------------------------------------------------------------------- cases --
def _store(name, T, Hq, Hk, D, dtype="bf16", norm=True, page=64, pad=0):
    return dict(name=name, op="store", T=T, Hq=Hq, Hk=Hk, D=D, dtype=dtype, norm=norm, page=page,
                pad=pad)


def _attend(name, B, lo, hi, Hq, Hk, D, dtype="bf16", nq=1, scores=False, page=64):
    return dict(name=name, op="attend", B=B, lo=lo, hi=hi, Hq=Hq, Hk=Hk, D=D, dtype=dtype, nq=nq,
                scores=scores, page=page)


def _evict(name, B, lo, hi, Hk, D, budget, recent, page=64):
    return dict(name=name, op="evict", B=B, lo=lo, hi=hi, Hk=Hk, D=D, budget=budget,
                recent=recent, page=page)


def listed():
    return [
        # One decode step of five sequences: launch latency.
        _store("store_t5", 5, 32, 8, 128),
        # A long prompt, the GQA layout's largest length.
        _store("store_t16384", 16384, 32, 8, 128),
        # fp32 rows stored as they are (a layerwise-normalised buffer), padded rows.
        _store("store_fp32_d64_t1037", 1037, 64, 8, 64, dtype="fp32", norm=False, page=16, pad=8),
        # One short conversation: launch latency.
        _attend("attend_b1_len301", 1, 301, 301, 32, 8, 128),
        # A decode batch of mixed contexts.
        _attend("attend_b64_len8192", 64, 37, 8192, 32, 8, 128),
        # Few long contexts, with the weights accumulated for eviction.
        _attend("attend_b4_len131072_scores", 4, 60001, 131072, 32, 8, 128, scores=True,
                page=128),
        # Verification of drafted tokens, every query head with its own key head.
        _attend("attend_fp16_d64_nq5", 16, 200, 4001, 16, 16, 64, dtype="fp16", nq=5, page=16),
        # Wide heads in fp32, with scores.
        _attend("attend_fp32_d256", 7, 1, 2049, 28, 4, 256, dtype="fp32", scores=True, page=32),
        # FP8 activations, a tensor-parallel rank's share of the heads.
        _attend("attend_fp8_b128", 128, 500, 2500, 8, 1, 128, dtype="fp8"),
        # One sequence a little over its budget.
        _evict("evict_b1_len301", 1, 301, 301, 8, 128, 256, 64),
        # A batch of prompts cut down after prefill.
        _evict("evict_b64_len8192", 64, 1500, 8192, 8, 128, 2048, 256),
        # Long contexts cut down.
        _evict("evict_b2_len131072", 2, 100003, 131072, 8, 128, 16384, 1024, page=128),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm, odd as often as not."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "attend", "attend", "evict"])
    D = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32", "fp8"])
    Hk = rng.choice([1, 2, 4, 8, 8, 16])
    if op == "store":
        T = _spread(rng, 1, max(2, 16384 * 6144 // ((Hk * 6) * D) // SIZES[dtype]))
        return dict(op="store", T=min(T, 16384), Hq=Hk * rng.choice([1, 2, 4]), Hk=Hk, D=D,
                    dtype=dtype, norm=rng.random() < 0.7, page=page, pad=rng.choice([0, 0, 16]))
    B = _spread(rng, 1, 64)
    top = max(64, min(131072, 3_000_000 * 128 // (B * Hk * D)))
    hi = _spread(rng, 16, top)
    lo = _spread(rng, 1, hi)
    if op == "evict":
        budget = _spread(rng, 8, max(9, hi // 2))
        return dict(op="evict", B=B, lo=lo, hi=hi, Hk=Hk, D=D, budget=budget,
                    recent=rng.randint(0, budget), page=page)
    group = rng.choice([1, 2, 4, 5, 8])
    nq = 1 if rng.random() < 0.6 else rng.randint(2, 6)
    return dict(op="attend", B=B, lo=lo, hi=hi, Hq=Hk * group, Hk=Hk, D=D, dtype=dtype, nq=nq,
                scores=rng.random() < 0.4, page=page)


def _lens(case):
    """Cached rows of each sequence: spread evenly over [lo, hi], the last the longest."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    lens = [lo + int((hi - lo) * ((i + 1) * 0.6180339887498949 % 1.0)) for i in range(B)]
    lens[-1] = hi
    return lens


def _nqs(case):
    """Query tokens of each sequence: 1 to nq, at most its cached rows but for the shortest."""
    return [case["nq"] if i % 3 == 0 else 1 + (i * 7) % case["nq"] for i in range(case["B"])]


# ------------------------------------------------------------------ inputs --
def _pack_rows(y):
    """Codes and {scale, mid} (before the row's norm factor) of rows y [..., D] in fp32."""
    lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    s = (hi * 0.5 - lo * 0.5) * (2.0 / 15.0)
    s = torch.where(s < 2.0 ** -126, torch.zeros_like(s), s)
    m = lo + 8.0 * s
    inv = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    codes = (torch.round((y - m) * inv).clamp(-8, 7) + 8).to(torch.uint8)
    return codes, s, m


def _nibbles(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _random_pool(g, pages, Hk, D, page):
    """A pool full of rows as the path meets them: normalised keys times a weight, values
    with a scale of their own for each row."""
    dev = g.device
    pool = torch.empty((pages, Hk, page // 16, 16 * D + 128), dtype=torch.uint8, device=dev)
    gk = 1 + 0.1 * torch.randn(D, generator=g, device=dev)
    step = max(1, (1 << 27) // (Hk * page * D))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        shape = (n, Hk, page // 16, 16, D)
        for which in range(2):
            y = torch.randn(shape, generator=g, device=dev)
            if which == 0:
                y *= gk * torch.rsqrt(y.square().mean(-1, keepdim=True))
            else:
                y *= torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=g, device=dev))
            codes, s, m = _pack_rows(y)
            at = which * 8 * D
            pool[p:p + n, ..., at:at + 8 * D] = _nibbles(codes).flatten(-2)
            at = 16 * D + 64 * which
            pool[p:p + n, ..., at:at + 64] = torch.cat([s, m], -1).bfloat16().view(
                torch.uint8).flatten(-2)
    return pool


def _random_qkv(g, T, heads, D, pad, dtype, norm):
    dev = g.device
    x = torch.randn((T, heads * D + pad), generator=g, device=dev)
    if not norm:  # rows that hold heads whose norm is done
        x *= 2.0
    else:
        x *= torch.exp(torch.randn((T, 1), generator=g, device=dev))
    if dtype == "fp8":
        x = x.clamp(-448, 448)
    return x.to(DTYPES[dtype])


def _tables(case, g, extra=0):
    """A page table over shuffled pages, and `extra` pages a sequence behind it."""
    lens, page = _lens(case), case["page"]
    need = [-(-n // page) for n in lens]
    total = sum(need) + extra * case["B"]
    order = torch.randperm(total, generator=g, device=g.device).to(torch.int32)
    table = torch.full((case["B"], max(need)), -1, dtype=torch.int32, device=g.device)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, order[at:].view(case["B"], extra), total


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = g.device
    Hk, D, page = case["Hk"], case["D"], case["page"]
    s = dict(case)
    if case["op"] == "store":
        T, Hq = case["T"], case["Hq"]
        pages = -(-T // page) + 2
        s["qkv"] = _random_qkv(g, T, Hq + 2 * Hk, D, case["pad"], case["dtype"], case["norm"])
        s["slots"] = torch.randperm(pages * page, generator=g, device=dev)[:T].contiguous()
        s["pool"] = torch.zeros((pages, Hk, page // 16, 16 * D + 128), dtype=torch.uint8,
                                device=dev)
        s["gq"] = s["gk"] = None
        if case["norm"]:
            s["gq"] = 1 + 0.1 * torch.randn(D, generator=g, device=dev)
            s["gk"] = 1 + 0.1 * torch.randn(D, generator=g, device=dev)
        return s
    s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=dev)
    if case["op"] == "attend":
        s["table"], _, pages = _tables(case, g)
        nqs = _nqs(case)
        s["T"] = sum(nqs)
        s["starts"] = torch.tensor([sum(nqs[:b]) for b in range(case["B"] + 1)],
                                   dtype=torch.int32, device=dev)
        s["qkv"] = _random_qkv(g, s["T"], case["Hq"] + 2 * Hk, D, 0, case["dtype"], False)
        s["pool"] = _random_pool(g, pages, Hk, D, page)
        s["sums"] = None
        if case["scores"]:
            s["sums"] = torch.rand((pages, Hk, page), generator=g, device=dev)
        return s
    keep = -(-case["budget"] // page)
    s["table"], s["to"], pages = _tables(case, g, keep)
    s["pool"] = _random_pool(g, pages, Hk, D, page)
    r = torch.rand((pages, Hk, page), generator=g, device=dev)
    s["sums"] = torch.where(r < 0.05, torch.zeros_like(r), -4.0 * torch.log(r) * r)
    return s


# -------------------------------------------------------------- plain form --
def _row_norm(x, gamma):
    return torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS), gamma


def _to(x, dtype):
    return (x.clamp(-448, 448) if dtype == torch.float8_e4m3fn else x).to(dtype)


def _slot_places(s, slots):
    page = s["page"]
    return slots // page, (slots % page) // 16, slots % 16


def _values(blocks, D, which):
    """The values, fp32 [..., 16, D], that blocks of 16 rows hold (0: keys, 1: values)."""
    codes = blocks[..., which * 8 * D:(which + 1) * 8 * D].unflatten(-1, (16, D // 2))
    codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8.0
    at = 16 * D + 64 * which
    par = blocks[..., at:at + 64].contiguous().view(torch.bfloat16).float().unflatten(-1, (16, 2))
    return par[..., 1:] + par[..., :1] * codes


def _plain_store(s):
    Hq, Hk, D, T = s["Hq"], s["Hk"], s["D"], s["T"]
    qkv, slots, pool = s["qkv"], s["slots"], s["pool"]
    x = qkv[:, :(Hq + 2 * Hk) * D].float().view(T, Hq + 2 * Hk, D)
    k, v = x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    factor = torch.ones_like(k[..., :1])
    if s["norm"]:
        q = x[:, :Hq]
        rq = torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS)
        factor = torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS)
        qkv[:, :Hq * D] = _to(q * rq * s["gq"], qkv.dtype).flatten(1)
        qkv[:, Hq * D:(Hq + Hk) * D] = _to(k * factor * s["gk"], qkv.dtype).flatten(1)
        k = k * s["gk"]
    page, block, row = _slot_places(s, slots)
    codes_k, sk, mk = _pack_rows(k)
    codes_v, sv, mv = _pack_rows(v)
    heads = torch.arange(Hk, device=qkv.device)
    p, h, b = page[:, None], heads[None], block[:, None]
    rows = pool.view(-1)
    base = ((p * Hk + h) * pool.shape[2] + b) * pool.shape[3]
    byte = torch.arange(D // 2, device=qkv.device)
    four = torch.arange(4, device=qkv.device)
    at = base[..., None] + row[:, None, None] * (D // 2) + byte
    rows[at] = _nibbles(codes_k)
    rows[at + 8 * D] = _nibbles(codes_v)
    at = base[..., None] + 16 * D + row[:, None, None] * 4 + four
    rows[at] = torch.cat([sk * factor, mk * factor], -1).bfloat16().view(torch.uint8)
    rows[at + 64] = torch.cat([sv, mv], -1).bfloat16().view(torch.uint8)
    got = pool[p, h, b]
    r = row[:, None, None, None].expand(T, Hk, 1, D)
    k = _values(got, D, 0).gather(2, r).squeeze(2)
    v = _values(got, D, 1).gather(2, r).squeeze(2)
    return {"qkv": qkv, "k": k.bfloat16().flatten(1), "v": v.bfloat16().flatten(1)}


def _plain_attend(s):
    Hq, Hk, D, page, B, n = s["Hq"], s["Hk"], s["D"], s["page"], s["B"], s["nq"]
    G, T, dev = Hq // Hk, s["T"], s["qkv"].device
    table = s["table"].clamp(min=0).long()
    blocks = s["pool"][table].transpose(1, 2).flatten(2, 3)  # [B, Hk, blocks, bytes]
    L = blocks.shape[2] * 16
    starts = s["starts"].long()
    count = starts[1:] - starts[:-1]
    i = torch.arange(n, device=dev)
    there = i < count[:, None]
    at = (starts[:-1, None] + i).clamp(max=T - 1)
    q = s["qkv"][:, :Hq * D][at].float().view(B, n, Hk, G, D).permute(0, 2, 1, 3, 4)
    q = q.reshape(B, Hk, n * G, D)
    w = q @ _values(blocks, D, 0).flatten(2, 3).transpose(-1, -2) * D ** -0.5
    sees = s["lens"].long()[:, None] - count[:, None] + i + 1  # rows that query i sees
    sees = torch.where(there, sees, torch.zeros_like(sees))
    hidden = torch.arange(L, device=dev) >= sees.repeat_interleave(G, 1)[:, None, :, None]
    w = w.masked_fill(hidden, float("-inf"))
    top = w.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    w = torch.exp(w - top)
    total = w.sum(-1, keepdim=True, dtype=torch.float64)
    w = w / torch.where(total > 0, total, torch.ones_like(total)).float()
    o = (w @ _values(blocks, D, 1).flatten(2, 3)).view(B, Hk, n, G, D).permute(0, 2, 1, 3, 4)
    lse = (top.double() + torch.log(total)).float().view(B, Hk, n, G).permute(0, 2, 1, 3)
    got = {"out": _to(o.reshape(B, n, Hq * D)[there], s["qkv"].dtype),
           "lse": lse.reshape(B, n, Hq)[there]}
    if s["scores"]:
        add = w.sum(2).view(B, Hk, -1, page).transpose(1, 2)
        s["sums"].index_put_((table,), add, accumulate=True)
        got["sums"] = s["sums"]
    return got


def _plain_evict(s):
    Hk, D, page, B, dev = s["Hk"], s["D"], s["page"], s["B"], s["pool"].device
    table, to, budget = s["table"].clamp(min=0).long(), s["to"].long(), s["budget"]
    lens = s["lens"].long()[:, None, None]
    sums = s["sums"][table].transpose(1, 2).flatten(2)  # [B, Hk, L]
    L = sums.shape[2]
    slot = torch.arange(L, device=dev)
    rank = torch.where(slot >= lens - s["recent"], torch.full_like(sums, float("inf")), sums)
    rank = torch.where(slot >= lens, torch.full_like(sums, float("-inf")), rank)
    kept = rank.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    new = lens.clamp(max=budget)
    place = torch.arange(kept.shape[2], device=dev)
    kept = torch.where(place < new, kept, torch.full_like(kept, L)).sort(-1).values
    b, h, at = (place < new).expand(kept.shape).nonzero(as_tuple=True)
    src = kept[b, h, at]
    p, t = table[b, src // page], to[b, at // page]
    got = {"lens": new.flatten().to(torch.int32),
           "kept": torch.full((B, Hk, budget), -1, dtype=torch.int32, device=dev)}
    got["kept"][b, h, at] = src.to(torch.int32)
    s["sums"][t, h, at % page] = s["sums"][p, h, src % page]
    pool = s["pool"]
    code = pool[..., :16 * D].unflatten(-1, (2, 16, D // 2))
    par = pool[..., 16 * D:].unflatten(-1, (2, 16, 4))
    code[t, h, at % page // 16, :, at % 16] = code[p, h, src % page // 16, :, src % 16]
    par[t, h, at % page // 16, :, at % 16] = par[p, h, src % page // 16, :, src % 16]
    # The moved rows are copies, byte for byte, so they come back as the bytes they are.
    return {**got, "pool": pool, "sums": s["sums"]}


# ----------------------------------------------------------- the operators --
def _own_store(s):
    import attention_qk_norm_b200 as qkn

    cache = qkn.KV4Cache(s["pool"], s["Hk"], s["D"], s["page"])
    qkn.qknorm_kv4_append(cache, s["qkv"], s["slots"], s["Hq"], s["gq"], s["gk"], EPS)
    k, v = qkn.qknorm_kv4_read(cache, s["slots"], dtype=torch.bfloat16)
    return {"qkv": s["qkv"], "k": k, "v": v}


def _own_attend(s):
    import attention_qk_norm_b200 as qkn

    cache = qkn.KV4Cache(s["pool"], s["Hk"], s["D"], s["page"], scores=s["sums"])
    if "workspace" not in s:  # a program's own, kept for its calls
        s["workspace"] = qkn.kv4_attention_workspace(cache, s["qkv"], s["Hq"], s["table"],
                                                     max_q=s["nq"], add_scores=s["scores"])
    out, lse = qkn.qknorm_kv4_attention(cache, s["qkv"], s["Hq"], s["table"], s["lens"],
                                        q_starts=s["starts"], max_q=s["nq"],
                                        add_scores=s["scores"], workspace=s["workspace"])
    got = {"out": out, "lse": lse}
    if s["scores"]:
        got["sums"] = s["sums"]
    return got


def _own_evict(s):
    import attention_qk_norm_b200 as qkn

    cache = qkn.KV4Cache(s["pool"], s["Hk"], s["D"], s["page"], scores=s["sums"])
    lens, kept = qkn.qknorm_kv4_evict(cache, s["table"], s["lens"], s["to"], s["budget"],
                                      s["recent"])
    return {"lens": lens, "kept": kept, "pool": s["pool"], "sums": s["sums"]}


def run(state):
    if own:
        return {"store": _own_store, "attend": _own_attend, "evict": _own_evict}[state["op"]](state)
    return {"store": _plain_store, "attend": _plain_attend,
            "evict": _plain_evict}[state["op"]](state)


def work(case):
    Hk, D = case["Hk"], case["D"]
    row = D + 8  # bytes of one cached token and head: two rows of codes, two pairs of parameters
    if case["op"] == "store":
        T, Hq, es = case["T"], case["Hq"], SIZES[case["dtype"]]
        heads = Hq + 2 * Hk if case["norm"] else 2 * Hk
        moved = T * D * es * (heads + (Hq + Hk if case["norm"] else 0))
        cached = T * Hk * row
        return {"bytes": moved + 2 * cached + T * 2 * Hk * D * 2 + 16 * T,
                "flops": T * D * (8 * heads + 4 * Hk)}
    lens = _lens(case)
    if case["op"] == "attend":
        nqs, Hq, es = _nqs(case), case["Hq"], SIZES[case["dtype"]]
        T = sum(nqs)
        cached = sum(lens) * Hk * row
        scored = 8 * sum(lens) * Hk if case["scores"] else 0
        pairs = sum(sum(max(0, n - k + i + 1) for i in range(k)) for n, k in zip(lens, nqs))
        return {"bytes": cached + scored + T * Hq * (2 * D * es + 4), "flops": pairs * Hq * 4 * D}
    kept = sum(min(n, case["budget"]) for n in lens) * Hk
    return {"bytes": 4 * sum(lens) * Hk + kept * (2 * row + 8) + 8 * case["B"],
            "flops": sum(lens) * Hk}


# ------------------------------------------------------------------- exact --
def _exact_rows(s, b, n, which):
    """Values of sequence b's first n rows, float64 [Hk, n, D], unpacked byte by byte."""
    D, page = s["D"], s["page"]
    t = torch.arange(n, device=s["pool"].device)
    blocks = s["pool"][s["table"][b].long()[t // page], :, (t % page) // 16].transpose(0, 1)
    r = t % 16
    byte = blocks.gather(2, (which * 8 * D + r[:, None] * (D // 2)
                             + torch.arange(D // 2, device=t.device)).expand(s["Hk"], -1, -1))
    codes = torch.empty(byte.shape[:2] + (D,), dtype=torch.float64, device=t.device)
    codes[..., 0::2] = (byte % 16).double()
    codes[..., 1::2] = torch.div(byte, 16, rounding_mode="floor").double()
    four = blocks.gather(2, (16 * D + 64 * which + r[:, None] * 4
                             + torch.arange(4, device=t.device)).expand(s["Hk"], -1, -1)).int()
    scale = ((four[..., 0] + 256 * four[..., 1]) << 16).view(torch.float32).double()
    mid = ((four[..., 2] + 256 * four[..., 3]) << 16).view(torch.float32).double()
    return scale[..., None] * (codes - 8) + mid[..., None]


def _exact_store(s):
    Hq, Hk, D, T = s["Hq"], s["Hk"], s["D"], s["T"]
    whole = s["qkv"].to(torch.float64)
    got = whole.clone()
    x = whole[:, :(Hq + 2 * Hk) * D].reshape(T, -1, D)
    k, v = x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    factor = 1.0
    if s["norm"]:
        rinv = (x[:, :Hq + Hk].square().mean(-1, keepdim=True) + EPS) ** -0.5
        factor = rinv[:, Hq:]
        got[:, :Hq * D] = (x[:, :Hq] * rinv[:, :Hq] * s["gq"].double()).reshape(T, -1)
        got[:, Hq * D:(Hq + Hk) * D] = (k * factor * s["gk"].double()).reshape(T, -1)
        k = (k.float() * s["gk"]).double()

    def held(y, factor):
        # A code is defined by steps in fp32: 16-bit rows put many values exactly half way
        # between two codes, and these steps say which one each gets.
        y = y.float()
        lo, hi = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
        step = (hi / 2 - lo / 2) * (2 / 15)
        mid = lo + 8 * step
        code = ((y - mid) * (1 / torch.where(step > 0, step, 1.0))).round().clamp(-8, 7).double()
        step, mid = ((p.double() * factor).bfloat16().double() for p in (step, mid))
        return (mid + step * code).reshape(T, -1)

    return {"qkv": got, "k": held(k, factor), "v": held(v, 1.0)}


def _exact_attend(s):
    Hq, Hk, D, page = s["Hq"], s["Hk"], s["D"], s["page"]
    G, dev = Hq // Hk, s["qkv"].device
    lens, starts = s["lens"].tolist(), s["starts"].tolist()
    out = torch.zeros((s["T"], Hk, G, D), dtype=torch.float64, device=dev)
    lse = torch.full((s["T"], Hk, G), float("-inf"), dtype=torch.float64, device=dev)
    sums = s["sums"].double() if s["scores"] else None
    for b, n in enumerate(lens):
        k, v = _exact_rows(s, b, n, 0), _exact_rows(s, b, n, 1)
        nq = starts[b + 1] - starts[b]
        for i in range(nq):
            sees, t = max(0, n - nq + i + 1), starts[b] + i
            if sees == 0:
                continue
            q = s["qkv"][t, :Hq * D].to(torch.float64).view(Hk, G, D)
            w = torch.einsum("hgd,hnd->hgn", q, k[:, :sees]) / math.sqrt(D)
            lse[t] = torch.logsumexp(w, -1)
            w = torch.softmax(w, -1)
            out[t] = torch.einsum("hgn,hnd->hgd", w, v[:, :sees])
            if sums is not None:
                at = torch.arange(sees, device=dev)
                sums[s["table"][b].long()[at // page], :, at % page] += w.sum(1).T
    got = {"out": out.reshape(s["T"], -1), "lse": lse.reshape(s["T"], Hq)}
    if sums is not None:
        got["sums"] = sums
    return got


def exact(case, seed):
    if case["op"] == "evict":  # a choice and copies: no computed numbers
        return None
    s = prepare(case, seed)
    return _exact_store(s) if case["op"] == "store" else _exact_attend(s)
