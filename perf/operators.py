"""Measured cases of the cache-append and 8-bit-cache attention operators.

Three operators of the serving path, each in its plain form (elementary torch
operations in fp32) and, where `own` is true, through the package:

  append   new tokens' K (with the rotary rotation of their positions) and V
           stored into the pages of their sequences, the queries rotated on the
           way; into a bf16 or fp32 pool
  append8  the same into a pool held in 8 bits (e4m3) with one power-of-two
           scale per (page of 16 tokens, KV head)
  attend8  the query tokens of every request attending over the request's
           pages of such a pool: prompts (causal) and single tokens
"""

import math
import random

import torch

own = False

PAGE = 16
POS = 8192          # positions of the rotary table
E4M3_MAX = 448.0


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one generated token of one request into a bf16 cache: latency alone
        dict(name="append_one", op="append", cache="bf16", n_seq=1, new_lo=1, new_hi=1, held_hi=1000, kv_heads=8,
             group=4, dim=128, rotate=True, fused=True, shape=1),
        # the prompts of 16 batched requests, sliced out of one fused projection
        dict(name="append_prompts", op="append", cache="bf16", n_seq=16, new_lo=32, new_hi=128, held_hi=700, kv_heads=8,
             group=4, dim=128, rotate=True, fused=True, shape=2),
        # fp32 cache of the small configuration's head size, ragged lengths
        dict(name="append_f32", op="append", cache="f32", n_seq=5, new_lo=1, new_hi=700, held_hi=100, kv_heads=4,
             group=2, dim=64, rotate=True, fused=False, shape=3),
        # one generation step of 64 requests into an 8-bit cache
        dict(name="append8_step", op="append8", cache="e4m3", n_seq=64, new_lo=1, new_hi=1, held_hi=2000, kv_heads=8,
             group=4, dim=128, rotate=True, fused=True, shape=4),
        # ragged prompts that continue pages already begun
        dict(name="append8_prompts", op="append8", cache="e4m3", n_seq=16, new_lo=32, new_hi=1024, held_hi=700,
             kv_heads=8, group=4, dim=128, rotate=True, fused=True, shape=5),
        # 32 precomputed chunks of 2,048 tokens written whole
        dict(name="append8_chunks", op="append8", cache="e4m3", n_seq=32, new_lo=2048, new_hi=2048, held_hi=0,
             kv_heads=8, group=0, dim=128, rotate=True, fused=False, shape=6),
        # one token of one request over a short context: latency alone
        dict(name="attend8_one", op="attend8", n_req=1, chunks=1, chunk_lo=500, chunk_hi=520, q_lo=1, q_hi=1, ctx_hi=100,
             kv_heads=8, group=4, causal=True, shape=7),
        # a generation step of 16 requests over 4-8 retrieved chunks each
        dict(name="attend8_step16", op="attend8", n_req=16, chunks=6, chunk_lo=256, chunk_hi=1024, q_lo=1, q_hi=1,
             ctx_hi=384, kv_heads=8, group=4, causal=True, shape=8),
        # a generation step of 64 requests with long contexts: HBM alone
        dict(name="attend8_step64", op="attend8", n_req=64, chunks=12, chunk_lo=512, chunk_hi=1536, q_lo=1, q_hi=1,
             ctx_hi=1024, kv_heads=8, group=4, causal=True, shape=9),
        # the 100-token query of one request over ten 1,000-token chunks
        dict(name="attend8_prompt", op="attend8", n_req=1, chunks=10, chunk_lo=1000, chunk_hi=1000, q_lo=100, q_hi=100,
             ctx_hi=0, kv_heads=8, group=4, causal=True, shape=10),
        # 16 requests' queries of 32-128 tokens over ragged chunks
        dict(name="attend8_prompts16", op="attend8", n_req=16, chunks=6, chunk_lo=256, chunk_hi=1024, q_lo=32,
             q_hi=128, ctx_hi=0, kv_heads=8, group=4, causal=True, shape=11),
        # 64 query heads, 256 query tokens over 32 chunks of 2,048
        dict(name="attend8_long", op="attend8", n_req=1, chunks=32, chunk_lo=2048, chunk_hi=2048, q_lo=256, q_hi=256,
             ctx_hi=0, kv_heads=8, group=8, causal=True, shape=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {}   # the largest listed bytes and flops of each operator
    for c in listed():
        w, m = work(c), most.setdefault(c["op"], [0.0, 0.0])
        m[:] = max(m[0], w["bytes"]), max(m[1], w["flops"])
    while True:
        op = rng.choice(["append", "append8", "attend8", "attend8"])
        if op == "attend8":
            single = rng.random() < 0.5
            q_hi = _log_int(rng, 1, 4) if single else _log_int(rng, 2, 400)
            lo = _log_int(rng, 1, 2500)
            c = dict(op=op, n_req=_log_int(rng, 1, 64), chunks=_log_int(rng, 1, 40), chunk_lo=lo,
                     chunk_hi=lo + rng.randrange(0, 1 + lo), q_lo=rng.randint(1, q_hi), q_hi=q_hi,
                     ctx_hi=rng.choice([0, 7, 60, 384]), kv_heads=rng.choice([1, 2, 4, 8, 16, 32]),
                     group=rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), causal=rng.random() < 0.85)
        else:
            hi = _log_int(rng, 1, 3 if rng.random() < 0.4 else 4000)
            cache = "e4m3" if op == "append8" else rng.choice(["bf16", "bf16", "f32"])
            c = dict(op=op, cache=cache, n_seq=_log_int(rng, 1, 64), new_lo=rng.randint(1, hi), new_hi=hi,
                     held_hi=rng.choice([0, 15, 200, 2000]), kv_heads=rng.choice([1, 2, 4, 8, 16, 32]),
                     group=rng.choice([0, 1, 2, 3, 4, 5, 7, 8]), dim=rng.choice([64, 128]) if cache == "f32" else 128,
                     rotate=rng.random() < 0.85, fused=rng.random() < 0.6)
        c["shape"] = rng.randrange(1, 1 << 30)
        w = work(c)
        if w["bytes"] <= most[op][0] and w["flops"] <= most[op][1]:
            return c


# ------------------------------------------------------------------- shapes

def _spread(r, n, lo, hi):
    return [r.randint(lo, hi) for _ in range(n)]


def _append_shape(c):
    """Per sequence: tokens held before the call, new tokens, position of slot 0."""
    r = random.Random(c["shape"])
    new = _spread(r, c["n_seq"], c["new_lo"], c["new_hi"])
    held = _spread(r, c["n_seq"], 0, c["held_hi"])
    pos0 = [r.randint(0, POS - h - n) for h, n in zip(held, new)]
    return held, new, pos0


def _attend_shape(c):
    """Per request: the lengths of its chunks (the last one is its own context,
    which ends in the query tokens) and its query tokens."""
    r = random.Random(c["shape"])
    q = _spread(r, c["n_req"], c["q_lo"], c["q_hi"])
    lens = [_spread(r, c["chunks"], c["chunk_lo"], c["chunk_hi"]) + [n + r.randint(0, c["ctx_hi"])] for n in q]
    return lens, q


def _prefix(xs):
    out = [0]
    for x in xs:
        out.append(out[-1] + x)
    return out


def work(case):
    c = case
    if c["op"] == "attend8":
        lens, q = _attend_shape(c)
        n = [sum(x) for x in lens]
        pages = sum(-(-x // PAGE) for xs in lens for x in xs)
        hq = c["kv_heads"] * c["group"]
        seen = sum(nq * nk - (nq * (nq - 1) // 2 if c["causal"] else 0) for nq, nk in zip(q, n))
        return {"bytes": float(sum(n) * c["kv_heads"] * 256 + pages * c["kv_heads"] * 8 + sum(q) * hq * 512 + pages * 4),
                "flops": float(4 * 128 * hq * seen)}
    held, new, _ = _append_shape(c)
    size_in = 4 if c["cache"] == "f32" else 2
    size_out = {"f32": 4, "bf16": 2, "e4m3": 1}[c["cache"]]
    row = c["kv_heads"] * c["dim"]
    total = sum(new)
    b = total * row * 2 * (size_in + size_out) + total * row * c["group"] * 2 * size_in
    b += total * (4 * c["dim"] if c["rotate"] else 0)
    if c["cache"] == "e4m3":
        b += sum((h + n - 1) // PAGE - h // PAGE + 1 for h, n in zip(held, new)) * c["kv_heads"] * 8
    return {"bytes": float(b), "flops": float(total * row * (1 + c["group"]) * 3)}


# ------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2 + 1)
    return g


def _channels(g, heads, dim, outliers=2):
    """Per (head, channel) scale of synthetic keys or values: lognormal, two
    outlier channels a head."""
    s = torch.exp(0.5 * torch.randn(heads, dim, generator=g, device="cuda"))
    at = torch.randint(0, dim, (heads, outliers), generator=g, device="cuda")
    return s.scatter(1, at, s.gather(1, at) * 8.0)


def _pow2_scale(amax, top):
    """The smallest power of two, at least 2^-24 and at most 2^top, whose 448
    multiples cover amax."""
    m, e = torch.frexp(amax)                      # amax = m 2^e, m in [0.5, 1)
    k = torch.where(m > 0.875, e - 8, e - 9)      # 448 = 0.875 * 2^9
    k = torch.where(amax == 0, torch.full_like(k, -24), k).clamp(-24, top)
    return ((k.to(torch.int32) + 127) << 23).view(torch.float32)


def _random_cache8(g, pages, heads, pages_at_once=4096):
    """Codes [1, pages, heads, 16, 128] and scales [1, pages, heads] of random
    keys (or values) with outlier channels."""
    ch = _channels(g, heads, 128)
    codes = torch.empty(1, pages, heads, PAGE, 128, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(1, pages, heads, device="cuda")
    for p0 in range(0, pages, pages_at_once):
        n = min(pages_at_once, pages - p0)
        x = torch.randn(n, heads, PAGE, 128, generator=g, device="cuda") * ch[:, None, :]
        s = _pow2_scale(x.abs().amax((2, 3)), 7)
        codes[0, p0:p0 + n] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn)
        scale[0, p0:p0 + n] = s
    return codes, scale


def _dev(xs):
    return torch.tensor(xs, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": dict(c)}
    H, G = c["kv_heads"], c["group"]
    if c["op"] == "attend8":
        lens, q = _attend_shape(c)
        flat = [x for xs in lens for x in xs]
        pages = [-(-x // PAGE) for x in flat]
        num_pages = sum(pages) + 3
        host = [_prefix([len(x) for x in lens]), _prefix(flat), _prefix(pages),
                torch.randperm(num_pages, generator=g, device="cuda")[: sum(pages)].to(torch.int32), _prefix(q)]
        s["req_chunk_off"], s["chunk_doc_off"], s["chunk_page_off"], s["q_off"] = (_dev(host[i]) for i in (0, 1, 2, 4))
        s["page_ids"] = host[3]
        s["max_doc"], s["max_q"] = max(sum(x) for x in lens), max(q)
        s["total_doc"], s["total_q"] = sum(flat), sum(q)
        s["k"], s["k_scale"] = _random_cache8(g, num_pages, H)
        s["v"], s["v_scale"] = _random_cache8(g, num_pages, H)
        s["q"] = torch.randn(sum(q), H * G, 128, generator=g, device="cuda").to(torch.bfloat16)
        if own:   # what a serving program keeps for a batch: the pool, the batch, its workspace and output
            import serving_prefill_b200 as sp
            s["pool"] = sp.KV8Pool(1, num_pages, H, 128, k=s["k"], v=s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"])
            s["batch"] = sp.Batch(*host)
            s["workspace"] = sp.new_workspace(s["pool"], s["batch"], H * G)
            s["o"] = torch.empty(sum(q), H * G, 128, dtype=torch.bfloat16, device="cuda")
        return s
    held, new, pos0 = _append_shape(c)
    D, T = c["dim"], sum(new)
    dt = torch.float32 if c["cache"] == "f32" else torch.bfloat16
    pages = [-(-(h + n) // PAGE) for h, n in zip(held, new)]
    num_pages = sum(pages) + 3
    s["tok_off"], s["page_off"] = _dev(_prefix(new)), _dev(_prefix(pages))
    s["start"], s["pos0"] = _dev(held), _dev(pos0)
    s["page_ids"] = torch.randperm(num_pages, generator=g, device="cuda")[: sum(pages)].to(torch.int32)
    heads = H * (G + 2)
    if c["fused"]:
        x = torch.randn(T, heads, D, generator=g, device="cuda").to(dt)
        x[:, H * G:H * (G + 1)] *= _channels(g, H, D).to(dt)
        x[:, H * (G + 1):] *= _channels(g, H, D).to(dt)
        s["q"], s["k"], s["v"] = x[:, :H * G], x[:, H * G:H * (G + 1)], x[:, H * (G + 1):]
    else:
        s["q"] = torch.randn(T, H * G, D, generator=g, device="cuda").to(dt)
        s["k"] = (torch.randn(T, H, D, generator=g, device="cuda") * _channels(g, H, D)).to(dt)
        s["v"] = (torch.randn(T, H, D, generator=g, device="cuda") * _channels(g, H, D)).to(dt)
    if G == 0:
        s["q"] = None
    s["rope"] = None
    if c["rotate"]:   # (cos, sin) of position p and pair i: p * 10000^(-2 i / D)
        theta = 10000.0 ** (-2.0 * torch.arange(D // 2, dtype=torch.float64, device="cuda") / D)
        ang = torch.arange(POS, dtype=torch.float64, device="cuda")[:, None] * theta
        s["rope"] = torch.stack([ang.cos(), ang.sin()], -1).float()
    if c["cache"] == "e4m3":
        s["pool_k"], s["pool_ks"] = _random_cache8(g, num_pages, H)
        s["pool_v"], s["pool_vs"] = _random_cache8(g, num_pages, H)
    else:
        shape = (1, num_pages, H, PAGE, D)
        s["pool_k"] = torch.randn(shape, generator=g, device="cuda").to(dt)
        s["pool_v"] = torch.randn(shape, generator=g, device="cuda").to(torch.float16 if dt == torch.bfloat16 else dt)
    if own:
        import serving_prefill_b200 as sp
        if c["cache"] == "e4m3":
            s["pool"] = sp.KV8Pool(1, num_pages, H, D, k=s["pool_k"], v=s["pool_v"], k_scale=s["pool_ks"],
                                   v_scale=s["pool_vs"])
        else:
            s["pool"] = sp.KVPool(1, num_pages, H, D, dtype=dt, k=s["pool_k"], v=s["pool_v"])
        s["seqs"] = sp.Append(s["tok_off"], s["start"], s["page_off"], s["page_ids"], pos0=s["pos0"], total_new=T)
        s["q_out"] = None if G == 0 else torch.empty(T, H * G, D, dtype=dt, device="cuda")
    return s


# ------------------------------------------------------------------- one pass

def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import serving_prefill_b200 as sp
        if op == "attend8":
            sp.rag_kv8_attn(s["pool"], 0, s["batch"], s["q"], s["o"], s["workspace"], causal=s["case"]["causal"])
            return s["o"]
        call = sp.rag_kv8_append if op == "append8" else sp.rag_kv_append
        call(s["pool"], 0, s["seqs"], s["k"], s["v"], rope=s["rope"], q=s["q"], q_out=s["q_out"])
        out = {"k": s["pool_k"], "v": s["pool_v"]}
        if op == "append8":
            out["k_scale"], out["v_scale"] = s["pool_ks"], s["pool_vs"]
        if s["q_out"] is not None:
            out["q"] = s["q_out"]
        return out
    return _plain_attend(s) if op == "attend8" else _plain_append(s)


def _rotate(x, cs):
    """Pairs (i, i + D/2) turned by the angle of cs = (cos, sin) [T, D/2, 2]."""
    h = x.shape[-1] // 2
    a, b, co, si = x[..., :h], x[..., h:], cs[:, None, :, 0], cs[:, None, :, 1]
    return torch.cat([a * co - b * si, b * co + a * si], -1)


def _plain_append(s):
    t = torch.arange(s["k"].shape[0], dtype=torch.int32, device="cuda")
    seq = torch.searchsorted(s["tok_off"][1:], t, right=True)
    at = s["start"][seq] + t - s["tok_off"][seq]            # token's index in its sequence
    page = s["page_ids"][s["page_off"][seq] + torch.div(at, PAGE, rounding_mode="floor")].long()
    slot = (at % PAGE).long()
    k, v = s["k"].float(), s["v"].float()
    q = None if s["q"] is None else s["q"].float()
    if s["rope"] is not None:
        cs = s["rope"][s["pos0"][seq] + at]
        k = _rotate(k, cs)
        q = None if q is None else _rotate(q, cs)
    out = {}
    # tokens of the call in the same page: unit u is the n-th page of its sequence that the call touches
    n_unit = t.numel() // PAGE + 2 * s["start"].numel()
    first = torch.div(s["tok_off"][:-1], PAGE, rounding_mode="floor") + 2 * torch.arange(s["start"].numel(), device="cuda")
    unit = first[seq] + torch.div(at, PAGE, rounding_mode="floor") - torch.div(s["start"][seq], PAGE, rounding_mode="floor")
    lo = torch.full((n_unit,), PAGE, device="cuda").scatter_reduce(0, unit, slot, "amin")
    where = torch.zeros(n_unit, dtype=torch.long, device="cuda").scatter(0, unit, page)
    src = torch.where(lo < PAGE, torch.arange(n_unit, device="cuda"), unit[0])   # unused units repeat the first one
    where, lo = where[src], lo[src]
    for name, x, top in (("k", k, 127), ("v", v, 7)):
        pool = s["pool_" + name][0]
        held = torch.arange(PAGE, device="cuda")[None, :] < lo[:, None]            # slots filled by earlier calls
        keep = (held | (lo[:, None] > 0))[:, None, :, None]
        if s["case"]["op"] == "append8":
            scale = s["pool_" + name + "s"][0]
            big = x.abs().amax(-1)
            need = torch.zeros(n_unit, x.shape[1], device="cuda").scatter_reduce(0, unit[:, None].expand_as(big), big, "amax")
            need = _pow2_scale(need[src], top)
            old = scale[where]
            new = torch.where(lo[:, None] == 0, need, torch.maximum(old, need))
            codes = pool.view(torch.uint8)
            block = codes[where]
            was = block.view(torch.float8_e4m3fn).float() * (old / new)[:, :, None, None]
            was = torch.where(held[:, None, :, None], was.to(torch.float8_e4m3fn).view(torch.uint8), block)
            codes[where] = torch.where(keep, was, torch.zeros_like(was))
            scale[where] = new
            y = (x / new[unit][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
            codes[page, :, slot] = y.to(torch.float8_e4m3fn).view(torch.uint8)
            out[name + "_scale"] = s["pool_" + name + "s"]
        else:
            block = pool[where]
            pool[where] = torch.where(keep, block, torch.zeros_like(block))
            pool[page, :, slot] = x.to(pool.dtype)
        out[name] = s["pool_" + name]
    if q is not None:
        out["q"] = q.to(s["q"].dtype)
    return out


def _plain_attend(s):
    c = s["case"]
    H, G, B = c["kv_heads"], c["group"], c["n_req"]
    doc = torch.arange(s["total_doc"], dtype=torch.int32, device="cuda")
    ch = torch.searchsorted(s["chunk_doc_off"][1:], doc, right=True)
    off = doc - s["chunk_doc_off"][ch]
    page = s["page_ids"][s["chunk_page_off"][ch] + torch.div(off, PAGE, rounding_mode="floor")].long()
    slot = (off % PAGE).long()
    first = s["chunk_doc_off"][s["req_chunk_off"].long()]                  # [B + 1] first token of a request
    n_doc, n_q = first[1:] - first[:-1], s["q_off"][1:] - s["q_off"][:-1]
    n = torch.arange(s["max_doc"], device="cuda")
    j = torch.arange(s["max_q"], device="cuda")
    tok = (first[:-1, None] + n).clamp(max=s["total_doc"] - 1)             # [B, N]
    row = (s["q_off"][:-1, None] + j).clamp(max=s["total_q"] - 1)          # [B, Q]

    def dense(codes, scale):
        x = codes[0].view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).float() * scale[0][page][:, :, None]
        return x[tok].permute(0, 2, 1, 3)                                  # [B, H, N, 128]

    q = s["q"].float()[row].view(B, -1, H, G, 128).permute(0, 2, 1, 3, 4).reshape(B, H, -1, 128)
    x = torch.matmul(q, dense(s["k"], s["k_scale"]).transpose(2, 3)) / math.sqrt(128.0)
    x = x.view(B, H, s["max_q"], G, -1)
    limit = n_doc[:, None] - n_q[:, None] + j if c["causal"] else n_doc[:, None].expand(B, j.numel()) - 1
    seen = (n < n_doc[:, None, None]) & (n <= limit[:, :, None])           # [B, Q, N]
    x.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = torch.exp_(x.sub_(torch.where(m == -math.inf, 0.0, m)))
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, H, -1, x.shape[-1]), dense(s["v"], s["v_scale"])).view(B, H, -1, G, 128)
    o = o / torch.where(l == 0, 1.0, l)
    o = o.permute(0, 2, 1, 3, 4).reshape(B * s["max_q"], H * G, 128)
    t = torch.arange(s["total_q"], dtype=torch.int32, device="cuda")
    b = torch.searchsorted(s["q_off"][1:], t, right=True)
    return o[b * s["max_q"] + t - s["q_off"][b]].to(torch.bfloat16)


# ------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_attend(s) if case["op"] == "attend8" else _exact_append(s)


def _exact_attend(s):
    c = s["case"]
    lens, qs = _attend_shape(c)
    H, G = c["kv_heads"], c["group"]
    out = torch.empty(s["total_q"], H * G, 128, dtype=torch.float64, device="cuda")
    ids = s["page_ids"].long()
    p0 = q0 = 0
    for chunks, nq in zip(lens, qs):
        rows = []
        for n in chunks:
            at = torch.arange(n, device="cuda")
            rows.append(ids[p0 + at // PAGE] * PAGE + at % PAGE)
            p0 += -(-n // PAGE)
        rows = torch.cat(rows)
        n = rows.numel()
        hide = None
        if c["causal"]:
            hide = torch.arange(n, device="cuda")[None, :] > (n - nq + torch.arange(nq, device="cuda"))[:, None]
        for h in range(H):
            k, v = _rows8(s, "k", h, rows), _rows8(s, "v", h, rows)
            for i in range(h * G, (h + 1) * G):
                a = s["q"][q0:q0 + nq, i].double() @ k.T * 128.0 ** -0.5
                if hide is not None:
                    a.masked_fill_(hide, -math.inf)
                out[q0:q0 + nq, i] = torch.softmax(a, -1) @ v
        q0 += nq
    return out


def _rows8(s, name, h, rows):
    page, slot = rows // PAGE, rows % PAGE
    x = s[name][0].view(torch.uint8)[page, h, slot].view(torch.float8_e4m3fn).double()
    return x * s[name + "_scale"][0, page, h].double()[:, None]


def _exact_append(s):
    c = s["case"]
    held, new, pos0 = _append_shape(c)
    D = c["dim"]
    ids = s["page_ids"].tolist()
    k, v = s["k"].double(), s["v"].double()
    q = None if s["q"] is None else s["q"].double()
    if s["rope"] is not None:
        p = torch.cat([a + h + torch.arange(n, device="cuda") for a, h, n in zip(pos0, held, new)])
        z = torch.complex(*s["rope"].double()[p].unbind(-1))[:, None, :]
        turn = lambda x: torch.cat([(w := torch.complex(x[..., :D // 2], x[..., D // 2:]) * z).real, w.imag], -1)  # noqa: E731
        k, q = turn(k), None if q is None else turn(q)
    out = {}
    for name, x, top in (("k", k, 127), ("v", v, 7)):
        pool = s["pool_" + name].double()
        scale = s["pool_" + name + "s"].double() if c["op"] == "append8" else None
        t0 = p0 = 0
        for h, n in zip(held, new):
            for a in range(h // PAGE, (h + n - 1) // PAGE + 1):      # the pages of the sequence that get tokens
                lo, hi = max(h, a * PAGE), min(h + n, (a + 1) * PAGE)
                page, rows = ids[p0 + a], x[t0 + lo - h:t0 + hi - h].transpose(0, 1)
                if lo == a * PAGE:
                    pool[0, page] = 0
                if scale is not None:
                    m, e = torch.frexp(rows.abs().amax((1, 2)) / E4M3_MAX)      # m in [0.5, 1): 2^e, or 2^(e-1) at a power of two
                    e = torch.where(m == 0, -24, torch.where(m == 0.5, e - 1, e)).clamp(-24, top)
                    need = torch.ldexp(torch.ones_like(m), e)
                    grown = need if lo == a * PAGE else torch.maximum(need, scale[0, page])
                    pool[0, page, :, :lo % PAGE] *= (scale[0, page] / grown)[:, None, None]
                    scale[0, page] = grown
                    rows = rows / grown[:, None, None]
                pool[0, page, :, lo % PAGE:lo % PAGE + hi - lo] = rows
            t0 += n
            p0 += -(-(h + n) // PAGE)
        out[name] = pool
        if scale is not None:
            out[name + "_scale"] = scale
    if q is not None:
        out["q"] = q
    return out
