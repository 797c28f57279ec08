"""The 16-bit append and the 16-bit attention together: chunks, prompt and
generated tokens appended to a bf16 pool, the attention reading what was written."""

import pytest
import torch

import serving_prefill_b200 as sp
from kv8_support import check, reference

pytestmark = pytest.mark.gpu


def test_prompt_then_generation_on_a_16_bit_pool():
    """Two requests: retrieved chunks appended at their positions, then a prompt
    and 20 tokens. Each call appends the new tokens (K and Q turned on the way;
    the turned K, which the attention takes as its query block's own, comes out
    of the same call as further heads of q) and attends over what was cached
    before. Outputs are held to fp64 attention over the pool's contents and the
    tokens' own K, V; the bounds of the 8-bit attention count every rounding of
    this one too (weights and partial rows in fp16, the output in bf16, fp32
    sums) and more. The pool is held to the values it was given: half a step of
    bf16 for K (2^-8, and fp32's 6 * 2^-24 of the row's largest in the turn), V
    exactly (bf16 values within fp16's normal range)."""
    H, G, layers, steps = 2, 4, 2, 20
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    chunks, prompt = [[90, 40], [33]], [21, 7]
    docs = [sum(c) for c in chunks]
    counts = [[-(-n // 16) for n in c] + [-(-(p + steps) // 16)] for c, p in zip(chunks, prompt)]
    total = sum(map(sum, counts))
    ids = torch.randperm(total + 2).tolist()
    pages, at = [], 0
    for cs in counts:
        row = []
        for n in cs:
            row.append(ids[at:at + n])
            at += n
        pages.append(row)
    pool = sp.KVPool(layers, total + 2, H, 128)
    pool.k.fill_(float("nan"))
    pool.v.fill_(float("nan"))
    rope = sp.rag_rope_cos_sin(10000.0, 128, 512)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    given = {}

    def turn(x, pos):
        x, cs = x.double(), rope[pos].double()
        a, c = x[:, :64], x[:, 64:]
        return torch.cat([a * cs[:, 0] - c * cs[:, 1], c * cs[:, 0] + a * cs[:, 1]], -1)

    def note(layer, k, v, where):
        for r, (b, pos) in enumerate(where):
            given[layer, b, pos] = turn(k[r], pos), v[r].double(), k[r].double().abs().max()

    for layer in range(layers):
        for b, cs in enumerate(chunks):
            pos = 0
            for c, n in enumerate(cs):
                k, v = rnd(n, H, 128), rnd(n, H, 128)
                sp.rag_kv_append(pool, layer, sp.Append([0, n], [0], [0, len(pages[b][c])], pages[b][c], pos0=[pos]),
                                 k, v, rope=rope, device_err=err)
                note(layer, k, v, [(b, pos + i) for i in range(n)])
                pos += n

    def held(layer, b, own):
        ks, vs = [], []
        for pg, n in zip(pages[b], chunks[b] + [own]):
            for dst, x in ((ks, pool.k), (vs, pool.v)):
                dst.append(x[layer][pg].double().permute(0, 2, 1, 3).reshape(-1, H, 128)[:n])
        return torch.cat(ks).cpu(), torch.cat(vs).cpu()

    ctx = [pages[b][-1] for b in range(2)]
    page_off = [0, len(ctx[0]), len(ctx[0]) + len(ctx[1])]

    def batch(own, n_q):
        doc, page, ids = [0], [0], []
        for b in range(2):
            for n, p in zip(chunks[b] + [own[b]], pages[b]):
                doc.append(doc[-1] + n)
                page.append(page[-1] + -(-n // 16))
                ids += p[: -(-n // 16)]
        return sp.Batch([0, 3, 5], doc, page, ids, [0, n_q[0], sum(n_q)])

    own = [0, 0]
    for n_q in [prompt] + [[1, 1]] * steps:
        T = sum(n_q)
        seqs = sp.Append([0, n_q[0], T], own, page_off, ctx[0] + ctx[1], pos0=docs)
        b0 = batch(own, n_q)
        for layer in range(layers):
            x = rnd(T, H * (G + 2), 128)                    # one fused projection: q heads, k heads, v heads
            k, v = x[:, H * G:H * (G + 1)], x[:, H * (G + 1):]
            turned = torch.empty(T, H * (G + 1), 128, dtype=torch.bfloat16, device="cuda")
            sp.rag_kv_append(pool, layer, seqs, k, v, rope=rope, q=x[:, :H * (G + 1)], q_out=turned, device_err=err)
            where = [(b, docs[b] + own[b] + i) for b in range(2) for i in range(n_q[b])]
            note(layer, k, v, where)
            q, kq, vq = (t.contiguous() for t in (turned[:, :H * G], turned[:, H * G:], v))
            o, lse = torch.empty_like(q), torch.empty(T, H * G, device="cuda")
            ws = sp.new_workspace(pool, b0, H * G)
            sp.rag_fused_prefill_attn(pool, layer, b0, q, kq, vq, o, ws, row_lse=lse)
            assert sp.rag_last_device_error(ws) == (0, 0)
            dense, r = [], 0
            for b in range(2):
                kk, vv = held(layer, b, own[b])
                # what the append stored for the new tokens is what it gave out as their turned K
                new = held(layer, b, own[b] + n_q[b])[0][-n_q[b]:]
                mine = slice(r, r + n_q[b])
                assert torch.equal(new, kq[mine].double().cpu())
                dense.append((torch.cat([kk, kq[mine].double().cpu()]), torch.cat([vv, vq[mine].double().cpu()])))
                r += n_q[b]
            check((o.double().cpu(), lse.double().cpu()),
                  reference(dense, n_q, q.double().cpu(), H, G, True, 128.0 ** -0.5))
        own = [a + n for a, n in zip(own, n_q)]
    assert int(err.item()) == 0
    for layer in range(layers):
        for b in range(2):
            kk, vv = held(layer, b, own[b])
            for pos in range(kk.shape[0]):
                k, v, big = (t.cpu() for t in given[layer, b, pos])
                assert ((kk[pos] - k).abs() <= k.abs() * 2.0 ** -8 + 6 * 2.0 ** -24 * big).all()
                assert ((vv[pos] - v).abs() <= 2.0 ** -25).all()
