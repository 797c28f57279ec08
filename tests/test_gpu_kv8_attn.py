"""Attention over the 8-bit pool on the GPU, against fp64."""

import pytest
import torch

import serving_prefill_b200 as sp
from kv8_support import AttnCase, check, reference

pytestmark = pytest.mark.gpu

# (KV heads, query heads a KV head, [(chunk lengths, query tokens)])
PROMPTS = {
    "one_page": (2, 4, [([16], 16)]),
    "ragged": (2, 4, [([100, 33, 1, 15, 17], 10), ([250], 33), ([16, 16, 5], 1)]),
    "two_q_tiles": (1, 4, [([300, 70], 61)]),
    "three_blocks": (2, 8, [([700], 100), ([40, 41], 80)]),
    "mha": (4, 1, [([130, 20], 140), ([7], 3)]),
    "mqa": (1, 32, [([200, 9], 11)]),
    "group_3": (2, 3, [([90, 90], 50), ([33], 20)]),
    "group_5": (1, 5, [([90, 64], 60)]),
    "group_7": (2, 7, [([333], 40), ([20], 19)]),
    "group_128": (1, 128, [([60, 7], 5)]),
    "group_100": (1, 100, [([60, 7], 3)]),
    "long_split": (2, 4, [([1000] * 5, 70)]),
    "many_chunks": (1, 4, [([3 + i % 5 for i in range(90)], 30), ([1], 1)]),
    "self_prompt": (2, 2, [([500], 500)]),
    "more_queries_than_keys": (2, 4, [([5], 40), ([], 7), ([64], 64), ([1], 1)]),
    "no_queries": (2, 4, [([50], 0), ([60], 30), ([], 0)]),
}
SINGLE = {
    "one_token": (8, 4, [([100], 1)]),
    "one_key": (2, 4, [([1], 1)]),
    "step": (8, 4, [([300, 77, 12], 1), ([16], 1), ([900, 1], 1), ([33] * 7, 1)]),
    "mha_step": (32, 1, [([200, 31], 1), ([50], 1)]),
    "group_16": (2, 16, [([500, 10], 1), ([129], 1)]),
    "group_3": (2, 3, [([300, 11], 1), ([128], 1)]),
    "group_7": (4, 7, [([150, 150], 2), ([16], 1)]),
    "four_tokens": (2, 4, [([200, 90], 4), ([3], 2), ([600], 3)]),
    "five_of_three": (1, 3, [([140], 5), ([2], 5)]),
    "sixteen_of_one": (4, 1, [([300, 300], 16), ([10], 16)]),
    "empty_requests": (2, 4, [([], 1), ([40], 1), ([], 2), ([40], 0)]),
    "many_chunks": (2, 4, [([1 + i % 19 for i in range(130)], 1)]),
    "long": (2, 4, [([1024] * 12, 1)]),
}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", list(PROMPTS))
def test_prompts(name, causal):
    case = AttnCase(*PROMPTS[name], seed=len(name))
    check(case.run(causal), case.reference(causal))
    assert sp.rag_last_device_error(case.ws) == (0, 0)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", list(SINGLE))
def test_short_query_blocks(name, causal):
    case = AttnCase(*SINGLE[name], seed=len(name))
    check(case.run(causal), case.reference(causal))
    assert sp.rag_last_device_error(case.ws) == (0, 0)


@pytest.mark.parametrize("seed", [0, 1])
def test_many_items_a_block_of_every_kind(seed):
    """More work items than SMs, one- and two-tile query blocks and single
    tokens mixed, so that a block walks items of every kind in turn."""
    import random
    r = random.Random(seed)
    reqs = [([r.randint(1, 400) for _ in range(r.randint(1, 5))], r.choice([1, 2, 20, 33, 60, 64, 70, 100, 129]))
            for _ in range(24)]
    case = AttnCase(8, 4, reqs, seed=seed)
    check(case.run(True), case.reference(True))
    assert sp.rag_last_device_error(case.ws) == (0, 0)


PAGE_OOB, GEOMETRY, RANGE = 3, 8, 9
SHORT = [([300, 77, 12], 1), ([500, 33], 2), ([90], 1), ([260, 16], 4)]
LONG = [([300, 77, 12], 40), ([500, 33], 70), ([90], 9), ([260, 16], 33)]


def others(case, got, want, skip):
    """Every request but `skip` is as the reference has it."""
    q0 = 0
    for b, (_, nq) in enumerate(case.reqs):
        if b != skip and nq:
            check([x[q0:q0 + nq] for x in got], [x[q0:q0 + nq] for x in want])
        q0 += nq


@pytest.mark.parametrize("reqs", [SHORT, LONG], ids=["short", "long"])
def test_a_page_outside_the_pool_is_masked_and_reported(reqs):
    case = AttnCase(2, 4, reqs, seed=1)
    want = case.reference()
    ids = list(case.arrays[3])
    ids[2], ids[-1] = case.kc.shape[1] + 7, -3
    case.batch = sp.Batch(*case.arrays[:3], ids, case.arrays[4])
    got = case.run()
    assert sp.rag_last_device_error(case.ws) == (PAGE_OOB, 1)
    assert torch.isfinite(got[0]).all()
    q0 = 0
    for b, (_, nq) in enumerate(case.reqs):
        if b in (1, 2):
            check([x[q0:q0 + nq] for x in got], [x[q0:q0 + nq] for x in want])
        q0 += nq
    assert sp.rag_last_device_error(case.ws) == (0, 0)      # read and cleared


@pytest.mark.parametrize("reqs", [SHORT, LONG], ids=["short", "long"])
@pytest.mark.parametrize("extra", [1, -1])
def test_a_chunk_with_a_page_too_many_or_too_few_is_reported(reqs, extra):
    case = AttnCase(2, 4, reqs, seed=2)
    want = case.reference()
    rc, cd, cp, ids, qo = [list(x) for x in case.arrays]
    c = 3                                                    # request 1's first chunk
    ids = ids[:cp[c + 1]] + [ids[-1]] + ids[cp[c + 1]:] if extra > 0 else ids[:cp[c + 1] - 1] + ids[cp[c + 1]:]
    cp = cp[:c + 1] + [x + extra for x in cp[c + 1:]]
    case.batch = sp.Batch(rc, cd, cp, ids, qo)
    if extra < 0:                                            # keep the host's maxima: the device has to find it
        case.batch.c.max_pages = max(case.batch.c.max_pages, -(-max(case.batch.doc_lens) // 16))
        case.batch.c.num_page_refs = max(case.batch.c.num_page_refs, case.batch.c.max_pages)
    case.ws = sp.new_workspace(case.pool, case.batch, 8)
    got = case.run()
    st, bits = sp.rag_last_device_error(case.ws)
    assert st == GEOMETRY and bits == 2
    others(case, got, want, skip=1 if extra < 0 else -1)     # a page too many holds no token: still exact


@pytest.mark.parametrize("reqs", [SHORT, LONG], ids=["short", "long"])
def test_a_scale_that_is_none_is_reported(reqs):
    for bad, which in ((float("nan"), "k"), (0.0, "v"), (-1.0, "k"), (float("inf"), "v"), (256.0, "v")):
        case = AttnCase(2, 4, reqs, seed=3)
        want = case.reference()
        scale = case.pool.k_scale if which == "k" else case.pool.v_scale
        scale[1, case.pages[0][0], 1] = bad                  # request 0's first page
        got = case.run()
        assert sp.rag_last_device_error(case.ws) == (RANGE, 8)
        assert torch.isfinite(got[0]).all()
        others(case, got, want, skip=0)


@pytest.mark.parametrize("reqs", [SHORT, LONG], ids=["short", "long"])
def test_rows_of_nan_and_infinite_queries_stay_their_own(reqs):
    case = AttnCase(2, 4, reqs, seed=4)
    want = case.reference()
    case.q[2, 3, 17] = float("nan")
    case.q[0, 5, 0] = float("inf")
    o, lse = case.run()
    hit = torch.zeros(case.total_q, 8, dtype=torch.bool)
    hit[2, 3] = hit[0, 5] = True
    assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
    O, L, bo, bl = want
    assert ((o - O).abs() <= bo)[~hit].all() and ((lse - L).abs() <= bl)[~hit].all()


@pytest.mark.parametrize("reqs", [SHORT, LONG], ids=["short", "long"])
def test_extreme_magnitudes(reqs):
    """A peaked softmax (scores in the thousands), a flat one, tiny and huge
    scales, and queries that span e4m3's whole range within a row."""
    for q_scale, exps in ((30.0, (-4, -1)), (1e-4, (-9, -4)), (1.0, (-24, -20)), (1.0, (-20, 3))):
        case = AttnCase(2, 4, reqs, seed=5, q_scale=q_scale, scale_exp=exps)
        case.q[:, :, ::7] *= 2.0 ** -9
        check(case.run(), case.reference())
        assert sp.rag_last_device_error(case.ws) == (0, 0)


@pytest.mark.parametrize("reqs", [SHORT, LONG], ids=["short", "long"])
def test_keys_that_grow_along_the_sequence_rescale_the_sums(reqs):
    """Each page's scale twice that of the one two before it: the running
    maximum jumps again and again, past every lazy threshold."""
    case = AttnCase(2, 4, reqs, seed=6)
    for c, pg in enumerate(case.pages):
        for i, x in enumerate(pg):
            case.ks[:, x] = 2.0 ** (-12 + min(i // 2, 9))
    case.pool.k_scale.copy_(torch.nan_to_num(case.ks, nan=1.0))
    check(case.run(), case.reference())


@pytest.mark.parametrize("reqs", [SHORT, LONG], ids=["short", "long"])
def test_own_scale_padding_rows_and_another_stream(reqs):
    case = AttnCase(2, 4, reqs, seed=7, pad_rows=3)
    want = case.reference(scale=0.03)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    check(case.run(sm_scale=0.03, stream=stream), want)
    assert (case.o[case.total_q:] == 7.0).all() and (case.lse[case.total_q:] == 7.0).all()


@pytest.mark.parametrize("reqs", [SHORT, LONG], ids=["short", "long"])
def test_repeated_chunks_and_page_placement(reqs):
    """A request that lists a chunk's pages twice, and shared pages between
    requests; the output does not depend on where pages lie."""
    case = AttnCase(2, 4, [(c + [c[0]], q) for c, q in reqs], seed=8, repeat=[(3, 0)])
    check(case.run(), case.reference())
    a, b = (AttnCase(2, 4, reqs, seed=9) for _ in range(2))
    perm = torch.randperm(b.kc.shape[1])
    inv = torch.argsort(perm)
    b.pool = sp.KV8Pool(2, b.kc.shape[1], 2, k=b.kc[:, perm].contiguous().view(torch.float8_e4m3fn).cuda(),
                        v=b.vc[:, perm].contiguous().view(torch.float8_e4m3fn).cuda(),
                        k_scale=b.ks[:, perm].contiguous().cuda(), v_scale=b.vs[:, perm].contiguous().cuda())
    b.batch = sp.Batch(*b.arrays[:3], [int(inv[i]) for i in b.arrays[3]], b.arrays[4])
    x, y = a.run(), b.run()
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


@pytest.mark.parametrize("reqs", [SHORT, LONG], ids=["short", "long"])
def test_the_same_call_gives_the_same_bits(reqs):
    case = AttnCase(8, 4, reqs * 5, seed=10)
    first = [x.clone() for x in case.run()]
    for _ in range(5):
        again = case.run()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("n_q", [1, 40])
def test_captured_call_follows_the_batch_within_its_capacities(n_q):
    """One captured call, its batch's device arrays rewritten between replays:
    lengths grow from nothing to the capacities, requests come and go."""
    reqs = [([400, 300], n_q), ([900], n_q), ([50, 20, 700], n_q)]
    case = AttnCase(2, 4, reqs, seed=11)
    case.run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sp.rag_kv8_attn(case.pool, 1, case.batch, case.q, case.o, case.ws, row_lse=case.lse)
    full = [list(x) for x in case.arrays]
    dense = case.dense()
    for frac in (0.0, 0.03, 0.4, 1.0):
        doc, page, ids = [0], [0], []
        keep = []
        for c, n in enumerate(case.lens):
            m = int(n * frac)
            keep.append(m)
            doc.append(doc[-1] + m)
            page.append(page[-1] + -(-m // 16))
            ids += case.pages[c][: -(-m // 16)]
        for t, x in zip(case.batch.dev, (full[0], doc, page, ids, full[4])):
            t[: len(x)] = torch.tensor(x, dtype=torch.int32)
        g.replay()
        torch.cuda.synchronize()
        part, c = [], 0
        for (k, v), (chunks, _) in zip(dense, reqs):
            rows, at = [], 0
            for n in chunks:
                rows += list(range(at, at + keep[c]))
                at += n
                c += 1
            part.append((k[rows], v[rows]))
        want = reference(part, [n_q] * 3, case.q.double().cpu(), 2, 4, True, 128.0 ** -0.5)
        check((case.o.double().cpu(), case.lse.double().cpu()), want)
    assert sp.rag_last_device_error(case.ws) == (0, 0)


def test_two_calls_at_once_with_a_workspace_each():
    a, b = AttnCase(8, 4, SHORT * 8, seed=12), AttnCase(4, 8, LONG * 3, seed=13)
    want = a.reference(), b.reference()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        sp.rag_kv8_attn(a.pool, 1, a.batch, a.q, a.o, a.ws, row_lse=a.lse, stream=s1)
        sp.rag_kv8_attn(b.pool, 1, b.batch, b.q, b.o, b.ws, row_lse=b.lse, stream=s2)
    torch.cuda.synchronize()
    check((a.o.double().cpu(), a.lse.double().cpu()), want[0])
    check((b.o.double().cpu(), b.lse.double().cpu()), want[1])


def test_calls_that_follow_one_another_on_one_workspace():
    """Calls back to back on one stream and one workspace (overlapping launches),
    each reading the output of the one before as its queries."""
    case = AttnCase(2, 4, LONG, seed=14)
    q1 = case.q.clone()
    o1 = case.run()[0]
    case.q.copy_(o1.to(torch.bfloat16))
    want = case.reference()
    case.q.copy_(q1)
    o2 = torch.empty_like(case.o)
    torch.cuda.synchronize()
    for _ in range(20):
        sp.rag_kv8_attn(case.pool, 1, case.batch, q1, case.o, case.ws)
        sp.rag_kv8_attn(case.pool, 1, case.batch, case.o, o2, case.ws, row_lse=case.lse)
    torch.cuda.synchronize()
    check((o2.double().cpu(), case.lse.double().cpu()), want)


def test_four_thousand_requests():
    reqs = [([1 + i % 37], 1 + (i % 3 == 0)) for i in range(4096)]
    case = AttnCase(1, 2, reqs, seed=15)
    check(case.run(), case.reference())
    case = AttnCase(1, 2, [(c, 9 * q) for c, q in reqs[:900]] , seed=15)
    check(case.run(), case.reference())
    assert sp.rag_last_device_error(case.ws) == (0, 0)


def test_pool_offsets_past_32_bits():
    H, P = 8, (1 << 31) // (8 * 16 * 128) + 64
    pool = sp.KV8Pool(1, P, H)
    x = torch.randn(40, H, 128, device="cuda").to(torch.bfloat16)
    pages = [P - 1, P - 3, P - 2]
    sp.rag_kv8_append(pool, 0, sp.Append([0, 40], [0], [0, 3], pages), x, x)
    q = torch.randn(40, 4 * H, 128, device="cuda").to(torch.bfloat16)
    k = (pool.k[0][pages].double() * pool.k_scale[0][pages].double()[..., None, None]).permute(0, 2, 1, 3)
    v = (pool.v[0][pages].double() * pool.v_scale[0][pages].double()[..., None, None]).permute(0, 2, 1, 3)
    dense = [(k.reshape(-1, H, 128)[:40].cpu(), v.reshape(-1, H, 128)[:40].cpu())]
    for n in (1, 40):
        b = sp.Batch([0, 1], [0, 40], [0, 3], pages, [0, n])
        o, lse = torch.empty_like(q[:n]), torch.empty(n, 4 * H, device="cuda")
        sp.rag_kv8_attn(pool, 0, b, q[:n].contiguous(), o, sp.new_workspace(pool, b, 4 * H), row_lse=lse)
        check((o.double().cpu(), lse.double().cpu()),
              reference(dense, [n], q[:n].double().cpu(), H, 4, True, 128.0 ** -0.5))


def test_prompt_then_generation():
    """The operators together as a server uses them: retrieved chunks and the
    prompt appended to an 8-bit pool with their rotation, the prompt attended,
    then 20 tokens, each appended to its request's last page and attended, all
    in one captured step whose arrays advance on the device. Every output is
    held to fp64 attention over what the pool holds, and the pool to the keys
    and values it was given."""
    H, G, layers = 2, 4, 2
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    chunks, prompt, steps = [[90, 40], [33]], [21, 7], 20
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
    pool = sp.KV8Pool(layers, total + 2, H)
    rope = sp.rag_rope_cos_sin(10000.0, 128, 512)
    given = {}                                   # (request, position) -> (k rotated, v) per layer, fp64

    def add(layer, seqs, k, v, where, **kw):
        sp.rag_kv8_append(pool, layer, seqs, k, v, rope=rope, **kw)
        for r, (b, pos) in enumerate(where):
            x, cs = k[r].double(), rope[pos].double()
            a, c = x[:, :64], x[:, 64:]
            given[layer, b, pos] = (torch.cat([a * cs[:, 0] - c * cs[:, 1], c * cs[:, 0] + a * cs[:, 1]], -1),
                                    v[r].double())

    for layer in range(layers):                  # the chunks, at their positions in the concatenation
        for b, cs in enumerate(chunks):
            pos = 0
            for c, n in enumerate(cs):
                add(layer, sp.Append([0, n], [0], [0, len(pages[b][c])], pages[b][c], pos0=[pos]), rnd(n, H, 128),
                    rnd(n, H, 128), [(b, pos + i) for i in range(n)])
                pos += n

    def held(layer, lens):
        out = []
        for b in range(2):
            ks, vs = [], []
            for pg, n in zip(pages[b], chunks[b] + [lens[b]]):
                for dst, x, s in ((ks, pool.k, pool.k_scale), (vs, pool.v, pool.v_scale)):
                    y = x[layer][pg].double() * s[layer][pg].double()[..., None, None]
                    dst.append(y.permute(0, 2, 1, 3).reshape(-1, H, 128)[:n])
            out.append((torch.cat(ks).cpu(), torch.cat(vs).cpu()))
        return out

    ctx_pages = [pages[b][-1] for b in range(2)]
    page_off = [0, len(ctx_pages[0]), len(ctx_pages[0]) + len(ctx_pages[1])]
    flat_ids = [x for row in pages for p in row for x in p]

    def arrays(lens):
        doc, page = [0], [0]
        for b in range(2):
            for n, p in zip(chunks[b] + [lens[b]], pages[b]):
                doc.append(doc[-1] + n)
                page.append(page[-1] + -(-n // 16))
        ids = [x for b in range(2) for n, p in zip(chunks[b] + [lens[b]], pages[b]) for x in p[: -(-n // 16)]]
        return doc, page, ids

    # the prompts
    T = sum(prompt)
    doc, page, ids_now = arrays(prompt)
    b0 = sp.Batch([0, 3, 5], doc, page, ids_now, [0, prompt[0], T])
    seqs = sp.Append([0, prompt[0], T], [0, 0], page_off, ctx_pages[0] + ctx_pages[1], pos0=docs)
    ws = sp.new_workspace(pool, b0, H * G)
    q, qr, o = rnd(T, H * G, 128), torch.empty(T, H * G, 128, dtype=torch.bfloat16, device="cuda"), None
    for layer in range(layers):
        where = [(b, docs[b] + i) for b in range(2) for i in range(prompt[b])]
        add(layer, seqs, rnd(T, H, 128), rnd(T, H, 128), where, q=q, q_out=qr)
        o, lse = torch.empty_like(qr), torch.empty(T, H * G, device="cuda")
        sp.rag_kv8_attn(pool, layer, b0, qr, o, ws, row_lse=lse)
        check((o.double().cpu(), lse.double().cpu()),
              reference(held(layer, prompt), prompt, qr.double().cpu(), H, G, True, 128.0 ** -0.5))
    assert sp.rag_last_device_error(ws) == (0, 0)

    # the generation: capacities of the last step, arrays of the current one
    doc, page, ids_now = arrays([p + steps for p in prompt])
    b1 = sp.Batch([0, 3, 5], doc, page, ids_now, [0, 1, 2])
    ws = sp.new_workspace(pool, b1, H * G)
    start = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    one = sp.Append([0, 1, 2], start, page_off, ctx_pages[0] + ctx_pages[1], pos0=docs)
    k, v, q = rnd(2, H, 128), rnd(2, H, 128), rnd(2, H * G, 128)
    qr, o = torch.empty_like(q), [torch.empty_like(q) for _ in range(layers)]
    lse = [torch.empty(2, H * G, device="cuda") for _ in range(layers)]

    def step():
        for layer in range(layers):
            sp.rag_kv8_append(pool, layer, one, k, v, rope=rope, q=q, q_out=qr)
            sp.rag_kv8_attn(pool, layer, b1, qr, o[layer], ws, row_lse=lse[layer])

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        k.copy_(rnd(2, H, 128) * (1 + i))        # magnitudes that make the pages' scales grow
        v.copy_(rnd(2, H, 128) * (1 + i))
        q.copy_(rnd(2, H * G, 128))
        lens = [p + i + 1 for p in prompt]
        doc, page, ids_now = arrays(lens)
        for t, x in zip(b1.dev, ([0, 3, 5], doc, page, ids_now, [0, 1, 2])):
            t[: len(x)] = torch.tensor(x, dtype=torch.int32)
        graph.replay()
        torch.cuda.synchronize()
        for layer in range(layers):
            for b in range(2):
                pos = docs[b] + prompt[b] + i
                cs = rope[pos].double()
                a, c = k[b].double()[:, :64], k[b].double()[:, 64:]
                given[layer, b, pos] = (torch.cat([a * cs[:, 0] - c * cs[:, 1], c * cs[:, 0] + a * cs[:, 1]], -1),
                                        v[b].double())
            want = reference(held(layer, lens), [1, 1], qr.double().cpu(), H, G, True, 128.0 ** -0.5)
            check((o[layer].double().cpu(), lse[layer].double().cpu()), want)
        start += 1
    assert sp.rag_last_device_error(ws) == (0, 0)
    # what the pool holds in the end: e4m3's half step of the value, twice (a
    # held code is rounded again, by an exact factor, only below the normal
    # range), plus its smallest step under the page's final scale
    for layer in range(layers):
        for b, (kk, vv) in enumerate(held(layer, [p + steps for p in prompt])):
            n = kk.shape[0]
            for i, (got, scale) in enumerate(((kk, pool.k_scale), (vv, pool.v_scale))):
                ref = torch.stack([given[layer, b, pos][i] for pos in range(n)]).cpu()
                top = float(scale[layer].max())
                assert ((got - ref).abs() <= ref.abs() / 16 + top * 2.0 ** -8).all()
