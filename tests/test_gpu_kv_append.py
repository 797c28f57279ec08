"""Append to paged caches on the GPU, against the fp64 oracle and, bit for bit,
against the same formula in fp32 (numpy)."""

import numpy as np
import pytest
import torch

import serving_prefill_b200 as sp
from oracle import append as oa

pytestmark = pytest.mark.gpu

D = {"bf16": 128, "e4m3": 128, "f32": 128, "f32_64": 64}


def table_np(dim, n_pos, base=10000.0):
    ang = np.arange(n_pos)[:, None] * base ** (-2.0 * np.arange(dim // 2) / dim)
    return np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32)


class Case:
    """Sequences (pages, start, n_new, pos0) on a pool whose pages start with
    arbitrary finite contents (and, past each sequence's held tokens, garbage
    that an earlier owner left)."""

    def __init__(self, kind, starts, news, H=2, G=3, fused=False, pad=0, seed=0, n_pos=4096, scale=1.0, rope=True):
        self.kind, self.H, self.d = kind, H, D[kind]
        self.dt = torch.float32 if kind.startswith("f32") else torch.bfloat16
        g = torch.Generator().manual_seed(seed)
        counts = [-(-(s + n) // 16) for s, n in zip(starts, news)]
        P = sum(counts) + 2
        perm = torch.randperm(P, generator=g).tolist()
        self.seqs, at = [], 0
        for i, (s, n, c) in enumerate(zip(starts, news, counts)):
            self.seqs.append((perm[at:at + c], s, n, 37 * i))
            at += c
        T = sum(news)
        rnd = lambda *sh: torch.randn(*sh, generator=g)  # noqa: E731
        x = (rnd(T + pad, H * (G + 2), self.d) * scale).to(self.dt)
        q, k, v = x[:, :H * G], x[:, H * G:H * G + H], x[:, H * G + H:]
        if not fused:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
            xs = [q.cuda(), k.cuda(), v.cuda()]
        else:
            xd = x.cuda()
            xs = [xd[:, :H * G], xd[:, H * G:H * G + H], xd[:, H * G + H:]]
        self.q, self.k, self.v = xs
        self.host = [t[:T].double().numpy() for t in (q, k, v)]
        self.table = table_np(self.d, n_pos) if rope else None
        self.rope = torch.from_numpy(self.table).cuda() if rope else None
        self.T, self.G, self.P = T, G, P
        shape = (2, P, H, 16, self.d)
        if kind == "e4m3":
            codes = torch.randint(0, 127, shape, generator=g).to(torch.uint8)
            codes2 = torch.randint(128, 255, shape, generator=g).to(torch.uint8)
            exps = torch.randint(-9, -5, shape[:3], generator=g)
            self.pool = sp.KV8Pool(2, P, H, k=codes.view(torch.float8_e4m3fn).cuda(),
                                   v=codes2.view(torch.float8_e4m3fn).cuda(), k_scale=torch.exp2(exps.float()).cuda(),
                                   v_scale=torch.exp2((exps - 1).float()).cuda())
        else:
            vdt = torch.float16 if kind == "bf16" else torch.float32
            self.pool = sp.KVPool(2, P, H, self.d, dtype=self.dt, k=rnd(*shape).to(self.dt).cuda(),
                                  v=rnd(*shape).to(vdt).cuda())
        self.arrays = (np.cumsum([0] + list(news)).tolist(), list(starts), np.cumsum([0] + counts).tolist(),
                       [p for s in self.seqs for p in s[0]], [s[3] for s in self.seqs])
        self.append_c = sp.Append(*self.arrays[:4], pos0=self.arrays[4], total_new=T + pad)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.q_out = torch.full((T + pad, H * G, self.d), 7.0, dtype=self.dt, device="cuda")

    def state(self):
        p = self.pool
        s = [p.k[1].double().cpu().numpy(), p.v[1].double().cpu().numpy()]
        return s + ([p.k_scale[1].double().cpu().numpy(), p.v_scale[1].double().cpu().numpy()]
                    if self.kind == "e4m3" else [None, None])

    def run(self, **kw):
        fn = sp.rag_kv8_append if self.kind == "e4m3" else sp.rag_kv_append
        args = dict(rope=self.rope, q=self.q, q_out=self.q_out, device_err=self.err)
        args.update(kw)
        fn(self.pool, 1, self.append_c, self.k, self.v, **args)
        torch.cuda.synchronize()

    def oracle(self, before):
        want = [None if x is None else x.copy() for x in before]
        _, k, v = self.host
        tab = None if self.table is None else self.table.astype(np.float64)
        oa.append(want[0], want[1], want[2], want[3], self.seqs, k, v, tab)
        return want

    def positions(self):
        return np.concatenate([[p0 + s + i for i in range(n)] for _, s, n, p0 in self.seqs if n] or [[]]).astype(int)


def half_step(kind, is_v):
    """(relative half step, absolute half step of the subnormals) of the stored type."""
    if kind == "e4m3":
        return 2.0 ** -4, 2.0 ** -10
    if kind == "bf16":
        return (2.0 ** -11, 2.0 ** -25) if is_v else (2.0 ** -8, 0.0)
    return 2.0 ** -24, 0.0


def check(case, before, after, want):
    """Stored values within one half step of the 64-bit ones, plus the fp32
    rounding of the rotation: each of a c and b s, and their sum, is off by at
    most 2^-24 of its magnitude, together at most 3 * 2^-24 * (|a| + |b|) with
    |a|, |b| <= the largest input magnitude."""
    big = max(np.abs(case.host[1]).max(initial=0), 1e-30)
    rel, sub = half_step(case.kind, False)
    turn = 3 * 2.0 ** -24 * 2 * big if case.table is not None else 0.0
    for name, i, is_v in (("k", 0, False), ("v", 1, True)):
        rel, sub = half_step(case.kind, is_v)
        got, ref = after[i], want[i]
        extra = 0.0 if is_v else turn
        if case.kind == "e4m3":
            gs, ws = after[2 + i], want[2 + i]
            # a scale may differ only where the 64-bit and the fp32 maximum lie on either side of a border
            edge = gs != ws
            assert edge.sum() == 0 or not is_v
            got, ref = got * gs[..., None, None], ref * ws[..., None, None]
            tol = rel * np.abs(ref) + sub * np.maximum(gs, ws)[..., None, None] + extra
            tol = np.where(edge[..., None, None], 2 * tol, tol)
        else:
            tol = rel * np.abs(ref) + sub + extra
        err = np.abs(got - ref)
        assert (err <= tol).all(), (name, np.argwhere(err > tol)[:4].tolist(), (err / np.maximum(tol, 1e-300)).max())
        # slots that no new token owns, and that no begun page zeroes, keep their bits
        touched = np.zeros(got.shape[:1] + got.shape[2:3], bool)
        for pages, s, n, _ in case.seqs:
            for t in range(s, s + n):
                touched[pages[t // 16], t % 16] = True
        keep = ~touched
        if case.kind != "e4m3":
            ref_keep = want[i].transpose(0, 2, 1, 3)[keep]
            np.testing.assert_array_equal(after[i].transpose(0, 2, 1, 3)[keep], ref_keep)


def check_q(case):
    got = case.q_out[:case.T].double().cpu().numpy()
    q, pos = case.host[0], case.positions()
    want = q if case.table is None else np.stack([oa.rotate(q[t], case.table[pos[t]].astype(np.float64))
                                                 for t in range(case.T)])
    rel = 2.0 ** -8 if case.dt == torch.bfloat16 else 2.0 ** -24
    tol = rel * np.abs(want) + 6 * 2.0 ** -24 * np.abs(q).max()
    assert (np.abs(got - want) <= tol).all()
    assert (case.q_out[case.T:] == 7.0).all()      # padding rows are left as they were


STARTS_NEWS = [
    ([0], [1]),
    ([5], [1]),
    ([15, 16, 0], [1, 1, 16]),
    ([0, 3, 31, 16, 7], [33, 0, 17, 1, 9]),
    ([0, 0, 1], [128, 15, 300]),
]


@pytest.mark.parametrize("fused,pad", [(False, 0), (True, 3)])
@pytest.mark.parametrize("starts,news", STARTS_NEWS)
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32", "f32_64"])
def test_append_matches_the_oracle(kind, starts, news, fused, pad):
    case = Case(kind, starts, news, fused=fused, pad=pad, seed=len(news))
    before = case.state()
    layer0 = [case.pool.k[0].clone(), case.pool.v[0].clone()]
    case.run()
    check(case, before, case.state(), case.oracle(before))
    check_q(case)
    assert int(case.err.item()) == 0
    assert torch.equal(case.pool.k[0].view(torch.uint8), layer0[0].view(torch.uint8))   # another layer's pages
    assert torch.equal(case.pool.v[0].view(torch.uint8), layer0[1].view(torch.uint8))


@pytest.mark.parametrize("H,G", [(1, 1), (8, 4), (3, 5), (32, 1), (4, 0)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_head_layouts_without_rotation(kind, H, G):
    case = Case(kind, [2, 0], [20, 5], H=H, G=max(G, 1), rope=False, seed=H)
    before = case.state()
    case.run(**({"q": None, "q_out": None} if G == 0 else {}))
    check(case, before, case.state(), case.oracle(before))
    if G:
        check_q(case)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32", "f32_64"])
def test_bits_are_the_fp32_formulas(kind):
    """Rotation in fp32 with each product and sum rounded, one rounding to the
    stored type: the same bits from numpy's fp32."""
    case = Case(kind, [0, 9], [400, 300], seed=3)
    before = case.state()
    case.run()
    after = case.state()
    q, k, v = case.host
    pos = case.positions()
    if kind.startswith("f32"):
        q32 = np.stack([oa.rotate(q[t].astype(np.float32), case.table[pos[t]]) for t in range(case.T)])
        np.testing.assert_array_equal(case.q_out[:case.T].cpu().numpy(), q32)
    k32 = np.stack([oa.rotate(k[t].astype(np.float32), case.table[pos[t]]) for t in range(case.T)])
    assert k32.dtype == np.float32
    want = [None if x is None else x.copy() for x in before]
    oa.append(want[0], want[1], want[2], want[3], case.seqs, k32.astype(np.float64), v, None)
    if kind == "e4m3":
        np.testing.assert_array_equal(after[2], want[2])
        np.testing.assert_array_equal(after[3], want[3])
        np.testing.assert_array_equal(after[0], oa.to_e4m3(want[0]))
        np.testing.assert_array_equal(after[1], oa.to_e4m3(want[1]))
    else:
        np.testing.assert_array_equal(after[0], torch.from_numpy(want[0]).float().to(case.dt).double().numpy())


def test_scale_grows_token_by_token_and_held_codes_follow():
    """32 tokens appended one at a time with magnitudes that double every two
    tokens and then fall: the scale follows the largest, held codes are rounded
    again by exact powers of two, so a value that stays within e4m3's normal
    range keeps its code's value."""
    case = Case("e4m3", [0], [32], H=2, G=1, rope=False)
    mag = torch.tensor([2.0 ** min(i // 2, 6) if i < 24 else 0.01 for i in range(32)])
    k = (case.k * mag[:, None, None].cuda().to(case.k.dtype)).contiguous()
    v = (case.v * mag[:, None, None].cuda().to(case.v.dtype)).contiguous()
    want = case.state()
    pages = case.seqs[0][0]
    for i in range(32):
        s = sp.Append([0, 1], [i], [0, 2], pages)
        sp.rag_kv8_append(case.pool, 1, s, k[i:i + 1], v[i:i + 1])
        kk, vv = k[i:i + 1].double().cpu().numpy(), v[i:i + 1].double().cpu().numpy()
        oa.append(want[0], want[1], want[2], want[3], [(pages, i, 1, 0)], kk, vv, None)
        want[0], want[1] = oa.to_e4m3(want[0]), oa.to_e4m3(want[1])
    got = case.state()
    for a, b in zip(got, want):
        np.testing.assert_array_equal(a, b)


def test_a_begun_page_keeps_nothing_of_its_earlier_owner():
    """Pages full of nan codes and of nan values: after a write of slot 0 every
    slot behind the new tokens is zero."""
    for kind in ("bf16", "e4m3", "f32"):
        case = Case(kind, [0, 16], [5, 3], seed=9)
        if kind == "e4m3":
            case.pool.k.view(torch.uint8).fill_(0x7F)
            case.pool.v.view(torch.uint8).fill_(0xFF)
            case.pool.k_scale.fill_(float("nan"))
        else:
            case.pool.k.fill_(float("nan"))
            case.pool.v.fill_(float("nan"))
        case.run()
        for pool in (case.pool.k, case.pool.v):
            x = pool[1].float()
            assert not x[case.seqs[0][0][0], :, 5:].any() and torch.isfinite(x[case.seqs[0][0][0]]).all()
            assert not x[case.seqs[1][0][1], :, 3:].any()
            assert torch.isnan(x[case.seqs[1][0][0]]).all()        # a page of the sequence the call does not touch
        assert int(case.err.item()) == 0


def test_infinities_and_nan():
    case = Case("e4m3", [0, 4], [20, 2], rope=False, seed=4)
    k, v = case.k, case.v
    k[3, 0, 7], k[5, 1, 0], v[2, 0, 1], v[2, 1, 5], v[20, 0, 3] = (float("inf"), float("nan"), float("-inf"),
                                                                   float("nan"), 60000.0)
    case.run()
    x = [(p[1].float() * s[1][..., None, None]).cpu() for p, s in ((case.pool.k, case.pool.k_scale),
                                                                  (case.pool.v, case.pool.v_scale))]
    p0 = case.seqs[0][0][0]
    sc = case.pool.k_scale[1].cpu(), case.pool.v_scale[1].cpu()
    assert x[0][p0, 0, 3, 7] == 448 * sc[0][p0, 0] and x[0][p0, 1, 5, 0] == 0
    assert x[1][p0, 0, 2, 1] == -448 * sc[1][p0, 0] and x[1][p0, 1, 2, 5] == 0
    assert sc[0][p0].max() < 1 and sc[1][p0].max() < 1          # the scale follows the finite values
    p1 = case.seqs[1][0][0]
    assert sc[1][p1, 0] == 128 and x[1][p1, 0, 4, 3] == 57344
    assert int(case.err.item()) == 8
    # a 16-bit pool keeps K's bits and saturates V, as its pool write does
    case = Case("bf16", [0], [4], rope=False)
    case.k[1, 0, 0], case.v[1, 0, 0] = float("nan"), 70000.0
    case.run()
    p0 = case.seqs[0][0][0]
    assert torch.isnan(case.pool.k[1, p0, 0, 1, 0]) and case.pool.v[1, p0, 0, 1, 0] == 65504
    assert int(case.err.item()) == 8


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_bad_pages_and_positions_are_skipped_and_reported(kind):
    case = Case(kind, [0, 0, 0], [20, 20, 20], seed=5)
    tok, start, po, ids, pos0 = case.arrays
    ids = list(ids)
    ids[po[0]] = case.P + 3                                     # sequence 0, page 0: outside the pool
    case.append_c = sp.Append(tok, start, po, ids, pos0=[0, 4096 - 10, 5])
    before = case.state()
    case.run()
    after = case.state()
    assert int(case.err.item()) == 3
    case.seqs = [(case.seqs[0][0], 16, 4, 0), (case.seqs[1][0], 0, 20, 4086), (case.seqs[2][0], 0, 20, 5)]
    np.testing.assert_array_equal(after[0][case.seqs[0][0][0]], before[0][case.seqs[0][0][0]])
    # positions past the table: zeros in the cache and in q_out
    p = case.seqs[1][0]
    assert not after[0][p[0], :, 10:].any() and not after[1][p[0], :, 10:].any() and not after[0][p[1]].any()
    assert after[0][p[0], :, :10].any()
    assert not case.q_out[30:40].any() and case.q_out[20:30].any()
    # sequence 2 is as the oracle has it
    want = [None if x is None else x.copy() for x in before]
    oa.append(want[0], want[1], want[2], want[3], [case.seqs[2]], case.host[1][40:], case.host[2][40:],
              case.table.astype(np.float64))
    for pg in case.seqs[2][0]:
        for i in range(2):
            got, ref = after[i][pg], want[i][pg]
            assert np.abs(got - ref).max() <= (np.abs(ref).max() * 2.0 ** -4 + 1e-6)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("what", ["start", "pages", "order", "total"])
def test_inconsistent_descriptors_are_reported_and_write_nothing(kind, what):
    case = Case(kind, [0, 3], [20, 20], seed=6)
    tok, start, po, ids, pos0 = case.arrays
    total = 40
    if what == "start":
        start = [0, -1]
    elif what == "pages":
        po = [0, 2, 3]                                          # one page too few for sequence 1
    elif what == "order":
        tok = [0, 20, 10]
    else:
        tok = [0, 20, 400]                                      # past total_new
    case.append_c = sp.Append(tok, start, po, ids, pos0=pos0, total_new=total)
    before = case.state()
    case.run()
    after = case.state()
    assert int(case.err.item()) == 2 or what == "order"         # order: no token belongs to the sequence
    for pg in case.seqs[1][0]:
        np.testing.assert_array_equal(after[0][pg], before[0][pg])
        np.testing.assert_array_equal(after[1][pg], before[1][pg])


@pytest.mark.parametrize("kind,H,n", [("bf16", 2, 20), ("e4m3", 2, 20), ("e4m3", 32, 700)])
def test_rows_before_the_first_sequence_are_reported(kind, H, n):
    """tok_off that does not begin at 0: its rows belong to the sequence all the
    same, the 16 before them to none (their q_out rows become zeros)."""
    case = Case(kind, [40], [n], H=H, G=1, seed=16)
    tok, start, po, ids, pos0 = case.arrays
    before = case.state()
    case.run()
    want, q_want = case.state(), case.q_out.clone()
    other = Case(kind, [40], [n], H=H, G=1, seed=16)
    pad = lambda x: torch.cat([torch.full_like(x[:16], 3.0), x])  # noqa: E731
    other.k, other.v, other.q = pad(other.k), pad(other.v), pad(other.q)
    other.q_out = torch.full_like(other.q, 7.0)
    other.append_c = sp.Append([16, 16 + n], start, po, ids, pos0=pos0)
    other.run()
    for x, y in zip(other.state(), want):
        np.testing.assert_array_equal(x, y)
    assert torch.equal(other.q_out[16:], q_want) and not other.q_out[:16].any()
    assert int(other.err.item()) == 2 and int(case.err.item()) == 0
    np.testing.assert_array_equal(before[0][ids[0]], want[0][ids[0]])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_captured_steps_advance_on_the_device(kind):
    """One captured append of one token per sequence, replayed 20 times while
    the device arrays advance, equals 20 calls."""
    a, b = (Case(kind, [0, 13], [20, 20], seed=8) for _ in range(2))
    for i in range(20):
        rows = [i, 20 + i]
        s = sp.Append([0, 1, 2], [i, 13 + i], a.arrays[2], a.arrays[3], pos0=a.arrays[4])
        fn = sp.rag_kv8_append if kind == "e4m3" else sp.rag_kv_append
        fn(a.pool, 1, s, a.k[rows], a.v[rows], rope=a.rope)
    start = torch.tensor([0, 13], dtype=torch.int32, device="cuda")
    k, v = b.k[[0, 20]].clone(), b.v[[0, 20]].clone()
    s = sp.Append([0, 1, 2], start, b.arrays[2], b.arrays[3], pos0=b.arrays[4])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn(b.pool, 1, s, k, v, rope=b.rope)
    for i in range(20):
        k.copy_(b.k[[i, 20 + i]])
        v.copy_(b.v[[i, 20 + i]])
        g.replay()
        start += 1
    torch.cuda.synchronize()
    for x, y in zip(a.state(), b.state()):
        np.testing.assert_array_equal(x, y)


def test_query_rotated_in_place_on_another_stream():
    case = Case("bf16", [0], [50], seed=2)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    q = case.q.clone()
    torch.cuda.synchronize()
    case.run(q=q, q_out=q, stream=stream)
    case.q_out[:50] = q
    check_q(case)


def test_table_of_rotations():
    for base, dim in ((10000.0, 128), (500000.0, 128), (10000.0, 64)):
        t = sp.rag_rope_cos_sin(base, dim, 70000).double().cpu().numpy()
        pos = np.array([0, 1, 2, 17, 4095, 69999])
        ang = pos[:, None] * base ** (-2.0 * np.arange(dim // 2) / dim)
        want = np.stack([np.cos(ang), np.sin(ang)], -1)
        # fp64 on both sides: the angle is off by a few 2^-53 of its size, the result by fp32's half step
        assert np.abs(t[pos] - want).max() <= 2.0 ** -25 + 8 * 2.0 ** -53 * 70000
    assert sp.rag_rope_cos_sin(10000.0, 128, 0).shape == (0, 64, 2)


def test_offsets_past_32_bits():
    """A pool of more than 2^31 bytes a tensor: the last page's block is where it should be."""
    H, P = 8, (1 << 31) // (8 * 16 * 128) + 40
    pool = sp.KV8Pool(1, P, H)
    k = torch.randn(20, H, 128, device="cuda").to(torch.bfloat16)
    s = sp.Append([0, 20], [0], [0, 2], [P - 1, P - 2])
    sp.rag_kv8_append(pool, 0, s, k, k)
    x = pool.k[0, P - 1].float() * pool.k_scale[0, P - 1][:, None, None]
    ref = k[:16].float().permute(1, 0, 2)
    assert ((x - ref).abs() <= ref.abs() / 16 + pool.k_scale[0, P - 1][:, None, None] * 2.0 ** -10).all()
    assert not pool.k[0, :100].view(torch.uint8).any()


# calls with many tokens stream their rows through shared memory
@pytest.mark.parametrize("fused,pad,rope", [(False, 0, True), (True, 5, True), (False, 0, False)])
@pytest.mark.parametrize("H,starts,news", [(32, [0, 5, 31, 16], [300, 1, 170, 160]), (3, [7, 0], [3000, 3400]),
                                           (1, [0], [19000]), (20, [3, 15, 0], [500, 17, 513]),
                                           (8, [3, 0], [1500, 1300])])
def test_streamed_calls(H, starts, news, fused, pad, rope):
    case = Case("e4m3", starts, news, H=H, G=2, fused=fused, pad=pad, seed=H, n_pos=20000, rope=rope)
    before = case.state()
    case.run()
    check(case, before, case.state(), case.oracle(before))
    check_q(case)
    assert int(case.err.item()) == 0


def test_streamed_calls_give_the_bits_of_small_ones():
    """The same tokens in one call and page by page: the same codes, scales and
    queries, whatever the kernel (a page's rows are all in one call either way)."""
    a, b = (Case("e4m3", [0, 8], [320, 312], H=32, G=1, seed=3) for _ in range(2))
    a.run()
    t = 0
    for pages, start, n, pos0 in b.seqs:
        at = start
        while at < start + n:
            m = min(16 - at % 16, start + n - at)
            s = sp.Append([0, m], [at], [0, len(pages)], pages, pos0=[pos0])
            sp.rag_kv8_append(b.pool, 1, s, b.k[t:t + m], b.v[t:t + m], rope=b.rope, q=b.q[t:t + m],
                              q_out=b.q_out[t:t + m])
            at, t = at + m, t + m
    for x, y in zip(a.state(), b.state()):
        np.testing.assert_array_equal(x, y)
    assert torch.equal(a.q_out, b.q_out)


# a sequence that appends nothing is not looked at: its start and pages may be anything
@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("n", [3, 3000])
def test_a_sequence_of_no_tokens_is_skipped(kind, n):
    case = Case(kind, [5, 0, 2], [n, 0, n], H=8, seed=n, n_pos=8192)
    tok, start, po, ids, pos0 = case.arrays
    before = case.state()
    case.run()
    want = case.state()
    other = Case(kind, [5, 0, 2], [n, 0, n], H=8, seed=n, n_pos=8192)
    bad = list(start)
    bad[1] = 1 << 20
    other.append_c = sp.Append(tok, bad, po, ids, pos0=pos0)
    other.run()
    for x, y in zip(other.state(), want):
        np.testing.assert_array_equal(x, y)
    assert torch.equal(other.q_out, case.q_out) and int(other.err.item()) == int(case.err.item()) == 0


def test_streamed_infinities_bad_pages_and_positions():
    case = Case("e4m3", [0, 4, 0], [400, 300, 300], H=32, G=1, seed=4)
    tok, start, po, ids, pos0 = case.arrays
    ids = list(ids)
    ids[po[0] + 1] = -1
    case.append_c = sp.Append(tok, start, po, ids, pos0=[pos0[0], pos0[1], 4096 - 20])
    case.k[3, 0, 7], case.k[5, 1, 0] = float("inf"), float("nan")
    case.v[402, 31, 1], case.v[402, 30, 2] = float("-inf"), float("nan")
    before = case.state()
    case.run()
    after = case.state()
    assert int(case.err.item()) == 1 | 2 | 8
    p0, p1, p2 = (s[0] for s in case.seqs)
    np.testing.assert_array_equal(after[0][p0[1]], before[0][p0[1]])
    assert after[0][p0[0], 1, 5, 0] == 0 and np.isfinite(after[0][p0[0]]).all() and np.isfinite(after[2][p0[0]]).all()
    assert after[1][p1[0], 31, 6, 1] == -448 and after[1][p1[0], 30, 6, 2] == 0
    assert after[0][p2[1], :, :4].any() and not after[0][p2[1], :, 4:].any() and not after[1][p2[5]].any()
    assert not case.q_out[720:].any() and case.q_out[719].any()
