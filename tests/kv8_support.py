"""Helpers of the 8-bit-cache tests: a pool with poisoned unused slots, a batch
over it, the fp64 reference and the bounds it is held to."""

from __future__ import annotations

import numpy as np
import torch

import serving_prefill_b200 as sp


class AttnCase:
    """reqs: list of (chunk lengths, query tokens). Pages are placed at random;
    the slots that hold no token, and the pages nobody refers to, hold nan codes
    and nan scales."""

    def __init__(self, H, G, reqs, seed=0, q_scale=1.0, layers=2, layer=1, repeat=(), pad_rows=0, scale_exp=(-9, -4)):
        g = torch.Generator().manual_seed(seed)
        self.H, self.G, self.reqs, self.layer = H, G, reqs, layer
        lens = [c for chunks, _ in reqs for c in chunks]
        counts = [-(-n // 16) for n in lens]
        P = sum(counts) + 3
        perm = torch.randperm(P, generator=g).tolist()
        pages, at = [], 0
        for n in counts:
            pages.append(perm[at:at + n])
            at += n
        for dst, src in repeat:                     # a chunk-list entry that repeats another's pages
            assert lens[dst] == lens[src]
            pages[dst] = pages[src]
        codes = [torch.randint(0, 127, (layers, P, H, 16, 128), generator=g, dtype=torch.int32).to(torch.uint8)
                 | (torch.randint(0, 2, (layers, P, H, 16, 128), generator=g, dtype=torch.int32).to(torch.uint8) << 7)
                 for _ in range(2)]
        # magnitudes like a quantised page's: most codes in the upper binades
        mags = [torch.randn(layers, P, H, 16, 128, generator=g) * 90 for _ in range(2)]
        codes = [m.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for m in mags]
        scales = [torch.exp2(torch.randint(*scale_exp, (layers, P, H), generator=g).float()) for _ in range(2)]
        live = torch.zeros(P, 16, dtype=torch.bool)
        for n, pg in zip(lens, pages):
            for i, x in enumerate(pg):
                live[x, : min(16, n - 16 * i)] = True
        for c in codes:
            c[~live[None, :, None, :, None].expand_as(c)] = 0x7F
        for s in scales:
            s[:, ~live.any(1)] = float("nan")
        self.kc, self.vc = codes
        self.ks, self.vs = scales
        self.pool = sp.KV8Pool(layers, P, H, k=codes[0].view(torch.float8_e4m3fn).cuda(),
                               v=codes[1].view(torch.float8_e4m3fn).cuda(), k_scale=scales[0].cuda(),
                               v_scale=scales[1].cuda())
        self.pages, self.lens = pages, lens
        q_lens = [q for _, q in reqs]
        cum = lambda xs: np.cumsum([0] + list(xs)).tolist()  # noqa: E731
        self.arrays = [cum([len(c) for c, _ in reqs]), cum(lens), cum([len(p) for p in pages]),
                       [x for p in pages for x in p], cum(q_lens)]
        self.batch = sp.Batch(*self.arrays)
        self.total_q = sum(q_lens)
        rows = max(self.total_q + pad_rows, 1)
        self.q = (torch.randn(rows, H * G, 128, generator=g) * q_scale).to(torch.bfloat16).cuda()
        self.o = torch.full((rows, H * G, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((rows, H * G), 7.0, device="cuda")
        self.ws = sp.new_workspace(self.pool, self.batch, H * G)

    def run(self, causal=True, **kw):
        sp.rag_kv8_attn(self.pool, self.layer, self.batch, self.q, self.o, self.ws, causal=causal, row_lse=self.lse, **kw)
        torch.cuda.synchronize()
        return self.o[: self.total_q].double().cpu(), self.lse[: self.total_q].double().cpu()

    def dense(self):
        """Per request the fp64 K and V [N, H, 128] of its cached tokens."""
        out, c = [], 0
        for chunks, _ in self.reqs:
            ks, vs = [], []
            for n in chunks:
                pg = torch.tensor(self.pages[c], dtype=torch.long)
                for dst, codes, sc in ((ks, self.kc, self.ks), (vs, self.vc, self.vs)):
                    x = codes[self.layer][pg].view(torch.float8_e4m3fn).double()
                    x = x * sc[self.layer][pg].double()[:, :, None, None]
                    dst.append(x.permute(0, 2, 1, 3).reshape(-1, self.H, 128)[:n])
                c += 1
            z = torch.zeros(0, self.H, 128, dtype=torch.float64)
            out.append((torch.cat(ks) if ks else z, torch.cat(vs) if vs else z))
        return out

    def reference(self, causal=True, scale=128.0 ** -0.5):
        return reference(self.dense(), [q for _, q in self.reqs], self.q.double().cpu(), self.H, self.G, causal, scale)


def reference(dense, q_lens, q, H, G, causal, scale):
    """fp64 O, lse and the bounds of their errors. The bounds count, per row:
    the output's bf16 half step (2^-8 of the value); the weights' and a split
    row's fp16 half steps (2^-11 each) against sum alpha |v|, where a weight
    below 2^-14 of the row's largest has fp16's subnormal half step, 2^-25 of
    that largest (whose share of the row is at most 1): 2^-25 sum |v| more; an
    output below fp16's normal range likewise 2^-24; and the scores'
    error d as a relative error of the weights (2 d): queries in two e4m3 parts
    are off by at most 2^-10 of a row scale that is below max|q| / 224, and
    fp32 sums of 256 products by 256 * 2^-24 of the sum of magnitudes."""
    O, L, bo, bl = [], [], [], []
    q0 = 0
    for (k, v), nq in zip(dense, q_lens):
        n = k.shape[0]
        for j in range(nq):
            see = min(max(n - nq + j + 1, 0), n) if causal else n
            qq = q[q0 + j].view(H, G, 128)
            if see == 0:
                O.append(torch.zeros(H * G, 128, dtype=torch.float64))
                L.append(torch.full((H * G,), -float("inf"), dtype=torch.float64))
                bo.append(torch.zeros(H * G, 128, dtype=torch.float64))
                bl.append(torch.zeros(H * G, dtype=torch.float64))
                continue
            kk, vv = k[:see], v[:see]
            s = torch.einsum("hgd,nhd->hgn", qq, kk) * scale
            a = torch.softmax(s, -1)
            o = torch.einsum("hgn,nhd->hgd", a, vv)
            av = torch.einsum("hgn,nhd->hgd", a, vv.abs())
            # only keys that carry weight matter for the score error: bound over all of them is the safe one
            d = scale * (qq.abs().amax(-1) * kk.abs().sum(-1).amax(0)[:, None] * 2.0 ** -10 / 224
                         + torch.einsum("hgd,nhd->hgn", qq.abs(), kk.abs()).amax(-1) * 2.0 ** -16)
            rel = 2 * 2.0 ** -11 + 2 * d + 2.0 ** -14
            O.append(o.reshape(H * G, 128))
            L.append(torch.logsumexp(s, -1).reshape(-1))
            floor = 2.0 ** -25 * vv.abs().sum(0)[:, None]
            bo.append((2.0 ** -8 * o.abs() + rel[..., None] * av + floor + 2.0 ** -24).reshape(H * G, 128))
            bl.append((d + 2.0 ** -14 + 2.0 ** -22 * s.abs().amax(-1)).reshape(-1))
        q0 += nq
    z = lambda xs, *sh: torch.stack(xs) if xs else torch.zeros(0, *sh, dtype=torch.float64)  # noqa: E731
    return z(O, H * G, 128), z(L, H * G), z(bo, H * G, 128), z(bl, H * G)


def check(got, want):
    o, lse = got
    O, L, bo, bl = want
    err = (o - O).abs()
    assert torch.isfinite(o).all(), f"{(~torch.isfinite(o)).sum()} values are not finite"
    bad = err > bo
    assert not bad.any(), (bad.nonzero()[:5].tolist(), float((err / bo.clamp(min=1e-300)).max()))
    none = torch.isinf(L)
    assert torch.equal(torch.isinf(lse) & (lse < 0), none)
    e = (lse - L).abs()[~none]
    assert (e <= bl[~none]).all(), float((e / bl[~none]).max())
