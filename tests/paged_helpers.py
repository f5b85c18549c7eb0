"""Plain fp64 forms of the rotary positions, the paged append and the attention over a paged
cache, and the batches their tests run (torch, any device)."""
from __future__ import annotations

import torch

import routed_sparse_attention_chunk_b200 as msa

HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # of a rounding, relative


def rotate64(x, cs, interleaved=False, transpose=False):
    """x [N, H, d], cs [N, rd/2, 2] (the table rows of the tokens): fp64."""
    x, cs = x.double(), cs.double()
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    if transpose:
        s = -s
    rd = 2 * c.shape[-1]
    y = x.clone()
    a, b = (x[..., 0:rd:2], x[..., 1:rd:2]) if interleaved else (x[..., :rd // 2], x[..., rd // 2:rd])
    u, w = a * c - b * s, a * s + b * c
    if interleaved:
        y[..., 0:rd:2], y[..., 1:rd:2] = u, w
    else:
        y[..., :rd // 2], y[..., rd // 2:rd] = u, w
    return y


def rotation_bound(x, cs, dtype, interleaved=False):
    """Elementwise error bound of a rotation in fp32 stored in dtype: two products and a sum, each
    rounded once (3 x 2^-24 of |a c| + |b s|), then the store's half step."""
    x, cs = x.double().abs(), cs.double().abs()
    mag = rotate64(x, torch.stack([cs[..., 0], -cs[..., 1]], -1), interleaved)  # |a||c| + |b||s| in the first half
    mag2 = rotate64(x, cs, interleaved)                                          # ... and in the second
    m = torch.maximum(mag, mag2)
    return 3 * 2.0 ** -24 * m + HALF_STEP[dtype] * (1 + 2.0 ** -20) * m


class Batch:
    """Ragged sequences over a cache of pages.  Everything the calls must not read is NaN: pages
    that belong to nobody, rows past a sequence's last token, and (as far outside) block-table
    entries past a sequence's last page."""

    def __init__(self, q_len, total, Hq, Hkv, d, page, dtype, device, seed=0, order="prhd", pad_rows=0, spare=3,
                 scale=0.5):
        g = torch.Generator(device=device).manual_seed(seed)
        self.q_len, self.total, self.page, self.dtype, self.device = list(q_len), list(total), page, dtype, device
        self.Hq, self.Hkv, self.d = Hq, Hkv, d
        B, N = len(q_len), sum(q_len)
        self.N, self.rows = N, N + pad_rows
        off = [0]
        for n in q_len:
            off.append(off[-1] + n)
        self.off = off
        self.q_off = torch.tensor(off, dtype=torch.int64, device=device)
        self.seq_len = torch.tensor(self.total, dtype=torch.int32, device=device)
        self.max_q = max(max(q_len), 1)
        npages = [-(-t // page) for t in self.total]
        P = sum(npages) + spare
        perm = torch.randperm(P, generator=torch.Generator().manual_seed(seed)).tolist()
        width = max(npages + [1]) + 1
        table = torch.full((B, width), 2 ** 31 - 1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(npages):
            table[b, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
            at += n
        self.table = table.to(device)
        self.P = P

        def pages():
            shape = {"prhd": (P, page, Hkv, d), "phrd": (P, Hkv, page, d), "pair": (P, 2, page, Hkv, d)}[order]
            return torch.full(shape, float("nan"), dtype=dtype, device=device)
        if order == "pair":
            both = pages()
            self.K, self.V = both[:, 0], both[:, 1]
        else:
            self.K, self.V = pages(), pages()
            if order == "phrd":
                self.K, self.V = self.K.transpose(1, 2), self.V.transpose(1, 2)
        rnd = lambda *s: (scale * torch.randn(s, generator=g, device=device)).to(dtype)
        self.kd, self.vd = [], []  # dense keys and values of every sequence
        for b in range(B):
            k, v = rnd(self.total[b], Hkv, d), rnd(self.total[b], Hkv, d)
            self.kd.append(k)
            self.vd.append(v)
            pg, row = self.slots(b, torch.arange(self.total[b]))
            self.K[pg, row], self.V[pg, row] = k, v
        self.Q = torch.full((self.rows, Hq, d), float("nan"), dtype=dtype, device=device)
        self.Q[:N] = rnd(N, Hq, d)
        self.rnd = rnd

    def slots(self, b, t):
        """Page and row of cache positions t of sequence b."""
        t = t.to(self.device)
        return self.table[b].long()[t // self.page], t % self.page

    def select(self, k, docs, max_chunks, seed=0, fixed=False):
        """A bank of `docs` documents of 1..max_chunks chunks and k of them for every sequence."""
        g = torch.Generator().manual_seed(seed)
        n = torch.full((docs,), max_chunks) if fixed else torch.randint(0, max_chunks + 1, (docs,), generator=g)
        n[0] = max(int(n[0]), 1)
        self.chunk_off = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)]).to(self.device)
        C = int(n.sum())
        self.Kbar, self.Vbar = self.rnd(C, self.Hkv, self.d), self.rnd(C, self.Hkv, self.d)
        self.idx = torch.stack([torch.randperm(docs, generator=g)[:k] for _ in self.q_len]).to(torch.int32).to(self.device)
        self.k = k
        return self

    def memory(self, b, Mmax):
        if not hasattr(self, "idx"):
            return [], False
        off = self.chunk_off.tolist()
        D = len(off) - 1
        rows = [c for j in self.idx[b].tolist() if 0 <= j < D for c in range(off[j], off[j + 1])]
        return rows[:Mmax], len(rows) > Mmax

    def attention64(self, Mmax=0, scale=None):
        """O [N, Hq, d], lse [Hq, N] and A = sum p |v| (the scale of the weights' rounding) in fp64."""
        G, sc = self.Hq // self.Hkv, scale or self.d ** -0.5
        O = torch.zeros((self.N, self.Hq, self.d), dtype=torch.float64, device=self.device)
        A, lse = torch.zeros_like(O), torch.full((self.Hq, self.N), -float("inf"), dtype=torch.float64, device=self.device)
        self.smax = 0.0  # largest sum |q||k| scale: the scale of the scores' fp32 rounding
        for b, (n, t) in enumerate(zip(self.q_len, self.total)):
            rows, _ = self.memory(b, Mmax)
            m = len(rows)
            for h in range(self.Hq):
                k, v = self.kd[b][:, h // G].double(), self.vd[b][:, h // G].double()
                if m:
                    k = torch.cat([self.Kbar[rows, h // G].double(), k])
                    v = torch.cat([self.Vbar[rows, h // G].double(), v])
                q = self.Q[self.off[b]:self.off[b] + n, h].double()
                if n == 0 or m + t == 0:
                    continue
                s = q @ k.T * sc
                self.smax = max(self.smax, float((q.abs() @ k.abs().T).max()) * sc)
                i, j = torch.arange(n, device=self.device)[:, None], torch.arange(m + t, device=self.device)[None]
                s.masked_fill_((j >= m) & (j > m + t - n + i), -float("inf"))  # memory rows are always visible
                some = s.amax(1) > -float("inf")
                l = torch.logsumexp(s, 1)
                p = torch.where(some[:, None], torch.exp(s - torch.where(some, l, 0.0)[:, None]), 0.0)
                sl = slice(self.off[b], self.off[b] + n)
                O[sl, h], A[sl, h], lse[h, sl] = p @ v, p @ v.abs(), l
        return O, lse, A

    def bounds(self, O, A, lse, keys):
        """Elementwise error bounds.  bf16: every weight rounded to bf16 (a half step of A in all),
        2^x to 7.5e-5, scores and sums in fp32, the store's half step of O.  fp32: d products and a
        sum per score, one rounding of the exponent's argument, a sum over the keys; all of A."""
        ds = (self.d + 4) * 2.0 ** -24 * self.smax  # of a score
        n = keys * 2.0 ** -24
        if self.dtype == torch.bfloat16:
            rel = 2.0 ** -8 + 7.5e-5 + 2 * ds + n
            return rel * A + 2.0 ** -8 * (O.abs() + rel * A) + 1e-30, 7.5e-5 + 2 * ds + n + 2.0 ** -22 * lse.abs()
        rel = 4 * ds + 2 * n + 16 * 2.0 ** -24
        return rel * A + 2.0 ** -24 * O.abs() + 1e-30, rel + 2.0 ** -22 * lse.abs()

    def run(self, Mmax=0, scale=0.0, want_lse=True, max_q=None, ws=None, O=None, flag=None):
        """msa.paged_attn of the batch: (O, lse, flag value is read by the caller)."""
        sel = hasattr(self, "idx")
        max_q = max_q or self.max_q
        n = msa.paged_attn_workspace_size(self.dtype, len(self.q_len), max_q, self.Hq, self.Hkv, self.d,
                                          self.k if sel else 0, Mmax)
        ws = ws if ws is not None else torch.full((n,), 255, dtype=torch.uint8, device=self.device)  # NaN bytes
        O = O if O is not None else torch.full((self.rows, self.Hq, self.d), 7.0, dtype=self.dtype, device=self.device)
        lse = torch.full((self.Hq, self.rows), 7.0, dtype=torch.float32, device=self.device) if want_lse else None
        flag = flag if flag is not None else torch.zeros(1, dtype=torch.int32, device=self.device)
        kw = dict(topk_idx=self.idx, doc_chunk_off=self.chunk_off, Kbar=self.Kbar, Vbar=self.Vbar, Mmax=Mmax) if sel else {}
        msa.paged_attn(self.Q, self.q_off, max_q, self.K, self.V, self.table, self.seq_len, O, ws, lse=lse,
                       scale=scale, err_flag=flag, **kw)
        return O, lse, flag

    def check(self, O, lse, Mmax=0, scale=None):
        Oo, lo, A = self.attention64(Mmax, scale)
        keys = max(self.total + [0]) + Mmax
        bo, bl = self.bounds(Oo, A, torch.nan_to_num(lo, neginf=0.0), keys)
        N = self.N
        err = (O[:N].double() - Oo).abs()
        assert torch.isfinite(O[:N].float()).all(), "O is not finite"
        assert (err <= bo).all(), f"O off by {float((err / bo).max()):.3g} x its bound"
        assert (O[N:] == 7).all(), "rows behind the last sequence were written"
        if lse is not None:
            none = lo == -float("inf")
            assert (lse[:, :N][none] == -float("inf")).all()
            el = (lse[:, :N].double() - lo).abs()[~none]
            assert (el <= bl[~none]).all(), f"lse off by {float((el / bl[~none]).max()):.3g} x its bound"
            assert (lse[:, N:] == 7).all()
