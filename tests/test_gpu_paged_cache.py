"""msa_paged_attn and msa_paged_append over caches of other strides, and over tables, lengths and
offsets that do not fit."""
import pytest
import torch

import routed_sparse_attention_chunk_b200 as msa

from .paged_helpers import Batch, rotate64, rotation_bound

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _flag(flag):
    torch.cuda.synchronize()
    return int(flag.item())


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("q_len,total,Hq,Hkv,d,page,bad", [
    ([1, 2, 1], [300, 129, 90], 8, 2, 128, 16, {1: [3]}),              # few rows
    ([3, 1], [1000, 64], 4, 1, 64, 128, {0: [0, 7], 1: [0]}),          # whole tiles, nothing left for one
    ([2, 1], [30000, 500], 8, 2, 128, 64, {0: [0, 200, 468]}),         # cut items, the last page
    ([30, 2, 70], [300, 129, 90], 8, 2, 128, 16, {0: [18], 1: [3], 2: [0, 5]}),  # blocks of rows, new tokens' pages
    ([200, 9], [640, 9], 12, 4, 64, 8, {0: [0, 1, 40, 79]}),
    ([130, 5], [9000, 300], 8, 2, 128, 256, {0: [1, 35]}),
])
def test_pages_outside_the_pool_read_as_zeros(dtype, q_len, total, Hq, Hkv, d, page, bad):
    """In every kernel the same: keys and values of 0, and a flag."""
    b = Batch(q_len, total, Hq, Hkv, d, page, dtype, DEV, seed=61, pad_rows=2)
    for n, (i, pages) in enumerate(bad.items()):
        for m, pi in enumerate(pages):
            b.table[i, pi] = (-1, 2 ** 31 - 1, b.P)[(n + m) % 3]
            b.kd[i][pi * page:(pi + 1) * page] = 0
            b.vd[i][pi * page:(pi + 1) * page] = 0
    for max_q in (None, 40 + b.max_q):
        O, lse, flag = b.run(max_q=max_q)
        assert _flag(flag) == msa.FLAG_INDEX_OOB
        b.check(O, lse)


def _append_changes(b, k, q_off):
    """Which new tokens' cache rows an append with these offsets changed, and the flag."""
    K0 = b.K.clone()
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    msa.paged_append(None, k, k, q_off, b.seq_len, b.table, b.K, b.V, err_flag=flag)
    changed = ~((b.K == K0) | (b.K.isnan() & K0.isnan())).flatten(2).all(2)
    b.K.copy_(K0)
    return _flag(flag), changed


@pytest.mark.parametrize("dtype", [F32, BF])
def test_append_skips_tokens_of_bad_offsets(dtype):
    """A token whose sequence's offsets leave [0, N] is not written, at either end."""
    b = Batch([2, 1, 3], [20, 5, 40], 4, 2, 64, 16, dtype, DEV, seed=65)
    k = b.rnd(b.N, 2, 64) + 3.0
    rows = lambda i: [tuple(int(x) for x in s) for s in zip(*b.slots(i, torch.arange(b.total[i] - b.q_len[i], b.total[i])))]  # noqa: E731
    flag, changed = _append_changes(b, k, b.q_off)
    assert flag == 0 and sorted(map(tuple, changed.nonzero().tolist())) == sorted(rows(0) + rows(1) + rows(2))
    for first in (-1, -2 ** 40):
        o = b.q_off.clone()
        o[0] = first
        flag, changed = _append_changes(b, k, o)
        assert flag == msa.FLAG_OFFSETS and sorted(map(tuple, changed.nonzero().tolist())) == sorted(rows(1) + rows(2))
    for last in (b.N + 1, 2 ** 40):
        o = b.q_off.clone()
        o[3] = last
        flag, changed = _append_changes(b, k, o)
        assert flag == msa.FLAG_OFFSETS and sorted(map(tuple, changed.nonzero().tolist())) == sorted(rows(0) + rows(1))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("layout", ["kv_per_head", "kv_per_row", "padded_heads"])
@pytest.mark.parametrize("page", [8, 16, 256])
@pytest.mark.parametrize("d", [64, 128])
def test_other_strides(dtype, layout, page, d):
    """K beside V within each head, within each row, and heads apart from one another."""
    for q_len in ([1, 1, 2], [60, 1, 5]):
        b = Batch(q_len, [300, 131, 90], 8, 2, d, page, dtype, DEV, seed=62)
        shape = {"kv_per_head": (b.P, page, 2, 2, d), "kv_per_row": (b.P, page, 2, 2, d),
                 "padded_heads": (2, b.P, page, 2, d + 16)}[layout]
        pool = torch.full(shape, float("nan"), dtype=dtype, device=DEV)
        if layout == "kv_per_head":
            K, V = pool[:, :, :, 0], pool[:, :, :, 1]
        elif layout == "kv_per_row":
            K, V = pool[:, :, 0], pool[:, :, 1]
        else:
            K, V = pool[0][..., :d], pool[1][..., :d]
        K.copy_(b.K)
        V.copy_(b.V)
        b.K, b.V = K, V
        O, lse, flag = b.run()
        assert _flag(flag) == 0
        b.check(O, lse)
        # and the append into it: the same rows as into a dense cache, nothing beside them
        k, v = b.rnd(b.rows, 2, d), b.rnd(b.rows, 2, d)
        Kd, Vd = K.clone(memory_format=torch.contiguous_format), V.clone(memory_format=torch.contiguous_format)
        before = pool.clone()
        msa.paged_append(None, k, v, b.q_off, b.seq_len, b.table, K, V, err_flag=flag)
        msa.paged_append(None, k, v, b.q_off, b.seq_len, b.table, Kd, Vd, err_flag=flag)
        assert _flag(flag) == 0
        same = lambda x, y: bool(((x == y) | (x.isnan() & y.isnan())).all())  # noqa: E731
        assert same(K, Kd) and same(V, Vd)
        if layout == "padded_heads":
            assert pool[..., d:].isnan().all()
        for i, n in enumerate(q_len):
            pg, row = b.slots(i, torch.arange(b.total[i] - n))
            K2 = before[:, :, :, 0] if layout == "kv_per_head" else before[:, :, 0] if layout == "kv_per_row" else before[0][..., :d]
            assert torch.equal(K[pg, row], K2[pg, row])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("q_len,total,d", [([1, 2], [64, 64], 128), ([40, 30], [128, 128], 128), ([3, 40], [48, 48], 64)])
def test_length_past_the_table_reads_the_table(dtype, q_len, total, d):
    """A length past max_pages * page is that length: the same bits, and a flag."""
    b = Batch(q_len, total, 8, 2, d, 16, dtype, DEV, seed=63)
    b.table = b.table[:, :total[0] // 16].contiguous()
    O1, lse1, flag = b.run()
    assert _flag(flag) == 0
    b.check(O1, lse1)
    b.seq_len[1] = total[1] + 1000
    O2, lse2, flag = b.run()
    assert _flag(flag) == msa.FLAG_INDEX_OOB
    assert torch.equal(O1, O2) and torch.equal(lse1, lse2)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("q_len,end,max_q", [([1, 1, 2, 1], 3, 4), ([40, 32, 60, 5], 92, 100)])
def test_decreasing_offsets_skip_their_sequence(dtype, q_len, end, max_q):
    """A sequence that ends before it begins is skipped; rows that only one other sequence claims hold."""
    b = Batch(q_len, [300, 129, 200, 90], 8, 2, 128, 16, dtype, DEV, seed=64)
    O1, lse1, _ = b.run(max_q=max_q)
    b.q_off[1] = end  # the first sequence takes the second's rows and some of the third's
    O2, lse2, flag = b.run(max_q=max_q)
    assert _flag(flag) == msa.FLAG_OFFSETS
    alone = slice(end, b.N)
    assert torch.equal(O1[alone], O2[alone]) and torch.equal(lse1[:, alone], lse2[:, alone])


def test_gradient_of_a_broadcast_input():
    """One head's row read for all heads: the rows' gradients, summed over the heads, are its own."""
    N, H, d = 20, 4, 64
    g = torch.Generator(device=DEV).manual_seed(66)
    one, w, u = (torch.randn(N, h, d, generator=g, device=DEV) for h in (1, H, 1))
    cs, pos = msa.rope_table_scaled("none", 1e6, d, 32).to(DEV), torch.arange(N, dtype=torch.int32, device=DEV)
    y, dx = torch.empty((N, H, d), device=DEV), torch.empty((N, H, d), device=DEV)
    msa.rope_backward(w, pos, cs, dx)
    rows = cs[pos.long()]
    assert ((dx.double() - rotate64(w, rows, transpose=True)).abs() <= rotation_bound(w, rows, F32)).all()
    # <w, rope(one + u / 4) - rope(one - u / 4)> 2 = <sum over heads of dx, u>: rounding as in a
    # difference of four roundings of |one| + |u| / 4 per term, times 2 |w|
    outs = []
    for x in (one + 0.25 * u, one - 0.25 * u):
        msa.rope(x.expand(N, H, d), pos, cs, y)
        outs.append(y.double())
    num = ((outs[0] - outs[1]) * 2 * w.double()).sum()
    ana = (dx.double().sum(1, keepdim=True) * u.double()).sum()
    scale = float(((one.abs() + u.abs()) * w.abs()).double().sum())
    assert abs(float(num - ana)) <= 32 * 2.0 ** -24 * scale


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("max_q", [4, 90])
def test_a_token_alone_and_in_a_batch(dtype, max_q):
    """The batch decides where a sequence's keys are cut and which kernel runs, so fp32 sums change
    their order and bf16 weights the reference they are rounded against; nothing else."""
    b = Batch([1, 3, 2, 1], [5000, 300, 20000, 40], 8, 2, 128, 16, dtype, DEV, seed=67)
    O1, lse1, _ = b.run(max_q=max_q)
    want, lo, A = b.attention64()
    bo, bl = b.bounds(want, A, lo, max(b.total))
    for i in range(4):
        one = Batch([1], [1], 8, 2, 128, 16, dtype, DEV, seed=1)
        sl = slice(b.off[i], b.off[i + 1])
        one.__dict__.update(q_len=[b.q_len[i]], total=[b.total[i]], N=b.q_len[i], rows=b.q_len[i], max_q=b.q_len[i],
                            Q=b.Q[sl].contiguous(), q_off=b.q_off[i:i + 2] - b.q_off[i], table=b.table[i:i + 1].contiguous(),
                            seq_len=b.seq_len[i:i + 1].contiguous(), K=b.K, V=b.V)
        O2, lse2, flag = one.run()
        assert _flag(flag) == 0
        assert ((O1[sl].double() - O2.double()).abs() <= 2 * bo[sl]).all()
        assert ((lse1[:, sl].double() - lse2.double()).abs() <= 2 * bl[:, sl]).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,q", [(4, 1), (5, 1), (1, 4), (8, 1), (4, 2), (9, 1), (3, 3), (16, 1), (4, 4), (17, 1), (3, 6)])
def test_rows_around_the_kernels_borders(dtype, d, G, q):
    """4, 5, 8, 9, 16, 17 rows per KV head: at and beside the counts at which another kernel takes the call."""
    b = Batch([q, 1, 0, q], [700, 40, 9, 129], 2 * G, 2, d, 32, dtype, DEV, seed=68).select(3, 9, 11, seed=8)
    O, lse, flag = b.run(40)
    assert _flag(flag) in (0, msa.FLAG_OVERFLOW)
    b.check(O, lse, 40)
