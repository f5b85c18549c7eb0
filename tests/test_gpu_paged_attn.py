"""msa_paged_attn against a plain fp64 form: ragged batches over a cache of pages, from one token
over one key to parts of prompts over thousands, with and without selected documents.  Everything
the call must not read (free pages, rows past a sequence's end, the workspace) holds NaN."""
import pytest
import torch

import routed_sparse_attention_chunk_b200 as msa

from .paged_helpers import Batch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _flag(flag):
    torch.cuda.synchronize()
    return int(flag.item())


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("q_len,total,Hq,Hkv,d,page", [
    ([1], [1], 8, 2, 128, 16),                               # one token, one key
    ([1, 1, 1], [128, 129, 127], 32, 8, 128, 16),            # around a tile's end
    ([1] * 5, [1, 2, 300, 1000, 64], 4, 4, 128, 8),          # G = 1
    ([1, 0, 1], [77, 500, 33], 14, 2, 128, 32),              # G = 7, a sequence without new tokens
    ([4, 1, 3], [1030, 40, 3], 32, 8, 128, 64),              # drafts: 16 rows
    ([2, 2], [256, 255], 64, 8, 128, 256),                   # G = 8 x 2 tokens
    ([1, 1], [700, 5], 5, 1, 64, 16),                        # small heads, G = 5
    ([33], [33], 8, 8, 64, 8),                               # a prompt, no history
    ([70, 1, 130], [300, 900, 130], 12, 4, 128, 16),         # parts of prompts among a token, G = 3
    ([257], [1000], 32, 8, 128, 128),                        # several blocks
    ([40, 1], [640, 257], 64, 1, 64, 32),                    # G = 64: two tokens a block
    ([5, 9], [5, 1], 8, 2, 128, 16),                         # lengths below the new tokens: no key for some
    ([3], [0], 8, 2, 128, 16),                               # nothing cached at all
    ([300, 300], [0, 17], 8, 4, 64, 64),
])
def test_ragged_batches(dtype, q_len, total, Hq, Hkv, d, page):
    b = Batch(q_len, total, Hq, Hkv, d, page, dtype, DEV, seed=1, pad_rows=3)
    O, lse, flag = b.run()
    assert _flag(flag) == 0
    b.check(O, lse)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("q_len,total,Hq,Hkv,d,page,k,Mmax", [
    ([1] * 4, [300, 1, 129, 64], 32, 8, 128, 16, 5, 80),
    ([1, 2], [40, 700], 8, 4, 128, 64, 16, 300),
    ([50, 1, 200], [50, 300, 999], 16, 4, 128, 32, 7, 200),
    ([20, 3], [20, 60], 6, 2, 64, 8, 3, 40),
    ([2], [0], 8, 2, 128, 16, 4, 60),                        # memory rows only
    ([130, 2], [100, 2], 8, 2, 128, 16, 4, 60),              # memory rows and no local key for some
    ([1], [50], 8, 2, 128, 16, 6, 0),                        # no room for memory rows
    ([1, 1], [200, 10], 32, 8, 128, 16, 9, 17),              # the selection overflows inside a run
])
def test_with_selected_documents(dtype, q_len, total, Hq, Hkv, d, page, k, Mmax):
    b = Batch(q_len, total, Hq, Hkv, d, page, dtype, DEV, seed=2, pad_rows=1).select(k, 40, 19, seed=3)
    O, lse, flag = b.run(Mmax)
    over = any(b.memory(i, Mmax)[1] for i in range(len(q_len)))
    assert _flag(flag) == (msa.FLAG_OVERFLOW if over else 0)
    b.check(O, lse, Mmax)


@pytest.mark.parametrize("order", ["phrd", "pair"])
@pytest.mark.parametrize("dtype,q_len,d", [(BF, [1, 1, 2], 128), (BF, [60, 1, 5], 128), (BF, [60, 1, 5], 64),
                                           (F32, [20, 1, 5], 64)])
def test_cache_strides(order, dtype, q_len, d):
    """Pages of [head, row] and pages that hold K beside V, queries inside a fused projection."""
    b = Batch(q_len, [200, 131, 90], 8, 2, d, 16, dtype, DEV, seed=4, order=order)
    wide = torch.full((b.rows, 13, d), float("nan"), dtype=dtype, device=DEV)
    wide[:, 3:11] = b.Q
    b.Q = wide[:, 3:11]
    O, lse, flag = b.run()
    assert _flag(flag) == 0
    b.check(O, lse)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
def test_page_sizes(dtype, page):
    for q_len in ([1, 1], [90, 40]):
        b = Batch(q_len, [391, 40], 8, 2, 128, page, dtype, DEV, seed=5)
        O, lse, flag = b.run()
        assert _flag(flag) == 0
        b.check(O, lse)


@pytest.mark.parametrize("dtype,q_len,total,Hq,Hkv,d", [
    (BF, [1], [40000], 4, 1, 128),           # one item cut by every border
    (BF, [1, 1, 1], [20000, 9, 3000], 32, 8, 128),
    (BF, [130], [20000], 8, 2, 128),
    (BF, [700, 1, 64], [5000, 12000, 64], 16, 4, 64),
    (F32, [3, 60], [9000, 2000], 8, 2, 128),
])
def test_long_caches(dtype, q_len, total, Hq, Hkv, d):
    b = Batch(q_len, total, Hq, Hkv, d, 64, dtype, DEV, seed=6)
    O, lse, flag = b.run()
    assert _flag(flag) == 0
    b.check(O, lse)


@pytest.mark.parametrize("q_len,total,Hq,Hkv,d", [
    ([300, 320], [420, 320], 32, 8, 128), ([20, 3], [180, 131], 20, 1, 64), ([9], [140], 33, 1, 128),
    ([5, 70], [300, 70], 64, 1, 64), ([30, 40], [33, 500], 6, 2, 64), ([33], [129], 32, 1, 128)])
def test_fp32_blocks_of_either_size(q_len, total, Hq, Hkv, d):
    """Blocks of 32 rows and of 64, chosen by the heads that fit and the size of the batch."""
    b = Batch(q_len, total, Hq, Hkv, d, 32, F32, DEV, seed=31).select(2, 9, 11, seed=8)
    O, lse, flag = b.run(20)
    assert _flag(flag) in (0, msa.FLAG_OVERFLOW)
    b.check(O, lse, 20)


@pytest.mark.parametrize("d", [64, 128])
def test_single_tokens_in_a_batch_with_parts(d):
    """Long runs of tiles where most rows of a block do not exist (their warps run ahead)."""
    b = Batch([1, 40, 1, 2, 1], [20001, 300, 20001, 16000, 9000], 8, 4, d, 128, BF, DEV, seed=19)
    for _ in range(3):
        O, lse, flag = b.run()
        assert _flag(flag) == 0
    b.check(O, lse)


def test_many_sequences():
    """More sequences than threads that plan the split, most of them tiny, some without new tokens."""
    g = torch.Generator().manual_seed(7)
    q_len = torch.randint(0, 3, (700,), generator=g).tolist()
    total = [n + int(c) for n, c in zip(q_len, torch.randint(0, 90, (700,), generator=g))]
    for Hq, Hkv, d in ((8, 2, 128), (8, 2, 64)):
        b = Batch(q_len, total, Hq, Hkv, d, 8, BF, DEV, seed=7, pad_rows=2)
        O, lse, flag = b.run()
        assert _flag(flag) == 0
        b.check(O, lse)


@pytest.mark.parametrize("q_len", [[1, 1, 1], [40, 200, 3]])
def test_large_scores_move_the_maximum(q_len):
    """Scores of some hundred, growing along the keys: the running maximum moves in most tiles."""
    b = Batch(q_len, [900, 700, 333], 8, 2, 128, 16, BF, DEV, seed=8, scale=2.0)
    O, lse, flag = b.run()
    assert _flag(flag) == 0
    b.check(O, lse)
    for i, kd in enumerate(b.kd):  # keys growing with the position
        kd *= torch.linspace(0.1, 3.0, kd.shape[0], device=DEV)[:, None, None].to(BF)
        pg, row = b.slots(i, torch.arange(b.total[i]))
        b.K[pg, row] = kd
    O, lse, flag = b.run(scale=0.25)
    assert _flag(flag) == 0
    b.check(O, lse, scale=0.25)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_max_q_is_only_a_bound(dtype):
    """A larger max_q selects another kernel, not another result."""
    b = Batch([1, 2, 1], [300, 129, 7], 8, 2, 128, 16, dtype, DEV, seed=9)
    for max_q in (2, 4, 5, 300):
        O, lse, flag = b.run(max_q=max_q)
        assert _flag(flag) == 0
        b.check(O, lse)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("q_len", [[1, 2, 1], [30, 2, 70]])
def test_device_flags(dtype, q_len):
    """What only the device can see is flagged, skipped or clamped, and the other sequences hold."""
    def fresh():
        return Batch(q_len, [300, 129, 90], 8, 2, 128, 16, dtype, DEV, seed=10)

    def check_others(b, O, lse, bad):
        Oo, lo, A = b.attention64()
        bo, bl = b.bounds(Oo, A, lo, 400)
        keep = torch.ones(b.N, dtype=torch.bool, device=DEV)
        keep[b.off[bad]:b.off[bad + 1]] = False
        assert ((O[:b.N].double() - Oo).abs() <= bo)[keep].all()
        assert ((lse[:, :b.N].double() - lo).abs() <= bl)[:, keep].all()

    for page in (-1, 10 ** 6):  # a page outside the pool
        b = fresh()
        b.table[1, 3] = page
        O, lse, flag = b.run()
        assert _flag(flag) == msa.FLAG_INDEX_OOB
        check_others(b, O, lse, 1)
    b = fresh()
    b.seq_len[2] = -4
    O, lse, flag = b.run()
    assert _flag(flag) == msa.FLAG_INDEX_OOB
    check_others(b, O, lse, 2)
    assert (O[b.off[2]:b.off[3]] == 0).all() and (lse[:, b.off[2]:b.off[3]] == -float("inf")).all()
    b = fresh()
    b.q_off[3] = b.N + 5  # past the packed rows
    O, lse, flag = b.run()
    assert _flag(flag) == msa.FLAG_OFFSETS
    check_others(b, O, lse, 2)
    assert (O[b.off[2]:] == 7).all()
    b = fresh()
    b.q_off[2] = 0  # decreasing
    b.q_off[1] = 1 if q_len[0] == 1 else 30
    O, lse, flag = b.run()
    assert _flag(flag) & msa.FLAG_OFFSETS
    b = fresh()
    O, lse, flag = b.run(max_q=1)  # sequences above the bound are skipped
    assert _flag(flag) == msa.FLAG_OFFSETS
    for i, n in enumerate(q_len):
        if n > 1:
            assert (O[b.off[i]:b.off[i + 1]] == 7).all()


def test_length_past_the_table_is_clamped():
    b = Batch([1, 1], [64, 30], 8, 2, 128, 16, BF, DEV, seed=11, spare=60)
    b.table = b.table[:, :4].contiguous()
    b.table[1] = torch.tensor([7, 7, 7, 7], device=DEV)
    b.seq_len[1] = 1000
    O, lse, flag = b.run()
    assert _flag(flag) == msa.FLAG_INDEX_OOB


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("q_len", [[1, 1], [100, 7]])
def test_bad_documents_are_skipped(dtype, q_len):
    b = Batch(q_len, [200, 140], 8, 2, 128, 16, dtype, DEV, seed=12).select(5, 30, 9, seed=12)
    b.idx[0, 1], b.idx[1, 4] = -1, 30
    O, lse, flag = b.run(60)
    assert _flag(flag) & msa.FLAG_INDEX_OOB
    b.check(O, lse, 60)


@pytest.mark.parametrize("q_len", [[1, 1, 2], [200, 1, 30]])
def test_same_bits_every_time(q_len):
    b = Batch(q_len, [3000, 129, 900], 16, 4, 128, 16, BF, DEV, seed=13)
    O, lse, _ = b.run()
    for _ in range(3):
        O2, lse2, _ = b.run()
        assert torch.equal(O, O2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("q_len", [[1, 1, 2], [150, 1, 30]])
def test_captured_and_replayed(q_len):
    """A captured call follows the lengths, the table and the values of the replay; two graphs and
    an eager call on another stream each use their own workspace."""
    b = Batch(q_len, [700, 129, 300], 16, 4, 128, 16, BF, DEV, seed=14).select(4, 20, 9, seed=1)
    c = Batch(q_len, [700, 129, 300], 16, 4, 128, 16, BF, DEV, seed=15).select(4, 20, 9, seed=2)
    ws = [torch.empty(msa.paged_attn_workspace_size(BF, 3, b.max_q, 16, 4, 128, 4, 40), dtype=torch.uint8, device=DEV)
          for _ in range(2)]
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    b.run(40, ws=ws[0], flag=flag)
    torch.cuda.synchronize()
    graphs = []
    for i, x in enumerate((b, c)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = x.run(40, ws=ws[i], flag=flag)
        graphs.append((g, x, out))
    # shorter sequences and other pages' values for the replay
    for g, x, out in graphs:
        x.total = [700 - 37, 129, 260]
        x.seq_len.copy_(torch.tensor(x.total, dtype=torch.int32))
        x.kd, x.vd = [k[:t] for k, t in zip(x.kd, x.total)], [v[:t] for v, t in zip(x.vd, x.total)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs[0][0].replay()
    with torch.cuda.stream(s):
        graphs[1][0].replay()
    torch.cuda.synchronize()
    assert int(flag.item()) == 0
    for g, x, out in graphs:
        x.check(out[0], out[1], 40)


def test_agrees_with_the_dense_layer_attention():
    """The same selection and local rows through msa_sparse_attn_indexed (dense local K / V)."""
    B, T, L, Hq, Hkv, d, k = 2, 48, 160, 32, 8, 128, 6
    b = Batch([T] * B, [L] * B, Hq, Hkv, d, 32, BF, DEV, seed=16).select(k, 30, 8, seed=4, fixed=True)
    Mmax = 8 * k
    O, lse, flag = b.run(Mmax)
    Kl, Vl = torch.stack(b.kd), torch.stack(b.vd)
    Q = b.Q.view(B, T, Hq, d)
    O2, lse2 = torch.empty_like(Q), torch.empty((B, Hq, T), device=DEV)
    ws = torch.empty(msa.sparse_attn_indexed_workspace_size(B, T, L, Hq, Hkv, d, k, Mmax), dtype=torch.uint8, device=DEV)
    msa.sparse_attn_indexed(Q, Kl, Vl, b.idx, b.chunk_off, b.Kbar, b.Vbar, Mmax, O2, ws, lse2, err_flag=flag)
    assert _flag(flag) == 0
    Oo, lo, A = b.attention64(Mmax)
    bo, bl = b.bounds(Oo, A, lo, L + Mmax)
    assert ((O.double() - O2.view_as(O).double()).abs() <= 2 * bo).all()
    assert ((lse.double() - lse2.transpose(0, 1).reshape(Hq, B * T).double()).abs() <= 2 * bl).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("q_len,total,d,max_q", [
    ([3], [300], 128, None), ([4, 1], [131, 90], 128, None), ([2], [2], 128, None),     # drafts
    ([70], [70], 128, None), ([200, 9], [640, 9], 128, None), ([150], [300], 64, None),  # parts of prompts
    ([3, 4], [257, 128], 128, 90)])
def test_values_that_are_not_finite(dtype, q_len, total, d, max_q):
    """Infinities and NaN in V of new tokens reach exactly the tokens that see them, dimension by
    dimension; in K, the tokens that see the key; in bank rows nobody selected, nobody."""
    inf, nan = float("inf"), float("nan")
    b = Batch(q_len, total, 8, 2, d, 16, dtype, DEV, seed=21).select(2, 12, 9, seed=3)
    Mmax = 18
    O0, lse0, _ = b.run(Mmax, max_q=max_q)
    b.check(O0, lse0, Mmax)
    picked = {c for i in range(len(q_len)) for c in b.memory(i, Mmax)[0]}
    rest = [c for c in range(b.Kbar.shape[0]) if c not in picked]
    b.Kbar[rest], b.Vbar[rest] = nan, inf
    marks = []  # (sequence, position, KV head, dimension, value)
    for i, (n, t) in enumerate(zip(q_len, total)):
        for back, g, x, val in ((1, 0, 3, inf), (1, 1, 5, nan), (n // 2 + 1, 0, 7, -inf), (n // 2 + 1, 0, 3, inf),
                                (n, 1, 60, inf), (max(n // 3, 1), 1, 60, -inf)):
            if back <= n and (i, t - back, g, x) not in [m[:4] for m in marks]:
                marks.append((i, t - back, g, x, val))
    clean = [v.clone() for v in b.vd]
    want, lo, A = None, None, None
    for i, pos, g, x, val in marks:
        clean[i][pos, g, x] = 0
        pg, row = b.slots(i, torch.tensor([pos]))
        b.V[pg, row, g, x] = val
    b.vd = clean
    want, lo, A = b.attention64(Mmax)
    bo, bl = b.bounds(want, A, lo, max(total) + Mmax)
    for i, pos, g, x, val in marks:
        first = b.off[i] + max(0, pos - (total[i] - q_len[i]))
        want[first:b.off[i + 1], 4 * g:4 * g + 4, x] += val  # inf - inf: NaN
    for _ in range(2):
        O, lse, flag = b.run(Mmax, max_q=max_q)
        assert _flag(flag) == 0
        odd = ~want.isfinite()
        got = O[:b.N].double()
        assert torch.equal(got.isnan()[odd], want.isnan()[odd])
        there = odd & ~want.isnan()
        assert torch.equal(got[there], want[there])
        assert (got - want).abs()[~odd].le(bo[~odd]).all()
        assert ((lse[:, :b.N].double() - lo).abs() <= bl).all()
    # a key that is not finite: its own token and the later ones, of its KV head
    i = 0
    b2 = Batch(q_len, total, 8, 2, d, 16, dtype, DEV, seed=21)
    pos = total[i] - 1 - q_len[i] // 2
    pg, row = b2.slots(i, torch.tensor([pos]))
    O1, _, _ = b2.run(max_q=max_q)
    b2.K[pg, row, 1, 2] = nan
    O2, _, flag = b2.run(max_q=max_q)
    assert _flag(flag) == 0
    first = b2.off[i] + pos - (total[i] - q_len[i])
    hit = torch.zeros(b2.N, 8, dtype=torch.bool, device=DEV)
    hit[first:b2.off[i + 1], 4:] = True
    assert O2[:b2.N][hit].isnan().all() and torch.equal(O2[:b2.N][~hit], O1[:b2.N][~hit])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("q_len,total,d", [([3, 1], [300, 140], 128), ([1, 2], [700, 40], 64), ([150, 4], [200, 600], 128),
                                           ([70], [300], 64)])
def test_query_that_is_not_finite(dtype, q_len, total, d):
    """A head of a token whose query holds a NaN is NaN; no other head or token changes by a bit."""
    b = Batch(q_len, total, 8, 2, d, 16, dtype, DEV, seed=41)
    O1, lse1, _ = b.run()
    tok, h = b.N // 2, 5
    b.Q[tok, h, 7] = float("nan")
    O2, lse2, flag = b.run()
    assert _flag(flag) == 0
    assert O2[tok, h].isnan().all() and lse2[h, tok].isnan()
    O2[tok, h], lse2[h, tok] = O1[tok, h], lse1[h, tok]
    assert torch.equal(O1, O2) and torch.equal(lse1, lse2)


@pytest.mark.parametrize("dtype,max_q", [(F32, 1), (BF, 1), (BF, 40)])
def test_no_new_tokens_at_all(dtype, max_q):
    """Sequences without new tokens leave everything as it was; rows before the first are nobody's."""
    b = Batch([0, 0, 0], [30, 0, 7], 8, 2, 128, 16, dtype, DEV, seed=22, pad_rows=4)
    O, lse, flag = b.run(max_q=max_q)
    assert _flag(flag) == 0 and (O == 7).all() and (lse == 7).all()
    b = Batch([1, 1], [30, 70], 8, 2, 128, 16, dtype, DEV, seed=22, pad_rows=2)
    b.Q = torch.cat([b.Q[2:], b.Q[:2]]).contiguous()
    b.q_off += 2
    O, lse, flag = b.run(max_q=max_q)
    assert _flag(flag) == 0 and (O[:2] == 7).all()
    b.Q, b.q_off = torch.cat([b.Q[2:], b.Q[:2]]), b.q_off - 2
    b.check(torch.cat([O[2:], O[:2]]), torch.cat([lse[:, 2:], lse[:, :2]], 1))


def test_without_lse():
    for q_len in ([1, 1], [40, 3]):
        b = Batch(q_len, [300, 40], 8, 2, 128, 16, BF, DEV, seed=23)
        O, none, flag = b.run(want_lse=False)
        assert none is None and _flag(flag) == 0
        b.check(O, None)


def test_a_key_selected_twice():
    """A document selected twice counts twice, as in msa_sparse_attn_indexed."""
    b = Batch([1, 60], [30, 90], 8, 2, 128, 16, BF, DEV, seed=24).select(3, 10, 5, seed=1)
    b.idx[:, 2] = b.idx[:, 0]
    O, lse, flag = b.run(30)
    assert _flag(flag) == 0
    b.check(O, lse, 30)


def test_launches_are_counted():
    b = Batch([1, 1], [40, 30], 8, 2, 128, 16, BF, DEV, seed=17)
    n = msa.kernel_launch_count()
    b.run()
    assert msa.kernel_launch_count() - n == 2  # the attention and the merge
    b.select(2, 5, 4)
    n = msa.kernel_launch_count()
    b.run(10)
    assert msa.kernel_launch_count() - n == 3  # and the plan of the selection


def test_cache_past_2_to_31_elements():
    """Byte and element offsets past 32 bits: pages at the end of a 6.4 GB pool."""
    page, Hkv, d = 256, 8, 128
    P = 2 ** 31 // (page * Hkv * d) + 2000
    b = Batch([1, 40], [600, 700], 32, Hkv, d, page, BF, DEV, seed=18)
    K = torch.zeros((P, page, Hkv, d), dtype=BF, device=DEV)
    V = torch.zeros_like(K)
    K[P - b.P:], V[P - b.P:] = b.K, b.V
    b.K, b.V = K, V
    b.table = torch.where(b.table < b.P, b.table + (P - b.P), b.table)
    for max_q in (40, 64):
        O, lse, flag = b.run(max_q=max_q)
        assert _flag(flag) == 0
        b.check(O, lse)
    one = Batch([1, 1], [600, 700], 32, Hkv, d, page, BF, DEV, seed=18)
    K[P - one.P:], V[P - one.P:] = one.K, one.V
    one.K, one.V = K, V
    one.table = torch.where(one.table < one.P, one.table + (P - one.P), one.table)
    O, lse, flag = one.run()
    assert _flag(flag) == 0
    one.check(O, lse)
