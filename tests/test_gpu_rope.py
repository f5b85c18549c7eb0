"""msa_rope, msa_rope_backward and msa_paged_append against their formulas in fp64, the gradient
against differences as well, and a serving loop that uses them with msa_paged_attn."""
import pytest
import torch

import routed_sparse_attention_chunk_b200 as msa

from .paged_helpers import Batch, HALF_STEP, rotate64, rotation_bound

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
LAYOUTS = [msa.ROPE_HALF, msa.ROPE_INTERLEAVED]


def _table(rd, n, method="none", **kw):
    return msa.rope_table_scaled(method, 1e6, rd, n, **kw).to(DEV)


def _randn(*shape, dtype, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N,H,d,rd", [(1, 1, 64, 64), (1, 40, 128, 128), (7, 3, 128, 32), (333, 10, 64, 16),
                                      (50, 5, 256, 64), (9, 2, 48, 48), (1000, 40, 128, 96)])
def test_rotation_and_its_adjoint(layout, dtype, N, H, d, rd):
    x = _randn(N, H, d, dtype=dtype)
    cs = _table(rd, 4000, "yarn", factor=4.0, orig_len=1000, lo=1, hi=32)
    pos = torch.randint(0, 4000, (N,), generator=torch.Generator().manual_seed(1)).to(torch.int32).to(DEV)
    pos[0] = 3999
    rows = cs[pos.long()]
    inter = layout == msa.ROPE_INTERLEAVED
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    for f, transpose in ((msa.rope, False), (msa.rope_backward, True)):
        y = torch.full_like(x, float("nan"))
        f(x, pos, cs, y, layout=layout, err_flag=flag)
        want = rotate64(x, rows, inter, transpose)
        assert ((y.double() - want).abs() <= rotation_bound(x, rows, dtype, inter)).all()
        assert torch.equal(y[..., rd:], x[..., rd:])
        z = x.clone()
        f(z, pos, cs, z, layout=layout, err_flag=flag)  # in place
        assert torch.equal(z, y)
    assert flag.item() == 0


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", [F32, BF])
def test_strided_views(layout, dtype):
    """Heads of a fused projection in, [head, token] rows out; other heads and rows untouched."""
    N, H, d = 37, 6, 64
    qkv = _randn(N, H + 5, d, dtype=dtype, seed=2)
    x = qkv[:, 2:2 + H]
    out = torch.full((H, N + 2, d), 9.0, dtype=dtype, device=DEV)
    y = out.transpose(0, 1)[1:1 + N]
    cs = _table(32, 64)
    pos = torch.arange(N, dtype=torch.int32, device=DEV)
    msa.rope(x, pos, cs, y, layout=layout)
    ref = torch.empty((N, H, d), dtype=dtype, device=DEV)
    msa.rope(x.contiguous(), pos, cs, ref, layout=layout)
    assert torch.equal(y, ref)
    assert (out[:, 0] == 9).all() and (out[:, -1] == 9).all()
    before = qkv.clone()
    msa.rope(x, pos, cs, x, layout=layout)  # in place inside the projection
    assert torch.equal(x, ref) and torch.equal(qkv[:, :2], before[:, :2]) and torch.equal(qkv[:, 8:], before[:, 8:])


def test_broadcast_input():
    """One head's row read for all heads, and its gradient: the sum over the heads."""
    N, H, d = 20, 4, 64
    one = _randn(N, 1, d, dtype=F32, seed=3)
    cs, pos = _table(64, 32), torch.arange(N, dtype=torch.int32, device=DEV)
    y = torch.empty((N, H, d), device=DEV)
    msa.rope(one.expand(N, H, d), pos, cs, y)
    want = rotate64(one, cs[pos.long()])
    assert ((y.double() - want).abs() <= rotation_bound(one, cs[pos.long()], F32)).all()


@pytest.mark.parametrize("layout", LAYOUTS)
def test_gradient_against_differences(layout):
    """<w, rope(x + e u) - rope(x - e u)> / 2e = <rope_backward(w), u>: the map is linear, so the
    difference has no truncation error and e = 1/4 keeps its rounding at a few 2^-24 of the sums."""
    N, H, d, rd = 11, 3, 64, 32
    x, u, w = (_randn(N, H, d, dtype=F32, seed=s) for s in (4, 5, 6))
    cs, pos = _table(rd, 100, "linear", factor=2.0), torch.arange(N, dtype=torch.int32, device=DEV) * 9
    out = [torch.empty_like(x) for _ in range(3)]
    msa.rope(x + 0.25 * u, pos, cs, out[0], layout=layout)
    msa.rope(x - 0.25 * u, pos, cs, out[1], layout=layout)
    msa.rope_backward(w, pos, cs, out[2], layout=layout)
    num = ((out[0].double() - out[1].double()) * 2 * w.double()).sum()
    ana = (out[2].double() * u.double()).sum()
    # each of the N H d terms: two rotations (4 roundings of |x| + |u|/4 sums) times 2 |w|, and dx's own
    scale = float(((x.abs() + u.abs()) * w.abs()).double().sum())
    assert abs(float(num - ana)) <= 32 * 2.0 ** -24 * scale


def test_rows_with_positions_outside_the_table():
    x = _randn(6, 2, 64, dtype=BF)
    cs = _table(64, 10)
    pos = torch.tensor([0, -1, 9, 10, 2 ** 31 - 1, 5], dtype=torch.int32, device=DEV)
    y = torch.full_like(x, 3.0)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    msa.rope(x, pos, cs, y, err_flag=flag)
    assert flag.item() == msa.FLAG_INDEX_OOB
    good = [0, 2, 5]
    assert (y[[1, 3, 4]] == 3).all()
    rows = cs[pos[good].long()]
    assert ((y[good].double() - rotate64(x[good], rows)).abs() <= rotation_bound(x[good], rows, BF)).all()
    msa.rope(x[:0], pos[:0], cs, y[:0])  # no tokens: nothing launched


def test_training_step_in_a_graph_beside_eager_work():
    """Forward and backward captured together and replayed while eager gradients of the same
    tensors are alive."""
    x, w = _randn(64, 8, 128, dtype=BF, seed=7), _randn(64, 8, 128, dtype=BF, seed=8)
    cs, pos = _table(128, 64), torch.arange(64, dtype=torch.int32, device=DEV)
    y, dx, ye, dxe = (torch.empty_like(x) for _ in range(4))
    msa.rope(x, pos, cs, ye)
    msa.rope_backward(w, pos, cs, dxe)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        msa.rope(x, pos, cs, y)
        msa.rope_backward(w, pos, cs, dx)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, ye) and torch.equal(dx, dxe)


def _append_ref(b, q, k, v, pos, cs, inter):
    K, V = b.K.double(), b.V.double()
    rows = cs[pos]
    kr = rotate64(k, rows, inter)
    bound = rotation_bound(k, rows, k.dtype, inter)
    BK = torch.zeros_like(K)
    for i, n in enumerate(b.q_len):
        sl = slice(b.off[i], b.off[i] + n)
        pg, row = b.slots(i, torch.arange(b.total[i] - n, b.total[i]))
        K[pg, row], V[pg, row], BK[pg, row] = kr[sl], v[sl].double(), bound[sl]
    return K, V, BK, rotate64(q, rows, inter), rotation_bound(q, rows, q.dtype, inter)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("q_len,total,d,page,order,rd", [
    ([1], [1], 64, 8, "prhd", 64), ([1] * 5, [1, 16, 17, 32, 300], 128, 16, "prhd", 128),
    ([5, 0, 40, 1], [5, 9, 100, 128], 128, 32, "phrd", 32), ([300, 2], [300, 257], 64, 256, "pair", 16),
    ([7, 7], [7, 8], 128, 8, "prhd", 96)])
def test_append(layout, dtype, q_len, total, d, page, order, rd):
    Hq, Hkv = 6, 2
    b = Batch(q_len, total, Hq, Hkv, d, page, dtype, DEV, seed=9, order=order, pad_rows=2)
    qkv = _randn(b.rows, Hq + 2 * Hkv, d, dtype=dtype, seed=10)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    cs = _table(rd, 400)
    N = b.N
    at = torch.cat([torch.arange(t - n, t) for n, t in zip(q_len, total)]).to(DEV)
    inter = layout == msa.ROPE_INTERLEAVED
    K0, V0 = b.K.clone(), b.V.clone()
    Kw, Vw, BK, qw, bq = _append_ref(b, q[:N], k[:N], v[:N], at, cs, inter)
    q_out = torch.full((b.rows, Hq, d), 5.0, dtype=dtype, device=DEV)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    msa.paged_append(q, k, v, b.q_off, b.seq_len, b.table, b.K, b.V, rope_cs=cs, q_out=q_out, layout=layout,
                     err_flag=flag)
    assert flag.item() == 0
    same = lambda x, y: ((x == y) | (x.isnan() & y.isnan())).all()  # noqa: E731
    hit = BK > 0
    assert ((b.K.double() - Kw).abs() <= BK)[hit].all()
    assert same(b.K.double()[~hit], Kw[~hit]) and same(b.V.double(), Vw)
    assert ((q_out[:N].double() - qw).abs() <= bq).all() and (q_out[N:] == 5).all()

    # without a rotation, and without queries: copies
    b.K.copy_(K0)
    b.V.copy_(V0)
    msa.paged_append(None, k, v, b.q_off, b.seq_len, b.table, b.K, b.V, err_flag=flag)
    for i, n in enumerate(q_len):
        pg, row = b.slots(i, torch.arange(total[i] - n, total[i]))
        assert torch.equal(b.K[pg, row], k[b.off[i]:b.off[i] + n]) and torch.equal(b.V[pg, row], v[b.off[i]:b.off[i] + n])
    # rotary positions of the caller's own
    pos = torch.zeros(b.rows, dtype=torch.int32, device=DEV)
    pos[:N] = 399 - at.to(torch.int32)
    b.K.copy_(K0)
    Kw, _, BK, qw, bq = _append_ref(b, q[:N], k[:N], v[:N], pos[:N].long(), cs, inter)
    msa.paged_append(q, k, v, b.q_off, b.seq_len, b.table, b.K, b.V, rope_cs=cs, q_out=q, pos=pos, layout=layout,
                     err_flag=flag)  # the queries in place
    hit = BK > 0
    assert flag.item() == 0 and ((b.K.double() - Kw).abs() <= BK)[hit].all()
    assert ((q[:N].double() - qw).abs() <= bq).all()


def test_append_skips_and_flags():
    b = Batch([2, 1, 1], [20, 5, 40], 4, 2, 64, 16, BF, DEV, seed=11)
    k = _randn(4, 2, 64, dtype=BF, seed=12)
    def run(cs=None, **kw):
        K0, V0 = b.K.clone(), b.V.clone()
        flag = torch.zeros(1, dtype=torch.int32, device=DEV)
        a = dict(q_off=b.q_off, seq_len=b.seq_len, table=b.table)
        a.update(kw)
        msa.paged_append(None, k, k, a["q_off"], a["seq_len"], a["table"], b.K, b.V, rope_cs=cs, err_flag=flag)
        changed = [i for i in range(4) if not torch.equal(_rows(b, i, b.K), _rows_of(K0, b, i))]
        b.K.copy_(K0)
        b.V.copy_(V0)
        return int(flag.item()), changed

    def _rows_of(K, b, i):
        s = [0, 0, 1, 2][i]
        pg, row = b.slots(s, torch.tensor([b.total[s] - b.q_len[s] + i - b.off[s]]))
        return K[pg, row]

    def _rows(b, i, K):
        return _rows_of(K, b, i)
    assert run() == (0, [0, 1, 2, 3])
    t = b.table.clone()
    t[2, 2] = -1
    assert run(table=t) == (msa.FLAG_INDEX_OOB, [0, 1, 2])
    t[2, 2] = b.P
    assert run(table=t) == (msa.FLAG_INDEX_OOB, [0, 1, 2])
    assert run(cs=_table(64, 19)) == (msa.FLAG_INDEX_OOB, [0, 2])  # positions 19 and 39 are past the table
    s = b.seq_len.clone()
    s[0] = 1  # its first token would sit before position 0
    f, c = run(seq_len=s)
    assert f == msa.FLAG_OFFSETS and 3 in c and 2 in c
    s[0] = 10 ** 6  # past the block table
    f, c = run(seq_len=s)
    assert f == msa.FLAG_INDEX_OOB and c == [2, 3]
    o = b.q_off.clone()
    o[3] = 9
    assert run(q_off=o)[0] == msa.FLAG_OFFSETS
    o = b.q_off + 1
    assert run(q_off=o)[0] == msa.FLAG_OFFSETS  # its last sequence passes the packed rows
    o = b.q_off.clone()
    o[1] = 4  # decreasing after it
    assert run(q_off=o)[0] & msa.FLAG_OFFSETS
    o = torch.tensor([1, 2, 3, 4], device=DEV)  # the first row is nobody's: nothing is wrong
    assert run(q_off=o)[0] == 0


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [64, 128])
def test_serving_loop(dtype, d):
    """Prompts in parts, then single tokens: each step appends (with the rotation) and attends over
    the selected documents and the cache; against fp64 attention over the keys and values the
    library itself stored, step by step, and the stored rows against the rotated projections."""
    Hq, Hkv, page, k = 8, 2, 16, 3
    steps = [[37, 5, 0], [20, 1, 70], [1, 1, 1], [1, 1, 1], [3, 0, 1]]
    B, width = 3, 12
    P = B * width + 2
    K = torch.full((P, page, Hkv, d), float("nan"), dtype=dtype, device=DEV)
    V = torch.full_like(K, float("nan"))
    table = torch.randperm(P, generator=torch.Generator().manual_seed(3))[:B * width].view(B, width).to(torch.int32).to(DEV)
    cs = _table(d, width * page, "ntk", factor=2.0)
    done = [0] * B
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    raw = [[] for _ in range(B)]
    bank = Batch([1] * B, [1] * B, Hq, Hkv, d, page, dtype, DEV, seed=20).select(k, 12, 9, seed=5)
    for t, q_len in enumerate(steps):
        N = sum(q_len)
        qkv = _randn(N, Hq + 2 * Hkv, d, dtype=dtype, seed=30 + t) * 0.5
        q, kk, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        done = [a + n for a, n in zip(done, q_len)]
        off = torch.tensor([0] + list(torch.tensor(q_len).cumsum(0)), dtype=torch.int64, device=DEV)
        seq_len = torch.tensor(done, dtype=torch.int32, device=DEV)
        q_out = torch.empty((N, Hq, d), dtype=dtype, device=DEV)
        msa.paged_append(q, kk, v, off, seq_len, table, K, V, rope_cs=cs, q_out=q_out, err_flag=flag)
        b = Batch.__new__(Batch)
        b.__dict__.update(q_len=q_len, total=list(done), page=page, dtype=dtype, device=DEV, Hq=Hq, Hkv=Hkv, d=d, N=N,
                          rows=N, off=off.tolist(), q_off=off, seq_len=seq_len, max_q=max(q_len), table=table, K=K,
                          V=V, Q=q_out, idx=bank.idx, chunk_off=bank.chunk_off, Kbar=bank.Kbar, Vbar=bank.Vbar, k=k)
        O, lse, _ = b.run(20, flag=flag)
        b.kd, b.vd = [], []
        for i in range(B):
            raw[i].append((kk[b.off[i]:b.off[i + 1]], v[b.off[i]:b.off[i + 1]]))
            pg, row = b.slots(i, torch.arange(done[i]))
            b.kd.append(K[pg, row])
            b.vd.append(V[pg, row])
            want = torch.cat([x for x, _ in raw[i]])
            assert ((b.kd[i].double() - rotate64(want, cs[:done[i]])).abs() <= rotation_bound(want, cs[:done[i]], dtype)).all()
            assert torch.equal(b.vd[i], torch.cat([x for _, x in raw[i]]))
        assert int(flag.item()) in (0, msa.FLAG_OVERFLOW)
        b.check(O, lse, 20)
