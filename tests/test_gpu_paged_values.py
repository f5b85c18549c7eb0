"""msa_paged_attn where keys and values are not finite: they reach the tokens that see them, and no
bit of any other output."""
import pytest
import torch

from .paged_helpers import Batch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


def _put(b, pages, i, pos, g, x, val):
    pg, row = b.slots(i, torch.tensor([pos]))
    pages[pg, row, g, x] = val


def _same(x, y):
    return bool(((x == y) | (x.isnan() & y.isnan())).all())


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("q_len,total,Hq,Hkv,d,page", [
    ([3, 1, 2], [300, 140, 77], 8, 2, 128, 16),             # few rows, an item a CTA
    ([3, 1, 2], [300, 140, 77], 8, 2, 64, 16),
    ([3, 1, 2, 4], [41000, 900, 20000, 4], 8, 2, 128, 64),  # few rows, items cut by the split
    ([2, 1, 2], [30000, 90, 9000], 8, 2, 64, 64),
    ([70, 30, 9], [200, 30, 300], 8, 2, 128, 16),           # blocks of rows
    ([300, 200, 64], [9000, 200, 700], 16, 4, 128, 32),     # ... cut
    ([150, 30, 290], [6000, 30, 700], 12, 4, 64, 8),
    ([40, 9], [64, 9], 8, 8, 64, 8),                        # one head a group
])
def test_values_touch_only_what_sees_them(dtype, q_len, total, Hq, Hkv, d, page):
    """Infinities and NaN in new tokens' values of the first sequence: the outputs of that dimension
    and KV head from their token on, and bit for bit nothing else."""
    b = Batch(q_len, total, Hq, Hkv, d, page, dtype, DEV, seed=51)
    O1, lse1, _ = b.run()
    b.check(O1, lse1)
    n, t, G = q_len[0], total[0], Hq // Hkv
    first = t - n
    marks = [(t - 1, 0, 3, INF), (t - 1, 1, d - 1, NAN), (first + n // 2, 0, 5, -INF), (first + n // 2, 0, 3, INF),
             (first + 1, 1, 8, INF), (first + n // 3, 1, 8, -INF), (first, 0, 17, INF)]
    hit = {}
    for pos, g, x, val in marks:
        _put(b, b.V, 0, pos, g, x, val)
        hit[(pos, g, x)] = val
    add = torch.zeros(b.N, Hq, d, dtype=torch.float64, device=DEV)
    for (pos, g, x), val in hit.items():
        add[b.off[0] + pos - first:b.off[1], g * G:(g + 1) * G, x] += val  # inf - inf: NaN
    for _ in range(2):
        O2, lse2, flag = b.run()
        assert int(flag.item()) == 0
        assert _same(lse1, lse2)
        odd = ~add.isfinite()
        got = O2[:b.N].double()
        assert _same(got[odd], add[odd])
        assert torch.equal(O2[:b.N][~odd], O1[:b.N][~odd])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("q_len,total,Hq,Hkv,d", [
    ([3, 1, 2], [300, 140, 77], 8, 2, 128), ([200, 30, 9], [700, 30, 300], 8, 2, 128), ([300, 40], [20000, 90], 4, 4, 64),
    ([130, 5], [90, 5], 4, 4, 128)])
def test_a_sequence_without_a_finite_value(dtype, q_len, total, Hq, Hkv, d):
    """All new values of the first sequence are infinite or NaN: its tokens that see one are not finite in
    any dimension, its lse and the other sequences keep their bits."""
    b = Batch(q_len, total, Hq, Hkv, d, 16, dtype, DEV, seed=54)
    O1, lse1, _ = b.run()
    n, t = q_len[0], total[0]
    for val in (INF, NAN):
        pg, row = b.slots(0, torch.arange(max(t - n, 0), t))
        b.V[pg, row] = val
        O2, lse2, flag = b.run()
        assert int(flag.item()) == 0 and torch.equal(lse1, lse2)
        sees = torch.arange(n, device=DEV) + t - n >= 0
        assert not O2[:n][sees].isfinite().any()
        assert torch.equal(O2[n:], O1[n:]) and torch.equal(O2[:n][~sees], O1[:n][~sees])


MINUS_INF = [
    ([3, 2], [300, 140], 128, None, 1), ([3, 2], [300, 140], 64, None, 1), ([3, 2], [300, 140], 128, 60, 1),
    ([2, 1], [700, 200], 128, None, 128), ([2, 1], [700, 200], 64, None, 128), ([2, 1], [700, 200], 128, 60, 128),
    ([1, 1], [20000, 300], 128, None, 300), ([90, 40], [300, 140], 128, None, 128), ([90, 40], [300, 140], 64, None, 1)]


def _minus_infinity(dtype, q_len, total, d, max_q, keys, poison):
    """The first keys of a sequence score -inf: what is left is the softmax over the others, also
    where another sequence of the batch holds a value that is not finite."""
    b = Batch(q_len, total, 8, 2, d, 16, dtype, DEV, seed=52)
    b.Q[:b.N, :, 0] = 1.0
    b.attention64()
    smax = b.smax
    b.kd[0][:keys, :, 0] = -INF
    pg, row = b.slots(0, torch.arange(keys))
    b.K[pg, row] = b.kd[0][:keys]
    want, lo, A = b.attention64()
    b.smax = smax
    bo, bl = b.bounds(want, A, lo, max(total))
    if poison:
        _put(b, b.V, 1, total[1] - 1, 0, 3, INF)
        want[b.off[2] - 1, :4, 3] = INF
    O, lse, flag = b.run(max_q=max_q)
    assert int(flag.item()) == 0
    got, fin = O[:b.N].double(), want.isfinite()
    assert _same(got[~fin], want[~fin])
    assert ((got - want).abs() <= bo)[fin].all()
    assert ((lse[:, :b.N].double() - lo).abs() <= bl).all()


@pytest.mark.parametrize("poison", [False, True])
@pytest.mark.parametrize("q_len,total,d,max_q,keys", MINUS_INF)
def test_keys_of_score_minus_infinity_weigh_nothing(q_len, total, d, max_q, keys, poison):
    _minus_infinity(BF, q_len, total, d, max_q, keys, poison)


@pytest.mark.parametrize("poison", [False, True])
@pytest.mark.parametrize("q_len,total,d,max_q,keys", MINUS_INF)
def test_fp32_keys_of_score_minus_infinity_weigh_nothing(q_len, total, d, max_q, keys, poison):
    _minus_infinity(F32, q_len, total, d, max_q, keys, poison)


HARDLY = [(*c, where) for c in [
    ([1], [300], 128), ([1], [300], 64), ([2], [300], 128), ([4], [300], 128), ([3], [40000], 128), ([70], [300], 128),
    ([70], [300], 64), ([130], [9000], 128)] for where in ("first", "middle", "new", "new_low_first")[:3 + (c[0][0] > 1)]]


def _hardly_weighs(dtype, q_len, total, d, where, val):
    """A weight is above 0 however small it is: a value that is not finite makes the output of its
    dimension not finite, also where the weight is no fp32 number.  lse and the other dimensions hold."""
    b = Batch(q_len, total, 8, 2, d, 16, dtype, DEV, seed=53)
    n, t = q_len[0], total[0]
    pos = {"first": 0, "middle": (t - n) // 2, "new": t - 1 - n // 3, "new_low_first": t - n}[where]
    b.Q[:b.N] = 1.0  # the key of `pos` scores 0, all others 220 nats and more
    b.kd[0] = (b.kd[0].float().abs() + 220.0 / d ** 0.5).to(dtype)
    b.kd[0][pos] = 0
    pg, row = b.slots(0, torch.arange(t))
    b.K[pg, row] = b.kd[0]
    O1, lse1, flag = b.run()
    b.check(O1, lse1)
    _put(b, b.V, 0, pos, 1, 9, val)
    O2, lse2, flag = b.run()
    assert int(flag.item()) == 0 and torch.equal(lse1, lse2)
    sees = torch.arange(n, device=DEV) + t - n >= pos
    assert not O2[:n][sees][:, 4:, 9].isfinite().any()
    O2[:n, 4:, 9] = torch.where(sees[:, None], O1[:n, 4:, 9], O2[:n, 4:, 9])
    assert torch.equal(O1[:n], O2[:n])


@pytest.mark.parametrize("q_len,total,d,where", HARDLY)
@pytest.mark.parametrize("val", [INF, NAN])
def test_a_value_that_hardly_weighs_is_still_seen(q_len, total, d, where, val):
    _hardly_weighs(BF, q_len, total, d, where, val)



@pytest.mark.parametrize("q_len,total,d,where", HARDLY)
@pytest.mark.parametrize("val", [INF, NAN])
def test_fp32_a_value_that_hardly_weighs_is_still_seen(q_len, total, d, where, val):
    _hardly_weighs(F32, q_len, total, d, where, val)
