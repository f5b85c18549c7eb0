"""msa_paged_attn and msa_paged_append over caches of other strides, and over tables, lengths and
offsets that do not fit."""
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
