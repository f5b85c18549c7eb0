"""Rotary positions and the paged cache without a GPU: the scaled tables against their formulas, and
the refusals of the C entry points and of the binding (nothing is launched)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import routed_sparse_attention_chunk_b200 as msa
from routed_sparse_attention_chunk_b200 import _lib

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
FAKE = 0x10000  # 16-byte aligned, never dereferenced


def _freqs(method, theta, rd, factor, orig, lo, hi):
    i = np.arange(rd // 2, dtype=np.float64)
    f = theta ** (-2 * i / rd)
    if method == "linear":
        return f / factor, 1.0
    if method == "ntk":
        return (theta * factor ** (rd / (rd - 2))) ** (-2 * i / rd), 1.0
    if method == "bands":
        s = np.clip((orig * f / (2 * math.pi) - lo) / (hi - lo), 0, 1)
        return f * s + f / factor * (1 - s), 1.0
    if method == "yarn":
        x = lambda r: rd * math.log(orig / (2 * math.pi * r)) / (2 * math.log(theta))  # noqa: E731
        a, b = max(math.floor(x(hi)), 0), min(math.ceil(x(lo)), rd - 1)
        if b <= a:
            b = a + 0.001
        t = np.clip((i - a) / (b - a), 0, 1)
        return f * (1 - t) + f / factor * t, 0.1 * math.log(factor) + 1
    return f, 1.0


@pytest.mark.parametrize("rd,theta", [(16, 1e4), (64, 1e6), (128, 5e5)])
@pytest.mark.parametrize("method,factor,orig,lo,hi", [
    ("none", 1.0, 0, 0, 0), ("linear", 4.0, 0, 0, 0), ("ntk", 8.0, 0, 0, 0), ("yarn", 4.0, 4096, 1, 32),
    ("yarn", 1.0, 4096, 1, 32), ("yarn", 16.0, 10, 1, 32), ("bands", 8.0, 8192, 1, 4)])
def test_scaled_tables(rd, theta, method, factor, orig, lo, hi):
    n = 700
    t = msa.rope_table_scaled(method, theta, rd, n, factor, orig, lo, hi).numpy()
    f, mag = _freqs(method, theta, rd, factor, orig, lo, hi)
    ang = np.arange(n)[:, None] * f
    # one rounding to fp32 of values up to mag (a half step of at most 2^-24 mag), and fp64's own on
    # angles up to 700 (a few 1e-13)
    tol = 2.0 ** -24 * mag + 1e-12
    assert np.abs(t[..., 0] - mag * np.cos(ang)).max() <= tol
    assert np.abs(t[..., 1] - mag * np.sin(ang)).max() <= tol


def test_unscaled_table_is_the_pool_s():
    assert torch.equal(msa.rope_table_scaled("none", 1e6, 128, 300), msa.rope_table(1e6, 128, 300))


def test_far_positions_keep_their_angle():
    n = 200_001
    t = msa.rope_table_scaled("linear", 1e4, 16, n, factor=2.0).numpy()
    ang = (n - 1) * (1e4 ** (-2 * np.arange(8) / 16)) / 2.0
    assert np.abs(t[-1, :, 0] - np.cos(ang)).max() <= 2.0 ** -24 + 1e-10


def test_table_refusals():
    buf = (ctypes.c_float * 64)()

    def call(method=0, theta=1e4, rd=16, n=2, factor=2.0, orig=100.0, lo=1.0, hi=4.0, out=buf):
        return _lib.load().msa_rope_table_scaled_host(method, theta, rd, n, factor, orig, lo, hi, out)
    for m in range(5):
        assert call(method=m) == OK
    for bad in (dict(method=5), dict(method=-1), dict(theta=0.0), dict(theta=float("nan")), dict(rd=15), dict(rd=0),
                dict(n=0), dict(out=None), dict(method=1, factor=0.5), dict(method=1, factor=float("inf")),
                dict(method=2, factor=float("nan")), dict(method=2, rd=2), dict(method=3, orig=0.0),
                dict(method=3, lo=4.0), dict(method=3, theta=1.0), dict(method=4, lo=0.0), dict(method=4, hi=1.0)):
        assert call(**bad) == INVALID, bad
    assert call(method=0, factor=0.0) == OK  # read by the scaled methods only
    with pytest.raises(ValueError):
        msa.rope_table_scaled("other", 1e4, 16, 2)
    with pytest.raises(msa.MSAError):
        msa.rope_table_scaled("linear", 1e4, 16, 2, factor=0.0)


def _rope(fn="msa_rope", **kw):
    a = dict(dt=1, x=FAKE, xt=512, xh=64, N=3, H=8, d=64, pos=FAKE, cs=FAKE, max_len=10, rd=64, layout=0,
             out=FAKE + 1024, ot=512, oh=64, flag=None)
    a.update(kw)
    return getattr(_lib.load(), fn)(*a.values(), None)


@pytest.mark.parametrize("fn", ["msa_rope", "msa_rope_backward"])
def test_rope_refusals(fn):
    assert _rope(fn, N=0, x=None, out=None, pos=None) == OK  # no tokens: nothing launched
    for bad in (dict(dt=2), dict(N=-1), dict(N=1 << 31), dict(H=0), dict(x=None), dict(pos=None), dict(cs=None),
                dict(out=None), dict(x=FAKE + 2), dict(out=FAKE + 8), dict(cs=FAKE + 4), dict(max_len=0), dict(rd=0),
                dict(rd=80), dict(rd=15), dict(layout=2), dict(xt=-8), dict(xt=511), dict(xh=60), dict(ot=4),
                dict(N=5, ot=0), dict(N=5, ot=256), dict(N=5, oh=32), dict(N=5, out=FAKE, xt=1024),
                dict(N=5, out=FAKE, xh=128, xt=1024, ot=1024)):
        assert _rope(fn, **bad) == INVALID, bad
    for bad in (dict(d=72, rd=16), dict(d=2048, xh=2048, xt=1 << 14, oh=2048, ot=1 << 14), dict(rd=24), dict(rd=8)):
        assert _rope(fn, **bad) == UNSUPPORTED, bad


CACHE = dict(K=FAKE, V=FAKE, num_pages=9, page=16, ps=16 * 128, rs=128, hs=64, table=FAKE, max_pages=4, seq_len=FAKE)
BAD_CACHE = [dict(K=None), dict(V=None), dict(K=FAKE + 8), dict(num_pages=0), dict(num_pages=0x7fffffff), dict(page=0),
             dict(ps=1000), dict(rs=64), dict(hs=32), dict(hs=65), dict(rs=126), dict(ps=0), dict(table=None),
             dict(max_pages=0), dict(max_pages=1 << 28), dict(seq_len=None), dict(q_off=None), dict(N=-1), dict(B=-1),
             dict(dt=3), dict(Hkv=0)]
UNSUP_CACHE = [dict(page=4, ps=4 * 128), dict(page=12, ps=12 * 128), dict(page=512, ps=512 * 128),
               dict(d=96, hs=96, rs=192, ps=16 * 192)]


def _append(**kw):
    a = dict(dt=1, q=FAKE, qs=256, qo=FAKE + 64, qos=256, Hq=4, k=FAKE, ks=128, v=FAKE, vs=128, N=3, B=3, q_off=FAKE,
             Hkv=2, d=64, pos=None, cs=FAKE, max_len=10, rd=64, layout=0)
    a.update({k: v for k, v in CACHE.items()})
    a["flag"] = None
    a.update(kw)
    return _lib.load().msa_paged_append(*a.values(), None)


def test_append_refusals():
    none = dict(N=0, k=None, v=None, q=None, qo=None)  # no tokens: nothing launched
    assert _append(**none) == OK and _append(B=0) == OK
    assert _append(**none, Hq=0) == OK and _append(**none, cs=None, rd=0, max_len=0) == OK
    assert _append(**none, ps=2 * 16 * 128) == OK            # K beside V in a page
    assert _append(**none, rs=64, hs=16 * 64) == OK          # [head, row] pages
    for bad in BAD_CACHE + [dict(k=None), dict(v=None), dict(k=FAKE + 2), dict(ks=-8), dict(vs=60), dict(Hq=0),
                            dict(qo=None), dict(q=FAKE + 8), dict(qs=12), dict(N=2, qos=128), dict(rd=66),
                            dict(max_len=0), dict(layout=5), dict(N=2, q=FAKE + 64, qs=512)]:
        assert _append(**bad) == INVALID, bad
    for bad in UNSUP_CACHE + [dict(rd=24)]:
        assert _append(**bad) == UNSUPPORTED, bad


def _attn(**kw):
    a = dict(dt=1, Q=FAKE, qs=256, N=3, B=3, max_q=1, q_off=FAKE, Hq=4, Hkv=2, d=64)
    a.update({k: v for k, v in CACHE.items()})
    a.update(idx=FAKE, k=2, off=FAKE, D=5, C=20, Kbar=FAKE, Vbar=FAKE, Mmax=16, scale=0.0, O=FAKE, lse=None, ws=FAKE,
             wsb=1 << 40, flag=None)
    a.update(kw)
    return _lib.load().msa_paged_attn(*a.values(), None)


def test_attention_refusals():
    assert _attn(N=0, Q=None, O=None) == OK and _attn(B=0) == OK
    assert _attn(N=0, k=0, idx=None, off=None, Kbar=None, Vbar=None, D=0) == OK
    for bad in BAD_CACHE + [dict(max_q=0), dict(Hq=0), dict(Hq=3), dict(k=-1), dict(Mmax=-1), dict(Q=None),
                            dict(Q=FAKE + 8), dict(qs=4), dict(O=None), dict(O=FAKE + 2), dict(idx=None),
                            dict(off=None), dict(Kbar=None), dict(Vbar=FAKE + 8), dict(D=0), dict(C=-1)]:
        assert _attn(**bad) == INVALID, bad
    for bad in UNSUP_CACHE + [dict(Hq=130), dict(k=70000)]:
        assert _attn(**bad) == UNSUPPORTED, bad
    assert _attn(N=2, ws=None) == WORKSPACE
    assert _attn(N=2, wsb=100) == WORKSPACE
    assert _attn(N=2, ws=FAKE + 4) == WORKSPACE


def test_workspace_size():
    f = msa.paged_attn_workspace_size
    assert f(torch.bfloat16, 4, 1, 32, 8, 128) > 0
    assert f(torch.bfloat16, 4, 1, 32, 8, 128, 16, 128) > f(torch.bfloat16, 4, 1, 32, 8, 128)
    assert f(torch.bfloat16, 4, 100, 32, 8, 128) > f(torch.bfloat16, 4, 1, 32, 8, 128)
    for bad in (dict(B=-1), dict(max_q=0), dict(Hkv=0), dict(k=-1), dict(Mmax=-1)):
        a = dict(dtype=torch.float32, B=1, max_q=1, Hq=4, Hkv=2, d=64, k=0, Mmax=0)
        a.update(bad)
        assert f(*a.values()) == 0


def test_binding_takes_no_cpu_tensors(device0):
    x, pos, cs = torch.zeros(2, 2, 64), torch.zeros(2, dtype=torch.int32), torch.zeros(4, 32, 2)
    with pytest.raises(ValueError):
        msa.rope(x, pos, cs, torch.zeros_like(x))


class _Fake:
    """What the binding looks at of a CUDA tensor."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.bfloat16, strides=None, device=0):
        self.shape, self.dtype, self._device = torch.Size(shape), dtype, device
        self._st = strides or tuple(int(np.prod(shape[i + 1:])) for i in range(len(shape)))

    def stride(self, i=None):
        return self._st if i is None else self._st[i]

    def dim(self):
        return len(self.shape)

    def numel(self):
        return int(np.prod(self.shape))

    def get_device(self):
        return self._device

    def is_contiguous(self):
        return self._st == tuple(int(np.prod(self.shape[i + 1:])) for i in range(len(self.shape)))

    def data_ptr(self):
        return FAKE

    @property
    def nbytes(self):
        return 2 * self.numel()


@pytest.fixture
def device0(monkeypatch):
    monkeypatch.setattr(msa, "_cuda_dev", lambda: 0)


def test_binding_refusals(device0):
    i32, i64, f32 = torch.int32, torch.int64, torch.float32
    x, pos, cs = _Fake(3, 2, 64), _Fake(3, dtype=i32), _Fake(9, 32, 2, dtype=f32)

    def rope(**kw):
        a = dict(x=x, pos=pos, rope_cs=cs, out=_Fake(3, 2, 64))
        a.update(kw)
        msa.rope(**a)
    for bad in (dict(out=_Fake(3, 2, 32)), dict(pos=_Fake(2, dtype=i32)), dict(rope_cs=_Fake(9, 32, 3, dtype=f32)),
                dict(x=_Fake(3, 2, 64, strides=(128, 1, 2))), dict(out=_Fake(3, 2, 64, device=1)),
                dict(pos=_Fake(3, dtype=i32, strides=(2,)))):
        with pytest.raises(ValueError):
            rope(**bad)
    for bad in (dict(out=_Fake(3, 2, 64, dtype=f32)), dict(pos=_Fake(3, dtype=i64)), dict(x=_Fake(3, 2, 64, dtype=torch.float16)),
                dict(rope_cs=_Fake(9, 32, 2))):
        with pytest.raises(TypeError):
            rope(**bad)

    pages = _Fake(5, 16, 2, 64)
    base = dict(q=_Fake(3, 4, 64), k=x, v=_Fake(3, 2, 64), q_off=_Fake(3, dtype=i64), seq_len=_Fake(2, dtype=i32),
                block_table=_Fake(2, 4, dtype=i32), Kpages=pages, Vpages=_Fake(5, 16, 2, 64), q_out=_Fake(3, 4, 64),
                rope_cs=cs)
    for bad in (dict(v=_Fake(2, 2, 64)), dict(q=_Fake(3, 4, 32)), dict(q_out=None), dict(Kpages=_Fake(5, 16, 4, 64)),
                dict(Vpages=_Fake(5, 16, 2, 64, strides=(4096, 128, 64, 1))), dict(Vpages=_Fake(6, 16, 2, 64)),
                dict(q_off=_Fake(2, dtype=i64)), dict(block_table=_Fake(3, 4, dtype=i32)),
                dict(k=_Fake(3, 2, 64, strides=(256, 128, 1))), dict(pos=_Fake(4, dtype=i32)),
                dict(seq_len=_Fake(2, dtype=i32, device=1))):
        with pytest.raises(ValueError):
            msa.paged_append(**{**base, **bad})
    for bad in (dict(q_off=_Fake(3, dtype=i32)), dict(seq_len=_Fake(2, dtype=i64)), dict(v=_Fake(3, 2, 64, dtype=f32)),
                dict(Kpages=_Fake(5, 16, 2, 64, dtype=f32))):
        with pytest.raises(TypeError):
            msa.paged_append(**{**base, **bad})

    att = dict(Q=_Fake(3, 4, 64), q_off=_Fake(3, dtype=i64), max_q=2, Kpages=pages, Vpages=_Fake(5, 16, 2, 64),
               block_table=_Fake(2, 4, dtype=i32), seq_len=_Fake(2, dtype=i32), O=_Fake(3, 4, 64), ws=_Fake(1 << 20))
    sel = dict(topk_idx=_Fake(2, 3, dtype=i32), doc_chunk_off=_Fake(8, dtype=i64), Kbar=_Fake(20, 2, 64),
               Vbar=_Fake(20, 2, 64), Mmax=8)
    for bad in (dict(O=_Fake(3, 4, 32)), dict(lse=_Fake(3, 4, dtype=f32)), dict(Kpages=_Fake(5, 16, 2, 32)),
                dict(O=_Fake(3, 4, 64, strides=(512, 64, 1))), dict(sel, topk_idx=_Fake(3, 3, dtype=i32)),
                dict(sel, Kbar=_Fake(20, 4, 64)), dict(sel, Vbar=_Fake(19, 2, 64)), dict(ws=_Fake(8, device=1))):
        with pytest.raises(ValueError):
            msa.paged_attn(**{**att, **bad})
