"""Refusals of the paged pool's operators and of the sampler, without a GPU:
every call here fails its checks before the library touches CUDA, and the
pure-host answers (sizes) are the layout's."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import outlier_split_bit_b200 as sp
from outlier_split_bit_b200 import _lib
from outlier_split_bit_b200 import build as libbuild

import serving_reference as ref

FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return _lib.load()


def _pool(H=2, D=128, P=16, n=8, mass=FAKE, **other):
    f = dict(k_codes=FAKE, k_scales=FAKE, k_zeros=FAKE, v_codes=FAKE, v_scales=FAKE, v_zeros=FAKE, mass=mass)
    f.update(other)
    return _lib.KVPool(H, D, P, n, *f.values())


def test_pool_sizes(L):
    got = [ctypes.c_size_t() for _ in range(4)]
    r = [ctypes.byref(g) for g in got]
    assert L.spectra_kv_pool_sizes(3, 96, 32, 7, *r) == _lib.OK
    slots = 3 * 32 * 7
    assert [g.value for g in got] == [slots * 48, slots * 6, slots * 4, slots * 4]
    for bad in [(0, 96, 32, 7), (3, 100, 32, 7), (3, 288, 32, 7), (3, 0, 32, 7), (3, 96, 24, 7), (3, 96, 8, 7),
                (3, 96, 2048, 7), (3, 96, 32, 0), (1, 32, 1024, 1 << 21)]:
        assert L.spectra_kv_pool_sizes(*bad, *r) == _lib.ERR_SHAPE, bad
    assert L.spectra_kv_pool_sizes(3, 96, 32, 7, None, *r[1:]) == _lib.ERR_INVALID_ARG


def test_append_refusals(L):
    def call(pool=None, k=FAKE, v=FAKE, n=4, ks=256, vs=256, slots=FAKE):
        return L.spectra_kv_pool_append(ctypes.byref(pool if pool is not None else _pool()), k, v, n, ks, vs, slots,
                                        None)

    assert call(n=0, k=None, slots=None) == _lib.OK
    assert call(n=-1) == _lib.ERR_INVALID_ARG
    assert call(k=None) == call(v=None) == call(slots=None) == _lib.ERR_INVALID_ARG
    assert call(ks=255) == call(vs=248) == call(ks=-256) == _lib.ERR_SHAPE
    assert call(ks=260) == call(k=FAKE + 8) == call(v=FAKE + 2) == call(slots=FAKE + 2) == _lib.ERR_ALIGN
    assert call(n=1 << 30) == _lib.ERR_SHAPE
    assert call(_pool(P=48)) == call(_pool(D=48)) == call(_pool(H=0)) == call(_pool(n=0)) == _lib.ERR_SHAPE
    assert call(_pool(v_zeros=None)) == call(_pool(k_codes=None)) == _lib.ERR_INVALID_ARG
    assert call(_pool(k_scales=FAKE + 8)) == call(_pool(mass=FAKE + 4)) == _lib.ERR_ALIGN
    assert L.spectra_kv_pool_append(None, FAKE, FAKE, 1, 256, 256, FAKE, None) == _lib.ERR_INVALID_ARG


def test_read_refusals(L):
    def call(pool=None, slots=FAKE, n=4, k=FAKE, v=FAKE, dt=1):
        return L.spectra_kv_pool_read(ctypes.byref(pool if pool is not None else _pool()), slots, n, k, v, dt, None)

    assert call(n=0, slots=None) == _lib.OK
    assert call(n=-1) == call(slots=None) == call(k=None, v=None) == call(dt=2) == _lib.ERR_INVALID_ARG
    assert call(k=FAKE + 8) == call(v=FAKE + 4) == call(slots=FAKE + 1) == _lib.ERR_ALIGN
    assert call(_pool(P=0)) == _lib.ERR_SHAPE


def _query(**other):
    f = dict(pages=FAKE, lengths=FAKE, q_start=FAKE, n_seq=3, max_pages=5, n_rows=7, max_q=4, n_q_heads=12, window=0,
             scale=0.1, softcap=0.0, q=FAKE, slopes=None, out=64 * FAKE, out_dtype=1, update_mass=0, lse=None)
    f.update(other)
    return _lib.PagedQuery(*f.values())


def test_attention_refusals(L):
    def call(pool=None, ws=FAKE, wsb=1 << 40, **other):
        return L.spectra_attention_paged(ctypes.byref(pool if pool is not None else _pool()),
                                         ctypes.byref(_query(**other)), ws, wsb, None)

    assert call(n_seq=0) == call(n_rows=0) == _lib.OK
    assert call(n_seq=-1) == call(n_rows=-1) == call(out_dtype=3) == _lib.ERR_INVALID_ARG
    for name in ("pages", "lengths", "q", "out"):
        assert call(**{name: None}) == _lib.ERR_INVALID_ARG, name
    assert call(ws=None) == _lib.ERR_INVALID_ARG
    for name in ("scale", "softcap"):
        assert call(**{name: float("nan")}) == call(**{name: float("inf")}) == _lib.ERR_INVALID_ARG
    assert call(softcap=-1.0) == _lib.ERR_INVALID_ARG
    assert call(_pool(mass=None), update_mass=1) == _lib.ERR_INVALID_ARG
    assert call(n_q_heads=11) == call(n_q_heads=0) == call(n_q_heads=2 * 65) == _lib.ERR_SHAPE
    assert call(window=-1) == call(max_q=0) == call(max_pages=0) == call(n_seq=70000) == _lib.ERR_SHAPE
    assert call(max_pages=(1 << 26) + 1) == call(q_start=None) == call(n_rows=1 << 29) == _lib.ERR_SHAPE
    for name in ("q", "out"):
        assert call(**{name: FAKE + 8}) == _lib.ERR_ALIGN, name
    for name in ("pages", "lengths", "q_start", "slopes", "lse"):
        assert call(**{name: FAKE + 2}) == _lib.ERR_ALIGN, name
    assert call(ws=FAKE + 8) == _lib.ERR_ALIGN
    size = 7 * 12 * 128 * 2
    assert call(out=FAKE) == call(out=FAKE + size - 16) == call(out=FAKE - 2 * size + 16, out_dtype=0) == \
        _lib.ERR_INVALID_ARG  # over q
    need = L.spectra_attention_paged_workspace_size(ctypes.byref(_pool()), 7, 12)
    assert need > 0 and call(wsb=need - 1) == _lib.ERR_BUFFER_TOO_SMALL
    assert L.spectra_attention_paged(None, ctypes.byref(_query()), FAKE, need, None) == _lib.ERR_INVALID_ARG
    assert L.spectra_attention_paged(ctypes.byref(_pool()), None, FAKE, need, None) == _lib.ERR_INVALID_ARG
    for bad in ((None, 7, 12), (ctypes.byref(_pool(D=40)), 7, 12), (ctypes.byref(_pool()), -1, 12),
                (ctypes.byref(_pool()), 7, 13)):
        assert L.spectra_attention_paged_workspace_size(*bad) == 0


def test_evict_refusals(L):
    def call(pool=None, pages=FAKE, mp=9, lengths=FAKE, n=3, dst=FAKE, dmp=4, budget=50, recent=8, new=2 * FAKE, ws=FAKE,
             wsb=1 << 40):
        return L.spectra_kv_evict(ctypes.byref(pool if pool is not None else _pool()), pages, mp, lengths, n, dst, dmp,
                                  budget, recent, new, ws, wsb, None)

    assert call(n=0) == _lib.OK
    assert call(n=-1) == call(_pool(mass=None)) == _lib.ERR_INVALID_ARG
    assert call(pages=None) == call(lengths=None) == call(dst=None) == call(new=None) == _lib.ERR_INVALID_ARG
    assert call(ws=None) == _lib.ERR_INVALID_ARG
    assert call(new=FAKE) == call(new=FAKE + 8) == call(new=FAKE - 8) == _lib.ERR_INVALID_ARG  # overlaps lengths
    assert call(budget=0) == call(recent=-1) == call(recent=51) == call(dmp=3) == call(mp=0) == _lib.ERR_SHAPE
    assert call(dmp=0) == call(n=70000) == call(mp=(1 << 26) + 1) == _lib.ERR_SHAPE
    assert call(pages=FAKE + 2) == call(dst=FAKE + 1) == call(ws=FAKE + 4) == call(new=2 * FAKE + 2) == _lib.ERR_ALIGN
    need = L.spectra_kv_evict_workspace_size(ctypes.byref(_pool()), 3, 9, 50)
    assert need > 0 and call(wsb=need - 1) == _lib.ERR_BUFFER_TOO_SMALL
    assert L.spectra_kv_evict_workspace_size(ctypes.byref(_pool()), 3, 0, 50) == 0
    assert L.spectra_kv_evict_workspace_size(ctypes.byref(_pool()), 3, 9, 0) == 0


def test_sample_refusals(L):
    def call(x=FAKE, rows=2, vocab=1000, stride=1000, u=FAKE, t=None, k=None, p=None, m=None, ids=FAKE, lp=None):
        return L.spectra_sample(x, rows, vocab, stride, u, t, k, p, m, ids, lp, None)

    assert call(rows=0, x=None) == _lib.OK
    assert call(x=None) == call(u=None) == call(ids=None) == _lib.ERR_INVALID_ARG
    assert call(rows=-1) == call(vocab=0) == call(vocab=524289, stride=600000) == call(stride=999) == _lib.ERR_SHAPE
    assert call(x=FAKE + 2) == call(t=FAKE + 1) == call(k=FAKE + 2) == call(lp=FAKE + 3) == _lib.ERR_ALIGN


def test_binding_refuses_wrong_tensors():
    """Types, shapes, strides and host tensors are refused by name before a call."""
    with pytest.raises(ValueError, match="codes"):
        z = torch.zeros
        sp.KVPool.from_buffers(1, 32, 16, 1, z(256, dtype=torch.uint8), z(16, dtype=torch.int16),
                               z(16, dtype=torch.int32), z(256, dtype=torch.uint8), z(16, dtype=torch.int16),
                               z(16, dtype=torch.int32))
    with pytest.raises(sp.SpectraError):
        sp.KVPool.sizes(1, 33, 16, 1)
    with pytest.raises(ValueError, match="logits"):
        sp.spectra_sample(torch.zeros(2, 5), torch.zeros(2))


# ---------------------------------------------------------------- the reference itself

def test_reference_layout_by_hand():
    """One vector's words, by the layout's formulas, on one channel at a time."""
    p = ref.Pool(2, 64, 16, 3)
    for which, bits in (("k", 32), ("v", 16)):
        for ch in (0, 7, 8, 31, 32, 45, 63):
            codes = np.zeros(64, np.uint8)
            codes[ch] = 9
            p.put(which, 37, 1, codes, np.array([0x3C00, 0x4000], np.uint16), [3, 5])
            slot = (37 // 16 * 2 + 1) * 16 + 37 % 16
            g, c = ch // 32, ch % 32
            words = p.codes[which].view(np.uint32 if bits == 32 else np.uint16).ravel()
            per = bits // 4  # channels of a word
            want = slot * (64 // per) + c // per * 2 + g
            assert np.flatnonzero(words).tolist() == [want] and words[want] == 9 << (4 * (c % per))
            value = np.repeat([-3.0 * 1.0, -5.0 * 2.0], 32)
            value[ch] += 9 * (1.0, 2.0)[g]
            assert np.array_equal(p.value(which, 37, 1), value)
            assert p.zeros[which][slot] == 3 | 5 << 4
        p.codes[which][:] = 0


def test_reference_sample_by_hand():
    x = np.log(np.array([1.0, 4.0, 2.0, 1.0]))
    assert [ref.sample(x, u)[0] for u in (0.0, 0.12, 0.13, 0.62, 0.63, 0.87, 0.88)] == [0, 0, 1, 1, 2, 2, 3]
    assert [ref.sample(x, u, top_k=2)[0] for u in (0.0, 0.66, 0.67)] == [1, 1, 2]
    assert [ref.sample(x, 0.999, top_k=3)[0], ref.sample(x, 0.0, top_k=3)[0]] == [2, 0]  # the tie's lower index stays
    assert ref.sample(x, 0.99, top_p=0.49)[0] == 1 and ref.sample(x, 0.99, top_p=0.51)[0] == 2
    assert ref.sample(x, 0.99, min_p=0.3)[0] == 2 and ref.sample(x, 0.99, min_p=0.6)[0] == 1
    assert ref.sample(x, 0.99, temperature=0.0)[0] == 1
    assert ref.sample(np.array([-np.inf, np.nan]), 0.5)[0] == -1


def test_reference_attention_is_the_oracles():
    """The paged form of one sequence, one token, is the oracle's decode attention."""
    rng = np.random.default_rng(3)
    H, D, P, T = 2, 64, 16, 37
    cache = {w: oracle.kv_cache(H, T, D) for w in "kv"}
    p = ref.Pool(H, D, P, 5, rng)
    pages = [[4, 0, 2]]
    bits = {}
    for w in "kv":
        x = rng.standard_normal((T, H, D)).astype(np.float32)
        bits[w] = (x.view(np.uint32) >> 16).astype(np.uint16)
        oracle.kv_quantize(cache[w], bits[w], 0)
    p.append(bits["k"], bits["v"], [pages[0][t // P] * P + t % P for t in range(T)])
    q = (rng.standard_normal((1, 4, D)).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    want, _, _ = oracle.attention(cache["k"], cache["v"], q[0], T, 0.125)
    q64 = (q.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    out, lse, add, *_ = ref.attention(p, pages, [T], q64, [0, 1], 0.125)
    assert np.allclose(out[0], want, rtol=1e-12, atol=1e-12)
    assert np.isclose(add.sum(), 4.0) and np.isfinite(lse).all()


def test_fp32_quotient_rounds_like_the_double_one():
    """The append's codes use rint of an FP32 quotient where the definition has
    a double one; equal for every BF16 numerator and FP16 scale whose quotient
    can occur (at most 15 * 2^9 in magnitude), on a sample of 2^8 scales."""
    rng = np.random.default_rng(5)
    v = (np.arange(1 << 16, dtype=np.uint32) << 16).view(np.float32)
    v = v[np.isfinite(v)]
    scales = np.unique(np.concatenate([rng.integers(1, 0x7C00, 200), [1, 2, 3, 5, 0x3FF, 0x400, 0x401, 0x7BFF],
                                       rng.integers(1, 0x400, 48)])).astype(np.uint16)
    for s in scales.view(np.float16):
        S = np.float32(s)
        x = v[np.abs(v.astype(np.float64)) <= 15 * 2.0 ** 9 * float(S)]
        with np.errstate(under="ignore"):
            assert np.array_equal(np.rint(x / S).astype(np.float64), np.rint(x.astype(np.float64) / float(S)))
