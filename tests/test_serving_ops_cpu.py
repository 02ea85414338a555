"""Host-side checks of the operators over caller-held caches: every refusal that needs no
device is given before any device work (these addresses are never read)."""
import ctypes

import pytest

A = 1 << 20                                     # an aligned address


@pytest.fixture(scope="module")
def qd():
    import __graft_entry__
    __graft_entry__.build_library()
    import transformer_autoregressive_decode_gb300 as m
    return m


def cache(qd, **kw):
    f = dict(k=A, v=2 * A, k_scale=3 * A, v_scale=4 * A, format=qd.QD_KV_Q8, n_streams=2, n_kv_heads=2, smax=32,
             head_dim=64, stream_stride=2 * 32 * 64, head_stride=32 * 64, row_stride=64, scale_stream_stride=64,
             scale_head_stride=32)
    f.update(kw)
    return qd.qd_kv_cache(*(f[n] for n, _ in qd.qd_kv_cache._fields_))


def _has_device():
    import torch
    return torch.cuda.is_available()


BAD_CACHE = [(dict(k=None), "EINVAL"), (dict(v=None), "EINVAL"), (dict(k_scale=None), "EINVAL"), (dict(v_scale=2), "EINVAL"),
             (dict(k=A + 8), "EINVAL"), (dict(format=2), "EINVAL"), (dict(n_streams=0), "EINVAL"), (dict(smax=0), "EINVAL"),
             (dict(n_kv_heads=0), "EINVAL"), (dict(head_dim=96), "EUNSUPPORTED"), (dict(row_stride=48), "EINVAL"),
             (dict(row_stride=72), "EINVAL"), (dict(head_stride=-64), "EINVAL"), (dict(stream_stride=4104), "EINVAL"),
             (dict(scale_head_stride=-1), "EINVAL"), (dict(format=0, head_stride=4), "EINVAL")]


@pytest.mark.parametrize("kw,want", BAD_CACHE)
def test_bad_caches(qd, kw, want):
    c = cache(qd, **kw)
    at = ctypes.addressof(c)
    want = getattr(qd, "QD_" + want)
    assert qd._lib.qd_kv_append(at, A, A, 0, 1, 64, 64, 64, A, None, None) == want
    assert qd._lib.qd_kv_read(at, A, A, 0, 1, 64, 64, 64, A, None, None) == want
    assert qd._lib.qd_attn_cached(at, None, 0, A, 64, 64, A, 64, 64, 0, 1, 2, 1.0, A, None, 32, None, 0, None) == want
    if "n_streams" in kw or "stream_stride" in kw:
        return                                  # unread for a prefix, or checked with it alike
    good = cache(qd)
    assert qd._lib.qd_attn_cached(ctypes.addressof(good), at, 1, A, 64, 64, A, 64, 64, 0, 1, 2, 1.0, A, None, 32, A,
                                  1 << 20, None) in (want, qd.QD_EINVAL)


ROWS = [dict(k_rows=None), dict(v_rows=None), dict(k_rows=A + 4), dict(dtype=3), dict(n=0), dict(stream=-64), dict(token=6),
        dict(head=2), dict(lengths=None), dict(lengths=A + 1), dict(n_new=A + 2)]


@pytest.mark.parametrize("kw", ROWS)
def test_bad_rows(qd, kw):
    f = dict(k_rows=A, v_rows=A, dtype=1, n=1, stream=64, token=64, head=64, lengths=A, n_new=None)
    f.update(kw)
    c = cache(qd)
    for fn in (qd._lib.qd_kv_append, qd._lib.qd_kv_read):
        assert fn(ctypes.addressof(c), *f.values(), None) == qd.QD_EINVAL


def test_rows_over_each_other(qd):
    """What a call writes must have places of its own; what it only reads may be shared."""
    f = dict(k_rows=A, v_rows=2 * A, dtype=1, n=2, stream=256, token=128, head=64, lengths=A, n_new=None)
    for kw in (dict(v_rows=A), dict(stream=0), dict(token=0), dict(head=0), dict(token=32)):
        assert qd._lib.qd_kv_read(ctypes.addressof(cache(qd)), *dict(f, **kw).values(), None) == qd.QD_EINVAL
    for kw in (dict(stream_stride=0), dict(head_stride=0), dict(v=A), dict(v_scale=3 * A), dict(scale_head_stride=0),
               dict(scale_stream_stride=0)):
        assert qd._lib.qd_kv_append(ctypes.addressof(cache(qd, **kw)), *f.values(), None) == qd.QD_EINVAL
    g = dict(prefix=None, plen=0, q=A, qs=256, qt=128, out=2 * A, os=256, ot=128, dtype=1, n=2, heads=2, scale=1.0, lengths=A,
             n_new=None, most=32, ws=None, wb=0)
    for kw in (dict(out=A), dict(os=0), dict(ot=0), dict(ot=64), dict(os=64)):
        assert qd._lib.qd_attn_cached(ctypes.addressof(cache(qd)), *dict(g, **kw).values(), None) == qd.QD_EINVAL
    if not _has_device():                       # these pass the checks of their arguments
        for kw in (dict(), dict(qs=0), dict(qt=0), dict(qs=0, qt=0)):
            assert qd._lib.qd_attn_cached(ctypes.addressof(cache(qd)), *dict(g, **kw).values(), None) == qd.QD_ECUDA
        for kw in (dict(), dict(v_rows=A), dict(stream=0), dict(head=0)):
            assert qd._lib.qd_kv_append(ctypes.addressof(cache(qd)), *dict(f, **kw).values(), None) == qd.QD_ECUDA
        for kw in (dict(stream_stride=0), dict(head_stride=0), dict(v=A)):
            assert qd._lib.qd_kv_read(ctypes.addressof(cache(qd, **kw)), *f.values(), None) == qd.QD_ECUDA


ATTN = [(dict(q=None), "EINVAL"), (dict(out=None), "EINVAL"), (dict(q=A + 8), "EINVAL"), (dict(qt=4), "EINVAL"), (dict(os=-8), "EINVAL"),
        (dict(dtype=2), "EINVAL"), (dict(n=0), "EINVAL"), (dict(n=65), "EUNSUPPORTED"), (dict(heads=3), "EINVAL"), (dict(heads=0), "EINVAL"),
        (dict(scale=float("nan")), "EINVAL"), (dict(scale=float("inf")), "EINVAL"), (dict(lengths=None), "EINVAL"), (dict(most=0), "EINVAL"),
        (dict(most=33), "EINVAL"), (dict(plen=4), "EINVAL"), (dict(plen=-1), "EINVAL")]


@pytest.mark.parametrize("kw,want", ATTN)
def test_bad_attention(qd, kw, want):
    f = dict(prefix=None, plen=0, q=A, qs=64, qt=64, out=A, os=64, ot=64, dtype=1, n=1, heads=2, scale=1.0, lengths=A,
             n_new=None, most=32, ws=None, wb=0)
    f.update(kw)
    c = cache(qd)
    assert qd._lib.qd_attn_cached(ctypes.addressof(c), *f.values(), None) == getattr(qd, "QD_" + want)


def test_prefix_must_fit_the_cache(qd):
    c = cache(qd)
    for kw, plen in ((dict(n_kv_heads=1), 4), (dict(head_dim=128, row_stride=128), 4), ({}, 33)):
        p = cache(qd, **kw)
        assert qd._lib.qd_attn_cached(ctypes.addressof(c), ctypes.addressof(p), plen, A, 64, 64, A, 64, 64, 1, 1, 2, 1.0, A,
                                      None, 32, A, 1 << 20, None) == qd.QD_EINVAL


@pytest.mark.parametrize("kw,n,want", [({}, dict(T=0), "EINVAL"), ({}, dict(heads=3), "EINVAL"), ({}, dict(heads=1), "EINVAL"),
                                       (dict(head_dim=80), {}, "EUNSUPPORTED"), ({}, dict(T=65), "EUNSUPPORTED"),
                                       ({}, dict(plen=-1), "EINVAL"), ({}, dict(plen=5), "EINVAL"), ({}, dict(dtype=7), "EINVAL"),
                                       ({}, dict(most=33), "EINVAL"), (dict(n_streams=1 << 23), dict(T=8), "EUNSUPPORTED")])
def test_workspace_refusals(qd, kw, n, want):
    f = dict(prefix=None, plen=0, dtype=1, T=1, heads=2, most=32)
    f.update(n)
    c, out = cache(qd, **kw), ctypes.c_size_t(5)
    assert qd._lib.qd_attn_cached_workspace(ctypes.addressof(c), *f.values(), ctypes.byref(out)) == getattr(qd, "QD_" + want)


VERIFY = [dict(p=None), dict(p=A + 2), dict(ids=None), dict(u=None), dict(out=None), dict(acc=None), dict(ps=-1), dict(pr=-1),
          dict(q=A, qs=-1), dict(q=A + 1), dict(nd=A + 3), dict(B=0), dict(T=0), dict(T=65), dict(V=0), dict(V=524289)]


@pytest.mark.parametrize("kw", VERIFY)
def test_bad_verification(qd, kw):
    f = dict(p=A, ps=16, pr=8, q=None, qs=0, qr=0, ids=A, nd=None, u=A, B=1, T=1, V=8, out=A, acc=A)
    f.update(kw)
    assert qd._lib.qd_verify_drafts(*f.values(), None) == qd.QD_EINVAL


def test_scratch_lives_as_long_as_its_address_is_noted(qd):
    """A stream's scratch goes only when another takes its place (no such device: no call finds it)."""
    import gc
    import weakref

    class Memory:
        pass

    ops = qd._setup_ops()
    a, b = Memory(), Memory()
    wa, wb = weakref.ref(a), weakref.ref(b)
    assert ops.keep(99, 7, a, A, 256)
    del a
    gc.collect()
    assert wa() is not None
    assert ops.keep(99, 7, b, 2 * A, 512)
    del b
    gc.collect()
    assert wa() is None and wb() is not None
