"""Refusals of the operators over caller-held caches that need no device: layouts in which a call's writes would lie
over each other, sizes past the kernels' counters, workspaces that are less than they say (these addresses are never read)."""
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
    """2 streams x 3 heads x 32 positions of 64, contiguous, the scales too."""
    f = dict(k=A, v=2 * A, k_scale=3 * A, v_scale=4 * A, format=qd.QD_KV_Q8, n_streams=2, n_kv_heads=3, smax=32,
             head_dim=64, stream_stride=3 * 32 * 64, head_stride=32 * 64, row_stride=64, scale_stream_stride=96,
             scale_head_stride=32)
    f.update(kw)
    return qd.qd_kv_cache(*(f[n] for n, _ in qd.qd_kv_cache._fields_))


@pytest.fixture(scope="module")
def accepted(qd):
    """What a call answers that passed every check of its arguments, where there is no device to go on with."""
    import torch
    if torch.cuda.is_available():
        return None                             # there the made-up addresses are refused next
    return qd.QD_ECUDA


def check(qd, accepted, got, over):
    if over:
        assert got == qd.QD_EINVAL
    elif accepted is not None:
        assert got == accepted


def append(qd, c):
    return qd._lib.qd_kv_append(ctypes.addressof(c), A, A, 0, 1, 192, 192, 64, A, None, None)


# (cache, written over each other?)
LAYOUTS = [
    (dict(), False),
    (dict(head_stride=64), True),                                            # head 1's row j is head 0's row j + 1
    (dict(head_stride=31 * 64), True),                                       # head 1 begins on head 0's last row
    (dict(stream_stride=32 * 64), True),                                     # stream 1 is head 1
    (dict(stream_stride=2 * 32 * 64 + 31 * 64), True),
    (dict(head_stride=64, row_stride=3 * 64), False),                        # positions before heads
    (dict(head_stride=64, row_stride=2 * 64), True),
    (dict(stream_stride=64, head_stride=2 * 64, row_stride=6 * 64), False),  # streams innermost
    (dict(stream_stride=64, head_stride=64, row_stride=6 * 64), True),
    (dict(head_stride=40 * 64, stream_stride=3 * 40 * 64), False),           # spare rows behind every head
    (dict(v=A + 16), True),
    (dict(v=A + 64), True),                                                  # v's row j is k's row j + 1
    (dict(v=A + 64, row_stride=128, head_stride=32 * 128, stream_stride=3 * 32 * 128), False),   # k and v side by side
    (dict(k=A + 64, v=A, row_stride=128, head_stride=32 * 128, stream_stride=3 * 32 * 128), False),
    (dict(v=A + 3 * 32 * 64, stream_stride=2 * 3 * 32 * 64), False),         # [streams, 2, heads, ...]
    (dict(v=A + 2 * 32 * 64, stream_stride=2 * 3 * 32 * 64), True),
    (dict(v=A + 2 * 3 * 32 * 64), False),                                    # right behind
    (dict(v=A + 2 * 3 * 32 * 64 - 16), True),
    (dict(scale_head_stride=1), True),
    (dict(scale_head_stride=31), True),
    (dict(scale_stream_stride=1), True),
    (dict(scale_stream_stride=95), True),
    (dict(scale_stream_stride=32, scale_head_stride=64), False),
    (dict(v_scale=3 * A + 4), True),
    (dict(v_scale=3 * A + 192 * 4), False),
    (dict(v_scale=3 * A + 191 * 4), True),
    (dict(v_scale=3 * A + 32 * 4, scale_head_stride=64, scale_stream_stride=192), False),
    (dict(k_scale=None, v_scale=None, format=0, k=A, v=A + 2 * 2 * 3 * 32 * 64), False),
    (dict(k_scale=None, v_scale=None, format=0, k=A, v=A + 2 * 3 * 32 * 64), True),
    (dict(n_streams=1, stream_stride=0, scale_stream_stride=0), False),
    (dict(n_kv_heads=1, head_stride=0, scale_head_stride=0), False),
    (dict(smax=1, head_stride=64, stream_stride=192, scale_head_stride=1, scale_stream_stride=3), False),
    (dict(stream_stride=(1 << 62) // 64 * 64, n_streams=1 << 10), True),     # past 64 bits: no such memory
]


@pytest.mark.parametrize("kw,over", LAYOUTS)
def test_caches_that_lie_over_themselves(qd, accepted, kw, over):
    got = append(qd, cache(qd, **kw))
    check(qd, accepted, got, over)


# rows of 64 bf16 (128 bytes): 3 heads, 4 tokens, 2 streams
ROWS = [
    (dict(), False),
    (dict(head=64, token=64), True),
    (dict(head=64, token=128), True),
    (dict(head=256, token=64), False),                       # heads outside tokens
    (dict(head=192, token=64), True),
    (dict(stream=192), True),
    (dict(stream=768 - 64), True),
    (dict(v_rows=A + 16), True),
    (dict(v_rows=A + 128), True),
    (dict(v_rows=A + 3 * 128, token=6 * 64, stream=4 * 6 * 64), False),    # two parts of a fused projection
    (dict(v_rows=A + 2 * 128, token=6 * 64, stream=4 * 6 * 64), True),
]


@pytest.mark.parametrize("kw,over", ROWS)
def test_rows_read_over_each_other(qd, accepted, kw, over):
    f = dict(k_rows=A, v_rows=2 * A, dtype=1, n=4, stream=768, token=192, head=64, lengths=A, n_new=None)
    f.update(kw)
    c = cache(qd)
    got = qd._lib.qd_kv_read(ctypes.addressof(c), *f.values(), None)
    check(qd, accepted, got, over)


# q and out: 6 heads of 64 bf16 (768 bytes), 3 tokens, 2 streams
OUTS = [
    (dict(), False),
    (dict(os=384, ot=384), True),
    (dict(os=2 * 384, ot=384), True),
    (dict(os=384, ot=2 * 384), False),                       # tokens outside streams
    (dict(out=A + 16), True),                                # q and out alike, 8 elements apart
    (dict(out=A + 768), True),                               # out's token t is q's t + 1
    (dict(out=A + 3 * 768), True),
    (dict(out=A + 2 * 3 * 768), False),
    (dict(q=A + 2 * 3 * 768, out=A), False),
    (dict(out=A + 768, qt=768, ot=768, qs=3 * 768, os=3 * 768), False),    # side by side
    (dict(q=A, qs=0, qt=0, out=A + 768), False),             # one query for all, its result behind it
    (dict(q=A + 768, qs=0, qt=0, out=A), True),              # one query for all among the results
    (dict(q=A + 16, out=A, qs=3 * 400, qt=400), True),       # other strides, the same bytes
]


@pytest.mark.parametrize("kw,over", OUTS)
def test_results_over_each_other_or_the_queries(qd, accepted, kw, over):
    f = dict(prefix=None, plen=0, q=A, qs=3 * 384, qt=384, out=2 * A, os=3 * 384, ot=384, dtype=1, n=3, heads=6, scale=1.0,
             lengths=A, n_new=None, most=32, ws=None, wb=0)
    f.update(kw)
    c = cache(qd)
    got = qd._lib.qd_attn_cached(ctypes.addressof(c), *f.values(), None)
    check(qd, accepted, got, over)


# -------------------------------------------------------------------- sizes past the kernels' counters

FAR = 2 ** 31 - 1


@pytest.mark.parametrize("most,plen", [(FAR, 0), (FAR - 1023, 0), (32, FAR), (32, FAR - 126), (FAR, FAR)])
def test_positions_past_the_counters(qd, most, plen):
    """A reader's cache may hold that many rows (K and V may be the same ones)."""
    c = cache(qd, smax=FAR, stream_stride=0, head_stride=0)
    p = cache(qd, smax=FAR, n_streams=1, stream_stride=0, head_stride=0)
    n = ctypes.c_size_t(0)
    at = (ctypes.addressof(c), ctypes.addressof(p) if plen else None, plen)
    assert qd._lib.qd_attn_cached_workspace(*at, 1, 1, 3, most, ctypes.byref(n)) == qd.QD_EUNSUPPORTED
    assert qd._lib.qd_attn_cached(*at, A, 192, 192, 2 * A, 192, 192, 1, 1, 3, 1.0, A, None, most, A, 1 << 30,
                                  None) == qd.QD_EUNSUPPORTED


@pytest.mark.parametrize("tokens", [FAR, FAR - 2 ** 20 + 1])
def test_tokens_past_the_counters(qd, tokens):
    """One row for all tokens (a stride of 0), as appending allows, and as many rows apart as reading asks for."""
    c = cache(qd)
    assert qd._lib.qd_kv_append(ctypes.addressof(c), A, A, 1, tokens, 0, 0, 64, A, None, None) == qd.QD_EUNSUPPORTED
    c = cache(qd, n_streams=1, n_kv_heads=1)
    assert qd._lib.qd_kv_read(ctypes.addressof(c), A, 1 << 50, 1, tokens, 0, 64, 0, A, None, None) == qd.QD_EUNSUPPORTED


# --------------------------------------------------------------------------------- the binding

def test_a_workspace_that_is_less_than_it_counts(qd):
    """An expanded tensor counts bytes that it does not have."""
    import torch
    k = torch.zeros((2, 2, 32, 64), dtype=torch.bfloat16)
    view = qd.KvCache(k, k.clone())
    q = torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16)
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 30), torch.zeros(1 << 12, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError):
            qd.qd_attn_cached(q, view, torch.zeros(2, dtype=torch.int32), torch.zeros_like(q), workspace=ws)


def test_scratch_is_given_back(qd):
    """All that the binding holds for streams goes at once, and is asked for anew afterwards (no such device)."""
    import gc
    import weakref

    class Memory:
        pass

    ops = qd._setup_ops()
    held = [Memory() for _ in range(3)]
    refs = [weakref.ref(x) for x in held]
    for i, x in enumerate(held):
        assert ops.keep(98, i, x, A, 256)
    del held, x
    gc.collect()
    assert all(r() is not None for r in refs)
    qd.release_scratch()
    gc.collect()
    assert all(r() is None for r in refs)
    again = Memory()
    assert ops.keep(98, 0, again, A, 256)
    qd.release_scratch()
    qd.release_scratch()                                  # nothing left: nothing to do


# ------------------------------------------------------------------------------- verification's arrays

# 3 streams of 4 drafts: ids 48 bytes, u and out_ids 60, n_draft and n_accepted 12
ARRAYS = [
    (dict(), False),
    (dict(acc=6 * A), True),                                 # n_accepted over n_draft: some CTAs would read the new count
    (dict(out=4 * A), True),                                 # out_ids over draft_ids: rows of another pitch
    (dict(out=4 * A + 44), True),
    (dict(out=4 * A + 48), False),
    (dict(out=4 * A - 56), True),
    (dict(out=4 * A - 60), False),
    (dict(out=5 * A), True),
    (dict(acc=5 * A + 56), True),
    (dict(acc=5 * A + 60), False),
    (dict(out=6 * A - 56), True),
    (dict(acc=7 * A + 56), True),                            # n_accepted in out_ids
    (dict(acc=7 * A + 60), False),
    (dict(acc=4 * A + 40), True),
]


@pytest.mark.parametrize("kw,over", ARRAYS)
def test_verification_over_what_it_reads(qd, accepted, kw, over):
    f = dict(p=2 * A, ps=40, pr=8, q=3 * A, qs=32, qr=8, ids=4 * A, nd=6 * A, u=5 * A, B=3, T=4, V=8, out=7 * A, acc=8 * A)
    f.update(kw)
    check(qd, accepted, qd._lib.qd_verify_drafts(*f.values(), None), over)
