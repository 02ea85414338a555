"""Refusals of the calls over a cache in pages that need no device (the addresses are never read)."""
import ctypes

import pytest

A = 1 << 24                                     # an aligned address; arrays stand A apart


@pytest.fixture(scope="module")
def qd():
    import __graft_entry__
    __graft_entry__.build_library()
    import transformer_autoregressive_decode_gb300 as m
    return m


@pytest.fixture(scope="module")
def accepted(qd):
    """What a call answers that passed every check of its arguments, where there is no device to go on with."""
    import torch
    if torch.cuda.is_available():
        return None                             # there the made-up addresses are refused next
    return qd.QD_ECUDA


def pool(qd, **kw):
    """6 pages x 2 heads x 16 positions of 64, contiguous, the scales too."""
    f = dict(k=20 * A, v=21 * A, k_scale=22 * A, v_scale=23 * A, format=qd.QD_KV_Q8, n_streams=6, n_kv_heads=2, smax=16,
             head_dim=64, stream_stride=2 * 16 * 64, head_stride=16 * 64, row_stride=64, scale_stream_stride=32,
             scale_head_stride=16)
    f.update(kw)
    return qd.qd_kv_cache(*(f[n] for n, _ in qd.qd_kv_cache._fields_))


def rope(qd, cache=True, **kw):
    """8 tokens of 4 streams, 4 query and 2 key heads, a fused fp32 projection, bf16 results, 8-bit pages."""
    f = dict(q=A, k=A + 4 * 64 * 4, v=A + 6 * 64 * 4, q_stride=512, k_stride=512, v_stride=512, q_out=2 * A, k_out=3 * A, v_out=4 * A,
             q_out_stride=256, k_out_stride=128, v_out_stride=128, dtype=qd.QD_F32, out_dtype=qd.QD_BF16, n_tokens=8, n_q_heads=4,
             n_kv_heads=2, head_dim=64, q_gamma=5 * A, k_gamma=5 * A, eps=1e-6, cos=6 * A, sin=7 * A, rope_rows=64, positions=None,
             mrope_h=0, lengths=8 * A, offsets=None, n_new=None, n_streams=4, pages=None, page_table=9 * A, table_stride=2,
             table_pages=2)
    c = pool(qd, **kw.pop("pool", {}))
    if cache:
        f["pages"] = ctypes.addressof(c)
    f.update(kw)
    r = qd.qd_rope_rows(*(f[n] for n, _ in qd.qd_rope_rows._fields_))
    return qd._lib.qd_qk_norm_rope(ctypes.addressof(r), None)


EINVAL, EUNS, OK = "QD_EINVAL", "QD_EUNSUPPORTED", None
B16 = dict(dtype=1, q_stride=512, k_stride=512, v_stride=512, k=A + 4 * 64 * 2, v=A + 6 * 64 * 2)
ROPE = [
    (dict(), OK),
    (dict(k_out=None, v_out=None), OK),
    (dict(cos=None, sin=None), OK),
    (dict(q_gamma=None, k_gamma=None), OK),
    (dict(cache=False, v=None, v_out=None), OK),
    (dict(cache=False, lengths=None, n_streams=0, positions=10 * A), OK),
    (dict(positions=10 * A, mrope_h=10), OK),
    (dict(offsets=10 * A, n_tokens=7), OK),
    (dict(n_new=10 * A), OK),
    (dict(**B16, q_out=A, q_out_stride=512, k_out=B16["k"], k_out_stride=512, v_out=B16["v"], v_out_stride=512), OK),    # in place
    (dict(n_tokens=4, **dict(B16, q_stride=1024, k_stride=1024, v_stride=1024), q_out=A + 512 * 2, q_out_stride=1024), OK),   # beside
    (dict(q=None), EINVAL), (dict(k=None), EINVAL), (dict(q_out=None), EINVAL),
    (dict(v=None, v_out=None), EINVAL),                          # pages want v
    (dict(cache=False, v=None), EINVAL),                         # and so does v_out
    (dict(dtype=2), EINVAL), (dict(out_dtype=-1), EINVAL),
    (dict(n_tokens=0), EINVAL), (dict(n_q_heads=0), EINVAL), (dict(n_kv_heads=0), EINVAL),
    (dict(head_dim=96), EUNS), (dict(n_tokens=(1 << 30) + 4), EUNS),
    (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL),
    (dict(sin=None), EINVAL), (dict(rope_rows=0), EINVAL), (dict(cos=6 * A + 4), EINVAL),
    (dict(mrope_h=10), EINVAL), (dict(mrope_h=11, positions=10 * A), EINVAL), (dict(mrope_h=-1, positions=10 * A), EINVAL),
    (dict(cache=False, lengths=None), EINVAL),                   # no positions at all
    (dict(lengths=None, positions=10 * A), EINVAL),              # pages without lengths
    (dict(cache=False, lengths=None, positions=10 * A, offsets=11 * A), EINVAL),
    (dict(offsets=10 * A, n_new=11 * A), EINVAL),
    (dict(n_tokens=7), EINVAL),                                  # not a whole number a stream
    (dict(n_streams=0), EINVAL),
    (dict(q_stride=514), EINVAL), (dict(q=A + 8), EINVAL), (dict(q_out_stride=252), EINVAL), (dict(q_out_stride=128), EINVAL),
    (dict(k_out_stride=64), EINVAL), (dict(lengths=8 * A + 2), EINVAL), (dict(page_table=9 * A + 1), EINVAL),
    (dict(q_out=A), EINVAL),                                     # over fp32 rows, in another type
    (dict(k_out=2 * A), EINVAL), (dict(k_out=2 * A + 256, k_out_stride=256), EINVAL),
    (dict(v_out=3 * A), EINVAL),
    (dict(**B16, q_out=A + 16, q_out_stride=512), EINVAL),       # in place, but shifted
    (dict(**B16, q_out=A, q_out_stride=256), EINVAL),            # in place, but packed
    (dict(page_table=None), EINVAL), (dict(table_pages=0), EINVAL), (dict(table_stride=-1), EINVAL),
    (dict(pool=dict(smax=24)), EUNS), (dict(pool=dict(smax=8)), EUNS), (dict(pool=dict(n_kv_heads=1)), EINVAL),
    (dict(pool=dict(smax=1 << 20, row_stride=64, head_stride=1 << 26, stream_stride=1 << 27, scale_head_stride=1 << 20,
                    scale_stream_stride=1 << 21, v=1 << 40, v_scale=1 << 41), table_pages=2048), EUNS),
    (dict(pool=dict(head_dim=128, row_stride=128, head_stride=2048, stream_stride=4096)), EINVAL),
    (dict(pool=dict(stream_stride=16 * 64)), EINVAL),            # page 1 is head 1
    (dict(pool=dict(v=20 * A)), EINVAL), (dict(pool=dict(scale_head_stride=8)), EINVAL),
    (dict(pool=dict(k=20 * A + 8)), EINVAL),
]


@pytest.mark.parametrize("kw, want", ROPE)
def test_rope_refusals(qd, accepted, kw, want):
    got = rope(qd, **kw)
    if want:
        assert got == getattr(qd, want)
    elif accepted is not None:
        assert got == accepted


def test_rope_host_tensors_are_refused(qd):
    import torch
    q, k = torch.zeros(2, 4, 64), torch.zeros(2, 2, 64)
    pos = torch.zeros(2, dtype=torch.int32)
    cos = torch.zeros(8, 32)
    with pytest.raises(qd.QDError):
        qd.qd_qk_norm_rope(q, k, torch.zeros(2, 4, 64), cos, cos, positions=pos)


@pytest.mark.parametrize("bad", ["heads", "type", "cos", "gamma", "offsets", "positions", "table", "pages", "float lengths"])
def test_rope_marshalling(qd, bad):
    import torch
    z, i = torch.zeros, torch.int32
    c = qd.KvCache(z(4, 2, 16, 64, dtype=torch.bfloat16), z(4, 2, 16, 64, dtype=torch.bfloat16))
    a = dict(q=z(4, 4, 64), k=z(4, 2, 64), q_out=z(4, 4, 64), cos=z(8, 32), sin=z(8, 32), lengths=z(2, dtype=i), v=z(4, 2, 64),
             q_gamma=z(64), pages=c, page_table=z(2, 2, dtype=i))
    a |= {"heads": dict(q=z(4, 64, 4).transpose(1, 2)), "type": dict(k=z(4, 2, 64, dtype=torch.bfloat16)), "cos": dict(cos=z(8, 64)),
          "gamma": dict(q_gamma=z(32)), "offsets": dict(offsets=z(2, dtype=i)), "positions": dict(positions=z(4, dtype=i), mrope_h=3),
          "table": dict(page_table=z(3, 2, dtype=i)), "pages": dict(pages=None), "float lengths": dict(lengths=z(2))}[bad]
    with pytest.raises(ValueError):
        qd.qd_qk_norm_rope(a.pop("q"), a.pop("k"), a.pop("q_out"), **a)


def paged(qd, **kw):
    """4 streams of 2 tokens, 4 query and 2 key heads, fp32."""
    f = dict(table=9 * A, table_stride=2, table_pages=2, n_streams=4, q=A, qs=512, qt=256, out=2 * A, os=512, ot=256, dtype=0, n_tokens=2,
             n_q_heads=4, scale=0.125, lengths=8 * A, n_new=None, max_length=32, ws=None, ws_bytes=0)
    c = pool(qd, **kw.pop("pool", {}))
    f.update(kw)
    return qd._lib.qd_attn_paged(ctypes.addressof(c), *f.values(), None)


PAGED = [
    (dict(), OK), (dict(n_new=10 * A), OK), (dict(dtype=1), OK), (dict(max_length=1), OK), (dict(table_stride=0), OK),
    (dict(table=None), EINVAL), (dict(table=9 * A + 2), EINVAL), (dict(table_pages=0), EINVAL), (dict(table_stride=-2), EINVAL),
    (dict(n_streams=0), EINVAL), (dict(max_length=33), EINVAL), (dict(max_length=0), EINVAL), (dict(dtype=3), EINVAL),
    (dict(n_tokens=0), EINVAL), (dict(n_tokens=65), EUNS), (dict(n_q_heads=3), EINVAL), (dict(n_q_heads=1), EINVAL),
    (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL),
    (dict(q=None), EINVAL), (dict(out=None), EINVAL), (dict(lengths=None), EINVAL), (dict(q=A + 8), EINVAL), (dict(qt=258), EINVAL),
    (dict(out=A), EINVAL), (dict(out=A + 1024), EINVAL), (dict(ot=128), EINVAL), (dict(os=256), EINVAL), (dict(n_new=10 * A + 1), EINVAL),
    (dict(pool=dict(smax=48)), EUNS), (dict(pool=dict(head_dim=32)), EUNS), (dict(pool=dict(k=None)), EINVAL),
    (dict(pool=dict(k_scale=None)), EINVAL), (dict(pool=dict(format=2)), EINVAL),
    (dict(n_streams=(1 << 22) + 1), EUNS),      # 2 tokens x 2 heads of each key head x 2^22 streams are the 2^24 rows allowed
    (dict(table_pages=1 << 27, max_length=1 << 20), EUNS),
]


@pytest.mark.parametrize("kw, want", PAGED)
def test_paged_refusals(qd, accepted, kw, want):
    got = paged(qd, **kw)
    if want:
        assert got == getattr(qd, want)
    elif accepted is not None:
        assert got == accepted


@pytest.mark.parametrize("bad", ["streams", "heads", "table", "type", "lengths", "long", "workspace"])
def test_paged_marshalling(qd, bad):
    import torch
    z, i = torch.zeros, torch.int32
    c = qd.KvCache(z(4, 2, 16, 64, dtype=torch.bfloat16), z(4, 2, 16, 64, dtype=torch.bfloat16))
    a = dict(q=z(2, 1, 4, 64), table=z(2, 2, dtype=i), lengths=z(2, dtype=i), out=z(2, 1, 4, 64))
    more = {}
    if bad == "workspace":
        more = dict(workspace=z(1, dtype=torch.uint8).expand(1 << 20))
    else:
        a |= {"streams": dict(out=z(3, 1, 4, 64)), "heads": dict(q=z(2, 1, 64, 4).transpose(2, 3)), "table": dict(table=z(2, 2)),
              "type": dict(out=z(2, 1, 4, 64, dtype=torch.bfloat16)), "lengths": dict(lengths=z(3, dtype=i)),
              "long": dict(table=z(2, 1, dtype=i).expand(2, 2))}[bad]
    with pytest.raises(ValueError):
        qd.qd_attn_paged(a["q"], c, a["table"], a["lengths"], a["out"], **more)


def attend_prompt(qd, **kw):
    """100 tokens, 4 query and 2 key heads of 64, slices of a fused projection; results elsewhere."""
    f = dict(q=A, qs=512, k=A + 512, ks=512, v=A + 768, vs=512, out=2 * A, os=256, n=100, m=100, qh=4, kvh=2, hd=64, scale=0.125,
             offsets=8 * A, kv_offsets=None, seqs=3, ws=None, ws_bytes=0)
    f.update(kw)
    return qd._lib.qd_attn_prompt(*f.values(), None)


PROMPT = [
    (dict(), OK), (dict(kv_offsets=9 * A, m=200, k=3 * A, v=4 * A), OK), (dict(n=1, m=1, qs=0, ks=0, vs=0, os=0), OK), (dict(scale=-1.0), OK),
    (dict(out=A + 1024 + 512, os=1024, qs=1024, ks=1024, vs=1024), OK),      # between the rows
    (dict(q=None), EINVAL), (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(out=None), EINVAL), (dict(offsets=None), EINVAL),
    (dict(n=0), EINVAL), (dict(m=0), EINVAL), (dict(seqs=0), EINVAL), (dict(qh=3), EINVAL), (dict(qh=1), EINVAL), (dict(kvh=0), EINVAL),
    (dict(hd=96), EUNS), (dict(qh=258), EUNS), (dict(m=200), EINVAL), (dict(seqs=(1 << 24) + 1), EUNS),
    (dict(n=(1 << 30) + 1, m=(1 << 30) + 1), EUNS),
    (dict(scale=float("inf")), EINVAL), (dict(q=A + 8), EINVAL), (dict(qs=508), EINVAL), (dict(qs=248), EINVAL), (dict(ks=120), EINVAL),
    (dict(os=128), EINVAL), (dict(qs=-512), EINVAL), (dict(vs=(1 << 37) + 8), EINVAL), (dict(offsets=8 * A + 2), EINVAL),
    (dict(kv_offsets=8 * A + 1), EINVAL),
    (dict(out=A), EINVAL), (dict(out=A, os=512), EINVAL), (dict(out=A + 512, os=512), EINVAL), (dict(out=A + 1024 * 10), EINVAL),
    (dict(out=A + 512, os=512, k=3 * A, v=4 * A, ks=128, vs=128), OK),
]


@pytest.mark.parametrize("kw, want", PROMPT)
def test_prompt_refusals(qd, accepted, kw, want):
    got = attend_prompt(qd, **kw)
    if want:
        assert got == getattr(qd, want)
    elif accepted is not None:
        assert got == accepted


@pytest.mark.parametrize("bad", ["type", "heads", "keys", "offsets", "kv", "none", "workspace"])
def test_prompt_marshalling(qd, bad):
    import torch
    z, i, h = torch.zeros, torch.int32, torch.bfloat16
    a = dict(q=z(4, 4, 64, dtype=h), k=z(4, 2, 64, dtype=h), v=z(4, 2, 64, dtype=h), out=z(4, 4, 64, dtype=h), offsets=z(2, dtype=i))
    more = {}
    if bad == "workspace":
        more = dict(workspace=z(1, dtype=torch.uint8).expand(1 << 20))
    else:
        a |= {"type": dict(q=z(4, 4, 64)), "heads": dict(out=z(4, 64, 4, dtype=h).transpose(1, 2)), "keys": dict(v=z(5, 2, 64, dtype=h)),
              "offsets": dict(offsets=z(2)), "kv": dict(k=z(5, 2, 64, dtype=h), v=z(5, 2, 64, dtype=h)), "none": dict(offsets=None)}[bad]
    with pytest.raises(ValueError):
        qd.qd_attn_prompt(*a.values(), **more)


def test_prompt_without_rows(qd):
    """Nothing to do: no call is made (a call on host memory would be refused)."""
    import torch
    z, h = torch.zeros, torch.bfloat16
    qd.qd_attn_prompt(z(0, 4, 64, dtype=h), z(0, 2, 64, dtype=h), z(0, 2, 64, dtype=h), z(0, 4, 64, dtype=h), z(3, dtype=torch.int32))
    qd.qd_qk_norm_rope(z(0, 4, 64), z(0, 2, 64), z(0, 4, 64), positions=z(0, dtype=torch.int32))
