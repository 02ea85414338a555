"""The operators over caller-held caches on the GPU against plain 64-bit forms: writing and
reading rows (bit for bit), attention (within the bounds of ``_serving_ref``), the
verification of drafts (whole numbers, equal), and a decode loop of all of them."""
import math

import numpy as np
import pytest
import torch

from tests import _serving_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(cuda_ok):
    import __graft_entry__
    __graft_entry__.build()
    yield


@pytest.fixture(scope="module")
def qd():
    import transformer_autoregressive_decode_gb300 as m
    return m


WIDE_ROWS = 48                                   # rows of a key head from which a prefix goes to the wide kernel


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ----------------------------------------------------------------------------- rows

def _empty_cache(B, H, S, D, q8, order="bhs"):
    """A cache and its scales full of rubbish, in memory order bhs or bsh."""
    shape = (B, H, S, D) if order == "bhs" else (B, S, H, D)

    def lay(x):
        return x if order == "bhs" else x.transpose(1, 2)
    if q8:
        k, v = (lay(torch.randint(-128, 128, shape, dtype=torch.int8, device="cuda")) for _ in range(2))
        ks, vs = (torch.full((B, H, S), math.nan, device="cuda") for _ in range(2))
        return k, v, ks, vs
    k, v = (lay(torch.full(shape, math.nan, dtype=torch.bfloat16, device="cuda")) for _ in range(2))
    return k, v, None, None


ROWS = [  # B, T, H, D, S, lengths, n_new
    (1, 1, 1, 64, 1, [1], None),
    (3, 1, 8, 128, 40, [1, 40, 17], [1, 0, 1]),
    (4, 5, 2, 64, 33, [5, 3, 33, 20], [5, 5, 2, 0]),            # the second begins before position 0
    (2, 37, 3, 128, 50, [37, 61], [37, 40]),                    # n_new above the call's rows; past the end
    (5, 130, 4, 64, 200, [130, 131, 150, 200, 7], [130, 1, 77, 130, 7]),
]


@pytest.mark.parametrize("case", range(len(ROWS)))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("order", ["bhs", "bsh"])
def test_rows_written_and_read(qd, case, dtype, q8, order):
    B, T, H, D, S, lengths, n_new = ROWS[case]
    g = gen(case)
    fused = (torch.randn((B, T, 3, H, D), generator=g) * torch.exp(2 * torch.randn((B, T, 3, H, 1), generator=g))).to(dtype)
    fused[0, 0, 1, 0] = 0.0                                       # a row of zeros
    if T > 2:
        fused[0, 1, 1, 0, 3], fused[0, 2, 2, 0, 5] = math.inf, math.nan
        fused[0, 1, 2, 0] = fused[0, 1, 2, 0] * 0 + 1e-38
    dev = fused.cuda()
    k, v, ks, vs = _empty_cache(B, H, S, D, q8, order)
    before = [None if x is None else x.clone() for x in (k, v, ks, vs)]
    view = qd.KvCache(k, v, ks, vs)
    ln, nn = ints(lengths), None if n_new is None else ints(n_new)
    qd.qd_kv_append(view, dev[:, :, 1], dev[:, :, 2], ln, n_new=nn)
    back = [torch.full((B, T, H, D), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    qd.qd_kv_read(view, ln, *back, n_new=nn)
    torch.cuda.synchronize()
    for part, (c, s, c0, s0, got) in enumerate([(k, ks, before[0], before[2], back[0]), (v, vs, before[1], before[3], back[1])]):
        want, want_s = c0.cpu().clone(), None if s0 is None else s0.cpu().clone()
        read = torch.full((B, T, H, D), 7.0, dtype=dtype)
        for b in range(B):
            n = T if n_new is None else min(n_new[b], T)
            for t in range(n):
                pos = lengths[b] - n + t
                if not 0 <= pos < S:
                    continue
                row = fused[b, t, 1 + part].float()
                if q8:
                    codes, scale = ref.quantise_rows(row.numpy())
                    want[b, :, pos] = torch.from_numpy(codes)
                    want_s[b, :, pos] = torch.from_numpy(scale)
                    read[b, t] = (torch.from_numpy(codes).float() * torch.from_numpy(scale)[:, None]).to(dtype)
                else:
                    want[b, :, pos] = row.bfloat16()
                    read[b, t] = row.bfloat16().to(dtype)
        if q8:
            assert torch.equal(c.cpu(), want)
            assert np.array_equal(s.cpu().numpy(), want_s.numpy(), equal_nan=True)
        else:
            assert np.array_equal(c.cpu().float().numpy(), want.float().numpy(), equal_nan=True)
        assert np.array_equal(got.cpu().float().numpy(), read.float().numpy(), equal_nan=True)


# ------------------------------------------------------------------------ attention

def _filled(g, B, H, S, D, q8, loud=1.0):
    """(device cache view parts, 64-bit values)"""
    x = [torch.randn((B, H, S, D), generator=g) * torch.exp(0.7 * torch.randn((B, H, S, 1), generator=g)) * loud for _ in range(2)]
    if q8:
        parts = [ref.quantise_rows(a.numpy()) for a in x]
        vals = [torch.from_numpy(c).double() * torch.from_numpy(s).double()[..., None] for c, s in parts]
        dev = [torch.from_numpy(parts[0][0]).cuda(), torch.from_numpy(parts[1][0]).cuda(),
               torch.from_numpy(parts[0][1]).cuda(), torch.from_numpy(parts[1][1]).cuda()]
        return dev, vals
    x = [a.bfloat16() for a in x]
    return [x[0].cuda(), x[1].cuda(), None, None], [a.double() for a in x]


def _spoil(dev, lengths, S):
    """NaN and infinity in every place that no query sees."""
    for b, n in enumerate(lengths):
        n = max(n, 0)
        if n >= S:
            continue
        if dev[2] is None:
            dev[0][b, :, n:], dev[1][b, :, n:] = math.nan, math.inf
        else:
            dev[2][b, :, n:], dev[3][b, :, n:] = math.inf, math.nan


def _check(qd, B, T, G, H, D, S, lengths, n_new, q8, dtype, P=0, p8=None, seed=0, q_scale=1.0, loud=1.0, scale=None,
           order="bhs", max_length=None):
    g = gen(seed)
    dev, (k, v) = _filled(g, B, H, S, D, q8, loud)
    _spoil(dev, lengths, S)
    if order == "bsh":
        dev = [None if x is None else x.transpose(1, 2).contiguous().transpose(1, 2) if x.dim() == 4 else x for x in dev]
    view = qd.KvCache(*dev)
    fused = (torch.randn((B, T, G * H + 2 * H, D), generator=g) * q_scale).to(dtype)
    q = fused[:, :, :G * H]
    nn = [min(n, T) for n in n_new] if n_new else [T] * B
    for b in range(B):
        fused[b, nn[b]:] = math.nan                              # queries not in use
    pre, pk, pv = None, None, None
    if P:
        pdev, (pk, pv) = _filled(g, 1, H, P + 3, D, q8 if p8 is None else p8, loud)
        _spoil(pdev, [P], P + 3)
        pre, pk, pv = qd.KvCache(*pdev), pk[0, :, :P], pv[0, :, :P]
    out = torch.full((B, T, G * H, D), 7.0, dtype=dtype, device="cuda")
    qd.qd_attn_cached(fused.cuda()[:, :, :G * H], view, ints(lengths), out, n_new=ints(n_new) if n_new else None, prefix=pre,
                      prefix_length=P if P else None, scale=scale, max_length=max_length)
    torch.cuda.synchronize()
    want, mag, spread = ref.attend(q, k, v, [max(n, 0) for n in lengths], nn, D ** -0.5 if scale is None else scale, pk, pv)
    got = out.cpu().double()
    unused = torch.isnan(want)
    assert torch.equal(got[unused], torch.full_like(got[unused], 7.0))
    pq = q8 if p8 is None else p8
    bf16 = dtype == torch.bfloat16
    # the prefix goes to the wide kernel; and from 9 rows on, a bf16 cache or prefix gets one bf16 part of each probability
    wide = bool(P) and bf16 and B * T * G >= (WIDE_ROWS if pq else 9)
    tol = ref.attend_bound(want, mag, spread, max(lengths) + P, D, dtype, q8, bf16 and not q8 and T * G > 8)
    if P:
        tol = torch.maximum(tol, ref.attend_bound(want, mag, spread, max(lengths) + P, D, dtype, pq, wide))
    bad = ~((got - want).abs() <= tol) & ~unused
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float(((got - want).abs() / tol)[~unused].max()):.3g} of the bound"
    return got


LENGTHS = [1, 0, 15, 16, 17, 63, 64, 65, 127, 200]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 3, 8])
def test_single_tokens(qd, dtype, q8, D, G):
    _check(qd, len(LENGTHS), 1, G, 2, D, 200, LENGTHS, None, q8, dtype, seed=G)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,G", [(2, 1), (5, 2), (3, 3), (8, 4), (64, 1), (11, 8)])
def test_drafted_tokens(qd, dtype, q8, D, T, G):
    """Several new tokens, some streams with fewer, with none, with less cache than tokens."""
    lengths = [1, 0, 5, 16, 33, 64, 90, 3]
    n_new = [T, T, min(3, T), 0, T, 1, T, T + 9]
    _check(qd, 8, T, G, 2, D, 90, lengths, n_new, q8, dtype, seed=T)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("q8,p8", [(True, True), (False, False), (True, False), (False, True)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P,T,G", [(1, 1, 1), (17, 1, 2), (130, 4, 2), (333, 3, 3)])
def test_shared_prefix(qd, dtype, q8, p8, D, P, T, G):
    lengths = [0, 1, 7, 40, 64]
    _check(qd, 5, T, G, 2, D, 64, lengths, [min(T, n) for n in lengths], q8, dtype, P=P, p8=p8, seed=P)


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,T,G,P", [(24, 1, 2, 1), (48, 1, 1, 127), (64, 1, 2, 128), (33, 1, 4, 129), (13, 5, 3, 700),
                                     (10, 8, 8, 515), (50, 2, 3, 1300)])
def test_many_rows_over_a_prefix(qd, q8, D, B, T, G, P):
    """Tiles of 128 rows, one alone (every other chunk to each half) or in pairs, partly filled, with unused rows between."""
    g = gen(P)
    lengths = torch.randint(0, 20, (B,), generator=g).tolist()
    n_new = torch.randint(0, T + 1, (B,), generator=g).tolist() if T > 1 else None
    if n_new:
        n_new = [min(a, b) for a, b in zip(n_new, lengths)]
    _check(qd, B, T, G, 2, D, 20, lengths, n_new, q8, torch.bfloat16, P=P, p8=q8, seed=P)
    if T > 1:
        _check(qd, B, T, G, 2, D, 20, lengths, None, q8, torch.bfloat16, P=P, p8=q8, seed=P + 1, q_scale=4.0)


@pytest.mark.parametrize("q8,dtype,B,T,G,P", [(True, torch.float32, 24, 4, 2, 3000), (False, torch.float32, 9, 3, 3, 4100),
                                             (False, torch.bfloat16, 5, 1, 3, 30000), (True, torch.bfloat16, 22, 1, 2, 3500)])
def test_prefix_in_a_pass_of_its_own(qd, q8, dtype, B, T, G, P):
    """Too long for every stream to read, and too few or too exact rows for the tcgen05 cores."""
    g = gen(P)
    lengths = torch.randint(0, 40, (B,), generator=g).tolist()
    _check(qd, B, T, G, 2, 64, 40, lengths, [min(T, n) for n in lengths], q8, dtype, P=P, p8=q8, seed=P)


def test_no_rows_in_use_over_a_prefix(qd):
    _check(qd, 30, 2, 2, 2, 128, 20, [0] * 30, [0] * 30, True, torch.bfloat16, P=300, p8=True)
    _check(qd, 30, 2, 2, 2, 128, 20, [3] * 30, [0] * 29 + [1], False, torch.bfloat16, P=300, p8=False)


def test_a_prefix_that_begins_with_hidden_keys(qd):
    """Keys of -infinity first, then scores far below zero: the reference comes from the first that count."""
    g = gen(18)
    B, P, D = 64, 300, 128
    k = torch.full((1, 1, P, D), 0.0)
    k[0, 0, :, 0] = -500.0 + torch.rand((P,), generator=g)
    k[0, 0, :150] = -math.inf
    v = torch.randn((1, 1, P, D), generator=g).bfloat16()
    k = k.bfloat16()
    own, _ = _filled(g, B, 1, 4, D, False)
    q = torch.zeros((B, 1, 1, D)).bfloat16()
    q[..., 0] = 1.0
    q[...] = q + 2.0 ** -100                                        # nothing times an infinity
    out = torch.empty((B, 1, 1, D), dtype=torch.bfloat16, device="cuda")
    qd.qd_attn_cached(q.cuda(), qd.KvCache(*own), ints([0] * B), out, prefix=qd.KvCache(k.cuda(), v.cuda()), scale=1.0)
    want, mag, spread = ref.attend(q[:1], k[:, :, 150:].double(), v[:, :, 150:].double(), [150], [1], 1.0)
    assert ((out.cpu().double() - want).abs() <= ref.attend_bound(want, mag, spread, P, D, torch.bfloat16, False, True)).all()


@pytest.mark.parametrize("q8", [True, False])
def test_growing_scores_over_a_prefix(qd, q8):
    """Keys in order of their score: the reference moves in every chunk, O with it."""
    g = gen(17)
    B, P, D = 64, 1000, 128
    q = torch.randn((B, 1, 1, D), generator=g).bfloat16()
    q[:] = q[:1]
    ramp = torch.linspace(-30, 90, P)
    k = (ramp[:, None] * q[0, 0, 0].float() / q[0, 0, 0].float().square().sum())[None, None]
    v = torch.randn((1, 1, P, D), generator=g) * torch.linspace(3, 0.1, P)[:, None]
    if q8:
        (kc, ks), (vc, vs) = ref.quantise_rows(k.numpy()), ref.quantise_rows(v.numpy())
        pre = [torch.from_numpy(x).cuda() for x in (kc, vc, ks, vs)]
        k, v = (torch.from_numpy(c).double() * torch.from_numpy(s).double()[..., None] for c, s in ((kc, ks), (vc, vs)))
    else:
        pre = [k.bfloat16().cuda(), v.bfloat16().cuda(), None, None]
        k, v = k.bfloat16().double(), v.bfloat16().double()
    own, _ = _filled(g, B, 1, 4, D, q8)
    out = torch.empty((B, 1, 1, D), dtype=torch.bfloat16, device="cuda")
    qd.qd_attn_cached(q.cuda(), qd.KvCache(*own), ints([0] * B), out, prefix=qd.KvCache(*pre), scale=1.0)
    want, mag, spread = ref.attend(q[:1], k, v, [P], [1], 1.0)
    tol = ref.attend_bound(want, mag, spread, P, D, torch.bfloat16, q8, True)
    assert ((out.cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_long_axis_is_split_and_joined(qd, q8, dtype):
    _check(qd, 1, 1, 2, 2, 128, 3001, [2999], None, q8, dtype, seed=3)
    _check(qd, 2, 1, 2, 1, 64, 16, [16, 2], None, q8, dtype, P=4001, p8=q8, seed=4)


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("q_scale,loud", [(30.0, 1.0), (1e-3, 1.0), (1.0, 1e4), (1.0, 1e-6)])
def test_sharp_flat_loud_and_faint(qd, q8, dtype, q_scale, loud):
    """One position takes all, all are alike, and values far from 1 (the scores stay in reach)."""
    _check(qd, 3, 2, 2, 2, 64, 300, [300, 177, 31], None, q8, dtype, seed=7, q_scale=q_scale, loud=loud,
           scale=0.125 / loud)


@pytest.mark.parametrize("q8", [True, False])
def test_memory_order_of_positions_before_heads(qd, q8):
    _check(qd, 3, 2, 2, 4, 64, 70, [70, 12, 33], None, q8, torch.bfloat16, order="bsh", seed=9, max_length=70)


def test_growing_scores_move_the_reference(qd):
    """Keys in order of their score, so that the running maximum moves at every step."""
    for q8 in (True, False):
        g = gen(11)
        q = torch.randn((1, 1, 2, 64), generator=g)
        ramp = torch.linspace(0, 60, 500)
        k = (ramp[:, None] * q[0, 0, 0] / q[0, 0, 0].square().sum())[None, None].repeat(1, 2, 1, 1)
        v = torch.randn((1, 2, 500, 64), generator=g)
        if q8:
            (kc, ks), (vc, vs) = ref.quantise_rows(k.numpy()), ref.quantise_rows(v.numpy())
            dev = [torch.from_numpy(x).cuda() for x in (kc, vc, ks, vs)]
            k, v = (torch.from_numpy(c).double() * torch.from_numpy(s).double()[..., None] for c, s in ((kc, ks), (vc, vs)))
        else:
            dev = [k.bfloat16().cuda(), v.bfloat16().cuda(), None, None]
            k, v = k.bfloat16().double(), v.bfloat16().double()
        out = torch.empty((1, 1, 2, 64), device="cuda")
        qd.qd_attn_cached(q.cuda(), qd.KvCache(*dev), ints([500]), out, scale=1.0)
        want, mag, spread = ref.attend(q, k, v, [500], [1], 1.0)
        tol = ref.attend_bound(want, mag, spread, 500, 64, torch.float32, q8)
        assert ((out.cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("G,D", [(2, 128), (5, 128), (5, 64), (2, 64)])
def test_a_new_token_that_is_not_finite_reaches_only_those_that_see_it(qd, dtype, q8, G, D):
    g = gen(12)
    B, T, H, S = 2, 4, 2, 50
    dev, (k, v) = _filled(g, B, H, S, D, q8)
    lengths = [50, 19]
    for b, n in enumerate(lengths):
        if q8:
            dev[3][b, :, n - 2] = math.nan
        else:
            dev[1][b, :, n - 2, 5] = math.inf
        if q8:
            dev[2][b, :, n - 1] = math.nan
        else:
            dev[0][b, :, n - 1, 7] = math.nan
    q = torch.randn((B, T, G * H, D), generator=g).to(dtype)
    out = torch.zeros((B, T, G * H, D), dtype=dtype, device="cuda")
    qd.qd_attn_cached(q.cuda(), qd.KvCache(*dev), ints(lengths), out)
    got = out.cpu().double()
    want, mag, spread = ref.attend(q[:, :2], k, v, [n - 2 for n in lengths], [2, 2], D ** -0.5)
    tol = ref.attend_bound(want, mag, spread, 50, D, dtype, q8, not q8 and dtype == torch.bfloat16 and T * G > 8)
    assert ((got[:, :2] - want).abs() <= tol).all()
    if q8:
        assert torch.isnan(got[:, 2]).all()
    else:
        # p stands in two or three parts, the last often 0: 0 x infinity is NaN, so an infinity
        # that is seen gives one or the other (qd.h says so)
        assert not torch.isfinite(got[:, 2, :, 5]).any() and torch.isfinite(got[:, 2, :, :5]).all()
    assert torch.isnan(got[:, 3]).all()


@pytest.mark.parametrize("q8,dtype", [(True, torch.bfloat16), (True, torch.float32), (False, torch.bfloat16)])
def test_scores_of_minus_infinity_everywhere_give_zeros(qd, q8, dtype):
    """Products that overflow: every weight is 0, and so is the result.  (fp32 queries over a
    bf16 cache have parts of both signs, whose products overflow to infinity less infinity: NaN.)"""
    big = torch.full((1, 1, 20, 64), 3e38)
    k, v = (big, torch.ones_like(big)) if not q8 else (torch.full((1, 1, 20, 64), 127.0), torch.ones_like(big))
    scales = [torch.full((1, 1, 20), 2e36, device="cuda"), torch.ones((1, 1, 20), device="cuda")] if q8 else []
    dev = [x.to(torch.int8 if q8 else torch.bfloat16).cuda() for x in (k, v)] + scales
    q = torch.full((1, 1, 1, 64), -3e38, dtype=dtype, device="cuda")
    out = torch.full((1, 1, 1, 64), 7.0, dtype=dtype, device="cuda")
    qd.qd_attn_cached(q, qd.KvCache(*dev), ints([20]), out)
    assert torch.equal(out, torch.zeros_like(out))


def test_keys_of_minus_infinity_hide_a_position(qd):
    """bf16 rows over a bf16 cache: a key of -infinity against positive queries has weight 0."""
    g = gen(14)
    dev, (k, v) = _filled(g, 1, 1, 40, 64, False)
    q = torch.rand((1, 1, 2, 64), generator=g).bfloat16() + 0.5
    dev[0][0, 0, 3:30] = -math.inf
    out = torch.full((1, 1, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    qd.qd_attn_cached(q.cuda(), qd.KvCache(*dev), ints([40]), out)
    keep = [0, 1, 2, *range(30, 40)]
    want, mag, spread = ref.attend(q, k[:, :, keep], v[:, :, keep], [13], [1], 0.125)
    assert ((out.cpu().double() - want).abs() <= ref.attend_bound(want, mag, spread, 40, 64, torch.bfloat16, False)).all()
    qd.qd_attn_cached(q.cuda(), qd.KvCache(*dev), ints([40]), out, prefix=qd.KvCache(dev[0][:, :, 3:30], dev[1][:, :, 3:30]))
    assert ((out.cpu().double() - want).abs() <= ref.attend_bound(want, mag, spread, 40, 64, torch.bfloat16, False)).all()


def test_offsets_past_32_bits(qd):
    """Streams and heads more than 2^32 bytes into the cache."""
    g = gen(13)
    B, H, S, D = 2, 2, 40, 128
    dev, (k, v) = _filled(g, B, H, S, D, True)
    big = [torch.zeros(5 * 2 ** 30, dtype=torch.int8, device="cuda") for _ in range(2)]
    far = [x.as_strided((B, H, S, D), (2 ** 31 + 2 ** 29, 2 ** 31 + 256, 2 * D, 1)) for x in big]
    lengths, q = [40, 23], torch.randn((B, 1, H, D), generator=g).bfloat16()
    for x, y in zip(far, dev):
        x.copy_(y)
    out = torch.zeros((B, 1, H, D), dtype=torch.bfloat16, device="cuda")
    qd.qd_attn_cached(q.cuda(), qd.KvCache(far[0], far[1], dev[2], dev[3]), ints(lengths), out)
    want, mag, spread = ref.attend(q, k, v, lengths, [1, 1], D ** -0.5)
    assert ((out.cpu().double() - want).abs() <= ref.attend_bound(want, mag, spread, 40, D, torch.bfloat16, True)).all()
    back = [torch.zeros((B, 1, H, D), device="cuda") for _ in range(2)]
    qd.qd_kv_read(qd.KvCache(far[0], far[1], dev[2], dev[3]), ints(lengths), *back)
    for b, n in enumerate(lengths):
        assert torch.equal(back[0][b, 0].cpu().double(), k[b, :, n - 1].float().double())


def test_results_repeat_bit_for_bit(qd):
    a = _check(qd, 3, 2, 2, 2, 128, 700, [700, 3, 555], None, True, torch.float32, P=900, p8=True, seed=21)
    b = _check(qd, 3, 2, 2, 2, 128, 700, [700, 3, 555], None, True, torch.float32, P=900, p8=True, seed=21)
    assert torch.equal(a, b)


# --------------------------------------------------------------------- verification

def _probs(g, shape):
    return torch.softmax(3 * torch.randn(shape, generator=g), -1)


def _verify(qd, p, ids, u, q=None, n_draft=None):
    B, T = ids.shape
    out, acc = torch.full((B, T + 1), 77, dtype=torch.int32, device="cuda"), torch.full((B,), 77, dtype=torch.int32, device="cuda")
    qd.qd_verify_drafts(p.cuda(), ids.cuda(), u.cuda(), out, acc, draft_probs=None if q is None else q.cuda(),
                        n_draft=None if n_draft is None else ints(n_draft))
    w_out, w_acc = ref.verify(p.numpy(), ids.numpy(), u.numpy(), None if q is None else q.numpy(), n_draft)
    assert np.array_equal(acc.cpu().numpy(), w_acc)
    assert np.array_equal(out.cpu().numpy(), w_out)
    return w_out, w_acc


@pytest.mark.parametrize("drafter", ["probs", "ids"])
@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (3, 1, 5), (7, 4, 127), (5, 8, 2048), (9, 3, 4099), (2, 64, 300), (3, 2, 151936)])
def test_drafts_are_verified(qd, B, T, V, drafter):
    g = gen(V + T)
    p = _probs(g, (B, T + 1, V))
    q = torch.softmax(torch.log(p[:, :T]) + 0.5 * torch.randn((B, T, V), generator=g), -1) if drafter == "probs" else None
    ids = torch.stack([torch.multinomial(q[b] if q is not None else p[b, :T], 1, generator=g)[:, 0] for b in range(B)]).int()
    u = torch.rand((B, T + 1), generator=g)
    n = torch.randint(0, T + 1, (B,), generator=g).tolist()
    n[0] = T + 5
    _verify(qd, p, ids, u, q, n)
    if drafter == "ids":
        u[:, :T] *= p[:, :T].gather(2, ids.long()[..., None])[..., 0] * 1.3
    _verify(qd, p, ids, u, q)


def test_edges_of_verification(qd):
    g = gen(5)
    p = _probs(g, (8, 4, 1000))
    q = p[:, :3].clone()
    ids = p[:, :3].argmax(-1).int()
    u = torch.rand((8, 4), generator=g) * 0.99
    _, acc = _verify(qd, p, ids, u, q)                              # q = p: u < 1 always passes
    assert (acc == 3).all()
    u[1, 0] = 1.0                                                   # not below: fails with nothing left of p - q
    u[2, 3], u[3, 3] = 0.0, 1.0 - 2.0 ** -24                        # the first and the last weight
    ids[4, 1], ids[5, 2] = -1, 1000                                 # ids outside the vocabulary
    q[6, 0] = 0.0                                                   # q(x) = 0 < p(x): passes
    p[7] = 0.0                                                      # no weight at all
    p[0, 3, 10], p[0, 3, 11], p[0, 3, 12] = math.nan, -1.0, 3.0     # not probabilities
    out, acc = _verify(qd, p, ids, u, q)
    assert acc.tolist() == [3, 0, 3, 3, 1, 2, 3, 0] and out[7, 0] == -1
    _verify(qd, p, ids, u)                                          # and for drafts that were not sampled


def test_rows_at_odd_addresses(qd):
    g = gen(6)
    B, T, V = 3, 2, 1001
    base, qb = _probs(g, (B, T + 1, V + 2)), _probs(g, (B, T, V + 4))
    p, q = base.cuda()[:, :, 1:V + 1], qb.cuda()[:, :, 3:V + 3]
    ids = torch.randint(0, V, (B, T), generator=g).int()
    u = torch.rand((B, T + 1), generator=g)
    out, acc = torch.zeros((B, T + 1), dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    qd.qd_verify_drafts(p, ids.cuda(), u.cuda(), out, acc, draft_probs=q)
    w_out, w_acc = ref.verify(p.cpu().numpy(), ids.numpy(), u.numpy(), q.cpu().numpy())
    assert np.array_equal(out.cpu().numpy(), w_out) and np.array_equal(acc.cpu().numpy(), w_acc)


def test_drawn_tokens_follow_the_target(qd):
    """The point of the scheme: whatever the drafter, the first token is distributed as p."""
    g = gen(8)
    V, N = 11, 40000
    p, q = _probs(g, (V,)) * 0 + torch.softmax(torch.randn(V, generator=g), -1), torch.softmax(torch.randn(V, generator=g), -1)
    ids = torch.multinomial(q, N, replacement=True, generator=g)[:, None].int()
    out, acc = torch.zeros((N, 2), dtype=torch.int32, device="cuda"), torch.zeros(N, dtype=torch.int32, device="cuda")
    qd.qd_verify_drafts(p.cuda().expand(N, 2, V), ids.cuda(), torch.rand((N, 2), generator=g).cuda(), out, acc,
                        draft_probs=q.cuda().expand(N, 1, V))
    share = torch.bincount(out[:, 0].cpu().long(), minlength=V).double() / N
    # a share of N draws has deviation sqrt(p (1 - p) / N); six of them for 11 shares
    assert ((share - p.double()).abs() <= 6 * (p.double() * (1 - p.double()) / N).sqrt()).all()


# ----------------------------------------------------------------- refusals, and a run

def test_refusals(qd):
    k = torch.zeros((2, 2, 32, 64), dtype=torch.int8, device="cuda")
    s = torch.zeros((2, 2, 32), device="cuda")
    view = qd.KvCache(k, k.clone(), s, s.clone())
    q = torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    out, ln = torch.zeros_like(q), ints([3, 4])

    def status(fn):
        with pytest.raises(qd.QDError) as e:
            fn()
        return e.value.status

    assert status(lambda: qd.qd_attn_cached(q, view, ln, out, max_length=33)) == qd.QD_EINVAL
    assert status(lambda: qd.qd_attn_cached(q, view, ln, out, max_length=0)) == qd.QD_EINVAL
    assert status(lambda: qd.qd_attn_cached(q, view, ln.cpu(), out)) == qd.QD_EINVAL          # host lengths
    assert status(lambda: qd.qd_attn_cached(q.cpu(), view, ln, out)) == qd.QD_EINVAL
    assert status(lambda: qd.qd_attn_cached(q, view, ln, out, scale=math.inf)) == qd.QD_EINVAL
    many = torch.zeros((2, 65, 4, 64), dtype=torch.bfloat16, device="cuda")
    assert status(lambda: qd.qd_attn_cached(many, view, ln, many.clone())) == qd.QD_EUNSUPPORTED
    three = torch.zeros((2, 1, 3, 64), dtype=torch.bfloat16, device="cuda")
    assert status(lambda: qd.qd_attn_cached(three, view, ln, three.clone())) == qd.QD_EINVAL    # 3 heads over 2
    b = torch.zeros((1, 2, 32, 64), dtype=torch.bfloat16, device="cuda")
    pre = qd.KvCache(b, b.clone())                                # another format: a pass of its own
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    assert status(lambda: qd.qd_attn_cached(q, view, ln, out, prefix=pre, workspace=small)) == qd.QD_EINVAL
    assert status(lambda: qd.qd_attn_cached(q, view, ln, out, prefix=pre, prefix_length=33,
                                            workspace=torch.empty(1 << 22, dtype=torch.uint8, device="cuda"))) == qd.QD_EINVAL
    odd = torch.zeros(2 * 4 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(2, 1, 4, 64)
    assert status(lambda: qd.qd_attn_cached(odd, view, ln, out)) == qd.QD_EINVAL               # not 16-byte aligned
    rows = torch.zeros((2, 1, 2, 64), device="cuda")
    assert status(lambda: qd.qd_kv_append(view, rows, rows.cpu().clone(), ln)) == qd.QD_EINVAL
    p, u = torch.ones((2, 2, 8), device="cuda") / 8, torch.zeros((2, 2), device="cuda")
    ids, o, a = ints([[0], [1]]), ints([[0, 0], [0, 0]]), ints([0, 0])
    assert status(lambda: qd.qd_verify_drafts(p.cpu(), ids, u, o, a)) == qd.QD_EINVAL
    with pytest.raises(ValueError):
        qd.qd_verify_drafts(p[:, :1], ids, u, o, a)
    with pytest.raises(ValueError):
        qd.KvCache(k, k.clone())
    with pytest.raises(ValueError):
        qd.qd_kv_append(view, rows, rows.clone(), ln.long())
    out_before = out.clone()
    torch.cuda.synchronize()
    assert torch.equal(out, out_before)


def test_a_decode_loop_of_all_of_them_captured(qd):
    """Append, attend behind a prefix, verify: one graph replayed while the streams grow by
    what was accepted, against the 64-bit forms step by step; two graphs with their own workspaces."""
    g = gen(31)
    B, T, H, G, D, S, P, V = 3, 3, 2, 2, 64, 64, 50, 97
    pdev, (pk, pv) = _filled(g, 1, H, P, D, True)
    pre = qd.KvCache(*pdev)
    k, v = (torch.zeros((B, H, S, D), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((B, H, S), device="cuda") for _ in range(2))
    view = qd.KvCache(k, v, ks, vs)
    fused = torch.zeros((B, T, (G + 2) * H, D), dtype=torch.bfloat16, device="cuda")
    q, kn, vn = fused[:, :, :G * H], fused[:, :, G * H:(G + 1) * H], fused[:, :, (G + 1) * H:]
    lengths, new = ints([0] * B), ints([0] * B)
    p, dq = torch.zeros((B, T + 1, V), device="cuda"), torch.zeros((B, T, V), device="cuda")
    ids, u = torch.zeros((B, T), dtype=torch.int32, device="cuda"), torch.zeros((B, T + 1), device="cuda")
    outs = [torch.zeros((B, T, G * H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    oi, acc = torch.zeros((B, T + 1), dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    need = qd.qd_attn_cached_workspace(view, True, T, G * H, prefix=pre)
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]

    def step(i):
        qd.qd_kv_append(view, kn, vn, lengths, n_new=new)
        qd.qd_attn_cached(q, view, lengths, outs[i], n_new=new, prefix=pre, workspace=ws[i])
        qd.qd_verify_drafts(p, ids, u, oi, acc, draft_probs=dq, n_draft=new)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(0)
        step(1)
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            step(i)
    have = [0] * B
    kv = [torch.zeros((B, H, S, D), dtype=torch.float64) for _ in range(2)]
    for it in range(6):
        n = torch.randint(0, T + 1, (B,), generator=g).tolist()
        n[it % B] = T
        f = torch.randn((B, T, (G + 2) * H, D), generator=g).bfloat16()
        pp, dd = _probs(g, (B, T + 1, V)), _probs(g, (B, T, V))
        ii = torch.randint(0, V, (B, T), generator=g).int()
        uu = torch.rand((B, T + 1), generator=g)
        for dst, src in ((fused, f), (p, pp), (dq, dd), (ids, ii), (u, uu), (new, ints(n)),
                         (lengths, ints([a + b for a, b in zip(have, n)]))):
            dst.copy_(src)
        graphs[it % 2].replay()
        torch.cuda.synchronize()
        for b in range(B):
            for t in range(n[b]):
                for part, at in ((0, G), (1, G + 1)):
                    c, s = ref.quantise_rows(f[b, t, at * H:(at + 1) * H].float().numpy())
                    kv[part][b, :, have[b] + t] = torch.from_numpy(c).double() * torch.from_numpy(s).double()[:, None]
        want, mag, spread = ref.attend(f[:, :, :G * H], kv[0], kv[1], [a + b for a, b in zip(have, n)], n, D ** -0.5, pk[0], pv[0])
        got, used = outs[it % 2].cpu().double(), ~torch.isnan(want)
        tol = ref.attend_bound(want, mag, spread, S + P, D, torch.bfloat16, True)
        assert ((got - want).abs() <= tol)[used].all()
        w_out, w_acc = ref.verify(pp.numpy(), ii.numpy(), uu.numpy(), dd.numpy(), n)
        assert np.array_equal(oi.cpu().numpy(), w_out) and np.array_equal(acc.cpu().numpy(), w_acc)
        have = [h + int(a) for h, a in zip(have, w_acc)]           # the rejected rows are written over


def test_another_stream(qd):
    """Work on a stream of the caller's, the workspace from torch's allocator on that stream."""
    g = gen(41)
    pdev, (pk, pv) = _filled(g, 1, 2, 200, 64, False)
    dev, (k, v) = _filled(g, 2, 2, 64, 64, False)
    q = torch.randn((2, 1, 4, 64), generator=g).bfloat16()
    qc, out, ln = q.cuda(), torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16, device="cuda"), ints([64, 9])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(20):
        qd.qd_attn_cached(qc, qd.KvCache(*dev), ln, out, prefix=qd.KvCache(*pdev), stream=s)
    s.synchronize()
    want, mag, spread = ref.attend(q, k, v, [64, 9], [1, 1], 0.125, pk[0], pv[0])
    assert ((out.cpu().double() - want).abs() <= ref.attend_bound(want, mag, spread, 264, 64, torch.bfloat16, False)).all()


def test_scratch_of_two_streams_and_of_a_capture(qd):
    """Calls without a workspace at the same time on two streams, and a replayed capture beside them: each has memory
    of its own, and the results stay bit for bit."""
    g = gen(43)
    B, P = 40, 4000
    dev, _ = _filled(g, B, 2, 300, 64, True)
    pdev, _ = _filled(g, 1, 2, P, 64, True)
    view, pre = qd.KvCache(*dev), qd.KvCache(*pdev)
    ln = ints(torch.randint(1, 300, (B,), generator=g).tolist())
    qs = [torch.randn((B, 1, 4, 64), generator=g).bfloat16().cuda() for _ in range(3)]
    assert qd.qd_attn_cached_workspace(view, True, 1, 4, prefix=pre) > 0

    def call(q, out):
        qd.qd_attn_cached(q, view, ln, out, prefix=pre)
    want = []
    for q in qs:
        o = torch.empty_like(q)
        call(q, o)
        want.append(o)
    torch.cuda.synchronize()
    outs = [torch.zeros_like(q) for q in qs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(qs[2], outs[2])
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(30):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                call(qs[i], outs[i])
        with torch.cuda.stream(streams[2]):
            graph.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_two_host_threads_on_one_stream(qd):
    import threading
    g = gen(44)
    dev, _ = _filled(g, 6, 2, 700, 64, False)
    pdev, _ = _filled(g, 1, 2, 30000, 64, False)
    view, pre, ln = qd.KvCache(*dev), qd.KvCache(*pdev), ints([700, 1, 30, 444, 0, 64])
    assert qd.qd_attn_cached_workspace(view, True, 1, 4, prefix=pre) > 0
    qs = [torch.randn((6, 1, 4, 64), generator=g).bfloat16().cuda() for _ in range(2)]
    outs, want = [torch.zeros_like(q) for q in qs], [torch.zeros_like(q) for q in qs]
    for q, o in zip(qs, want):
        qd.qd_attn_cached(q, view, ln, o, prefix=pre)

    def work(i):
        for _ in range(200):
            qd.qd_attn_cached(qs[i], view, ln, outs[i], prefix=pre)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


FIRST_IN_A_CAPTURE = """
import torch, sys
import transformer_autoregressive_decode_gb300 as qd
def i(v): return torch.tensor(v, dtype=torch.int32, device="cuda")
torch.manual_seed(1)
k = torch.randn((40, 2, 300, 64), device="cuda").bfloat16()
p = torch.randn((1, 2, 5000, 64), device="cuda").bfloat16()
view, pre = qd.KvCache(k, k.clone()), qd.KvCache(p, p.clone())
q = torch.randn((40, 2, 4, 64), device="cuda").bfloat16()
outs = [torch.zeros_like(q) for _ in range(2)]
ln = i([300] * 40)
def work(out):
    qd.qd_kv_append(view, q[:, :, :2], q[:, :, 2:], ln)
    qd.qd_attn_cached(q, view, ln, out, prefix=pre)
    qd.qd_attn_cached(q[:1], one, ln[:1], out1)
one, out1 = qd.KvCache(k[:1], k[:1]), torch.zeros_like(q[:1])
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    work(outs[0])
g.replay()
torch.cuda.synchronize()
work(outs[1])
torch.cuda.synchronize()
assert torch.equal(outs[0], outs[1]) and bool(outs[0].float().abs().sum() > 0)
print("captured first")
"""


def test_the_first_call_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_IN_A_CAPTURE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


# ------------------------------------------------------------------------ the ends of the arguments

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [0, 33])
def test_row_groups_without_a_row_in_use(qd, dtype, q8, D, P):
    """Runs that skip the row groups of tokens that n_new leaves out: none, one or all of a stream's in use."""
    B, T, G, H, S = 40, 6, 8, 4, 130
    g = gen(P + D)
    lengths = torch.randint(0, S + 1, (B,), generator=g).tolist()
    n_new = torch.randint(0, T + 1, (B,), generator=g).tolist()
    n_new[:2] = n_new[-2:] = [0] * 2
    n_new[10:13], lengths[5] = [T, 1, 0], 0
    _check(qd, B, T, G, H, D, S, lengths, n_new, q8, dtype, P=P, p8=q8, seed=P)


INT_MIN, INT_MAX = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("q8", [True, False])
def test_counts_beyond_their_ends(qd, q8):
    """Lengths and counts are taken as the nearest end; rows outside the cache are not written."""
    B, T, H, D, S = 5, 4, 2, 64, 40
    g = gen(77)
    dev, _ = _filled(g, B, H, S, D, q8)
    before = [None if x is None else x.clone() for x in dev]
    view = qd.KvCache(*dev)
    rows = torch.randn((B, T, H, D), generator=g).cuda()
    far, nn = ints([INT_MIN, INT_MAX, INT_MIN + 2, -1, S + T]), ints([INT_MAX, INT_MAX, T, 2, INT_MAX])
    qd.qd_kv_append(view, rows, rows, far, n_new=nn)
    back = [torch.full((B, T, H, D), 7.0, device="cuda") for _ in range(2)]
    qd.qd_kv_read(view, far, *back, n_new=nn)
    assert all(x is None or torch.equal(x, y) for x, y in zip(dev, before))
    assert all(bool((x == 7.0).all()) for x in back)
    q = torch.randn((B, T, 2 * H, D), generator=g).cuda()
    got, want = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
    qd.qd_attn_cached(q, view, far, got, n_new=ints([INT_MAX, INT_MIN, T, 2, INT_MAX]), max_length=S)
    qd.qd_attn_cached(q, view, ints([0, S, 0, 0, S]), want, n_new=ints([T, 0, T, 2, T]), max_length=S)
    assert torch.equal(got, want)
    assert bool((got[[0, 2]] == 0).all()) and bool((got[1] == 7.0).all()) and bool((got[3, 2:] == 7.0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("q8", [True, False])
def test_queries_and_caches_shared_by_streams(qd, q8, dtype):
    """What is only read may be broadcast: one query for all streams, one cache for all."""
    B, T, G, H, D, S = 6, 3, 2, 2, 128, 90
    g = gen(78)
    dev, _ = _filled(g, 1, H, S, D, q8)
    one = [None if x is None else x.expand(B, *x.shape[1:]) for x in dev]
    all_ = [None if x is None else x.contiguous() for x in one]
    q = torch.randn((1, 1, G * H, D), generator=g).to(dtype).cuda().expand(B, T, G * H, D)
    ln = ints([90, 17, 3, 64, 65, 0])
    got, want = (torch.empty((B, T, G * H, D), dtype=dtype, device="cuda") for _ in range(2))
    qd.qd_attn_cached(q, qd.KvCache(*one), ln, got)
    qd.qd_attn_cached(q.contiguous(), qd.KvCache(*all_), ln, want)
    assert torch.equal(got, want)


@pytest.mark.parametrize("q8,dtype", [(True, torch.bfloat16), (False, torch.bfloat16), (True, torch.float32)])
@pytest.mark.parametrize("captured", [False, True])
def test_the_streams_own_pass_sees_what_was_written_just_before(qd, q8, dtype, captured):
    """Every step writes rows, lengths and queries directly before the call over a long prefix; the same call on
    finished inputs gives the same bits (the pass beside the prefix's must not read anything older)."""
    B, G, H, D, S, P = 48, 2, 4, 128, 96, 2900
    g = gen(91)
    dev, _ = _filled(g, B, H, S, D, q8)
    pdev, _ = _filled(g, 1, H, P, D, q8)
    view, pre = qd.KvCache(*dev), qd.KvCache(*pdev)
    steps = 40
    rows = torch.randn((steps, 2, B, 1, H, D), generator=g).to(dtype).cuda()
    qs = torch.randn((steps, B, 1, G * H, D), generator=g).to(dtype).cuda()
    row, q = torch.empty_like(rows[0]), torch.empty_like(qs[0])
    ln = torch.zeros((B,), dtype=torch.int32, device="cuda")
    out, again = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty((qd.qd_attn_cached_workspace(view, dtype == torch.bfloat16, 1, G * H, prefix=pre),), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0

    def step():
        ln.add_(1)
        qd.qd_kv_append(view, row[0], row[1], ln)
        qd.qd_attn_cached(q, view, ln, out, prefix=pre, workspace=ws)

    if captured:
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        ln.zero_()
    for i in range(steps):
        row.copy_(rows[i])
        q.copy_(qs[i])
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        qd.qd_attn_cached(q, view, ln, again, prefix=pre, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(out, again), i
