"""Attention over caller-held caches, path by path: every case says which way its prefix goes (read by the
streams' own pass, in a pass of a few rows at a time, or on the tcgen05 cores) and checks it by the workspace that the
call asks for, so that a moved threshold fails here instead of emptying the test.  A prefix of the other format
than the cache's is never read by the streams' own pass, whatever its length."""
import math

import pytest
import torch

from tests import _serving_ref as ref
from tests.test_gpu_serving_ops import _filled, _spoil, gen, ints

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


def route(qd, view, pre, P, bf16, T, QH):
    """'inline', 'narrow' or 'wide', from the workspace: the tcgen05 kernel keeps two records of 128 rows for every SM at
    least, the narrow pass (ref, sum) and an fp32 row for each row of the batch, key head and split, and nothing else is added."""
    H, D = view.shape[1], view.shape[3]
    more = qd.qd_attn_cached_workspace(view, bf16, T, QH, prefix=pre, prefix_length=P)
    none = qd.qd_attn_cached_workspace(view, bf16, T, QH)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if more - none >= 2 * sms * 128 * (8 + 4 * D):
        return "wide"

    def up(n):
        return (n + 255) // 256 * 256
    rows = H * view.shape[0] * T * (QH // H)
    if more - none in [up(rows * s * 8) + up(rows * s * 4 * D) for s in range(1, 33)]:
        return "narrow"
    return "inline"


def bound(want, mag, spread, n, D, dtype, q8, wide=False):
    """ref.attend_bound with the bits that qd.h promises for the probabilities at any number of rows: 16 over bf16
    rows (two bf16 parts) and 22 over 8-bit rows (two fp16 parts) for bf16 queries.  The floor of 8-bit rows as there:
    the spacing of fp16's smallest numbers, against a largest weight of 2^10, of 2^2 where `wide`."""
    mag, top = mag[..., :D], mag[..., D:]
    bf16 = dtype == torch.bfloat16
    step = torch.finfo(dtype).eps / 2
    part_p, part_q = (2.0 ** -22, 0.0 if bf16 else 2.0 ** -22) if q8 else (2.0 ** -16, 0.0) if bf16 else (2.0 ** -24, 2.0 ** -24)
    ds = spread * (part_q + (D + 8) * 2.0 ** -23)
    rel = 2 * part_p + 2 * torch.expm1(2 * ds) + 2.0 ** -20 + 2 * (n + 64) * 2.0 ** -23
    floor = n * 2.0 ** (-27 if wide else -35) * top if q8 else 0.0
    return step * (out_abs(want) + mag * rel) + mag * rel + floor * 1.01 + 1e-30


def out_abs(x):
    return torch.nan_to_num(x).abs()


def run(qd, way, B, T, G, H, D, S, lengths, n_new, q8, dtype, P=0, p8=None, seed=0, q_scale=1.0, change=None,
        queries=None):
    """A call of this way against the 64-bit form; `change` may alter (dev, values) of cache and prefix, `queries` the queries."""
    g = gen(seed)
    dev, kv = _filled(g, B, H, S, D, q8)
    pdev, pkv = _filled(g, 1, H, P + 3, D, p8) if P else (None, None)
    if change:
        change(dev, kv, pdev, pkv)
    _spoil(dev, lengths, S)
    nn = [min(n, T) for n in n_new] if n_new else [T] * B
    q = (torch.randn((B, T, G * H, D), generator=g) * q_scale).to(dtype)
    if queries:
        queries(q)
    for b in range(B):
        q[b, nn[b]:] = math.nan
    view, pre, pk, pv = qd.KvCache(*dev), None, None, None
    if P:
        _spoil(pdev, [P], P + 3)
        pre, pk, pv = qd.KvCache(*pdev), pkv[0][0, :, :P], pkv[1][0, :, :P]
        assert route(qd, view, pre, P, dtype == torch.bfloat16, T, G * H) == way
    out = torch.full((B, T, G * H, D), 7.0, dtype=dtype, device="cuda")
    qd.qd_attn_cached(q.cuda(), view, ints(lengths), out, n_new=ints(n_new) if n_new else None, prefix=pre,
                      prefix_length=P if P else None)
    torch.cuda.synchronize()
    want, mag, spread = ref.attend(q, kv[0], kv[1], lengths, nn, D ** -0.5, pk, pv)
    got, unused = out.cpu().double(), torch.isnan(want)
    assert torch.equal(got[unused], torch.full_like(got[unused], 7.0))
    n = max(lengths) + P
    tol = bound(want, mag, spread, n, D, dtype, q8)
    if P:
        tol = torch.maximum(tol, bound(want, mag, spread, n, D, dtype, p8, way == "wide"))
    bad = ~((got - want).abs() <= tol) & ~unused
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float(((got - want).abs() / tol)[~unused].max()):.3g} of the bound"


# ------------------------------------------------- the probabilities keep their bits at any number of rows

def cancel(dev, kv, pdev, pkv):
    """Position 2 i + 1's value is the negative of position 2 i's (codes, or bf16): every result is a small difference of large
    terms, where it shows if probabilities were cut short."""
    for parts, values in ((dev, kv), (pdev, pkv)):
        if parts is None:
            continue
        n = parts[1].shape[2] // 2 * 2
        parts[1][:, :, 1:n:2] = -parts[1][:, :, :n:2]
        if parts[3] is not None:
            parts[3][:, :, 1:n:2] = parts[3][:, :, :n:2]
        values[1][:, :, 1:n:2] = -values[1][:, :, :n:2]


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,G", [(1, 2), (1, 8), (4, 2), (3, 5), (9, 8)])
def test_terms_that_cancel_over_own_caches(qd, q8, D, T, G):
    lengths = [20, 8, 12, 2, 16, 10]
    run(qd, None, 6, T, G, 2, D, 20, lengths, [min(T, n) for n in lengths], q8, torch.bfloat16, seed=T + 9, q_scale=0.05, change=cancel)


@pytest.mark.parametrize("p8", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("way,B,T,G", [("narrow", 3, 1, 2), ("narrow", 12, 1, 2), ("wide", 24, 1, 2), ("wide", 40, 4, 2)])
def test_terms_that_cancel_over_a_prefix(qd, p8, D, way, B, T, G):
    run(qd, way, B, T, G, 2, D, 8, [0] * B, None, not p8, torch.bfloat16, P=20, p8=p8, seed=B + 9, q_scale=0.05, change=cancel)


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,G", [(1, 2), (4, 2), (3, 3), (4, 4), (5, 8), (9, 8)])
def test_probabilities_over_own_caches(qd, q8, D, T, G):
    """2 to 72 rows a key head, few positions: where an element's terms cancel, a part that was left out shows."""
    lengths = [20, 7, 12, 2, 16, 9]
    run(qd, None, 6, T, G, 2, D, 20, lengths, [min(T, n) for n in lengths], q8, torch.bfloat16, seed=T)


@pytest.mark.parametrize("p8", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,T,G", [(3, 1, 2), (12, 1, 2), (3, 3, 5)])
def test_probabilities_over_a_prefix_of_few_rows(qd, p8, D, B, T, G):
    run(qd, "narrow", B, T, G, 2, D, 8, [0] * B, None, not p8, torch.bfloat16, P=20, p8=p8, seed=B)


@pytest.mark.parametrize("p8", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,T,G", [(24, 1, 2), (64, 1, 2), (40, 4, 2)])
def test_probabilities_over_a_prefix_of_many_rows(qd, p8, D, B, T, G):
    run(qd, "wide", B, T, G, 2, D, 8, [0] * B, None, not p8, torch.bfloat16, P=20, p8=p8, seed=B)


# ---------------------------------------------------------------- scores in fp32, scales of either sign

def loud_channel(dev, kv, pdev, pkv):
    """8-bit keys with one loud channel, as rotated and normalised keys have: the row's scale comes from it and the other
    codes are small."""
    for parts, values in ((dev, kv), (pdev, pkv)):
        if parts is None or parts[2] is None:
            continue
        x = values[0].float()
        x[..., 11] = 60.0 * x.abs().amax(-1)
        c, s = ref.quantise_rows(x.numpy())
        parts[0].copy_(torch.from_numpy(c))
        parts[2].copy_(torch.from_numpy(s))
        values[0] = torch.from_numpy(c).double() * torch.from_numpy(s).double()[..., None]


def quiet_there(q):
    """Queries that do not look at that channel."""
    q[..., 11] = 0.0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("way,B,T,G", [(None, 6, 1, 2), (None, 6, 4, 4), ("narrow", 4, 1, 2), ("wide", 32, 1, 2)])
def test_scores_beside_a_loud_channel(qd, dtype, D, way, B, T, G):
    """The scores' error goes by the products that a query has, not by the row's largest key."""
    if way == "wide" and dtype == torch.float32:
        way = "narrow"
    lengths = [20] * B if way is None else [0] * B
    run(qd, way, B, T, G, 2, D, 20, lengths, None, way is None, dtype, P=20 if way else 0, p8=True, seed=B + T, q_scale=6.0,
        change=loud_channel, queries=quiet_there)


def negative_scales(dev, kv, pdev, pkv):
    """An element stands for code * scale, whatever the scale's sign: values 2^12 loud with every other scale negative, the
    keys' too."""
    for parts, values in ((dev, kv), (pdev, pkv)):
        if parts is None or parts[2] is None:
            continue
        for i in range(2):
            sign = torch.ones(parts[2 + i].shape)
            sign[..., i::2] = -1.0
            if i == 1:
                sign *= 4096.0
            parts[2 + i].mul_(sign.cuda())
            values[i] = values[i] * sign.double()[..., None]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("way,B,T,G", [(None, 6, 1, 2), (None, 6, 4, 4), ("narrow", 4, 1, 2), ("wide", 32, 1, 2)])
def test_scales_of_either_sign(qd, dtype, D, way, B, T, G):
    if way == "wide" and dtype == torch.float32:
        way = "narrow"
    lengths = [40, 1, 2, 33, 17, 9] if way is None else [0] * B
    run(qd, way, B, T, G, 2, D, 40, lengths, [min(T, n) for n in lengths] if way is None else None, way is None, dtype,
        P=150 if way else 0, p8=True, seed=B + T, change=negative_scales)


# ------------------------------------------------------------------------------------- host threads

FIRST_CALLS_MEET = """
import ctypes, threading, torch
import transformer_autoregressive_decode_gb300 as qd
# ctypes lets go of the interpreter's lock, so the library's first calls run at the same time; head_dim 64 and 128, both formats
torch.zeros(1, device="cuda")
jobs = []
for d in (64, 128):
    for dt in (torch.int8, torch.bfloat16):
        # long enough that the workspace goes by the SMs and the CTAs that each holds
        k = torch.zeros((1, 2, 4000, d), dtype=dt, device="cuda").expand(300, 2, 4000, d)
        s = [torch.ones((1, 2, 4000), device="cuda").expand(300, 2, 4000) for _ in range(2)] if dt == torch.int8 else []
        jobs.append(qd.KvCache(k, k, *s))
got = [[] for _ in range(8)]
gate = threading.Barrier(8)
def work(i):
    n = ctypes.c_size_t(0)
    gate.wait()
    for v in jobs:
        st = qd._lib.qd_attn_cached_workspace(v.addr, None, 0, 1, 1, 4, 4000, ctypes.byref(n))
        got[i].append((st, n.value))
t = [threading.Thread(target=work, args=(i,)) for i in range(8)]
[x.start() for x in t]
[x.join() for x in t]
assert all(g == got[0] for g in got) and all(st == 0 and n > 0 for st, n in got[0]), got
print("alike")
"""


def test_first_calls_of_host_threads():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS_MEET], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "alike" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]


# --------------------------------------------------------------- a prefix's own passes, shape by shape

@pytest.mark.parametrize("p8", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,T,G,P", [(24, 1, 2, 1), (48, 1, 1, 127), (33, 1, 2, 129), (64, 1, 2, 128), (43, 1, 3, 700), (64, 2, 2, 257),
                                     (50, 2, 3, 1300), (13, 5, 3, 515), (10, 8, 8, 64)])
def test_wide_prefix(qd, p8, D, B, T, G, P):
    """48 to 640 rows a key head: a tile of 128 rows alone (every other chunk of 128 keys to each half), full, one row into the
    next, an odd number of tiles; unused rows left out, or all in use; the streams' caches in the other format beside it."""
    g = gen(P)
    lengths = torch.randint(0, 20, (B,), generator=g).tolist()
    n_new = [min(int(a), b) for a, b in zip(torch.randint(0, T + 1, (B,), generator=g), lengths)] if T > 1 else None
    run(qd, "wide", B, T, G, 2, D, 20, lengths, n_new, not p8, torch.bfloat16, P=P, p8=p8, seed=P)
    if T > 1:
        run(qd, "wide", B, T, G, 2, D, 20, lengths, None, not p8, torch.bfloat16, P=P, p8=p8, seed=P + 1, q_scale=4.0)


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("D,B,T,G,P", [(64, 60, 1, 2, 6000), (128, 60, 1, 2, 6000), (64, 20, 6, 3, 5400)])
def test_wide_prefix_of_the_caches_format(qd, q8, D, B, T, G, P):
    """Long enough that the streams do not read it themselves; several chunks a CTA."""
    lengths = torch.randint(T, 30, (B,), generator=gen(P)).tolist()
    run(qd, "wide", B, T, G, 3, D, 30, lengths, None, q8, torch.bfloat16, P=P, p8=q8, seed=P)


@pytest.mark.parametrize("p8", [True, False])
@pytest.mark.parametrize("n_new", [None, "some", "none", "one"])
def test_wide_prefix_of_more_streams_than_it_lists(qd, p8, n_new):
    """Above 2048 streams unused rows are not left out of the tiles."""
    B = 2100
    lengths = torch.randint(0, 4, (B,), generator=gen(5)).tolist()
    used = {None: None, "some": [b % 2 for b in range(B)], "none": [0] * B, "one": [0] * (B - 1) + [1]}[n_new]
    run(qd, "wide", B, 1, 1, 1, 64, 4, lengths, used, not p8, torch.bfloat16, P=150, p8=p8, seed=5)


@pytest.mark.parametrize("p8", [True, False])
@pytest.mark.parametrize("n_new", ["none", "one", "last"])
def test_wide_prefix_with_next_to_no_rows_in_use(qd, p8, n_new):
    B, T = 30, 2
    used = {"none": [0] * B, "one": [1] + [0] * (B - 1), "last": [0] * (B - 1) + [2]}[n_new]
    run(qd, "wide", B, T, 2, 2, 128, 20, [3] * B, used, not p8, torch.bfloat16, P=300, p8=p8, seed=3)


@pytest.mark.parametrize("p8", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("way,dtype,B,T,G", [("wide", torch.bfloat16, 24, 1, 2), ("wide", torch.bfloat16, 40, 2, 2),
                                            ("narrow", torch.bfloat16, 4, 1, 2), ("narrow", torch.float32, 30, 1, 2)])
def test_scores_that_rise_in_steps(qd, p8, D, way, dtype, B, T, G):
    """The reference has to move between the chunks of a prefix, and in the middle of one, over what that chunk has written
    already: keys in four levels, each with a quarter of the dims to itself, so that what the earlier levels left
    stands alone there."""
    P, jump = 700, 10.0 if p8 else 45.0
    level = torch.zeros(P + 3)
    for at in (192, 448, 512):
        level[at:] += 1

    def steps(dev, kv, pdev, pkv):
        g = gen(77)
        d = torch.zeros(D)
        d[::2] = 1.0                                                        # the direction of the scores; the queries' below
        k = (level * jump * D ** 0.5 / (D // 2))[:, None] * d + 0.1 * torch.randn((2, P + 3, D), generator=g)
        v = torch.randn((2, P + 3, D), generator=g)
        v *= (torch.arange(D) * 4 // D == level[:, None]).float()
        for i, x in enumerate((k[None], v[None])):
            if p8:
                c, s = ref.quantise_rows(x.numpy())
                pdev[i].copy_(torch.from_numpy(c))
                pdev[2 + i].copy_(torch.from_numpy(s))
                pkv[i] = torch.from_numpy(c).double() * torch.from_numpy(s).double()[..., None]
            else:
                pdev[i].copy_(x.bfloat16())
                pkv[i] = x.bfloat16().double()

    def ones(q):
        q[:] = q[:1, :1, :1]
        q[..., ::2] = 1.0

    run(qd, way, B, T, G, 2, D, 8, [0] * B, None, not p8, dtype, P=P, p8=p8, seed=B, change=steps, queries=ones)


@pytest.mark.parametrize("way,B", [("wide", 64), ("narrow", 4)])
def test_a_prefix_that_begins_with_hidden_keys(qd, way, B):
    """Keys of -infinity first, then scores far below zero: the reference comes from the first that count."""
    g = gen(18)
    P, D = 300, 128
    k = torch.zeros((1, 1, P, D))
    k[0, 0, :, 0] = -500.0 + torch.rand((P,), generator=g)
    k[0, 0, :150] = -math.inf
    v, k = torch.randn((1, 1, P, D), generator=g).bfloat16(), k.bfloat16()
    own, _ = _filled(g, B, 1, 4, D, True)
    q = torch.zeros((B, 1, 1, D))
    q[..., 0] = 1.0
    q = (q + 2.0 ** -100).bfloat16()                                          # nothing times an infinity
    view, pre = qd.KvCache(*own), qd.KvCache(k.cuda(), v.cuda())
    assert route(qd, view, pre, P, True, 1, 1) == way
    out = torch.empty((B, 1, 1, D), dtype=torch.bfloat16, device="cuda")
    qd.qd_attn_cached(q.cuda(), view, ints([0] * B), out, prefix=pre, scale=1.0)
    want, mag, spread = ref.attend(q[:1], k[:, :, 150:].double(), v[:, :, 150:].double(), [150], [1], 1.0)
    assert ((out.cpu().double() - want).abs() <= bound(want, mag, spread, P, D, torch.bfloat16, False)).all()


@pytest.mark.parametrize("p8", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype,B,T,G,P", [(torch.float32, 5, 1, 2, 3000), (torch.float32, 24, 4, 2, 333), (torch.float32, 9, 3, 3, 17),
                                           (torch.bfloat16, 5, 1, 3, 4100), (torch.bfloat16, 3, 5, 3, 130)])
def test_narrow_prefix(qd, p8, D, dtype, B, T, G, P):
    """Too few rows, or fp32 ones: a few rows of the batch at a time, the positions split over CTAs where they are many."""
    lengths = torch.randint(0, 40, (B,), generator=gen(P)).tolist()
    run(qd, "narrow", B, T, G, 2, D, 40, lengths, [min(T, n) for n in lengths], not p8, dtype, P=P, p8=p8, seed=P)


@pytest.mark.parametrize("q8", [True, False])
def test_narrow_prefix_of_the_caches_format(qd, q8):
    """Rows that fill a quarter or half of a tile stream by stream, and all of it together."""
    B, P = 64, 21000 if q8 else 10600
    run(qd, "narrow", B, 1, 1, 2, 64, 6, [b % 7 for b in range(B)], None, q8, torch.float32, P=P, p8=q8, seed=1)


@pytest.mark.parametrize("way,dtype,B,T", [("wide", torch.bfloat16, 40, 1), ("narrow", torch.float32, 40, 1)])
def test_prefix_passes_of_three_streams_at_a_time(qd, way, dtype, B, T):
    """Eager calls on two streams and a replayed capture on a third, no workspace given: the results stay bit for bit."""
    g = gen(45)
    dev, _ = _filled(g, B, 2, 300, 64, True)
    pdev, _ = _filled(g, 1, 2, 4000, 64, False)
    view, pre = qd.KvCache(*dev), qd.KvCache(*pdev)
    assert route(qd, view, pre, 4000, dtype == torch.bfloat16, T, 4) == way
    ln = ints(torch.randint(1, 300, (B,), generator=g).tolist())
    qs = [torch.randn((B, T, 4, 64), generator=g).to(dtype).cuda() for _ in range(3)]

    def call(q, out):
        qd.qd_attn_cached(q, view, ln, out, prefix=pre)
    want = [torch.empty_like(q) for q in qs]
    for q, o in zip(qs, want):
        call(q, o)
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


@pytest.mark.parametrize("dtype,D,rows", [(torch.float32, 128, 8), (torch.float32, 64, 16), (torch.bfloat16, 128, 16)])
def test_narrow_prefix_leaves_out_unused_rows(qd, dtype, D, rows):
    """A group of `rows` rows of the batch in which none is in use is not worked: its partials, which stand first in the
    workspace, (ref, sum) of [key head][row of the batch], stay as they were."""
    B, T, G, H, P, n_new = 5, 4, 2, 2, 20, [4, 0, 1, 0, 0]
    g = gen(8)
    q8 = dtype == torch.bfloat16
    dev, kv = _filled(g, B, H, 8, D, q8)
    pdev, pkv = _filled(g, 1, H, P, D, not q8)
    view, pre = qd.KvCache(*dev), qd.KvCache(*pdev)
    assert route(qd, view, pre, P, q8, T, G * H) == "narrow"
    ws = torch.full((qd.qd_attn_cached_workspace(view, q8, T, G * H, prefix=pre),), 0xAB, dtype=torch.uint8, device="cuda")
    q = torch.randn((B, T, G * H, D), generator=g).to(dtype)
    out = torch.full((B, T, G * H, D), 7.0, dtype=dtype, device="cuda")
    qd.qd_attn_cached(q.cuda(), view, ints([4] * B), out, n_new=ints(n_new), prefix=pre, workspace=ws)
    want, mag, spread = ref.attend(q, kv[0], kv[1], [4] * B, n_new, D ** -0.5, pkv[0][0], pkv[1][0])
    used = ~torch.isnan(want)
    assert ((out.cpu().double() - want).abs() <= bound(want, mag, spread, P + 4, D, dtype, False))[used].all()
    assert bool((out.cpu()[~used] == 7.0).all())
    n = B * T * G
    notes = ws.cpu()[:H * n * 8].view(H, n, 8)
    live = torch.tensor([t < n_new[b] for b in range(B) for t in range(T) for _ in range(G)])
    for r0 in range(0, n, rows):
        untouched = bool((notes[:, r0:r0 + rows] == 0xAB).all())
        assert untouched == (not live[r0:r0 + rows].any()), r0


@pytest.mark.parametrize("way,q8,dtype,T", [("wide", True, torch.bfloat16, 1), ("wide", False, torch.bfloat16, 3), ("narrow", True, torch.float32, 2),
                                            ("narrow", False, torch.float32, 1)])
@pytest.mark.parametrize("captured", [False, True])
def test_inputs_written_just_before_a_prefix_of_its_own_pass(qd, way, q8, dtype, T, captured):
    """Rows, lengths, counts and queries change directly before every call, whose pass over the streams' caches begins
    while the prefix's runs; the same call on finished inputs gives the same bits."""
    B, G, H, D, S, P, steps = 40, 2, 4, 128, 130, 2900, 30
    g = gen(92)
    dev, _ = _filled(g, B, H, S, D, q8)
    pdev, _ = _filled(g, 1, H, P, D, not q8)
    view, pre = qd.KvCache(*dev), qd.KvCache(*pdev)
    assert route(qd, view, pre, P, dtype == torch.bfloat16, T, G * H) == way
    rows = torch.randn((steps, 2, B, T, H, D), generator=g).to(dtype).cuda()
    qs = torch.randn((steps, B, T, G * H, D), generator=g).to(dtype).cuda()
    counts = torch.randint(0, T + 1, (steps, B), generator=g, dtype=torch.int32).cuda()
    at, row, q = torch.zeros((1,), dtype=torch.long, device="cuda"), torch.empty_like(rows[0]), torch.empty_like(qs[0])
    ln, nn = torch.zeros((B,), dtype=torch.int32, device="cuda"), torch.zeros((B,), dtype=torch.int32, device="cuda")
    out, again = torch.zeros_like(q), torch.zeros_like(q)
    ws = torch.empty((qd.qd_attn_cached_workspace(view, dtype == torch.bfloat16, T, G * H, prefix=pre),), dtype=torch.uint8, device="cuda")

    def step():
        row.copy_(rows.index_select(0, at)[0])
        nn.copy_(counts.index_select(0, at)[0])
        ln.add_(nn)
        q.copy_(qs.index_select(0, at)[0])
        qd.qd_kv_append(view, row[0], row[1], ln, n_new=nn)
        qd.qd_attn_cached(q, view, ln, out, n_new=nn, prefix=pre, workspace=ws)
        at.add_(1)

    if captured:
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        at.zero_()
        ln.zero_()
        out.zero_()
    for i in range(steps):
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        qd.qd_attn_cached(q, view, ln, again, n_new=nn, prefix=pre, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(out, again), i


def test_scratch_is_given_back_and_taken_anew(qd):
    g = gen(46)
    B = 40
    dev, _ = _filled(g, B, 2, 8, 64, True)
    pdev, _ = _filled(g, 1, 2, 600, 64, False)
    view, pre = qd.KvCache(*dev), qd.KvCache(*pdev)
    q, ln = torch.randn((B, 1, 4, 64), generator=g).bfloat16().cuda(), ints([8] * B)
    outs = [torch.zeros_like(q) for _ in range(2)]
    qd.release_scratch()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    qd.qd_attn_cached(q, view, ln, outs[0], prefix=pre)
    assert torch.cuda.memory_allocated() > before
    qd.release_scratch()                                  # the call may still run: its memory stays the stream's
    assert torch.cuda.memory_allocated() == before
    qd.qd_attn_cached(q, view, ln, outs[1], prefix=pre)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and bool(outs[0].float().abs().sum() > 0)
    qd.release_scratch()


@pytest.mark.parametrize("way,p8,B", [("wide", True, 24), ("wide", False, 24), ("narrow", True, 4), ("narrow", False, 4)])
def test_prefix_offsets_past_32_bits(qd, way, p8, B):
    """A prefix whose second head stands more than 2^32 bytes on, and whose rows are far apart."""
    g = gen(13)
    H, P, D, G = 2, 200, 128, 2
    e = 1 if p8 else 2
    (pdev, pkv), (dev, kv) = _filled(g, 1, H, P, D, p8), _filled(g, B, H, 4, D, not p8)
    step, row = 2 ** 32 // e + 2 ** 27, 2 ** 20
    far = []
    for x in pdev[:2]:
        y = torch.zeros(step + P * row, dtype=x.dtype, device="cuda").as_strided((1, H, P, D), (0, step, row, 1))
        far.append(y.copy_(x))
    view, pre = qd.KvCache(*dev), qd.KvCache(*far, *pdev[2:])
    q = torch.randn((B, 1, G * H, D), generator=g).bfloat16()
    out = torch.zeros((B, 1, G * H, D), dtype=torch.bfloat16, device="cuda")
    assert route(qd, view, pre, P, True, 1, G * H) == way
    qd.qd_attn_cached(q.cuda(), view, ints([4] * B), out, prefix=pre)
    want, mag, spread = ref.attend(q, kv[0], kv[1], [4] * B, [1] * B, D ** -0.5, pkv[0][0], pkv[1][0])
    tol = torch.maximum(bound(want, mag, spread, P + 4, D, torch.bfloat16, p8, way == "wide"),
                        bound(want, mag, spread, P + 4, D, torch.bfloat16, not p8))
    assert ((out.cpu().double() - want).abs() <= tol).all()
