"""qd_qk_norm_rope against a 64-bit form: types, layouts, pages, rows that are not in use, captures, streams."""
import numpy as np
import pytest
import torch

from tests._paged_ref import norm_rope, norm_rope_bound, place
from tests._serving_ref import quantise_rows

pytestmark = pytest.mark.gpu
EPS = 1e-6
MARK = 77.0                                     # what stands where nothing may be written


@pytest.fixture(scope="module")
def qd(cuda_ok):
    import transformer_autoregressive_decode_gb300 as m
    return m


def make(lengths, new, qh, kvh, hd, page, fmt, dtype, out, seed=0, slack=0, T=None, rows=None):
    """The call's tensors: packed where T is None, else T rows a stream.  slack: spare rows behind the last sequence."""
    g = torch.Generator().manual_seed(seed)
    B = len(lengths)
    N = (sum(new) + slack) if T is None else B * T
    fused = torch.randn((N, qh + 2 * kvh, hd), generator=g) * (0.1 + 3 * torch.rand((N, qh + 2 * kvh, 1), generator=g))
    if N > 2:
        fused[1, 0] = 0                         # a row of zeros (eps alone under the root)
        fused[2] *= 1e-4
    x = fused.to(dtype).cuda()
    per = max(1, (max(lengths, default=1) + page - 1) // page)
    n_pages = B * per + 1
    table = torch.randperm(n_pages, generator=g)[:B * per].reshape(B, per).to(torch.int32)
    rows = rows or max(lengths) + 3
    angle = torch.arange(rows, dtype=torch.float64)[:, None] * 1e6 ** (-torch.arange(0, hd, 2, dtype=torch.float64) / hd)
    st = dict(x=x, q=x[:, :qh], k=x[:, qh:qh + kvh], v=x[:, qh + kvh:], N=N, table=table.cuda(), cos=angle.cos().float().cuda(),
              sin=angle.sin().float().cuda(), lengths=torch.tensor(lengths, dtype=torch.int32).cuda(),
              q_gamma=(0.5 + torch.rand(hd, generator=g)).cuda(), k_gamma=(0.5 + torch.rand(hd, generator=g)).cuda())
    st |= {n: torch.full((N, h, hd), MARK, dtype=out).cuda() for n, h in (("q_out", qh), ("k_out", kvh), ("v_out", kvh))}
    if fmt == "q8":
        st |= {n: torch.full((n_pages, kvh, page, hd), 77, dtype=torch.int8).cuda() for n in ("kp", "vp")}
        st |= {n: torch.full((n_pages, kvh, page), MARK).cuda() for n in ("ks", "vs")}
    else:
        st |= {n: torch.full((n_pages, kvh, page, hd), MARK, dtype=torch.bfloat16).cuda() for n in ("kp", "vp")}
        st |= dict(ks=None, vs=None)
    if T is None:
        st["offsets"], st["n_new"] = torch.tensor([0, *np.cumsum(new)], dtype=torch.int32).cuda(), None
    else:
        st["offsets"], st["n_new"] = None, torch.tensor(new, dtype=torch.int32).cuda()
    return st


def call(qd, st, pages=True, **kw):
    a = {n: st[n] for n in ("cos", "sin", "lengths", "v", "k_out", "v_out", "q_gamma", "k_gamma", "offsets", "n_new")}
    if pages:
        a |= dict(pages=qd.KvCache(st["kp"], st["vp"], st["ks"], st["vs"]), page_table=st["table"])
    a |= kw
    qd.qd_qk_norm_rope(st["q"], st["k"], st["q_out"], eps=EPS, **a)


def rows_of(lengths, new, T):
    """Row of every new token."""
    at = np.concatenate([[0], np.cumsum(new)]) if T is None else np.arange(len(new) + 1) * T
    return [int(at[b]) + t for b in range(len(new)) for t in range(new[b])]


def check(st, lengths, new, T=None, pos=None, mrope_h=0, gammas=True, rotate=True, written=None):
    """Everything that the call wrote, and that it wrote nothing else.  written: which of the tokens reach the pages (all)."""
    hd = st["q"].shape[2]
    page = st["kp"].shape[2]
    rows = rows_of(lengths, new, T)
    at = [lengths[b] - new[b] + t for b in range(len(new)) for t in range(new[b])]
    c = s = None
    if rotate:
        if mrope_h:
            d = torch.arange(hd // 2)
            p = pos[torch.where(d < 3 * mrope_h, d % 3, 0)][:, rows].T.long()
            c, s = st["cos"].cpu()[p, d], st["sin"].cpu()[p, d]
        else:
            p = torch.tensor(at) if pos is None else pos[rows].long()
            c, s = st["cos"].cpu()[p], st["sin"].cpu()[p]
    want = {}
    for name in "qk":
        want[name] = norm_rope(st[name][rows].cpu(), st[name + "_gamma"].cpu() if gammas else None, EPS, c, s)
    v = st["v"][rows].cpu().double()
    want["v"] = (v, v.abs() * 0)
    idle = sorted(set(range(st["N"])) - set(rows))
    for name in "qkv":
        got = st[name + "_out"].cpu()
        assert (got[idle].double() == MARK).all()
        y, size = want[name]
        near = norm_rope_bound(size, hd) * (0 if name == "v" else 1)
        bound = near + torch.finfo(got.dtype).eps / 2 * (y.abs() + near)
        assert ((got[rows].double() - y).abs() <= bound).all(), name
    # the pages
    written = written or [True] * len(rows)
    where = [w for w, on in zip(place(lengths, new, page), written) if on]
    keep = torch.tensor([i for i, on in enumerate(written) if on], dtype=torch.long)
    table = st["table"].cpu()
    pg = torch.tensor([int(table[b, i]) for b, i, _ in where], dtype=torch.long)
    r = torch.tensor([w[2] for w in where], dtype=torch.long)
    rest = torch.ones((st["kp"].shape[0], page), dtype=torch.bool)
    rest[pg, r] = False
    for name, held, scale in (("k", "kp", "ks"), ("v", "vp", "vs")):
        cells = st[held].cpu()
        y, size = (t[keep] for t in want[name])
        near = norm_rope_bound(size, hd) * (0 if name == "v" else 1)
        got = cells[pg, :, r]
        if st[scale] is None:
            assert ((got.double() - y).abs() <= near + 2.0 ** -8 * (y.abs() + near)).all()
            assert (cells.transpose(1, 2)[rest].double() == MARK).all()
            continue
        sc = st[scale].cpu()
        assert (cells.transpose(1, 2)[rest] == 77).all() and (sc.transpose(1, 2)[rest] == MARK).all()
        if name == "v":                         # given rows: the definition bit for bit
            codes, scales = quantise_rows(y.float().numpy())
            assert np.array_equal(got.numpy(), codes) and np.array_equal(sc[pg, :, r].numpy(), scales)
            continue
        # half a code, what the row is off by, and the scale's and the quotient's roundings on up to 127 codes
        s64 = sc[pg, :, r].double()[..., None]
        assert ((got.double() * s64 - y).abs() <= 0.5 * s64 + near + 127 * s64 * 4 * 2.0 ** -24).all()
        top = y.abs().amax(-1)
        assert ((sc[pg, :, r].double() * 127 - top).abs() <= near.amax(-1) + top * 2 * 2.0 ** -24).all()


F, H = torch.float32, torch.bfloat16
SHAPES = [  # lengths, new, T, qh, kvh, hd, page
    ([1], [1], 1, 1, 1, 64, 16),
    ([5, 1, 300], [1, 1, 1], 1, 16, 8, 128, 16),
    ([17, 0, 4, 129], [3, 0, 1, 2], 3, 6, 2, 128, 64),
    ([16, 33, 1, 0, 48], [16, 33, 1, 0, 48], None, 16, 8, 128, 16),
    ([70, 200], [7, 131], None, 5, 5, 64, 32),
    ([260], [257], None, 40, 8, 128, 256),
    ([9, 9, 9], [4, 4, 4], 4, 24, 1, 64, 16),
]


@pytest.mark.parametrize("fmt", ["bf16", "q8"])
@pytest.mark.parametrize("dtype, out", [(F, F), (F, H), (H, H), (H, F)])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{s[3]}h{s[5]}")
def test_values(qd, shape, dtype, out, fmt):
    lengths, new, T, qh, kvh, hd, page = shape
    st = make(lengths, new, qh, kvh, hd, page, fmt, dtype, out, T=T, slack=3)
    call(qd, st)
    check(st, lengths, new, T)


@pytest.mark.parametrize("how", ["plain positions", "three streams", "no rotation", "no norm", "no cache", "no streams"])
def test_forms(qd, how):
    lengths, new, T = [40, 3, 25], [7, 3, 20], None
    st = make(lengths, new, 8, 2, 128, 16, "bf16", F, H, rows=64)
    N = st["N"]
    g = torch.Generator().manual_seed(3)
    if how == "plain positions":
        pos = torch.randint(0, 64, (N,), generator=g, dtype=torch.int32)
        call(qd, st, positions=pos.cuda())
        check(st, lengths, new, T, pos=pos)
    elif how == "three streams":
        pos = torch.randint(0, 64, (3, N), generator=g, dtype=torch.int32)
        for h in (20, 5, 21):
            call(qd, st, positions=pos.cuda(), mrope_h=h)
            check(st, lengths, new, T, pos=pos, mrope_h=h)
    elif how == "no rotation":
        call(qd, st, cos=None, sin=None)
        check(st, lengths, new, T, rotate=False)
    elif how == "no norm":
        call(qd, st, q_gamma=None, k_gamma=None)
        check(st, lengths, new, T, gammas=False)
    else:
        pos = torch.randint(0, 64, (N,), generator=g, dtype=torch.int32)
        more = dict(positions=pos.cuda())
        if how == "no streams":
            more |= dict(lengths=None, offsets=None)
        call(qd, st, pages=False, **more)
        check(st, lengths, new, T, pos=pos, written=[False] * N)


def test_rows_without_v_or_k_out(qd):
    st = make([9, 9], [1, 1], 4, 2, 64, 16, "bf16", H, H, T=1)
    call(qd, st, pages=False, v=None, v_out=None, k_out=None)
    assert (st["k_out"].cpu() == MARK).all() and (st["v_out"].cpu() == MARK).all() and not (st["q_out"].cpu() == MARK).any()


@pytest.mark.parametrize("hd", [64, 128])
def test_in_place_and_between(qd, hd):
    lengths, new = [30, 11], [12, 11]
    a, b = (make(lengths, new, 6, 2, hd, 16, "q8", H, H) for _ in "ab")
    call(qd, a)
    x = b["x"].clone()
    for n in "qkv":
        b[n + "_out"] = b[n]
    call(qd, b)
    for n in "qkv":
        assert torch.equal(a[n + "_out"], b[n])
    assert torch.equal(a["kp"], b["kp"]) and torch.equal(a["vs"], b["vs"])
    # results between the rows of another array
    wide = torch.full((23, 20, hd), MARK, dtype=H).cuda()
    wide[:, :10] = x
    b |= dict(q=wide[:, :6], k=wide[:, 6:8], v=wide[:, 8:10], q_out=wide[:, 10:16], k_out=wide[:, 16:18], v_out=wide[:, 18:])
    call(qd, b)
    assert torch.equal(wide[:, 10:16], a["q_out"]) and torch.equal(wide[:, 16:18], a["k_out"]) and torch.equal(wide[:, :10], x)


@pytest.mark.parametrize("fmt", ["bf16", "q8"])
def test_places_outside(qd, fmt):
    """Positions behind the tables, pages outside the pool, counts and lengths that make no sense."""
    lengths, new = [40, 3, 25, 20], [7, 3, 20, 2]
    st = make(lengths, new, 4, 2, 64, 16, fmt, F, F, rows=64)
    st["table"][0, 2] = -1                      # positions 32 .. 47 of stream 0: its tokens from 33 on
    st["table"][2, 0] = st["kp"].shape[0]       # positions 0 .. 15 of stream 2
    on = [t[1] != 2 if t[0] == 0 else t[0] != 2 or t[1] != 0 for t in place(lengths, new, 16)]
    assert 0 < sum(on) < len(on)
    call(qd, st)
    check(st, lengths, new, None, written=on)
    # a length past the table's pages: rotated as usual, written nowhere
    st = make([40], [4], 2, 1, 64, 16, fmt, F, F, rows=64)
    st["table"] = st["table"][:, :2].contiguous()
    call(qd, st)
    check(st, [40], [4], None, written=[False] * 4)
    # a position outside cos and sin: NaN, by token
    st = make([6], [6], 2, 1, 64, 16, "bf16", F, F, rows=64)
    call(qd, st, positions=torch.tensor([0, -1, 63, 64, 5, 1 << 30], dtype=torch.int32).cuda())
    nan = st["q_out"].cpu().isnan()
    assert nan[[1, 3, 5]].all() and not nan[[0, 2, 4]].any() and not st["v_out"].isnan().any()


def test_rows_that_are_not_finite(qd):
    st = make([4], [4], 2, 2, 64, 16, "q8", F, F)
    st["x"][1, 2, 5] = float("inf")             # key head 0
    st["x"][2, 5, 7] = float("nan")             # value head 1
    call(qd, st)
    p = int(st["table"][0, 0])
    ks, vs = st["ks"].cpu()[p], st["vs"].cpu()[p]
    assert ks[0, 1].isnan() and not ks[0, [0, 2, 3]].isnan().any() and not ks[1, :4].isnan().any()
    assert vs[1, 2].isnan() and not vs[0, :4].isnan().any()
    assert (st["kp"].cpu()[p, 0, 1] == 0).all() and (st["vp"].cpu()[p, 1, 2] == 0).all()


def test_page_order_and_strides(qd):
    """Pools of [pages, page, heads, dim], tables with longer rows, spare tokens' strides."""
    lengths, new = [50, 18], [50, 2]
    a, b = (make(lengths, new, 4, 2, 128, 16, "bf16", H, H) for _ in "ab")
    call(qd, a)
    kp, vp = (torch.full((b["kp"].shape[0], 16, 2, 128), MARK, dtype=H).cuda() for _ in "kv")
    b["kp"], b["vp"] = kp.transpose(1, 2), vp.transpose(1, 2)
    wide = torch.full((2, 9), -5, dtype=torch.int32).cuda()
    wide[:, :b["table"].shape[1]] = b["table"]
    b["table"] = wide[:, :b["table"].shape[1]]
    call(qd, b)
    assert torch.equal(a["kp"], b["kp"]) and torch.equal(a["vp"], b["vp"]) and torch.equal(a["q_out"], b["q_out"])


def test_far_pages(qd):
    """A pool whose last pages stand more than 2^32 bytes from its first."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("memory")
    page, n = 1024, 4200                        # 4200 x 8 x 1024 x 128 codes: 4.4 GB each
    kp, vp = (torch.zeros((n, 8, page, 128), dtype=torch.int8, device="cuda") for _ in "kv")
    ks, vs = (torch.zeros((n, 8, page), device="cuda") for _ in "kv")
    st = make([5000, 20], [3, 20], 16, 8, 128, page, "q8", F, H)
    far = torch.tensor([[n - 1, n - 2, n - 3, n - 4, n - 5], [7, 6, 5, 4, 3]], dtype=torch.int32)
    qd.qd_qk_norm_rope(st["q"], st["k"], st["q_out"], st["cos"], st["sin"], st["lengths"], v=st["v"], q_gamma=st["q_gamma"], k_gamma=st["k_gamma"],
                       eps=EPS, offsets=st["offsets"], pages=qd.KvCache(kp, vp, ks, vs), page_table=far.cuda())
    at = [(n - 5, 4997 - 4096 + t) for t in range(3)] + [(7, t) for t in range(20)]
    codes, scales = quantise_rows(st["v"].float().cpu().numpy())
    for i, (p, r) in enumerate(at):
        assert np.array_equal(vp[p, :, r].cpu().numpy(), codes[i]) and np.array_equal(vs[p, :, r].cpu().numpy(), scales[i])
    assert int((vs != 0).sum()) == 23 * 8 and int((ks != 0).sum()) == 23 * 8


def test_captured_steps_grow(qd):
    lengths, new = [14, 30, 3], [1, 1, 1]
    st = make([20, 36, 9], new, 16, 8, 128, 16, "bf16", H, H, T=1)
    st["lengths"].copy_(torch.tensor(lengths))
    graph = torch.cuda.CUDAGraph()
    call(qd, st)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call(qd, st)
    for n in ("kp", "vp"):
        st[n].fill_(MARK)
    for step in range(4):
        st["x"].copy_(torch.randn(st["x"].shape, generator=torch.Generator().manual_seed(step)).to(H))
        for n in ("kp", "vp"):
            st[n].fill_(MARK)
        st["lengths"].copy_(torch.tensor([n + step for n in lengths]))
        graph.replay()
        torch.cuda.synchronize()
        check(st, [n + step for n in lengths], new, 1)


def test_two_streams(qd):
    sts = [make([200, 90], [200, 90], 16, 8, 128, 16, "bf16", F, H, seed=i) for i in range(2)]
    side = [torch.cuda.Stream() for _ in sts]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, s in zip(sts, side):
            call(qd, st, stream=s)
    with torch.cuda.stream(side[0]):
        call(qd, sts[0])
    torch.cuda.synchronize()
    for st in sts:
        check(st, [200, 90], [200, 90])
