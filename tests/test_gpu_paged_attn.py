"""qd_attn_paged against a 64-bit form, and bit for bit against qd_attn_cached over the same positions laid out
contiguously: types, page sizes, lengths from 0, shared and foreign pages, rubbish in unseen places, captures, streams."""
import numpy as np
import pytest
import torch

from tests._serving_ref import attend, attend_bound, quantise_rows

pytestmark = pytest.mark.gpu
F, H = torch.float32, torch.bfloat16
MARK = 55.0


@pytest.fixture(scope="module")
def qd(cuda_ok):
    import transformer_autoregressive_decode_gb300 as m
    return m


class Case:
    """A cache laid out contiguously and the same in pages in random order, of a pool with pages to spare full of NaN."""

    def __init__(self, lengths, new, T, qh, kvh, hd, page, fmt, dtype, seed=0, most=None):
        g = torch.Generator().manual_seed(seed)
        B = len(lengths)
        most = most or max(max(lengths), 1)
        per = (most + page - 1) // page
        S = per * page
        k = torch.randn((B, kvh, S, hd), generator=g) * (1 + 2 * (torch.rand((1, kvh, 1, hd), generator=g) > 0.9))
        v = torch.randn((B, kvh, S, hd), generator=g) * (0.25 + torch.rand((B, kvh, S, 1), generator=g))
        n = B * per + 3
        ids = torch.randperm(n, generator=g)
        table = ids[:B * per].reshape(B, per)
        self.lengths, self.new, self.most, self.page, self.fmt = lengths, new, most, page, fmt
        self.q = (1.5 * torch.randn((B, T, qh, hd), generator=g)).to(dtype)
        seen = torch.arange(S) < torch.tensor(lengths)[:, None]            # positions that hold something
        if fmt == "q8":
            (kc, ks), (vc, vs) = (quantise_rows(t.numpy()) for t in (k, v))
            kc, ks, vc, vs = (torch.from_numpy(t) for t in (kc, ks, vc, vs))
            self.k64, self.v64 = kc.double() * ks.double()[..., None], vc.double() * vs.double()[..., None]
            ks, vs = (torch.where(seen[:, None], t, torch.full_like(t, float("nan"))) for t in (ks, vs))
            cont = (kc, vc, ks, vs)
        else:
            k, v = k.to(H), v.to(H)
            self.k64, self.v64 = k.double(), v.double()
            cont = tuple(torch.where(seen[:, None, :, None], t, torch.full_like(t, float("nan"))) for t in (k, v)) + (None, None)
        self.cont = tuple(None if t is None else t.cuda() for t in cont)

        def paged(t):
            if t is None:
                return None
            p = torch.full((n, kvh, page, *t.shape[3:]), 77 if t.dtype == torch.int8 else float("nan"), dtype=t.dtype)
            for b in range(B):
                p[table[b]] = t[b].reshape(kvh, per, page, *t.shape[3:]).transpose(0, 1)
            return p.cuda()
        self.pool = tuple(paged(t) for t in cont)
        self.table = table.to(torch.int32).cuda()
        # what is named beyond a stream's length is not looked at
        for b in range(B):
            self.table[b, (lengths[b] + page - 1) // page:] = -7
        self.len_d = torch.tensor(lengths, dtype=torch.int32).cuda()
        self.new_d = torch.tensor(new, dtype=torch.int32).cuda()

    def run(self, qd, **kw):
        q = self.q.cuda()
        out = torch.full_like(q, MARK)
        qd.qd_attn_paged(q, qd.KvCache(*self.pool), self.table, self.len_d, out, n_new=self.new_d, max_length=self.most, **kw)
        return out

    def run_contiguous(self, qd, **kw):
        q = self.q.cuda()
        out = torch.full_like(q, MARK)
        qd.qd_attn_cached(q, qd.KvCache(*self.cont), self.len_d, out, n_new=self.new_d, max_length=self.most, **kw)
        return out

    def check(self, out):
        scale = self.q.shape[3] ** -0.5
        want, mag, spread = attend(self.q, self.k64, self.v64, self.lengths, self.new, scale)
        got = out.cpu().double()
        used = ~want.isnan()
        bound = attend_bound(want, mag, spread, max(self.lengths), self.q.shape[3], self.q.dtype, self.fmt == "q8")
        assert (got[~used] == MARK).all()
        off = ((got - want).abs() - bound)[used]
        assert (off <= 0).all(), float(off.max())


SHAPES = [  # lengths, new, T, qh, kvh, hd, page
    ([1], [1], 1, 2, 2, 64, 16),
    ([600], [1], 1, 16, 8, 128, 16),
    ([0, 1, 15, 16, 17, 31, 32, 33], [0, 1, 1, 1, 1, 1, 1, 1], 1, 4, 2, 128, 16),
    ([130, 0, 64, 65, 3], [3, 0, 4, 2, 3], 4, 6, 2, 64, 32),
    ([257, 5, 140], [1, 5, 0], 5, 24, 1, 128, 128),
    ([33, 70], [8, 8], 8, 8, 8, 64, 64),
    ([2000] + [50, 900] * 8, [1] * 17, 1, 8, 4, 128, 16),
    ([700] * 24 + [1] * 40, [2] * 24 + [1] * 40, 2, 8, 8, 64, 64),
]


@pytest.mark.parametrize("fmt", ["bf16", "q8"])
@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}of{max(s[0])}x{s[2]}x{s[3]}h{s[5]}p{s[6]}")
def test_values(qd, shape, dtype, fmt):
    c = Case(*shape, fmt, dtype)
    out = c.run(qd)
    c.check(out)
    assert torch.equal(out, c.run_contiguous(qd))


@pytest.mark.parametrize("fmt", ["bf16", "q8"])
@pytest.mark.parametrize("page", [16, 32, 256, 2048])
@pytest.mark.parametrize("lengths, T, qh, kvh, hd", [([30000, 17, 9000], 1, 32, 8, 128), ([5000] * 30, 1, 8, 2, 64),
                                                     ([300, 2, 1500, 800] * 16, 3, 12, 4, 64), ([2500, 1000] * 20, 2, 16, 2, 128)])
def test_shared_out(qd, lengths, T, qh, kvh, hd, page, fmt):
    """Sizes at which the tiles are shared out over all warps, runs that begin and end inside pages."""
    new = [min(n, T) for n in lengths]
    for dtype in (H, F):
        c = Case(lengths, new, T, qh, kvh, hd, page, fmt, dtype)
        assert qd.qd_attn_paged_workspace(qd.KvCache(*c.pool), len(lengths), c.table.shape[1], dtype == H, T, qh, c.most) > 0
        assert torch.equal(c.run(qd), c.run_contiguous(qd))


def test_shared_out_values(qd):
    c = Case([4000, 17, 900] + [3] * 20, [1] * 23, 1, 16, 8, 128, 32, "q8", F)
    assert qd.qd_attn_paged_workspace(qd.KvCache(*c.pool), 23, c.table.shape[1], False, 1, 16, c.most) > 0
    c.check(c.run(qd))


@pytest.mark.parametrize("page_id", [-1, 1 << 30, None])
@pytest.mark.parametrize("fmt", ["bf16", "q8"])
@pytest.mark.parametrize("lengths", [[100, 90, 40], [9000, 4000, 300] + [20] * 30], ids=["clusters", "shared out"])
def test_pages_outside_the_pool(qd, lengths, fmt, page_id):
    c = Case(lengths, [2] * len(lengths), 2, 8, 4, 64, 16, fmt, H)
    want = c.run(qd)
    c.table[1, 2] = c.pool[0].shape[0] if page_id is None else page_id
    got = c.run(qd)
    assert got[1].isnan().all()
    keep = [0] + list(range(2, len(lengths)))
    assert torch.equal(got[keep], want[keep])


def test_streams_share_pages(qd):
    """A common prompt's pages named by every stream."""
    c = Case([80, 70, 75], [1, 1, 1], 1, 4, 2, 128, 16, "bf16", H)
    for t in c.cont[:2]:
        t[1:, :, :64] = t[:1, :, :64]
    c.table[1:, :4] = c.table[:1, :4]
    assert torch.equal(c.run(qd), c.run_contiguous(qd))


def test_orders_and_strides(qd):
    c = Case([90, 33], [2, 1], 2, 8, 4, 128, 32, "bf16", F)
    want = c.run(qd)
    c.pool = tuple(None if t is None else t.transpose(1, 2).contiguous().transpose(1, 2) for t in c.pool)   # pages of whole tokens
    wide = torch.full((2, 12), -9, dtype=torch.int32).cuda()
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide[:, :c.table.shape[1]]
    assert torch.equal(c.run(qd), want)
    # queries and results of a fused projection
    q = torch.zeros((2, 2, 24, 128)).cuda()
    q[:, :, 3:11] = c.q.cuda()
    qd.qd_attn_paged(q[:, :, 3:11], qd.KvCache(*c.pool), c.table, c.len_d, q[:, :, 13:21], n_new=c.new_d, max_length=c.most)
    used = want != MARK
    assert torch.equal(q[:, :, 13:21][used], want[used]) and (q[:, :, 13:21][~used] == 0).all()


def test_far_pages(qd):
    """Pages more than 2^32 bytes apart."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("memory")
    n, page = 4200, 1024
    c = Case([1500, 3000], [1, 1], 1, 16, 8, 128, page, "bf16", H)
    want = c.run(qd)
    far = [3, n - 1, n - 2, 2000, n - 7]
    k, v = (torch.empty((n, 8, page, 128), dtype=H, device="cuda") for _ in "kv")
    table = torch.full_like(c.table, -1)
    for at, (b, i) in zip(far, [(0, 0), (0, 1), (1, 0), (1, 1), (1, 2)]):
        k[at], v[at] = c.pool[0][int(c.table[b, i])], c.pool[1][int(c.table[b, i])]
        table[b, i] = at
    c.pool, c.table = (k, v, None, None), table
    assert torch.equal(c.run(qd), want)


@pytest.mark.parametrize("lengths", [[20, 40, 1], [6000, 2500] + [30] * 40], ids=["clusters", "shared out"])
def test_captured_steps_grow(qd, lengths):
    """One graph serves growing streams, whose pages and lengths change between replays."""
    B = len(lengths)
    full = Case([n + 40 for n in lengths], [1] * B, 1, 8, 4, 64, 16, "bf16", H)
    q, out = full.q.cuda(), torch.full((B, 1, 8, 64), MARK, dtype=H).cuda()
    view = qd.KvCache(*full.pool)
    lens, table = torch.tensor(lengths, dtype=torch.int32).cuda(), full.table.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qd.qd_attn_paged(q, view, table, lens, out, max_length=full.most)
    for step in (0, 1, 39):
        lens.copy_(torch.tensor([n + step for n in lengths]))
        table.copy_(full.table)
        for b in range(B):
            table[b, (lengths[b] + step + 15) // 16:] = -1
        out.fill_(MARK)
        graph.replay()
        torch.cuda.synchronize()
        now = out.clone()
        ref = torch.full_like(out, MARK)
        qd.qd_attn_cached(q, qd.KvCache(*full.cont), lens, ref, max_length=full.most)
        assert torch.equal(now, ref)


def test_two_streams_and_workspaces(qd):
    cs = [Case([5000, 300] + [9] * 40, [1] * 42, 1, 16, 8, 64, 16, "q8", H, seed=i) for i in range(2)]
    want = [c.run(qd) for c in cs]
    side = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for c, s in zip(cs, side):
            with torch.cuda.stream(s):
                outs.append(c.run(qd))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, want[i % 2])
    # a workspace of the caller's, and one that is too small
    c = cs[0]
    need = qd.qd_attn_paged_workspace(qd.KvCache(*c.pool), 42, c.table.shape[1], True, 1, 16, c.most)
    assert torch.equal(c.run(qd, workspace=torch.empty(need, dtype=torch.uint8, device="cuda")), want[0])
    with pytest.raises(qd.QDError):
        c.run(qd, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


def test_new_tokens_that_are_not_finite(qd):
    """A drafted token's infinite value reaches the queries that see it and no other."""
    for fmt in ("bf16", "q8"):
        c = Case([50, 20], [4, 4], 4, 4, 2, 64, 16, fmt, H)
        want = c.run(qd)
        p, r = int(c.table[0, 48 // 16]), 48 % 16          # stream 0, token 2
        if fmt == "q8":
            c.pool[3][p, 1, r] = float("inf")
        else:
            c.pool[1][p, 1, r, 7] = float("inf")
        got = c.run(qd)
        assert torch.equal(got[1], want[1]) and torch.equal(got[0, :2], want[0, :2]) and torch.equal(got[0, :, :2], want[0, :, :2])
        assert not got[0, 2:, 2:, 7].isfinite().any()


def test_empty_and_odd_lengths(qd):
    """Lengths below zero and above the bound are taken as the nearest end; no position seen gives zeros."""
    c = Case([64, 64, 64], [1, 1, 1], 1, 4, 2, 64, 16, "bf16", F)
    want = c.run(qd)
    c.len_d.copy_(torch.tensor([-5, 1000, 0]))
    got = c.run(qd)
    assert (got[0] == 0).all() and (got[2] == 0).all() and torch.equal(got[1], want[1])


@pytest.mark.parametrize("rows", [1, 64])
def test_infinite_scales_of_contiguous_caches(qd, rows):
    """A row whose scale is infinite makes what sees it infinite or NaN, not zero: in a stream's own cache and in a prefix
    (a few rows at a time, or many on the tensor cores)."""
    B = rows
    c = Case([40] * B, [1] * B, 1, 16, 8, 64, 16, "q8", H)
    c.cont[3][0, 1, 5] = float("inf")
    assert not c.run_contiguous(qd)[0, 0, 2:4].isfinite().any()
    p = Case([2000], [1], 1, 16, 8, 64, 16, "q8", H)
    p.cont[3][0, 1, 1500] = float("inf")
    own = Case([40] * B, [1] * B, 1, 16, 8, 64, 16, "q8", H)
    got = own.run_contiguous(qd, prefix=qd.KvCache(*p.cont), prefix_length=1990)
    assert not got[:, 0, 2:4].isfinite().any() and got[:, 0, :2].isfinite().all()
