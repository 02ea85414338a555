"""qd_attn_prompt against a 64-bit form: lengths from none, chunks with earlier keys, head groups that fill a tile or do not,
values that are not finite in unseen places, scores that outgrow their reference, layouts, captures, streams."""
import numpy as np
import pytest
import torch

from tests._paged_ref import prompt, prompt_bound, prompt_norm_bound

pytestmark = pytest.mark.gpu
H = torch.bfloat16
MARK = 33.0


@pytest.fixture(scope="module")
def qd(cuda_ok):
    import transformer_autoregressive_decode_gb300 as m
    return m


def make(lens, klens, qh, kvh, hd, seed=0, slack=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    N, M = sum(lens) + slack, (sum(klens) if klens else sum(lens)) + slack
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    loud = 1 + 2 * (torch.rand((1, kvh, hd), generator=g, device="cuda") > 0.94)
    st = dict(q=(1.5 * rnd(N, qh, hd)).to(H), k=(rnd(M, kvh, hd) * loud).to(H), v=rnd(M, kvh, hd).to(H),
              out=torch.full((N, qh, hd), MARK, dtype=H, device="cuda"))
    st["offs"] = [0, *np.cumsum(lens).tolist()]
    st["koffs"] = [0, *np.cumsum(klens).tolist()] if klens else st["offs"]
    st["offsets"] = torch.tensor(st["offs"], dtype=torch.int32).cuda()
    st["kv_offsets"] = torch.tensor(st["koffs"], dtype=torch.int32).cuda() if klens else None
    return st


def call(qd, st, **kw):
    qd.qd_attn_prompt(st["q"], st["k"], st["v"], st["out"], st["offsets"], kv_offsets=st["kv_offsets"], **kw)
    return st["out"]


def check(st, scale=None, norm=True):
    hd = st["q"].shape[2]
    want, mag, noise, spread = prompt(st["q"], st["k"], st["v"], st["offs"], st["koffs"], hd ** -0.5 if scale is None else scale)
    got = st["out"].double()
    used = ~want[:, 0, 0].isnan()
    assert (got[~used] == MARK).all()
    most = max(b - a for a, b in zip(st["koffs"], st["koffs"][1:]))
    off = ((got - want).abs() - prompt_bound(want, mag, spread, most, hd))[used]
    assert (off <= 0).all(), float(off.max())
    if norm and used.any():
        assert (got - want)[used].norm() <= prompt_norm_bound(want[used], noise[used])


SHAPES = [  # lens, klens, qh, kvh, hd
    ([1], None, 1, 1, 64),
    ([1], None, 16, 8, 128),
    ([64], None, 16, 8, 128),
    ([128], None, 2, 2, 128),
    ([129, 127, 128], None, 4, 4, 64),
    ([257], None, 1, 1, 128),
    ([500], None, 6, 2, 128),                               # 3 heads a group: 126 rows a tile
    ([333, 2], None, 5, 1, 64),                             # 5: 125 rows
    ([200], None, 7, 1, 128),
    ([90, 31], None, 24, 2, 64),                            # 12: 120 rows
    ([70], None, 128, 1, 64),                               # a token a tile
    ([9], None, 100, 1, 128),
    ([700], None, 32, 4, 128),
    ([0, 3, 0, 0, 130, 1, 0], None, 4, 2, 128),             # sequences of none
    ([1, 2, 3, 5, 8, 13, 21, 34, 55, 89, 144, 233], None, 8, 2, 64),
    ([40, 300], [900, 1300], 4, 2, 128),                    # chunks of longer prompts
    ([1, 1, 1], [1000, 1, 129], 8, 4, 64),                  # single tokens
    ([130, 64], [131, 64 + 127], 3, 3, 128),
    ([200, 50], [70, 50], 4, 2, 64),                        # more queries than keys: the first see none
    ([300, 20, 5], [0, 10, 5], 2, 1, 128),                  # no keys at all
    ([300], [150], 1, 1, 128),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{'-'.join(map(str, s[0]))[:24]}x{s[2]}of{s[3]}h{s[4]}{'k' if s[1] else ''}")
def test_values(qd, shape):
    st = make(*shape, slack=5)
    call(qd, st)
    check(st, norm=st["q"].numel() > 20000)


@pytest.mark.parametrize("lens, klens, qh, kvh, hd", [
    ([2000, 1], None, 16, 8, 128), ([512] * 8, None, 16, 8, 128), (list(range(1, 600, 17)), None, 8, 8, 64), ([3000], None, 32, 4, 128),
    ([100] * 70, None, 6, 2, 64), ([700, 300, 1000], [3000, 5000, 1000], 12, 4, 128), ([1] * 400, None, 4, 4, 64),
    ([4100], None, 4, 4, 64), ([40] * 1500, None, 1, 1, 64), ([9000], None, 6, 6, 128), ([1900, 2000], [2500, 4001], 18, 6, 64),
    ([20000, 17, 3000], None, 4, 2, 64), ([5000, 4000], [6000, 4000], 40, 8, 128), ([33] * 300, [33 + i for i in range(300)], 16, 8, 64)])
def test_many_pairs(qd, lens, klens, qh, kvh, hd):
    """More pairs of tiles than SMs, dealt out by every CTA for itself or, beyond 256 pairs or 16 an SM, taken from a sorted list."""
    st = make(lens, klens, qh, kvh, hd, slack=3)
    N, M = st["q"].shape[0], st["k"].shape[0]
    pairs = N // (2 * (128 // (qh // kvh))) + len(lens)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    listed = pairs > 256 or len(lens) > 256 or pairs * kvh > 16 * sms
    cut = not listed and pairs * kvh <= sms + sms // 4 and M >= 2048 * len(lens)      # may be cut into pieces
    assert (qd.qd_attn_prompt_workspace(N, M, len(lens), qh, kvh, hd) > 0) == (listed or cut)
    call(qd, st)
    check(st)


@pytest.mark.parametrize("lens, klens, qh, kvh, hd", [
    ([3000], None, 1, 1, 128), ([5000], None, 2, 2, 64), ([1], [9000], 4, 2, 64), ([300], [7000], 8, 2, 128), ([128, 256], [4000, 8000], 3, 3, 64),
    ([1, 64, 0, 700], [4097, 6400, 10, 5000], 4, 4, 128), ([2300, 40, 1], None, 6, 2, 64), ([600] * 6, [3600] * 6, 8, 8, 128), ([250], [3000], 100, 1, 64),
    ([50], [3], 1, 1, 64), ([600, 300], [100, 9000], 2, 2, 64), ([897, 400, 30], [141, 8000, 0], 3, 1, 128)])
def test_pieces(qd, lens, klens, qh, kvh, hd):
    """Few pairs over long keys: cut into equal runs of chunks, joined."""
    st = make(lens, klens, qh, kvh, hd, slack=2)
    call(qd, st)
    check(st)
    if klens and sum(klens) > 3000:             # pieces in which a row sees nothing, and rising scores between them
        st["k"][:, :, :] *= 0.2
        at = st["koffs"][-1] - 1
        st["k"][at] = st["q"][st["offs"][-1] - 1, ::qh // kvh] * 5.0
        call(qd, st)
        check(st, norm=False)


def test_pieces_and_values_that_are_not_finite(qd):
    st = make([300], [7000], 8, 2, 128, slack=60)
    want = call(qd, st).clone()
    st["v"][7000:], st["v"][6900, 1, 5] = float("nan"), float("inf")
    st["out"].fill_(MARK)
    call(qd, st)
    got = st["out"]
    mask = torch.zeros(got.shape, dtype=torch.bool, device="cuda")
    mask[200:300, 4:, 5] = True                 # query i sees keys up to 6700 + i
    assert not got[mask].isfinite().any() and (got[300:] == MARK).all()
    assert torch.equal(got[:300][~mask[:300]], want[:300][~mask[:300]])


@pytest.mark.parametrize("hd", [64, 128])
def test_scales(qd, hd):
    for scale in (0.0, -0.3, 2.0):
        st = make([300, 50], None, 4, 2, hd)
        call(qd, st, scale=scale)
        check(st, scale=scale, norm=False)


@pytest.mark.parametrize("at", [40, 70, 127, 128, 200, 390, 449])
def test_rising_scores(qd, at):
    """A key whose score is beyond 2^80 times the ones before it: in a first half, a second half, a later chunk, the last key."""
    st = make([450], None, 4, 2, 128)
    st["k"][:, :, :] *= 0.1
    st["k"][at] = st["q"][449, ::2] * 5.0
    call(qd, st)
    check(st, norm=False)
    st["k"][at] = -st["k"][at]                  # and far below them
    call(qd, st)
    check(st, norm=False)


def test_every_chunk_rises(qd):
    st = make([700], None, 2, 2, 64)
    st["q"][:] = 1.0
    st["k"][:] = (torch.arange(700, device="cuda", dtype=torch.float32)[:, None, None] * 0.2).to(H)   # scores up to 1120 in natural units
    call(qd, st)
    check(st, norm=False)
    st["k"][:] = -st["k"]
    call(qd, st)
    check(st, norm=False)


def test_lowest_scores(qd):
    """All scores far below zero, and all -infinity up to a later key."""
    st = make([300], None, 2, 1, 64)
    st["q"][:], st["k"][:] = 8.0, -30.0
    call(qd, st)
    check(st, norm=False)
    st["k"][:200] = float("-inf")
    call(qd, st)
    got = st["out"]
    assert not got[:200].isfinite().any()       # every weight is 0 / 0 there: the plain form's NaN
    want = torch.cumsum(st["v"][200:].double(), 0) / torch.arange(1, 101, device="cuda")[:, None, None]
    assert (got[200:].double() - want).abs().max() < 0.05 and got[200:].isfinite().all()


@pytest.mark.parametrize("qh, kvh, hd", [(1, 1, 64), (4, 2, 128), (6, 2, 64)])
@pytest.mark.parametrize("what", ["inf", "nan", "-inf"])
def test_unseen_values_that_are_not_finite(qd, what, qh, kvh, hd):
    lens = [150, 60, 260]
    st = make(lens, None, qh, kvh, hd, slack=8)
    call(qd, st)
    want = st["out"].clone()
    at = [(0, 100), (1, 59), (2, 0), (2, 128), (2, 200)]
    for b, j in at:
        st["v"][st["offs"][b] + j, kvh - 1, 3] = float(what)
    st["v"][sum(lens):] = float(what)           # behind the last sequence, where a tile of keys reaches
    st["out"].fill_(MARK)
    call(qd, st)
    G = qh // kvh
    for b in range(3):
        rows = slice(st["offs"][b], st["offs"][b + 1])
        first = min(j for s, j in at if s == b)
        i = torch.arange(lens[b], device="cuda")
        got, ref = st["out"][rows], want[rows]
        mask = torch.zeros(got.shape, dtype=torch.bool, device="cuda")
        mask[i >= first, -G:, 3] = True
        assert not got[mask].isfinite().any()
        assert torch.equal(got[~mask], ref[~mask])
    assert (st["out"][sum(lens):] == MARK).all()


def test_unseen_keys_that_are_not_finite(qd):
    st = make([150, 60], None, 4, 2, 64, slack=8)
    call(qd, st)
    want = st["out"].clone()
    st["k"][100], st["k"][210:] = float("nan"), float("nan")
    call(qd, st)
    assert torch.equal(st["out"][:100], want[:100]) and torch.equal(st["out"][150:], want[150:])
    assert st["out"][100:150].isnan().all()


def test_fused_rows_and_results_between(qd):
    st = make([77, 300], None, 4, 2, 128)
    want = call(qd, st).clone()
    wide = torch.full((377, 14, 128), MARK, dtype=H, device="cuda")
    wide[:, :4], wide[:, 4:6], wide[:, 6:8] = st["q"], st["k"], st["v"]
    before = wide.clone()
    st |= dict(q=wide[:, :4], k=wide[:, 4:6], v=wide[:, 6:8], out=wide[:, 9:13])
    call(qd, st)
    assert torch.equal(wide[:, 9:13], want)
    before[:, 9:13] = want
    assert torch.equal(wide, before)


def test_far_rows(qd):
    """Tokens more than 2^32 bytes apart."""
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("memory")
    n, stride = 600, 1 << 23                    # 16 MB a token: 10 GB
    big = torch.empty(n * stride, dtype=H, device="cuda")
    st = make([n - 10], None, 2, 1, 64)
    want = call(qd, st).clone()
    view = lambda at, h: big.as_strided((n - 10, h, 64), (stride, 64, 1), at + 10 * stride)  # noqa: E731
    far = dict(q=view(0, 2), k=view(1024, 1), v=view(2048, 1), out=view(4096, 2))
    for x in "qkv":
        far[x].copy_(st[x])
    st |= far
    call(qd, st)
    assert torch.equal(st["out"], want)


@pytest.mark.parametrize("offs", [[-5, 40, 100], [0, 60, 20], [0, 50, 1 << 30], [30, 30, 30], [50, 10, 90]])
def test_offsets_that_make_no_sense(qd, offs):
    """Taken into the rows there are; a sequence that ends before it begins is empty."""
    st = make([60, 40], None, 4, 2, 64)
    st["offsets"].copy_(torch.tensor(offs))
    call(qd, st)
    lo = [min(max(o, 0), 100) for o in offs]
    st["offs"] = st["koffs"] = lo
    if lo == sorted(lo):
        check(st, norm=False)
    else:
        rows = torch.zeros(100, dtype=torch.bool)
        for a, b in zip(lo, lo[1:]):
            rows[a:max(a, b)] = True
        assert (st["out"].cpu()[~rows] == MARK).all() and st["out"].isfinite().all()


@pytest.mark.parametrize("lens", [[64, 30], [700, 900, 300], [100] * 260], ids=["a pair an SM", "several", "list"])
def test_captured_calls(qd, lens):
    """A graph's replays with other lengths and values, and two calls in it."""
    st = make(lens, None, 16, 8, 128)
    second = make(lens, None, 16, 8, 128, seed=5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(qd, st)
        call(qd, second)
    g = torch.Generator().manual_seed(1)
    for _ in range(3):
        for x in (st, second):
            n = torch.randint(0, sum(lens) + 1, (len(lens) - 1,), generator=g).sort().values.tolist()
            x["offs"] = x["koffs"] = [0, *n, sum(lens)]
            x["offsets"].copy_(torch.tensor(x["offs"]))
            x["v"].copy_(torch.randn(x["v"].shape, generator=g).to(H))
            x["out"].fill_(MARK)
        graph.replay()
        torch.cuda.synchronize()
        check(st)
        check(second)


def test_streams_and_workspaces(qd):
    sts = [make(lens, None, 16, 8, 128, seed=i) for i, lens in enumerate(([800, 600, 77], [100] * 270))]
    side = [torch.cuda.Stream() for _ in sts]
    torch.cuda.synchronize()
    for _ in range(4):
        for st, s in zip(sts, side):
            with torch.cuda.stream(s):
                call(qd, st)
    call(qd, sts[0], stream=side[0])
    torch.cuda.synchronize()
    for st in sts:
        check(st)
    st = make([9000, 20000, 77, 5000], None, 16, 8, 128)   # 34077 // 128 + 4 = 270 pairs: a list
    need = qd.qd_attn_prompt_workspace(34077, 34077, 4, 16, 8, 128)
    want = call(qd, st).clone()
    call(qd, st, workspace=torch.full((need,), 255, dtype=torch.uint8, device="cuda"))
    assert torch.equal(st["out"], want)
    with pytest.raises(qd.QDError):
        call(qd, st, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


def test_the_same_whatever_the_batch(qd):
    """A sequence's result does not depend on what is packed beside it."""
    st = make([300, 700, 45], None, 8, 2, 128)
    want = call(qd, st).clone()
    for b in range(3):
        i0, i1 = st["offs"][b], st["offs"][b + 1]
        out = torch.empty_like(want[i0:i1])
        qd.qd_attn_prompt(st["q"][i0:i1], st["k"][i0:i1], st["v"][i0:i1], out, torch.tensor([0, i1 - i0], dtype=torch.int32).cuda())
        assert torch.equal(out, want[i0:i1])


def test_pairs_whose_first_tile_has_no_keys(qd):
    """Tiles that see nothing beside ones that do, pair after pair in the same CTA: many sequences of more queries than keys."""
    lens = [200 + 3 * i for i in range(60)]
    klens = [70 + i for i in range(60)]
    st = make(lens, klens, 32, 16, 128)
    for _ in range(3):
        st["out"].fill_(MARK)
        call(qd, st)
        check(st)
