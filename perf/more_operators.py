"""A decoder layer's attention over a paged cache, measured: prompts brought in, and decoded.

Three operators, as a serving program's layer uses them between its projections:

* ``rotate`` -- ``qd_qk_norm_rope``: a fused projection's queries and keys normalised head by head and rotated to
                their positions, in one pass that also writes the keys and values into the cache's pages.
* ``prompt`` -- ``qd_attn_prompt``: causal attention over whole prompts of different lengths that stand packed one after
                the other, or over later chunks of prompts whose earlier keys are at hand.
* ``paged``  -- ``qd_attn_paged``: attention of each stream's new token (or a few drafted ones) over a cache in pages.

Shapes are those of the decoders that the repository runs (16 query / 8 key heads of 128, 8 / 8 of 64, prompts of 8 x 512, 64
streams of 256 to 2048 positions, three interleaved position streams), and generic grouped heads.

Norm and rotation, per head of h = head_dim: x' = x / sqrt(mean(x^2) + eps) * gamma, then for d < h / 2, with c and s
of the token's position in the tables, y[d] = x'[d] c - x'[d + h/2] s and y[d + h/2] = x'[d + h/2] c + x'[d] s.  With three
position streams frequency d < 3 n takes stream d % 3, the others the first.  Values are not changed.

Pages: position j of stream b stands in row j % page_size of page table[b][j / page_size].  8-bit rows: s = fp32(max|x| /
127), r = fp32(127 / max|x|), code = nearest integer (ties to even) to fp32(x r), the value it stands for is code s; a
row under 2^-116 throughout is zero.

Prompts: queries offsets[b] .. offsets[b + 1] - 1 are the newest of sequence b, whose keys are kv_offsets[b] ..
kv_offsets[b + 1] - 1; the last query sees all of them, each one before it one key less.

Decoding: stream b holds lengths[b] positions, the newest n_new[b] of which are its queries' own; query t sees the
positions j < lengths[b] - (n_new[b] - 1 - t).  The rows t >= n_new[b] of an output are left as they were.
"""
import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step's projection of 64 streams in one layer: all latency
        dict(name="rotate step 64x1", op="rotate", B=64, T=1, lo=100, hi=300, qh=16, kvh=8, hd=128, page=16, fmt="bf16",
             dtype="bf16", out="bf16", norm=True, mrope=False, packed=False),
        # prompts of up to 512, from the framework's fp32 activations into an 8-bit cache
        dict(name="rotate prompts 8x512 f32", op="rotate", B=8, T=0, lo=300, hi=512, qh=16, kvh=8, hd=128, page=64, fmt="q8",
             dtype="f32", out="bf16", norm=True, mrope=False, packed=True),
        # a large prefill batch of prompts with images: three position streams, many query heads
        dict(name="rotate prompts 16x2500", op="rotate", B=16, T=0, lo=1000, hi=2500, qh=32, kvh=8, hd=128, page=32,
             fmt="bf16", dtype="bf16", out="bf16", norm=True, mrope=True, packed=True),
        # one short prompt: latency
        dict(name="prompt 1x64", op="prompt", B=1, lo=64, hi=64, past=0, qh=16, kvh=8, hd=128),
        # the batched prefill's shape
        dict(name="prompt 8x512", op="prompt", B=8, lo=512, hi=512, past=0, qh=16, kvh=8, hd=128),
        # many short ragged prompts, heads of 64 that are not grouped
        dict(name="prompt 37 ragged", op="prompt", B=37, lo=1, hi=701, past=0, qh=8, kvh=8, hd=64),
        # the next chunk of a few long prompts, three query heads a key head
        dict(name="prompt chunks 3x1000", op="prompt", B=3, lo=700, hi=1000, past=5000, qh=12, kvh=4, hd=128),
        # one long document
        dict(name="prompt 1x8192", op="prompt", B=1, lo=8192, hi=8192, past=0, qh=32, kvh=8, hd=128),
        # one stream decoding alone: latency of a short cache
        dict(name="paged 1x600", op="paged", B=1, T=1, qh=16, kvh=8, hd=128, lo=600, hi=600, page=16, fmt="bf16",
             dtype="bf16", ragged=False),
        # 64 ragged streams, one token each, 8-bit pages
        dict(name="paged 64 q8", op="paged", B=64, T=1, qh=16, kvh=8, hd=128, lo=257, hi=2048, page=64, fmt="q8",
             dtype="bf16", ragged=False),
        # drafted tokens: up to 5 queries a stream, an odd batch, heads of 64, fp32 activations
        dict(name="paged 37x5 f32", op="paged", B=37, T=5, qh=8, kvh=8, hd=64, lo=1, hi=512, page=32, fmt="bf16",
             dtype="f32", ragged=True),
        # a few very long streams of grouped heads in small pages: the axis has to be split
        dict(name="paged 3x65536", op="paged", B=3, T=1, qh=32, kvh=8, hd=128, lo=40000, hi=65536, page=16,
             fmt="bf16", dtype="bf16", ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "prompt", "prompt", "paged", "paged"])
    kvh, hd = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    if op == "rotate":
        packed = rng.random() < 0.6
        B = _log(rng, 1, 40 if packed else 96)
        hi = _log(rng, 2, 4000) if packed else _log(rng, 8, 400)
        while packed and B * hi > 40000:
            hi = (hi + 1) // 2
        return dict(op=op, B=B, T=0 if packed else rng.choice([1, 1, 2, 3, 5]), lo=rng.randint(1, hi), hi=hi,
                    qh=kvh * rng.choice([1, 2, 3, 4]), kvh=kvh, hd=hd, page=rng.choice([16, 32, 64, 128]),
                    fmt=rng.choice(["bf16", "q8"]), dtype=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "bf16", "f32"]),
                    norm=rng.random() < 0.8, mrope=rng.random() < 0.3, packed=packed)
    if op == "prompt":
        B, hi = _log(rng, 1, 48), _log(rng, 1, 8192)
        past = rng.choice([0, 0, _log(rng, 1, 8000)])
        qh = kvh * rng.choice([1, 2, 3, 4, 5, 8])
        while B * hi > 40000 or B * hi * (hi + past) * qh > 2.1e9:
            hi, past = (hi + 1) // 2, past // 2
        return dict(op=op, B=B, lo=rng.randint(1, hi), hi=hi, past=past, qh=qh, kvh=kvh, hd=hd)
    B, T = _log(rng, 1, 96), rng.choice([1, 1, 1, 2, 3, 4, 5, 7, 8])
    hi = _log(rng, 8, 16000)
    while B * hi > 160000:
        hi = (hi + 1) // 2
    return dict(op=op, B=B, T=T, qh=kvh * rng.choice([1, 2, 3, 4, 8]), kvh=kvh, hd=hd, lo=rng.randint(1, hi), hi=hi,
                page=rng.choice([16, 32, 64, 128, 256]), fmt=rng.choice(["bf16", "q8"]),
                dtype=rng.choice(["bf16", "bf16", "f32"]), ragged=rng.random() < 0.5)


# ----------------------------------------------------------------------------------------- inputs

def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _spread(B, lo, hi):
    """B lengths from lo to hi."""
    return [hi - (hi - lo) * i // max(1, B - 1) for i in range(B)]


def _lengths(g, B, lo, hi):
    """The same for every seed, in another order."""
    n = torch.tensor(_spread(B, lo, hi), device="cuda", dtype=torch.int32)
    return n[torch.randperm(B, generator=g, device="cuda")]


def _offsets(n):
    return torch.cat([torch.zeros_like(n[:1]), n.cumsum(0).to(torch.int32)])


def _quantise(x):
    """Rows of the last axis as codes and scales, in the arithmetic that the file's head gives."""
    top = x.abs().amax(-1)
    live = top >= 2.0 ** -116
    most, none = torch.full_like(top, 127.0), torch.zeros_like(top)     # tensors: a quotient by a number is a product
    scale = torch.where(live, top / most, none)
    by = torch.where(live, most / torch.where(live, top, most), none)
    return torch.round(x * by[..., None]).to(torch.int8), scale


def _table(g, B, hi, page):
    """Pages of B streams of up to hi positions, in no order."""
    n = (hi + page - 1) // page
    return torch.randperm(B * n, generator=g, device="cuda").to(torch.int32).reshape(B, n)


def _keys(g, shape):
    """Keys with a few loud channels, as normalised and rotated keys have."""
    loud = 1.0 + 2.0 * (torch.rand((shape[-3], 1, shape[-1]), generator=g, device="cuda") > 0.94)
    return torch.randn(shape, generator=g, device="cuda") * loud


def _pool(g, pages, kvh, page, hd, fmt):
    """Filled pages [pages, kvh, page, hd], a part at a time."""
    parts = {"k": [], "v": [], "ks": [], "vs": []}
    step = max(1, (1 << 28) // (kvh * page * hd))
    for p in range(0, pages, step):
        shape = (min(step, pages - p), kvh, page, hd)
        k = _keys(g, shape)
        v = torch.randn(shape, generator=g, device="cuda") * (0.25 + torch.rand((*shape[:3], 1), generator=g, device="cuda"))
        if fmt == "q8":
            (k, ks), (v, vs) = _quantise(k), _quantise(v)
            parts["ks"].append(ks)
            parts["vs"].append(vs)
        else:
            k, v = k.bfloat16(), v.bfloat16()
        parts["k"].append(k)
        parts["v"].append(v)
    return {n: torch.cat(p) if p else None for n, p in parts.items()}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    st = {"case": case}
    B, qh, kvh, hd = (case[k] for k in ("B", "qh", "kvh", "hd"))
    if case["op"] == "rotate":
        hi, page, T = case["hi"], case["page"], case["T"]
        st["lengths"] = n = _lengths(g, B, case["lo"], hi)
        st["table"] = _table(g, B, hi, page)
        if case["packed"]:                                  # whole prompts: every position is new
            st["offsets"], st["new"] = _offsets(n), n
            N = int(st["offsets"][-1])
        else:
            st["offsets"], N = None, B * T
            new = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if T > 1 else torch.ones_like(n)
            st["new"] = torch.minimum(new, n)
        # the rows stand in a fused projection [N, q + k + v], as a decoder's product leaves them
        fused = torch.randn((N, qh + 2 * kvh, hd), generator=g, device="cuda")
        fused *= 0.2 + 2.0 * torch.rand((N, qh + 2 * kvh, 1), generator=g, device="cuda")
        fused = fused.to(_type(case["dtype"]))
        st["q"], st["k"], st["v"] = fused[:, :qh], fused[:, qh:qh + kvh], fused[:, qh + kvh:]
        st["gammas"] = [0.5 + torch.rand((hd,), generator=g, device="cuda") if case["norm"] else None for _ in "qk"]
        rate = 1.0e6 ** (-torch.arange(0, hd, 2, device="cuda", dtype=torch.float64) / hd)
        angle = torch.arange(hi, device="cuda", dtype=torch.float64)[:, None] * rate
        st["cos"], st["sin"] = angle.cos().float(), angle.sin().float()
        st["pos"] = None
        if case["mrope"]:
            st["pos"] = torch.randint(0, hi, (3, N), generator=g, device="cuda", dtype=torch.int32)
        st["q_out"] = torch.zeros((N, qh, hd), device="cuda", dtype=_type(case["out"]))
        pages = st["table"].numel()
        of = torch.int8 if case["fmt"] == "q8" else torch.bfloat16
        st["pool"] = {n: torch.zeros((pages, kvh, page, hd), device="cuda", dtype=of) for n in "kv"}
        st["pool"] |= {n + "s": torch.zeros((pages, kvh, page), device="cuda") if case["fmt"] == "q8" else None for n in "kv"}
    elif case["op"] == "prompt":
        n = _lengths(g, B, case["lo"], case["hi"])
        st["offsets"] = _offsets(n)
        N = int(st["offsets"][-1])
        if case["past"]:                                    # queries of a chunk, keys of all so far
            st["kv_offsets"] = _offsets(n + torch.randint(0, case["past"] + 1, (B,), generator=g, device="cuda", dtype=torch.int32))
            M = int(st["kv_offsets"][-1])
            q = 1.5 * torch.randn((N, qh, hd), generator=g, device="cuda")
            st["q"] = q.bfloat16()
            st["k"] = _keys(g, (M, kvh, 1, hd))[:, :, 0].bfloat16()
            st["v"] = torch.randn((M, kvh, hd), generator=g, device="cuda").bfloat16()
        else:                                               # slices of one projection
            st["kv_offsets"] = None
            fused = torch.randn((N, qh + 2 * kvh, hd), generator=g, device="cuda")
            fused[:, :qh] *= 1.5
            fused[:, qh:qh + kvh] = _keys(g, (N, kvh, 1, hd))[:, :, 0]
            fused = fused.bfloat16()
            st["q"], st["k"], st["v"] = fused[:, :qh], fused[:, qh:qh + kvh], fused[:, qh + kvh:]
        st["out"] = torch.zeros((N, qh, hd), device="cuda", dtype=torch.bfloat16)
    else:
        T, page = case["T"], case["page"]
        st["lengths"] = n = _lengths(g, B, case["lo"], case["hi"])
        new = torch.full((B,), T, device="cuda", dtype=torch.int32)
        if case["ragged"]:
            new = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        st["new"] = torch.minimum(new, n)
        st["table"] = _table(g, B, case["hi"], page)
        st["pool"] = _pool(g, st["table"].numel(), kvh, page, hd, case["fmt"])
        st["q"] = (1.5 * torch.randn((B, T, qh, hd), generator=g, device="cuda")).to(_type(case["dtype"]))
        st["out"] = torch.zeros((B, T, qh, hd), device="cuda", dtype=_type(case["dtype"]))
    return st


# ------------------------------------------------------------------------------- the passes

def run(state):
    return {"rotate": _rotate, "prompt": _prompt, "paged": _paged}[state["case"]["op"]](state)


def _view(state):
    """The framework's view of the pages; a serving program keeps it with them."""
    import transformer_autoregressive_decode_gb300 as qd
    if "view" not in state:
        c = state["pool"]
        state["view"] = qd.KvCache(c["k"], c["v"], c["ks"], c["vs"])
    return state["view"]


def _values(c, name):
    x = c[name].float()
    return x if c[name + "s"] is None else x * c[name + "s"][..., None]


def _held(st):
    """What the pages hold: bf16 rows as they are, 8-bit rows as bf16 of the values that they stand for."""
    c = st["pool"]
    return {n: c[n] if c["ks"] is None else _values(c, n).bfloat16() for n in "kv"}


def _tokens(st):
    """Stream and index among its new tokens of every token row, and whether the row is in use."""
    N, new = st["q"].shape[0], st["new"].long()
    row = torch.arange(N, device="cuda")
    if st["offsets"] is None:
        T = N // new.shape[0]
        b, t = row // T, row % T
        return b, t, t < new[b]
    b = torch.searchsorted(st["offsets"][1:].long(), row, right=True)
    return b, row - st["offsets"].long()[b], torch.ones_like(row, dtype=torch.bool)


def _rotated(x, gamma, c, s):
    x = x.float()
    if gamma is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma
    a, b = x.chunk(2, -1)
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _rotate(st):
    case = st["case"]
    if own:
        import transformer_autoregressive_decode_gb300 as qd
        qd.qd_qk_norm_rope(st["q"], st["k"], st["q_out"], st["cos"], st["sin"], st["lengths"], v=st["v"], q_gamma=st["gammas"][0],
                           k_gamma=st["gammas"][1], eps=EPS, offsets=st["offsets"],
                           n_new=None if st["offsets"] is not None else st["new"], positions=st["pos"],
                           mrope_h=case["hd"] // 8 if case["mrope"] else 0, pages=_view(st), page_table=st["table"])
        return {"q": st["q_out"]} | _held(st)
    b, t, used = _tokens(st)
    at = st["lengths"].long()[b] - st["new"].long()[b] + t                      # positions in the cache
    if st["pos"] is None:
        c, s = st["cos"][at.clamp(max=case["hi"] - 1)], st["sin"][at.clamp(max=case["hi"] - 1)]
    else:
        d = torch.arange(case["hd"] // 2, device="cuda")
        r = st["pos"].long()[torch.where(d < 3 * (case["hd"] // 8), d % 3, torch.zeros_like(d))].T
        c, s = st["cos"][r, d], st["sin"][r, d]
    c, s = c[:, None], s[:, None]
    q = _rotated(st["q"], st["gammas"][0], c, s).to(st["q_out"].dtype)
    st["q_out"].copy_(torch.where(used[:, None, None], q, st["q_out"]))
    rows = {"k": _rotated(st["k"], st["gammas"][1], c, s), "v": st["v"].float()}
    on = torch.nonzero(used)[:, 0]
    page, slot = st["table"].long()[b[on], at[on] // case["page"]], at[on] % case["page"]
    codes, scale = zip(*(_quantise(rows[n][on]) if case["fmt"] == "q8" else (rows[n][on].bfloat16(), None) for n in "kv"))
    st["pool"]["k"][page, :, slot], st["pool"]["v"][page, :, slot] = codes
    if case["fmt"] == "q8":
        st["pool"]["ks"][page, :, slot], st["pool"]["vs"][page, :, slot] = scale
    return {"q": st["q_out"]} | _held(st)


def _prompt(st):
    case, q = st["case"], st["q"]
    if own:
        import transformer_autoregressive_decode_gb300 as qd
        qd.qd_attn_prompt(q, st["k"], st["v"], st["out"], st["offsets"], kv_offsets=st["kv_offsets"])
        return st["out"]
    B, qh, kvh, hd = (case[k] for k in ("B", "qh", "kvh", "hd"))
    offs = st["offsets"].long()
    koffs = offs if st["kv_offsets"] is None else st["kv_offsets"].long()
    L, M = case["hi"], case["hi"] + case["past"]
    i, j = torch.arange(L, device="cuda"), torch.arange(M, device="cuda")
    n, m = offs.diff(), koffs.diff()
    at = (offs[:-1, None] + i).clamp(max=q.shape[0] - 1)                        # sequences padded to the longest
    to = (koffs[:-1, None] + j).clamp(max=st["k"].shape[0] - 1)
    x = q[at].float().reshape(B, L, kvh, qh // kvh, hd).permute(0, 2, 3, 1, 4).reshape(B, kvh, -1, hd)
    k, v = st["k"][to].float().transpose(1, 2), st["v"][to].float().transpose(1, 2)
    s = torch.matmul(x, k.transpose(2, 3)).div_(math.sqrt(hd)).reshape(B, kvh, -1, L, M)
    seen = j < (m[:, None] - n[:, None] + 1 + i)[..., None]                     # [B, L, M]
    s.masked_fill_(~seen[:, None, None], -math.inf)
    p = s.sub_(s.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(p.reshape(B, kvh, -1, M), v).reshape(B, kvh, -1, L, hd) / p.sum(-1, keepdim=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, L, qh, hd).to(q.dtype)
    st["out"][at[i < n[:, None]]] = o[i < n[:, None]]
    return st["out"]


def _paged(st):
    case, q, lengths, new = st["case"], st["q"], st["lengths"], st["new"]
    if own:
        import transformer_autoregressive_decode_gb300 as qd
        qd.qd_attn_paged(q, _view(st), st["table"], lengths, st["out"], n_new=new, max_length=case["hi"])
        return st["out"]
    B, T, qh, hd = q.shape
    kvh, n = case["kvh"], st["table"].shape[1] * case["page"]
    x = q.float().reshape(B, T, kvh, qh // kvh, hd).permute(0, 2, 3, 1, 4).reshape(B, kvh, -1, hd)   # rows (head, t)
    own_pages = {a: None if t is None else t[st["table"].long()].transpose(1, 2).reshape(B, kvh, n, *t.shape[3:])
                 for a, t in st["pool"].items()}
    s = torch.matmul(x, _values(own_pages, "k").transpose(2, 3)) / math.sqrt(hd)
    t = torch.arange(T, device="cuda")
    seen = torch.arange(n, device="cuda") < (lengths[:, None] - (new[:, None] - 1 - t))[..., None]        # [B, T, n]
    s = s.reshape(B, kvh, -1, T, n).masked_fill(~seen[:, None, None], -math.inf).reshape(B, kvh, -1, n)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    o, total = torch.matmul(p, _values(own_pages, "v")), p.sum(-1, keepdim=True)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.reshape(B, kvh, qh // kvh, T, hd).permute(0, 3, 1, 2, 4).reshape(B, T, qh, hd).to(q.dtype)
    return torch.where((t < new[:, None])[..., None, None], o, st["out"])


# ----------------------------------------------------------------------------------- work and truth

def work(case):
    B, qh, kvh, hd = (case[k] for k in ("B", "qh", "kvh", "hd"))
    lengths = _spread(B, case["lo"], case["hi"])
    n = sum(lengths)
    if case["op"] == "rotate":
        n = n if case["packed"] else B * (1 if case["T"] == 1 else case["T"] / 2)
        e, o = (2 if case[k] == "bf16" else 4 for k in ("dtype", "out"))
        row = hd * 2 if case["fmt"] == "bf16" else hd + 4
        return {"bytes": n * ((qh + 2 * kvh) * hd * e + qh * hd * o + 2 * kvh * row), "flops": n * (qh + kvh) * hd * 8}
    if case["op"] == "prompt":
        pairs = sum(i * (i + 1) for i in lengths) / 2 + n * case["past"] / 2
        keys = n + B * case["past"] / 2
        return {"bytes": 2 * hd * (2 * qh * n + 2 * kvh * keys), "flops": 4 * hd * qh * pairs}
    row = 2 * (hd * 2 if case["fmt"] == "bf16" else hd + 4)
    new = B * (case["T"] / 2 if case["ragged"] else case["T"])
    e = 2 if case["dtype"] == "bf16" else 4
    return {"bytes": n * kvh * row + 2 * new * qh * hd * e, "flops": 4 * qh * hd * (n / B) * new}


def exact(case, seed):
    st = prepare(case, seed)
    return {"rotate": _rotate64, "prompt": _prompt64, "paged": _paged64}[case["op"]](case, st)


def _rotate64(case, st):
    """Stream after stream; what 8-bit rows stand for has no 64-bit value (a code may fall either side of a half)."""
    N, T, hd = st["q"].shape[0], case["T"], case["hd"]
    lengths, new, table = st["lengths"].tolist(), st["new"].tolist(), st["table"].tolist()
    half, page = hd // 2, case["page"]
    out = st["q_out"].double()
    pool = {n: st["pool"][n].double() for n in "kv"} if case["fmt"] == "bf16" else {"k": None, "v": None}
    start = 0
    for b in range(case["B"]):
        rows = slice(start, start + new[b])
        start += new[b] if case["packed"] else T
        if not new[b]:
            continue
        at = torch.arange(lengths[b] - new[b], lengths[b], device="cuda")
        angle = [[st[n][at, m] if st["pos"] is None else st[n][st["pos"][m % 3 if m < 3 * (hd // 8) else 0, rows].long(), m]
                  for m in range(half)] for n in ("cos", "sin")]
        c, s = (torch.stack(a, 1).double()[:, None] for a in angle)
        made = {}
        for name, gamma in zip("qk", st["gammas"]):
            x = st[name][rows].double()
            if gamma is not None:
                x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / hd + EPS) * gamma.double()
            y = torch.empty_like(x)
            y[..., :half] = c * x[..., :half] - s * x[..., half:]
            y[..., half:] = s * x[..., :half] + c * x[..., half:]
            made[name] = y
        out[rows] = made["q"]
        if case["fmt"] == "bf16":
            on = torch.tensor(table[b], device="cuda")[at // page]
            pool["k"][on, :, at % page] = made["k"]
            pool["v"][on, :, at % page] = st["v"][rows].double()
    return {"q": out} | pool


def _prompt64(case, st):
    """One sequence, one query head and some hundred queries after the other."""
    qh, kvh, hd = (case[k] for k in ("qh", "kvh", "hd"))
    offs = st["offsets"].tolist()
    koffs = offs if st["kv_offsets"] is None else st["kv_offsets"].tolist()
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        n, m = offs[b + 1] - offs[b], koffs[b + 1] - koffs[b]
        step = max(1, min(n, (1 << 27) // m))
        for h in range(qh):
            k, v = (st[x][koffs[b]:koffs[b + 1], h // (qh // kvh)].double() for x in "kv")
            for i in range(0, n, step):
                to = min(n, i + step)
                most = m - n + to                               # keys that the last of these queries sees
                s = st["q"][offs[b] + i:offs[b] + to, h].double() @ k[:most].T * hd ** -0.5
                s += torch.full_like(s, -math.inf).triu_(m - n + i + 1)
                e = torch.exp(s - s.max(1, keepdim=True).values)
                out[offs[b] + i:offs[b] + to, h] = (e @ v[:most]) / e.sum(1, keepdim=True)
    return out


def _paged64(case, st):
    """One stream and one key head after the other."""
    qh, kvh, hd = (case[k] for k in ("qh", "kvh", "hd"))
    lengths, new, page = st["lengths"].tolist(), st["new"].tolist(), case["page"]
    q, c = st["q"].double(), st["pool"]
    out = st["out"].double().clone()
    for b in range(case["B"]):
        j = torch.arange(lengths[b], device="cuda")
        on, slot = st["table"][b].long()[j // page], j % page
        for h in range(kvh):
            k, v = (c[x][on, h, slot].double() * (1.0 if c["ks"] is None else c[x + "s"][on, h, slot, None].double()) for x in "kv")
            heads = slice(h * (qh // kvh), (h + 1) * (qh // kvh))
            for t in range(new[b]):
                n = lengths[b] - (new[b] - 1 - t)
                s = q[b, t, heads] @ k[:n].T * hd ** -0.5
                e = torch.exp(s - s.max(1, keepdim=True).values)
                out[b, t, heads] = (e @ v[:n]) / e.sum(1, keepdim=True)
    return out
