"""A layer's attention as a serving program runs it: prompts through the norm and rotation into pages and the prompt's attention,
then steps over the pages, against a 64-bit form of the whole; eager and captured, with pages handed out as the streams grow."""
import pytest
import torch

from tests._paged_ref import norm_rope

pytestmark = pytest.mark.gpu
H = torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module")
def qd(cuda_ok):
    import transformer_autoregressive_decode_gb300 as m
    return m


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("fmt", ["bf16", "q8"])
@pytest.mark.parametrize("dtype, qh, kvh, hd, page", [(torch.float32, 16, 8, 128, 16), (H, 6, 2, 64, 64)])
def test_prompts_and_steps(qd, dtype, qh, kvh, hd, page, fmt, captured):
    g = torch.Generator(device="cuda").manual_seed(7)
    prompts, steps, most = [130, 1, 77], 20, 160
    B, N = len(prompts), sum(prompts)
    per = (most + page - 1) // page
    n_pages = B * per + 2
    code = torch.int8 if fmt == "q8" else H
    kp, vp = (torch.zeros((n_pages, kvh, page, hd), dtype=code, device="cuda") for _ in "kv")
    ks, vs = ((torch.zeros((n_pages, kvh, page), device="cuda") for _ in "kv") if fmt == "q8" else (None, None))
    pages = qd.KvCache(kp, vp, ks, vs)
    free = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32).tolist()
    table = torch.full((B, per), -1, dtype=torch.int32, device="cuda")
    held = [0] * B

    def grow(b, n):
        while held[b] * page < n:
            table[b, held[b]] = free.pop()
            held[b] += 1

    angle = torch.arange(most, device="cuda", dtype=torch.float64)[:, None] * 1e6 ** (-torch.arange(0, hd, 2, device="cuda", dtype=torch.float64) / hd)
    cos, sin = angle.cos().float(), angle.sin().float()
    gq, gk = (0.5 + torch.rand(hd, generator=g, device="cuda") for _ in "qk")
    heads = qh + 2 * kvh
    x = torch.randn((N, heads, hd), generator=g, device="cuda").to(dtype)
    offsets = torch.tensor([0, 130, 131, 208], dtype=torch.int32, device="cuda")
    lengths = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    for b in range(B):
        grow(b, prompts[b])
    q = torch.empty((N, qh, hd), dtype=H, device="cuda")
    k, v = (torch.empty((N, kvh, hd), dtype=H, device="cuda") for _ in "kv")
    out = torch.empty_like(q)

    def prefill():
        qd.qd_qk_norm_rope(x[:, :qh], x[:, qh:qh + kvh], q, cos, sin, lengths, v=x[:, qh + kvh:], k_out=k, v_out=v, q_gamma=gq, k_gamma=gk,
                           eps=EPS, offsets=offsets, pages=pages, page_table=table)
        qd.qd_attn_prompt(q, k, v, out, offsets)

    y = torch.empty((B, heads, hd), dtype=dtype, device="cuda")
    q1 = torch.empty((B, qh, hd), dtype=H, device="cuda")
    o1 = torch.empty((B, 1, qh, hd), dtype=H, device="cuda")

    def step():
        qd.qd_qk_norm_rope(y[:, :qh], y[:, qh:qh + kvh], q1, cos, sin, lengths, v=y[:, qh + kvh:], q_gamma=gq, k_gamma=gk, eps=EPS, pages=pages,
                           page_table=table)
        qd.qd_attn_paged(q1[:, None], pages, table, lengths, o1, max_length=most)

    def runner(f):
        if not captured:
            return f
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f()
        return graph.replay

    def exact(rows, pos, gamma):
        return norm_rope(rows, gamma, EPS, cos[pos], sin[pos])[0]

    # the 64-bit layer: keys and values of all positions so far
    keys, values = [], []
    runner(prefill)()
    # relative to the results' size: bf16 queries, keys, values, probabilities and results round by 2^-8 at most each (2^-8 / sqrt(3) in the mean), 8-bit
    # keys and values by half a code, 1 / 254 of a row's largest, about 3 of its mean size
    room = 5 * 2.0 ** -8 + (2 * 3 / 254 if fmt == "q8" else 0)

    def near(got, want):
        assert got.isfinite().all() and float((got.double() - want).norm() / want.norm()) < room

    for b in range(B):
        i0, n = int(offsets[b]), prompts[b]
        pos = torch.arange(n, device="cuda")
        qe, ke = exact(x[i0:i0 + n, :qh], pos, gq), exact(x[i0:i0 + n, qh:qh + kvh], pos, gk)
        ve = x[i0:i0 + n, qh + kvh:].double()
        keys.append(ke), values.append(ve)
        kk, vv = (t.repeat_interleave(qh // kvh, 1) for t in (ke, ve))
        s = torch.einsum("ihd,jhd->hij", qe, kk) * hd ** -0.5
        p = torch.softmax(s.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), float("-inf")), -1)
        near(out[i0:i0 + n], torch.einsum("hij,jhd->ihd", p, vv))
    lengths.add_(1)
    for b in range(B):
        grow(b, prompts[b] + 1)
    run = None
    for t in range(steps):
        y.copy_(torch.randn((B, heads, hd), generator=g, device="cuda"))
        if run is None:
            run = runner(step)
        run()
        for b in range(B):
            pos = torch.tensor([prompts[b] + t], device="cuda")
            qe = exact(y[b:b + 1, :qh], pos, gq)[0]
            keys[b] = torch.cat([keys[b], exact(y[b:b + 1, qh:qh + kvh], pos, gk)])
            values[b] = torch.cat([values[b], y[b:b + 1, qh + kvh:].double()])
            kk, vv = (z.repeat_interleave(qh // kvh, 1) for z in (keys[b], values[b]))
            p = torch.softmax(torch.einsum("hd,jhd->hj", qe, kk) * hd ** -0.5, -1)
            near(o1[b, 0], torch.einsum("hj,jhd->hd", p, vv))
        lengths.add_(1)
        for b in range(B):
            grow(b, min(prompts[b] + t + 2, most))
