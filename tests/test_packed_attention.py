"""Causal attention over packed sequences (qwen3_op_attention_packed_plan, qwen3_op_attention_prefill_packed) against float64,
and a run of the packed and paged operators together.

Tolerance: probabilities are rounded to bf16 for the product with V (2^-8 of each, so 2^-8 of the weighted |v|), the result to
bf16 (2^-8 of itself). Scores are fp32 sums of dh products (off by dh 2^-23 of their terms' sum, below 2^-15 of the largest
|q||k| here), exponents and sums add a few 2^-22: 2^-13 (1 + largest score term) of the weighted |v| covers them.
"""
import numpy as np
import pytest
import torch

from qwen3_decoder_transformer_gb300 import build as B

HEADS = [(8, 4, 64), (16, 8, 128), (4, 4, 128), (3, 1, 64)]
FORMS = [1, 4096, 8192]  # values of `longest` on both sides of what picks the kernel's form


@pytest.fixture(scope="module")
def bd():
    B.build()
    from qwen3_decoder_transformer_gb300 import binding
    binding.lib()
    return binding


def _cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _ref(q, k, v):
    """q [lq, Hq, dh], k, v [lk, Hkv, dh] (host) -> result and bound, float64."""
    q, k, v = (t.double().numpy() for t in (q, k, v))
    lq, Hq, dh = q.shape
    lk, Hkv, _ = k.shape
    ref, tol = np.zeros((lq, Hq, dh)), np.zeros((lq, Hq, dh))
    if lk == 0:
        return ref, tol
    see = np.arange(lk) <= np.arange(lq)[:, None] + lk - lq
    for h in range(Hq):
        j = h // (Hq // Hkv)
        x = q[:, h] @ k[:, j].T / dh ** 0.5
        size = (np.abs(q[:, h]) @ np.abs(k[:, j]).T / dh ** 0.5 * see).max() if see.any() else 0.0
        x = np.where(see, x, -np.inf)
        top = x.max(1, keepdims=True)
        p = np.where(see, np.exp(x - np.where(np.isfinite(top), top, 0)), 0)
        z = p.sum(1, keepdims=True)
        p = np.where(z > 0, p / np.where(z > 0, z, 1), 0)
        ref[:, h] = p @ v[:, j]
        tol[:, h] = 2.0 ** -8 * np.abs(ref[:, h]) + (2.0 ** -8 + 2.0 ** -13 * (1 + 2.0 ** -4 * size)) * (p @ np.abs(v[:, j]))
    return ref, tol


def _plan(bd, cu_q, cu_k, nq, nk, S):
    plan = torch.full((bd.attention_packed_plan_bytes(nq, S),), 255, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bd.op_attention_packed_plan(cu_q, cu_k, nq, nk, plan, err=err)
    return plan, err


def _inputs(heads, lq, lk, seed, tail=0):
    Hq, Hkv, dh = heads
    gen = torch.Generator().manual_seed(seed)
    mk = lambda n, h: torch.randn(n + tail, h, dh, generator=gen).to(torch.bfloat16)  # noqa: E731
    return mk(sum(lq), Hq), mk(sum(lk), Hkv), mk(sum(lk), Hkv)


def _run(bd, q, k, v, lq, lk, longest, stream=None):
    cu_q, cu_k = _cu(lq), _cu(lk)
    plan, err = _plan(bd, cu_q, cu_k, q.shape[0], k.shape[0], len(lq))
    out = torch.full((q.shape[0], q.shape[1] * q.shape[2]), 7.0, dtype=torch.bfloat16, device="cuda")
    bd.op_attention_prefill_packed(q, k, v, plan, longest, out, err=err, stream=stream)
    torch.cuda.synchronize()
    return out, int(err.item())


def _check(out, q, k, v, lq, lk):
    n = 0
    m = 0
    for a, b in zip(lq, lk):
        ref, tol = _ref(q[n:n + a], k[m:m + b], v[m:m + b])
        y = out[n:n + a].cpu().double().numpy().reshape(ref.shape)
        assert np.all(np.abs(y - ref) <= tol), (a, b, float((np.abs(y - ref) / np.where(tol > 0, tol, 1e-30)).max()))
        n += a
        m += b
    assert torch.all(out[n:] == 7.0)  # rows behind the last sequence


@pytest.mark.gpu
@pytest.mark.parametrize("longest", FORMS)
@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_prompts(bd, heads, longest):
    lens = [1, 127, 0, 128, 129, 2, 300, 640]
    q, k, v = _inputs(heads, lens, lens, longest + heads[0], tail=5)
    out, err = _run(bd, q.cuda(), k.cuda(), v.cuda(), lens, lens, longest)
    assert err == 0
    _check(out, q, k, v, lens, lens)


@pytest.mark.gpu
@pytest.mark.parametrize("longest", FORMS)
@pytest.mark.parametrize("heads", HEADS[:3], ids=str)
def test_histories(bd, heads, longest):
    """Queries behind a history, single tokens, sequences without queries, and queries before the first key."""
    lq = [1, 5, 130, 0, 200, 1, 7, 3]
    lk = [700, 5, 513, 40, 60, 1, 0, 128]
    q, k, v = _inputs(heads, lq, lk, longest + heads[0])
    out, err = _run(bd, q.cuda(), k.cuda(), v.cuda(), lq, lk, longest)
    assert err == 0
    _check(out, q, k, v, lq, lk)


@pytest.mark.gpu
@pytest.mark.parametrize("longest", FORMS)
@pytest.mark.parametrize("dh", [64, 128])
def test_long(bd, dh, longest):
    lens = [1500, 2300]
    q, k, v = _inputs((2, 1, dh), lens, lens, dh)
    q *= 4  # scores that move the running maximum
    out, err = _run(bd, q.cuda(), k.cuda(), v.cuda(), lens, lens, longest)
    assert err == 0
    _check(out, q, k, v, lens, lens)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1e-8, 300.0, 1e7])
@pytest.mark.parametrize("dh", [64, 128])
def test_sizes_of_scores(bd, dh, scale):
    lens = [200, 90]
    q, k, v = _inputs((4, 2, dh), lens, lens, 5)
    q = (q.float() * scale).to(torch.bfloat16)
    q[3] = 0
    out, err = _run(bd, q.cuda(), k.cuda(), v.cuda(), lens, lens, 200)
    assert err == 0
    _check(out, q, k, v, lens, lens)


@pytest.mark.gpu
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_and_values_at_their_limits(bd, dh, sign):
    """Scores just below 2^30, whose rounding in fp32 gives a row's weights a factor of up to 2^64 either way, beside values of
    2^55 over the visible keys: the result is the value of the row's largest score, to the roundings of its weight and of itself."""
    # the pair of bf16 values whose product, in log2 units, is furthest above (below) its fp32 rounding
    sl2 = np.float32(np.float32(1.4426950408889634) / np.sqrt(np.float32(dh)))
    a = np.arange(128, 256, dtype=np.float64)
    s = a[:, None] * a * 2.0 ** np.floor(30 + np.log2(dh) / 2 - np.log2(a[:, None] * a))
    x = s * np.float64(sl2)  # (40 bits: exact)
    off = np.where(s / dh ** 0.5 < 2.0 ** 30, (x - np.float32(x)) * sign, -1.0)
    i, j = np.unravel_index(off.argmax(), off.shape)
    assert off[i, j] > 56
    n, heads = 200, (4, 2, dh)
    q, k, v = (torch.zeros(n, h, dh) for h in (4, 2, 2))
    q[:, :, 0], k[0, :, 0] = a[i], s[i, j] / a[i]  # key 0 has all of the weight
    v[:] = torch.randn(n, 2, dh, generator=torch.Generator().manual_seed(1)).clamp(-1, 1) * 2.0 ** 55 / n
    q, k, v = (t.to(torch.bfloat16) for t in (q, k, v))
    out, err = _run(bd, q.cuda(), k.cuda(), v.cuda(), [n], [n], n)
    assert err == 0
    ref = v[0].double()[None, :, None].expand(n, 2, 2, dh).reshape(n, -1)
    assert torch.all((out.cpu().double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -8 + 2.0 ** -15) * ref.abs())


@pytest.mark.gpu
@pytest.mark.parametrize("S", [1, 33, 2000])
def test_many_sequences(bd, S):
    lens = [(i * 7919 + 5) % 23 for i in range(S)]
    q, k, v = _inputs((2, 2, 64), lens, lens, S, tail=1)
    out, err = _run(bd, q.cuda(), k.cuda(), v.cuda(), lens, lens, 64)
    assert err == 0
    _check(out, q, k, v, lens, lens)


@pytest.mark.gpu
@pytest.mark.parametrize("longest", FORMS)
def test_other_sequences_do_not_leak(bd, longest):
    """NaN and infinities in every other sequence, and behind the last one."""
    heads, lens = (8, 4, 64), [60, 200, 70, 128, 1, 90]
    q, k, v = _inputs(heads, lens, lens, 3, tail=40)
    ends = np.cumsum([0] + lens)
    for i in (0, 2, 4):
        for t, x in ((q, float("nan")), (k, float("inf")), (v, float("nan"))):
            t[ends[i]:ends[i + 1]] = x
    for t in (q, k, v):
        t[ends[-1]:] = float("nan")
    out, err = _run(bd, q.cuda(), k.cuda(), v.cuda(), lens, lens, longest)
    assert err == 0
    for i in (1, 3, 5):
        a, b = ends[i], ends[i + 1]
        ref, tol = _ref(q[a:b], k[a:b], v[a:b])
        y = out[a:b].cpu().double().numpy().reshape(ref.shape)
        assert np.all(np.abs(y - ref) <= tol)


@pytest.mark.gpu
def test_later_tiles_of_the_same_sequence_do_not_leak(bd):
    """Values behind the 128-row tile that a query belongs to may hold anything."""
    lens = [300]
    q, k, v = _inputs((2, 1, 128), lens, lens, 4)
    v[256:] = float("nan")
    k[256:] = float("inf")
    out, err = _run(bd, q.cuda(), k.cuda(), v.cuda(), lens, lens, 300)
    assert err == 0
    ref, tol = _ref(q[:256], k[:256], v[:256])
    assert np.all(np.abs(out[:256].cpu().double().numpy().reshape(ref.shape) - ref) <= tol)


@pytest.mark.gpu
@pytest.mark.parametrize("longest", FORMS[:2])
def test_rows_before_the_first_sequence(bd, longest):
    """Bounds that begin behind row 0: the rows in front belong to no sequence."""
    heads, lens, front = (8, 4, 128), [70, 0, 131], 37
    q, k, v = _inputs(heads, lens, lens, 6, tail=front)
    for t in (q, k, v):
        t[:front] = float("nan")
    cu = _cu(lens) + front
    plan, err = _plan(bd, cu, cu, q.shape[0], k.shape[0], 3)
    out = torch.full((q.shape[0], 8 * 128), 7.0, dtype=torch.bfloat16, device="cuda")
    bd.op_attention_prefill_packed(q.cuda(), k.cuda(), v.cuda(), plan, longest, out, err=err)
    assert int(err.item()) == 0 and torch.all(out[:front] == 7.0)
    _check(out[front:], q[front:], k[front:], v[front:], lens, lens)


@pytest.mark.gpu
@pytest.mark.parametrize("heads", HEADS[:2], ids=str)
def test_views_of_qkv_rows(bd, heads):
    """Queries, keys and values read in place from packed rows, with a stride of their own."""
    Hq, Hkv, dh = heads
    lens = [50, 200, 13]
    n, width = sum(lens), (Hq + 2 * Hkv) * dh + 16
    rows = torch.randn(n, width, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    cut = lambda t: (t[:, :Hq * dh].view(n, Hq, dh) if t.is_contiguous() else None)  # noqa: E731
    part = lambda t, a, h: t.as_strided((n, h, dh), (width, dh, 1), a)  # noqa: E731
    d = rows.cuda()
    views = [(part(rows, a, h), part(d, a, h)) for a, h in ((0, Hq), (Hq * dh, Hkv), ((Hq + Hkv) * dh, Hkv))]
    assert cut(rows) is not None
    out, err = _run(bd, *[x[1] for x in views], lens, lens, 256)
    assert err == 0
    _check(out, *[x[0] for x in views], lens, lens)


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [(16, 1, 64), (64, 1, 128), (128, 1, 64), (24, 1, 64), (256, 1, 64)], ids=str)
def test_large_groups(bd, heads):
    """Groups whose tiles have fewer tokens than the plan's finest list."""
    lq, lk = [1, 17, 0, 16, 40, 3], [30, 17, 9, 200, 40, 2]
    q, k, v = _inputs(heads, lq, lk, heads[0], tail=2)
    out, err = _run(bd, q.cuda(), k.cuda(), v.cuda(), lq, lk, 200)
    assert err == 0
    _check(out, q, k, v, lq, lk)


@pytest.mark.gpu
@pytest.mark.parametrize("longest", FORMS[:2])
@pytest.mark.parametrize("heads", [(16, 8, 128), (32, 8, 128), (8, 8, 64)], ids=str)
def test_many_items_a_cta(bd, heads, longest):
    """Ten and more tiles a CTA with one to three key tiles each, and histories in front of some: every accumulator, stage of Q and
    list of sums is used again and again."""
    lq = [300 - (i * 37) % 90 for i in range(24)] + [128, 1, 0, 257]
    lk = [n + (i % 3) * 60 for i, n in enumerate(lq)]
    q, k, v = _inputs(heads, lq, lk, heads[0] + longest, tail=3)
    out, err = _run(bd, q.cuda(), k.cuda(), v.cuda(), lq, lk, longest)
    assert err == 0
    _check(out, q, k, v, lq, lk)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,S,n,longest", [((32, 8, 128), 1100, 20, 4096), ((8, 8, 128), 10500, 3, 1), ((8, 8, 64), 10500, 3, 1),
                                               ((8, 8, 64), 10500, 2, 4096)], ids=str)
def test_more_items_than_are_looked_up_at_the_start(bd, heads, S, n, longest):
    """More tiles a CTA than its table holds (48 in the long form at head_dim 128, 512 otherwise; 152 CTAs): the others are found
    one by one. Sequences of one length, so that the reference takes them all at once."""
    Hq, Hkv, dh = heads
    lens = [n] * S
    q, k, v = _inputs(heads, lens, lens, S + n, tail=2)
    out, err = _run(bd, q.cuda(), k.cuda(), v.cuda(), lens, lens, longest)
    assert err == 0 and torch.all(out[S * n:] == 7.0)
    a = q[:S * n].cuda().double().view(S, n, Hkv, Hq // Hkv, dh)
    b, w = (t[:S * n].cuda().double().view(S, n, Hkv, dh) for t in (k, v))
    x = torch.einsum("sihgd,sjhd->shgij", a, b) / dh ** 0.5
    size = (torch.einsum("sihgd,sjhd->shgij", a.abs(), b.abs()).tril() / dh ** 0.5).amax(dim=(3, 4))
    x.masked_fill_(torch.ones(n, n, device="cuda").triu(1).bool(), float("-inf"))
    p = torch.softmax(x, dim=-1)
    ref, weighted = (torch.einsum("shgij,sjhd->sihgd", p, t) for t in (w, w.abs()))
    # (the bound of _ref)
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -13 * (1 + 2.0 ** -4 * size))[:, None, :, :, None] * weighted
    assert torch.all((out[:S * n].double().view(ref.shape) - ref).abs() <= tol)


@pytest.mark.gpu
def test_one_long_prompt(bd):
    """A prompt of 40,000 tokens (66 tiles a CTA, up to 313 key tiles each), on sampled rows."""
    n, Hq, Hkv, dh = 40000, 32, 8, 128
    gen = torch.Generator(device="cuda").manual_seed(40)
    q, k, v = (torch.randn(n, h, dh, generator=gen, device="cuda").to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    out, err = _run(bd, q, k, v, [n], [n], n)
    assert err == 0
    for i in (0, 1, 127, 128, 4095, 17000, 31999, 32000, 39935, 39936, 39999):
        ref, tol = _ref(q[i:i + 1].cpu(), k[:i + 1].cpu(), v[:i + 1].cpu())
        assert np.all(np.abs(out[i].cpu().double().numpy().reshape(ref.shape) - ref) <= tol), i


@pytest.mark.gpu
@pytest.mark.parametrize("lq,more", [([300, 0, 1, 129, 4097, 64], 0), ([4096, 4098, 5], 3), ([9000], 2000),
                                     ([3] * 1030 + [5000] + [2] * 20 + [6000], 1)])
def test_plan_lists(bd, lq, more):
    """Each of the four lists has every 128, 64, 32 and 16 rows of every sequence once, by falling numbers of key tiles."""
    lk = [n + more for n in lq]
    nq, nk = sum(lq), sum(lk)
    plan, err = _plan(bd, _cu(lq), _cu(lk), nq, nk, len(lq))
    raw = plan.cpu().numpy()
    assert int(err.item()) == 0
    counts, firsts = raw[:16].view(np.int32), raw[16:48].view(np.int64)
    items = raw[256:].view(np.int32).reshape(-1, 4)
    for level in range(4):
        rows = 128 >> level
        want, q0, k0 = [], 0, 0
        for a, b in zip(lq, lk):
            want += [(q0 + t, min(rows, a - t), k0, b - a + t) for t in range(0, a, rows)]
            q0, k0 = q0 + a, k0 + b
        got = items[firsts[level]:firsts[level] + counts[level]]
        assert sorted(map(tuple, got.tolist())) == sorted(want)
        tiles = np.minimum(-(-(got[:, 3] + got[:, 1]) // 128), 1023)
        assert np.all(np.diff(tiles) <= 0)


@pytest.mark.gpu
def test_plan_flags_bad_bounds(bd):
    """Sequences with bounds out of order or range are left out, their rows untouched; the others are right."""
    lens = [40, 50, 30, 20]
    q, k, v = _inputs((4, 4, 64), lens, lens, 7)
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    for cu in ([0, 40, 90, 120, 500], [0, 40, 90, 80, 140], [-5, 40, 90, 120, 140]):
        cu_q, cu_k = torch.tensor(cu, dtype=torch.int32, device="cuda"), _cu(lens)
        plan, err = _plan(bd, cu_q, cu_k, 140, 140, 4)
        assert int(err.item()) == 4
        out = torch.full((140, 256), 7.0, dtype=torch.bfloat16, device="cuda")
        bd.op_attention_prefill_packed(qd, kd, vd, plan, 64, out)
        ref, tol = _ref(q[40:90], k[40:90], v[40:90])
        y = out[40:90].cpu().double().numpy().reshape(ref.shape)
        assert np.all(np.abs(y - ref) <= tol)
    assert torch.all(out[:40] == 7.0)
    # sequences that overlap: more tiles than the plan has room for
    cu_q = torch.tensor([0, 140] * 8, dtype=torch.int32, device="cuda")
    plan, err = _plan(bd, cu_q, cu_q, 140, 140, 15)
    assert int(err.item()) == 4
    bd.op_attention_prefill_packed(qd, kd, vd, plan, 64, out)
    torch.cuda.synchronize()


@pytest.mark.gpu
@pytest.mark.parametrize("longest", FORMS)
def test_plan_of_other_rows(bd, longest):
    """A plan for more rows than the call has, and one that was never made: rows that the call has not are not written."""
    heads, lens = (4, 2, 64), [40, 50, 30]
    q, k, v = (t.cuda() for t in _inputs(heads, lens, lens, 5))
    plan, _ = _plan(bd, _cu(lens), _cu(lens), 120, 120, 3)
    whole = torch.full((120, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    bd.op_attention_prefill_packed(q, k, v, plan, longest, whole)
    out = torch.full((120, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    bd.op_attention_prefill_packed(q[:60], k, v, plan, longest, out[:60])
    torch.cuda.synchronize()
    assert torch.equal(out[:60], whole[:60]) and torch.all(out[60:] == 7.0)
    for fill in (0, 127, 255):
        plan.fill_(fill)
        bd.op_attention_prefill_packed(q[:60], k, v, plan, longest, out[:60])
        torch.cuda.synchronize()
        assert torch.all(out[60:] == 7.0)


@pytest.mark.gpu
def test_no_rows_and_no_keys(bd):
    q = torch.randn(3, 4, 64).to(torch.bfloat16).cuda()
    none = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    out, err = _run(bd, q, none, none, [3], [0], 1)
    assert err == 0 and torch.all(out == 0)
    out, err = _run(bd, q[:0], none, none, [0], [0], 1)
    assert err == 0 and out.numel() == 0


@pytest.mark.gpu
def test_streams_and_graph(bd):
    """Bit-equal results on two streams that share a plan, and from a graph that makes the plan and follows its bounds."""
    lens = [100, 700, 33]
    q, k, v = (t.cuda() for t in _inputs((16, 8, 128), lens, lens, 2))
    cu = _cu(lens)
    plan, _ = _plan(bd, cu, cu, 833, 833, 3)
    base, _ = _run(bd, q, k, v, lens, lens, 700)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.zeros_like(base) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o in zip(streams, outs):
            bd.op_attention_prefill_packed(q, k, v, plan, 700, o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, base) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        bd.op_attention_packed_plan(cu, cu, 833, 833, plan)
        bd.op_attention_prefill_packed(q, k, v, plan, 700, outs[0])
    outs[0].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], base)
    cu.copy_(_cu([400, 400, 33]))
    graph.replay()
    torch.cuda.synchronize()
    want, _ = _run(bd, q, k, v, [400, 400, 33], [400, 400, 33], 700)
    assert torch.equal(outs[0], want)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,page", [((16, 8, 128), 16), ((8, 4, 64), 64)], ids=str)
def test_prompts_then_tokens(bd, heads, page):
    """A serving loop's attention: prompts of different lengths appended and attended to, then single tokens over the
    cache, then a second prompt over the history read back; each step against float64 on what the cache holds."""
    Hq, Hkv, dh = heads
    lens = [37, 5, 150, 64]
    S, extra, more = len(lens), 6, 20
    reach = -(-(max(lens) + extra + more) // page)
    n_pages = S * reach
    table = torch.randperm(n_pages, generator=torch.Generator().manual_seed(1)).int().view(S, reach).cuda()
    size = bd.paged4_page_bytes(page, dh)
    kp, vp = (torch.full((n_pages, Hkv, size), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
    cs = torch.empty(512, dh, dtype=torch.bfloat16, device="cuda")
    bd.op_rope_table(1e6, dh, 512, cs)
    gen = torch.Generator().manual_seed(2)
    gamma = [(1 + 0.1 * torch.randn(dh, generator=gen)).to(torch.bfloat16).cuda() for _ in range(2)]
    width = (Hq + 2 * Hkv) * dh
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def append(counts, start):
        n = sum(counts)
        qkv = torch.randn(n, width, generator=gen).to(torch.bfloat16).cuda()
        q = torch.empty(n, Hq, dh, dtype=torch.bfloat16, device="cuda")
        k = torch.empty(n, Hkv, dh, dtype=torch.bfloat16, device="cuda")
        cu = _cu(counts)
        bd.op_append_paged4(qkv, cu, torch.tensor(start, dtype=torch.int32, device="cuda"), cs, kp, vp, table, q, k_out=k,
                            q_gamma=gamma[0], k_gamma=gamma[1], err=err)
        return q, k, qkv.as_strided((n, Hkv, dh), (width, dh, 1), (Hq + Hkv) * dh), cu

    def read(counts):
        n = sum(counts)
        k = torch.empty(n, Hkv, dh, dtype=torch.bfloat16, device="cuda")
        v = torch.empty_like(k)
        bd.op_read_paged4(kp, vp, table, _cu(counts), torch.zeros(S, dtype=torch.int32, device="cuda"), k, v, err=err)
        return k, v

    q, k, v, cu = append(lens, [0] * S)
    plan, _ = _plan(bd, cu, cu, q.shape[0], q.shape[0], S)
    out = torch.full((q.shape[0], Hq * dh), 7.0, dtype=torch.bfloat16, device="cuda")
    bd.op_attention_prefill_packed(q, k, v, plan, max(lens), out, err=err)
    _check(out, q.cpu(), k.cpu(), v.cpu(), lens, lens)
    # the cache holds the same keys, to half a step of 1/15 of a group's range
    kc, vc = read(lens)
    for a, b in ((k, kc), (v, vc)):
        a, b = a.float().unflatten(-1, (-1, 64)), b.float().unflatten(-1, (-1, 64))
        span = a.amax(-1, keepdim=True) - a.amin(-1, keepdim=True)
        assert torch.all((a - b).abs() <= span / 30 * 1.03 + 2.0 ** -7 * a.abs().amax(-1, keepdim=True))
    work = torch.empty(bd.attention_decode_paged4_workspace(S, Hq, Hkv, dh), dtype=torch.uint8, device="cuda")
    at = list(lens)
    for _ in range(extra):
        q, _, _, _ = append([1] * S, at)
        len0 = torch.tensor(at, dtype=torch.int32, device="cuda")
        out = torch.empty(S, Hq * dh, dtype=torch.bfloat16, device="cuda")
        bd.op_attention_decode_paged4(q, kp, vp, table, len0, work, out, err=err)
        at = [n + 1 for n in at]
        kc, vc = (t.cpu() for t in read(at))
        n = 0
        for b in range(S):
            ref, tol = _ref(q[b:b + 1].cpu(), kc[n:n + at[b]], vc[n:n + at[b]])
            # the values read back are rounded to bf16 (2^-8 of each), which moves the scores by 2^-8 of their terms, and
            # through them the weights by as much
            qq, kk = q[b].double().cpu().abs(), kc[n:n + at[b]].double().abs()
            size = max(float((kk[:, h // (Hq // Hkv)] @ qq[h]).max()) for h in range(Hq)) / dh ** 0.5
            big = vc[n:n + at[b]].double().abs().max().item()
            y = out[b].cpu().double().numpy().reshape(ref.shape)
            assert np.all(np.abs(y - ref) <= tol + 2.0 ** -8 * big * (2 + 2 * size))
            n += at[b]
    # a second turn: its keys appended, the whole history read back, attention with the history in front
    q, _, _, cu_q = append([more] * S, at)
    at = [n + more for n in at]
    kc, vc = read(at)
    cu_k = _cu(at)
    plan, _ = _plan(bd, cu_q, cu_k, q.shape[0], kc.shape[0], S)
    out = torch.full((q.shape[0], Hq * dh), 7.0, dtype=torch.bfloat16, device="cuda")
    bd.op_attention_prefill_packed(q, kc, vc, plan, max(at), out, err=err)
    _check(out, q.cpu(), kc.cpu(), vc.cpu(), [more] * S, at)
    assert int(err.item()) == 0


# ------------------------------------------------------------------------------------------------------------ refusals

def test_library_refuses(bd):
    """Argument checks on the host: nothing is launched (the addresses are never dereferenced)."""
    L, p, size = bd.lib(), 4096, 1 << 20

    def plan(**c):
        a = dict(cu_q=p, cu_k=p, S=3, Nq=100, Nk=100, plan=p, bytes=size)
        a.update(c)
        return L.qwen3_op_attention_packed_plan(*[a[n] for n in ("cu_q", "cu_k", "S", "Nq", "Nk", "plan", "bytes")], None, None)

    for c in (dict(cu_q=None), dict(cu_k=None), dict(S=-1), dict(Nq=-1), dict(Nk=-1), dict(Nq=2 ** 30 + 1), dict(plan=None),
              dict(plan=p + 8), dict(bytes=bd.attention_packed_plan_bytes(100, 3) - 1), dict(bytes=0)):
        assert plan(**c) == 5, c
    assert bd.attention_packed_plan_bytes(-1, 3) == 0 and bd.attention_packed_plan_bytes(5, -1) == 0
    assert bd.attention_packed_plan_bytes(2 ** 40, 1) == 0

    def attend(**c):
        a = dict(q=p, ldq=512, k=p, ldk=256, v=p, ldv=256, Nq=100, Nk=100, Hq=8, Hkv=4, dh=64, plan=p, bytes=size, longest=100,
                 out=p)
        a.update(c)
        return L.qwen3_op_attention_prefill_packed(*[a[n] for n in ("q", "ldq", "k", "ldk", "v", "ldv", "Nq", "Nk", "Hq", "Hkv",
                                                                    "dh", "plan", "bytes", "longest", "out")], None, None)

    for c in (dict(q=None), dict(k=None), dict(v=None), dict(plan=None), dict(out=None), dict(q=p + 8), dict(k=p + 2), dict(v=p + 4),
              dict(out=p + 8), dict(plan=p + 4), dict(ldq=504), dict(ldk=255), dict(ldv=260), dict(ldk=2 ** 38), dict(Nq=-1),
              dict(Nk=-1), dict(Hq=0), dict(Hq=6), dict(Hkv=0), dict(dh=96), dict(bytes=100), dict(bytes=1 << 40)):
        assert attend(**c) == 5, c
    assert attend(Nq=0) == 0


def test_binding_refuses(bd):
    bf, i32 = torch.bfloat16, torch.int32
    cu, plan = torch.zeros(4, dtype=i32), torch.zeros(4096, dtype=torch.uint8)
    base = dict(cu_q=cu, cu_k=cu, Nq=10, Nk=10, plan=plan)
    for change in (dict(cu_q=cu[0]), dict(cu_q=cu[:3]), dict(cu_k=cu.long()), dict(plan=None), dict(plan=plan[::2]), {}):
        with pytest.raises(ValueError):
            bd.op_attention_packed_plan(**{**base, **change})
    q, k, v = torch.zeros(10, 8, 64, dtype=bf), torch.zeros(10, 4, 64, dtype=bf), torch.zeros(10, 4, 64, dtype=bf)
    base = dict(q=q, k=k, v=v, plan=plan, longest=10, out=torch.zeros(10, 512, dtype=bf))
    for change in (dict(q=q[0]), dict(q=q.float()), dict(q=q.transpose(0, 1)), dict(k=k[:, :3]), dict(k=k[:9]), dict(v=v.float()),
                   dict(k=torch.zeros(10, 4, 128, dtype=bf)), dict(k=k[:, :0], v=v[:, :0]), dict(out=base["out"][:9]),
                   dict(out=base["out"].float()), dict(plan=None), dict(err=torch.zeros(1)), {}):
        with pytest.raises(ValueError):
            bd.op_attention_prefill_packed(**{**base, **change})


@pytest.mark.parametrize("longest,field", [(-5, 0), (0, 0), (77, 77), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1),
                                           (2 ** 63, 2 ** 31 - 1), (-2 ** 70, 0), (2 ** 200, 2 ** 31 - 1)])
def test_longest_is_any_whole_number(bd, longest, field):
    """A hint: what passes the field is its limit."""
    q, out = torch.zeros(3, 8, 64, dtype=torch.bfloat16), torch.zeros(3, 512, dtype=torch.bfloat16)
    block = bd._checks().attention_prefill_packed(q, q, q, torch.zeros(4096, dtype=torch.uint8), longest, out, None)
    assert int.from_bytes(block[88:92], "little") == field
