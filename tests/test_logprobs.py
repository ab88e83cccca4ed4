"""Token log probabilities, entropy and top alternatives (qwen3_op_token_logprobs) against float64.

Tolerances: with d = x - max, the kernel's terms are e^d with an exponent rounded to fp32 (relative error of e^d up to
|d| 2^-24 log2(e) plus the exponential's 2 ulp), summed over at most a few hundred elements a thread and a tree of
joins. Terms that matter have |d| <= 30, so s and t carry a relative error below 30 * 1.5 * 2^-24 + 20 * 2^-24 < 4e-6;
log s is then off by 4e-6 absolute, and x - max and the last difference by half an ulp of the result each. So a log
probability is within 1e-5 + 2^-23 |value|, and the entropy, log s - t / s with |t / s| <= log V, within
1e-5 + 4e-6 log V. Indices are exact.
"""
import math

import numpy as np
import pytest
import torch

from qwen3_decoder_transformer_gb300 import TINY, build as B


@pytest.fixture(scope="module")
def bd():
    B.build()
    from qwen3_decoder_transformer_gb300 import binding
    binding.lib()
    return binding


def _ref(x, tokens, k):
    """x: host float tensor (values as the kernel sees them)."""
    x = x.double()
    lsm = torch.log_softmax(x, dim=1)
    p = lsm.exp()
    ent = -torch.where(p > 0, p * lsm, torch.zeros_like(p)).sum(1)
    order = torch.from_numpy(np.argsort(-x.numpy(), axis=1, kind="stable")[:, :k].copy())
    return lsm.gather(1, tokens.long()[:, None])[:, 0], ent, order.int(), lsm.gather(1, order)


def _run(bd, x, tokens, k, stream=None):
    M = x.shape[0]
    out = dict(logprob=torch.full((M,), 7.0, device="cuda"), entropy=torch.full((M,), 7.0, device="cuda"),
               top_ids=torch.full((M, k), -7, dtype=torch.int32, device="cuda"),
               top_logprobs=torch.full((M, k), 7.0, device="cuda"))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bd.op_token_logprobs(x, tokens, err=err, stream=stream, **out)
    torch.cuda.synchronize()
    return [out[n].cpu() for n in ("logprob", "entropy", "top_ids", "top_logprobs")] + [int(err.item())]


def _check(got, ref, V):
    lp, ent, ids, tops, err = got
    rlp, rent, rids, rtops = ref
    assert err == 0
    assert torch.equal(ids, rids)
    for a, r in ((lp, rlp), (tops, rtops)):
        both = torch.isinf(r) & (a.double() == r)
        assert torch.all(both | ((a.double() - r).abs() <= 1e-5 + 2.0 ** -23 * r.abs()))
    assert torch.all((ent.double() - rent).abs() <= 1e-5 + 4e-6 * math.log(max(V, 2)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,V,k,pad", [(1, 1, 1, 0), (3, 2, 2, 1), (2, 7, 7, 0), (5, 33, 32, 3), (1, 1024, 32, 0),
                                       (4, 4099, 20, 5), (7, 32003, 5, 1), (1, 151936, 32, 0), (64, 151936, 5, 0),
                                       (200, 9001, 1, 0), (33, 50000, 0, 7), (700, 2050, 32, 0)])
def test_against_float64(bd, dtype, M, V, k, pad):
    g = torch.Generator().manual_seed(M * 1000 + V)
    full = (torch.randn(M, V + pad, generator=g) * 4).to(dtype)
    tokens = torch.randint(0, V, (M,), generator=g, dtype=torch.int32)
    tokens[0] = V - 1
    x = full.cuda()[:, :V]
    got = _run(bd, x, tokens.cuda(), k)
    _check(got, _ref(full[:, :V].float(), tokens, k), V)


@pytest.mark.gpu
@pytest.mark.parametrize("offset", [1, 2, 3, 5])
def test_unaligned_rows(bd, offset):
    """Rows that start off a 16-byte boundary, each row at another offset (an odd row stride)."""
    V, M, k = 5001, 6, 8
    for dtype in (torch.float32, torch.bfloat16):
        flat = (torch.randn(offset + M * (V + 2), generator=torch.Generator().manual_seed(offset)) * 3).to(dtype)
        x = flat.cuda()[offset:].reshape(M, V + 2)[:, :V]
        tokens = torch.arange(M, dtype=torch.int32)
        got = _run(bd, x, tokens.cuda(), k)
        _check(got, _ref(flat[offset:].reshape(M, V + 2)[:, :V].float(), tokens, k), V)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 40, 400])
@pytest.mark.parametrize("kind", ["ascending", "descending", "constant", "two values", "one peak", "clustered", "masked"])
def test_orders_and_ties(bd, kind, M):
    """Rows whose order or ties could defeat the candidate threshold; masked rows hold -inf and the lowest value."""
    V, k = 30011, 32
    if kind == "ascending":
        row = torch.linspace(-20, 5, V)
    elif kind == "descending":
        row = torch.linspace(5, -20, V)
    elif kind == "constant":
        row = torch.full((V,), -3.25)
    elif kind == "two values":
        row = (torch.arange(V) % 3 == 1).float()
    elif kind == "one peak":
        row = torch.zeros(V)
        row[V // 2 + 17] = 60.0
    elif kind == "clustered":  # 4000 large values that the spread sample of the row may miss
        row = torch.full((V,), -30.0)
        row[9000:13000] = torch.rand(4000, generator=torch.Generator().manual_seed(1))
    else:
        row = torch.full((V,), float("-inf"))
        row[::3] = torch.finfo(torch.float32).min
        row[100:140] = torch.arange(40).float() / 7
    full = row.repeat(M, 1)
    tokens = torch.full((M,), 120, dtype=torch.int32)
    _check(_run(bd, full.cuda(), tokens.cuda(), k), _ref(full, tokens, k), V)


@pytest.mark.gpu
def test_rows_without_a_distribution(bd):
    """NaN, +inf, or only -inf in a row: NaN values, ordered indices; the other rows are untouched by them."""
    V, k = 20000, 4
    x = torch.randn(5, V, generator=torch.Generator().manual_seed(3))
    x[1, [700, 30]] = float("nan")
    x[2, 5000] = float("inf")
    x[3, :] = float("-inf")
    tokens = torch.tensor([1, 2, 3, 4, 5], dtype=torch.int32)
    lp, ent, ids, tops, err = _run(bd, x.cuda(), tokens.cuda(), k)
    assert err == 0
    for r in (1, 2, 3):
        assert torch.isnan(lp[r]) and torch.isnan(ent[r]) and torch.isnan(tops[r]).all()
    assert ids[1].tolist()[:2] == [30, 700]
    assert ids[2, 0] == 5000
    assert ids[3].tolist() == [0, 1, 2, 3]
    rest = [0, 4]
    ref = _ref(x[rest], tokens[rest], k)
    _check((lp[rest], ent[rest], ids[rest], tops[rest], err), ref, V)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,V", [(2, 40), (1, 30011), (70, 30011), (400, 5003)])
def test_masked_rows(bd, dtype, M, V):
    """Rows in which a mask leaves fewer tokens than alternatives are asked for (none, one, a few, scattered or at the ends):
    the alternatives go on with the masked tokens in index order."""
    k = 20
    g = torch.Generator().manual_seed(V + M)
    full = torch.full((M, V), float("-inf"))
    for r in range(M):
        n = [1, 2, 7, 19, 20, 21, 3][r % 7]
        at = torch.randperm(V, generator=g)[:n] if r % 3 else torch.arange(V - n, V)
        full[r, at] = torch.randn(n, generator=g) * 5
    full = full.to(dtype)
    tokens = full.float().argmax(1).int()
    got = _run(bd, full.cuda(), tokens.cuda(), k)
    _check(got, _ref(full.float(), tokens, k), V)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 30, 1300])
@pytest.mark.parametrize("kind", ["lowest", "zero", "levels"])
def test_ties_at_the_threshold(bd, dtype, M, kind):
    """Most of a row has one value, by a mask of the type's lowest value or otherwise, and it is the last alternatives'
    value too: its tokens follow in index order, from wherever in the row they start."""
    V, k = 20011, 20
    g = torch.Generator().manual_seed(M)
    low = {"lowest": torch.finfo(dtype).min, "zero": -0.0, "levels": -2.0}[kind]
    full = torch.full((M, V), low, dtype=dtype)
    for r in range(M):
        n = [0, 1, 5, 19, 20, 21][r % 6]
        at = torch.randperm(V, generator=g)[:n] if r % 2 else torch.arange(V - n, V)
        full[r, at] = (torch.randn(n, generator=g).abs() + 1).to(dtype)
        if kind == "levels":  # the ties start late, behind lower values
            full[r, :[0, 9000, 19950][r % 3]] = -3.0
        if kind == "zero":  # both zeros are one value
            full[r, ::7] = full[r, ::7].clamp(min=0.0) + 0.0
    tokens = full.float().argmax(1).int()
    _check(_run(bd, full.cuda(), tokens.cuda(), k), _ref(full.float(), tokens, k), V)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,V,k", [(1, 1, 1), (3, 4, 4), (5, 33, 32), (1, 30011, 20), (40, 30011, 32), (200, 9001, 5),
                                   (1300, 2050, 4)])
def test_nan_at_the_first_tokens(bd, dtype, M, V, k):
    """Token 0 is an alternative like any other when its logit is NaN: alone, with others, and in rows of NaN only (a
    diverged model's), down to as many alternatives as tokens. NaN first, ties to the lowest index, no id outside [0, V)."""
    g = torch.Generator().manual_seed(V + M)
    full = (torch.randn(M, V, generator=g) * 3).to(dtype)
    for r in range(M):
        kind = (r + (M == 1)) % 5
        if kind == 0:
            full[r, 0] = float("nan")
        elif kind == 1:
            full[r, :] = float("nan")
        elif kind == 2:
            full[r, torch.tensor([0, V // 2, V - 1])] = float("nan")
        elif kind == 3:
            full[r, 0], full[r, V - 1] = float("inf"), float("nan")
    tokens = torch.zeros(M, dtype=torch.int32)
    lp, ent, ids, tops, err = _run(bd, full.cuda(), tokens.cuda(), k)
    x = full.float().numpy()
    order = np.argsort(-np.where(np.isnan(x), np.inf, x), axis=1, kind="stable")
    nan_first = np.argsort(~np.take_along_axis(np.isnan(x), order, 1), axis=1, kind="stable")
    want = torch.from_numpy(np.take_along_axis(order, nan_first, 1)[:, :k].copy()).int()
    assert err == 0
    assert int(ids.min()) >= 0 and int(ids.max()) < V
    assert torch.equal(ids, want)
    none = ~torch.isfinite(full.float()).all(1)
    assert torch.isnan(lp[none]).all() and torch.isnan(ent[none]).all() and torch.isnan(tops[none]).all()
    if (~none).any():
        rest = ~none
        _check((lp[rest], ent[rest], ids[rest], tops[rest], err), _ref(full[rest].float(), tokens[rest], k), V)


@pytest.mark.gpu
def test_bad_tokens_flagged(bd):
    x = torch.randn(4, 1000, generator=torch.Generator().manual_seed(4))
    tokens = torch.tensor([0, -1, 1000, 999], dtype=torch.int32)
    lp, ent, ids, tops, err = _run(bd, x.cuda(), tokens.cuda(), 2)
    assert err & 1
    assert torch.isnan(lp[1]) and torch.isnan(lp[2]) and torch.isfinite(lp[[0, 3]]).all()
    assert torch.isfinite(ent).all()


@pytest.mark.gpu
def test_parts_left_out_and_neighbours_untouched(bd):
    """Each output alone, and rows behind the last one as they were."""
    M, V, k = 3, 2000, 6
    x = torch.randn(M, V, generator=torch.Generator().manual_seed(5))
    tokens = torch.tensor([5, 6, 7], dtype=torch.int32)
    ref = _ref(x, tokens, k)
    xd, td = x.cuda(), tokens.cuda()
    lp = torch.full((M + 2,), 7.0, device="cuda")
    bd.op_token_logprobs(xd, td, logprob=lp[:M])
    ent = torch.full((M + 2,), 7.0, device="cuda")
    bd.op_token_logprobs(xd, entropy=ent[:M])
    ids = torch.full((M + 2, k), -7, dtype=torch.int32, device="cuda")
    bd.op_token_logprobs(xd, top_ids=ids[:M])
    tops = torch.full((M + 2, k), 7.0, device="cuda")
    bd.op_token_logprobs(xd, top_logprobs=tops[:M])
    torch.cuda.synchronize()
    for t in (lp, ent, ids.float().abs(), tops):
        assert torch.all(t[M:] == 7)
    _check((lp[:M].cpu(), ent[:M].cpu(), ids[:M].cpu(), tops[:M].cpu(), 0), ref, V)
    bd.op_token_logprobs(xd[:0], td[:0], logprob=lp[:0])  # no rows


@pytest.mark.gpu
def test_captured_on_another_stream_and_repeatable(bd):
    M, V, k = 20, 151936, 20
    x = (torch.randn(M, V, generator=torch.Generator().manual_seed(6)) * 3).to(torch.bfloat16).cuda()
    tokens = torch.arange(M, dtype=torch.int32, device="cuda")
    out = [torch.empty(M, device="cuda"), torch.empty(M, device="cuda"),
           torch.empty(M, k, dtype=torch.int32, device="cuda"), torch.empty(M, k, device="cuda")]
    bd.op_token_logprobs(x, tokens, *out)
    first = [t.clone() for t in out]
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            bd.op_token_logprobs(x, tokens, *out)
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, first):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_two_streams(bd):
    """Calls of one row (a cluster of sixteen CTAs), of 30 and of 700 rows on two streams at once: each as alone."""
    g = torch.Generator().manual_seed(7)
    calls = []
    for M, V in ((1, 151936), (30, 50001), (700, 4099)):
        x = (torch.randn(M, V, generator=g) * 3).cuda()
        tok = torch.randint(0, V, (M,), generator=g, dtype=torch.int32).cuda()
        outs = [(torch.zeros(M, device="cuda"), torch.zeros(M, device="cuda"),
                 torch.zeros(M, 9, dtype=torch.int32, device="cuda"), torch.zeros(M, 9, device="cuda")) for _ in range(2)]
        calls.append((x, tok, outs))
    want = []
    for x, tok, outs in calls:
        bd.op_token_logprobs(x, tok, *outs[0])
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs[0]])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in range(30):
        for n, s in enumerate(streams):
            x, tok, outs = calls[(i + n) % 3]
            bd.op_token_logprobs(x, tok, *outs[n], stream=s)
    torch.cuda.synchronize()
    for w, (_, _, outs) in zip(want, calls):
        assert all(torch.equal(a, b) for o in outs for a, b in zip(o, w))


@pytest.mark.gpu
def test_with_greedy_on_model_logits(bd):
    """On the logits of a prefill (all rows): the first alternative is the greedy token, and the log probability of the
    given tokens sums to the sequence's score."""
    from qwen3_decoder_transformer_gb300 import synth
    w = synth.make_weights(TINY, 0)
    w = {k: ([t.cuda() for t in v] if isinstance(v, list) else (None if v is None else v.cuda())) for k, v in w.items()}
    T, V = 40, TINY["vocab"]
    m = bd.Model(TINY, w, max_batch=1, capacity=T, max_tokens=T)
    ids = synth.make_ids(V, 1, T, 9).cuda()
    logits = torch.empty(T, V, device="cuda")
    m.prefill(ids, logits, all_rows=True)
    nxt = torch.empty(T, dtype=torch.int32, device="cuda")
    bd.op_greedy(logits, nxt)
    lp = torch.empty(T - 1, device="cuda")
    top = torch.empty(T - 1, 3, dtype=torch.int32, device="cuda")
    bd.op_token_logprobs(logits[:-1], ids[0, 1:].contiguous(), logprob=lp, top_ids=top)
    torch.cuda.synchronize()
    assert torch.equal(top[:, 0], nxt[:-1])
    ref = torch.log_softmax(logits[:-1].double(), 1).gather(1, ids[0, 1:].long()[:, None])[:, 0]
    assert torch.all((lp.double() - ref).abs() <= 1e-5 + 2.0 ** -23 * ref.abs())
    m.close()


# ------------------------------------------------------------------------------------------------ refusals (CPU)

def test_library_refuses(bd):
    import ctypes
    L = bd.lib()
    p = ctypes.c_void_p(64)  # never dereferenced: every call is refused on the host
    def call(logits=p, kind=0, ld=100, M=2, V=100, tokens=p, k=3, lp=p, ids=p):
        return L.qwen3_op_token_logprobs(logits, kind, ld, M, V, tokens, k, lp, None, ids, None, None, None)
    assert call(logits=None) == 5
    assert call(kind=2) == 5
    assert call(ld=99) == 5
    assert call(M=-1) == 5 and call(M=(1 << 27) + 1) == 5
    assert call(V=0) == 5
    assert call(k=33) == 5 and call(k=-1) == 5 and call(V=2, k=3) == 5
    assert call(tokens=None) == 5 and call(lp=None) == 5
    assert call(logits=ctypes.c_void_p(66)) == 5 and call(logits=ctypes.c_void_p(65), kind=1) == 5


def test_binding_refuses(bd):
    x, t, lp = torch.zeros(2, 10), torch.zeros(2, dtype=torch.int32), torch.zeros(2)
    ids = torch.zeros(2, 3, dtype=torch.int32)
    bad = [dict(logits=x.half()), dict(logits=x[0]), dict(logits=torch.zeros(10, 2).t()), dict(tokens=t.long()),
           dict(tokens=t[:1]), dict(logprob=None), dict(tokens=None), dict(entropy=torch.zeros(2, dtype=torch.float64)),
           dict(top_ids=ids.float()), dict(top_ids=torch.zeros(2, 11, dtype=torch.int32)),
           dict(top_ids=ids, top_logprobs=torch.zeros(2, 4)), dict(logprob=torch.zeros(4)[::2]),
           dict(logits=x.expand(2, 10)[:1].expand(2, 10)), dict(err=torch.zeros(2, dtype=torch.int32)),
           {}]  # the last: host tensors
    with pytest.raises(ValueError, match="2\\^27"):  # sizes past the library's integers
        bd.op_token_logprobs(torch.empty((1 << 32) + 1, 1, device="meta"), entropy=lp)
    for change in bad:
        kw = dict(logits=x, tokens=t, logprob=lp)
        kw.update(change)
        with pytest.raises(ValueError):
            bd.op_token_logprobs(**kw)
