"""Decode attention over a shared prefix, and attention with a sliding window and sinks (prefill and single-token form),
against softmax attention in float64 over the visible keys.

Tolerance. The kernels differ from the exact result by the rounding of the probabilities to bf16, half a step each
(relative 2^-8), the rounding of the result (2^-8 of it), and fp32 arithmetic. So |got - ref| <= 2^-8 |ref| +
(2^-8 + e) sum_i p_i |v_i| for every element, the sum computed in float64 beside the reference. e covers the scores: an
fp32 score in log2 units, |x| <= X, is off by at most about 10 roundings, 10 * 2^-24 X, and moves p by 0.7 of that: 4e-6 for
the ordinary cases (X about 10), 6e-4 for X = 1500; 1e-6 absolute for the rest.
"""
import pytest
import torch

from qwen3_decoder_transformer_gb300 import build as B

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def bd():
    B.build()
    from qwen3_decoder_transformer_gb300 import binding
    binding.lib()
    return binding


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _attend(q, k, v):
    """q [G, dh], k, v [n, dh] -> (exact result, sum of p |v|), float64; no keys: zeros."""
    if k.shape[0] == 0:
        z = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
        return z, z
    w = torch.softmax(q.double() @ k.double().T / q.shape[1] ** 0.5, dim=1)
    return w @ v.double(), w @ v.double().abs()


def _close(got, ref, spread, e=4e-6):
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + e) * spread + 1e-6
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((got.double() - ref).abs() / tol).nan_to_num(1e9).max()))


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------- shared prefix, decode

def _shared_case(bd, Bn, Hq, Hkv, dh, P, cap, lens, meta=None, prefix_cap=None, seed=0, poison=True, scale=1.0):
    g = _gen(seed)
    prefix_cap = P if prefix_cap is None else prefix_cap
    q = _normal(g, Bn, Hq, dh, scale=scale)
    kp, vp = _normal(g, Hkv, max(prefix_cap, 1), dh), _normal(g, Hkv, max(prefix_cap, 1), dh)
    k, v = _normal(g, Bn, Hkv, cap, dh), _normal(g, Bn, Hkv, cap, dh)
    G = Hq // Hkv
    ps, psh, pads = (meta[0], meta[1], meta[2:]) if meta else (0, 0, [0] * Bn)
    ref = torch.empty(Bn, Hq, dh, dtype=torch.float64, device="cuda")
    spread = torch.empty_like(ref)
    seen = torch.zeros(Bn, cap, dtype=torch.bool, device="cuda")
    for b in range(Bn):
        n = min((lens[b] if len(lens) > 1 else lens[0]) + 1, cap)
        for s in range(psh, n):
            seen[b, s] = not (ps <= s < ps + pads[b])
        for h in range(Hkv):
            kk = torch.cat([kp[h, :P], k[b, h][seen[b]]])
            vv = torch.cat([vp[h, :P], v[b, h][seen[b]]])
            ref[b, h * G:(h + 1) * G], spread[b, h * G:(h + 1) * G] = _attend(q[b, h * G:(h + 1) * G], kk, vv)
    if poison:  # rows that nobody sees
        for t in (k, v):
            t.masked_fill_(~seen[:, None, :, None], float("nan"))
        kp[:, P:], vp[:, P:] = float("nan"), float("nan")
    work = torch.full((bd.attention_decode_shared_workspace(Bn, Hq, Hkv, dh, P) // 4 + 64,), float("nan"), device="cuda")
    out = torch.full((Bn + 1, Hq * dh), 7.0, dtype=torch.bfloat16, device="cuda")
    err = _err()
    bd.op_attention_decode_shared(q, kp if prefix_cap else None, vp if prefix_cap else None, k, v,
                                  torch.tensor(lens, dtype=torch.int32, device="cuda"), work, out[:Bn],
                                  prefix_len=P if prefix_cap else None, err=err,
                                  seq_meta=torch.tensor(meta, dtype=torch.int32, device="cuda") if meta else None)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert torch.all(out[Bn] == 7.0)
    assert torch.isnan(work[-64:]).all()  # scratch behind its stated size
    _close(out[:Bn].reshape(Bn, Hq, dh), ref, spread, 4e-6 if scale == 1.0 else 6e-4)


@gpu
@pytest.mark.parametrize("P", [0, 1, 15, 127, 128, 129, 582, 1000, 5000])
@pytest.mark.parametrize("Bn,Hq,Hkv,dh", [(1, 8, 4, 64), (5, 16, 8, 128), (33, 32, 8, 128)])
def test_shared_prefix_lengths(bd, Bn, Hq, Hkv, dh, P):
    lens = [(b * 37) % 70 - (1 if b == 2 else 0) for b in range(Bn)]
    if Bn > 2:
        lens[2] = -1  # a sequence without own keys
    _shared_case(bd, Bn, Hq, Hkv, dh, P, 70, lens, prefix_cap=P + (3 if P % 2 else 0), seed=P + Bn)


@gpu
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (3, 1), (8, 8), (10, 2), (12, 2), (14, 2), (8, 1), (16, 2)])
@pytest.mark.parametrize("Bn", [1, 17, 70, 150])
def test_shared_head_groups(bd, Hq, Hkv, Bn):
    """Groups of 1 to 8 query heads; batches over the row-tile borders (floor(128 / G) sequences a tile)."""
    _shared_case(bd, Bn, Hq, Hkv, 128 if Bn != 70 else 64, 300, 40, [(b * 11) % 40 for b in range(Bn)], seed=Hq + Bn)


@gpu
@pytest.mark.parametrize("cap,own", [(1, 0), (16, 15), (17, 16), (700, 699), (5000, 4999)])
@pytest.mark.parametrize("Bn", [1, 20])
def test_shared_own_lengths(bd, cap, own, Bn):
    """One length for all (len0 of one element), and lengths past the cache."""
    _shared_case(bd, Bn, 16, 8, 128, 200, cap, [own], seed=cap)
    _shared_case(bd, Bn, 16, 8, 128, 200, cap, [own + 50], seed=cap + 1)


@gpu
def test_shared_framework_layout(bd):
    """The layout qwen3_share_prefix leaves: the prefix in sequence 0's cache, own slots from psh, padding at ps. The
    same call through qwen3_op_attention_decode, which reads the prefix once per sequence, gives the same result to
    two roundings."""
    g = _gen(3)
    Bn, Hq, Hkv, dh, cap, n = 6, 16, 8, 128, 1024, 700
    psh, ps, pads = 256, 300, [0, 17, 250, 3, 0, 100]
    q, kc, vc = _normal(g, Bn, Hq, dh), _normal(g, Bn, Hkv, cap, dh), _normal(g, Bn, Hkv, cap, dh)
    meta = torch.tensor([ps, psh] + pads, dtype=torch.int32, device="cuda")
    len_t = torch.tensor([n - 1], dtype=torch.int32, device="cuda")
    old, new = (torch.empty(Bn, Hq * dh, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w0 = torch.empty(bd.attention_decode_workspace(Bn, Hq, dh, cap), dtype=torch.uint8, device="cuda")
    bd.op_attention_decode(q, kc, vc, len_t, w0, old, seq_meta=meta)
    work = torch.empty(bd.attention_decode_shared_workspace(Bn, Hq, Hkv, dh, psh), dtype=torch.uint8, device="cuda")
    bd.op_attention_decode_shared(q, kc[0], vc[0], kc, vc, len_t, work, new, prefix_len=psh, seq_meta=meta)
    for b in range(Bn):
        own = [s for s in range(psh, n) if not ps <= s < ps + pads[b]]
        for h in range(Hkv):
            k = torch.cat([kc[0, h, :psh], kc[b, h, own]])
            v = torch.cat([vc[0, h, :psh], vc[b, h, own]])
            ref, spread = _attend(q[b, 2 * h:2 * h + 2], k, v)
            for o in (old, new):
                _close(o.reshape(Bn, Hq, dh)[b, 2 * h:2 * h + 2], ref, spread)


@gpu
@pytest.mark.parametrize("ps,psh,pads", [(0, 0, [5, 0, 39]), (10, 0, [0, 30, 7]), (130, 128, [0, 20, 33])])
def test_shared_padding(bd, ps, psh, pads):
    _shared_case(bd, 3, 8, 2, 64, 150, 200, [180], meta=[ps, psh] + pads, seed=ps)


@gpu
@pytest.mark.parametrize("Bn,Hq,Hkv,dh,P", [(600, 8, 8, 64, 15), (520, 16, 8, 128, 1 + 15), (70, 3, 1, 128, 1000), (150, 6, 1, 64, 500),
                                            (41, 10, 2, 128, 900), (33, 14, 2, 128, 1100), (9, 16, 2, 64, 4000),
                                            (1, 1, 1, 128, 70000), (1, 8, 1, 64, 66001), (2, 16, 8, 128, 4097),
                                            (2, 16, 8, 128, 4096), (64, 16, 8, 128, 128), (65, 16, 8, 128, 128)])
def test_shared_read_once_or_by_each(bd, Bn, Hq, Hkv, dh, P):
    """Sizes at and past the border between a prefix read once for the batch and one that each sequence reads for itself
    (65,536 keys over all kv heads), groups of 1 to 8 heads."""
    _shared_case(bd, Bn, Hq, Hkv, dh, P, 40, [(b * 11) % 41 - 1 for b in range(Bn)], seed=Hq + Bn, prefix_cap=P + 5)


@gpu
@pytest.mark.parametrize("Bn,Hq,Hkv,dh,P,cap", [(2, 10, 2, 128, 20000, 3000), (1, 7, 1, 64, 70000, 5000), (37, 4, 4, 64, 30000, 140),
                                                (19, 12, 4, 128, 9000, 300), (3, 8, 1, 128, 30000, 900), (9, 9, 3, 64, 6000, 600)])
def test_shared_own_keys_of_several_ctas(bd, Bn, Hq, Hkv, dh, P, cap):
    """Own keys split over a cluster beside a long prefix: the cluster's parts and the records of many chunks in one join."""
    _shared_case(bd, Bn, Hq, Hkv, dh, P, cap, [(b * 131 + cap - 2) % cap for b in range(Bn)], seed=Bn)
    _shared_case(bd, Bn, Hq, Hkv, dh, P, cap, [cap - 1], seed=Bn + 1,
                 meta=[cap // 3, 0] + [(17 * b + 5) % (cap // 2) for b in range(Bn)])


@gpu
def test_shared_many_own_keys_without_a_prefix(bd):
    lens = [(b * 53) % 700 for b in range(64)]
    _shared_case(bd, 64, 16, 8, 128, 0, 700, lens)
    _shared_case(bd, 64, 16, 8, 128, 0, 700, lens, prefix_cap=9, seed=1)


@gpu
@pytest.mark.parametrize("Bn,Hq,Hkv", [(3, 8, 2), (40, 8, 8)])
def test_shared_short_prefix_and_padding(bd, Bn, Hq, Hkv):
    """A layout with padding beside a prefix of every form."""
    for P in (1, 100, 700):
        _shared_case(bd, Bn, Hq, Hkv, 128, P, 200, [180], meta=[130, 128] + [(7 * b) % 45 for b in range(Bn)], seed=P)


@gpu
def test_shared_large_scores(bd):
    """Scores of a few hundred: the running maxima of chunks, warps and CTAs differ widely."""
    _shared_case(bd, 9, 16, 8, 128, 3000, 300, [(b * 97) % 300 for b in range(9)], seed=5, scale=60.0)


@gpu
def test_shared_repeatable_captured_and_two_streams(bd):
    """Bit-equal results from repeated calls, from a graph captured on a side stream, and from calls on two streams at once
    with a workspace each."""
    g = _gen(11)
    Bn, Hq, Hkv, dh, P, cap = 24, 32, 8, 128, 3000, 256
    q, kp, vp = _normal(g, Bn, Hq, dh), _normal(g, Hkv, P, dh), _normal(g, Hkv, P, dh)
    k, v = _normal(g, Bn, Hkv, cap, dh), _normal(g, Bn, Hkv, cap, dh)
    lens = torch.randint(0, cap, (Bn,), device="cuda", dtype=torch.int32)
    size = bd.attention_decode_shared_workspace(Bn, Hq, Hkv, dh, P)
    works = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty(Bn, Hq * dh, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    bd.op_attention_decode_shared(q, kp, vp, k, v, lens, works[0], outs[0])
    first = outs[0].clone()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, w, o in zip(streams, works, outs):
            bd.op_attention_decode_shared(q, kp, vp, k, v, lens, w, o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        bd.op_attention_decode_shared(q, kp, vp, k, v, lens, works[0], outs[0])
    for step in range(3):
        outs[0].zero_()
        lens.add_(-1)  # the lengths are read on the device: a replay sees the new ones
        graph.replay()
        bd.op_attention_decode_shared(q, kp, vp, k, v, lens, works[1], outs[1])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1])


# ------------------------------------------------------------------------------------- sliding window and sinks

def _row(s, sink_rows, ring):
    return s if not ring or s < sink_rows else sink_rows + (s - sink_rows) % ring


def _sinks_case(bd, Bn, T, Hq, Hkv, dh, starts, window, sinks, rolling, cap=None, decode=False, seed=0, extra=0, scale=1.0):
    g = _gen(seed)
    sink_rows = bd.attention_sink_rows(sinks)
    assert sink_rows == (sinks + 127) // 128 * 128
    ring = 0
    if rolling:
        ring = (window + T - 1 + 127) // 128 * 128 + 128 * extra
        cap = sink_rows + ring
    elif cap is None:
        cap = max(max(starts) + T, 1)
    q = _normal(g, Bn, Hq, T, dh, scale=scale)
    k, v = _normal(g, Bn, Hkv, cap, dh), _normal(g, Bn, Hkv, cap, dh)
    G = Hq // Hkv
    ref = torch.zeros(Bn, T, Hq, dh, dtype=torch.float64, device="cuda")
    spread = torch.zeros_like(ref)
    seen = torch.zeros(Bn, cap, dtype=torch.bool, device="cuda")
    rows = range(T) if T <= 6 else sorted({0, 1, T // 3, T // 2, T - 2, T - 1, min(T - 1, 127), min(T - 1, 128), min(T - 1, 200)})
    for b in range(Bn):
        start = starts[b] if len(starts) > 1 else starts[0]
        if start < 0:
            continue
        lo = max(0, start - window + 1)
        for s in list(range(min(sinks, lo))) + list(range(lo, min(start + T, cap) if not ring else start + T)):
            seen[b, _row(s, sink_rows, ring)] = True
        for t in rows:
            i = start + t
            slots = [s for s in range(0, min(sinks, i + 1))] + list(range(max(sinks, i - window + 1, 0), i + 1))
            if not ring:
                slots = [s for s in slots if s < cap]
            at = torch.tensor([_row(s, sink_rows, ring) for s in slots], device="cuda")
            for h in range(Hkv):
                ref[b, t, h * G:(h + 1) * G], spread[b, t, h * G:(h + 1) * G] = _attend(
                    q[b, h * G:(h + 1) * G, t], k[b, h][at], v[b, h][at])
    for x in (k, v):  # rows that no query of the call sees
        x.masked_fill_(~seen[:, None, :, None], float("nan"))
    out = torch.full((Bn * T + 1, Hq * dh), 7.0, dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor(starts, dtype=torch.int32, device="cuda")
    err = _err()
    if decode:
        bd.op_attention_decode_sinks(q[:, :, 0].contiguous(), k, v, lens, out[:Bn], window, sinks, rolling=rolling, err=err)
    else:
        bd.op_attention_prefill_sinks(q, k, v, lens, out[:Bn * T], window, sinks, rolling=rolling, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert torch.all(out[Bn * T] == 7.0)
    got = out[:Bn * T].reshape(Bn, T, Hq, dh)
    assert torch.isfinite(got).all()
    rows = list(rows)
    _close(got[:, rows], ref[:, rows], spread[:, rows])


@gpu
@pytest.mark.parametrize("rolling", [False, True], ids=["full", "rolling"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (16, 1), (100, 0), (128, 128), (129, 300), (1000, 4), (4096, 130)])
@pytest.mark.parametrize("Bn,Hq,Hkv,dh", [(1, 16, 8, 128), (3, 8, 4, 64), (40, 32, 8, 128)])
def test_sinks_decode(bd, Bn, Hq, Hkv, dh, window, sinks, rolling):
    """Sequences at their own lengths: one of one key, one inside the window, one inside the sinks, several far past."""
    starts = [0, window // 2, max(0, sinks - 2), 3 * window + 7, 5000] * 8
    starts = starts[:Bn] if Bn > 1 else [3 * window + 200]
    if Bn > 4:
        starts[4] = -1  # a sequence that is not in use
    _sinks_case(bd, Bn, 1, Hq, Hkv, dh, starts, window, sinks, rolling, decode=True, seed=window + sinks)


@gpu
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (8, 8), (10, 2), (12, 2), (14, 2), (8, 1)])
def test_sinks_decode_head_groups(bd, Hq, Hkv):
    _sinks_case(bd, 5, 1, Hq, Hkv, 64, [900, 10, 300, 299, 301], 300, 5, False, decode=True, seed=Hq)


@gpu
@pytest.mark.parametrize("Bn,window,dh", [(1, 2500, 64), (1, 1100, 128), (3, 2500, 128), (20, 5000, 64), (130, 2500, 64)])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (5, 1), (6, 1), (7, 1), (8, 1), (8, 4)])
def test_sinks_decode_clusters(bd, Bn, window, dh, Hq, Hkv):
    """Sequences split over two to sixteen CTAs, by any group of heads, down to one key each."""
    _sinks_case(bd, Bn, 1, Hq, Hkv, dh, [(b * 611 + window + 40) % (window + 300) for b in range(Bn)], window, 7, False,
                decode=True, seed=Hq)


@gpu
def test_sinks_decode_one_length_and_past_the_cache(bd):
    _sinks_case(bd, 3, 1, 16, 8, 128, [777], 200, 4, False, decode=True, cap=1000)
    _sinks_case(bd, 3, 1, 16, 8, 128, [999], 2000, 4, False, decode=True, cap=1000)
    _sinks_case(bd, 2, 1, 16, 8, 128, [2 ** 30], 200, 4, True, decode=True)  # a ring turned often


@gpu
@pytest.mark.parametrize("rolling", [False, True], ids=["full", "rolling"])
@pytest.mark.parametrize("T,start,window,sinks", [(1, 0, 1, 0), (1, 500, 64, 4), (2, 127, 128, 1), (64, 1000, 100, 4),
                                                  (127, 0, 50, 200), (128, 300, 129, 128), (300, 0, 64, 0),
                                                  (333, 777, 256, 130), (1000, 0, 300, 4), (700, 5000, 2048, 300)])
@pytest.mark.parametrize("Hq,Hkv,dh", [(8, 4, 64), (6, 2, 128)])
def test_sinks_prefill(bd, Hq, Hkv, dh, T, start, window, sinks, rolling):
    _sinks_case(bd, 2, T, Hq, Hkv, dh, [start, start // 3], window, sinks, rolling, seed=T + window, extra=int(rolling))


@gpu
@pytest.mark.parametrize("window,dh,start", [(4096, 128, 0), (4000, 64, 3000), (8192, 128, 9000), (9000, 64, 0)])
def test_sinks_prefill_long_windows(bd, window, dh, start):
    """The forms the kernel takes for windows from 4096 and 8192 keys, over more items than SMs."""
    _sinks_case(bd, 1, 5000, 8, 2, dh, [start], window, 20, False, seed=window)
    _sinks_case(bd, 1, 700, 8, 2, dh, [start + 20000], window, 20, True, seed=window)


@gpu
def test_sinks_prefill_without_sinks_is_the_windowed_prefill(bd):
    """sinks = 0 on a full cache is the sliding window of qwen3_op_attention_prefill (another kernel, which adds in another
    order): every row of both is within the tolerance of float64."""
    g = _gen(4)
    Bn, Hq, Hkv, dh, T, cap, start, window = 2, 8, 4, 128, 500, 700, 150, 200
    q, k, v = _normal(g, Bn, Hq, T, dh), _normal(g, Bn, Hkv, cap, dh), _normal(g, Bn, Hkv, cap, dh)
    len0 = torch.tensor([start], dtype=torch.int32, device="cuda")
    a, b = (torch.empty(Bn * T, Hq * dh, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bd.op_attention_prefill(q, k, v, len0, a, window=window)
    bd.op_attention_prefill_sinks(q, k, v, len0, b, window, 0)
    i, j = torch.arange(start, start + T, device="cuda")[:, None], torch.arange(cap, device="cuda")
    kk, vv = (x.double().repeat_interleave(Hq // Hkv, dim=1) for x in (k, v))
    x = torch.einsum("bhtd,bhnd->bhtn", q.double(), kk) / dh ** 0.5
    p = torch.softmax(x.masked_fill((j > i) | (i - j >= window), float("-inf")), dim=3)
    ref, spread = (torch.einsum("bhtn,bhnd->bthd", p, y) for y in (vv, vv.abs()))
    for o in (a, b):
        _close(o.reshape(Bn, T, Hq, dh), ref, spread)


@gpu
def test_sinks_windows_past_32_bits(bd):
    """A window or a number of sinks that no 32-bit integer holds is a limit that hides nothing, not its lower bits."""
    g = _gen(15)
    Bn, Hq, Hkv, dh, T, cap = 1, 4, 2, 64, 140, 500
    q, k, v = _normal(g, Bn, Hq, T, dh), _normal(g, Bn, Hkv, cap, dh), _normal(g, Bn, Hkv, cap, dh)
    len0 = torch.tensor([cap - T], dtype=torch.int32, device="cuda")
    outs = []
    for window, sinks in ((cap, 0), (2 ** 33 + 3, 0), (2 ** 31, 0), (3, 2 ** 40)):
        o = torch.empty(Bn * T, Hq * dh, dtype=torch.bfloat16, device="cuda")
        d = torch.empty(Bn, Hq * dh, dtype=torch.bfloat16, device="cuda")
        bd.op_attention_prefill_sinks(q, k, v, len0, o, window, sinks)
        bd.op_attention_decode_sinks(q[:, :, 0].contiguous(), k, v, len0, d, window, sinks)
        outs.append((o, d))
    torch.cuda.synchronize()
    G = Hq // Hkv
    for h in range(Hkv):
        for t in (0, T - 1):
            n = cap - T + t + 1
            ref, spread = _attend(q[0, h * G:(h + 1) * G, t], k[0, h, :n], v[0, h, :n])
            for o, d in outs:
                _close(o.reshape(T, Hq, dh)[t, h * G:(h + 1) * G], ref, spread)
                if t == 0:
                    _close(d.reshape(Hq, dh)[h * G:(h + 1) * G], ref, spread)
    for window, sinks in ((5 - 2 ** 32, 0), (5, 3 - 2 ** 32)):
        with pytest.raises(bd.Qwen3Error):
            bd.op_attention_prefill_sinks(q, k, v, len0, o, window, sinks)


@gpu
def test_sinks_captured_and_repeatable(bd):
    g = _gen(12)
    Bn, Hq, Hkv, dh, window, sinks = 2, 32, 8, 128, 1000, 4
    cap = bd.attention_sink_rows(sinks) + 1152
    k, v = _normal(g, Bn, Hkv, cap, dh), _normal(g, Bn, Hkv, cap, dh)
    lens = torch.tensor([5000, 20], dtype=torch.int32, device="cuda")
    qd, qp = _normal(g, Bn, Hq, dh), _normal(g, Bn, Hq, 100, dh)
    od = torch.empty(Bn, Hq * dh, dtype=torch.bfloat16, device="cuda")
    op = torch.empty(Bn * 100, Hq * dh, dtype=torch.bfloat16, device="cuda")

    def calls():
        bd.op_attention_decode_sinks(qd, k, v, lens, od, window, sinks, rolling=True)
        bd.op_attention_prefill_sinks(qp, k, v, lens, op, window, sinks, rolling=True)

    calls()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        calls()
    for _ in range(3):
        calls()
        want = od.clone(), op.clone()
        od.zero_(), op.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(od, want[0]) and torch.equal(op, want[1])
        lens.add_(1)


@gpu
def test_sinks_decode_on_two_streams(bd):
    """Calls that take clusters of sixteen and of four CTAs, and a prefill, on two streams at once: each as alone."""
    g = _gen(16)
    calls = []
    for Bn, Hq, Hkv, dh, cap, T in ((1, 32, 8, 128, 5000, 1), (10, 16, 8, 64, 3000, 1), (1, 16, 8, 128, 2000, 300)):
        k, v = _normal(g, Bn, Hkv, cap, dh), _normal(g, Bn, Hkv, cap, dh)
        lens = torch.randint(cap // 2, cap - T, (Bn,), device="cuda", dtype=torch.int32)
        out = torch.zeros(2, Bn * T, Hq * dh, dtype=torch.bfloat16, device="cuda")
        q = _normal(g, Bn, Hq, T, dh) if T > 1 else _normal(g, Bn, Hq, dh)
        op = bd.op_attention_prefill_sinks if T > 1 else bd.op_attention_decode_sinks
        calls.append((op, q, k, v, lens, out, min(cap, 4096)))
    want = []
    for op, q, k, v, lens, out, window in calls:
        op(q, k, v, lens, out[0], window, 4)
        torch.cuda.synchronize()
        want.append(out[0].clone())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in range(30):
        for n, s in enumerate(streams):
            op, q, k, v, lens, out, window = calls[(i + n) % 3]
            op(q, k, v, lens, out[n], window, 4, stream=s)
    torch.cuda.synchronize()
    for w, c in zip(want, calls):
        assert torch.equal(c[5][0], w) and torch.equal(c[5][1], w)


@gpu
def test_streaming_loop(bd):
    """The operators as a streaming server uses them: chunks of a prompt, then tokens, appended to a rolling buffer with
    sinks; every result equals attention in float64 over the whole history, and the prefill form agrees on one token."""
    g = _gen(13)
    Bn, Hq, Hkv, dh, window, sinks, chunk = 2, 8, 4, 64, 150, 10, 100
    total = 900
    G = Hq // Hkv
    ks, vs = _normal(g, Bn, Hkv, total, dh), _normal(g, Bn, Hkv, total, dh)
    sink_rows = bd.attention_sink_rows(sinks)
    ring = (window + chunk - 1 + 127) // 128 * 128
    kc = torch.full((Bn, Hkv, sink_rows + ring, dh), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    pos = 0
    for T in [chunk] * 6 + [1] * 130 + [37, 1]:
        at = torch.tensor([_row(s, sink_rows, ring) for s in range(pos, pos + T)], device="cuda")
        kc[:, :, at], vc[:, :, at] = ks[:, :, pos:pos + T], vs[:, :, pos:pos + T]
        q = _normal(g, Bn, Hq, T, dh)
        len0 = torch.tensor([pos], dtype=torch.int32, device="cuda")
        out = torch.empty(Bn * T, Hq * dh, dtype=torch.bfloat16, device="cuda")
        if T == 1:
            bd.op_attention_decode_sinks(q[:, :, 0].contiguous(), kc, vc, len0, out, window, sinks, rolling=True)
        if T > 1 or pos % 40 == 0:
            other = torch.empty_like(out)
            bd.op_attention_prefill_sinks(q, kc, vc, len0, other, window, sinks, rolling=True)
        for t in ([0] if T == 1 else [0, T // 2, T - 1]):
            i = pos + t
            slots = list(range(min(sinks, i + 1))) + list(range(max(sinks, i - window + 1), i + 1))
            for b in range(Bn):
                for h in range(Hkv):
                    ref, spread = _attend(q[b, h * G:(h + 1) * G, t], ks[b, h, slots], vs[b, h, slots])
                    outs = ([out] if T == 1 else []) + ([other] if T > 1 or pos % 40 == 0 else [])
                    for o in outs:
                        _close(o.reshape(Bn, T, Hq, dh)[b, t, h * G:(h + 1) * G], ref, spread)
        pos += T


@gpu
def test_shared_then_scored(bd):
    """A decode step over a shared prefix as a server runs it: append, attention, projection to logits, scores."""
    g = _gen(14)
    Bn, Hq, Hkv, dh, P, cap, V = 12, 8, 4, 64, 300, 40, 1000
    d = Hq * dh
    kp, vp = _normal(g, Hkv, P, dh), _normal(g, Hkv, P, dh)
    kc = torch.zeros(Bn, Hkv, cap, dh, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    head = _normal(g, V, d, scale=0.2)
    table = torch.empty(P + cap, dh, dtype=torch.bfloat16, device="cuda")
    bd.op_rope_table(1e6, dh, P + cap, table)
    gamma = torch.ones(dh, dtype=torch.bfloat16, device="cuda")
    work = torch.empty(bd.attention_decode_shared_workspace(Bn, Hq, Hkv, dh, P), dtype=torch.uint8, device="cuda")
    q = torch.empty(Bn, Hq, dh, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(Bn, d, dtype=torch.bfloat16, device="cuda")
    logits = torch.empty(Bn, V, device="cuda")
    lp, ids = torch.empty(Bn, device="cuda"), torch.empty(Bn, 4, dtype=torch.int32, device="cuda")
    tops, nxt = torch.empty(Bn, 4, device="cuda"), torch.empty(Bn, dtype=torch.int32, device="cuda")
    for step in range(3):
        qkv = _normal(g, Bn, (Hq + 2 * Hkv) * dh)
        len0 = torch.tensor([step], dtype=torch.int32, device="cuda")
        bd.op_qknorm_rope_append(qkv, Bn, 1, Hq, Hkv, dh, gamma, gamma, table[P:], len0, 1e-6, q, kc, vc)
        bd.op_attention_decode_shared(q, kp, vp, kc, vc, len0, work, out)
        bd.op_gemm(out, head, bd.EPI_F32, logits)
        bd.op_greedy(logits, nxt)
        bd.op_token_logprobs(logits, nxt, logprob=lp, top_ids=ids, top_logprobs=tops)
        torch.cuda.synchronize()
        for b in range(Bn):
            for h in range(Hkv):
                ref, spread = _attend(q[b, 2 * h:2 * h + 2], torch.cat([kp[h], kc[b, h, :step + 1]]),
                                      torch.cat([vp[h], vc[b, h, :step + 1]]))
                _close(out.reshape(Bn, Hq, dh)[b, 2 * h:2 * h + 2], ref, spread)
        assert torch.equal(ids[:, 0], nxt) and torch.equal(tops[:, 0], lp)
        ref = torch.log_softmax(logits.double(), 1).gather(1, nxt.long()[:, None])[:, 0]
        assert torch.all((lp.double() - ref).abs() <= 1e-5 + 2.0 ** -23 * ref.abs())


# ------------------------------------------------------------------------------------------------ refusals (CPU)

def test_library_refuses(bd):
    import ctypes
    L = bd.lib()
    p, odd = ctypes.c_void_p(64), ctypes.c_void_p(72)  # never dereferenced

    def shared(q=p, kp=p, vp=p, pc=100, P=100, kc=p, vc=p, B=2, Hq=8, Hkv=4, dh=64, cap=10, len0=p, st=0, work=p, out=p,
               size=1 << 30):
        return L.qwen3_op_attention_decode_shared(q, kp, vp, pc, P, kc, vc, B, Hq, Hkv, dh, cap, len0, st, None, work, size,
                                                  out, None, None)
    for kw in (dict(q=None), dict(kc=None), dict(vc=None), dict(len0=None), dict(out=None), dict(kp=None), dict(vp=None),
               dict(work=None), dict(P=101), dict(P=-1), dict(B=-1), dict(B=65536), dict(Hq=9), dict(Hq=36), dict(dh=96),
               dict(cap=0), dict(st=2), dict(q=odd), dict(kp=odd), dict(vc=odd), dict(work=odd), dict(Hkv=0),
               dict(size=bd.attention_decode_shared_workspace(2, 8, 4, 64, 100) - 1)):
        assert shared(**kw) == 5, kw
    ws = bd.attention_decode_shared_workspace
    assert ws(2, 8, 4, 64, 0) == 0 and ws(0, 8, 4, 64, 10) == 0 and ws(2, 36, 4, 64, 10) == 0
    # one key tile and one row tile: a 128-row record for each kv head, and the own keys' result for each query row
    assert ws(2, 8, 4, 64, 10) == (4 * 128 * 66 + 2 * 8 * 68) * 4

    def sinks(decode, q=p, kc=p, vc=p, B=1, T=4, Hq=8, Hkv=4, dh=64, cap=512, len0=p, st=0, window=100, sinks=4, roll=1,
              out=p):
        if decode:
            return L.qwen3_op_attention_decode_sinks(q, kc, vc, B, Hq, Hkv, dh, cap, len0, st, window, sinks, roll, out,
                                                     None, None)
        return L.qwen3_op_attention_prefill_sinks(q, kc, vc, B, T, Hq, Hkv, dh, cap, len0, st, window, sinks, roll, out,
                                                  None, None)
    for kw in (dict(q=None), dict(kc=None), dict(vc=None), dict(len0=None), dict(out=None), dict(B=-1), dict(Hq=9),
               dict(dh=32), dict(cap=0), dict(st=-1), dict(window=0), dict(sinks=-1), dict(roll=2), dict(q=odd),
               dict(kc=odd), dict(vc=odd), dict(cap=513), dict(cap=128), dict(window=385, T=1), dict(sinks=385),
               dict(window=2 ** 30, cap=2 ** 30)):
        for decode in (True, False):
            assert sinks(decode, **kw) == 5, (decode, kw)
    for decode in (True, False):  # slot numbers past 2^30
        assert sinks(decode, roll=0, cap=2 ** 30 + 1) == 5 and sinks(decode, cap=2 ** 30 + 128) == 5
    assert shared(cap=2 ** 30 + 1) == 5 and shared(P=2 ** 30 + 1, pc=2 ** 30 + 1) == 5
    assert sinks(False, window=382, T=4) == 5  # ring of 384 < window + T - 1
    assert sinks(False, T=513, roll=0) == 5
    assert sinks(False, T=-1) == 5 and sinks(False, T=2 ** 30, B=64, roll=0) == 5
    assert sinks(True, Hq=36) == 5 and sinks(True, B=65536) == 5
    assert bd.attention_sink_rows(0) == 0 and bd.attention_sink_rows(1) == 128 and bd.attention_sink_rows(129) == 256


def test_binding_refuses(bd):
    bf, i32 = torch.bfloat16, torch.int32
    q, kc, vc = torch.zeros(2, 8, 64, dtype=bf), torch.zeros(2, 4, 10, 64, dtype=bf), torch.zeros(2, 4, 10, 64, dtype=bf)
    kp, vp = torch.zeros(4, 30, 64, dtype=bf), torch.zeros(4, 30, 64, dtype=bf)
    len0, out = torch.zeros(1, dtype=i32), torch.zeros(2, 512, dtype=bf)
    work = torch.zeros(1 << 16, dtype=torch.uint8)
    base = dict(q=q, k_prefix=kp, v_prefix=vp, k_cache=kc, v_cache=vc, len0=len0, work=work, out=out)
    for change in (dict(q=q[0]), dict(q=q.float()), dict(q=q.transpose(0, 1)), dict(k_cache=kc[:1]), dict(v_cache=vc[:, :, :5]),
                   dict(k_cache=kc.transpose(1, 2).contiguous().transpose(1, 2)), dict(len0=torch.zeros(3, dtype=i32)),
                   dict(len0=torch.zeros(2)), dict(len0=torch.zeros(2, 1, dtype=i32)), dict(out=out[:1]), dict(out=out.float()),
                   dict(k_prefix=kp[:3]), dict(v_prefix=None), dict(k_prefix=None), dict(prefix_len=31),
                   dict(prefix_len=-1), dict(work=None), dict(work=work[:100]), dict(k_prefix=kp.permute(1, 0, 2)),
                   dict(seq_meta=torch.zeros(3, dtype=i32)), {}):
        with pytest.raises(ValueError):
            bd.op_attention_decode_shared(**{**base, **change})
    base = dict(q=q, k_cache=kc, v_cache=vc, len0=len0, out=out, window=5, sinks=1)
    for change in (dict(q=q[0]), dict(k_cache=kc[:, :3]), dict(v_cache=vc.float()), dict(len0=len0.long()),
                   dict(out=out[:, :500]), {}):
        with pytest.raises(ValueError):
            bd.op_attention_decode_sinks(**{**base, **change})
    base["q"] = torch.zeros(2, 8, 3, 64, dtype=bf)
    base["out"] = torch.zeros(6, 512, dtype=bf)
    for change in (dict(q=q), dict(out=out), dict(q=base["q"].transpose(1, 2)), dict(err=torch.zeros(1)), {}):
        with pytest.raises(ValueError):
            bd.op_attention_prefill_sinks(**{**base, **change})
