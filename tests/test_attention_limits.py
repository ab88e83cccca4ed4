"""Attention with a sliding window and sinks, and over a shared prefix, at the limits of their arguments: scores whose
maximum rises from tile to tile, large values, lengths past the cache, and own slots at the border of the rule for who reads a
prefix.

Tolerance as in test_attention_ranges: half a step of bf16 for each probability and for the result, and e for scores of up
to X in log2 units, 10 fp32 roundings of them: e = 0.7 * 10 * 2^-24 X. Scaling the sums to a larger maximum adds a few
fp32 roundings a tile, far below the half step.
"""
import math

import pytest
import torch

from tests.test_attention_ranges import _attend, _close, _err, _gen, _normal, _row, _shared_case, bd  # noqa: F401

gpu = pytest.mark.gpu


def _call(bd, q, k, v, starts, window, sinks, rolling, decode):
    """Output [B, T, Hq, dh] of a call, rows behind it checked."""
    Bn, Hq, T, dh = q.shape
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
    return out[:Bn * T].reshape(Bn, T, Hq, dh)


def _check_rows(got, q, k, v, starts, window, sinks, sink_rows, ring, rows, X):
    """Rows `rows` of every sequence against float64 attention over the slots that they see, scores up to X (log2)."""
    Bn, Hq, T, dh = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    for b in range(Bn):
        for t in rows:
            i = starts[b] + t
            slots = list(range(min(sinks, i + 1))) + list(range(max(sinks, i - window + 1, 0), i + 1))
            at = torch.tensor([_row(s, sink_rows, ring) for s in slots], device="cuda")
            for h in range(Hkv):
                ref, spread = _attend(q[b, h * G:(h + 1) * G, t], k[b, h][at], v[b, h][at])
                _close(got[b, t, h * G:(h + 1) * G], ref, spread, 7 * 2.0 ** -24 * X)


@gpu
@pytest.mark.parametrize("rolling", [False, True], ids=["full", "rolling"])
@pytest.mark.parametrize("dh,Hq,Hkv", [(64, 4, 2), (128, 8, 2)])
@pytest.mark.parametrize("T,start,window,sinks,period,rise", [
    (300, 0, 1000, 0, 128, 9.0), (200, 700, 640, 4, 128, 12.0), (130, 500, 400, 130, 128, 20.0), (1, 900, 900, 5, 64, 9.0),
    (1, 620, 300, 4, 32, 8.5), (150, 333, 500, 7, 64, 6.0), (1, 895, 900, 0, 64, 9.0), (1, 575, 520, 4, 32, 8.5)])
def test_sinks_scores_that_rise(bd, dh, Hq, Hkv, T, start, window, sinks, period, rise, rolling):
    """Scores rise by `rise` log2 units every `period` slots, so that a row's running maximum grows again and again and the
    earlier tiles' sums are scaled by 2^-rise each time. Every other stretch of slots has one high key among low ones:
    the 128 of the stretch before it keep a share of the sum that a wrong factor would show, and the values fall by 2^-rise from
    stretch to stretch, so that every stretch keeps a share of the output."""
    g = _gen(T + start + period)
    Bn = 2
    sink_rows = bd.attention_sink_rows(sinks) if rolling else 0
    ring = (window + T - 1 + 127) // 128 * 128 if rolling else 0
    starts = [start, max(0, start - 77)]
    cap = sink_rows + ring if rolling else start + T
    q = torch.ones(Bn, Hq, T, dh, device="cuda") + 0.1 * torch.randn(Bn, Hq, T, dh, generator=g, device="cuda")
    sign = torch.where(torch.rand(dh, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    q = (q * sign).to(torch.bfloat16)
    k, v = torch.empty(Bn, Hkv, cap, dh, device="cuda"), torch.empty(Bn, Hkv, cap, dh, device="cuda")
    k.fill_(float("nan"))
    v.fill_(float("nan"))
    X = 0.0
    for b in range(Bn):
        n = starts[b] + T
        first = max(0, starts[b] - window + 1)
        for s in list(range(min(sinks, first))) + list(range(first, n)):  # later slots replace earlier ones in a ring
            step = 0 if s < first else (s - first) // period
            level = rise * step
            if step % 2 and (s - first) % period != period // 2:
                level -= 40.0
            X = max(X, abs(level) + 10.0)
            noise = 0.3 * torch.randn(Hkv, dh, generator=g, device="cuda")
            at = _row(s, sink_rows, ring)
            k[b, :, at] = level / math.log2(math.e) / dh ** 0.5 * sign + noise
            v[b, :, at] = torch.randn(Hkv, dh, generator=g, device="cuda") * 2.0 ** min(
                100.0, rise * ((n - first) // period - step))  # (bf16 ends at 2^128)
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    # among the rows, those whose last stretch is one high key after a full one
    ends = {t for t in range(T) for s in starts if (s + t - max(0, s - window + 1)) % (2 * period) == 2 * period - 1}
    rows = sorted({0, 1 % T, T // 2, T - 1, min(T - 1, 127), min(T - 1, 128)} | ends)
    for decode in ([True, False] if T == 1 else [False]):
        got = _call(bd, q, k, v, starts, window, sinks, rolling, decode)
        assert torch.isfinite(got).all()
        _check_rows(got, q, k, v, starts, window, sinks, sink_rows, ring, rows, 2 * X)


@gpu
@pytest.mark.parametrize("rolling", [False, True], ids=["full", "rolling"])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("T,start,window,sinks", [(260, 500, 400, 4), (1, 2000, 1500, 130)])
def test_sinks_large_scores(bd, dh, T, start, window, sinks, rolling):
    """Scores of a few hundred, in no order: a row's weight moves from key to key over the tiles."""
    g = _gen(dh + T)
    Bn, Hq, Hkv = 2, 8, 4
    sink_rows = bd.attention_sink_rows(sinks) if rolling else 0
    ring = (window + T - 1 + 127) // 128 * 128 if rolling else 0
    cap = sink_rows + ring if rolling else start + T
    q = _normal(g, Bn, Hq, T, dh, scale=60.0)
    k, v = _normal(g, Bn, Hkv, cap, dh), _normal(g, Bn, Hkv, cap, dh)
    for decode in ([True, False] if T == 1 else [False]):
        got = _call(bd, q, k, v, [start, start // 3], window, sinks, rolling, decode)
        _check_rows(got, q, k, v, [start, start // 3], window, sinks, sink_rows, ring, sorted({0, T // 2, T - 1}), 1500.0)


@gpu
@pytest.mark.parametrize("dh", [64, 128])
def test_large_values(bd, dh):
    """Values as large as the sums before the division allow: fp32 sums of weights up to 2^8 times the largest one, so
    |v| times the number of keys below 2^119. 1,100 keys of nearly equal weight and |v| in [2^107, 2^108)."""
    g = _gen(dh + 1)
    Bn, Hq, Hkv, n = 2, 8, 4, 1100
    q, k = _normal(g, Bn, Hq, 1, dh, scale=0.1), _normal(g, Bn, Hkv, n, dh)
    sign = torch.where(torch.rand(Bn, Hkv, 1, dh, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    v = (sign * (1 + 0.99 * torch.rand(Bn, Hkv, n, dh, generator=g, device="cuda")) * 2.0 ** 107).to(torch.bfloat16)
    for decode in (True, False):
        got = _call(bd, q, k, v, [n - 1] * 2, 1000, 4, False, decode)
        _check_rows(got, q, k, v, [n - 1] * 2, 1000, 4, 0, 0, [0], 10.0)
    for P in (100, 1000):  # read by each, and once
        Bs = 70
        qs = _normal(g, Bs, Hq, dh, scale=0.1)
        ks, vs = k[0, :, P:P + 90].repeat(Bs, 1, 1, 1).contiguous(), v[0, :, P:P + 90].repeat(Bs, 1, 1, 1).contiguous()
        work = torch.empty(bd.attention_decode_shared_workspace(Bs, Hq, Hkv, dh, P), dtype=torch.uint8, device="cuda")
        out = torch.empty(Bs, Hq * dh, dtype=torch.bfloat16, device="cuda")
        bd.op_attention_decode_shared(qs, k[0, :, :P].contiguous(), v[0, :, :P].contiguous(), ks, vs,
                                      torch.tensor([89], dtype=torch.int32, device="cuda"), work, out)
        torch.cuda.synchronize()
        for b in (0, Bs // 2, Bs - 1):
            for h in range(Hkv):
                ref, spread = _attend(qs[b, 2 * h:2 * h + 2], k[0, h, :P + 90], v[0, h, :P + 90])
                _close(out.reshape(Bs, Hq, dh)[b, 2 * h:2 * h + 2], ref, spread)


@gpu
@pytest.mark.parametrize("dh", [64, 128])
def test_sinks_lengths_past_the_limits(bd, dh):
    """A length beyond the cache counts as the longest that fits (2^30 in a rolling buffer); a negative one counts as 0 in a
    prefill and gives zeros in decode. Each equals the call with the length that it counts as, and float64."""
    g = _gen(dh)
    Bn, Hq, Hkv, cap, window, sinks = 3, 8, 4, 500, 150, 4
    k, v = _normal(g, Bn, Hkv, cap, dh), _normal(g, Bn, Hkv, cap, dh)
    for T in (1, 3, 140):
        q = _normal(g, Bn, Hq, T, dh)
        last = cap - T
        given, counts = [last + 40, last + 1, 2 ** 31 - 1], [last] * 3
        for decode in ([True, False] if T == 1 else [False]):
            got = _call(bd, q, k, v, given, window, sinks, False, decode)
            assert torch.equal(got, _call(bd, q, k, v, counts, window, sinks, False, decode))
            _check_rows(got, q, k, v, counts, window, sinks, 0, 0, sorted({0, T - 1}), 10.0)
        got = _call(bd, q, k, v, [-5, -1, -2 ** 31], window, sinks, False, False)
        _check_rows(got, q, k, v, [0] * 3, window, sinks, 0, 0, sorted({0, T // 2, T - 1}), 10.0)
    q = _normal(g, Bn, Hq, 1, dh)
    got = _call(bd, q, k, v, [cap, -1, -2 ** 31], window, sinks, False, True)
    assert torch.all(got[1:] == 0)
    _check_rows(got[:1], q[:1], k[:1], v[:1], [cap - 1], window, sinks, 0, 0, [0], 10.0)
    # a ring turned up to the largest slot
    sink_rows, ring = 128, 384
    k, v = _normal(g, Bn, Hkv, sink_rows + ring, dh), _normal(g, Bn, Hkv, sink_rows + ring, dh)
    given, counts = [2 ** 30 + 77, 2 ** 30, 2 ** 31 - 1], [2 ** 30] * 3
    for T in (1, 200):
        q = _normal(g, Bn, Hq, T, dh)
        for decode in ([True, False] if T == 1 else [False]):
            got = _call(bd, q, k, v, given, window, sinks, True, decode)
            assert torch.equal(got, _call(bd, q, k, v, counts, window, sinks, True, decode))
            _check_rows(got, q, k, v, counts, window, sinks, sink_rows, ring, sorted({0, T - 1}), 10.0)


@gpu
@pytest.mark.parametrize("Bn,Hq,Hkv,P,cap", [(64, 16, 8, 128, 256), (64, 16, 8, 128, 258), (64, 16, 8, 128, 512),
                                             (2, 8, 8, 4096, 8192), (2, 8, 8, 4096, 8194), (16, 8, 4, 600, 2896),
                                             (16, 8, 4, 600, 2898)])
def test_shared_own_slots_at_the_border(bd, Bn, Hq, Hkv, P, cap):
    """A prefix is read by each sequence only while the pairs of sequence and kv head times P are at most 2^16 and, counted
    with half of the own slots, at most 2^17: sizes on both sides of the second border, with and without a layout."""
    _shared_case(bd, Bn, Hq, Hkv, 64, P, cap, [(b * 37 + cap - 3) % cap for b in range(Bn)], seed=cap)
    if cap <= 512:
        _shared_case(bd, Bn, Hq, Hkv, 128, P, cap + P, [cap - 1], seed=cap, meta=[130, 128] + [(7 * b) % 45 for b in range(Bn)])


# ------------------------------------------------------------------------------------------------ refusals (CPU)

def test_prefill_refuses_items_past_the_kernels_counters(bd):  # noqa: F811
    """Query tiles x heads x sequences are counted in 32 bits, a round of CTAs past the last one included."""
    import ctypes
    p = ctypes.c_void_p(64)  # never dereferenced: the call is refused on the host
    L = bd.lib()
    for Hq, Bn in ((2 ** 16 - 1, 2 ** 15), (2 ** 31 - 1, 1), (1, 2 ** 31 - 1), (2 ** 31 - 300, 1)):
        assert L.qwen3_op_attention_prefill_sinks(p, p, p, Bn, 1, Hq, Hq, 64, 512, p, 0, 100, 4, 0, p, None, None) == 5
