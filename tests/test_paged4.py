"""The paged 4-bit cache: append (qwen3_op_append_paged4), read (qwen3_op_read_paged4) and decode attention
(qwen3_op_attention_decode_paged4) against float64.

Tolerances. A bf16 result is off by half a step, 2^-8 of its value at most.
  Rotated heads: fp32 products and sums of a few terms of the size |a| + |b| of the rotated pair, after a norm whose sum of
  up to 128 squares is off by at most 128 * 2^-24 of itself (half of that in its root): 2^-16 (|a| + |b|) covers both.
  Cached values: a code stands for a value within half a scale of it; the fp32 key that is quantised is off as above.
  Decode: the reference takes the cache's own bytes, so K and V are exact. A weight (probability times scale) is rounded to fp16,
  2^-11 of itself, and below fp16's normal range by 2^-25 where the head's largest is 2^13 or more: 2^-38 of the largest
  weight for each key, times codes up to 15. A product of 16 keys adds 17 terms to an fp32 sum, each cut off below 2^-24 of
  the largest: 2^-20 of the sum's terms a product, and as much for the joins and changes of range. Scores are four such
  products a group of dims (2^-18 of their terms), a few fp32 operations and an exponential: 2^-17 (1 + the largest score's
  terms) of every weight.
"""
import struct

import numpy as np
import pytest
import torch

from qwen3_decoder_transformer_gb300 import build as B

HEADS = [(8, 4, 64), (16, 8, 128), (4, 4, 128), (12, 4, 64), (12, 4, 128), (32, 8, 128), (16, 2, 64), (8, 1, 128)]
PAGES = [16, 32, 64, 128, 256]
EPS = 1e-6


@pytest.fixture(scope="module")
def bd():
    B.build()
    from qwen3_decoder_transformer_gb300 import binding
    binding.lib()
    return binding


# ------------------------------------------------------------------------------------------------ the cache in numpy

def _unpack(pages, page, dh):
    """pages [P, Hkv, bytes] uint8 (host) -> codes [P, Hkv, page, dh], scale and minimum [P, Hkv, page, dh / 64] (float64)."""
    raw = pages.numpy()
    P, H, _ = raw.shape
    c = raw[:, :, :page * dh // 2].reshape(P, H, page, dh // 2)
    codes = np.stack([c & 15, c >> 4], axis=-1).reshape(P, H, page, dh)
    side = np.ascontiguousarray(raw[:, :, page * dh // 2:]).view(np.uint16).reshape(P, H, page, dh // 64, 2)
    side = (side.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return codes, side[..., 0], side[..., 1]


def _values(pages, page, dh):
    codes, scale, low = _unpack(pages, page, dh)
    with np.errstate(invalid="ignore", over="ignore"):
        return np.repeat(low, 64, axis=-1) + np.repeat(scale, 64, axis=-1) * codes


def _rows(values, table, page, slots, b):
    """values [P, Hkv, page, dh] -> the slots of sequence b, [n, Hkv, dh]."""
    return values[table[b, slots // page], :, slots % page]


class Cache:
    """A page pool on the GPU with every byte 255 (codes 15, scales and minima NaN), and shuffled page tables."""

    def __init__(self, Hkv, dh, page, lens, seed, spare=2):
        rng = np.random.default_rng(seed)
        counts = [-(-n // page) for n in lens]
        self.page, self.dh, self.Hkv = page, dh, Hkv
        n_pages = sum(counts) + spare
        order = rng.permutation(n_pages)
        # entries that no call needs are far out of range
        self.table = np.full((len(lens), max(1, max(counts, default=1)) + 1), 2 ** 30, dtype=np.int32)
        at = 0
        for b, n in enumerate(counts):
            self.table[b, :n] = order[at:at + n]
            at += n
        size = page * (dh // 2 + dh // 16)
        self.k = torch.full((n_pages, Hkv, size), 255, dtype=torch.uint8, device="cuda")
        self.v = torch.full((n_pages, Hkv, size), 255, dtype=torch.uint8, device="cuda")
        self.dtable = torch.from_numpy(self.table).cuda()

    def fill(self, lens, seed, spread=1.0):
        """Random codes with scales and minima of either sign's size in the slots below lens."""
        gen = torch.Generator().manual_seed(seed)
        page, dh = self.page, self.dh
        for pages in (self.k, self.v):
            host = pages.cpu()
            P, H, _ = host.shape
            codes = torch.randint(0, 256, (P, H, page, dh // 2), generator=gen, dtype=torch.uint8)
            scale = (torch.rand(P, H, page, dh // 64, generator=gen) + 0.1) * 0.3 * spread
            low = -7.5 * scale * (1 + 0.3 * torch.randn(P, H, page, dh // 64, generator=gen))
            side = torch.stack([scale, low], dim=-1).to(torch.bfloat16).view(torch.uint8).reshape(P, H, page, -1)
            hv = host[:, :, :page * dh // 2].view(P, H, page, dh // 2)
            sv = host[:, :, page * dh // 2:].view(P, H, page, dh // 16)
            for b, n in enumerate(lens):
                s = np.arange(max(n, 0))
                at, off = torch.from_numpy(self.table[b, s // page]).long(), torch.from_numpy(s % page)
                hv[at, :, off] = codes[at, :, off]
                sv[at, :, off] = side[at, :, off]
            pages.copy_(host)
        return self


def _cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _table(dh, n):
    """[n, dh] bf16 cos and sin on the host."""
    w = 1e6 ** (-np.arange(0, dh, 2) / dh)
    a = np.arange(n)[:, None] * w
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], axis=1)).to(torch.bfloat16)


def _rotated(x, gamma, cs):
    """x [n, H, dh] float64, cs [n, dh]: norm, rotation; and the size of the terms."""
    if gamma is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS) * gamma
    h = x.shape[-1] // 2
    a, b, c, s = x[..., :h], x[..., h:], cs[:, None, :h], cs[:, None, h:]
    size = np.abs(a) + np.abs(b)
    return np.concatenate([a * c - b * s, b * c + a * s], -1), np.concatenate([size, size], -1)


def _append(bd, heads, page, lens, start, pad=0, norm=True, seed=0, scale=1.0, ld_extra=0, qkv=None, n_pos=None, cache=None,
            stream=None):
    Hq, Hkv, dh = heads
    n = sum(lens)
    ends = [a + k for a, k in zip(start, lens)]
    c = cache or Cache(Hkv, dh, page, ends, seed)
    gen = torch.Generator().manual_seed(seed)
    width = (Hq + 2 * Hkv) * dh
    if qkv is None:
        qkv = (torch.randn(n + pad, width + ld_extra, generator=gen) * scale).to(torch.bfloat16)
    g = [(1 + 0.1 * torch.randn(dh, generator=gen)).to(torch.bfloat16) if norm else None for _ in range(2)]
    cs = _table(dh, n_pos or max(1, max(ends, default=1)))
    dq = qkv.cuda()[:, :width]
    q_out = torch.full((n + pad, Hq, dh), 7.0, dtype=torch.bfloat16, device="cuda")
    k_out = torch.full((n + pad, Hkv, dh), 7.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu, st = _cu(lens), torch.tensor(start, dtype=torch.int32, device="cuda")
    args = dict(q_gamma=None if g[0] is None else g[0].cuda(), k_gamma=None if g[1] is None else g[1].cuda(), eps=EPS, err=err)
    bd.op_append_paged4(dq, cu, st, cs.cuda(), c.k, c.v, c.dtable, q_out, k_out=k_out, stream=stream, **args)
    torch.cuda.synchronize()
    return dict(cache=c, qkv=qkv[:, :width], g=g, cs=cs, q=q_out.cpu(), k=k_out.cpu(), err=int(err.item()), cu=cu, start=st)


def _positions(lens, start):
    return np.concatenate([np.arange(a, a + n) for a, n in zip(start, lens)]).astype(int) if lens else np.zeros(0, int)


def _check_append(r, heads, lens, start):
    Hq, Hkv, dh = heads
    n = sum(lens)
    pos = _positions(lens, start)
    x = r["qkv"][:n].double().numpy().reshape(n, Hq + 2 * Hkv, dh)
    cs = r["cs"].double().numpy()[pos]
    g = [None if t is None else t.double().numpy() for t in r["g"]]
    c = r["cache"]
    for got, part, gamma in ((r["q"], x[:, :Hq], g[0]), (r["k"], x[:, Hq:Hq + Hkv], g[1])):
        ref, size = _rotated(part, gamma, cs)
        y = got[:n].double().numpy()
        assert np.all(np.abs(y - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -16 * size)
        assert torch.all(got[n:] == 7.0)  # behind the last sequence
    seq = np.repeat(np.arange(len(lens)), lens)
    for pages, is_k in ((c.k, True), (c.v, False)):
        codes, scale, low = _unpack(pages.cpu(), c.page, dh)
        at, off = c.table[seq, pos // c.page], pos % c.page
        codes, scale, low = codes[at, :, off], scale[at, :, off], low[at, :, off]
        if is_k:
            ref, size = _rotated(x[:, Hq:Hq + Hkv], g[1], cs)
        else:
            ref = x[:, Hq + Hkv:]
            size = np.zeros_like(ref)
        gr = ref.reshape(n, Hkv, dh // 64, 64)
        slack = 2.0 ** -16 * size.reshape(gr.shape).max(-1)
        mn, mx = gr.min(-1), gr.max(-1)
        # rounded down (up) to bf16: below (above) by less than a step, 2^-7 of the value
        assert np.all(low <= mn + slack) and np.all(low >= mn - 2.0 ** -7 * np.abs(mn) - slack)
        want = (mx - low) / 15
        assert np.all(scale >= want * (1 - 2.0 ** -20) - slack) and np.all(scale <= want * (1 + 2.0 ** -7) + slack)
        val = low[..., None] + scale[..., None] * codes.reshape(gr.shape)
        assert np.all(np.abs(val - gr) <= scale[..., None] * (0.5 + 2.0 ** -18) + slack[..., None])
        if not is_k:  # bf16 inputs: exactly the definition
            q = np.where(scale[..., None] > 0, (gr - low[..., None]) / np.where(scale > 0, scale, 1)[..., None], 0)
            assert np.array_equal(codes.reshape(gr.shape), np.clip(np.rint(q), 0, 15))
    # every other byte of the pages is as it was
    for pages in (c.k, c.v):
        host = pages.cpu().numpy().copy()
        P, H, _ = host.shape
        cv = host[:, :, :c.page * dh // 2].reshape(P, H, c.page, dh // 2)
        sv = host[:, :, c.page * dh // 2:].reshape(P, H, c.page, dh // 16)
        at, off = c.table[seq, pos // c.page], pos % c.page
        cv[at, :, off] = 255
        sv[at, :, off] = 255
        assert np.all(cv == 255) and np.all(sv == 255)


# ---------------------------------------------------------------------------------------------------- append and read

@pytest.mark.gpu
@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_append(bd, heads, page):
    lens, start = [1, 0, 40, 3, 0, 17, 300], [0, 5, 33, 15, 0, 255, 1]
    r = _append(bd, heads, page, lens, start, pad=3, norm=page != 32, seed=page + heads[0], scale=1.0 if page < 64 else 5.0)
    assert r["err"] == 0
    _check_append(r, heads, lens, start)


@pytest.mark.gpu
@pytest.mark.parametrize("seqs", [1, 2, 31, 32, 33, 64, 1023, 1025, 1100])
def test_append_decode_batches(bd, seqs):
    """One row a sequence, over the sizes at which the search for a row's sequence takes another step."""
    heads, start = (4, 2, 64), [(i * 37) % 50 for i in range(seqs)]
    r = _append(bd, heads, 16, [1] * seqs, start, pad=2, seed=seqs)
    assert r["err"] == 0
    _check_append(r, heads, [1] * seqs, start)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,n", [((32, 8, 128), 150), ((32, 8, 128), 300), ((16, 8, 128), 801), ((32, 8, 128), 2600),
                                     ((4, 4, 64), 5003)], ids=str)
def test_append_splits(bd, heads, n):
    """Tokens shared by several warps, and warps with several tokens, over the ends of sequences and pages."""
    lens, start = [n // 3, 0, n // 3 + 1, n - n // 3 * 2 - 1], [7, 0, 30, 0]
    r = _append(bd, heads, 16, lens, start, pad=5, seed=n)
    assert r["err"] == 0
    _check_append(r, heads, lens, start)


@pytest.mark.gpu
def test_append_rows_further_apart_and_no_keys_out(bd):
    heads, lens, start = (8, 4, 64), [9, 2], [3, 30]
    r = _append(bd, heads, 16, lens, start, ld_extra=24, seed=3)
    _check_append(r, heads, lens, start)
    c = Cache(4, 64, 16, [12, 32], 3)
    q = torch.zeros(11, 8, 64, dtype=torch.bfloat16, device="cuda")
    bd.op_append_paged4(r["qkv"].contiguous().cuda(), r["cu"], r["start"], r["cs"].cuda(), c.k, c.v, c.dtable, q,
                        q_gamma=r["g"][0].cuda(), k_gamma=r["g"][1].cuda(), eps=EPS)
    assert torch.equal(q.cpu(), r["q"]) and torch.equal(c.k.cpu(), r["cache"].k.cpu())


@pytest.mark.gpu
def test_rows_before_the_first_sequence(bd):
    """Bounds that begin behind row 0: the rows in front belong to no sequence and are left as they were."""
    heads, lens, start, front = (8, 4, 64), [9, 0, 30], [3, 1, 20], 5
    ref = _append(bd, heads, 16, lens, start, seed=8)
    c = Cache(4, 64, 16, [a + n for a, n in zip(start, lens)], 8)
    qkv = torch.cat([torch.full((front, 16 * 64), float("nan"), dtype=torch.bfloat16), ref["qkv"]]).cuda()
    q = torch.full((front + 39, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    k = torch.full((front + 39, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = ref["cu"] + front
    bd.op_append_paged4(qkv, cu, ref["start"], ref["cs"].cuda(), c.k, c.v, c.dtable, q, k_out=k, q_gamma=ref["g"][0].cuda(),
                        k_gamma=ref["g"][1].cuda(), eps=EPS, err=err)
    assert torch.equal(q[front:].cpu(), ref["q"]) and torch.equal(k[front:].cpu(), ref["k"])
    assert torch.all(q[:front] == 7.0) and torch.all(k[:front] == 7.0)
    assert torch.equal(c.k, ref["cache"].k) and torch.equal(c.v, ref["cache"].v)
    kr, vr = torch.full_like(k, 7.0), torch.full_like(k, 7.0)
    bd.op_read_paged4(c.k, c.v, c.dtable, cu, ref["start"], kr, vr, err=err)
    assert torch.all(kr[:front] == 7.0) and torch.all(vr[:front] == 7.0) and torch.isfinite(kr[front:].float()).all()
    assert int(err.item()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["q", "k"])
def test_append_with_one_gamma(bd, which):
    """A norm of the queries alone, or of the keys alone: each as with both or none."""
    heads, lens, start = (8, 4, 64), [9, 30], [3, 20]
    both = _append(bd, heads, 16, lens, start, seed=9)
    none = _append(bd, heads, 16, lens, start, seed=9, norm=False, qkv=both["qkv"])
    c = Cache(4, 64, 16, [12, 50], 9)
    q = torch.empty(39, 8, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.empty(39, 4, 64, dtype=torch.bfloat16, device="cuda")
    g = {which + "_gamma": both["g"]["qk".index(which)].cuda()}
    bd.op_append_paged4(both["qkv"].contiguous().cuda(), both["cu"], both["start"], both["cs"].cuda(), c.k, c.v, c.dtable, q,
                        k_out=k, eps=EPS, **g)
    a, b = (both, none) if which == "q" else (none, both)
    assert torch.equal(q.cpu(), a["q"]) and torch.equal(k.cpu(), b["k"])
    assert torch.equal(c.k, b["cache"].k) and torch.equal(c.v, both["cache"].v)


@pytest.mark.gpu
def test_append_values_at_the_edges(bd):
    """Groups of one value, of both signs, of zeros, of very large and of subnormal values; NaN and infinities."""
    heads, dh = (2, 2, 64), 64
    width = 6 * dh
    x = torch.randn(9, width, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    v = x.view(9, 6, dh)
    v[0, 4] = 3.0
    v[1, 4] = 0.0
    v[2, 4] = -2.5
    v[3, 4, :32] = 1e-40
    v[3, 4, 32:] = -3e-39
    v[4, 4] *= 1e37
    v[5, 4, 7] = float("nan")
    v[6, 4, 8] = float("inf")
    v[7, 4, 9] = float("-inf")
    v[8, 4, 0], v[8, 4, 1] = 3e38, -3e38  # their difference is past fp32
    r = _append(bd, heads, 16, [9], [0], norm=False, qkv=x)
    codes, scale, low = _unpack(r["cache"].v.cpu(), 16, dh)
    at = r["cache"].table[0, 0]
    codes, scale, low = codes[at, 0, :9], scale[at, 0, :9, 0], low[at, 0, :9, 0]
    assert np.all(np.isnan(scale[5:])) and np.all(np.isnan(low[5:]))
    ref = v[:5, 4].double().numpy()
    val = low[:5, None] + scale[:5, None] * codes[:5]
    assert np.all(np.abs(val - ref) <= scale[:5, None] * (0.5 + 2.0 ** -18))
    assert np.array_equal(val[:3], ref[:3])
    # the other head of the same rows is untouched by it
    c2, s2, l2 = _unpack(r["cache"].v.cpu(), 16, dh)
    assert np.all(np.isfinite(s2[at, 1, :9])) and np.all(np.isfinite(l2[at, 1, :9]))


@pytest.mark.gpu
@pytest.mark.parametrize("dh", [64, 128])
def test_append_quotients_beside_a_tie(bd, dh):
    """Values less than 2^-20 of a scale on either side of the middle between two codes take the nearer code, those in the middle the
    even one. The differences to the minimum are exact in fp32, and the scale is 2."""
    lows = [-1.0, -3.0, -5.0, -15.0]  # 0 lies in the middle of codes 0 and 1, 1 and 2, 2 and 3, 7 and 8
    x = torch.zeros(len(lows), 3 * dh, dtype=torch.bfloat16)
    v = x[:, 2 * dh:].view(len(lows), dh // 64, 64)
    for i, low in enumerate(lows):
        step = 2.0 ** (np.floor(np.log2(-low)) - 23)  # of fp32 at the difference
        v[i, :, 0], v[i, :, 1] = low, low + 30
        for j, d in enumerate((1, -1, 2, -2, 3, -3, 4, -4)):
            v[i, :, 2 + j] = d * step
    r = _append(bd, (1, 1, dh), 16, [len(lows)], [0], norm=False, qkv=x)
    codes, scale, low = _unpack(r["cache"].v.cpu(), 16, dh)
    at = r["cache"].table[0, 0]
    assert np.all(scale[at, 0, :len(lows)] == 2) and np.all(low[at, 0, :len(lows)] == np.array(lows)[:, None])
    q = (v.double().numpy() - np.array(lows)[:, None, None]) / 2  # exact
    assert np.array_equal(codes[at, 0, :len(lows)].reshape(q.shape), np.rint(q))


@pytest.mark.gpu
def test_append_flags_what_it_cannot_place(bd):
    heads, lens = (8, 4, 64), [4, 4, 4, 4]
    ref = _append(bd, heads, 16, lens, [14, 3, 5, 9], seed=5, n_pos=64)
    assert ref["err"] == 0

    def again(start, table=None, n_pos=64, cu=None):
        c = Cache(4, 64, 16, [18, 7, 9, 13], 5)
        if table is not None:
            c.dtable = torch.from_numpy(table(c.table.copy())).cuda()
        q = torch.full((16, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        k = torch.full((16, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        bd.op_append_paged4(ref["qkv"].contiguous().cuda(), ref["cu"] if cu is None else cu,
                            torch.tensor(start, dtype=torch.int32, device="cuda"), ref["cs"].cuda()[:n_pos].contiguous(), c.k,
                            c.v, c.dtable, q, k_out=k, q_gamma=ref["g"][0].cuda(), k_gamma=ref["g"][1].cuda(), eps=EPS, err=err)
        return q.cpu(), c, int(err.item())

    def bad(t):
        t[0, 1] = -1          # slots 16, 17 of sequence 0
        t[2, 0] = 1 << 20
        return t

    q, c, err = again([14, 3, 5, 9], bad)
    assert err == 4 and torch.equal(q, ref["q"])  # the rows without a page still get their outputs
    got, want = _values(c.k.cpu(), 16, 64), _values(ref["cache"].k.cpu(), 16, 64)
    for b, s in ((0, [14, 15]), (1, [3, 4, 5, 6]), (3, [9, 10, 11, 12])):
        assert np.array_equal(_rows(got, c.table, 16, np.array(s), b), _rows(want, c.table, 16, np.array(s), b))
    assert np.all(np.isnan(_rows(got, c.table, 16, np.array([5, 6, 7, 8]), 2)))
    # slots that are negative, past the rotation table, past the page table's reach
    q, c, err = again([-2, 60, 5, 2 ** 31 - 2])
    assert err == 4
    assert torch.all(q[:2] == 7.0) and not torch.any(q[2:4] == 7.0)
    assert torch.all(q[12:] == 7.0) and torch.equal(q[8:12], ref["q"][8:12])
    q, c, err = again([14, 3, 5, 9], n_pos=8)
    assert err == 4 and torch.all(q[0:4] == 7.0) and torch.equal(q[4:8], ref["q"][4:8]) and torch.all(q[11] == 7.0)


@pytest.mark.gpu
@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("heads", HEADS[:5], ids=str)
def test_read(bd, heads, page):
    _, Hkv, dh = heads
    lens, start = [1, 0, 60, 5, 200], [0, 3, 20, 250, 31]
    ends = [a + n for a, n in zip(start, lens)]
    c = Cache(Hkv, dh, page, ends, page).fill(ends, page)
    n = sum(lens)
    k = torch.full((n + 2, Hkv, dh), 7.0, dtype=torch.bfloat16, device="cuda")
    v, err = k.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    bd.op_read_paged4(c.k, c.v, c.dtable, _cu(lens), torch.tensor(start, dtype=torch.int32, device="cuda"), k, v, err=err)
    assert int(err.item()) == 0
    seq, pos = np.repeat(np.arange(len(lens)), lens), _positions(lens, start)
    for got, pages in ((k, c.k), (v, c.v)):
        val = _values(pages.cpu(), page, dh)[c.table[seq, pos // page], :, pos % page]
        # the sum is rounded to fp32 (2^-24 of it), then to bf16
        assert np.all(np.abs(got[:n].cpu().double().numpy() - val) <= 2.0 ** -8 * np.abs(val) * (1 + 2.0 ** -14))
        assert torch.all(got[n:] == 7.0)


@pytest.mark.gpu
def test_read_leaves_what_it_cannot_find(bd):
    c = Cache(2, 64, 16, [40, 40], 1).fill([40, 40], 1)
    c.dtable[0, 1] = -5
    k = torch.full((80, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    v, err = k.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    bd.op_read_paged4(c.k, c.v, c.dtable, _cu([40, 40]), torch.zeros(2, dtype=torch.int32, device="cuda"), k, v, err=err)
    assert int(err.item()) == 4
    assert torch.all(k[16:32] == 7.0) and torch.all(v[16:32] == 7.0)
    assert not torch.any(k[:16].float() == 7.0) and torch.isfinite(k[32:].float()).all()


# ---------------------------------------------------------------------------------------------------- decode attention

def _decode(bd, q, c, len0, work=None, stream=None, out=None):
    Bq, Hq, dh = q.shape
    if out is None:
        out = torch.full((Bq, Hq * dh), 7.0, dtype=torch.bfloat16, device="cuda")
    if work is None:
        work = torch.full((bd.attention_decode_paged4_workspace(Bq, Hq, c.Hkv, dh),), 255, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bd.op_attention_decode_paged4(q, c.k, c.v, c.dtable, len0, work, out, err=err, stream=stream)
    torch.cuda.synchronize()
    return out, int(err.item())


def _ref_decode(q, c, lens, cap=None):
    """Result and bound [B, Hq, dh] for q (host bf16)."""
    Bq, Hq, dh = q.shape
    codes_k, scale_k, low_k = _unpack(c.k.cpu(), c.page, dh)
    codes_v, scale_v, low_v = _unpack(c.v.cpu(), c.page, dh)
    ref, tol = np.zeros((Bq, Hq, dh)), np.zeros((Bq, Hq, dh))
    g = Hq // c.Hkv
    for b, n in enumerate(lens):
        if n <= 0:
            continue
        s = np.arange(n)
        pick = lambda a: a[c.table[b, s // c.page], :, s % c.page]  # noqa: E731
        sk, lk = np.repeat(pick(scale_k), 64, -1), np.repeat(pick(low_k), 64, -1)
        k = lk + sk * pick(codes_k)
        sv, lv, cv = np.repeat(pick(scale_v), 64, -1), np.repeat(pick(low_v), 64, -1), pick(codes_v)
        v = lv + sv * cv
        for h in range(Hq):
            j = h // g
            qq = q[b, h].double().numpy()
            x = k[:, j] @ qq / dh ** 0.5
            size = ((np.abs(lk[:, j]) + sk[:, j] * pick(codes_k)[:, j]) @ np.abs(qq)).max() / dh ** 0.5
            p = np.exp(x - x.max())
            p /= p.sum()
            ref[b, h] = p @ v[:, j]
            w, low = sv[:, j] * cv[:, j], np.abs(lv[:, j])
            steps = -(-n // 16) + 16
            tol[b, h] = (2.0 ** -8 * np.abs(ref[b, h]) + 2.0 ** -11 * (p @ w) + n * 15 * 2.0 ** -38 * (p[:, None] * sv[:, j]).max() +
                         steps * 2.0 ** -20 * (p @ (w + low)) + 2.0 ** -17 * (1 + size) * (p @ (w + low)))
    return ref, tol


def _check_decode(got, q, c, lens):
    ref, tol = _ref_decode(q, c, lens)
    y = got.cpu().double().numpy().reshape(ref.shape)
    assert np.all(np.abs(y - ref) <= tol), float((np.abs(y - ref) / np.where(tol > 0, tol, 1)).max())


@pytest.mark.gpu
@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_decode(bd, heads, page):
    Hq, Hkv, dh = heads
    lens = [1, 15, 16, 17, 0, 31, 32, 33, 100, 257, 700]
    c = Cache(Hkv, dh, page, lens, page + dh).fill(lens, page)
    q = torch.randn(len(lens), Hq, dh, generator=torch.Generator().manual_seed(page)).to(torch.bfloat16)
    len0 = torch.tensor([n - 1 for n in lens], dtype=torch.int32, device="cuda")
    out, err = _decode(bd, q.cuda(), c, len0)
    assert err == 0
    _check_decode(out, q, c, lens)


@pytest.mark.gpu
@pytest.mark.parametrize("B_", [1, 2, 7, 255, 256, 257, 383, 384, 385, 600, 1500])
@pytest.mark.parametrize("heads", [(8, 4, 64), (16, 8, 128)], ids=str)
def test_decode_batches(bd, heads, B_):
    """Batches past the strips in which lengths are counted, with empty sequences among them."""
    Hq, Hkv, dh = heads
    lens = [(i * 131) % 97 for i in range(B_)]
    lens[0] = 61
    c = Cache(Hkv, dh, 16, lens, B_).fill(lens, B_)
    q = torch.randn(B_, Hq, dh, generator=torch.Generator().manual_seed(B_)).to(torch.bfloat16)
    len0 = torch.tensor([n - 1 if n else -1 - i for i, n in enumerate(lens)], dtype=torch.int32, device="cuda")
    out, err = _decode(bd, q.cuda(), c, len0)
    assert err == 0
    _check_decode(out, q, c, lens)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,lens,page", [((8, 1, 128), [20011], 64), ((4, 4, 64), [30000, 1], 256),
                                             ((32, 8, 128), [5000, 3000, 40], 16), ((16, 2, 64), [9999], 32),
                                             ((16, 8, 128), [130], 64), ((16, 2, 128), [2500], 128), ((32, 8, 128), [9000], 16),
                                             ((8, 1, 64), [60000], 32), ((32, 8, 128), [20000, 0, 20000], 64)], ids=str)
def test_decode_long(bd, heads, lens, page):
    Hq, Hkv, dh = heads
    c = Cache(Hkv, dh, page, lens, page).fill(lens, page)
    q = torch.randn(len(lens), Hq, dh, generator=torch.Generator().manual_seed(page)).to(torch.bfloat16)
    out, err = _decode(bd, q.cuda(), c, torch.tensor([n - 1 for n in lens], dtype=torch.int32, device="cuda"))
    assert err == 0
    _check_decode(out, q, c, lens)


@pytest.mark.gpu
@pytest.mark.parametrize("q_scale,spread", [(30.0, 1.0), (1e-6, 1.0), (1.0, 1e4), (1e10, 1e-10), (1.0, 1e-3), (1e8, 1.0)])
def test_decode_sizes_of_values(bd, q_scale, spread):
    """Scores far apart, all alike, and values of other sizes."""
    heads, lens = (12, 4, 128), [300, 64]
    c = Cache(4, 128, 32, lens, 9).fill(lens, 9, spread)
    q = (torch.randn(2, 12, 128, generator=torch.Generator().manual_seed(9)) * q_scale).to(torch.bfloat16)
    q[0, 3] = 0
    q[0, 4, 1:] = 0
    out, err = _decode(bd, q.cuda(), c, torch.tensor([299, 63], dtype=torch.int32, device="cuda"))
    assert err == 0
    _check_decode(out, q, c, lens)


def _smaller_values(c, powers):
    """Multiply the scales and minima of V by 2^-powers[s] (exact), s: the slot, of every sequence."""
    host = c.v.cpu()
    side = host[:, :, c.page * c.dh // 2:].view(torch.bfloat16).view(*host.shape[:2], c.page, c.dh // 64, 2)
    s = np.arange(len(powers))
    by = torch.from_numpy(2.0 ** -np.asarray(powers, dtype=np.float64)).float()
    for b in range(c.table.shape[0]):
        have = c.table[b, s // c.page] < 2 ** 30
        at, off = torch.from_numpy(c.table[b, s // c.page][have]).long(), torch.from_numpy((s % c.page)[have])
        side[at, :, off] = (side[at, :, off].float() * by[torch.from_numpy(have)][:, None, None, None]).to(torch.bfloat16)
    c.v.copy_(host)


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [(16, 8, 128), (12, 4, 64), (8, 1, 128)], ids=str)
@pytest.mark.parametrize("power", [45, 50, 62, 75, 84, 86, 100, 114])
@pytest.mark.parametrize("q_scale", [1.0, 30.0])
def test_decode_small_values(bd, heads, power, q_scale):
    """Values down to 2^-114: their codes count as those of any other size do, also where scores far above the ones before come."""
    Hq, Hkv, dh = heads
    lens = [700, 64, 3]
    c = Cache(Hkv, dh, 16, lens, 21).fill(lens, 21)
    _smaller_values(c, [power] * 700)
    q = (torch.randn(3, Hq, dh, generator=torch.Generator().manual_seed(21)) * q_scale).to(torch.bfloat16)
    out, err = _decode(bd, q.cuda(), c, torch.tensor([n - 1 for n in lens], dtype=torch.int32, device="cuda"))
    assert err == 0
    _check_decode(out, q, c, lens)


@pytest.mark.gpu
@pytest.mark.parametrize("step", [0.01, 0.1])
def test_decode_small_values_and_rising_scores(bd, step):
    """Small values whose scores grow along the sequence, past the running maximum in every unit or past its range."""
    c = Cache(2, 64, 64, [2048], 23).fill([2048], 23)
    _smaller_values(c, [90] * 2048)
    host = c.k.cpu()
    side = host[:, :, 64 * 32:].view(torch.bfloat16).view(*host.shape[:2], 64, 2)
    s = np.arange(2048)
    at, off = torch.from_numpy(c.table[0, s // 64]).long(), torch.from_numpy(s % 64)
    side[at, :, off, 1] = (torch.from_numpy(s).float() * step).to(torch.bfloat16)[:, None].expand(-1, 2)
    c.k.copy_(host)
    q = torch.full((1, 8, 64), 0.5).to(torch.bfloat16)
    out, err = _decode(bd, q.cuda(), c, torch.tensor([2047], dtype=torch.int32, device="cuda"))
    assert err == 0
    _check_decode(out, q, c, [2048])


@pytest.mark.gpu
@pytest.mark.parametrize("order", ["falling", "rising", "one large", "one large, unseen", "zeros first"])
@pytest.mark.parametrize("heads", [(16, 8, 128), (12, 4, 64), (8, 1, 128)], ids=str)
def test_decode_values_of_many_sizes(bd, heads, order):
    """Values whose sizes change along a sequence by up to 2^110, and a key of large values that some heads' scores leave nothing of."""
    Hq, Hkv, dh = heads
    n = 900
    c = Cache(Hkv, dh, 64, [n], 22).fill([n], 22)
    s = np.arange(n)
    powers = {"falling": s * 110 // n, "rising": 110 - s * 110 // n, "zeros first": np.where(s < 200, 1000, 90)}.get(
        order, np.where(s == 450, 0, 90))
    _smaller_values(c, powers)
    q = torch.randn(1, Hq, dh, generator=torch.Generator().manual_seed(22)).to(torch.bfloat16)
    if order == "one large, unseen":  # key 450 is -30 in every dim: scores of -300 and less for a positive query
        host = c.k.cpu()
        side = host[:, :, 64 * dh // 2:].view(torch.bfloat16).view(*host.shape[:2], 64, dh // 64, 2)
        side[int(c.table[0, 7]), :, 2, :, 0], side[int(c.table[0, 7]), :, 2, :, 1] = 0.0, -30.0
        c.k.copy_(host)
        q[0, ::2] = 1.25
        q[0, ::2, ::3] = 0.5
    out, err = _decode(bd, q.cuda(), c, torch.tensor([n - 1], dtype=torch.int32, device="cuda"))
    assert err == 0
    _check_decode(out, q, c, [n])


@pytest.mark.gpu
def test_decode_rising_scores(bd):
    """Keys that grow along the sequence: the running maximum moves in every unit."""
    lens = [4096]
    c = Cache(2, 64, 64, lens, 4).fill(lens, 4)
    host = c.k.cpu()
    P, H, _ = host.shape
    side = host[:, :, 64 * 32:].view(torch.bfloat16).view(P, H, 64, 2)
    s = np.arange(4096)
    at, off = torch.from_numpy(c.table[0, s // 64]).long(), torch.from_numpy(s % 64)
    low = (torch.from_numpy(s).float() * 0.01).to(torch.bfloat16)
    side[at, :, off, 1] = low[:, None].expand(-1, H)
    c.k.copy_(host)
    q = torch.full((1, 8, 64), 0.5).to(torch.bfloat16)
    out, err = _decode(bd, q.cuda(), c, torch.tensor([4095], dtype=torch.int32, device="cuda"))
    assert err == 0
    _check_decode(out, q, c, lens)


@pytest.mark.gpu
def test_decode_length_past_the_table(bd):
    """A length that the page table does not reach counts as its last slot; negative ones give zeros."""
    c = Cache(4, 64, 16, [48, 48, 48], 2).fill([48] * 3, 2)
    c.dtable = c.dtable[:, :3].contiguous()
    q = torch.randn(3, 8, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    out, err = _decode(bd, q.cuda(), c, torch.tensor([2 ** 31 - 1, -2 ** 31, 48], dtype=torch.int32, device="cuda"))
    assert err == 0
    _check_decode(out, q, c, [48, 0, 48])


@pytest.mark.gpu
def test_decode_bad_page_and_nan_stay_in_their_sequence(bd):
    heads, lens = (8, 4, 64), [100, 70, 50]
    c = Cache(4, 64, 16, lens, 6).fill(lens, 6)
    q = torch.randn(3, 8, 64, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
    len0 = torch.tensor([n - 1 for n in lens], dtype=torch.int32, device="cuda")
    good, err = _decode(bd, q.cuda(), c, len0)
    assert err == 0
    keep = int(c.dtable[1, 2])
    for bad in (-1, c.k.shape[0], 2 ** 31 - 1):
        c.dtable[1, 2] = bad
        out, err = _decode(bd, q.cuda(), c, len0)
        assert err == 4
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    c.dtable[1, 2] = keep
    # a key (scale, minimum) of NaN in kv head 2 of sequence 0, slot 40
    side = c.k[:, :, 16 * 32:].view(torch.bfloat16)
    side[int(c.table[0, 2]), 2, 8 * 2:8 * 2 + 2] = float("nan")
    out, err = _decode(bd, q.cuda(), c, len0)
    assert err == 0
    o = out.view(3, 8, 64)
    assert torch.isnan(o[0, 4:6]).all()
    g = good.view(3, 8, 64)
    assert torch.equal(o[0, :4], g[0, :4]) and torch.equal(o[0, 6:], g[0, 6:]) and torch.equal(o[1:], g[1:])


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [(8, 4, 64), (16, 4, 128), (8, 1, 128)], ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_decode_bad_query_stays_in_its_head(bd, heads, bad):
    """A query value of NaN or infinity makes that head NaN, and no other."""
    Hq, Hkv, dh = heads
    lens = [900, 20, 64]
    c = Cache(Hkv, dh, 32, lens, 11).fill(lens, 11)
    q = torch.randn(3, Hq, dh, generator=torch.Generator().manual_seed(11)).to(torch.bfloat16)
    q[0, 1, 5] = bad
    q[2, Hq - 1] = bad
    out, err = _decode(bd, q.cuda(), c, torch.tensor([n - 1 for n in lens], dtype=torch.int32, device="cuda"))
    assert err == 0
    o = out.view(3, Hq, dh).cpu()
    assert torch.isnan(o[0, 1]).all() and torch.isnan(o[2, Hq - 1]).all()
    q[0, 1, 5] = 0
    q[2, Hq - 1] = 0
    ref, tol = _ref_decode(q, c, lens)
    good = np.ones((3, Hq), dtype=bool)
    good[0, 1] = good[2, Hq - 1] = False
    assert np.all((np.abs(o.double().numpy() - ref) <= tol)[good])


@pytest.mark.gpu
@pytest.mark.parametrize("slot", [3, 500, 899])
def test_decode_bad_value_stays_in_its_dims(bd, slot):
    """A NaN pair of V makes its 64 dims of its kv head NaN."""
    lens = [900]
    c = Cache(2, 128, 64, lens, 12).fill(lens, 12)
    q = torch.randn(1, 8, 128, generator=torch.Generator().manual_seed(12)).to(torch.bfloat16)
    ref, tol = _ref_decode(q, c, lens)
    side = c.v[:, :, 64 * 64:].view(torch.bfloat16)
    side[int(c.table[0, slot // 64]), 1, (slot % 64) * 4 + 2:(slot % 64) * 4 + 4] = float("nan")
    out, err = _decode(bd, q.cuda(), c, torch.tensor([899], dtype=torch.int32, device="cuda"))
    assert err == 0
    o = out.view(1, 8, 128).cpu().double().numpy()
    assert np.isnan(o[0, 4:, 64:]).all()
    near = np.abs(o - ref) <= tol
    assert near[0, :4].all() and near[0, 4:, :64].all()


@pytest.mark.gpu
def test_steps_in_a_graph(bd):
    """A decode step (append and attention of every sequence) captured once and replayed as the lengths grow over the ends of units
    and pages, against the same calls made one by one on a second cache; each capture has its workspace."""
    heads, page, S, steps = (16, 8, 128), 16, 3, 9
    Hq, Hkv, dh = heads
    lens = [60, 127, 1]
    first = Cache(Hkv, dh, page, [n + steps for n in lens], 13).fill(lens, 13)
    pages = [(first.k, first.v), (first.k.clone(), first.v.clone())]
    cs = torch.empty(300, dh, dtype=torch.bfloat16, device="cuda")
    bd.op_rope_table(1e6, dh, 300, cs)
    gen = torch.Generator().manual_seed(13)
    cu = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    size = bd.attention_decode_paged4_workspace(S, Hq, Hkv, dh)
    qkv = torch.empty(S, (Hq + 2 * Hkv) * dh, dtype=torch.bfloat16, device="cuda")
    at = torch.empty(S, dtype=torch.int32, device="cuda")
    bufs = [(torch.empty(S, Hq, dh, dtype=torch.bfloat16, device="cuda"), torch.empty(size, dtype=torch.uint8, device="cuda"),
             torch.empty(S, Hq * dh, dtype=torch.bfloat16, device="cuda")) for _ in range(2)]

    def step(i):
        (kp, vp), (q, work, out) = pages[i], bufs[i]
        bd.op_append_paged4(qkv, cu, at, cs, kp, vp, first.dtable, q)
        bd.op_attention_decode_paged4(q, kp, vp, first.dtable, at, work, out)

    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        step(0)
    for i in range(steps):
        qkv.copy_(torch.randn(qkv.shape, generator=gen).to(torch.bfloat16))
        at.copy_(torch.tensor([n + i for n in lens], dtype=torch.int32))
        graph.replay()
        step(1)
        torch.cuda.synchronize()
        assert torch.equal(bufs[0][0], bufs[1][0]) and torch.equal(bufs[0][2], bufs[1][2])
    assert torch.equal(pages[0][0], pages[1][0]) and torch.equal(pages[0][1], pages[1][1])
    _check_decode(bufs[0][2], bufs[0][0].cpu(), first, [n + steps for n in lens])


@pytest.mark.gpu
def test_decode_repeats_streams_and_graph(bd):
    """Bit-equal results from repeated calls with any workspace contents, on two streams at once, from a replayed graph; and the
    graph follows lengths that change."""
    lens = [3000, 1, 513, 90] * 3
    c = Cache(8, 128, 16, lens, 8).fill(lens, 8)
    q = torch.randn(12, 16, 128, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    len0 = torch.tensor([n - 1 for n in lens], dtype=torch.int32, device="cuda")
    base, _ = _decode(bd, q, c, len0)
    size = bd.attention_decode_paged4_workspace(12, 16, 8, 128)
    for fill in (0, 255, 127):
        out, _ = _decode(bd, q, c, len0, work=torch.full((size,), fill, dtype=torch.uint8, device="cuda"))
        assert torch.equal(out, base)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    works = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in streams]
    outs = [torch.zeros_like(base) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, w, o in zip(streams, works, outs):
            bd.op_attention_decode_paged4(q, c.k, c.v, c.dtable, len0, w, o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, base) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        bd.op_attention_decode_paged4(q, c.k, c.v, c.dtable, len0, works[0], outs[0])
    outs[0].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], base)
    len0 -= 1
    graph.replay()
    torch.cuda.synchronize()
    want, _ = _decode(bd, q, c, len0)
    assert torch.equal(outs[0], want)


@pytest.mark.gpu
def test_pool_past_32_bits(bd):
    """A pool of 4.4 GB a tensor whose last pages are in use: appended, read back and attended to."""
    heads, page = (16, 8, 128), 256
    n_pages, size = 30000, 256 * 72
    k = torch.empty(n_pages, 8, size, dtype=torch.uint8, device="cuda")
    v = torch.empty_like(k)
    assert k.numel() > 2 ** 32
    lens, start = [300, 1], [0, 40]
    small = Cache(8, 128, page, [300, 41], 3)
    _append(bd, heads, page, [300, 41], [0, 0], seed=4, cache=small)
    far = small.table.copy()
    used = np.unique(far[far < 2 ** 30])
    for i, p in enumerate(used):
        far[small.table == p] = n_pages - 1 - i
        k[n_pages - 1 - i] = small.k[p]
        v[n_pages - 1 - i] = small.v[p]
    big = Cache(8, 128, page, [1, 1], 3)
    big.k, big.v, big.table, big.dtable = k, v, far, torch.from_numpy(far).cuda()
    qkv = torch.randn(301, 32 * 128, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    cs = _table(128, 300).cuda()
    res = []
    for c in (small, big):
        q, kr = torch.zeros(301, 16, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(301, 8, 128, dtype=torch.bfloat16, device="cuda")
        vr, err = torch.zeros_like(kr), torch.zeros(1, dtype=torch.int32, device="cuda")
        cu, st = _cu(lens), torch.tensor(start, dtype=torch.int32, device="cuda")
        bd.op_append_paged4(qkv, cu, st, cs, c.k, c.v, c.dtable, q, err=err)
        bd.op_read_paged4(c.k, c.v, c.dtable, cu, st, kr, vr, err=err)
        out, e = _decode(bd, q[-2:].contiguous(), c, torch.tensor([299, 40], dtype=torch.int32, device="cuda"))
        assert e == 0 and int(err.item()) == 0
        res.append((q, kr, vr, out))
    assert all(torch.equal(a, b) for a, b in zip(*res))
    assert torch.isfinite(res[0][3].float()).all() and torch.any(res[0][1] != 0)


@pytest.mark.gpu
@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("heads", [(8, 1, 128), (16, 2, 128), (8, 8, 64), (16, 2, 64), (10, 5, 64), (9, 3, 128)], ids=str)
def test_read_forms(bd, heads, page):
    """The rows that a warp takes at once, for kv heads on both sides of each form."""
    _, Hkv, dh = heads
    lens, start = [3, 0, 130, 70], [page - 1, 9, 0, 2 * page + 5]
    ends = [a + n for a, n in zip(start, lens)]
    c = Cache(Hkv, dh, page, ends, page).fill(ends, page)
    n = sum(lens)
    k = torch.full((n + 3, Hkv, dh), 7.0, dtype=torch.bfloat16, device="cuda")
    v, err = k.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    bd.op_read_paged4(c.k, c.v, c.dtable, _cu(lens), torch.tensor(start, dtype=torch.int32, device="cuda"), k, v, err=err)
    assert int(err.item()) == 0
    seq, pos = np.repeat(np.arange(len(lens)), lens), _positions(lens, start)
    for got, pages in ((k, c.k), (v, c.v)):
        val = _values(pages.cpu(), page, dh)[c.table[seq, pos // page], :, pos % page]
        # the sum is rounded to fp32 (2^-24 of it), then to bf16
        assert np.all(np.abs(got[:n].cpu().double().numpy() - val) <= 2.0 ** -8 * np.abs(val) * (1 + 2.0 ** -14))
        assert torch.all(got[n:] == 7.0)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("heads,lens", [((5, 1, 128), [9000, 100]), ((12, 2, 64), [3000, 0, 700]), ((7, 1, 64), [20000]),
                                        ((7, 1, 128), [5000, 1, 2000]), ((40, 8, 128), [2100, 65, 900]),
                                        ((24, 4, 128), [64, 65, 63, 800])], ids=str)
def test_decode_odd_groups(bd, heads, lens, page):
    """Groups of five to seven query heads, with sequences that are cut between warps and between CTAs."""
    Hq, Hkv, dh = heads
    c = Cache(Hkv, dh, page, lens, page).fill(lens, page)
    q = torch.randn(len(lens), Hq, dh, generator=torch.Generator().manual_seed(page)).to(torch.bfloat16)
    out, err = _decode(bd, q.cuda(), c, torch.tensor([n - 1 for n in lens], dtype=torch.int32, device="cuda"))
    assert err == 0
    _check_decode(out, q, c, lens)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,lens,page", [((8, 1, 128), [20011], 64), ((4, 2, 64), [9000, 1, 4000], 16),
                                             ((12, 4, 128), [2500, 2500], 32), ((7, 1, 64), [30000], 128)], ids=str)
def test_decode_counts_every_unit_once(bd, heads, lens, page):
    """One key in every 64 has nearly all of the weight, and a value in a dim of its own (which up to eight share): a unit
    that is left out, or taken twice, changes that dim by an eighth of it at least, against a bound of about a hundredth."""
    Hq, Hkv, dh = heads
    c = Cache(Hkv, dh, page, lens, page)
    for pages, is_k in ((c.k, True), (c.v, False)):
        host = pages.cpu()
        codes = host[:, :, :page * dh // 2].view(*host.shape[:2], page, dh // 2)
        side = host[:, :, page * dh // 2:].view(torch.bfloat16).view(*host.shape[:2], page, dh // 64, 2)
        for b, n in enumerate(lens):
            s = np.arange(n)
            unit = s // 64
            # (the last unit's key is its first one)
            marked = s == unit * 64 + np.where((unit + 1) * 64 <= n, unit * 29 % 64, 0)
            at, off = torch.from_numpy(c.table[b, s // page]).long(), torch.from_numpy(s % page)
            m = torch.from_numpy(marked)
            row = torch.zeros(n, dh // 2, dtype=torch.uint8)
            if is_k:  # scores of 2 sqrt(dh) and the negative of it, 32 and more apart
                pair = torch.where(m, 2.0, -2.0).to(torch.bfloat16)
                side[at, :, off] = torch.stack([torch.zeros_like(pair), pair], -1)[:, None, None].expand(n, host.shape[1], dh // 64, 2)
            else:
                dim = unit[marked] % dh
                row[np.nonzero(marked)[0], dim // 2] = torch.from_numpy(np.where(dim % 2, 0xf0, 0x0f).astype(np.uint8))
                side[at, :, off] = torch.tensor([1.0, 0.0], dtype=torch.bfloat16).expand(n, host.shape[1], dh // 64, 2)
            codes[at, :, off] = row[:, None].expand(n, host.shape[1], dh // 2)
        pages.copy_(host)
    q = torch.ones(len(lens), Hq, dh, dtype=torch.bfloat16)
    out, err = _decode(bd, q.cuda(), c, torch.tensor([n - 1 for n in lens], dtype=torch.int32, device="cuda"))
    assert err == 0
    _check_decode(out, q, c, lens)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,page", [((16, 8, 128), 16), ((8, 4, 64), 64), ((40, 8, 128), 32)], ids=str)
def test_appended_tokens_are_attended_to(bd, heads, page):
    """Prompts, then single tokens: after every append the attention of all sequences, the new key among those it sees, against
    float64 on the cache's own bytes. The new key is the query itself times 8 in every other sequence, so that it has most of the weight."""
    Hq, Hkv, dh = heads
    lens, steps = [37, 5, 150, 64], 4
    ends = [n + steps for n in lens]
    c = Cache(Hkv, dh, page, ends, 17)
    _append(bd, heads, page, lens, [0] * 4, seed=17, cache=c)
    gen = torch.Generator().manual_seed(18)
    for i in range(steps):
        at = [n + i for n in lens]
        qkv = torch.randn(4, (Hq + 2 * Hkv) * dh, generator=gen)
        x = qkv.view(4, Hq + 2 * Hkv, dh)
        x[::2, Hq:Hq + Hkv] = 8 * x[::2, :Hq:Hq // Hkv]
        r = _append(bd, heads, page, [1] * 4, at, norm=False, qkv=qkv.to(torch.bfloat16), cache=c)
        assert r["err"] == 0
        out, err = _decode(bd, r["q"].cuda(), c, torch.tensor(at, dtype=torch.int32, device="cuda"))
        assert err == 0
        _check_decode(out, r["q"], c, [n + 1 for n in at])


# ------------------------------------------------------------------------------------------------------------ refusals

def test_page_bytes(bd):
    for page in PAGES:
        assert bd.paged4_page_bytes(page, 128) == page * 72 and bd.paged4_page_bytes(page, 64) == page * 36
    for page, dh in ((0, 128), (8, 128), (24, 128), (512, 128), (64, 96), (-16, 64), (2 ** 40, 128)):
        assert bd.paged4_page_bytes(page, dh) == 0


def test_library_refuses(bd):
    """Argument checks on the host: nothing is launched (the addresses are never dereferenced)."""
    L, p = bd.lib(), 4096

    def append(**c):
        a = dict(qkv=p, ld=1024, N=3, cu=p, start=p, S=1, Hq=8, Hkv=4, dh=64, qg=p, kg=p, cs=p, n_pos=10, q=p, k=p, kp=p, vp=p,
                 n_pages=4, page=16, table=p, max_pages=2)
        a.update(c)
        return L.qwen3_op_append_paged4(a["qkv"], a["ld"], a["N"], a["cu"], a["start"], a["S"], a["Hq"], a["Hkv"], a["dh"], a["qg"],
                                        a["kg"], 1e-6, a["cs"], a["n_pos"], a["q"], a["k"], a["kp"], a["vp"], a["n_pages"],
                                        a["page"], a["table"], a["max_pages"], None, None)

    for c in (dict(qkv=None), dict(ld=1023), dict(ld=1016), dict(ld=1028), dict(N=-1), dict(N=2 ** 30 + 1), dict(cu=None),
              dict(start=None), dict(S=-1), dict(Hq=0), dict(Hq=7), dict(Hkv=0), dict(dh=96), dict(cs=None), dict(n_pos=0),
              dict(q=None), dict(kp=None), dict(vp=None), dict(n_pages=0), dict(page=8), dict(page=48), dict(page=512),
              dict(table=None), dict(max_pages=0), dict(qkv=p + 2), dict(q=p + 8), dict(k=p + 8), dict(kp=p + 8), dict(vp=p + 1),
              dict(cs=p + 2), dict(qg=p + 2), dict(kg=p + 2), dict(Hq=65536 * 4)):
        assert append(**c) == 5, c
    assert append(N=0) == 0 and append(S=0) == 0

    def read(**c):
        a = dict(kp=p, vp=p, n_pages=4, page=16, table=p, max_pages=2, cu=p, start=p, S=1, N=3, Hkv=4, dh=64, k=p, v=p)
        a.update(c)
        return L.qwen3_op_read_paged4(*[a[n] for n in ("kp", "vp", "n_pages", "page", "table", "max_pages", "cu", "start", "S", "N",
                                                       "Hkv", "dh", "k", "v")], None, None)

    for c in (dict(kp=None), dict(vp=None), dict(kp=p + 8), dict(n_pages=0), dict(page=20), dict(table=None), dict(max_pages=0),
              dict(cu=None), dict(start=None), dict(S=-1), dict(N=-1), dict(Hkv=0), dict(dh=32), dict(k=None), dict(v=None),
              dict(k=p + 2), dict(v=p + 8)):
        assert read(**c) == 5, c
    assert read(N=0) == 0 and read(S=0) == 0

    size = 1 << 30

    def decode(**c):
        a = dict(q=p, kp=p, vp=p, n_pages=4, page=16, table=p, max_pages=2, len0=p, B=2, Hq=8, Hkv=4, dh=64, work=p, bytes=size,
                 out=p)
        a.update(c)
        return L.qwen3_op_attention_decode_paged4(*[a[n] for n in ("q", "kp", "vp", "n_pages", "page", "table", "max_pages", "len0",
                                                                   "B", "Hq", "Hkv", "dh", "work", "bytes", "out")], None, None)

    for c in (dict(q=None), dict(kp=None), dict(vp=None), dict(n_pages=0), dict(page=17), dict(table=None), dict(max_pages=0),
              dict(len0=None), dict(B=-1), dict(B=65536), dict(Hq=9), dict(Hq=36), dict(Hkv=0), dict(dh=80), dict(work=None),
              dict(out=None), dict(q=p + 8), dict(out=p + 2), dict(work=p + 4), dict(bytes=0), dict(bytes=1000),
              dict(B=65535, max_pages=2 ** 26)):
        assert decode(**c) == 5, c
    assert decode(B=0) == 0
    assert bd.attention_decode_paged4_workspace(0, 8, 4, 64) == 0
    assert bd.attention_decode_paged4_workspace(1, 36, 4, 64) == 0


APPEND_ARGS, READ_ARGS, DECODE_ARGS, PACKED_ARGS = (struct.Struct(f) for f in (
    "PqiPPiiiiPPfPiPPPPiiPiP", "PPiiPiPPiiiiPPP", "PPPiiPiPiiiiPNPP", "PqPqPqiiiiiPNiPP"))  # the header's argument blocks


def test_argument_blocks(bd):
    """Argument blocks: every field, wrong by itself, is refused as in the direct call, and the right ones are taken (a call
    without rows does nothing)."""
    L, p, size = bd.lib(), 4096, 1 << 30
    # (the row count, field `rows`, stays 0: nothing is launched)
    forms = ((L.qwen3_op_append_paged4_block, APPEND_ARGS, L.qwen3_op_append_paged4, 2,
              [p, 1024, 0, p, p, 1, 8, 4, 64, p, p, 1e-6, p, 10, p, p, p, p, 4, 16, p, 2, 0]),
             (L.qwen3_op_read_paged4_block, READ_ARGS, L.qwen3_op_read_paged4, 9,
              [p, p, 4, 16, p, 2, p, p, 1, 0, 4, 64, p, p, 0]),
             (L.qwen3_op_attention_decode_paged4_block, DECODE_ARGS, L.qwen3_op_attention_decode_paged4, 8,
              [p, p, p, 4, 16, p, 2, p, 0, 8, 4, 64, p, size, p, 0]),
             (L.qwen3_op_attention_prefill_packed_block, PACKED_ARGS, L.qwen3_op_attention_prefill_packed, 6,
              [p, 512, p, 256, p, 256, 0, 100, 8, 4, 64, p, 1 << 20, 100, p, 0]))
    for block, layout, direct, rows, args in forms:
        assert args[rows] == 0
        assert block(layout.pack(*args), None) == 0 and direct(*args, None) == 0
        assert block(None, None) == 5
        refused = 0
        for i in range(len(args)):
            for bad in (0, -1, 7, p + 2):
                wrong = list(args)
                wrong[i] = bad
                if i == rows:
                    continue
                try:
                    packed = layout.pack(*wrong)
                except (OverflowError, struct.error):  # no such pointer or size
                    continue
                want = direct(*wrong, None)
                assert want in (0, 5) and block(packed, None) == want, (block.__name__, i, bad)
                refused += want == 5
        assert refused > len(args)


def _fields(layout, got):
    return layout.unpack(got.ljust(layout.size, b"\0"))


@pytest.mark.parametrize("one", [False, True])
def test_packed_blocks(bd, one):
    """The binding's blocks hold the fields of the header's, from tensors of any of the allowed strides; no rows, no block."""
    bf, i32, u8, c = torch.bfloat16, torch.int32, torch.uint8, bd._checks()
    N = 1 if one else 6
    z = lambda *shape, dtype=bf: torch.zeros(shape, dtype=dtype)  # noqa: E731
    kp, vp, table = z(5, 4, 16 * 72, dtype=u8), z(5, 4, 16 * 72, dtype=u8), z(2, 3, dtype=i32)
    cu, start, err, work = z(3, dtype=i32), z(2, dtype=i32), z(1, dtype=i32), z(333, dtype=torch.float64)
    qkv, cs, q, k, v, g = z(N, 2100)[:, :2048], z(9, 128), z(N, 8, 128), z(N, 4, 128), z(N, 4, 128), z(128)
    at = lambda *ts: [0 if t is None else t.data_ptr() for t in ts]  # noqa: E731
    for k_out, gq, e in ((k, g, None), (None, None, err)):
        got = _fields(APPEND_ARGS, c.append_paged4(qkv, cu, start, cs, kp, vp, table, q, k_out, gq, g, 0.25, e))
        want = at(qkv) + [2048 if one else 2100, N] + at(cu, start) + [2, 8, 4, 128] + at(gq, g) + [0.25] + at(cs) + [9] + \
            at(q, k_out, kp, vp) + [5, 16] + at(table) + [3] + at(e)
        assert list(got) == want
        got = _fields(READ_ARGS, c.read_paged4(kp, vp, table, cu, start, k, v, e))
        assert list(got) == at(kp, vp) + [5, 16] + at(table) + [3] + at(cu, start) + [2, N, 4, 128] + at(k, v, e)
        B = z(2, 8, 128)
        got = _fields(DECODE_ARGS, c.attention_decode_paged4(B, kp, vp, table, start, work, z(2, 1024), e))
        assert list(got)[:-2] == at(B, kp, vp) + [5, 16] + at(table) + [3] + at(start) + [2, 8, 4, 128] + at(work) + [2664]
        heads = qkv.as_strided((N, 4, 128), (2100, 128, 1), 1024)
        out = z(N, 1024)
        got = _fields(PACKED_ARGS, c.attention_prefill_packed(q, heads, v, work, 77, out, e))
        assert list(got) == at(q) + [1024] + at(heads) + [512 if one else 2100] + at(v) + [512, N, N, 8, 4, 128] + at(work) + \
            [2664, 77] + at(out, e)
    assert c.append_paged4(qkv[:0], cu, start, cs, kp, vp, table, q[:0], None, None, None, 0.25, None) == b""
    assert c.read_paged4(kp, vp, table, cu, start, k[:0], v[:0], None) == b""
    assert c.attention_decode_paged4(B[:0], kp, vp, table[:0], start[:0], work, z(0, 1024), None) == b""
    assert c.attention_prefill_packed(q[:0], k, v, work, 77, z(0, 1024), None) == b""
    for bad in (None, 3, "q", [q], q.to_sparse()):
        assert c.read_paged4(kp, vp, table, cu, start, bad, v, None) is None
        assert c.attention_prefill_packed(q, k, v, bad, 77, out, None) is None
    with pytest.raises(TypeError):
        c.read_paged4(kp, vp)
    with pytest.raises(TypeError):
        c.append_paged4(qkv, cu, start, cs, kp, vp, table, q, None, None, None, "eps", None)
    with pytest.raises(TypeError):
        c.attention_prefill_packed(q, k, v, work, None, out, None)


def test_binding_refuses(bd):
    bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
    kp, vp = torch.zeros(5, 4, 16 * 36, dtype=u8), torch.zeros(5, 4, 16 * 36, dtype=u8)
    table, cu, start = torch.zeros(2, 3, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32)
    base = dict(qkv=torch.zeros(6, 1024, dtype=bf), cu=cu, start=start, cos_sin=torch.zeros(9, 64, dtype=bf), k_pages=kp,
                v_pages=vp, page_table=table, q_out=torch.zeros(6, 8, 64, dtype=bf), k_out=torch.zeros(6, 4, 64, dtype=bf),
                q_gamma=torch.zeros(64, dtype=bf), k_gamma=torch.zeros(64, dtype=bf))
    pages = (dict(k_pages=kp[0]), dict(k_pages=kp.float()), dict(v_pages=vp[:4]), dict(k_pages=kp[:, :, :-1], v_pages=vp[:, :, :-1]),
             dict(page_table=table[0]), dict(page_table=table.long()), dict(page_table=table[:, :0]), dict(v_pages=None))
    for change in pages + (dict(qkv=base["qkv"].float()), dict(qkv=base["qkv"][:5]), dict(qkv=base["qkv"][:, :1000]),
                           dict(qkv=torch.zeros(1024, 6, dtype=bf).t()), dict(cu=cu[:2]), dict(cu=cu.long()),
                           dict(start=torch.zeros(3, dtype=i32)), dict(cos_sin=torch.zeros(9, 32, dtype=bf)),
                           dict(q_out=base["q_out"].float()), dict(q_out=base["q_out"][:, :7]), dict(k_out=base["k_out"][:5]),
                           dict(q_gamma=torch.zeros(32, dtype=bf)), dict(k_gamma=torch.zeros(64)), dict(err=torch.zeros(1)), {}):
        with pytest.raises(ValueError):
            bd.op_append_paged4(**{**base, **change})
    base = dict(k_pages=kp, v_pages=vp, page_table=table, cu=cu, start=start, k_out=torch.zeros(6, 4, 64, dtype=bf),
                v_out=torch.zeros(6, 4, 64, dtype=bf))
    for change in pages + (dict(k_out=base["k_out"][:, :3]), dict(v_out=base["v_out"][:5]), dict(k_out=base["k_out"].float()),
                           dict(cu=cu[:1]), {}):
        with pytest.raises(ValueError):
            bd.op_read_paged4(**{**base, **change})
    base = dict(q=torch.zeros(2, 8, 64, dtype=bf), k_pages=kp, v_pages=vp, page_table=table, len0=start,
                work=torch.zeros(10, dtype=u8), out=torch.zeros(2, 512, dtype=bf))
    for change in pages + (dict(q=base["q"][0]), dict(q=base["q"].float()), dict(q=torch.zeros(2, 36, 64, dtype=bf)),
                           dict(q=torch.zeros(3, 8, 64, dtype=bf)), dict(len0=cu), dict(len0=start.long()), dict(work=None),
                           dict(out=base["out"][:1]), dict(out=base["out"].float()), {}):
        with pytest.raises(ValueError):
            bd.op_attention_decode_paged4(**{**base, **change})
