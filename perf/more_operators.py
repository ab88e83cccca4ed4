"""Cases for the operators of a paged cache held in 4 bits and of packed prompts, each in plain torch and through the library:
appending keys and values (with head norms and rotation), reading them back, decode attention over the pages, and causal
attention over packed sequences of different lengths.

A page holds `page` tokens of one kv head in 4 bits: the codes [page, dh / 2] (two a byte, the lower nibble first), then for each
token and 64 dims a scale and a minimum in bf16: value = min + scale * code. A case is one call as a serving loop makes it.
"""
import random

import torch

own = False

# (query heads, kv heads, head_dim): the tiny, 0.6B and 8B stacks of this repository, and groups of 1, 3 and 8 query heads
HEADS = [(8, 4, 64), (16, 8, 128), (32, 8, 128), (8, 8, 64), (12, 4, 128), (16, 2, 128)]
POSITIONS = 40960
EPS = 1e-6
GROUP = 64


def listed():
    return [
        # ---- append: head norms, rotation and 4-bit pages; the cached values are read back
        # one sequence's decode step: latency
        dict(name="append 1 token 8b", op="append", heads=2, page=16, seqs=1, tokens=1, start=5000, pad=0, norm=True),
        # a decode batch of 64, padded to 72 rows
        dict(name="append 64 tokens 0.6b", op="append", heads=1, page=64, seqs=64, tokens=64, start=4096, pad=8, norm=True),
        # nine prompts of different lengths, 32,768 tokens in all
        dict(name="append 32768 prompt tokens 8b", op="append", heads=2, page=64, seqs=9, tokens=32768, start=0, pad=0,
             norm=True),
        # ---- read: slots of the cache as bf16 rows
        # the end of one sequence, to look at or to go on from
        dict(name="read 200 of 1 sequence 0.6b", op="read", heads=1, page=16, seqs=1, tokens=200, start=700),
        # the histories of 16 chats, before their next prompts
        dict(name="read 16 histories 8b", op="read", heads=2, page=64, seqs=16, tokens=100000, start=0),
        # ---- decode attention over the pages
        # one sequence: latency
        dict(name="decode 1 @ 4096 8b", op="decode", heads=2, page=16, seqs=1, longest=4096),
        # many short answers of a small model
        dict(name="decode 200 @ 300 tiny", op="decode", heads=0, page=32, seqs=200, longest=300),
        # the 0.6B batch of 64
        dict(name="decode 64 @ 4096 0.6b", op="decode", heads=1, page=16, seqs=64, longest=4096),
        # the 8B long-context batch
        dict(name="decode 16 @ 32768 8b", op="decode", heads=2, page=64, seqs=16, longest=32768),
        # ---- packed causal attention
        # a few short prompts
        dict(name="packed 6 prompts 0.6b", op="packed", heads=1, seqs=6, tokens=1500, history=0),
        # the next turns of 16 chats over their histories
        dict(name="packed 16 turns over histories 8b", op="packed", heads=2, seqs=16, tokens=5000, history=4096),
        # three long prompts
        dict(name="packed 3 long prompts 8b", op="packed", heads=2, seqs=3, tokens=17000, history=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["append", "read", "decode", "packed"])
    heads, page = rng.randrange(len(HEADS)), rng.choice([16, 32, 64, 128, 256])
    if op == "append":
        seqs = _log_int(rng, 1, 128)
        tokens = seqs if rng.random() < 0.4 else _log_int(rng, 1, 32768)
        return dict(op=op, heads=heads, page=page, seqs=seqs, tokens=tokens, start=rng.choice([0, _log_int(rng, 1, 4096)]),
                    pad=rng.choice([0, rng.randint(1, 40)]), norm=rng.random() < 0.7)
    if op == "read":
        return dict(op=op, heads=heads, page=page, seqs=_log_int(rng, 1, 64), tokens=_log_int(rng, 1, 65536),
                    start=rng.choice([0, _log_int(rng, 1, 4096)]))
    if op == "decode":
        seqs = _log_int(rng, 1, 256)
        return dict(op=op, heads=heads, page=page, seqs=seqs, longest=_log_int(rng, 1, min(32768, 524288 // seqs)))
    seqs = _log_int(rng, 1, 32)
    return dict(op=op, heads=heads, seqs=seqs, tokens=_log_int(rng, 1, 8192), history=rng.choice([0, 0, _log_int(rng, 1, 2048)]))


# ------------------------------------------------------------------------------------------------ geometry of a case

def _lengths(total, n):
    """total spread unevenly over n sequences; some are empty when it is small."""
    w = [1 + (i * 7919 + 13) % 29 for i in range(n)]
    ends = [0]
    for i in range(n):
        ends.append(ends[-1] + w[i])
    cut = [total * e // ends[-1] for e in ends]
    return [b - a for a, b in zip(cut, cut[1:])]


def _spread(longest, n):
    """Lengths of n sequences up to the longest, the first one of it."""
    return [longest - (i * 613) % (longest // 2 + 1) for i in range(n)]


def _slots(case):
    """(first slot, slots) of each sequence that the call appends, reads or attends to."""
    if case["op"] == "decode":
        return [(0, n) for n in _spread(case["longest"], case["seqs"])]
    lens = _lengths(case["tokens"], case["seqs"])
    if case["op"] == "append" and case["tokens"] == case["seqs"]:
        lens = [1] * case["seqs"]
    return list(zip(_spread(case["start"], case["seqs"]), lens))


def _histories(case):
    return _spread(case["history"], case["seqs"]) if case["history"] else [0] * case["seqs"]


def _kv_bytes(dh):
    return dh // 2 + dh // GROUP * 4


def work(case):
    hq, hkv, dh = HEADS[case["heads"]]
    if case["op"] == "packed":
        pairs = keys = 0
        for n, h in zip(_lengths(case["tokens"], case["seqs"]), _histories(case)):
            pairs += n * h + n * (n + 1) // 2
            keys += n + h if n else 0
        return {"bytes": 4 * dh * (case["tokens"] * hq + keys * hkv), "flops": 4 * dh * hq * pairs}
    n = sum(k for _, k in _slots(case))
    if case["op"] == "append":  # the cached values count once, as they are returned
        return {"bytes": n * dh * 2 * ((hq + 2 * hkv) + (hq + hkv) + 2 * hkv), "flops": n * dh * (8 * (hq + hkv) + 8 * 2 * hkv)}
    if case["op"] == "read":
        return {"bytes": 2 * n * hkv * (_kv_bytes(dh) + 2 * dh), "flops": 4 * n * hkv * dh}
    return {"bytes": 2 * n * hkv * _kv_bytes(dh) + 4 * case["seqs"] * hq * dh, "flops": 4 * n * hq * dh}


# --------------------------------------------------------------------------------------------- pages in plain torch

def _down(x):
    """fp32 to the nearest bf16 value not above it (as fp32)."""
    bits = x.contiguous().view(torch.int32)
    cut = bits & -65536
    return torch.where((bits < 0) & (cut != bits), cut + 65536, cut).view(torch.float32)


def _quantize(x):
    """x [.., dh] fp32 -> codes [.., dh] (0..15) and scale, min [.., dh / 64], as the cache defines them."""
    g = x.unflatten(-1, (-1, GROUP))
    low = _down(g.amin(dim=-1))
    scale = -_down(-((g.amax(dim=-1) - low) / torch.full_like(low, 15)))  # (a division, not a product with 1 / 15)
    codes = ((g - low[..., None]) / torch.where(scale > 0, scale, 1)[..., None]).round_().clamp_(0, 15)
    return codes.flatten(-2), scale, low


def _parts(pages, page, dh):
    """Views of the pages' codes [P, Hkv, page, dh / 2] and scales and minima [P, Hkv, page, dh / 64, 2] (bf16)."""
    p, h, _ = pages.shape
    codes = pages[:, :, :page * dh // 2].view(p, h, page, dh // 2)
    side = pages.view(torch.bfloat16)[:, :, page * dh // 4:].view(p, h, page, dh // GROUP, 2)
    return codes, side


def _store(pages, page, dh, at, off, x):
    """Put x [n, Hkv, dh] into rows `off` of pages `at`."""
    codes, scale, low = _quantize(x)
    c = codes.to(torch.uint8)
    cv, sv = _parts(pages, page, dh)
    cv[at, :, off] = c[..., 0::2] | (c[..., 1::2] << 4)
    sv[at, :, off] = torch.stack([scale, low], dim=-1).to(torch.bfloat16)


def _load(pages, page, dh, at, off):
    """The values [n, Hkv, dh] of rows `off` of pages `at`, in fp32."""
    cv, sv = _parts(pages, page, dh)
    c = cv[at, :, off]
    c = torch.stack([c & 15, c >> 4], dim=-1).flatten(-2).float()
    s = sv[at, :, off].float()
    v = c.unflatten(-1, (-1, GROUP)) * s[..., 0:1] + s[..., 1:2]
    return v.flatten(-2)


# ------------------------------------------------------------------------------------------------------------ inputs

def _rope_table(dh):
    """[POSITIONS, dh] bf16: cos and sin of the dh / 2 pair angles, theta 1e6."""
    w = (1e6 ** (-torch.arange(0, dh, 2, device="cuda", dtype=torch.float64) / dh)).float()
    a = (torch.arange(POSITIONS, device="cuda").float()[:, None] * w).double()
    return torch.cat([a.cos(), a.sin()], dim=1).float().to(torch.bfloat16)


def _cumulative(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, device="cuda", dtype=torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)

    hq, hkv, dh = HEADS[case["heads"]]
    if case["op"] == "packed":
        lens, hist = _lengths(case["tokens"], case["seqs"]), _histories(case)
        cu_q, cu_k = _cumulative(lens), _cumulative([a + b for a, b in zip(lens, hist)])
        longest = max(a + b for a, b in zip(lens, hist))
        nq, nk = sum(lens), sum(lens) + sum(hist)
        st = dict(case=case, q=normal(nq, hq, dh), k=normal(nk, hkv, dh), v=normal(nk, hkv, dh), cu_q=cu_q, cu_k=cu_k,
                  longest_q=max(lens), longest=longest, out=torch.empty(nq, hq * dh, device="cuda", dtype=torch.bfloat16))
        if own:  # made once for a batch, for all layers
            from qwen3_decoder_transformer_gb300 import binding
            st["plan"] = torch.empty(binding.attention_packed_plan_bytes(nq, case["seqs"]), device="cuda", dtype=torch.uint8)
            binding.op_attention_packed_plan(cu_q, cu_k, nq, nk, st["plan"])
        return st
    page, slots = case["page"], _slots(case)
    counts = [-(-(a + n) // page) for a, n in slots]
    pool = sum(counts) + 3
    order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((case["seqs"], max(1, max(counts))), -1, device="cuda", dtype=torch.int32)
    at = 0
    for b, n in enumerate(counts):  # entries behind a sequence's pages are never read
        table[b, :n] = order[at:at + n]
        at += n
    size = page * _kv_bytes(dh)
    k_pages = torch.zeros(pool, hkv, size, device="cuda", dtype=torch.uint8)
    v_pages = torch.zeros(pool, hkv, size, device="cuda", dtype=torch.uint8)
    if case["op"] != "append":  # a filled cache
        every = torch.arange(pool, device="cuda").repeat_interleave(page)
        row = torch.arange(page, device="cuda").repeat(pool)
        for p in (k_pages, v_pages):
            for c in range(0, pool * page, 65536):
                e, r = every[c:c + 65536], row[c:c + 65536]
                _store(p, page, dh, e, r, torch.randn(e.numel(), hkv, dh, generator=gen, device="cuda"))
    n = sum(k for _, k in slots)
    st = dict(case=case, k_pages=k_pages, v_pages=v_pages, table=table, n=n, cu=_cumulative([k for _, k in slots]),
              start=torch.tensor([a for a, _ in slots], device="cuda", dtype=torch.int32))
    if case["op"] == "decode":
        st.update(q=normal(case["seqs"], hq, dh), out=torch.empty(case["seqs"], hq * dh, device="cuda", dtype=torch.bfloat16),
                  len0=torch.tensor([k - 1 for _, k in slots], device="cuda", dtype=torch.int32))
        if own:  # the scratch that a serving loop allocates once for its batch
            from qwen3_decoder_transformer_gb300 import binding
            st["work"] = torch.empty(binding.attention_decode_paged4_workspace(case["seqs"], hq, hkv, dh), device="cuda",
                                     dtype=torch.uint8)
        return st
    st.update(k_out=torch.zeros(n, hkv, dh, device="cuda", dtype=torch.bfloat16),
              v_out=torch.zeros(n, hkv, dh, device="cuda", dtype=torch.bfloat16))
    if case["op"] == "append":
        rows = n + case["pad"]
        st.update(qkv=normal(rows, (hq + 2 * hkv) * dh), table_rope=_rope_table(dh),
                  q_out=torch.zeros(rows, hq, dh, device="cuda", dtype=torch.bfloat16),
                  k_rot=torch.zeros(rows, hkv, dh, device="cuda", dtype=torch.bfloat16),
                  q_gamma=(1 + 0.1 * normal(dh)) if case["norm"] else None,
                  k_gamma=(1 + 0.1 * normal(dh)) if case["norm"] else None)
    return st


# -------------------------------------------------------------------------------------------------------- plain forms

def _rows(st):
    """Sequence, slot, page and row within the page of each of the call's n tokens."""
    t = torch.arange(st["n"], device=st["cu"].device)
    s = torch.searchsorted(st["cu"][1:].contiguous(), t.to(torch.int32), right=True)
    slot = st["start"][s].long() + t - st["cu"][s]
    page = st["case"]["page"]
    return s, slot, st["table"][s, slot // page].long(), slot % page


def _plain_append(st):
    hq, hkv, dh = HEADS[st["case"]["heads"]]
    n, page = st["n"], st["case"]["page"]
    _, slot, at, off = _rows(st)
    x = st["qkv"][:n].float().view(n, hq + 2 * hkv, dh)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if st["q_gamma"] is not None:
        q = q * torch.rsqrt(q.square().mean(dim=-1, keepdim=True) + EPS) * st["q_gamma"].float()
        k = k * torch.rsqrt(k.square().mean(dim=-1, keepdim=True) + EPS) * st["k_gamma"].float()
    cs = st["table_rope"][slot].float()[:, None]
    cos, sin = cs[..., :dh // 2], cs[..., dh // 2:]

    def rotate(y):
        a, b = y[..., :dh // 2], y[..., dh // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)

    q, k = rotate(q), rotate(k)
    st["q_out"][:n] = q.to(torch.bfloat16)
    st["k_rot"][:n] = k.to(torch.bfloat16)
    _store(st["k_pages"], page, dh, at, off, k)
    _store(st["v_pages"], page, dh, at, off, v)
    return (st["q_out"], st["k_rot"], _load(st["k_pages"], page, dh, at, off).to(torch.bfloat16),
            _load(st["v_pages"], page, dh, at, off).to(torch.bfloat16))


def _plain_read(st):
    dh = HEADS[st["case"]["heads"]][2]
    _, _, at, off = _rows(st)
    return tuple(_load(st[p], st["case"]["page"], dh, at, off).to(torch.bfloat16) for p in ("k_pages", "v_pages"))


def _plain_decode(st):
    hq, hkv, dh = HEADS[st["case"]["heads"]]
    b, n, page = st["case"]["seqs"], st["case"]["longest"], st["case"]["page"]
    slot = torch.arange(n, device="cuda")
    at = st["table"].long().clamp(min=0)[:, slot // page]                      # [b, n]
    off = (slot % page).expand(b, n)
    k = _load(st["k_pages"], page, dh, at.reshape(-1), off.reshape(-1)).view(b, n, hkv, dh).transpose(1, 2)
    q = st["q"].float().view(b, hkv, hq // hkv, dh) * dh ** -0.5
    x = torch.matmul(q, k.transpose(2, 3))
    seen = slot <= st["len0"][:, None]
    x = x.masked_fill_(~seen[:, None, None], float("-inf"))
    x = x.sub_(x.amax(dim=-1, keepdim=True)).exp_()
    z = x.sum(dim=-1, keepdim=True)
    del k
    v = _load(st["v_pages"], page, dh, at.reshape(-1), off.reshape(-1)).view(b, n, hkv, dh).transpose(1, 2)
    return (torch.matmul(x, v) / z).reshape(b, hq * dh).to(torch.bfloat16)


def _plain_packed(st):
    """Sequences padded to the longest one."""
    hq, hkv, dh = HEADS[st["case"]["heads"]]
    s, nq, nk = st["case"]["seqs"], st["longest_q"], st["longest"]
    cu_q, cu_k = st["cu_q"].long(), st["cu_k"].long()
    lq, lk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    i, j = torch.arange(nq, device="cuda"), torch.arange(nk, device="cuda")
    iq = (cu_q[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    ik = (cu_k[:-1, None] + j).clamp(max=st["k"].shape[0] - 1)
    q = st["q"][iq].float().view(s, nq, hkv, hq // hkv, dh).permute(0, 2, 3, 1, 4).reshape(s, hkv, -1, dh) * dh ** -0.5
    k, v = st["k"][ik].float().transpose(1, 2), st["v"][ik].float().transpose(1, 2)
    x = torch.matmul(q, k.transpose(2, 3)).view(s, hkv, hq // hkv, nq, nk)
    seen = j <= (i + (lk - lq)[:, None])[:, :, None]                            # [s, nq, nk]
    x.masked_fill_(~seen[:, None, None], float("-inf"))
    x.sub_(x.amax(dim=-1, keepdim=True)).exp_()
    z = x.sum(dim=-1, keepdim=True)
    o = torch.matmul(x.view(s, hkv, -1, nk), v).view(s, hkv, hq // hkv, nq, dh) / z
    o = o.permute(0, 3, 1, 2, 4).reshape(s, nq, hq * dh)
    return o[i < lq[:, None]].to(torch.bfloat16)


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        from qwen3_decoder_transformer_gb300 import binding
        if op == "append":
            binding.op_append_paged4(state["qkv"], state["cu"], state["start"], state["table_rope"], state["k_pages"],
                                     state["v_pages"], state["table"], state["q_out"], k_out=state["k_rot"],
                                     q_gamma=state["q_gamma"], k_gamma=state["k_gamma"], eps=EPS)
        if op in ("append", "read"):
            binding.op_read_paged4(state["k_pages"], state["v_pages"], state["table"], state["cu"], state["start"],
                                   state["k_out"], state["v_out"])
            if op == "read":
                return state["k_out"], state["v_out"]
            return state["q_out"], state["k_rot"], state["k_out"], state["v_out"]
        if op == "decode":
            binding.op_attention_decode_paged4(state["q"], state["k_pages"], state["v_pages"], state["table"], state["len0"],
                                               state["work"], state["out"])
        else:
            binding.op_attention_prefill_packed(state["q"], state["k"], state["v"], state["plan"], state["longest"],
                                                state["out"])
        return state["out"]
    if op == "append":
        return _plain_append(state)
    if op == "read":
        return _plain_read(state)
    if op == "decode":
        return _plain_decode(state)
    return _plain_packed(state)


# --------------------------------------------------------------------------------------------------------------- exact

def _attend64(q, k, v, scale, first):
    """q [hkv, g, t, dh] over k, v [hkv, n, dh] in fp64; query i sees keys up to first + i."""
    x = torch.einsum("hgtd,hnd->hgtn", q, k) * scale
    i, j = torch.arange(q.shape[2], device="cuda"), torch.arange(k.shape[1], device="cuda")
    x.masked_fill_(j > first + i[:, None], float("-inf"))
    return torch.einsum("hgtn,hnd->hgtd", torch.softmax(x, dim=-1), v)


def _cached64(pages, table, b, a, n, page, dh):
    """Slots a .. a + n - 1 of sequence b, [n, hkv, dh] in fp64, page by page."""
    rows = []
    for p in range(a // page, -(-(a + n) // page)):
        raw = pages[int(table[b, p])]                                            # [hkv, bytes]
        h = raw.shape[0]
        c = raw[:, :page * dh // 2].reshape(h, page, dh // 2)
        c = torch.stack([c % 16, c // 16], dim=-1).reshape(h, page, dh // GROUP, GROUP).double()
        s = raw[:, page * dh // 2:].contiguous().view(torch.bfloat16).reshape(h, page, dh // GROUP, 2).double()
        rows.append((s[..., 1:] + s[..., :1] * c).reshape(h, page, dh).transpose(0, 1))
    lo = a // page * page
    return torch.cat(rows)[a - lo:a - lo + n] if rows else torch.zeros(0, pages.shape[1], dh, device="cuda", dtype=torch.float64)


def _nearby(x):
    """What the cache keeps of x [n, hkv, dh] (fp64)."""
    g = x.reshape(*x.shape[:-1], -1, GROUP)

    def bf16_below(y):
        e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -126)))
        step = torch.exp2(e - 7)
        return torch.floor(y / step) * step

    lo = bf16_below(g.min(dim=-1, keepdim=True).values)
    sc = -bf16_below(-(g.max(dim=-1, keepdim=True).values - lo) / 15)
    code = torch.where(sc > 0, torch.round((g - lo) / sc), torch.zeros_like(g)).clamp(0, 15)
    return (lo + sc * code).reshape(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    hq, hkv, dh = HEADS[case["heads"]]
    if case["op"] == "packed":
        if work(case)["flops"] > 4e12:
            return None  # beyond what fp64 units do in the time
        out, iq, ik = [], 0, 0
        for n, h in zip(_lengths(case["tokens"], case["seqs"]), _histories(case)):
            k, v = (st[x][ik:ik + n + h].double().transpose(0, 1) for x in ("k", "v"))
            for a in range(0, n, 512):
                e = min(n, a + 512)
                q = st["q"][iq + a:iq + e].double().reshape(e - a, hkv, hq // hkv, dh).permute(1, 2, 0, 3)
                o = _attend64(q, k[:, :h + e], v[:, :h + e], dh ** -0.5, h + a)
                out.append(o.permute(2, 0, 1, 3).reshape(e - a, hq * dh))
            iq, ik = iq + n, ik + n + h
        return torch.cat(out)
    if sum(n for _, n in _slots(case)) // case["page"] > 20000:
        return None
    table, page = st["table"].cpu(), case["page"]
    if case["op"] == "append":
        n = st["n"]
        slot = torch.cat([torch.arange(a, a + k, device="cuda") for a, k in _slots(case)])
        x = st["qkv"][:n].double().reshape(n, hq + 2 * hkv, dh)
        ang = st["table_rope"].double()[slot]
        cos, sin = ang[:, None, :dh // 2], ang[:, None, dh // 2:]
        pair = []
        for y, g in ((x[:, :hq], st["q_gamma"]), (x[:, hq:hq + hkv], st["k_gamma"])):
            if g is not None:
                y = y / torch.sqrt((y * y).sum(dim=-1, keepdim=True) / dh + EPS) * g.double()
            z = torch.complex(y[..., :dh // 2], y[..., dh // 2:]) * torch.complex(cos, sin)
            pair.append(torch.cat([z.real, z.imag], dim=-1))
        padded = [torch.cat([y, torch.zeros(case["pad"], y.shape[1], dh, device="cuda", dtype=torch.float64)]) for y in pair]
        return padded[0], padded[1], _nearby(pair[1]), _nearby(x[:, hq + hkv:])
    if case["op"] == "read":
        return tuple(torch.cat([_cached64(st[p], table, b, a, n, page, dh) for b, (a, n) in enumerate(_slots(case))])
                     for p in ("k_pages", "v_pages"))
    out = []
    for b, (a, n) in enumerate(_slots(case)):
        k, v = (_cached64(st[p], table, b, a, n, page, dh).transpose(0, 1) for p in ("k_pages", "v_pages"))
        q = st["q"][b].double().reshape(hkv, hq // hkv, 1, dh)
        out.append(_attend64(q, k, v, dh ** -0.5, n - 1).reshape(hq * dh))
    return torch.stack(out)


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(6)]:
        print(c, work(c))
