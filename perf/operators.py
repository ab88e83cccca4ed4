"""Cases for the serving operators: token log probabilities, decode attention over a shared prefix, and attention with a
sliding window and sink tokens (prefill and single-token form), each in plain torch and through the library.

A case is one call as a serving loop makes it; see listed(). K/V caches hold [.., slots, head_dim] bf16 as the library's.
"""
import random

import torch

own = False

# (query heads, kv heads, head_dim): the tiny, 0.6B and 8B stacks of this repository, and groups of 1, 3 and 8 query heads
HEADS = [(8, 4, 64), (16, 8, 128), (32, 8, 128), (8, 8, 64), (12, 4, 128), (16, 2, 128)]


def listed():
    return [
        # ---- log probabilities of the sampled token with entropy and alternatives
        # one sequence's decode step at the full vocabulary: latency
        dict(name="logprobs 1x151936 k20", op="logprobs", rows=1, vocab=151936, top_k=20, dtype="float32", pad=0),
        # a decode batch of 64, as an API that returns five alternatives asks for it
        dict(name="logprobs 64x151936 k5", op="logprobs", rows=64, vocab=151936, top_k=5, dtype="float32", pad=0),
        # scoring a 2048-token prompt from all rows' logits (prefill with all rows)
        dict(name="logprobs 2048x151936 k1", op="logprobs", rows=2048, vocab=151936, top_k=1, dtype="float32", pad=0),
        # bf16 logits of an odd vocabulary in padded rows: ties, unaligned rows
        dict(name="logprobs 333x32003 bf16 k32", op="logprobs", rows=333, vocab=32003, top_k=32, dtype="bfloat16", pad=10),
        # ---- decode attention, prefix shared by the batch
        # a few prompts over the 582-token shared start of the classification notebook: latency
        dict(name="shared 4 @ 582", op="shared", batch=4, heads=1, prefix=582, own_max=48),
        # the 0.6B batch of 64 over a 4096-token start
        dict(name="shared 64 @ 4096 0.6b", op="shared", batch=64, heads=1, prefix=4096, own_max=512),
        # 64 answers over a 32768-token document, 8B heads
        dict(name="shared 64 @ 32768 8b", op="shared", batch=64, heads=2, prefix=32768, own_max=1024),
        # many short answers: 200 sequences, 800 query rows a kv head, tensor bound
        dict(name="shared 200 @ 16384 8b", op="shared", batch=200, heads=2, prefix=16384, own_max=64),
        # ---- sliding window with sinks: prefill and single tokens
        # a 2048-token prompt, short window, 0.6B heads
        dict(name="sinks prefill 1x2048 w512", op="sinks_prefill", batch=1, tokens=2048, heads=1, start=0, window=512,
             sinks=4, rolling=False),
        # a 16384-token prompt through a 4096 window, 8B heads
        dict(name="sinks prefill 1x16384 w4096", op="sinks_prefill", batch=1, tokens=16384, heads=2, start=0,
             window=4096, sinks=128, rolling=False),
        # one sequence far past its window, from a rolling buffer: latency
        dict(name="sinks decode 1 w4096", op="sinks_decode", batch=1, heads=2, start=32768, window=4096, sinks=4,
             rolling=True),
        # the 0.6B batch of 64 at its own lengths
        dict(name="sinks decode 64 w4096", op="sinks_decode", batch=64, heads=1, start=6000, window=4096, sinks=4,
             rolling=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["logprobs", "shared", "sinks_prefill", "sinks_decode"])
    if op == "logprobs":
        vocab = rng.choice([151936, _log_int(rng, 1000, 152000)])
        rows = _log_int(rng, 1, 2048)
        return dict(op=op, rows=rows, vocab=vocab, top_k=rng.randint(0, 32), dtype=rng.choice(["float32", "bfloat16"]),
                    pad=rng.choice([0, rng.randint(1, 64)]))
    heads = rng.randrange(len(HEADS))
    if op == "shared":
        return dict(op=op, batch=_log_int(rng, 1, 128), heads=heads, prefix=_log_int(rng, 16, 32768),
                    own_max=_log_int(rng, 1, 1024))
    window, sinks = _log_int(rng, 16, 4096), rng.choice([0, 1, 4, rng.randint(1, 300)])
    rolling = rng.random() < 0.5
    if op == "sinks_decode":
        return dict(op=op, batch=_log_int(rng, 1, 64), heads=heads, start=_log_int(rng, 1, 8192), window=window,
                    sinks=sinks, rolling=rolling)
    batch = rng.choice([1, 1, 2, 5])
    return dict(op=op, batch=batch, tokens=max(1, _log_int(rng, 1, 8192) // batch), heads=heads,
                start=rng.choice([0, _log_int(rng, 1, 8192)]), window=window, sinks=sinks, rolling=rolling)


# ------------------------------------------------------------------------------------------------ geometry of a case

def _own_lengths(case):
    """Own keys of each sequence: 1 .. own_max, spread over the batch."""
    return [1 + (b * 7919) % case["own_max"] for b in range(case["batch"])]


def _starts(case):
    """Cache slots before the call: sequences stop at their own lengths, the first at the longest."""
    return [max(0, case["start"] - (b * 613) % (case["start"] // 4 + 1)) for b in range(case["batch"])]


def _sink_rows(case):
    """Cache rows that keep the first slots in a rolling buffer: the sinks in whole 128-row tiles."""
    return (case["sinks"] + 127) // 128 * 128


def _cache_rows(case, tokens):
    if not case["rolling"]:
        return case["start"] + tokens
    return _sink_rows(case) + (case["window"] + tokens - 1 + 127) // 128 * 128


def _rows_of(slots, case, rows):
    """Cache row of each slot (a tensor of slots)."""
    if not case["rolling"]:
        return slots
    r0 = _sink_rows(case)
    return torch.where(slots < r0, slots, r0 + (slots - r0) % (rows - r0))


def _pairs(case):
    """Visible (query, key) pairs and visible keys over the batch, each counted once."""
    w, s, t = case["window"], case["sinks"], case.get("tokens", 1)
    pairs = keys = 0
    for n in _starts(case):
        for i in range(n, n + t):
            lo = max(0, i - w + 1)
            pairs += i - lo + 1 + min(s, lo)
        first = max(0, n - w + 1)
        keys += n + t - first + min(s, first)
    return pairs, keys


def work(case):
    if case["op"] == "logprobs":
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": case["rows"] * (case["vocab"] * size + 4 + 8 + 8 * case["top_k"]),
                "flops": 6 * case["rows"] * case["vocab"]}
    hq, hkv, dh = HEADS[case["heads"]]
    if case["op"] == "shared":
        n = sum(_own_lengths(case))
        return {"bytes": 4 * hkv * dh * (case["prefix"] + n) + 4 * case["batch"] * hq * dh,
                "flops": 4 * dh * hq * (case["batch"] * case["prefix"] + n)}
    pairs, keys = _pairs(case)
    return {"bytes": 4 * hkv * dh * keys + 4 * case["batch"] * case.get("tokens", 1) * hq * dh,
            "flops": 4 * dh * hq * pairs}


# ------------------------------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)

    if case["op"] == "logprobs":
        m, v, k = case["rows"], case["vocab"], case["top_k"]
        full = torch.empty(m, v + case["pad"], device="cuda", dtype=getattr(torch, case["dtype"]))
        full.normal_(0.0, 3.0, generator=gen)  # logits spread as a language model's, a few tokens well above the rest
        tokens = torch.randint(0, v, (m,), generator=gen, device="cuda", dtype=torch.int32)
        return dict(case=case, logits=full[:, :v], tokens=tokens,
                    logprob=torch.empty(m, device="cuda"), entropy=torch.empty(m, device="cuda"),
                    top_ids=torch.empty(m, k, device="cuda", dtype=torch.int32),
                    top_logprobs=torch.empty(m, k, device="cuda"))
    hq, hkv, dh = HEADS[case["heads"]]
    b = case["batch"]
    if case["op"] == "shared":
        lens = _own_lengths(case)
        st = dict(case=case, q=normal(b, hq, dh), k_prefix=normal(hkv, case["prefix"], dh),
                  v_prefix=normal(hkv, case["prefix"], dh), k=normal(b, hkv, case["own_max"], dh),
                  v=normal(b, hkv, case["own_max"], dh), out=torch.empty(b, hq * dh, device="cuda", dtype=torch.bfloat16),
                  len0=torch.tensor([n - 1 for n in lens], device="cuda", dtype=torch.int32))
        if own:  # the scratch that a serving loop allocates once for its batch and prefix
            from qwen3_decoder_transformer_gb300 import binding
            st["work"] = torch.empty(binding.attention_decode_shared_workspace(b, hq, hkv, dh, case["prefix"]),
                                     device="cuda", dtype=torch.uint8)
        return st
    t = case.get("tokens", 1)
    rows = _cache_rows(case, t)
    q = normal(b, hq, t, dh) if case["op"] == "sinks_prefill" else normal(b, hq, dh)
    return dict(case=case, q=q, k=normal(b, hkv, rows, dh), v=normal(b, hkv, rows, dh),
                out=torch.empty(b * t, hq * dh, device="cuda", dtype=torch.bfloat16),
                len0=torch.tensor(_starts(case), device="cuda", dtype=torch.int32))


# -------------------------------------------------------------------------------------------------------- plain forms

def _plain_logprobs(st):
    x, k = st["logits"].float(), st["case"]["top_k"]
    top = x.max(dim=1, keepdim=True).values
    d = x - top
    e = d.exp()
    z = e.sum(dim=1, keepdim=True)
    logz = z.log()
    lp = d.gather(1, st["tokens"].long()[:, None]) - logz
    entropy = logz - (e * d).sum(dim=1, keepdim=True) / z
    val, idx = x.sort(dim=1, descending=True, stable=True)  # stable: ties go to the lowest index
    return lp[:, 0], entropy[:, 0], idx[:, :k].to(torch.int32), val[:, :k] - top - logz


def _plain_shared(st):
    b, hq, dh = st["q"].shape
    hkv, cap = st["k"].shape[1], st["k"].shape[2]
    q = st["q"].float().reshape(b, hkv, hq // hkv, dh) * dh ** -0.5
    sp = torch.matmul(q.transpose(0, 1).reshape(hkv, -1, dh), st["k_prefix"].float().transpose(1, 2))
    sp = sp.reshape(hkv, b, hq // hkv, -1).transpose(0, 1)
    so = torch.matmul(q, st["k"].float().transpose(2, 3))
    seen = torch.arange(cap, device=q.device) <= st["len0"][:, None]
    so = so.masked_fill(~seen[:, None, None, :], float("-inf"))
    s = torch.cat([sp, so], dim=3)
    e = (s - s.max(dim=3, keepdim=True).values).exp()
    p = e / e.sum(dim=3, keepdim=True)
    n = sp.shape[3]
    op = torch.matmul(p[..., :n].transpose(0, 1).reshape(hkv, -1, n), st["v_prefix"].float())
    op = op.reshape(hkv, b, hq // hkv, dh).transpose(0, 1)
    return (op + torch.matmul(p[..., n:], st["v"].float())).reshape(b, hq * dh).to(torch.bfloat16)


def _plain_sinks(st):
    """Queries in blocks of up to 1024; each block gathers the sinks and the slots any of its rows sees."""
    case, q = st["case"], st["q"]
    if q.dim() == 3:
        q = q[:, :, None, :]
    b, hq, t, dh = q.shape
    hkv, rows = st["k"].shape[1], st["k"].shape[2]
    g, w, s = hq // hkv, case["window"], case["sinks"]
    nb = min(t, 1024)
    blocks = (t + nb - 1) // nb
    dev = q.device
    at = torch.arange(blocks * nb, device=dev).clamp(max=t - 1).reshape(blocks, nb)
    slot_q = st["len0"].long()[:, None, None] + at                       # [b, blocks, nb]
    first = slot_q[:, :, :1] - w + 1                                      # oldest slot the block's first row sees
    near = first + torch.arange(w + nb - 1, device=dev)                   # [b, blocks, w + nb - 1]
    far = torch.arange(s, device=dev).expand(b, blocks, s)
    far = torch.where(far < first.clamp(min=0), far, -1)                  # a sink that the near part holds counts once
    slots = torch.cat([far, near], dim=2)
    i, j = slot_q[..., None], slots[:, :, None, :]
    seen = (j >= 0) & (j <= i) & ((i - j < w) | (j < s))                  # [b, blocks, nb, keys]
    idx = _rows_of(slots.clamp(min=0), case, rows).clamp(max=rows - 1)
    pick = torch.arange(b, device=dev)[:, None, None]
    k = st["k"].transpose(1, 2)[pick, idx].float().permute(0, 3, 1, 2, 4)  # [b, hkv, blocks, keys, dh]
    v = st["v"].transpose(1, 2)[pick, idx].float().permute(0, 3, 1, 2, 4)
    qb = q[:, :, at.reshape(-1)].float().reshape(b, hkv, g, blocks, nb, dh) * dh ** -0.5
    qb = qb.permute(0, 1, 3, 2, 4, 5).reshape(b, hkv, blocks, g * nb, dh)
    x = torch.matmul(qb, k.transpose(3, 4)).reshape(b, hkv, blocks, g, nb, -1)
    x = x.masked_fill_(~seen[:, None, :, None], float("-inf"))
    x = x.sub_(x.max(dim=5, keepdim=True).values).exp_()
    z = x.sum(dim=5, keepdim=True).reshape(b, hkv, blocks, g * nb, 1)
    o = torch.matmul(x.reshape(b, hkv, blocks, g * nb, -1), v) / z
    o = o.reshape(b, hkv, blocks, g, nb, dh).permute(0, 2, 4, 1, 3, 5).reshape(b, blocks * nb, hq * dh)
    return o[:, :t].reshape(b * t, hq * dh).to(torch.bfloat16)


def run(state):
    op = state["case"]["op"]
    if own:
        from qwen3_decoder_transformer_gb300 import binding
        c = state["case"]
        if op == "logprobs":
            binding.op_token_logprobs(state["logits"], state["tokens"], state["logprob"], entropy=state["entropy"],
                                      top_ids=state["top_ids"], top_logprobs=state["top_logprobs"])
            return state["logprob"], state["entropy"], state["top_ids"], state["top_logprobs"]
        if op == "shared":
            binding.op_attention_decode_shared(state["q"], state["k_prefix"], state["v_prefix"], state["k"], state["v"],
                                               state["len0"], state["work"], state["out"])
        elif op == "sinks_prefill":
            binding.op_attention_prefill_sinks(state["q"], state["k"], state["v"], state["len0"], state["out"],
                                               c["window"], c["sinks"], rolling=c["rolling"])
        else:
            binding.op_attention_decode_sinks(state["q"], state["k"], state["v"], state["len0"], state["out"],
                                              c["window"], c["sinks"], rolling=c["rolling"])
        return state["out"]
    if op == "logprobs":
        return _plain_logprobs(state)
    if op == "shared":
        return _plain_shared(state)
    return _plain_sinks(state)


# --------------------------------------------------------------------------------------------------------------- exact

def _attend64(q, keys, values):
    """softmax(q k^T / sqrt(dh)) v in fp64: q [hkv, rows, dh], keys and values [hkv, n, dh]."""
    w = torch.softmax(torch.einsum("hrd,hnd->hrn", q, keys) / q.shape[-1] ** 0.5, dim=-1)
    return torch.einsum("hrn,hnd->hrd", w, values)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "logprobs":
        m, k = case["rows"], case["top_k"]
        lps, ents, ids, tops = [], [], [], []
        for r in range(0, m, 128):
            x = st["logits"][r:r + 128].double()
            lsm = torch.log_softmax(x, dim=1)
            lps.append(lsm.gather(1, st["tokens"][r:r + 128].long()[:, None])[:, 0])
            ents.append(-(lsm.exp() * lsm).sum(dim=1))
            order = torch.argsort(-x, dim=1, stable=True)[:, :k]
            ids.append(order.to(torch.int32))
            tops.append(lsm.gather(1, order))
        return torch.cat(lps), torch.cat(ents), torch.cat(ids), torch.cat(tops)
    hq, hkv, dh = HEADS[case["heads"]]
    if case["op"] == "shared":
        out = []
        for b, n in enumerate(_own_lengths(case)):
            keys = torch.cat([st["k_prefix"], st["k"][b, :, :n]], dim=1).double()
            values = torch.cat([st["v_prefix"], st["v"][b, :, :n]], dim=1).double()
            out.append(_attend64(st["q"][b].double().reshape(hkv, hq // hkv, dh), keys, values).reshape(hq * dh))
        return torch.stack(out)
    if _pairs(case)[0] * hq * dh * 4 > 4e12:
        return None  # beyond what fp64 units do in the time
    t, w, s = case.get("tokens", 1), case["window"], case["sinks"]
    rows = st["k"].shape[2]
    q = st["q"].reshape(case["batch"], hkv, hq // hkv, t, dh)
    out = torch.empty(case["batch"], t, hq, dh, dtype=torch.float64, device="cuda")
    step = 1 if t == 1 else 256
    for b, n in enumerate(_starts(case)):
        for a in range(0, t, step):
            e = min(t, a + step)
            lo = max(0, n + a - w + 1)
            slots = list(range(min(s, lo))) + list(range(lo, n + e))  # every slot some row of the block sees
            sl = torch.tensor(slots, device="cuda")
            at = _rows_of(sl, case, rows)
            kk, vv = st["k"][b][:, at].double(), st["v"][b][:, at].double()
            i = torch.arange(n + a, n + e, device="cuda")[:, None]
            hidden = (sl > i) | ((i - sl >= w) & (sl >= s))
            for h in range(hkv):
                x = torch.einsum("gtd,nd->gtn", q[b, h, :, a:e].double(), kk[h]) / dh ** 0.5
                x.masked_fill_(hidden, float("-inf"))
                o = torch.einsum("gtn,nd->gtd", torch.softmax(x, dim=-1), vv[h])
                out[b, a:e, h * (hq // hkv):(h + 1) * (hq // hkv)] = o.transpose(0, 1)
    return out.reshape(case["batch"] * t, hq * dh)


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(6)]:
        print(c, work(c))
