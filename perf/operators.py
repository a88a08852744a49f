"""Cases of the dense operators over a RecSA token cache, for measurement.

Four operators: attention over all visible tokens of the cache (a decode step's single
tokens, or a chunk of new tokens), the same with a sliding window and sinks, the attention
weight each cache slot receives, and the eviction of slots by that weight.  `own` chooses
between the plain form (elementary torch operations in 32 bits) and the framework's calls.

The cache holds keys before RoPE; token t is rotated to position t when it is scored.
"""

import math

import torch

own = False

D = 128
HALF = 64
BASE = 1.0e6
SCALE = 1.0 / math.sqrt(D)


# --------------------------------------------------------------------------- cases


def listed():
    return [
        # the tiny decode workload: 16 independent queries over one short cache (latency)
        dict(name="decode_tiny", op="attend", batch=1, kv=1, group=4, length=4096, queries=16, causal=False,
             page=0, ragged=False, sinks=0, window=0, fp32=True),
        # one decode step of eight long sequences of the 131K decode workload's head shape
        dict(name="decode_131k", op="attend", batch=8, kv=8, group=4, length=131072, queries=1, causal=False,
             page=0, ragged=False, sinks=0, window=0, fp32=False),
        # a serving batch: uneven sequences in pages of 16 tokens, eight query heads a group
        dict(name="decode_ragged_paged", op="attend", batch=24, kv=4, group=8, length=19001, queries=1, causal=False,
             page=16, ragged=True, sinks=0, window=0, fp32=False),
        # short chunks of a continuous batch over paged caches of uneven length
        dict(name="chunk_paged", op="attend", batch=4, kv=8, group=4, length=8205, queries=130, causal=True,
             page=64, ragged=True, sinks=0, window=0, fp32=False),
        # a long prompt's chunk over what came before it, at the 32/8 head shape
        dict(name="chunk_large", op="append_attend", batch=1, kv=8, group=4, length=32768, queries=4096, causal=True,
             page=0, ragged=False, sinks=0, window=0, fp32=False),
        # single tokens of a windowed layer: a short read from many sequences (latency)
        dict(name="window_decode", op="attend", batch=32, kv=8, group=4, length=16384, queries=1, causal=False,
             page=0, ragged=False, sinks=4, window=1024, fp32=False),
        # a windowed layer's prompt chunk
        dict(name="window_chunk", op="append_attend", batch=1, kv=8, group=4, length=18000, queries=2048, causal=True,
             page=0, ragged=False, sinks=4, window=1024, fp32=False),
        # verification of a few draft tokens in a windowed layer, 32-bit output, odd sizes
        dict(name="window_verify_fp32", op="attend", batch=6, kv=2, group=2, length=5001, queries=5, causal=True,
             page=32, ragged=True, sinks=3, window=777, fp32=True),
        # the last queries of a prompt judge which of its tokens are worth keeping
        dict(name="weights_prompt", op="weights", batch=1, kv=8, group=4, length=32768, queries=64, causal=True,
             page=0, ragged=False, sinks=0, window=0, fp32=True),
        # the weights one decode step adds
        dict(name="weights_step", op="weights", batch=4, kv=8, group=4, length=65536, queries=1, causal=False,
             page=0, ragged=False, sinks=0, window=0, fp32=True),
        # a short cache cut to half (latency)
        dict(name="evict_short", op="evict", batch=2, kv=4, group=4, length=2051, keep=1024, page=16, ragged=True,
             sinks=4, recent=64),
        # long caches cut to a quarter
        dict(name="evict_long", op="evict", batch=4, kv=8, group=4, length=131072, keep=32768, page=0, ragged=False,
             sinks=4, recent=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "chunk", "chunk", "window", "window", "weights", "evict"])
    kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
    page = rng.choice([0, 0, 16, 64, 256])
    ragged = rng.random() < 0.4
    if op == "evict":
        length = _log(rng, 600, 131072)
        batch = max(1, min(_log(rng, 1, 16), (32 * 131072) // (length * kv)))
        keep = max(64, int(length * rng.uniform(0.1, 0.9)))
        return dict(op="evict", batch=batch, kv=kv, group=group, length=length, keep=keep, page=page, ragged=ragged,
                    sinks=rng.choice([0, 4, 16]), recent=rng.randrange(0, min(keep - 16, 1024) + 1))
    if op == "weights":
        queries = rng.choice([1, 1, 2, 8, 17, 32, 64])
        length = _log(rng, 512, 65536)
        batch = max(1, min(_log(rng, 1, 16), int(2.0e9 / (length * kv * group * queries * 4.0)),
                           (32 * 65536) // (length * kv)))
        return dict(op="weights", batch=batch, kv=kv, group=group, length=length, queries=queries,
                    causal=queries > 1, page=page, ragged=ragged, sinks=0, window=0, fp32=True)
    sinks = window = 0
    if op == "window":
        sinks, window = rng.choice([0, 1, 4, 16]), _log(rng, 32, 4096)
    chunk = op == "chunk" or (op == "window" and rng.random() < 0.5)
    if chunk:
        queries = _log(rng, 2, 4000)
        length = _log(rng, max(queries, 256), 30000)
        queries = min(queries, int(4.0e9 / (length * kv * group)))
        batch = max(1, min(_log(rng, 1, 8), int(5.0e8 / (queries * float(length) * kv * group))))
    else:
        queries = rng.choice([1, 1, 1, 4])
        length = _log(rng, 256, 131072)
        batch = max(1, min(_log(rng, 1, 64), (64 * 131072) // (length * kv * 2)))
    fp32 = rng.random() < (0.15 if chunk else 0.3)
    append = chunk and page == 0 and not ragged and rng.random() < 0.5
    return dict(op="append_attend" if append else "attend", batch=batch, kv=kv, group=group, length=length,
                queries=queries, causal=chunk, page=page, ragged=ragged, sinks=sinks, window=window, fp32=fp32)


# --------------------------------------------------------------------------- inputs


def _lengths(c, g):
    """Tokens of each sequence: the case's length, or uneven ones up to it (the first the longest)."""
    B, L = c["batch"], c["length"]
    if not c["ragged"]:
        return torch.full((B,), L, dtype=torch.int64, device="cuda")
    lens = (torch.rand(B, generator=g, device="cuda", dtype=torch.float64) * L).long().clamp(1, L)
    lens[0] = L
    return lens


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, H, G, L = c["batch"], c["kv"], c["group"], c["length"]
    Hq = H * G
    cap = -(-L // c["page"]) * c["page"] if c["page"] else L
    s = dict(c, cap=cap)
    s["lens"] = _lengths(c, g)
    # uneven magnitudes of the channels, as keys and values have
    ks = torch.empty(1, H, 1, D, device="cuda").uniform_(0.5, 2.0, generator=g).bfloat16()
    vs = torch.empty(1, H, 1, D, device="cuda").uniform_(0.5, 2.0, generator=g).bfloat16()

    def rows(n0, n2, scale):
        x = torch.empty(n0, H, n2, D, device="cuda", dtype=torch.bfloat16)
        return x.normal_(generator=g).mul_(scale)

    if c["page"]:
        pps = cap // c["page"]
        pages = B * pps + 3
        s["table"] = torch.randperm(pages, generator=g, device="cuda")[: B * pps].to(torch.int32).view(B, pps)
        s["k"], s["v"] = rows(pages, c["page"], ks), rows(pages, c["page"], vs)
    else:
        s["table"] = None
        s["k"], s["v"] = rows(B, cap, ks), rows(B, cap, vs)
    if c["op"] == "evict":
        # accumulated weights have a long tail; equal ones occur among the untouched slots
        w = torch.empty(B, H, cap, device="cuda").exponential_(1.0, generator=g).pow_(3.0)
        s["w"] = torch.where(w < 0.01, torch.zeros_like(w), w)
        s["to_k"] = torch.empty(B, H, c["keep"], D, device="cuda", dtype=torch.bfloat16)
        s["to_v"] = torch.empty_like(s["to_k"])
        s["to_w"] = torch.zeros(B, H, c["keep"], device="cuda")
        s["kept"] = torch.empty(B, H, c["keep"], device="cuda", dtype=torch.int32)
    else:
        n = c["queries"]
        s["q"] = torch.empty(B, n, Hq, D, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
        if c["op"] == "weights":
            s["w"] = torch.zeros(B, H, cap, device="cuda")
        else:
            s["out"] = torch.empty(B, n, Hq, D, device="cuda", dtype=torch.float32 if c["fp32"] else torch.bfloat16)
        if c["op"] == "append_attend":
            s["k_new"] = torch.empty(B, n, H, D, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
            s["v_new"] = torch.empty(B, n, H, D, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    if own:
        _plan(s)
    return s


def _plan(s):
    """What a user's program keeps: parameters, the cache handles, the workspace and the view."""
    import hierarchical_sparse_attention_build_b200 as R

    s["R"] = R
    s["p"] = R.params(num_kv_heads=s["kv"], num_q_heads=s["kv"] * s["group"], branching=16, top_k=8, rope_base=BASE)
    seq = s["lens"].clone() if s["ragged"] else None
    s["cache"] = R.TokenCache(s["p"], s["k"], s["v"], s["length"], seq_len=seq, page_table=s["table"])
    if s["op"] == "evict":
        s["into"] = R.TokenCache(s["p"], s["to_k"], s["to_v"], 0, seq_len=None if seq is None else seq.clone())
    else:
        s["ws"] = R.DenseWorkspace(s["p"], s["batch"], s["cap"], "cuda")
        s["view"] = R.View(sinks=s["sinks"], window=s["window"], causal=s["causal"], own_token=s["causal"])


# --------------------------------------------------------------------------- the plain form


def _angles(pos):
    """cos and sin of position x frequency, fp32 [..., 64]; the angle itself in 64 bits."""
    f = BASE ** (-(2.0 * torch.arange(HALF, device=pos.device, dtype=torch.float64)) / D)
    a = pos.double()[..., None] * f
    return a.cos().float(), a.sin().float()


def _rope(x, cs):
    lo, hi = x[..., :HALF], x[..., HALF:]
    return torch.cat([lo * cs[0] - hi * cs[1], hi * cs[0] + lo * cs[1]], dim=-1)


def _tokens(s, pool):
    """The cache's rows in token order, [B][H][cap][128]."""
    if s["table"] is None:
        return pool
    B, pps = s["table"].shape
    x = pool[s["table"].long().view(-1)].view(B, pps, s["kv"], s["page"], D)
    return x.permute(0, 2, 1, 3, 4).reshape(B, s["kv"], pps * s["page"], D)


def _positions(s):
    """Position of each query, [B][n]."""
    n = s["queries"]
    p = s["lens"][:, None] + torch.zeros(n, dtype=torch.int64, device="cuda")
    return p - n + 1 + torch.arange(n, device="cuda") if s["causal"] else p


def _probs(s):
    """Softmax weights [B][H][n * G][cap] of every query row (query-major) over the cache's slots."""
    B, H, G, n = s["batch"], s["kv"], s["group"], s["queries"]
    t = torch.arange(s["cap"], device="cuda")
    p = _positions(s)
    k = _rope(_tokens(s, s["k"]).float(), _angles(t))
    q = s["q"].float().view(B, n, H, G, D)

    def scores(pos, keys):
        c, sn = _angles(pos)
        r = _rope(q, (c[:, :, None, None], sn[:, :, None, None])) * SCALE
        return r.permute(0, 2, 1, 3, 4).reshape(B, H, n * G, D) @ keys.transpose(-1, -2)

    x = scores(p, k)
    pe = p[:, :, None]
    seen = t < pe
    if s["window"]:
        m = s["sinks"]
        if m:  # sinks sit at their rank before the window's tokens
            x[..., :m] = scores(torch.minimum(p, torch.tensor(m + s["window"], device="cuda")), k[..., :m, :])
        seen = seen & ((t < m) | (t >= pe - s["window"]))
    hidden = ~seen.repeat_interleave(G, dim=1)[:, None]
    x.masked_fill_(hidden, -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = x.sum(-1, keepdim=True)
    return x.div_(torch.where(total == 0, torch.ones_like(total), total))


def _plain_attend(s):
    B, H, G, n = s["batch"], s["kv"], s["group"], s["queries"]
    o = _probs(s) @ _tokens(s, s["v"]).float()
    o = o.view(B, H, n, G, D).permute(0, 2, 1, 3, 4).reshape(B, n, H * G, D)
    return o if s["fp32"] else o.bfloat16()


def _plain_append(s):
    at = s["length"] - s["queries"]
    s["k"][:, :, at: s["length"]] = s["k_new"].transpose(1, 2)
    s["v"][:, :, at: s["length"]] = s["v_new"].transpose(1, 2)


def _plain_weights(s):
    B, H, cap = s["batch"], s["kv"], s["cap"]
    w = _probs(s).sum(2)
    live = torch.arange(cap, device="cuda") < s["lens"][:, None]
    return torch.where(live[:, None].expand(B, H, cap), w, s["w"])


def _plain_evict(s):
    B, H, keep, cap = s["batch"], s["kv"], s["keep"], s["cap"]
    t = torch.arange(cap, device="cuda")
    n = s["lens"][:, None]
    forced = (t < s["sinks"]) | (t >= n - s["recent"])
    rank = torch.where(forced, torch.full((), math.inf, device="cuda"), torch.zeros((), device="cuda"))[:, None] + s["w"]
    rank = torch.where((t < n)[:, None], rank, torch.full((), -math.inf, device="cuda"))
    order = rank.sort(dim=-1, descending=True, stable=True).indices  # ties: the lower slot first
    m = torch.minimum(n, torch.tensor(keep, device="cuda"))[:, None]  # slots kept of each sequence
    j = torch.arange(keep, device="cuda")
    top = order[..., :keep] if keep <= cap else torch.nn.functional.pad(order, (0, keep - cap))
    kept = torch.where(j < m, top, torch.full((), cap, device="cuda")).sort(dim=-1).values
    src = torch.where(j < m, kept, torch.zeros((), dtype=torch.int64, device="cuda"))
    row = src[..., None].expand(B, H, keep, D)
    live = (j < m).expand(B, H, keep)
    s["to_k"].copy_(torch.where(live[..., None], _tokens(s, s["k"]).gather(2, row), s["to_k"]))
    s["to_v"].copy_(torch.where(live[..., None], _tokens(s, s["v"]).gather(2, row), s["to_v"]))
    s["to_w"].copy_(torch.where(live, s["w"].gather(2, src), s["to_w"]))
    kept = torch.where(live, kept, torch.full((), -1, device="cuda", dtype=torch.int64)).to(torch.int32)
    return _evicted(s, kept)


def _evicted(s, kept):
    """Kept slots and, for each sequence's kept rows, the compacted cache and weights (rows past them zeroed)."""
    if not s["ragged"]:
        return kept, s["to_k"], s["to_v"], s["to_w"]
    live = (torch.arange(s["keep"], device="cuda") < s["lens"][:, None])[:, None]
    return (kept, torch.where(live[..., None], s["to_k"], 0), torch.where(live[..., None], s["to_v"], 0),
            torch.where(live, s["to_w"], 0))


# --------------------------------------------------------------------------- one pass


def run(state):
    s = state
    op = s["op"]
    if not own:
        if op == "evict":
            return _plain_evict(s)
        if op == "weights":
            return _plain_weights(s)
        if op == "append_attend":
            _plain_append(s)
            return _plain_attend(s), s["k"], s["v"]
        return _plain_attend(s)
    R = s["R"]
    if op == "evict":
        R.evict(s["p"], s["cache"], s["w"], s["keep"], s["kept"], into=s["into"], into_weights=s["to_w"],
                sinks=s["sinks"], recent=s["recent"])
        return _evicted(s, s["kept"])
    if op == "weights":
        R.accumulate_weights(s["p"], s["cache"], s["q"], s["w"], s["ws"], s["view"], accumulate=False)
        return s["w"]
    if op == "append_attend":
        s["cache"].length = s["length"] - s["queries"]
        R.dense_prefill_chunk(s["p"], s["cache"], s["k_new"], s["v_new"], s["q"], s["out"], s["ws"], s["view"])
        return s["out"], s["k"], s["v"]
    R.dense_attend(s["p"], s["cache"], s["q"], s["out"], s["ws"], s["view"])
    return s["out"]


# --------------------------------------------------------------------------- floors


def work(case):
    c = case
    B, H, G, L = c["batch"], c["kv"], c["group"], c["length"]
    mean = L * (0.5 + 0.5 / B) if c["ragged"] else float(L)  # expected tokens of a sequence
    if c["op"] == "evict":
        kept = min(float(c["keep"]), mean)
        return {"bytes": B * H * (mean * 4 + kept * (2 * 512 + 12)), "flops": 0.0}
    n = c["queries"]
    seen = mean - (n - 1) / 2.0 if c["causal"] else mean  # tokens a query sees, on average
    union = mean
    if c["window"]:
        seen = min(seen, float(c["window"] + c["sinks"]))
        union = min(union, float(c["window"] + c["sinks"] + (n - 1 if c["causal"] else 0)))
    seen = max(seen, 1.0)
    rows = B * n * H * G
    if c["op"] == "weights":
        return {"bytes": B * H * mean * (256 + 4) + rows * 256, "flops": rows * seen * 2 * D}
    extra = B * n * H * 1024 if c["op"] == "append_attend" else 0
    return {"bytes": B * H * union * 512 + rows * (256 + (512 if c["fp32"] else 256)) + extra,
            "flops": rows * seen * 4 * D}


# --------------------------------------------------------------------------- the definition, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    B, H, G = s["batch"], s["kv"], s["group"]
    lens = s["lens"].tolist()
    if s["op"] == "evict":
        return _exact_evict(s, lens)
    n, L = s["queries"], s["length"]
    freq = torch.tensor([BASE ** (-2.0 * i / D) for i in range(HALF)], dtype=torch.float64, device="cuda")

    def turn(x, pos):  # rotate rows x [m][128] to positions pos [m], as complex numbers
        z = torch.complex(x[:, :HALF], x[:, HALF:])
        a = pos.double()[:, None] * freq
        z = z * torch.polar(torch.ones_like(a), a)
        return torch.cat([z.real, z.imag], dim=1)

    if s["op"] == "append_attend":
        k_all, v_all = s["k"].clone(), s["v"].clone()
        k_all[:, :, L - n:L] = s["k_new"].permute(0, 2, 1, 3)
        v_all[:, :, L - n:L] = s["v_new"].permute(0, 2, 1, 3)
    w = torch.zeros(B, H, s["cap"], dtype=torch.float64, device="cuda") if s["op"] == "weights" else None
    out = None if w is not None else torch.zeros(B, n, H * G, D, dtype=torch.float64, device="cuda")
    step = max(1, min(n, int(1.5e9 / (8 * G * L))))
    for b in range(B):
        m = lens[b]
        for h in range(H):
            if s["op"] == "append_attend":
                k, v = k_all[b, h, :m].double(), v_all[b, h, :m].double()
            elif s["table"] is None:
                k, v = s["k"][b, h, :m].double(), s["v"][b, h, :m].double()
            else:
                pages = s["table"][b].long()
                k = s["k"][pages, h].reshape(-1, D)[:m].double()
                v = s["v"][pages, h].reshape(-1, D)[:m].double()
            t = torch.arange(m, device="cuda")
            kr = turn(k, t)
            for i0 in range(0, n, step):
                i1 = min(n, i0 + step)
                p = torch.full((i1 - i0,), m, dtype=torch.int64, device="cuda")
                if s["causal"]:
                    p = torch.arange(m - n + i0 + 1, m - n + i1 + 1, device="cuda")
                p = p.repeat_interleave(G)
                q = s["q"][b, i0:i1, h * G:(h + 1) * G].double().reshape(-1, D)
                x = turn(q, p) @ kr.T * SCALE
                see = t[None] < p[:, None]
                if s["window"]:
                    far = t[None] < p[:, None] - s["window"]
                    sink = (t < s["sinks"])[None]
                    at = torch.clamp(p, max=s["sinks"] + s["window"])
                    x = torch.where(far & sink, turn(q, at) @ kr.T * SCALE, x)
                    see = see & (~far | sink)
                x = torch.where(see, x, torch.full_like(x, -math.inf))
                e = torch.softmax(x, dim=1)
                e = torch.where(see.any(1, keepdim=True), e, torch.zeros_like(e))
                if w is not None:
                    w[b, h, :m] += e.sum(0)
                else:
                    out[b, i0:i1, h * G:(h + 1) * G] = (e @ v).view(i1 - i0, G, D)
                del x, e, see
    if w is not None:
        return w
    if s["op"] == "append_attend":
        return out, k_all.double(), v_all.double()
    return out


def _exact_evict(s, lens):
    B, H, keep = s["batch"], s["kv"], s["keep"]
    kept = torch.full((B, H, keep), -1, dtype=torch.int32, device="cuda")
    k = torch.zeros(B, H, keep, D, dtype=torch.float64, device="cuda")
    v, w = torch.zeros_like(k), torch.zeros(B, H, keep, dtype=torch.float64, device="cuda")
    for b in range(B):
        m = lens[b]
        for h in range(H):
            free = torch.arange(min(s["sinks"], m), max(m - s["recent"], min(s["sinks"], m)), device="cuda")
            sure = torch.ones(m, dtype=torch.bool, device="cuda")
            sure[free] = False
            room = min(keep, m) - int(sure.sum())
            best = free[torch.argsort(s["w"][b, h, free].double(), descending=True, stable=True)[:room]]
            sure[best] = True
            at = sure.nonzero()[:, 0]
            c = at.numel()
            kept[b, h, :c] = at.int()
            if s["table"] is None:
                kk, vv = s["k"][b, h], s["v"][b, h]
            else:
                pages = s["table"][b].long()
                kk, vv = s["k"][pages, h].reshape(-1, D), s["v"][pages, h].reshape(-1, D)
            k[b, h, :c], v[b, h, :c], w[b, h, :c] = kk[at].double(), vv[at].double(), s["w"][b, h, at].double()
    return kept, k, v, w
