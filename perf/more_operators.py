"""The operators of a grouped-query layer in the paged serving step, as measured cases: the append
of new keys and values to a cache held in 8 bits with a scale for each block of tokens and head,
the read-back of that cache, the scores of its blocks from their mean keys, and the attention of
new tokens over all that they see or over the blocks selected for them.

Each case is one call of one operator.  Where ``own`` is false ``run`` computes the plain form
in elementary torch operations (32 bits, rounded once at the end); where it is true it calls
the framework's entry points.
"""
import math

import torch

own = False
DEV = "cuda"
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
DT = {"bf16": BF16, "f32": F32}
SIZE = {"bf16": 2, "f32": 4}
E_MIN = -64                     # least exponent of a scale


# ------------------------------------------------------------------ cases
def _case(name, op, B, Hq, Hkv, ps, ctx, new, D=128, dt="bf16", **more):
    return dict(name=name, op=op, B=B, Hq=Hq, Hkv=Hkv, D=D, dt=dt, page_size=ps, ctx_lo=ctx[0],
                ctx_hi=ctx[1], new_lo=new[0], new_hi=new[1], **more)


def listed():
    return [
        # a decode step's 64 new tokens into partly filled blocks: latency
        _case("append_decode", "append", 64, 64, 8, 64, (100, 16000), (1, 1)),
        # a large prefill step's keys and values, ragged prompts that begin and end inside blocks
        _case("append_chunk", "append", 24, 64, 8, 64, (0, 5000), (500, 4900)),
        # one request's prefix brought back to 16 bits, an odd length
        _case("read_prefix", "read", 1, 32, 4, 16, (0, 0), (1001, 1001)),
        # prefixes of a batch brought back for a pass over plain keys and values
        _case("read_batch", "read", 12, 64, 8, 64, (0, 0), (900, 9000)),
        # which blocks a decode step's tokens look at, on the longest contexts
        _case("scores_decode", "scores", 4, 64, 8, 64, (262100, 262143), (1, 1), sink_blocks=1,
              local_blocks=2),
        # the same for every token of a prompt chunk
        _case("scores_chunk", "scores", 1, 64, 4, 64, (14336, 14336), (2048, 2048),
              sink_blocks=1, local_blocks=2),
        # one request's decode token on a short context: latency
        _case("attend_one", "attend", 1, 64, 8, 16, (256, 256), (1, 1), window=0, sinks=0, K=0),
        # a decode batch on ragged contexts
        _case("attend_decode", "attend", 64, 64, 8, 64, (4096, 16000), (1, 1), window=0, sinks=0,
              K=0),
        # a prompt chunk on a long context
        _case("attend_chunk", "attend", 1, 64, 4, 64, (14336, 14336), (2048, 2048), window=0,
              sinks=0, K=0),
        # a local layer in a mixed step: prompt chunks beside decodes, window and first tokens
        _case("attend_window", "attend", 16, 32, 8, 32, (0, 8000), (1, 250), window=1024, sinks=4,
              K=0),
        # decode tokens on the longest contexts, each KV head on its 32 selected blocks
        _case("attend_blocks_decode", "attend", 4, 64, 8, 64, (262100, 262143), (1, 1), window=0,
              sinks=0, K=32),
        # every token of a prompt chunk on its own 32 blocks
        _case("attend_blocks_chunk", "attend", 1, 64, 4, 64, (14336, 14336), (1024, 1024),
              window=0, sinks=0, K=32),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "read", "scores", "scores", "attend", "attend", "attend",
                     "blocks", "blocks"])
    D = rng.choice([128, 128, 128, 64])
    Hkv = rng.choice([1, 2, 4, 4, 8, 8])
    G = rng.choice([g for g in (1, 2, 4, 5, 8, 8, 16) if g * Hkv <= 128])
    ps = rng.choice([16, 32, 48, 64, 64, 128])
    dt = rng.choice(["bf16"] * 5 + ["f32"])
    head = dict(Hq=G * Hkv, Hkv=Hkv, D=D, dt=dt, page_size=ps)
    if op in ("append", "read"):
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, 60000 // B))
        ctx = 0 if op == "read" else _log(rng, 1, 8000) - 1
        return dict(head, op=op, B=B, ctx_lo=ctx // 3, ctx_hi=ctx, new_lo=max(1, hi // 9),
                    new_hi=hi)
    kind = rng.choice(["decode", "decode", "chunk", "mixed", "tiny"])
    if kind == "tiny" or dt == "f32":
        head |= dict(D=rng.choice([64, 32, 80]), dt="f32", page_size=16)
        B, ctx, new = rng.randint(1, 3), (0, _log(rng, 1, 256)), (1, _log(rng, 1, 100))
    elif kind == "decode":
        B, top = _log(rng, 1, 48), _log(rng, 16, 16000)
        ctx, new = (max(1, top // 4), top), (1, rng.choice([1, 1, 1, 2, 3]))
    elif kind == "chunk":
        n, top = _log(rng, 16, 1024), _log(rng, 1, 8192)
        B, ctx, new = 1, (top, top), (n, n)
    else:
        B, ctx, new = _log(rng, 2, 16), (0, _log(rng, 16, 6000)), (1, _log(rng, 2, 200))
    if op == "blocks" and B * new[1] * Hkv > 4096:
        new = (1, max(1, 4096 // (B * Hkv)))
    head |= dict(B=B, ctx_lo=ctx[0], ctx_hi=ctx[1], new_lo=new[0], new_hi=new[1])
    if op == "scores":
        return dict(head, op="scores", sink_blocks=rng.choice([0, 1, 2]),
                    local_blocks=rng.choice([0, 1, 4]))
    if op == "blocks":
        return dict(head, op="attend", window=0, sinks=0, K=_log(rng, 1, max(1, 2048 // ps)))
    window, sinks = rng.choice([(0, 0), (0, 0), (_log(rng, 64, 1024), rng.choice([0, 4, 130]))])
    return dict(head, op="attend", window=window, sinks=sinks, K=0)


def _lengths(case):
    """The requests' lengths: part of the case (every seed has the same ones), spread over the
    case's ranges by a fixed rule, long and short mixed."""
    B = case["B"]

    def spread(lo, hi, mul):
        return [lo + (b * mul + mul // 2) % B * (hi - lo) // max(1, B - 1) if B > 1 else hi
                for b in range(B)]
    ctx = spread(case["ctx_lo"], case["ctx_hi"], 7)
    new = spread(case["new_lo"], case["new_hi"], 5)
    if case["op"] == "attend" and case["new_hi"] > 1 and B > 2:   # decodes beside the chunks
        new = [1 if b % 3 == 2 else n for b, n in enumerate(new)]
    return ctx, new


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op, ps, B, Hq, Hkv, D = (case[k] for k in ("op", "page_size", "B", "Hq", "Hkv", "D"))
    ctx, new = _lengths(case)
    total = [c + n for c, n in zip(ctx, new)]
    blocks = [-(-t // ps) for t in total]
    n_pages, T, dt = sum(blocks) + 3, sum(new), DT[case["dt"]]

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=DEV) * std

    p = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, max(blocks) + 1), -1, dtype=torch.int32, device=DEV)
    col = torch.arange(table.shape[1], device=DEV)
    first = i32([0] + blocks).long().cumsum(0)[:-1]
    held = col[None, :] < i32(blocks)[:, None]
    table[held] = p[(first[:, None] + col[None, :])[held]]
    cu = [0]
    for k in new:
        cu.append(cu[-1] + k)
    s = dict(case=case, table=table, seq_lens=i32(total), cu_new=i32(cu), n_max=max(new),
             s_max=max(total), sm_scale=1.0 / math.sqrt(D))

    def cache(std):
        """Codes of normal rows, some heads and blocks larger than others, with the scales of
        their largest elements; page by page in bounded pieces."""
        codes = torch.empty((n_pages, Hkv, ps, D), dtype=E4M3, device=DEV)
        scale = torch.empty((n_pages, Hkv), device=DEV)
        for lo in range(0, n_pages, 8192):
            x = normal(min(8192, n_pages - lo), Hkv, ps, D, std=std)
            x *= torch.exp2(normal(x.shape[0], Hkv, 1, 1, std=0.5))
            c, e = _quantise(x, x.abs().amax((2, 3)))
            codes[lo:lo + 8192], scale[lo:lo + 8192] = c, torch.exp2(e)
        return codes, scale

    if op == "scores":
        # means of 64 keys or so, some far from zero: keys have a common part
        mean = normal(n_pages, Hkv, D, std=0.4) + normal(1, Hkv, D, std=0.5)
        s |= dict(k_mean=mean.to(BF16), q=normal(T, Hq, D, std=2.0).to(dt),
                  scores=torch.zeros((T, Hkv, table.shape[1]), device=DEV))
        return s
    s["k_pages"], s["k_scale"] = cache(1.0)
    s["v_pages"], s["v_scale"] = cache(0.7)
    if op == "append":
        # some tokens are larger than what their block holds: scales grow
        up = torch.exp2(normal(T, Hkv, 1, std=0.7))
        s |= dict(k_new=(normal(T, Hkv, D) * up).to(dt),
                  v_new=(normal(T, Hkv, D, std=0.7) * up).to(dt),
                  k_mean=normal(n_pages, Hkv, D, std=0.4).to(BF16))
        return s
    if op == "read":
        s |= dict(k_out=torch.zeros((T, Hkv, D), dtype=dt, device=DEV),
                  v_out=torch.zeros((T, Hkv, D), dtype=dt, device=DEV))
        return s
    s |= dict(q=normal(T, Hq, D, std=2.0).to(dt),
              out=torch.zeros((T, Hq, D), dtype=dt, device=DEV),
              lse=torch.zeros((T, Hq), dtype=F32, device=DEV), block_ids=None,
              ws=torch.empty(128 << 20, dtype=torch.uint8, device=DEV))
    if case["K"]:
        # each token's own block, then others of those before it, in no order; -1 where it has
        # too few
        pos = torch.cat([torch.arange(c, c + n, device=DEV) for c, n in zip(ctx, new)])
        mine = (pos // ps)[:, None, None]
        nb = table.shape[1]
        key = torch.rand((T, Hkv, nb), generator=g, device=DEV)
        key = torch.where(col < mine, key, torch.where(col == mine, 2.0, -1.0))
        top, ids = key.topk(min(case["K"], nb), -1)
        ids = torch.where(top >= 0, ids, -1).to(torch.int32)
        pad = ids.new_full((T, Hkv, case["K"] - ids.shape[2]), -1)
        s["block_ids"] = torch.cat([ids, pad], -1).contiguous()
    return s


def _quantise(x, largest):
    """Codes of x [n, Hkv, ps, D] and the exponent [n, Hkv] of their scale: the least (E_MIN at
    least) with ``largest`` within 448 of it."""
    m, e = torch.frexp(largest)
    e = torch.where(m <= 0.875, e - 9, e - 8).float()              # 448 = 0.875 * 2^9
    e = torch.where(largest > 0, e.clamp(min=E_MIN), float(E_MIN))
    return (x * torch.exp2(-e)[..., None, None]).to(E4M3), e


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return {"append": _own_append, "read": _own_read, "scores": _own_scores,
                "attend": _own_attend}[op](s)
    if op == "attend":
        return _attend_blocks(s) if s["case"]["K"] else _attend(s)
    return {"append": _append, "read": _read, "scores": _scores}[op](s)


def _own_append(s):
    from sparse_attention_indexer_kpool_gb300 import ops
    ops.dsa_gqa_append(s["k_new"], s["v_new"], s["k_pages"], s["v_pages"], s["k_scale"],
                       s["v_scale"], s["table"], s["seq_lens"], s["cu_new"], k_mean=s["k_mean"])
    return s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["k_mean"]


def _own_read(s):
    from sparse_attention_indexer_kpool_gb300 import ops
    ops.dsa_gqa_read(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["table"],
                     s["seq_lens"], s["cu_new"], s["k_out"], s["v_out"])
    return s["k_out"], s["v_out"]


def _own_scores(s):
    from sparse_attention_indexer_kpool_gb300 import ops
    c = s["case"]
    ops.dsa_gqa_block_scores(s["q"], s["k_mean"], s["table"], s["seq_lens"], c["page_size"],
                             s["cu_new"], c["sink_blocks"], c["local_blocks"], s["sm_scale"],
                             s["scores"])
    return s["scores"]


def _own_attend(s):
    from sparse_attention_indexer_kpool_gb300 import ops
    c = s["case"]
    ops.dsa_gqa_attend(s["q"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["table"],
                       s["seq_lens"], s["cu_new"], c["window"], c["sinks"], s["sm_scale"],
                       s["out"], s["lse"], s["ws"], block_ids=s["block_ids"])
    return s["out"], s["lse"]


def _append(s):
    ps = s["case"]["page_size"]
    cu, lens = s["cu_new"].long(), s["seq_lens"].long()
    n = cu[1:] - cu[:-1]
    ctx = lens - n
    # the blocks that the step touches, [B, most of them], and the positions in them
    most = (s["n_max"] - 1) // ps + 2
    blk = ctx[:, None] // ps + torch.arange(most, device=DEV)
    seq, i = torch.nonzero((blk * ps < lens[:, None]) & (n > 0)[:, None], as_tuple=True)
    blk = blk[seq, i]
    page = s["table"].long()[seq, blk]
    pos = blk[:, None] * ps + torch.arange(ps, device=DEV)
    old = pos < ctx[seq, None]
    fresh = ~old & (pos < lens[seq, None])
    src = torch.where(fresh, cu[seq, None] + pos - ctx[seq, None], 0)
    whole = (blk + 1) * ps <= lens[seq]

    def write(new, pages, scale):
        x = torch.where(fresh[:, None, :, None], new[src].float().transpose(1, 2), 0.0)
        finite = torch.isfinite(x)
        _, e = _quantise(x[:, :, :0], torch.where(finite, x.abs(), 0.0).amax((2, 3)))
        before = torch.where(old.any(1)[:, None], torch.frexp(scale[page])[1].float() - 1.0,
                             float(E_MIN))
        e = torch.maximum(e, before)
        x = torch.where(finite, x * torch.exp2(-e)[..., None, None], float("nan"))
        held = pages.view(torch.uint8)[page]
        moved = held.view(E4M3).float() * torch.exp2(before - e)[..., None, None]
        codes = torch.where(old[:, None, :, None], moved, x).to(E4M3).view(torch.uint8)
        codes = torch.where((old | fresh)[:, None, :, None], codes, held)
        pages, scale = pages.view(torch.uint8).clone(), scale.clone()
        pages[page], scale[page] = codes, torch.exp2(e)
        return pages.view(E4M3), scale, codes.view(E4M3).float(), torch.exp2(e)

    k_pages, k_scale, codes, up = write(s["k_new"], s["k_pages"], s["k_scale"])
    v_pages, v_scale, _, _ = write(s["v_new"], s["v_pages"], s["v_scale"])
    mean = (codes.sum(2) * (up / ps)[..., None]).to(BF16)
    k_mean = s["k_mean"].clone()
    k_mean[page[whole]] = mean[whole]
    return k_pages, v_pages, k_scale, v_scale, k_mean


def _read(s):
    ps = s["case"]["page_size"]
    cu, t = s["cu_new"].long(), torch.arange(s["k_out"].shape[0], device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = t - cu[seq]
    page = s["table"].long()[seq, pos // ps]

    def get(pages, scale):
        codes = pages.view(torch.uint8)[page, :, pos % ps].view(E4M3).float()
        return (codes * scale[page][..., None]).to(DT[s["case"]["dt"]])
    return get(s["k_pages"], s["k_scale"]), get(s["v_pages"], s["v_scale"])


def _tokens(s):
    """Sequence and position of every new token."""
    cu, lens = s["cu_new"].long(), s["seq_lens"].long()
    t = torch.arange(s["q"].shape[0], device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return seq, lens[seq] - cu[seq + 1] + t


def _scores(s):
    c = s["case"]
    ps, Hkv, D = c["page_size"], c["Hkv"], c["D"]
    (T, Hq, _), (B, nb) = s["q"].shape, s["table"].shape
    cu, lens = s["cu_new"].long(), s["seq_lens"].long()
    n, n_max = cu[1:] - cu[:-1], s["n_max"]
    i = torch.arange(n_max, device=DEV)
    live = i[None, :] < n[:, None]
    src = torch.where(live, cu[:-1, None] + i[None, :], 0)
    q = s["q"][src].float().view(B, n_max, Hkv, Hq // Hkv, D)
    q = q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    means = s["k_mean"][s["table"].long().clamp(min=0)].float()    # [B, nb, Hkv, D]
    z = (q @ means.permute(0, 2, 3, 1)).view(B, Hkv, n_max, Hq // Hkv, nb) * s["sm_scale"]
    pos = (lens - n)[:, None] + i[None, :]                         # [B, n_max]
    blk = torch.arange(nb, device=DEV)
    see = ((blk * ps + ps - 1) <= pos[..., None])[:, None, :, None, :]
    z = z.masked_fill(~see, -math.inf)
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    total = e.sum(-1, keepdim=True)
    mass = torch.where(total > 0, e / total, 0.0).sum(3)           # [B, Hkv, n_max, nb]
    mine = (pos // ps)[:, None, :, None]
    forced = (blk <= mine) & ((blk < c["sink_blocks"]) | (blk > mine - c["local_blocks"]))
    mass = torch.where(see[:, :, :, 0], mass, -math.inf).masked_fill(forced, math.inf)
    return mass.transpose(1, 2)[live]                              # [T, Hkv, nb]


def _attend(s):
    c = s["case"]
    ps, Hq, Hkv, D = c["page_size"], c["Hq"], c["Hkv"], c["D"]
    T, B, n_max, s_max = s["q"].shape[0], s["table"].shape[0], s["n_max"], s["s_max"]
    cu, lens = s["cu_new"].long(), s["seq_lens"].long()
    n, G = cu[1:] - cu[:-1], Hq // Hkv
    # the sequences' keys and values, padded to the longest
    pos = torch.arange(s_max, device=DEV)
    page = s["table"].long()[:, pos // ps].clamp(min=0)
    held = (pos[None, :] < lens[:, None])[..., None, None]

    def rows(pages, scale):                                        # [B * Hkv, s_max, D]
        x = pages.view(torch.uint8)[page, :, pos % ps].view(E4M3).float() * scale[page][..., None]
        return torch.where(held, x, 0.0).transpose(1, 2).reshape(B * Hkv, s_max, D)
    # the new tokens' queries, padded to the most of them
    i = torch.arange(n_max, device=DEV)
    live = i[None, :] < n[:, None]
    src = torch.where(live, cu[:-1, None] + i[None, :], 0)
    q = s["q"][src].float().view(B, n_max, Hkv, G, D).transpose(1, 2).reshape(B * Hkv, -1, D)
    z = torch.bmm(q, rows(s["k_pages"], s["k_scale"]).transpose(1, 2))
    z = z.view(B, Hkv, n_max, G, s_max).mul_(s["sm_scale"])
    at = (lens - n)[:, None] + i[None, :]
    see = pos <= at[..., None]
    if c["window"]:
        see &= (pos > at[..., None] - c["window"]) | (pos < c["sinks"])
    z.masked_fill_(~(see & live[..., None])[:, None, :, None, :], -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = z.sub_(m).exp_()
    total = e.sum(-1, keepdim=True)
    o = torch.bmm(e.view(B * Hkv, n_max * G, s_max), rows(s["v_pages"], s["v_scale"]))
    o = torch.where(total > 0, o.view(B, Hkv, n_max, G, D) / total, 0.0)
    lse = (m + total.log()).squeeze(-1)                            # [B, Hkv, n_max, G]
    return (o.transpose(1, 2)[live].reshape(T, Hq, D).to(s["q"].dtype),
            lse.transpose(1, 2)[live].reshape(T, Hq))


def _attend_blocks(s):
    c = s["case"]
    ps, Hq, Hkv, D = c["page_size"], c["Hq"], c["Hkv"], c["D"]
    T, ids = s["q"].shape[0], s["block_ids"].long()
    seq, at = _tokens(s)
    page = s["table"].long()[seq[:, None, None], ids.clamp(min=0)]
    pos = (ids[..., None] * ps + torch.arange(ps, device=DEV)).flatten(2)
    see = (pos <= at[:, None, None]) & (ids >= 0).repeat_interleave(ps, -1)
    head = torch.arange(Hkv, device=DEV)[None, :, None]

    def rows(pages, scale):                                        # [T, Hkv, K * ps, D]
        x = pages.view(torch.uint8)[page, head].view(E4M3).float()
        x *= scale[page, head][..., None, None]
        return x.flatten(2, 3).masked_fill_(~see[..., None], 0.0)
    q = s["q"].float().view(T, Hkv, Hq // Hkv, D)
    z = (q @ rows(s["k_pages"], s["k_scale"]).transpose(2, 3)) * s["sm_scale"]
    z = z.masked_fill(~see[:, :, None, :], -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = torch.exp(z - m)
    total = e.sum(-1, keepdim=True)
    o = torch.where(total > 0, (e @ rows(s["v_pages"], s["v_scale"])) / total, 0.0)
    return o.reshape(T, Hq, D).to(s["q"].dtype), (m + total.log()).reshape(T, Hq)


# ------------------------------------------------------------------ what a pass cannot do without
def _visible(case):
    """(new token, key) pairs per KV head, and keys that some new token sees."""
    ctx, new = _lengths(case)
    W, S, K, ps = case.get("window", 0), case.get("sinks", 0), case.get("K", 0), case["page_size"]
    pairs = rows = 0
    for c, n in zip(ctx, new):
        seen = 0
        for i in range(n):
            p = c + i
            if K:
                seen += min(K - 1, p // ps) * ps + p % ps + 1
            else:
                lo = max(0, p - W + 1) if W else 0
                seen += p + 1 - lo + min(S, lo)
        pairs += seen
        lo = max(0, c - W + 1) if W else 0
        rows += min(seen, c + n - lo + min(S, lo))
    return pairs, rows


def work(case):
    ctx, new = _lengths(case)
    Hq, Hkv, D, ps, size = case["Hq"], case["Hkv"], case["D"], case["page_size"], SIZE[case["dt"]]
    T = sum(new)
    if case["op"] == "append":
        touched = sum(-(-(c + n) // ps) - c // ps for c, n in zip(ctx, new))
        whole = sum((c + n) // ps - c // ps for c, n in zip(ctx, new))
        return dict(bytes=Hkv * (2 * T * D * (size + 1) + 8 * touched + 2 * whole * D), flops=0)
    if case["op"] == "read":
        touched = sum(-(-n // ps) for n in new)
        return dict(bytes=Hkv * (2 * T * D * (size + 1) + 8 * touched), flops=0)
    if case["op"] == "scores":
        nb = max(-(-(c + n) // ps) for c, n in zip(ctx, new)) + 1
        pairs = sum((c + i + 1) // ps for c, n in zip(ctx, new) for i in range(n))
        means = sum((c + n) // ps for c, n in zip(ctx, new))
        return dict(bytes=2 * means * Hkv * D + T * Hq * D * size + 4 * T * Hkv * nb,
                    flops=2 * pairs * Hq * D)
    pairs, rows = _visible(case)
    return dict(bytes=Hkv * (rows * 2 * D + 8 * -(-rows // ps)) + T * Hq * (2 * D * size + 4)
                + 4 * T * Hkv * case["K"], flops=4 * pairs * Hq * D)


# ------------------------------------------------------------------ 64 bits
def _two(e):
    """2^e in 64 bits, exactly (the 32-bit function is exact at whole numbers)."""
    return torch.exp2(e.float()).double()


def _grid(x):
    """The E4M3 value nearest to x (64 bits; ties to the even code), |x| <= 448."""
    e = (torch.frexp(x)[1] - 1).clamp(min=-6).double()
    step = _two(e - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    op, ps, Hq, Hkv, D = (case[k] for k in ("op", "page_size", "Hq", "Hkv", "D"))
    ctx, new = _lengths(case)
    G = Hq // Hkv
    if op == "attend" and 4 * _visible(dict(case, window=0))[0] * Hq * D > 6e12:
        return None
    s = prepare(case, seed)
    table = s["table"].tolist()
    if op == "append":
        def write(new_rows, pages, scale):
            pages, scale = pages.double(), scale.double()
            at = 0
            for b, (c, n) in enumerate(zip(ctx, new)):
                for j in range(c // ps, -(-(c + n) // ps)):
                    lo, hi = max(c, j * ps), min(c + n, j * ps + ps)
                    x = new_rows[at + lo - c:at + hi - c].double().transpose(0, 1)
                    a = x.abs().amax((1, 2))
                    e = torch.ceil(torch.log2(a / 448.0)).clamp(min=E_MIN)
                    e = torch.where(a > 448.0 * _two(e), e + 1, e)
                    e = torch.where(a <= 448.0 * _two(e - 1), e - 1, e).clamp(min=E_MIN)
                    pg, o = table[b][j], lo - j * ps
                    if o:
                        before = torch.log2(scale[pg]).round()
                        e = torch.maximum(e, before)
                        up = _two(before - e)[:, None, None]
                        pages[pg, :, :o] = _grid(pages[pg, :, :o] * up)
                    pages[pg, :, o:o + hi - lo] = _grid(x / _two(e)[:, None, None])
                    scale[pg] = _two(e)
                at += n
            return pages, scale
        if sum(new) > 70000:
            return None
        k_pages, k_scale = write(s["k_new"], s["k_pages"], s["k_scale"])
        v_pages, v_scale = write(s["v_new"], s["v_pages"], s["v_scale"])
        mean = s["k_mean"].double()
        for b, (c, n) in enumerate(zip(ctx, new)):
            pg = torch.tensor(table[b][c // ps:(c + n) // ps], dtype=torch.long, device=DEV)
            mean[pg] = k_pages[pg].mean(2) * k_scale[pg][..., None]
        return k_pages, v_pages, k_scale, v_scale, mean

    def rows(pages, scale, b, t):                                  # [Hkv, positions, D]
        pg = s["table"][b].long()[t // ps]
        x = pages.view(torch.uint8)[pg, :, t % ps].view(E4M3).double()
        return (x * scale[pg].double()[..., None]).transpose(0, 1)
    if op == "read":
        t = [torch.arange(n, device=DEV) for n in new]
        return tuple(torch.cat([rows(s[a + "_pages"], s[a + "_scale"], b, t[b]).transpose(0, 1)
                                for b in range(len(new))]) for a in "kv")
    if op == "scores":
        nb = s["table"].shape[1]
        out = torch.full((sum(new), Hkv, nb), -math.inf, dtype=torch.float64, device=DEV)
        at = 0
        for b, (c, n) in enumerate(zip(ctx, new)):
            q = s["q"][at:at + n].double().view(n, Hkv, G, D).transpose(0, 1).reshape(Hkv, -1, D)
            k = s["k_mean"][s["table"][b].long().clamp(min=0)].double().permute(1, 2, 0)
            z = (q @ k).view(Hkv, n, G, nb) * s["sm_scale"]
            p = c + torch.arange(n, device=DEV)
            done = torch.arange(nb, device=DEV)[None, :] < ((p + 1) // ps)[:, None]
            z = z.masked_fill(~done[None, :, None, :], -math.inf)
            mass = torch.softmax(z, -1).nan_to_num(0.0).sum(2).transpose(0, 1)
            got = torch.where(done[:, None, :], mass, -math.inf)
            i, at_blk = torch.arange(nb, device=DEV)[None, :], (p // ps)[:, None]
            near = (at_blk >= i) & ((i < case["sink_blocks"]) | (at_blk < i + case["local_blocks"]))
            out[at:at + n] = got.masked_fill(near[:, None, :], math.inf)
            at += n
        return out
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    at = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        t = torch.arange(c + n, device=DEV)
        if case["K"]:
            t = torch.arange(-(-(c + n) // ps) * ps, device=DEV)
        k, v = rows(s["k_pages"], s["k_scale"], b, t), rows(s["v_pages"], s["v_scale"], b, t)
        step = max(1, min(128, (1 << 27) // (len(t) * Hq)))
        for lo in range(0, n, step):
            hi = min(n, lo + step)
            p = c + torch.arange(lo, hi, device=DEV)
            q = s["q"][at + lo:at + hi].double().view(hi - lo, Hkv, G, D)
            z = torch.einsum("thgd,hsd->thgs", q, k) * s["sm_scale"]
            hide = (t[None, :] > p[:, None])[:, None, :]
            if case["window"]:
                hide = hide | ((t[None, :] <= p[:, None] - case["window"])
                               & (t[None, :] >= case["sinks"]))[:, None, :]
            if case["K"]:
                ids = s["block_ids"][at + lo:at + hi].long()
                listed_at = torch.zeros((hi - lo, Hkv, len(t) // ps + 1), device=DEV)
                listed_at.scatter_(2, torch.where(ids < 0, len(t) // ps, ids), 1.0)
                hide = hide | (listed_at[..., :-1].repeat_interleave(ps, -1) == 0)
            z = z.masked_fill(hide[:, :, None, :], -math.inf)
            lse[at + lo:at + hi] = torch.logsumexp(z, -1).reshape(hi - lo, Hq)
            w = torch.softmax(z, -1).nan_to_num(0.0)
            out[at + lo:at + hi] = torch.einsum("thgs,hsd->thgd", w, v).reshape(hi - lo, Hq, D)
        at += n
    return out, lse
