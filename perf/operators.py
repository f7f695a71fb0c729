"""The paged serving step's operators as measured cases: the step plan (block tables and slot
maps from request lengths), the append of new latent rows to the paged cache, and the
attention of the new tokens over that cache (causal, optionally a sliding window and sinks).

Each case is one call of one operator.  Where ``own`` is false ``run`` computes the plain form
in elementary torch operations (32 bits, rounded once at the end); where it is true it calls
the framework's entry points.
"""
import math

import torch

own = False
DEV = "cuda"
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
DT = {"bf16": BF16, "f32": F32, "e4m3": E4M3}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the plan of a decode step: 64 running requests, one new token each
        dict(name="plan_decode", op="plan", B=64, T=64, page_size=64, ctx_lo=100, ctx_hi=65536,
             new_lo=1, new_hi=1, pad=0, keys=True),
        # the plan of a mixed step: 512 requests, chunks of prompts beside decodes, padded to a
        # fixed token count as a captured step has it
        dict(name="plan_mixed", op="plan", B=512, T=65536, page_size=16, ctx_lo=0, ctx_hi=4096,
             new_lo=1, new_hi=240, pad=1000, keys=False),
        # a decode step's 64 new rows into a bf16 cache
        dict(name="append_decode_bf16", op="append", T=64, L=512, dt="bf16", kv="bf16",
             page_size=64, drop=0),
        # a prefill step's rows into a bf16 cache, an odd number, some dropped (padding)
        dict(name="append_chunk_bf16", op="append", T=16383, L=512, dt="bf16", kv="bf16",
             page_size=16, drop=37),
        # a large prefill step's rows quantised into an E4M3 cache
        dict(name="append_chunk_e4m3", op="append", T=65536, L=512, dt="bf16", kv="e4m3",
             page_size=64, drop=0),
        # the fp32 verification geometry: 4 heads of latent 64, a short prompt in one chunk
        dict(name="attend_f32_tiny", op="attend", B=1, Hm=4, L=64, dt="f32", kv="f32",
             page_size=16, ctx_lo=0, ctx_hi=0, new_lo=200, new_hi=200, window=0, sinks=0),
        # one request's decode token on a short context: latency
        dict(name="attend_decode_one", op="attend", B=1, Hm=64, L=512, dt="bf16", kv="bf16",
             page_size=64, ctx_lo=256, ctx_hi=256, new_lo=1, new_hi=1, window=0, sinks=0),
        # a decode batch on ragged contexts
        dict(name="attend_decode_bf16", op="attend", B=64, Hm=64, L=512, dt="bf16", kv="bf16",
             page_size=64, ctx_lo=4096, ctx_hi=16000, new_lo=1, new_hi=1, window=0, sinks=0),
        # the same with a quarter of the heads (a tensor-parallel share) on an E4M3 cache
        dict(name="attend_decode_e4m3", op="attend", B=64, Hm=16, L=512, dt="bf16", kv="e4m3",
             page_size=16, ctx_lo=4096, ctx_hi=16000, new_lo=1, new_hi=1, window=0, sinks=0),
        # a prompt chunk on a long context
        dict(name="attend_chunk_bf16", op="attend", B=1, Hm=64, L=512, dt="bf16", kv="bf16",
             page_size=64, ctx_lo=14336, ctx_hi=14336, new_lo=2048, new_hi=2048, window=0,
             sinks=0),
        # a mixed step: prompt chunks of many sizes beside decode tokens, E4M3 cache
        dict(name="attend_mixed_e4m3", op="attend", B=12, Hm=64, L=512, dt="bf16", kv="e4m3",
             page_size=64, ctx_lo=0, ctx_hi=5000, new_lo=1, new_hi=300, window=0, sinks=0),
        # a local layer: sliding window with the first tokens visible, chunks beside decodes
        dict(name="attend_window_bf16", op="attend", B=16, Hm=64, L=512, dt="bf16", kv="bf16",
             page_size=32, ctx_lo=0, ctx_hi=8000, new_lo=1, new_hi=128, window=512, sinks=4),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "append", "attend", "attend", "attend", "attend"])
    ps = rng.choice([16, 32, 48, 64])
    if op == "plan":
        B = _log(rng, 1, 1024)
        hi = max(1, min(240, 60000 // B))
        new, pad = _log(rng, 1, hi), _log(rng, 1, 2000) - 1
        return dict(op="plan", B=B, T=B * new + pad, page_size=ps, ctx_lo=0,
                    ctx_hi=_log(rng, 1, 65536), new_lo=1, new_hi=new, pad=pad,
                    keys=rng.random() < 0.5)
    if op == "append":
        T = _log(rng, 1, 65536)
        return dict(op="append", T=T, L=512, dt="bf16", kv=rng.choice(["bf16", "e4m3"]),
                    page_size=ps, drop=rng.randint(0, T // 8))
    kind = rng.choice(["decode", "decode", "chunk", "mixed", "tiny"])
    if kind == "tiny":
        n = _log(rng, 1, 256)
        return dict(op="attend", B=rng.randint(1, 3), Hm=4, L=64, dt="f32", kv="f32",
                    page_size=16, ctx_lo=0, ctx_hi=_log(rng, 1, 256), new_lo=1, new_hi=n,
                    window=rng.choice([0, 0, 40]), sinks=rng.choice([0, 3]))
    Hm = rng.choice([16, 32, 64, 64, 64, 128])
    kv = rng.choice(["bf16", "e4m3"])
    window, sinks = rng.choice([(0, 0), (0, 0), (_log(rng, 64, 1024), rng.choice([0, 4, 130]))])
    if kind == "decode":
        B = _log(rng, 1, 64)
        top = _log(rng, 16, 16000)
        ctx, new = [max(1, top // 4), top], [1, rng.choice([1, 1, 1, 2, 3])]
    elif kind == "chunk":
        B = 1
        n = _log(rng, 16, 1024)
        ctx, new = [_log(rng, 1, 8192)] * 2, [n, n]
    else:
        B = _log(rng, 2, 16)
        ctx, new = [0, _log(rng, 16, 6000)], [1, _log(rng, 2, 256)]
    return dict(op="attend", B=B, Hm=Hm, L=512, dt="bf16", kv=kv, page_size=ps, ctx_lo=ctx[0],
                ctx_hi=ctx[1], new_lo=new[0], new_hi=new[1], window=window, sinks=sinks)


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
    if case["op"] == "plan":
        left = case["T"] - case["pad"]
        for b in range(B):
            new[b] = min(new[b], max(0, left))
            left -= new[b]
    return ctx, new


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    def perm(n):
        return torch.randperm(n, generator=g, device=DEV).to(torch.int32)

    def normal(shape, dtype, std=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)

    def codes(shape):  # E4M3 codes as a quantised row holds them: its largest at 448
        x = torch.randn(shape, generator=g, device=DEV)
        return (x / x.abs().amax(1, keepdim=True) * 448.0).to(E4M3)

    s = dict(case=case)
    if case["op"] == "plan":
        ctx, new = _lengths(case)
        ps, B, T = case["page_size"], case["B"], case["T"]
        have = [-(-c // ps) for c in ctx]
        need = sum(-(-(c + n) // ps) - h for c, n, h in zip(ctx, new, have))
        width = max(-(-(c + n) // ps) for c, n in zip(ctx, new)) + 1
        n_pages = sum(have) + need + 100
        p = perm(n_pages)
        table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        col = torch.arange(width, device=DEV)
        first = i32([0] + have).long().cumsum(0)[:-1]
        own_block = col[None, :] < i32(have)[:, None]
        table[own_block] = p[(first[:, None] + col[None, :])[own_block]]
        begin = 17
        free = torch.cat([p[:begin], p[sum(have):]])  # entries before `begin` are taken already
        e = lambda n: torch.empty(n, dtype=torch.int32, device=DEV)  # noqa: E731
        s |= dict(ctx=i32(ctx), new=i32(new), free=free, begin=i32([begin]), table=table,
                  n_pages=n_pages, base=perm(B) * 70000 if case["keys"] else None,
                  seq_lens=e(B), cu_new=e(B + 1), q_seq=e(T), q_pos=e(T), kv_rows=e(T),
                  key_rows=e(T) if case["keys"] else None, end=e(1))
        return s
    if case["op"] == "append":
        T, L, ps = case["T"], case["L"], case["page_size"]
        n_pages = -(-T // ps) + 5
        rows = perm(n_pages)[:-(-T // ps), None] * ps + torch.arange(ps, device=DEV)
        rows = rows.reshape(-1)[:T].to(torch.int32).contiguous()
        if case["drop"]:
            rows[perm(T)[:case["drop"]].long()] = -1
        n = n_pages * ps
        kv = DT[case["kv"]]
        s |= dict(x=normal((T, L), DT[case["dt"]]), rows=rows,
                  pages=codes((n, L)) if kv == E4M3 else normal((n, L), kv),
                  scale=torch.rand(n, generator=g, device=DEV) if kv == E4M3 else None)
        return s
    ctx, new = _lengths(case)
    ps, B, Hm, L = case["page_size"], case["B"], case["Hm"], case["L"]
    total = [c + n for c, n in zip(ctx, new)]
    blocks = [-(-t // ps) for t in total]
    n_pages = sum(blocks) + 3
    p = perm(n_pages)
    table = torch.full((B, max(blocks) + 1), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b in range(B):
        table[b, :blocks[b]] = p[at:at + blocks[b]]
        at += blocks[b]
    n, T = n_pages * ps, sum(new)
    act, kv = DT[case["dt"]], DT[case["kv"]]
    cu = [0]
    for k in new:
        cu.append(cu[-1] + k)
    s |= dict(q=normal((T, Hm, L), act, 2.0),
              pages=codes((n, L)) if kv == E4M3 else normal((n, L), kv),
              scale=(torch.rand(n, generator=g, device=DEV) + 3.0) / 448.0 if kv == E4M3 else None,
              table=table, seq_lens=i32(total), cu_new=i32(cu), sm_scale=1.0 / math.sqrt(L),
              n_max=max(new), s_max=max(total),
              out=torch.zeros((T, Hm, L), dtype=act, device=DEV),
              lse=torch.zeros((T, Hm), dtype=F32, device=DEV))
    if own:  # the workspace that a user's program keeps
        from sparse_attention_indexer_kpool_gb300 import ops
        s["ws"] = torch.empty(max(16, ops.mla_paged_chunk_workspace_bytes(s["q"], s["pages"])),
                              dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return {"plan": _own_plan, "append": _own_append, "attend": _own_attend}[s["case"]["op"]](s)
    return {"plan": _plan, "append": _append, "attend": _attend}[s["case"]["op"]](s)


def _own_plan(s):
    from sparse_attention_indexer_kpool_gb300 import ops
    ops.dsa_paged_plan(s["ctx"], s["new"], s["free"], s["begin"], s["n_pages"],
                       s["case"]["page_size"], s["table"], s["seq_lens"], s["cu_new"], s["q_seq"],
                       s["q_pos"], s["kv_rows"], s["end"], row_base=s["base"],
                       key_rows=s["key_rows"])
    return _plan_outputs(s["table"], s["seq_lens"], s["cu_new"], s["q_seq"], s["q_pos"],
                         s["kv_rows"], s["end"], s["key_rows"])


def _plan_outputs(table, seq_lens, cu_new, q_seq, q_pos, kv_rows, end, key_rows):
    got = dict(table=table, seq_lens=seq_lens, cu_new=cu_new, q_seq=q_seq, q_pos=q_pos,
               kv_rows=kv_rows, end=end)
    return got if key_rows is None else got | dict(key_rows=key_rows)


def _own_append(s):
    from sparse_attention_indexer_kpool_gb300 import ops
    ops.dsa_paged_append(s["x"], s["rows"], s["pages"], s["scale"])
    return (s["pages"],) if s["scale"] is None else (s["pages"], s["scale"])


def _own_attend(s):
    from sparse_attention_indexer_kpool_gb300 import ops
    c = s["case"]
    ops.dsa_mla_paged_chunk(s["q"], s["pages"], s["scale"], s["table"], s["seq_lens"],
                            c["page_size"], s["cu_new"], c["window"], c["sinks"], s["sm_scale"],
                            s["out"], s["lse"], s["ws"])
    return s["out"], s["lse"]


def _plan(s):
    ps, T = s["case"]["page_size"], s["case"]["T"]
    ctx, new = s["ctx"].long(), s["new"].long()
    B = ctx.numel()
    cu = torch.zeros(B + 1, dtype=torch.long, device=DEV)
    cu[1:] = new.cumsum(0)
    seq_lens = ctx + new
    have = (ctx + ps - 1) // ps
    need = (seq_lens + ps - 1) // ps - have
    first = need.cumsum(0) - need                      # of the free pages that the step takes
    begin = s["begin"].long()
    col = torch.arange(s["table"].shape[1], device=DEV)[None, :]
    fresh = (col >= have[:, None]) & (col < (have + need)[:, None])
    src = (begin + first[:, None] + col - have[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][src], s["table"])
    t = torch.arange(T, device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    live = seq < B
    seq = seq.clamp(max=B - 1)
    pos = ctx[seq] + t - cu[seq]
    blk = (pos // ps).clamp(max=table.shape[1] - 1)
    row = table[seq, blk].long() * ps + pos % ps

    def out(x, empty):
        return torch.where(live, x, empty).to(torch.int32)
    key = None if s["base"] is None else out(s["base"].long()[seq] + pos, -1)
    return _plan_outputs(table, seq_lens.to(torch.int32), cu.to(torch.int32), out(seq, 0),
                         out(pos, -1), out(row, -1),
                         (begin + need.sum()).to(torch.int32), key)


def _append(s):
    x, rows, pages = s["x"].float(), s["rows"].long(), s["pages"]
    n, L = pages.shape
    live = rows >= 0
    dst = torch.where(live, rows, n)                   # dropped rows go to a row behind the cache
    if s["scale"] is None:
        grown = torch.cat([pages, pages.new_empty(1, L)])
        grown[dst] = x.to(pages.dtype)
        return (grown[:n],)
    finite = torch.isfinite(x)
    scale = torch.where(finite, x.abs(), 0.0).amax(1) / 448.0
    scale = torch.where(scale > 0, scale, 1.0)
    q = torch.where(finite, (x / scale[:, None]).clamp(-448.0, 448.0), float("nan")).to(E4M3)
    grown = torch.cat([pages.view(torch.uint8), torch.empty((1, L), dtype=torch.uint8, device=DEV)])
    grown[dst] = q.view(torch.uint8)
    scales = torch.cat([s["scale"], s["scale"].new_empty(1)])
    scales[dst] = scale
    return grown[:n].view(E4M3), scales[:n]


def _attend(s):
    c = s["case"]
    ps, Hm, L = c["page_size"], c["Hm"], c["L"]
    T, (B, width) = s["q"].shape[0], s["table"].shape
    n_max, s_max = s["n_max"], s["s_max"]
    cu, lens = s["cu_new"].long(), s["seq_lens"].long()
    n = cu[1:] - cu[:-1]
    # the sequences' rows, padded to the longest
    pos = torch.arange(s_max, device=DEV)
    rows = s["table"].long()[:, pos // ps].clamp(min=0) * ps + pos % ps
    kv = s["pages"][rows].float() if s["scale"] is None else (
        s["pages"].view(torch.uint8)[rows].view(E4M3).float() * s["scale"][rows][..., None])
    kv = torch.where((pos[None, :] < lens[:, None])[..., None], kv, 0.0)
    # the new tokens' queries, padded to the most of them
    i = torch.arange(n_max, device=DEV)
    live = i[None, :] < n[:, None]
    src = torch.where(live, cu[:-1, None] + i[None, :], 0)
    q = s["q"][src].float().reshape(B, n_max * Hm, L)
    z = torch.bmm(q, kv.transpose(1, 2)).view(B, n_max, Hm, s_max).mul_(s["sm_scale"])
    at = (lens - n)[:, None] + i[None, :]
    see = pos <= at[..., None]
    if c["window"]:
        see &= (pos > at[..., None] - c["window"]) | (pos < c["sinks"])
    z.masked_fill_(~(see & live[..., None])[:, :, None, :], -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = z.sub_(m).exp_()
    total = e.sum(-1, keepdim=True)
    o = torch.bmm(e.view(B, n_max * Hm, s_max), kv).view(B, n_max, Hm, L)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (m + total.log()).squeeze(-1)
    dst = torch.where(live, src, T).reshape(-1)        # padding goes to a row behind the last
    out = torch.empty((T + 1, Hm, L), dtype=s["q"].dtype, device=DEV)
    out[dst] = o.reshape(-1, Hm, L).to(out.dtype)
    lses = torch.empty((T + 1, Hm), dtype=F32, device=DEV)
    lses[dst] = lse.reshape(-1, Hm)
    return out[:T], lses[:T]


# ------------------------------------------------------------------ what a pass cannot do without
def _visible(case):
    """Per new token: how many keys it sees; per sequence: how many rows anyone sees."""
    ctx, new = _lengths(case)
    W, S = case["window"], case["sinks"]
    pairs = rows = 0
    for c, n in zip(ctx, new):
        if W == 0:
            pairs += n * c + n * (n + 1) // 2
            rows += c + n
            continue
        for i in range(n):
            p = c + i
            lo = max(0, p - W + 1)
            pairs += p + 1 - lo + min(S, lo)
        lo = max(0, c - W + 1)
        rows += c + n - lo + min(S, lo)
    return pairs, rows, sum(new)


def work(case):
    if case["op"] == "plan":
        ctx, new = _lengths(case)
        ps = case["page_size"]
        pages = sum(-(-(c + n) // ps) + (-c // ps) for c, n in zip(ctx, new))
        seq = case["B"] * (2 + 2 + (1 if case["keys"] else 0)) + 3
        return dict(bytes=4 * (seq + 2 * pages + case["T"] * (4 if case["keys"] else 3)), flops=0)
    size = {"bf16": 2, "f32": 4, "e4m3": 1}
    if case["op"] == "append":
        live = case["T"] - case["drop"]
        per = case["L"] * (size[case["dt"]] + size[case["kv"]]) + (4 if case["kv"] == "e4m3" else 0)
        return dict(bytes=4 * case["T"] + live * per, flops=0)
    pairs, rows, T = _visible(case)
    Hm, L = case["Hm"], case["L"]
    per_row = L * size[case["kv"]] + (4 if case["kv"] == "e4m3" else 0)
    return dict(bytes=rows * per_row + T * Hm * (2 * L * size[case["dt"]] + 4),
                flops=4 * pairs * Hm * L)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    if case["op"] == "plan":
        return None                                    # whole numbers
    s = prepare(case, seed)
    if case["op"] == "append":
        if case["kv"] != "e4m3":
            pages = s["pages"].double()
            for lo in range(0, case["T"], 8192):
                r = s["rows"][lo:lo + 8192].long()
                pages[r[r >= 0]] = s["x"][lo:lo + 8192][r >= 0].double()
            return (pages,)
        scale = s["scale"].double()
        live = s["rows"] >= 0
        scale[s["rows"][live].long()] = s["x"][live].double().abs().amax(1) / 448.0
        pages = s["pages"].double()
        pages[s["rows"][live].long()] = (
            s["x"][live].double() / scale[s["rows"][live].long()][:, None])
        return pages, scale
    ctx, new = _lengths(case)
    ps, Hm, L, W = case["page_size"], case["Hm"], case["L"], case["window"]
    pairs = _visible(dict(case, window=0))[0]
    if 4 * pairs * Hm * L > 6e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        t = torch.arange(c + n, device=DEV)
        row = s["table"][b, t // ps].long() * ps + t % ps
        keys = s["pages"].view(torch.uint8)[row].view(E4M3).double() if s["scale"] is not None \
            else s["pages"][row].double()
        if s["scale"] is not None:
            keys = keys * s["scale"][row].double()[:, None]
        for lo in range(0, n, 128):
            hi = min(n, lo + 128)
            p = c + torch.arange(lo, hi, device=DEV)
            logits = (s["q"][at + lo:at + hi].double().reshape(-1, L) @ keys.T) * s["sm_scale"]
            hide = t[None, :] > p[:, None]
            if W:
                hide |= (t[None, :] <= p[:, None] - W) & (t[None, :] >= case["sinks"])
            logits = logits.view(hi - lo, Hm, -1).masked_fill(hide[:, None, :], -math.inf)
            lse[at + lo:at + hi] = torch.logsumexp(logits, -1)
            w = torch.softmax(logits, -1)
            out[at + lo:at + hi] = (w.view(-1, c + n) @ keys).view(hi - lo, Hm, L)
        at += n
    return out, lse
