"""Plain 64-bit forms of the grouped-query layer's operators, on CPU tensors."""
import math

import torch

E_MIN, E_MAX = -64, 120
F8 = torch.float8_e4m3fn


def two(e):
    return torch.exp2(e.double()) if isinstance(e, torch.Tensor) else 2.0 ** e


def grid(x):
    """The E4M3 value nearest to x (ties to even), |x| <= 448; NaN stays NaN."""
    e = (torch.frexp(x)[1] - 1).clamp(min=-6)
    step = 2.0 ** (e - 3).double()
    return torch.round(x / step) * step


def exponent(a):
    """The least exponent >= E_MIN with a <= 448 * 2^e."""
    if a == 0:
        return E_MIN
    e = math.ceil(math.log2(a / 448.0)) + 1
    while a <= 448.0 * 2.0 ** (e - 1):
        e -= 1
    return max(e, E_MIN)


def values(codes):
    """Codes (float8_e4m3fn or uint8) as 64-bit values."""
    return codes.view(torch.uint8).view(F8).float().double()


def append(new, pages, scale, table, lens, cu, ps, means=None):
    """``pages`` [n_pages, Hkv, ps, D] 64-bit values of the codes and ``scale`` [n_pages, Hkv]
    64-bit, moved on in place by the rows ``new`` [T, Hkv, D]; ``means`` [n_pages, Hkv, D]."""
    n_pages, Hkv = scale.shape
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        ctx = lens[b] - n
        if n == 0:
            continue
        for j in range(ctx // ps, (lens[b] - 1) // ps + 1):
            lo, hi = max(ctx, j * ps), min(lens[b], j * ps + ps)
            page = table[b][j] if j < len(table[b]) else -1
            if not 0 <= page < n_pages:
                continue
            o = lo - j * ps
            x = new[cu[b] + lo - ctx:cu[b] + hi - ctx].double()
            for h in range(Hkv):
                y = x[:, h]
                fin = torch.isfinite(y)
                a = float(torch.where(fin, y.abs(), 0.0).max())
                e = exponent(a)
                if o:
                    e0 = round(math.log2(float(scale[page, h])))
                    e = max(e, e0)
                    pages[page, h, :o] = grid(pages[page, h, :o] * 2.0 ** (e0 - e))
                pages[page, h, o:o + hi - lo] = torch.where(fin, grid(y * 2.0 ** -e), math.nan)
                scale[page, h] = 2.0 ** e
                if means is not None and hi == j * ps + ps:
                    means[page, h] = pages[page, h].mean(0) * 2.0 ** e


def rows(pages, scale, table_row, pos):
    """[len(pos), Hkv, D] values at positions of one sequence; NaN where there is no page."""
    n_pages, Hkv, ps, D = pages.shape
    out = torch.full((len(pos), Hkv, D), math.nan, dtype=torch.float64)
    for i, p in enumerate(pos):
        page = table_row[p // ps] if p // ps < len(table_row) else -1
        if 0 <= page < n_pages:
            out[i] = pages[page, :, p % ps] * scale[page][:, None]
    return out


def scores(q, means, table, lens, cu, ps, sinks, local, sm, NB):
    """[T, Hkv, NB] and the largest |z| sum of products (for tolerances)."""
    T, Hq, D = q.shape
    Hkv = means.shape[1]
    G = Hq // Hkv
    out = torch.full((T, Hkv, NB), math.nan, dtype=torch.float64)
    big = 0.0
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            p, t = lens[b] - n + i, cu[b] + i
            if p < 0:
                out[t] = -math.inf
                continue
            cand = [j for j in range(min((p + 1) // ps, NB, len(table[b])))
                    if 0 <= table[b][j] < means.shape[0]]
            out[t] = -math.inf
            if cand:
                m = means[[table[b][j] for j in cand]].double()          # [n, Hkv, D]
                for h in range(Hkv):
                    qq = q[t, h * G:h * G + G].double()
                    z = qq @ m[:, h].T * sm
                    big = max(big, float((qq.abs() @ m[:, h].abs().T).max()) * abs(sm))
                    out[t, h, cand] = torch.softmax(z, -1).sum(0)
            for j in range(min(NB, p // ps + 1)):
                if j < sinks or j > p // ps - local:
                    out[t, :, j] = math.inf
    return out, big


def attend(q, kp, ks, vp, vs, table, lens, cu, sm, window=0, sinks=0, ids=None):
    """out [T, Hq, D], lse [T, Hq], and for tolerances the absolute weighted values [T, Hq, D], the
    number of keys times the largest weight times its value's scale [T, Hq], and the largest sum
    of |products| of a logit; rows without a sequence are NaN."""
    T, Hq, D = q.shape
    n_pages, Hkv, ps, _ = kp.shape
    G = Hq // Hkv
    out = torch.full((T, Hq, D), math.nan, dtype=torch.float64)
    mass = torch.zeros((T, Hq, D), dtype=torch.float64)
    top = torch.zeros((T, Hq), dtype=torch.float64)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64)
    big = 0.0
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        k_all = rows(kp, ks, table[b], range(max(lens[b], 0)))
        v_all = rows(vp, vs, table[b], range(max(lens[b], 0)))
        held = [0 <= (table[b][t // ps] if t // ps < len(table[b]) else -1) < n_pages
                for t in range(max(lens[b], 0))]
        for i in range(n):
            p, t = lens[b] - n + i, cu[b] + i
            for h in range(Hkv):
                if ids is None:
                    see = [x for x in range(p + 1)
                           if window == 0 or x > p - window or x < sinks]
                else:
                    see = [x for j in ids[t, h].tolist() if j >= 0
                           for x in range(j * ps, min(j * ps + ps, p + 1))]
                see = [x for x in see if held[x]]
                hs = slice(h * G, h * G + G)
                if not see:
                    out[t, hs], lse[t, hs] = 0.0, -math.inf
                    continue
                qq, k, v = q[t, hs].double(), k_all[see, h], v_all[see, h]
                z = qq @ k.T * sm
                big = max(big, float((qq.abs() @ k.abs().T).nan_to_num(0.0).max()) * abs(sm))
                w = torch.softmax(z, -1)
                out[t, hs], lse[t, hs] = w @ v, torch.logsumexp(z, -1)
                mass[t, hs] = w @ v.abs()
                s = torch.stack([vs[table[b][x // ps], h] for x in see])
                top[t, hs] = (w * s).amax(-1) * len(see)
    return out, lse, mass, top, big


def attend_dense(q, kp, ks, vp, vs, table, lens, cu, sm, window=0, sinks=0):
    """``attend`` without lists, a sequence and KV head at a time on the tensors' device; every
    position needs a page."""
    T, Hq, D = q.shape
    Hkv, ps = kp.shape[1], kp.shape[2]
    G, dev = Hq // Hkv, q.device
    out = torch.full((T, Hq, D), math.nan, dtype=torch.float64, device=dev)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64, device=dev)
    mass, top, big = torch.zeros_like(out), torch.zeros_like(lse), 0.0
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        x = torch.arange(lens[b], device=dev)
        page = torch.tensor(table[b], device=dev)[x // ps]
        p = lens[b] - n + torch.arange(n, device=dev)
        see = x[None, :] <= p[:, None]
        if window:
            see &= (x[None, :] > p[:, None] - window) | (x[None, :] < sinks)
        for h in range(Hkv):
            k = kp[page, h, x % ps] * ks[page, h][:, None]
            v = vp[page, h, x % ps] * vs[page, h][:, None]
            bad = torch.isnan(v)
            qq = q[cu[b]:cu[b + 1], h * G:h * G + G].double()
            z = torch.einsum("tgd,sd->tgs", qq, k) * sm
            most = (qq.abs().flatten(0, 1) @ k.abs().T).nan_to_num(0.0).max()
            big = max(big, float(most) * abs(sm))
            z = z.masked_fill(~see[:, None, :], -math.inf)
            w = torch.softmax(z, -1)
            o = torch.einsum("tgs,sd->tgd", w, v.nan_to_num(0.0))
            hit = (see.double() @ bad.double()) > 0          # [n, D]
            rows = slice(cu[b], cu[b + 1]), slice(h * G, h * G + G)
            out[rows] = o.masked_fill(hit[:, None, :], math.nan)
            mass[rows] = torch.einsum("tgs,sd->tgd", w, v.nan_to_num(0.0).abs())
            lse[rows] = torch.logsumexp(z, -1)
            top[rows] = (w * vs[page, h]).amax(-1) * lens[b]
    return out, lse, mass, top, big


def bound_of_bf16(want, mass, top, big, n, D):
    """How far the bf16 path's outputs may be from ``attend``'s: a logit is a sum of D products in
    fp32 (cut off where fp32 rounds: two half steps a term) and a few more roundings; a weight is
    2^z (2^-22) over a sum of n.  Then the weight's rounding to fp16's 11 bits, 2^-11 of it; where
    it is below fp16's normal numbers, and where weights that are written are scaled down, 2^-25 of
    the row's largest at most, a code of at most 448 and n keys; and the output's to bf16, 2^-8."""
    dz = big * (2 * D + 8) * 2.0 ** -24
    w = 2 * dz + n * 2.0 ** -24 + 2.0 ** -20
    return (2.0 ** -8 * want.abs() + 2 * w * (mass + want.abs()) + 2.0 ** -11 * mass
            + 448 * 2.0 ** -25 * top[..., None] + 2.0 ** -126)


def weights_rounded_to(dtype, z, v, s):
    """Outputs [G, D] of logits ``z`` [G, n], values ``v`` [n, D] of scales ``s`` [n], with weights
    times scales rounded to ``dtype`` for the products and not for the sum."""
    w = torch.exp(z - z.amax(-1, keepdim=True))
    held = 4.0 * w * s / (w * s).amax(-1, keepdim=True)
    return (held.to(dtype).double() / held.nan_to_num(1.0) * w) @ v / w.sum(-1, keepdim=True)
