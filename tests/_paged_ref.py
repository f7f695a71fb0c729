"""Plain 64-bit forms of the paged step's operators (tests only), and the bounds
that their rounding gives."""
import math

import torch

DEV_BAD_PAGE, DEV_BAD_LENGTH, DEV_NO_PAGE, DEV_TOKEN_CAP = 256, 512, 1024, 2048
INT_MAX = 2 ** 31 - 1


def plan(ctx, new, free, begin, n_pages, page_size, table, T, base=None):
    """The step plan on Python integers.  ``table``: list of rows (changed in place).
    Returns a dict of lists and the status bits."""
    B, width = len(ctx), len(table[0]) if table else 0
    st, cu, n_eff, c_eff = 0, [0], [], []
    for b in range(B):
        c, n = ctx[b], new[b]
        if n < 0 or c < 0 or c + n > INT_MAX:
            st |= DEV_BAD_LENGTH
            n, c = 0, max(c, 0)
        kept = min(n, T - cu[-1])
        if kept < n:
            st |= DEV_TOKEN_CAP
        cu.append(cu[-1] + kept)
        n_eff.append(kept)
        c_eff.append(c)
    if begin < 0:
        st |= DEV_BAD_LENGTH
    avail = 0 if begin < 0 else max(0, len(free) - begin)
    taken = 0
    old = [list(r) for r in table]
    for b in range(B):
        have, after = -(-c_eff[b] // page_size), -(-(c_eff[b] + n_eff[b]) // page_size)
        if n_eff[b] > 0 and after > width:
            st |= DEV_NO_PAGE
        for blk in range(have, min(after, width)):
            if taken < avail:
                page = free[begin + taken]
                if not 0 <= page < n_pages:
                    st, page = st | DEV_BAD_PAGE, -1
            else:
                st, page = st | DEV_NO_PAGE, -1
            table[b][blk] = page
            taken += 1
    q_seq, q_pos, rows, keys = [], [], [], []
    for b in range(B):
        have = -(-c_eff[b] // page_size)
        for i in range(n_eff[b]):
            p = c_eff[b] + i
            blk = p // page_size
            page = table[b][blk] if blk < width else -1
            if blk < min(have, width) and not 0 <= old[b][blk] < n_pages:
                st, page = st | DEV_BAD_PAGE, -1
            q_seq.append(b)
            q_pos.append(p)
            rows.append(-1 if page < 0 else page * page_size + p % page_size)
            keys.append(-1 if base is None else base[b] + p)
    pad = T - len(q_seq)
    return dict(cu_new=cu, seq_lens=[c + n for c, n in zip(c_eff, n_eff)], table=table,
                q_seq=q_seq + [0] * pad, q_pos=q_pos + [-1] * pad, kv_rows=rows + [-1] * pad,
                key_rows=keys + [-1] * pad, free_end=begin + min(taken, avail)), st


def values(pages, row_scale):
    """The cache rows' values in 64 bits."""
    if row_scale is None:
        return pages.double()
    p = pages.view(torch.float8_e4m3fn) if pages.dtype == torch.uint8 else pages
    return p.float().double() * row_scale.double()[:, None]


def attend(q_lat, rows64, table, seq_lens, page_size, cu_new, window, sinks, sm_scale):
    """out, lse in 64 bits, with the sum of |p c| and the largest |logit| term sums that the
    bounds need.  ``rows64`` [n_rows, L]; a position without a page is skipped."""
    T, Hm, L = q_lat.shape
    dev = q_lat.device
    n_pages = rows64.shape[0] // page_size
    out = torch.zeros((T, Hm, L), dtype=torch.float64, device=dev)
    mag = torch.zeros_like(out)
    lse = torch.full((T, Hm), -math.inf, dtype=torch.float64, device=dev)
    dot = torch.zeros((T, Hm), dtype=torch.float64, device=dev)
    seen = torch.zeros(T, dtype=torch.long, device=dev)
    cu, lens, tab = cu_new.tolist(), seq_lens.tolist(), table.to(dev).long()
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        pos = torch.arange(max(lens[b], 0), device=dev)
        blk = pos // page_size
        page = torch.where(blk < tab.shape[1], tab[b][blk.clamp(max=tab.shape[1] - 1)], -1)
        row = page * page_size + pos % page_size
        paged = (page >= 0) & (page < n_pages)
        for i in range(n):
            p = lens[b] - n + i
            see = paged & (pos <= p)
            if window:
                see &= (pos > p - window) | (pos < sinks)
            pr = row[see]
            if pr.numel() == 0:
                continue
            r = cu[b] + i
            c = rows64[pr]
            q = q_lat[r].double()
            z = (q @ c.T) * sm_scale
            lse[r] = torch.logsumexp(z, -1)
            w = torch.softmax(z, -1)
            out[r] = w @ c
            mag[r] = w @ c.abs()
            dot[r] = ((q.abs() @ c.abs().T) * abs(sm_scale)).amax(-1)
            seen[r] = pr.numel()
    return out, lse, mag, dot, seen


def attend_bounds(ref, dtype, L, dz_more=0.0, out_more=0.0):
    """Largest errors of an attention that keeps logits, sums and outputs in fp32.
    A logit is a sum of L fp32 products: off by at most dz = L 2^-24 sum|q c| (twice that
    where the order is not known) and 2^-21 of itself for the base-2 scaling and the
    exponential; a weight by that relatively, so is their sum.  A weight is rounded to bf16
    for the second product (2^-8) in the bf16 kernels, the sum over n positions adds
    n 2^-23, the result is rounded once.  ``dz_more`` [T, Hm]: what the logits may be off by
    beside that; ``out_more``: the outputs (``underflow``)."""
    out, lse, mag, dot, seen = ref
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    dz = 2 * L * 2.0 ** -24 * dot + 2.0 ** -21 * dot + dz_more
    n = seen.double()[:, None]
    rel = 2 * dz + n * 2.0 ** -23 + 2.0 ** -20 + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
    tol_out = rel[..., None] * mag * 1.01 + half * out.abs() + 1e-30 + out_more
    tol_lse = dz + n * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * torch.where(
        torch.isfinite(lse), lse.abs(), 0.0)
    return tol_out, tol_lse


def underflow(pages, row_scale, act):
    """What E5M2 weights lose of the smallest ones, per latent column (E4M3 pages under bf16
    activations).  A weight w_t times its row's scale r_t, relative to a reference that the
    largest of these products reaches, is held times 2^8 in three parts of E5M2, whose least
    step is 2^-16: off by at most 3 * 2^-17 in all where a part falls below the normal range, so
    the sum over keys by e = 3 * 2^-25 sum_t |code_t|.  The sum of the weights is at least that of
    the key whose product reaches the reference, 1 / r: the output is off by at most e max r."""
    if row_scale is None or act != torch.bfloat16:
        return 0.0
    codes = pages.view(torch.float8_e4m3fn) if pages.dtype == torch.uint8 else pages
    keep = torch.isfinite(row_scale)
    codes = torch.nan_to_num(codes.float()[keep]).abs().double().sum(0)
    return 3 * 2.0 ** -25 * codes * row_scale[keep].double().max()


def check_attend(out, lse, ref, dtype, L, rows=None, dz_more=0.0, out_more=0.0):
    tol_out, tol_lse = attend_bounds(ref, dtype, L, dz_more, out_more)
    want_out, want_lse = ref[0], ref[1]
    if rows is not None:
        out, lse, want_out, want_lse, tol_out, tol_lse = (
            x[rows] for x in (out, lse, want_out, want_lse, tol_out, tol_lse))
    err = (out.double() - want_out).abs() - tol_out
    assert not bool((err > 0).any()) and not bool(torch.isnan(err).any()), \
        f"out beyond its bound by {err.max().item():.3g}"
    fin = torch.isfinite(want_lse)
    assert torch.equal(torch.isfinite(lse), fin) and bool((lse[~fin] == -math.inf).all())
    err = (lse.double() - want_lse)[fin].abs() - tol_lse[fin]
    assert not bool((err > 0).any()), f"lse beyond its bound by {err.max().item():.3g}"


def quantise(x):
    """E4M3 codes and scales of rows, as dsa_paged_append defines them (fp32 divisions; a
    division by a Python number may be done as a product with its reciprocal, so 448 is a
    tensor)."""
    x = x.float()
    fin = torch.isfinite(x)
    s = torch.where(fin, x.abs(), torch.zeros_like(x)).amax(1)
    s = s / torch.full_like(s, 448.0)
    s = torch.where(s > 0, s, torch.ones_like(s))
    q = (x / s[:, None]).clamp(-448.0, 448.0)
    q = torch.where(fin, q, torch.full_like(q, float("nan")))
    return q.to(torch.float8_e4m3fn), s
