"""The paged serving step on the GPU: the plan against integers, the append against
fp32 divisions, the chunk attention against 64 bits within the bounds of its
roundings, and the three together with the selection that they feed."""
import math
import random
import threading

import pytest
import torch

from sparse_attention_indexer_kpool_gb300 import ops, pipeline, synth
from sparse_attention_indexer_kpool_gb300.synth import Geometry
from tests import _paged_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
WIDE = 320_000     # positions of a table whose width lets a few tokens' keys be many
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- plan
def run_plan(ctx, new, free, begin, n_pages, ps, table, T, base=None, in_place=False):
    c, fb = i32(ctx), i32([begin])
    tab = i32(table)
    B = len(ctx)
    e = lambda n: torch.full((n,), -77, dtype=torch.int32, device=DEV)  # noqa: E731
    lens, end = (c, fb) if in_place else (e(B), e(1))
    out = dict(seq_lens=lens, cu_new=e(B + 1), q_seq=e(T), q_pos=e(T), kv_rows=e(T))
    keys = e(T) if base is not None else None
    st = i32([0])
    ops.dsa_paged_plan(c, i32(new), i32(free), fb, n_pages, ps, tab, out["seq_lens"],
                       out["cu_new"], out["q_seq"], out["q_pos"], out["kv_rows"], end,
                       row_base=None if base is None else i32(base), key_rows=keys, status=st)
    torch.cuda.synchronize()
    got = {k: v.tolist() for k, v in out.items()}
    got |= dict(table=tab.tolist(), free_end=end.item())
    if keys is not None:
        got["key_rows"] = keys.tolist()
    return got, st.item()


def check_plan(*args, **kw):
    in_place = kw.pop("in_place", False)
    ctx, new, free, begin, n_pages, ps, table, T = args
    got, st = run_plan(*args, **kw, in_place=in_place)
    want, want_st = ref.plan(ctx, new, free, begin, n_pages, ps, [list(r) for r in table], T, **kw)
    for k in got:
        assert got[k] == want[k], k
    assert st == want_st


def random_plan(seed, B, ps, new_hi, ctx_hi, slack, width_cut=0):
    rng = random.Random(seed)
    ctx = [rng.randint(0, ctx_hi) for _ in range(B)]
    new = [rng.randint(0, new_hi) for _ in range(B)]
    have = [-(-c // ps) for c in ctx]
    after = [-(-(c + n) // ps) for c, n in zip(ctx, new)]
    width = max(1, max(after) - width_cut)
    n_pages = sum(have) + sum(after) + 50
    ids = list(range(n_pages))
    rng.shuffle(ids)
    table, at = [], 0
    for h in have:
        table.append((ids[at:at + h] + [-1] * width)[:width])
        at += h
    free = ids[at:at + 3 + sum(after) - sum(have) + slack]
    base = [rng.randint(0, 10 ** 6) for _ in range(B)]
    return ctx, new, free, 3, n_pages, ps, table, sum(new), base


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,ps,new_hi,ctx_hi,T_off", [
    (1, 1, 1, 0, 0), (1, 64, 5000, 300, 9), (3, 7, 40, 100, 0), (64, 64, 1, 65000, 0),
    (255, 16, 3, 900, 100), (256, 5, 30, 60, -11), (1025, 16, 4, 200, 1), (8192, 48, 2, 100, 3),
    (300, 16, 200, 50, 5000)])
def test_plan(B, ps, new_hi, ctx_hi, T_off, in_place):
    ctx, new, free, begin, n_pages, ps, table, T, base = random_plan(B, B, ps, new_hi, ctx_hi, 5)
    T = max(0, T + T_off)
    check_plan(ctx, new, free, begin, n_pages, ps, table, T, base=base, in_place=in_place)
    check_plan(ctx, new, free, begin, n_pages, ps, table, T, in_place=in_place)


def test_plan_with_nothing_new_and_no_room():
    check_plan([5, 0, 9], [0, 0, 0], [], 0, 4, 4, [[0, 1, -1], [-1] * 3, [2, 3, 0]], 0)
    check_plan([5, 0, 9], [0, 0, 0], [1], 0, 4, 4, [[0, 1, -1], [-1] * 3, [2, 3, 0]], 5)
    check_plan([5, 0, 9], [3, 2, 2], [3], 0, 4, 4, [[0, 1, -1], [-1] * 3, [2, 3, 0]], 0)


def test_plan_faults_are_flagged_and_contained():
    ctx, new, free, begin, n_pages, ps, table, T, base = random_plan(5, 40, 8, 20, 60, -30)
    check_plan(ctx, new, free, begin, n_pages, ps, table, T, base=base)          # list used up
    check_plan(ctx, new, free, -4, n_pages, ps, table, T)                        # no list at all
    check_plan(ctx, new, free, len(free) + 9, n_pages, ps, table, T)             # begins past it
    ctx, new, free, begin, n_pages, ps, table, T, base = random_plan(6, 40, 8, 20, 60, 5, 3)
    check_plan(ctx, new, free, begin, n_pages, ps, table, T, base=base)          # narrow table
    ctx, new, free, begin, n_pages, ps, table, T, base = random_plan(7, 9, 8, 20, 60, 5)
    bad = list(ctx), list(new)
    bad[1][2], bad[0][4], bad[0][5], bad[1][6] = -3, -1, 2 ** 31 - 2, 2 ** 31 - 1
    check_plan(bad[0], bad[1], free, begin, n_pages, ps, table, T)
    for k in range(begin, len(free), 2):
        free[k] = [-1, n_pages, -2 ** 31, 2 ** 31 - 1][k % 4]
    for row in table[::2]:
        row[0:2] = [n_pages + 3, -9][:len(row)]
    check_plan(ctx, new, free, begin, n_pages, ps, table, T)


@pytest.mark.parametrize("lens_in_place,list_in_place", [(True, False), (False, True)])
def test_plan_half_in_place(lens_in_place, list_in_place):
    ctx, new, free, begin, n_pages, ps, table, T, base = random_plan(8, 3000, 16, 4, 300, 9)
    c, fb, tab, B = i32(ctx), i32([begin]), i32(table), 3000
    e = lambda n: torch.full((n,), -77, dtype=torch.int32, device=DEV)  # noqa: E731
    out = dict(seq_lens=c if lens_in_place else e(B), cu_new=e(B + 1), q_seq=e(T), q_pos=e(T),
               kv_rows=e(T))
    end = fb if list_in_place else e(1)
    ops.dsa_paged_plan(c, i32(new), i32(free), fb, n_pages, ps, tab, out["seq_lens"],
                       out["cu_new"], out["q_seq"], out["q_pos"], out["kv_rows"], end)
    want, _ = ref.plan(ctx, new, free, begin, n_pages, ps, [list(r) for r in table], T)
    assert all(out[k].tolist() == want[k] for k in out)
    assert tab.tolist() == want["table"] and end.item() == want["free_end"]


def test_plan_at_the_end_of_the_positions():
    """Positions just below 2^31, behind many other tokens of the step."""
    hi = 2 ** 31 - 1
    ctx, new = [0, hi - 3, hi - 700, 5], [5000, 3, 700, 1]
    ps = 1 << 20
    table = [[-1] * 2048, list(range(2048)), list(range(2047, -1, -1)), [0] + [-1] * 2047]
    check_plan(ctx, new, [7, 9], 0, 2047, ps, table, 5800)


def test_calls_from_two_threads():
    """The plan and the generic attention at different sizes from two threads, a stream each."""
    jobs, got = [], {}
    for B, L in ((8192, 1024), (4200, 520)):
        p = random_plan(B, B, 16, 2, 40, 5)
        s = make([70, 9], [3, 2], Hm=2, L=L, act=F32, kv=F32, ps=16, seed=L)
        jobs.append((B, L, p, s, [i32(x) for x in (p[0], p[1], p[2], [p[3]], p[6])]))
    torch.cuda.synchronize()

    def work(B, p, s, inputs):
        ctx, new, free, begin, table = inputs
        with torch.cuda.stream(torch.cuda.Stream()):
            e = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)  # noqa: E731
            runs = []
            for _ in range(20):
                tab, rows = table.clone(), e(p[7])
                ops.dsa_paged_plan(ctx, new, free, begin, p[4], p[5], tab, e(B), e(B + 1), e(p[7]),
                                   e(p[7]), rows, e(1))
                o, ls = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:2], device=DEV)
                ops.dsa_mla_paged_chunk(s["q"], s["pages"], None, s["table"], s["lens"], 16,
                                        s["cu"], 0, 0, s["sm"], o, ls)
                runs.append((rows, tab, o, ls))
            torch.cuda.current_stream().synchronize()
            got[B] = runs

    threads = [threading.Thread(target=work, args=(B, p, s, x)) for B, _, p, s, x in jobs]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    for B, L, p, s, _ in jobs:
        want, _ = ref.plan(p[0], p[1], p[2], p[3], p[4], p[5], [list(r) for r in p[6]], p[7])
        exp = reference(s)
        for rows, tab, o, ls in got[B]:
            assert rows.tolist() == want["kv_rows"] and tab.tolist() == want["table"]
            ref.check_attend(o, ls, exp, F32, L, rows=torch.arange(5, device=DEV))


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("L", [8, 64, 248, 512, 520, 1024])
@pytest.mark.parametrize("act", [BF, F32])
@pytest.mark.parametrize("kv", [BF, F32, F8])
def test_append(L, act, kv):
    g = torch.Generator(device=DEV).manual_seed(L)
    for T, n_rows in ((1, 5), (77, 200)):
        x = torch.randn((T, L), generator=g, device=DEV).to(act)
        x *= torch.logspace(-30, 30, T, device=DEV)[:, None].to(act)   # every scale
        if T > 1:
            x[3] = 0
            x[4, 1], x[5, 0], x[5, L - 1], x[6] = math.nan, math.inf, -math.inf, math.nan
            x[7] = 1e-44 if act == F32 else 0
            x[8, 2] = -x[8].abs().max() * 2                            # the largest is negative
        rows = torch.randperm(n_rows, generator=g, device=DEV)[:T].to(torch.int32)
        if T > 1:
            rows[10:20] = -1
            rows[30], rows[31] = n_rows, 2 ** 31 - 1                   # dropped and flagged
        pages = torch.randn((n_rows, L), generator=g, device=DEV).to(kv)
        scale = torch.rand(n_rows, generator=g, device=DEV) if kv == F8 else None
        want, want_s = pages.clone(), None if scale is None else scale.clone()
        live = (rows >= 0) & (rows < n_rows)
        at = rows[live].long()
        if kv == F8:
            codes, s = ref.quantise(x[live])
            want.view(torch.uint8)[at] = codes.view(torch.uint8)
            want_s[at] = s
        else:
            want[at] = x[live].to(kv)
        st = i32([0])
        ops.dsa_paged_append(x, rows, pages, scale, status=st)
        torch.cuda.synchronize()
        assert st.item() == (ops.DEV_BAD_PAGE if T > 1 else 0)
        assert torch.equal(torch.nan_to_num(pages.float(), nan=12345.0),
                           torch.nan_to_num(want.float(), nan=12345.0))
        if kv == F8:
            assert torch.equal(scale, want_s)


@pytest.mark.parametrize("kv,L,act", [(BF, 512, BF), (F8, 512, BF), (F32, 1024, F32)])
@pytest.mark.parametrize("ps", [64, 5])
def test_rows_past_32_bits(kv, L, act, ps):
    """A cache whose elements pass 2^31 (2^32 bytes and more but for E4M3): rows appended to its
    last pages and attended to."""
    n_pages = -(-(2 ** 31 + 2 ** 24) // (L * ps))
    pages = torch.empty((n_pages * ps, L), dtype=kv, device=DEV)
    scale = torch.empty(n_pages * ps, device=DEV) if kv == F8 else None
    g = torch.Generator(device=DEV).manual_seed(24)
    n = 150
    x = torch.randn((n, L), generator=g, device=DEV).to(act)
    blocks = -(-n // ps)
    table = torch.arange(n_pages - 1, n_pages - 1 - blocks, -1, device=DEV).to(torch.int32)[None]
    p = torch.arange(n, device=DEV)
    rows = table[0].long()[p // ps] * ps + p % ps
    assert int(rows.min()) * L > 2 ** 31
    st = i32([0])
    ops.dsa_paged_append(x, rows.to(torch.int32), pages, scale, status=st)
    used = pages[rows.min():]                       # (the last pages, in 64 bits)
    first = int(rows.min()) // ps * ps
    vals = ref.values(pages[first:], None if scale is None else scale[first:])
    have = vals[rows - first]
    tol = x.double().abs() * (2.0 ** -4 if kv == F8 else 2.0 ** -8)
    if kv == F8:
        tol = torch.maximum(tol, 2.0 ** -10 * scale[rows].double()[:, None]) * 1.001
    assert bool(((have - x.double()).abs() <= tol).all()) and used.shape[0] >= n
    for Hm in ((64, 16) if act == BF else (4,)):
        q = torch.randn((9, Hm, L), generator=g, device=DEV).to(act)
        for width in (0, WIDE):
            tab = torch.full((1, max(blocks, -(-width // ps))), -1, dtype=torch.int32, device=DEV)
            tab[:, :blocks] = table
            s = dict(q=q, pages=pages, scale=scale, table=tab, lens=i32([n]), cu=i32([0, 9]),
                     ps=ps, sm=1.0 / math.sqrt(L), T=9)
            out, lse, status = attend(s)
            assert status == 0
            near = dict(s, table=torch.where(tab >= 0, tab - first // ps, tab))
            want = ref.attend(q, vals, near["table"], s["lens"], ps, s["cu"], 0, 0, s["sm"])
            more = ref.underflow(pages[rows], None if scale is None else scale[rows], act)
            ref.check_attend(out, lse, want, act, L, out_more=more)
    assert st.item() == 0


# ---------------------------------------------------------------- chunk attention
def make(lens, new, *, Hm=64, L=512, act=BF, kv=BF, ps=64, seed=0, pad=3, q_std=1.0,
         hidden=math.nan, width=0):
    """A paged cache whose rows outside the sequences hold ``hidden``; the table has room for
    ``width`` positions at least (wide tables may take another kernel)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    blocks = [-(-max(t, 0) // ps) for t in lens]
    n_pages = sum(blocks) + 2
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    cols = max(max(blocks + [1]) + 1, -(-width // ps))
    table = torch.full((len(lens), cols), -1, dtype=torch.int32, device=DEV)
    n = n_pages * ps
    x = torch.randn((n, L), generator=g, device=DEV)
    used = torch.zeros(n, dtype=torch.bool, device=DEV)
    at = 0
    for b, t in enumerate(lens):
        table[b, :blocks[b]] = perm[at:at + blocks[b]]
        at += blocks[b]
        p = torch.arange(max(t, 0), device=DEV)
        used[table[b].long()[p // ps] * ps + p % ps] = True
    x[~used] = hidden
    if kv == F8:
        pages, scale = ref.quantise(x)
        scale[~used] = hidden
    else:
        pages, scale = x.to(kv), None
    T = sum(new) + pad
    cu = [0]
    for k in new:
        cu.append(cu[-1] + k)
    q = (torch.randn((T, Hm, L), generator=g, device=DEV) * q_std).to(act)
    return dict(q=q, pages=pages, scale=scale, table=table, lens=i32(lens), cu=i32(cu), ps=ps,
                sm=1.0 / math.sqrt(L), T=T)


make_step = make


def attend(s, window=0, sinks=0, stream=None, ws=None, out=None, lse=None):
    T, Hm, L = s["q"].shape
    out = torch.full_like(s["q"], 7.0) if out is None else out
    lse = torch.full((T, Hm), 7.0, dtype=F32, device=DEV) if lse is None else lse
    st = i32([0])
    n = ops.mla_paged_chunk_workspace_bytes(s["q"], s["pages"])
    if ws is None:  # what a workspace held before does not matter
        ws = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device=DEV)
    ops.dsa_mla_paged_chunk(s["q"], s["pages"], s["scale"], s["table"], s["lens"], s["ps"],
                            s["cu"], window, sinks, s["sm"], out, lse, ws, st, stream)
    torch.cuda.synchronize()
    return out, lse, st.item()


def reference(s, window=0, sinks=0):
    return ref.attend(s["q"], ref.values(s["pages"], s["scale"]), s["table"], s["lens"], s["ps"],
                      s["cu"], window, sinks, s["sm"])


def check(s, window=0, sinks=0, status=0):
    out, lse, st = attend(s, window, sinks)
    assert st == status
    live = s["cu"][-1].item()
    r = reference(s, window, sinks)
    ref.check_attend(out, lse, r, s["q"].dtype, s["q"].shape[2],
                     rows=torch.arange(live, device=DEV),
                     out_more=ref.underflow(s["pages"], s["scale"], s["q"].dtype))
    assert bool((out[live:] == 7.0).all()) and bool((lse[live:] == 7.0).all())
    return out, lse


LENS = [([1], [1]), ([127, 128, 129, 1], [1, 1, 1, 1]), ([300], [300]), ([0, 5, 0], [0, 5, 0]),
        ([1000, 3, 130, 700, 64], [1, 3, 2, 9, 64]), ([2500, 17], [130, 0]),
        ([513, 256, 255], [3, 7, 1])]
MASKS = [(0, 0), (0, 5), (1, 0), (64, 4), (100, 130), (700, 1), (128, 1000)]
GEOS = [(64, 512, BF, BF), (64, 512, BF, F8), (16, 512, BF, BF), (128, 512, BF, F8),
        (33, 512, BF, BF), (1, 512, BF, F8), (80, 512, BF, BF), (4, 64, F32, F32),
        (5, 40, BF, F8), (3, 1024, F32, F8), (2, 512, F32, BF), (2, 512, BF, F32)]


@pytest.mark.parametrize("Hm,L,act,kv", GEOS)
@pytest.mark.parametrize("which", range(len(LENS)))
def test_chunk(Hm, L, act, kv, which):
    lens, new = LENS[which]
    for j, (window, sinks) in enumerate(MASKS):
        ps = (64, 16, 1, 48, 5, 128, 8)[(which + j) % 7]
        s = make(lens, new, Hm=Hm, L=L, act=act, kv=kv, ps=ps, seed=which * 10 + j)
        check(s, window, sinks)


@pytest.mark.parametrize("Hm", [64, 128, 33, 80])
@pytest.mark.parametrize("which", range(len(LENS)))
def test_chunk_wide_tables(Hm, which):
    """Two row blocks share their keys: chunks of two tokens and more (or more than 64 heads)
    that may see many positions."""
    lens, new = LENS[which]
    for j, (window, sinks) in enumerate([(0, 0), (1, WIDE), (64, WIDE), (100, 2 ** 31 - 1),
                                         (WIDE, 0), (WIDE, 7), (2 ** 31 - 1, 2 ** 31 - 1)]):
        ps = (64, 16, 48, 8, 128, 24)[(which + j) % 6]
        check(make(lens, new, Hm=Hm, ps=ps, seed=which * 10 + j, width=WIDE, pad=0), window, sinks)


def test_chunk_wide_tables_long_windows():
    s = make([5000, 2600, 2300], [200, 3, 120], seed=16, q_std=2.0)
    for window, sinks in ((2047, 2), (2100, 5), (2500, 300), (1, 2500), (4990, 1), (64, 4000),
                          (100, 1990), (700, 1400)):
        check(s, window, sinks)


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("B,hi,new", [(1, 9000, 1), (3, 20000, 1), (160, 700, 1), (40, 2000, 3)])
def test_chunk_decode_split_over_the_card(B, hi, new, kv):
    rng = random.Random(B)
    lens = [rng.randint(new, hi) for _ in range(B)]
    s = make(lens, [new] * B, kv=kv, seed=B, q_std=2.0)
    check(s)
    check(s, 512, 4)


@pytest.mark.parametrize("kv", [BF, F8])
def test_chunk_many_tokens(kv):
    s = make([900, 1500, 40], [300, 200, 40], kv=kv, seed=3, q_std=2.0)
    check(s)
    check(s, 200, 9)


@pytest.mark.parametrize("act,kv,L", [(BF, BF, 512), (BF, F8, 512), (F32, F32, 64)])
def test_chunk_rising_and_falling_logits(act, kv, L):
    """Keys whose logits climb (and fall) by hundreds along the sequence: the running
    maximum has to move, far apart tiles must not overflow or vanish."""
    for sign, Hm, width in ((1.0, 16, 0), (-1.0, 16, 0), (1.0, 64, WIDE), (-1.0, 64, WIDE)):
        s = make([1300], [4], Hm=Hm, L=L, act=act, kv=kv, seed=4, width=width, pad=0)
        ramp = torch.linspace(-6.0, 6.0, 1300, device=DEV) * sign
        p = torch.arange(1300, device=DEV)
        rows = s["table"][0].long()[p // s["ps"]] * s["ps"] + p % s["ps"]
        direction = torch.randn(L, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV)
        x = ramp[:, None] * direction[None, :] + 0.05 * torch.randn((1300, L), device=DEV)
        if kv == F8:
            codes, sc = ref.quantise(x)
            s["pages"].view(torch.uint8)[rows] = codes.view(torch.uint8)
            s["scale"][rows] = sc
        else:
            s["pages"][rows] = x.to(kv)
        s["q"] = (direction * 2).to(act).expand(s["T"], Hm, L).contiguous()
        check(s)
        check(s, 300, 7)


@pytest.mark.parametrize("Hm", [64, 40, 100])
def test_chunk_wide_tables_short_rows_one_after_the_other(Hm):
    """Hundreds of row tiles of two to four key tiles: the first outputs of one may not reach
    the accumulators before every warp has read those of the one before."""
    rng = random.Random(Hm)
    lens = [rng.choice((80, 100, 128, 200, 256)) for _ in range(500)]
    new = [rng.choice((1, 2, 2, 2, 3)) for _ in lens]
    s = make(lens, new, Hm=Hm, ps=16, seed=28, width=WIDE, pad=0, q_std=2.0)
    want = check(s)
    for _ in range(20):
        out, lse, st = attend(s)
        assert st == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("Hm", [64, 40, 100])
def test_chunk_wide_tables_rows_of_one_tile(Hm):
    """Hundreds of row tiles of a single key tile, whose sums differ widely: no row may be
    normalised by the next one's."""
    rng = random.Random(Hm)
    lens = [rng.randint(2, 64) for _ in range(900)]
    s = make(lens, [2] * 900, Hm=Hm, ps=16, seed=29, width=WIDE, pad=0, q_std=4.0)
    want = check(s)
    for _ in range(20):
        out, lse, st = attend(s)
        assert st == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("n,m,window", [(400, 6, 50), (2500, 320, 2060)])
@pytest.mark.parametrize("act,kv,Hm,L", [(BF, BF, 64, 512), (BF, F8, 16, 512), (F32, F32, 4, 64)])
def test_chunk_later_tokens_do_not_reach_earlier_ones(act, kv, Hm, L, n, m, window):
    """NaN, infinities and the type's largest values in the rows of later tokens, outside
    the window and behind the sequence leave the others as they are."""
    for fill in (math.nan, math.inf, -math.inf, torch.finfo(kv).max):
        s = make([n], [m], Hm=Hm, L=L, act=act, kv=kv, ps=16, seed=6, hidden=fill)
        want, want_lse, _ = attend(s, window, 3)
        p = torch.arange(n, device=DEV)
        rows = s["table"][0].long()[p // 16] * 16 + p % 16
        hide = torch.zeros(n, dtype=torch.bool, device=DEV)
        hide[n - 3:] = True                  # the chunk's last three tokens
        hide[3:n - m - window + 1] = True    # outside every window
        s["pages"][rows[hide]] = torch.full((), fill, device=DEV).to(kv)
        if kv == F8:
            s["scale"][rows[hide]] = fill
        out, lse, _ = attend(s, window, 3)
        k = m - 3
        assert torch.equal(out[:k], want[:k]) and torch.equal(lse[:k], want_lse[:k])
        if math.isnan(fill):                 # and it reaches those that see it
            assert torch.isnan(out[k:m].float()).all()


@pytest.mark.parametrize("window,m", [(0, 6), (2100, 6), (2100, 320)])
@pytest.mark.parametrize("act,Hm,L,width", [(BF, 64, 512, 0), (BF, 64, 512, WIDE),
                                            (BF, 40, 512, WIDE), (F32, 4, 64, 0)])
def test_chunk_infinite_keys(act, Hm, L, width, window, m):
    """Infinities in the last token's key, and in the one that leaves the window with it.  Where a
    query makes its logit minus infinity its weight is 0, and 0 times infinity NaN: in those
    latent columns alone.  Other queries' logits are infinite or NaN, and their outputs NaN.  A
    token that does not see the key keeps every bit."""
    n, ps = 2500, 16
    s = make([n], [m], Hm=Hm, L=L, act=act, kv=act, ps=ps, seed=31, width=width, pad=0)
    d = [7, L - 20]                                     # (one in each half of the columns)
    h = torch.arange(Hm, device=DEV)
    signs = torch.where(h % 4 == 1, 1, -1), torch.where(h % 4 == 2, -1, 1)
    for col, sign in zip(d, signs):
        s["q"][:, :, col] = (s["q"][:, :, col].abs() + 0.5) * sign
    want, want_lse, _ = attend(s, window, 3)
    p = torch.arange(n, device=DEV)
    rows = s["table"][0].long()[p // ps] * ps + p % ps
    keys = [n - 1] + ([n - 1 - window] if window else [])
    for k in keys:
        s["pages"][rows[k], d[0]] = math.inf
        s["pages"][rows[k], d[1]] = -math.inf
    out, lse, st = attend(s, window, 3)
    assert st == 0
    low = (h % 4 == 0) | (h % 4 == 3)                   # minus infinity in both columns
    for i in range(m):
        at = n - m + i
        see = (p <= at) & ((p > at - window) | (p < 3) if window else True)
        if not any(bool(see[k]) for k in keys):
            assert torch.equal(out[i], want[i]) and torch.equal(lse[i], want_lse[i])
            continue
        assert torch.isnan(out[i][~low].float()).all()
        see[keys] = False
        one = rows[see].to(torch.int32)[None]
        exp = ref.attend(s["q"][i:i + 1, low], ref.values(s["pages"], None), one,
                         i32([one.shape[1]]), 1, i32([0, 1]), 0, 0, s["sm"])
        got = out[i:i + 1, low]
        assert torch.isnan(got[:, :, d].float()).all(), (i, "columns")
        got[:, :, d] = exp[0][:, :, d].to(act)
        ref.check_attend(got, lse[i:i + 1, low], exp, act, L)


@pytest.mark.parametrize("width", [0, WIDE])
@pytest.mark.parametrize("act,kv,Hm,L", [(BF, BF, 64, 512), (BF, F8, 64, 512), (F32, F32, 4, 64)])
def test_chunk_faults_are_flagged_and_contained(act, kv, Hm, L, width):
    def make(*a, **kw):
        return make_step(*a, **kw, width=width)

    s = make([500, 100, 60], [3, 100, 2], Hm=Hm, L=L, act=act, kv=kv, ps=16, seed=7)
    n_pages = s["pages"].shape[0] // 16
    s["table"][0, 3], s["table"][0, 20], s["table"][1, 0] = -1, n_pages, 2 ** 31 - 1
    s["table"][2, :] = -5                              # nothing at all
    check(s, status=ops.DEV_BAD_PAGE)
    s = make([500, 100], [3, 100], Hm=Hm, L=L, act=act, kv=kv, ps=16, seed=8)
    s["table"] = s["table"][:, :10].contiguous()       # too narrow for the first
    check(s, status=ops.DEV_BAD_PAGE)
    s = make([5, 9, -3], [8, 9, 2], Hm=Hm, L=L, act=act, kv=kv, ps=16, seed=9)
    check(s, status=ops.DEV_BAD_LENGTH)                # rows before position 0 see nothing
    s = make([50, 60], [10, 20], Hm=Hm, L=L, act=act, kv=kv, ps=16, seed=10, pad=0)
    s["cu"] = i32([-4, 10, 1000])                      # cut to the rows that exist
    out, lse, st = attend(s)
    assert st & ops.DEV_BAD_LENGTH and torch.isfinite(out.float()).all()
    s["cu"] = i32([20, 3, 7])
    assert attend(s)[2] & ops.DEV_BAD_LENGTH


@pytest.mark.parametrize("act,kv,Hm,L,width", [(BF, BF, 64, 512, 0), (BF, BF, 128, 512, 3200),
                                               (BF, F8, 16, 512, 0), (F32, F32, 4, 64, 0)])
def test_chunk_rows_of_many_sequences_at_once_do_not_multiply(act, kv, Hm, L, width):
    """Ends that rise and fall would give every row to thousands of sequences: flagged, and
    over soon."""
    s = make([900] + [0] * 8191, [600] + [0] * 8191, Hm=Hm, L=L, act=act, kv=kv, ps=16, seed=26,
             width=width, pad=0)
    s["cu"] = i32([0, 600] * 4096 + [0])
    s["lens"] = i32([900] * 8192)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    attend(s)
    start.record()
    st = attend(s)[2]
    end.record()
    torch.cuda.synchronize()
    assert st & ops.DEV_BAD_LENGTH and start.elapsed_time(end) < 100.0


@pytest.mark.parametrize("act,kv,Hm,L", [(BF, BF, 64, 512), (BF, BF, 16, 512), (BF, F8, 64, 512),
                                         (F32, F32, 4, 64)])
def test_chunk_many_sequences_of_which_few_have_tokens(act, kv, Hm, L):
    """8,192 sequences with five tokens among them; none at all; no lse; codes as bytes."""
    lens, new = [0] * 8192, [0] * 8192
    for b, n, k in ((0, 40, 1), (17, 300, 2), (8191, 129, 2)):
        lens[b], new[b] = n, k
    s = make(lens, new, Hm=Hm, L=L, act=act, kv=kv, ps=16, seed=25)
    out, _ = check(s)
    check(dict(s, cu=i32([0] * 8193)))
    T, got = s["T"], torch.full_like(s["q"], 7.0)
    ws = torch.empty(ops.mla_paged_chunk_workspace_bytes(s["q"], s["pages"]), dtype=torch.uint8,
                     device=DEV)
    pages = s["pages"].view(torch.uint8) if kv == F8 else s["pages"]
    ops.dsa_mla_paged_chunk(s["q"], pages, s["scale"], s["table"], s["lens"], 16, s["cu"], 0, 0,
                            s["sm"], got, None, ws if ws.numel() else None)
    torch.cuda.synchronize()
    assert torch.equal(got, out) and T == 8


@pytest.mark.parametrize("act,kv,Hm,L,width", [(BF, BF, 64, 512, 0), (BF, BF, 64, 512, WIDE),
                                               (BF, F8, 64, 512, 0), (BF, F8, 16, 512, 0),
                                               (F32, F32, 4, 64, 0)])
def test_chunk_softmax_scales(act, kv, Hm, L, width):
    """No scale, a negative one, and one that leaves a weight or two."""
    for sm in (0.0, -0.05, 1.5):
        s = make([700, 90], [6, 3], Hm=Hm, L=L, act=act, kv=kv, seed=22, width=width)
        s["sm"] = sm
        check(s)
        check(s, 100, 3)


@pytest.mark.parametrize("Hm,ps", [(64, 64), (16, 16), (64, 5)])
def test_chunk_e4m3_queries_with_a_large_element(Hm, ps):
    """A query element far above the others, in a latent column where the keys are small, so
    that the others make the logits.  The queries' 8-bit parts are off by at most 2^-21 of a
    row's largest element (the widened rows' kernel: not at all): 2^-21 max|q| sum|c| of a
    logit."""
    s = make([900, 40], [5, 3], Hm=Hm, kv=F8, ps=ps, seed=23)
    vals = ref.values(s["pages"], s["scale"])
    vals[:, 7] *= 1e-4
    codes, scale = ref.quantise(torch.nan_to_num(vals).float())
    s["pages"], s["scale"] = codes, scale
    for big in (30.0, 1000.0, 30000.0):
        s["q"][:, :, 7] = big
        s["q"][:, ::2, 7] = -big
        out, lse, st = attend(s)
        assert st == 0
        live = int(s["cu"][-1])
        largest = ref.values(s["pages"], s["scale"]).abs().sum(1).max()
        more = 2.0 ** -21 * s["q"].double().abs().amax(2) * largest * s["sm"]
        ref.check_attend(out, lse, reference(s), BF, 512, rows=torch.arange(live, device=DEV),
                         dz_more=more, out_more=ref.underflow(s["pages"], s["scale"], BF))


@pytest.mark.parametrize("act,Hm,L,ps,width", [(BF, 64, 512, 16, 0), (BF, 64, 512, 16, WIDE),
                                               (BF, 16, 512, 5, 0), (F32, 4, 64, 16, 0)])
def test_chunk_logits_all_minus_infinity(act, Hm, L, ps, width):
    """As nothing seen, but for the latent column of the infinity."""
    s = make([1], [1], Hm=Hm, L=L, act=act, kv=act, ps=ps, seed=37, width=width, pad=0)
    s["q"][:, :, 5] = -1.0
    s["pages"][s["table"][0, 0].long() * ps, 5] = math.inf
    out, lse, st = attend(s)
    rest = torch.arange(L, device=DEV) != 5
    assert st == 0 and bool((lse == -math.inf).all()) and bool((out[:, :, rest] == 0).all())
    assert torch.isnan(out[:, :, 5].float()).all()


def e4m3_step(rows, scales=None, Hm=64, ps=64, n_new=3, seed=32, q=None):
    """One sequence whose cache holds the given rows (E4M3 codes made from them; ``scales``: of
    the codes of rows with a largest magnitude of 448) and its last tokens' queries."""
    n = rows.shape[0]
    s = make([n], [n_new], Hm=Hm, kv=F8, ps=ps, seed=seed, pad=0, hidden=0.0)
    codes, sc = ref.quantise(rows)
    p = torch.arange(n, device=DEV)
    at = s["table"][0].long()[p // ps] * ps + p % ps
    s["pages"].view(torch.uint8)[at] = codes.view(torch.uint8)
    s["scale"].fill_(1.0)
    s["scale"][at] = sc if scales is None else scales
    if q is not None:
        s["q"] = q.to(BF).contiguous()
    return s, at


def check_e4m3(s, at, zero=(), shift=0):
    """Against 64 bits; what E5M2 weights lose is relative to the largest weight times row scale
    of the rows seen that are not zero.  The comparison is made 2^shift higher, by rows times
    that and queries divided by it (which leaves the logits)."""
    out, lse, st = attend(s)
    assert st == 0
    out = out.double() * 2.0 ** shift
    assert torch.isfinite(out).all()
    s = dict(s, q=s["q"].double() * 2.0 ** -shift, scale=s["scale"].double() * 2.0 ** shift)
    keep = torch.ones(at.shape[0], dtype=torch.bool, device=DEV)
    keep[list(zero)] = False
    more = 0.0
    if s["ps"] % 8 == 0:
        # a product u = weight * scale at the reference or above is 2^8 and more in E5M2; the
        # output is the sum of u * code over the sum of the weights, so it is off by at most 3 *
        # 2^-25 sum|code| max(u) / sum of the weights, max(u) over rows that are not zero
        vals = ref.values(s["pages"], s["scale"])[at]
        z = torch.einsum("thl,nl->thn", s["q"].double(), vals) * s["sm"]
        n, m = at.shape[0], s["T"]
        see = torch.arange(n, device=DEV)[None] <= n - m + torch.arange(m, device=DEV)[:, None]
        w = torch.softmax(z.masked_fill(~see[:, None], -math.inf), -1)
        u = (w * s["scale"][at].double())[:, :, keep].amax(-1)
        codes = s["pages"][at].float().abs().double().sum(0)
        more = 3 * 2.0 ** -25 * codes * u[..., None]
    ref.check_attend(out, lse, reference(s), BF, 512, out_more=more)
    return out


@pytest.mark.parametrize("Hm,ps", [(64, 64), (16, 64), (32, 64), (64, 5)])
@pytest.mark.parametrize("size,toward", [(0.01, 0.0), (1e-2, -9.0), (1e-3, -4.0), (1e-5, 0.0),
                                         (1e-5, 3.0)])
def test_chunk_e4m3_zero_rows(Hm, ps, size, toward):
    """All-zero rows (stored with a scale of 1) among small ones: their weights count, their
    scale does not.  ``toward``: the small rows' logits against the zero rows', base e."""
    g = torch.Generator(device=DEV).manual_seed(33)
    n, zero = 700, [0, 5, 130, 131, 500, 698]
    rows = torch.randn((n, 512), generator=g, device=DEV) * size
    rows[:, 3] = 2.0 * size
    rows[zero] = 0.0
    q = torch.randn((3, Hm, 512), generator=g, device=DEV) * 0.1
    q[:, :, 3] = toward * math.sqrt(512.0) / (2.0 * size)
    s, at = e4m3_step(rows, Hm=Hm, ps=ps, q=q)
    assert bool((s["scale"][at[zero]] == 1.0).all())
    check_e4m3(s, at, zero)


@pytest.mark.parametrize("Hm,ps", [(64, 64), (16, 64), (32, 64), (64, 5)])
@pytest.mark.parametrize("size", [-90, -104, -118, -125, -130])
def test_chunk_e4m3_small_queries(Hm, ps, size):
    """Queries of 2^size (2^-130: multiples of the least bf16 value), a softmax scale and row
    scales that make their logits ordinary."""
    g = torch.Generator(device=DEV).manual_seed(35)
    rows = torch.randn((300, 512), generator=g, device=DEV)
    q = torch.randn((3, Hm, 512), generator=g, device=DEV) * 2.0 ** size
    s, at = e4m3_step(rows, torch.full((300,), 2.0 ** 110, device=DEV), Hm=Hm, ps=ps, q=q)
    s["sm"] *= 2.0 ** (-118 - size)
    check_e4m3(s, at, shift=-110)


@pytest.mark.parametrize("Hm,ps", [(64, 64), (16, 64), (32, 64), (64, 5)])
@pytest.mark.parametrize("lo,hi,zeros", [(-30, 0, 0), (-10, 0, 0), (-62, -58, 0), (-70, -70, 0),
                                         (-100, -100, 0), (-100, -100, 4), (-115, -80, 0),
                                         (40, 60, 0), (100, 110, 0), (95, 110, 4)])
def test_chunk_e4m3_row_scales_of_every_size(Hm, ps, lo, hi, zeros):
    """Row scales of 2^lo to 2^hi, in every order, with all-zero rows of scale 1 among them;
    on one CTA's share (700 rows) and on many (9,000)."""
    for n, n_new in ((700, 3), (9000, 1)):
        g = torch.Generator(device=DEV).manual_seed(34)
        zero = list(range(0, n, n // zeros)) if zeros else []
        rows = torch.randn((n, 512), generator=g, device=DEV)
        rows[zero] = 0.0
        lg = lo + (hi - lo) * torch.rand(n, generator=g, device=DEV)
        scales = torch.exp2(lg)
        scales[zero] = 1.0
        q = torch.randn((n_new, Hm, 512), generator=g, device=DEV) * 2.0 ** (-8 - hi)
        s, at = e4m3_step(rows, scales, Hm=Hm, ps=ps, n_new=n_new, q=q)
        check_e4m3(s, at, zero, shift=-hi)


@pytest.mark.parametrize("Hm,ps", [(64, 64), (16, 64), (32, 64), (64, 5)])
@pytest.mark.parametrize("first,last,zeros", [(-60, 0, 0), (0, -60, 0), (-100, -100, 300),
                                              (-20, -100, 40), (60, 0, 130)])
def test_chunk_e4m3_row_scales_along_the_sequence(Hm, ps, first, last, zeros):
    """Row scales from 2^first to 2^last, behind ``zeros`` all-zero rows of scale 1, under 300
    tokens: several tiles of a row one after the other in a CTA."""
    n = 700
    g = torch.Generator(device=DEV).manual_seed(36)
    rows = torch.randn((n, 512), generator=g, device=DEV)
    scales = torch.exp2(torch.linspace(first, last, n, device=DEV))
    rows[:zeros], scales[:zeros] = 0.0, 1.0
    q = torch.randn((300, Hm, 512), generator=g, device=DEV) * 2.0 ** (-8 - max(first, last))
    s, at = e4m3_step(rows, scales, Hm=Hm, ps=ps, n_new=300, q=q)
    check_e4m3(s, at, range(zeros), shift=-max(first, last))


@pytest.mark.parametrize("n", [1, 3, 200, 9000])
def test_chunk_e4m3_nothing_but_zero_rows(n):
    """Every logit is 0: out 0 and lse log n, the sum of n ones being exact."""
    s, _ = e4m3_step(torch.zeros((n, 512), device=DEV), n_new=1)
    out, lse, st = attend(s)
    assert st == 0 and bool((out == 0).all())
    assert bool(((lse.double() - math.log(n)).abs() <= 2.0 ** -21 + 2.0 ** -22 * math.log(n)).all())


@pytest.mark.parametrize("act,kv,Hm,L", [(BF, BF, 64, 512), (BF, F8, 16, 512), (F32, F32, 4, 64)])
@pytest.mark.parametrize("cols", [3, WIDE // 16])
def test_chunk_lengths_past_the_table_cost_no_more_than_it(act, kv, Hm, L, cols):
    """A length far behind the table's width: flagged, and the tokens see the positions that
    the table has (with a window that has left them: the sinks alone)."""
    ps = 16
    s = make([cols * ps, 40], [1, 40], Hm=Hm, L=L, act=act, kv=kv, ps=ps, seed=17, pad=0)
    s["table"] = s["table"][:, :cols].contiguous()
    long = dict(s, lens=i32([2 ** 31 - 1, 40]))
    for window, sinks in ((0, 0), (2 ** 31 - 1, 0), (1000, 20), (7, 2 ** 31 - 1)):
        out, lse, st = attend(long, window, sinks)
        assert st == ops.DEV_BAD_PAGE
        see = cols * ps if window in (0, 2 ** 31 - 1) else min(sinks, cols * ps)
        first = dict(s, lens=i32([see, 40]), q=s["q"][:1], cu=i32([0, 1, 1]), T=1)
        ref.check_attend(out[:1], lse[:1], reference(first), act, L)
        rest = dict(s, lens=i32([0, 40]), cu=i32([0, 0, 40]), q=s["q"][1:], T=40)
        ref.check_attend(out[1:], lse[1:], reference(rest, window, sinks), act, L)


@pytest.mark.parametrize("kv", [BF, F8])
def test_chunk_of_2_to_the_31_positions(kv):
    """The longest sequence that the lengths can say, on pages of an odd size: 2^24 tiles whose
    last one's rows count past an int.  One page serves all blocks, its rows are alike, so the
    output is a row.  A CTA adds up 2^24 / SMs tiles of eight products in fp32, each sum off by
    at most 2^-23 of itself: 2^4 / SMs of the output in all, a sixteenth of that (one addition
    a tile, 2^-24) of the sum, half as much again for the roundings of weights and result."""
    ps, n = 1001, 2 ** 31 - 1
    g = torch.Generator(device=DEV).manual_seed(30)
    row = torch.randn((1, 512), generator=g, device=DEV)
    pages, scale = ref.quantise(row) if kv == F8 else (row.to(kv), None)
    pages = pages.view(torch.uint8).repeat(ps, 1).view(kv)
    scale = None if scale is None else scale.repeat(ps)
    table = torch.zeros((1, -(-n // ps)), dtype=torch.int32, device=DEV)
    q = torch.randn((1, 16, 512), generator=g, device=DEV).to(BF)
    s = dict(q=q, pages=pages, scale=scale, table=table, lens=i32([n]), cu=i32([0, 1]), ps=ps,
             sm=1.0 / math.sqrt(512), T=1)
    out, lse, st = attend(s)
    assert st == 0
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rel = 16.0 / sms * (1 + 1 / 16 + 0.5)
    want = ref.values(pages, scale)[0]
    assert bool(((out.double() - want).abs() <= rel * want.abs()).all())
    z = (q[0].double() @ want) * s["sm"]
    assert bool((lse[0].double() - z - math.log(n)).abs().max() <= 1.0 / sms + 1e-3)


@pytest.mark.parametrize("kv,Hm,width,ps", [(BF, 64, 0, 64), (BF, 64, WIDE, 64), (BF, 16, 0, 5),
                                            (F8, 64, 0, 64), (F8, 16, 0, 5)])
def test_chunk_gives_up_and_recovers(kv, Hm, width, ps):
    """The failure drill: no tile arrives, the first waits run out after a millisecond, the
    call returns and says so, and the next one is as before."""
    s = make([700, 300], [20, 30], Hm=Hm, kv=kv, ps=ps, seed=18, width=width)
    want = attend(s)
    ops.dsa_set_failure_drill(ops.DSA_DRILL_SKIP_ARM)
    try:
        assert attend(s)[2] == 64            # DSA_DEV_TIMEOUT
    finally:
        ops.dsa_set_failure_drill(0)
    got = attend(s)
    assert got[2] == want[2] == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("width", [0, WIDE])
@pytest.mark.parametrize("kv", [BF, F8])
def test_chunk_infinite_and_nan_queries_stay_in_their_rows(kv, width):
    s = make([300, 40], [5, 3], kv=kv, seed=11, width=width)
    want, want_lse, _ = attend(s)
    s["q"][1, 7] = math.nan
    s["q"][6, 0, 3] = math.inf
    out, lse, _ = attend(s)
    keep = torch.ones((s["T"], 64), dtype=torch.bool, device=DEV)
    keep[1, 7] = keep[6, 0] = False
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], want_lse[keep])
    assert torch.isnan(out[1, 7].float()).all() and torch.isnan(out[6, 0].float()).all()


def test_chunk_same_bits_every_time_and_beside_other_calls():
    a = make([3100, 20, 777], [5, 20, 300], seed=12, width=WIDE)   # (row blocks share their keys)
    b = make([90, 9000], [1, 1], kv=F8, seed=13)
    want_a, want_b = attend(a), attend(b)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(3):
        for x, st in zip((a, b), streams):
            T, Hm, L = x["q"].shape
            out, lse = torch.full_like(x["q"], 7.0), torch.full((T, Hm), 7.0, device=DEV)
            ws = torch.empty(max(16, ops.mla_paged_chunk_workspace_bytes(x["q"], x["pages"])),
                             dtype=torch.uint8, device=DEV)
            torch.cuda.synchronize()
            ops.dsa_mla_paged_chunk(x["q"], x["pages"], x["scale"], x["table"], x["lens"],
                                    x["ps"], x["cu"], 0, 0, x["sm"], out, lse, ws, None, st)
            got.append((out, lse, ws))
    torch.cuda.synchronize()
    for i, (out, lse, _) in enumerate(got):
        want = (want_a, want_b)[i % 2]
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("kv,Hm,width", [(BF, 64, WIDE), (BF, 128, WIDE), (F8, 64, 0), (F8, 16, 0)])
def test_chunk_captured_follows_lengths(kv, Hm, width):
    """A captured call replayed after its lengths and the step's rows have changed."""
    first = make([900, 40, 300], [30, 2, 8], Hm=Hm, kv=kv, seed=27, width=width, pad=0)
    s = {k: v.clone() if torch.is_tensor(v) else v for k, v in first.items()}
    out, lse = torch.full_like(s["q"], 7.0), torch.full((40, Hm), 7.0, device=DEV)
    ws = torch.empty(ops.mla_paged_chunk_workspace_bytes(s["q"], s["pages"]), dtype=torch.uint8,
                     device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.dsa_mla_paged_chunk(s["q"], s["pages"], s["scale"], s["table"], s["lens"], s["ps"],
                                s["cu"], 0, 0, s["sm"], out, lse, ws)
    for now in (first, dict(first, lens=i32([899, 39, 64]), cu=i32([0, 3, 39, 40]))):
        s["lens"].copy_(now["lens"])
        s["cu"].copy_(now["cu"])
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        want = reference(now)
        ref.check_attend(out, lse, want, BF, 512, rows=torch.arange(int(now["cu"][-1]), device=DEV),
                         out_more=ref.underflow(s["pages"], s["scale"], BF))


@pytest.mark.parametrize("kv", [BF, F8])
def test_step_captured_and_replayed(kv):
    """plan -> append -> attention in one CUDA graph, lengths and free list in place: each
    replay is the next decode step.  The steps one by one, uncaptured, give the same."""
    L, Hm, ps, B = 512, 64, 16, 5
    g = torch.Generator(device=DEV).manual_seed(14)
    lens0 = [0, 31, 16, 200, 5]
    x = torch.randn((4, B, L), generator=g, device=DEV).to(BF)
    q = torch.randn((4, B, Hm, L), generator=g, device=DEV).to(BF)

    def state():
        s = make(lens0, [0] * B, kv=kv, ps=ps, seed=15, pad=B, hidden=0.0)
        n_pages = s["pages"].shape[0] // ps + 40
        grow = torch.zeros((40 * ps, L), dtype=kv, device=DEV)
        s["pages"] = torch.cat([s["pages"].view(torch.uint8), grow.view(torch.uint8)]).view(kv)
        if s["scale"] is not None:
            s["scale"] = torch.cat([s["scale"], torch.zeros(40 * ps, device=DEV)])
        s["free"] = torch.arange(n_pages - 40, n_pages, device=DEV).to(torch.int32)
        s["begin"], s["one"] = i32([0]), i32([1] * B)
        for k in ("q_seq", "q_pos", "rows"):
            s[k] = i32([0] * B)
        s["x"], s["out"] = torch.empty_like(x[0]), torch.empty_like(q[0])
        s["lse"] = torch.empty((B, Hm), dtype=F32, device=DEV)
        s["q"] = torch.empty_like(q[0])
        s["ws"] = torch.empty(max(16, ops.mla_paged_chunk_workspace_bytes(s["q"], s["pages"])),
                              dtype=torch.uint8, device=DEV)
        s["st"] = i32([0])
        return s

    def step(s):
        ops.dsa_paged_plan(s["lens"], s["one"], s["free"], s["begin"], s["pages"].shape[0] // ps,
                           ps, s["table"], s["lens"], s["cu"], s["q_seq"], s["q_pos"], s["rows"],
                           s["begin"], status=s["st"])
        ops.dsa_paged_append(s["x"], s["rows"], s["pages"], s["scale"], status=s["st"])
        ops.dsa_mla_paged_chunk(s["q"], s["pages"], s["scale"], s["table"], s["lens"], ps,
                                s["cu"], 0, 0, s["sm"], s["out"], s["lse"], s["ws"], s["st"])

    def outputs(s, i):
        s["x"].copy_(x[i])
        s["q"].copy_(q[i])

    eager, want = state(), []
    for i in range(4):
        outputs(eager, i)
        step(eager)
        want.append((eager["out"].clone(), eager["lse"].clone()))
    s = state()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(s)
    assert s["lens"].tolist() == lens0                 # captured, not run
    for i in range(4):
        outputs(s, i)
        graph.replay()
        assert torch.equal(s["out"], want[i][0]) and torch.equal(s["lse"], want[i][1])
    assert s["lens"].tolist() == [n + 4 for n in lens0] and s["st"].item() == 0
    assert s["begin"].item() == sum(-(-(n + 4) // ps) - -(-n // ps) for n in lens0)
    # the cache holds the appended rows, and the attention read them
    p = torch.full((B,), 3, device=DEV) + i32(lens0)
    rows = s["table"].gather(1, (p // ps).long()[:, None])[:, 0] * ps + p % ps
    have = ref.values(s["pages"], s["scale"])[rows.long()]
    tol = (2.0 ** -4 if kv == F8 else 2.0 ** -8) * x[3].double().abs()
    if kv == F8:  # codes below 2^-6 are 2^-9 apart
        tol = torch.maximum(tol, 2.0 ** -10 * s["scale"][rows.long()].double()[:, None]) * 1.001
    assert bool(((have - x[3].double()).abs() <= tol).all())
    chk = dict(s, T=B)
    ref.check_attend(s["out"], s["lse"], reference(chk), BF, L)


@pytest.mark.parametrize("e4m3", [False, True])
def test_step_as_a_serving_loop_runs_it(e4m3):
    """The framework's own step (pipeline.PagedStep): a plan with the slots of the key cache,
    the append, the dense attention, and the selection with its attention on the plan's
    sequences and positions.  A chunk first, then two decode steps."""
    geo = Geometry(D=128, H=32, kpool=4, select_k=64, out_width=320, Hm=64, L=512, dtype="bf16")
    lengths, ps = [1203, 23, 50], 16
    new = [[5, 20, 1], [1, 1, 1], [1, 1, 1]]           # the rest is in the cache before
    ctx0 = [n - sum(s[b] for s in new) for b, n in enumerate(lengths)]
    bt = synth.make_batch(geo, lengths, [3, 0, 1], device=DEV, seed=19)
    full = synth.paged_cache(bt.kv, bt.cu_seqlens, ps, e4m3=e4m3, seed=20)
    # the cache as it was before the steps: their rows and pages are not there yet
    cu = bt.cu_seqlens.tolist()
    pages = torch.zeros_like(full.pages.view(torch.uint8)).view(full.pages.dtype)
    scale = None if full.row_scale is None else torch.zeros_like(full.row_scale)
    table, free = torch.full_like(full.block_table, -1), []
    for b in range(3):
        held = -(-ctx0[b] // ps)
        table[b, :held] = full.block_table[b, :held]
        p = torch.arange(ctx0[b], device=DEV)
        rows = table[b].long()[p // ps] * ps + p % ps
        pages.view(torch.uint8)[rows] = full.pages.view(torch.uint8)[rows]
        if scale is not None:
            scale[rows] = full.row_scale[rows]
        free += full.block_table[b, held:-(-lengths[b] // ps)].tolist()
    cache = synth.PagedCache(pages, scale, table, i32(ctx0), ps)
    step = pipeline.PagedStep.alloc(cache, i32(free + [0]), 26, 64, bt=bt)
    buf = pipeline.LayerBuffers.alloc(bt)
    pipeline.compress(bt, buf)                         # (pools by their tokens: later ones hidden)
    g = torch.Generator(device=DEV).manual_seed(21)
    done = list(ctx0)
    for n in new:
        T = sum(n)
        pipeline.plan_step(cache, step, i32(n), row_base=bt.cu_seqlens[:3].contiguous())
        pos = [done[b] + i for b in range(3) for i in range(n[b])]
        seq = [b for b in range(3) for _ in range(n[b])]
        done = [d + k for d, k in zip(done, n)]
        assert cache.seq_lens.tolist() == done
        assert step.q_seq[:T].tolist() == seq and step.q_pos[:T].tolist() == pos
        keys = [cu[b] + p for b, p in zip(seq, pos)]
        assert step.key_rows.tolist() == keys + [-1] * (26 - T)
        x = torch.zeros((26, 512), dtype=BF, device=DEV)
        x[:T] = bt.kv[torch.tensor(keys, device=DEV)]
        q_lat = torch.randn((26, 64, 512), generator=g, device=DEV).to(BF)
        pipeline.append_step(cache, step, x)
        pipeline.attend_step(cache, step, q_lat, bt.sm_scale)
        torch.cuda.synchronize()
        vals = ref.values(cache.pages, cache.row_scale)
        want = ref.attend(q_lat, vals, cache.block_table, cache.seq_lens, ps, step.cu_new, 0, 0,
                          bt.sm_scale)
        live = torch.arange(T, device=DEV)
        ref.check_attend(step.out, step.lse, want, BF, 512, rows=live)
        # the selection of the same tokens, and its attention
        q = torch.randn((26, 32, 128), generator=g, device=DEV).to(BF)
        w = torch.randn((26, 32), generator=g, device=DEV)
        pipeline.select_step(bt, buf, step, q, w)
        pipeline.attend_selected_step(cache, step, q_lat, bt.sm_scale)
        torch.cuda.synchronize()
        ids = step.token_ids.tolist()
        assert all(t == -1 for row in ids[T:] for t in row)
        rows64 = []
        for r in range(T):
            t = torch.tensor([t for t in ids[r] if t >= 0], dtype=torch.long, device=DEV)
            assert t.numel() == 0 or int(t.max()) <= pos[r]
            assert t.numel() >= min(256, (pos[r] + 1 - bt.pads[seq[r]]) // 4 * 4)
            rows64.append(cache.block_table[seq[r]].long()[t // ps] * ps + t % ps)
        # the same formula over the selected rows, one row of pages a token
        width = max(len(r) for r in rows64)
        one = torch.full((T, width), -1, dtype=torch.int32, device=DEV)
        for r, rr in enumerate(rows64):
            one[r, :len(rr)] = rr.to(torch.int32)
        want = ref.attend(q_lat[:T], vals, one, i32([len(r) for r in rows64]), 1,
                          i32(list(range(T + 1))), 0, 0, bt.sm_scale)
        ref.check_attend(step.out[:T], step.lse[:T], want, BF, 512)
    assert int(step.status.item()) == 0 and int(buf.status.item()) == 0
    assert cache.block_table.tolist() == full.block_table.tolist()
    assert step.free_begin.item() == len(free)
