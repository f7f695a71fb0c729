"""The grouped-query layer of the paged step on the GPU, against plain 64-bit forms: the append
and the read-back exactly, block scores and attention within the bounds of their roundings, and
the whole step in a captured graph."""
import math
import random
import threading

import pytest
import torch

from sparse_attention_indexer_kpool_gb300 import ops, pipeline, synth
from tests import _gqa_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
NAN_CODE = 0x7f
# half a step of a rounding, relative to the value
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Case:
    """A random cache: sequences of ``lens`` tokens on shuffled pages, the last ``new`` of each
    new.  Rows behind a sequence's end and spare pages hold NaN codes under NaN scales."""

    def __init__(self, seed, lens, new, Hkv, ps, D, spread=3, poison=True, width=None):
        g = torch.Generator().manual_seed(seed)
        self.g, self.lens, self.new, self.Hkv, self.ps, self.D = g, lens, new, Hkv, ps, D
        blocks = [max(0, -(-n // ps)) for n in lens]
        self.n_pages = sum(blocks) + 3
        perm = torch.randperm(self.n_pages, generator=g).tolist()
        width = max(blocks + [1]) + 1 if width is None else width
        self.table, at = [], 0
        for k in blocks:
            self.table.append((perm[at:at + k] + [-1] * width)[:width])
            at += k
        self.cu = [0]
        for n in new:
            self.cu.append(self.cu[-1] + n)
        self.T = self.cu[-1]
        self.codes, self.scale = {}, {}
        for a in "kv":
            x = torch.randn((self.n_pages, Hkv, ps, D), generator=g)
            e = torch.randint(-spread, spread + 1, (self.n_pages, Hkv), generator=g)
            c = (x / x.abs().amax((2, 3), keepdim=True) * 440.0).to(F8).view(torch.uint8)
            s = torch.exp2(e.float() - 6.0)
            if poison:
                used = torch.zeros(self.n_pages, ps, dtype=torch.bool)
                for b, n in enumerate(lens):
                    for t in range(max(n, 0)):
                        if t // ps < width:
                            used[self.table[b][t // ps], t % ps] = True
                c[~used[:, None, :].expand(-1, Hkv, -1)] = NAN_CODE
                s[~used.any(1)] = math.nan
            self.codes[a], self.scale[a] = c, s

    def normal(self, *shape, std=1.0, dtype=BF):
        return (torch.randn(shape, generator=self.g) * std).to(dtype)

    def put(self):
        """(k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, cu_new) on the GPU."""
        c, s = self.codes, self.scale
        return (c["k"].clone().to(DEV).view(F8), c["v"].clone().to(DEV).view(F8),
                s["k"].clone().to(DEV), s["v"].clone().to(DEV), i32(self.table), i32(self.lens),
                i32(self.cu))

    def plain(self, a):
        return ref.values(self.codes[a]), self.scale[a].double()


def spread_lens(seed, B, hi, new_hi):
    rng = random.Random(seed)
    new = [rng.randint(0, new_hi) for _ in range(B)]
    return [n + rng.randint(0, hi) for n in new], new


# ---------------------------------------------------------------- append
def check_append(c, k_new, v_new, mean=True, fault=0, T_pad=0):
    args = c.put()
    kp, vp, ks, vs, table, lens, cu = args
    k_mean = torch.full((c.n_pages, c.Hkv, c.D), 7.0, dtype=BF, device=DEV)
    st = i32([0])
    pad = lambda x: torch.cat([x, x.new_full((T_pad,) + x.shape[1:], 99.0)]).to(DEV)  # noqa: E731
    ops.dsa_gqa_append(pad(k_new), pad(v_new), *args, k_mean=k_mean if mean else None, status=st)
    torch.cuda.synchronize()
    assert st.item() == fault
    want_mean = torch.full((c.n_pages, c.Hkv, c.D), 7.0, dtype=torch.float64)
    for a, new, got, got_s in (("k", k_new, kp, ks), ("v", v_new, vp, vs)):
        pages, scale = c.plain(a)
        ref.append(new, pages, scale, c.table, c.lens, c.cu, c.ps,
                   want_mean if a == "k" and mean else None)
        assert torch.equal(got_s.cpu().double().nan_to_num(-1.0), scale.nan_to_num(-1.0)), a
        x = ref.values(got.cpu())
        assert torch.equal(torch.isnan(x), torch.isnan(pages)), a
        assert torch.equal(x.nan_to_num(), pages.nan_to_num()), a
    m = k_mean.cpu().double()
    assert torch.equal(torch.isnan(m), torch.isnan(want_mean))
    # one rounding to bf16 of a sum of ps codes in fp32 (each at most 448 of the scale), times
    # 2^e / ps rounded once and the product rounded once
    m, want_mean = m.nan_to_num(), want_mean.nan_to_num()
    tol = want_mean.abs() * (HALF[BF] + 2.0 ** -22) + c.ps * 2.0 ** -24 * want_mean.abs().max()
    assert bool(((m - want_mean).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,hi,new_hi,Hkv,ps,D", [
    (1, 0, 1, 1, 16, 16), (1, 0, 200, 2, 16, 64), (5, 100, 1, 8, 64, 128), (7, 90, 70, 3, 32, 80),
    (3, 300, 300, 4, 64, 128), (2, 40, 500, 2, 48, 256), (40, 30, 9, 1, 16, 32),
    (2, 1500, 1200, 2, 1024, 48)])
def test_append(B, hi, new_hi, Hkv, ps, D, dtype):
    lens, new = spread_lens(B + ps, B, hi, new_hi)
    if sum(new) == 0:
        lens[0], new[0] = lens[0] + 1, 1
    c = Case(ps + D, lens, new, Hkv, ps, D)
    up = torch.exp2(torch.randn((c.T, Hkv, 1), generator=c.g) * 2.0)   # some scales grow
    x, y = c.normal(c.T, Hkv, D, dtype=F32) * up, c.normal(c.T, Hkv, D, dtype=F32) * up
    check_append(c, x.to(dtype), y.to(dtype), T_pad=5)
    check_append(c, x.to(dtype), y.to(dtype), mean=False)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_extreme_values(dtype):
    """Zeros, tiny and huge rows, exact powers and maxima at the borders of an exponent, infinities
    and NaN."""
    tops = [0.0, 448.0, 449.0, 447.0, 1.75, 1.7578125, 2.0 ** -70, 2.0 ** -56, 448 * 2.0 ** -64,
            2.0 ** -126, 2.0 ** -140, 3.0e38, 2.0 ** 127, 1.0e-30, math.inf, math.nan]
    lens = [16 + 5] * len(tops)
    c = Case(3, lens, [20] * len(tops), 2, 16, 32)
    x = torch.randn((c.T, 2, 32), generator=c.g).clamp(-3, 3) / 3.0
    for i, top in enumerate(tops):
        blk = x[c.cu[i]:c.cu[i + 1]]
        if math.isfinite(top):
            blk *= top
            blk[::4, :, 5] = top
        else:
            blk[3, 1, 7] = top
            blk[18, 0, 9] = -top
    check_append(c, x.to(dtype), (-x).to(dtype))


def test_append_in_pieces_and_again():
    """Tokens appended one by one and in chunks end at the same scales; codes differ where a value
    below 2^-6 of the scale was rounded twice.  The same call again changes nothing."""
    n, Hkv, ps, D = 150, 2, 64, 64
    g = torch.Generator().manual_seed(5)
    x = (torch.randn((n, Hkv, D), generator=g) * torch.exp2(torch.randn((n, 1, 1), generator=g))
         ).to(BF)
    whole = Case(1, [n], [n], Hkv, ps, D)
    done = {}
    for name, cuts in (("whole", [n]), ("pieces", [1, 2, 3, 64, 65, 100, 128, 129, 149, 150])):
        kp, vp, ks, vs, table, _, _ = whole.put()
        mean = torch.zeros((whole.n_pages, Hkv, D), dtype=BF, device=DEV)
        at = 0
        for cut in cuts:
            for _ in range(2):
                ops.dsa_gqa_append(x[at:cut].to(DEV), x[at:cut].to(DEV), kp, vp, ks, vs, table,
                                   i32([cut]), i32([0, cut - at]), k_mean=mean)
            at = cut
        done[name] = [t.cpu() for t in (kp, ks, mean)] + [vp.cpu(), vs.cpu()]
    for i in (1, 4):
        assert torch.equal(done["whole"][i].nan_to_num(-1.0), done["pieces"][i].nan_to_num(-1.0))
    pages, scale = ref.values(done["whole"][0]), done["whole"][1].double()
    other = ref.values(done["pieces"][0])
    for t in range(n):
        pg = whole.table[0][t // ps]
        a, b = pages[pg, :, t % ps], other[pg, :, t % ps]
        # twice half of E4M3's least step, 2^-9
        assert bool(((a - b).abs() <= torch.where(a.abs() < 2.0 ** -6, 2.0 ** -9, 0.0)).all())


def test_append_faults():
    c = Case(2, [40, 70, 33, 200], [10, 70, 2, 30], 2, 16, 32)
    c.table[0][2] = 10 ** 6
    c.table[1][0], c.table[1][3] = -5, c.n_pages
    x = c.normal(c.T, 2, 32)
    check_append(c, x, x, fault=ops.DEV_BAD_PAGE)
    narrow = Case(4, [40, 70], [10, 70], 2, 16, 32, width=3)
    x = narrow.normal(narrow.T, 2, 32)
    check_append(narrow, x, x, fault=ops.DEV_BAD_PAGE)
    # fewer positions than new tokens: the rows before position 0 go nowhere
    c = Case(6, [12], [12], 1, 16, 32)
    x = c.normal(20, 1, 32).to(DEV)
    kp, vp, ks, vs, table, lens, _ = c.put()
    st = i32([0])
    ops.dsa_gqa_append(x, x, kp, vp, ks, vs, table, lens, i32([0, 20]), status=st)
    assert st.item() == ops.DEV_BAD_LENGTH
    pages, scale = c.plain("k")
    ref.append(x[8:].cpu(), pages, scale, c.table, [12], [0, 12], 16)
    assert torch.equal(ref.values(kp.cpu()).nan_to_num(), pages.nan_to_num())
    # nothing to do
    before = kp.view(torch.uint8).clone()
    ops.dsa_gqa_append(x, x, kp, vp, ks, vs, table, lens, i32([0, 0]), status=st)
    ops.dsa_gqa_append(x[:0], x[:0], kp, vp, ks, vs, table, lens, i32([0, 0]), status=st)
    assert torch.equal(kp.view(torch.uint8), before)


# ---------------------------------------------------------------- read
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,hi,Hkv,ps,D", [(1, 1, 1, 16, 16), (3, 100, 2, 16, 64),
                                           (9, 300, 8, 64, 128), (2, 90, 3, 48, 80)])
def test_read(B, hi, Hkv, ps, D, dtype):
    rng = random.Random(B + ps)
    lens = [rng.randint(1, hi) for _ in range(B)]
    c = Case(D, lens, [0] * B, Hkv, ps, D)
    begin = [rng.randint(0, n - 1) for n in lens]
    count = [rng.randint(0, n - f) for n, f in zip(lens, begin)]
    for first in (begin, None):
        cu = [0]
        for n in count:
            cu.append(cu[-1] + n)
        T = cu[-1] + 3
        kp, vp, ks, vs, table, sl, _ = c.put()
        out = [torch.full((T, Hkv, D), 5.0, dtype=dtype, device=DEV) for _ in "kv"]
        st = i32([0])
        ops.dsa_gqa_read(kp, vp, ks, vs, table, sl, i32(cu), *out,
                         begin=None if first is None else i32(first), status=st)
        assert st.item() == 0
        for a, got in zip("kv", out):
            pages, scale = c.plain(a)
            got = got.cpu().double()
            for b in range(B):
                f = 0 if first is None else first[b]
                want = ref.rows(pages, scale, c.table[b], range(f, f + count[b]))
                assert torch.equal(got[cu[b]:cu[b + 1]], want)   # exact: 4 bits times 2^e
            assert bool((got[cu[-1]:] == 5.0).all())


def test_read_faults():
    c = Case(1, [40, 20], [0, 0], 2, 16, 32)
    c.table[0][1] = 999
    kp, vp, ks, vs, table, lens, _ = c.put()
    out = [torch.full((40, 2, 32), 5.0, device=DEV) for _ in "kv"]
    st = i32([0])
    ops.dsa_gqa_read(kp, vp, ks, vs, table, lens, i32([0, 36, 40]), *out, begin=i32([-1, 18]),
                     status=st)
    assert st.item() == ops.DEV_BAD_PAGE | ops.DEV_BAD_LENGTH
    pages, scale = c.plain("v")
    want = torch.cat([torch.zeros((1, 2, 32), dtype=torch.float64),
                      ref.rows(pages, scale, c.table[0], range(35)).nan_to_num(),
                      ref.rows(pages, scale, c.table[1], range(18, 20)),
                      torch.zeros((2, 2, 32), dtype=torch.float64)])
    assert torch.equal(out[1].cpu().double(), want)


# ---------------------------------------------------------------- block scores
def check_scores(c, G, dtype, sinks, local, NB=None, fault=0, std=2.0, T_pad=2):
    q = c.normal(c.T + T_pad, c.Hkv * G, c.D, std=std, dtype=dtype)
    means = c.normal(c.n_pages, c.Hkv, c.D, std=0.5)
    held = torch.zeros(c.n_pages, dtype=torch.bool)
    for b, n in enumerate(c.lens):
        for j in range(min(max(n, 0) // c.ps, len(c.table[b]))):
            if 0 <= c.table[b][j] < c.n_pages:
                held[c.table[b][j]] = True
    means[~held] = math.nan                       # incomplete and spare blocks
    NB = len(c.table[0]) if NB is None else NB
    sm = 1.0 / math.sqrt(c.D)
    out = torch.full((c.T + T_pad, c.Hkv, NB), 5.0, device=DEV)
    st = i32([0])
    ops.dsa_gqa_block_scores(q.to(DEV), means.to(DEV), i32(c.table), i32(c.lens), c.ps, i32(c.cu),
                             sinks, local, sm, out, status=st)
    torch.cuda.synchronize()
    assert st.item() == fault
    want, big = ref.scores(q[:c.T], means, c.table, c.lens, c.cu, c.ps, sinks, local, sm, NB)
    got = out.cpu().double()
    assert bool((got[c.T:] == 5.0).all())
    got, fin = got[:c.T], torch.isfinite(want)
    assert torch.equal(got[~fin], want[~fin])
    # a logit is a sum of D products in fp32 (the tensor cores add in another order and cut off
    # where fp32 rounds: twice a half step a term), in base 2 by a factor rounded twice, and the
    # maximum's taken off; the weight is 2^z (2^-22) over a sum of NB of them; G are added
    dz = big * (2 * c.D * 2.0 ** -24 + 8 * 2.0 ** -24)
    tol = want[fin].abs() * (4 * dz + (NB + G) * 2.0 ** -24 + 2.0 ** -20) + 2.0 ** -126
    assert bool(((got[fin] - want[fin]).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens,new,Hkv,G,ps,D,sinks,local", [
    ([1], [1], 1, 1, 16, 16, 0, 0), ([40, 15, 16], [1, 1, 1], 2, 4, 16, 64, 1, 1),
    ([700, 90, 33], [1, 30, 33], 2, 8, 16, 128, 1, 2), ([1200], [70], 1, 16, 32, 128, 0, 1),
    ([500, 0, 320], [2, 0, 40], 3, 5, 16, 80, 2, 0), ([400], [3], 2, 32, 16, 64, 1, 1),
    ([900, 900], [16, 17], 1, 128, 64, 128, 0, 3), ([2100], [9], 8, 2, 16, 64, 1, 4)])
def test_scores(lens, new, Hkv, G, ps, D, sinks, local, dtype):
    check_scores(Case(ps + G, lens, new, Hkv, ps, D), G, dtype, sinks, local)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scores_narrow_and_faults(dtype):
    c = Case(7, [300, 200], [20, 3], 2, 16, 64)
    check_scores(c, 8, dtype, 1, 1, NB=7, fault=ops.DEV_POOL_RANGE)
    check_scores(c, 8, dtype, 1, 1, NB=40)
    check_scores(c, 8, dtype, 0, 2, std=60.0)     # weights far below the largest
    c.table[0][3] = -9
    check_scores(c, 8, dtype, 0, 1, fault=ops.DEV_BAD_PAGE)
    c = Case(8, [300, 200], [20, 3], 2, 16, 64, width=5)
    check_scores(c, 8, dtype, 1, 1, NB=9, fault=ops.DEV_BAD_PAGE | ops.DEV_POOL_RANGE)


# ---------------------------------------------------------------- attention
def run_attend(c, q, sm, window=0, sinks=0, ids=None, put=None, **kw):
    args = put or c.put()
    T, Hq, D = q.shape
    out = torch.full((T, Hq, D), 5.0, dtype=q.dtype, device=DEV)
    lse = torch.full((T, Hq), 5.0, device=DEV)
    st = i32([0])
    qd = q.to(DEV)
    n = ops.gqa_attend_workspace_bytes(qd, args[0])
    ws = torch.full((max(n, 16),), 0xff, dtype=torch.uint8, device=DEV)
    ops.dsa_gqa_attend(qd, *args, window, sinks, sm, out, lse, ws,
                       block_ids=None if ids is None else ids.to(DEV), status=st, **kw)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu(), st.item()


def check_attend(c, G, dtype, window=0, sinks=0, K=0, std=2.0, fault=0, ids=None, T_pad=2):
    Hq = c.Hkv * G
    q = c.normal(c.T + T_pad, Hq, c.D, std=std, dtype=dtype)
    sm = 1.0 / math.sqrt(c.D)
    if K:
        ids = random_ids(c, K, T_pad)
    out, lse, st = run_attend(c, q, sm, window, sinks, ids)
    assert st == fault
    assert bool((out[c.T:] == 5.0).all()) and bool((lse[c.T:] == 5.0).all())
    compare(c, q, sm, out, lse, dtype, window, sinks, ids)


def compare(c, q, sm, out, lse, dtype, window=0, sinks=0, ids=None, dense=False):
    kp, ks = c.plain("k")
    vp, vs = c.plain("v")
    if dense:
        want, want_lse, mass, top, big = ref.attend_dense(
            q[:c.T].to(DEV), kp.to(DEV), ks.to(DEV), vp.to(DEV), vs.to(DEV), c.table, c.lens, c.cu,
            sm, window, sinks)
        want, want_lse, mass, top = want.cpu(), want_lse.cpu(), mass.cpu(), top.cpu()
    else:
        want, want_lse, mass, top, big = ref.attend(
            q[:c.T], kp, ks, vp, vs, c.table, c.lens, c.cu, sm, window, sinks,
            None if ids is None else ids[:c.T])
    out, lse = out[:c.T].double(), lse[:c.T].double()
    n = max(c.lens + [1]) if ids is None else ids.shape[2] * c.ps
    # A logit: D products added in fp32 (in the tensor cores: cut off, two half steps a term),
    # its factors rounded a few times, the reference's taken off.  A weight: 2^z (2^-22), and on
    # the bf16 path its rounding to fp16, 2^-8 of itself at most; sums of n.  The output: rounded
    # once.  fp16 ends: a weight times its value's scale is held times 2^2 of the reference, which
    # is at most the row's largest such product, in steps of 2^-24, so that it is off by 2^-27 of
    # the largest at most, times a code of at most 448, for each of n keys.
    dz = big * (2 * c.D * 2.0 ** -24 + 8 * 2.0 ** -24)
    w = 2 * dz + n * 2.0 ** -24 + 2.0 ** -20
    lost = 2.0 ** -8 if dtype == BF else 0.0
    tol = HALF[dtype] * want.abs() + (2 * w + lost) * (mass + want.abs()) + 2.0 ** -126
    if dtype == BF:
        tol = tol + 448 * 2.0 ** -27 * top[..., None]
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(out), nan)
    worst = ((out - want).abs() - tol)[~nan]
    assert worst.numel() == 0 or float(worst.max()) <= 0.0
    fin = torch.isfinite(want_lse)
    assert torch.equal(torch.isnan(lse), torch.isnan(want_lse))
    assert torch.equal(lse[~fin].nan_to_num(7.0), want_lse[~fin].nan_to_num(7.0))
    ltol = w + want_lse[fin].abs() * 2.0 ** -22
    assert bool(((lse[fin] - want_lse[fin]).abs() <= ltol).all())


def random_ids(c, K, T_pad=0):
    """Own block somewhere in the list, others at random, some entries empty, one row all empty."""
    rng = random.Random(c.T)
    ids = torch.full((c.T + T_pad, c.Hkv, K), -1, dtype=torch.int32)
    for b, n in enumerate(c.new):
        for i in range(n):
            mine = (c.lens[b] - n + i) // c.ps
            for h in range(c.Hkv):
                pick = rng.sample(range(mine + 1), min(mine + 1, rng.randint(0, K)))
                if mine not in pick and pick:
                    pick[0] = mine
                pick += [-1] * (K - len(pick))
                rng.shuffle(pick)
                ids[c.cu[b] + i, h] = torch.tensor(pick, dtype=torch.int32)
    if c.T:
        ids[c.T - 1, 0] = -1
    return ids


SHAPES = [  # lens, new, Hkv, G, ps, D
    ([1], [1], 1, 1, 16, 16), ([1, 17, 16, 33], [1, 1, 1, 1], 2, 4, 16, 64),
    ([300, 0, 5, 1000], [1, 0, 5, 1], 2, 8, 64, 128), ([257], [1], 8, 8, 16, 128),
    ([130, 200], [40, 3], 1, 16, 32, 128), ([90, 500, 64], [90, 2, 64], 3, 5, 48, 128),
    ([400], [2], 1, 128, 16, 64), ([333, 20], [1, 20], 2, 20, 128, 64),
    ([150, 70], [30, 70], 2, 3, 16, 80), ([200], [9], 1, 7, 64, 256), ([700], [1], 1, 1, 16, 32)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (40, 0), (64, 3), (20, 70)])
@pytest.mark.parametrize("lens,new,Hkv,G,ps,D", SHAPES)
def test_attend(lens, new, Hkv, G, ps, D, window, sinks, dtype):
    check_attend(Case(ps + G, lens, new, Hkv, ps, D), G, dtype, window, sinks)


def check_dense(c, G, window=0, sinks=0, std=2.0, q=None, sm=None):
    q = c.normal(c.T + 1, c.Hkv * G, c.D, std=std) if q is None else q
    sm = 1.0 / math.sqrt(c.D) if sm is None else sm
    out, lse, st = run_attend(c, q, sm, window, sinks)
    assert st == 0
    assert bool((out[c.T:] == 5.0).all()) and bool((lse[c.T:] == 5.0).all())
    compare(c, q, sm, out, lse, BF, window, sinks, dense=True)


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 0), (300, 200), (1, 1), (700, 5)])
@pytest.mark.parametrize("lens,new,Hkv,G,ps,D", [
    ([1500], [700], 2, 16, 64, 128), ([900, 40, 1, 400], [300, 40, 1, 129], 1, 8, 32, 128),
    ([600, 333], [64, 333], 2, 5, 48, 128), ([520], [520], 1, 64, 16, 128),
    ([300, 1100], [17, 90], 4, 1, 128, 64), ([700], [200], 1, 128, 64, 64),
    ([2100], [33], 8, 3, 256, 128), ([4000, 3000, 5], [9, 60, 5], 2, 12, 64, 64)])
def test_attend_chunks(lens, new, Hkv, G, ps, D, window, sinks):
    check_dense(Case(ps + G, lens, new, Hkv, ps, D), G, window, sinks)


@pytest.mark.parametrize("window", [0, 400])
def test_attend_chunks_rising_logits(window):
    """Keys that grow along the sequence, so that references are raised again and again, in the
    middle of a tile and over several of them; and some that fall."""
    for grow in (8.0, -8.0):
        c = Case(41, [1300, 700], [200, 90], 1, 16, 128, spread=0)
        for row, n in zip(c.table, c.lens):
            blocks = -(-n // 16)
            for j in range(blocks):
                c.scale["k"][row[j]] = 2.0 ** (-7 + round(grow * j / blocks))
        check_dense(c, 16, window)
    # single keys far above the rest, at every place of a tile
    c = Case(42, [700], [150], 1, 64, 128, spread=0)
    for t in range(0, 700, 37):
        c.codes["k"][c.table[0][t // 64], 0, t % 64] = 0x7e     # 448
    q = c.normal(c.T + 1, 16, 128).abs()
    check_dense(c, 16, window, q=q, sm=0.5)


def test_attend_chunks_scales_far_apart():
    for lo, hi in ((-64, 100), (-30, 30), (-64, -64), (40, 100)):
        c = Case(43, [500, 300], [80, 90], 1, 16, 128)
        e = torch.randint(0, 2, c.scale["v"].shape, generator=c.g) * (hi - lo) + lo
        c.scale["v"] = torch.where(torch.isnan(c.scale["v"]), c.scale["v"], torch.exp2(e.float()))
        c.codes["v"][c.table[0][1], 0] = 0
        check_dense(c, 8)
        c.scale["k"] = torch.where(torch.isnan(c.scale["k"]), c.scale["k"], 2.0 ** 2)
        check_dense(c, 8, std=0.1)


def test_attend_chunks_nan():
    """NaN codes in keys and values at many places, on and beside the diagonal and the window's
    edge: what sees them is NaN, nothing else."""
    for window, sinks in ((0, 0), (130, 0), (60, 20)):
        c = Case(44, [700, 260], [300, 200], 2, 64, 128)
        rng = random.Random(3)
        for b, n in enumerate(c.lens):
            for _ in range(12):
                t = rng.randrange(n - c.new[b] // 2, n)
                row = c.codes["v"][c.table[b][t // 64], rng.randrange(2), t % 64]
                row[rng.randrange(128)] = 0x7f
            t = n - 20
            c.codes["k"][c.table[b][t // 64], 1, t % 64, 5] = 0xff
        c.codes["v"][c.table[0][0], 0, 3, 77] = 0xff
        q = c.normal(c.T + 1, 16, 128)
        q[7, 2, 9], q[250, 12, 0] = math.nan, -math.inf
        out, lse, st = run_attend(c, q, 0.1, window, sinks)
        assert bool(torch.isnan(out[7, 2]).all()) and bool(torch.isnan(lse[250, 12]).all())
        q[7, 2], q[250, 12] = 0.0, 0.0
        clean = run_attend(c, q, 0.1, window, sinks)
        compare(c, q, 0.1, clean[0], clean[1], BF, window, sinks, dense=True)
        for t, h in ((7, 2), (250, 12)):
            out[t, h], lse[t, h] = clean[0][t, h], clean[1][t, h]
        assert torch.equal(out.nan_to_num(9.0), clean[0].nan_to_num(9.0))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [1, 3, 10])
@pytest.mark.parametrize("lens,new,Hkv,G,ps,D", SHAPES)
def test_attend_blocks(lens, new, Hkv, G, ps, D, K, dtype):
    check_attend(Case(ps + G, lens, new, Hkv, ps, D), G, dtype, K=K)


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
@pytest.mark.parametrize("lens,new,Hkv,G,ps,D", SHAPES[:8] + [
    ([5000, 1, 3000, 700], [1, 1, 2, 1], 2, 8, 64, 128), ([9000], [1], 1, 16, 16, 128),
    ([4000, 2500], [2, 3], 4, 4, 32, 64)])
def test_attend_by_shares(lens, new, Hkv, G, ps, D, window, sinks):
    """The same under a table so wide that a step's keys may be many: their tiles are then shared
    out over all warps and the partials joined by a second kernel."""
    c = Case(ps + G, lens, new, Hkv, ps, D, width=40_000 // ps)
    if max(lens) > 2000:
        check_dense(c, G, window, sinks)
    else:
        check_attend(c, G, BF, window, sinks)


@pytest.mark.parametrize("K", [40, 300])
def test_attend_blocks_by_shares(K):
    """Long lists, and more row tiles than SMs."""
    c = Case(50, [900, 300, 40], [20, 30, 2], 4, 16, 128)
    check_attend(c, 8, BF, K=K)
    c = Case(51, [5000], [1], 2, 16, 128)
    check_attend(c, 16, BF, K=K)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_blocks_listed_oddly(dtype):
    """The same block twice counts twice; blocks behind the token's own are not seen; past the
    table they are no error where the token does not reach them."""
    c = Case(11, [100, 40], [2, 1], 2, 16, 128)
    ids = torch.tensor([[0, 0, 6], [5, 6, 99], [2, 1, 1]], dtype=torch.int32)
    ids = ids[:, None, :].repeat(1, 2, 1).contiguous()
    ids[0, 1] = torch.tensor([-3, 2 ** 31 - 1, -2 ** 31])
    check_attend(c, 8, dtype, ids=ids, T_pad=0)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_faults(dtype):
    for K in (0, 20):
        c = Case(12, [300, 120], [3, 30], 2, 16, 128)
        c.table[0][2], c.table[0][9], c.table[1][7] = -1, 10 ** 6, c.n_pages
        check_attend(c, 8, dtype, fault=ops.DEV_BAD_PAGE,
                     ids=None if not K else torch.arange(K, dtype=torch.int32).expand(
                         c.T + 2, 2, K).contiguous())
    narrow = Case(13, [300, 120], [3, 30], 2, 16, 128, width=4)
    check_attend(narrow, 8, dtype, fault=ops.DEV_BAD_PAGE)
    check_attend(narrow, 8, dtype, fault=ops.DEV_BAD_PAGE, window=30, sinks=5)
    # rows without a position see nothing
    c = Case(14, [5], [5], 1, 16, 128)
    q = c.normal(9, 8, 128, dtype=dtype)
    kp, vp, ks, vs, table, lens, _ = c.put()
    out, lse, st = run_attend(c, q, 0.1, put=(kp, vp, ks, vs, table, lens, i32([0, 9])))
    assert st == ops.DEV_BAD_LENGTH
    assert bool((out[:4] == 0).all()) and bool((lse[:4] == -math.inf).all())
    c.lens, c.new, c.cu, c.T = [5], [5], [0, 5], 5
    compare(c, q[4:], 0.1, out[4:], lse[4:], dtype)
    # a length below zero, no new tokens anywhere, fewer tokens than rows
    kp, vp, ks, vs, table, lens, _ = c.put()
    for ln, cu in (([-7], [0, 9]), ([5], [0, 0]), ([5], [9, 9])):
        out, lse, st = run_attend(c, q, 0.1, put=(kp, vp, ks, vs, table, i32(ln), i32(cu)))
        if ln[0] < 0:
            assert bool((out == 0).all()) and bool((lse == -math.inf).all())
        else:
            assert st == 0 and bool((out == 5.0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [0, 6])
def test_attend_scales_far_apart(K, dtype):
    """Blocks whose scales lie far apart: keys large and small, values at both ends of the range
    of exponents, zero blocks."""
    for lo, hi, width in ((-64, 100, 7), (-30, 30, 7), (-64, -64, 7), (-64, 100, 3000)):
        c = Case(15, [80, 90], [2, 1], 2, 16, 128, width=width)
        used = ~torch.isnan(c.scale["v"])
        e = torch.randint(0, 2, c.scale["v"].shape, generator=c.g) * (hi - lo) + lo
        c.scale["v"] = torch.where(used, torch.exp2(e.float()), c.scale["v"])
        c.codes["v"][c.table[0][1], 0] = 0
        check_attend(c, 8, dtype, K=K)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_large_logits_and_queries(dtype):
    """Logits of hundreds, rising and falling along the keys; query rows of very different sizes."""
    c = Case(16, [200, 150], [2, 1], 2, 16, 128)
    for a in c.scale:
        c.scale[a] = torch.where(torch.isnan(c.scale[a]), c.scale[a], 2.0 ** -6)
    q = c.normal(3, 16, 128, std=20.0, dtype=dtype)
    q[0, 3] *= 2.0 ** 40
    q[0, 4] *= 2.0 ** -60
    q[1, 5, ::2] *= 2.0 ** -20
    q[2, 0] = 0
    q[2, 1, 7] = 2.0 ** 13 * q[2, 1].abs().max()
    sm = torch.full((), 1.0 / math.sqrt(128)).item()
    q[0, 3] *= 2.0 ** -38
    out, lse, st = run_attend(c, q, sm)
    assert st == 0
    for t in range(3):  # the bound on a logit's error is a row's own
        b = 0 if t < 2 else 1
        for h in range(16):
            one = Case.__new__(Case)
            one.__dict__.update(c.__dict__, T=1, cu=[0, 1], new=[1], table=[c.table[b]],
                                lens=[c.lens[b] - (1 - t if b == 0 else 0)])
            one.codes = {a: x[:, h // 8:h // 8 + 1] for a, x in c.codes.items()}
            one.scale = {a: x[:, h // 8:h // 8 + 1] for a, x in c.scale.items()}
            one.Hkv = 1
            compare(one, q[t:t + 1, h:h + 1], sm, out[t:t + 1, h:h + 1], lse[t:t + 1, h:h + 1],
                    dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [0, 4])
def test_nan_stays_with_what_sees_it(K, dtype):
    """A NaN key reaches every row that sees it and no other; a NaN value its column only."""
    c = Case(17, [50, 60], [20, 1], 2, 16, 128)
    blk, row = 35 // 16, 35 % 16
    c.codes["k"][c.table[0][blk], 0, row, 3] = NAN_CODE
    c.codes["v"][c.table[0][blk], 1, row, 9] = 0x80 | NAN_CODE
    ids = None
    if K:
        ids = torch.arange(K, dtype=torch.int32).expand(23, 2, K).contiguous()
    check_attend(c, 8, dtype, ids=ids)
    q = c.normal(21, 16, 128, dtype=dtype)
    q[3, 2, 5], q[20, 11, 0] = math.nan, math.inf
    out, lse, st = run_attend(c, q, 0.1, ids=None if ids is None else ids[:21].contiguous())
    assert bool(torch.isnan(out[3, 2]).all()) and bool(torch.isnan(out[20, 11]).all())
    assert not bool(torch.isnan(out[3, 3]).any()) and not bool(torch.isnan(out[20, 10]).any())
    assert not bool(torch.isnan(out[2]).any()) and not bool(torch.isnan(out[4, 8:, 10:]).any())


def test_attend_deterministic_and_without_lse():
    c = Case(18, [3000, 40, 700], [1, 40, 3], 2, 64, 128)
    q = c.normal(c.T, 16, 128)
    first = run_attend(c, q, 0.09)
    for _ in range(3):
        again = run_attend(c, q, 0.09)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    args = c.put()
    out = torch.empty_like(q, device=DEV)
    ws = torch.empty(max(16, ops.gqa_attend_workspace_bytes(out, args[0])), dtype=torch.uint8,
                     device=DEV)
    ops.dsa_gqa_attend(q.to(DEV), *args, 0, 0, 0.09, out, None, ws)
    assert torch.equal(out.cpu(), first[0])


def test_attend_many_sequences():
    rng = random.Random(1)
    lens = [rng.choice([0, 1, 2, 16, 17, 40]) for _ in range(8192)]
    new = [min(n, 1) for n in lens]
    c = Case(19, lens, new, 1, 16, 64, poison=False)
    check_attend(c, 4, BF)


def test_attend_cache_beyond_32_bits():
    """Pages past 2^32 bytes of codes."""
    n_pages, Hkv, ps, D = 70_000, 8, 64, 128
    gen = torch.Generator(device=DEV).manual_seed(2)
    pages = torch.randint(0, 0x77, (n_pages, Hkv, ps, D), dtype=torch.uint8, device=DEV,
                          generator=gen)
    scale = torch.full((n_pages, Hkv), 2.0 ** -7, device=DEV)
    table = [[n_pages - 1 - 3 * i for i in range(6)]]
    q = torch.randn((2, 64, D), generator=torch.Generator().manual_seed(3)).to(BF)
    c = Case.__new__(Case)
    c.__dict__.update(T=2, cu=[0, 2], new=[2], lens=[6 * ps - 9], Hkv=Hkv, ps=ps, D=D,
                      table=[list(range(6))])
    cp = pages[table[0]].cpu()
    c.codes, c.scale = dict(k=cp, v=cp), dict(k=scale[table[0]].cpu(), v=scale[table[0]].cpu())
    put = (pages, pages, scale, scale, i32(table), i32(c.lens), i32(c.cu))
    out, lse, st = run_attend(c, q, 0.05, put=put)
    assert st == 0
    compare(c, q, 0.05, out, lse, BF)
    ids = i32([[[5, 0, 3]] * 8] * 2)
    out, lse, st = run_attend(c, q, 0.05, ids=ids.cpu(), put=put)
    compare(c, q, 0.05, out, lse, BF, ids=ids.cpu())
    k_out = torch.zeros((20, Hkv, D), dtype=BF, device=DEV)
    ops.dsa_gqa_read(*put[:6], i32([0, 20]), k_out, torch.zeros_like(k_out), begin=i32([300]))
    want = ref.rows(ref.values(cp), scale[:6].cpu().double(), list(range(6)), range(300, 320))
    assert torch.equal(k_out.cpu().double(), want)
    x = torch.randn((9, Hkv, D), generator=torch.Generator().manual_seed(4)).to(BF)
    v_pages, v_scale = pages.clone(), scale.clone()
    ops.dsa_gqa_append(x.to(DEV), x.to(DEV), pages, v_pages, scale, v_scale, *put[4:6], i32([0, 9]))
    kp, ks = ref.values(cp), c.scale["k"].double()
    ref.append(x, kp, ks, c.table, c.lens, [0, 9], ps)
    assert torch.equal(ref.values(pages[table[0]].cpu()), kp)
    assert torch.equal(ref.values(v_pages[table[0]].cpu()), kp)


# ---------------------------------------------------------------- the step
def test_step_in_a_graph():
    """Plan, append, block selection and attention of two layers' forms, step after step: eager
    steps and replays of one captured step agree, and both with the plain forms."""
    B, Hkv, G, ps, D, K = 3, 2, 8, 16, 128, 4
    sm = 1.0 / math.sqrt(D)
    starts = [70, 0, 33]
    gen = torch.Generator().manual_seed(9)
    T = 8
    steps = [([1, 5, 1], 7), ([1, 1, 1], 3), ([2, 3, 0], 5), ([1, 1, 6], 8)]
    data = [[torch.randn((T, h, D), generator=gen).to(BF) for h in (Hkv, Hkv, Hkv * G)]
            for _ in range(len(steps) + 1)]
    first = [torch.randn((sum(starts), Hkv, D), generator=gen).to(BF).to(DEV) for _ in "kv"]

    def fresh():
        cache = synth.GqaCache.alloc(40, Hkv, ps, D, B, 9)
        step = pipeline.GqaStep.alloc(cache, torch.randperm(
            40, generator=torch.Generator().manual_seed(1)).to(torch.int32).to(DEV), T, Hkv * G,
            select_k=K)
        fill = pipeline.GqaStep.alloc(cache, step.free_pages, sum(starts), Hkv * G)
        pipeline.plan_step(cache, fill, i32(starts))
        pipeline.append_gqa_step(cache, fill, *first)
        step.free_begin.copy_(fill.free_begin)
        bufs = [torch.zeros((T, h, D), dtype=BF, device=DEV) for h in (Hkv, Hkv, Hkv * G)]
        return cache, step, i32([0] * B), bufs, torch.zeros_like(step.out)

    def one(cache, step, new, bufs, dense):
        pipeline.plan_step(cache, step, new)
        pipeline.append_gqa_step(cache, step, bufs[0], bufs[1])
        pipeline.attend_gqa_step(cache, step, bufs[2], sm)
        dense.copy_(step.out)
        pipeline.select_blocks_step(cache, step, bufs[2], sm, 1, 1)
        pipeline.attend_gqa_step(cache, step, bufs[2], sm, selected=True)

    eager, graphed = fresh(), fresh()
    side = torch.cuda.Stream()
    warm = fresh()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one(*warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one(*graphed)
    lens = list(starts)
    for (new, n), x in zip(steps, data):
        for cache, step, nl, bufs, dense in (eager, graphed):
            nl.copy_(i32(new))
            for buf, y in zip(bufs, x):
                buf.copy_(y.to(DEV))
        one(*eager)
        graph.replay()
        torch.cuda.synchronize()
        ctx, lens = lens, [a + b for a, b in zip(lens, new)]
        (ca, sa, _, _, da), (cb, sb, _, _, db) = eager, graphed
        assert sa.status.item() == sb.status.item() == 0
        assert torch.equal(ca.seq_lens.cpu(), torch.tensor(lens, dtype=torch.int32))
        for a, b in ((ca.k_pages.view(torch.uint8), cb.k_pages.view(torch.uint8)),
                     (ca.v_pages.view(torch.uint8), cb.v_pages.view(torch.uint8)),
                     (ca.k_scale, cb.k_scale), (ca.k_mean, cb.k_mean), (da, db),
                     (sa.out, sb.out), (sa.lse, sb.lse), (sa.block_ids[:n], sb.block_ids[:n])):
            assert torch.equal(a, b)
        c = Case.__new__(Case)
        cu = [0]
        for k in new:
            cu.append(cu[-1] + k)
        c.__dict__.update(T=n, cu=cu, new=new, lens=lens, Hkv=Hkv, ps=ps, D=D,
                          table=ca.block_table.cpu().tolist())
        c.codes = dict(k=ca.k_pages.cpu().view(torch.uint8), v=ca.v_pages.cpu().view(torch.uint8))
        c.scale = dict(k=ca.k_scale.cpu(), v=ca.v_scale.cpu())
        ids = sa.block_ids.cpu()
        compare(c, x[2], sm, sa.out.cpu(), sa.lse.cpu(), BF, ids=ids)
        kp, ks = c.plain("k")
        vp, vs = c.plain("v")
        want, _, mass, _, _ = ref.attend(x[2][:n], kp, ks, vp, vs, c.table, lens, cu, sm)
        tol = 2.0 ** -7 * (mass + want.abs()) + 2.0 ** -10
        assert bool(((da.cpu().double()[:n] - want).abs() <= tol).all())
        # the selection: the scores' own top, own and first block always in it
        got, _ = ref.scores(x[2][:n], ca.k_mean.cpu(), c.table, lens, cu, ps, 1, 1, sm, 9)
        for b in range(B):
            for i in range(new[b]):
                mine = (ctx[b] + i) // ps
                for h in range(Hkv):
                    row = [j for j in ids[cu[b] + i, h].tolist() if j >= 0]
                    assert len(row) == min(K, mine + 1) and mine in row and 0 in row
                    s = got[cu[b] + i, h]
                    rest = [j for j in range(mine) if j not in row]
                    for j in row:
                        for k in rest:
                            assert s[j] >= s[k] - 1e-5


def test_two_threads_and_streams():
    """Two threads' calls at once, each on its own stream and workspace, give what one gives."""
    cases = [Case(20 + i, [900, 50], [1, 6], 2, 16, 128) for i in range(2)]
    qs = [c.normal(c.T, 16, 128) for c in cases]
    want = [run_attend(c, q, 0.09) for c, q in zip(cases, qs)]
    got, errs = [None, None], []

    def work(i):
        try:
            s = torch.cuda.Stream()
            args, q = cases[i].put(), qs[i].to(DEV)
            out = torch.empty_like(q)
            lse = torch.empty(q.shape[:2], device=DEV)
            ws = torch.empty(max(16, ops.gqa_attend_workspace_bytes(q, args[0])),
                             dtype=torch.uint8, device=DEV)
            torch.cuda.synchronize()
            for _ in range(50):
                ops.dsa_gqa_attend(q, *args, 0, 0, 0.09, out, lse, ws, stream=s)
            s.synchronize()
            got[i] = out.cpu(), lse.cpu()
        except Exception as e:  # noqa: BLE001
            errs.append(e)
    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errs
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_refused_tensors():
    """What the binding refuses with a ValueError or TypeError, on the GPU's tensors."""
    c = Case(30, [40], [2], 2, 16, 32)
    kp, vp, ks, vs, table, lens, cu = c.put()
    q = torch.zeros((2, 4, 32), dtype=BF, device=DEV)
    out, lse = torch.zeros_like(q), torch.zeros((2, 4), device=DEV)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)
    good = dict(q=q, kp=kp, vp=vp, ks=ks, vs=vs, table=table, lens=lens, cu=cu, out=out, lse=lse,
                ids=None)

    def call(**kw):
        a = dict(good, **kw)
        ops.dsa_gqa_attend(a["q"], a["kp"], a["vp"], a["ks"], a["vs"], a["table"], a["lens"],
                           a["cu"], 0, 0, 0.1, a["out"], a["lse"], ws, block_ids=a["ids"])
    call()
    for kw in (dict(q=q.cpu()), dict(q=q[:, ::2]), dict(q=q[..., :16].contiguous()),
               dict(out=out[:1]), dict(lse=lse[:1]), dict(ks=ks[:1]), dict(vs=vs.double()),
               dict(kp=kp.float()), dict(vp=vp[:1]), dict(cu=cu[:1]), dict(cu=cu.long()),
               dict(table=table[0]), dict(lens=lens.repeat(2)), dict(kp=kp.transpose(1, 2)),
               dict(ids=table), dict(ids=torch.zeros((2, 2, 0), dtype=torch.int32, device=DEV)),
               dict(ids=torch.zeros((2, 1, 3), dtype=torch.int32, device=DEV)),
               dict(out=out.float())):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    with pytest.raises(ops.DsaError):
        ops.dsa_gqa_attend(q[:, :3].contiguous(), kp, vp, ks, vs, table, lens, cu, 0, 0, 0.1,
                           out[:, :3].contiguous(), lse[:, :3].contiguous(), ws)


@pytest.mark.parametrize("lens,new,Hkv,G,ps,D,sinks,local", [
    ([5000, 3, 0, 2300], [200, 3, 0, 60], 2, 8, 16, 128, 1, 2),
    ([4200], [460], 1, 1, 16, 128, 0, 0), ([2500, 900], [300, 160], 1, 2, 16, 64, 2, 1),
    ([700, 700], [100, 60], 3, 4, 16, 64, 0, 1),
    ([1900, 40], [230, 1], 2, 5, 16, 128, 1, 0), ([3000], [120], 4, 16, 16, 128, 1, 4),
    ([900], [900], 1, 32, 64, 128, 0, 2), ([2060], [250], 2, 20, 16, 64, 3, 200),
    ([460], [460], 1, 8, 256, 64, 1, 1)])
def test_scores_of_chunks(lens, new, Hkv, G, ps, D, sinks, local):
    check_scores(Case(ps + G, lens, new, Hkv, ps, D), G, BF, sinks, local)


def test_scores_of_chunks_narrow_and_faults():
    c = Case(9, [2300, 700], [200, 30], 2, 16, 64)
    check_scores(c, 8, BF, 1, 1, NB=133, fault=ops.DEV_POOL_RANGE)
    check_scores(c, 8, BF, 1, 1, NB=400)
    check_scores(c, 8, BF, 0, 2, std=60.0)
    c.table[0][3], c.table[0][130], c.table[1][2] = -9, 10 ** 6, c.n_pages
    check_scores(c, 8, BF, 0, 1, fault=ops.DEV_BAD_PAGE)
    c = Case(10, [2300, 700], [200, 30], 2, 16, 64, width=5)
    check_scores(c, 8, BF, 1, 1, NB=9, fault=ops.DEV_BAD_PAGE | ops.DEV_POOL_RANGE)


def test_scores_of_chunks_nan():
    """A query with a NaN reaches its token's scores of its KV head, a NaN mean the rows that have
    its block as a candidate."""
    c = Case(11, [2300, 700], [200, 30], 2, 16, 128)
    q, means = c.normal(230, 8, 128, std=2.0), c.normal(c.n_pages, 2, 128, std=0.5)

    def scores(q, means):
        out = torch.empty((230, 2, len(c.table[0])), device=DEV)
        ops.dsa_gqa_block_scores(q.to(DEV), means.to(DEV), i32(c.table), i32(c.lens), 16,
                                 i32(c.cu), 1, 1, 0.1, out)
        return out.cpu()
    plain = scores(q, means)
    q[77, 6, 100] = math.nan
    means[c.table[1][43], 0, 5] = math.nan             # complete with the last 13 tokens or so
    got = scores(q, means)
    row = torch.isnan(got)
    cand = torch.isfinite(plain)
    want = torch.zeros_like(row)
    want[77, 1] = cand[77, 1]
    for t in range(200, 230):
        if 700 - 230 + t + 1 >= 44 * 16:
            want[t, 0] = cand[t, 0]
    assert torch.equal(row, want)
    assert torch.equal(got[~row], plain[~row])


def test_chunks_with_a_negative_scale():
    """sm_scale < 0 is the negated query's, bit for bit."""
    c = Case(12, [900, 300], [200, 60], 2, 16, 128)
    q = c.normal(c.T, 16, 128)
    one, two = run_attend(c, q, -0.2), run_attend(c, -q, 0.2)
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    means = c.normal(c.n_pages, 2, 128, std=0.5).to(DEV)
    out = [torch.empty((c.T, 2, len(c.table[0])), device=DEV) for _ in range(2)]
    for x, sm, o in ((q, -0.2, out[0]), (-q, 0.2, out[1])):
        ops.dsa_gqa_block_scores(x.to(DEV), means, i32(c.table), i32(c.lens), 16, i32(c.cu), 1, 1,
                                 sm, o)
    assert torch.equal(*out)


@pytest.mark.parametrize("D", [64, 128])
def test_attend_chunks_small_and_zero_queries(D):
    c = Case(13, [700, 400], [150, 33], 2, 16, D)
    q = c.normal(c.T + 1, 10, D, std=2.0)
    q[3], q[40, 2], q[160, 9, 1:] = 0.0, q[40, 2] * 2.0 ** -90, 0.0
    q[41, 1, ::3] *= 2.0 ** -30
    check_dense(c, 5, q=q)
    check_dense(c, 5, 90, 20, q=q)


@pytest.mark.parametrize("tokens", [200, 1])
def test_kernels_give_up_and_recover(tokens):
    """A wait that runs out ends the call with a flagged status; the context stays usable, and the
    same call made afterwards gives what it gave before."""
    c = Case(14, [2300, 700], [tokens, 30], 2, 16, 128)
    q, means = c.normal(c.T, 16, 128), c.normal(c.n_pages, 2, 128, std=0.5).to(DEV)

    def both():
        st = i32([0])
        scores = torch.zeros((c.T, 2, len(c.table[0])), device=DEV)
        ops.dsa_gqa_block_scores(q.to(DEV), means, i32(c.table), i32(c.lens), 16, i32(c.cu), 1, 1,
                                 0.1, scores, status=st)
        out, lse, bits = run_attend(c, q, 0.1)
        return scores.cpu(), out, lse, bits, st.item()
    first = both()
    assert first[3:] == (0, 0)
    ops.dsa_set_failure_drill(ops.DSA_DRILL_SKIP_ARM)
    try:
        _, _, _, bits, st = both()
    finally:
        ops.dsa_set_failure_drill(0)
    if tokens > 1:  # (a decode step's kernels wait for loads alone, which no drill withholds)
        assert bits == st == ops.DEV_TIMEOUT
    again = both()
    assert again[3:] == (0, 0) and all(torch.equal(a, b) for a, b in zip(first[:3], again[:3]))


def offset(x, n):
    """A copy of x that begins n bytes behind a multiple of 256."""
    buf = torch.empty(x.numel() * x.element_size() + 256, dtype=torch.uint8, device=DEV)
    y = buf[n:n + x.numel() * x.element_size()].view(x.dtype).view(x.shape)
    y.copy_(x)
    assert y.data_ptr() % 256 == n
    return y


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,ps,new", [(128, 64, 200), (64, 16, 3), (80, 32, 70)])
def test_tensors_on_16_bytes(D, ps, new, dtype):
    """Activations that begin on an odd multiple of 16 bytes, each by itself: the same bits."""
    c = Case(15, [new + 90, new + 5], [new, new], 2, ps, D)
    k, v = (c.normal(c.T, 2, D, dtype=dtype).to(DEV) for _ in "kv")
    want = None
    for at in ((0, 0), (16, 0), (0, 16), (48, 80)):
        kp, vp, ks, vs, table, lens, cu = c.put()
        ops.dsa_gqa_append(offset(k, at[0]), offset(v, at[1]), kp, vp, ks, vs, table, lens, cu)
        out = [offset(torch.zeros((sum(c.lens), 2, D), dtype=dtype, device=DEV), n) for n in at]
        ops.dsa_gqa_read(kp, vp, ks, vs, table, lens, i32([0, c.lens[0], sum(c.lens)]), *out)
        got = [x.clone() for x in (kp.view(torch.uint8), vp.view(torch.uint8), *out)]
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("lens,new", [([700, 300], [150, 60]), ([700, 300], [1, 2])])
def test_a_scale_of_zero_weighs_all_alike(lens, new):
    c = Case(16, lens, new, 2, 16, 128)
    for window, sinks in ((0, 0), (90, 20)):
        check_dense(c, 8, window, sinks, sm=0.0)
    means = c.normal(c.n_pages, 2, 128).to(DEV)
    out = torch.empty((c.T, 2, len(c.table[0])), device=DEV)
    ops.dsa_gqa_block_scores(c.normal(c.T, 16, 128).to(DEV), means, i32(c.table), i32(c.lens), 16,
                             i32(c.cu), 0, 1, 0.0, out)
    got = out.cpu()
    for b, t in ((0, c.cu[1] - 1), (1, c.T - 1)):
        n = c.lens[b] // 16 - (c.lens[b] % 16 == 0)     # the own block is forced
        want = torch.full((2, n), 8.0 / (c.lens[b] // 16))
        assert torch.allclose(got[t, :, :n], want, rtol=2.0 ** -20, atol=0.0)


def test_chunks_in_a_graph_with_other_lengths():
    """Chunk kernels captured once: replays follow lengths and step boundaries that changed, and a
    step that shrank to decode tokens."""
    c = Case(17, [2300, 900], [200, 100], 2, 16, 128)
    kp, vp, ks, vs, table, lens, cu = c.put()
    q = c.normal(300, 16, 128).to(DEV)
    means = c.normal(c.n_pages, 2, 128).to(DEV)
    out, lse = torch.zeros((300, 16, 128), dtype=BF, device=DEV), torch.zeros((300, 16), device=DEV)
    scores = torch.zeros((300, 2, len(c.table[0])), device=DEV)
    ws = torch.empty(ops.gqa_attend_workspace_bytes(q, kp), dtype=torch.uint8, device=DEV)

    def step():
        ops.dsa_gqa_block_scores(q, means, table, lens, 16, cu, 1, 1, 0.1, scores)
        ops.dsa_gqa_attend(q, kp, vp, ks, vs, table, lens, cu, 0, 0, 0.1, out, lse, ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n, edges in (([2300, 900], [0, 200, 300]), ([2299, 33], [0, 200, 210]),
                     ([400, 900], [0, 1, 2]), ([2300, 0], [0, 300, 300]), ([17, 900], [0, 0, 300])):
        lens.copy_(i32(n))
        cu.copy_(i32(edges))
        for x in (out, lse, scores):
            x.fill_(3.0)
        graph.replay()
        got = [x.clone() for x in (out, lse, scores)]
        for x in (out, lse, scores):
            x.fill_(3.0)
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, lse, scores)))
        assert bool((out[edges[-1]:] == 3.0).all()) and bool((scores[edges[-1]:] == 3.0).all())
        d = Case.__new__(Case)
        d.__dict__.update(c.__dict__, lens=n, cu=edges, T=edges[-1],
                          new=[b - a for a, b in zip(edges, edges[1:])])
        compare(d, q.cpu(), 0.1, out.cpu(), lse.cpu(), BF, dense=True)
