"""Edges of the grouped-query calls on the GPU: boundaries, lengths, scales and logits at the ends
of their ranges, what a weight's rounding may cost, more rows than a grid has in y, and waits that
run out."""
import math

import math

import pytest
import torch

from sparse_attention_indexer_kpool_gb300 import ops, pipeline, synth
from tests import _gqa_ref as ref
from tests.test_gpu_gqa import (BF, DEV, F8, F32, Case, compare, i32, random_ids,
                                run_attend)

pytestmark = pytest.mark.gpu
LOW, HIGH = -2 ** 31, 2 ** 31 - 1
# geometries, new tokens of two sequences and activation types that take each form of the calls
FORMS = [(2, 8, 16, 128, (200, 90), BF), (8, 8, 16, 64, (3, 2), BF), (2, 8, 64, 128, (40, 90), BF),
         (1, 4, 32, 80, (30, 9), F32), (2, 8, 1024, 128, (300, 70), BF)]


@pytest.mark.parametrize("Hkv,G,ps,D,new,dtype", FORMS)
def test_boundaries_far_apart(Hkv, G, ps, D, new, dtype):
    """Boundaries of the token axis that lie 2^31 and more apart are faults like any others:
    nothing outside the step is read or written, and a sequence whose end lies before its
    beginning has no rows."""
    c = Case(60 + D, [new[0] + 50, new[1] + 20], list(new), Hkv, ps, D)
    T, edge = c.T, new[0]
    k, v, q = (c.normal(T, h, D, dtype=dtype).to(DEV) for h in (Hkv, Hkv, Hkv * G))
    means = c.normal(c.n_pages, Hkv, D).to(DEV)

    def run(cu):
        kp, vp, ks, vs, table, lens, _ = c.put()
        st = [i32([0]) for _ in range(4)]
        mean = means.clone()
        ops.dsa_gqa_append(k, v, kp, vp, ks, vs, table, lens, i32(cu), k_mean=mean, status=st[0])
        back = [torch.full((T + 4, Hkv, D), 5.0, dtype=dtype, device=DEV) for _ in "kv"]
        ops.dsa_gqa_read(kp, vp, ks, vs, table, lens, i32(cu), *(x[2:-2] for x in back),
                         status=st[1])
        scores = torch.full((T + 4, Hkv, len(c.table[0])), 5.0, device=DEV)
        ops.dsa_gqa_block_scores(q, means, table, lens, ps, i32(cu), 0, 1, 0.1, scores[2:-2],
                                 status=st[2])
        out = torch.full((T + 4, Hkv * G, D), 5.0, dtype=dtype, device=DEV)
        lse = torch.full((T + 4, Hkv * G), 5.0, device=DEV)
        ws = torch.empty(max(16, ops.gqa_attend_workspace_bytes(q, kp)), dtype=torch.uint8,
                         device=DEV)
        ops.dsa_gqa_attend(q, kp, vp, ks, vs, table, lens, i32(cu), 0, 0, 0.1, out[2:-2],
                           lse[2:-2], ws, status=st[3])
        torch.cuda.synchronize()
        for x in (*back, scores, out, lse):
            assert bool((x[:2] == 5.0).all()) and bool((x[-2:] == 5.0).all())
        return ([x.view(torch.uint8) for x in (kp, vp)] + [ks, vs, mean], back, scores, out,
                [x.item() for x in st])
    held, back, scores, out, st = run([0, edge, LOW])
    want = run([0, edge, edge])
    assert want[4] == [0] * 4 and st[1:] == [ops.DEV_BAD_LENGTH] * 3
    for x, y in zip(held, want[0]):
        assert torch.equal(x.nan_to_num(-1.0), y.nan_to_num(-1.0))
    for x, y in zip([*back, scores], [*want[1], want[2]]):
        assert torch.equal(x, y)
    assert bool((out[2 + edge:] == 5.0).all())
    for cu in ([LOW, edge, HIGH], [HIGH, edge, LOW], [HIGH, LOW, HIGH], [0, HIGH, LOW]):
        st = run(cu)[4]
        assert st[1:] == [ops.DEV_BAD_LENGTH] * 3, cu
    got = run([0, edge, edge])
    assert got[4] == [0] * 4 and torch.equal(got[3], want[3])


# forms of the append: a warp a token's block, a CTA a block (elements in registers; read twice)
@pytest.mark.parametrize("T,B,Hkv,ps,D", [
    (5, 4, 2, 16, 64), (5, 300, 2, 16, 64), (400, 4, 2, 16, 128), (900, 300, 2, 16, 128),
    (400, 4, 1, 32, 80)])
def test_append_reports_every_faulty_sequence(T, B, Hkv, ps, D):
    """Lengths below the new tokens' number, zero and negative ones, and boundaries that fall, are
    negative or past the step: reported whichever sequence has them, the last included."""
    kp, vp = (torch.zeros((3, Hkv, ps, D), dtype=torch.uint8, device=DEV).view(F8) for _ in "kv")
    ks, vs = torch.ones((3, Hkv), device=DEV), torch.ones((3, Hkv), device=DEV)
    table = torch.full((B, 1), -1, dtype=torch.int32, device=DEV)
    x = torch.ones((T, Hkv, D), dtype=BF, device=DEV)

    def status(cu, lens):
        st = i32([0])
        ops.dsa_gqa_append(x, x, kp, vp, ks, vs, table, i32(lens), i32(cu), status=st)
        return st.item()
    part = [0] + [min(T, 2 + i) for i in range(B - 1)] + [T]
    good = [T + 40] * B
    assert status(part, good) == ops.DEV_BAD_PAGE           # (no sequence has a page)
    for b in (0, 1, B - 1):
        n = part[b + 1] - part[b]
        for ln in (n - 1, 0, -1, -5, LOW):
            if n > 0:
                assert status(part, good[:b] + [ln] + good[b + 1:]) & ops.DEV_BAD_LENGTH, (b, ln)
        # without new tokens any length is right
        if b < B - 1:
            none = [T if i > b + 1 else 0 for i in range(B + 1)]
            assert status(none, good[:b] + [-3] + good[b + 1:]) == ops.DEV_BAD_PAGE, b
    for b, edge in ((0, -3), (0, LOW), (B, T + 1), (B, HIGH), (B - 1, T + 5), (2, -1), (B, 0)):
        cu = list(part)
        cu[b] = edge
        assert status(cu, good) & ops.DEV_BAD_LENGTH, (b, edge)
    # where no slot is the faulty sequence's own
    for cu in ([0, T - 1, T + 4], [-3, 0, T], [0, T, 2, T], [0, T, T - 1], [T, 0, 0]):
        cu = cu + [cu[-1]] * (B + 1 - len(cu))
        assert status(cu, good) & ops.DEV_BAD_LENGTH, cu
    assert not bool(kp.view(torch.uint8).any()) and not bool(vp.view(torch.uint8).any())


def top_by_sort(scores, K):
    """Score descending, then the smaller index; -1 for what is no candidate."""
    Q, P = scores.shape
    order = torch.sort(scores.nan_to_num(-math.inf, math.inf, -math.inf), dim=1, descending=True,
                       stable=True)
    ids = torch.where(order.values > -math.inf, order.indices, -1)[:, :K].to(torch.int32)
    return torch.nn.functional.pad(ids, (0, max(0, K - P)), value=-1)


@pytest.mark.parametrize("Q,P,K", [(65_535, 33, 7), (65_536, 33, 7), (200_001, 20, 32),
                                   (70_000, 257, 32), (3, 40_000, 100), (152, 70_000, 64)])
def test_topk_of_many_rows(Q, P, K):
    g = torch.Generator(device=DEV).manual_seed(Q + P)
    s = torch.randint(-6, 7, (Q, P), generator=g, device=DEV).float()
    s[s == -6] = -math.inf
    s[s == 6] = math.inf
    s[::5] = torch.randn(s[::5].shape, generator=g, device=DEV)
    ids = torch.full((Q + 1, K), 77, dtype=torch.int32, device=DEV)
    ops.dsa_topk_pools(s, K, ids[:Q], None)
    assert torch.equal(ids[:Q], top_by_sort(s, K))
    assert bool((ids[Q] == 77).all())


def test_blocks_of_a_long_prompt():
    """9,000 new tokens of 8 KV heads select their blocks: 72,000 rows in one step."""
    T, Hkv, G, ps, D, K = 9000, 8, 1, 64, 64, 6
    cache = synth.GqaCache.alloc(150, Hkv, ps, D, 2, 142)
    step = pipeline.GqaStep.alloc(cache, torch.arange(150, dtype=torch.int32, device=DEV), T,
                                  Hkv * G, select_k=K)
    g = torch.Generator().manual_seed(4)
    k, v, q = (torch.randn((T, Hkv, D), generator=g).to(BF).to(DEV) for _ in "kvq")
    pipeline.plan_step(cache, step, i32([T - 5, 5]))
    pipeline.append_gqa_step(cache, step, k, v)
    pipeline.select_blocks_step(cache, step, q, 0.125)
    pipeline.attend_gqa_step(cache, step, q, 0.125, selected=True)
    torch.cuda.synchronize()
    assert step.status.item() == 0
    ids = step.block_ids
    assert torch.equal(ids.view(T * Hkv, K), top_by_sort(step.scores.view(T * Hkv, -1), K))
    mine = torch.cat([torch.arange(T - 5), torch.arange(5)]).to(DEV) // ps
    assert bool((ids == mine[:, None, None]).any(2).all()) and bool((ids[..., 0] == 0).all())
    assert bool((ids <= mine[:, None, None]).all())
    # the last tokens' attention, from the cache that the step wrote
    c = Case.__new__(Case)
    t = torch.arange(T - 9, T)
    c.__dict__.update(T=4, cu=[0, 4], new=[4], lens=[T - 5], Hkv=Hkv, ps=ps, D=D,
                      table=cache.block_table[:1].cpu().tolist())
    c.codes = dict(k=cache.k_pages.cpu().view(torch.uint8),
                   v=cache.v_pages.cpu().view(torch.uint8))
    c.scale = dict(k=cache.k_scale.cpu(), v=cache.v_scale.cpu())
    compare(c, q[t[:4]].cpu(), 0.125, step.out[t[:4]].cpu(), step.lse[t[:4]].cpu(), BF,
            ids=ids[t[:4]].cpu())


@pytest.mark.parametrize("first,low", [(1.0, -math.inf), (2.0 ** 127, -2.0 ** 10)])
@pytest.mark.parametrize("lens,new,dtype", [([2300, 700], [200, 30], BF), ([2300, 700], [2, 1], BF),
                                            ([2300, 700], [2, 1], F32)])
@pytest.mark.parametrize("struck", [[5], list(range(40)), list(range(30, 140, 3)),
                                    list(range(200))])
def test_scores_with_logits_of_minus_infinity(lens, new, dtype, first, low, struck):
    """A block whose logit is minus infinity weighs nothing, in every form of the scores, wherever
    it stands; where there are only such blocks all weigh nothing."""
    c = Case(80, lens, new, 2, 16, 128)
    G, sm = 8, 0.1
    q, means = c.normal(c.T, 16, 128, dtype=dtype), c.normal(c.n_pages, 2, 128, std=0.5)
    q[..., 0], means[..., 0] = first, 0.0
    hit = [j for j in struck if j < len(c.table[0]) and c.table[0][j] >= 0]
    means[[c.table[0][j] for j in hit], :, 0] = low
    NB = len(c.table[0])
    out = torch.empty((c.T, 2, NB), device=DEV)
    st = i32([0])
    ops.dsa_gqa_block_scores(q.to(DEV), means.to(DEV), i32(c.table), i32(c.lens), 16, i32(c.cu), 0,
                             0, sm, out, status=st)
    assert st.item() == 0
    got = out.cpu().double()
    qq, mm = q[..., 1:].double().view(c.T, 2, G, 127), means[..., 1:].double()
    for b in range(2):
        page = [p for p in c.table[b] if p >= 0]
        z = torch.einsum("thgd,jhd->thgj", qq[c.cu[b]:c.cu[b + 1]], mm[page]) * sm
        # of the logits' size, as where all weigh something (the first element adds 0 to them)
        big = float(torch.einsum("thgd,jhd->thgj", qq.abs(), mm[page].abs()).max()) * sm
        dz = big * (2 * 128 + 8) * 2.0 ** -24
        for i in range(new[b]):
            n = (lens[b] - new[b] + i + 1) // 16
            x = z[i, :, :, :n].clone()
            if b == 0:
                x[..., [j for j in hit if j < n]] = -math.inf
            want = torch.softmax(x, -1).nan_to_num(0.0).sum(1)      # (all minus infinity: zeros)
            y = got[c.cu[b] + i]
            tol = want * (4 * dz + (NB + G) * 2.0 ** -24 + 2.0 ** -20) + 2.0 ** -126
            assert bool(((y[:, :n] - want).abs() <= tol).all()), (b, i)
            assert bool((y[:, n:] == -math.inf).all())


@pytest.mark.parametrize("G", [8, 16])
@pytest.mark.parametrize("lens,new,width,K", [
    ([2300, 700], [1, 2], 150, 0),              # a cluster a row tile
    ([2300, 700], [1, 2], 2500, 0),             # warps on equal shares, and a join
    ([2300, 700, 90], [60, 40, 9], 150, 20)])   # the same on lists
def test_decode_attention_gives_up_and_recovers(lens, new, width, K, G):
    """The waits of the decode attention run out under a drill: the call ends with a flagged
    status, the context stays usable, and the same call afterwards gives what it gave before."""
    c = Case(81, lens, new, 2, 16, 128, width=width)
    q = c.normal(c.T, 2 * G, 128)
    ids = random_ids(c, K) if K else None
    first = run_attend(c, q, 0.1, ids=ids)
    assert first[2] == 0
    ops.dsa_set_failure_drill(ops.DSA_DRILL_SKIP_ARM)
    try:
        for _ in range(2):
            assert run_attend(c, q, 0.1, ids=ids)[2] == ops.DEV_TIMEOUT
    finally:
        ops.dsa_set_failure_drill(0)
    again = run_attend(c, q, 0.1, ids=ids)
    assert again[2] == 0
    assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


PLACES = [  # lens, new, table width, K, type: a cluster a row tile, shares, lists, chunks, generic
    ([300, 90], [2, 1], None, 0, BF), ([300, 90], [2, 1], 2500, 0, BF),
    ([300, 90], [40, 30], None, 6, BF), ([300, 90], [40, 30], None, 0, BF),
    ([120, 40], [3, 2], None, 0, F32)]


def check_in_place(c, q, sm, K, dtype):
    ids = random_ids(c, K) if K else None
    out, lse, st = run_attend(c, q, sm, ids=ids)
    assert st == 0
    compare(c, q, sm, out, lse, dtype, ids=ids)


@pytest.mark.parametrize("lens,new,width,K,dtype", PLACES)
@pytest.mark.parametrize("e_q,lo,hi", [(-17, -64, 11), (-118, -64, 112), (-122, 100, 116),
                                       (-125, 119, 119), (58, -64, -64)])
def test_attend_queries_and_key_scales_far_apart(lens, new, width, K, dtype, e_q, lo, hi):
    """Logits of ordinary size from queries and keys' scales at opposite ends of their ranges, and
    blocks whose keys are next to nothing beside them."""
    c = Case(90 + K, lens, new, 2, 16, 128, width=width)
    e = torch.randint(0, 2, c.scale["k"].shape, generator=c.g) * (hi - lo) + lo
    c.scale["k"] = torch.where(torch.isnan(c.scale["k"]), c.scale["k"], torch.exp2(e.float()))
    q = (c.normal(c.T, 16, 128, dtype=F32) * 2.0 ** e_q).to(dtype)
    check_in_place(c, q, 1.0 / math.sqrt(128), K, dtype)


@pytest.mark.parametrize("lens,new,width,K,dtype", PLACES)
def test_attend_value_scales_at_both_ends(lens, new, width, K, dtype):
    """Values' scales of 2^-64 and 2^120 side by side (codes up to 112: their values are numbers of
    the outputs' type)."""
    c = Case(91 + K, lens, new, 2, 16, 128, width=width)
    e = torch.randint(0, 2, c.scale["v"].shape, generator=c.g) * 184 - 64
    c.scale["v"] = torch.where(torch.isnan(c.scale["v"]), c.scale["v"], torch.exp2(e.float()))
    c.codes["v"] = (ref.values(c.codes["v"]) / 4.0).float().to(F8).view(torch.uint8)
    check_in_place(c, c.normal(c.T, 16, 128, std=2.0, dtype=dtype), 1.0 / math.sqrt(128), K, dtype)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,new,width,K", [
    ([2, 3, 5, 9, 40], [1] * 5, None, 0), ([2, 3, 5, 9, 40], [1] * 5, 2500, 0),
    ([40, 30, 7], [40, 30, 7], None, 2), ([60, 50], [60, 50], None, 0)])
def test_weights_have_eleven_bits(lens, new, width, K, D):
    """Logits next to each other and values that cancel: a weight's own rounding is then most of
    what an output may be off, and eight bits of it would be too few (the bound's own test)."""
    c = Case(92 + K, lens, new, 2, 16, D, spread=1, width=width)
    G, sm = 8, 1.0 / math.sqrt(D)
    q = c.normal(c.T, 2 * G, D, std=0.02)
    ids = random_ids(c, K) if K else None
    out, lse, st = run_attend(c, q, sm, ids=ids)
    assert st == 0
    want, _, mass, top, big = ref.attend(q, *c.plain("k"), *c.plain("v"), c.table, c.lens, c.cu, sm,
                                         ids=ids)
    n = max(lens) if ids is None else K * 16
    tol = ref.bound_of_bf16(want, mass, top, big, n, D)
    assert bool(((out.double() - want).abs() <= tol).all())
    compare(c, q, sm, out, lse, BF, ids=ids)


@pytest.mark.parametrize("lens,new,width,K,dtype", PLACES)
@pytest.mark.parametrize("e_q,e_k,sm", [(62, 50, 2.0 ** -125), (-64, -50, 2.0 ** 107)])
def test_attend_softmax_scales_near_the_ends(lens, new, width, K, dtype, e_q, e_k, sm):
    """Logits of ordinary size by a softmax scale next to fp32's least normal number, or a huge
    one."""
    c = Case(93 + K, lens, new, 2, 16, 128, width=width)
    c.scale["k"] = torch.where(torch.isnan(c.scale["k"]), c.scale["k"], 2.0 ** e_k)
    q = (c.normal(c.T, 16, 128, dtype=F32) * 2.0 ** e_q).to(dtype)
    check_in_place(c, q, sm, K, dtype)
