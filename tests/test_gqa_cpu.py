"""The grouped-query entry points refuse what they cannot do, on the host, before any CUDA call;
and the tests' plain forms on hand-worked values."""
import ctypes
import dataclasses
import math
import os
import re
import subprocess

import pytest
import torch

from sparse_attention_indexer_kpool_gb300 import _lib, build, pipeline
from tests import _gqa_ref as ref
from tests.test_abi_cpu import A, ERR, header_define


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


KV = dict(kp=A, vp=A, ks=A, vs=A, table=A, lens=A, n_pages=100, ps=64, width=8, Hkv=8, D=128)
BAD = [dict(n_pages=0), dict(ps=0), dict(width=0), dict(Hkv=0), dict(D=0), dict(kp=None),
       dict(vp=None), dict(ks=None), dict(vs=None), dict(table=None), dict(lens=None)]
ODD = [dict(ps=8), dict(ps=24), dict(ps=1040), dict(D=8), dict(D=100), dict(D=272),
       dict(n_pages=1 << 20, ps=1024), dict(B=header_define("DSA_PLAN_MAX_B") + 1)]
SLANT = [dict(kp=A + 8), dict(vp=A + 8), dict(ks=A + 2), dict(vs=A + 2), dict(table=A + 2),
         dict(lens=A + 2), dict(st=A + 2), dict(cu=A + 2)]


def kv_of(a):
    return ctypes.byref(_lib.GqaKv(a["kp"], a["vp"], a["ks"], a["vs"], a["table"], a["lens"],
                                   a["n_pages"], a["ps"], a["width"], a["Hkv"], a["D"]))


def check(lib, call, bad, odd, slant):
    n = lib.dsa_kernel_launches()
    for kw in bad:
        assert call(lib, **kw) == ERR["DSA_ERR_INVALID_ARG"], kw
    for kw in odd:
        assert call(lib, **kw) == ERR["DSA_ERR_UNSUPPORTED"], kw
    for kw in slant:
        assert call(lib, **kw) == ERR["DSA_ERR_MISALIGNED"], kw
    assert call(lib, T=0) == ERR["DSA_OK"]
    assert call(lib, B=0) == ERR["DSA_OK"]
    assert lib.dsa_kernel_launches() == n


def append(lib, **kw):
    a = dict(KV, x=A, y=A, cu=A, T=4, B=2, dt=0, mean=None, st=None, kv=True)
    a.update(kw)
    return lib.dsa_gqa_append(a["x"], a["y"], a["cu"], a["T"], a["B"], a["dt"],
                              kv_of(a) if a["kv"] else None, a["mean"], a["st"], None)


def test_append_validation(lib):
    check(lib, append, BAD + [dict(T=-1), dict(B=-1), dict(dt=2), dict(x=None), dict(y=None),
                              dict(cu=None), dict(kv=False)],
          ODD + [dict(Hkv=129)], SLANT + [dict(x=A + 8), dict(y=A + 4), dict(mean=A + 8)])


def read(lib, **kw):
    a = dict(KV, x=A, y=A, cu=A, begin=None, T=4, B=2, dt=0, st=None, kv=True)
    a.update(kw)
    return lib.dsa_gqa_read(kv_of(a) if a["kv"] else None, a["cu"], a["begin"], a["T"], a["B"],
                            a["dt"], a["x"], a["y"], a["st"], None)


def test_read_validation(lib):
    check(lib, read, BAD + [dict(T=-1), dict(B=-1), dict(dt=7), dict(x=None), dict(y=None),
                            dict(cu=None), dict(kv=False)],
          ODD, SLANT + [dict(x=A + 8), dict(y=A + 8), dict(begin=A + 2)])


def scores(lib, **kw):
    a = dict(q=A, mean=A, table=A, lens=A, cu=A, T=4, B=2, Hq=64, Hkv=8, D=128, n_pages=100,
             ps=64, width=8, sink=1, local=1, sm=0.1, NB=8, dt=0, out=A, st=None)
    a.update(kw)
    return lib.dsa_gqa_block_scores(
        a["q"], a["mean"], a["table"], a["lens"], a["cu"], a["T"], a["B"], a["Hq"], a["Hkv"],
        a["D"], a["n_pages"], a["ps"], a["width"], a["sink"], a["local"], a["sm"], a["NB"],
        a["dt"], a["out"], a["st"], None)


def test_scores_validation(lib):
    check(lib, scores, [dict(T=-1), dict(B=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=63), dict(D=0),
                        dict(n_pages=0), dict(ps=0), dict(width=0), dict(sink=-1), dict(local=-1),
                        dict(NB=0), dict(dt=3), dict(sm=math.nan), dict(sm=math.inf),
                        dict(q=None), dict(mean=None), dict(table=None), dict(lens=None),
                        dict(cu=None), dict(out=None)],
          ODD + [dict(Hq=136), dict(T=1 << 26)],
          [dict(q=A + 8), dict(mean=A + 8), dict(table=A + 2), dict(lens=A + 2), dict(cu=A + 2),
           dict(out=A + 2), dict(st=A + 2)])


def attend(lib, **kw):
    a = dict(KV, q=A, cu=A, ids=None, K=0, T=4, B=2, Hq=64, window=0, sinks=0, sm=0.1, dt=0,
             out=A, lse=A, ws=A, nbytes=1 << 30, st=None, kv=True)
    a.update(kw)
    return lib.dsa_gqa_attend(a["q"], kv_of(a) if a["kv"] else None, a["cu"], a["ids"], a["K"],
                              a["T"], a["B"], a["Hq"], a["window"], a["sinks"], a["sm"], a["dt"],
                              a["out"], a["lse"], a["ws"], a["nbytes"], a["st"], None)


def test_attend_validation(lib):
    check(lib, attend, BAD + [
        dict(T=-1), dict(B=-1), dict(Hq=0), dict(Hq=60), dict(window=-1), dict(sinks=-1),
        dict(sm=math.nan), dict(dt=2), dict(K=-1), dict(K=3), dict(ids=A), dict(kv=False),
        dict(ids=A, K=3, window=5), dict(ids=A, K=3, sinks=5), dict(q=None), dict(out=None),
        dict(cu=None)],
        ODD + [dict(Hq=136), dict(T=1 << 26), dict(ids=A, K=1 << 26)],
        SLANT + [dict(q=A + 8), dict(out=A + 8), dict(lse=A + 2), dict(ids=A + 2, K=1),
                 dict(ws=A + 8)])
    need = lib.dsa_gqa_attend_workspace_size(4, 64, 8, 128, 0)
    if need:
        assert attend(lib, nbytes=need - 1) == ERR["DSA_ERR_WORKSPACE"]
        assert attend(lib, ws=None) == ERR["DSA_ERR_WORKSPACE"]
    for bad in ((0, 64, 8, 128, 0), (4, 60, 8, 128, 0), (4, 64, 0, 128, 0), (4, 64, 8, 0, 0),
                (4, 64, 8, 128, 2)):
        assert lib.dsa_gqa_attend_workspace_size(*bad) == 0


# ---------------------------------------------------------------- the plain forms
def test_grid_is_the_e4m3_type():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().double()
    codes = codes[torch.isfinite(codes)]
    assert torch.equal(ref.grid(codes), codes)
    x = torch.cat([codes, (codes[1:] + codes[:-1]) / 2, torch.randn(5000).double() * 100,
                   torch.randn(5000).double() * 0.01]).clamp(-448, 448)
    assert torch.equal(ref.grid(x), x.float().to(torch.float8_e4m3fn).float().double())


@pytest.mark.parametrize("a,e", [(0.0, -64), (448.0, 0), (448.5, 1), (224.0, -1), (1.0, -8),
                                 (1.75, -8), (1.76, -7), (2.0 ** -56, -64), (3.3e38, 120)])
def test_exponent(a, e):
    assert ref.exponent(a) == e
    assert a <= 448.0 * 2.0 ** e and (e == -64 or a > 448.0 * 2.0 ** (e - 1))


def test_append_by_hand():
    # pages of two rows; one row before (values 448 and 2^-9 at scale 1), one new row up to 896
    pages = torch.tensor([[[[448.0, 2.0 ** -9], [5.0, 5.0]]]], dtype=torch.float64)
    scale = torch.ones((1, 1), dtype=torch.float64)
    means = torch.zeros((1, 1, 2), dtype=torch.float64)
    ref.append(torch.tensor([[[896.0, -100.0]]]), pages, scale, [[0]], [2], [0, 1], 2, means)
    assert scale.item() == 2.0
    # 448 becomes 224 of twice the scale; 2^-10 is a tie of 0 and 2^-9: to even, 0; -50 is -48 or
    # -52: the middle, to even (-48 = 1.5 * 32, -52 = 1.625 * 32)
    assert pages[0, 0].tolist() == [[224.0, 0.0], [448.0, -48.0]]
    assert means[0, 0].tolist() == [672.0, -48.0]


def test_scores_and_attention_by_hand():
    means = torch.tensor([[[1.0, 0.0]], [[0.0, 1.0]], [[9.0, 9.0]]])
    q = torch.tensor([[[0.0, math.log(3.0)], [0.0, 0.0]]])
    s, _ = ref.scores(q, means, [[0, 1, 2]], [5], [0, 1], 2, 0, 0, 1.0, 4)
    assert torch.allclose(s[0, 0, :2], torch.tensor([0.25 + 0.5, 0.75 + 0.5]).double(), atol=1e-7)
    assert s[0, 0, 2:].tolist() == [-math.inf, -math.inf]
    s, _ = ref.scores(q, means, [[0, 1, 2]], [5], [0, 1], 2, 1, 1, 1.0, 4)
    assert s[0, 0, 0] == math.inf and s[0, 0, 2] == math.inf and s[0, 0, 3] == -math.inf
    kp = torch.tensor([[[[0.0, 0.0], [0.0, 1.0]]], [[[8.0, 8.0], [1.0, 1.0]]]]).double()
    one = torch.ones((2, 1), dtype=torch.float64)
    out, lse, *_ = ref.attend(q, kp, one, kp, one, [[0, 1]], [2], [0, 1], 1.0)
    assert torch.allclose(out[0, 0], torch.tensor([0.0, 0.75]).double(), atol=1e-7)
    assert torch.allclose(lse[0], torch.tensor([4.0, 2.0]).log().double(), atol=1e-7)
    out, lse, *_ = ref.attend(q, kp, one, kp, one, [[0, 1]], [2], [0, 1], 1.0,
                                ids=torch.tensor([[[0, 0, -1]]]))
    assert torch.allclose(lse[0], torch.tensor([8.0, 4.0]).log().double(), atol=1e-7)
    out, lse, *_ = ref.attend(q, kp, one, kp, one, [[0, 1]], [2], [0, 1], 1.0,
                                ids=torch.tensor([[[-1, 1, -1]]]))
    assert out.abs().max() == 0 and bool((lse == -math.inf).all())


def test_scores_of_more_blocks_than_positions_have(lib):
    assert scores(lib, NB=(1 << 27) + 1) == ERR["DSA_ERR_UNSUPPORTED"]
    assert scores(lib, NB=1 << 27, T=0) == 0


def test_attend_lists_of_more_rows_than_counted(lib):
    assert attend(lib, ids=A, K=(1 << 24) + 1) == ERR["DSA_ERR_UNSUPPORTED"]
    assert attend(lib, ids=A, K=1 << 24, T=0) == 0


CSRC = os.path.join(os.path.dirname(build.__file__), "csrc")


def gqa_kernels():
    """(file, source from a kernel's __global__ to the next one or the file's end)"""
    for name in sorted(os.listdir(CSRC)):
        if name.startswith("gqa"):
            text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
            for body in text.split("__global__")[1:]:
                yield name, body


def test_dependents_start_behind_the_tensor_memory():
    """A kernel lets its dependents start behind a barrier that follows its allocation of tensor
    memory: a dependent's CTA beside one that still waits for its columns could take them, and
    itself wait for that grid."""
    found = 0
    for name, body in gqa_kernels():
        if "tmem_alloc<" not in body:
            continue
        found += 1
        alloc = body.index("tmem_alloc<")
        # (find_share ends with a barrier)
        barrier = re.compile(r"__syncthreads\w*\(|find_share\(p, c\);").search(body, alloc)
        triggers = [m.start() for m in re.finditer(r"pdl_launch_dependents\(\)", body)]
        assert triggers and all(t > barrier.start() for t in triggers), name
    assert found == 2


def test_barriers_are_fenced_where_they_are_made():
    """A thread that makes a barrier fences it itself: another thread's fence, or a block-wide
    barrier, does not show it to the copies that complete on it."""
    found = 0
    for name, body in gqa_kernels():
        opened, inside = [], []          # blocks that are open; (place, condition's block) of each
        for m in re.finditer(r"[{}]|mbar_init\(&|fence_mbar_init\(\)", body):
            if m.group() == "{":
                opened.append(m.start())
            elif m.group() == "}":
                opened = opened[:-1]
            else:
                under = [at for at in opened if re.search(r"\bif \([^{};]*\) $", body[:at])]
                inside.append((m.group(), under[-1] if under else None))
        fenced = {block for what, block in inside if what.startswith("fence")}
        for what, block in inside:
            if what.startswith("mbar"):
                found += 1
                assert block is not None and block in fenced, name
    assert found


def test_topk_takes_the_rows_of_a_long_prompt(lib):
    """T * Hkv rows of block scores: more than a grid has in y.  (Refused for its pointer, which is
    looked at behind the sizes: nothing is launched.)"""
    n = lib.dsa_kernel_launches()
    bad = ERR["DSA_ERR_INVALID_ARG"]
    for rows in (65_536, 8 * 65_536, 2 ** 31 - 1):
        assert lib.dsa_topk_pools(None, rows, 64, 32, A, None, 0, None) == bad
        assert lib.dsa_topk_pools_workspace_size(rows, 64, 32) == 0
    assert lib.dsa_kernel_launches() == n


def test_every_cluster_kernel_asks_for_itself(lib):
    """How many clusters fit at once is kept for each of the decode kernel's eight cluster forms:
    they differ in shared memory and registers."""
    names = subprocess.run(["nm", "-C", os.path.join(build.BUILD, "gqa_split.o")], text=True,
                           capture_output=True, check=True).stdout
    kept = re.findall(r"clusters_of<&\(void dsa::\(anonymous namespace\)::gqa_split_kernel"
                      r"<(\d+, \d+, \d+), true>[^\n]*\)::held$", names, re.M)
    assert len(set(kept)) == 8


def test_the_bound_of_the_bf16_path_is_that_of_fp16_weights():
    """The bound that the GPU's attention is held to passes weights rounded to fp16 and none rounded
    to bf16 (planted here, in the plain form)."""
    g = torch.Generator().manual_seed(6)
    for n in (2, 3, 5, 9, 40):
        z = torch.randn((16, n), generator=g).double() * 0.05
        s = torch.exp2(torch.randint(-3, 4, (n,), generator=g).double())
        v = torch.randn((n, 128), generator=g).double() * 100.0 * s[:, None]
        w = torch.softmax(z, -1)
        want, mass, top = w @ v, w @ v.abs(), (w * s).amax(-1) * n
        tol = ref.bound_of_bf16(want, mass, top, 0.2, n, 128)
        fails = {}
        for dtype in (torch.float16, torch.bfloat16):
            out = ref.weights_rounded_to(dtype, z, v, s).to(torch.bfloat16).double()
            fails[dtype] = int(((out - want).abs() > tol).sum())
        assert fails[torch.float16] == 0 and fails[torch.bfloat16] > 0, (n, fails)


def test_a_step_without_a_selection_is_not_attended_to_densely():
    """Selected blocks asked of a step that was allocated without a selection: refused, not
    answered with attention over everything."""
    kw = {f.name: None for f in dataclasses.fields(pipeline.GqaStep)}
    step = pipeline.GqaStep(**kw)
    with pytest.raises(ValueError, match="select_k"):
        pipeline.attend_gqa_step(None, step, None, 0.1, selected=True)
    with pytest.raises(ValueError, match="select_k"):
        pipeline.select_blocks_step(None, step, None, 0.1)
