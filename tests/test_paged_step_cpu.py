"""The paged step's entry points refuse what they cannot do, on the host, before
any CUDA call; and the tests' plain plan on hand-worked steps."""
import ctypes

import pytest
import torch

from sparse_attention_indexer_kpool_gb300 import _lib, build, ops
from tests import _paged_ref as ref
from tests.test_abi_cpu import A, ERR, header_define


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_status_bits():
    for name in ("BAD_LENGTH", "NO_PAGE", "TOKEN_CAP", "BAD_PAGE"):
        assert header_define(f"DSA_DEV_{name}") == getattr(ops, f"DEV_{name}") \
            == getattr(ref, f"DEV_{name}")


def plan(lib, **kw):
    a = dict(ctx=A, new=A, free=A, begin=A, base=None, B=4, T=16, n_free=8, n_pages=100, ps=16,
             width=8, table=A, lens=A, cu=A, qs=A, qp=A, rows=A, keys=None, end=A, st=None)
    a.update(kw)
    return lib.dsa_paged_plan(a["ctx"], a["new"], a["free"], a["begin"], a["base"], a["B"], a["T"],
                              a["n_free"], a["n_pages"], a["ps"], a["width"], a["table"],
                              a["lens"], a["cu"], a["qs"], a["qp"], a["rows"], a["keys"],
                              a["end"], a["st"], None)


def test_plan_validation(lib):
    n = lib.dsa_kernel_launches()
    for kw in (dict(B=-1), dict(T=-1), dict(n_free=-1), dict(n_pages=0), dict(ps=0),
               dict(width=0), dict(ctx=None), dict(new=None), dict(free=None), dict(begin=None),
               dict(table=None), dict(lens=None), dict(cu=None), dict(qs=None), dict(qp=None),
               dict(rows=None), dict(end=None), dict(base=A), dict(keys=A)):
        assert plan(lib, **kw) == ERR["DSA_ERR_INVALID_ARG"], kw
    assert plan(lib, n_pages=1 << 20, ps=1 << 12) == ERR["DSA_ERR_UNSUPPORTED"]
    assert plan(lib, B=header_define("DSA_PLAN_MAX_B") + 1) == ERR["DSA_ERR_UNSUPPORTED"]
    assert plan(lib, T=header_define("DSA_PLAN_MAX_T") + 1) == ERR["DSA_ERR_UNSUPPORTED"]
    assert plan(lib, B=1 << 10, width=1 << 20) == ERR["DSA_ERR_UNSUPPORTED"]
    for name in ("ctx", "new", "free", "begin", "table", "lens", "cu", "qs", "qp", "rows", "end",
                 "st"):
        assert plan(lib, **{name: A + 2}) == ERR["DSA_ERR_MISALIGNED"], name
    assert plan(lib, B=0) == ERR["DSA_OK"]
    assert lib.dsa_kernel_launches() == n


def append(lib, **kw):
    a = dict(x=A, rows=A, T=4, L=512, dt=0, pages=A, scale=None, n_pages=10, ps=16, kd=0, st=None)
    a.update(kw)
    return lib.dsa_paged_append(a["x"], a["rows"], a["T"], a["L"], a["dt"], a["pages"], a["scale"],
                                a["n_pages"], a["ps"], a["kd"], a["st"], None)


def test_append_validation(lib):
    n = lib.dsa_kernel_launches()
    for kw in (dict(T=-1), dict(L=0), dict(n_pages=0), dict(ps=0), dict(dt=2), dict(kd=7),
               dict(kd=2), dict(scale=A), dict(x=None), dict(rows=None), dict(pages=None)):
        assert append(lib, **kw) == ERR["DSA_ERR_INVALID_ARG"], kw
    for kw in (dict(L=500), dict(L=1032), dict(n_pages=1 << 20, ps=1 << 12)):
        assert append(lib, **kw) == ERR["DSA_ERR_UNSUPPORTED"], kw
    for kw in (dict(x=A + 8), dict(pages=A + 8), dict(rows=A + 2), dict(st=A + 2),
               dict(kd=2, scale=A + 2)):
        assert append(lib, **kw) == ERR["DSA_ERR_MISALIGNED"], kw
    assert append(lib, T=0) == ERR["DSA_OK"]
    assert lib.dsa_kernel_launches() == n


def chunk(lib, **kw):
    a = dict(q=A, pages=A, scale=None, table=A, lens=A, n_pages=100, ps=64, width=8, kd=0, cu=A,
             T=4, B=2, Hm=64, L=512, window=0, sinks=0, sm=0.04, dt=0, out=A, lse=A, ws=A,
             nbytes=1 << 30, st=None, kv=True)
    a.update(kw)
    kv = _lib.PagedKv(a["pages"], a["scale"], a["table"], a["lens"], a["n_pages"], a["ps"],
                      a["width"], a["kd"])
    return lib.dsa_mla_paged_chunk(a["q"], ctypes.byref(kv) if a["kv"] else None, a["cu"], a["T"],
                                   a["B"], a["Hm"], a["L"], a["window"], a["sinks"], a["sm"],
                                   a["dt"], a["out"], a["lse"], a["ws"], a["nbytes"], a["st"],
                                   None)


def test_chunk_validation(lib):
    n = lib.dsa_kernel_launches()
    for kw in (dict(T=-1), dict(B=-1), dict(Hm=0), dict(L=0), dict(window=-1), dict(sinks=-1),
               dict(sm=float("inf")), dict(sm=float("nan")), dict(dt=2), dict(kd=7), dict(kd=2),
               dict(scale=A), dict(n_pages=0), dict(ps=0), dict(width=0), dict(q=None),
               dict(pages=None), dict(table=None), dict(lens=None), dict(cu=None),
               dict(out=None), dict(kv=False)):
        assert chunk(lib, **kw) == ERR["DSA_ERR_INVALID_ARG"], kw
    for kw in (dict(L=500), dict(L=1032), dict(Hm=129), dict(n_pages=1 << 20, ps=1 << 12),
               dict(T=1 << 26), dict(B=header_define("DSA_PLAN_MAX_B") + 1)):
        assert chunk(lib, **kw) == ERR["DSA_ERR_UNSUPPORTED"], kw
    for kw in (dict(q=A + 8), dict(pages=A + 8), dict(out=A + 8), dict(table=A + 2),
               dict(lens=A + 2), dict(cu=A + 2), dict(lse=A + 2), dict(st=A + 2),
               dict(kd=2, scale=A + 2), dict(ws=A + 8)):
        assert chunk(lib, **kw) == ERR["DSA_ERR_MISALIGNED"], kw
    assert chunk(lib, T=0) == ERR["DSA_OK"]
    assert chunk(lib, B=0) == ERR["DSA_OK"]
    need = lib.dsa_mla_paged_chunk_workspace_size(4, 64, 512, 0, 0)
    if need:
        assert chunk(lib, nbytes=need - 1) == ERR["DSA_ERR_WORKSPACE"]
        assert chunk(lib, ws=None) == ERR["DSA_ERR_WORKSPACE"]
    assert lib.dsa_mla_paged_chunk_workspace_size(4, 64, 512, 1, 1) == 0      # fp32: generic
    assert lib.dsa_mla_paged_chunk_workspace_size(0, 64, 512, 0, 0) == 0
    assert lib.dsa_kernel_launches() == n


def test_binding_refuses_buffers_of_other_sizes(lib):
    """The library cannot see how long a buffer is; the binding can."""
    i = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    good = dict(ctx_lens=i(3), new_lens=i(3), free_pages=i(4), free_begin=i(1), n_pages=9,
                page_size=16, block_table=torch.zeros((3, 5), dtype=torch.int32), seq_lens=i(3),
                cu_new=i(4), q_seq=i(7), q_pos=i(7), kv_rows=i(7), free_end=i(1))
    for name, bad in (("new_lens", i(2)), ("free_begin", i(2)), ("seq_lens", i(4)),
                      ("cu_new", i(3)), ("q_pos", i(6)), ("kv_rows", i(8)), ("free_end", i(0)),
                      ("block_table", torch.zeros((2, 5), dtype=torch.int32)), ("row_base", i(2)),
                      ("key_rows", i(6))):
        with pytest.raises(ValueError, match=name):
            ops.dsa_paged_plan(**{**good, name: bad})
    with pytest.raises(ValueError, match="CUDA tensor"):     # no CPU path
        ops.dsa_paged_plan(**good)
    x, pages = torch.zeros((4, 64)), torch.zeros((32, 64))
    with pytest.raises(ValueError, match="kv_rows"):
        ops.dsa_paged_append(x, i(3), pages)
    with pytest.raises(ValueError, match="L"):
        ops.dsa_paged_append(x, i(4), torch.zeros((32, 32)))
    with pytest.raises(ValueError, match="row_scale"):
        ops.dsa_paged_append(x, i(4), pages.to(torch.float8_e4m3fn), torch.zeros(31))
    q = torch.zeros((4, 2, 64))
    good = dict(q_lat=q, pages=pages, row_scale=None, block_table=torch.zeros((1, 2),
                dtype=torch.int32), seq_lens=i(1), page_size=16, cu_new=i(2), window=0, sinks=0,
                sm_scale=1.0, out=torch.zeros_like(q), lse=torch.zeros((4, 2)))
    for name, bad in (("cu_new", i(3)), ("out", torch.zeros(3)), ("lse", torch.zeros((4, 3))),
                      ("seq_lens", i(2)), ("page_size", 15), ("pages", torch.zeros((32, 32)))):
        with pytest.raises(ValueError):
            ops.dsa_mla_paged_chunk(**{**good, name: bad})


def test_plain_plan_by_hand():
    # two requests, pages of 4: 5 cached + 4 new (blocks 0, 1 held, block 2 new), 0 + 1
    table = [[7, 3, -1, -1], [-1, -1, -1, -1]]
    got, st = ref.plan([5, 0], [4, 1], [9, 2, 5, 6], 1, 10, 4, table, 6, base=[100, 200])
    assert st == 0
    assert got["cu_new"] == [0, 4, 5] and got["seq_lens"] == [9, 1]
    assert got["table"] == [[7, 3, 2, -1], [5, -1, -1, -1]] and got["free_end"] == 3
    assert got["q_seq"] == [0, 0, 0, 0, 1, 0] and got["q_pos"] == [5, 6, 7, 8, 0, -1]
    assert got["kv_rows"] == [13, 14, 15, 8, 20, -1]
    assert got["key_rows"] == [105, 106, 107, 108, 200, -1]
    # cut at T, and no page left for the second block
    got, st = ref.plan([0, 3], [6, 9], [4], 0, 10, 4, [[-1, -1], [1, -1]], 7)
    assert st == ref.DEV_TOKEN_CAP | ref.DEV_NO_PAGE
    assert got["cu_new"] == [0, 6, 7] and got["seq_lens"] == [6, 4]
    assert got["kv_rows"] == [16, 17, 18, 19, -1, -1, 7] and got["free_end"] == 1
