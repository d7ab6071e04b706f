"""CPU checks of the caches in pages: struct layouts, workspace sizes, refusals before any launch, and the oracle itself."""

import ctypes

import numpy as np
import pytest
import torch

from long_context_decode_c4a_b200 import _lib, ops
from oracle import paged_oracle as PO
from tests.test_abi_cpu import _c_offsets

ARG, SUP, WS = _lib.CSA_ERR_INVALID_ARG, _lib.CSA_ERR_UNSUPPORTED, _lib.CSA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


@pytest.mark.parametrize("cls,cname", [(_lib.PageTableArg, "csa_page_table"), (_lib.PagedCacheArg, "csa_paged_cache"),
                                       (_lib.Attn8Args, "csa_attn8_args")])
def test_struct_layout_matches_header(cls, cname):
    fields = [f for f, _ in cls._fields_]
    size, offs = _c_offsets(cname, fields)
    assert ctypes.sizeof(cls) == size
    assert [getattr(cls, f).offset for f in fields] == offs


def test_packed_attention_arguments():
    values = [4096 + i for i in range(9)] + [1 << 33, -(1 << 40), 1, 2, 3, 4, 1e4, 0.5, 5, 6, 7, 8, 1]
    a = _lib.Attn8Args.from_buffer_copy(_lib.pack_attn8(*values))
    assert [getattr(a, f) for f, _ in _lib.Attn8Args._fields_] == values


def test_status_string(lib):
    assert lib.csa_status_string(_lib.CSA_ERR_NO_PAGES) == b"not enough free pages"


def test_workspace_size(lib):
    n = ctypes.c_size_t()
    assert lib.csa_workspace_size(_lib.CSA_WS_PAGES, 64, 128, 10000, 0, ctypes.byref(n)) == 0
    assert n.value >= 256 + 4 * 10000 * 4 + 64 * 128 * 4 and n.value % 256 == 0
    assert lib.csa_workspace_size(_lib.CSA_WS_PAGES, 1 << 20, 1 << 12, 8, 0, ctypes.byref(n)) == SUP


P = 4096   # a pointer that is never followed


def table(**kw):
    return _lib.PageTableArg(**dict(dict(slots=4, max_pages=8, num_pages=32, page_size=64, table=P, refs=P), **kw))


def cache8(**kw):
    return _lib.PagedCacheArg(**dict(dict(d=512, block=16, pages=P, scales=P), **kw))


def cache16(**kw):
    return _lib.PagedCacheArg(**dict(dict(d=128, block=0, pages=P, scales=None), **kw))


def calls(lib, pt, c8, c16, ws=P, ws_bytes=1 << 20):
    """Every call with good arguments but for what the test gives: its name and what it returns."""
    pt, c8, c16 = (ctypes.byref(x) if x is not None else None for x in (pt, c8, c16))
    yield "append8", lambda B=2, S=4, ratio=4, start=P, rows=P, stride=512 * 9, n=9: lib.csa_cache_append(
        pt, c8, B, S, ratio, start, rows, stride, n, ws, ws_bytes, None)
    yield "append16", lambda: lib.csa_cache_append(pt, c16, 2, 4, 4, P, P, 128 * 9, 9, ws, ws_bytes, None)
    yield "read", lambda B=2, n=5, idx=P, out=P: lib.csa_cache_read(pt, c8, B, n, idx, out, ws, ws_bytes, None)
    yield "reserve", lambda entries=P: lib.csa_pages_reserve(pt, entries, ws, ws_bytes, None)
    yield "fork", lambda n=1, parent=P, entries=P: lib.csa_pages_fork(pt, c8, n, parent, entries, ws, ws_bytes, None)
    yield "compact", lambda n=1, map=P, live=P: lib.csa_pages_compact(pt, c8, n, map, live, ws, ws_bytes, None)
    yield "scores", lambda B=2, S=1, H=64, ratio=4, q=P, scores=P: lib.csa_indexer_scores_paged(
        pt, c16, B, S, H, ratio, P, q, P, scores, ws, ws_bytes, None)
    yield "topk", lambda B=2, S=1, H=64, ratio=4, k=16, idx=P: lib.csa_indexer_topk_paged(
        pt, c16, B, S, H, ratio, k, P, P, P, idx, None, ws, ws_bytes, None)
    def attn(fn, B=2, S=1, H=128, rd=64, base=1e4, scale=0.1, ratio=4, q=P, ring=P, stride=512 * 128, cap=128, win=128, idx=P, k=8):
        addr = lambda x: ctypes.cast(x, ctypes.c_void_p).value if x is not None else None  # noqa: E731
        a = _lib.Attn8Args(addr(pt), addr(c8), P, q, ring, idx, P, P, ws, ws_bytes, stride, B, S, H, rd, base, scale, ratio, cap, win, k, 0)
        return fn(ctypes.addressof(a), None)
    yield "list", lambda **kw: attn(lib.csa_sparse_attn8, **kw)
    yield "range", lambda **kw: attn(lib.hca_attn8, **kw)


@pytest.mark.parametrize("bad,code", [
    (dict(slots=0), ARG), (dict(max_pages=0), ARG), (dict(num_pages=0), ARG), (dict(page_size=8), SUP), (dict(page_size=48), SUP),
    (dict(page_size=2048), SUP), (dict(table=None), ARG), (dict(refs=None), ARG), (dict(table=P + 2), ARG),
    (dict(num_pages=1 << 25), SUP), (dict(max_pages=1 << 25), SUP), (dict(slots=1 << 20, max_pages=1 << 12), SUP)])
def test_bad_tables(lib, bad, code):
    for name, call in calls(lib, table(**bad), cache8(), cache16()):
        assert call() == code, name


def test_null_structs(lib):
    for name, call in calls(lib, None, cache8(), cache16()):
        assert call() == ARG, name
    for name, call in calls(lib, table(), None, None):
        if name != "reserve":
            assert call() == ARG, name


@pytest.mark.parametrize("bad,code", [
    (dict(pages=None), ARG), (dict(pages=P + 8), ARG), (dict(d=256), SUP), (dict(block=0), SUP), (dict(block=3), SUP), (dict(block=128), SUP),
    (dict(scales=P + 4), ARG)])
def test_bad_8_bit_caches(lib, bad, code):
    for name, call in calls(lib, table(), cache8(**bad), cache16()):
        if name not in ("append16", "scores", "topk", "reserve"):
            assert call() == code, name
    small = table(page_size=16)
    for name, call in calls(lib, small, cache8(block=32), cache16()):
        if name not in ("append16", "scores", "topk", "reserve"):
            assert call() == SUP, name


@pytest.mark.parametrize("bad,code", [(dict(pages=None), ARG), (dict(d=12), SUP), (dict(d=520), SUP)])
def test_bad_bf16_caches(lib, bad, code):
    for name, call in calls(lib, table(), cache8(), cache16(**bad)):
        if name in ("append16", "scores", "topk"):
            assert call() == code, name


def test_the_wrong_kind_of_cache(lib):
    for name, call in calls(lib, table(), cache16(), cache8()):
        if name in ("scores", "topk", "list", "range"):
            assert call() == ARG, name
    for name, call in calls(lib, table(), cache8(), cache16(d=64)):
        if name in ("scores", "topk"):
            assert call() == SUP, name


def test_workspaces(lib):
    for ws, n in ((None, 1 << 20), (P + 128, 1 << 20), (P, 255)):
        for name, call in calls(lib, table(), cache8(), cache16(), ws, n):
            if name not in ("scores", "topk"):   # these look at the device first
                assert call() == WS, name
    for name, call in calls(lib, table(), cache8(), cache16(), P, 256):
        if name in ("reserve", "fork", "compact"):
            assert call() == WS, name


@pytest.mark.parametrize("name,bad,code", [
    ("append8", dict(B=0), ARG), ("append8", dict(B=5), ARG), ("append8", dict(S=0), ARG), ("append8", dict(ratio=0), ARG), ("append8", dict(start=None), ARG),
    ("append8", dict(rows=P + 8), ARG), ("append8", dict(stride=4), ARG), ("append8", dict(n=0), ARG),
    ("read", dict(n=0), ARG), ("read", dict(idx=None), ARG), ("read", dict(out=P + 2), ARG), ("read", dict(B=5), ARG),
    ("reserve", dict(entries=None), ARG), ("fork", dict(n=-1), ARG), ("fork", dict(n=1025), ARG), ("fork", dict(parent=None), ARG),
    ("fork", dict(entries=P + 1), ARG), ("compact", dict(map=None), ARG), ("compact", dict(live=None), ARG),
    ("scores", dict(H=48), SUP), ("scores", dict(B=5), ARG), ("scores", dict(S=0), ARG), ("scores", dict(scores=None), ARG), ("scores", dict(ratio=0), ARG),
    ("topk", dict(k=0), SUP), ("topk", dict(k=4096), SUP), ("topk", dict(idx=None), ARG),
    ("list", dict(B=5), ARG), ("list", dict(S=0), ARG), ("list", dict(H=0), SUP), ("list", dict(H=129), SUP), ("list", dict(rd=3), SUP),
    ("list", dict(rd=130), SUP), ("list", dict(base=0.0), ARG), ("list", dict(scale=float("nan")), ARG), ("list", dict(ratio=0), ARG),
    ("list", dict(q=P + 8), ARG), ("list", dict(ring=None), ARG), ("list", dict(stride=512 * 128 + 4), ARG), ("list", dict(stride=512), ARG),
    ("list", dict(cap=100), ARG), ("list", dict(win=0), SUP), ("list", dict(win=1025, cap=2000), SUP), ("list", dict(idx=None), ARG),
    ("list", dict(k=0), SUP), ("list", dict(k=2049), SUP), ("range", dict(B=0), ARG), ("range", dict(H=200), SUP)])
def test_bad_arguments(lib, name, bad, code):
    assert dict(calls(lib, table(), cache8(), cache16()))[name](**bad) == code


def test_attention_without_arguments(lib):
    assert lib.csa_sparse_attn8(None, None) == ARG and lib.hca_attn8(None, None) == ARG


def test_bindings_refuse_host_tensors():
    with pytest.raises(ValueError, match="CUDA"):
        ops.PageTable(torch.zeros(2, 2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), 16)


# ------------------------------------------------------------------------------------------------ the oracle


def test_oracle_codes_are_the_format():
    assert np.array_equal(PO.CODES, torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy())
    x = torch.randn(20000, generator=torch.Generator().manual_seed(0)) * torch.exp(2 * torch.randn(20000, generator=torch.Generator().manual_seed(1)))
    x = x.clamp(-448, 448)
    assert np.array_equal(PO.e4m3(x.double().numpy()), x.to(torch.float8_e4m3fn).double().numpy())
    for a, s in ((0.0, 2.0 ** -100), (448.0, 1.0), (449.0, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8)):
        assert PO.block_scale(a) == s


def test_oracle_fork_keeps_no_page_that_another_has():
    """A partly filled last page that somebody else still reads is copied: slot 2 takes 9 of slot 0's 16 entries, slot 1 keeps them all."""
    tab, refs = [[0], [0], [-1]], [2, 0, 0]
    assert PO.fork(tab, refs, 16, [-1, 1, 0], [9, 16, 0]) == [(0, 1)]
    assert tab == [[-1], [0], [1]] and refs == [1, 1, 0]
    tab, refs = [[0], [-1]], [2, 0]      # ... or a holder outside the table
    assert PO.fork(tab, refs, 16, [-1, 0], [9, 0]) == [(0, 1)]
    assert tab == [[-1], [1]] and refs == [1, 1]
    tab, refs = [[0], [0], [-1], [-1]], [2, 0, 0]   # two parents of one page that both leave: its lowest heir keeps it
    assert PO.fork(tab, refs, 16, [-1, -1, 1, 0], [9, 7, 0, 0]) == [(0, 1)]
    assert tab == [[-1], [-1], [0], [1]] and refs == [1, 1, 0]


def test_oracle_fork_and_compact_by_hand():
    """Two prompts; slot 1 becomes a sample of slot 0, slot 2 leaves, slot 3 takes slot 2's place in the middle of a page."""
    tab, refs = [[0, 1, -1], [-1, -1, -1], [5, 4, -1], [2, -1, -1]], [1, 1, 1, 0, 1, 1, 0]
    moves = PO.fork(tab, refs, 16, [0, 0, -1, 2], [20, 0, 25, 9])
    assert tab == [[0, 1, -1], [0, 2, -1], [-1, -1, -1], [5, 4, -1]]   # page 2 was freed by the same call
    assert moves == [(1, 2)] and refs == [2, 1, 1, 0, 1, 1, 0]
    moves, where, live = PO.compact(tab, refs)
    assert (moves, live) == ([(5, 3)], 5) and where == [0, 1, 2, -1, 4, 3, -1]
    assert tab[3] == [3, 4, -1] and refs == [2, 1, 1, 1, 1, 0, 0]
    with pytest.raises(PO.NoPages):
        PO.reserve(tab, refs, 16, [48, 48, 48, 0])
