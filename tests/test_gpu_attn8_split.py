"""Attention over an 8-bit cache in pages where a query's candidates are really split over several CTA pairs and merged."""

import math

import numpy as np
import pytest
import torch

from oracle import csa_oracle as O
from tests.parity import np64
from tests.test_gpu_attn8 import D, Plain, check_close, i32, make_q, run_case

pytestmark = pytest.mark.gpu

FORMS = ("list", "range")
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def ops():
    from long_context_decode_c4a_b200 import ops
    return ops


class Split(Plain):
    """Plain of at least five tiles, the least that one request is split at; whether it was shows in the workspace."""

    def run(self, split=True, form="list", scale=None):
        partials = self.ws[256:]
        partials.fill_(0x5A)
        out = super().run(split, form, scale)
        assert bool((partials != 0x5A).any()) == split
        return out


# ------------------------------------------------------------------------------------------------ sinks


def test_sinks(ops):
    """A sink of any size; +inf takes the whole weight, NaN makes its head NaN: however the candidates are split."""
    p = Split(ops, E=640)
    p.sink[:4] = torch.tensor([-INF, 1e4, -1e4, 60.0])
    p.check()
    want, tol, _ = p.want()
    p.sink[5], p.sink[6] = INF, NAN
    rest = [h for h in range(128) if h not in (5, 6)]
    for form in FORMS:
        for split in (True, False):
            out = p.run(split, form)
            assert (out[5] == 0).all() and out[6].isnan().all()
            check_close(out[rest], want[rest], tol[rest], f"{form} split={split}")


@pytest.mark.parametrize("sink", [INF, NAN, 3e38, -INF])
def test_padding_query_with_any_sink(ops, sink):
    """No candidate: zero, whatever the sink."""
    p = Split(ops, E=640)
    p.sink.fill_(sink)
    p.t = -1
    for form in FORMS:
        for split in (True, False):
            assert (p.run(split, form) == 0).all()


@pytest.mark.parametrize("split", [True, False])
def test_infinite_sink_in_the_contiguous_form(ops, split):
    """sparse_attn's partials go through the same merge."""
    g = torch.Generator().manual_seed(3)
    E, W, H, t = 640, 16, 32, 4 * 640 + 3
    q, ring = make_q(g, 1, 1, H, D).cuda(), torch.randn(1, W, D, generator=g).to(torch.bfloat16).cuda()
    cache, sink = torch.randn(1, E, D, generator=g).to(torch.bfloat16).cuda(), torch.randn(H, generator=g).cuda()
    idx = torch.arange(E, dtype=torch.int32, device="cuda").view(1, 1, E)
    ws = ops.workspace(ops._lib.CSA_WS_SPARSE_ATTN, 1, 1, 1, 1)
    outs = []
    for s5 in (1.0, INF):
        sink[5] = s5
        ws[256:].fill_(0x5A)
        out = torch.empty(1, 1, H, D, dtype=torch.float32, device="cuda")
        ops.sparse_attn(i32([[t]]), q, ring, cache, idx, sink, W, out=out, ws=ws if split else ws[:256])
        assert bool((ws[256:] != 0x5A).any()) == split
        outs.append(out[0, 0])
    assert (outs[1][5] == 0).all()
    rest = [h for h in range(H) if h != 5]
    assert torch.equal(outs[0][rest], outs[1][rest])


# ------------------------------------------------------------------------------------------------ hard rows


@pytest.mark.parametrize("scale", [-0.5, 0.0, 1e-6, 3.0])
def test_other_scales(ops, scale):
    p = Split(ops, E=640)
    want, tol, _ = p.want(scale=scale)
    for form in FORMS:
        for split in (True, False):
            check_close(p.run(split, form, scale), want, tol, f"{form} split={split} scale={scale}")


def test_lists_that_leave_little(ops):
    """A list of 640 places, few of them taken: whole splits are left without a candidate."""
    p = Split(ops, E=640)
    p.idx.fill_(-1)
    p.check(forms=("list",))                     # the window alone
    p.idx[0, 0, 633] = 639
    p.check(forms=("list",))
    p.idx[0, 0, 3:9] = 42                        # the same entry six times counts six times
    p.check(forms=("list",))
    p.idx[0, 0, 200:] = -1                       # ends long before the list does
    p.check(forms=("list",))
    p.sink.fill_(-INF)
    p.check(forms=("list",))


@pytest.mark.parametrize("pages", [[0], [9], [2, 3, 4, 5], list(range(10))])
def test_zero_scales_do_not_count(ops, pages):
    """Some splits' rows, or every entry's, left out by a scale of zero."""
    p = Split(ops, E=640)
    t = p.cache.book.table[0].long()
    for i in pages:
        p.cache.scales[t[i]] = 0.0
    p.check([e for e in range(640) if e // 64 not in pages])
    p.sink.fill_(-INF)
    p.check([e for e in range(640) if e // 64 not in pages])


def test_extreme_magnitudes(ops):
    """q and rows near the ends of their ranges; a page of tiny scales, a split of them, beside ordinary ones."""
    p = Split(ops, E=640)
    t = p.cache.book.table[0].long()
    p.cache.scales[t[1]] = 2.0 ** -100
    p.check()
    for i in range(6):
        p.cache.scales[t[i]] = 2.0 ** -100
    p.check()
    p.q[0, 0, 3] *= 2.0 ** -90
    p.q[0, 0, 4] = 0
    p.ring[0, 2] = 0
    p.ring[0, 3] *= 2.0 ** -110
    p.check()


def test_what_is_not_a_number(ops):
    """NaN and infinities reach the heads and queries that read them, and no others, in whichever split they lie."""
    for page in (0, 4, 9):
        p = Split(ops, E=640)
        t = p.cache.book.table[0].long()
        p.cache.pages.view(torch.uint8)[t[page], 5, 77] = 0x7F           # a NaN code
        p.idx[p.idx // 64 == page] = -1
        p.check([e for e in range(640) if e // 64 != page], forms=("list",))
        p.idx[0, 0, 100] = 64 * page + 5
        for split in (True, False):
            for form in FORMS:
                assert p.run(split, form)[:, 77].isnan().all()
        p = Split(ops, E=640)
        p.cache.scales[t[page], 1] = NAN
        for split in (True, False):
            for form in FORMS:
                assert p.run(split, form).isnan().all()
    p = Split(ops, E=640)
    want, tol, _ = p.want()
    p.q[0, 0, 9, 100], p.q[0, 0, 10, 100] = NAN, INF
    rest = [h for h in range(128) if h not in (9, 10)]
    for split in (True, False):
        for form in FORMS:
            out = p.run(split, form)
            assert out[9].isnan().all() and out[10].isnan().all()
            check_close(out[rest], want[rest], tol[rest], f"{form} split={split}")
    p = Split(ops, E=640)
    p.ring[0, 5, 5] = NAN
    for split in (True, False):
        for form in FORMS:
            assert p.run(split, form).isnan().all()


# ------------------------------------------------------------------------------------------------ every entry counts


@pytest.mark.parametrize("B,S,H,W,page,block,pos,ratio", [
    (1, 1, 128, 128, 64, 16, [5], 128),
    (1, 1, 128, 128, 32, 1, [200002], 128),
    (3, 1, 64, 128, 64, 32, [127, 128, 9000], 128),
    (1, 1, 128, 16, 16, 2, [19999], 4),
    (75, 1, 128, 128, 1024, 64, [5000 + i for i in range(75)], 4),
    (1, 50, 32, 128, 64, 16, [350], 4),
    (1, 39, 128, 100, 64, 16, [380], 4),
])
def test_range_in_32_bits(ops, B, S, H, W, page, block, pos, ratio):
    """The range form's fp32 output, held to the mean square of independent roundings too."""
    run_case(ops, B=B, S=S, H=H, W=W, page=page, block=block, pos=pos, ratio=ratio, dtype=torch.float32)


@pytest.mark.parametrize("E", [300, 640, 1000, 5000])
def test_no_entry_is_missing(ops, E):
    """The mean square tells a range that ends one entry early from the whole one."""
    p = Split(ops, E=E)
    want, tol, var = p.want(range(E))
    limit = 2.0 ** -16 * var                     # independent roundings of the weights, each within 2^-8 of itself
    short = p.want(range(E - 1))[0]
    assert np.mean((short - want) ** 2) > 2 * limit
    for form in FORMS if E <= 2048 else ("range",):
        for split in (True, False):
            out = p.run(split, form)
            check_close(out, want, tol, f"{form} split={split}")
            assert np.mean((np64(out) - want) ** 2) <= limit


# ------------------------------------------------------------------------------------------------ long tails


@pytest.mark.parametrize("W", [1, 128])
@pytest.mark.parametrize("f", [1.1875, 1.265625, 1.28125, 1.34375])
def test_long_tail_behind_one_large_weight(ops, f, W):
    """262144 visible entries of weights around 2^-19.4 to 2^-21.9 of the largest, most of a quarter of its mass: they count.
    All but one page hold the same 64 rows, so the sums are taken over those."""
    g = torch.Generator().manual_seed(int(64 * f))
    places, page = 4096, 64
    book = ops.PageTable(i32([[0] + [1] * (places - 1)]), i32([1, places - 1]), page)
    u = torch.ones(D)
    u[1::2] = -1
    rows = (torch.randint(0, 2, (2, page, D // 2), generator=g) * 2.0 - 1).repeat_interleave(2, -1)   # no part along u
    rows[1, :, :16] += (torch.randint(-1, 2, (page, 1), generator=g) * 0.25 * u[:16])                 # or a little: l within 0.18
    rows[0, 7] = u * 0.5                                                                               # the large one
    cache = ops.PagedCache(book, rows.to(torch.float8_e4m3fn).cuda(), torch.ones(2, page // 16, device="cuda"))
    rows = rows.to(torch.float8_e4m3fn).double().numpy()
    H = 8
    q = (u * f).to(torch.bfloat16).expand(1, 1, H, D).contiguous()
    ring, sink = torch.zeros(1, W, D, dtype=torch.bfloat16), torch.full((H,), -INF)
    out = torch.empty(1, 1, H, D, dtype=torch.float32, device="cuda")
    ws = ops.workspace(ops._lib.CSA_WS_HCA_ATTN, 1, 1, 1, 1)
    c = np.concatenate([np.zeros((1, D)), rows.reshape(-1, D)])
    n = np.array([W] + [1] * page + [places - 1] * page, dtype=np.float64)
    l = np64(q[0, 0, 0]) @ c.T / math.sqrt(D)
    w = np.exp(l - l.max())
    ref = O.rope(((n * w) @ c / (n * w).sum())[None], 4 * places * page - 1, 64, 10000.0, inverse=True)[0]
    # A weight's P is w 2^-head, head what the reference is above the maximum: -0.75 for the 4097 tiles or more of one pair, 1 for a
    # sixteenth of them. Below 2^-18 its second piece alone has it: three bits, 2^-3 of itself at most, and 2^-25 for fp16's
    # step below 2^-14. Else it is off by 2^-8 of itself, or 2^-22 and 2^-4 of itself. The denominator has it whole. Scores and
    # additions: 2^-13.
    for head, part in ((-0.75, ws[:256]), (1.0, ws)):
        P = w * 2.0 ** -head
        dP = np.where(P < 2.0 ** -18, P * 2.0 ** -3 + 2.0 ** -25, np.minimum(2.0 ** -8 * P + 2.0 ** -22, 2.0 ** -4 * P))
        tol = (n * (dP * 2.0 ** head + 2.0 ** -13 * w)) @ np.abs(c) / (n * w).sum()
        tol[D - 64:] = tol[D - 64:].reshape(-1, 2).sum(-1).repeat(2)
        ops.hca_attn8(i32([[4 * places * page - 1]]), q.cuda(), ring.cuda(), cache, sink.cuda(), W, ratio=4, out=out, ws=part)
        assert ops.device_status(ws) == 0
        for h in range(H):
            check_close(out[0, 0, h], ref, tol, f"head={head}")
