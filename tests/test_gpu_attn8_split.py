"""Attention over an 8-bit cache in pages where a query's candidates are really split over several CTA pairs and merged."""

import math

import numpy as np
import pytest
import torch

from oracle import csa_oracle as O
from tests.parity import np64
from tests.test_gpu_attn8 import BOUNDS, D, Plain, check_close, i32, make_cache, make_q, reference

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
