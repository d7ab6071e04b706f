"""Split-candidate attention where the rotated dims do not begin at a multiple of 4."""

import math

import pytest
import torch

from oracle import csa_oracle as O
from tests.parity import assert_attn_close, np64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rope_dim", [2, 6, 64])
def test_split_attention_rotates_from_any_even_dim(rope_dim):
    from long_context_decode_c4a_b200 import ops
    g = torch.Generator().manual_seed(rope_dim)
    t, W, E, H = 4 * 500 + 3, 128, 500, 16
    q = torch.randn(1, 1, H, 512, generator=g).to(torch.bfloat16)
    ring, cache = torch.randn(1, W, 512, generator=g).to(torch.bfloat16), torch.randn(1, E, 512, generator=g).to(torch.bfloat16)
    idx, sink = torch.arange(E, dtype=torch.int32).view(1, 1, E), torch.randn(H, generator=g)
    out = torch.empty(1, 1, H, 512, dtype=torch.float32, device="cuda")
    ops.sparse_attn(torch.tensor([[t]], dtype=torch.int32, device="cuda"), q.cuda(), ring.cuda(), cache.cuda(), idx.cuda(), sink.cuda(),
                    W, out=out, rope_dim=rope_dim)
    ref = O.attend_query(np64(q[0, 0]), t, W, np64(ring[0]), W, np64(cache[0]), range(E), np64(sink), 1 / math.sqrt(512), rope_dim, 10000.0)
    assert_attn_close(out[0, 0], ref, f"rope_dim={rope_dim}")
