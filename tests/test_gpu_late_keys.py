"""Whole-scene attention when one late key's logit is hundreds of log2 units above every key before it and the rows
of a warp are alike, so that no other row notices: the offset of the softmax is then far below that logit, where a
2^x whose exponent is added as an integer has no exponent bits left.

Tolerances as in test_gpu_streaming.py: P and O rounded to bf16 (2^-8 each), exponentials off by 7.5e-5 and logits by
the rounding of an fp32 sum of 64 exact products, both entering P and the sum."""
import numpy as np
import pytest
import torch

import oracle
import streaming_ref as ref
from feed_forward_view_vggt_b200 import attn

pytestmark = pytest.mark.gpu
D = 64


def scene(n, h, w, heads, at, seed=5):
    """Shape, q (all rows alike), k (with one late key along q), v."""
    shape = attn.vggt_shape(n, 5, h, w, heads, D)
    rows = n * (5 + h * w)
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(rows, heads, D, generator=g).bfloat16() for _ in range(3))
    q[:] = q[0].clone()
    k[at] = 40 * q[0].float()
    return shape, q.cuda(), k.cuda(), v.cuda()


def logit_error(q, k, at):
    return 64 * 2.0 ** -24 * (q.double().abs() * k[at].double().abs()).sum(-1).max().item() * D ** -0.5


def check(got, want, spread, off):
    tol = 2.0 ** -8 * (1.01 * want.abs() + 1.12 * spread) + 2 * off * spread + 1e-30
    worst = ((got.double() - want).abs() / tol).max().item()
    assert worst <= 1.0, worst


@pytest.mark.parametrize("n,h,w", [(6, 12, 12), (8, 14, 14)])
@pytest.mark.parametrize("at", [640, 643, 647, 655])
def test_global(n, h, w, at):
    shape, q, k, v = scene(n, h, w, 4, at)
    got = attn.global_(q, k, v, shape)
    assert attn.vggt_check()[0] == attn.VGGT_OK
    rows = q.shape[0]
    want, _, spread = ref.attention(q, [k], [v], [0, rows], [rows], 0)
    check(got, want, spread, logit_error(q, k, at))


@pytest.mark.parametrize("slot", [128, 131, 135, 143])
def test_frame(slot):
    n, h, w = 3, 16, 16
    L = 5 + h * w
    shape, q, k, v = scene(n, h, w, 4, L + slot)  # of the second frame
    got = attn.frame(q, k, v, shape)
    assert attn.vggt_check()[0] == attn.VGGT_OK
    cu = [L * i for i in range(n + 1)]
    split = lambda t: [t[cu[i]:cu[i + 1]] for i in range(n)]  # noqa: E731
    want, _, spread = ref.attention(q, split(k), split(v), cu, [L] * n, 0)
    check(got, want, spread, logit_error(q, k, L + slot))


@pytest.mark.parametrize("slot", [0, 2, 4])
def test_sga(slot):
    # special tokens are kept: with 2 x 2 of 12 x 12 those of frame 4 are kept keys 164 to 168
    n, h, w, heads = 6, 12, 12, 4
    at = 4 * (5 + h * w) + slot
    shape, q, k, v = scene(n, h, w, heads, at)
    got = attn.sga(q, k, v, attn.SgaIndex(shape, 2, 2))
    assert attn.vggt_check()[0] == attn.VGGT_OK
    bits = [t.cpu().contiguous().view(torch.int16).numpy().view(np.uint16) for t in (q, k, v)]
    want, _ = oracle.sga_attention(*bits, oracle.Shape(n, 5, h, w, heads, D), 2, 2, rows=np.arange(q.shape[0]))
    # the late key has nearly all the weight of every row: A = sum p |v| / l is |v| of it
    want = torch.as_tensor(want, dtype=torch.float64, device="cuda")
    assert torch.allclose(want, v[at].double().expand_as(want), atol=1e-12)
    check(got, want, want.abs(), logit_error(q, k, at))
