"""NaN and infinities in the FP8 block-scaled operators: they spoil what reads their block, nothing else, and the
status word reports them."""
import numpy as np
import pytest
import torch

import fp8_reference as ref
import microscaling_quantized_linear_b200 as nvq
from test_gpu_fp8_block import activation, operand, randn, same

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def spoiled(M, K, seed):
    """Values with a NaN, an infinity and a negative one in three blocks of their own."""
    x = activation(M, K, seed)
    x[1, K - 3], x[2, 5], x[M - 1, K // 2] = NAN, -INF, INF
    return x


def reported():
    return nvq.device_status() == nvq.NVQ_STATUS_NONFINITE


@pytest.mark.parametrize("M,K", [(5, 144), (130, 272), (300, 520)])
def test_quantizers_keep_nonfinite_values_in_their_blocks(M, K):
    """Every orientation, bit for bit the definition: a NaN scale, an infinite one, codes of NaN where they stand."""
    x = spoiled(M, K, M)
    xd, xf = x.cuda(), x.float().numpy()
    for fn, want in ((nvq.fp8_block_quantize, ref.rows_quantize), (nvq.fp8_block_quantize_columns, ref.columns_quantize),
                     (nvq.fp8_block_quantize_weight, ref.tiles_quantize)):
        codes, scales = fn(xd)
        assert reported()
        c, s = want(xf)
        same(scales, s)
        c = np.where(np.isnan(xf) | np.isinf(xf), c & 0x7F, c)           # the sign of a NaN code says nothing
        got = codes.cpu().numpy()
        same(torch.from_numpy(np.where((got & 0x7F) == 0x7F, got & 0x7F, got)), c)
    both = nvq.fp8_block_quantize_both(xd)
    assert reported()
    for got, want in zip(both, (*nvq.fp8_block_quantize(xd), *nvq.fp8_block_quantize_columns(xd))):
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
    assert reported()


def test_weight_gradient_of_spoiled_columns():
    M, N, K = 300, 264, 272
    dy, x = randn(M, N, seed=1), spoiled(M, K, 2)
    dw = nvq.fp8_block_linear_wgrad(*nvq.fp8_block_quantize_columns(dy.cuda()), *nvq.fp8_block_quantize_columns(x.cuda()))
    assert reported()
    bad = torch.isnan(dw)
    cols = [K - 3, 5, K // 2]
    assert bad[:, cols].all()
    bad[:, cols] = False
    assert not bad.any() and torch.isfinite(dw[:, [c for c in range(K) if c not in cols]]).all()


@pytest.mark.parametrize("M", [4, 40, 300])
def test_input_gradient_of_spoiled_tiles(M):
    """A NaN in a weight: its 128 input columns are NaN, the others are not."""
    w = randn(264, 272, seed=3, std=0.05)
    w[200, 130] = NAN
    q = nvq.fp8_block_quantize_weight(w.cuda())
    assert reported()
    dx = nvq.fp8_block_linear_dgrad(*operand(M, 264, "rows", 1, False), *q)
    assert torch.isnan(dx[:, 128:256]).all()
    assert torch.isfinite(dx[:, :128]).all() and torch.isfinite(dx[:, 256:]).all()


@pytest.mark.parametrize("M", [4, 40, 300])
def test_gated_linear_of_spoiled_rows_and_tiles(M):
    K, F = 272, 384
    a, w = activation(M, K, 1), randn(2 * F, K, seed=2, std=0.05)
    wq = nvq.fp8_block_quantize_weight(w.cuda())
    clean = nvq.fp8_block_gated_linear(*nvq.fp8_block_quantize(a.cuda()), *wq, save=True)
    assert nvq.device_status() == 0
    a[1, 200], a[2, 3] = NAN, INF
    aq = nvq.fp8_block_quantize(a.cuda())
    assert reported()
    codes, scales, gu = nvq.fp8_block_gated_linear(*aq, *wq, save=True)
    assert reported()
    rows = [r for r in range(M) if r not in (1, 2)]
    assert torch.isnan(gu[1:3]).all() and torch.isnan(scales[:, 1:3]).all()
    assert torch.equal(codes[rows], clean[0][rows]) and torch.equal(scales[:, rows], clean[1][:, rows])
    assert torch.equal(gu[rows], clean[2][rows])
    # a NaN in a tile of up: one block of every row of H
    a[1, 200], a[2, 3] = 0, 0
    w[F + 130, 3] = NAN
    wq = nvq.fp8_block_quantize_weight(w.cuda())
    nvq.device_status()
    aq = nvq.fp8_block_quantize(a.cuda())
    codes, scales, gu = nvq.fp8_block_gated_linear(*aq, *wq, save=True)
    assert reported()
    assert torch.isnan(scales[1]).all() and torch.isfinite(scales[[0, 2]]).all()
    assert torch.isnan(gu[:, F + 128:F + 256]).all() and torch.isfinite(gu[:, :F]).all()


@pytest.mark.parametrize("which,value", [("dh", NAN), ("dh", INF), ("up", NAN), ("up", -INF), ("gate", NAN), ("gate", INF), ("gate", -INF)])
def test_gated_backward_of_spoiled_inputs(which, value):
    """Row blocks and columns that read the value are not finite; the rest keep their bits."""
    M, F, r, c = 300, 384, 140, 129 + 17
    gu, dh = randn(M, 2 * F, seed=1, std=2.0), randn(M, F, seed=2)
    gu[:, 144:152] = 0.5                                    # one path for the octet, with the value or without
    gu[r, 144:152] = 60.0
    clean = nvq.fp8_block_gated_backward(dh.cuda(), gu.cuda())
    assert nvq.device_status() == 0
    (dh if which == "dh" else gu)[r, c + (F if which == "up" else 0)] = value
    got = nvq.fp8_block_gated_backward(dh.cuda(), gu.cuda())
    assert reported()
    bad = {"dh": (True, True, False), "up": (True, False, True), "gate": (True, True, True)}[which]   # dG, dU, H
    (rc, rs), (cc, cs), (hc, hs) = got
    nonfinite = lambda t: ~torch.isfinite(t)                # noqa: E731
    want = torch.zeros_like(rs, dtype=torch.bool)
    want[1, r], want[F // 128 + 1, r] = bad[0], bad[1]
    assert torch.equal(nonfinite(rs), want)
    want = torch.zeros_like(cs, dtype=torch.bool)
    want[1, c], want[1, F + c] = bad[0], bad[1]
    assert torch.equal(nonfinite(cs), want)
    want = torch.zeros_like(hs, dtype=torch.bool)
    want[1, c] = bad[2]
    assert torch.equal(nonfinite(hs), want)
    rows = [i for i in range(M) if i != r]
    assert torch.equal(rc[rows], clean[0][0][rows]) and torch.equal(rs[:, rows], clean[0][1][:, rows])
    for t, ts, u, us, n, spoilt in ((cc[:, :F], cs[:, :F], *(x[:, :F] for x in clean[1]), F, bad[0]),
                                    (cc[:, F:], cs[:, F:], *(x[:, F:] for x in clean[1]), F, bad[1]), (hc, hs, *clean[2], F, bad[2])):
        cols = [i for i in range(n) if i != c or not spoilt]
        assert torch.equal(t[:, cols], u[:, cols]) and torch.equal(ts[:, cols], us[:, cols])
        assert torch.equal(t[:128], u[:128]) and torch.equal(t[256:], u[256:])
