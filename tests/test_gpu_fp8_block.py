"""FP8 with one FP32 scale per block of 128 on the GPU, against 64-bit plain forms."""
import numpy as np
import pytest
import torch

import fp8_reference as ref
import microscaling_quantized_linear_b200 as nvq

pytestmark = pytest.mark.gpu

CUDA = "cuda"
U_BF16 = 2.0 ** -8          # half a BF16 step, relative
U_E4M3 = 2.0 ** -4          # half an E4M3 step, relative (normal codes); 2^-10 absolute below


def np32(t):
    return t.float().cpu().numpy()


def randn(*shape, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (std * torch.randn(*shape, generator=g)).bfloat16()


def activation(M, K, seed=0):
    """Normal values, channels of different size, some zero rows and zero blocks."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * torch.exp(torch.randn(1, K, generator=g))
    if M > 4:
        x[3] = 0
    x[-1, :128] = 0
    return x.bfloat16()


def sum_bound(abs_sum, T):
    """Error of an FP32 sum of T terms taken in blocks of 128: each of the at most
    128 additions of a block and ceil(T / 128) of blocks, and the scale products,
    off by at most 2^-23 of the sum of magnitudes (truncation allowed)."""
    return (128 + -(-T // 128) + 4) * 2.0 ** -23 * abs_sum


def check(out, want, bound, unit=U_BF16):
    got = out.double().cpu().numpy()
    inside(got, want, bound + unit * (np.abs(want) + bound))


def inside(got, want, tol):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%d of %d outside, worst %.3g of the tolerance at %s" % (
        bad.sum(), bad.size, np.nanmax(np.abs(got - want) / np.maximum(tol, 1e-300)), np.argwhere(bad)[:4].tolist())


def same(t, want):
    got = t.cpu().numpy()
    got = got.view(np.uint8) if got.dtype != np.float32 else got
    np.testing.assert_array_equal(got, want)


# ------------------------------------------------------------------ quantizers

SHAPES = [(1, 8), (130, 136), (1, 16), (1, 4096), (2, 128), (3, 144), (17, 112), (127, 256), (128, 128), (129, 272), (300, 1040), (513, 64)]


@pytest.mark.parametrize("M,K", SHAPES)
def test_quantize_matches_definition_bit_for_bit(M, K):
    x = activation(M, K, seed=M + K)
    xd, xf = x.to(CUDA), x.float().numpy()
    codes, scales = nvq.fp8_block_quantize(xd)
    c, s = ref.rows_quantize(xf)
    same(codes, c), same(scales, s)
    codes, scales = nvq.fp8_block_quantize_columns(xd)
    c2, s2 = ref.columns_quantize(xf)
    same(codes, c2), same(scales, s2)
    for got, want in zip(nvq.fp8_block_quantize_both(xd), (c, s, c2, s2)):
        same(got, want)
    codes, scales = nvq.fp8_block_quantize_weight(xd)
    c, s = ref.tiles_quantize(xf)
    same(codes, c), same(scales, s)
    assert nvq.device_status() == 0


@pytest.mark.parametrize("exp", [-133, -126, -101, -100, -99, 0, 100, 127])
def test_quantize_extreme_magnitudes(exp):
    """Subnormal, tiny (scale 0 below 2^-100) and huge blocks."""
    x = randn(5, 256, seed=exp & 0xFF).clamp(-1.5, 1.5)
    x[2, 7] = 1.5
    x = (x.double() * 2.0 ** exp).float().bfloat16()
    assert torch.isfinite(x.float()).all()
    c, s = ref.rows_quantize(x.float().numpy())
    codes, scales = nvq.fp8_block_quantize(x.to(CUDA))
    same(codes, c), same(scales, s)


def test_quantize_pitched_offset_and_given_outputs():
    big = randn(200, 512, seed=9).to(CUDA)
    x = big[3:150, 64:64 + 272]                         # pitch 512, 16-byte aligned start
    c, s = ref.rows_quantize(np32(x))
    codes = torch.full((147, 272), 0xEE, dtype=torch.uint8, device=CUDA)
    scales = torch.full((3, 147), -1.0, device=CUDA)
    r = nvq.fp8_block_quantize(x, codes=codes, scales=scales)
    assert r[0] is codes and r[1] is scales
    same(codes, c), same(scales, s)
    c, s = ref.tiles_quantize(np32(x))
    codes, scales = nvq.fp8_block_quantize_weight(x)
    same(codes, c), same(scales, s)


def test_quantize_writes_nothing_past_its_outputs():
    x = activation(131, 144, seed=4).to(CUDA)
    for cells, fn in ((3 * 0 + 2 * 131, nvq.fp8_block_quantize), (2 * 144, nvq.fp8_block_quantize_columns)):
        codes = torch.full((131 * 144 + 4096,), 0xEE, dtype=torch.uint8, device=CUDA)
        scales = torch.full((cells + 1024,), -1.0, device=CUDA)
        shape = (2, 131) if fn is nvq.fp8_block_quantize else (2, 144)
        fn(x, codes=codes[:131 * 144].view(131, 144), scales=scales[:cells].view(shape))
        assert (codes[131 * 144:] == 0xEE).all() and (scales[cells:] == -1.0).all()
        assert (scales[:cells] >= 0).all()


def test_quantize_nonfinite_blocks():
    """A NaN or infinity spoils its own block only, and the status word says so."""
    x = randn(4, 384, seed=3)
    x[1, 130] = float("nan")
    x[2, 5] = float("-inf")
    codes, scales = nvq.fp8_block_quantize(x.to(CUDA))
    assert nvq.device_status() == nvq.NVQ_STATUS_NONFINITE
    c, s = ref.rows_quantize(x.float().numpy())
    same(scales, s)
    v = ref.value(codes, scales, "rows")
    bad = np.isnan(v)
    assert bad[1, 128:256].all() and bad[2, :128].any() and not np.isfinite(v[2, 5])
    bad[1, 128:256] = bad[2, :128] = False
    assert not bad.any()
    out = nvq.fp8_block_linear(codes, scales, *nvq.fp8_block_quantize_weight(randn(16, 384, seed=1).to(CUDA)))
    assert torch.isnan(out[1:3]).all() and torch.isfinite(out[[0, 3]]).all()


def test_empty_batch():
    x = torch.empty(0, 256, dtype=torch.bfloat16, device=CUDA)
    codes, scales = nvq.fp8_block_quantize(x)
    assert codes.shape == (0, 256) and scales.shape == (2, 0)
    rc, rs, cc, cs = nvq.fp8_block_quantize_both(x)
    assert cc.shape == (0, 256) and cs.shape == (0, 256)
    w = nvq.fp8_block_quantize_weight(randn(256, 256).to(CUDA))
    assert nvq.fp8_block_linear(codes, scales, *w).shape == (0, 256)
    assert nvq.fp8_block_linear_dgrad(codes, scales, *w).shape == (0, 256)
    h, hs, gu = nvq.fp8_block_gated_linear(codes, scales, *w, save=True)
    assert h.shape == (0, 128) and hs.shape == (1, 0) and gu.shape == (0, 256)
    out = torch.full((256, 256), 3.0, device=CUDA)
    nvq.fp8_block_linear_wgrad(cc, cs, cc, cs, out=out, accumulate=True)
    assert (out == 3).all()
    nvq.fp8_block_linear_wgrad(cc, cs, cc, cs, out=out)
    assert (out == 0).all()


# ------------------------------------------------------------------ products

def exact_codes(rows, cols, seed):
    """Codes of the values -2 .. 2 in steps of 1/2: products and sums are exact in FP32."""
    g = np.random.default_rng(seed)
    return torch.from_numpy(ref.e4m3_code(g.integers(-4, 5, (rows, cols)).astype(np.float32) / 2))


def pow2_scales(shape, seed):
    return torch.from_numpy(np.exp2(np.random.default_rng(seed).integers(-2, 3, shape)).astype(np.float32))


def operand(rows, cols, kind, seed, exact):
    if exact:
        c = exact_codes(rows, cols, seed)
        s = pow2_scales(nvq.fp8_block_scale_shape(kind, rows, cols), seed + 1)
        return c.to(CUDA), s.to(CUDA)
    x = (activation(rows, cols, seed) if kind != "tiles" else randn(rows, cols, seed=seed, std=0.05)).to(CUDA)
    return {"rows": nvq.fp8_block_quantize, "columns": nvq.fp8_block_quantize_columns,
            "tiles": nvq.fp8_block_quantize_weight}[kind](x)


def product_bounds(A, B, T, exact):
    """A [R, T], B [C, T] in FP64 -> (value, bound of the FP32 sum)."""
    want = A @ B.T
    return want, (0.0 if exact else sum_bound(np.abs(A) @ np.abs(B).T, T))


LINEAR = [(1, 8, 16), (1, 264, 128), (1, 4096, 1024), (2, 136, 144), (8, 520, 2048), (16, 256, 384), (17, 248, 400),
          (31, 1032, 656), (32, 128, 128), (33, 384, 272), (64, 264, 1040), (65, 264, 512), (127, 128, 112), (128, 256, 256),
          (129, 264, 384), (200, 1288, 528), (256, 256, 2048), (257, 520, 144), (513, 776, 640), (1000, 2056, 336),
          (5, 9224, 20496), (40, 264, 8208), (600, 8200, 2320)]                            # more tiles than CTA pairs, more blocks than any ring


@pytest.mark.parametrize("exact", [True, False], ids=["exact", "random"])
@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear(M, N, K, exact):
    a, w = operand(M, K, "rows", 1, exact), operand(N, K, "tiles", 2, exact)
    bias = randn(N, seed=5).to(CUDA)
    want, bound = product_bounds(ref.value(*a, "rows"), ref.value(*w, "tiles"), K, exact)
    check(nvq.fp8_block_linear(*a, *w), want, bound)
    want = want + bias.double().cpu().numpy()
    check(nvq.fp8_block_linear(*a, *w, bias=bias), want, bound + 2.0 ** -24 * np.abs(want))
    assert nvq.device_status() == 0


BACKWARD = [(1, 8, 16), (70, 136, 144), (300, 1032, 272), (1, 16, 16), (3, 256, 144), (64, 272, 400), (100, 144, 272), (128, 256, 384), (129, 400, 256), (257, 528, 1040),
            (700, 1296, 784), (1024, 512, 512), (2500, 272, 528), (600, 2320, 8208), (2320, 600, 8208)]


@pytest.mark.parametrize("exact", [True, False], ids=["exact", "random"])
@pytest.mark.parametrize("M,N,K", BACKWARD)
def test_dgrad(M, N, K, exact):
    dy, w = operand(M, N, "rows", 1, exact), operand(N, K, "tiles", 2, exact)
    want, bound = product_bounds(ref.value(*dy, "rows"), ref.value(*w, "tiles").T, N, exact)
    check(nvq.fp8_block_linear_dgrad(*dy, *w), want, bound)
    assert nvq.device_status() == 0


@pytest.mark.parametrize("exact", [True, False], ids=["exact", "random"])
@pytest.mark.parametrize("M,N,K", BACKWARD)
def test_wgrad(M, N, K, exact):
    dy, x = operand(M, N, "columns", 1, exact), operand(M, K, "columns", 2, exact)
    want, bound = product_bounds(ref.value(*dy, "columns").T, ref.value(*x, "columns").T, M, exact)
    out = nvq.fp8_block_linear_wgrad(*dy, *x)
    assert out.dtype == torch.float32
    check(out, want, bound, unit=2.0 ** -24)
    again = nvq.fp8_block_linear_wgrad(*dy, *x, out=out.clone(), accumulate=True)
    check(again, 2 * want, 2 * bound, unit=2.0 ** -23)
    assert nvq.device_status() == 0


@pytest.mark.parametrize("M", [5, 40, 300])
def test_linear_writes_only_its_output(M):
    """A pitched output: rows and columns around it stay as they were."""
    a, w = operand(M, 272, "rows", 1, True), operand(264, 272, "tiles", 2, True)
    big = torch.full((M + 4, 400), 7.0, dtype=torch.bfloat16, device=CUDA)
    out = big[2:2 + M, 8:272]
    assert nvq.fp8_block_linear(*a, *w, out=out) is out
    assert torch.equal(out.contiguous(), nvq.fp8_block_linear(*a, *w))
    big[2:2 + M, 8:272] = 7.0
    assert (big == 7).all()
    dy = operand(M, 264 + 8, "rows", 3, True)
    w2 = operand(272, 272, "tiles", 2, True)
    out = big[2:2 + M, 8:280]
    nvq.fp8_block_linear_dgrad(*dy, *w2, out=out)
    big[2:2 + M, 8:280] = 7.0
    assert (big == 7).all()
    acc = torch.full((300, 400), 7.0, device=CUDA)
    nvq.fp8_block_linear_wgrad(*operand(M, 272, "columns", 1, True), *operand(M, 144, "columns", 2, True),
                               out=acc[4:276, 16:160])
    acc[4:276, 16:160] = 7.0
    assert (acc == 7).all()


def test_extreme_scales():
    """Scales far from one, and zero, on either side."""
    a, w = operand(40, 384, "rows", 1, True), operand(136, 384, "tiles", 2, True)
    a[1].mul_(2.0 ** 60)
    w[1].mul_(2.0 ** -50)
    a[1][1, 7] = 0
    w[1][1, 2] = 0
    want, _ = product_bounds(ref.value(*a, "rows"), ref.value(*w, "tiles"), 384, True)
    check(nvq.fp8_block_linear(*a, *w), want, 0.0)


def test_all_codes_times_one():
    """Every E4M3 code passes the product unchanged (times one, one term each)."""
    codes = torch.zeros(256, 128, dtype=torch.uint8)
    codes[:, 5] = torch.arange(256, dtype=torch.uint8)
    eye = torch.zeros(128, 128, dtype=torch.uint8)
    eye[:, 5] = 0x38                                    # 1.0
    one = lambda *s: torch.ones(*s, device=CUDA)        # noqa: E731
    out = nvq.fp8_block_linear(codes.to(CUDA), one(1, 256), eye.to(CUDA), one(1, 1))
    v = ref.e4m3_value(np.arange(256))
    got = out.double().cpu().numpy()
    np.testing.assert_array_equal(np.isnan(got[:, 0]), np.isnan(v))
    ok = ~np.isnan(v)
    np.testing.assert_array_equal(got[ok], np.repeat(v[ok][:, None], 128, 1))


# ------------------------------------------------------------------ gated block

def e4m3_step_bound(v, scales, kind):
    """Half a code step around v: 2^-4 of |v|, and never less than 2^-10 scales."""
    s = ref.value(np.full(v.shape, 0x38, np.uint8), scales, kind)
    return U_E4M3 * np.abs(v) + 2.0 ** -10 * s


GATED = [(1, 128, 16), (1, 1408, 1024), (3, 256, 144), (16, 384, 528), (17, 128, 272), (32, 640, 2048), (33, 256, 400),
         (64, 128, 128), (100, 384, 1040), (129, 256, 272), (300, 512, 784), (640, 1408, 400), (1, 12288, 272), (7, 640, 16400), (48, 256, 4112), (600, 4224, 2320)]


def sigmoid_error(g):
    """Relative error of the kernel's sigmoid: exp of a rounded argument (|g| 2^-23)
    with a few units of its own, one addition, one reciprocal."""
    return (np.abs(g) + 8) * 2.0 ** -22


@pytest.mark.parametrize("save", [False, True])
@pytest.mark.parametrize("M,F,K", GATED)
def test_gated_linear(M, F, K, save):
    a, w = operand(M, K, "rows", 1, False), operand(2 * F, K, "tiles", 2, False)
    A, W = ref.value(*a, "rows"), ref.value(*w, "tiles")
    gu, e = product_bounds(A, W, K, False)
    codes, scales, saved = nvq.fp8_block_gated_linear(*a, *w, save=save)
    assert (saved is not None) == save
    if save:
        check(saved, gu, e)
    gate, up = gu[:, :F], gu[:, F:]
    h = ref.silu(gate) * up
    # |SiLU'| < 1.1
    eh = 1.1 * e[:, :F] * np.abs(up) + np.abs(ref.silu(gate)) * e[:, F:] + e[:, :F] * e[:, F:] + sigmoid_error(gate) * np.abs(h)
    pad = lambda t: t.reshape(M, F // 128, 128)         # noqa: E731
    amax, ea = np.abs(pad(h)).max(2).T, pad(eh).max(2).T
    s = scales.double().cpu().numpy()
    inside(s, amax / 448, ea / 448 + 2.0 ** -23 * amax / 448)
    got = ref.value(codes, scales, "rows")
    # a code may be that of any value within eh, and its scale off by the same
    inside(got, h, e4m3_step_bound(np.abs(h) + eh, scales, "rows") + eh * (1 + U_E4M3) + 2.0 ** -20 * np.abs(h))
    assert nvq.device_status() == 0


@pytest.mark.parametrize("M", [3, 70])
def test_gated_linear_whose_gate_times_up_passes_fp32(M):
    """SiLU(gate) * up is finite where gate * up is not: -80 and -200 times 2^120."""
    a = torch.zeros(M, 128, dtype=torch.bfloat16)
    a[:, 0] = 1
    w = torch.zeros(256, 128, dtype=torch.bfloat16)
    w[:64, 0], w[64:128, 0], w[128:, 0] = -80.0, -200.0, 2.0 ** 120
    w_codes, w_scales = nvq.fp8_block_quantize_weight(w.to(CUDA))
    codes, scales, gu = nvq.fp8_block_gated_linear(*nvq.fp8_block_quantize(a.to(CUDA)), w_codes, w_scales, save=True)
    gate = ref.value(w_codes, w_scales, "tiles")[:128, 0]
    h = np.broadcast_to(ref.silu(gate) * 2.0 ** 120, (M, 128))
    e = 2 * sigmoid_error(gate) * np.abs(h) + 2.0 ** -20 * np.abs(h)
    assert np.abs(h).max() > 1 and nvq.device_status() == 0
    assert torch.isfinite(scales).all()
    inside(ref.value(codes, scales, "rows"), h, e4m3_step_bound(np.abs(h) + e, scales, "rows") + 2 * e)


def test_gated_linear_of_zero_rows_is_zero():
    a = nvq.fp8_block_quantize(torch.zeros(70, 256, dtype=torch.bfloat16, device=CUDA))
    codes, scales, gu = nvq.fp8_block_gated_linear(*a, *operand(512, 256, "tiles", 2, False), save=True)
    assert (scales == 0).all() and (gu == 0).all() and ((codes & 0x7F) == 0).all()


@pytest.mark.parametrize("M,F", [(1, 128), (2, 384), (31, 256), (128, 128), (129, 640), (300, 1408)])
def test_gated_backward(M, F):
    gu, dh = randn(M, 2 * F, seed=1, std=3.0), activation(M, F, seed=2)
    gu[0, :8] = torch.tensor([0.0, -0.0, 90.0, -90.0, 300.0, -300.0, -1.28125, 20.0]).bfloat16()
    got = nvq.fp8_block_gated_backward(dh.to(CUDA), gu.to(CUDA))
    G, U, D = (t.double().numpy() for t in (gu[:, :F], gu[:, F:], dh))
    dg, du, h = ref.gated_grads(D, G, U)
    sig = 1 / (1 + np.exp(-G))
    se = sigmoid_error(G) + 2.0 ** -21
    e = np.concatenate((np.abs(D * U) * sig * (2 + 3 * np.abs(G)) * se, np.abs(du) * se), 1)
    d = np.concatenate((dg, du), 1)
    for (codes, scales), v, ev, kind in ((got[0], d, e, "rows"), (got[1], d, e, "columns"), (got[2], h, np.abs(h) * se, "columns")):
        R, C = v.shape
        assert tuple(codes.shape) == (R, C) and tuple(scales.shape) == nvq.fp8_block_scale_shape(kind, R, C)
        blocks = lambda t: (np.stack([t[:, i:i + 128].max(1) for i in range(0, C, 128)]) if kind == "rows"     # noqa: E731
                            else np.stack([t[i:i + 128].max(0) for i in range(0, R, 128)]))
        s, amax, ea = scales.double().cpu().numpy(), blocks(np.abs(v)), blocks(ev)
        # a block below 2^-100 is zero by definition; exp(-g) overflows for g < -88,
        # where sigma < 2^-126 and |dH|, |up| < 2^10, |g| < 2^9 leave less than 2^-97
        inside(s, amax / 448, (ea + 2.0 ** -23 * amax + 2.0 ** -97) / 448)
        q = ref.value(codes, scales, kind)
        inside(q, v, e4m3_step_bound(np.abs(v) + ev, scales, kind) + ev * (1 + U_E4M3) + 2.0 ** -20 * np.abs(v) + 2.0 ** -97)
    assert nvq.device_status() == 0


def test_gated_backward_pitched_inputs():
    gu, dh = randn(70, 600, seed=1).to(CUDA)[:, 16:528], randn(70, 400, seed=2).to(CUDA)[:, 8:264]
    for x, y in zip(nvq.fp8_block_gated_backward(dh, gu), nvq.fp8_block_gated_backward(dh.contiguous(), gu.contiguous())):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_gated_backward_against_differences():
    """dH . H's derivative along random directions, by central differences of the 64-bit formula."""
    M, F = 9, 256
    gu, dh = randn(M, 2 * F, seed=1), randn(M, F, seed=2)
    (rc, rs), _, _ = nvq.fp8_block_gated_backward(dh.to(CUDA), gu.to(CUDA))
    grad = ref.value(rc, rs, "rows")
    G, D = gu.double().numpy(), dh.double().numpy()
    f = lambda z: (D * ref.silu(z[:, :F]) * z[:, F:]).sum(1)      # noqa: E731
    for seed in range(3):
        v = np.random.default_rng(seed).standard_normal(G.shape)
        want = (f(G + 1e-5 * v) - f(G - 1e-5 * v)) / 2e-5
        # every code off by at most half a step (its block's largest code has 448)
        tol = (e4m3_step_bound(grad, rs, "rows") * 1.07 * np.abs(v)).sum(1)
        inside((grad * v).sum(1), want, tol + 1e-6)


# ------------------------------------------------------------------ together

def test_feed_forward_forward_and_backward():
    """A gated feed-forward block's training step out of the operators, each
    product against FP64 on the operands it was given."""
    M, K, F = 200, 272, 384
    x, dy = activation(M, K, 1).to(CUDA), randn(M, K, seed=7, std=1e-3).to(CUDA)
    wgu = nvq.fp8_block_quantize_weight(randn(2 * F, K, seed=2, std=0.05).to(CUDA))
    wd = nvq.fp8_block_quantize_weight(randn(K, F, seed=3, std=0.05).to(CUDA))
    xr, xs, xc, xcs = nvq.fp8_block_quantize_both(x)
    h, hs, gu = nvq.fp8_block_gated_linear(xr, xs, *wgu, save=True)
    y = nvq.fp8_block_linear(h, hs, *wd)
    want, b = product_bounds(ref.value(h, hs, "rows"), ref.value(*wd, "tiles"), F, False)
    check(y, want, b)
    dr, drs, dc, dcs = nvq.fp8_block_quantize_both(dy)
    dh = nvq.fp8_block_linear_dgrad(dr, drs, *wd)
    want, b = product_bounds(ref.value(dr, drs, "rows"), ref.value(*wd, "tiles").T, K, False)
    check(dh, want, b)
    rows, cols, hc = nvq.fp8_block_gated_backward(dh, gu)
    dwd = nvq.fp8_block_linear_wgrad(dc, dcs, *hc)
    want, b = product_bounds(ref.value(dc, dcs, "columns").T, ref.value(*hc, "columns").T, M, False)
    check(dwd, want, b, unit=2.0 ** -24)
    dx = nvq.fp8_block_linear_dgrad(*rows, *wgu)
    want, b = product_bounds(ref.value(*rows, "rows"), ref.value(*wgu, "tiles").T, 2 * F, False)
    check(dx, want, b)
    dwgu = nvq.fp8_block_linear_wgrad(*cols, xc, xcs)
    want, b = product_bounds(ref.value(*cols, "columns").T, ref.value(xc, xcs, "columns").T, M, False)
    check(dwgu, want, b, unit=2.0 ** -24)
    assert nvq.device_status() == 0


def _step(x, w, wgu):
    a = nvq.fp8_block_quantize(x)
    y = nvq.fp8_block_linear(*a, *w)
    h, hs, gu = nvq.fp8_block_gated_linear(*a, *wgu, save=True)
    rc, rs, cc, cs = nvq.fp8_block_quantize_both(y)
    dx = nvq.fp8_block_linear_dgrad(rc, rs, *w)
    back = nvq.fp8_block_gated_backward(gu[:, :gu.shape[1] // 2], gu)
    dw = nvq.fp8_block_linear_wgrad(cc, cs, *back[2])
    return [y, h, hs, gu, dx, dw, *back[0], *back[1]]


@pytest.mark.parametrize("M", [1, 24, 200])
def test_graph_replay_and_other_stream(M):
    """Captured and replayed on new inputs, and run on a stream other than the current one: the same bits."""
    w = nvq.fp8_block_quantize_weight(randn(272, 400, seed=2, std=0.05).to(CUDA))
    wgu = nvq.fp8_block_quantize_weight(randn(512, 400, seed=3, std=0.05).to(CUDA))
    xs = [activation(M, 400, s).to(CUDA) for s in range(3)]
    want = [_step(x, w, wgu) for x in xs]
    x = xs[0].clone()
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        outs = _step(x, w, wgu)
    for i in (1, 2, 0):
        x.copy_(xs[i])
        g.replay()
        torch.cuda.synchronize()
        for got, ex in zip(outs, want[i]):
            assert torch.equal(got, ex)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    codes, scales = nvq.fp8_block_quantize(xs[1], stream=s)
    y = nvq.fp8_block_linear(codes, scales, *w, stream=s)
    h, hs, _ = nvq.fp8_block_gated_linear(codes, scales, *wgu, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for got, ex in zip((y, h, hs), want[1]):
        assert torch.equal(got, ex)


def test_two_streams_at_once():
    """Calls on two streams share nothing: repeated side by side they give the same bits as alone."""
    w = nvq.fp8_block_quantize_weight(randn(1024, 2048, seed=2, std=0.05).to(CUDA))
    a = [nvq.fp8_block_quantize(activation(m, 2048, m).to(CUDA)) for m in (4, 300)]
    want = [nvq.fp8_block_linear(*x, *w) for x in a]
    streams = [torch.cuda.Stream() for _ in a]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            got[i].append(nvq.fp8_block_linear(*a[i], *w, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(t, want[i]) for t in got[i])


def test_float8_dtype_views_are_taken():
    a, w = operand(9, 256, "rows", 1, True), operand(136, 256, "tiles", 2, True)
    f8 = torch.float8_e4m3fn
    assert torch.equal(nvq.fp8_block_linear(a[0].view(f8), a[1], w[0].view(f8), w[1]), nvq.fp8_block_linear(*a, *w))


# ------------------------------------------------------------------ layers, failure, debug build

@pytest.mark.parametrize("M", [1, 20, 300])
def test_linear_layer(M):
    K, N = 272, 400
    w, b, x, dy = randn(N, K, seed=1, std=0.05).to(CUDA), randn(N, seed=2).to(CUDA), activation(M, K, 3).to(CUDA), randn(M, N, seed=4).to(CUDA)
    layer = nvq.BlockFp8Linear(w, b)
    y, saved = layer.forward(x)
    assert torch.equal(y, layer(x))
    a = nvq.fp8_block_quantize(x)
    assert torch.equal(y, nvq.fp8_block_linear(*a, *nvq.fp8_block_quantize_weight(w), bias=b))
    dx, dw, db = layer.backward(dy, saved)
    X, W, D = (t.double().cpu().numpy() for t in (x, w, dy))
    # three quantizations' half steps: relative to the sums of magnitudes
    q = 2 * U_E4M3 + U_E4M3 ** 2 + 2.0 ** -8
    inside(dx.double().cpu().numpy(), D @ W, q * (np.abs(D) @ np.abs(W)) + 2.0 ** -9 * np.abs(D).max() * np.abs(W).max() * N)
    inside(dw.double().cpu().numpy(), D.T @ X, q * (np.abs(D.T) @ np.abs(X)) + 2.0 ** -9 * np.abs(D).max() * np.abs(X).max() * M)
    inside(db.double().cpu().numpy(), D.sum(0), M * 2.0 ** -24 * np.abs(D).sum(0))
    again = layer.backward(dy, saved, dw=dw.clone())[1]
    inside(again.double().cpu().numpy(), 2 * dw.double().cpu().numpy(), 2.0 ** -23 * np.abs(dw.double().cpu().numpy()))
    layer.update(2 * w)
    assert torch.equal(layer(x), nvq.fp8_block_linear(*a, *nvq.fp8_block_quantize_weight(2 * w), bias=b))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2, saved2 = layer.forward(x, stream=s)
    g2 = layer.backward(dy, saved2, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y2, layer(x)) and torch.equal(g2[1], dw) and torch.equal(g2[2], db)


def test_layers_take_an_empty_batch():
    """Outputs without rows, weight gradients of zeros."""
    layer, x = nvq.BlockFp8Linear(randn(264, 272).to(CUDA), randn(264).to(CUDA)), torch.empty(0, 272, dtype=torch.bfloat16, device=CUDA)
    y, saved = layer.forward(x)
    dx, dw, db = layer.backward(y, saved)
    assert y.shape == layer(x).shape == (0, 264) and dx.shape == (0, 272) and (dw == 0).all() and (db == 0).all()
    ff = nvq.BlockFp8GatedFF(randn(512, 272).to(CUDA), randn(264, 256).to(CUDA))
    y, saved = ff.forward(x)
    dx, dwgu, dwd = ff.backward(y, saved)
    assert y.shape == ff(x).shape == (0, 264) and dx.shape == (0, 272)
    assert dwgu.shape == (512, 272) and dwd.shape == (264, 256) and (dwgu == 0).all() and (dwd == 0).all()


def test_linear_of_an_output_past_32_bits():
    """70,016 x 32,776 values: offsets pass 2^31; the last rows and columns, exactly."""
    M, N, K = 70016, 32776, 144
    a, w = operand(M, K, "rows", 1, True), operand(N, K, "tiles", 2, True)
    out = nvq.fp8_block_linear(*a, *w)
    B = ref.value(*w, "tiles")
    for i in (0, 65530, M - 40):
        rows = ref.value(a[0][i:i + 40], a[1][:, i:i + 40].contiguous(), "rows")
        check(out[i:i + 40], rows @ B.T, 0.0)


@pytest.mark.parametrize("M", [1, 20, 300])
def test_gated_ff_layer(M):
    K, F, N = 272, 384, 256
    wgu, wd = randn(2 * F, K, seed=1, std=0.05).to(CUDA), randn(N, F, seed=2, std=0.05).to(CUDA)
    x, dy = activation(M, K, 3).to(CUDA), randn(M, N, seed=4).to(CUDA)
    ff = nvq.BlockFp8GatedFF(wgu, wd)
    y, saved = ff.forward(x)
    assert torch.equal(y, ff(x))
    h, hs, _ = nvq.fp8_block_gated_linear(*nvq.fp8_block_quantize(x), *nvq.fp8_block_quantize_weight(wgu))
    assert torch.equal(y, nvq.fp8_block_linear(h, hs, *nvq.fp8_block_quantize_weight(wd)))
    dx, dwgu, dwd = ff.backward(dy, saved)
    # the gradients of the BF16 block, to the accuracy that E4M3 operands leave: 2-norms within 15 %
    # (each of at most five quantizations on a path is within 2^-4 of each value)
    p = [t.double().requires_grad_() for t in (x, wgu, wd)]
    gu = p[0] @ p[1].t()
    out = (torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]) @ p[2].t()
    out.backward(dy.double())
    for got, want in zip((y, dx, dwgu, dwd), (out.detach(), p[0].grad, p[1].grad, p[2].grad)):
        assert (got.double() - want).norm() <= 0.15 * want.norm()
    again = ff.backward(dy, saved, dw_gate_up=dwgu.clone(), dw_down=dwd.clone())
    assert torch.equal(again[0], dx) and torch.allclose(again[1], 2 * dwgu, rtol=2.0 ** -22, atol=0) and torch.allclose(again[2], 2 * dwd, rtol=2.0 ** -22, atol=0)
    with pytest.raises(ValueError, match="rows"):
        nvq.BlockFp8GatedFF(wgu, wgu)


def test_timeout_is_reported_and_leaves_the_context_usable():
    """With a wait limit of 1 ns a product may give up; it says so and returns, and the next is right."""
    big = [(operand(m, 4096, "rows", 1, False), operand(4096, 4096, "tiles", 2, False)) for m in (8, 2000)]
    want = [nvq.fp8_block_linear(*a, *w) for a, w in big]
    assert nvq.device_status() == 0
    for (a, w), y in zip(big, want):
        nvq.set_wait_limit(1)
        try:
            nvq.fp8_block_linear(*a, *w)
            assert nvq.device_status() in (0, nvq.NVQ_STATUS_TIMEOUT)
        finally:
            nvq.set_wait_limit(0)
        assert torch.equal(nvq.fp8_block_linear(*a, *w), y)
        assert nvq.device_status() == 0


DEBUG_RUN = """
import sys
sys.path[:0] = [%r, %r]
import torch
import microscaling_quantized_linear_b200 as nvq
import test_gpu_fp8_block as t
assert nvq.DEBUG_BUILD
for M, K in t.SHAPES:
    t.test_quantize_matches_definition_bit_for_bit(M, K)
for M, N, K in [(1, 264, 128), (17, 248, 400), (65, 264, 512), (257, 520, 144), (1000, 2056, 336)]:
    t.test_linear(M, N, K, True)
for M, N, K in [(1, 8, 16), (300, 1032, 272), (129, 400, 256), (700, 1296, 784)]:
    t.test_dgrad(M, N, K, True)
    t.test_wgrad(M, N, K, True)
for M, F, K in [(3, 256, 144), (33, 256, 400), (300, 512, 784)]:
    t.test_gated_linear(M, F, K, True)
for M, F in [(1, 128), (129, 640)]:
    t.test_gated_backward(M, F)
assert nvq.device_status() == 0
print("clean")
"""


def test_debug_build_finds_no_access_out_of_bounds():
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    out = subprocess.run([sys.executable, "-c", DEBUG_RUN % (os.path.dirname(here), here)], env=dict(os.environ, NVQ_DEBUG="1"),
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "clean" in out.stdout, out.stdout[-2000:] + out.stderr[-4000:]


CAPTURE_FIRST = """
import sys
sys.path[:0] = [%r, %r]
import torch
import microscaling_quantized_linear_b200 as nvq
x = torch.randn(300, 256, device="cuda").bfloat16()
t = torch.randn(8, 256, device="cuda").bfloat16()
w = torch.randn(512, 256, device="cuda").bfloat16()
def step():
    wq = nvq.fp8_block_quantize_weight(w)
    rc, rs, cc, cs = nvq.fp8_block_quantize_both(x)
    h, hs, gu = nvq.fp8_block_gated_linear(rc, rs, *wq, save=True)
    back = nvq.fp8_block_gated_backward(x, gu)
    y = nvq.fp8_block_linear(rc, rs, *wq)
    return [h, hs, gu, y, nvq.fp8_block_linear_dgrad(*back[0], *wq), nvq.fp8_block_linear_wgrad(*back[1], cc, cs),
            nvq.fp8_block_linear(*nvq.fp8_block_quantize(t), *wq)]
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = step()
g.replay()
torch.cuda.synchronize()
for a, b in zip(out, step()):
    assert torch.equal(a, b)
assert nvq.device_status() == 0
print("same")
"""


def test_first_calls_may_be_captured():
    """In a fresh process every entry point's first call is inside a graph capture."""
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    out = subprocess.run([sys.executable, "-c", CAPTURE_FIRST % (os.path.dirname(here), here)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "same" in out.stdout, out.stdout[-2000:] + out.stderr[-4000:]
