"""The FP8 block-scaled operators at the ends of their ranges, against 64-bit plain forms."""
import numpy as np
import numpy as np
import pytest
import torch

import fp8_reference as ref
import microscaling_quantized_linear_b200 as nvq
from test_gpu_fp8_block import check, e4m3_step_bound, inside, operand, product_bounds, sigmoid_error

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ scales

@pytest.mark.parametrize("big", [105, -109])
@pytest.mark.parametrize("M,N,K", [(40, 136, 272), (300, 400, 528)])
def test_products_of_opposing_scales(M, N, K, big):
    """One operand's scales near the end of FP32, the other's bringing their product back, and codes of 256 to
    448 of one sign, whose blocks sum to 2^24: exact, in steps of 2^12."""
    small = -60 if big > 0 else 64
    for op, kinds, shapes in ((nvq.fp8_block_linear, ("rows", "tiles"), ((M, K), (N, K))),
                              (nvq.fp8_block_linear_dgrad, ("rows", "tiles"), ((M, N), (N, K))),
                              (nvq.fp8_block_linear_wgrad, ("columns", "columns"), ((M, N), (M, K)))):
        for ea, eb in ((big, small), (small, big)):
            a, b = (operand(*s, k, i, True) for i, (s, k) in enumerate(zip(shapes, kinds)))
            for codes, _ in (a, b):
                codes.bitwise_and_(7).bitwise_or_(0x78).clamp_(max=0x7E)
            a[1].mul_(2.0 ** ea)
            b[1].mul_(2.0 ** eb)
            A, B = ref.value(*a, kinds[0]), ref.value(*b, kinds[1])
            if op is nvq.fp8_block_linear_dgrad:
                B, T = B.T, N
            elif op is nvq.fp8_block_linear_wgrad:
                A, B, T = A.T, B.T, M
            else:
                T = K
            want, _ = product_bounds(A, B, T, True)
            check(op(*a, *b), want, 0.0, unit=2.0 ** -24 if op is nvq.fp8_block_linear_wgrad else 2.0 ** -8)
    assert nvq.device_status() == 0


# ------------------------------------------------------------------ gates

# gates (multiples of 4 that E4M3 holds at a block scale of 1/2); below -87 SiLU is 0 by definition, where it is
# less than |g| 2^-125
GATES = [-208.0, -176.0, -160.0, -144.0, -128.0, -112.0, -104.0, -96.0, -88.0, -80.0, -40.0, -8.0, 0.0, 8.0, 96.0, 224.0]


def cut(g):
    """What taking sigma below -87 as 0 changes, relative to |g|."""
    return np.where(g < -87, 2.0 ** -125, 0.0)


@pytest.mark.parametrize("up", [0, 60, 120, 126])
@pytest.mark.parametrize("M", [3, 70])
def test_gated_linear_of_far_gates(M, up):
    """A row of A times one gate and 2^up: H to the accuracy of the sigmoid."""
    a = torch.zeros(M, 128, dtype=torch.bfloat16)
    a[:, 0] = 1
    for gate in GATES:
        w = torch.zeros(256, 128, dtype=torch.bfloat16)
        w[:128, 0], w[128:, 0] = gate, 2.0 ** up
        w[0, 1] = 224.0                                     # keeps the gates' block scale at 1/2; A has zeros there
        wc, ws = nvq.fp8_block_quantize_weight(w.cuda())
        codes, scales, gu = nvq.fp8_block_gated_linear(*nvq.fp8_block_quantize(a.cuda()), wc, ws, save=True)
        assert (gu[:, 1:128] == gate).all() and (gu[:, 128:] == 2.0 ** up).all()
        g = np.float64(gate)
        h = np.full((M, 128), ref.silu(g) * 2.0 ** up)
        if h[0, 0] >= 2.0 ** 128:                           # H is an FP32 number: infinite
            assert torch.isinf(scales).all() and nvq.device_status() == nvq.NVQ_STATUS_NONFINITE
            continue
        # 2^-100: the definition takes a block below it as zero
        e = 2 * sigmoid_error(g) * np.abs(h) + 2.0 ** -20 * np.abs(h) + abs(g) * cut(g) * 2.0 ** up + 2.0 ** -100
        inside(scales.double().cpu().numpy(), np.full((1, M), abs(h[0, 0]) / 448), e.max() / 448)
        inside(ref.value(codes, scales, "rows"), h, e4m3_step_bound(np.abs(h) + e, scales, "rows") + 2 * e)
    assert nvq.device_status() == 0


# (dH, gate, up): products that pass FP32's range where the results do not, gates far on either side
FAR = [(2.0 ** -20, 1.5 * 2.0 ** 127, 1.0), (1.0, 2.0 ** 110, 2.0 ** -30), (2.0 ** -3, 100.0, 2.0 ** 120), (1.0, -40.0, 2.0 ** 126),
       (2.0 ** 10, -40.0, 2.0 ** 126), (2.0 ** 100, -60.0, 2.0 ** 60), (2.0 ** 127, -85.0, 2.0 ** 100), (1.9921875 * 2.0 ** 127, 1.5, 0.25),
       (0.25, 1.5, 1.9921875 * 2.0 ** 126), (2.0 ** 100, -30.0, 2.0 ** -90), (2.0 ** -100, -30.0, 2.0 ** 120), (2.0 ** 90, -1.28125, 2.0 ** 38),
       (1.0, -100.0, 2.0 ** 100), (1.0, -2.0 ** 120, 2.0 ** 100), (2.0 ** 64, 0.0, 2.0 ** 63), (2.0 ** 120, -86.5, -2.0 ** 110)]


@pytest.mark.parametrize("dh,gate,up", FAR)
def test_gated_backward_at_the_ends_of_the_range(dh, gate, up):
    one = lambda v, n: torch.full((2, n), v, dtype=torch.bfloat16, device="cuda")      # noqa: E731
    got = nvq.fp8_block_gated_backward(one(dh, 128), torch.cat((one(gate, 128), one(up, 128)), 1))
    g = np.float64(gate)
    s = 0.5 * (1 + np.tanh(g / 2)) if g > -30 else np.exp(g)
    one_minus = np.exp(-g) if g > 30 else 1 - s
    want = np.array([dh * up * s * (1 + g * one_minus), dh * g * s, g * s * up])
    # as for ordinary inputs: the sigmoid's error, times what 1 + g (1 - s) makes of it (g (1 - s) is at most 0.3 above 1)
    se = sigmoid_error(min(abs(g), 90.0)) + 2.0 ** -21
    err = np.array([abs(dh * up) * s * (2 + 3 * min(abs(g), 90.0)) * se, abs(want[1]) * se, abs(want[2]) * se])
    err += cut(g) * (np.abs([dh * up, dh, up]) * (1 + abs(g))) + 2.0 ** -100
    status = 0
    for (codes, scales), which, kind in ((got[0], (0, 1), "rows"), (got[1], (0, 1), "columns"), (got[2], (2,), "columns")):
        for n, i in enumerate(which):
            sc = scales[n] if kind == "rows" else scales[0, 128 * n:128 * n + 128]
            if abs(want[i]) >= 2.0 ** 128:
                assert torch.isinf(sc).all()
                status = nvq.NVQ_STATUS_NONFINITE
                continue
            inside(sc.double().cpu().numpy(), np.float64(abs(want[i]) / 448), (err[i] + 2.0 ** -23 * abs(want[i])) / 448)
            v = ref.e4m3_value(codes[:, 128 * n:128 * n + 128].cpu().numpy()) * (sc.double().cpu().numpy()[:, None] if kind == "rows" else sc.double().cpu().numpy())
            inside(v, want[i], 2.0 ** -20 * abs(want[i]) + 2 * err[i])     # a block's largest magnitude has the code 448
    assert nvq.device_status() == status


@pytest.mark.parametrize("far", [60.0, 100.0, 2.0 ** 120, -2.0 ** 120])
def test_gated_backward_far_values_leave_the_others_alone(far):
    """One far gate, with an up whose product with it passes FP32: the rest of the tile, gates above 43 among it,
    keeps its bits."""
    g = torch.Generator().manual_seed(3)
    gu, dh = torch.randn(300, 512, generator=g).bfloat16(), torch.randn(300, 256, generator=g).bfloat16()
    gu[:, 40:44] = 50.0
    (rc, rs), (cc, cs), (hc, hs) = nvq.fp8_block_gated_backward(dh.cuda(), gu.cuda())
    gu[5, 17], gu[5, 256 + 17] = far, 2.0 ** 100
    (rc2, rs2), (cc2, cs2), (hc2, hs2) = nvq.fp8_block_gated_backward(dh.cuda(), gu.cuda())
    nvq.device_status()
    rows, cols = [r for r in range(300) if r != 5], [c for c in range(512) if c not in (17, 256 + 17)]
    assert torch.equal(rc[rows], rc2[rows]) and torch.equal(rs[:, rows], rs2[:, rows])
    assert torch.equal(rc[5, 128:256], rc2[5, 128:256]) and torch.equal(rc[5, 384:], rc2[5, 384:])
    assert torch.equal(cc[:, cols], cc2[:, cols]) and torch.equal(cs[:, cols], cs2[:, cols])
    assert torch.equal(cc[128:], cc2[128:]) and torch.equal(hc[128:], hc2[128:])
    assert torch.equal(hc[:, [c for c in range(256) if c != 17]], hc2[:, [c for c in range(256) if c != 17]])


def test_gated_backward_values_beside_a_far_one_keep_their_bits():
    """up times a gate of 20 passes FP32 for one value of many octets: its neighbours' gradients and H stay, to the bit."""
    g = torch.Generator().manual_seed(4)
    gu, dh = torch.randn(256, 512, generator=g).bfloat16(), torch.randn(256, 256, generator=g).bfloat16()
    gu[:, 9:256:16] = 20.0
    _, (cc, cs), (hc, hs) = nvq.fp8_block_gated_backward(dh.cuda(), gu.cuda())
    gu[:, 256 + 9::16] = 2.0 ** 126
    dh[:, 9::16] = 2.0 ** -60
    _, (cc2, cs2), (hc2, hs2) = nvq.fp8_block_gated_backward(dh.cuda(), gu.cuda())
    assert torch.isinf(hs2[:, 9::16]).all() and nvq.device_status() == nvq.NVQ_STATUS_NONFINITE
    rest = [c for c in range(256) if c % 16 != 9]
    assert torch.equal(hc[:, rest], hc2[:, rest]) and torch.equal(hs[:, rest], hs2[:, rest])
    rest += [256 + c for c in rest]
    assert torch.equal(cc[:, rest], cc2[:, rest]) and torch.equal(cs[:, rest], cs2[:, rest])


def test_gated_backward_far_values_of_many_tiles_per_block():
    """20,480 tiles, some 139 to a thread block: far values early, late and in a block's first, its 128th and its last
    tiles are done carefully, and a NaN stays where it is."""
    M, F = 2, 128 * 20480
    g = torch.Generator("cuda").manual_seed(5)
    gu, dh = (torch.randn(M, n, generator=g, device="cuda").bfloat16() for n in (2 * F, F))
    clean = nvq.fp8_block_gated_backward(dh, gu)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = [0, 7, sms - 1, sms, 127 * sms + 5, 128 * sms, 130 * sms + 9, 20479]
    cols = torch.tensor([128 * t + 3 for t in tiles], device="cuda")
    gu[:, cols], gu[:, F + cols], dh[:, cols] = -40.0, 2.0 ** 126, 1.0
    gu[1, F + 128 * 50 + 9] = float("nan")
    (rc, rs), (cc, cs), (hc, hs) = nvq.fp8_block_gated_backward(dh, gu)
    assert nvq.device_status() == nvq.NVQ_STATUS_NONFINITE
    want = abs(ref.silu(np.float64(-40.0)) * 2.0 ** 126)
    inside(hs[0, cols].double().cpu().numpy(), np.float64(want / 448), (want * sigmoid_error(np.float64(40.0)) + 2.0 ** -23 * want) / 448)
    bad = ~torch.isfinite(hs)
    assert bad[0, 128 * 50 + 9] and bad.sum() == 1
    bad = ~torch.isfinite(cs)
    assert bad[0, 128 * 50 + 9] and bad.sum() == 1
    bad = ~torch.isfinite(rs)
    assert bad[50, 1] and bad.sum() == 1
    same = torch.ones(F, dtype=torch.bool, device="cuda")
    same[cols], same[128 * 50 + 9] = False, False
    assert torch.equal(hs[:, same], clean[2][1][:, same]) and torch.equal(hc[:, same], clean[2][0][:, same])
    same = torch.cat((same, same))
    assert torch.equal(cs[:, same], clean[1][1][:, same]) and torch.equal(cc[:, same], clean[1][0][:, same])


def test_gated_backward_where_the_derivative_of_silu_vanishes():
    """dgate around gate = -1.28, dH = up = 1: its error is the sigmoid's, not magnified by a rounded 1 - sigmoid.
    sigma is within 1.5 FP32 steps (2^-23), so that 1 + g - g sigma is off by |g| sigma 1.5 2^-23; three more roundings.
    One row: the column scales are |dgate| / 448 to FP32 precision."""
    g = torch.arange(0xBF80, 0xBFD0, dtype=torch.int32).to(torch.uint16).view(torch.bfloat16)      # -1.0 to -1.6171875
    gu = torch.cat((torch.cat((g, g[:128 - len(g)]))[None], torch.ones(1, 128, dtype=torch.bfloat16)), 1)
    _, (_, cs), _ = nvq.fp8_block_gated_backward(torch.ones(1, 128, dtype=torch.bfloat16, device="cuda"), gu.cuda())
    G = gu[0, :128].double().numpy()
    s = 1 / (1 + np.exp(-G))
    f = s * (1 + G * (1 - s))
    inside(cs[0, :128].double().cpu().numpy() * 448, np.abs(f), s * np.abs(G) * s * 1.5 * 2.0 ** -23 + 4 * 2.0 ** -24 * np.abs(f))
