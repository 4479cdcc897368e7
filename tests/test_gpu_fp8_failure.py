"""Waits of the FP8 block-scaled products that run out, without a fault.

nvq_set_wait_limit shortens the bounded waits between a kernel's roles, so that
some of them give up in the middle of a product.  Every call has to return and
leave the context usable: the status word says what happened, and the next call,
at the default limit, gives the bits that it gave before.
"""
import time

import pytest
import torch

import microscaling_quantized_linear_b200 as nvq

pytestmark = pytest.mark.gpu


def quantized(kind, rows, cols, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda").bfloat16()
    return {"rows": nvq.fp8_block_quantize, "columns": nvq.fp8_block_quantize_columns,
            "tiles": nvq.fp8_block_quantize_weight}[kind](x)


def linear(M, N, K):
    a, w = quantized("rows", M, K, 1), quantized("tiles", N, K, 2)
    return lambda: [nvq.fp8_block_linear(*a, *w)]


def dgrad(M, N, K):
    dy, w = quantized("rows", M, N, 1), quantized("tiles", N, K, 2)
    return lambda: [nvq.fp8_block_linear_dgrad(*dy, *w)]


def wgrad(M, N, K):
    dy, x = quantized("columns", M, N, 1), quantized("columns", M, K, 2)
    return lambda: [nvq.fp8_block_linear_wgrad(*dy, *x)]


def gated(M, F, K):
    a, w = quantized("rows", M, K, 1), quantized("tiles", 2 * F, K, 2)
    return lambda: list(nvq.fp8_block_gated_linear(*a, *w, save=True))


# few tokens (clusters that split the contracted axis); CTA pairs with a tile's loads all issued at once
# (four blocks) and with more blocks than stages; loads without a tensor map (N = 8 mod 16)
CALLS = [(linear, 8, 4096, 4096), (linear, 48, 4096, 4096), (dgrad, 8, 4096, 4096), (gated, 3, 4096, 4096),
         (linear, 2000, 4096, 512), (linear, 1000, 4096, 4096), (dgrad, 1000, 512, 4096), (dgrad, 1000, 4096, 2048),
         (dgrad, 700, 2056, 1552), (gated, 700, 1024, 512), (gated, 2000, 4096, 512), (gated, 1111, 1408, 2048), (wgrad, 512, 4096, 2048), (wgrad, 2048, 1024, 2048), (wgrad, 1111, 2056, 1552)]


def limited(call, limit_ns):
    """The status of a call whose waits are limited; its outputs are unspecified if one ran out."""
    nvq.set_wait_limit(limit_ns)
    try:
        call()
        return nvq.device_status()
    finally:
        nvq.set_wait_limit(0)


def same_bits(xs, ys):
    return all(torch.equal(x, y) for x, y in zip(xs, ys))


@pytest.mark.parametrize("make,M,N,K", CALLS, ids=lambda v: v.__name__ if callable(v) else str(v))
def test_products_return_when_their_waits_run_out(make, M, N, K):
    call = make(M, N, K)
    want = call()
    assert nvq.device_status() == 0
    for limit_ns in (1, 2000):
        assert limited(call, limit_ns) in (0, nvq.NVQ_STATUS_TIMEOUT)
        assert same_bits(call(), want) and nvq.device_status() == 0


@pytest.mark.parametrize("make,M,N,K", [(linear, 2000, 4096, 512), (linear, 1000, 4096, 4096), (dgrad, 700, 2056, 1552),
                                        (gated, 2000, 4096, 512), (wgrad, 1111, 2056, 1552)], ids=lambda v: v.__name__ if callable(v) else str(v))
def test_a_product_that_gives_up_returns_soon(make, M, N, K):
    """No CTA of a pair drains its loads for seconds after the other gave up: 10 ms for each of at most six
    stages is far from the 4 s that one of them would take."""
    call = make(M, N, K)
    want = call()
    torch.cuda.synchronize()
    for limit_ns in (1, 500, 1000, 2000, 4000):
        start = time.monotonic()
        limited(call, limit_ns)
        assert time.monotonic() - start < 1.0
    assert same_bits(call(), want) and nvq.device_status() == 0


@pytest.mark.parametrize("make,M,N,K", CALLS, ids=lambda v: v.__name__ if callable(v) else str(v))
def test_a_wait_of_one_nanosecond_runs_out_and_is_reported(make, M, N, K):
    """The first wait for operands from memory takes longer than that in every kernel."""
    call = make(M, N, K)
    want = call()
    assert nvq.device_status() == 0
    assert limited(call, 1) == nvq.NVQ_STATUS_TIMEOUT
    assert nvq.device_status() == 0                        # read clears it
    assert same_bits(call(), want) and nvq.device_status() == 0


@pytest.mark.parametrize("M,F,K", [(300, 256, 1024), (2000, 4096, 512), (600, 1408, 4096)])
def test_gated_warps_that_share_a_row_leave_together(M, F, K):
    """The two warps of a row's block meet at a barrier and wait for different accumulators before it: limits
    around the time of a stage make one give up where the other does not, at tiles early and late."""
    call = gated(M, F, K)
    want = call()
    seen = set()
    for limit_ns in (200, 500, 800, 1200, 1600, 2400, 3200, 5000):
        for _ in range(3):
            seen.add(limited(call, limit_ns))
    assert nvq.NVQ_STATUS_TIMEOUT in seen and seen <= {0, nvq.NVQ_STATUS_TIMEOUT}
    assert same_bits(call(), want) and nvq.device_status() == 0
