"""Host-side checks of the FP8 block-scaled entry points (no GPU): the C ABI
refuses bad arguments before it touches the device, and the binding refuses
tensors of a wrong type, shape or place before the library sees a pointer."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_reference as ref
import microscaling_quantized_linear_b200 as nvq

L = nvq._lib
NULL = None
P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
SHAPE, NUL, ALIGN = -2, -1, -3


def test_scale_counts_and_shapes():
    for kind, code in (("rows", 0), ("columns", 1), ("tiles", 2)):
        for r, c in ((1, 16), (128, 128), (129, 272), (300, 64)):
            s = nvq.fp8_block_scale_shape(kind, r, c)
            assert L.fp8_block_scales(code, r, c) == s[0] * s[1]
    assert L.fp8_block_scales(3, 128, 128) == 0 and L.fp8_block_scales(0, 0, 128) == 0
    with pytest.raises(ValueError):
        nvq.fp8_block_scale_shape("blocks", 1, 1)


def q(x=P, M=4, K=64, ld=64, rc=P, rs=P, cc=P, cs=P):
    return L.fp8_block_quantize(x, M, K, ld, rc, rs, cc, cs, NULL)


def test_quantize_refusals():
    assert q(K=20, ld=24) == SHAPE                    # K not a multiple of 8
    assert q(ld=56) == SHAPE and q(ld=68) == SHAPE    # pitch short, not a multiple of 8
    assert q(M=-1) == SHAPE and q(K=0, ld=0) == SHAPE
    assert q(M=1 << 20, K=1 << 12, ld=1 << 12) == SHAPE
    assert q(M=0, x=NULL) == 0
    assert q(x=NULL) == NUL and q(rs=NULL) == NUL and q(cc=NULL) == NUL
    assert q(rc=NULL, rs=NULL, cc=NULL, cs=NULL) == NUL
    assert q(x=ODD) == ALIGN and q(cs=ODD) == ALIGN and q(rc=ODD) == ALIGN
    w = lambda x=P, N=4, K=64, ld=64, c=P, s=P: L.fp8_block_quantize_weight(x, N, K, ld, c, s, NULL)      # noqa: E731
    assert w(K=36, ld=40) == SHAPE and w(c=NULL) == NUL and w(s=ODD) == ALIGN and w(N=0) == 0


def lin(a=P, sa=P, w=P, sw=P, bias=NULL, out=P, ldo=64, M=4, N=64, K=128):
    return L.fp8_block_linear(a, sa, w, sw, bias, out, ldo, M, N, K, NULL)


def test_linear_refusals():
    assert lin(N=60) == SHAPE and lin(N=0) == SHAPE and lin(N=-8) == SHAPE
    assert lin(K=120) == SHAPE and lin(ldo=56) == SHAPE and lin(ldo=66) == SHAPE and lin(M=-1) == SHAPE
    assert lin(N=1 << 20, K=1 << 12, ldo=1 << 20) == SHAPE
    assert lin(M=0, a=NULL, sa=NULL, out=NULL) == 0
    for k in ("a", "sa", "w", "sw", "out"):
        assert lin(**{k: NULL}) == NUL and lin(**{k: ODD}) == ALIGN
    assert lin(bias=ctypes.c_void_p(0x10001)) == ALIGN
    d = lambda M=4, N=64, K=64, ld=64, dy=P, out=P: L.fp8_block_linear_dgrad(dy, P, P, P, out, ld, M, N, K, NULL)     # noqa: E731
    assert d(N=68) == SHAPE and d(K=72, ld=72) == SHAPE and d(ld=60) == SHAPE and d(dy=NULL) == NUL and d(out=ODD) == ALIGN
    assert d(M=0, dy=NULL) == 0
    g = lambda M=4, N=64, K=64, ld=64, dy=P, out=P: L.fp8_block_linear_wgrad(dy, P, P, P, out, ld, 0, M, N, K, NULL)  # noqa: E731
    assert g(N=68) == SHAPE and g(K=72, ld=72) == SHAPE and g(ld=62) == SHAPE and g(dy=NULL) == NUL and g(out=ODD) == ALIGN
    assert g(M=0, out=NULL) == NUL


def test_gated_refusals():
    f = lambda M=4, F=128, K=64, ld=256, a=P, gu=P, h=P: L.fp8_block_gated_linear(a, P, P, P, h, P, gu, ld, M, F, K, NULL)  # noqa: E731
    assert f(F=64) == SHAPE and f(F=0) == SHAPE and f(K=72) == SHAPE and f(ld=128) == SHAPE and f(ld=260) == SHAPE
    assert f(a=NULL) == NUL and f(h=NULL) == NUL and f(gu=ODD) == ALIGN and f(M=0, a=NULL) == 0
    b = lambda M=4, F=128, ldh=128, ldg=256, dh=P, gu=P, rc=P: L.fp8_block_gated_backward(                          # noqa: E731
        dh, ldh, gu, ldg, rc, P, P, P, P, P, M, F, NULL)
    assert b(F=64) == SHAPE and b(ldh=120) == SHAPE and b(ldg=128) == SHAPE and b(ldh=132) == SHAPE
    assert b(dh=NULL) == NUL and b(rc=NULL) == NUL and b(gu=ODD) == ALIGN and b(M=0, dh=NULL) == 0


def codes(r, c):
    return torch.zeros(r, c, dtype=torch.uint8)


def scales(kind, r, c):
    return torch.zeros(nvq.fp8_block_scale_shape(kind, r, c))


def test_binding_refuses_before_the_library():
    bf = torch.zeros(4, 64, dtype=torch.bfloat16)
    for bad, msg in ((bf.float(), "bfloat16"), (bf.t(), "unit column stride"), (bf[0], "unit column stride")):
        for fn in (nvq.fp8_block_quantize, nvq.fp8_block_quantize_columns, nvq.fp8_block_quantize_both, nvq.fp8_block_quantize_weight):
            with pytest.raises(ValueError, match=msg):
                fn(bad)
    with pytest.raises(ValueError, match="CUDA tensor"):
        nvq.fp8_block_quantize(bf)
    with pytest.raises(ValueError, match="codes"):
        nvq.fp8_block_quantize(bf, codes=codes(4, 32))
    with pytest.raises(ValueError, match="scales"):
        nvq.fp8_block_quantize(bf, scales=torch.zeros(2, 4))
    a, w = (codes(4, 256), scales("rows", 4, 256)), (codes(64, 256), scales("tiles", 64, 256))
    ok = lambda: nvq.fp8_block_linear(*a, *w)                 # noqa: E731
    with pytest.raises(ValueError, match="CUDA tensor"):
        ok()
    for args in ((a[0].float(), a[1], *w), (a[0], a[1].t(), *w), (a[0], a[1], codes(64, 128), w[1]),
                 (a[0].t(), a[1], *w), (a[0], a[1].double(), *w), (a[0], a[1], w[0], torch.zeros(2, 2))):
        with pytest.raises(ValueError, match="expected|columns"):
            nvq.fp8_block_linear(*args)
    with pytest.raises(ValueError, match="columns"):
        nvq.fp8_block_linear(codes(4, 128), scales("rows", 4, 128), *w)
    with pytest.raises(ValueError, match="bias"):
        nvq.fp8_block_linear(*a, *w, bias=torch.zeros(32, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="out"):
        nvq.fp8_block_linear(*a, *w, out=torch.zeros(4, 32, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="rows"):
        nvq.fp8_block_linear_dgrad(*a, *w)
    c1, c2 = (codes(4, 64), scales("columns", 4, 64)), (codes(5, 32), scales("columns", 5, 32))
    with pytest.raises(ValueError, match="rows"):
        nvq.fp8_block_linear_wgrad(*c1, *c2)
    with pytest.raises(ValueError, match="accumulate"):
        nvq.fp8_block_linear_wgrad(*c1, *c1, accumulate=True)
    with pytest.raises(ValueError, match="multiple of 128"):
        nvq.fp8_block_gated_linear(*a, *w)
    with pytest.raises(ValueError, match="gate_up"):
        nvq.fp8_block_gated_backward(torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(4, 128, dtype=torch.bfloat16))


def test_layers_refuse_weights_that_no_call_could_take():
    w = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)     # noqa: E731
    for shape in ((12, 32), (16, 40)):
        with pytest.raises(ValueError, match="weight"):
            nvq.BlockFp8Linear(w(*shape))
    with pytest.raises(ValueError, match="bias"):
        nvq.BlockFp8Linear(w(16, 32), torch.zeros(16))
    for gate_up, down in (((256, 40), (16, 128)), ((256, 32), (12, 128)), ((128, 32), (16, 64)), ((256, 32), (16, 256))):
        with pytest.raises(ValueError, match="w_gate_up"):
            nvq.BlockFp8GatedFF(w(*gate_up), w(*down))


def test_reference_codes_agree_with_torch():
    """The tests' own E4M3 rounding against torch's cast, every code and ties."""
    v = ref.e4m3_value(np.arange(256)).astype(np.float32)
    f = np.isfinite(v)
    np.testing.assert_array_equal(ref.e4m3_code(v[f]), np.arange(256, dtype=np.uint8)[f])
    x = np.concatenate((np.sort(v[f]), (np.sort(v[f])[1:] + np.sort(v[f])[:-1]) / 2,
                        np.random.default_rng(0).standard_normal(5000).astype(np.float32) * 40))
    t = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(ref.e4m3_code(x), t)


def test_package_imports_with_a_torch_built_without_cuda():
    """torch's private CUDA functions are not there then; the package has to load and to refuse CPU tensors."""
    import os
    import subprocess
    import sys
    code = ("import torch\n"
            "for n in ('_cuda_getDevice', '_cuda_getCurrentRawStream'):\n"
            "    delattr(torch._C, n)\n"
            "import microscaling_quantized_linear_b200 as nvq\n"
            "assert nvq.fp8_block_scale_shape('rows', 3, 200) == (2, 3)\n"
            "try:\n"
            "    nvq.fp8_block_quantize(torch.zeros(4, 64, dtype=torch.bfloat16))\n"
            "except ValueError as e:\n"
            "    assert 'CUDA tensor' in str(e)\n"
            "    print('refused')\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "refused" in out.stdout, out.stdout + out.stderr
