"""The FP8 block-scaled operators as measured cases.

Codes are E4M3 (float8_e4m3fn).  Their FP32 scales cover blocks of 128:
  rows     one scale per 1 x 128 block along a row:    [ceil(C / 128), R] for an [R, C] matrix
  columns  one scale per 128 x 1 block along a column: [ceil(R / 128), C]
  tiles    one scale per 128 x 128 block (weights):    [ceil(R / 128), ceil(C / 128)]
Blocks at the end of a ragged matrix are short.  For a block with largest
magnitude b the scale is b / 448 and a code is E4M3(x * (448 / b)), to nearest
even; blocks with b < 2^-100 get the scale 0 and codes 0.

Operators:
  quantize        BF16 -> row-wise and (for training) column-wise codes and scales, or a weight's tile-wise ones
  linear          out[M, N] = A[M, K] . W[N, K]^T + bias, BF16
  linear_backward dX[M, K] = dY . W (BF16) and dW[N, K] = dY^T . X (FP32), from row-wise and column-wise codes
  gated           H = SiLU(A . Wg^T) * (A . Wu^T), quantized row-wise; training also keeps gate and up in BF16
  gated_backward  the gradients of gate and up, and H again, quantized as the following products read them
"""
import math

import torch

own = False

_NAMES = ("quantize", "linear", "linear_backward", "gated", "gated_backward")


def _lib():
    import microscaling_quantized_linear_b200 as nvq

    return nvq


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token's activation before a projection: the smallest call, all latency
        {"name": "quantize token", "op": "quantize", "M": 1, "K": 4096, "kind": "rows"},
        # a training step's activation: 1024 x 1024 image and text tokens by the feed-forward width, both orientations
        {"name": "quantize training", "op": "quantize", "M": 4608, "K": 12288, "kind": "both"},
        # a weight after an optimizer step, ragged in both directions
        {"name": "quantize weight", "op": "quantize", "M": 9224, "K": 4112, "kind": "weight"},
        # a single token through a square projection: streams the weight once
        {"name": "linear token", "op": "linear", "M": 1, "N": 4096, "K": 4096, "bias": False},
        # a few sequences decoding together, odd sizes, with a bias
        {"name": "linear batch", "op": "linear", "M": 29, "N": 9224, "K": 4112, "bias": True},
        # one image's tokens through the feed-forward's first projection
        {"name": "linear prompt", "op": "linear", "M": 4608, "N": 12288, "K": 4096, "bias": True},
        # a ragged batch of a small model in training
        {"name": "backward ragged", "op": "linear_backward", "M": 1111, "N": 2056, "K": 1552},
        # the feed-forward's second projection in training
        {"name": "backward training", "op": "linear_backward", "M": 4608, "N": 4096, "K": 12288},
        # a single token through a gated feed-forward block's first half
        {"name": "gated token", "op": "gated", "M": 1, "F": 12288, "K": 4096, "save": False},
        # one image's tokens in training: gate and up are kept
        {"name": "gated training", "op": "gated", "M": 4608, "F": 12288, "K": 4096, "save": True},
        # the same block's backward pass between its products, on a ragged batch of a small model
        {"name": "gated backward ragged", "op": "gated_backward", "M": 611, "F": 1408},
        # and at full size
        {"name": "gated backward training", "op": "gated_backward", "M": 4608, "F": 12288},
    ]


def _between(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(_NAMES)
    if op == "quantize":
        return {"op": op, "M": _between(rng, 1, 4608), "K": _between(rng, 64, 12288, 16),
                "kind": rng.choice(["rows", "both", "weight"])}
    if op == "linear":
        # token counts from decoding to prompts
        return {"op": op, "M": _between(rng, 1, 4608), "N": _between(rng, 256, 12288, 8), "K": _between(rng, 128, 4096, 16),
                "bias": rng.random() < 0.5}
    if op == "linear_backward":
        return {"op": op, "M": _between(rng, 64, 4608), "N": _between(rng, 256, 4096, 16), "K": _between(rng, 256, 12288, 16)}
    if op == "gated":
        return {"op": op, "M": _between(rng, 1, 4608), "F": _between(rng, 256, 12288, 128), "K": _between(rng, 128, 4096, 16),
                "save": rng.random() < 0.5}
    return {"op": op, "M": _between(rng, 1, 4608), "F": _between(rng, 256, 12288, 128)}


# ------------------------------------------------------------------ plain forms

def _blocks(x):
    """[R, C] FP32 -> [R, ceil(C / 128), 128], zeros past the end."""
    r, c = x.shape
    return torch.nn.functional.pad(x, (0, -c % 128)).view(r, (c + 127) // 128, 128)


def _scales(amax):
    """(scale, factor) of blocks by their largest magnitude."""
    zero = amax < 2.0 ** -100
    one = torch.ones_like(amax)
    return (torch.where(zero, torch.zeros_like(amax), amax / 448.0),
            torch.where(zero, torch.zeros_like(amax), 448.0 / torch.where(zero, one, amax)))


def _e4m3(v):
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _quantize_rows(x):
    """FP32 [R, C] -> codes [R, C], scales [ceil(C / 128), R]."""
    b = _blocks(x)
    s, f = _scales(b.abs().amax(2))
    return _e4m3((b * f[:, :, None]).reshape(x.shape[0], -1)[:, :x.shape[1]]).contiguous(), s.t().contiguous()


def _quantize_columns(x):
    """FP32 [R, C] -> codes [R, C], scales [ceil(R / 128), C]."""
    r, c = x.shape
    b = torch.nn.functional.pad(x, (0, 0, 0, -r % 128)).view((r + 127) // 128, 128, c)
    s, f = _scales(b.abs().amax(1))
    return _e4m3((b * f[:, None, :]).reshape(-1, c)[:r]).contiguous(), s


def _quantize_tiles(x):
    """FP32 [R, C] -> codes [R, C], scales [ceil(R / 128), ceil(C / 128)]."""
    r, c = x.shape
    b = torch.nn.functional.pad(x, (0, -c % 128, 0, -r % 128)).view((r + 127) // 128, 128, (c + 127) // 128, 128)
    s, f = _scales(b.abs().amax((1, 3)))
    return _e4m3((b * f[:, None, :, None]).reshape(b.shape[0] * 128, -1)[:r, :c]).contiguous(), s


def _rows_value(codes, scales):
    """FP32 values of row-wise codes."""
    return codes.view(torch.float8_e4m3fn).float() * scales.t().repeat_interleave(128, 1)[:, :codes.shape[1]]


def _columns_value(codes, scales):
    return codes.view(torch.float8_e4m3fn).float() * scales.repeat_interleave(128, 0)[:codes.shape[0]]


def _tiles_value(codes, scales):
    r, c = codes.shape
    return codes.view(torch.float8_e4m3fn).float() * scales.repeat_interleave(128, 0)[:r].repeat_interleave(128, 1)[:, :c]


def _plain(s):
    op = s["op"]
    if op == "quantize":
        x = s["x"].float()
        if s["kind"] == "weight":
            return _quantize_tiles(x)
        return _quantize_rows(x) if s["kind"] == "rows" else (*_quantize_rows(x), *_quantize_columns(x))
    if op == "linear":
        y = _rows_value(*s["a"]) @ _tiles_value(*s["w"]).t()
        return (y if s["bias"] is None else y + s["bias"].float()).bfloat16()
    if op == "linear_backward":
        dx = _rows_value(*s["dy_rows"]) @ _tiles_value(*s["w"])
        dw = _columns_value(*s["dy_columns"]).t() @ _columns_value(*s["x_columns"])
        return {"dx": dx.bfloat16(), "dw": dw}
    if op == "gated":
        gu = _rows_value(*s["a"]) @ _tiles_value(*s["w"]).t()
        gate, up = gu.chunk(2, 1)
        codes, scales = _quantize_rows(gate / (1 + torch.exp(-gate)) * up)
        return {"codes": codes, "scales": scales, "gate_up": gu.bfloat16() if s["save"] else None}
    gate, up = s["gate_up"].float().chunk(2, 1)
    dh = s["dh"].float()
    sig = 1 / (1 + torch.exp(-gate))
    d = torch.cat((dh * up * (sig * (1 + gate * (1 - sig))), dh * (gate * sig)), 1)
    return {"rows": _quantize_rows(d), "columns": _quantize_columns(d), "h_columns": _quantize_columns(gate * sig * up)}


# ------------------------------------------------------------------ the framework's operators

def _e4(codes):
    """E4M3 bytes as the values they stand for."""
    return codes.view(torch.float8_e4m3fn)


def _own(s):
    nvq = _lib()
    op = s["op"]
    if op == "quantize":
        if s["kind"] == "weight":
            codes, scales = nvq.fp8_block_quantize_weight(s["x"])
            return _e4(codes), scales
        if s["kind"] == "rows":
            codes, scales = nvq.fp8_block_quantize(s["x"])
            return _e4(codes), scales
        rc, rs, cc, cs = nvq.fp8_block_quantize_both(s["x"])
        return _e4(rc), rs, _e4(cc), cs
    if op == "linear":
        return nvq.fp8_block_linear(*s["a"], *s["w"], bias=s["bias"])
    if op == "linear_backward":
        return {"dx": nvq.fp8_block_linear_dgrad(*s["dy_rows"], *s["w"]),
                "dw": nvq.fp8_block_linear_wgrad(*s["dy_columns"], *s["x_columns"])}
    if op == "gated":
        codes, scales, gate_up = nvq.fp8_block_gated_linear(*s["a"], *s["w"], save=s["save"])
        return {"codes": _e4(codes), "scales": scales, "gate_up": gate_up}
    (rc, rs), (cc, cs), (hc, hs) = nvq.fp8_block_gated_backward(s["dh"], s["gate_up"])
    return {"rows": (_e4(rc), rs), "columns": (_e4(cc), cs), "h_columns": (_e4(hc), hs)}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ inputs

def _normal(g, rows, cols):
    return torch.randn(rows, cols, generator=g, device="cuda")


def _activation(g, rows, cols):
    """BF16 [rows, cols]: channels of different size, a few outliers, and padded rows that are zero."""
    x = _normal(g, rows, cols) * torch.exp(0.5 * _normal(g, 1, cols))
    x = torch.where(torch.rand(rows, cols, generator=g, device="cuda") < 0.001, 30 * x, x)
    if rows >= 64:
        x[rows - rows // 64:] = 0
    return x.bfloat16()


def _weight(g, rows, cols, std=0.02):
    return (std * _normal(g, rows, cols)).bfloat16()


def _bytes(codes, scales):
    return codes.view(torch.uint8), scales


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    op, M = case["op"], case["M"]
    s = {"op": op}
    if op == "quantize":
        s["kind"] = case["kind"]
        s["x"] = _weight(g, M, case["K"]) if case["kind"] == "weight" else _activation(g, M, case["K"])
    elif op == "linear":
        s["a"] = _bytes(*_quantize_rows(_activation(g, M, case["K"]).float()))
        s["w"] = _bytes(*_quantize_tiles(_weight(g, case["N"], case["K"]).float()))
        s["bias"] = (0.1 * _normal(g, 1, case["N"])[0]).bfloat16() if case["bias"] else None
    elif op == "linear_backward":
        dy = (1e-3 * _activation(g, M, case["N"]).float()).bfloat16().float()
        s["dy_rows"], s["dy_columns"] = _bytes(*_quantize_rows(dy)), _bytes(*_quantize_columns(dy))
        s["x_columns"] = _bytes(*_quantize_columns(_activation(g, M, case["K"]).float()))
        s["w"] = _bytes(*_quantize_tiles(_weight(g, case["N"], case["K"]).float()))
    elif op == "gated":
        s["save"] = case["save"]
        s["a"] = _bytes(*_quantize_rows(_activation(g, M, case["K"]).float()))
        s["w"] = _bytes(*_quantize_tiles(_weight(g, 2 * case["F"], case["K"]).float()))
    else:
        s["gate_up"] = (1.5 * _normal(g, M, 2 * case["F"])).bfloat16()
        s["dh"] = (1e-3 * _activation(g, M, case["F"]).float()).bfloat16()
    return s


# ------------------------------------------------------------------ what a pass cannot do without

def _up(n):
    return (n + 127) // 128


def work(case):
    op, M = case["op"], case["M"]
    if op == "quantize":
        K = case["K"]
        sides = {"rows": M * K + 4 * M * _up(K), "weight": M * K + 4 * _up(M) * _up(K),
                 "both": 2 * M * K + 4 * (M * _up(K) + K * _up(M))}
        return {"bytes": 2 * M * K + sides[case["kind"]], "flops": 2 * M * K}
    if op == "linear":
        N, K = case["N"], case["K"]
        return {"bytes": M * K + 4 * M * _up(K) + N * K + 4 * _up(N) * _up(K) + 2 * M * N + (2 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    if op == "linear_backward":
        N, K = case["N"], case["K"]
        dx = M * N + 4 * M * _up(N) + N * K + 4 * _up(N) * _up(K) + 2 * M * K
        dw = M * (N + K) + 4 * _up(M) * (N + K) + 4 * N * K
        return {"bytes": dx + dw, "flops": 4 * M * N * K}
    if op == "gated":
        F, K = case["F"], case["K"]
        return {"bytes": M * K + 4 * M * _up(K) + 2 * F * K + 8 * _up(F) * _up(K) + M * F + 4 * M * _up(F) + (4 * M * F if case["save"] else 0),
                "flops": 4 * M * F * K}
    F = case["F"]
    return {"bytes": 6 * M * F + 5 * M * F + 4 * (2 * M * _up(F) + 3 * F * _up(M)), "flops": 20 * M * F}


# ------------------------------------------------------------------ from the definition, in 64 bits

def _x_round(v):
    """Nearest E4M3 value, ties to even: 3 bits below the leading one, steps of 2^-9 below 2^-6."""
    _, e = torch.frexp(v)
    step = torch.exp2((e.double() - 4).clamp(min=-9.0))
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _x_quantize(x, rows, cols):
    """Codes' values and scales [row block, column block] of FP64 x in blocks of rows x cols."""
    r, c = x.shape
    nr, nc = -(-r // rows), -(-c // cols)
    big = x.new_zeros(nr * rows, nc * cols)
    big[:r, :c] = x
    big = big.view(nr, rows, nc, cols)
    amax = big.abs().amax((1, 3))
    live = amax >= 2.0 ** -100
    mul = torch.where(live, 448.0 / torch.where(live, amax, 1.0), 0.0)
    q = _x_round(big * mul[:, None, :, None]).view(nr * rows, nc * cols)[:r, :c]
    return q, torch.where(live, amax / 448.0, 0.0)


def _x_value(codes, scales, rows, cols):
    """FP64 values of codes whose scales are [row block, column block]."""
    r, c = codes.shape
    ri = torch.arange(r, device=codes.device) // rows
    ci = torch.arange(c, device=codes.device) // cols
    return codes.view(torch.float8_e4m3fn).double() * scales.double()[ri][:, ci]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["x"].double()
        if s["kind"] == "weight":
            return _x_quantize(x, 128, 128)
        codes, scales = _x_quantize(x, 1, 128)
        if s["kind"] == "rows":
            return codes, scales.t()
        return (codes, scales.t(), *_x_quantize(x, 128, 1))
    if op == "linear":
        y = _x_value(s["a"][0], s["a"][1].t(), 1, 128) @ _x_value(*s["w"], 128, 128).t()
        return y if s["bias"] is None else y + s["bias"].double()
    if op == "linear_backward":
        dy = _x_value(s["dy_rows"][0], s["dy_rows"][1].t(), 1, 128)
        return {"dx": dy @ _x_value(*s["w"], 128, 128),
                "dw": _x_value(*s["dy_columns"], 128, 1).t() @ _x_value(*s["x_columns"], 128, 1)}
    if op == "gated":
        F = case["F"]
        gu = _x_value(s["a"][0], s["a"][1].t(), 1, 128) @ _x_value(*s["w"], 128, 128).t()
        codes, scales = _x_quantize(gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:], 1, 128)
        return {"codes": codes, "scales": scales.t(), "gate_up": gu if case["save"] else None}
    F = case["F"]
    gate, up, dh = s["gate_up"][:, :F].double(), s["gate_up"][:, F:].double(), s["dh"].double()
    sig = torch.sigmoid(gate)
    silu = gate * sig
    d = torch.cat((dh * up * (sig + silu * torch.sigmoid(-gate)), dh * silu), 1)
    rows = _x_quantize(d, 1, 128)
    return {"rows": (rows[0], rows[1].t()), "columns": _x_quantize(d, 128, 1), "h_columns": _x_quantize(silu * up, 128, 1)}
