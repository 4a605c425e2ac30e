"""Plain 64-bit forms of the rotary, cross-attention and shared-prefix operators, and the
tolerances their tests derive from the arithmetic."""

import math

import torch

HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}

# fp32 work of a rotated element, relative to the magnitude of its pair: the norm's sum (13 steps of
# 2^-24, halved by the root) and its product (4 x 2^-24), the angle (half turns rounded to fp32 and
# the sine's own error: 2^-23 and 2^-22), two products and a sum (3 x 2^-24): below 2^-20.
ROPE_FP32 = 2.0 ** -20


def rope_rows(x, positions, table, interleaved, amplitude=1.0, weight=None, eps=1e-6):
    """(rotated rows, magnitudes of their pairs) of x [T, heads, D], both in 64 bits."""
    x = x.double().cpu()
    table = table.double().cpu()
    if weight is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double().cpu()
    rot = 2 * table.numel()
    turns = positions.double().cpu()[:, None] * table
    angle = 2 * math.pi * (turns - turns.round())
    c, s = torch.cos(angle)[:, None] * amplitude, torch.sin(angle)[:, None] * amplitude
    first = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    second = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    out, mag = x.clone(), x.abs()
    a, b = x[..., first], x[..., second]
    out[..., first], out[..., second] = a * c - b * s, b * c + a * s
    mag[..., first] = mag[..., second] = torch.hypot(a, b) * amplitude
    return out, mag


def assert_rope(got, want, mag, what=""):
    dt = got.dtype
    got = got.double().cpu()
    # one rounding to the type (2^-25: half a step among fp16's subnormals), and the fp32 work
    tol = 1.001 * HALF_STEP[dt] * want.abs() + ROPE_FP32 * mag + 2.0 ** -25
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {(got - want).abs().max():.3e}"


def attention(q, K, V, scale):
    """softmax(scale q K^T) V in 64 bits and the same with |V|: q [rows, H, D], K, V
    [tokens, Hkv, D]; zeros without tokens."""
    rows, H, D = q.shape
    if K.shape[0] == 0:
        z = torch.zeros((rows, H, D), dtype=torch.float64, device=q.device)
        return z, z
    G = H // K.shape[1]
    q, K, V = q.double(), K.double().repeat_interleave(G, 1), V.double().repeat_interleave(G, 1)
    w = torch.softmax(torch.einsum("rhd,thd->hrt", q, K) * scale, -1)
    return torch.einsum("hrt,thd->rhd", w, V), torch.einsum("hrt,thd->rhd", w, V.abs())


def tokens(cache, table, n):
    """The first n tokens that a block table (a list) names, [n, Hkv, D]."""
    _, Hkv, S, D = cache.shape
    if n == 0:
        return cache.new_zeros((0, Hkv, D))
    idx = torch.tensor(table[:-(-n // S)], dtype=torch.long, device=cache.device)
    return cache[idx].transpose(1, 2).reshape(-1, Hkv, D)[:n]


def assert_attention(got, want, absolute, dt, what=""):
    """got against want. Relative to sum w |V| (`absolute`): the weights' 16-bit terms (bf16 enters
    as value and residue, 2^-17; fp16 as one term, 2^-11), and the scores: 128 products of N(0, 1)
    pairs accumulated in fp32 are off by at most 128 x 2^-24 x 128 x E|qk| x scale ~ 5e-5 of a
    weight, twice that in the ratio, below 2^-13. Then the output's own rounding."""
    odt = got.dtype
    got = got.double()
    rel = (2.0 ** -17 if dt == torch.bfloat16 else 2.0 ** -11) + 2.0 ** -13
    tol = rel * absolute + 1.001 * HALF_STEP[odt] * want.abs() + 2.0 ** -25
    off = (got - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), \
        f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {(off / tol).max():.3g} x tolerance"
