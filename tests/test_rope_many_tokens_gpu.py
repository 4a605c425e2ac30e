"""The rotary kernel with several tokens per CTA (2, 4 and 8, from 8, 16 and 32 tokens per SM on),
the last CTA's fewer: every token against the 64-bit form, both layouts and the one for sizes that do
not divide, with and without norms, alone and into 16-bit and E4M3 caches, padding inside a CTA's tokens
and behind the last."""

import pytest
import torch

from paged_kv_cache_driven_b200 import binding
from reference64 import ROPE_FP32, assert_rope, rope_rows

pytestmark = pytest.mark.gpu
DEV = "cuda"
# tokens per SM, and tokens more than that: no multiple of a CTA's tokens
MANY = [(8, 1), (16, 3), (32, 65)]


def tokens_for(per_sm, more):
    return per_sm * torch.cuda.get_device_properties(0).multi_processor_count + more


def inputs(T, H, Hkv, D, dt, norm, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    qkv = torch.randn((T, H + 2 * Hkv, D), generator=g, device=DEV).to(dt)
    weights = [(1 + 0.3 * torch.randn(D, generator=g, device=DEV)).to(dt) if norm else None
               for _ in range(2)]
    # (no two tokens alike, so that a wrong token's angles show)
    pos = (torch.randperm(4 * T, generator=g, device=DEV)[:T] + 3).to(torch.int32)
    return qkv.split((H, Hkv, Hkv), 1), weights, pos


@pytest.mark.parametrize("norm", [False, True], ids=["plain", "normed"])
@pytest.mark.parametrize("D,rot,interleaved", [(128, 128, False), (64, 32, True), (80, 20, False),
                                               (256, 128, False), (96, 24, True)])
@pytest.mark.parametrize("per_sm,more", MANY)
def test_alone(per_sm, more, D, rot, interleaved, norm):
    T, H, Hkv = tokens_for(per_sm, more), 3, 2
    dt = torch.bfloat16 if norm else torch.float16
    (q, k, _), (qw, kw), pos = inputs(T, H, Hkv, D, dt, norm, per_sm + D)
    table = binding.pa_rope_table(rot)[0]
    qo, ko = torch.full_like(q, 7.0).contiguous(), torch.full_like(k, 7.0).contiguous()
    binding.pa_rope(qo, ko, q, k, pos, table.to(DEV), interleaved=interleaved, q_weight=qw,
                    k_weight=kw)
    torch.cuda.synchronize()
    assert binding.pa_get_device_error() == 0
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        assert_rope(got, *rope_rows(x, pos, table, interleaved, 1.0, w), f"{T} tokens")


@pytest.mark.parametrize("e4m3", [False, True], ids=["16bit", "e4m3"])
@pytest.mark.parametrize("D,rot,interleaved,norm", [(128, 128, False, True), (64, 64, True, False),
                                                    (80, 20, False, True), (128, 64, True, True)])
@pytest.mark.parametrize("per_sm,more", MANY)
def test_into_a_cache(per_sm, more, D, rot, interleaved, norm, e4m3):
    T, H, Hkv, S = tokens_for(per_sm, more), 2, 2, 16
    dt = torch.float16 if norm and not e4m3 else torch.bfloat16
    (q, k, v), (qw, kw), pos = inputs(T, H, Hkv, D, dt, norm, per_sm + D)
    table = binding.pa_rope_table(rot)[0]
    NB = -(-T // S) + 2
    g = torch.Generator(device=DEV).manual_seed(T)
    slots = torch.randperm(NB * S, generator=g, device=DEV)[:T]
    slots[5::7] = -1  # padding inside a CTA's tokens
    slots[-3:] = -1   # and behind the batch's last one
    shape = (2, NB, Hkv, S, D)
    cache = torch.randint(0, 120, shape, dtype=torch.uint8, device=DEV) if e4m3 else \
        torch.randn(shape, generator=g, device=DEV).to(dt)
    before = cache.clone()
    qo = torch.full_like(q, 7.0).contiguous()
    how = dict(interleaved=interleaved, q_weight=qw, k_weight=kw)
    ks, vs = 0.017, 0.02
    if e4m3:
        binding.pa_rope_append_fp8(qo, q, k, v, pos, slots, cache[0], cache[1], ks, vs,
                                   table.to(DEV), **how)
    else:
        binding.pa_rope_append(qo, q, k, v, pos, slots, cache[0], cache[1], table.to(DEV), **how)
    torch.cuda.synchronize()
    assert binding.pa_get_device_error() == 0
    assert_rope(qo, *rope_rows(q, pos, table, interleaved, 1.0, qw), f"q of {T} tokens")
    live = (slots >= 0).nonzero().flatten()
    at = slots[live]
    rows = [c.transpose(1, 2).reshape(NB * S, Hkv, D) for c in cache]
    want, mag = rope_rows(k[live], pos[live], table, interleaved, 1.0, kw)
    if e4m3:
        plain = before.clone()
        binding.pa_kv_append_fp8(k.contiguous(), v.contiguous(), slots, plain[0], plain[1], ks, vs)
        assert torch.equal(cache[1], plain[1])
        # the code nearest to value / scale (half a step: 2^-4 of it, 2^-10 among subnormals)
        y, m = (want / ks).clamp(-448, 448), mag / ks
        got = rows[0][at].view(torch.float8_e4m3fn).double().cpu()
        tol = 2.0 ** -4 * y.abs() + 2.0 ** -10 + 2 * ROPE_FP32 * m
        assert bool(((got - y).abs() <= tol).all())
    else:
        assert_rope(rows[0][at], want, mag, f"k of {T} tokens")
        assert torch.equal(rows[1][at], v[live])
    keep = torch.ones(NB * S, dtype=torch.bool, device=DEV)
    keep[at] = False
    for r, b in zip(rows, before):
        assert torch.equal(r[keep], b.transpose(1, 2).reshape(NB * S, Hkv, D)[keep])


def test_append_with_q_in_place():
    """q rotated where it lies in the fused projection while k and v go to the cache."""
    T, H, Hkv, D, S = 75, 6, 2, 128, 16
    (q, k, v), (qw, kw), pos = inputs(T, H, Hkv, D, torch.bfloat16, True, 1)
    table = binding.pa_rope_table(D)[0].to(DEV)
    slots = torch.arange(T, device=DEV)
    cache = torch.zeros((4, 5, Hkv, S, D), dtype=torch.bfloat16, device=DEV)
    want = torch.empty_like(q).contiguous()
    how = dict(q_weight=qw, k_weight=kw)
    binding.pa_rope_append(want, q, k, v, pos, slots, cache[0], cache[1], table, **how)
    k0, v0 = k.clone(), v.clone()
    binding.pa_rope_append(q, q, k, v, pos, slots, cache[2], cache[3], table, **how)
    assert torch.equal(q, want) and torch.equal(k, k0) and torch.equal(v, v0)
    assert torch.equal(cache[:2], cache[2:]) and binding.pa_get_device_error() == 0
