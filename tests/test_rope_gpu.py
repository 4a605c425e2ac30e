"""Rotary positions with per-head norms, alone (pa_rope) and on the way into the paged cache
(pa_rope_append, pa_rope_append_fp8), against a plain 64-bit form."""

import pytest
import torch

from paged_kv_cache_driven_b200 import binding
from reference64 import ROPE_FP32, assert_rope, rope_rows

pytestmark = pytest.mark.gpu
DEV = "cuda"
FAR = 2 ** 31 - 1


def inputs(T, H, Hkv, D, dt, seed=0, norm=True, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    qkv = (scale * torch.randn((T, H + 2 * Hkv, D), generator=g, device=DEV)).to(dt)
    q, k, v = qkv.split((H, Hkv, Hkv), 1)
    weights = [(1 + 0.3 * torch.randn(D, generator=g, device=DEV)).to(dt) if norm else None
               for _ in range(2)]
    return q, k, v, weights


def run(T, H, Hkv, D, rot, dt, interleaved=False, norm=True, positions=None, seed=0, amplitude=1.0,
        scale=1.0):
    q, k, v, (qw, kw) = inputs(T, H, Hkv, D, dt, seed, norm, scale)
    table, _ = binding.pa_rope_table(rot)
    if positions is None:
        positions = torch.arange(5, 5 + T)
    pos = positions.to(torch.int32).to(DEV)
    qo, ko = torch.full_like(q, 7.0).contiguous(), torch.full_like(k, 7.0).contiguous()
    binding.pa_rope(qo, ko, q, k, pos, table.to(DEV), interleaved=interleaved,
                    amplitude=amplitude, q_weight=qw, k_weight=kw)
    torch.cuda.synchronize()
    assert binding.pa_get_device_error() == 0
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        want, mag = rope_rows(x, pos, table, interleaved, amplitude, w)
        assert_rope(got, want, mag, f"T={T} H={H}/{Hkv} D={D} rot={rot} {interleaved} {norm}")
    return qo, ko


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 32), (80, 20), (96, 24), (128, 128), (128, 2),
                                   (256, 256), (256, 64), (8, 8), (40, 6)])
def test_layouts_and_sizes(D, rot, interleaved, dt):
    run(7, 5, 3, D, rot, dt, interleaved)


@pytest.mark.parametrize("T", [1, 2, 149, 700])
@pytest.mark.parametrize("H,Hkv", [(32, 32), (64, 8), (1, 1)])
def test_tokens_and_heads(T, H, Hkv):
    run(T, H, Hkv, 128, 128, torch.bfloat16, norm=T % 2 == 0)


def test_far_and_negative_positions():
    pos = torch.tensor([0, 1, -1, 123457, 1000003, 16777217, FAR, -FAR - 1])
    for interleaved in (False, True):
        run(8, 2, 2, 128, 128, torch.float16, interleaved, norm=False, positions=pos)


def test_amplitude_and_magnitudes():
    """An amplitude on the rotated part only; rows whose squares leave fp16's range."""
    run(5, 4, 2, 64, 32, torch.bfloat16, amplitude=1.3)
    run(5, 4, 2, 128, 128, torch.bfloat16, scale=1e15)
    run(5, 4, 2, 128, 128, torch.float16, scale=1e-3)


def test_zero_rows_and_one_sided_norms():
    q, k, _, (qw, kw) = inputs(3, 2, 2, 64, torch.bfloat16)
    q = q.clone()
    q[1] = 0
    table, _ = binding.pa_rope_table(64)
    pos = torch.arange(3, dtype=torch.int32, device=DEV)
    for a, b in ((qw, None), (None, kw)):
        qo, ko = torch.empty_like(q), torch.empty_like(k).contiguous()
        binding.pa_rope(qo, ko, q, k, pos, table.to(DEV), q_weight=a, k_weight=b)
        for got, x, w in ((qo, q, a), (ko, k, b)):
            want, mag = rope_rows(x, pos, table, False, 1.0, w)
            assert_rope(got, want, mag, "one norm")
        assert bool((qo[1] == 0).all())


def test_elements_past_the_rotation_keep_infinities():
    """Without a norm the elements past rot_dim are copied: an infinity beside them stays where it
    is and does not become NaN through a product with a zero sine."""
    for interleaved in (False, True):
        x = torch.randn((2, 1, 64), device=DEV).to(torch.bfloat16)
        x[0, 0, 40], x[1, 0, 63] = float("inf"), float("-inf")
        table, _ = binding.pa_rope_table(32)
        out, k = torch.empty_like(x), x[:, :0]
        binding.pa_rope(out, k, x, k, torch.arange(2, dtype=torch.int32, device=DEV),
                        table.to(DEV), interleaved=interleaved)
        assert torch.equal(out[..., 32:], x[..., 32:])


def test_in_place_on_a_fused_projection():
    """q and k rotated where they lie in a [T, H + 2 Hkv, D] projection; v is not touched, and a
    call with outputs of its own gives the same bits."""
    q, k, v, (qw, kw) = inputs(33, 8, 2, 128, torch.bfloat16, seed=3)
    table = binding.pa_rope_table(128)[0].to(DEV)
    pos = torch.arange(33, dtype=torch.int32, device=DEV)
    want = torch.empty(q.shape, dtype=q.dtype, device=DEV), torch.empty(k.shape, dtype=k.dtype,
                                                                       device=DEV)
    binding.pa_rope(*want, q, k, pos, table, q_weight=qw, k_weight=kw)
    v0 = v.clone()
    binding.pa_rope(q, k, q, k, pos, table, q_weight=qw, k_weight=kw)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, v0)


@pytest.mark.parametrize("kind", range(5))
def test_scalings(kind):
    """Each scaling's table rotates as its formula says, amplitude included."""
    table, amp = binding.pa_rope_table(64, 10000.0, kind, factor=4.0, low=1.0, high=32.0,
                                       original_len=2048)
    q, k, _, _ = inputs(9, 2, 1, 64, torch.float16, norm=False)
    pos = torch.arange(8000, 8009, dtype=torch.int32, device=DEV)
    qo, ko = torch.empty_like(q).contiguous(), torch.empty_like(k).contiguous()
    binding.pa_rope(qo, ko, q, k, pos, table.to(DEV), amplitude=amp)
    assert_rope(qo, *rope_rows(q, pos, table, False, amp), f"scaling {kind}")
    assert (kind == binding.PA_ROPE_YARN) == (amp != 1.0)


def slots_for(T, NB, S, seed=0, pad=()):
    g = torch.Generator().manual_seed(seed)
    slots = torch.randperm(NB * S, generator=g)[:T]
    for i in pad:
        slots[i] = -1
    return slots.to(DEV)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,H,Hkv,D,S,rot,interleaved", [
    (1, 4, 4, 128, 16, 128, False), (64, 40, 40, 128, 16, 128, False), (77, 8, 2, 64, 8, 64, True),
    (333, 16, 2, 128, 32, 64, False), (50, 5, 5, 80, 16, 20, False), (21, 3, 1, 256, 5, 256, True),
    (2000, 64, 8, 128, 16, 128, False)])
def test_append_is_rope_then_append(T, H, Hkv, D, S, rot, interleaved, dt):
    """q_out and the whole caches, bit for bit those of pa_rope followed by pa_kv_append; padded
    tokens (negative slots) leave the caches alone but have their q rotated."""
    q, k, v, (qw, kw) = inputs(T, H, Hkv, D, dt, seed=T)
    NB = -(-T // S) + 3
    pad = [i for i in range(T) if i % 9 == 4]
    slots = slots_for(T, NB, S, pad=pad)
    table = binding.pa_rope_table(rot)[0].to(DEV)
    pos = torch.arange(100, 100 + T, dtype=torch.int32, device=DEV)
    cache = torch.randn((2, NB, Hkv, S, D), device=DEV).to(dt)
    want_c = cache.clone()
    qo, ko = torch.empty_like(q).contiguous(), torch.empty_like(k).contiguous()
    how = dict(interleaved=interleaved, q_weight=qw, k_weight=kw)
    binding.pa_rope(qo, ko, q, k, pos, table, **how)
    binding.pa_kv_append(ko, v.contiguous(), slots, want_c[0], want_c[1])
    got_q = torch.empty_like(qo)
    binding.pa_rope_append(got_q, q, k, v, pos, slots, cache[0], cache[1], table, **how)
    torch.cuda.synchronize()
    assert binding.pa_get_device_error() == 0
    assert torch.equal(got_q, qo)
    assert torch.equal(cache.view(torch.int16), want_c.view(torch.int16))


@pytest.mark.parametrize("T,H,Hkv,D,S,rot,interleaved", [
    (1, 4, 4, 128, 16, 128, False), (77, 8, 2, 64, 8, 32, True), (50, 5, 5, 80, 16, 20, False),
    (300, 16, 4, 128, 16, 128, False)])
def test_append_e4m3(T, H, Hkv, D, S, rot, interleaved):
    dt = torch.bfloat16
    q, k, v, (qw, kw) = inputs(T, H, Hkv, D, dt, seed=T)
    NB = -(-T // S) + 2
    slots = slots_for(T, NB, S, pad=[T - 1] if T > 1 else [])
    table = binding.pa_rope_table(rot)[0]
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    k_scale, v_scale = 0.017, 0.02
    cache = torch.randint(0, 120, (2, NB, Hkv, S, D), dtype=torch.uint8, device=DEV)
    plain = cache.clone()
    before = cache.clone()
    qo = torch.empty_like(q).contiguous()
    how = dict(interleaved=interleaved, q_weight=qw, k_weight=kw)
    binding.pa_rope_append_fp8(qo, q, k, v, pos, slots, cache[0], cache[1], k_scale, v_scale,
                               table.to(DEV), **how)
    torch.cuda.synchronize()
    assert binding.pa_get_device_error() == 0
    assert_rope(qo, *rope_rows(q, pos, table, interleaved, 1.0, qw), "q")
    # v as pa_kv_append_fp8 stores it
    binding.pa_kv_append_fp8(k.contiguous(), v.contiguous(), slots, plain[0], plain[1], k_scale,
                             v_scale)
    assert torch.equal(cache[1], plain[1])
    # k: the code nearest to value / scale (half a step: 2^-4 of it, 2^-10 among subnormals)
    want, mag = rope_rows(k, pos, table, interleaved, 1.0, kw)
    y, m = (want / k_scale).clamp(-448, 448), mag / k_scale
    live = (slots >= 0).nonzero().flatten()
    at = slots[live]
    got = cache[0][at // S, :, at % S].view(torch.float8_e4m3fn).double().cpu()
    live = live.cpu()
    tol = 2.0 ** -4 * y[live].abs() + 2.0 ** -10 + 2 * ROPE_FP32 * m[live]
    assert bool(((got - y[live]).abs() <= tol).all())
    # everything that no slot names is as it was
    keep = torch.ones(NB * S, dtype=torch.bool, device=DEV)
    keep[at] = False
    for c, b in zip(cache, before):
        assert torch.equal(c.transpose(1, 2).reshape(NB * S, -1)[keep],
                           b.transpose(1, 2).reshape(NB * S, -1)[keep])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_every_value_over_many_scales(dt):
    """Every 16-bit value, infinities and NaN among them, over scales of all kinds (powers of two,
    mantissas of all ones, random ones, the ends of the range): v's codes are those of
    pa_kv_append_fp8, whose quotients are correctly rounded divisions."""
    Hkv, D, S = 4, 128, 16
    T = 65536 // (Hkv * D)
    v = torch.arange(65536, dtype=torch.int32, device=DEV).to(torch.int16).view(dt)
    v = v.reshape(T, Hkv, D)
    table = binding.pa_rope_table(D)[0].to(DEV)
    pos = torch.zeros(T, dtype=torch.int32, device=DEV)
    slots = torch.arange(T, device=DEV)
    q = torch.zeros((T, 0, D), dtype=dt, device=DEV)
    g = torch.Generator().manual_seed(0)
    scales = [1.0, 0.5, 2.0 ** -9, 2.0 ** -60, 2.0 ** 60, 2.0 - 2.0 ** -23, 2.0 ** -7 - 2.0 ** -31,
              1.0 + 2.0 ** -23, 3.0, 1.0 / 3.0]
    scales += (2.0 ** (20 * torch.rand(120, generator=g, dtype=torch.float64) - 14)).tolist()
    got, want = (torch.zeros((2, T // S, Hkv, S, D), dtype=torch.uint8, device=DEV)
                 for _ in range(2))
    for interleaved in (False, True):
        for s in scales:
            binding.pa_rope_append_fp8(q, q, v, v, pos, slots, got[0], got[1], s, s, table,
                                       interleaved=interleaved)
            binding.pa_kv_append_fp8(v, v, slots, want[0], want[1], s, s)
            assert torch.equal(got[1], want[1]), s
            # at position 0 the rotation changes no finite key
            finite = v.isfinite().all(-1)
            k = [c[0].transpose(1, 2).reshape(T, Hkv, D)[finite] for c in (got, want)]
            k = [x.view(torch.float8_e4m3fn).float() for x in k]  # (-0 may become 0)
            assert torch.equal(*k), s


def test_bad_slots_are_skipped_and_flagged():
    q, k, v, (qw, kw) = inputs(4, 2, 2, 64, torch.bfloat16)
    table = binding.pa_rope_table(64)[0].to(DEV)
    pos = torch.arange(4, dtype=torch.int32, device=DEV)
    cache = torch.zeros((2, 2, 2, 16, 64), device=DEV, dtype=torch.bfloat16)
    slots = torch.tensor([3, 32, 2 ** 40, 5], device=DEV)
    qo = torch.empty_like(q).contiguous()
    binding.pa_rope_append(qo, q, k, v, pos, slots, cache[0], cache[1], table)
    assert binding.pa_get_device_error() == binding.PA_DEVERR_SLOT
    rows = cache[1].transpose(1, 2).reshape(32, 2, 64)
    used = rows.abs().amax((1, 2)) > 0
    assert used.nonzero().flatten().tolist() == [3, 5]
    assert torch.equal(rows[3], v[0]) and torch.equal(rows[5], v[3])


def test_nothing_to_do():
    table = binding.pa_rope_table(64)[0].to(DEV)
    q, k, v, _ = inputs(0, 2, 2, 64, torch.bfloat16)
    pos = torch.zeros(0, dtype=torch.int32, device=DEV)
    binding.pa_rope(q, k, q, k, pos, table)
    cache = torch.zeros((2, 2, 2, 16, 64), device=DEV, dtype=torch.bfloat16)
    binding.pa_rope_append(q, q, k, v, pos, pos.long(), cache[0], cache[1], table)
    assert binding.pa_get_device_error() == 0


def test_captured_and_on_another_stream():
    q, k, v, (qw, kw) = inputs(17, 8, 2, 128, torch.bfloat16)
    table = binding.pa_rope_table(128)[0].to(DEV)
    pos = torch.arange(17, dtype=torch.int32, device=DEV)
    slots = slots_for(17, 4, 16)
    cache = torch.zeros((2, 4, 2, 16, 128), device=DEV, dtype=torch.bfloat16)
    want_c, want_q = cache.clone(), torch.empty_like(q).contiguous()
    binding.pa_rope_append(want_q, q, k, v, pos, slots, want_c[0], want_c[1], table, q_weight=qw,
                           k_weight=kw)
    got_q = torch.zeros_like(want_q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        binding.pa_rope_append(got_q, q, k, v, pos, slots, cache[0], cache[1], table, q_weight=qw,
                               k_weight=kw)
    assert bool((got_q == 0).all())
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got_q, want_q) and torch.equal(cache, want_c)
    pos += 5  # a replay reads the inputs as they are then
    graph.replay()
    binding.pa_rope_append(want_q, q, k, v, pos, slots, want_c[0], want_c[1], table, q_weight=qw,
                           k_weight=kw)
    torch.cuda.synchronize()
    assert torch.equal(got_q, want_q) and torch.equal(cache, want_c)


def test_binding_refusals():
    q, k, v, (qw, kw) = inputs(4, 4, 2, 64, torch.bfloat16)
    table = binding.pa_rope_table(64)[0].to(DEV)
    pos = torch.arange(4, dtype=torch.int32, device=DEV)
    qo, ko = torch.empty_like(q).contiguous(), torch.empty_like(k).contiguous()
    ok = dict(q_out=qo, k_out=ko, q=q, k=k, positions=pos, table=table)
    for bad in (dict(positions=pos.long()), dict(positions=pos[:3]), dict(table=table.float()),
                dict(table=table.cpu()), dict(k=k.half()), dict(q=q.float()),
                dict(q_out=qo[:3]), dict(q_weight=qw[:32]), dict(k_weight=kw.float()),
                dict(q=q.transpose(0, 1)), dict(k=k[..., ::2]), dict(positions=pos.cpu())):
        with pytest.raises(ValueError):
            binding.pa_rope(**{**ok, **bad})
    with pytest.raises(binding.PagedAttnError):  # rot_dim > D
        binding.pa_rope(**{**ok, "table": torch.zeros(33, dtype=torch.float64, device=DEV)})
    cache = torch.zeros((2, 2, 2, 16, 64), device=DEV, dtype=torch.bfloat16)
    slots = torch.arange(4, device=DEV)
    ok = dict(q_out=qo, q=q, k=k, v=v, positions=pos, slot_mapping=slots, k_cache=cache[0],
              v_cache=cache[1], table=table)
    for bad in (dict(slot_mapping=slots.int()), dict(k_cache=cache[0].half()), dict(v=v[:, :1]),
                dict(v_cache=cache[1][:1]), dict(k_cache=cache[0].transpose(1, 2)),
                dict(slot_mapping=slots[:2])):
        with pytest.raises(ValueError):
            binding.pa_rope_append(**{**ok, **bad})
    with pytest.raises(ValueError):
        binding.pa_rope_append_fp8(**ok, k_scale=1.0, v_scale=1.0)
    codes = {**ok, "k_cache": cache[0].to(torch.uint8), "v_cache": cache[1].to(torch.uint8)}
    with pytest.raises(binding.PagedAttnError):
        binding.pa_rope_append_fp8(**codes, k_scale=0.0, v_scale=1.0)
