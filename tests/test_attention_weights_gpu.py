"""How many bits of a softmax weight enter the second product of pa_cross and pa_decode_shared.

One token (the sink, V = 0) has score 0, a second kind of tokens (V = 1) has the score -c scale,
c a value of each query row, and the rest score so low that their weights are 0 in 32 bits. So a
row's exact output is n w / (1 + n w), w = exp(-c scale), in each of its columns: nothing
averages a weight's rounding away."""

import pytest
import torch

from paged_kv_cache_driven_b200 import binding
from test_shared_prefix_decode_gpu import Batch

pytestmark = pytest.mark.gpu
DEV = "cuda"
NONE = -60000.0  # times at least 1/8: a weight of 0


def queries(rows, H, D, dt, lo, hi, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.zeros((rows, H, D), device=DEV)
    q[..., 0] = lo + (hi - lo) * torch.rand((rows, H), generator=g, device=DEV)
    return q.to(dt)


def assert_weights(out, q, scale, n, dt, small=0.0):
    """Weights as two 16-bit terms: 2^-16 (bf16) or 2^-22 (fp16) of a weight. 32-bit work: the
    exponent, below 16, with three roundings (3 x 2^-24 x 16 x ln 2), 2^x (2^-22), up to 40 sums
    one after the other (2^-23 each in the product, 2^-24 beside it), quotient and merges
    (2 x 2^-22): together below 2^-16. small: the largest error from fp16's smallest steps,
    relative to a weight."""
    c = q[..., :1].double()
    w = n * torch.exp(-c * scale)
    want = (w / (1 + w)).expand(out.shape)
    rel = (2.0 ** -16 if dt == torch.bfloat16 else 2.0 ** -22 + small) + 2.0 ** -16
    off = (out.double() - want).abs() / want
    assert bool((off <= rel).all()), f"worst {off.max():.3g}, {off.max() / rel:.3g} x tolerance"


def cross(q, S, tokens, special, dt, partition):
    rows, H, D = q.shape
    NB = -(-tokens // S)
    k = torch.zeros((NB, H, S, D), device=DEV)
    v = torch.ones((NB, H, S, D), device=DEV)  # (every token but the sink)
    flat = k.transpose(1, 2).reshape(NB * S, H, D)
    flat[:, :, 0] = NONE
    flat[7, :, 0] = 0
    flat[special, :, 0] = -1
    k = flat.reshape(NB, S, H, D).transpose(1, 2).contiguous().to(dt)
    v[7 // S, :, 7 % S] = 0
    v = v.to(dt)
    bt = torch.arange(NB, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([tokens], dtype=torch.int32, device=DEV)
    start = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    out = torch.full((rows, H, D), 7.0, device=DEV)
    n = binding.pa_cross_workspace_bytes(1, rows, H, H, D, rows, tokens, partition)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV) if n else None
    binding.pa_cross(out, q, k, v, bt, lens, start, 0.125, rows, tokens, partition=partition,
                     workspace=ws)
    torch.cuda.synchronize()
    assert binding.pa_get_device_error() == 0
    return out


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("rows", [1, 40, 200])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_cross(D, rows, dt):
    q = queries(rows, 24, D, dt, 1, 22)
    for partition in (-1, 128):
        for token in (3, 100, 290):  # the sink's tile, another warpgroup's, another tile or part
            assert_weights(cross(q, 16, 300, [token], dt, partition), q, 0.125, 1, dt)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("D", [64, 128])
def test_many_small_weights(D, rows, dt):
    """600 weights around e^-10 beside a sink whose V is 0: fp16's smallest step, 2^-24, is
    2^-25 / 2^-14.5 of such a weight as it is, and has to lie at least 2^7 lower."""
    q = queries(rows, 4, D, dt, 79, 81)
    out = cross(q, 16, 700, list(range(20, 620)), dt, -1)
    assert_weights(out, q, 0.125, 600, dt, small=2.0 ** -25 / 2.0 ** (-14.7 + 7))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("H,Hkv,D", [(4, 4, 64), (16, 4, 64), (4, 4, 128), (16, 4, 128),
                                     (24, 1, 128), (8, 4, 256)])
def test_shared_prefix(H, Hkv, D, n, dt):
    """The special tokens in the shared part, then in the tails."""
    if (H // Hkv) * n > 16 and n == 3:
        n = 1
    for behind in (False, True):
        b = Batch([(256, [256 + 20 + i for i in range(n)])], H, Hkv, D, 16, dt)
        b.q = queries(n, H, D, dt, 1, 22, seed=n)
        b.k.zero_()
        b.k[..., 0] = NONE
        b.v.fill_(1)
        for t in b.tables:
            for token, key in ((7, 0), (130, -1)) if not behind else ((263, 0), (269, -1)):
                b.k[t[token // 16], :, token % 16, 0] = key
                b.v[t[token // 16], :, token % 16] = 0 if key == 0 else 1
        b.scale = 0.125
        out = b.run(torch.float32)
        assert binding.pa_get_device_error() == 0
        assert_weights(out, b.q, b.scale, 1, dt)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("rows", [1, 40, 200])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_beyond_the_integers(D, rows, dt):
    """Scores from 2^18 to 2^30, where 32-bit steps exceed what the weights are scaled by: equal scores
    give V's mean, a larger one takes all."""
    S, n = 16, 300
    NB = -(-n // S)
    g = torch.Generator(device=DEV).manual_seed(rows)
    v = torch.randn((NB, 4, S, D), generator=g, device=DEV).to(dt)
    bt = torch.arange(NB, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    start = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    V = v.transpose(1, 2).reshape(NB * S, 4, D)[:n].double()
    for size in (1000, 3000, 6000, 10000, 14000, 20000, 24000, 28000, 34000, 40000, 60000):
        q = torch.zeros((rows, 4, D), device=DEV, dtype=dt)
        q[..., 0] = size
        for top in (None, 5, 100, 200, 299):
            k = torch.zeros_like(v)
            k[..., 0] = size
            if top is not None:  # a step of the 16-bit types: scores higher by 2^7 and more
                k[top // S, :, top % S, 0] = size * 1.01
            for partition in (-1, 128):
                out = torch.full((rows, 4, D), 7.0, device=DEV)
                b = binding.pa_cross_workspace_bytes(1, rows, 4, 4, D, rows, n, partition)
                ws = torch.full((b,), 255, dtype=torch.uint8, device=DEV) if b else None
                binding.pa_cross(out, q, k, v, bt, lens, start, 0.125, rows, n,
                                 partition=partition, workspace=ws)
                want = V.mean(0) if top is None else V[top]
                off = (out.double() - want).abs().amax()
                # 32-bit sums of 300 values below 6
                assert bool(off <= 2.0 ** -15), f"{size} {top} {partition}: {off}"
    assert binding.pa_get_device_error() == 0
