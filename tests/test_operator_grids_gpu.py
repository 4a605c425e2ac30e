"""Grids of pa_cross and pa_decode_shared beyond what the smaller tests launch: requests that start
in descending order of length, many tail CTAs (the narrow form), and the most requests."""

import pytest
import torch

from paged_kv_cache_driven_b200 import binding
from reference64 import assert_attention, attention, tokens
from test_cross_gpu import check
from test_shared_prefix_decode_gpu import Batch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def uneven(B, last):
    """B lengths, no order in them, some of them equal; the last one is the longest, the shortest,
    none at all, or equal to the first."""
    kv = [(130, 64, 400, 129, 1, 257, 400, 0)[(5 * i + 2) % 8] for i in range(B)]
    kv[0] = 257
    kv[-1] = {"longest": 555, "shortest": 1, "none": 0, "tie": 257}[last]
    return kv


@pytest.mark.parametrize("last", ["longest", "shortest", "none", "tie"])
@pytest.mark.parametrize("B", [2, 3, 7, 31, 32])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_uneven_requests_beyond_a_wave(D, B, last):
    """More CTAs than run at once (two per SM at head size 64, else one; a CTA takes 128 query rows,
    at head size 128 up to 256), so the kernel takes the requests by their lengths."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    q = [(150, 17, 40, 129, 20)[i % 5] for i in range(B)]
    row_tiles = 1 if D == 128 else 2
    H = (2 if D == 64 else 1) * sms // (row_tiles * B) + 1
    check(q, uneven(B, last), H, H, D, 16, torch.bfloat16, partition=-1)


def wide_batch(D, S, shared, seed):
    tails = [0, 1, S - 1, S, S + 1, 97, 128, 5, 211]
    lens = [shared + tails[i % len(tails)] for i in range(24)]
    return Batch([(shared, lens[:19]), (shared // 2, lens[19:])], 32, 32, D, S, torch.bfloat16,
                 seed=seed)


@pytest.mark.parametrize("shared", [0, 96])
@pytest.mark.parametrize("D,S", [(64, 8), (64, 16), (64, 32), (128, 8), (128, 16), (256, 8)])
def test_many_tails_of_single_heads(D, S, shared):
    """768 tail CTAs and more, behind a shared part (launched to overlap it) and without one."""
    wide_batch(D, S, shared, D + S).check()


def test_the_most_requests():
    """65,534 requests behind one block, each with a tail of one token or none."""
    B, S, D = 65534, 16, 64
    g = torch.Generator(device=DEV).manual_seed(0)
    k, v = (torch.randn((B + 1, 1, S, D), generator=g, device=DEV).to(torch.bfloat16)
            for _ in range(2))
    q = torch.randn((B, 1, D), generator=g, device=DEV).to(torch.bfloat16)
    i = torch.arange(B, dtype=torch.int32, device=DEV)
    bt = torch.stack([torch.zeros_like(i), i + 1], 1)
    seq, sh = S + i % 2, torch.full_like(i, S)
    start = torch.tensor([0, B], dtype=torch.int32, device=DEV)
    n = binding.pa_decode_shared_workspace_bytes(B, 1, 1, 1, D, S, B, S, 1)
    out = torch.empty_like(q)
    binding.pa_decode_shared(out, q, k, v, bt, seq, sh, start, 0.125, B, S, 1,
                             workspace=torch.empty(n, dtype=torch.uint8, device=DEV))
    assert binding.pa_get_device_error() == 0
    for r in list(range(5)) + [127, 128, 32767, 32768, B - 2, B - 1]:
        K, V = (tokens(c, [0, r + 1], S + r % 2) for c in (k, v))
        assert_attention(out[r:r + 1], *attention(q[r:r + 1], K, V, 0.125), torch.bfloat16, str(r))
    with pytest.raises(binding.PagedAttnError):  # one more than there may be
        big = torch.zeros((B + 1, 1, D), device=DEV, dtype=torch.bfloat16)
        z = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
        binding.pa_decode_shared(big, big, k, v, z[:, None].repeat(1, 2), z, z, start, 0.125, B, S,
                                 1, workspace=torch.empty(n, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [3, 40])
def test_nan_stays_nan_in_grouped_heads(n, D):
    """Four query heads per KV head: a NaN in a shared key makes NaN of its group's four heads, one in
    a tail of its request's; an infinite score does the same; a tail that is all NaN in one unit
    of keys spoils no other request."""
    H, Hkv = 8, 2
    lens = [300 + i for i in range(n)]
    b = Batch([(256, lens), (128, [200, 0, 150])], H, Hkv, D, 16, torch.bfloat16, seed=n)
    good = b.run()
    b.q[n + 1] = float("nan")  # the request without tokens
    out = b.run()
    assert torch.equal(out, good) and bool((out[n + 1] == 0).all())
    want = torch.zeros_like(out, dtype=torch.bool)
    b.k[b.tables[1][17], 1, 5, 0] = float("nan")  # request 1's own token 277, second KV head
    want[1, 4:] = True
    b.k[b.tables[2][18], 0, :, 3] = float("nan")  # request 2's tokens 288 .. 301, first KV head
    want[2, :4] = True
    b.k[b.tables[0][16], 0, 2, 1] = float("inf")  # request 0's own token 258
    sign = b.q[0, :4, 1] > 0  # (q . K is +inf or -inf: NaN, or a weight of 0)
    want[0, :4][sign] = True
    out = b.run()
    assert torch.equal(out.isnan(), want)
    rest = ~want
    rest[0, :4] = False
    assert torch.equal(out[rest], good[rest])
    b.k[b.tables[n][3], 0, 1, 9] = float("nan")  # a shared token of the second group
    out = b.run()
    want[n, :4] = want[n + 2, :4] = True
    assert torch.equal(out.isnan(), want)


@pytest.mark.parametrize("H,Hkv", [(4, 4), (16, 2)])
def test_wider_bounds_than_needed(H, Hkv):
    Batch([(128, [140, 128, 150, 200]), (64, [70])], H, Hkv, 128, 16, torch.bfloat16).check(
        max_group=5, max_shared_len=176, max_tail_len=190)
