"""What a request of a group must not see (pa_decode_shared): infinities and NaN in the shared tokens
past its own length, against the 64-bit form of that request over its own tokens."""

import pytest
import torch

from paged_kv_cache_driven_b200 import binding
from reference64 import assert_attention, attention, tokens
from test_shared_prefix_decode_gpu import Batch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("n", [3, 5, 60])
@pytest.mark.parametrize("H,Hkv,D,S", [(4, 4, 64, 16), (4, 4, 128, 8), (8, 2, 128, 16),
                                       (10, 2, 64, 32), (4, 4, 256, 16), (8, 2, 256, 8)])
def test_values_past_a_short_request(H, Hkv, D, S, n, dt):
    """Requests that end inside the shared part: V behind their end, in their last block's key tile and
    in later ones and later partitions, holds infinities of both signs and NaN. The long requests
    see those, in the columns that hold them and nowhere else."""
    lens = [(100, 1100, 16, 1030, 7, 0, 333, 1024, 640)[i % 9] for i in range(n)]
    b = Batch([(1024, lens), (64, [70, 5])], H, Hkv, D, S, dt, seed=n)
    common = b.tables[lens.index(1100)]
    for token, col, value in ((8, 1, "inf"), (17, 3, "nan"), (104, 5, "-inf"), (105, 7, "inf"),
                              (700, 9, "nan"), (1000, 11, "-inf")):
        b.v[common[token // S], 0, token % S, col] = float(value)
    out = b.run(torch.float32)
    torch.cuda.synchronize()
    assert binding.pa_get_device_error() == 0
    G = H // Hkv
    for i, n_i in enumerate(b.lens):
        K, V = (tokens(c, b.tables[i], n_i) for c in (b.k, b.v))
        want, mag = attention(b.q[i:i + 1], K, V, b.scale)
        finite = want.isfinite()
        assert torch.equal(out[i:i + 1].isfinite(), finite), f"request {i} of {n_i} tokens"
        if n_i < 9:
            assert bool(finite.all())
        assert bool(finite[:, G:].all())  # (the values lie in the first KV head)
        assert_attention(out[i:i + 1][finite][None], want[finite][None], mag[finite][None], dt,
                         f"request {i}")


def test_a_short_request_that_sees_a_nan():
    """A NaN in a key that a short request sees stays NaN for it, beside masked infinities in V."""
    b = Batch([(512, [600, 100, 90])], 4, 4, 128, 16, torch.bfloat16)
    b.v[b.tables[0][20], :, 0, 0] = float("inf")
    b.k[b.tables[0][5], 2, 15, 0] = float("nan")  # token 95
    out = b.run()
    assert binding.pa_get_device_error() == 0
    want = torch.zeros(4, dtype=torch.bool, device=DEV)
    assert torch.equal(out[2].isnan().any(-1), want)
    want[2] = True
    assert torch.equal(out[1].isnan().any(-1), want) and bool(out[1, 2].isnan().all())


def test_bounds_of_zero_are_checked_too():
    """Lengths past a bound of zero, whose pass is then not launched: clamped and flagged."""
    def flags(b, **bounds):
        out = b.run(**bounds)
        torch.cuda.synchronize()
        return out, binding.pa_get_device_error()

    SEQ = binding.PA_DEVERR_SEQ_LEN
    b = Batch([(64, [64, 70, 64])], 4, 2, 64, 16, torch.bfloat16)
    good, err = flags(b)
    assert err == 0
    out, err = flags(b, max_tail_len=0)  # request 1's tail is 6 tokens
    assert err == SEQ and torch.equal(out[[0, 2]], good[[0, 2]])
    K, V = (tokens(c, b.tables[1], 64) for c in (b.k, b.v))
    assert_attention(out[1:2], *attention(b.q[1:2], K, V, b.scale), b.dt)
    # shared lengths beyond a bound of zero: nothing is shared, all of it is tail
    out, err = flags(b, max_shared_len=0, max_tail_len=70)
    assert err == SEQ
    for i, n in enumerate(b.lens):
        K, V = (tokens(c, b.tables[i], n) for c in (b.k, b.v))
        assert_attention(out[i:i + 1], *attention(b.q[i:i + 1], K, V, b.scale), b.dt)
    b.sh.zero_()
    assert flags(b, max_shared_len=0, max_tail_len=70)[1] == 0
    out, err = flags(b, max_shared_len=0, max_tail_len=0)
    assert err == SEQ and bool((out == 0).all())
    b.seq.copy_(torch.tensor([0, -3, 0]))
    out, err = flags(b, max_shared_len=0, max_tail_len=0)
    assert err == SEQ and bool((out == 0).all())
    b.seq.zero_()
    assert flags(b, max_shared_len=0, max_tail_len=0)[1] == 0
    b.sh[2] = -1
    assert flags(b, max_shared_len=0, max_tail_len=0)[1] == SEQ


@pytest.mark.parametrize("n", [2, 30])
def test_requests_outside_every_group_are_flagged(n):
    """Groups that do not cover the batch leave requests without their shared part."""
    b = Batch([(64, [70 + i for i in range(n)]), (32, [40, 50])], 2, 2, 64, 16, torch.bfloat16)
    good = b.run()
    assert binding.pa_get_device_error() == 0
    for starts, kept in (([0, n, n + 1], slice(0, n + 1)), ([1, n, n + 2], slice(1, n + 2)),
                         ([0, n], slice(0, n))):
        b.start = torch.tensor(starts, dtype=torch.int32, device=DEV)
        out = b.run()
        assert binding.pa_get_device_error() == binding.PA_DEVERR_SEQ_LEN
        assert torch.equal(out[kept], good[kept])
