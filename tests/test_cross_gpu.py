"""Cross attention over cached states (pa_cross) against a plain 64-bit form: ragged query and
key lengths (none, one, tile edges), every head size and block size, grouped heads, split and
unsplit keys, poisoned unused slots."""

import pytest
import torch

from paged_kv_cache_driven_b200 import binding, workloads
from reference64 import assert_attention, attention, tokens

pytestmark = pytest.mark.gpu
DEV = "cuda"


def case(q_lens, kv_lens, H, Hkv, D, S, dt, seed=0, **kw):
    c = workloads.decode_case(kv_lens, H=H, D=D, S=S, dtype=dt, seed=seed, device=DEV, Hkv=Hkv,
                              pool_blocks=sum(-(-n // S) for n in kv_lens) + 3, **kw)
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    q = torch.randn((sum(q_lens), H, D), generator=g, device=DEV).to(dt)
    starts = [0]
    for n in q_lens:
        starts.append(starts[-1] + n)
    return c, q, torch.tensor(starts, dtype=torch.int32, device=DEV)


def call(c, q, q_start, q_lens, kv_lens, odt=None, partition=0, max_q=None, max_kv=None, out=None,
         stream=None):
    T, H, D = q.shape
    Hkv = c.k_cache.shape[1]
    max_q = max(q_lens) if max_q is None else max_q
    max_kv = max(kv_lens) if max_kv is None else max_kv
    if out is None:
        out = torch.full_like(q, 7.0, dtype=odt or q.dtype)
    n = binding.pa_cross_workspace_bytes(len(kv_lens), T, H, Hkv, D, max_q, max_kv, partition)
    # whatever the workspace holds must not matter
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV) if n else None
    binding.pa_cross(out, q, c.k_cache, c.v_cache, c.block_tables, c.seq_lens, q_start, c.scale,
                     max_q, max_kv, partition=partition, workspace=ws, stream=stream)
    return out


def check(q_lens, kv_lens, H, Hkv, D, S, dt, odt=None, partition=0, seed=0, **kw):
    c, q, q_start = case(q_lens, kv_lens, H, Hkv, D, S, dt, seed)
    out = call(c, q, q_start, q_lens, kv_lens, odt, partition, **kw)
    torch.cuda.synchronize()
    assert binding.pa_get_device_error() == 0
    at = 0
    for i, n in enumerate(q_lens):
        K = tokens(c.k_cache, c.tables_host[i], kv_lens[i])
        V = tokens(c.v_cache, c.tables_host[i], kv_lens[i])
        want, mag = attention(q[at:at + n], K, V, c.scale)
        assert_attention(out[at:at + n], want, mag, dt, f"request {i}: {n} x {kv_lens[i]}")
        at += n
    return out


RAGGED_Q = [1, 0, 77, 128, 129, 300, 1]
RAGGED_KV = [300, 50, 1, 128, 129, 0, 1000]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("partition", [-1, 0, 128])
def test_ragged(D, dt, partition):
    check(RAGGED_Q, RAGGED_KV, 3, 3, D, 16, dt, partition=partition)


@pytest.mark.parametrize("S", [8, 16, 32, 64, 128])
def test_block_sizes(S):
    check([5, 200], [777, 130], 4, 2, 128, S, torch.bfloat16, partition=256)
    check([1, 1], [90, 1200], 2, 2, 64, S, torch.float16)


@pytest.mark.parametrize("S", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 256])
def test_block_sizes_many_rows(D, S):
    """Blocks shorter and longer than a key tile under whole row tiles, keys split and not."""
    for partition in (-1, 128):
        check([40, 200], [777, 130], 2, 2, D, S, torch.bfloat16, partition=partition)
    check([129, 17, 50], [64, 63, 193], 2, 1, D, S, torch.float16)


@pytest.mark.parametrize("B", [2, 7, 32, 33])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_more_than_a_wave_of_uneven_requests(D, B):
    """Lengths in an order of their own, with equal ones, none, and requests without queries,
    on more CTAs than run at once (up to 32 requests then start in descending order of length)."""
    kv = [(0, 130, 64, 400, 130, 1, 257)[(3 * i + 1) % 7] for i in range(B)]
    q = [(150, 17, 0, 129, 20)[i % 5] for i in range(B)]
    H = 12 if B > 2 else 160
    check(q, kv, H, H, D, 16, torch.bfloat16)
    check(q, [130] * B, H, H, D, 16, torch.float16)


@pytest.mark.parametrize("G", [1, 2, 5, 8, 16, 100, 128])
@pytest.mark.parametrize("q", [1, 3, 60, 300])
def test_grouped_heads(G, q):
    """Rows of a tile are (token, head) pairs: groups that divide 128 and groups that do not."""
    check([q, max(1, q // 2)], [200, 391], 2 * G, 2, 64, 16, torch.bfloat16, seed=G)


@pytest.mark.parametrize("kv", [1, 64, 127, 128, 129, 255, 256, 257, 384, 385, 640])
@pytest.mark.parametrize("q", [1, 128, 129, 256])
def test_key_tiles(q, kv):
    """One to six key tiles, whole and ragged, on one row tile and on two."""
    check([q], [kv], 1, 1, 128, 16, torch.bfloat16, partition=-1)


@pytest.mark.parametrize("odt", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("partition", [-1, 128])
def test_output_types(odt, partition):
    check([3, 150], [300, 500], 2, 1, 128, 16, torch.bfloat16, odt=odt, partition=partition)


def test_split_equals_unsplit_rows():
    """Single tokens over long states: the automatic split against one pass."""
    c, q, qs = case([1] * 4, [1500, 700, 1, 999], 20, 20, 64, 16, torch.bfloat16)
    a = call(c, q, qs, [1] * 4, [1500, 700, 1, 999], torch.float32)
    b = call(c, q, qs, [1] * 4, [1500, 700, 1, 999], torch.float32, partition=-1)
    n = binding.pa_cross_workspace_bytes(4, 4, 20, 20, 64, 1, 1500)
    assert n > 0
    # the same weights' terms; the sums over the keys in another order
    assert bool(((a - b).abs() <= 2.0 ** -14 * (1 + b.abs())).all())


def test_rows_outside_the_requests_stay():
    """Rows of q before q_start[0]'s and behind the last request's are left as they were."""
    c, q, qs = case([4, 6, 5], [100, 300, 40], 2, 2, 64, 16, torch.bfloat16)
    out = torch.full_like(q, 7.0)
    qs2 = torch.tensor([4, 4, 10, 10], dtype=torch.int32, device=DEV)  # only rows 4 .. 9
    for partition in (-1, 128):
        out.fill_(7.0)
        n = binding.pa_cross_workspace_bytes(3, 15, 2, 2, 64, 6, 300, partition)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
        binding.pa_cross(out, q, c.k_cache, c.v_cache, c.block_tables, c.seq_lens, qs2, c.scale, 6,
                         300, partition=partition, workspace=ws)
        torch.cuda.synchronize()
        assert bool((out[:4] == 7).all()) and bool((out[10:] == 7).all())
        K, V = (tokens(x, c.tables_host[1], 300) for x in (c.k_cache, c.v_cache))
        assert_attention(out[4:10], *attention(q[4:10], K, V, c.scale), torch.bfloat16)
    assert binding.pa_get_device_error() == 0


def test_wider_bounds_than_needed():
    check([3, 40], [100, 260], 2, 2, 128, 16, torch.bfloat16, max_q=43, max_kv=272)


def test_bad_inputs_are_flagged():
    q_lens, kv_lens = [4, 6], [100, 300]
    c, q, qs = case(q_lens, kv_lens, 2, 2, 64, 16, torch.bfloat16)
    good = call(c, q, qs, q_lens, kv_lens, partition=-1)
    bt = c.block_tables.clone()
    bt[0, 1] = c.k_cache.shape[0] + 3
    c2 = workloads.DecodeCase(q=c.q, k_cache=c.k_cache, v_cache=c.v_cache, block_tables=bt,
                              seq_lens=c.seq_lens, scale=c.scale)
    out = call(c2, q, qs, q_lens, kv_lens, partition=-1)
    assert binding.pa_get_device_error() == binding.PA_DEVERR_BLOCK_ID
    assert torch.equal(out[4:], good[4:])
    # a length past its bound is clamped to it, one below zero counts as none
    c2.block_tables = c.block_tables
    c2.seq_lens = torch.tensor([-5, 300], dtype=torch.int32, device=DEV)
    out = call(c2, q, qs, q_lens, kv_lens, partition=-1, max_kv=208)
    assert binding.pa_get_device_error() == binding.PA_DEVERR_SEQ_LEN
    assert bool((out[:4] == 0).all())
    K, V = (tokens(x, c.tables_host[1], 208) for x in (c.k_cache, c.v_cache))
    assert_attention(out[4:], *attention(q[4:], K, V, c.scale), torch.bfloat16)
    # inconsistent query ranges: that request is skipped
    for bad in ([0, 4, 11], [0, 4, 3], [-1, 4, 10]):
        out = call(c, q, torch.tensor(bad, dtype=torch.int32, device=DEV), q_lens, kv_lens,
                   partition=-1)
        assert binding.pa_get_device_error() == binding.PA_DEVERR_SEQ_LEN
    out = call(c, q, qs, q_lens, kv_lens, partition=-1, max_q=5)
    assert binding.pa_get_device_error() == binding.PA_DEVERR_SEQ_LEN
    assert torch.equal(out[:4], good[:4]) and bool((out[4:] == 7).all())


@pytest.mark.parametrize("q_len,partition", [(1, -1), (1, 128), (3, 0), (40, -1), (300, -1),
                                             (40, 128)])
@pytest.mark.parametrize("D", [64, 128])
def test_nan_stays_nan_where_it_belongs(D, q_len, partition):
    """A NaN in a key of a request, or in one query row, makes NaN of the rows that see it and of no
    others (zeros would hide it)."""
    q_lens, kv_lens = [q_len, q_len], [600, 500]
    c, q, qs = case(q_lens, kv_lens, 2, 2, D, 16, torch.bfloat16, seed=3)
    good = call(c, q, qs, q_lens, kv_lens, partition=partition)
    c.k_cache[c.tables_host[0][20], 1, 3, 5] = float("nan")  # token 323 of request 0, head 1
    bad_row = 2 * q_len - 1
    q[bad_row, 0, 7] = float("nan")
    out = call(c, q, qs, q_lens, kv_lens, partition=partition)
    want = torch.zeros(2 * q_len, 2, dtype=torch.bool, device=DEV)
    want[:q_len, 1] = True
    want[bad_row, 0] = True
    assert torch.equal(out.isnan().all(-1), want) and torch.equal(out.isnan().any(-1), want)
    assert torch.equal(out[~want], good[~want])


def test_captured_on_two_streams():
    """Two captured calls with workspaces of their own, replayed at the same time."""
    q_lens, kv_lens = [1] * 3, [900, 1500, 64]
    runs = []
    for seed in (1, 2):
        c, q, qs = case(q_lens, kv_lens, 8, 4, 64, 16, torch.bfloat16, seed)
        want = call(c, q, qs, q_lens, kv_lens)
        n = binding.pa_cross_workspace_bytes(3, 3, 8, 4, 64, 1, 1500)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        out, st, g = torch.zeros_like(want), torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=st):
            binding.pa_cross(out, q, c.k_cache, c.v_cache, c.block_tables, c.seq_lens, qs, c.scale,
                             1, 1500, workspace=ws)
        runs.append((g, st, out, want, ws, c, q, qs))
    for _ in range(5):
        for g, st, *_ in runs:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for _, _, out, want, *_ in runs:
        assert torch.equal(out, want)


def test_binding_refusals():
    c, q, qs = case([2], [40], 4, 2, 64, 16, torch.bfloat16)
    out = torch.empty_like(q)
    ok = dict(out=out, q=q, k_cache=c.k_cache, v_cache=c.v_cache, block_tables=c.block_tables,
              kv_lens=c.seq_lens, q_start=qs, scale=c.scale, max_q_len=2, max_kv_len=40)
    for bad in (dict(q=q.float()), dict(q=q.half()), dict(out=out[:1]), dict(q_start=qs[:1]),
                dict(q_start=qs.long()), dict(kv_lens=c.seq_lens.cpu()),
                dict(v_cache=c.v_cache[:1]), dict(block_tables=c.block_tables[0]),
                dict(q=q.transpose(0, 1)), dict(out=out.double())):
        with pytest.raises(ValueError):
            binding.pa_cross(**{**ok, **bad})
    for bad in (dict(scale=0.0), dict(max_kv_len=10 ** 6), dict(partition=100),
                dict(partition=-2)):
        with pytest.raises(binding.PagedAttnError):
            binding.pa_cross(**{**ok, **bad})
    long = case([1], [2000], 1, 1, 64, 16, torch.bfloat16)
    with pytest.raises(binding.PagedAttnError):  # a split without its workspace
        binding.pa_cross(torch.empty_like(long[1]), long[1], long[0].k_cache, long[0].v_cache,
                         long[0].block_tables, long[0].seq_lens, long[2], 0.1, 1, 2000)
    assert binding.pa_get_device_error() == 0
