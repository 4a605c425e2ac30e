"""Decode for batches that share prefixes (pa_decode_shared) against a plain 64-bit form of each
request over its own table: groups of one to many, several groups, shared lengths that end
inside a block, requests without tokens or without tails, grouped heads, poisoned slots."""

import math

import pytest
import torch

from paged_kv_cache_driven_b200 import binding
from reference64 import assert_attention, attention, tokens

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Batch:
    """groups: [(shared tokens, [length of each request])]; the whole blocks of the shared tokens
    are named by all tables of a group, the rest by each its own. Unused slots hold NaN."""

    def __init__(self, groups, H, Hkv, D, S, dt, seed=0):
        g = torch.Generator().manual_seed(seed)
        need = 4 + sum(sh // S + sum(-(-n // S) + 1 for n in lens) for sh, lens in groups)
        perm = torch.randperm(need, generator=g).tolist()
        self.tables, self.lens, self.shared, starts = [], [], [], [0]
        for sh, lens in groups:
            common = [perm.pop() for _ in range(sh // S)]
            for n in lens:
                nb = -(-n // S)
                table = common[:nb]
                self.tables.append(table + [perm.pop() for _ in range(nb - len(table))])
                self.lens.append(n)
                self.shared.append(sh)
            starts.append(starts[-1] + len(lens))
        B = len(self.lens)
        self.MB = max([len(t) for t in self.tables] + [max(s for s in self.shared) // S, 1])
        bt = torch.full((B, self.MB), -1, dtype=torch.int32)
        for i, t in enumerate(self.tables):
            bt[i, :len(t)] = torch.tensor(t, dtype=torch.int32)
        d = torch.Generator(device=DEV).manual_seed(seed)
        shape = (need, Hkv, S, D)
        self.k = torch.randn(shape, generator=d, device=DEV).to(dt)
        self.v = torch.randn(shape, generator=d, device=DEV).to(dt)
        used = torch.zeros((need, S), dtype=torch.bool)
        for t, n in zip(self.tables, self.lens):
            for j, b in enumerate(t):
                used[b, :max(0, min(S, n - j * S))] = True
        for c in (self.k, self.v):
            c.transpose(1, 2)[~used.to(DEV)] = float("nan")
        self.q = torch.randn((B, H, D), generator=d, device=DEV).to(dt)
        self.bt = bt.to(DEV)
        self.seq = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        self.sh = torch.tensor(self.shared, dtype=torch.int32, device=DEV)
        self.start = torch.tensor(starts, dtype=torch.int32, device=DEV)
        self.max_group = max(len(lens) for _, lens in groups)
        self.max_shared = max(self.shared)
        self.max_tail = max(n - min(n, s) // S * S for n, s in zip(self.lens, self.shared))
        self.scale, self.dt, self.H, self.Hkv, self.D, self.S = 1 / math.sqrt(D), dt, H, Hkv, D, S

    def workspace(self, **over):
        b = dict(max_group=self.max_group, max_shared_len=self.max_shared,
                 max_tail_len=self.max_tail, **over)
        n = binding.pa_decode_shared_workspace_bytes(
            len(self.lens), self.start.numel() - 1, self.H, self.Hkv, self.D, self.S, **b)
        return torch.full((n,), 255, dtype=torch.uint8, device=DEV) if n else None

    def run(self, odt=None, out=None, workspace=None, **over):
        if out is None:
            out = torch.full_like(self.q, 7.0, dtype=odt or self.dt)
        bounds = {**dict(max_group=self.max_group, max_shared_len=self.max_shared,
                         max_tail_len=self.max_tail), **over}
        if workspace is None:
            n = binding.pa_decode_shared_workspace_bytes(
                len(self.lens), self.start.numel() - 1, self.H, self.Hkv, self.D, self.S, **bounds)
            workspace = torch.full((n,), 255, dtype=torch.uint8, device=DEV) if n else None
        binding.pa_decode_shared(out, self.q, self.k, self.v, self.bt, self.seq, self.sh,
                                 self.start, self.scale, workspace=workspace, **bounds)
        return out

    def check(self, odt=None, what="", rows=None, **over):
        out = self.run(odt, **over)
        torch.cuda.synchronize()
        assert binding.pa_get_device_error() == 0
        for i in rows if rows is not None else range(len(self.lens)):
            K, V = (tokens(c, self.tables[i], self.lens[i]) for c in (self.k, self.v))
            want, mag = attention(self.q[i:i + 1], K, V, self.scale)
            assert_attention(out[i:i + 1], want, mag, self.dt, f"{what} request {i}")
        return out


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,Hkv", [(4, 4), (8, 1), (10, 2), (24, 1)])
def test_one_group(H, Hkv, D, dt):
    Batch([(320, [321, 330, 400, 357, 320])], H, Hkv, D, 16, dt).check()


@pytest.mark.parametrize("S", [8, 16, 32])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (8, 2)])
def test_several_groups(S, H, Hkv):
    """Groups of several sizes, one request alone, one sharing nothing, one group's prefix far
    longer than the others'."""
    Batch([(64, [70, 64, 65]), (0, [33]), (1024, [1024 + i for i in range(1, 8)]),
           (96, [500]), (0, [5, 200])], H, Hkv, 128, S, torch.bfloat16, seed=S).check()


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 127, 128, 129, 256, 257, 300])
def test_group_sizes(n):
    """One row tile, two, and more, whole and ragged."""
    Batch([(256, [256 + 1 + i % 37 for i in range(n)])], 1, 1, 64, 16, torch.bfloat16).check()


@pytest.mark.parametrize("G", [2, 3, 5, 7, 8, 16, 17, 40, 128])
def test_heads_per_group(G):
    Batch([(272, [280, 300, 273] * 5), (128, [150])], 2 * G, 2, 64, 16, torch.bfloat16).check()


@pytest.mark.parametrize("shared", [0, 16, 112, 128, 144, 256, 1000, 4096])
def test_shared_lengths(shared):
    Batch([(shared, [shared + 3, shared + 700, shared + 1])], 4, 4, 128, 16,
          torch.bfloat16).check()


def test_shared_length_inside_a_block():
    """Only whole blocks are taken from the group: the rest of a shared length that ends inside
    a block is read through each request's own table."""
    b = Batch([(80, [100, 93, 81])], 2, 2, 128, 16, torch.bfloat16)
    b.sh += 13  # 93: five whole blocks and 13 tokens
    b.check(max_shared_len=93)


def test_requests_without_tokens_or_tails():
    """Padding rows of the batch (length 0) give zeros; requests that end with the shared part,
    and a group whose first request is padding."""
    b = Batch([(64, [0, 64, 70, 0]), (32, [32, 32]), (48, [0])], 4, 2, 128, 16, torch.bfloat16)
    out = b.check()
    for i in (0, 3, 6):
        assert bool((out[i] == 0).all())
    everyone = Batch([(64, [64, 64])], 4, 2, 128, 16, torch.bfloat16)
    assert everyone.max_tail == 0
    everyone.check()
    none = Batch([(0, [0, 0, 0])], 4, 2, 128, 16, torch.bfloat16)
    assert bool((none.check() == 0).all())


def test_requests_shorter_than_the_shared_part():
    """A request whose length is below its group's shared length sees its own tokens only."""
    Batch([(512, [100, 600, 16, 513, 7])], 4, 4, 128, 16, torch.bfloat16).check()


@pytest.mark.parametrize("odt", [torch.float32, torch.float16, torch.bfloat16])
def test_output_types(odt):
    Batch([(192, [200, 333])], 8, 2, 128, 16, torch.bfloat16).check(odt)


def test_extreme_scores_and_masked_infinities():
    """Scores that spread over hundreds, in the shared part and in the tails; K and V of unused
    slots hold infinities."""
    b = Batch([(256, [300, 260, 270])], 4, 1, 128, 16, torch.bfloat16)
    b.q *= 30
    for c in (b.k, b.v):
        c[torch.isnan(c)] = float("inf")
    out = b.run(torch.float32)
    assert bool(torch.isfinite(out).all())
    for i in range(3):
        K, V = (tokens(c, b.tables[i], b.lens[i]) for c in (b.k, b.v))
        want, mag = attention(b.q[i:i + 1], K, V, b.scale)
        # scores 30 times as large: their error, and so the weights', is 30 times the derived one
        assert bool(((out[i:i + 1] - want).abs() <= (30 * 2.0 ** -13 + 2.0 ** -17) * mag).all())


@pytest.mark.parametrize("n", [3, 40])
def test_nan_stays_nan_where_it_belongs(n):
    """A NaN in a shared key makes NaN of its whole group, one in a tail of its request only;
    padding rows of q may hold anything."""
    lens = [300 + i for i in range(n)]
    b = Batch([(256, lens), (128, [200, 0, 150])], 4, 4, 64, 16, torch.bfloat16, seed=n)
    good = b.run()
    b.q[n + 1] = float("nan")  # the request without tokens
    out = b.run()
    assert torch.equal(out, good) and bool((out[n + 1] == 0).all())
    b.k[b.tables[1][17], 2, 5, 0] = float("nan")  # request 1's own token 277, head 2
    out = b.run()
    want = torch.zeros_like(out, dtype=torch.bool)
    want[1, 2] = True
    assert torch.equal(out.isnan(), want) and torch.equal(out[~want], good[~want])
    b.k[b.tables[n][3], 0, 1, 9] = float("nan")  # a shared token of the second group, head 0
    out = b.run()
    want[n, 0] = want[n + 2, 0] = True
    assert torch.equal(out.isnan(), want) and torch.equal(out[~want], good[~want])


def test_equals_grouped_decode():
    """The same call without sharing (pa_decode_gqa) on a batch of forked sequences, through the
    allocator: tables of pa_seq_fork, a private last block after copy-on-write."""
    S, D, H, Hkv = 16, 128, 8, 2
    alloc = binding.BlockAllocator(64, S)
    alloc.pa_seq_grow(0, 200)
    for child in range(1, 5):
        alloc.pa_seq_fork(0, child)
    for step in range(5):
        alloc.pa_prepare_step(list(range(5)), 1, 16)
    lens = [alloc.pa_seq_len(i) for i in range(5)]
    bt = alloc.pa_build_block_tables(range(5), 16).to(DEV)
    pairs = alloc.pa_alloc_take_copies().to(DEV)
    g = torch.Generator(device=DEV).manual_seed(0)
    k, v = (torch.randn((64, Hkv, S, D), generator=g, device=DEV).to(torch.bfloat16)
            for _ in range(2))
    binding.pa_copy_blocks(k, v, pairs)
    q = torch.randn((5, H, D), generator=g, device=DEV).to(torch.bfloat16)
    seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
    want, got = (torch.empty((5, H, D), device=DEV) for _ in range(2))
    n = binding.pa_decode_workspace_bytes(5, H, D, S, 256)
    binding.pa_decode_gqa(want, q, k, v, bt, seq, 0.1, 256,
                          workspace=torch.empty(n, dtype=torch.uint8, device=DEV))
    sh = torch.full((5,), 200, dtype=torch.int32, device=DEV)  # 12 whole blocks
    start = torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    n = binding.pa_decode_shared_workspace_bytes(5, 1, H, Hkv, D, S, 5, 200, 16)
    binding.pa_decode_shared(got, q, k, v, bt, seq, sh, start, 0.1, 5, 200, 16,
                             workspace=torch.empty(n, dtype=torch.uint8, device=DEV))
    assert binding.pa_get_device_error() == 0
    # both within 2^-13 + 2^-17 of the exact value relative to sum w |V| <= max |V|
    assert bool(((got - want).abs() <= 2 * (2.0 ** -13 + 2.0 ** -17) * v.float().abs().max()).all())


def test_bad_inputs_are_flagged():
    b = Batch([(64, [70, 80]), (32, [40, 50])], 2, 2, 64, 16, torch.bfloat16)
    good = b.run()
    seq = b.seq.clone()
    b.seq[1] = -4
    out = b.run()
    assert binding.pa_get_device_error() == binding.PA_DEVERR_SEQ_LEN
    assert torch.equal(out[2:], good[2:]) and torch.equal(out[0], good[0])
    b.seq.copy_(seq)
    b.seq[3] = 10 ** 6  # past the table: clamped, flagged
    out = b.run()
    assert binding.pa_get_device_error() & binding.PA_DEVERR_SEQ_LEN
    assert torch.equal(out[:3], good[:3])
    b.seq.copy_(seq)
    b.run(max_tail_len=9)  # request 1's tail is 16 tokens
    assert binding.pa_get_device_error() == binding.PA_DEVERR_SEQ_LEN
    b.sh[2] = -1
    b.run()
    assert binding.pa_get_device_error() == binding.PA_DEVERR_SEQ_LEN
    b.sh[2] = 32
    for bad in ([0, 3, 2], [0, 2, 5], [-1, 2, 4]):
        b.start = torch.tensor(bad, dtype=torch.int32, device=DEV)
        b.run()
        assert binding.pa_get_device_error() == binding.PA_DEVERR_SEQ_LEN
    b.start = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    b.run(max_group=1)
    assert binding.pa_get_device_error() == binding.PA_DEVERR_SEQ_LEN
    b.bt[0, 0] = 10 ** 6
    out = b.run()
    assert binding.pa_get_device_error() == binding.PA_DEVERR_BLOCK_ID
    assert torch.equal(out[2:], good[2:])


def test_captured_and_replayed_with_new_lengths():
    """A captured call reads lengths and tables as they are at each replay."""
    b = Batch([(128, [140, 130, 150, 133])], 8, 2, 128, 16, torch.bfloat16)
    bounds = dict(max_group=4, max_shared_len=128, max_tail_len=64)
    n = binding.pa_decode_shared_workspace_bytes(4, 1, 8, 2, 128, 16, 4, 128, 64)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    want = b.run(**bounds)
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run(out=out, workspace=ws, **bounds)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    b.seq -= 2
    want = b.run(**bounds)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert binding.pa_get_device_error() == 0


def test_a_step_as_it_is_served():
    """The operators together: the prompt's rotated keys appended, the sequences forked, then steps
    of rotated append and shared decode, and cross attention over encoder states that went into
    the same pool; each step against 64 bits on the cache as it is, the first keys against the
    rotation's own formula."""
    S, D, H, Hkv, n = 16, 128, 8, 2, 5
    dt = torch.bfloat16
    alloc = binding.BlockAllocator(128, S)
    g = torch.Generator(device=DEV).manual_seed(5)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV).to(dt)

    k_cache, v_cache = (torch.full((128, Hkv, S, D), float("nan"), device=DEV, dtype=dt)
                        for _ in range(2))
    table = binding.pa_rope_table(D)[0].to(DEV)
    qw, kw = (1 + 0.1 * normal(D)).to(dt), (1 + 0.1 * normal(D)).to(dt)
    how = dict(q_weight=qw, k_weight=kw)
    prompt, enc = 150, 333
    alloc.pa_seq_grow(0, prompt)
    qkv = normal(prompt, H + 2 * Hkv, D)
    slots = alloc.pa_build_slot_mapping([0], [0], [prompt]).to(DEV)
    q, k, v = qkv.split((H, Hkv, Hkv), 1)
    q_rot = torch.empty((prompt, H, D), device=DEV, dtype=dt)
    pos = torch.arange(prompt, dtype=torch.int32, device=DEV)
    binding.pa_rope_append(q_rot, q, k, v, pos, slots, k_cache, v_cache, table, **how)
    alloc.pa_seq_grow(100, enc)  # the encoder's states: their own sequence in the pool
    binding.pa_kv_append(normal(enc, Hkv, D), normal(enc, Hkv, D),
                         alloc.pa_build_slot_mapping([100], [0], [enc]).to(DEV), k_cache, v_cache)
    for c in range(1, n):
        alloc.pa_seq_fork(0, c)
    MB = 24
    enc_table = alloc.pa_build_block_tables([100] * n, MB).to(DEV)
    start = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    shared = torch.full((n,), prompt, dtype=torch.int32, device=DEV)
    one = torch.arange(n + 1, dtype=torch.int32, device=DEV)
    enc_lens = torch.full((n,), enc, dtype=torch.int32, device=DEV)
    ws = torch.empty(binding.pa_decode_shared_workspace_bytes(n, 1, H, Hkv, D, S, n, prompt, 64),
                     dtype=torch.uint8, device=DEV)
    wx = torch.empty(binding.pa_cross_workspace_bytes(n, n, H, Hkv, D, 1, enc), dtype=torch.uint8,
                     device=DEV)
    for step in range(20):
        new = torch.empty(n, dtype=torch.int64)
        tables = torch.empty((n, MB), dtype=torch.int32)
        lens = torch.empty(n, dtype=torch.int32)
        alloc.pa_prepare_step(list(range(n)), 1, MB, new, tables, lens)
        pairs = alloc.pa_alloc_take_copies()
        if len(pairs):
            binding.pa_copy_blocks(k_cache, v_cache, pairs.to(DEV))
        qkv = normal(n, H + 2 * Hkv, D)
        q, k, v = qkv.split((H, Hkv, Hkv), 1)
        seq = lens.to(DEV)
        q_rot = torch.empty((n, H, D), device=DEV, dtype=dt)
        binding.pa_rope_append(q_rot, q, k, v, seq - 1, new.to(DEV), k_cache, v_cache, table, **how)
        out = torch.empty_like(q_rot)
        binding.pa_decode_shared(out, q_rot, k_cache, v_cache, tables.to(DEV), seq, shared, start,
                                 0.1, n, prompt, 64, workspace=ws)
        x = torch.empty_like(out)
        binding.pa_cross(x, out, k_cache, v_cache, enc_table, enc_lens, one, 0.1, 1, enc,
                         workspace=wx)
        for i in range(n):
            t = alloc.pa_seq_block_table(i)
            K, V = (tokens(c, t, int(lens[i])) for c in (k_cache, v_cache))
            assert_attention(out[i:i + 1], *attention(q_rot[i:i + 1], K, V, 0.1), dt)
            t = alloc.pa_seq_block_table(100)
            K, V = (tokens(c, t, enc) for c in (k_cache, v_cache))
            assert_attention(x[i:i + 1], *attention(out[i:i + 1], K, V, 0.1), dt)
    assert binding.pa_get_device_error() == 0


def test_binding_refusals():
    b = Batch([(32, [40, 33])], 4, 2, 64, 16, torch.bfloat16)
    out = torch.empty_like(b.q)
    ok = dict(out=out, q=b.q, k_cache=b.k, v_cache=b.v, block_tables=b.bt, seq_lens=b.seq,
              shared_lens=b.sh, group_start=b.start, scale=0.1, max_group=2, max_shared_len=32,
              max_tail_len=8, workspace=b.workspace())
    for bad in (dict(shared_lens=b.sh.long()), dict(shared_lens=b.sh[:1]), dict(q=b.q.half()),
                dict(block_tables=b.bt[:1]), dict(out=out.double()), dict(seq_lens=b.seq.cpu()),
                dict(group_start=b.start[None])):
        with pytest.raises(ValueError):
            binding.pa_decode_shared(**{**ok, **bad})
    for bad in (dict(workspace=None), dict(scale=-1.0), dict(max_shared_len=10 ** 6),
                dict(max_tail_len=-1), dict(max_group=0), dict(group_start=b.start[:1])):
        with pytest.raises(binding.PagedAttnError):
            binding.pa_decode_shared(**{**ok, **bad})
    assert binding.pa_get_device_error() == 0
