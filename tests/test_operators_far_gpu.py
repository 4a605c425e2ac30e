"""The rotary, cross-attention and shared-prefix operators where offsets pass 32 bits, and captured
into a graph by a process that has made no call before."""

import subprocess
import sys

import pytest
import torch

from paged_kv_cache_driven_b200 import binding
from reference64 import assert_attention, assert_rope, attention, rope_rows, tokens

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def big():
    """K and V caches of more than 2^31 elements each; the first and the last blocks hold values."""
    NB, Hkv, S, D = 70000, 16, 16, 128
    assert NB * Hkv * S * D > 2 ** 31
    k, v = (torch.zeros((NB, Hkv, S, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    yield k, v
    del k, v
    torch.cuda.empty_cache()


def test_append_and_attention_behind_2_31_elements(big):
    k_cache, v_cache = big
    NB, Hkv, S, D = k_cache.shape
    H, n = 32, 200
    g = torch.Generator(device=DEV).manual_seed(1)
    qkv = torch.randn((n, H + 2 * Hkv, D), generator=g, device=DEV).to(torch.bfloat16)
    q, k, v = qkv.split((H, Hkv, Hkv), 1)
    table = [NB - 1 - 3 * j for j in range(-(-n // S))]  # the last blocks, out of order
    bt = torch.tensor([table], dtype=torch.int32, device=DEV)
    t = torch.arange(n, device=DEV)
    slots = torch.tensor(table, device=DEV)[t // S] * S + t % S
    assert int(slots.max()) * Hkv * D > 2 ** 31
    q_rot = torch.empty((n, H, D), dtype=torch.bfloat16, device=DEV)
    freq = binding.pa_rope_table(D)[0]
    binding.pa_rope_append(q_rot, q, k, v, t.int(), slots, k_cache, v_cache, freq.to(DEV))
    K, V = (tokens(c, table, n) for c in (k_cache, v_cache))
    assert torch.equal(V, v)
    assert_rope(K, *rope_rows(k, t, freq, False), "k")
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    for rows in (3, 8, 200):  # few rows, one row tile, two
        qs = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
        for partition in (-1, 128):
            m = binding.pa_cross_workspace_bytes(1, rows, H, Hkv, D, rows, n, partition)
            ws = torch.empty(m, dtype=torch.uint8, device=DEV) if m else None
            x = q_rot[:rows].contiguous()
            out = torch.empty_like(x)
            binding.pa_cross(out, x, k_cache, v_cache, bt, lens, qs, 0.1, rows, n,
                             partition=partition, workspace=ws)
            assert_attention(out, *attention(x, K, V, 0.1), torch.bfloat16, f"{rows} rows")
    for B in (4, 40):  # forked: 192 shared tokens, tails of 8
        out = torch.empty_like(q_rot[:B])
        m = binding.pa_decode_shared_workspace_bytes(B, 1, H, Hkv, D, S, B, 192, 16)
        binding.pa_decode_shared(
            out, q_rot[:B].contiguous(), k_cache, v_cache, bt.expand(B, -1).contiguous(),
            lens.expand(B).contiguous(), torch.full((B,), 192, dtype=torch.int32, device=DEV),
            torch.tensor([0, B], dtype=torch.int32, device=DEV), 0.1, B, 192, 16,
            workspace=torch.empty(m, dtype=torch.uint8, device=DEV))
        assert_attention(out, *attention(q_rot[:B], K, V, 0.1), torch.bfloat16, f"{B} requests")
    assert binding.pa_get_device_error() == 0


def test_rope_behind_2_31_elements():
    T, H, Hkv, D = 215000, 62, 9, 128
    assert T * (H + 2 * Hkv) * D > 2 ** 31
    qkv = torch.zeros((T, H + 2 * Hkv, D), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(2)
    qkv[-40:] = torch.randn((40, H + 2 * Hkv, D), generator=g, device=DEV).to(torch.bfloat16)
    last = qkv[-40:].clone()
    freq = binding.pa_rope_table(D)[0]
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    q, k, v = qkv.split((H, Hkv, Hkv), 1)
    binding.pa_rope(q, k, q, k, pos, freq.to(DEV))  # in place
    for got, x in ((q, last[:, :H]), (k, last[:, H:H + Hkv])):
        assert_rope(got[-40:], *rope_rows(x, pos[-40:], freq, False), "last tokens")
    assert torch.equal(v[-40:], last[:, H + Hkv:])
    assert bool((q[:-40] == 0).all())
    assert binding.pa_get_device_error() == 0


FIRST_CALLS = """
import torch
from paged_kv_cache_driven_b200 import binding as pa
D, S = 64, 16
def make(B, n):
    kc, vc = (torch.randn((64, 2, S, D), device="cuda").to(torch.bfloat16) for _ in range(2))
    bt = torch.randperm(64)[:B * n].reshape(B, n).int().cuda()
    return kc, vc, bt
kc, vc, bt = make(4, 8)
table = pa.pa_rope_table(D)[0].cuda()
lens = torch.full((4,), 120, dtype=torch.int32, device="cuda")
sh = torch.zeros(4, dtype=torch.int32, device="cuda")
pos, slots = lens - 1, (bt[:, 7].long() * S + 7)
one, grp = (torch.arange(n, dtype=torch.int32, device="cuda") for n in (5, 5))
qkv = torch.randn((4, 12, D), device="cuda").to(torch.bfloat16)
q, k, v = qkv.split((8, 2, 2), 1)
qo = torch.empty((4, 8, D), dtype=torch.bfloat16, device="cuda")
o1, o2 = torch.empty_like(qo), torch.empty_like(qo)
w1, w2 = (torch.empty(1 << 22, dtype=torch.uint8, device="cuda") for _ in range(2))
def step():
    pa.pa_rope_append(qo, q, k, v, pos, slots, kc, vc, table)
    pa.pa_cross(o1, qo, kc, vc, bt, lens, one, 0.1, 1, 128, workspace=w1)
    pa.pa_decode_shared(o2, qo, kc, vc, bt, lens, sh, grp, 0.1, 1, 16, 128, workspace=w2)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
torch.cuda.synchronize()
got = o1.clone(), o2.clone()
step()
torch.cuda.synchronize()
assert torch.equal(got[0], o1) and torch.equal(got[1], o2)
assert (o1.float() - o2.float()).abs().max() < 0.05  # the same attention two ways
assert pa.pa_get_device_error() == 0
print("same")
"""


def test_first_calls_captured():
    """A process whose first calls are inside a graph capture."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
