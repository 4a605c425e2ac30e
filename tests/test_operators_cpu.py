"""Rotary tables, and the host-side refusals and plans of pa_rope, pa_rope_append(_fp8), pa_cross and
pa_decode_shared: nothing here reaches a GPU."""

import ctypes
import math

import pytest
import torch

from paged_kv_cache_driven_b200 import binding, build

INVALID, OK = binding.PA_ERR_INVALID, binding.PA_OK
NULL = None
P = ctypes.c_void_p(16 * 1024)  # an aligned address that the host checks never dereference
ODD = ctypes.c_void_p(16 * 1024 + 8)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def freqs(rot, base=10000.0):
    return [base ** (-2.0 * j / rot) for j in range(rot // 2)]


def close(table, want):
    # a few roundings in 64 bits
    return all(abs(a * 2 * math.pi - b) <= 1e-13 * b for a, b in zip(table.tolist(), want))


def test_tables(lib):
    for rot in (2, 20, 64, 128, 256):
        t, amp = binding.pa_rope_table(rot)
        assert t.dtype == torch.float64 and t.numel() == rot // 2 and amp == 1.0
        assert close(t, freqs(rot))
    t, _ = binding.pa_rope_table(64, 500000.0)
    assert close(t, freqs(64, 500000.0))
    t, amp = binding.pa_rope_table(64, scaling=binding.PA_ROPE_LINEAR, factor=8.0)
    assert amp == 1.0 and close(t, [f / 8 for f in freqs(64)])
    t, amp = binding.pa_rope_table(64, scaling=binding.PA_ROPE_NTK, factor=4.0)
    assert amp == 1.0 and close(t, freqs(64, 10000.0 * 4.0 ** (64 / 62)))


def test_banded_tables(lib):
    rot, factor, low, high, n = 128, 8.0, 1.0, 4.0, 8192
    t, amp = binding.pa_rope_table(rot, 500000.0, binding.PA_ROPE_BANDS, factor, low, high, n)
    want = []
    for f in freqs(rot, 500000.0):
        wavelength = 2 * math.pi / f
        if wavelength < n / high:
            want.append(f)
        elif wavelength > n / low:
            want.append(f / factor)
        else:
            keep = (n / wavelength - low) / (high - low)
            want.append((1 - keep) * f / factor + keep * f)
    assert amp == 1.0 and close(t, want)


def test_yarn_tables(lib):
    rot, base, factor, low, high, n = 128, 10000.0, 4.0, 1.0, 32.0, 4096

    def pair(turns):
        return rot * math.log(n / (turns * 2 * math.pi)) / (2 * math.log(base))

    first, last = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
    t, amp = binding.pa_rope_table(rot, base, binding.PA_ROPE_YARN, factor, low, high, n)
    want = []
    for j, f in enumerate(freqs(rot, base)):
        ramp = min(max((j - first) / (last - first), 0.0), 1.0)
        want.append(f / factor * ramp + f * (1 - ramp))
    assert close(t, want)
    assert abs(amp - (0.1 * math.log(factor) + 1)) < 1e-6
    # the fastest pairs as they were, the slowest by the whole factor
    f = freqs(rot, base)
    assert abs(t[0] * 2 * math.pi - f[0]) < 1e-12
    assert abs(t[-1] * 2 * math.pi - f[-1] / factor) < 1e-12


@pytest.mark.parametrize("bad", [
    dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=-4), dict(base=1.0), dict(base=NAN),
    dict(scaling=9), dict(scaling=-1), dict(scaling=1, factor=0.5), dict(scaling=1, factor=INF),
    dict(scaling=2, rot_dim=2), dict(scaling=3), dict(scaling=3, original_len=100, low=0.0),
    dict(scaling=4, original_len=100, low=4.0, high=4.0), dict(scaling=4, original_len=NAN)])
def test_table_refusals(lib, bad):
    with pytest.raises(binding.PagedAttnError):
        binding.pa_rope_table(**{"rot_dim": 64, "factor": 2.0, **bad})
    amp = ctypes.c_float()
    assert lib.pa_rope_table(NULL, 64, 1e4, 0, 1.0, 1.0, 2.0, 0.0, ctypes.byref(amp)) == INVALID


def address(x):
    return 0 if x is None else x.value if isinstance(x, ctypes.c_void_p) else x


def rope_block(a, scales=(1.0, 1.0)):
    """The arguments of a rotary call as an argument block."""
    ptr = ["q_out", "qos", "k_out", "kos", "q", "qs", "k", "ks", "v", "vs", "slots", "kc", "vc",
           "pos", "table", "qw", "kw", "stream"]
    return binding._ROPE_ARGS.pack(
        *(address(a.get(n)) for n in ptr), *scales, a["amp"], a["eps"],
        *(a.get(n, 0) for n in ("rot", "il", "T", "H", "Hkv", "D", "S", "NB", "dt")))


def ranges_block(a):
    """The arguments of pa_cross or pa_decode_shared as an argument block."""
    a = {**a, "lens": a.get("lens", a.get("seq"))}
    ptr = ["out", "q", "k", "v", "bt", "lens", "start", "sh", "ws", "ws_bytes", "stream"]
    ints = ["out_dt", "MB", "B", "H", "Hkv", "D", "S", "NB", "dt", "T", "max_q", "max_kv",
            "partition", "NG", "max_group", "max_shared", "max_tail"]
    return binding._RANGES_ARGS.pack(*(address(a.get(n)) for n in ptr), a["scale"],
                                     *(a.get(n, 0) for n in ints))


ROPE = dict(q_out=P, qos=4 * 64, k_out=P, kos=2 * 64, q=P, qs=4 * 64, k=P, ks=2 * 64, pos=P,
            table=P, rot=64, il=0, amp=1.0, qw=NULL, kw=NULL, eps=1e-6, T=3, H=4, Hkv=2, D=64,
            dt=binding.PA_BF16, stream=NULL)


@pytest.mark.parametrize("bad", [
    dict(D=60), dict(D=0), dict(D=264, rot=64), dict(rot=0), dict(rot=65), dict(rot=66),
    dict(T=-1), dict(H=-1), dict(Hkv=-2), dict(dt=binding.PA_F32), dict(amp=NAN), dict(amp=INF),
    dict(eps=-1.0), dict(eps=NAN), dict(q=NULL), dict(k=NULL), dict(q_out=NULL), dict(k_out=NULL),
    dict(pos=NULL), dict(table=NULL), dict(q=ODD), dict(k=ODD), dict(q_out=ODD), dict(k_out=ODD),
    dict(qw=ODD), dict(kw=ODD), dict(qs=4 * 64 + 4), dict(qs=64), dict(ks=0), dict(kos=64),
    dict(qos=-256), dict(table=ctypes.c_void_p(16 * 1024 + 4)), dict(H=2 ** 29, qs=2 ** 36)])
def test_rope_refusals(lib, bad):
    assert lib.pa_rope(*{**ROPE, **bad}.values()) == INVALID
    assert lib.pa_rope_call(rope_block({**ROPE, **bad})) == INVALID


def test_rope_without_work(lib):
    assert lib.pa_rope(*{**ROPE, "T": 0, "q": NULL, "pos": NULL}.values()) == OK
    assert lib.pa_rope(*{**ROPE, "H": 0, "Hkv": 0, "q": NULL}.values()) == OK
    for none in (dict(T=0, q=NULL), dict(H=0, Hkv=0, k=NULL)):
        assert lib.pa_rope_call(rope_block({**ROPE, **none})) == OK
    for name in ("pa_rope_call", "pa_rope_append_call", "pa_rope_append_fp8_call",
                 "pa_cross_call", "pa_decode_shared_call"):
        assert getattr(lib, name)(None) == INVALID


APPEND = dict(q_out=P, qos=4 * 64, q=P, qs=4 * 64, k=P, ks=2 * 64, v=P, vs=2 * 64, pos=P, slots=P,
              kc=P, vc=P, table=P, rot=64, il=0, amp=1.0, qw=NULL, kw=NULL, eps=1e-6, T=3, H=4,
              Hkv=2, D=64, S=16, NB=4, dt=binding.PA_F16, stream=NULL)


@pytest.mark.parametrize("bad", [
    dict(Hkv=0), dict(S=0), dict(NB=-1), dict(v=NULL), dict(v=ODD), dict(vs=64), dict(vs=132),
    dict(slots=NULL), dict(kc=NULL), dict(vc=NULL), dict(kc=ODD), dict(vc=ODD), dict(D=72, rot=80),
    dict(rot=3), dict(T=-3), dict(q=NULL), dict(dt=9)])
def test_append_refusals(lib, bad):
    args = {**APPEND, **bad}
    assert lib.pa_rope_append(*args.values()) == INVALID
    head, tail = list(args.values())[:12], list(args.values())[12:]
    assert lib.pa_rope_append_fp8(*head, 1.0, 1.0, *tail) == INVALID
    assert lib.pa_rope_append_call(rope_block(args)) == INVALID
    assert lib.pa_rope_append_fp8_call(rope_block(args)) == INVALID
    for name in ("pa_rope_append_call", "pa_rope_append_fp8_call"):  # (the block itself is good)
        assert getattr(lib, name)(rope_block({**APPEND, "T": 0})) == OK


@pytest.mark.parametrize("scales", [(0.0, 1.0), (1.0, -1.0), (NAN, 1.0), (1.0, INF), (1e-19, 1.0),
                                    (1.0, 1e19)])
def test_append_fp8_scales(lib, scales):
    v = list(APPEND.values())
    assert lib.pa_rope_append_fp8(*v[:12], *scales, *v[12:]) == INVALID
    assert lib.pa_rope_append_fp8_call(rope_block(APPEND, scales)) == INVALID
    v = list({**APPEND, "D": 72, "qs": 288, "ks": 144, "vs": 144, "qos": 288}.values())
    assert lib.pa_rope_append_fp8(*v[:12], 1.0, 1.0, *v[12:]) == INVALID  # D % 16
    v = list({**APPEND, "T": 0}.values())
    assert lib.pa_rope_append_fp8(*v[:12], 1.0, 1.0, *v[12:]) == OK


CROSS = dict(out=P, out_dt=binding.PA_F32, q=P, k=P, v=P, bt=P, MB=8, lens=P, start=P, scale=0.1,
             B=2, H=8, Hkv=4, D=128, S=16, NB=16, dt=binding.PA_BF16, T=600, max_q=300, max_kv=100,
             partition=0, ws=NULL, ws_bytes=0, stream=NULL)


@pytest.mark.parametrize("bad", [
    dict(D=96), dict(D=32), dict(S=4), dict(S=24), dict(S=256), dict(dt=binding.PA_F32),
    dict(out_dt=7), dict(H=0), dict(Hkv=0), dict(H=9), dict(H=1032, Hkv=8), dict(B=-1),
    dict(H=65536, Hkv=1024), dict(B=70000), dict(T=-1), dict(max_q=-1), dict(max_kv=-1), dict(max_kv=129), dict(MB=-1),
    dict(MB=0, max_kv=0), dict(NB=0), dict(NB=-1), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=NAN), dict(scale=INF), dict(partition=-2), dict(partition=64), dict(partition=200),
    dict(out=NULL), dict(q=NULL), dict(k=NULL), dict(v=NULL), dict(bt=NULL), dict(lens=NULL),
    dict(start=NULL), dict(q=ODD), dict(out=ODD), dict(k=ODD), dict(v=ODD),
    dict(NB=2 ** 26, Hkv=8, H=8), dict(MB=2 ** 28, max_kv=10),
    dict(MB=2 ** 27 - 1, max_kv=2 ** 31 - 16),  # no room for a whole last key tile
    dict(MB=64, max_kv=1000, partition=128),    # a split without its workspace
    dict(MB=64, max_kv=1000, partition=128, ws=P, ws_bytes=1000),
    dict(MB=64, max_kv=1000, partition=128, ws=ODD, ws_bytes=2 ** 40)])
def test_cross_refusals(lib, bad):
    assert lib.pa_cross(*{**CROSS, **bad}.values()) == INVALID
    assert lib.pa_cross_call(ranges_block({**CROSS, **bad})) == INVALID


def test_cross_without_work(lib):
    for none in (dict(B=0), dict(T=0), dict(max_q=0)):
        assert lib.pa_cross(*{**CROSS, **none, "q": NULL, "out": NULL}.values()) == OK
        assert lib.pa_cross_call(ranges_block({**CROSS, **none, "q": NULL})) == OK


def slots(n_bytes, pairs, D):
    """Result slots per (row, head) that a workspace of n_bytes was sized for."""
    for np in range(1, 4096):
        n = pairs * np
        if (n * 8 + 255) // 256 * 256 + n * D * 4 == n_bytes:
            return np
    return None


def test_cross_plan(lib):
    ws = binding.pa_cross_workspace_bytes
    # enough row tiles for every SM (148 without a device): no split
    assert ws(16, 16 * 512, 32, 32, 128, 512, 1500) == 0
    # single tokens on few heads: split, over at most the key tiles there are
    n = slots(ws(1, 1, 8, 8, 128, 1, 8192), 8, 128)
    assert 8 < n <= 64
    assert slots(ws(1, 1, 8, 8, 128, 1, 128), 8, 128) is None  # one key tile
    # a given partition is taken as it is
    assert slots(ws(2, 6, 4, 2, 64, 3, 1000, 256), 24, 64) == 4
    assert ws(2, 6, 4, 2, 64, 3, 1000, -1) == 0
    for bad in ((0, 1, 4, 4, 64, 1, 1000), (1, 1, 4, 3, 64, 1, 1000), (1, 1, 4, 4, 96, 1, 1000)):
        assert ws(*bad) == 0


SHARED = dict(out=P, out_dt=binding.PA_BF16, q=P, k=P, v=P, bt=P, MB=64, seq=P, sh=P, start=P, NG=2,
              scale=0.1, B=4, H=8, Hkv=4, D=128, S=16, NB=16, dt=binding.PA_BF16, max_group=3,
              max_shared=512, max_tail=100, ws=P, ws_bytes=2 ** 40, stream=NULL)


@pytest.mark.parametrize("bad", [
    dict(D=96), dict(S=64), dict(S=4), dict(dt=binding.PA_F32), dict(out_dt=3), dict(H=0),
    dict(Hkv=3), dict(H=1032, Hkv=8), dict(B=-1), dict(B=65535), dict(NG=-1), dict(NG=65535),
    dict(H=65536, Hkv=1024),
    dict(NG=0), dict(max_group=0), dict(max_group=-1), dict(max_shared=-1), dict(max_tail=-1),
    dict(max_shared=1025), dict(max_tail=1025), dict(MB=0, max_shared=0, max_tail=0), dict(NB=0),
    dict(scale=0.0), dict(scale=NAN), dict(out=NULL), dict(q=NULL), dict(k=NULL), dict(v=NULL),
    dict(bt=NULL), dict(seq=NULL), dict(sh=NULL), dict(start=NULL), dict(q=ODD), dict(k=ODD),
    dict(v=ODD), dict(out=ODD), dict(ws=NULL), dict(ws=ODD), dict(ws_bytes=100),
    dict(NB=2 ** 28), dict(MB=2 ** 28)])
def test_shared_refusals(lib, bad):
    assert lib.pa_decode_shared(*{**SHARED, **bad}.values()) == INVALID
    assert lib.pa_decode_shared_call(ranges_block({**SHARED, **bad})) == INVALID


def test_shared_without_work(lib):
    assert lib.pa_decode_shared(*{**SHARED, "B": 0, "NG": 0, "q": NULL, "ws": NULL,
                                  "ws_bytes": 0}.values()) == OK
    assert lib.pa_decode_shared_call(ranges_block({**SHARED, "B": 0, "NG": 0, "ws": NULL})) == OK


def test_shared_workspace(lib):
    ws = binding.pa_decode_shared_workspace_bytes
    # the shared part's slots, then the tails' (one where nothing splits them)
    tails = slots(ws(64, 1, 40, 40, 128, 16, 64, 0, 100), 64 * 40, 128)
    alone = slots(ws(64, 1, 40, 40, 128, 16, 64, 2048, 0), 64 * 40, 128)
    both = slots(ws(64, 1, 40, 40, 128, 16, 64, 2048, 100), 64 * 40, 128)
    # alone the shared part is cut to fill the SMs (3 x 40 CTAs of 148); beside tails it leaves
    # some to them
    assert (tails, alone) == (1, 3) and tails < both < tails + alone
    # 64 query heads on 8 KV heads, 512 rows: two CTAs of two row tiles per KV head and part
    assert slots(ws(64, 1, 64, 8, 128, 16, 64, 32768, 0), 64 * 64, 128) == 9
    assert ws(64, 1, 40, 40, 128, 16, 64, 0, 0) == 0
    assert ws(0, 0, 40, 40, 128, 16, 64, 2048, 100) == 0
    assert ws(4, 1, 40, 40, 96, 16, 64, 2048, 100) == 0
    # a group cannot hold more requests than the batch
    assert ws(4, 1, 8, 8, 64, 16, 10 ** 6, 2048, 9) == ws(4, 1, 8, 8, 64, 16, 4, 2048, 9)
