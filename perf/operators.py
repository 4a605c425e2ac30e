"""The serving operators around the paged cache, as cases that can be measured: rotary positions
with per-head norms, the same fused with the append to the paged cache (16-bit and E4M3), cross
attention over cached encoder states, and decode for batches that share a prefix.

``run`` computes a case in plain torch (``own`` false) or through the library (``own`` true) on the
inputs of ``prepare``; ``exact`` is the definition in 64 bits; ``work`` counts what a pass has to
read, write and compute.
"""

import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _rope(name, T, H, Hkv, D, rot, layout, norm, dtype, far=0, factor=1.0):
    return dict(name=name, op="rope", T=T, H=H, Hkv=Hkv, D=D, rot=rot, layout=layout, norm=norm,
                dtype=dtype, far=far, factor=factor)


def _append(name, T, H, Hkv, D, S, rot, layout, norm, dtype, pad=0, fp8=False, factor=1.0):
    return dict(name=name, op="append", T=T, H=H, Hkv=Hkv, D=D, S=S, rot=rot, layout=layout,
                norm=norm, dtype=dtype, pad=pad, fp8=fp8, far=0, factor=factor)


def _cross(name, B, q_lo, q_hi, kv_lo, kv_hi, H, Hkv, D, S, dtype, lens):
    return dict(name=name, op="cross", B=B, q_lo=q_lo, q_hi=q_hi, kv_lo=kv_lo, kv_hi=kv_hi, H=H,
                Hkv=Hkv, D=D, S=S, dtype=dtype, lens=lens)


def _shared(name, groups, g_lo, g_hi, pre_lo, pre_hi, tail_lo, tail_hi, H, Hkv, D, S, dtype, lens):
    return dict(name=name, op="shared", groups=groups, g_lo=g_lo, g_hi=g_hi, pre_lo=pre_lo,
                pre_hi=pre_hi, tail_lo=tail_lo, tail_hi=tail_hi, H=H, Hkv=Hkv, D=D, S=S,
                dtype=dtype, lens=lens)


def listed():
    return [
        # one new token of one request, queries and keys normed and rotated: pure latency
        _rope("rope_one_token", 1, 32, 32, 128, 128, "half", True, "bf16"),
        # a long prompt at far positions, half of each head rotated, pairs side by side
        _rope("rope_prompt_partial", 20011, 32, 8, 64, 32, "pairs", False, "fp16", far=1000000,
              factor=8.0),
        # a decode step of 64 requests on 40 heads: one token each into the cache
        _append("append_step", 64, 40, 40, 128, 16, 128, "half", True, "bf16"),
        # the prompts of a serving step, 64 query heads on 8 KV heads, the last rows padding
        _append("append_prompts_grouped", 32003, 64, 8, 128, 16, 128, "half", True, "bf16", pad=29),
        # prompts of 32 heads into an E4M3 cache
        _append("append_prompts_e4m3", 12289, 32, 32, 128, 16, 128, "pairs", False, "bf16",
                fp8=True),
        # a decoder's single tokens over encoder states of some 1,500 rows
        _cross("cross_step", 8, 1, 1, 700, 1500, 20, 20, 64, 16, "fp16", 1),
        # decoder prompts over encoder states, ragged on both sides
        _cross("cross_prompts", 16, 30, 447, 200, 1500, 32, 32, 64, 16, "bf16", 2),
        # long decoder inputs over long encoder states, grouped heads: the tensor cores' case
        _cross("cross_long", 4, 1501, 2048, 6000, 8192, 32, 8, 128, 16, "bf16", 3),
        # the four continuations of one prompt, 32 heads: latency
        _shared("shared_four", 1, 4, 4, 1328, 1328, 1, 40, 32, 32, 128, 16, "bf16", 4),
        # a batch of 64 behind one system prompt on 40 heads
        _shared("shared_batch", 1, 64, 64, 2048, 2048, 1, 512, 40, 40, 128, 16, "bf16", 5),
        # eight documents, each asked several questions, head size 64
        _shared("shared_documents", 8, 3, 17, 1000, 4096, 5, 300, 32, 32, 64, 16, "fp16", 6),
        # a long shared context on 64 query heads over 8 KV heads
        _shared("shared_long_grouped", 1, 64, 64, 32768, 32768, 1, 2048, 64, 8, 128, 16, "bf16", 7),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "cross", "shared"])
    dtype = rng.choice(["bf16", "fp16"])
    D = rng.choice([64, 128])
    S = rng.choice([8, 16, 32])
    if op in ("rope", "append"):
        Hkv = rng.choice([4, 8, 32, 40])
        H = Hkv * rng.choice([1, 4, 8]) if Hkv <= 8 else Hkv
        rot = rng.choice([D, D, D // 2])
        layout = rng.choice(["half", "pairs"])
        norm = rng.random() < 0.5
        factor = rng.choice([1.0, 4.0])
        T = _log_int(rng, 1, 24000 if H <= 32 else 12000)
        if op == "rope":
            c = _rope("", T, H, Hkv, D, rot, layout, norm, dtype,
                      far=rng.choice([0, 100000]), factor=factor)
        else:
            c = _append("", T, H, Hkv, D, S, rot, layout, norm, dtype,
                        pad=min(rng.choice([0, 3, 17]), T - 1), fp8=rng.random() < 0.3,
                        factor=factor)
    elif op == "cross":
        B = _log_int(rng, 1, 16)
        Hkv = rng.choice([4, 8, 20, 32])
        H = Hkv * rng.choice([1, 4]) if Hkv <= 8 else Hkv
        q_hi = _log_int(rng, 1, 1024)
        kv_hi = _log_int(rng, 16, 4096)
        c = _cross("", B, max(1, q_hi // 2), q_hi, max(1, kv_hi // 3), kv_hi, H, Hkv, D, S, dtype,
                   rng.randrange(1 << 20))
    else:
        groups = _log_int(rng, 1, 8)
        Hkv = rng.choice([4, 8, 32, 40])
        H = Hkv * rng.choice([2, 5, 8]) if Hkv <= 8 else Hkv
        g_hi = _log_int(rng, 1, 64 // groups + 1)
        pre_hi = _log_int(rng, 64, 6000)
        tail_hi = _log_int(rng, 1, 600)
        c = _shared("", groups, max(1, g_hi // 3), g_hi, pre_hi // 2, pre_hi,
                    max(1, tail_hi // 4), tail_hi, H, Hkv, D, S, dtype, rng.randrange(1 << 20))
    del c["name"]
    return c


def _lengths(case):
    """The lengths of an attention case: drawn from the case alone, so that work() knows them."""
    rng = random.Random(case["lens"])
    if case["op"] == "cross":
        return ([rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["B"])],
                [rng.randint(case["kv_lo"], case["kv_hi"]) for _ in range(case["B"])])
    S = case["S"]
    sizes = [rng.randint(case["g_lo"], case["g_hi"]) for _ in range(case["groups"])]
    shared = [rng.randint(case["pre_lo"], case["pre_hi"]) // S * S for _ in sizes]
    tails = [[rng.randint(case["tail_lo"], case["tail_hi"]) for _ in range(n)] for n in sizes]
    return sizes, shared, tails


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _frequencies(case):
    """Turns per position of each pair (64 bits): base 10000, positions scaled by 1 / factor."""
    j = torch.arange(case["rot"] // 2, dtype=torch.float64)
    return 10000.0 ** (-2.0 * j / case["rot"]) / case["factor"] / (2.0 * math.pi)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    host = torch.Generator().manual_seed(int(seed))
    dt = _DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    s = dict(case=dict(case))
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    if case["op"] in ("rope", "append"):
        T = case["T"]
        s["table"] = _frequencies(case).to(dev)
        # what a fused projection leaves: queries, keys and values of a token side by side
        s["qkv"] = normal(T, H + 2 * Hkv, D)
        start = case["far"] + int(torch.randint(0, 4096, (1,), generator=host))
        s["positions"] = torch.arange(start, start + T, dtype=torch.int32, device=dev)
        s["q_weight"] = (1 + 0.1 * torch.randn(D, generator=g, device=dev)).to(dt) \
            if case["norm"] else None
        s["k_weight"] = (1 + 0.1 * torch.randn(D, generator=g, device=dev)).to(dt) \
            if case["norm"] else None
        s["q_out"] = torch.empty((T, H, D), dtype=dt, device=dev)
        if case["op"] == "rope":
            s["k_out"] = torch.empty((T, Hkv, D), dtype=dt, device=dev)
            return s
        S = case["S"]
        NB = -(-T // S) + 2
        perm = torch.randperm(NB, generator=host)
        t = torch.arange(T)
        slots = perm[t // S] * S + t % S
        if case["pad"]:
            slots[T - case["pad"]:] = -1
        s["slots"] = slots.to(torch.int64).to(dev)
        shape = (NB, Hkv, S, D)
        s["k_cache"], s["v_cache"] = normal(*shape), normal(*shape)
        if case["fp8"]:
            s["k_cache"] = s["k_cache"].to(torch.float8_e4m3fn).view(torch.uint8)
            s["v_cache"] = s["v_cache"].to(torch.float8_e4m3fn).view(torch.uint8)
            s["k_scale"], s["v_scale"] = 0.03125, 0.0234375
        return s

    S = case["S"]
    if case["op"] == "cross":
        q_lens, lens = _lengths(case)
        B = case["B"]
        starts = [0]
        for n in q_lens:
            starts.append(starts[-1] + n)
        s["T"], s["max_q"], s["max_kv"] = starts[-1], max(q_lens), max(lens)
        s["q_start"] = torch.tensor(starts, dtype=torch.int32, device=dev)
        owned = lens
        named = [(0, -1)] * B
        s["q"] = normal(s["T"], H, D)
    else:
        sizes, shared, tails = _lengths(case)
        starts, lens, named, owned = [0], [], [], []
        for j, n in enumerate(sizes):
            starts.append(starts[-1] + n)
            for k in range(n):
                lens.append(shared[j] + tails[j][k])
                named.append((shared[j] // S, j))
                owned.append(tails[j][k])
        B = len(lens)
        s["max_group"], s["max_shared"] = max(sizes), max(shared)
        s["max_tail"] = max(owned)
        s["group_start"] = torch.tensor(starts, dtype=torch.int32, device=dev)
        s["shared_lens"] = torch.tensor([shared[j] for _, j in named], dtype=torch.int32,
                                        device=dev)
        s["q"] = normal(B, H, D)
    # physical blocks in a random order; the blocks of a shared prefix are named by every table
    prefix_blocks = [p // S for p in shared] if case["op"] == "shared" else []
    need = sum(prefix_blocks) + sum(-(-n // S) for n in owned)
    perm = torch.randperm(need, generator=host).to(torch.int32)
    MB = max(-(-n // S) for n in lens)
    tables = torch.full((B, MB), -1, dtype=torch.int32)
    at, firsts = 0, []
    for n in prefix_blocks:
        firsts.append(at)
        at += n
    for i in range(B):
        n0, j = named[i]
        if n0:
            tables[i, :n0] = perm[firsts[j]:firsts[j] + n0]
        n1 = -(-owned[i] // S)
        tables[i, n0:n0 + n1] = perm[at:at + n1]
        at += n1
    s["block_tables"] = tables.to(dev)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["k_cache"], s["v_cache"] = normal(need, Hkv, S, D), normal(need, Hkv, S, D)
    s["out"] = torch.empty_like(s["q"])
    s["scale"] = 1.0 / math.sqrt(D)
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _norm_rotate(x, weight, turns, rot, layout):
    """x [T, heads, D] in 32 bits: normed per head (where there is a weight), the first `rot`
    elements rotated by `turns` [T, rot / 2] (64 bits: positions may be far)."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
    angle = 2.0 * math.pi * (turns - torch.round(turns))
    c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    r, rest = x[..., :rot], x[..., rot:]
    if layout == "half":
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * c - b * s, b * c + a * s), -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    return torch.cat((r, rest), -1)


def _plain_rope(s):
    c = s["case"]
    H, Hkv = c["H"], c["Hkv"]
    q, k, v = s["qkv"].split((H, Hkv, Hkv), 1)
    turns = s["positions"].double()[:, None] * s["table"]
    q = _norm_rotate(q, s["q_weight"], turns, c["rot"], c["layout"])
    k = _norm_rotate(k, s["k_weight"], turns, c["rot"], c["layout"])
    dt = s["qkv"].dtype
    if c["op"] == "rope":
        return {"q": q.to(dt), "k": k.to(dt)}
    S = c["S"]
    live = s["slots"] >= 0
    slots = s["slots"][live]
    blk, off = slots // S, slots % S
    k, v = k[live], v[live]
    if c["fp8"]:
        k = (k / s["k_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (v.float() / s["v_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    s["k_cache"][blk, :, off] = k.to(s["k_cache"].dtype)
    s["v_cache"][blk, :, off] = v
    return _with_caches(s, q.to(dt))


def _with_caches(s, q):
    k, v = s["k_cache"], s["v_cache"]
    if s["case"]["fp8"]:
        k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
    return {"q": q, "k_cache": k, "v_cache": v}


def _gather(cache, tables, lens):
    """Rows of the tables' blocks as [n, Hkv, tokens, D] in 32 bits, zero past each length."""
    n, MB = tables.shape
    _, Hkv, S, D = cache.shape
    x = cache[tables.clamp(min=0).long()].float()
    x = x.permute(0, 2, 1, 3, 4).reshape(n, Hkv, MB * S, D)
    live = torch.arange(MB * S, device=cache.device) < lens[:, None]
    return torch.where(live[:, None, :, None], x, 0.0), live


def _plain_cross(s):
    c = s["case"]
    B, H, Hkv, D = c["B"], c["H"], c["Hkv"], c["D"]
    K, live = _gather(s["k_cache"], s["block_tables"], s["seq_lens"])
    V, _ = _gather(s["v_cache"], s["block_tables"], s["seq_lens"])
    t = torch.arange(s["max_q"], device=K.device)
    n = s["q_start"][1:] - s["q_start"][:-1]
    row = (s["q_start"][:-1, None] + t).clamp(max=s["T"] - 1).long()
    q = s["q"][row].float().permute(0, 2, 1, 3).reshape(B, Hkv, -1, D)  # a group's heads share K
    x = q @ K.transpose(-1, -2) * s["scale"]
    x = x.masked_fill(~live[:, None, None], -math.inf)
    w = torch.exp(x - x.amax(-1, keepdim=True))
    o = (w @ V / w.sum(-1, keepdim=True)).reshape(B, H, -1, D).permute(0, 2, 1, 3)
    return o[t < n[:, None]].to(s["q"].dtype)


def _plain_shared(s):
    c = s["case"]
    H, Hkv, D, S = c["H"], c["Hkv"], c["D"], c["S"]
    B, G, NG = s["q"].shape[0], H // Hkv, c["groups"]
    dev = s["q"].device
    first = s["group_start"][:-1].long()
    group = torch.searchsorted(s["group_start"][1:].contiguous(),
                               torch.arange(B, device=dev, dtype=torch.int32), right=True)
    place = torch.arange(B, device=dev) - first[group]
    # the prefixes, once for each group
    tables = s["block_tables"][first][:, :max(1, s["max_shared"] // S)]
    plen = s["shared_lens"][first]
    K, live = _gather(s["k_cache"], tables, plen)
    V, _ = _gather(s["v_cache"], tables, plen)
    q = s["q"].float().reshape(B, Hkv, G, D)
    qg = torch.zeros((NG, s["max_group"], Hkv, G, D), device=dev)
    qg[group, place] = q
    x = (qg.permute(0, 2, 1, 3, 4).reshape(NG, Hkv, -1, D) @ K.transpose(-1, -2)) * s["scale"]
    x = x.masked_fill(~live[:, None, None], -math.inf)
    x = x.reshape(NG, Hkv, s["max_group"], G, -1).permute(0, 2, 1, 3, 4)[group, place]
    # the tails, one for each request
    nb = -(-s["max_tail"] // S)
    at = (s["shared_lens"] // S)[:, None] + torch.arange(nb, device=dev)
    tables = s["block_tables"].gather(1, at.clamp(max=s["block_tables"].shape[1] - 1).long())
    Kt, live_t = _gather(s["k_cache"], tables, s["seq_lens"] - s["shared_lens"])
    Vt, _ = _gather(s["v_cache"], tables, s["seq_lens"] - s["shared_lens"])
    y = (q @ Kt.transpose(-1, -2)) * s["scale"]
    y = y.masked_fill(~live_t[:, None, None], -math.inf)
    m = torch.maximum(x.amax(-1, keepdim=True), y.amax(-1, keepdim=True))
    x, y = torch.exp(x - m), torch.exp(y - m)
    xg = torch.zeros((NG, s["max_group"], Hkv, G, x.shape[-1]), device=dev)
    xg[group, place] = x
    o = xg.permute(0, 2, 1, 3, 4).reshape(NG, Hkv, -1, x.shape[-1]) @ V
    o = o.reshape(NG, Hkv, s["max_group"], G, D).permute(0, 2, 1, 3, 4)[group, place]
    o = (o + y @ Vt) / (x.sum(-1, keepdim=True) + y.sum(-1, keepdim=True))
    return o.reshape(B, H, D).to(s["q"].dtype)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _own(s):
    import paged_kv_cache_driven_b200 as pa

    c = s["case"]
    H, Hkv, D = c["H"], c["Hkv"], c["D"]
    if c["op"] in ("rope", "append"):
        q, k, v = s["qkv"].split((H, Hkv, Hkv), 1)
        how = dict(interleaved=c["layout"] == "pairs", q_weight=s["q_weight"],
                   k_weight=s["k_weight"], eps=1e-6)
        if c["op"] == "rope":
            pa.pa_rope(s["q_out"], s["k_out"], q, k, s["positions"], s["table"], **how)
            return {"q": s["q_out"], "k": s["k_out"]}
        if c["fp8"]:
            pa.pa_rope_append_fp8(s["q_out"], q, k, v, s["positions"], s["slots"], s["k_cache"],
                                  s["v_cache"], s["k_scale"], s["v_scale"], s["table"], **how)
        else:
            pa.pa_rope_append(s["q_out"], q, k, v, s["positions"], s["slots"], s["k_cache"],
                              s["v_cache"], s["table"], **how)
        return _with_caches(s, s["q_out"])
    if c["op"] == "cross":
        if "workspace" not in s:  # a program keeps it from call to call
            n = pa.pa_cross_workspace_bytes(c["B"], s["T"], H, Hkv, D, s["max_q"], s["max_kv"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
        pa.pa_cross(s["out"], s["q"], s["k_cache"], s["v_cache"], s["block_tables"],
                    s["seq_lens"], s["q_start"], s["scale"], s["max_q"], s["max_kv"],
                    workspace=s["workspace"])
        return s["out"]
    if "workspace" not in s:
        n = pa.pa_decode_shared_workspace_bytes(s["q"].shape[0], c["groups"], H, Hkv, D, c["S"],
                                                s["max_group"], s["max_shared"], s["max_tail"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    pa.pa_decode_shared(s["out"], s["q"], s["k_cache"], s["v_cache"], s["block_tables"],
                        s["seq_lens"], s["shared_lens"], s["group_start"], s["scale"],
                        s["max_group"], s["max_shared"], s["max_tail"], workspace=s["workspace"])
    return s["out"]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "cross":
        return _plain_cross(state)
    if op == "shared":
        return _plain_shared(state)
    return _plain_rope(state)


# ---------------------------------------------------------------------------
# the definition in 64 bits, and the work
# ---------------------------------------------------------------------------

def _exact_rows(x, weight, positions, freq, rot, layout):
    x = x.double()
    if weight is not None:
        x = x / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * weight.double()
    out = x.clone()
    angle = torch.outer(positions.double(), freq * 2 * math.pi)
    z = torch.polar(torch.ones_like(angle), angle)[:, None]
    first = slice(0, rot // 2) if layout == "half" else slice(0, rot, 2)
    second = slice(rot // 2, rot) if layout == "half" else slice(1, rot, 2)
    turned = torch.complex(x[..., first], x[..., second]) * z
    out[..., first], out[..., second] = turned.real, turned.imag
    return out


def _exact_attention(q, K, V, scale):
    """q [rows, H, D] over K, V [tokens, Hkv, D]."""
    G = q.shape[1] // K.shape[1]
    K, V = K.repeat_interleave(G, 1), V.repeat_interleave(G, 1)
    w = torch.softmax(torch.einsum("rhd,thd->hrt", q, K) * scale, -1)
    return torch.einsum("hrt,thd->rhd", w, V)


def exact(case, seed):
    s = prepare(case, seed)
    H, Hkv = case["H"], case["Hkv"]
    if case["op"] in ("rope", "append"):
        freq = _frequencies(case).to("cuda")
        how = (s["positions"], freq, case["rot"], case["layout"])
        q = _exact_rows(s["qkv"][:, :H], s["q_weight"], *how)
        k = _exact_rows(s["qkv"][:, H:H + Hkv], s["k_weight"], *how)
        if case["op"] == "rope":
            return {"q": q, "k": k}
        caches = [s["k_cache"], s["v_cache"]]
        rows = [k, s["qkv"][:, H + Hkv:].double()]
        if case["fp8"]:  # the stored value before it is rounded to eight bits
            caches = [x.view(torch.float8_e4m3fn) for x in caches]
            rows = [(r / sc).clamp(-448, 448) for r, sc in zip(rows, (s["k_scale"], s["v_scale"]))]
        caches = [x.double() for x in caches]
        used = torch.nonzero(s["slots"] >= 0).flatten()
        where = s["slots"][used]
        for cache, r in zip(caches, rows):
            cache[where // case["S"], :, where % case["S"]] = r[used]
        return {"q": q, "k_cache": caches[0], "v_cache": caches[1]}
    tables, lens = s["block_tables"], s["seq_lens"].tolist()

    def rows_of(cache, i):
        S = case["S"]
        n = lens[i]
        x = cache[tables[i, :-(-n // S)].long()].double()
        return x.transpose(1, 2).reshape(-1, Hkv, case["D"])[:n]

    out = []
    starts = s["q_start"].tolist() if case["op"] == "cross" else list(range(len(lens) + 1))
    for i in range(len(lens)):
        out.append(_exact_attention(s["q"][starts[i]:starts[i + 1]].double(),
                                    rows_of(s["k_cache"], i), rows_of(s["v_cache"], i),
                                    s["scale"]))
    return torch.cat(out)


def work(case):
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    if case["op"] in ("rope", "append"):
        T = case["T"]
        heads = T * (H + Hkv) * D
        flops = heads * (3 if case["rot"] == D else 2) + (4 * heads if case["norm"] else 0)
        moved = 2 * 2 * heads + 4 * T + 8 * (case["rot"] // 2)
        if case["op"] == "append":
            live = T - case["pad"]
            rows = live * Hkv * D
            moved = (2 * T * H * D * 2 + 2 * rows * 2 + 2 * rows * (1 if case["fp8"] else 2)
                     + 12 * T + 8 * (case["rot"] // 2))
        return {"bytes": moved, "flops": flops}
    if case["op"] == "cross":
        q_lens, lens = _lengths(case)
        tokens, pairs, rows = sum(lens), sum(a * b for a, b in zip(q_lens, lens)), sum(q_lens)
    else:
        sizes, shared, tails = _lengths(case)
        rows = sum(sizes)
        own_tokens = sum(sum(t) for t in tails)
        tokens = sum(shared) + own_tokens
        pairs = sum(n * p for n, p in zip(sizes, shared)) + own_tokens
    return {"bytes": 4 * tokens * Hkv * D + 4 * rows * H * D, "flops": 4 * pairs * H * D}
