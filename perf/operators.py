"""Operators around the packed KV cache, as measured cases: their inputs, a plain form in elementary torch operations,
the calls a user makes of the library, and their definition in 64 bits.

  norm_rope  RMS norm of every query and key head with the position rotation in the same pass (one or three position axes)
  extend     attention of n new query tokens per sequence over a packed cache, causal among the new tokens
  bounds     per 64-token block and KV head the channelwise minimum and maximum of the dequantised, rotated keys
  sparse     decode over the blocks that an upper bound from those minima and maxima selects: selection and attention
"""
from __future__ import annotations

import functools
import math

import numpy as np
import torch

own = False

D = 128          # head dimension of the library
BLOCK = 64       # tokens of a block that has bounds
GROUP = 32       # channels of a value group
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding step of a batch of eight long conversations: latency counts
        dict(name="norm_rope step", op="norm_rope", batch=8, tokens=1, hq=28, hk=4, dtype="bf16", axes=1, far=32768,
             interleaved=False, rot=128, weights=True),
        # a prompt's chunk of the largest head layout
        dict(name="norm_rope prompt", op="norm_rope", batch=1, tokens=8192, hq=64, hk=8, dtype="bf16", axes=1, far=131072,
             interleaved=False, rot=128, weights=True),
        # images and video: positions in time, height and width, an odd number of tokens
        dict(name="norm_rope three axes", op="norm_rope", batch=3, tokens=1777, hq=12, hk=2, dtype="f16", axes=3, far=4096,
             interleaved=True, rot=128, weights=True),
        # a short conversation's step: the smallest call
        dict(name="extend short", op="extend", batch=1, tokens=1, hq=12, hkv=2, length=333, ragged=False, mode="prod", bits=3,
             vbits=2, dtype="bf16"),
        # one token over the longest context
        dict(name="extend stream", op="extend", batch=1, tokens=1, hq=64, hkv=8, length=131072, ragged=False, mode="prod",
             bits=4, vbits=4, dtype="bf16"),
        # checking five drafted tokens for each of eight sequences of their own lengths
        dict(name="extend verify", op="extend", batch=8, tokens=5, hq=28, hkv=4, length=32768, ragged=True, mode="prod", bits=3,
             vbits=2, dtype="bf16"),
        # a chunk of a long prompt
        dict(name="extend chunk", op="extend", batch=1, tokens=2048, hq=28, hkv=4, length=16384, ragged=False, mode="mse",
             bits=4, vbits=4, dtype="bf16"),
        # first chunks of three prompts, nothing cached before them, odd lengths, two key groups
        dict(name="extend first", op="extend", batch=3, tokens=999, hq=12, hkv=2, length=999, ragged=False, mode="grouped",
             bits=3, vbits=4, dtype="f16"),
        # a step over the longest context that reads a sixteenth of it
        dict(name="sparse stream", op="sparse", batch=1, hq=64, hkv=8, length=131072, ragged=False, mode="prod", bits=4, vbits=4,
             dtype="bf16", select=128, sink=1, recent=4),
        # a step of eight sequences of their own lengths
        dict(name="sparse batch", op="sparse", batch=8, hq=28, hkv=4, length=32768, ragged=True, mode="prod", bits=3, vbits=2,
             dtype="bf16", select=48, sink=1, recent=2),
        # bounds of whole prompts, once written
        dict(name="bounds prompt", op="bounds", batch=8, hkv=4, length=32768, ragged=True, mode="prod", bits=3, tokens=32768),
        # bounds after one more token of each sequence
        dict(name="bounds step", op="bounds", batch=8, hkv=4, length=32768, ragged=True, mode="mse", bits=4, tokens=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    return rng.choice([(12, 2), (28, 4), (64, 8), (8, 8), (5, 1), (6, 3)])


def _keys(rng):
    mode = rng.choice(["mse", "prod", "grouped"])
    return mode, rng.randint(*{"mse": (1, 4), "prod": (2, 4), "grouped": (1, 3)}[mode])


def draw(rng):
    op = rng.choice(["norm_rope", "extend", "extend", "sparse", "bounds"])
    hq, hkv = _heads(rng)
    mode, bits = _keys(rng)
    dtype = rng.choice(["bf16", "f16"])
    if op == "norm_rope":
        tokens = _log(rng, 1, 8000)
        return dict(op=op, batch=max(1, min(rng.randint(1, 8), 8000 // tokens)), tokens=tokens, hq=hq, hk=hkv,
                    dtype=rng.choice(["bf16", "f16", "f32"]), axes=rng.choice([1, 2, 3]), far=_log(rng, 100, 1000000),
                    interleaved=rng.random() < 0.5, rot=rng.choice([128, 128, 64, 96]), weights=rng.random() < 0.8)
    length = _log(rng, 1, 60000)
    batch = max(1, min(rng.randint(1, 8), 900000 // (length * hkv)))
    if op == "extend":
        most = max(1, min(length, 300_000_000 // (batch * hq * length)))
        return dict(op=op, batch=batch, tokens=min(2048, _log(rng, 1, most)), hq=hq, hkv=hkv, length=length,
                    ragged=rng.random() < 0.5, mode=mode, bits=bits, vbits=rng.choice([2, 4]), dtype=dtype)
    if op == "sparse":
        sink, recent = rng.randint(0, 2), rng.randint(1, 4)
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, length=length, ragged=rng.random() < 0.5, mode=mode, bits=bits,
                    vbits=rng.choice([2, 4]), dtype=dtype, select=sink + recent + _log(rng, 1, 200), sink=sink, recent=recent)
    return dict(op=op, batch=batch, hkv=hkv, length=length, ragged=rng.random() < 0.5, mode=mode, bits=bits,
                tokens=min(length, _log(rng, 1, length)))


# ------------------------------------------------------------------------------------------- tables of a quantizer

def _splitmix(seed, tag, n):
    """n outputs of SplitMix64 on the stream `tag` of a quantizer's seed, as Python integers."""
    mask, state, got = (1 << 64) - 1, seed ^ (tag << 56), []
    for _ in range(n):
        state = (state + 0x9E3779B97F4A7C15) & mask
        z = ((state ^ (state >> 30)) * 0xBF58476D1CE4E5B9) & mask
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & mask
        got.append(z ^ (z >> 31))
    return got


def _signs(seed, tag, n):
    return [-1.0 if z >> 63 else 1.0 for z in _splitmix(seed, tag, n)]


@functools.lru_cache(None)
def _levels(bits):
    """The levels of the Lloyd-Max quantizer of N(0,1), ascending, by the fixed point level = mean of its cell."""
    phi = lambda x: math.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)   # noqa: E731
    tail = lambda x: 0.5 * math.erfc(x / math.sqrt(2))                # noqa: E731
    half = 1 << (bits - 1)
    c = [(k + 0.5) * 3 / half for k in range(half)]
    moved = 1.0
    while moved >= 1e-14:
        t = [0.0] + [(a + b) / 2 for a, b in zip(c, c[1:])]
        mass = [(phi(t[k]) - (phi(t[k + 1]) if k + 1 < half else 0.0)) / (tail(t[k]) - (tail(t[k + 1]) if k + 1 < half else 0.0))
                for k in range(half)]
        moved = max(abs(a - b) for a, b in zip(mass, c))
        c = mass
    return [-x for x in reversed(c)] + c


def _width(bits):
    return 4 if bits == 3 else bits


@functools.lru_cache(None)
def _hadamard(n):
    i = np.arange(n)
    ones = np.array([bin(x).count("1") for x in range(n)])
    return 1.0 - 2.0 * (ones[i[:, None] & i[None, :]] & 1)


OUTLIERS = tuple(range(1, D, 4))   # the outlier channels of a grouped quantizer
SEED = 7                           # the quantizer's seed (that of its layer)


@functools.lru_cache(None)
def _tables(mode, bits):
    """Groups of channels (channels, code bits, rotation matrix in 64 bits) and, for prod, the sketch matrix."""
    if mode == "grouped":
        rest = tuple(c for c in range(D) if c not in OUTLIERS)
        parts = []
        for channels, b, tag in ((OUTLIERS, bits + 1, 3), (rest, bits, 4)):
            n = len(channels)
            m = np.kron(np.eye(n // 32), _hadamard(32)) / math.sqrt(32) * np.array(_signs(SEED, tag, n))
            parts.append((channels, b, m))
        return parts, None
    m = _hadamard(D) / math.sqrt(D) * np.array(_signs(SEED, 1, D))
    sketch = None
    if mode == "prod":
        z = _splitmix(SEED, 2, 2 * D * D)
        sketch = np.array([math.sqrt(-2 * math.log(((a >> 11) + 1) * 2.0 ** -53)) * math.cos(2 * math.pi * ((b >> 11) * 2.0 ** -53))
                           for a, b in zip(z[0::2], z[1::2])]).astype(np.float16).astype(np.float64).reshape(D, D)
    return [(tuple(range(D)), bits - 1 if mode == "prod" else bits, m)], sketch


@functools.lru_cache(None)
def _on_gpu(mode, bits, dtype):
    """The same on the GPU: [(channels, code bits, levels / sqrt(channels), rotation)], sketch."""
    parts, sketch = _tables(mode, bits)
    t = lambda x: torch.tensor(x, dtype=torch.float64, device="cuda").to(dtype)   # noqa: E731
    got = [(torch.tensor(c, device="cuda"), b, t([v / math.sqrt(len(c)) for v in _levels(b)]), t(m)) for c, b, m in parts]
    return got, None if sketch is None else t(sketch)


@functools.lru_cache(None)
def _quantizer(mode, bits):
    """The library's quantizer: a program builds one per layer and keeps it."""
    import kv_cache_vector_fwht_b200 as tq
    return tq.tq_build_codebook(D, bits, mode, SEED, list(OUTLIERS) if mode == "grouped" else None)


# ---------------------------------------------------------------------------------------------------- the inputs

def _pack(codes, width):
    per = 8 // width
    c = codes.view(codes.shape[0], -1, per)
    got = c[..., 0].clone()
    for f in range(1, per):
        got |= c[..., f] << (f * width)
    return got


def _lengths(case, seed):
    if not case["ragged"]:
        return [case["length"]] * case["batch"]
    r = np.random.default_rng(seed + 17)
    return [case["length"]] + [int(x) for x in r.integers(max(1, case["length"] // 4), case["length"] + 1, case["batch"] - 1)]


def _cache(case, seed, g):
    """Planes of a packed cache whose keys and values are Gaussian rows of norms a factor of four apart, as quantising writes
    them: level codes of unit Gaussian coordinates, 16-bit norms, random sketch signs, values rounded per group."""
    capacity = (case["length"] + 15) // 16 * 16 + 16
    rows = case["batch"] * case["hkv"] * capacity
    parts, sketch = _tables(case["mode"], case["bits"])
    idx, lost = [], 0.0
    for channels, b, _ in parts:
        lv = torch.tensor(_levels(b), device="cuda", dtype=torch.float32)
        u = torch.randn(rows, len(channels), generator=g, device="cuda")
        codes = torch.bucketize(u, (lv[1:] + lv[:-1]) / 2, out_int32=True)
        lost = ((u - lv[codes]) ** 2).mean().sqrt()   # the residual's size for a unit coordinate
        idx.append(_pack(codes.to(torch.uint8), _width(b)))
        del u, codes
    norm = math.sqrt(D) * (0.5 + 1.5 * torch.rand(rows, 1, generator=g, device="cuda"))
    norms = norm if case["mode"] == "mse" else torch.cat([norm, norm * lost * (0.9 + 0.2 * torch.rand(rows, 1, generator=g, device="cuda"))], 1) \
        if case["mode"] == "prod" else torch.cat([norm, 1.3 * norm.flip(0)], 1)
    s = dict(capacity=capacity, lengths=_lengths(case, seed), k_idx=torch.cat(idx, 1), k_norms=norms.half(), k_signs=None,
             mode=case["mode"], bits=case["bits"], batch=case["batch"], hkv=case["hkv"])
    if sketch is not None:
        s["k_signs"] = torch.randint(0, 256, (rows, D // 8), generator=g, device="cuda", dtype=torch.uint8)
    if "vbits" in case:
        top = (1 << case["vbits"]) - 1
        v = torch.randn(rows, D // GROUP, GROUP, generator=g, device="cuda")
        low = v.amin(2)
        step = ((v.amax(2) - low) / top).half()
        low = low.half()
        codes = ((v - low[..., None].float()) / step[..., None].float()).round().clamp(0, top).to(torch.uint8)
        s.update(vbits=case["vbits"], v_q=_pack(codes.view(rows, D), case["vbits"]), v_params=torch.stack([low, step], 2))
    return s


def _handle(s):
    """The library's cache with these planes."""
    import kv_cache_vector_fwht_b200 as tq
    q = _quantizer(s["mode"], s["bits"])
    c = tq.KVCache(q, s["batch"], s["hkv"], s["capacity"], value_bits=s.get("vbits", 0))
    for name in ("k_idx", "k_signs", "k_norms", "v_q", "v_params"):
        if s.get(name) is not None:
            plane = getattr(c, name)
            plane.copy_(s[name].view(plane.dtype))
            s[name] = plane.view(s[name].dtype)
    c.set_lengths(s["lengths"])
    return q, c


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    if case["op"] == "norm_rope":
        B, n, hq, hk = case["batch"], case["tokens"], case["hq"], case["hk"]
        dt = DTYPES[case["dtype"]]
        # the projection's output: queries, keys and values of a token side by side
        x = (2 * torch.randn(B, n, (hq + 2 * hk) * D, generator=g, device="cuda")).to(dt)
        pairs = case["rot"] // 2
        start = torch.randint(0, max(1, case["far"] - n), (case["axes"], B, 1), generator=g, device="cuda", dtype=torch.int32)
        spread = torch.randint(0, n, (case["axes"], B, n), generator=g, device="cuda", dtype=torch.int32)
        pos = start + (torch.arange(n, device="cuda", dtype=torch.int32) if case["axes"] == 1 else spread)
        s = dict(op="norm_rope", pos=pos.contiguous(), eps=1e-6, interleaved=case["interleaved"],
                 inv_freq=(1e6 ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs)).float(),
                 axis_of_freq=[i * case["axes"] // pairs for i in range(pairs)],
                 q=x[..., :hq * D].view(B, n, hq, D).transpose(1, 2), k=x[..., hq * D:(hq + hk) * D].view(B, n, hk, D).transpose(1, 2),
                 wq=None, wk=None)
        if case["weights"]:
            s["wq"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
            s["wk"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
        if own:   # the step's output buffers
            s["q_out"], s["k_out"] = torch.empty((B, hq, n, D), dtype=dt, device="cuda"), torch.empty((B, hk, n, D), dtype=dt, device="cuda")
        return s
    s = _cache(case, seed, g)
    s["op"] = case["op"]
    blocks = -(-s["capacity"] // BLOCK)
    if case["op"] == "bounds":
        s["tokens"] = case["tokens"]
        s["bounds"] = torch.zeros(case["batch"], case["hkv"], blocks, 2, D, dtype=torch.float16, device="cuda")
    else:
        shape = (case["batch"], case["hq"], case["tokens"], D) if case["op"] == "extend" else (case["batch"], case["hq"], D)
        s["query"] = (2 * torch.randn(shape, generator=g, device="cuda")).to(DTYPES[case["dtype"]])
    if case["op"] == "sparse":
        s.update(select=case["select"], sink=case["sink"], recent=case["recent"])
        # bounds as a block's 64 Gaussian coordinates have them, around a mean of their own
        mid = 0.6 * torch.randn(case["batch"], case["hkv"], blocks, 1, D, generator=g, device="cuda")
        wide = 1.5 + 1.5 * torch.rand(case["batch"], case["hkv"], blocks, 2, D, generator=g, device="cuda")
        s["bounds"] = (mid + wide * torch.tensor([[-1.0], [1.0]], device="cuda")).half()
    if own:   # the layer's quantizer and cache, the program's workspace and output buffers
        import kv_cache_vector_fwht_b200 as tq
        s["quantizer"], s["cache"] = _handle(s)
        if case["op"] != "bounds":
            s["out"] = torch.empty_like(s["query"])
        if case["op"] == "extend":
            s["workspace"] = tq.alloc_extend_workspace(s["cache"], case["hq"], case["tokens"])
        if case["op"] == "sparse":
            s["workspace"] = tq.alloc_blocks_workspace(s["cache"], case["hq"], case["select"])
            s["ids"] = torch.empty((case["batch"], case["hkv"], case["select"]), dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------- the plain forms

def _unpack(packed, width):
    per = 8 // width
    f = [(packed >> (width * i)) & ((1 << width) - 1) for i in range(per)]
    return torch.stack(f, -1).flatten(-2)


def _rotated_keys(s, idx, norms):
    """Dequantised keys in the rotated coordinates of each channel group, 32 bits: the groups' channels side by side."""
    parts, _ = _on_gpu(s["mode"], s["bits"], torch.float32)
    got, at = [], 0
    for i, (channels, b, lv, _) in enumerate(parts):
        size = len(channels) * _width(b) // 8
        codes = _unpack(idx[..., at:at + size], _width(b)).int()
        got.append(lv[codes] * norms[..., i:i + 1].float())
        at += size
    return torch.cat(got, -1)


def _rotated_query(s, x, dtype):
    parts, _ = _on_gpu(s["mode"], s["bits"], dtype)
    return torch.cat([x.to(dtype)[..., channels] @ m.T for channels, _, _, m in parts], -1)


def _of_cache(s, name, rows=None):
    """A plane as (sequence, KV head, token, bytes)."""
    t = s[name].view(s["batch"], s["hkv"], s["capacity"], -1)
    return t if rows is None else torch.gather(t, 2, rows[..., None].expand(-1, -1, -1, t.shape[-1]))


def _attend(s, query, rows, keep):
    """Attention of query (B, heads, n, D) over the cache's rows (None: all of them); keep: (B, 1 or KV heads, n, rows)."""
    B, H, n, _ = query.shape
    hkv = s["hkv"]
    norms = _of_cache(s, "k_norms", rows)
    keys = _rotated_keys(s, _of_cache(s, "k_idx", rows), norms)
    q = _rotated_query(s, query, torch.float32)
    if s["mode"] == "prod":
        _, sketch = _on_gpu(s["mode"], s["bits"], torch.float32)
        sign = 2.0 * _unpack(_of_cache(s, "k_signs", rows), 1).float() - 1
        keys = torch.cat([keys, norms[..., 1:2].float() * sign], -1)
        q = torch.cat([q, (math.sqrt(math.pi / 2) / D) * (q @ sketch.T)], -1)
    q = q.view(B, hkv, H // hkv * n, -1)
    score = (q @ keys.transpose(-1, -2)).view(B, hkv, H // hkv, n, -1) / math.sqrt(D)
    score.masked_fill_(~keep[:, :, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min(-1e30)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    params = _of_cache(s, "v_params", rows).view(B, hkv, -1, D // GROUP, 2).float()
    codes = _unpack(_of_cache(s, "v_q", rows), s["vbits"]).view(B, hkv, -1, D // GROUP, GROUP).float()
    v = (params[..., :1] + codes * params[..., 1:]).flatten(-2)
    out = (p.view(B, hkv, -1, p.shape[-1]) @ v).view(B, hkv, H // hkv, n, D)
    return (out / total.clamp_min(1e-30)).view(B, H, n, D).to(query.dtype)


def _on_device(values, dtype):
    return torch.tensor(values, dtype=dtype).cuda()


def _plain_extend(s):
    n = s["query"].shape[2]
    at = torch.arange(s["capacity"], device="cuda")
    end = _on_device(s["lengths"], torch.int64)[:, None] - n + 1 + torch.arange(n, device="cuda")
    return _attend(s, s["query"], None, (at < end[..., None])[:, None])


def _plain_select(s):
    """The blocks attended, ascending, -1 behind them. The scores are sums of products of 11-bit and exact numbers, held in
    64 bits, so that the order of near equals does not hang on the order of a sum."""
    B, H, _ = s["query"].shape
    q = _rotated_query(s, s["query"], torch.float64).view(B, s["hkv"], H // s["hkv"], D)
    lo, hi = s["bounds"].double().unbind(3)
    score = (q.clamp_min(0) @ hi.transpose(-1, -2) + q.clamp_max(0) @ lo.transpose(-1, -2)).amax(2)
    blocks = lo.shape[2]
    used = (_on_device(s["lengths"], torch.int64)[:, None, None] + BLOCK - 1) // BLOCK
    at = torch.arange(blocks, device="cuda")
    always = (at < s["sink"]) | (at >= used - s["recent"])
    score = torch.where(always, math.inf, score).masked_fill(at >= used, -math.inf)
    # of equals the lowest first; what always counts and what does not exist are told apart by their infinities
    order = score.sort(dim=-1, descending=True, stable=True).indices[..., :s["select"]]
    order = torch.where(order < used, order, blocks).sort(-1).values
    ids = torch.full((B, s["hkv"], s["select"]), -1, dtype=torch.int32, device="cuda")
    ids[..., :order.shape[-1]] = torch.where(order < blocks, order, -1).int()
    return ids


def _plain_sparse(s):
    ids = _plain_select(s)
    rows = (ids.long()[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")).flatten(-2)
    keep = (rows >= 0) & (rows < _on_device(s["lengths"], torch.int64)[:, None, None])
    out = _attend(s, s["query"][:, :, None], rows.clamp(0, s["capacity"] - 1), keep[:, :, None])
    return ids, out[:, :, 0]


def _plain_bounds(s):
    B, hkv = s["batch"], s["hkv"]
    keys = _rotated_keys(s, _of_cache(s, "k_idx"), _of_cache(s, "k_norms"))
    length = _on_device(s["lengths"], torch.int64)[:, None]
    blocks = s["bounds"].shape[2]
    keys = torch.nn.functional.pad(keys, (0, 0, 0, blocks * BLOCK - s["capacity"]))
    there = (torch.arange(blocks * BLOCK, device="cuda") < length)[:, None, :, None]
    lo = torch.where(there, keys, math.inf).view(B, hkv, blocks, BLOCK, D).amin(3)
    hi = torch.where(there, keys, -math.inf).view(B, hkv, blocks, BLOCK, D).amax(3)
    at = torch.arange(blocks, device="cuda")
    new = (at >= (length - s["tokens"]).clamp_min(0) // BLOCK) & (at * BLOCK < length)
    return torch.where(new[:, None, :, None, None], torch.stack([lo, hi], 3).half(), s["bounds"])


def _plain_norm_rope(s):
    pairs = len(s["axis_of_freq"])
    axis = _on_device(s["axis_of_freq"], torch.int64)
    # angles of far positions need 64 bits
    angle = s["pos"].double()[axis].permute(1, 2, 0) * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    first, second = (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if s["interleaved"] else (slice(0, pairs), slice(pairs, 2 * pairs))
    got = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * w.float()
        z = y.clone()
        z[..., first] = y[..., first] * cos - y[..., second] * sin
        z[..., second] = y[..., second] * cos + y[..., first] * sin
        got.append(z.to(x.dtype).contiguous())
    return tuple(got)


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "norm_rope":
        return _plain_norm_rope(s)
    if s["op"] == "extend":
        return _plain_extend(s)
    if s["op"] == "bounds":
        return _plain_bounds(s)
    return _plain_sparse(s)


def _run_own(s):
    import kv_cache_vector_fwht_b200 as tq
    if s["op"] == "norm_rope":
        tq.tq_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["pos"], s["inv_freq"], q_weight=s["wq"], k_weight=s["wk"],
                        eps=s["eps"], axis_of_freq=s["axis_of_freq"], interleaved=s["interleaved"])
        return s["q_out"], s["k_out"]
    if s["op"] == "extend":
        tq.tq_extend_attention(s["quantizer"], s["cache"], s["query"], s["out"], s["workspace"])
        return s["out"]
    if s["op"] == "bounds":
        tq.tq_block_bounds(s["quantizer"], s["cache"], s["bounds"], s["tokens"])
        return s["bounds"]
    tq.tq_select_blocks(s["quantizer"], s["cache"], s["bounds"], s["query"], s["ids"], s["workspace"], n_sink=s["sink"],
                        n_recent=s["recent"])
    tq.tq_decode_attention_blocks(s["quantizer"], s["cache"], s["query"], s["ids"], s["out"], s["workspace"])
    return s["ids"], s["out"]


# ------------------------------------------------------------------------------------------------------- the work

def work(case):
    if case["op"] == "norm_rope":
        size = torch.empty(0, dtype=DTYPES[case["dtype"]]).element_size()
        tokens = case["batch"] * case["tokens"]
        values = tokens * (case["hq"] + case["hk"]) * D
        return {"bytes": 2 * size * values + 4 * case["axes"] * tokens + 2 * case["rot"] + (2 * D * size if case["weights"] else 0),
                "flops": values * (4 + 3 * case["rot"] / D)}
    parts, sketch = _tables(case["mode"], case["bits"])
    key = sum(len(c) * _width(b) // 8 for c, b, _ in parts) + (2 if case["mode"] == "mse" else 4)
    row = key + (D // 8 if sketch is not None else 0) + (D * case["vbits"] // 8 + 16 if "vbits" in case else 0)
    # ragged lengths are a case's own: their mean stands for them
    mean = case["length"] if not case["ragged"] else case["length"] * (1 + (case["batch"] - 1) * 0.625) / case["batch"]
    pairs = case["batch"] * case["hkv"]
    if case["op"] == "bounds":
        rows = pairs * min(mean, case["tokens"] + BLOCK / 2)
        return {"bytes": rows * key + pairs * max(1, min(mean, case["tokens"]) / BLOCK) * 4 * D, "flops": rows * 3 * D}
    n = case.get("tokens", 1)
    answers = case["batch"] * case["hq"] * n * D * 2 * 2
    if case["op"] == "extend":
        seen = sum(max(0.0, mean - n + 1 + t) for t in range(n))
        return {"bytes": pairs * mean * row + answers, "flops": 4 * D * case["batch"] * case["hq"] * seen}
    blocks = mean / BLOCK
    read = min(mean, case["select"] * BLOCK)
    return {"bytes": pairs * (blocks * 4 * D + read * row) + answers + 4 * pairs * case["select"],
            "flops": case["batch"] * case["hq"] * (2 * D * blocks + 4 * D * read)}


# ---------------------------------------------------------------------------------------- the definition in 64 bits

def _exact_keys(s, b, h, rows):
    """Keys of one (sequence, KV head) in the original coordinates: norm * rotation^T levels, and for prod the sketch's part."""
    parts, sketch = _on_gpu(s["mode"], s["bits"], torch.float64)
    idx, norms = _of_cache(s, "k_idx")[b, h, rows], _of_cache(s, "k_norms")[b, h, rows].double()
    keys, at = torch.zeros(len(rows), D, dtype=torch.float64, device="cuda"), 0
    for i, (channels, bits, lv, m) in enumerate(parts):
        w = _width(bits)
        size = len(channels) * w // 8
        byte = idx[:, at:at + size].long().repeat_interleave(8 // w, 1)
        codes = (byte >> (torch.arange(len(channels), device="cuda") * w % 8)) % (1 << w)
        keys[:, channels] = norms[:, i:i + 1] * (lv[codes] @ m)
        at += size
    if sketch is not None:
        bits = (_of_cache(s, "k_signs")[b, h, rows].long().repeat_interleave(8, 1) >> (torch.arange(D, device="cuda") % 8)) % 2
        keys += norms[:, 1:2] * (math.sqrt(math.pi / 2) / D) * ((2.0 * bits.double() - 1) @ sketch @ parts[0][3])
    return keys


def _exact_values(s, b, h, rows):
    w = s["vbits"]
    byte = _of_cache(s, "v_q")[b, h, rows].long().repeat_interleave(8 // w, 1)
    codes = (byte >> (torch.arange(D, device="cuda") * w % 8)) % (1 << w)
    low, step = _of_cache(s, "v_params")[b, h, rows].double().view(-1, D // GROUP, 2).repeat_interleave(GROUP, 1).unbind(2)
    return low + codes * step


def _exact_attention(query, keys, values, ends):
    """query (heads, n, D) over keys and values (rows, D); row t of n sees the first ends[t] of them."""
    out = torch.zeros(query.shape, dtype=torch.float64, device="cuda")
    hidden = torch.arange(len(keys), device="cuda") >= ends[:, None]
    for j in range(query.shape[0]):
        p = torch.softmax((query[j].double() @ keys.T / math.sqrt(D)).masked_fill(hidden, -math.inf), -1)
        out[j] = torch.nan_to_num(p, nan=0.0) @ values   # a row that sees nothing has no weights
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        got = []
        for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
            x = x.double()
            if w is not None:
                x = x / (x.square().sum(-1, keepdim=True) / D + s["eps"]).sqrt() * w.double()
            pairs = case["rot"] // 2
            turned = x[..., :2 * pairs]
            z = torch.complex(*(turned.unflatten(-1, (pairs, 2)).unbind(-1) if s["interleaved"] else turned.unflatten(-1, (2, pairs)).unbind(-2)))
            angle = torch.stack([s["pos"][a].double() * f for a, f in zip(s["axis_of_freq"], s["inv_freq"].double())], -1)[:, None]
            z = z * torch.polar(torch.ones_like(angle), angle)
            z = torch.stack([z.real, z.imag], -1 if s["interleaved"] else -2).flatten(-2)
            got.append(torch.cat([z, x[..., 2 * pairs:]], -1))
        return tuple(got)
    B, hkv, lengths = s["batch"], s["hkv"], s["lengths"]
    if case["op"] == "bounds":
        parts, _ = _on_gpu(s["mode"], s["bits"], torch.float64)
        want = s["bounds"].double()
        for b in range(B):
            first = max(0, lengths[b] - s["tokens"]) // BLOCK
            for h in range(hkv):
                rows = torch.arange(first * BLOCK, lengths[b], device="cuda")
                if len(rows):
                    keys = _exact_keys(dict(s, mode="mse", bits=s["bits"] - 1, k_signs=None) if s["mode"] == "prod" else s, b, h, rows)
                    turned = torch.cat([keys[:, channels] @ m.T for channels, _, _, m in parts], 1)
                    for i in range(-(-len(rows) // BLOCK)):
                        part = turned[i * BLOCK:(i + 1) * BLOCK]
                        want[b, h, first + i, 0], want[b, h, first + i, 1] = part.amin(0), part.amax(0)
        return want
    query = s["query"].double().view(B, hkv, -1, case.get("tokens", 1), D)
    out = torch.zeros(query.shape, dtype=torch.float64, device="cuda")
    ids = None
    for b in range(B):
        for h in range(hkv):
            if case["op"] == "extend":
                rows = torch.arange(lengths[b], device="cuda")
                ends = lengths[b] - query.shape[3] + 1 + torch.arange(query.shape[3], device="cuda")
            else:
                used = -(-lengths[b] // BLOCK)
                lo, hi = s["bounds"][b, h, :used].double().unbind(1)
                q = _rotated_query(s, query[b, h, :, 0], torch.float64)
                score = ((hi + lo) / 2 @ q.T + (hi - lo) / 2 @ q.abs().T).amax(1)
                score[:s["sink"]] = math.inf
                score[max(0, used - s["recent"]):] = math.inf
                ids = score.topk(min(used, s["select"])).indices.sort().values
                rows = (ids[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")).flatten()
                rows = rows[rows < lengths[b]]
                ends = torch.tensor([len(rows)], device="cuda")
            out[b, h] = _exact_attention(query[b, h], _exact_keys(s, b, h, rows), _exact_values(s, b, h, rows), ends)
    out = out.view(s["query"].shape)
    return out if case["op"] == "extend" else (None, out)
