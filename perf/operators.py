"""Measured cases of the operators around one serving step of the paged KV cache.

build_batch            block tables, slot mapping, positions and offsets of a batch from request lengths
qk_norm_rope           RMS norm of every query and key head and rotary positions (one or several axes), one pass
qkv_norm_rope_write    the same, with the keys and values stored into the paged cache
paged_cross_attention  attention of decoder tokens to an encoder's cached states (every cache format),
                       optionally limited to a range of them per query token

listed() and draw() give the cases, prepare() their inputs, run() one pass: with `own` false in elementary
torch operations, with `own` true by the calls a user of paged_quantized_kv_cache_b200 makes. exact() computes
the same outputs in 64 bits.
"""
import math

import torch

own = False

BLOCK = 16
FORMATS = {"fp16": 0, "bf16": 1, "fp8_e4m3": 2, "fp8_e5m2": 3, "fp4_e2m1": 4}
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
FP8 = {"fp8_e4m3": (torch.float8_e4m3fn, 448.0), "fp8_e5m2": (torch.float8_e5m2, 57344.0)}
# query heads, KV heads, head size of the decode workloads' layers and of the small ones in the tests
HEADS = ((32, 8, 128), (64, 8, 128), (8, 2, 64), (8, 8, 64), (16, 2, 64))


# ---- cases ----------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 16 running requests: one token each, a new block now and then
        {"name": "batch-decode-16", "op": "batch", "requests": 16, "new_lo": 1, "new_hi": 1, "past": 4096, "pad": 0},
        # 96 requests in one padded step: most prefill a ragged chunk of up to 512 tokens behind what they have
        {"name": "batch-chunks-96", "op": "batch", "requests": 96, "new_lo": 1, "new_hi": 512, "past": 7680, "pad": 500},
        # the tables of 512 whole prompts laid down at once
        {"name": "batch-prompts-512", "op": "batch", "requests": 512, "new_lo": 256, "new_hi": 1024, "past": 0, "pad": 0},
        # one token of one request with time/height/width positions: the latency of a step
        {"name": "norm-rope-1", "op": "norm", "dtype": "bf16", "tokens": 1, "hq": 32, "hkv": 8, "d": 128,
         "rot": 128, "axes": 3, "interleaved": False, "norm": True, "past": 32768},
        # a prompt of text and images, positions on three axes
        {"name": "norm-rope-8191", "op": "norm", "dtype": "bf16", "tokens": 8191, "hq": 32, "hkv": 8, "d": 128,
         "rot": 128, "axes": 3, "interleaved": False, "norm": True, "past": 32768},
        # 64 running requests, one token each, keys and values into the cache
        {"name": "norm-rope-write-64", "op": "write", "dtype": "bf16", "tokens": 64, "hq": 32, "hkv": 8, "d": 128,
         "rot": 128, "axes": 1, "interleaved": False, "norm": True, "past": 32768},
        # eight 512-token chunks and a ragged one of the layer with 64 query heads: fp16, half of each head rotated in
        # neighbouring pairs, positions on two axes
        {"name": "norm-rope-write-4133", "op": "write", "dtype": "fp16", "tokens": 4133, "hq": 64, "hkv": 8, "d": 128,
         "rot": 64, "axes": 2, "interleaved": True, "norm": True, "past": 8192},
        # one decoder token of 16 requests, each reading its audio or image states of some 1500 positions
        {"name": "cross-1-bf16", "op": "cross", "format": "bf16", "dtype": "bf16", "batch": 16, "q_lo": 1, "q_hi": 1,
         "kv_lo": 1400, "kv_hi": 1500, "hq": 32, "hkv": 8, "d": 128, "ranges": False},
        # the same from an FP8 cache with longer states
        {"name": "cross-1-fp8", "op": "cross", "format": "fp8_e4m3", "dtype": "bf16", "batch": 64, "q_lo": 1, "q_hi": 1,
         "kv_lo": 2048, "kv_hi": 6404, "hq": 32, "hkv": 8, "d": 128, "ranges": False},
        # a prompt's 512-token chunks, every token limited to the images before it (some see none)
        {"name": "cross-chunk-bf16", "op": "cross", "format": "bf16", "dtype": "bf16", "batch": 16, "q_lo": 300, "q_hi": 512,
         "kv_lo": 3203, "kv_hi": 6404, "hq": 32, "hkv": 8, "d": 128, "ranges": True},
        # a few tokens of the small layer over short states in fp16
        {"name": "cross-short-fp16", "op": "cross", "format": "fp16", "dtype": "fp16", "batch": 4, "q_lo": 3, "q_hi": 40,
         "kv_lo": 1, "kv_hi": 577, "hq": 8, "hkv": 2, "d": 64, "ranges": True},
        # chunks over the 4-bit cache with its outlier channels
        {"name": "cross-chunk-fp4", "op": "cross", "format": "fp4_e2m1", "dtype": "bf16", "batch": 8, "q_lo": 129, "q_hi": 512,
         "kv_lo": 1000, "kv_hi": 4096, "hq": 32, "hkv": 8, "d": 128, "ranges": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("batch", "norm", "write", "cross", "cross"))
    if op == "batch":
        requests = _log(rng, 1, 512)
        whole = rng.random() < 0.3
        hi = _log(rng, 1, 1024)
        return {"op": op, "requests": requests, "new_lo": rng.randint(0, hi), "new_hi": hi,
                "past": 0 if whole else _log(rng, 1, 32768), "pad": rng.choice((0, 0, rng.randint(1, 1000)))}
    hq, hkv, d = rng.choice(HEADS)
    if op != "cross":
        return {"op": op, "dtype": rng.choice(("bf16", "fp16")), "tokens": _log(rng, 1, 8191 if hq <= 32 else 4133), "hq": hq,
                "hkv": hkv, "d": d, "rot": rng.choice((0, d // 4, d // 2, d - 8, d, d)), "axes": rng.choice((1, 1, 2, 3)),
                "interleaved": rng.random() < 0.3, "norm": rng.random() < 0.8, "past": _log(rng, 64, 32768)}
    fmt = rng.choice(tuple(FORMATS))
    kv_hi, q_hi = _log(rng, 1, 6404), _log(rng, 1, 512)
    kv_lo, q_lo = rng.randint(0, kv_hi), rng.randint(0, q_hi)
    return {"op": op, "format": fmt, "dtype": fmt if fmt in TYPES else rng.choice(("bf16", "fp16")), "batch": _log(rng, 1, 16),
            "q_lo": q_lo, "q_hi": q_hi, "kv_lo": kv_lo, "kv_hi": kv_hi, "hq": min(hq, 32), "hkv": hkv, "d": d,
            "ranges": rng.random() < 0.4}


# ---- inputs ---------------------------------------------------------------------------------------------------------

def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, dtype=torch.int64)


def _spread(lo, hi, n):
    """n lengths from hi down to lo: every seed's batch has the same ones, in another order."""
    return [hi - i * (hi - lo) // max(1, n - 1) for i in range(n)]


def _host(seed):
    return torch.Generator().manual_seed(int(seed) * 2 + 1)


def _gpu(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 2)


def _blocks(tokens):
    return (tokens + BLOCK - 1) // BLOCK


def _cuda(t, dtype=torch.int32):
    return t.to(dtype).cuda()


def _batch_lengths(case, seed):
    g = _host(seed)
    n = case["requests"]
    new = torch.tensor(_spread(case["new_lo"], case["new_hi"], n))[torch.randperm(n, generator=g)]
    start = _ints(g, 0, case["past"], n) if case["past"] else torch.zeros(n, dtype=torch.int64)
    return start, new, g


def _prepare_batch(case, seed):
    start, new, g = _batch_lengths(case, seed)
    n = case["requests"]
    have, need = _blocks(start), _blocks(start + new)
    most = _blocks(case["past"] + case["new_hi"]) + 1
    num_blocks = int(need.sum()) + 64
    ids = torch.randperm(num_blocks, generator=g)
    fresh = int((need - have).sum())
    held = ids[fresh:fresh + int(have.sum())]
    tables = torch.full((n, most), -1, dtype=torch.int64)
    tables[torch.arange(most)[None, :] < have[:, None]] = held
    capacity = int(new.sum()) + case["pad"]
    empty = lambda k: torch.empty(k, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"case": case, "start": _cuda(start), "new": _cuda(new), "ids": _cuda(ids[:fresh]), "tables": _cuda(tables),
            "num_blocks": num_blocks, "slots": empty(capacity), "positions": empty(capacity), "cu": empty(n + 1),
            "lens": empty(n), "err": torch.zeros(1, dtype=torch.int32, device="cuda")}


def _axes_of(case):
    """The axis of every rotated pair: the axes take turns in thirds of the pairs' order, as blocks."""
    pairs = case["rot"] // 2
    return torch.arange(pairs) * case["axes"] // max(1, pairs)


def _prepare_rows(case, seed):
    g, h = _gpu(seed), _host(seed)
    t, hq, hkv, d, rot = (case[k] for k in ("tokens", "hq", "hkv", "d", "rot"))
    dtype = TYPES[case["dtype"]]
    # the projection's output: queries, keys and values of a token side by side, channels of different size
    size = 0.25 + torch.rand((hq + 2 * hkv) * d, generator=g, device="cuda") * 2
    qkv = (torch.randn(t, (hq + 2 * hkv) * d, generator=g, device="cuda") * size).to(dtype)
    count = case["past"] + t
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / max(1, rot))
    angle = torch.arange(count, dtype=torch.float64, device="cuda")[:, None] * freq
    table = torch.cat((angle.cos(), angle.sin()), dim=1).to(torch.float32).contiguous()
    begin = int(_ints(h, 0, case["past"], 1))
    i = torch.arange(t)
    # one axis counts tokens; the others walk the rows and columns of a picture behind the same start
    places = [begin + i, begin + i // 37 % 24, begin + i % 37]
    positions = torch.stack([p.clamp(max=count - 1) for p in places[:case["axes"]]])
    weight = lambda: (1 + 0.2 * torch.randn(d, generator=g, device="cuda")) if case["norm"] else None  # noqa: E731
    axes = _axes_of(case)
    s = {"case": case, "qkv": qkv, "table": table, "positions": _cuda(positions), "axes": axes.cuda(),
         "axes_bytes": bytes(axes.tolist()), "qw": weight(), "kw": weight(),
         "q_out": torch.empty(t, hq, d, dtype=dtype, device="cuda"), "err": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if case["op"] == "norm":
        s["k_out"] = torch.empty(t, hkv, d, dtype=dtype, device="cuda")
        return s
    blocks = _blocks(t) + 3
    ids = torch.randperm(blocks, generator=h)
    offset = int(_ints(h, 0, BLOCK - 1, 1))
    p = offset + i
    s["slots"] = _cuda(ids[p // BLOCK] * BLOCK + p % BLOCK)
    s["cache"] = torch.zeros(blocks, hkv, 2, BLOCK, d, dtype=dtype, device="cuda")
    return s


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# token of (pair row, nibble) of a 4-bit block's values
PAIR_TOKENS = [[2 * (p // 2) + 8 * (p % 2), 2 * (p // 2) + 8 * (p % 2) + 1] for p in range(8)]


def _e2m1(y):
    """The code whose value is nearest (between two, the even code)."""
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=y.device)
    a = y.abs()
    up, down = torch.bucketize(a, edges, right=True), torch.bucketize(a, edges)
    code = torch.where(up % 2 == 0, up, down)
    return (code + 8 * (y < 0)).to(torch.uint8)


def _prepare_cache(case, g, blocks):
    """Cache arrays in the layout of the format, of normal keys and values."""
    hkv, d, fmt = case["hkv"], case["d"], case["format"]
    x = torch.randn(blocks, hkv, 2, BLOCK, d, generator=g, device="cuda")
    if fmt in TYPES:
        return {"cache": x.to(TYPES[fmt])}
    if fmt in FP8:
        dtype, most = FP8[fmt]
        scale = x.abs().amax(dim=(3, 4)) / most
        codes = (x / scale[..., None, None]).to(dtype).view(torch.uint8)
        return {"cache": codes, "scales": torch.cat((scale, torch.zeros_like(scale)), dim=2).contiguous()}
    channels = torch.rand(hkv, 2, d, generator=g, device="cuda").argsort(dim=2)[:, :, :2].sort(dim=2).values
    at = channels[None, :, :, None, :].expand(blocks, hkv, 2, BLOCK, 2)
    values = x.gather(4, at) * 16
    x = x.scatter(4, at, 0.0)
    scale = (x.view(blocks, hkv, 2, BLOCK, d // 16, 16).abs().amax(dim=5) / 6).to(torch.float8_e4m3fn)
    s = scale.to(torch.float32).repeat_interleave(16, dim=4)
    code = _e2m1(torch.where(s > 0, x / s, torch.zeros_like(x)))
    k = code[:, :, 0, :, 0::2] | (code[:, :, 0, :, 1::2] << 4)
    pair = code[:, :, 1][:, :, torch.tensor(PAIR_TOKENS, device="cuda")]  # [blocks][hkv][8][2][d]
    v = pair[:, :, :, 0] | (pair[:, :, :, 1] << 4)
    v = torch.cat((v[..., :d // 2], v[..., d // 2:]), dim=2)
    index = torch.full((blocks, hkv, 2, 8), 255, dtype=torch.uint8, device="cuda")
    index[..., :2] = channels.to(torch.uint8)
    value = torch.zeros(blocks, hkv, 2, BLOCK, 4, dtype=torch.float16, device="cuda")
    value[..., :2] = values.to(torch.float16)
    return {"cache": torch.stack((k, v), dim=2).contiguous(), "scales": scale.view(torch.uint8).contiguous(),
            "outliers_idx": index, "outliers_val": value}


def _cross_lengths(case, seed):
    h = _host(seed)
    n = case["batch"]
    q = torch.tensor(_spread(case["q_lo"], case["q_hi"], n))[torch.randperm(n, generator=h)]
    kv = torch.tensor(_spread(case["kv_lo"], case["kv_hi"], n))[torch.randperm(n, generator=h)]
    return q, kv, h


def _cross_ranges(case, q, kv, h):
    """A token sees the states of up to three pictures behind one another, and one in eight sees none."""
    n = int(q.sum())
    length = kv.repeat_interleave(q)
    piece = (length + 3) // 4
    lo = torch.randint(0, 4, (n,), generator=h) * piece
    hi = torch.minimum(length, lo + torch.randint(1, 4, (n,), generator=h) * piece)
    none = torch.randint(0, 8, (n,), generator=h) == 0
    return torch.stack((lo, torch.where(none, lo, hi)), dim=1)


def _prepare_cross(case, seed):
    g = _gpu(seed)
    q, kv, h = _cross_lengths(case, seed)
    n = case["batch"]
    nblk = _blocks(kv)
    blocks = int(nblk.sum()) + 5
    most = max(1, int(nblk.max()))
    ids = torch.randperm(blocks, generator=h)[:int(nblk.sum())]
    tables = torch.full((n, most), -1, dtype=torch.int64)
    tables[torch.arange(most)[None, :] < nblk[:, None]] = ids
    cu = torch.cat((torch.zeros(1, dtype=torch.int64), q.cumsum(0)))
    dtype = TYPES[case["dtype"]]
    x = torch.randn(int(cu[-1]), case["hq"], case["d"], generator=g, device="cuda").to(dtype)
    s = {"case": case, "q": x, "cu": _cuda(cu), "most_q": int(q.max()), "tables": _cuda(tables), "kv": _cuda(kv), "blocks": blocks,
         "ranges": _cuda(_cross_ranges(case, q, kv, h)) if case["ranges"] else None, "scale": 1 / math.sqrt(case["d"]),
         "out": torch.empty_like(x), "err": torch.zeros(1, dtype=torch.int32, device="cuda")}
    s.update(_prepare_cache(case, g, blocks))
    return s


def prepare(case, seed):
    if case["op"] == "batch":
        return _prepare_batch(case, seed)
    if case["op"] == "cross":
        return _prepare_cross(case, seed)
    return _prepare_rows(case, seed)


# ---- one pass -------------------------------------------------------------------------------------------------------

def _plain_batch(s):
    start, new, tables = s["start"].long(), s["new"].long(), s["tables"]
    n, most = tables.shape
    capacity = s["slots"].numel()
    have, need = (start + 15) // 16, (start + new + 15) // 16
    cu = torch.cat((new.new_zeros(1), new.cumsum(0)))
    first = (need - have).cumsum(0) - (need - have)
    j = torch.arange(most, device=tables.device)
    fresh = (j >= have[:, None]) & (j < need[:, None])
    ids = torch.cat((s["ids"], s["ids"].new_zeros(1)))
    at = torch.where(fresh, first[:, None] + j - have[:, None], s["ids"].numel())
    tables.copy_(torch.where(fresh, ids[at], tables))
    i = torch.arange(capacity, device=tables.device)
    b = torch.searchsorted(cu[1:], i, right=True).clamp(max=n - 1)
    used = i < cu[-1]
    position = torch.where(used, start[b] + i - cu[b], 0)
    slot = tables[b, position // 16].long() * 16 + position % 16
    return {"tables": tables, "slots": torch.where(used, slot, -1).int(), "positions": position.int(), "cu": cu.int(),
            "lens": (start + new).int()}


def _plain_rotate(x, s, weight):
    """RMS norm of the rows of x (when there is a weight) and the rotation of their first `rot` channels."""
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + 1e-6) * weight
    if not rot:
        return x
    place = s["positions"].long()[s["axes"]].t()
    pair = torch.arange(half, device=x.device)
    cos, sin = s["table"][place, pair][:, None], s["table"][place, pair + half][:, None]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if case["interleaved"] else (x[..., :half], x[..., half:rot])
    y, z = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((y, z), dim=-1).flatten(-2) if case["interleaved"] else torch.cat((y, z), dim=-1)
    return torch.cat((turned, x[..., rot:]), dim=-1)


def _split(s):
    case = s["case"]
    t, hq, hkv, d = (case[k] for k in ("tokens", "hq", "hkv", "d"))
    q, k, v = s["qkv"].split((hq * d, hkv * d, hkv * d), dim=1)
    return q.view(t, hq, d), k.view(t, hkv, d), v.view(t, hkv, d)


def _plain_rows(s):
    q, k, v = _split(s)
    dtype = q.dtype
    turned_q, turned_k = _plain_rotate(q, s, s["qw"]).to(dtype), _plain_rotate(k, s, s["kw"]).to(dtype)
    if s["case"]["op"] == "norm":
        return {"q": turned_q, "k": turned_k}
    slot = s["slots"].long()
    s["cache"][slot // 16, :, 0, slot % 16] = turned_k
    s["cache"][slot // 16, :, 1, slot % 16] = v
    return {"q": turned_q, "cache": s["cache"]}


def _plain_states(s):
    """Keys and values [batch][blocks][hkv][2][16][d] in 32 bits, through the block tables."""
    fmt = s["case"]["format"]
    id = s["tables"].long().clamp(min=0)
    x = s["cache"][id]
    if fmt in TYPES:
        return x.float()
    if fmt in FP8:
        return x.view(FP8[fmt][0]).float() * s["scales"][id][..., :2, None, None]
    d = s["case"]["d"]
    value = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=x.device)
    low, high = value[(x & 15).long()], value[(x >> 4).long()]
    k = torch.stack((low[:, :, :, 0], high[:, :, :, 0]), dim=-1).flatten(-2)
    v = torch.stack((low[:, :, :, 1], high[:, :, :, 1]), dim=-2)  # [...][16 rows][nibble][d / 2]
    v = torch.cat((v[..., :8, :, :], v[..., 8:, :, :]), dim=-1)   # [...][pair][nibble][d]
    token = torch.tensor(PAIR_TOKENS, device=x.device).flatten()
    v = v.flatten(-3, -2)[..., token.argsort(), :]
    y = torch.stack((k, v), dim=3)
    y = (y.unflatten(-1, (d // 16, 16)) * s["scales"].view(torch.float8_e4m3fn).float()[id][..., None]).flatten(-2)
    index = s["outliers_idx"][id][..., None, :4].long()
    kept = index < d
    at = torch.where(kept, index, d).expand(*y.shape[:-1], 4)
    y = torch.cat((y, y.new_zeros(*y.shape[:-1], 1)), dim=-1)
    return y.scatter(-1, at, s["outliers_val"][id].float())[..., :d]


def _plain_cross(s):
    case = s["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    q, cu, kv = s["q"], s["cu"].long(), s["kv"].long()
    n = kv.numel()
    x = _plain_states(s)
    length = x.shape[1] * BLOCK
    x = x.permute(3, 0, 2, 1, 4, 5).reshape(2, n, hkv, length, d)
    row = cu[:-1, None] + torch.arange(s["most_q"], device=q.device)
    used = row < cu[1:, None]
    at = torch.where(used, row, q.shape[0] - 1)
    rows = q.float()[at].view(n, -1, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
    t = torch.arange(length, device=q.device)
    seen = (t < kv[:, None])[:, None, None, None, :]
    if s["ranges"] is not None:
        r = s["ranges"].long()[at]
        seen = seen & ((t >= r[..., :1]) & (t < r[..., 1:]))[:, None, None]
    score = (rows @ x[0].transpose(-1, -2)).view(n, hkv, hq // hkv, -1, length) * s["scale"]
    score = torch.where(seen, score, -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    weight = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = weight.sum(dim=-1, keepdim=True)
    values = torch.where((t < kv[:, None])[:, None, :, None], x[1], 0.0)
    out = (weight.view(n, hkv, -1, length) @ values).view(n, hkv, hq // hkv, -1, d)
    out = out / torch.where(total > 0, total, 1.0)
    out = out.permute(0, 3, 1, 2, 4).reshape(n, -1, hq, d)
    i = torch.arange(q.shape[0], device=q.device)
    b = torch.searchsorted(cu[1:], i, right=True)
    return {"out": out[b, i - cu[b]].to(q.dtype)}


def _cache_of(pq, s, fmt, blocks):
    case = s["case"]
    flat = lambda t: None if t is None else t.view(torch.uint8).view(-1)  # noqa: E731
    return pq.KVCache(FORMATS[fmt], blocks, case["hkv"], case["d"], flat(s["cache"]), flat(s.get("scales")),
                      flat(s.get("outliers_idx")), flat(s.get("outliers_val")))


def _own(s):
    import paged_quantized_kv_cache_b200 as pq
    case = s["case"]
    if case["op"] == "batch":
        pq.build_batch(s["start"], s["new"], s["ids"], s["tables"], s["num_blocks"], s["slots"], s["positions"], s["cu"],
                       s["lens"], s["err"])
        return {k: s[k] for k in ("tables", "slots", "positions", "cu", "lens")}
    if case["op"] == "cross":
        pq.paged_cross_attention(s["q"], s["cu"], s["most_q"], _cache_of(pq, s, case["format"], s["blocks"]), s["tables"],
                                 s["kv"], s["scale"], s["out"], s["err"], kv_ranges=s["ranges"])
        return {"out": s["out"]}
    q, k, v = _split(s)
    rotary = pq.Rotary(s["table"], s["axes_bytes"], case["interleaved"])
    if case["op"] == "norm":
        pq.qk_norm_rope(q, k, s["positions"], rotary, s["q_out"], s["k_out"], s["err"], q_weight=s["qw"], k_weight=s["kw"])
        return {"q": s["q_out"], "k": s["k_out"]}
    pq.qkv_norm_rope_write(q, k, v, s["positions"], rotary, s["q_out"], s["slots"],
                           _cache_of(pq, s, case["dtype"], s["cache"].shape[0]), s["err"], q_weight=s["qw"], k_weight=s["kw"])
    return {"q": s["q_out"], "cache": s["cache"]}


def run(state):
    if own:
        return _own(state)
    if state["case"]["op"] == "batch":
        return _plain_batch(state)
    if state["case"]["op"] == "cross":
        return _plain_cross(state)
    return _plain_rows(state)


# ---- what a pass cannot do without ----------------------------------------------------------------------------------

def work(case):
    if case["op"] == "batch":
        n = case["requests"]
        tokens = sum(_spread(case["new_lo"], case["new_hi"], n))
        fresh = tokens / BLOCK
        return {"bytes": 4 * (2 * n + 2 * fresh + 2 * (tokens + case["pad"]) + 2 * n + 1 + (n if case["past"] else 0)), "flops": 0}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "cross":
        n = case["batch"]
        q, kv = sum(_spread(case["q_lo"], case["q_hi"], n)), sum(_spread(case["kv_lo"], case["kv_hi"], n))
        fmt = case["format"]
        state = 2 * d * 2 if fmt in TYPES else 2 * d + 1 if fmt in FP8 else d + d // 8 + 17
        share = 0.365 if case["ranges"] else 1.0  # of the states, what a token sees on average
        return {"bytes": 4 * q * hq * d + kv * hkv * state, "flops": 4 * q * (kv / n) * share * hq * d}
    t = case["tokens"]
    rows = (2 * (hq + hkv) if case["op"] == "norm" else 2 * (hq + 2 * hkv)) * t * d * 2
    return {"bytes": rows + t * 4 * (case["axes"] + case["rot"] + (case["op"] == "write")), "flops": 8 * t * (hq + hkv) * d}


# ---- the same in 64 bits --------------------------------------------------------------------------------------------

def _exact_batch(case, seed):
    s = _prepare_batch(case, seed)
    start, new, _ = _batch_lengths(case, seed)
    tables, ids = s["tables"].cpu().long(), s["ids"].cpu().long().tolist()
    capacity = s["slots"].numel()
    slots, positions, cu, lens, at, taken = [], [], [0], [], 0, 0
    for b in range(case["requests"]):
        first, count = int(start[b]), int(new[b])
        for j in range(-(-first // BLOCK), -(-(first + count) // BLOCK)):
            tables[b, j] = ids[taken]
            taken += 1
        for p in range(first, first + count):
            positions.append(p)
        p = torch.arange(first, first + count)
        slots.append(tables[b, p // BLOCK] * BLOCK + p % BLOCK)
        at += count
        cu.append(at)
        lens.append(first + count)
    slots.append(torch.full((capacity - at,), -1))
    whole = lambda v: torch.as_tensor(v).int().cuda()  # noqa: E731
    return {"tables": whole(tables), "slots": whole(torch.cat(slots)), "positions": whole(positions + [0] * (capacity - at)),
            "cu": whole(cu), "lens": whole(lens)}


def _exact_rows(case, seed):
    s = _prepare_rows(case, seed)
    t, hq, hkv, d, rot = (case[k] for k in ("tokens", "hq", "hkv", "d", "rot"))
    x = s["qkv"].double().view(t, hq + 2 * hkv, d)
    place = s["positions"].long()
    done = []
    for lo, hi, weight in ((0, hq, s["qw"]), (hq, hq + hkv, s["kw"])):
        y = x[:, lo:hi].clone()
        if weight is not None:
            y = y / (y.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt() * weight.double()
        z = y.clone()
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
            p = place[i * case["axes"] // (rot // 2)]
            c, e = s["table"][p, i].double()[:, None], s["table"][p, rot // 2 + i].double()[:, None]
            z[..., a] = y[..., a] * c - y[..., b] * e
            z[..., b] = y[..., a] * e + y[..., b] * c
        done.append(z)
    if case["op"] == "norm":
        return {"q": done[0], "k": done[1]}
    cache = s["cache"].double()
    slot = s["slots"].long()
    for h in range(hkv):
        cache[slot // BLOCK, h, 0, slot % BLOCK] = done[1][:, h]
        cache[slot // BLOCK, h, 1, slot % BLOCK] = x[:, hq + hkv + h]
    return {"q": done[0], "cache": cache}


def _exact_state(case, s, id, which):
    """The keys (which = 0) or values (1) of blocks `id`: [hkv][16 len(id)][d] in 64 bits, by the layout's words."""
    fmt, d, hkv = case["format"], case["d"], case["hkv"]
    x = s["cache"][id][:, :, which]
    if fmt in FP8:
        x = x.view(FP8[fmt][0]).double() * s["scales"][id][:, :, which, None, None].double()
    elif fmt == "fp4_e2m1":
        y = torch.zeros(len(id), hkv, BLOCK, d, dtype=torch.float64, device=x.device)
        sign = lambda c: torch.where(c >= 8, -1.0, 1.0)  # noqa: E731
        value = lambda c: sign(c) * torch.tensor(E2M1, dtype=torch.float64, device=x.device)[(c & 7).long()]  # noqa: E731
        for token in range(BLOCK):
            if which == 0:
                y[:, :, token, 0::2], y[:, :, token, 1::2] = value(x[:, :, token] & 15), value(x[:, :, token] >> 4)
            else:
                p = token // 2 * 2 if token < 8 else (token - 8) // 2 * 2 + 1
                move = 4 * (token % 2)
                y[:, :, token, :d // 2] = value((x[:, :, p] >> move) & 15)
                y[:, :, token, d // 2:] = value((x[:, :, 8 + p] >> move) & 15)
        scale = s["scales"][id][:, :, which].view(torch.float8_e4m3fn).double()
        for c in range(d):
            y[..., c] *= scale[..., c // 16]
        for h in range(hkv):
            for r in range(4):
                c = int(s["outliers_idx"][0, h, which, r])
                if c < d:
                    y[:, h, :, c] = s["outliers_val"][id][:, h, which, :, r].double()
        x = y
    return x.double().permute(1, 0, 2, 3).reshape(hkv, -1, d)


def _exact_cross(case, seed):
    s = _prepare_cross(case, seed)
    g = case["hq"] // case["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    cu = s["cu"].tolist()
    for b, length in enumerate(s["kv"].tolist()):
        rows = slice(cu[b], cu[b + 1])
        if length == 0 or rows.start == rows.stop:
            continue
        id = s["tables"][b, :-(-length // BLOCK)].long()
        k, v = (_exact_state(case, s, id, w)[:, :length] for w in (0, 1))
        seen = None
        if s["ranges"] is not None:
            t = torch.arange(length, device="cuda")
            seen = (t >= s["ranges"][rows, :1]) & (t < s["ranges"][rows, 1:])
        for h in range(case["hq"]):
            score = s["q"][rows, h].double() @ k[h // g].t() * s["scale"]
            if seen is not None:
                score[~seen] = -math.inf
            p = torch.softmax(score, dim=-1).nan_to_num(nan=0.0)
            out[rows, h] = p @ v[h // g]
    return {"out": out}


def exact(case, seed):
    if case["op"] == "batch":
        return _exact_batch(case, seed)
    if case["op"] == "cross":
        return _exact_cross(case, seed)
    return _exact_rows(case, seed)
