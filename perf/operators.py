"""Cases, plain forms and 64-bit definitions of three operators of the paged KV cache.

  rope    kv_append_rope: q and k are turned by their positions' angles, k and v go to their
          slots of the paged pool (16-bit, or quantized on the way)
  cross   paged_cross_attn: every row of a ragged batch attends to all cached states of its
          own sequence, which are of another length (a decoder against an encoder's states)
  groups  paged_decode_attn_groups: one decode step of a batch whose sequences come in groups,
          each group sharing a prefix of its own, attended once for the whole group

With ``own`` false the operators are computed by elementary torch operations in 32 bits; with
``own`` true by the library.
"""
import random

import torch

own = False

BLOCK = 16
DTYPE = {"f16": 0, "bf16": 1, "int8": 2, "int4": 3, "fp8": 4}    # the library's dtype codes
LIMIT = {"int8": 127.0, "int4": 7.0, "fp8": 448.0}
TORCH16 = {"f16": torch.float16, "bf16": torch.bfloat16}
MAX_POSITIONS = 131072


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token of one sequence: the latency of the smallest step (8B head shape)
        {"name": "rope one token", "op": "rope", "pool": "bf16", "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "inter": False, "tokens": 1, "run": 1, "fused": True, "pad": 0},
        # a decode step of 170 sequences, 70B head shape, over an int8 cache, padded to 176
        {"name": "rope decode int8", "op": "rope", "pool": "int8", "hq": 64, "hkv": 8, "d": 128, "rot": 128,
         "inter": False, "tokens": 176, "run": 1, "fused": True, "pad": 6},
        # one engine step of prefill chunks of 1,021 tokens, neighbouring pairs, half the dims turned
        {"name": "rope chunks fp8", "op": "rope", "pool": "fp8", "hq": 32, "hkv": 8, "d": 128, "rot": 64,
         "inter": True, "tokens": 4084, "run": 1021, "fused": False, "pad": 0},
        # the largest prefill step, 70B head shape, bf16 cache
        {"name": "rope prefill bf16", "op": "rope", "pool": "bf16", "hq": 64, "hkv": 8, "d": 128, "rot": 128,
         "inter": False, "tokens": 16384, "run": 4096, "fused": True, "pad": 0},

        # a single-token step of 8 sequences against short encoder states (latency), heads of 64
        {"name": "cross one token", "op": "cross", "pool": "f16", "hq": 16, "hkv": 16, "d": 64, "batch": 8,
         "rows_lo": 1, "rows_hi": 1, "ctx_lo": 0, "ctx_hi": 700, "pad": 0},
        # beam search: 1 to 5 hypotheses of each of 64 sequences, int8 states of up to 4,500
        {"name": "cross beams int8", "op": "cross", "pool": "int8", "hq": 32, "hkv": 8, "d": 128, "batch": 64,
         "rows_lo": 1, "rows_hi": 5, "ctx_lo": 1500, "ctx_hi": 4500, "pad": 3},
        # teacher forcing / decoder prompts of odd lengths, heads of 64 without grouping
        {"name": "cross prompts d64", "op": "cross", "pool": "bf16", "hq": 16, "hkv": 16, "d": 64, "batch": 16,
         "rows_lo": 33, "rows_hi": 448, "ctx_lo": 64, "ctx_hi": 1500, "pad": 5},
        # long documents scored against long states, 70B head shape
        {"name": "cross long bf16", "op": "cross", "pool": "bf16", "hq": 64, "hkv": 8, "d": 128, "batch": 6,
         "rows_lo": 700, "rows_hi": 1024, "ctx_lo": 2000, "ctx_hi": 6000, "pad": 0},

        # two system prompts over eight sequences (8B head shape): latency
        {"name": "groups of 4", "op": "groups", "pool": "bf16", "hq": 32, "hkv": 8, "d": 128, "groups": 2,
         "size_lo": 4, "size_hi": 4, "prefix_lo": 512, "prefix_hi": 1024, "suffix_lo": 1, "suffix_hi": 100},
        # an uneven batch on a heads-of-64 model, some groups without a prefix
        {"name": "groups uneven d64", "op": "groups", "pool": "f16", "hq": 32, "hkv": 4, "d": 64, "groups": 12,
         "size_lo": 1, "size_hi": 17, "prefix_lo": 0, "prefix_hi": 3000, "suffix_lo": 1, "suffix_hi": 700},
        # 8 system prompts of about 4,000 tokens, 32 sequences on each (70B head shape)
        {"name": "groups of 32 bf16", "op": "groups", "pool": "bf16", "hq": 64, "hkv": 8, "d": 128, "groups": 8,
         "size_lo": 32, "size_hi": 32, "prefix_lo": 3900, "prefix_hi": 4100, "suffix_lo": 200, "suffix_hi": 500},
        # long documents behind fp8 caches, a few questions on each
        {"name": "groups long fp8", "op": "groups", "pool": "fp8", "hq": 64, "hkv": 8, "d": 128, "groups": 4,
         "size_lo": 3, "size_hi": 6, "prefix_lo": 24000, "prefix_hi": 40000, "suffix_lo": 20, "suffix_hi": 900},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["rope", "cross", "groups"])
    hq, hkv = rng.choice([(32, 8), (64, 8), (16, 16), (32, 4), (8, 2), (12, 4)])
    d = rng.choice([64, 128])
    c = {"op": op, "pool": rng.choice(["bf16", "f16", "int8", "fp8", "int4"]), "hq": hq, "hkv": hkv, "d": d}
    if op == "rope":
        if c["pool"] == "int4":
            c["pool"] = "int8"
        t = _log(rng, 1, 12000)
        c.update(rot=rng.choice([d, d, d // 2]), inter=rng.random() < 0.5, tokens=t, run=_log(rng, 1, t),
                 fused=rng.random() < 0.5, pad=rng.choice([0, min(t - 1, rng.randint(0, 9))]))
    elif op == "cross":
        hi = _log(rng, 1, 900)
        b = max(1, min(_log(rng, 1, 128), 4096 // hi))
        ctx = _log(rng, 20, min(6000, 24000 // b + 600))
        c.update(batch=b, rows_lo=rng.randint(1, hi), rows_hi=hi, ctx_lo=rng.randint(0, ctx), ctx_hi=ctx,
                 pad=rng.randint(0, 7))
    else:
        hi = _log(rng, 1, 40)
        n = max(1, min(_log(rng, 1, 32), 200 // hi))
        pre = _log(rng, 16, min(40000, 400000 // (n * hi)))
        suf = _log(rng, 1, 900)
        c.update(groups=n, size_lo=rng.randint(1, hi), size_hi=hi, prefix_lo=rng.randint(0, pre), prefix_hi=pre,
                 suffix_lo=rng.randint(1, suf), suffix_hi=suf)
    return c


def _spread(case, what, n, lo, hi):
    """n whole numbers in [lo, hi] that go with the case alone; the largest is hi."""
    r = random.Random("%s %d %d %d" % (what, n, lo, hi))
    v = [r.randint(lo, hi) for _ in range(n)]
    v[r.randrange(n)] = hi
    return v


def _starts(v):
    s = [0]
    for x in v:
        s.append(s[-1] + x)
    return s


def _row_bytes(pool, d):
    return {"f16": 2 * d, "bf16": 2 * d, "int8": d, "fp8": d, "int4": d // 2}[pool]


def _sizes(case):
    """The lengths of a case: of its sequences, groups and tables."""
    if case["op"] == "rope":
        t, run = case["tokens"], case["run"]
        real = t - case["pad"]
        lens = [min(run, real - i) for i in range(0, real, run)]
        return {"lens": lens, "real": real}
    if case["op"] == "cross":
        rows = _spread(case, "rows", case["batch"], case["rows_lo"], case["rows_hi"])
        ctx = _spread(case, "ctx", case["batch"], case["ctx_lo"], case["ctx_hi"])
        return {"rows": rows, "ctx": ctx}
    sizes = _spread(case, "sizes", case["groups"], case["size_lo"], case["size_hi"])
    prefix = [p // BLOCK * BLOCK for p in _spread(case, "prefix", case["groups"], case["prefix_lo"], case["prefix_hi"])]
    suffix = _spread(case, "suffix", sum(sizes), case["suffix_lo"], case["suffix_hi"])
    ctx, i = [], 0
    for n, p in zip(sizes, prefix):
        ctx += [p + s for s in suffix[i:i + n]]
        i += n
    return {"sizes": sizes, "prefix": prefix, "suffix": suffix, "ctx": ctx}


def work(case):
    z, hq, hkv, d = _sizes(case), case["hq"], case["hkv"], case["d"]
    row = _row_bytes(case["pool"], d)
    scale = 8.0 / BLOCK if case["pool"] in LIMIT else 0.0   # a K and a V scale for every block and head
    if case["op"] == "rope":
        n = z["real"]
        moved = n * (2 * hq * d * 2 + 2 * hkv * d * 2 + 2 * hkv * row + case["rot"] * 4 + 8) + n * hkv * scale
        return {"bytes": moved, "flops": n * (hq + hkv) * case["rot"] * 3}
    if case["op"] == "cross":
        rows, ctx = z["rows"], z["ctx"]
        cached = sum(ctx) * hkv * (2 * row + scale) + sum(ctx) / BLOCK * 4
        pairs = sum(r * c for r, c in zip(rows, ctx))
        return {"bytes": cached + sum(rows) * hq * d * 4, "flops": 4 * d * hq * pairs}
    held = sum(z["prefix"]) + sum(z["suffix"])
    return {"bytes": held * hkv * (2 * row + scale) + held / BLOCK * 4 + sum(z["sizes"]) * hq * d * 4,
            "flops": 4 * d * hq * sum(z["ctx"])}


# ----------------------------------------------------------------- inputs --

def _side(case, shape, gen, dev):
    """One of K and V as a cache of earlier tokens holds it, and its scales."""
    x = torch.randn(*shape, case["d"], generator=gen, device=dev)
    if case["pool"] in TORCH16:
        return x.to(TORCH16[case["pool"]]), None
    spread = {"int8": 40, "fp8": 120, "int4": 2.5}[case["pool"]]
    x = (x * spread).clamp(-LIMIT[case["pool"]], LIMIT[case["pool"]])
    if case["pool"] == "fp8":
        x = x.to(torch.float8_e4m3fn).view(torch.uint8)
    elif case["pool"] == "int8":
        x = x.round().to(torch.int8).view(torch.uint8)
    else:
        x = x.round().to(torch.int32) & 15
        x = (x[..., 0::2] | (x[..., 1::2] << 4)).to(torch.uint8)
    return x.contiguous(), (torch.rand(*shape[:3], generator=gen, device=dev) + 0.5) / spread


def _pool(case, blocks, gen, dev):
    """K and V of one layer, [1][blocks][heads][16][row]."""
    shape = (1, blocks, case["hkv"], BLOCK)
    (k, ks), (v, vs) = _side(case, shape, gen, dev), _side(case, shape, gen, dev)
    return {"k": k, "v": v, "ks": ks, "vs": vs}


def _handle(case, s):
    """The handle that a program keeps on its pool."""
    from paged_kv_cache_431_b200 import pkv
    status = torch.zeros(1, dtype=torch.int32, device=s["k"].device)
    return pkv.KVPool(s["k"], s["v"], DTYPE[case["pool"]], case["d"], s["ks"], s["vs"], device_status=status)


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=dev).manual_seed(seed + 1)
    z, hq, hkv, d = _sizes(case), case["hq"], case["hkv"], case["d"]
    dt16 = TORCH16.get(case["pool"], torch.bfloat16)
    s = {"case": case, "scale": d ** -0.5}

    def i32(v):
        return torch.as_tensor(v, dtype=torch.int32).to(dev)

    if case["op"] == "rope":
        t, lens = case["tokens"], z["lens"]
        # every sequence goes on from a position of its own, in the middle of a block
        first = [int(x) for x in torch.randint(0, MAX_POSITIONS - max(lens), (len(lens),), generator=host)]
        need = [(p + n - 1) // BLOCK - p // BLOCK + 1 for p, n in zip(first, lens)]
        blocks = sum(need) + 8
        s.update(_pool(case, blocks, gen, dev))
        at, ends = torch.tensor(first), torch.tensor(_starts(need)[:-1])
        seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens))
        inner = torch.arange(len(seq)) - torch.tensor(_starts(lens)[:-1])[seq]
        pos = at[seq] + inner
        perm = torch.randperm(blocks, generator=host)
        slot = perm[ends[seq] + pos // BLOCK - at[seq] // BLOCK] * BLOCK + pos % BLOCK
        pad = case["pad"]
        s["positions"] = i32(torch.cat([pos, torch.zeros(pad, dtype=torch.long)]))
        s["slots"] = i32(torch.cat([slot, torch.full((pad,), -1)]))
        if case["fused"]:    # one projection's output holds q, k and v of a token side by side
            x = torch.randn(t, (hq + 2 * hkv) * d, generator=gen, device=dev).to(dt16)
            q, k, v = x.split([hq * d, hkv * d, hkv * d], dim=1)
        else:
            q, k, v = (torch.randn(t, h * d, generator=gen, device=dev).to(dt16) for h in (hq, hkv, hkv))
        s.update(q=q.unflatten(1, (hq, d)), kn=k.unflatten(1, (hkv, d)), vn=v.unflatten(1, (hkv, d)))
        half = case["rot"] // 2
        angle = torch.arange(MAX_POSITIONS, dtype=torch.float64, device=dev)[:, None] * \
            500000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
        s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["out"] = torch.zeros(t, hq, d, dtype=dt16, device=dev)
    else:
        if case["op"] == "cross":
            ctx, rows = z["ctx"], sum(z["rows"]) + case["pad"]
            shared = [0] * len(ctx)
        else:
            ctx, rows = z["ctx"], len(z["ctx"])
            shared = [p // BLOCK for n, p in zip(z["sizes"], z["prefix"]) for _ in range(n)]
        width = max(1, max(-(-c // BLOCK) for c in ctx))
        blocks = sum(-(-c // BLOCK) - m for c, m in zip(ctx, shared)) + 8
        blocks += sum(p // BLOCK for p in z.get("prefix", []))
        s.update(_pool(case, blocks, gen, dev))
        perm = torch.randperm(blocks, generator=host).to(torch.int32)
        tables = torch.full((len(ctx), width), -1, dtype=torch.int32)
        used, b = 0, 0
        for i in range(len(z.get("sizes", ctx))):
            members = range(b, b + z["sizes"][i]) if "sizes" in z else [i]
            common = shared[b] if "sizes" in z else 0
            for m in members:
                n = -(-ctx[m] // BLOCK)
                tables[m, :common] = perm[used:used + common]
            used += common
            for m in members:
                n = -(-ctx[m] // BLOCK)
                tables[m, common:n] = perm[used:used + n - common]
                used += n - common
            b += len(members)
        s.update(tables=tables.to(dev), ctx=i32(ctx))
        s["q"] = (2 * torch.randn(rows, hq, d, generator=gen, device=dev)).to(dt16)
        s["out"] = torch.zeros_like(s["q"])
        if case["op"] == "cross":
            s.update(starts=i32(_starts(z["rows"])), max_rows=max(z["rows"]), max_ctx=max(ctx))
        else:
            s.update(starts=i32(_starts(z["sizes"])), prefix=i32(z["prefix"]), max_size=max(z["sizes"]),
                     max_prefix=max(z["prefix"]), max_suffix=max(z["suffix"]))
    if own:
        s["pool"] = _handle(case, s)
    return s


# -------------------------------------------------------------- plain forms --

def _values(case, x):
    """The numbers that a pool's codes stand for, before their scale; [blocks][heads][16][d]."""
    x = x[0]
    if case["pool"] in TORCH16:
        return x.float()
    if case["pool"] == "int8":
        return x.view(torch.int8).float()
    if case["pool"] == "fp8":
        return x.view(torch.float8_e4m3fn).float()
    n = torch.stack([x & 15, x >> 4], -1).flatten(-2).to(torch.int32)
    return ((n ^ 8) - 8).float()


def _turn(x, cs, inter):
    """Rotates the first dims of x [tokens][heads][d] by the angles whose cosines and sines cs holds."""
    half = cs.shape[1] // 2
    c, sn = cs[:, None, :half], cs[:, None, half:]
    turned, kept = x[..., :2 * half].float(), x[..., 2 * half:].float()
    if inter:
        a, b = turned[..., 0::2], turned[..., 1::2]
        new = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    else:
        a, b = turned[..., :half], turned[..., half:]
        new = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    return torch.cat([new, kept], -1)


def _store(case, pool, scales, x, slots):
    """Writes rows x [tokens][heads][d] to their slots; negative slots are padding."""
    n, h, dev = pool.shape[1], pool.shape[2], pool.device
    blk = torch.where(slots < 0, n, slots // BLOCK).long()
    off = torch.where(slots < 0, 0, slots % BLOCK).long()
    if case["pool"] in TORCH16:
        grown = torch.cat([pool[0], torch.zeros_like(pool[0, :1])])
        grown[blk, :, off] = x
        pool[0].copy_(grown[:n])
        return
    limit = torch.tensor(LIMIT[case["pool"]], device=dev)
    x = x.float()
    amax = torch.zeros(n + 1, h, device=dev).scatter_reduce_(0, blk[:, None].expand(-1, h), x.abs().amax(-1), "amax")
    hit = torch.zeros(n + 1, device=dev).index_add_(0, blk, torch.ones_like(blk, dtype=torch.float32)) > 0
    fresh = torch.zeros(n + 1, device=dev).index_add_(0, blk, (off == 0).float()) > 0
    stored = torch.cat([scales[0], torch.zeros_like(scales[0, :1])])
    old = torch.where(fresh[:, None], 0.0, stored)
    new = torch.where(hit[:, None], torch.maximum(old, amax / limit), stored)

    def code(y):
        y = torch.minimum(torch.maximum(y, -limit), limit)
        return y.to(torch.float8_e4m3fn).float() if case["pool"] == "fp8" else y.round()

    held = torch.cat([_values(case, pool), torch.zeros(1, h, BLOCK, x.shape[-1], device=dev)])
    grows = (hit[:, None] & (new > old) & (old > 0))[..., None, None]
    held = torch.where(grows, code(held * old[..., None, None] / new[..., None, None]), held)
    s = new[blk][..., None]
    held[blk, :, off] = torch.where(s > 0, code(x / s), 0.0)
    kind = torch.float8_e4m3fn if case["pool"] == "fp8" else torch.int8
    pool[0].copy_(held[:n].to(kind).view(torch.uint8))
    scales[0].copy_(new[:n])


def _plain_rope(s):
    case, slots = s["case"], s["slots"]
    cs = s["table"][s["positions"].long()]
    q = _turn(s["q"], cs, case["inter"]).to(s["q"].dtype)
    s["out"].copy_(torch.where((slots < 0)[:, None, None], s["out"], q))
    _store(case, s["k"], s["ks"], _turn(s["kn"], cs, case["inter"]).to(s["kn"].dtype), slots)
    _store(case, s["v"], s["vs"], s["vn"], slots)


def _gather(case, x, scales, tables):
    """One of K and V of every sequence, padded to the widest table: [sequences][heads][keys][d] in 32 bits."""
    x = _values(case, x)
    if scales is not None:
        x = x * scales[0][..., None, None]
    return x[tables.clamp(min=0).long()].transpose(1, 2).flatten(2, 3)


def _attend(q, k, v, seen, scale):
    """q [b][heads][rows][d] against k, v [b][heads][keys][d]; seen [b][keys]. Rows that see nothing are 0."""
    seen = seen[:, None, None, :]
    x = torch.where(seen, q @ k.transpose(-1, -2) * scale, -torch.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isfinite(top), top, 0.0))
    total = p.sum(-1, keepdim=True)
    return (p @ torch.where(seen.transpose(-1, -2), v, 0.0)) / torch.where(total > 0, total, 1.0)


def _plain_cross(s):
    case = s["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    k, v = _gather(case, s["k"], s["ks"], s["tables"]), _gather(case, s["v"], s["vs"], s["tables"])
    seen = torch.arange(k.shape[2], device=k.device) < s["ctx"][:, None]
    starts, n = s["starts"].long(), s["max_rows"]
    at = starts[:-1, None] + torch.arange(n, device=k.device)
    there = at < starts[1:, None]
    at = torch.where(there, at, 0)
    q = s["q"][at].float()                                             # [b][rows][hq][d]
    b = q.shape[0]
    q = q.view(b, n, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).flatten(2, 3)
    o = _attend(q, k, v, seen, s["scale"])
    o = o.view(b, hkv, n, hq // hkv, d).transpose(1, 2).reshape(b, n, hq, d).to(s["q"].dtype)
    rows = s["q"].shape[0]
    whole = torch.cat([s["out"], s["out"][:1]])                       # the last row takes what is padding
    whole[torch.where(there, at, rows)] = o
    s["out"].copy_(whole[:rows])


def _plain_groups(s):
    case = s["case"]
    k, v = _gather(case, s["k"], s["ks"], s["tables"]), _gather(case, s["v"], s["vs"], s["tables"])
    seen = torch.arange(k.shape[2], device=k.device) < s["ctx"][:, None]
    q = s["q"].float().unflatten(1, (case["hkv"], -1))
    s["out"].copy_(_attend(q, k, v, seen, s["scale"]).flatten(1, 2))


def _whole(s):
    """What the pass left, with codes as the 8-bit numbers that they are."""
    case = s["case"]
    if case["op"] != "rope":
        return {"out": s["out"]}
    kind = {"int8": torch.int8, "fp8": torch.float8_e4m3fn}.get(case["pool"])
    r = {"q": s["out"], "k": s["k"] if kind is None else s["k"].view(kind), "v": s["v"] if kind is None else s["v"].view(kind)}
    if kind is not None:
        r.update(ks=s["ks"], vs=s["vs"])
    return r


def run(s):
    case = s["case"]
    if own:
        from paged_kv_cache_431_b200 import pkv
        if case["op"] == "rope":
            pkv.kv_append_rope(s["pool"], 0, s["q"], s["kn"], s["vn"], s["positions"], s["table"], s["slots"],
                               q_out=s["out"], interleaved=case["inter"])
        elif case["op"] == "cross":
            pkv.paged_cross_attn(s["pool"], 0, s["q"], s["starts"], s["tables"], s["ctx"], s["scale"],
                                 s["max_rows"], s["max_ctx"], out=s["out"])
        else:
            pkv.paged_decode_attn_groups(s["pool"], 0, s["q"], s["tables"], s["ctx"], s["starts"], s["prefix"],
                                         s["scale"], s["max_size"], s["max_prefix"], s["max_suffix"], out=s["out"])
    else:
        {"rope": _plain_rope, "cross": _plain_cross, "groups": _plain_groups}[case["op"]](s)
    return _whole(s)


# -------------------------------------------------------- 64-bit definitions --

def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return _exact_rope(case, s) if case["op"] == "rope" else {"out": _exact_attention(case, s)}


def _exact_rope(case, s):
    d, rot = case["d"], case["rot"]
    live = (s["slots"] >= 0).nonzero()[:, 0]
    slots = s["slots"][live].long()
    cs = s["table"].double()[s["positions"][live].long()]
    turn = torch.complex(cs[:, :rot // 2], cs[:, rot // 2:])[:, None]

    def rotated(x):
        x = x[live].double()
        if case["inter"]:
            first, second = torch.arange(0, rot, 2), torch.arange(1, rot, 2)
        else:
            first, second = torch.arange(rot // 2), torch.arange(rot // 2, rot)
        w = torch.complex(x[..., first], x[..., second]) * turn
        x[..., first], x[..., second] = w.real, w.imag
        return x

    q = s["out"].double()
    q[live] = rotated(s["q"])
    r = {"q": q, "k": None, "v": None}
    for name, rows in (("k", rotated(s["kn"])), ("v", s["vn"][live].double())):
        pool, scales = s[name][0], s[name + "s"]
        if scales is None:
            by_slot = pool.double().transpose(1, 2).reshape(-1, case["hkv"], d)
            by_slot[slots] = rows
            r[name] = by_slot.view(-1, BLOCK, case["hkv"], d).transpose(1, 2)[None]
            continue
        limit = LIMIT[case["pool"]]
        rows = rows.to(s["kn"].dtype).double()      # a row is stored as the model's type holds it
        scale = scales[0].double()
        blk = slots // BLOCK
        started = torch.zeros(len(pool), dtype=torch.bool, device=pool.device)
        started[blk[slots % BLOCK == 0]] = True
        old = torch.where(started[:, None], 0.0, scale)
        top = torch.full_like(scale, -1.0).index_reduce(0, blk, rows.abs().amax(-1), "amax")
        scale = torch.where(top >= 0, torch.maximum(old, top / limit), scale)
        if case["pool"] == "fp8":
            def near(y):
                return y.clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
            codes = pool.view(torch.float8_e4m3fn).double()
            more = (top >= 0) & (scale > old) & (old > 0)
            again = near(codes * (old / scale.clamp(min=1e-300))[..., None, None])
            codes = torch.where(more[..., None, None], again, codes)
            by_slot = codes.transpose(1, 2).reshape(-1, case["hkv"], d)
            by_slot[slots] = near(rows / scale[blk][..., None].clamp(min=1e-300))
            r[name] = by_slot.view(-1, BLOCK, case["hkv"], d).transpose(1, 2)[None]
        r[name + "s"] = scale[None]
    return r


def _exact_attention(case, s):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    out = s["out"].double()
    tables, ctx = s["tables"].cpu(), s["ctx"].tolist()
    if case["op"] == "cross":
        starts = s["starts"].tolist()
    else:
        starts = list(range(len(ctx) + 1))
    pools = []
    for x, sc in ((s["k"], s["ks"]), (s["v"], s["vs"])):
        x = x[0]
        if case["pool"] == "int4":
            low, high = (x & 15).to(torch.int8), (x >> 4).to(torch.int8)
            x = torch.empty(*x.shape[:-1], d, dtype=torch.int8, device=x.device)
            x[..., 0::2], x[..., 1::2] = low, high
            x = torch.where(x > 7, x - 16, x)
        elif case["pool"] == "int8":
            x = x.view(torch.int8)
        elif case["pool"] == "fp8":
            x = x.view(torch.float8_e4m3fn)
        pools.append((x, None if sc is None else sc[0]))
    for b, n in enumerate(ctx):
        if n == 0:
            out[starts[b]:starts[b + 1]] = 0.0
            continue
        used = tables[b, :(n + BLOCK - 1) // BLOCK].long().to(out.device)
        held = []
        for x, sc in pools:
            x = x.view(torch.uint8)[used].view(x.dtype).double() if x.dtype == torch.float8_e4m3fn else x[used].double()
            if sc is not None:
                x = x * sc[used].double()[:, :, None, None]
            held.append(x.permute(1, 0, 2, 3).reshape(hkv, -1, d)[:, :n])
        k, v = held
        q = s["q"][starts[b]:starts[b + 1]].double()
        for g in range(hkv):
            heads = slice(g * (hq // hkv), (g + 1) * (hq // hkv))
            w = torch.softmax(torch.matmul(q[:, heads], k[g].t()) * s["scale"], -1)
            out[starts[b]:starts[b + 1], heads] = torch.matmul(w, v[g])
    return out
