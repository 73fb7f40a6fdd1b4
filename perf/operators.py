"""Measured cases of the paged-cache operators of a decode step.

Four operators of ``paged_kv_cache_464_b200.capi``, each with a plain form in
elementary torch operations:

* ``append``  ``rope_and_cache`` / ``rope_and_cache_fp8``: rotate q and the new
  keys by their positions and write keys and values to their cache slots.
* ``shared``  ``decode_shared_prefix``: decode attention of groups of sequences
  that share a long prefix.
* ``bounds``  ``update_block_bounds``: per-channel minimum and maximum of the
  keys of every block that got new tokens.
* ``sparse``  ``select_blocks`` then ``decode_selected``: choose each query's
  blocks by those bounds, then attend to the chosen blocks only.
"""
import math
import random

import torch

own = False   # set by the tools: False = the plain forms, True = the framework's kernels

BS = 16       # tokens per cache block
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ROW = {"f32": 64, "f16": 128, "bf16": 128}    # head_dim: a (token, KV head) row is 256 bytes


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 32 sequences: one new token each, latency counts
        dict(name="append decode 32", op="append", type="bf16", cache="same", heads=32, kv_heads=8, tokens=32, chunk=1,
             padding=0, rotary=128, interleaved=False, base=500000.0, far=131072),
        # a prefill step: 16 chunks of 512 tokens, 32/8 heads
        dict(name="append chunks 8192", op="append", type="bf16", cache="same", heads=32, kv_heads=8, tokens=8192,
             chunk=512, padding=0, rotary=128, interleaved=False, base=500000.0, far=8192),
        # a padded prefill step into an E4M3 cache, adjacent pairs, part of each head rotated
        dict(name="append fp8 padded 4093", op="append", type="f16", cache="fp8", heads=32, kv_heads=8, tokens=4093,
             chunk=341, padding=37, rotary=64, interleaved=True, base=10000.0, far=32768),
        # a handful of requests over one system prompt, eight grouped heads
        dict(name="shared 5 x 4000", op="shared", type="bf16", heads=64, kv_heads=8, groups="5", prefix="4000",
             suffix_lo=1, suffix_hi=130, mix=3),
        # the shared-prefix decode workload: 128 sequences, a 1024-token prefix, suffixes U[16, 512]
        dict(name="shared 128 x 1024", op="shared", type="bf16", heads=32, kv_heads=8, groups="128", prefix="1024",
             suffix_lo=16, suffix_hi=512, mix=4),
        # three groups of unequal size, one of them without a prefix, one KV head per query head
        dict(name="shared groups 47 mha", op="shared", type="f16", heads=32, kv_heads=32, groups="29,11,7",
             prefix="2048,1520,0", suffix_lo=0, suffix_hi=300, mix=5),
        # many questions to one long document
        dict(name="shared 64 x 32768", op="shared", type="bf16", heads=32, kv_heads=8, groups="64", prefix="32768",
             suffix_lo=16, suffix_hi=512, mix=6),
        # one decode step of 256 sequences: one block of each has a new token
        dict(name="bounds decode 256", op="bounds", type="bf16", kv_heads=8, seqs=256, context_lo=128,
             context_hi=2048, new_lo=1, new_hi=1, mix=7),
        # a prefill step of 16 chunks of 512 tokens
        dict(name="bounds chunks 16 x 512", op="bounds", type="bf16", kv_heads=8, seqs=16, context_lo=512,
             context_hi=2047, new_lo=512, new_hi=512, mix=8),
        # one long request
        dict(name="sparse 1 x 32768", op="sparse", type="bf16", heads=64, kv_heads=8, seqs=1, context_lo=32768,
             context_hi=32768, selected=64, sink=1, recent=4, mix=9),
        # the long-context decode workload: 8 sequences of 32768 tokens, 64/8 heads
        dict(name="sparse 8 x 32768", op="sparse", type="bf16", heads=64, kv_heads=8, seqs=8, context_lo=32768,
             context_hi=32768, selected=128, sink=1, recent=8, mix=10),
        # a mixed batch: some sequences have fewer blocks than are chosen
        dict(name="sparse 61 mixed", op="sparse", type="f16", heads=32, kv_heads=8, seqs=61, context_lo=1,
             context_hi=8192, selected=33, sink=2, recent=2, mix=11),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "shared", "bounds", "sparse"])
    ty = rng.choice(["bf16", "f16"] if op == "shared" else ["bf16", "f16", "f32"])
    mix = rng.randrange(1 << 30)
    kv = rng.choice([1, 2, 3, 4, 5, 8])
    group = rng.choice([1, 2, 4, 8])
    if op == "append":
        tokens = _log(rng, 1, 8192)
        chunk = max(1, tokens // rng.choice([1, 3, 8, 64]))
        d = ROW[ty]
        return dict(op=op, type=ty, cache=rng.choice(["same", "same", "fp8"]) if ty != "f32" else "same",
                    heads=kv * group, kv_heads=kv, tokens=tokens, chunk=chunk, padding=rng.choice([0, 0, 1, tokens // 9]),
                    rotary=rng.choice([d, d, d // 2, d // 4]), interleaved=rng.random() < 0.4,
                    base=rng.choice([10000.0, 500000.0]), far=max(_log(rng, 512, 131072), tokens))
    if op == "shared":
        n = rng.choice([1, 1, 1, 2, 5])
        sizes, prefixes = [], []
        for _ in range(n):
            size = _log(rng, 1, max(1, 160 // n))
            # every sequence's context, read as often as there are sequences, stays below the largest case's
            sizes.append(size)
            prefixes.append(BS * rng.choice([_log(rng, 1, 1024), _log(rng, 1, 1024), 0] if n > 1 else [_log(rng, 1, 1024)]))
        while sum(sizes) * (max(prefixes) + 600) * kv > 64 * 33280 * 8:
            sizes = [max(1, s // 2) for s in sizes]
        lo = rng.choice([0, 1, 16])
        return dict(op=op, type=ty, heads=kv * group, kv_heads=kv, groups=",".join(map(str, sizes)),
                    prefix=",".join(map(str, prefixes)), suffix_lo=lo, suffix_hi=lo + _log(rng, 1, 500), mix=mix)
    if op == "bounds":
        seqs = _log(rng, 1, 256)
        hi = _log(rng, 2, max(2, min(8192, 500000 // seqs)))
        new = rng.choice([1, 1, _log(rng, 1, hi)])
        return dict(op=op, type=ty, kv_heads=kv, seqs=seqs, context_lo=max(1, hi // 5), context_hi=hi,
                    new_lo=rng.choice([0, new]), new_hi=new, mix=mix)
    seqs = _log(rng, 1, 64)
    hi = _log(rng, 64, max(64, min(32768, 262144 // seqs)))
    sink, recent = rng.choice([0, 1, 3]), rng.choice([1, 2, 8])
    return dict(op=op, type=ty, heads=kv * group, kv_heads=kv, seqs=seqs, context_lo=max(1, hi // rng.choice([1, 2, 50])),
                context_hi=hi, selected=sink + recent + _log(rng, 1, 150), sink=sink, recent=recent, mix=mix)


def _between(case, n, lo, hi, salt):
    """n lengths of [lo, hi], the case's own (the amount of work is part of the case)."""
    rng = random.Random(case["mix"] * 8 + salt)
    return [rng.randint(lo, hi) for _ in range(n)]


def _shared_lens(case):
    sizes = [int(x) for x in case["groups"].split(",")]
    prefixes = [int(x) for x in case["prefix"].split(",")]
    suffix = _between(case, sum(sizes), case["suffix_lo"], case["suffix_hi"], 0)
    per_seq = [p for s, p in zip(sizes, prefixes) for _ in range(s)]
    return sizes, prefixes, per_seq, suffix


def work(case):
    ty = TYPES[case["type"]]
    es, d = ty.itemsize, ROW[case["type"]]
    row = es * d
    if case["op"] == "append":
        t = case["tokens"] - case["padding"]
        out_row = d if case["cache"] == "fp8" else row
        angles = min(t, case["far"]) * case["rotary"] * 4
        return {"bytes": t * (case["heads"] * 2 * row + case["kv_heads"] * 2 * (row + out_row)) + angles + t * 16,
                "flops": t * (case["heads"] + case["kv_heads"]) * case["rotary"] * 3}
    if case["op"] == "shared":
        sizes, prefixes, per_seq, suffix = _shared_lens(case)
        once = sum(p for s, p in zip(sizes, prefixes) if s) + sum(suffix)
        total = sum(per_seq) + sum(suffix)
        return {"bytes": once * case["kv_heads"] * 2 * row + 2 * len(suffix) * case["heads"] * row,
                "flops": 4 * total * case["heads"] * d}
    if case["op"] == "bounds":
        ctx, new = _bounds_lens(case)
        blocks = sum(-(-c // BS) - (c - n) // BS for c, n in zip(ctx, new) if n)
        tokens = sum(c - (c - n) // BS * BS for c, n in zip(ctx, new) if n)
        return {"bytes": (tokens + 2 * blocks) * case["kv_heads"] * row, "flops": 2 * tokens * case["kv_heads"] * d}
    ctx = _between(case, case["seqs"], case["context_lo"], case["context_hi"], 0)
    blocks = [-(-c // BS) for c in ctx]
    kept = sum(min(c, case["selected"] * BS) for c in ctx)
    return {"bytes": (sum(blocks) + kept) * case["kv_heads"] * 2 * row + 2 * len(ctx) * case["heads"] * row
            + 2 * len(ctx) * case["kv_heads"] * case["selected"] * 4,
            "flops": (2 * sum(blocks) + 4 * kept) * case["heads"] * d}


def _bounds_lens(case):
    ctx = _between(case, case["seqs"], case["context_lo"], case["context_hi"], 0)
    new = [min(c, n) for c, n in zip(ctx, _between(case, case["seqs"], case["new_lo"], case["new_hi"], 1))]
    return ctx, new


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, shape, ty):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(ty)


def _ints(values, ty=torch.int32):
    return torch.tensor(values, device="cuda", dtype=ty)


def _tables(g, blocks, spare=8):
    """Shuffled physical ids for sequences of `blocks` blocks each; -1 past a sequence's last."""
    most, total = max(1, max(blocks)), sum(blocks)
    perm = torch.randperm(total + spare, generator=g, device="cuda").to(torch.int32)
    first = torch.cumsum(_ints([0] + blocks[:-1]), 0)
    col = torch.arange(most, device="cuda")
    at = first[:, None] + col
    live = col < _ints(blocks)[:, None]
    return torch.where(live, perm[torch.where(live, at, 0).long()], -1).to(torch.int32).contiguous(), total + spare


def _stale(cache, tables, lens):
    """What a cache holds past a sequence's end: the slots of its last block that have no token yet."""
    last = (torch.clamp(lens, min=1) - 1) // BS
    block = torch.gather(tables, 1, last[:, None].long())[:, 0]
    dead = torch.arange(BS, device="cuda") >= ((lens - 1) % BS + 1)[:, None]
    use = (block >= 0) & (lens > 0)
    at = torch.where(use, block, 0).long()
    rows = cache[at]
    filled = torch.where((dead & use[:, None])[:, :, None, None], torch.full_like(rows, float("nan")), rows)
    cache[at[use]] = filled[use]


def prepare(case, seed):
    g = _gen(seed)
    ty, d = TYPES[case["type"]], ROW[case["type"]]
    hkv = case["kv_heads"]
    s = dict(case)
    if case["op"] == "append":
        t, pad, heads, r = case["tokens"], case["padding"], case["heads"], case["rotary"]
        live = t - pad
        s["qkv"] = _randn(g, (t, heads + 2 * hkv, d), ty)      # one projection's output
        chunks = -(-live // case["chunk"]) if live else 1
        start = torch.randint(0, max(1, case["far"] - case["chunk"] + 1), (chunks,), generator=g, device="cuda")
        i = torch.arange(live, device="cuda")
        pos = start[i // case["chunk"]] + i % case["chunk"]
        pool = -(-live // BS) + 8
        # a chunk fills its blocks in order; a decode step's tokens each go to a block of their own
        if case["chunk"] == 1:
            pool = live + 8
            block = torch.randperm(pool, generator=g, device="cuda")[:live]
            slot = block * BS + pos % BS
        else:
            slot = torch.randperm(pool, generator=g, device="cuda")[i // BS] * BS + i % BS
        fill = torch.full((pad,), -1, device="cuda", dtype=torch.int64)
        s["positions"], s["slots"] = torch.cat([pos, fill]), torch.cat([slot, fill])
        angle = torch.arange(case["far"], device="cuda", dtype=torch.float64)[:, None] * torch.pow(
            torch.tensor(case["base"], device="cuda", dtype=torch.float64),
            -torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        kind = torch.float8_e4m3fn if case["cache"] == "fp8" else ty
        s["k_cache"] = torch.zeros((pool, BS, hkv, d), device="cuda", dtype=torch.float32).to(kind)
        s["v_cache"] = s["k_cache"].clone()
        s["q_out"] = torch.zeros((t, heads, d), device="cuda", dtype=ty)
        s["k_scale"], s["v_scale"] = 0.0125, 0.0125
        return s
    if case["op"] == "shared":
        sizes, prefixes, per_seq, suffix = _shared_lens(case)
        own_blocks = [-(-x // BS) for x in suffix]
        tails, pool = _tables(g, own_blocks)
        n_prefix = [p // BS for p in prefixes]
        perm = torch.randperm(pool + sum(n_prefix), generator=g, device="cuda").to(torch.int32)
        most = max(1, max(p // BS + b for p, b in zip(per_seq, own_blocks)))
        tables = torch.full((len(suffix), most), -1, device="cuda", dtype=torch.int32)
        at, row = pool, 0
        for size, n in zip(sizes, n_prefix):
            tables[row:row + size, :n] = perm[at:at + n]
            for b in range(row, row + size):
                tables[b, n:n + own_blocks[b]] = perm[tails[b, :own_blocks[b]].long()]
            at, row = at + n, row + size
        lens = [p + x for p, x in zip(per_seq, suffix)]
        s["tables"], s["lens"] = tables, _ints(lens)
        starts = [0]
        for size in sizes:
            starts.append(starts[-1] + size)
        s["group_start"], s["prefix_lens"] = _ints(starts), _ints(prefixes)
        s["max_prefix"], s["max_suffix"], s["max_size"] = max(prefixes), max(suffix), max(sizes)
        pool += sum(n_prefix)
        s["k_cache"] = _randn(g, (pool, BS, hkv, d), ty)
        s["v_cache"] = _randn(g, (pool, BS, hkv, d), ty)
        _stale(s["k_cache"], tables, s["lens"])
        _stale(s["v_cache"], tables, s["lens"])
        s["q"] = _randn(g, (len(lens), case["heads"], d), ty)
        s["out"] = torch.empty_like(s["q"])
        s["scale"] = d ** -0.5
        return s
    if case["op"] == "bounds":
        ctx, new = _bounds_lens(case)
        s["tables"], pool = _tables(g, [-(-c // BS) for c in ctx])
        s["lens"], s["new"] = _ints(ctx), _ints(new)
        s["max_new"] = max(new)
        s["k_cache"] = _randn(g, (pool, BS, hkv, d), ty)
        _stale(s["k_cache"], s["tables"], s["lens"])
        s["bounds"] = torch.zeros((pool, 2, hkv, d), device="cuda", dtype=ty)
        return s
    ctx = _between(case, case["seqs"], case["context_lo"], case["context_hi"], 0)
    s["tables"], pool = _tables(g, [-(-c // BS) for c in ctx])
    s["lens"] = _ints(ctx)
    # keys of neighbouring tokens have something in common, so that blocks differ in what they offer a query
    common = torch.randn((pool, 1, hkv, d), generator=g, device="cuda")
    s["k_cache"] = (0.6 * torch.randn((pool, BS, hkv, d), generator=g, device="cuda") + 0.8 * common).to(ty)
    s["v_cache"] = _randn(g, (pool, BS, hkv, d), ty)
    s["q"] = _randn(g, (len(ctx), case["heads"], d), ty)
    # the bounds as the cache has them: full blocks from all tokens, a last block from those it holds
    s["bounds"] = torch.stack([s["k_cache"].amin(1), s["k_cache"].amax(1)], 1)
    ids, rows, live = _last_blocks(s["k_cache"], s["tables"], s["lens"])
    low = torch.where(live, rows, float("inf")).amin(1)
    high = torch.where(live, rows, float("-inf")).amax(1)
    s["bounds"][ids] = torch.stack([low, high], 1)
    s["max_context"] = max(ctx)
    _stale(s["k_cache"], s["tables"], s["lens"])
    _stale(s["v_cache"], s["tables"], s["lens"])
    s["chosen"] = torch.empty((len(ctx), hkv, case["selected"]), device="cuda", dtype=torch.int32)
    s["out"] = torch.empty_like(s["q"])
    s["scale"] = d ** -0.5
    return s


def _last_blocks(cache, tables, lens):
    ids = torch.gather(tables, 1, ((lens - 1) // BS)[:, None].long())[:, 0].long()
    live = torch.arange(BS, device="cuda") <= ((lens - 1) % BS)[:, None]
    return ids, cache[ids], live[:, :, None, None]


# ------------------------------------------------------------------ one pass
def run(s):
    return _OWN[s["op"]](s) if own else _PLAIN[s["op"]](s)


def _split(s):
    heads, hkv = s["heads"], s["kv_heads"]
    return s["qkv"][:, :heads], s["qkv"][:, heads:heads + hkv], s["qkv"][:, heads + hkv:]


def _own_append(s):
    from paged_kv_cache_464_b200 import capi
    q, k, v = _split(s)
    if s["cache"] == "fp8":
        capi.rope_and_cache_fp8(q, k, v, s["positions"], s["cos_sin"], s["k_cache"], s["v_cache"], s["slots"],
                                s["k_scale"], s["v_scale"], s["q_out"], interleaved=s["interleaved"])
    else:
        capi.rope_and_cache(q, k, v, s["positions"], s["cos_sin"], s["k_cache"], s["v_cache"], s["slots"], s["q_out"],
                            interleaved=s["interleaved"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_shared(s):
    from paged_kv_cache_464_b200 import capi
    if "workspace" not in s:   # a serving loop's scratch, kept from step to step
        need = capi.decode_shared_prefix_workspace_bytes(len(s["lens"]), len(s["prefix_lens"]), s["heads"],
                                                         s["kv_heads"], s["q"].shape[2], s["max_prefix"],
                                                         s["max_suffix"], s["max_size"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return capi.decode_shared_prefix(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["group_start"],
                                     s["prefix_lens"], s["scale"], s["out"], max_prefix_len=s["max_prefix"],
                                     max_suffix_len=s["max_suffix"], max_group_size=s["max_size"],
                                     workspace=s["workspace"])


def _own_bounds(s):
    from paged_kv_cache_464_b200 import capi
    capi.update_block_bounds(s["k_cache"], s["bounds"], s["tables"], s["lens"], s["new"], max_new_len=s["max_new"])
    return s["bounds"]


def _own_sparse(s):
    from paged_kv_cache_464_b200 import capi
    if "workspace" not in s:
        n, hkv, d = len(s["lens"]), s["kv_heads"], s["q"].shape[2]
        need = max(capi.select_blocks_workspace_bytes(n, hkv, s["max_context"]),
                   capi.decode_selected_workspace_bytes(n, s["heads"], hkv, d, s["selected"]))
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    capi.select_blocks(s["q"], s["bounds"], s["tables"], s["lens"], s["chosen"], sink_blocks=s["sink"],
                       recent_blocks=s["recent"], max_context_len=s["max_context"], workspace=s["workspace"])
    capi.decode_selected(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["chosen"], s["scale"], s["out"],
                         workspace=s["workspace"])
    return {"chosen": s["chosen"], "out": s["out"]}


def _plain_rotate(x, cos, sin, rotary, interleaved):
    x = x.float()
    turned, rest = x[..., :rotary], x[..., rotary:]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if interleaved else turned.chunk(2, -1)
    c, d = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([c, d], -1).flatten(-2) if interleaved else torch.cat([c, d], -1)
    return torch.cat([turned, rest], -1)


def _plain_append(s):
    q, k, v = _split(s)
    at = s["cos_sin"][s["positions"].clamp(min=0)]
    cos, sin = (x[:, None, :] for x in at.chunk(2, -1))
    live = s["positions"] >= 0
    turned = _plain_rotate(q, cos, sin, s["rotary"], s["interleaved"]).to(q.dtype)
    s["q_out"].copy_(torch.where(live[:, None, None], turned, s["q_out"]))
    k, v = _plain_rotate(k, cos, sin, s["rotary"], s["interleaved"]), v.float()
    if s["cache"] == "fp8":
        k, v = (k / s["k_scale"]).clamp(-448, 448), (v / s["v_scale"]).clamp(-448, 448)
    use = s["slots"] >= 0
    for cache, rows in ((s["k_cache"], k), (s["v_cache"], v)):
        flat = cache.view(-1, *cache.shape[2:])
        if s["cache"] == "fp8":   # one byte each: the codes move as bytes
            flat.view(torch.uint8)[s["slots"][use]] = rows[use].to(cache.dtype).view(torch.uint8)
        else:
            flat[s["slots"][use]] = rows[use].to(cache.dtype)
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attention(s, mask):
    """softmax(scale q K^T) V in 32 bits over the tokens that mask [S, 1 or Hkv, tokens] leaves."""
    q = s["q"]
    n, heads, d = q.shape
    hkv = s["kv_heads"]
    at = s["tables"].clamp(min=0).long()
    length = at.shape[1] * BS
    live = (torch.arange(length, device="cuda") < s["lens"][:, None])[:, :, None, None]
    k = torch.where(live, s["k_cache"][at].view(n, length, hkv, d), 0).float()
    score = torch.einsum("bgid,btgd->bgit", q.view(n, hkv, -1, d).float(), k) * s["scale"]
    del k
    score = torch.where(mask[:, :, None], score, float("-inf"))
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - torch.where(top == float("-inf"), 0, top))
    total = weight.sum(-1)
    del score
    v = torch.where(live, s["v_cache"][at].view(n, length, hkv, d), 0).float()
    out = torch.einsum("bgit,btgd->bgid", weight, v)
    out = torch.where(total[..., None] > 0, out / total[..., None], 0)
    return out.reshape(n, heads, d).to(q.dtype)


def _plain_shared(s):
    length = s["tables"].shape[1] * BS
    return _plain_attention(s, (torch.arange(length, device="cuda") < s["lens"][:, None])[:, None])


def _plain_bounds(s):
    lens, new = s["lens"], s["new"]
    first, end = (lens - new) // BS, (lens + BS - 1) // BS
    block = first[:, None] + torch.arange(-(-s["max_new"] // BS) + 1, device="cuda")
    use = (block < end[:, None]) & (new > 0)[:, None]
    ids = torch.gather(s["tables"], 1, block.clamp(max=s["tables"].shape[1] - 1).long())
    ids, block = ids[use].long(), block[use]
    token = block[:, None] * BS + torch.arange(BS, device="cuda")
    live = (token < lens[:, None].expand(use.shape)[use][:, None])[:, :, None, None]
    rows = s["k_cache"][ids].float()
    low = torch.where(live, rows, float("inf")).amin(1)
    high = torch.where(live, rows, float("-inf")).amax(1)
    s["bounds"][ids] = torch.stack([low, high], 1).to(s["bounds"].dtype)
    return s["bounds"]


def _plain_sparse(s):
    q = s["q"]
    n, heads, d = q.shape
    hkv = s["kv_heads"]
    blocks = s["tables"].shape[1]
    at = s["bounds"][s["tables"].clamp(min=0).long()].double()      # [S, blocks, 2, Hkv, D]
    rows = q.view(n, hkv, -1, d).double()
    # sum_d max(q_d low_d, q_d high_d): where q_d >= 0 it is q_d high_d, else q_d low_d
    score = (torch.einsum("bgid,bjgd->bgij", rows.clamp(min=0), at[:, :, 1])
             + torch.einsum("bgid,bjgd->bgij", rows.clamp(max=0), at[:, :, 0])).amax(2)
    count = ((s["lens"] + BS - 1) // BS)[:, None, None]
    j = torch.arange(blocks, device="cuda")
    score = torch.where((j < s["sink"]) | (j >= count - s["recent"]), float("inf"), score)
    score = torch.where(j < count, score, float("-inf"))
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :s["selected"]]
    order = torch.where(order < count, order, blocks)
    order = torch.sort(order, -1).values
    pick = torch.full((n, hkv, s["selected"]), -1, device="cuda", dtype=torch.int32)
    pick[..., :order.shape[-1]] = torch.where(order < blocks, order, -1)
    s["chosen"].copy_(pick)
    mask = torch.zeros((n, hkv, blocks + 1), device="cuda", dtype=torch.bool)
    mask.scatter_(2, order, True)
    mask = mask[..., :blocks].repeat_interleave(BS, 2)
    length = torch.arange(blocks * BS, device="cuda") < s["lens"][:, None]
    s["out"].copy_(_plain_attention(s, mask & length[:, None]))
    return {"chosen": s["chosen"], "out": s["out"]}


_PLAIN = {"append": _plain_append, "shared": _plain_shared, "bounds": _plain_bounds, "sparse": _plain_sparse}
_OWN = {"append": _own_append, "shared": _own_shared, "bounds": _own_bounds, "sparse": _own_sparse}


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "bounds":
        out = s["bounds"].double()
        for b in range(s["seqs"]):
            length, new = int(s["lens"][b]), int(s["new"][b])
            for j in range((length - new) // BS if new else 1 << 30, -(-length // BS)):
                block = int(s["tables"][b, j])
                rows = s["k_cache"][block, :min(BS, length - j * BS)].double()
                out[block, 0], out[block, 1] = rows.min(0).values, rows.max(0).values
        return out
    return _exact_attention(s)


def _exact_append(s):
    q, k, v = (x.double() for x in _split(s))
    r = s["rotary"]
    live = s["positions"] >= 0
    # the table's entries are inputs
    half = s["cos_sin"].double()[s["positions"].clamp(min=0)]
    turn = torch.complex(half[:, :r // 2], half[:, r // 2:])[:, None, :]

    def rotate(x):
        out = x.clone()
        if s["interleaved"]:
            z = torch.view_as_complex(x[..., :r].reshape(*x.shape[:2], r // 2, 2).contiguous()) * turn
            out[..., 0:r:2], out[..., 1:r:2] = z.real, z.imag
        else:
            z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * turn
            out[..., :r // 2], out[..., r // 2:r] = z.real, z.imag
        return out

    q_out = torch.where(live[:, None, None], rotate(q), s["q_out"].double())
    k, use = rotate(k), s["slots"] >= 0
    if s["cache"] == "fp8":
        k, v = (k / s["k_scale"]).clamp(-448, 448), (v / s["v_scale"]).clamp(-448, 448)
    caches = []
    for cache, rows in ((s["k_cache"], k), (s["v_cache"], v)):
        whole = torch.zeros(cache.shape, device="cuda", dtype=torch.float64)
        whole.view(-1, *cache.shape[2:])[s["slots"][use]] = rows[use]
        caches.append(whole)
    return {"q": q_out, "k_cache": caches[0], "v_cache": caches[1]}


def _exact_attention(s):
    n, heads, d = s["q"].shape
    hkv = s["kv_heads"]
    group = heads // hkv
    out = torch.zeros((n, heads, d), device="cuda", dtype=torch.float64)
    chosen = torch.full((n, hkv, s["selected"]), -1, device="cuda", dtype=torch.int32) if s["op"] == "sparse" else None
    for b in range(n):
        length = int(s["lens"][b])
        if length == 0:
            continue
        blocks = -(-length // BS)
        ids = s["tables"][b, :blocks].long()
        k = s["k_cache"][ids].reshape(blocks * BS, hkv, d)[:length].double()
        v = s["v_cache"][ids].reshape(blocks * BS, hkv, d)[:length].double()
        q = s["q"][b].double().reshape(hkv, group, d)
        for g in range(hkv):
            keep = torch.ones(length, dtype=torch.bool, device="cuda")
            if chosen is not None:
                low, high = s["bounds"][ids, 0, g].double(), s["bounds"][ids, 1, g].double()
                best = torch.maximum(q[g][:, None] * low, q[g][:, None] * high).sum(-1).max(0).values
                j = torch.arange(blocks, device="cuda")
                best[(j < s["sink"]) | (j >= blocks - s["recent"])] = float("inf")
                pick = torch.argsort(best, descending=True, stable=True)[:s["selected"]].sort().values
                chosen[b, g, :len(pick)] = pick.int()
                kept = torch.zeros(blocks, dtype=torch.bool, device="cuda")
                kept[pick] = True
                keep = kept.repeat_interleave(BS)[:length]
            weight = torch.softmax(s["scale"] * (q[g] @ k[keep, g].T), -1)
            out[b, g * group:(g + 1) * group] = weight @ v[keep, g]
    return out if chosen is None else {"chosen": chosen, "out": out}
