"""Cases, plain forms and 64-bit values of the serving-step operators around the paged cache.

One step of drafting and verifying with a paged KV cache runs, on the GPU and without a host round trip:

  tree_masks     parents of a tree of drafted tokens -> packed ancestor masks and positions
  rope           rotary positions on q and k, with the cache write of the rotated k and of v (bf16 or E4M3 pools)
  tree           attention of the drafted tokens over the cache and over their ancestors in the tree
  extend         block tables grown from a free list, slot maps and positions, from the requests' lengths

``own`` False computes the plain forms with elementary torch operations, True calls the library.
"""
import math

import numpy as np
import torch

own = False

TWO_PI = 2.0 * math.pi


# --------------------------------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------------------------------

def _tree(name, batch, heads, kv_heads, dim, block, lo, hi, nodes, ragged):
    return {"name": name, "op": "tree", "batch": batch, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "block": block, "lo": lo, "hi": hi, "nodes": nodes, "ragged": ragged}


def _rope(name, tokens, heads, kv_heads, dim, rotary, interleaved, scaling, pool, start, block):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rotary": rotary, "interleaved": interleaved, "scaling": scaling, "pool": pool, "start": start,
            "block": block}


def _extend(name, batch, lo, hi, add_lo, add_hi, block, path):
    return {"name": name, "op": "extend", "batch": batch, "lo": lo, "hi": hi, "add_lo": add_lo, "add_hi": add_hi,
            "block": block, "path": path}


def _masks(name, batch, nodes, ragged, width):
    return {"name": name, "op": "masks", "batch": batch, "nodes": nodes, "ragged": ragged, "width": width}


def listed():
    return [
        # four short requests of the tiny shape with eight drafted tokens each: latency alone counts
        _tree("tree tiny", 4, 4, 2, 64, 16, 1, 47, 8, False),
        # a served batch with grouped heads, chat lengths, 32 drafted tokens at most: bound by the cache's bytes
        _tree("tree gqa chat", 64, 32, 8, 128, 32, 60, 4096, 32, True),
        # one key head for each query head, odd lengths, trees of different sizes
        _tree("tree mha ragged", 24, 32, 32, 128, 16, 128, 2048, 61, True),
        # few requests with a long cache: the work is split over the cache's length
        _tree("tree long", 8, 64, 8, 128, 16, 32768, 32768, 16, False),
        # many query rows for each key head: bound by the products and the exponentials
        _tree("tree wide", 4, 64, 8, 128, 16, 6000, 8190, 64, False),
        # one decode step of a batch far into a long context
        _rope("rope decode", 64, 32, 8, 128, 128, False, "parts", "bf16", 100000, 32),
        # a prompt of several thousand tokens, written to the cache as it is rotated
        _rope("rope prompt", 8192, 32, 8, 128, 128, False, "wavelength", "bf16", 0, 32),
        # interleaved pairs, a quarter of the head rotated, pools in 8 bits, an odd number of tokens
        _rope("rope interleaved fp8", 3001, 40, 40, 128, 32, True, "linear", "fp8", 777, 16),
        # after verification: up to six accepted tokens of a drafted path for each request
        _extend("extend accepted", 256, 1, 4096, 0, 6, 16, 33),
        # prompts of a whole batch enter the cache at once
        _extend("extend prompts", 64, 0, 0, 17, 4096, 16, 0),
        # masks of a few small trees, and of a batch of large ones
        _masks("masks small", 4, 8, False, 3),
        _masks("masks large", 256, 256, True, 24),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "rope", "extend", "masks"])
    if op == "tree":
        heads, kv_heads, dim = rng.choice([(4, 2, 64), (8, 8, 64), (32, 32, 128), (32, 8, 128), (64, 8, 128),
                                           (40, 40, 128), (8, 4, 128), (8, 2, 64)])
        hi = _log_int(rng, 1, 32768)
        nodes = _log_int(rng, 1, 128)
        # the bytes of the cache and the products stay below the largest listed case
        most = min(64, 262144 // hi, int(4 * 8190 * 64 * 64 / (hi * heads * nodes)), 262144 * 8 * 128 // (hi * kv_heads * dim))
        batch = _log_int(rng, 1, max(1, most))
        while nodes > 1 and batch * hi * heads * nodes > 8 * 32768 * 64 * 16:
            nodes = max(1, nodes // 2)
        return _tree("", batch, heads, kv_heads, dim, rng.choice([8, 16, 32, 64]), _log_int(rng, 1, hi), hi, nodes,
                     rng.random() < 0.5) | {"name": "tree drawn"}
    if op == "rope":
        heads, kv_heads, dim = rng.choice([(4, 2, 64), (32, 32, 128), (32, 8, 128), (64, 8, 128), (40, 40, 128),
                                           (8, 2, 64)])
        tokens = _log_int(rng, 1, 8192 * 48 // (heads + 2 * kv_heads))
        rotary = rng.choice([r for r in (16, 32, 64, 96, 128) if r <= dim])
        return _rope("rope drawn", tokens, heads, kv_heads, dim, rotary, rng.random() < 0.5,
                     rng.choice(["none", "linear", "ntk", "parts", "wavelength"]), rng.choice(["bf16", "fp8"]),
                     rng.choice([0, _log_int(rng, 1, 1000000)]), rng.choice([8, 16, 32, 64]))
    if op == "extend":
        if rng.random() < 0.5:
            nodes = rng.randint(1, 64)
            return _extend("extend drawn", _log_int(rng, 1, 512), 1, _log_int(rng, 1, 8192), 0,
                           rng.randint(1, min(8, nodes)), rng.choice([8, 16, 32, 64]), nodes)
        hi = _log_int(rng, 1, 8192)
        return _extend("extend drawn", max(1, min(_log_int(rng, 1, 512), 131072 // hi)), 0, rng.choice([0, 500]),
                       rng.randint(0, hi), hi, rng.choice([8, 16, 32, 64]), 0)
    return _masks("masks drawn", _log_int(rng, 1, 256), _log_int(rng, 1, 256), rng.random() < 0.5, rng.randint(1, 32))


def _spaced(lo, hi, n):
    """n lengths from lo to hi, spread over their logarithm; they follow from the case alone."""
    if n == 1 or lo == hi:
        return [hi] * n
    a = max(lo, 1)
    got = [int(round(a * (max(hi, 1) / a) ** (i / (n - 1)))) for i in range(n)]
    got[0], got[-1] = lo, hi
    return got


def _ramp(lo, hi, n):
    """n counts from lo to hi in even steps."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)] if n > 1 else [hi]


def _counts(case):
    b, n = case["batch"], case["nodes"]
    return _ramp(max(1, n // 3), n, b) if case["ragged"] else [n] * b


# --------------------------------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------------------------------

def _ints(values):
    return torch.tensor(np.asarray(values, dtype=np.int32), device="cuda")


def _parents(rng, counts, width):
    """Each node hangs below one of the `width` nodes before it; about one in eight starts from the cache itself."""
    out = []
    for n in counts:
        p = [max(-1, i - 1 - int(rng.integers(0, width))) if rng.random() > 0.125 else -1 for i in range(n)]
        out += p
    return np.asarray(out, dtype=np.int32)


def _packed(parents, counts, words):
    """The ancestors of each node and the node itself, 32 nodes in a word, and the depths."""
    masks, depth, at = np.zeros((sum(counts), words), np.uint32), np.zeros(sum(counts), np.int32), 0
    for n in counts:
        for i in range(n):
            p = int(parents[at + i])
            if p >= 0:
                masks[at + i] = masks[at + p]
                depth[at + i] = depth[at + p] + 1
            masks[at + i, i // 32] |= np.uint32(1 << (i % 32))
        at += n
    return masks.view(np.int32), depth


def turns_of(rotary, scaling):
    """Frequencies of the rotary pairs in turns for each position, in 64 bits, and the factor on the rotated values."""
    base, factor, original = 500000.0, 8.0, 8192.0
    i = np.arange(rotary // 2, dtype=np.float64)
    f, gain = base ** (-2.0 * i / rotary), 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "ntk":
        f = (base * factor ** (rotary / (rotary - 2.0))) ** (-2.0 * i / rotary)
    elif scaling == "parts":
        at = [rotary * math.log(original / (r * TWO_PI)) / (2.0 * math.log(base)) for r in (32.0, 1.0)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rotary - 1)
        ramp = np.clip((i - low) / max(high - low, 0.001), 0.0, 1.0)
        f = f / factor * ramp + f * (1.0 - ramp)
        gain = 0.1 * math.log(factor) + 1.0
    elif scaling == "wavelength":
        turns = original * f / TWO_PI
        keep = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        f = f / factor * (1.0 - keep) + f * keep
    return f / TWO_PI, gain


def prepare(case, seed):
    rng = np.random.default_rng([seed, 11])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)

    s = dict(case)
    if case["op"] == "tree":
        B, Hq, Hkv, d, bs = (case[k] for k in ("batch", "heads", "kv_heads", "dim", "block"))
        lens = rng.permutation(_spaced(case["lo"], case["hi"], B))
        counts = [int(n) for n in rng.permutation(_counts(case))]
        blocks = -(-lens // bs)
        nb, wide = int(blocks.sum()) + 3, int(blocks.max())
        order, tables, at = rng.permutation(nb), np.full((B, wide), -1), 0
        for b in range(B):
            tables[b, :blocks[b]] = order[at:at + blocks[b]]
            at += blocks[b]
        masks, _ = _packed(_parents(rng, counts, 6), counts, -(-max(counts) // 32))
        rows = sum(counts)
        kv = normal(rows, 2, Hkv, d)
        s.update(q=normal(rows, Hq, d), k_tree=kv[:, 0], v_tree=kv[:, 1], k_cache=normal(nb, Hkv, bs, d),
                 v_cache=normal(nb, Hkv, bs, d), tables=_ints(tables), lens=_ints(lens),
                 cu=_ints(np.concatenate([[0], np.cumsum(counts)])), masks=torch.tensor(masks, device="cuda"),
                 max_len=int(lens.max()), max_nodes=max(counts), scale=1.0 / math.sqrt(d))
    elif case["op"] == "rope":
        T, Hq, Hkv, d, bs = (case[k] for k in ("tokens", "heads", "kv_heads", "dim", "block"))
        qkv = normal(T, Hq + 2 * Hkv, d)  # one projection's output: q, k and v side by side in each row
        nb = -(-T // bs) + 2
        slots = rng.permutation(nb * bs)[:T] if T <= 64 else (
            rng.permutation(nb)[np.arange(T) // bs] * bs + np.arange(T) % bs)
        slots[rng.integers(0, T, size=T // 50)] = -1  # padding tokens
        positions = case["start"] + (rng.integers(0, 4096, size=T) if T <= 64 else np.arange(T))
        turns, gain = turns_of(case["rotary"], case["scaling"])
        fp8 = case["pool"] == "fp8"
        pool = torch.zeros(2, nb, Hkv, bs, d, device="cuda", dtype=torch.uint8 if fp8 else torch.bfloat16)
        s.update(qkv=qkv, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], k_cache=pool[0], v_cache=pool[1],
                 slots=_ints(slots), positions=_ints(positions), turns=torch.tensor(turns, device="cuda"), gain=gain,
                 k_scale=0.03125, v_scale=0.015625)
    elif case["op"] == "extend":
        B, bs = case["batch"], case["block"]
        lens = rng.permutation(_spaced(case["lo"], case["hi"], B)) if case["hi"] else np.zeros(B, np.int64)
        add = rng.permutation(_ramp(case["add_lo"], case["add_hi"], B))
        old, new = -(-lens // bs), -(-(lens + add) // bs)
        total = int(new.sum())
        order = rng.permutation(total + 9)
        wide, at = max(1, int(new.max())), 0
        tables = np.full((B, wide), -1)
        for b in range(B):
            tables[b, :old[b]] = order[at:at + old[b]]
            at += old[b]
        s.update(tables=_ints(tables), lens=_ints(lens), add=_ints(add), free=_ints(np.concatenate([[0, 0, 0], order[at:]])),
                 cursor=_ints([3]), num_blocks=total + 9, lens_out=_ints(np.zeros(B)), cursor_out=_ints([0]))
        if case["path"]:
            n = case["path"]
            path = np.full((B, max(1, case["add_hi"])), -1)
            for b in range(B):
                path[b, :add[b]] = np.sort(rng.permutation(n)[:add[b]])
            s.update(cu_rows=_ints(np.arange(B + 1) * n), path=_ints(path), rows=B * n)
        else:
            s.update(cu_rows=None, path=None, rows=int(add.sum()) + 5)
    else:
        counts = [int(n) for n in rng.permutation(_counts(case))]
        s.update(parents=_ints(_parents(rng, counts, case["width"])), cu=_ints(np.concatenate([[0], np.cumsum(counts)])),
                 lens=_ints(rng.integers(0, 5000, size=case["batch"])), max_nodes=max(counts), rows=sum(counts))
    return s


# --------------------------------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------------------------------

def _row_of(cu, rows):
    """The request of each row, and the row's number within it."""
    r = torch.arange(rows, device="cuda")
    b = (r[:, None] >= cu[None, 1:-1]).sum(1)
    return b, r - cu.long()[b]


def plain_tree(s):
    B, Hq, Hkv, d, bs = (s[k] for k in ("batch", "heads", "kv_heads", "dim", "block"))
    G, N, rows = Hq // Hkv, s["max_nodes"], s["q"].shape[0]
    blocks = -(-s["max_len"] // bs)
    table = s["tables"][:, :blocks].long().clamp(min=0)

    def context(pool):  # the cached rows in order: [B, Hkv, tokens, d]
        return pool[table].permute(0, 2, 1, 3, 4).reshape(B, Hkv, blocks * bs, d).float()

    cu = s["cu"].long()
    node = torch.arange(N, device="cuda")
    at = (cu[:-1, None] + node).clamp(max=rows - 1)  # [B, N]
    here = node < (cu[1:] - cu[:-1])[:, None]
    k = torch.cat([context(s["k_cache"]), s["k_tree"][at].permute(0, 2, 1, 3).float()], 2)
    v = torch.cat([context(s["v_cache"]), s["v_tree"][at].permute(0, 2, 1, 3).float()], 2)
    q = s["q"][at].float().reshape(B, N, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, d)
    score = torch.matmul(q, k.transpose(2, 3)).view(B, Hkv, N, G, -1) * s["scale"]
    cached = torch.arange(blocks * bs, device="cuda") < s["lens"].long()[:, None]  # [B, tokens]
    bits = (s["masks"][at][:, :, node // 32] >> (node % 32).int()) & 1  # [B, N, N]
    seen = torch.cat([cached[:, None].expand(B, N, -1), (bits != 0) & here[:, None]], 2)[:, None, :, None]
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = weight.sum(-1, keepdim=True)
    weight = (weight / torch.where(total == 0, 1.0, total)).view(B, Hkv, N * G, -1)
    out = torch.matmul(weight, v).view(B, Hkv, N, G, d).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, d)
    b, i = _row_of(cu, rows)
    return out[b, i].to(torch.bfloat16)


def _rotated(x, s):
    """x [T, H, d] in 32 bits with the first `rotary` values of each head rotated; angles in 64 bits."""
    r = s["rotary"]
    angle = s["positions"].double()[:, None, None] * s["turns"] * TWO_PI
    c, n = (torch.cos(angle) * s["gain"]).float(), (torch.sin(angle) * s["gain"]).float()
    x = x.float()
    if s["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([turned, x[..., r:]], -1)


def plain_rope(s):
    q, k, v = _rotated(s["q"], s).to(torch.bfloat16), _rotated(s["k"], s), s["v"].float()
    T, bs = s["tokens"], s["block"]
    keep = s["slots"] >= 0
    slot = torch.where(keep, s["slots"], 0).long()
    pools = []
    for new, pool, scale in ((k, s["k_cache"], s["k_scale"]), (v, s["v_cache"], s["v_scale"])):
        if s["pool"] == "fp8":
            new = (new * (1.0 / scale)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            new = new.to(torch.bfloat16)
        row = torch.full((pool.shape[0] * bs,), T, device="cuda")
        row = row.index_put((slot[keep],), torch.arange(T, device="cuda")[keep]).view(-1, 1, bs, 1)
        h, e = torch.arange(pool.shape[1], device="cuda").view(1, -1, 1, 1), torch.arange(pool.shape[3], device="cuda")
        pool.copy_(torch.where(row < T, new[row.clamp(max=T - 1), h, e], pool))
        pools.append(pool.view(torch.float8_e4m3fn) if s["pool"] == "fp8" else pool)
    return {"q": q, "k_cache": pools[0], "v_cache": pools[1]}


def plain_extend(s):
    bs, rows = s["block"], s["rows"]
    lens, add, tables = s["lens"].long(), s["add"].long(), s["tables"]
    old, new = (lens + bs - 1) // bs, (lens + add + bs - 1) // bs
    ends = torch.cumsum(new - old, 0)
    first = s["cursor"].long() + ends - (new - old)  # where each request's blocks start in the free list
    j = torch.arange(tables.shape[1], device="cuda")
    fresh = (j >= old[:, None]) & (j < new[:, None])
    taken = s["free"][torch.where(fresh, first[:, None] + j - old[:, None], 0)]
    tables.copy_(torch.where(fresh, taken, tables))
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(add, 0)])
    if s["path"] is None:
        b, i = _row_of(cu, rows)
        here = torch.arange(rows, device="cuda") < cu[-1]
    else:
        b, node = _row_of(s["cu_rows"], rows)
        step = torch.arange(s["path"].shape[1], device="cuda")
        hit = (s["path"][b] == node[:, None]) & (step < add[b][:, None])
        here, i = hit.any(1), hit.int().argmax(1)
    at = torch.where(here, lens[b] + i, 0)
    slot = torch.where(here, tables[b, at // bs].long() * bs + at % bs, -1)
    return {"tables": tables, "lens": (lens + add).int(), "cursor": (s["cursor"] + ends[-1]).int(),
            "slots": slot.int(), "positions": at.int(), "cu": cu.int()}


def plain_masks(s):
    B, N, rows = s["batch"], s["max_nodes"], s["rows"]
    cu, node = s["cu"].long(), torch.arange(s["max_nodes"], device="cuda")
    here = node < (cu[1:] - cu[:-1])[:, None]
    parent = torch.where(here, s["parents"][(cu[:-1, None] + node).clamp(max=rows - 1)].long(), -1)
    reach = ((parent[:, :, None] == node) | (node[:, None] == node)).float()  # a node, and its parent
    for _ in range(max(1, math.ceil(math.log2(max(N, 2))))):  # twice as many generations each time
        reach = (torch.matmul(reach, reach) > 0).float()
    words = -(-N // 32)
    bits = torch.nn.functional.pad(reach, (0, words * 32 - N)).view(B, N, words, 32).long()
    packed = (bits << torch.arange(32, device="cuda")).sum(-1).int()
    b, i = _row_of(cu, rows)
    return {"masks": packed[b, i], "positions": (s["lens"][b] + reach.sum(-1).int()[b, i] - 1).int()}


# --------------------------------------------------------------------------------------------------
# The library's calls
# --------------------------------------------------------------------------------------------------

def own_tree(s):
    import paged_kv_cache_349_b200 as pa
    if "workspace" not in s:  # kept by a program that serves this shape
        size = pa.pa_decode_tree_workspace_size(s["batch"], s["q"].shape[0], s["heads"], s["kv_heads"], s["dim"],
                                                s["block"], s["max_len"], s["max_nodes"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    out = torch.empty_like(s["q"])
    pa.pa_decode_tree(out, s["q"], s["k_tree"], s["v_tree"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["cu"],
                      s["masks"], max_seq_len=s["max_len"], max_nodes=s["max_nodes"], scale=s["scale"],
                      workspace=s["workspace"])
    return out


def own_rope(s):
    import paged_kv_cache_349_b200 as pa
    q = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    if s["pool"] == "fp8":
        pa.pa_rope_and_cache_fp8(s["q"], q, s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], s["positions"],
                                 s["turns"], interleaved=s["interleaved"], gain=s["gain"], k_scale=s["k_scale"],
                                 v_scale=s["v_scale"])
        return {"q": q, "k_cache": s["k_cache"].view(torch.float8_e4m3fn), "v_cache": s["v_cache"].view(torch.float8_e4m3fn)}
    pa.pa_rope_and_cache(s["q"], q, s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], s["positions"], s["turns"],
                         interleaved=s["interleaved"], gain=s["gain"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def own_extend(s):
    import paged_kv_cache_349_b200 as pa
    slots = torch.empty(s["rows"], dtype=torch.int32, device="cuda")
    positions = torch.empty(s["rows"], dtype=torch.int32, device="cuda")
    cu = torch.empty(s["batch"] + 1, dtype=torch.int32, device="cuda")
    pa.pa_extend_tables(s["tables"], s["lens"], s["add"], s["free"], s["cursor"], num_blocks=s["num_blocks"],
                        block_size=s["block"], seq_lens_out=s["lens_out"], cursor_out=s["cursor_out"],
                        slot_mapping=slots, positions=positions, cu_tokens=cu, cu_rows=s["cu_rows"], path=s["path"])
    return {"tables": s["tables"], "lens": s["lens_out"], "cursor": s["cursor_out"], "slots": slots,
            "positions": positions, "cu": cu}


def own_masks(s):
    import paged_kv_cache_349_b200 as pa
    masks = torch.empty(s["rows"], -(-s["max_nodes"] // 32), dtype=torch.int32, device="cuda")
    positions = torch.empty(s["rows"], dtype=torch.int32, device="cuda")
    pa.pa_tree_masks(masks, positions, s["parents"], s["cu"], s["lens"], max_nodes=s["max_nodes"])
    return {"masks": masks, "positions": positions}


def run(state):
    op = state["op"]
    if own:
        return {"tree": own_tree, "rope": own_rope, "extend": own_extend, "masks": own_masks}[op](state)
    return {"tree": plain_tree, "rope": plain_rope, "extend": plain_extend, "masks": plain_masks}[op](state)


# --------------------------------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------------------------------

def work(case):
    if case["op"] == "tree":
        B, Hq, Hkv, d, bs = (case[k] for k in ("batch", "heads", "kv_heads", "dim", "block"))
        lens, counts = _spaced(case["lo"], case["hi"], B), _counts(case)
        rows, words = sum(counts), -(-max(counts) // 32)
        cached = sum(lens)
        # the lengths and the trees are dealt to the requests in an order of the seed: the mean pairing
        pairs = cached * rows / B + rows
        return {"bytes": 4 * d * Hkv * (cached + rows) + 4 * d * Hq * rows + 4 * sum(-(-n // bs) for n in lens)
                + 4 * rows * words + 8 * B + 4, "flops": 4 * d * Hq * pairs}
    if case["op"] == "rope":
        T, Hq, Hkv, d = (case[k] for k in ("tokens", "heads", "kv_heads", "dim"))
        cell = 1 if case["pool"] == "fp8" else 2
        kept = T - T // 50
        return {"bytes": T * (4 * Hq * d + 8) + kept * (4 * Hkv * d + 2 * Hkv * d * cell) + 4 * case["rotary"],
                "flops": 3 * T * case["rotary"] * (Hq + Hkv)}
    if case["op"] == "extend":
        B, bs = case["batch"], case["block"]
        lens = _spaced(case["lo"], case["hi"], B) if case["hi"] else [0] * B
        add = _ramp(case["add_lo"], case["add_hi"], B)
        # each request takes at least this many blocks, whichever order the seed deals them in
        fresh = sum(a // bs for a in add)
        rows = B * case["path"] if case["path"] else sum(add) + 5
        return {"bytes": 16 * B + 8 * fresh + 8 * rows + (4 * B * case["add_hi"] if case["path"] else 0), "flops": 0}
    rows = sum(_counts(case))
    words = -(-max(_counts(case)) // 32)
    return {"bytes": 8 * rows + 4 * rows * words + 8 * case["batch"] + 4, "flops": 0}


# --------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------------------------------

def exact(case, seed):
    """Attention and rotation in 64 bits, request by request and pair by pair; whole numbers have no such value."""
    if case["op"] == "tree":
        s = prepare(case, seed)
        Hq, Hkv, d, bs = (case[k] for k in ("heads", "kv_heads", "dim", "block"))
        G = Hq // Hkv
        cu, lens = s["cu"].tolist(), s["lens"].tolist()
        masks = s["masks"].cpu().numpy().view(np.uint32)
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for b in range(case["batch"]):
            L, lo, hi = lens[b], cu[b], cu[b + 1]
            n = hi - lo
            pages = s["tables"][b, :-(-L // bs)].long()
            k = s["k_cache"][pages].transpose(1, 2).reshape(-1, Hkv, d)[:L].double()
            v = s["v_cache"][pages].transpose(1, 2).reshape(-1, Hkv, d)[:L].double()
            k, v = torch.cat([k, s["k_tree"][lo:hi].double()]), torch.cat([v, s["v_tree"][lo:hi].double()])
            bit = np.unpackbits(masks[lo:hi].view(np.uint8), axis=1, bitorder="little")[:, :n].astype(bool)
            ban = torch.cat([torch.zeros(n, L, dtype=torch.bool), torch.tensor(~bit)], 1).cuda()
            for h in range(Hkv):
                q = s["q"][lo:hi, h * G:(h + 1) * G].double()
                e = torch.einsum("ngd,td->gnt", q, k[:, h]) * s["scale"]
                e = torch.softmax(e.masked_fill(ban, -math.inf), -1)
                out[lo:hi, h * G:(h + 1) * G] = torch.einsum("gnt,td->ngd", e.nan_to_num(0.0), v[:, h])
        return out
    if case["op"] == "rope":
        s = prepare(case, seed)
        r, bs = case["rotary"], case["block"]
        spin = torch.polar(torch.full((), s["gain"], dtype=torch.float64, device="cuda"),
                           s["positions"].double()[:, None] * s["turns"] * TWO_PI)[:, None]

        def turn(x):
            x = x.double().clone()
            lo, hi = (slice(0, r, 2), slice(1, r, 2)) if case["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
            z = torch.complex(x[..., lo], x[..., hi]) * spin
            x[..., lo], x[..., hi] = z.real, z.imag
            return x

        got = {"q": turn(s["q"])}
        keep = s["slots"] >= 0
        slot = s["slots"][keep].long()
        for name, new, scale in (("k_cache", turn(s["k"]), s["k_scale"]), ("v_cache", s["v"].double(), s["v_scale"])):
            pool = torch.zeros(s[name].shape, dtype=torch.float64, device="cuda")
            new = new[keep]
            pool[slot // bs, :, slot % bs] = (new / scale).clamp(-448.0, 448.0) if case["pool"] == "fp8" else new
            got[name] = pool
        return got
    return None
