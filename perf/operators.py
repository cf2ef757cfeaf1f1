"""The operators around a paged KV cache held in 4 bits, as a serving step uses them.

  norm_rope   per-head RMS norm of queries and keys with the rotation of their
              positions (one axis, or time/height/width), alone or with the
              step's K/V written into the bf16 or the 4-bit cache in one pass
  write_q4    quantise K/V rows into the 4-bit cache, and read rows back
  decode_q4   one query token per sequence against the 4-bit cache
  prefill_q4  packed prompts, chunks and prefix hits against the 4-bit cache
  blocks      fork and free sequences' pages, compact a pool, copy pages

The 4-bit format: groups of 16 consecutive dims of one head's row share a
scale s (e4m3) and hold e2m1 codes, value = code * s * tensor_scale.
`own` chooses between the framework's kernels and the plain forms below.
"""

import math
import random

import torch

own = False

BS = 256     # tokens of a block
D = 128      # head dim
GROUP = 16   # dims that share a scale
DEV = "cuda"
EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # The 256 rows of a decode step of a 16/8-head model: q and k of the fused
        # projection normalised and rotated, k and v put into the bf16 cache.
        {"name": "norm_rope.step_bf16", "op": "norm_rope", "n": 256, "hq": 16, "hkv": 8, "into": "bf16", "rot": 128,
         "axes": 1, "interleaved": False, "far": 32768, "ts": 1.0},
        # A 16384-token step of prompts with images and video (three position
        # axes) into the 4-bit cache.
        {"name": "norm_rope.prefill_q4", "op": "norm_rope", "n": 16384, "hq": 16, "hkv": 8, "into": "q4", "rot": 128,
         "axes": 3, "interleaved": False, "far": 1000000, "ts": 1.0},
        # Four new tokens: the smallest step.
        {"name": "write_q4.4", "op": "write_q4", "n": 4, "hkv": 8, "ts": 1.0},
        # Four prompts of 8192 tokens written at once.
        {"name": "write_q4.32768", "op": "write_q4", "n": 32768, "hkv": 8, "ts": 0.25},
        # A handful of short sequences: launch latency and merging count.
        {"name": "decode_q4.4", "op": "decode_q4", "batch": 4, "lo": 1, "hi": 600, "pad": 0, "hq": 16, "hkv": 8,
         "ts": 1.0},
        # The ordinary decode batch.
        {"name": "decode_q4.256", "op": "decode_q4", "batch": 256, "lo": 100, "hi": 2048, "pad": 0, "hq": 16,
         "hkv": 8, "ts": 1.0},
        # Long contexts, four query heads to a kv head.
        {"name": "decode_q4.long", "op": "decode_q4", "batch": 64, "lo": 8192, "hi": 32768, "pad": 0, "hq": 32,
         "hkv": 8, "ts": 0.5},
        # A step of 16384 new tokens of ragged prompts, some with cached prefixes.
        {"name": "prefill_q4.chunked", "op": "prefill_q4", "seqs": 40, "lo": 100, "hi": 1024, "hits": 0.3,
         "new": 0, "budget": 16384, "hq": 16, "hkv": 8, "ts": 1.0},
        # Two whole prompts of 8192 tokens.
        {"name": "prefill_q4.8192", "op": "prefill_q4", "seqs": 2, "lo": 8192, "hi": 8192, "hits": 0.0,
         "new": 0, "budget": 16384, "hq": 32, "hkv": 8, "ts": 1.0},
        # The last 16 tokens of four long prompts (or 16 drafted ones to verify).
        {"name": "prefill_q4.tail", "op": "prefill_q4", "seqs": 4, "lo": 8192, "hi": 32768, "hits": 0.0, "new": 16,
         "budget": 16384, "hq": 16, "hkv": 8, "ts": 1.0},
        # Parallel sampling: 24 children share their parents' pages, copy the last
        # one in all 28 layers, and are given up again.
        {"name": "blocks.fork", "op": "fork", "batch": 16, "forks": 24, "lo": 100, "hi": 600, "layers": 28, "hkv": 8},
        # A half empty pool of four layers moved together.
        {"name": "blocks.compact", "op": "compact", "batch": 120, "lo": 100, "hi": 1024, "blocks": 640, "layers": 4,
         "hkv": 8},
    ]


HEADS = ((16, 8), (32, 8), (64, 8), (8, 8), (12, 4), (4, 2), (16, 1), (15, 3), (14, 7))


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    op = rng.choice(("norm_rope", "norm_rope", "write_q4", "decode_q4", "decode_q4", "prefill_q4", "prefill_q4",
                     "fork", "compact"))
    hq, hkv = rng.choice(HEADS)
    ts = rng.choice((1.0, 0.25, 2.0, 0.3))
    if op == "norm_rope":
        axes = rng.choice((1, 1, 3))
        return {"op": op, "n": _log(rng, 1, 16384), "hq": hq, "hkv": hkv, "into": rng.choice(("none", "bf16", "q4")),
                "rot": rng.choice((32, 64, 96, 128, 128)), "axes": axes, "interleaved": rng.random() < 0.3,
                "far": _log(rng, 100, 4000000), "ts": ts}
    if op == "write_q4":
        return {"op": op, "n": _log(rng, 1, 32768), "hkv": hkv, "ts": ts}
    if op == "decode_q4":
        batch = _log(rng, 1, 512)
        hi = _log(rng, 1, min(32768, 1200000 // batch))
        return {"op": op, "batch": batch, "lo": rng.randint(1, hi), "hi": hi, "pad": rng.choice((0, 0, 3, 12)),
                "hq": hq, "hkv": hkv, "ts": ts}
    if op == "prefill_q4":
        new = rng.choice((0, 0, _log(rng, 1, 100)))
        hi = _log(rng, 1, 32768 if new else 8192)
        seqs = _log(rng, 1, max(1, min(64, (131072 if new else 16384) // hi)))
        return {"op": op, "seqs": seqs, "lo": rng.randint(1, hi), "hi": hi, "hits": rng.choice((0.0, 0.3, 1.0)),
                "new": new, "budget": 16384, "hq": hq if new or hq < 64 else 32, "hkv": hkv, "ts": ts}
    if op == "fork":
        return {"op": op, "batch": _log(rng, 1, 64), "forks": _log(rng, 1, 48), "lo": 1, "hi": _log(rng, 1, 700),
                "layers": rng.randint(1, 14), "hkv": hkv}
    batch = _log(rng, 1, 128)
    return {"op": op, "batch": batch, "lo": 1, "hi": _log(rng, 1, 1000), "blocks": batch * 4 + rng.randint(1, 127),
            "layers": rng.randint(1, 4), "hkv": hkv}


# ------------------------------------------------------------------ lengths, the same for every seed
def _rng(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(case):
    r = _rng(case)
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]


def _prompts(case):
    """(length, cached) of the sequences of a prefill step: some continue after cached blocks."""
    r = _rng(case)
    got, left = [], case["budget"]
    for i in range(case["seqs"]):
        length = r.randint(case["lo"], case["hi"])
        cached = max(0, length - case["new"]) if case["new"] else 0
        if case["new"] == 0 and r.random() < case["hits"] and length > 1:
            cached = r.randint(1, length - 1) if i == 0 else min(BS * r.randint(1, 3), (length - 1) // BS * BS)
        if length - cached > left:
            break
        left -= length - cached
        got.append((length, cached))
    return got


def _sections(case):
    """Pairs that follow the time, height and width positions."""
    half = case["rot"] // 2
    return (half,) if case["axes"] == 1 else (half // 4, half * 3 // 8, half - half // 4 - half * 3 // 8)


def _forked(case):
    r = _rng({**case, "op": "parents"})
    lens = _lengths(case)
    return [r.randrange(case["batch"]) for _ in range(case["forks"])], lens


def work(case):
    op = case["op"]
    if op == "norm_rope":
        rows = {"none": 2 * (case["hq"] + case["hkv"]) * D * 2, "bf16": 2 * (case["hq"] + 2 * case["hkv"]) * D * 2,
                # k and v rows in, codes and scales out and read back as rows
                "q4": 2 * case["hq"] * D * 2 + 2 * case["hkv"] * 2 * (D * 2 + 72)}[case["into"]]
        return {"bytes": case["n"] * (rows + 4 * case["axes"] + (0 if case["into"] == "none" else 4)),
                "flops": case["n"] * (case["hq"] + case["hkv"]) * D * 8}
    if op == "write_q4":  # rows in, codes and scales out; codes and scales in, rows out
        return {"bytes": 2 * case["n"] * (2 * case["hkv"] * (2 * D + 72) + 4), "flops": case["n"] * case["hkv"] * D * 8}
    if op == "decode_q4":
        t = sum(_lengths(case))
        return {"bytes": t * case["hkv"] * 144 + (case["batch"] + case["pad"]) * case["hq"] * D * 4,
                "flops": 4 * t * case["hq"] * D}
    if op == "prefill_q4":
        p = _prompts(case)
        pairs = sum((c + 1 + n) * (n - c) // 2 for n, c in p)
        return {"bytes": sum(n for n, _ in p) * case["hkv"] * 144 + sum(n - c for n, c in p) * case["hq"] * D * 4,
                "flops": 4 * pairs * case["hq"] * D}
    page = BS * case["hkv"] * D * 2
    if op == "fork":
        parents, lens = _forked(case)
        moved = [p for p in parents if lens[p] % BS]
        entries = sum(-(-lens[p] // BS) for p in parents)
        return {"bytes": (len(moved) + len(set(moved))) * 2 * case["layers"] * page + entries * 16, "flops": entries}
    live = sum(-(-n // BS) for n in _lengths(case))
    moved = round(live * max(0, case["blocks"] - live) / case["blocks"])
    return {"bytes": moved * 2 * case["layers"] * page * 2 + 8 * (case["blocks"] + live), "flops": case["blocks"]}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rows(g, *shape):
    """Activations: N(0,1) with a few dims of every head several times larger."""
    x = torch.randn(shape, generator=g, device=DEV)
    x[..., 5::37] *= 6.0
    return x.to(torch.bfloat16)


def _tables(g, lens, blocks):
    """Every sequence's blocks from a shuffled pool, -1 behind them."""
    need = [-(-n // BS) for n in lens]
    perm = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    width = max([1] + need)
    count = torch.tensor(need, device=DEV)
    first = torch.cumsum(count, 0) - count
    col = torch.arange(width, device=DEV)
    at = (first[:, None] + col).clamp(max=blocks - 1)
    return torch.where(col < count[:, None], perm[at], torch.full_like(at, -1, dtype=torch.int32)).contiguous()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _empty_q4(blocks, hkv):
    d = torch.zeros((2, blocks, BS, hkv, D // 2), dtype=torch.uint8, device=DEV)
    s = torch.zeros((2, blocks, BS, hkv, D // GROUP), dtype=torch.uint8, device=DEV)
    return d, s


def _filled_q4(g, blocks, hkv, ts):
    d, s = _empty_q4(blocks, hkv)
    step = max(1, 4096 // hkv)
    for kv in range(2):
        for b in range(0, blocks, step):
            m = min(step, blocks - b)
            d[kv, b:b + m], s[kv, b:b + m] = _quantise(_rows(g, m, BS, hkv, D).float(), ts)
    return d, s


def prepare(case, seed):
    g = _gen(seed)
    op, s = case["op"], {"case": dict(case)}
    if op in ("norm_rope", "write_q4"):
        n, hkv = case["n"], case["hkv"]
        blocks = -(-n // BS) + 2
        s["slots"] = torch.randperm(blocks * BS, generator=g, device=DEV)[:n].to(torch.int32)
        if op == "write_q4" or case["into"] == "q4":
            s["data"], s["scales"] = _empty_q4(blocks, hkv)
        elif case["into"] == "bf16":
            s["cache"] = torch.zeros((2, blocks, BS, hkv, D), dtype=torch.bfloat16, device=DEV)
    if op == "norm_rope":
        hq, rot = case["hq"], case["rot"]
        s["qkv"] = _rows(g, n, hq + 2 * hkv, D)
        s["wq"], s["wk"] = ((1 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16) for _ in range(2))
        s["positions"] = torch.randint(0, case["far"], (case["axes"], n), generator=g, device=DEV, dtype=torch.int32)
        s["inv_freq"] = torch.tensor([1e6 ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64, device=DEV)
        # the same frequencies in turns per position, as 64-bit fractions of a turn
        s["freqs"] = torch.tensor([round(1e6 ** (-2.0 * i / rot) / (2 * math.pi) * 2.0 ** 64) for i in range(rot // 2)],
                                  dtype=torch.int64, device=DEV)
    elif op == "write_q4":
        s["kv"] = _rows(g, n, 2 * hkv, D)
    elif op == "decode_q4":
        lens = _lengths(case)
        blocks = int(1.1 * sum(-(-n // BS) for n in lens)) + 1
        s["data"], s["scales"] = _filled_q4(g, blocks, case["hkv"], case["ts"])
        pads = case["pad"]  # rows that fill a captured batch: no context, no blocks
        s["tables"] = torch.nn.functional.pad(_tables(g, lens, blocks), (0, 0, 0, pads), value=-1)
        s["lens"], s["max_len"] = _ints(lens + [0] * pads), max(lens)
        s["q"] = torch.randn((len(lens) + pads, case["hq"], D), generator=g, device=DEV).to(torch.bfloat16)
    elif op == "prefill_q4":
        prompts = _prompts(case)
        lens, new = [n for n, _ in prompts], [n - c for n, c in prompts]
        blocks = int(1.1 * sum(-(-n // BS) for n in lens)) + 1
        s["data"], s["scales"] = _filled_q4(g, blocks, case["hkv"], case["ts"])
        s["tables"] = _tables(g, lens, blocks)
        s["cu_q"] = _ints([sum(new[:i]) for i in range(len(new) + 1)])
        s["cu_k"] = _ints([sum(lens[:i]) for i in range(len(lens) + 1)])
        s["max_q"], s["max_k"] = max(new), max(lens)
        s["q"] = torch.randn((sum(new), case["hq"], D), generator=g, device=DEV).to(torch.bfloat16)
    else:
        lens = _lengths(case)
        live = sum(-(-n // BS) for n in lens)
        blocks = live + case["forks"] + 1 if op == "fork" else max(case["blocks"], live + 1)
        s["tables"], s["lens"] = _tables(g, lens, blocks), _ints(lens)
        s["ref"] = torch.zeros(blocks, dtype=torch.int32, device=DEV)
        s["ref"][s["tables"][s["tables"] >= 0].long()] = 1
        s["cache"] = torch.empty((2 * case["layers"], blocks, BS, case["hkv"], D), dtype=torch.bfloat16, device=DEV)
        for plane in s["cache"]:
            plane.copy_(torch.randn(plane.shape, generator=g, device=DEV))
        if op == "fork":
            s["parents"] = _ints(_forked(case)[0])
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return {"norm_rope": _norm_rope, "write_q4": _write_q4, "decode_q4": _decode_q4, "prefill_q4": _prefill_q4,
            "fork": _fork, "compact": _compact}[s["case"]["op"]](s)


def _q4(s):
    import paged_kv_cache_304_gb300 as pkv
    if "q4" not in s:
        d, c, ts = s["data"], s["scales"], s["case"]["ts"]
        s["q4"] = pkv.Q4Cache(d[0], c[0], d[1], c[1], k_scale=ts, v_scale=ts)
    return pkv, s["q4"]


def _norm_rope(s):
    c = s["case"]
    hq, hkv, n = c["hq"], c["hkv"], c["n"]
    q, k, v = s["qkv"][:, :hq], s["qkv"][:, hq:hq + hkv], s["qkv"][:, hq + hkv:]
    if own:
        import paged_kv_cache_304_gb300 as pkv
        a = (s["wq"], s["wk"], EPS, s["freqs"], s["positions"])
        more = {"interleaved": c["interleaved"], "sections": _sections(c)}
        if c["into"] == "none":
            return pkv.qk_norm_rope(q, k, *a, **more)
        if c["into"] == "bf16":
            return pkv.qk_norm_rope_write(q, k, v, *a, s["slots"], s["cache"][0], s["cache"][1], **more), s["cache"]
        _, q4 = _q4(s)
        return (pkv.qk_norm_rope_write_q4(q, k, v, *a, s["slots"], q4, **more),
                *pkv.kv_cache_read_q4(q4, s["slots"]))
    axis = torch.arange(c["axes"], device=DEV).repeat_interleave(torch.tensor(_sections(c), device=DEV))
    angle = s["positions"].double()[axis].T * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    out = []
    for x, w in ((q, s["wq"]), (k, s["wk"])):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        r = x[..., :c["rot"]]
        a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else r.chunk(2, -1)
        a, b = a * cos - b * sin, b * cos + a * sin
        r = torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)
        out.append(torch.cat((r, x[..., c["rot"]:]), -1).to(torch.bfloat16))
    if c["into"] == "none":
        return tuple(out)
    if c["into"] == "bf16":
        flat = s["cache"].view(2, -1, hkv, D)
        flat[0, s["slots"].long()] = out[1]
        flat[1, s["slots"].long()] = v
        return out[0], s["cache"]
    return (out[0], *_store_and_read(s, out[1], v))


def _write_q4(s):
    hkv = s["case"]["hkv"]
    k, v = s["kv"][:, :hkv], s["kv"][:, hkv:]
    if own:
        pkv, q4 = _q4(s)
        pkv.kv_cache_write_q4(k, v, s["slots"], q4)
        return pkv.kv_cache_read_q4(q4, s["slots"])
    return _store_and_read(s, k, v)


def _decode_q4(s):
    c = s["case"]
    scale = 1 / math.sqrt(D)
    if own:
        pkv, q4 = _q4(s)
        if "workspace" not in s:
            s["workspace"] = pkv.decode_q4_workspace(s["q"].shape[0], c["hq"], c["hkv"], DEV)
        return pkv.paged_attn_decode_q4(s["q"], q4, s["lens"], s["tables"], scale, workspace=s["workspace"],
                                        max_context_len=s["max_len"])
    b, hkv = s["q"].shape[0], c["hkv"]
    k, v = (_gather(s, kv, s["tables"], s["max_len"]) for kv in range(2))       # [B, L, Hkv, D]
    q = s["q"].float().view(b, hkv, -1, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * scale
    seen = torch.arange(x.shape[-1], device=DEV) < s["lens"][:, None, None, None]
    return _softmax_times(x, seen, v.permute(0, 2, 1, 3)).to(torch.bfloat16).view(b, -1, D)


def _prefill_q4(s):
    c = s["case"]
    scale = 1 / math.sqrt(D)
    if own:
        pkv, q4 = _q4(s)
        if "workspace" not in s:
            s["workspace"] = pkv.prefill_q4_workspace(s["q"].shape[0], s["tables"].shape[0], s["max_q"], s["max_k"],
                                                      c["hq"], c["hkv"], DEV)
        return pkv.paged_attn_prefill_q4(s["q"], q4, s["cu_q"], s["cu_k"], s["tables"], scale, s["max_q"], s["max_k"],
                                         workspace=s["workspace"])
    hq, hkv, n = c["hq"], c["hkv"], s["tables"].shape[0]
    k, v = (_gather(s, kv, s["tables"], s["max_k"]) for kv in range(2))         # [S, L, Hkv, D]
    count, total = s["cu_q"].diff().long(), s["cu_k"].diff().long()
    row = torch.arange(s["max_q"], device=DEV)
    real = row < count[:, None]                                                 # [S, maxq]
    q = s["q"].float()[(s["cu_q"][:-1, None] + row).clamp(max=s["q"].shape[0] - 1).long()]
    q = q.view(n, s["max_q"], hkv, hq // hkv, D).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, D)
    x = (torch.matmul(q, k.permute(0, 2, 3, 1)) * scale).view(n, hkv, hq // hkv, s["max_q"], -1)
    last = (total - count)[:, None] + row                                       # the last key that a row sees
    seen = torch.arange(x.shape[-1], device=DEV) <= last[:, None, None, :, None]
    o = _softmax_times(x, seen, v.permute(0, 2, 1, 3)[:, :, None])              # [S, Hkv, G, maxq, D]
    return o.permute(0, 3, 1, 2, 4).reshape(n, s["max_q"], hq, D)[real].to(torch.bfloat16)


def _fork(s):
    if own:
        import paged_kv_cache_304_gb300 as pkv
        tables, lens, src, dst = pkv.fork_blocks(s["tables"], s["lens"], s["parents"], s["ref"])
        pkv.copy_blocks(s["cache"], src, dst, block_dim=1)
        pkv.free_blocks(tables, lens, s["ref"])
    else:
        parents = s["parents"].long()
        lens, tables = s["lens"][parents], s["tables"][parents].clone()
        used, part = (lens + BS - 1) // BS, lens % BS > 0
        dst = torch.full_like(lens, -1)
        src = torch.where(part, tables.gather(1, (used - 1).clamp(min=0).long()[:, None])[:, 0], dst)
        free = torch.nonzero(s["ref"] == 0)[:, 0].to(torch.int32)
        dst = torch.where(part, free[(torch.cumsum(part, 0) - 1).clamp(min=0)], dst)
        at = torch.nonzero(part)[:, 0]
        tables[at, used[at].long() - 1] = dst[at]
        held = tables[torch.arange(tables.shape[1], device=DEV) < used[:, None]].long()
        s["ref"].index_add_(0, held, torch.ones_like(held, dtype=torch.int32))
        s["cache"][:, dst[at].long()] = s["cache"][:, src[at].long()]
        s["ref"].index_add_(0, held, torch.full_like(held, -1, dtype=torch.int32))
    return {"tables": tables, "lens": lens, "src": src, "dst": dst, "ref": s["ref"], "cache": s["cache"]}


def _compact(s):
    if own:
        import paged_kv_cache_304_gb300 as pkv
        tables, ref, src, dst, moves = pkv.compact_blocks(s["tables"], s["lens"], s["ref"])
        pkv.copy_blocks(s["cache"], src, dst, block_dim=1)
    else:
        blocks = s["ref"].shape[0]
        live, ids = s["ref"] > 0, torch.arange(blocks, device=DEV, dtype=torch.int32)
        kept = live.sum()
        holes, movers = ids[~live & (ids < kept)], ids[live & (ids >= kept)]
        moves = torch.full((1,), movers.numel(), dtype=torch.int32, device=DEV)
        src = torch.nn.functional.pad(movers, (0, blocks // 2 - movers.numel()), value=-1)
        dst = torch.nn.functional.pad(holes, (0, blocks // 2 - holes.numel()), value=-1)
        to = ids.clone()
        to[movers.long()] = holes
        inside = torch.arange(s["tables"].shape[1], device=DEV) < ((s["lens"] + BS - 1) // BS)[:, None]
        tables = torch.where(inside, to[s["tables"].clamp(min=0).long()], s["tables"])
        ref = s["ref"].clone()
        ref[holes.long()] = s["ref"][movers.long()]
        ref[movers.long()] = 0
        s["cache"][:, holes.long()] = s["cache"][:, movers.long()]
    return {"tables": tables, "ref": ref, "src": src, "dst": dst, "moves": moves, "cache": s["cache"]}


# ------------------------------------------------------------------ the plain 4-bit format
def _quantise(x, ts):
    """Rows [..., 128] in 32 bits to packed codes [..., 64] and e4m3 scales [..., 8] (as bytes)."""
    y = (x * (torch.ones((), dtype=torch.float32) / ts).item()).unflatten(-1, (-1, GROUP))
    s = (y.abs().amax(-1, keepdim=True) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    z = y / s.float()
    m = z.abs()
    # nearest code, ties to the even one
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = torch.where(s.float() > 0, code | ((z < 0).to(torch.uint8) << 3), torch.zeros_like(code)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.squeeze(-1).view(torch.uint8)


def _values(data, scales, ts):
    """The values that packed codes and scales stand for, in 32 bits."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    x = torch.stack((lut[(data & 15).int()], lut[(data >> 4).int()]), -1).flatten(-2)
    return x * (scales.view(torch.float8_e4m3fn).float() * ts).repeat_interleave(GROUP, -1)


def _store_and_read(s, k, v):
    """Codes and scales of k and v into the cache at the slots, and the values that the slots then hold."""
    ts, at, got = s["case"]["ts"], s["slots"].long(), []
    for kv, x in enumerate((k, v)):
        data, scales = s["data"][kv].flatten(0, 1), s["scales"][kv].flatten(0, 1)
        data[at], scales[at] = _quantise(x.float(), ts)
        got.append(_values(data[at], scales[at], ts).to(torch.bfloat16))
    return tuple(got)


def _gather(s, kv, tables, longest):
    """The first `longest` positions of every sequence, [S, L, Hkv, D] in 32 bits."""
    t = tables[:, :-(-longest // BS)].clamp(min=0).long()
    return _values(s["data"][kv][t], s["scales"][kv][t], s["case"]["ts"]).flatten(1, 2)[:, :longest]


def _softmax_times(x, seen, v):
    """softmax over the seen keys times v; rows that see nothing give zeros."""
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))


# ------------------------------------------------------------------ the definitions in 64 bits
def _to_grid(x, low, bits, top):
    """x >= 0 to the nearest value with `bits` bits behind the leading one (ties to even), steps of 2^low at least."""
    e = torch.floor(torch.log2(x.clamp(min=2.0 ** (low + bits)))).clamp(min=low + bits)
    step = torch.exp2(e - bits)
    return torch.minimum(torch.round(x / step) * step, torch.full_like(x, top))


def _held64(x, ts):
    """What 4 bits keep of rows [..., 128] of 64-bit numbers."""
    y = (x / ts).reshape(*x.shape[:-1], -1, GROUP)
    s = _to_grid(y.abs().max(-1, keepdim=True).values / 6.0, -9, 3, 448.0)
    z = torch.where(s > 0, y.abs() / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(y))
    return (_to_grid(z, -1, 1, 6.0) * torch.sign(y) * s * ts).reshape(x.shape)


def _cache64(s, kv, blocks):
    """The named blocks' rows [n * 256, Hkv, 128] in 64 bits, from the bits of the codes and scales."""
    d, c = s["data"][kv][blocks].flatten(0, 1).int(), s["scales"][kv][blocks].flatten(0, 1).int()
    n = torch.stack((d % 16, d // 16), -1).reshape(*d.shape[:-1], D)
    m, e = (n % 2).double(), (n // 2 % 4).double()
    x = torch.where(e > 0, torch.exp2(e - 1) * (1 + m / 2), m / 2) * (1 - 2 * (n // 8))
    m, e = (c % 8).double(), (c // 8 % 16).double()
    sc = torch.where(e > 0, torch.exp2(e - 7) * (1 + m / 8), torch.exp2(e - 9) * m)
    return x * sc.repeat_interleave(GROUP, -1) * s["case"]["ts"]


def _attend64(q, k, v, cached):
    """Causal attention of one sequence in 64 bits: q [n, Hq, D] at positions cached.., k and v [L, Hkv, D]."""
    n, hq, _ = q.shape
    g = hq // k.shape[1]
    out = torch.empty((n, hq, D), dtype=torch.float64, device=DEV)
    keys = torch.arange(k.shape[0], device=DEV)
    for r in range(0, n, 2048):
        hidden = keys[None] > cached + torch.arange(r, min(n, r + 2048), device=DEV)[:, None]
        for h in range(hq):
            x = (q[r:r + 2048, h].double() @ k[:, h // g].T) / math.sqrt(D)
            p = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
            out[r:r + 2048, h] = p @ v[:, h // g]
    return out


def exact(case, seed):
    op = case["op"]
    if op in ("fork", "compact"):
        return None  # whole numbers and copies
    s = prepare(case, seed)
    if op == "write_q4":
        x = _held64(s["kv"].double(), case["ts"])
        return x[:, :case["hkv"]], x[:, case["hkv"]:]
    if op == "norm_rope":
        hq, hkv, rot = case["hq"], case["hkv"], case["rot"]
        pos, first, parts = s["positions"].double(), 0, []
        for a, m in enumerate(_sections(case)):
            parts.append(pos[a][:, None] * s["inv_freq"][None, first:first + m])
            first += m
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), torch.cat(parts, 1))[:, None]
        x = s["qkv"].double()
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        got = []
        for x, w in ((q, s["wq"]), (k, s["wk"])):
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / D + EPS) * w.double()
            if case["interleaved"]:
                z = turn * torch.complex(x[..., 0:rot:2], x[..., 1:rot:2])
                x[..., 0:rot:2], x[..., 1:rot:2] = z.real, z.imag
            else:
                z = turn * torch.complex(x[..., :rot // 2], x[..., rot // 2:rot])
                x[..., :rot // 2], x[..., rot // 2:rot] = z.real, z.imag
            got.append(x)
        if case["into"] == "none":
            return tuple(got)
        if case["into"] == "bf16":
            cache = s["cache"].double()
            for kv, x in enumerate((got[1], v)):
                cache[kv].view(-1, hkv, D)[s["slots"].long()] = x
            return got[0], cache
        # the operator rounds k to the model's type before it is quantised
        return got[0], _held64(got[1].to(torch.bfloat16).double(), case["ts"]), _held64(v, case["ts"])
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    if op == "decode_q4":
        for b, n in enumerate(_lengths(case)):
            blocks = s["tables"][b, :-(-n // BS)].long()
            k, v = (_cache64(s, kv, blocks)[:n] for kv in range(2))
            out[b:b + 1] = _attend64(s["q"][b:b + 1], k, v, n - 1)
        return out
    at = 0
    for b, (n, cached) in enumerate(_prompts(case)):
        blocks = s["tables"][b, :-(-n // BS)].long()
        k, v = (_cache64(s, kv, blocks)[:n] for kv in range(2))
        out[at:at + n - cached] = _attend64(s["q"][at:at + n - cached], k, v, cached)
        at += n - cached
    return out
