"""Four operators of a serving step over a paged KV cache, as cases to measure.

  rope    rotary positions of one or several axes (time, height, width) applied to q
          and to the new K rows, K and V written straight into their cache slots
  scored  attention over the paged cache that also adds each cached row's share of the
          attention to a ledger: scores[seq, kv head, row] += sum over the head's query
          rows of softmax weight
  evict   eviction by those scores: every KV head of a sequence longer than `budget`
          keeps its `sinks` first and `recent` last positions and, of the others, the
          highest scores; kept rows from behind the budget fill the holes before it
  verify  acceptance of drafted tokens against the target's probabilities from given
          random numbers, the replacement token, and the cache length after rejection

Layouts: caches [blocks, kv heads, block size, head dim], block tables int32
[seqs, blocks per seq], ledgers [seqs, kv heads, rows] with row t of sequence i in
block table[i, t // block size].  With `own` false every operator is written out in
elementary torch operations.
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # a few sequences' new tokens, plain one-axis positions: launch latency
        dict(name="rope_few_tokens", op="rope", tokens=8, hq=32, hkv=8, d=128, bs=16, dtype="fp16",
             axes=1, rot=128, inter=False, fp8=False, packed=False),
        # a step of chunked prompts (16 x 512 tokens) with image positions, q/k/v slices
        # of one fused projection's output
        dict(name="rope_chunk_3axis", op="rope", tokens=8192, hq=32, hkv=8, d=128, bs=16,
             dtype="bf16", axes=3, rot=128, inter=False, fp8=False, packed=True),
        # an odd number of prompt tokens into an FP8 cache, adjacent pairs, half rotated
        dict(name="rope_chunk_fp8", op="rope", tokens=4099, hq=32, hkv=32, d=128, bs=16,
             dtype="fp16", axes=2, rot=64, inter=True, fp8=True, packed=False),
        # three short sequences: latency
        dict(name="scored_tiny", op="scored", seqs=3, q_len=1, hq=4, hkv=4, d=64, bs=16,
             dtype="fp16", lens="fixed", lo=17, hi=37, splits=1, fp8=False),
        # grouped-query decode of a batch with a long-tailed spread of lengths
        dict(name="scored_gqa", op="scored", seqs=64, q_len=1, hq=32, hkv=8, d=128, bs=16,
             dtype="bf16", lens="lognormal", lo=1500, hi=8192, splits=1, fp8=False),
        # few long sequences, split over their length
        dict(name="scored_long", op="scored", seqs=4, q_len=1, hq=32, hkv=8, d=128, bs=16,
             dtype="bf16", lens="fixed", lo=32768, hi=32768, splits=16, fp8=False),
        # one KV head per query head over an FP8 cache
        dict(name="scored_mha_fp8", op="scored", seqs=32, q_len=1, hq=32, hkv=32, d=128, bs=16,
             dtype="fp16", lens="uniform", lo=512, hi=4096, splits=1, fp8=True),
        # prompts in chunks: the ledger's first entries come from here
        dict(name="scored_chunk", op="scored", seqs=4, q_len=1024, hq=32, hkv=8, d=128, bs=16,
             dtype="bf16", lens="uniform", lo=2048, hi=8192, splits=1, fp8=False),
        # steady state: every step one row over budget in every sequence
        dict(name="evict_step", op="evict", seqs=64, hkv=8, d=128, bs=16, dtype="bf16", fp8=False,
             lens="fixed", lo=1025, hi=1025, budget=1024, sinks=4, recent=256),
        # after the prompts: from their whole lengths down to the budget
        dict(name="evict_prompts", op="evict", seqs=16, hkv=8, d=128, bs=16, dtype="bf16",
             fp8=False, lens="uniform", lo=4097, hi=32768, budget=2048, sinks=4, recent=512),
        # one sequence, one drafted token, a small vocabulary: latency
        dict(name="verify_one", op="verify", seqs=1, k=1, vocab=32000, ragged=False, sure=False),
        # a batch of seven drafted tokens each over a large vocabulary, some with fewer
        dict(name="verify_batch", op="verify", seqs=64, k=7, vocab=131071, ragged=True, sure=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "scored", "scored", "evict", "verify"])
    if op == "rope":
        hkv = rng.choice([1, 2, 4, 8, 32])
        fp8 = rng.random() < 0.35
        d = 128 if fp8 else rng.choice([64, 128])
        c = dict(op=op, hq=hkv * rng.choice([1, 2, 4] if hkv < 32 else [1]), hkv=hkv, d=d,
                 bs=rng.choice([8, 16, 32]), dtype=rng.choice(["fp16", "bf16"]),
                 axes=rng.choice([1, 2, 3]), rot=rng.choice([d, d, d // 2, d // 4 * 3]),
                 inter=rng.random() < 0.5, fp8=fp8, packed=rng.random() < 0.5)
        most = 8192 * 48 * 128 // ((c["hq"] + 2 * hkv) * d)
        c["tokens"] = _log(rng, 1, min(16384, most))
        return c
    if op == "scored":
        hkv = rng.choice([1, 2, 4, 8, 32])
        fp8 = rng.random() < 0.3
        kind = rng.choice(["one", "one", "verify", "chunk"])
        c = dict(op=op, seqs=_log(rng, 1, 64), hq=hkv * rng.choice([1, 2, 3, 4, 8] if hkv < 32 else [1]),
                 hkv=hkv, d=128 if fp8 else rng.choice([64, 128]), bs=rng.choice([8, 16, 16, 32]),
                 dtype=rng.choice(["fp16", "bf16"]), lens=rng.choice(["uniform", "lognormal"]),
                 splits=rng.choice([1, 1, 2, 5]), fp8=fp8,
                 q_len=1 if kind == "one" else rng.randint(2, 16) if kind == "verify" else _log(rng, 17, 1024))
        hi = _log(rng, 40, 16384)
        if c["lens"] == "uniform":
            c["lo"], c["hi"] = rng.randint(1, hi), hi
        else:
            c["lo"], c["hi"] = max(1, hi // 4), hi
        while c["seqs"] > 1 and (c["seqs"] * hi * hkv * c["d"] > 64 * 4096 * 8 * 128 or
                                 c["seqs"] * c["hq"] * c["q_len"] * hi > 4 * 32 * 1024 * 4096):
            c["seqs"] //= 2
        while c["seqs"] * c["hq"] * c["q_len"] * hi > 4 * 32 * 1024 * 4096:
            c["q_len"] = (c["q_len"] + 1) // 2
        return c
    if op == "evict":
        fp8 = rng.random() < 0.3
        hkv = rng.choice([1, 2, 4, 8, 32])
        c = dict(op=op, seqs=_log(rng, 1, 64), hkv=hkv, d=rng.choice([64, 128]) if not fp8 else 128,
                 bs=rng.choice([8, 16, 32]), dtype=rng.choice(["fp16", "bf16"]), fp8=fp8,
                 budget=_log(rng, 16, 4096))
        c["sinks"] = rng.randint(0, min(8, c["budget"] // 4))
        c["recent"] = rng.randint(0, c["budget"] // 2)
        if rng.random() < 0.4:  # a few rows over budget
            c["lens"], c["lo"] = "uniform", c["budget"]
            c["hi"] = c["budget"] + rng.randint(1, 8)
        else:
            c["lens"], c["lo"] = "uniform", max(1, c["budget"] // 2)
            c["hi"] = c["budget"] + _log(rng, 1, 32768 - c["budget"])
        while c["seqs"] > 1 and c["seqs"] * c["hi"] * hkv * c["d"] > 16 * 18000 * 8 * 128:
            c["seqs"] //= 2
        return c
    k = rng.randint(1, 8)
    c = dict(op=op, k=k, vocab=_log(rng, 1000, 160000), ragged=rng.random() < 0.5,
             sure=rng.random() < 0.3)
    c["seqs"] = _log(rng, 1, max(1, min(64, 64 * 8 * 131072 // ((k + 1) * c["vocab"]))))
    return c


def _lens(c):
    """The sequences' lengths: a case's own, whatever the seed of its values."""
    r = random.Random(c["seqs"] * 1000003 + c["hi"])
    if c["lens"] == "lognormal":
        got = [min(c["hi"], max(1, round(c["lo"] * math.exp(0.5 * r.gauss(0, 1))))) for _ in range(c["seqs"])]
    elif c["lens"] == "fixed":
        got = [c["lo"] if i % 2 == 0 else c["hi"] for i in range(c["seqs"])]
    else:
        got = [r.randint(c["lo"], c["hi"]) for _ in range(c["seqs"])]
    return got


def work(c):
    if c["op"] == "rope":
        t, d, cache = c["tokens"], c["d"], 1 if c["fp8"] else 2
        return {"bytes": t * d * (c["hq"] * 4 + 2 * c["hkv"] * (2 + cache)) + t * (4 * c["axes"] + 8),
                "flops": t * (c["hq"] + c["hkv"]) * c["rot"] * 3}
    if c["op"] == "scored":
        lens, cache = _lens(c), 1 if c["fp8"] else 2
        g = c["hq"] // c["hkv"]
        seen = sum(sum(max(0, l - c["q_len"] + u + 1) for u in range(c["q_len"])) for l in lens)
        kv = sum(lens) * c["hkv"] * 2 * c["d"] * cache
        qo = c["seqs"] * c["q_len"] * c["hq"] * c["d"] * 2 * 2
        ledger = sum(lens) * c["hkv"] * 8
        return {"bytes": kv + qo + ledger + 4 * sum(-(-l // c["bs"]) for l in lens),
                "flops": seen * c["hkv"] * g * c["d"] * 4}
    if c["op"] == "evict":
        row = 2 * c["d"] * (1 if c["fp8"] else 2)
        total = 0.0
        for l in _lens(c):
            b = min(l, c["budget"])
            total += 8 * l + 8 * b
            if l > c["budget"]:
                # kept rows from behind the budget: the last `recent`, and of the rest
                # as large a share as lies there
                late = min(c["recent"], l - b)
                rest = b - c["sinks"] - c["recent"]
                free = l - c["sinks"] - c["recent"]
                behind = max(0, l - b - late)
                moved = late + (rest * behind / free if free > 0 else 0)
                total += 2 * row * moved
        return {"bytes": total * c["hkv"] + 4 * c["seqs"] * 3, "flops": 0}
    # the drafted tokens' entries, then one vocabulary row of each distribution
    return {"bytes": c["seqs"] * (c["vocab"] * 4 * (1 if c["sure"] else 2) + (c["k"] + 1) * 24),
            "flops": c["seqs"] * c["vocab"] * 3}


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _pool(c, lens, g):
    """Caches of normal values, a block table over a random permutation of the pool."""
    bs = c["bs"]
    per = [-(-l // bs) for l in lens]
    width, used = max(1, max(per)), sum(per)
    blocks = used + 8
    order = torch.randperm(blocks, generator=g, device="cuda", dtype=torch.int32)
    table = torch.empty(len(lens), width, dtype=torch.int32, device="cuda")
    table[:] = order[used]  # entries past a sequence's end: a block of nobody's
    at = 0
    for i, n in enumerate(per):
        table[i, :n] = order[at:at + n]
        at += n
    shape = (blocks, c["hkv"], bs, c["d"])
    k, v = (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) for _ in range(2))
    if c["fp8"]:
        scales = [torch.rand(c["hkv"], generator=g, device="cuda") * 0.03 + 0.02 for _ in range(2)]
        k, v = ((x / s[:, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
                for x, s in zip((k, v), scales))
    else:
        scales = [None, None]
        k, v = k.to(DTYPES[c["dtype"]]), v.to(DTYPES[c["dtype"]])
    return k, v, table, scales[0], scales[1]


def prepare(c, seed):
    g = _gen(seed)
    s = {"c": c}
    if c["op"] == "rope":
        t, d, hq, hkv, half = c["tokens"], c["d"], c["hq"], c["hkv"], c["rot"] // 2
        pool = {**c, "seqs": 1}
        s["k_cache"], s["v_cache"], table, s["k_scale"], s["v_scale"] = _pool(pool, [t + 13], g)
        at = torch.arange(t, device="cuda") + 13  # the tokens begin inside a block
        s["slots"] = table[0, at // c["bs"]].long() * c["bs"] + at % c["bs"]
        if t > 4:
            s["slots"][t // 2] = -1  # a padding row: no cache slot
        dt = DTYPES[c["dtype"]]
        if c["packed"]:
            qkv = torch.randn(t, hq + 2 * hkv, d, generator=g, device="cuda").to(dt)
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        else:
            s["q"], s["k"], s["v"] = (torch.randn(t, h, d, generator=g, device="cuda").to(dt)
                                      for h in (hq, hkv, hkv))
        s["q_out"] = torch.empty(t, hq, d, dtype=dt, device="cuda")
        # far positions on every axis, as behind a long context
        first = torch.randint(0, 1 << 20, (c["axes"], 1), generator=g, device="cuda")
        step = torch.randint(0, 3, (c["axes"], t), generator=g, device="cuda")
        s["positions"] = (first + step.cumsum(1)).to(torch.int32).contiguous()
        f = [10000.0 ** (-i / half) for i in range(half)]
        s["inv_freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        s["pair_axis"] = (torch.arange(half, device="cuda") * c["axes"] // half).to(torch.int32)
        # turns per position in units of 2^-64 of a turn
        s["turns"] = torch.tensor([int(round(x / (2 * math.pi) * 2.0 ** 64)) for x in f],
                                  dtype=torch.int64, device="cuda")
        return s
    if c["op"] == "scored":
        lens = _lens(c)
        s["lens"] = lens
        s["k_cache"], s["v_cache"], s["table"], s["k_scale"], s["v_scale"] = _pool(c, lens, g)
        s["context_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        # some rows were evicted before: the sequences are longer than their caches
        s["seq_lens"] = s["context_lens"] + torch.randint(0, 100, (c["seqs"],), generator=g,
                                                         device="cuda", dtype=torch.int32)
        dt = DTYPES[c["dtype"]]
        s["q"] = (2 * torch.randn(c["seqs"], c["q_len"], c["hq"], c["d"], generator=g, device="cuda")).to(dt)
        s["out"] = torch.empty_like(s["q"])
        rows = s["table"].shape[1] * c["bs"]
        s["scores"] = torch.rand(c["seqs"], c["hkv"], rows, generator=g, device="cuda")
        s["row_pos"] = torch.arange(rows, device="cuda", dtype=torch.int32).repeat(c["seqs"], c["hkv"], 1)
        s["scale"] = c["d"] ** -0.5
        # room for the splits' partial results and the scores of up to 16 query tokens
        per_row = c["splits"] * c["hq"] * c["q_len"] * (c["d"] + 2) * 4
        raw = c["hq"] * c["q_len"] * (rows + 16) * 4 if c["q_len"] <= 16 else 0
        s["workspace"] = torch.empty(c["seqs"] * (per_row + raw) + 4096, dtype=torch.uint8, device="cuda")
        return s
    if c["op"] == "evict":
        lens = _lens(c)
        s["lens"] = lens
        s["k_cache"], s["v_cache"], s["table"], _, _ = _pool(c, lens, g)
        s["context_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["seq_lens"] = s["context_lens"] + 7  # rows that earlier calls evicted
        n, h, rows = c["seqs"], c["hkv"], s["table"].shape[1] * c["bs"]
        # a few rows draw most of the attention, some none at all
        scores = torch.exp(2 * torch.randn(n, h, rows, generator=g, device="cuda"))
        scores[torch.rand(n, h, rows, generator=g, device="cuda") < 0.05] = 0
        s["scores"] = scores
        pos = torch.arange(rows, device="cuda", dtype=torch.int32).repeat(n, h, 1)
        s["row_pos"] = torch.where(pos >= c["sinks"], pos + 7, pos)
        s["scores_out"] = torch.zeros_like(scores)
        s["row_pos_out"] = torch.zeros_like(s["row_pos"])
        s["new_lens"] = torch.zeros(n, dtype=torch.int32, device="cuda")
        s["workspace"] = torch.empty(n * h * (rows + 64) * 8 + 4096, dtype=torch.uint8, device="cuda")
        return s
    n, k, v = c["seqs"], c["k"], c["vocab"]
    logits = 2 * torch.randn(n, k + 1, v, generator=g, device="cuda")
    s["target"] = torch.softmax(logits, -1)
    noise = torch.randn(n, k, v, generator=g, device="cuda")
    draft = torch.softmax(logits[:, :k] + 0.7 * noise, -1)
    race = -torch.rand(n, k, v, generator=g, device="cuda").clamp_min(1e-30).log()
    s["tokens"] = (draft / race).argmax(-1).to(torch.int32)
    s["draft"] = None if c["sure"] else draft
    s["accept_u"] = torch.rand(n, k, generator=g, device="cuda")
    s["sample_u"] = torch.rand(n, generator=g, device="cuda")
    s["draft_lens"] = torch.randint(0, k + 1, (n,), generator=g, device="cuda", dtype=torch.int32) \
        if c["ragged"] else None
    s["context_lens"] = torch.randint(k + 1, 4096, (n,), generator=g, device="cuda", dtype=torch.int32)
    s["out_tokens"] = torch.empty(n, k + 1, dtype=torch.int32, device="cuda")
    s["accepted"] = torch.empty(n, dtype=torch.int32, device="cuda")
    s["new_lens"] = torch.empty(n, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------------------- runs
def run(s):
    return {"rope": _run_rope, "scored": _run_scored, "evict": _run_evict,
            "verify": _run_verify}[s["c"]["op"]](s)


def _codes(s, name):
    """A cache as it is returned: the values that its elements stand for."""
    return s[name].view(torch.float8_e4m3fn) if s["c"]["fp8"] else s[name]


def _rotate(x, cos, sin, inter):
    half = cos.shape[-1]
    x = x.float()
    rot, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (rot[..., 0::2], rot[..., 1::2]) if inter else (rot[..., :half], rot[..., half:])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    rot = torch.stack((ra, rb), -1).flatten(-2) if inter else torch.cat((ra, rb), -1)
    return torch.cat((rot, rest), -1)


def _run_rope(s):
    c = s["c"]
    if own:
        import paged_kv_cache_20_gb300 as pa
        pa.pa_rope_append(s["q_out"], s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"],
                          s["positions"], s["slots"], s["turns"], s["pair_axis"],
                          interleaved=c["inter"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    else:
        # angles in 64 bits: far positions lose their fraction in 32
        angle = s["positions"][s["pair_axis"].long()].double() * s["inv_freq"][:, None]
        cos, sin = angle.cos().float().t()[:, None], angle.sin().float().t()[:, None]
        s["q_out"].copy_(_rotate(s["q"], cos, sin, c["inter"]))
        k, v = _rotate(s["k"], cos, sin, c["inter"]), s["v"].float()
        live = s["slots"] >= 0
        slots = s["slots"][live]
        blk, off = slots // c["bs"], slots % c["bs"]
        if c["fp8"]:
            k, v = k / s["k_scale"][:, None], v / s["v_scale"][:, None]
            k, v = (x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
        s["k_cache"][blk, :, off] = k[live].to(s["k_cache"].dtype)
        s["v_cache"][blk, :, off] = v[live].to(s["v_cache"].dtype)
    return {"q": s["q_out"], "k_cache": _codes(s, "k_cache"), "v_cache": _codes(s, "v_cache")}


def _gather(s, name, scale, t):
    """Rows 0..t-1 of every sequence: [seqs, t, kv heads, head dim] in 32 bits."""
    c, at = s["c"], torch.arange(t, device="cuda")
    x = s[name][s["table"][:, at // c["bs"]].long(), :, at % c["bs"]]
    if c["fp8"]:
        return x.view(torch.float8_e4m3fn).float() * scale[:, None]
    return x.float()


def _run_scored(s):
    c = s["c"]
    if own:
        import paged_kv_cache_20_gb300 as pa
        pa.pa_decode_scored(s["out"], s["scores"], s["q"], s["k_cache"], s["v_cache"], s["table"],
                            s["context_lens"], s["scale"], q_len=c["q_len"], num_splits=c["splits"],
                            workspace=s["workspace"], row_pos=s["row_pos"], seq_lens=s["seq_lens"],
                            k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"out": s["out"], "scores": s["scores"], "row_pos": s["row_pos"]}
    n, u, hq, d = s["q"].shape
    t, h = max(s["lens"]), c["hkv"]
    at, lens = torch.arange(t, device="cuda"), s["context_lens"][:, None]
    alive = at < lens                                                     # [n, t]
    q = s["q"].float().view(n, u, h, hq // h, d)
    k = _gather(s, "k_cache", s["k_scale"], t)
    x = torch.einsum("nuhgd,nthd->nhgut", q, k) * s["scale"]
    del k
    # query token j sees rows up to len - q_len + j
    sees = at < (lens - u + 1 + torch.arange(u, device="cuda"))[:, :, None]   # [n, u, t]
    x.masked_fill_(~sees[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(top.masked_fill(top == -math.inf, 0)).exp_()
    total = p.sum(-1, keepdim=True)
    p = p.div_(total.masked_fill(total == 0, 1))
    v = _gather(s, "v_cache", s["v_scale"], t).masked_fill(~alive[:, :, None, None], 0)
    s["out"].copy_(torch.einsum("nhgut,nthd->nuhgd", p, v).reshape(n, u, hq, d))
    share = p.sum((2, 3))                                                 # [n, h, t]
    new = (at >= lens - u) & alive
    was = s["scores"][:, :, :t]
    s["scores"][:, :, :t] = torch.where(alive[:, None], torch.where(new[:, None], 0, was) + share, was)
    pos = (at - lens + s["seq_lens"][:, None]).to(torch.int32)
    s["row_pos"][:, :, :t] = torch.where(new[:, None], pos[:, None], s["row_pos"][:, :, :t])
    return {"out": s["out"], "scores": s["scores"], "row_pos": s["row_pos"]}


def _run_evict(s):
    c = s["c"]
    if own:
        import paged_kv_cache_20_gb300 as pa
        pa.pa_evict(s["k_cache"], s["v_cache"], s["scores"], s["row_pos"], s["table"],
                    s["context_lens"], s["seq_lens"], c["budget"], sinks=c["sinks"],
                    recent=c["recent"], scores_out=s["scores_out"], row_pos_out=s["row_pos_out"],
                    new_lens=s["new_lens"], workspace=s["workspace"])
    else:
        n, h, rows = s["scores"].shape
        at, lens = torch.arange(rows, device="cuda"), s["context_lens"][:, None, None]
        pos = s["row_pos"]
        safe = (pos < c["sinks"]) | (pos >= s["seq_lens"][:, None, None] - c["recent"])
        rank = s["scores"].masked_fill(safe, math.inf).masked_fill(at >= lens, -math.inf)
        order = rank.sort(dim=-1, descending=True, stable=True)[1]  # ties: the lowest row
        kept = torch.zeros_like(safe).scatter_(-1, order[..., :c["budget"]], True)
        kept = (kept | (lens <= c["budget"])) & (at < lens)
        hole = ~kept & (at < c["budget"]) & (at < lens)
        move = kept & (at >= c["budget"]) & (lens > c["budget"])
        # the i-th kept row from behind the budget goes to the i-th hole of its head
        i, j, to = hole.nonzero(as_tuple=True)
        _, _, frm = move.nonzero(as_tuple=True)
        to_blk, frm_blk = (s["table"][i, x // c["bs"]].long() for x in (to, frm))
        stay = kept & (at < c["budget"])
        s["scores_out"].copy_(torch.where(stay, s["scores"], s["scores_out"]))
        s["row_pos_out"].copy_(torch.where(stay, pos, s["row_pos_out"]))
        s["scores_out"][i, j, to] = s["scores"][i, j, frm]
        s["row_pos_out"][i, j, to] = pos[i, j, frm]
        # (the cache as 16-byte pieces: elements are moved, not read)
        kc, vc = (s[x].view(torch.int64) for x in ("k_cache", "v_cache"))
        kc[to_blk, j, to % c["bs"]] = kc[frm_blk, j, frm % c["bs"]]
        vc[to_blk, j, to % c["bs"]] = vc[frm_blk, j, frm % c["bs"]]
        s["new_lens"].copy_(s["context_lens"].clamp_max(c["budget"]))
    return {"k_cache": _codes(s, "k_cache"), "v_cache": _codes(s, "v_cache"),
            "scores": s["scores_out"], "row_pos": s["row_pos_out"], "new_lens": s["new_lens"]}


def _run_verify(s):
    c = s["c"]
    if own:
        import paged_kv_cache_20_gb300 as pa
        pa.pa_verify_drafts(s["target"], s["draft"], s["tokens"], s["accept_u"], s["sample_u"],
                            draft_lens=s["draft_lens"], context_lens=s["context_lens"],
                            out_tokens=s["out_tokens"], num_accepted=s["accepted"],
                            new_lens=s["new_lens"])
    else:
        n, k = c["seqs"], c["k"]
        here, at = torch.arange(n, device="cuda"), torch.arange(k + 1, device="cuda")
        given = at.new_full((n,), k) if s["draft_lens"] is None else s["draft_lens"].long()
        x = s["tokens"].long()[..., None]
        # 64 bits: a product next to its border, a sum over the vocabulary
        p = s["target"][:, :k].gather(-1, x)[..., 0].double()
        q = 1.0 if c["sure"] else s["draft"].gather(-1, x)[..., 0].double()
        ok = (s["accept_u"].double() * q < p) & (at[:k] < given[:, None])
        count = ok.long().cumprod(-1).sum(-1)
        w = s["target"][here, count].double()
        if c["sure"]:
            less = torch.zeros_like(w).scatter_(1, x[here, count.clamp_max(k - 1)], 1.0)
        else:
            less = s["draft"][here, count.clamp_max(k - 1)].double()
        w = torch.where((count < given)[:, None], (w - less).clamp_min(0), w)
        total = w.cumsum(-1)
        pick = (total <= s["sample_u"].double()[:, None] * total[:, -1:]).sum(-1)
        last = (c["vocab"] - 1) - (w.flip(-1) > 0).long().argmax(-1)
        pick = torch.minimum(pick, last).to(torch.int32)
        tokens = torch.cat((s["tokens"], pick[:, None]), -1)
        tokens = torch.where(at < count[:, None], tokens, -1)
        s["out_tokens"].copy_(torch.where(at == count[:, None], pick[:, None], tokens))
        s["accepted"].copy_(count)
        s["new_lens"].copy_(s["context_lens"] - (k - count))
    return {"tokens": s["out_tokens"], "accepted": s["accepted"], "new_lens": s["new_lens"]}


# --------------------------------------------------------------------- 64-bit results
def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        return _exact_rope(s)
    if c["op"] == "scored":
        return _exact_scored(s)
    return None  # rows moved bit for bit and whole numbers: nothing is rounded


def _exact_rope(s):
    c = s["c"]
    half = c["rot"] // 2
    theta = s["inv_freq"] * s["positions"].double().t()[:, s["pair_axis"].long()]
    turn = torch.polar(torch.ones_like(theta), theta)[:, None]

    def spun(x):
        y = x.double().clone()
        if c["inter"]:
            z = torch.complex(y[..., 0:c["rot"]:2], y[..., 1:c["rot"]:2]) * turn
            y[..., 0:c["rot"]:2], y[..., 1:c["rot"]:2] = z.real, z.imag
        else:
            z = torch.complex(y[..., :half], y[..., half:c["rot"]]) * turn
            y[..., :half], y[..., half:c["rot"]] = z.real, z.imag
        return y

    caches = []
    for name, rows, scale in (("k_cache", spun(s["k"]), s["k_scale"]),
                              ("v_cache", s["v"].double(), s["v_scale"])):
        if c["fp8"]:  # codes: which ones the rounding picks is the operator's, not an error
            caches.append(None)
            continue
        pool = s[name].double().transpose(1, 2).reshape(-1, c["hkv"], c["d"])
        keep = (s["slots"] >= 0).nonzero()[:, 0]
        pool.index_copy_(0, s["slots"][keep], rows[keep])
        caches.append(pool.view(-1, c["bs"], c["hkv"], c["d"]).transpose(1, 2).contiguous())
    return {"q": spun(s["q"]), "k_cache": caches[0], "v_cache": caches[1]}


def _exact_scored(s):
    c = s["c"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    scores = s["scores"].double()
    g = c["hq"] // c["hkv"]
    for i, length in enumerate(s["lens"]):
        blocks = s["table"][i, :-(-length // c["bs"])].long()

        def rows(name, scale):
            x = s[name][blocks]
            x = x.view(torch.float8_e4m3fn).to(torch.float64) * scale.double()[:, None, None] \
                if c["fp8"] else x.double()
            return x.transpose(0, 1).reshape(c["hkv"], -1, c["d"])[:, :length]

        k, v = rows("k_cache", s["k_scale"]), rows("v_cache", s["v_scale"])
        first = length - c["q_len"]
        scores[i, :, max(0, first):length] = 0
        for h in range(c["hkv"]):
            for j in range(g):
                x = s["q"][i, :, h * g + j].double() @ k[h].t() * s["scale"]
                col = torch.arange(length, device="cuda")
                row = torch.arange(c["q_len"], device="cuda")[:, None]
                x = torch.where(col <= first + row, x, -math.inf)
                w = torch.softmax(x, -1).nan_to_num(0.0)  # a query that sees nothing
                out[i, :, h * g + j] = w @ v[h]
                scores[i, h, :length] += w.sum(0)
    return {"out": out, "scores": scores, "row_pos": None}
