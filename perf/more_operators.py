"""Operators around an 8-bit paged KV cache and the step's end, as cases to measure.

  append  this step's K/V rows quantised into a cache of e4m3 codes with one scale for
          every block and KV head: the scale is the smallest power of two that holds
          the block's rows, grows with them, and older rows are brought to the new one
  attend  attention over that cache: value = code * scale of its block and head
  pages   the pool's bookkeeping on the device: blocks freed, reserved, forked
          (full blocks shared, the partial last one copied) and compacted, by counts
          of the table entries that refer to each block
  logits  penalties for repeated tokens, biases and grammar masks on a step's logits
          (every draft position behind the drafts before it), and the probabilities
          that the verification of drafts takes

Layouts: caches [blocks, kv heads, block size, head dim], scales fp32 [blocks, kv heads,
2] (K, V), block tables int32 [seqs, blocks per seq] with -1 for no block, reference
counts int32 [blocks].  With `own` false every operator is written out in elementary
torch operations.
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
LEAST, MOST = 2.0 ** -40, 2.0 ** 40  # block scales lie between


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step's one new token a sequence: latency
        dict(name="append_step", op="append", seqs=64, q_len=1, hkv=8, d=128, bs=16, dtype="bf16",
             lens="uniform", lo=512, hi=4096, packed=False),
        # a step of chunked prompts, k and v slices of one fused projection's output
        dict(name="append_prompts", op="append", seqs=16, q_len=512, hkv=32, d=128, bs=16, dtype="fp16",
             lens="uniform", lo=509, hi=4099, packed=True),
        # three short sequences: latency
        dict(name="attend_tiny", op="attend", seqs=3, q_len=1, hq=4, hkv=4, d=128, bs=16, dtype="fp16",
             lens="fixed", lo=17, hi=37, splits=1),
        # grouped-query decode of a batch with a long-tailed spread of lengths
        dict(name="attend_gqa", op="attend", seqs=64, q_len=1, hq=32, hkv=8, d=128, bs=16, dtype="bf16",
             lens="lognormal", lo=1500, hi=8192, splits=1),
        # one KV head per query head
        dict(name="attend_mha", op="attend", seqs=32, q_len=1, hq=32, hkv=32, d=128, bs=16, dtype="fp16",
             lens="uniform", lo=512, hi=4096, splits=1),
        # few long sequences, split over their length
        dict(name="attend_long", op="attend", seqs=4, q_len=1, hq=32, hkv=8, d=128, bs=32, dtype="bf16",
             lens="fixed", lo=32768, hi=32768, splits=16),
        # prompts in chunks over what is cached already
        dict(name="attend_chunk", op="attend", seqs=4, q_len=1024, hq=32, hkv=8, d=128, bs=16,
             dtype="bf16", lens="uniform", lo=2048, hi=8192, splits=1),
        # a beam step: the losing beams' blocks freed, the winners forked, tails copied
        dict(name="pages_beam", op="pages", kind="fork", parents=16, children=3, lens="uniform", lo=500,
             hi=4000, hkv=8, d=128, bs=16, bytes=2, blocks=8192),
        # continuous batching in a large pool: finished sequences go, prompts come,
        # everyone else grows by a step
        dict(name="pages_turnover", op="pages", kind="turnover", seqs=256, lens="uniform", lo=64,
             hi=12000, bs=16, blocks=131072),
        # a pool with holes after many requests, moved to its front with data and scales
        dict(name="pages_compact", op="pages", kind="compact", seqs=64, lens="uniform", lo=200,
             hi=4000, hkv=8, d=128, bs=16, bytes=1, blocks=16384),
        # one sequence, the token after its answer so far: latency
        dict(name="logits_one", op="logits", seqs=1, rows=1, vocab=32000, dtype="fp16", hist=700, bias=4,
             masked=False, probs=True),
        # a batch of seven drafted tokens each over a large vocabulary, under grammars
        dict(name="logits_batch", op="logits", seqs=64, rows=8, vocab=131071, dtype="bf16", hist=4096,
             bias=32, masked=True, probs=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "pages", "logits"])
    if op == "append":
        hkv = rng.choice([1, 2, 4, 8, 32])
        c = dict(op=op, seqs=_log(rng, 1, 128), q_len=rng.choice([1, 1, rng.randint(2, 16), _log(rng, 17, 2048)]),
                 hkv=hkv, d=128, bs=rng.choice([8, 16, 32]), dtype=rng.choice(["fp16", "bf16"]),
                 lens="uniform", packed=rng.random() < 0.5)
        while c["seqs"] > 1 and c["seqs"] * c["q_len"] * hkv > 16 * 512 * 32:
            c["seqs"] //= 2
        c["hi"] = _log(rng, 40, 8192)
        c["lo"] = rng.randint(1, c["hi"])
        while c["seqs"] > 1 and c["seqs"] * c["hi"] * hkv > 64 * 8192 * 8:
            c["seqs"] //= 2
        return c
    if op == "attend":
        hkv = rng.choice([1, 2, 4, 8, 32])
        kind = rng.choice(["one", "one", "verify", "chunk"])
        c = dict(op=op, seqs=_log(rng, 1, 64), hq=hkv * rng.choice([1, 2, 3, 4, 8] if hkv < 32 else [1]),
                 hkv=hkv, d=128, bs=rng.choice([8, 16, 16, 32]), dtype=rng.choice(["fp16", "bf16"]),
                 lens=rng.choice(["uniform", "lognormal"]), splits=rng.choice([1, 1, 2, 5]),
                 q_len=1 if kind == "one" else rng.randint(2, 16) if kind == "verify" else _log(rng, 17, 1024))
        hi = _log(rng, 40, 16384)
        c["lo"], c["hi"] = (rng.randint(1, hi) if c["lens"] == "uniform" else max(1, hi // 4)), hi
        while c["seqs"] > 1 and (c["seqs"] * hi * hkv > 64 * 4096 * 8 or
                                 c["seqs"] * c["hq"] * c["q_len"] * hi > 4 * 32 * 1024 * 4096):
            c["seqs"] //= 2
        while c["seqs"] * c["hq"] * c["q_len"] * hi > 4 * 32 * 1024 * 4096:
            c["q_len"] = (c["q_len"] + 1) // 2
        return c
    if op == "pages":
        kind = rng.choice(["fork", "turnover", "compact"])
        bs = rng.choice([8, 16, 32])
        c = dict(op=op, kind=kind, bs=bs, lens="uniform", hi=_log(rng, 40, 8000))
        c["lo"] = rng.randint(1, c["hi"])
        if kind == "turnover":
            c["seqs"] = _log(rng, 1, 256)
            c["blocks"] = c["seqs"] * (c["hi"] // bs + 2) + _log(rng, 1, 65536)
            return c
        c["hkv"], c["bytes"] = rng.choice([1, 2, 4, 8, 32]), rng.choice([1, 2])
        c["d"] = 128 if c["bytes"] == 1 else rng.choice([64, 128])
        most = (1 << 30) // (2 * c["hkv"] * bs * c["d"] * c["bytes"])
        if kind == "fork":
            c["parents"], c["children"] = _log(rng, 1, 32), rng.randint(1, 8)
            rows = c["parents"] * (1 + c["children"])
        else:
            c["seqs"] = rows = _log(rng, 1, 128)
        while c["hi"] > 40 and rows * (c["hi"] // bs + 2) > most // 2:
            c["hi"] //= 2
        c["lo"] = min(c["lo"], c["hi"])
        c["blocks"] = rows * (c["hi"] // bs + 2) + _log(rng, 1, min(4096, most // 4))
        return c
    c = dict(op=op, rows=rng.choice([1, 1, rng.randint(2, 9)]), vocab=_log(rng, 1000, 160000),
             dtype=rng.choice(["fp16", "bf16", "fp32"]), hist=_log(rng, 1, 8192), bias=rng.choice([0, 3, 300]),
             masked=rng.random() < 0.5, probs=rng.random() < 0.7)
    c["seqs"] = _log(rng, 1, max(1, min(128, 64 * 8 * 131072 // (c["rows"] * c["vocab"]))))
    return c


def _lens(c, n=None):
    """The sequences' lengths: a case's own, whatever the seed of its values."""
    n = c["seqs"] if n is None else n
    r = random.Random(n * 1000003 + c["hi"])
    if c["lens"] == "lognormal":
        return [min(c["hi"], max(1, round(c["lo"] * math.exp(0.5 * r.gauss(0, 1))))) for _ in range(n)]
    if c["lens"] == "fixed":
        return [c["lo"] if i % 2 == 0 else c["hi"] for i in range(n)]
    return [r.randint(c["lo"], c["hi"]) for _ in range(n)]


def _turnover(c):
    """(blocks held, tokens kept, tokens wanted) of every sequence."""
    r = random.Random(c["seqs"] * 7 + c["hi"])
    out = []
    for n in _lens(c):
        if r.random() < 0.2:  # finished; another prompt takes its row
            out.append((n, 0, r.randint(1, c["hi"])))
        elif r.random() < 0.2:  # drafts rejected, or rows evicted
            keep = r.randint(1, n)
            out.append((n, keep, min(c["hi"], keep + 8)))
        else:
            out.append((n, n, min(c["hi"], n + 8)))
    return out


def work(c):
    if c["op"] == "append":
        rows = sum(min(n, c["q_len"]) for n in _lens(c))
        blocks = sum(-(-n // c["bs"]) - max(0, n - c["q_len"]) // c["bs"] for n in _lens(c))
        return {"bytes": 2 * rows * c["hkv"] * c["d"] * 3 + blocks * (c["hkv"] * 16 + 4) + 4 * c["seqs"],
                "flops": 4 * rows * c["hkv"] * c["d"]}
    if c["op"] == "attend":
        lens, g = _lens(c), c["hq"] // c["hkv"]
        seen = sum(sum(max(0, n - c["q_len"] + u + 1) for u in range(c["q_len"])) for n in lens)
        blocks = sum(-(-n // c["bs"]) for n in lens)
        return {"bytes": sum(lens) * c["hkv"] * 2 * c["d"] + blocks * (c["hkv"] * 8 + 4) +
                c["seqs"] * (c["q_len"] * c["hq"] * c["d"] * 4 + 4),
                "flops": seen * c["hkv"] * g * c["d"] * 4}
    if c["op"] == "pages":
        if c["kind"] == "turnover":
            moves = _turnover(c)
            freed = sum(-(-a // c["bs"]) - -(-min(a, k) // c["bs"]) for a, k, _ in moves)
            taken = sum(max(0, -(-w // c["bs"]) - -(-k // c["bs"])) for _, k, w in moves)
            held = sum(-(-max(a, w) // c["bs"]) for a, _, w in moves)
            return {"bytes": 4 * (c["blocks"] + held + 2 * freed + 2 * taken + 2 * c["seqs"]), "flops": 0}
        page = 2 * c["hkv"] * c["bs"] * c["d"] * c["bytes"] + (8 * c["hkv"] if c["bytes"] == 1 else 0)
        if c["kind"] == "fork":
            lens = _lens(c, c["parents"])
            tails = sum(c["children"] for n in lens if n % c["bs"])
            shared = sum(n // c["bs"] for n in lens)
            # the pool's counts to find free blocks, the rows' entries read and written,
            # the shared blocks' counts, the tails' data
            return {"bytes": 4 * c["blocks"] + 4 * shared * (3 + 2 * c["children"]) + 2 * page * tails,
                    "flops": 0}
        # live blocks lie anywhere in the pool: those behind its front part move
        live = sum(-(-n // c["bs"]) for n in _lens(c))
        moved = live * (c["blocks"] - live) / c["blocks"]
        return {"bytes": 2 * page * moved + 8 * c["blocks"] + 8 * live, "flops": 0}
    n, elt = c["seqs"] * c["rows"] * c["vocab"], DTYPES[c["dtype"]].itemsize
    return {"bytes": n * (elt + (4 if c["probs"] else elt)) + (n // 8 if c["masked"] else 0) +
            c["seqs"] * (4 * c["hist"] + 8 * c["bias"]), "flops": n * 4}


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _need(top):
    """The smallest power of two s with top <= 448 s (448 = 0.875 * 2^9), as bits."""
    m, e = torch.frexp(top)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-40, 40)
    e = torch.where(top > 0, e, -40)
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _e4m3(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _pool(c, lens, g):
    """Quantised caches of normal values, a few tokens and channels far larger than the
    rest, and a block table over a random permutation of the pool."""
    bs, h, d = c["bs"], c["hkv"], c["d"]
    per = [-(-n // bs) for n in lens]
    width, used = max(1, max(per)), sum(per)
    blocks = used + 8
    order = torch.randperm(blocks, generator=g, device="cuda", dtype=torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(per):
        table[i, :n] = order[at:at + n]
        at += n
    caches, scales = [], []
    for _ in range(2):
        x = torch.randn(blocks, h, bs, d, generator=g, device="cuda")
        big = torch.rand(blocks, h, bs, 1, generator=g, device="cuda") < 0.01
        x = torch.where(big, 20 * x, x) * (1 + 7 * (torch.rand(1, h, 1, d, generator=g, device="cuda") < 0.02))
        s = _need(x.abs().amax((2, 3)))
        caches.append(_e4m3(x / s[:, :, None, None]).view(torch.uint8))
        scales.append(s)
        del x
    return caches[0], caches[1], torch.stack(scales, -1).contiguous(), table


def prepare(c, seed):
    g = _gen(seed)
    s = {"c": c}
    if c["op"] in ("append", "attend"):
        lens = _lens(c)
        s["lens"] = lens
        s["k_cache"], s["v_cache"], s["kv_scales"], s["table"] = _pool(c, lens, g)
        s["context_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        n, u, dt = c["seqs"], c["q_len"], DTYPES[c["dtype"]]
        if c["op"] == "append":
            h, d = c["hkv"], c["d"]
            new = torch.randn(n * u, 6 * h if c["packed"] else 2 * h, d, generator=g, device="cuda")
            new = torch.where(torch.rand(n * u, 1, 1, generator=g, device="cuda") < 0.05, 10 * new, new).to(dt)
            s["k_new"], s["v_new"] = new[:, -2 * h:-h], new[:, -h:]
            if not c["packed"]:
                s["k_new"], s["v_new"] = s["k_new"].contiguous(), s["v_new"].contiguous()
            return s
        s["q"] = (0.7 * torch.randn(n, u, c["hq"], c["d"], generator=g, device="cuda")).to(dt)
        s["out"] = torch.empty_like(s["q"])
        s["scale"] = c["d"] ** -0.5
        s["workspace"] = torch.empty(c["splits"] * n * u * c["hq"] * (c["d"] + 2) * 4 + 4096, dtype=torch.uint8,
                                     device="cuda")
        return s
    if c["op"] == "pages":
        return _prepare_pages(c, s, g)
    n, r, v = c["seqs"], c["rows"], c["vocab"]
    s["logits"] = (3 * torch.randn(n, r, v, generator=g, device="cuda")).to(DTYPES[c["dtype"]])
    s["out"] = torch.empty(n, r, v, dtype=torch.float32 if c["probs"] else s["logits"].dtype, device="cuda")
    # a few tokens come again and again, as in text
    s["history"] = (torch.rand(n, c["hist"], generator=g, device="cuda") ** 4 * v).to(torch.int32).clamp_max(v - 1)
    s["history_lens"] = torch.randint(0, c["hist"] + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
    s["history_lens"][0] = c["hist"]
    s["prompt_lens"] = s["history_lens"] // 2
    s["drafts"] = torch.randint(0, v, (n, r - 1), generator=g, device="cuda", dtype=torch.int32) if r > 1 else None
    one = torch.rand(4, n, generator=g, device="cuda")
    s["repetition"], s["presence"] = 1 + 0.3 * one[0], 0.5 * one[1]
    s["frequency"], s["temperature"] = 0.5 * one[2], 0.5 + one[3]
    if n > 3:
        s["temperature"][n // 2] = 0  # one that takes the best token
    s["bias_ids"] = s["bias_values"] = None
    if c["bias"]:
        s["bias_ids"] = torch.randint(0, v, (n, c["bias"]), generator=g, device="cuda", dtype=torch.int32)
        s["bias_values"] = 4 * torch.randn(n, c["bias"], generator=g, device="cuda")
    s["mask"] = None
    if c["masked"]:  # grammars leave anything from a few tokens to nearly all
        part = torch.rand(n, r, 1, generator=g, device="cuda") ** 2
        words = -(-v // 32)
        bits = torch.rand(n, r, words * 32, generator=g, device="cuda") < part
        lane = torch.arange(32, device="cuda")
        word = (bits.view(n, r, words, 32).long() << lane).sum(-1)
        s["mask"] = torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)
        del bits, word
    return s


def _caches(c, s, g):
    shape = (c["blocks"], c["hkv"], c["bs"], c["d"])
    for name in ("k_cache", "v_cache"):
        if c["bytes"] == 1:
            s[name] = torch.randint(0, 127, shape, generator=g, device="cuda", dtype=torch.uint8)
        else:
            s[name] = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.float16)
    s["kv_scales"] = torch.rand(c["blocks"], c["hkv"], 2, generator=g, device="cuda") if c["bytes"] == 1 else None


def _prepare_pages(c, s, g):
    # which blocks the pool's live table entries hold, in the order they were taken
    ids = torch.randperm(c["blocks"], generator=g, device="cuda").tolist()

    def table_of(lens, width):
        rows, at = [], 0
        for n in lens:
            per = -(-n // c["bs"])
            rows.append(ids[at:at + per] + [-1] * (width - per))
            at += per
        return rows, at

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    width = c["hi"] // c["bs"] + 2
    if c["kind"] == "turnover":
        moves = _turnover(c)
        rows, _ = table_of([m[0] for m in moves], width)
        s["table"] = i32(rows)
        s["keep"], s["want"] = i32([m[1] for m in moves]), i32([m[2] for m in moves])
        s["missing"] = i32([0])
    elif c["kind"] == "fork":
        lens = _lens(c, c["parents"])
        k = c["children"]
        rows, at = table_of(lens, width)
        ctx = list(lens)
        src, dst = [], []
        for p, n in enumerate(lens):
            for j in range(k):  # the beams of the step before: the same prompt's blocks, an own tail
                rows.append(list(rows[p]))
                full, tail = n // c["bs"], n % c["bs"]
                if tail:
                    rows[-1][full] = ids[at]
                    at += 1
                ctx.append(n)
                src.append(p)
                dst.append(c["parents"] + p * k + j)
        s["table"], s["context_lens"] = i32(rows), i32(ctx)
        s["src"], s["dst"] = i32(src), i32(dst)
        s["keep"] = i32(lens + [0] * len(dst))
        s["pairs"] = torch.zeros(2, len(dst), dtype=torch.int32, device="cuda")
        s["counts"] = torch.zeros(2, dtype=torch.int32, device="cuda")
        _caches(c, s, g)
    else:
        rows, _ = table_of(_lens(c), width)
        s["table"] = i32(rows)
        s["table_out"] = torch.empty_like(s["table"])
        s["refs_out"] = torch.empty(c["blocks"], dtype=torch.int32, device="cuda")
        s["pairs"] = torch.zeros(2, c["blocks"] // 2, dtype=torch.int32, device="cuda")
        s["counts"] = torch.zeros(2, dtype=torch.int32, device="cuda")
        _caches(c, s, g)
    flat = s["table"].flatten()
    s["refs"] = torch.bincount(flat[flat >= 0].long(), minlength=c["blocks"]).to(torch.int32)
    s["workspace"] = torch.empty(8 * c["blocks"] + 4096, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------- runs
def run(s):
    return {"append": _run_append, "attend": _run_attend, "pages": _run_pages,
            "logits": _run_logits}[s["c"]["op"]](s)


def _codes(t):
    return t.view(torch.float8_e4m3fn)


def _run_append(s):
    c = s["c"]
    if own:
        import paged_kv_cache_20_gb300 as pa
        pa.pa_append_kv_block_scaled(s["k_cache"], s["v_cache"], s["kv_scales"], s["k_new"], s["v_new"],
                                     s["table"], s["context_lens"], q_len=c["q_len"])
    else:
        n, u, bs, h, d = c["seqs"], c["q_len"], c["bs"], c["hkv"], c["d"]
        first = s["context_lens"].long() - u                                    # [n]
        lb = first.clamp_min(0)[:, None] // bs + torch.arange((u - 1) // bs + 2, device="cuda")   # [n, t]
        pos = lb[:, :, None] * bs + torch.arange(bs, device="cuda")             # [n, t, bs]
        new = (pos >= first[:, None, None]) & (pos < s["context_lens"][:, None, None])
        i, t = new.any(-1).nonzero(as_tuple=True)                               # touched blocks
        blk = s["table"][i, lb[i, t]].long()
        new, pos = new[i, t], pos[i, t]                                         # [m, bs]
        token = (pos - first[i][:, None]).clamp(0, u - 1) + i[:, None] * u
        older = pos < first[i][:, None]
        for at, (cache, rows) in enumerate((("k_cache", "k_new"), ("v_cache", "v_new"))):
            x = s[rows][token].float().transpose(1, 2)                          # [m, h, bs, d]
            need = _need((x.abs().amax(-1) * new[:, None]).amax(-1))            # [m, h]
            was = s["kv_scales"][blk, :, at].clamp(LEAST, MOST)
            scale = torch.where(older.any(-1)[:, None], torch.maximum(was, need), need)
            codes = s[cache][blk]
            moved = _e4m3(codes.view(torch.float8_e4m3fn).float() * (was / scale)[:, :, None, None])
            fresh = _e4m3(x / scale[:, :, None, None])
            codes = torch.where(new[:, None, :, None], fresh.view(torch.uint8),
                                torch.where(older[:, None, :, None], moved.view(torch.uint8), codes))
            s[cache][blk] = codes
            s["kv_scales"][blk, :, at] = scale
    return {"k_cache": _codes(s["k_cache"]), "v_cache": _codes(s["v_cache"]), "kv_scales": s["kv_scales"]}


def _run_attend(s):
    c = s["c"]
    if own:
        import paged_kv_cache_20_gb300 as pa
        return pa.pa_decode_block_scaled(s["out"], s["q"], s["k_cache"], s["v_cache"], s["kv_scales"], s["table"],
                                         s["context_lens"], s["scale"], q_len=c["q_len"], num_splits=c["splits"],
                                         workspace=s["workspace"])
    n, u, hq, d = s["q"].shape
    t, h = max(s["lens"]), c["hkv"]
    at, lens = torch.arange(t, device="cuda"), s["context_lens"][:, None]
    blk = s["table"][:, at // c["bs"]].clamp_min(0).long()                      # [n, t]

    def rows(name, which):
        x = s[name][blk, :, at % c["bs"]].view(torch.float8_e4m3fn).float()     # [n, t, h, d]
        return x * s["kv_scales"][blk, :, which, None]

    q = s["q"].float().view(n, u, h, hq // h, d)
    k = rows("k_cache", 0)
    x = torch.einsum("nuhgd,nthd->nhgut", q, k) * s["scale"]
    del k
    # query token j sees rows up to len - q_len + j
    sees = at < (lens - u + 1 + torch.arange(u, device="cuda"))[:, :, None]     # [n, u, t]
    x.masked_fill_(~sees[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(top.masked_fill(top == -math.inf, 0)).exp_()
    total = p.sum(-1, keepdim=True)
    p = p.div_(total.masked_fill(total == 0, 1))
    v = rows("v_cache", 1).masked_fill(~(at < lens)[:, :, None, None], 0)
    s["out"].copy_(torch.einsum("nhgut,nthd->nuhgd", p, v).reshape(n, u, hq, d))
    return s["out"]


def _free(table, refs, keep, bs):
    at = torch.arange(table.shape[1], device="cuda")
    gone = (at >= ((keep + bs - 1) // bs)[:, None]) & (table >= 0)
    refs.index_add_(0, table[gone].long(), torch.full_like(table[gone], -1))
    table[gone] = -1


def _run_pages(s):
    c, bs = s["c"], s["c"]["bs"]
    if own:
        import paged_kv_cache_20_gb300 as pa
    if c["kind"] == "turnover":
        if own:
            pa.pa_free_blocks(s["table"], s["refs"], s["keep"], bs)
            pa.pa_reserve_blocks(s["table"], s["refs"], s["want"], bs, missing=s["missing"], workspace=s["workspace"])
        else:
            _free(s["table"], s["refs"], s["keep"], bs)
            at = torch.arange(s["table"].shape[1], device="cuda")
            empty = (at < ((s["want"] + bs - 1) // bs)[:, None]) & (s["table"] < 0)
            i, j = empty.nonzero(as_tuple=True)
            free = (s["refs"] == 0).nonzero()[:i.shape[0], 0]
            i, j = i[:free.shape[0]], j[:free.shape[0]]
            s["table"][i, j] = free.to(torch.int32)
            s["refs"][free] = 1
            s["missing"].copy_(empty.sum() - free.shape[0])
        return {"table": s["table"], "refs": s["refs"], "missing": s["missing"]}
    pairs, counts = s["pairs"], s["counts"]
    if c["kind"] == "fork":
        if own:
            pa.pa_free_blocks(s["table"], s["refs"], s["keep"], bs)
            pa.pa_fork_blocks(s["table"], s["context_lens"], s["refs"], s["src"], s["dst"], bs, src_blocks=pairs[0],
                              dst_blocks=pairs[1], counts=counts, workspace=s["workspace"])
            pa.pa_copy_pages(s["k_cache"], s["v_cache"], pairs[0], pairs[1], counts, kv_scales=s["kv_scales"])
        else:
            _free(s["table"], s["refs"], s["keep"], bs)
            src, dst = s["src"].long(), s["dst"].long()
            lens, rows = s["context_lens"][src], s["table"][src]
            at = torch.arange(rows.shape[1], device="cuda")
            full = at < (lens // bs)[:, None]
            shared = rows[full].long()
            s["refs"].index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
            tail = (lens % bs > 0).nonzero()[:, 0]
            free = (s["refs"] == 0).nonzero()[:tail.shape[0], 0]
            got = tail[:free.shape[0]]
            child = torch.where(full, rows, -1)
            child[got, (lens // bs)[got].long()] = free.to(torch.int32)
            s["refs"][free] = 1
            s["table"][dst] = child
            ok = lens.clone()
            ok[tail[free.shape[0]:]] = lens[tail[free.shape[0]:]] // bs * bs
            s["context_lens"][dst] = ok
            pairs[0, :got.shape[0]] = rows[got, (lens // bs)[got].long()]
            pairs[1, :got.shape[0]] = free.to(torch.int32)
            counts.copy_(torch.tensor([got.shape[0], tail.shape[0] - got.shape[0]], dtype=torch.int32))
            _copy_pages(s, got.shape[0])
        return {"table": s["table"], "context_lens": s["context_lens"], "refs": s["refs"], "pairs": pairs,
                "counts": counts, **_pool_outputs(s)}
    if own:
        pa.pa_compact_blocks(s["table"], s["refs"], block_tables_out=s["table_out"], ref_counts_out=s["refs_out"],
                             src_blocks=pairs[0], dst_blocks=pairs[1], counts=counts, workspace=s["workspace"])
        pa.pa_copy_pages(s["k_cache"], s["v_cache"], pairs[0], pairs[1], counts, kv_scales=s["kv_scales"])
    else:
        used = s["refs"] > 0
        live = int(used.sum())
        frm = used[live:].nonzero()[:, 0] + live
        to = (~used[:live]).nonzero()[:, 0]
        name = torch.arange(c["blocks"], device="cuda", dtype=torch.int32)
        name[frm] = to.to(torch.int32)
        s["table_out"].copy_(torch.where(s["table"] >= 0, name[s["table"].clamp_min(0).long()], s["table"]))
        s["refs_out"].copy_(s["refs"])
        s["refs_out"][to] = s["refs"][frm]
        s["refs_out"][frm] = 0
        n = frm.shape[0]
        pairs[0, :n], pairs[1, :n] = frm.to(torch.int32), to.to(torch.int32)
        counts.copy_(torch.tensor([n, live], dtype=torch.int32))
        _copy_pages(s, n)
    return {"table": s["table_out"], "refs": s["refs_out"], "pairs": pairs, "counts": counts, **_pool_outputs(s)}


def _copy_pages(s, n):
    frm, to = s["pairs"][0, :n].long(), s["pairs"][1, :n].long()
    for name in ("k_cache", "v_cache"):
        # (the cache as 8-byte pieces: elements are moved, not read)
        x = s[name].view(torch.int64)
        x[to] = x[frm]
    if s["kv_scales"] is not None:
        s["kv_scales"][to] = s["kv_scales"][frm]


def _pool_outputs(s):
    if s["kv_scales"] is None:
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return {"k_cache": _codes(s["k_cache"]), "v_cache": _codes(s["v_cache"]), "kv_scales": s["kv_scales"]}


def _run_logits(s):
    c = s["c"]
    if own:
        import paged_kv_cache_20_gb300 as pa
        return pa.pa_adjust_logits(s["out"], s["logits"], history=s["history"], history_lens=s["history_lens"],
                                   prompt_lens=s["prompt_lens"], drafts=s["drafts"], repetition=s["repetition"],
                                   presence=s["presence"], frequency=s["frequency"], bias_ids=s["bias_ids"],
                                   bias_values=s["bias_values"], mask=s["mask"],
                                   temperature=s["temperature"] if c["probs"] else None, probs=c["probs"])
    n, r, v = s["logits"].shape
    at = torch.arange(c["hist"], device="cuda")
    ids = s["history"].long()
    there = at < s["history_lens"][:, None]
    given = there & (at < s["prompt_lens"][:, None])
    prompt = torch.zeros(n, v, device="cuda").scatter_add_(1, ids, given.float()) > 0
    count = torch.zeros(n, v, device="cuda").scatter_add_(1, ids, (there & ~given).float())
    x = s["logits"].float()
    out = torch.empty_like(x)
    for j in range(r):
        if j > 0:
            count.scatter_add_(1, s["drafts"][:, j - 1:j].long(), torch.ones(n, 1, device="cuda"))
        y = x[:, j]
        rep = s["repetition"][:, None]
        y = torch.where(prompt | (count > 0), torch.where(y > 0, y / rep, y * rep), y)
        y = y - (count * s["frequency"][:, None]) - (count > 0) * s["presence"][:, None]
        if s["bias_ids"] is not None:
            for b in range(c["bias"]):  # (in the list's order: one token may have several)
                y = y.scatter_add(1, s["bias_ids"][:, b:b + 1].long(), s["bias_values"][:, b:b + 1])
        out[:, j] = y
    if s["mask"] is not None:
        tok = torch.arange(v, device="cuda")
        out.masked_fill_((s["mask"][:, :, tok // 32] >> (tok % 32).to(torch.int32)) & 1 == 0, -math.inf)
    if not c["probs"]:
        s["out"].copy_(out)
        return s["out"]
    top = out.amax(-1, keepdim=True)
    best = torch.zeros_like(out).scatter_(-1, out.argmax(-1, keepdim=True), 1.0) * (top > -math.inf)
    t = s["temperature"][:, None, None]
    p = out.sub_(top.masked_fill(top == -math.inf, 0)).div_(t.masked_fill(t <= 0, 1)).exp_()
    total = p.sum(-1, keepdim=True)
    s["out"].copy_(torch.where(t > 0, p / total.masked_fill(total == 0, 1), best))
    return s["out"]


# --------------------------------------------------------------------- 64-bit results
def exact(c, seed):
    if c["op"] == "pages":
        return None  # whole numbers, and blocks moved bit for bit: nothing is rounded
    s = prepare(c, seed)
    if c["op"] == "append":
        return _exact_append(s)
    if c["op"] == "attend":
        return _exact_attend(s)
    return _exact_logits(s)


def _exact_append(s):
    """The scales; which codes the rounding picks is the operator's, not an error."""
    c, u, bs = s["c"], s["c"]["q_len"], s["c"]["bs"]
    scales = s["kv_scales"].double()
    for i, n in enumerate(s["lens"]):
        first = max(0, n - u)
        lo = first // bs
        hi = -(-n // bs)
        if hi <= lo:
            continue
        blk = s["table"][i, lo:hi].long()
        for which, rows in enumerate((s["k_new"], s["v_new"])):
            x = rows[i * u + first - (n - u):(i + 1) * u].double().abs().amax(-1)       # [new, h]
            full = torch.zeros((hi - lo) * bs, x.shape[1], dtype=torch.float64, device="cuda")
            full[first - lo * bs:first - lo * bs + x.shape[0]] = x
            top = full.view(hi - lo, bs, -1).amax(1)
            need = torch.exp2(torch.ceil(torch.log2(top.clamp_min(1e-300) / 448)).clamp(-40, 40))
            if first > lo * bs:
                need[0] = torch.maximum(need[0], scales[blk[0], :, which])
            scales[blk, :, which] = need
    return {"k_cache": None, "v_cache": None, "kv_scales": scales}


def _exact_attend(s):
    c = s["c"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    g = c["hq"] // c["hkv"]
    for i, length in enumerate(s["lens"]):
        blocks = s["table"][i, :-(-length // c["bs"])].long()

        def rows(name, which):
            x = s[name][blocks].view(torch.float8_e4m3fn).to(torch.float64)
            x = x * s["kv_scales"][blocks, :, which].double()[:, :, None, None]
            return x.transpose(0, 1).reshape(c["hkv"], -1, c["d"])[:, :length]

        k, v = rows("k_cache", 0), rows("v_cache", 1)
        col = torch.arange(length, device="cuda")
        row = torch.arange(c["q_len"], device="cuda")[:, None]
        for h in range(c["hkv"]):
            for j in range(g):
                x = s["q"][i, :, h * g + j].double() @ k[h].t() * s["scale"]
                x = torch.where(col <= length - c["q_len"] + row, x, -math.inf)
                out[i, :, h * g + j] = torch.softmax(x, -1).nan_to_num(0.0) @ v[h]
    return out


def _exact_logits(s):
    c = s["c"]
    n, r, v = s["logits"].shape
    if n * r * v > 1 << 27:
        return None
    out = torch.empty(n, r, v, dtype=torch.float64, device="cuda")
    for i in range(n):
        h, p = int(s["history_lens"][i]), int(s["prompt_lens"][i])
        seq = s["history"][i, :h].long()
        prompt = torch.bincount(seq[:p], minlength=v)
        rep, pres, freq = (float(s[k][i]) for k in ("repetition", "presence", "frequency"))
        extra = torch.zeros(v, dtype=torch.float64, device="cuda")
        if s["bias_ids"] is not None:
            extra.index_add_(0, s["bias_ids"][i].long(), s["bias_values"][i].double())
        for j in range(r):
            said = seq[p:] if j == 0 else torch.cat((seq[p:], s["drafts"][i, :j].long()))
            count = torch.bincount(said, minlength=v)
            y = s["logits"][i, j].double()
            known = (prompt + count) > 0
            y = torch.where(known & (y > 0), y / rep, torch.where(known, y * rep, y))
            y = y - freq * count - pres * count.clamp_max(1) + extra
            if s["mask"] is not None:
                w = s["mask"][i, j].long() & 0xffffffff
                on = ((w[:, None] >> torch.arange(32, device="cuda")) & 1).flatten()[:v] > 0
                y = torch.where(on, y, -math.inf)
            if c["probs"]:
                t = float(s["temperature"][i])
                if not bool((y > -math.inf).any()):
                    y = torch.zeros_like(y)
                elif t > 0:
                    y = torch.softmax(y / t, -1)
                else:
                    y = torch.nn.functional.one_hot(y.argmax(), v).double()
            out[i, j] = y
    return out
