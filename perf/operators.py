"""Cases for measuring the serving operators around the paged cache: the fused
query/key norm, rotation and cache write; the cache in 8-bit floating point,
written, read back and attended; attention for trees of drafted tokens, and
the move of an accepted path.

``run`` computes a case either with elementary torch operations in 32 bits
(``own`` false) or with this library's calls (``own`` true).
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 16
E4M3_MAX = 448.0
EXP_LO, EXP_HI = -50, 50            # range of a row's scale exponent


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step's tokens of a 64-sequence batch, before attention: the launch counts, not the bytes
        dict(name="norm_rope_decode", op="norm_rope", tokens=64, hq=32, hkv=8, d=128, rot=128, axes=1, norm=True,
             interleaved=False, dtype="bf16", pos_hi=4096),
        # an image-and-text prompt in one pass: three position axes (time, height, width), a ragged token count
        dict(name="norm_rope_prompt_axes", op="norm_rope", tokens=16381, hq=32, hkv=8, d=128, rot=128, axes=3,
             norm=True, interleaved=False, dtype="bf16", pos_hi=131072),
        # a decode step's new tokens of the GQA batch quantised into the cache, and their blocks read back
        dict(name="quantise_decode", op="quantise", seqs=256, new=1, hkv=8, d=128, dtype="bf16"),
        # whole prompts of a 13B-class model quantised as they are written, then read back for prefill
        dict(name="quantise_prompt", op="quantise", seqs=13, new=1261, hkv=40, d=128, dtype="bf16"),
        # four short sequences: the smallest decode step
        dict(name="decode_e4m3_tiny", op="decode", seqs=4, hq=8, hkv=8, d=64, lo=1, hi=64, dist="uniform", lens=1),
        # the GQA serving batch: 256 sequences of ragged lengths around 1000
        dict(name="decode_e4m3_gqa8b", op="decode", seqs=256, hq=32, hkv=8, d=128, lo=32, hi=4096,
             dist="lognormal", lens=2),
        # few sequences with very long contexts
        dict(name="decode_e4m3_long", op="decode", seqs=8, hq=64, hkv=8, d=128, lo=32768, hi=131072,
             dist="uniform", lens=3),
        # four short sequences with a handful of drafts each
        dict(name="tree_tiny", op="tree", seqs=4, hq=8, hkv=8, d=64, lo=1, hi=64, dist="uniform", nlo=1, nhi=8,
             lens=4),
        # a serving batch verifying trees of up to 32 drafted tokens
        dict(name="tree_gqa8b", op="tree", seqs=64, hq=32, hkv=8, d=128, lo=32, hi=4096, dist="lognormal", nlo=9,
             nhi=32, lens=5),
        # long contexts verifying trees of 16 tokens at eight query heads to a cache head
        dict(name="tree_long", op="tree", seqs=8, hq=64, hkv=8, d=128, lo=32768, hi=131072, dist="uniform", nlo=16,
             nhi=16, lens=6),
        # the accepted path of one layer, four sequences
        dict(name="accept_tiny", op="accept", seqs=4, layers=1, hkv=8, d=64, n=8, most=4, dtype="f32"),
        # every layer of the GQA model after a verification step of the whole batch
        dict(name="accept_layers", op="accept", seqs=64, layers=32, hkv=8, d=128, n=33, most=6, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope", "quantise", "decode", "decode", "tree", "tree", "accept"])
    d = rng.choice([64, 128])
    hkv, g = rng.choice([(8, 4), (8, 8), (8, 1), (40, 1), (2, 16), (5, 3), (1, 7), (4, 5)])
    if op == "norm_rope":
        return dict(op=op, tokens=_log_int(rng, 1, 16000 // max(1, hkv * (g + 2) // 48)), hq=hkv * g, hkv=hkv, d=d,
                    rot=rng.choice([d, d, d // 2]), axes=rng.choice([1, 1, 2, 3]), norm=rng.random() < 0.7,
                    interleaved=rng.random() < 0.4, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    pos_hi=_log_int(rng, 64, 1000000))
    if op == "quantise":
        seqs = _log_int(rng, 1, 256)
        return dict(op=op, seqs=seqs, new=_log_int(rng, 1, max(1, 15000 // seqs)), hkv=hkv, d=d,
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op in ("decode", "tree"):
        seqs = _log_int(rng, 1, 256 if op == "decode" else 64)
        # tokens in all are bounded by the largest listed case
        hi = _log_int(rng, 16, max(17, min(131072, (500000 if op == "decode" else 300000) * 8 // (hkv * seqs))))
        c = dict(op=op, seqs=seqs, hq=hkv * g, hkv=hkv, d=d, lo=rng.randint(1, hi), hi=hi, dist="uniform",
                 lens=rng.randrange(1 << 30))
        if op == "tree":
            c["nhi"] = _log_int(rng, 1, max(1, min(96, int(2.5e11 / (4 * d * seqs * hkv * g * (hi + 96))))))
            c["nlo"] = rng.randint(0, c["nhi"])
        return c
    n = _log_int(rng, 1, 64)
    return dict(op=op, seqs=_log_int(rng, 1, 64), layers=rng.randint(1, 32), hkv=hkv if hkv < 40 else 8, d=d, n=n,
                most=rng.randint(1, min(n, 8)), dtype=rng.choice(["bf16", "bf16", "f32"]))


# ---------------------------------------------------------------------------
# sizes that a case fixes whatever the seed
# ---------------------------------------------------------------------------
def _drafts(case):
    """Drafted tokens of every sequence."""
    rng = random.Random(case["lens"] + 1)
    return [case["nhi"]] + [rng.randint(case["nlo"], case["nhi"]) for _ in range(case["seqs"] - 1)]


def _contexts(case):
    """Context lengths; a tree's drafts come on top of the drawn context."""
    rng = random.Random(case["lens"])
    if case["dist"] == "lognormal":
        lens = [min(case["hi"], max(case["lo"], round(rng.lognormvariate(math.log(1000.0), 0.8))))
                for _ in range(case["seqs"])]
    else:
        lens = [rng.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    if case["op"] == "tree":
        lens = [a + b for a, b in zip(lens, _drafts(case))]
    return lens


def work(case):
    if case["op"] == "norm_rope":
        e = 2 if case["dtype"] == "bf16" else 4
        rows = case["hq"] + 2 * case["hkv"]
        per_token = 2 * rows * case["d"] * e + 8 * (case["axes"] + 1)
        flops = (case["hq"] + case["hkv"]) * case["d"] * (7 if case["norm"] else 3)
        return {"bytes": case["tokens"] * per_token, "flops": case["tokens"] * flops}
    if case["op"] == "quantise":
        e = 2 if case["dtype"] == "bf16" else 4
        tok = case["seqs"] * case["new"]
        blocks = sum(-(-case["new"] // BLOCK) for _ in range(case["seqs"]))
        row = 2 * case["hkv"] * case["d"]
        tile = 2 * case["hkv"] * (case["d"] + 1)
        return {"bytes": tok * (row * e + tile) + blocks * BLOCK * (tile + row * 2),
                "flops": 3 * tok * row + blocks * BLOCK * row}
    if case["op"] == "decode":
        tok = sum(_contexts(case))
        return {"bytes": tok * 2 * case["hkv"] * (case["d"] + 1) + 4 * case["seqs"] * case["hq"] * case["d"],
                "flops": 4 * tok * case["hq"] * case["d"]}
    if case["op"] == "tree":
        lens, ns = _contexts(case), _drafts(case)
        tok = sum(a for a, n in zip(lens, ns) if n)
        rows = sum(ns)
        return {"bytes": tok * 4 * case["hkv"] * case["d"] + 4 * rows * case["hq"] * case["d"],
                "flops": sum(4 * a * n for a, n in zip(lens, ns)) * case["hq"] * case["d"]}
    e = 2 if case["dtype"] == "bf16" else 4
    moved = case["seqs"] * max(1, case["most"] // 2)
    return {"bytes": 4 * moved * case["layers"] * case["hkv"] * case["d"] * e, "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _tables(lens, rng):
    """Shuffled physical blocks for sequences of these lengths: tables and pool size."""
    need = [-(-n // BLOCK) for n in lens]
    nb = sum(need) + 2
    perm = rng.permutation(nb)
    tables = np.zeros((len(lens), max(1, max(need))), dtype=np.int32)
    at = 0
    for s, k in enumerate(need):
        tables[s, :k] = perm[at:at + k]
        at += k
    return tables, nb


def _normal(gen, shape, dtype, gain=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * gain).to(dtype)


def _e4m3_pool(gen, nb, hkv, d):
    """A filled cache of e4m3 tiles: 16 rows of d codes, then the rows' 16 scale bytes."""
    cache = torch.empty(nb, hkv, BLOCK * (d + 1), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (hkv * BLOCK * d))
    for lo in range(0, nb, step):
        n = min(step, nb - lo)
        # rows differ in size by a few powers of two
        x = torch.randn(n, hkv, BLOCK, d, generator=gen, device="cuda")
        x = x * torch.exp2(torch.randint(-2, 3, (n, hkv, BLOCK, 1), generator=gen, device="cuda").float() * 0.5)
        m, ex = torch.frexp(x.abs().amax(-1))
        e = (ex - 1 - torch.where(2 * m <= 1.75, 8, 7)).clamp(EXP_LO, EXP_HI)
        code = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        cache[lo:lo + n, :, :BLOCK * d] = code.reshape(n, hkv, BLOCK * d)
        cache[lo:lo + n, :, BLOCK * d:] = (e + 127).to(torch.uint8)
    return cache


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)

    def dev(a, dtype=None):
        t = torch.as_tensor(np.ascontiguousarray(a))
        return (t if dtype is None else t.to(dtype)).cuda()

    op, d, hkv = case["op"], case["d"], case["hkv"]
    st = dict(case=case)
    if op == "norm_rope":
        t, hq, dt = case["tokens"], case["hq"], _DTYPE[case["dtype"]]
        nb = -(-t // BLOCK) + 3
        half = case["rot"] // 2
        freq = 1e6 ** (-np.arange(half) / half)
        pos = rng.integers(0, case["pos_hi"], size=(case["axes"], t))
        return st | dict(
            qkv=_normal(gen, (t, (hq + 2 * hkv) * d), dt),     # the projection's output, q, k and v side by side
            q_weight=_normal(gen, (d,), torch.float32, 0.1).add_(1.0).to(dt),
            k_weight=_normal(gen, (d,), torch.float32, 0.1).add_(1.0).to(dt),
            positions=dev(pos, torch.int64), inv_freq=dev(freq, torch.float32),
            axes=dev(np.arange(half) * case["axes"] // half, torch.int32),
            slots=dev(rng.permutation(nb * BLOCK)[:t], torch.int64),
            q_out=torch.zeros(t, hq, d, dtype=dt, device="cuda"),
            k_cache=torch.zeros(nb, hkv, BLOCK, d, dtype=dt, device="cuda"),
            v_cache=torch.zeros(nb, hkv, BLOCK, d, dtype=dt, device="cuda"))
    if op == "quantise":
        lens = [case["new"]] * case["seqs"]
        tables, nb = _tables(lens, rng)
        t = sum(lens)
        at = np.arange(case["new"])
        slots = (tables[:, at // BLOCK].astype(np.int64) * BLOCK + at % BLOCK).reshape(-1)
        used = tables.reshape(-1)
        scratch = rng.permutation(len(used))
        return st | dict(
            k=_normal(gen, (t, hkv, d), _DTYPE[case["dtype"]]), v=_normal(gen, (t, hkv, d), _DTYPE[case["dtype"]]),
            slots=dev(slots, torch.int64), pairs=dev(np.stack([used, scratch], 1), torch.int64),
            # zeroed tiles with the scale 1, as a fresh cache is
            k_cache=torch.zeros(nb, hkv, BLOCK * (d + 1), dtype=torch.uint8, device="cuda"),
            v_cache=torch.zeros(nb, hkv, BLOCK * (d + 1), dtype=torch.uint8, device="cuda"),
            k_back=torch.zeros(len(used), hkv, BLOCK, d, dtype=torch.bfloat16, device="cuda"),
            v_back=torch.zeros(len(used), hkv, BLOCK, d, dtype=torch.bfloat16, device="cuda"))
    if op in ("decode", "tree"):
        lens = _contexts(case)
        tables, nb = _tables(lens, rng)
        ns = _drafts(case) if op == "tree" else [1] * case["seqs"]
        rows = sum(ns)
        st |= dict(tables=dev(tables), lens=dev(np.array(lens, dtype=np.int32)), max_len=max(lens),
                   q=_normal(gen, (rows, case["hq"], d), torch.bfloat16),
                   out=torch.zeros(rows, case["hq"], d, dtype=torch.bfloat16, device="cuda"),
                   scale=d ** -0.5)
        if op == "decode":
            return st | dict(k_cache=_e4m3_pool(gen, nb, hkv, d), v_cache=_e4m3_pool(gen, nb, hkv, d))
        words = -(-max(1, case["nhi"]) // 64)
        mask = np.zeros((rows, words), dtype=np.uint64)
        start = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
        for s, n in enumerate(ns):
            for i in range(n):                     # node i hangs on an earlier one, seldom far back
                r = start[s] + i
                if i:
                    mask[r] = mask[start[s] + int(rng.integers(max(0, i - 6), i))]
                mask[r, i // 64] |= np.uint64(1 << (i % 64))
        return st | dict(k_cache=_normal(gen, (nb, hkv, BLOCK, d), torch.bfloat16),
                         v_cache=_normal(gen, (nb, hkv, BLOCK, d), torch.bfloat16),
                         starts=dev(start), mask=dev(mask.view(np.int64)), nmax=max(1, max(ns)))
    # accept
    n, most, seqs = case["n"], case["most"], case["seqs"]
    lens = [n + 1 + (17 * s) % 80 for s in range(seqs)]
    tables, nb = _tables(lens, rng)
    # a path keeps node 0 and goes down through nodes behind the accepted positions
    paths = np.zeros((seqs, most), dtype=np.int32)
    count = rng.integers(1, most + 1, size=seqs).astype(np.int32)
    for s in range(seqs):
        a = int(count[s])
        tail = np.sort(rng.choice(np.arange(a, n), size=min(a - 1, n - a), replace=False)) if n > a else []
        count[s] = 1 + len(tail)
        paths[s, 1:1 + len(tail)] = tail
    k_all = _normal(gen, (case["layers"], nb, hkv, BLOCK, d), _DTYPE[case["dtype"]])
    v_all = _normal(gen, (case["layers"], nb, hkv, BLOCK, d), _DTYPE[case["dtype"]])
    return st | dict(tables=dev(tables), lens=dev(np.array(lens, dtype=np.int32)),
                     starts=dev(np.arange(seqs + 1, dtype=np.int32) * n), paths=dev(paths), count=dev(count),
                     new_lens=torch.zeros(seqs, dtype=torch.int32, device="cuda"),
                     k_all=k_all, v_all=v_all, k_caches=list(k_all.unbind(0)), v_caches=list(v_all.unbind(0)))


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_norm_rope(st):
    case = st["case"]
    t, hq, hkv, d, half = case["tokens"], case["hq"], case["hkv"], case["d"], case["rot"] // 2
    x = st["qkv"].view(t, hq + 2 * hkv, d)
    angle = st["positions"].double()[st["axes"].long()] * st["inv_freq"].double()[:, None]      # [half, t]
    cos, sin = angle.cos().float().t()[:, None], angle.sin().float().t()[:, None]               # [t, 1, half]

    def turned(rows, weight):
        y = rows.float()
        if case["norm"]:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
        r, rest = y[..., :2 * half], y[..., 2 * half:]
        if case["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = r[..., :half], r[..., half:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([r, rest], -1).to(rows.dtype)

    blk, off = st["slots"] // BLOCK, st["slots"] % BLOCK
    st["k_cache"][blk, :, off] = turned(x[:, hq:hq + hkv], st["k_weight"])
    st["v_cache"][blk, :, off] = x[:, hq + hkv:]
    return turned(x[:, :hq], st["q_weight"])


def _plain_codes(x):
    """e4m3 codes and scale bytes of the rows of x."""
    x = x.float()
    m, ex = torch.frexp(x.abs().amax(-1))
    e = ex - 1 - torch.where(2 * m <= 1.75, 8, 7)
    e = torch.where(m == 0, 0, e).clamp(EXP_LO, EXP_HI)
    y = torch.ldexp(x, -e[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
    return y.to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def _plain_values(tiles, d):
    """The values that e4m3 tiles [..., 16 (d + 1)] stand for, [..., 16, d] in fp32."""
    codes = tiles[..., :BLOCK * d].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (BLOCK, d))
    return torch.ldexp(codes, tiles[..., BLOCK * d:].int()[..., None] - 127)


def _plain_quantise(st):
    d = st["case"]["d"]
    blk, off = st["slots"] // BLOCK, st["slots"] % BLOCK

    def through(rows, cache, back):
        codes, scales = _plain_codes(rows)
        cache[:, :, :BLOCK * d].unflatten(-1, (BLOCK, d))[blk, :, off] = codes
        cache[:, :, BLOCK * d:][blk, :, off] = scales
        src, dst = st["pairs"].unbind(1)
        back[dst] = _plain_values(cache[src], d).to(back.dtype)

    through(st["k"], st["k_cache"], st["k_back"])
    through(st["v"], st["v_cache"], st["v_back"])


def _gathered(st, cache):
    """Every sequence's rows in order, padded to the longest: [S, L, Hkv, d] in fp32, zeros past the end."""
    at = torch.arange(st["max_len"], device="cuda")
    live = at[None] < st["lens"][:, None]
    blk = torch.where(live, st["tables"].long()[:, at // BLOCK], 0)
    if cache.dtype == torch.uint8:
        d = st["case"]["d"]
        codes = cache[:, :, :BLOCK * d].unflatten(-1, (BLOCK, d))[blk, :, at % BLOCK]
        e = cache[:, :, BLOCK * d:][blk, :, at % BLOCK].int() - 127
        x = torch.ldexp(codes.view(torch.float8_e4m3fn).float(), e[..., None])
    else:
        x = cache[blk, :, at % BLOCK].float()
    return torch.where(live[:, :, None, None], x, 0.0), live


def _plain_attention(st):
    case = st["case"]
    seqs, hq, hkv, d = case["seqs"], case["hq"], case["hkv"], case["d"]
    k, live = _gathered(st, st["k_cache"])
    v, _ = _gathered(st, st["v_cache"])
    if case["op"] == "decode":
        n, row = 1, torch.arange(seqs, device="cuda")
        q = st["q"].float()[:, None]
        see = live[:, None]
    else:
        n, starts = st["nmax"], st["starts"].long()
        i = torch.arange(n, device="cuda")
        mine = i[None] < (starts[1:] - starts[:-1])[:, None]                                     # [S, n]
        rows = torch.where(mine, starts[:-1, None] + i[None], 0)
        row = torch.nonzero(mine.reshape(-1))[:, 0]
        q = st["q"].float()[rows]                                                                # [S, n, Hq, d]
        # position p of a sequence is draft p - base; earlier positions are seen by every row
        base = st["lens"].long() - (starts[1:] - starts[:-1])
        j = torch.arange(st["max_len"], device="cuda")[None] - base[:, None]                     # [S, L]
        word = (j.clamp(0, n - 1) // 64)[:, None].expand(-1, n, -1)
        bit = (st["mask"][rows].gather(2, word) >> (j.clamp(0, n - 1) % 64)[:, None]) & 1
        see = ((j < 0)[:, None] | (bit != 0)) & live[:, None]                                    # [S, n, L]
    q = q.view(seqs, n, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(seqs, hkv, n * (hq // hkv), d)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(st["scale"])
    s = s.masked_fill_(~see.repeat_interleave(hq // hkv, 1)[:, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, 1.0)
    o = o.view(seqs, hkv, n, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(seqs * n, hq, d)
    return o[row].to(torch.bfloat16)


def _plain_accept(st):
    seqs, most = st["paths"].shape
    base = st["lens"] - (st["starts"][1:] - st["starts"][:-1])
    j = torch.arange(most, device="cuda")
    take = j[None] < st["count"][:, None]
    s = torch.nonzero(take)[:, 0]
    src = (base[:, None] + st["paths"])[take].long()
    dst = (base[:, None] + j[None])[take].long()
    sb, db = st["tables"].long()[s, src // BLOCK], st["tables"].long()[s, dst // BLOCK]

    for cache in (st["k_all"], st["v_all"]):
        cache[:, db, :, dst % BLOCK] = cache[:, sb, :, src % BLOCK]
    st["new_lens"].copy_(base + st["count"])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    case = state["case"]
    op, d, hkv = case["op"], case["d"], case["hkv"]
    if own:
        from paged_kv_cache_177_gb300 import binding as B
    if op == "norm_rope":
        if own:
            t, hq = case["tokens"], case["hq"]
            q, k, v = state["qkv"].view(t, hq + 2 * hkv, d).split([hq, hkv, hkv], 1)
            weights = dict(q_weight=state["q_weight"], k_weight=state["k_weight"], eps=1e-6) if case["norm"] else {}
            q_out = B.qk_norm_rope_append(state["q_out"], q, k, v, state["positions"], state["inv_freq"],
                                          state["slots"], state["k_cache"], state["v_cache"], axes=state["axes"],
                                          interleaved=case["interleaved"], **weights)
        else:
            q_out = _plain_norm_rope(state)
        return q_out, state["k_cache"], state["v_cache"]
    if op == "quantise":
        if own:
            B.kv_append_e4m3(state["k"], state["v"], state["slots"], state["k_cache"], state["v_cache"])
            B.dequantize_blocks(state["k_back"], state["v_back"], state["k_cache"], state["v_cache"], state["pairs"],
                                check=False)
        else:
            _plain_quantise(state)
        return state["k_back"], state["v_back"]
    if op == "decode":
        if own:
            if "workspace" not in state:           # kept by the program for all its steps
                need = B.e4m3_workspace_bytes(case["seqs"], case["hq"], hkv, d, state["max_len"])
                state["workspace"] = torch.zeros(max(16, need), dtype=torch.uint8, device="cuda")
            return B.paged_decode_attention_e4m3(state["out"], state["q"], state["k_cache"], state["v_cache"],
                                                 state["tables"], state["lens"], state["scale"],
                                                 max_context_len=state["max_len"], workspace=state["workspace"])
        return _plain_attention(state)
    if op == "tree":
        if own:
            if "workspace" not in state:
                need = B.tree_workspace_bytes(case["seqs"], case["hq"], hkv, d, state["nmax"], state["max_len"])
                state["workspace"] = torch.zeros(max(16, need), dtype=torch.uint8, device="cuda")
            return B.paged_tree_attention(state["out"], state["q"], state["k_cache"], state["v_cache"],
                                          state["tables"], state["lens"], state["starts"], state["mask"],
                                          state["scale"], max_query_len=state["nmax"],
                                          max_context_len=state["max_len"], workspace=state["workspace"])
        return _plain_attention(state)
    if own:
        if "ptrs" not in state:                    # the layers' pointers, laid out once
            state["ptrs"] = (B.layer_pointers(state["k_caches"]), B.layer_pointers(state["v_caches"]))
        B.kv_accept_layers(state["k_caches"], state["v_caches"], state["tables"], state["lens"], state["starts"],
                           state["paths"], state["count"], state["new_lens"], ptrs=state["ptrs"])
    else:
        _plain_accept(state)
    return state["k_all"], state["v_all"], state["new_lens"]


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    op, d, hkv = case["op"], case["d"], case["hkv"]
    if op == "norm_rope":
        t, hq, half = case["tokens"], case["hq"], case["rot"] // 2
        x = st["qkv"].double().view(t, -1, d)
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        if case["norm"]:
            q = q / ((q * q).sum(-1, keepdim=True) / d + 1e-6).sqrt() * st["q_weight"].double()
            k = k / ((k * k).sum(-1, keepdim=True) / d + 1e-6).sqrt() * st["k_weight"].double()
        lead = torch.arange(half, device="cuda")
        first, second = (2 * lead, 2 * lead + 1) if case["interleaved"] else (lead, lead + half)
        theta = torch.stack([st["positions"][a].double() * f for a, f in
                             zip(st["axes"].tolist(), st["inv_freq"].double().tolist())], 1)[:, None]
        out = []
        for y in (q, k):
            z = torch.view_as_complex(torch.stack([y[..., first], y[..., second]], -1))
            z = torch.view_as_real(z * torch.polar(torch.ones_like(theta), theta))
            y = y.clone()
            y[..., first], y[..., second] = z[..., 0], z[..., 1]
            out.append(y)
        flat = torch.zeros(st["k_cache"].shape[0] * BLOCK, hkv, d, dtype=torch.float64, device="cuda")
        vflat = flat.clone()
        flat[st["slots"]], vflat[st["slots"]] = out[1], v
        kc = flat.view(-1, BLOCK, hkv, d).transpose(1, 2).contiguous()
        vc = vflat.view(-1, BLOCK, hkv, d).transpose(1, 2).contiguous()
        return out[0], kc, vc
    if op == "quantise":
        # the nearest of the finite codes' values, by search, ties to the even code
        codes = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
        mid = (codes[1:] + codes[:-1]) / 2

        def stand_for(x):
            x = x.double()
            top = x.abs().amax(-1, keepdim=True)
            e = torch.ceil(torch.log2(top / 448))
            e = torch.where(top > 448 * torch.exp2(e), e + 1, torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e))
            e = torch.where(top == 0, 0.0, e).clamp(EXP_LO, EXP_HI)
            y = x.abs() * torch.exp2(-e)
            lo = torch.searchsorted(mid, y, right=False)
            hi = torch.searchsorted(mid, y, right=True)
            pick = torch.where(lo % 2 == 0, lo, hi)
            return torch.sign(x) * codes[pick] * torch.exp2(e)

        src, dst = st["pairs"].unbind(1)
        back = []
        for rows in (st["k"], st["v"]):
            flat = torch.zeros(st["k_cache"].shape[0] * BLOCK, hkv, d, dtype=torch.float64, device="cuda")
            flat[st["slots"]] = torch.cat([stand_for(r) for r in rows.split(4096)])
            res = torch.zeros(st["k_back"].shape, dtype=torch.float64, device="cuda")
            res[dst] = flat.view(-1, BLOCK, hkv, d).transpose(1, 2)[src]
            back.append(res)
        return tuple(back)
    if op in ("decode", "tree"):
        starts = st["starts"].tolist() if op == "tree" else list(range(case["seqs"] + 1))
        g = case["hq"] // hkv
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        for s, length in enumerate(st["lens"].tolist()):
            n = starts[s + 1] - starts[s]
            if n == 0 or length == 0:
                continue
            rows = slice(starts[s], starts[s + 1])
            blocks = st["tables"][s, :-(-length // BLOCK)].long()
            see = torch.ones(n, length, dtype=torch.bool, device="cuda")
            if op == "tree":
                words = st["mask"][rows].cpu().numpy().view(np.uint64)
                bits = np.unpackbits(words.view(np.uint8), axis=1, bitorder="little")[:, :n]
                see[:, length - n:] = torch.from_numpy(bits.astype(bool)).cuda()
            for h in range(hkv):
                kv = []
                for cache in (st["k_cache"], st["v_cache"]):
                    tile = cache[blocks, h]
                    if op == "decode":
                        c = tile[:, :BLOCK * d].contiguous().view(torch.float8_e4m3fn).double().view(-1, BLOCK, d)
                        tile = c * torch.exp2(tile[:, BLOCK * d:].double() - 127)[..., None]
                    kv.append(tile.double().reshape(-1, d)[:length])
                qh = st["q"][rows, h * g:(h + 1) * g].double()
                w = torch.softmax((qh @ kv[0].T * st["scale"]).masked_fill(~see[:, None], -math.inf), -1)
                out[rows, h * g:(h + 1) * g] = torch.nan_to_num(w) @ kv[1]
        return out
    return None
