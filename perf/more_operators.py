"""Cases for measuring the operators around a model whose attention scores are
transformed (capped by a tanh, biased by distance, cut to a window, with a
prefix seen from both sides), a batch that shares a long prefix, and the
verification of drafted tokens from given random numbers.

``run`` computes a case either with elementary torch operations (``own``
false: 32 bits, and 64 where a random number is held against a sum) or with
this library's calls (``own`` true).
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 16


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # four short sequences in fp32: the smallest decode step, where the launch counts
        dict(name="scored_decode_tiny", op="decode", seqs=4, hq=8, hkv=8, d=64, dtype="f32", lo=1, hi=64,
             dist="uniform", lens=1, cap=30.0, window=0, alibi=True, gain=4.0),
        # a decode step of a GQA model that caps its scores: 256 sequences of ragged lengths around 1000
        dict(name="scored_decode_capped", op="decode", seqs=256, hq=32, hkv=8, d=128, dtype="bf16", lo=32, hi=4096,
             dist="lognormal", lens=2, cap=50.0, window=0, alibi=False, gain=4.0),
        # a decode step of a layer that sees the last 4096 tokens of longer contexts
        dict(name="scored_decode_window", op="decode", seqs=64, hq=32, hkv=8, d=128, dtype="bf16", lo=2048, hi=16384,
             dist="uniform", lens=3, cap=50.0, window=4096, alibi=False, gain=4.0),
        # a decode step of a 13B-class model whose scores fall off with distance
        dict(name="scored_decode_alibi", op="decode", seqs=64, hq=40, hkv=40, d=128, dtype="bf16", lo=16, hi=2048,
             dist="lognormal", lens=4, cap=0.0, window=0, alibi=True, gain=1.0),
        # four short prompts whose beginning is seen from both sides
        dict(name="scored_prefill_tiny", op="prefill", seqs=4, hq=8, hkv=8, d=64, lo=1, hi=64, nlo=1, nhi=64,
             whole=True, lens=5, cap=30.0, window=0, alibi=True, prefix=True, gain=4.0),
        # whole prompts of ragged lengths through a layer with a window and capped scores
        dict(name="scored_prefill_prompts", op="prefill", seqs=32, hq=32, hkv=8, d=128, lo=64, hi=2048, nlo=64,
             nhi=2048, whole=True, lens=6, cap=50.0, window=1024, alibi=False, prefix=False, gain=4.0),
        # chunks of long prompts after tens of thousands of cached tokens, capped scores
        dict(name="scored_prefill_chunks", op="prefill", seqs=8, hq=32, hkv=8, d=128, lo=16384, hi=32768, nlo=512,
             nhi=512, whole=False, lens=7, cap=50.0, window=0, alibi=False, prefix=False, gain=4.0),
        # eight requests under a system prompt of 256 tokens
        dict(name="common_prefix_small", op="common", seqs=8, hq=8, hkv=8, d=64, groups=1, shared=256, lo=1, hi=64,
             lens=8),
        # a serving batch under one long system prompt: 128 requests, 16K shared tokens, a few hundred own each
        dict(name="common_prefix_system", op="common", seqs=128, hq=32, hkv=8, d=128, groups=1, shared=16384, lo=16,
             hi=1024, lens=9),
        # four sequences with chains of up to four drafts from a draft model
        dict(name="verify_tiny", op="verify", seqs=4, vocab=32003, nlo=2, nhi=5, tree=False, draft=True, lens=10,
             dtype="f32"),
        # a batch verifying trees that a draft model filled, several samples to a node
        dict(name="verify_trees", op="verify", seqs=64, vocab=131072, nlo=9, nhi=32, tree=True, draft=True, lens=11,
             dtype="f32"),
        # a large batch verifying chains that were looked up, with no draft probabilities
        dict(name="verify_lookup", op="verify", seqs=256, vocab=131072, nlo=2, nhi=6, tree=False, draft=False,
             lens=12, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "prefill", "prefill", "prefill", "common", "common", "verify",
                     "verify"])
    d = rng.choice([64, 128])
    hkv, g = rng.choice([(8, 4), (8, 8), (8, 1), (40, 1), (2, 16), (5, 3), (1, 7), (4, 5)])
    seed = rng.randrange(1 << 30)
    scores = dict(cap=rng.choice([0.0, 5.0, 30.0, 50.0]), alibi=rng.random() < 0.5,
                  window=rng.choice([0, 0, 1, _log_int(rng, 2, 8192)]), gain=rng.choice([1.0, 4.0]))
    if op == "decode":
        seqs = _log_int(rng, 1, 256)
        hi = _log_int(rng, 16, max(17, min(65536, 250000 * 8 // (hkv * seqs))))
        return dict(op=op, seqs=seqs, hq=hkv * g, hkv=hkv, d=d, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    lo=rng.randint(1, hi), hi=hi, dist="uniform", lens=seed, **scores)
    if op == "prefill":
        seqs = _log_int(rng, 1, 32)
        # (new tokens times context) times heads is bounded by the largest listed case
        hi = _log_int(rng, 16, 16384)
        nhi = _log_int(rng, 1, max(1, min(hi, 2048, int(8 * 512 * 32 * 24000 / (seqs * hkv * g * hi)))))
        return dict(op=op, seqs=seqs, hq=hkv * g, hkv=hkv, d=d, lo=rng.randint(nhi, hi), hi=hi, nlo=rng.randint(0, nhi),
                    nhi=nhi, whole=False, lens=seed, prefix=rng.random() < 0.5, **scores)
    if op == "common":
        seqs = _log_int(rng, 1, 128)
        tokens = 130 * 17000 * 8 // (hkv * seqs)           # a sequence's, of the largest listed case's in all
        shared = BLOCK * _log_int(rng, 1, max(1, min(1024, tokens // (2 * BLOCK))))
        hi = _log_int(rng, 1, max(2, min(8192, tokens // 2, 60000 * 8 // (hkv * seqs))))
        return dict(op=op, seqs=seqs, hq=hkv * g, hkv=hkv, d=d, groups=rng.choice([1, 1, min(2, seqs), min(5, seqs)]),
                    shared=shared, lo=rng.randint(1, hi), hi=hi, lens=seed)
    tree = rng.random() < 0.5
    seqs = _log_int(rng, 1, 64)
    nhi = _log_int(rng, 1, 32)
    return dict(op=op, seqs=seqs, vocab=_log_int(rng, 100, max(200, min(200000, 64 * 32 * 131072 // (seqs * nhi)))),
                nlo=rng.randint(0, nhi), nhi=nhi, tree=tree, draft=rng.random() < 0.5, lens=seed,
                dtype=rng.choice(["f32", "f32", "bf16"]))


# ---------------------------------------------------------------------------
# sizes that a case fixes whatever the seed
# ---------------------------------------------------------------------------
def _rows(case):
    """New tokens (prefill) or drafts (verify) of every sequence."""
    rng = random.Random(case["lens"] + 1)
    if case["op"] == "prefill" and case["whole"]:
        return _contexts(case)
    return [case["nhi"]] + [rng.randint(case["nlo"], case["nhi"]) for _ in range(case["seqs"] - 1)]


def _contexts(case):
    rng = random.Random(case["lens"])
    if case.get("dist") == "lognormal":
        middle = 1000.0 if case["hkv"] < 40 else 400.0
        return [min(case["hi"], max(case["lo"], round(rng.lognormvariate(math.log(middle), 0.8))))
                for _ in range(case["seqs"])]
    lens = [rng.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    return [case["shared"] + n for n in lens] if case["op"] == "common" else lens


def _prefixes(case):
    """Tokens at the beginning of every prompt that are seen from both sides."""
    rng = random.Random(case["lens"] + 2)
    return [rng.randint(0, n) if case["prefix"] else 0 for n in _contexts(case)]


def _groups(case):
    """First sequence of every group, and the end."""
    return [case["seqs"] * i // case["groups"] for i in range(case["groups"] + 1)]


def _seen(case):
    """Prefill: (query, key) pairs that are visible, and keys that any query of their sequence sees."""
    pairs = keys = 0
    window = case["window"] or 1 << 30
    for length, n, pre in zip(_contexts(case), _rows(case), _prefixes(case)):
        if n == 0:
            continue
        pos = np.arange(length - n, length, dtype=np.int64)
        lo = np.maximum(0, pos - window + 1)
        hi = np.minimum(np.maximum(pos, pre - 1), pos + window - 1)
        pairs += int((hi - lo + 1).sum())
        keys += int(hi.max() - lo.min() + 1)
    return pairs, keys


def work(case):
    if case["op"] == "verify":
        e = 2 if case["dtype"] == "bf16" else 4
        # the next token of a sequence comes from one row of the target, less one row of the draft
        rows = case["seqs"] * (2 if case["draft"] else 1)
        return {"bytes": rows * case["vocab"] * e + sum(_rows(case)) * 24, "flops": 2 * rows * case["vocab"]}
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    if case["op"] == "decode":
        e = 2 if case["dtype"] == "bf16" else 4
        tok = sum(min(n, case["window"] or n) for n in _contexts(case))
        return {"bytes": tok * 2 * hkv * d * e + 2 * case["seqs"] * hq * d * e, "flops": 4 * tok * hq * d}
    if case["op"] == "prefill":
        pairs, keys = _seen(case)
        return {"bytes": keys * 4 * hkv * d + 4 * sum(_rows(case)) * hq * d, "flops": 4 * pairs * hq * d}
    lens = _contexts(case)
    own_tokens = sum(lens) - case["seqs"] * case["shared"]
    return {"bytes": (own_tokens + case["groups"] * case["shared"]) * 4 * hkv * d + 4 * case["seqs"] * hq * d,
            "flops": 4 * sum(lens) * hq * d}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _tables(lens, rng, shared=0, groups=None):
    """Shuffled physical blocks for sequences of these lengths, the first ``shared`` of a group's the same ones."""
    need = [-(-n // BLOCK) for n in lens]
    of_group = np.zeros(len(lens), dtype=np.int64)
    for z in range(len(groups) - 1 if groups else 0):
        of_group[groups[z]:groups[z + 1]] = z
    common = shared * (len(groups) - 1 if groups else 0)
    nb = common + sum(n - shared for n in need) + 2
    perm = rng.permutation(nb)
    tables = np.zeros((len(lens), max(1, max(need))), dtype=np.int32)
    at = common
    for s, n in enumerate(need):
        tables[s, :shared] = perm[of_group[s] * shared:(of_group[s] + 1) * shared]
        tables[s, shared:n] = perm[at:at + n - shared]
        at += n - shared
    return tables, nb


def _normal(gen, shape, dtype, gain=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * gain).to(dtype)


def _pool(gen, nb, hkv, d, dtype):
    cache = torch.empty(nb, hkv, BLOCK, d, dtype=dtype, device="cuda")
    step = max(1, (1 << 28) // (hkv * BLOCK * d))
    for lo in range(0, nb, step):
        cache[lo:lo + step] = _normal(gen, cache[lo:lo + step].shape, dtype)
    return cache


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)

    def dev(a, dtype=None):
        t = torch.as_tensor(np.ascontiguousarray(a))
        return (t if dtype is None else t.to(dtype)).cuda()

    op, seqs = case["op"], case["seqs"]
    st = dict(case=case)
    if op == "verify":
        ns, v = _rows(case), case["vocab"]
        total = sum(ns)
        start = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
        parents = np.full(total, -1, dtype=np.int32)
        for s, n in enumerate(ns):                  # row 0 is the last token that was chosen; drafts hang below it
            for i in range(1, n):
                parents[start[s] + i] = int(rng.integers(max(0, i - 3), i)) if case["tree"] else i - 1
        dt = _DTYPE[case["dtype"]]
        target = torch.empty(total, v, dtype=dt, device="cuda")
        draft = torch.empty(total, v, dtype=dt, device="cuda") if case["draft"] else None
        guess = torch.zeros(total, 8, dtype=torch.int64, device="cuda")    # samples of each row's draft distribution
        for lo in range(0, total, 256):
            logits = torch.randn(min(256, total - lo), v, generator=gen, device="cuda") * 3.0
            target[lo:lo + 256] = torch.softmax(logits, -1)
            near = torch.softmax(logits + 0.7 * torch.randn(logits.shape, generator=gen, device="cuda"), -1).to(dt)
            if draft is not None:
                draft[lo:lo + 256] = near
            guess[lo:lo + 256] = torch.multinomial(near.float(), 8, replacement=True, generator=gen)
        rows = np.arange(total)
        parent_row = np.where(parents >= 0, np.repeat(start[:-1], ns) + parents, rows)
        tokens = guess.cpu().numpy()[parent_row, rng.integers(0, 8, size=total)]
        return st | dict(
            tokens=dev(tokens), parents=dev(parents), starts=dev(start), target=target, draft=draft,
            uniforms=torch.rand(total, generator=gen, device="cuda"),
            final=torch.rand(seqs, generator=gen, device="cuda"), nmax=max(1, max(ns)),
            accepted=torch.zeros(seqs, max(1, max(ns)), dtype=torch.int32, device="cuda"),
            count=torch.zeros(seqs, dtype=torch.int32, device="cuda"),
            chosen=torch.zeros(seqs, dtype=torch.int64, device="cuda"))
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    lens = _contexts(case)
    dt = _DTYPE[case.get("dtype", "bf16")]
    groups = _groups(case) if op == "common" else None
    tables, nb = _tables(lens, rng, case["shared"] // BLOCK if groups else 0, groups)
    ns = _rows(case) if op == "prefill" else [1] * seqs
    st |= dict(tables=dev(tables), lens=dev(np.array(lens, dtype=np.int32)), max_len=max(lens), scale=d ** -0.5,
               q=_normal(gen, (sum(ns), hq, d), dt, case.get("gain", 1.0)),
               out=torch.zeros(sum(ns), hq, d, dtype=dt, device="cuda"),
               k_cache=_pool(gen, nb, hkv, d, dt), v_cache=_pool(gen, nb, hkv, d, dt), slopes=None, prefixes=None)
    if case.get("alibi"):
        st["slopes"] = dev(2.0 ** (-8.0 * np.arange(1, hq + 1) / hq), torch.float32)
    if op == "prefill":
        st |= dict(starts=dev(np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)), nmax=max(1, max(ns)),
                   ns=ns, host_lens=lens)
        if case["prefix"]:
            st["prefixes"] = dev(np.array(_prefixes(case), dtype=np.int32))
    if op == "common":
        st |= dict(starts=dev(np.array(groups, dtype=np.int32)), group_max=max(np.diff(groups)),
                   shared=dev(np.full(case["groups"], case["shared"] // BLOCK, dtype=np.int32)))
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_scores(case, raw, distance, slopes):
    """Scores [..., Hq-major rows, keys] from scaled products, in place where it can be."""
    if case.get("cap"):
        raw = raw.div_(case["cap"]).tanh_().mul_(case["cap"])
    if slopes is not None:
        raw = raw.sub_(slopes * distance)
    return raw


def _plain_decode(st):
    """Every sequence's visible keys side by side, padded to the most."""
    case = st["case"]
    seqs, hq, hkv, d = case["seqs"], case["hq"], case["hkv"], case["d"]
    window = case.get("window") or st["max_len"]
    span = min(window, st["max_len"])
    first = (st["lens"].long() - span).clamp(min=0)
    at = first[:, None] + torch.arange(span, device="cuda")
    live = at < st["lens"][:, None]
    blk = torch.where(live, st["tables"].long().gather(1, (at // BLOCK).clamp(max=st["tables"].shape[1] - 1)), 0)

    def rows(cache):
        return torch.where(live[:, :, None, None], cache[blk, :, at % BLOCK].float(), 0.0)

    q = st["q"].float().view(seqs, hkv, hq // hkv, d)
    s = torch.matmul(q, rows(st["k_cache"]).permute(0, 2, 3, 1)).mul_(st["scale"])
    slopes = None if st["slopes"] is None else st["slopes"].view(1, hkv, -1, 1)
    s = _plain_scores(case, s, (st["lens"][:, None] - 1 - at).float()[:, None, None], slopes)
    s = s.masked_fill_(~live[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    o = torch.matmul(p, rows(st["v_cache"]).permute(0, 2, 1, 3)) / p.sum(-1, keepdim=True)
    return o.reshape(seqs, hq, d).to(st["q"].dtype)


def _plain_prefill(st):
    case = st["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    out = torch.zeros_like(st["q"])
    row = 0
    for s, (n, length) in enumerate(zip(st["ns"], st["host_lens"])):
        if n == 0:
            continue
        blocks = st["tables"][s, :-(-length // BLOCK)].long()
        k, v = (c[blocks].transpose(0, 1).reshape(hkv, -1, d)[:, :length].float()
                for c in (st["k_cache"], st["v_cache"]))
        pos = torch.arange(length - n, length, device="cuda")[:, None]
        key = torch.arange(length, device="cuda")[None]
        see = key <= pos
        if st["prefixes"] is not None:
            see = see | (key < st["prefixes"][s])
        if case["window"]:
            see = see & ((pos - key).abs() < case["window"])
        q = st["q"][row:row + n].float().view(n, hkv, -1, d).permute(1, 2, 0, 3)                 # [Hkv, g, n, d]
        step = max(1, (1 << 28) // (hq * length))
        for lo in range(0, n, step):
            w = torch.matmul(q[:, :, lo:lo + step], k[:, None].transpose(-1, -2)).mul_(st["scale"])
            slopes = None if st["slopes"] is None else st["slopes"].view(hkv, -1, 1, 1)
            w = _plain_scores(case, w, (pos[lo:lo + step] - key).abs().float(), slopes)
            w = w.masked_fill_(~see[lo:lo + step], -math.inf)
            w = w.sub_(w.amax(-1, keepdim=True)).exp_()
            o = torch.matmul(w, v[:, None]) / w.sum(-1, keepdim=True)
            out[row + lo:row + min(n, lo + step)] = o.permute(2, 0, 1, 3).reshape(-1, hq, d).to(out.dtype)
        row += n
    return out


def _plain_verify(st):
    case = st["case"]
    seqs, most = st["accepted"].shape
    start = st["starts"].long()
    n = start[1:] - start[:-1]
    s = torch.arange(seqs, device="cuda")
    last = max(0, st["tokens"].shape[0] - 1)
    node = torch.zeros_like(n)                                   # the accepted draft that the walk stands at
    count = (n > 0).long()
    path = torch.where(n[:, None] > 0, 0, -1).repeat(1, most)
    path[:, 1:] = -1
    left = st["target"][start[:-1].clamp(max=last)].double()     # what the walk may still draw there, ...
    mass = torch.ones(seqs, dtype=torch.float64, device="cuda")  # ... its sum (one, as long as nothing was refused)
    for i in range(1, st["nmax"]):
        row = (start[:-1] + i).clamp(max=last)
        there = (i < n) & (st["parents"][row] == node)
        token = st["tokens"][row]
        have = left[s, token]
        at = (start[:-1] + node).clamp(max=last)
        bar = st["uniforms"][row].double() * mass
        if st["draft"] is not None:
            bar = bar * st["draft"][at, token].double()
        yes, no = there & (bar < have), there & ~(bar < have)
        if st["draft"] is not None:
            less = torch.clamp(left - mass[:, None] * st["draft"][at].double(), min=0.0)
        else:
            less = left.scatter(1, token[:, None], 0.0)
        less = torch.where(no[:, None], less, left)
        total = less.sum(-1)
        no = no & (total > 0)                                    # (nothing left: what was there stands)
        left = torch.where(no[:, None], less, left)
        mass = torch.where(no, total, mass)
        node = torch.where(yes, i, node)
        path[s, count.clamp(max=most - 1)] = torch.where(yes, i, path[s, count.clamp(max=most - 1)])
        count = count + yes
        left = torch.where(yes[:, None], st["target"][row].double(), left)
        mass = torch.where(yes, 1.0, mass)
    grown = left.cumsum(-1)
    pick = (grown <= st["final"].double()[:, None] * grown[:, -1:]).sum(-1)
    st["accepted"].copy_(path)
    st["count"].copy_(count)
    st["chosen"].copy_(torch.where(n > 0, pick, -1))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _workspace(state, need):
    """Scratch that a program keeps for all its steps."""
    if "workspace" not in state:
        state["workspace"] = torch.zeros(max(16, need), dtype=torch.uint8, device="cuda")
    return state["workspace"]


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        from paged_kv_cache_177_gb300 import binding as B
    if op == "verify":
        if own:
            B.verify_drafts(state["accepted"], state["count"], state["chosen"], state["tokens"], state["parents"],
                            state["starts"], state["target"], state["uniforms"], state["final"],
                            draft_probs=state["draft"], max_query_len=state["nmax"])
        else:
            _plain_verify(state)
        return state["accepted"], state["count"], state["chosen"]
    if not own:
        return _plain_prefill(state) if op == "prefill" else _plain_decode(state)
    args = (state["out"], state["q"], state["k_cache"], state["v_cache"], state["tables"], state["lens"])
    sizes = (case["seqs"], case["hq"], case["hkv"], case["d"])
    if op == "common":
        work_space = _workspace(state, B.common_prefix_workspace_bytes(*sizes))
        return B.paged_decode_attention_common_prefix(*args, state["scale"], state["starts"], state["shared"],
                                                      max_group_size=int(state["group_max"]),
                                                      max_context_len=state["max_len"], workspace=work_space)
    scores = dict(softcap=case["cap"], window=case["window"], slopes=state["slopes"])
    if op == "decode":
        work_space = _workspace(state, B.workspace_bytes(*sizes, state["max_len"]))
        return B.paged_decode_attention_scored(*args, state["scale"], max_context_len=state["max_len"],
                                               workspace=work_space, **scores)
    return B.paged_prefill_attention_scored(*args, state["starts"], state["scale"], prefix_lens=state["prefixes"],
                                            max_query_len=state["nmax"], max_context_len=state["max_len"], **scores)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_verify(case, st):
    tokens, parents, starts = (st[k].tolist() for k in ("tokens", "parents", "starts"))
    u, final = st["uniforms"].double().tolist(), st["final"].double().tolist()
    accepted = torch.full_like(st["accepted"], -1)
    count, chosen = torch.zeros_like(st["count"]), torch.full_like(st["chosen"], -1)
    for s in range(case["seqs"]):
        base, n = starts[s], starts[s + 1] - starts[s]
        if n == 0:
            continue
        path = [0]
        while True:
            p = st["target"][base + path[-1]].double().cpu().numpy()
            q = st["draft"][base + path[-1]].double().cpu().numpy() if case["draft"] else None
            children = [i for i in range(path[-1] + 1, n) if parents[base + i] == path[-1]]
            now, refused = p, False
            step = None
            for c in children:
                x = tokens[base + c]
                ratio = now[x] / (now.sum() if refused else 1.0)
                if u[base + c] * (1.0 if q is None else q[x]) < ratio:
                    step = c
                    break
                if q is None:
                    rest = now.copy()
                    rest[x] = 0.0
                else:
                    rest = np.maximum(now / (now.sum() if refused else 1.0) - q, 0.0)
                if rest.sum() > 0:
                    now, refused = rest, True
            if step is None:
                break
            path.append(step)
        grown = np.cumsum(now)
        chosen[s] = int(np.searchsorted(grown, final[s] * grown[-1], side="right"))
        count[s] = len(path)
        accepted[s, :len(path)] = torch.tensor(path, dtype=torch.int32)
    return accepted, count, chosen


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "verify":
        return _exact_verify(case, st)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g = hq // hkv
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    ns = st["ns"] if case["op"] == "prefill" else [1] * case["seqs"]
    window = case.get("window") or 1 << 30
    row = 0
    for s, length in enumerate(st["lens"].tolist()):
        n = ns[s]
        if n == 0:
            continue
        blocks = st["tables"][s, :-(-length // BLOCK)].long()
        pre = int(st["prefixes"][s]) if st["prefixes"] is not None else 0
        pos = torch.arange(length - n, length, device="cuda")
        far = torch.arange(length, device="cuda")[None] - pos[:, None]                  # key - query
        see = ((far <= 0) | (far + pos[:, None] < pre)) & (far.abs() < window)
        for h in range(hkv):
            k, v = (c[blocks, h].double().reshape(-1, d)[:length] for c in (st["k_cache"], st["v_cache"]))
            for e in range(h * g, (h + 1) * g):
                z = st["q"][row:row + n, e].double() @ k.T * st["scale"]
                if case.get("cap"):
                    z = case["cap"] * torch.tanh(z / case["cap"])
                if st["slopes"] is not None:
                    z = z - st["slopes"][e].double() * far.abs()
                out[row:row + n, e] = torch.softmax(z.masked_fill(~see, -math.inf), -1) @ v
        row += n
    return out
