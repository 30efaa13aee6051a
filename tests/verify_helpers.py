"""The walk of verify_drafts in 64 bits (numpy), straight from its definition,
and small trees of drafts for its tests."""
import numpy as np
import torch


def walk(n, parents, tokens, target, draft, uniforms, final, max_accepted):
    """One sequence: rows kept, token that follows.  target, draft: [n, V] float64 (draft None: certain drafts);
    parents and tokens may hold anything; the remaining distribution is normalised at every refusal."""
    vocab = target.shape[1]
    clean = lambda x: np.where(np.isnan(x) | (x < 0), 0.0, x)
    path = [0]
    while True:
        p = clean(target[path[-1]])
        q = None if draft is None else clean(draft[path[-1]])
        rest, refused, took = p, False, None
        if len(path) < max_accepted:
            for i in range(path[-1] + 1, n):
                if parents[i] != path[-1]:
                    continue
                x = int(tokens[i])
                known = 0 <= x < vocab
                total = rest.sum() if refused else 1.0
                have = rest[x] / total if known and total > 0 else 0.0
                if known and uniforms[i] * (1.0 if q is None else q[x]) < have:
                    took = i
                    break
                after = rest.copy()
                if q is not None:
                    after = np.maximum(rest / total - q, 0.0)
                elif known:
                    after[x] = 0.0
                if after.sum() > 0:
                    rest, refused = after, True
        if took is None:
            break
        path.append(took)
    grown = np.cumsum(rest)
    if not grown[-1] > 0:
        return path, -1
    return path, int(np.searchsorted(grown, final * grown[-1], side="right"))


def walk_all(start, parents, tokens, target, draft, uniforms, final, max_accepted):
    f = lambda t: None if t is None else t.detach().double().cpu().numpy()
    target, draft, uniforms, final = f(target), f(draft), f(uniforms), f(final)
    start, parents, tokens = (t.cpu().numpy() for t in (start, parents, tokens))
    accepted = np.full((len(start) - 1, max_accepted), -1, dtype=np.int32)
    count, following = np.zeros(len(start) - 1, dtype=np.int32), np.full(len(start) - 1, -1, dtype=np.int64)
    for s in range(len(start) - 1):
        rows = slice(start[s], start[s + 1])
        n = start[s + 1] - start[s]
        if n <= 0:
            continue
        path, following[s] = walk(n, parents[rows], tokens[rows], target[rows], None if draft is None else draft[rows],
                                  uniforms[rows], final[s], max_accepted)
        count[s] = len(path)
        accepted[s, :len(path)] = path
    return accepted, count, following


def trees(seed, ns, vocab, with_draft, dtype=torch.float32, back=3, sharp=3.0, device="cuda"):
    """Trees of ns[s] rows: parents a few rows back at most, tokens drawn from the draft's distribution behind the
    parent.  Returns (start, parents, tokens, target, draft, uniforms, final), draft None without ``with_draft``."""
    rng = np.random.default_rng(seed)
    start = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    total = int(start[-1])

    def soft(x):
        e = np.exp(x - x.max(-1, keepdims=True))
        return e / e.sum(-1, keepdims=True)

    logits = rng.standard_normal((total, vocab)) * sharp
    target = soft(logits)
    near = soft(logits + 0.7 * rng.standard_normal((total, vocab)))
    parents, tokens = np.full(total, -1, dtype=np.int32), np.zeros(total, dtype=np.int64)
    for s, n in enumerate(ns):
        for i in range(1, n):
            up = int(rng.integers(max(0, i - back), i))
            parents[start[s] + i] = up
            tokens[start[s] + i] = rng.choice(vocab, p=near[start[s] + up])
    t = lambda a, dt=None: torch.from_numpy(np.ascontiguousarray(a)).to(device, dt)
    return (t(start), t(parents), t(tokens), t(target, dtype), t(near, dtype) if with_draft else None,
            t(rng.random(total), torch.float32).clamp(max=1 - 2 ** -24),
            t(rng.random(len(ns)), torch.float32).clamp(max=1 - 2 ** -24))
