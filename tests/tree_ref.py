"""Plain 64-bit forms of the operators on a tree of drafts (test infrastructure): loops over
sequences and rows, written from the definitions in include/svd_tree.h."""
from __future__ import annotations

import math

import torch


def ancestors(parent, j):
    out = []
    while j >= 0:
        out.append(j)
        j = parent[j]
    return out


def parents_of(parent, B, n):
    if parent is None:
        return [[j - 1 for j in range(n)] for _ in range(B)]
    return parent.tolist()


def random_tree(B, n, seed, kind="tree"):
    """[B, n] int32 parents on the CPU: a tree, a chain, a star or a forest without a common root."""
    g = torch.Generator().manual_seed(seed)
    rows = []
    for _ in range(B):
        r = [-1]
        for j in range(1, n):
            if kind == "chain":
                r.append(j - 1)
            elif kind == "star":
                r.append(0)
            else:
                lo = -1 if kind == "forest" else 0
                r.append(int(torch.randint(max(lo, j - 9), j, (1,), generator=g)))
        rows.append(r)
    return torch.tensor(rows, dtype=torch.int32).view(B, n)


def attention(q, k_new, v_new, cache_k, cache_v, page_table, cache_len, parent=None, n_nodes=None, scale=None):
    """(out, lse, tol_out, tol_lse) in fp64 on q's device.

    The tolerances follow from the arithmetic.  u = eps / 2 of the tensors' type bounds the rounding
    of a softmax weight before the matrix product, and the rounding of the result.  A score is an fp32 sum of D
    exact products (2^-23 each relative to the sum of magnitudes, tensor-core accumulation may
    truncate), scaled and brought to base 2 (2^-22 of its size), and goes through an approximate
    exp2 (2^-21): a weight is off by e = 2^-23 D sum|q k| scale + 2^-22 |s| + 2^-21 relative, its
    normalised value by 2 e, and the sum over T keys adds T 2^-24.  Weights below the type's
    normal range are off by half its smallest step instead."""
    B, n, Hq, D = q.shape
    Hkv, G, page = k_new.shape[2], q.shape[2] // k_new.shape[2], cache_k.shape[1]
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    dev, f64 = q.device, torch.float64
    fi = torch.finfo(q.dtype)
    u, tiny = fi.eps / 2, fi.smallest_normal * fi.eps / 2
    out = torch.zeros(q.shape, dtype=f64, device=dev)
    lse = torch.full((B, n, Hq), -math.inf, dtype=f64, device=dev)
    tol, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    par = parents_of(parent, B, n)
    for b in range(B):
        L, used = int(cache_len[b]), n if n_nodes is None else int(n_nodes[b])
        if L:
            t = torch.arange(L, device=dev)
            pg = page_table[b].to(dev).long()[t // page]
            kc, vc = cache_k[pg, t % page].to(f64), cache_v[pg, t % page].to(f64)
        for j in range(used):
            anc = ancestors(par[b], j)
            for hk in range(Hkv):
                k, v = k_new[b, anc, hk].to(f64), v_new[b, anc, hk].to(f64)
                if L:
                    k, v = torch.cat([kc[:, hk], k]), torch.cat([vc[:, hk], v])
                hs = slice(hk * G, (hk + 1) * G)
                qq = q[b, j, hs].to(f64)
                s = qq @ k.T * scale
                m = s.amax(1, keepdim=True)
                p = torch.exp(s - m)
                l = p.sum(1, keepdim=True)
                out[b, j, hs] = p @ v / l
                lse[b, j, hs] = (m + l.log()).squeeze(1)
                mag = (qq.abs() @ k.abs().T).amax(1, keepdim=True) * abs(scale)
                e = 2.0 ** -23 * D * mag + 2.0 ** -22 * s.abs().amax(1, keepdim=True) + 2.0 ** -21
                T = k.shape[0]
                tol[b, j, hs] = (u * out[b, j, hs].abs() + (p @ v.abs() / l) * (u + 2 * e + T * 2.0 ** -24)
                                 + tiny * (1 + v.abs().sum(0) / l))
                tol_l[b, j, hs] = (2 * e + T * 2.0 ** -24 + 2.0 ** -22 * lse[b, j, hs].abs().unsqueeze(1)).squeeze(1)
    return out, lse, tol, tol_l


def counts(B, n, V, history, prompt_len, hist_len, node_tok, parent, dev):
    """(count, seen): [B, n, V] fp64 and bool."""
    c = torch.zeros((B, n, V), dtype=torch.float64, device=dev)
    seen = torch.zeros((B, n, V), dtype=torch.bool, device=dev)
    par = parents_of(parent, B, n)
    for b in range(B):
        if history is not None:
            S = history.shape[1]
            hl = S if hist_len is None else min(max(int(hist_len[b]), 0), S)
            pl = 0 if prompt_len is None else min(max(int(prompt_len[b]), 0), hl)
            for i, tok in enumerate(history[b, :hl].tolist()):
                if 0 <= tok < V:
                    seen[b, :, tok] = True
                    if i >= pl:
                        c[b, :, tok] += 1
        if node_tok is not None:
            toks = node_tok[b].tolist()
            for j in range(n):
                for i in ancestors(par[b], j):
                    if 0 <= toks[i] < V:
                        c[b, j, toks[i]] += 1
                        seen[b, j, toks[i]] = True
    return c, seen


def allowed(mask, n, V):
    """[B, n, V] bool from packed words."""
    w = mask.to(torch.int64) & 0xffffffff
    v = torch.arange(V, device=mask.device)
    return (((w[..., v // 32] >> (v % 32)) & 1) != 0).expand(-1, n, -1)


def process(logits, *, history=None, prompt_len=None, hist_len=None, node_tok=None, parent=None, repetition=None,
            frequency=None, presence=None, bias_tok=None, bias_val=None, mask=None, mask_value=-32768.0):
    """(z, tolerance): four fp32 operations (2^-24 of each operand) and one rounding to bf16 (2^-8)."""
    B, n, V = logits.shape
    dev, f64 = logits.device, torch.float64
    c, seen = counts(B, n, V, history, prompt_len, hist_len, node_tok, parent, dev)
    per = lambda t, d: torch.full((B, 1, 1), d, dtype=f64, device=dev) if t is None else t.to(f64).view(B, 1, 1)  # noqa: E731
    r, f, p = per(repetition, 1.0), per(frequency, 0.0), per(presence, 0.0)
    x = logits.to(f64)
    x1 = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
    add = torch.zeros((B, 1, V), dtype=f64, device=dev)
    if bias_tok is not None:
        for b in range(B):
            for tok, val in zip(bias_tok[b].tolist(), bias_val[b].tolist()):
                if 0 <= tok < V:
                    add[b, 0, tok] += val
    z = x1 - f * c - p * (c > 0) + add
    tol = 2.0 ** -8 * z.abs() + 4 * 2.0 ** -24 * (x1.abs() + f.abs() * c + p.abs() + add.abs())
    if mask is not None:
        ok = allowed(mask, n, V)
        mv = torch.tensor(mask_value).to(torch.bfloat16).to(f64).item()
        z = torch.where(ok, z, torch.full_like(z, mv))
        tol = torch.where(ok, tol, torch.zeros_like(tol))
    return z, tol


def process_grad(dz, logits, *, history=None, prompt_len=None, hist_len=None, node_tok=None, parent=None,
                 repetition=None, mask=None):
    B, n, V = logits.shape
    _, seen = counts(B, n, V, history, prompt_len, hist_len, node_tok, parent, logits.device)
    r = 1.0 if repetition is None else repetition.double().view(B, 1, 1)
    d = dz.double()
    d = torch.where(seen, torch.where(logits.double() > 0, d / r, d * r), d)
    return d if mask is None else torch.where(allowed(mask, n, V), d, torch.zeros_like(d))


def verify(y, node_tok, parent=None, n_nodes=None):
    """The walk, sequence by sequence: lists (path, emitted)."""
    B, n = node_tok.shape
    par, tok = parents_of(parent, B, n), node_tok.tolist()
    paths, toks = [], []
    for b in range(B):
        used = n if n_nodes is None else int(n_nodes[b])
        path, em = [], []
        if used > 0:
            cur = 0
            while True:
                path.append(cur)
                em.append(int(y[b, cur]))
                nxt = [c for c in range(1, used) if par[b][c] == cur and tok[b][c] == em[-1] and tok[b][c] >= 0]
                if not nxt:
                    break
                cur = nxt[0]
        paths.append(path)
        toks.append(em)
    return paths, toks
