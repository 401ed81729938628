"""Cases that measure the tree-of-drafts operators: attention of the drafted nodes over the paged cache, logits
processing (penalties, biases, grammar masks) with its gradient, acceptance over the tree, append to the cache.

A case names its operator in ``op``; ``run`` makes one pass, in plain torch operations or, with ``own`` set, through
the framework's entry points."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token of one request: a decode step without drafts, where latency counts
        dict(name="attention_decode_b1", op="attention", B=1, n=1, tree=False, Hq=32, Hkv=8, D=128, page=16, lo=1000,
             hi=1000, dtype="bf16"),
        # a batch of 32 verifying blocks of 16 drafts (17 nodes) over ragged contexts
        dict(name="attention_chain_b32", op="attention", B=32, n=17, tree=False, Hq=32, Hkv=8, D=128, page=16, lo=1,
             hi=4096, dtype="bf16"),
        # wide trees of a few long-context requests, narrow heads: many rows for each key
        dict(name="attention_tree_b4_long", op="attention", B=4, n=64, tree=True, Hq=64, Hkv=8, D=64, page=64,
             lo=28001, hi=32768, dtype="fp16"),
        # full serving concurrency, blocks of 16 drafts
        dict(name="attention_tree_b128", op="attention", B=128, n=17, tree=True, Hq=32, Hkv=8, D=128, page=64, lo=500,
             hi=6000, dtype="bf16"),
        # the tiny workload's logits: blocks of 8 drafts behind their root
        dict(name="process_tiny", op="process", B=4, n=9, tree=False, V=1024, hist=300, bias=8, mask="row"),
        # greedy verification of 32 blocks under a grammar
        dict(name="process_b32", op="process", B=32, n=17, tree=True, V=151936, hist=2048, bias=64, mask="row"),
        # the gradient of the distillation loss on its way to the drafter's raw logits
        dict(name="process_grad_b32", op="grad", B=32, n=16, tree=False, V=151936, hist=2048, bias=0, mask="row",
             dtype="bf16"),
        dict(name="process_grad_b6_fp32", op="grad", B=6, n=16, tree=False, V=128256, hist=700, bias=0, mask="seq",
             dtype="fp32"),
        # greedy acceptance over trees
        dict(name="verify_tiny", op="verify", B=4, n=9, tree=True, V=1024),
        dict(name="verify_b64", op="verify", B=64, n=33, tree=True, V=151936),
        # the accepted paths of a full batch go into the cache
        dict(name="append_path_b128", op="append", B=128, n=17, path=True, Hkv=8, D=128, page=16, hi=1500, dtype="bf16"),
        # the keys and values of prompts
        dict(name="append_prompt_b8", op="append", B=8, n=4001, path=False, Hkv=8, D=128, page=64, hi=700, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "process", "grad", "verify", "append"])
    n, tree = rng.choice([1, 2, 5, 9, 17, 33, rng.randint(1, 64)]), rng.random() < 0.5
    B = _log(rng, 1, 128)
    if op == "attention":
        Hkv = rng.choice([1, 2, 4, 8])
        D = rng.choice([64, 80, 96, 128])
        Hq = Hkv * rng.choice([1, 3, 4, 7, 8])
        hi = _log(rng, 16, 32768)
        while B * hi * Hkv * D > 300e6 or B * hi * Hq * n > 250e6:
            B, hi = max(1, B // 2), max(16, hi // 2 + 1)
        return dict(op=op, B=B, n=n, tree=tree, Hq=Hq, Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128]),
                    lo=rng.choice([0, 1, hi // 2, hi]), hi=hi, dtype=rng.choice(["bf16", "fp16"]))
    if op == "append":
        path = rng.random() < 0.5
        return dict(op=op, B=B if path else max(1, B // 8), n=n if path else _log(rng, 1, 4000), path=path,
                    Hkv=rng.choice([1, 2, 8]), D=rng.choice([64, 96, 128]), page=rng.choice([16, 32, 64, 128]),
                    hi=_log(rng, 1, 1500), dtype=rng.choice(["bf16", "fp16"]))
    V = rng.choice([1024, 128256, 151936, _log(rng, 500, 152000)])
    while B * n * V > 80e6:
        B, n = max(1, B // 2), max(1, n * 3 // 4)
    if op == "verify":
        return dict(op=op, B=B, n=n, tree=tree, V=V)
    c = dict(op=op, B=B, n=n, tree=tree, V=V, hist=_log(rng, 1, 4096), bias=rng.choice([0, 0, 5, 200]) if op == "process" else 0,
             mask=rng.choice(["none", "row", "seq"]))
    if op == "grad":
        c["dtype"] = rng.choice(["bf16", "fp32"])
    return c


def _tree(B, n, tree, g):
    """Parents of every node: a chain, or each node under one of the (up to) eight nodes before it."""
    j = torch.arange(n, device="cuda", dtype=torch.int32).expand(B, n)
    if not tree:
        return (j - 1).contiguous()
    back = (torch.rand((B, n), generator=g, device="cuda") * 8).to(torch.int32)
    return torch.where(j == 0, -1, torch.clamp(j - 1 - back, min=0)).to(torch.int32).contiguous()


def _lens(B, lo, hi, g):
    return (lo + (torch.rand(B, generator=g, device="cuda") * (hi - lo + 1)).to(torch.int32)).clamp(max=hi).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    c, B, n = case, case["B"], case["n"]
    rand = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    randn = lambda *s, dt=torch.float32: torch.randn(s, generator=g, device="cuda", dtype=dt)  # noqa: E731
    st = dict(case=c)
    if c["op"] in ("attention", "append"):
        dt = DTYPES[c["dtype"]]
        room = c["hi"] + (n if c["op"] == "append" else 0)
        per = -(-room // c["page"])
        st["page_table"] = torch.randperm(B * per, generator=g, device="cuda").to(torch.int32).view(B, per)
        for x in ("cache_k", "cache_v"):
            st[x] = randn(B * per, c["page"], c["Hkv"], c["D"], dt=dt)
        st["k_new"], st["v_new"] = (randn(B, n, c["Hkv"], c["D"], dt=dt) for _ in range(2))
        st["cache_len"] = _lens(B, c.get("lo", 0), c["hi"], g)
        if c["op"] == "attention":
            st["q"] = (1.5 * randn(B, n, c["Hq"], c["D"])).to(dt)
            st["parent"] = _tree(B, n, c["tree"], g)
        elif c["path"]:
            # strictly rising node indices, as an accepted path has them; at least the root
            keep = rand(B, n) < 0.4
            keep[:, 0] = True
            j = torch.where(keep, torch.arange(n, device="cuda"), 10 * n).sort(1).values
            st["path"] = torch.where(j < n, j, -1).to(torch.int32)
            st["count"] = keep.sum(1).to(torch.int32)
        else:
            st["path"], st["count"] = None, _lens(B, max(1, n // 2), n, g)
        return st
    V = c["V"]
    # logits as the workloads have them: normal noise on a head-and-tail bias over the ids
    base = -torch.log(torch.randperm(V, generator=g, device="cuda").float() + 1.0)
    st["logits"] = (2.0 * randn(B, n, V) + base).to(torch.bfloat16)
    st["parent"] = _tree(B, n, c["tree"], g)
    if c["op"] == "verify":
        # drafted tokens that often are the target's choice at their parent
        y = st["logits"].float().argmax(-1)
        right = y.gather(1, st["parent"].clamp(min=0).long())
        st["node_tok"] = torch.where(rand(B, n) < 0.7, right, (rand(B, n) * V).long()).to(torch.int32)
        return st
    S = c["hist"]
    st["node_tok"] = ((rand(B, n) ** 2) * V).to(torch.int32).clamp(max=V - 1)
    st["history"] = ((rand(B, S) ** 3) * V).to(torch.int32).clamp(max=V - 1)
    st["hist_len"] = _lens(B, S // 2, S, g)
    st["prompt_len"] = (rand(B) * (st["hist_len"] + 1)).to(torch.int32).minimum(st["hist_len"])
    st["repetition"], st["frequency"], st["presence"] = 1.0 + 0.3 * rand(B), 0.5 * rand(B), 0.5 * rand(B)
    if c["bias"]:
        st["bias_tok"] = torch.stack([torch.randperm(V, generator=g, device="cuda")[:c["bias"]] for _ in range(B)]).to(torch.int32)
        st["bias_val"] = 4.0 * randn(B, st["bias_tok"].shape[1])
    else:
        st["bias_tok"] = st["bias_val"] = None
    if c["mask"] == "none":
        st["mask"] = None
    else:
        # grammars that allow half of the ids, an eighth, or all but a few
        shape = (B, n if c["mask"] == "row" else 1, -(-V // 32))
        bits = lambda: torch.randint(-2**31, 2**31, shape, generator=g, device="cuda", dtype=torch.int64)  # noqa: E731
        a, b, d, kind = bits(), bits(), bits(), torch.arange(B, device="cuda").view(B, 1, 1) % 3
        st["mask"] = torch.where(kind == 0, a, torch.where(kind == 1, a & b & d, a | b | d)).to(torch.int32)
    if c["op"] == "grad":
        st["dz"] = (0.01 * randn(B, n, V)).to(DTYPES[c["dtype"]])
    return st


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------
def _ancestors(parent):
    """[B, n, n]: whether node i is j itself or on the way from the root to j."""
    n = parent.shape[1]
    up = (parent.unsqueeze(2) == torch.arange(n, device=parent.device)).float()
    return torch.linalg.matrix_power(up + torch.eye(n, device=parent.device), n) > 0


def _attention(s):
    c, q = s["case"], s["q"].float()
    B, n, Hq, D = q.shape
    Hkv, L = c["Hkv"], c["hi"]
    pages = s["page_table"].long()
    kc, vc = (s[x][pages].reshape(B, -1, Hkv, D)[:, :L].float() for x in ("cache_k", "cache_v"))
    k, v = torch.cat([kc, s["k_new"].float()], 1), torch.cat([vc, s["v_new"].float()], 1)
    seen = (torch.arange(L, device="cuda") < s["cache_len"].unsqueeze(1)).unsqueeze(1).expand(B, n, L)
    seen = torch.cat([seen, _ancestors(s["parent"])], 2)
    rows = q.view(B, n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    x = rows @ k.permute(0, 2, 3, 1) / math.sqrt(D)
    x = x.view(B, Hkv, Hq // Hkv, n, L + n).masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, -1, L + n) @ v.permute(0, 2, 1, 3)).view(B, Hkv, Hq // Hkv, n, D) / total
    lse = (top + total.log()).squeeze(-1)
    return dict(out=o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D).to(s["q"].dtype),
                lse=lse.permute(0, 3, 1, 2).reshape(B, n, Hq).contiguous())


def _counts(s, n, V):
    """For every row: the count of each id among the generated tokens, and whether it was seen at all."""
    B, S = s["history"].shape
    at, h = torch.arange(S, device="cuda"), s["history"].long()
    hist, prompt = (at < s["hist_len"].unsqueeze(1)), (at < s["prompt_len"].unsqueeze(1))
    zero = torch.zeros((B, V), device="cuda")
    made = zero.scatter_add(1, h, (hist & ~prompt).float())
    given = zero.scatter_add(1, h, prompt.float())
    path = torch.zeros((B, n, V), device="cuda")
    path.scatter_add_(2, s["node_tok"].long().unsqueeze(1).expand(B, n, n), _ancestors(s["parent"]).float())
    count = path + made.unsqueeze(1)
    return count, (count > 0) | (given > 0).unsqueeze(1)


def _allowed(mask, V):
    bits = (mask.unsqueeze(-1) >> torch.arange(32, device=mask.device, dtype=torch.int32)) & 1
    return bits.reshape(mask.shape[0], mask.shape[1], -1)[..., :V] != 0


def _process(s):
    x = s["logits"].float()
    B, n, V = x.shape
    count, seen = _counts(s, n, V)
    per = lambda name: s[name].view(B, 1, 1)  # noqa: E731
    x = torch.where(seen, torch.where(x > 0, x / per("repetition"), x * per("repetition")), x)
    x = x - per("frequency") * count
    x = x - per("presence") * (count > 0).float()
    if s["bias_tok"] is not None:
        x = x + torch.zeros((B, V), device="cuda").scatter_add(1, s["bias_tok"].long(), s["bias_val"]).unsqueeze(1)
    if s["mask"] is not None:
        x = torch.where(_allowed(s["mask"], V), x, -math.inf)
    out = x.to(torch.bfloat16)
    return dict(out=out, argmax=_first_argmax(out))


def _first_argmax(x):
    """Lowest index of the largest value."""
    hit = x == x.amax(-1, keepdim=True)
    return torch.where(hit, torch.arange(x.shape[-1], device=x.device, dtype=torch.int32), x.shape[-1]).amin(-1)


def _grad(s):
    B, n, V = s["dz"].shape
    _, seen = _counts(s, n, V)
    r = s["repetition"].view(B, 1, 1)
    d = s["dz"].float()
    d = torch.where(seen, torch.where(s["logits"].float() > 0, d / r, d * r), d)
    if s["mask"] is not None:
        d = torch.where(_allowed(s["mask"], V), d, 0.0)
    return dict(dlogits=d.to(s["dz"].dtype))


def _verify(s):
    y, tok, up = _first_argmax(s["logits"].float()), s["node_tok"], s["parent"]
    B, n = tok.shape
    j = torch.arange(n, device="cuda")
    match = (tok == y.gather(1, up.clamp(min=0).long())) & (up >= 0)
    same = (up.unsqueeze(2) == up.unsqueeze(1)) & (tok.unsqueeze(2) == tok.unsqueeze(1))
    first = ~(same & (j.view(1, 1, n) < j.view(1, n, 1))).any(2)
    ok = (match & first) | (j == 0)
    taken = (ok.unsqueeze(1) | ~_ancestors(up)).all(2) & _ancestors(up)[:, :, 0]
    order = torch.where(taken, j, n).sort(1).values
    count = taken.sum(1, keepdim=True)
    path = torch.where(order < n, order, -1)
    last = path.gather(1, count - 1)
    after = torch.cat([path[:, 1:], torch.full((B, 1), -1, device="cuda")], 1)
    emitted = torch.where(after >= 0, tok.gather(1, after.clamp(min=0)).long(), -1)
    emitted = torch.where(j == count - 1, y.gather(1, last).long(), emitted)
    i32 = lambda t: t.to(torch.int32)  # noqa: E731
    return dict(target_argmax=y, path=i32(path), n_path=i32(count[:, 0]), accept_len=i32(count[:, 0] - 1),
                emitted=i32(emitted), n_emitted=i32(count[:, 0]))


def _append(s):
    B, n, Hkv, D = s["k_new"].shape
    page = s["cache_k"].shape[1]
    i = torch.arange(n, device="cuda").expand(B, n)
    # entries behind a sequence's count write its first entry once more
    i = torch.where(i < s["count"].unsqueeze(1), i, 0)
    node = i if s["path"] is None else s["path"].long().gather(1, i)
    at = s["cache_len"].unsqueeze(1) + i
    slot = s["page_table"].long().gather(1, at // page) * page + at % page
    pick = node[:, :, None, None].expand(B, n, Hkv, D)
    for new, cache in (("k_new", "cache_k"), ("v_new", "cache_v")):
        s[cache].view(-1, Hkv, D)[slot.view(-1)] = s[new].gather(1, pick).view(-1, Hkv, D)
    return dict(cache_k=s["cache_k"], cache_v=s["cache_v"], new_len=s["cache_len"] + s["count"])


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def _handle(s):
    """The operator's call object, which a program makes once for its buffers and calls every step."""
    from speculative_decoding_verify_distill_b200 import api

    op = s["case"]["op"]
    if op == "attention":
        return api.TreeAttention(s["q"], s["k_new"], s["v_new"], s["cache_k"], s["cache_v"], s["page_table"],
                                 s["cache_len"], parent=s["parent"], lse=True)
    if op == "verify":
        return api.TreeVerify(s["node_tok"], logits=s["logits"], parent=s["parent"])
    if op == "append":
        return api.CacheAppend(s["k_new"], s["v_new"], s["cache_k"], s["cache_v"], s["page_table"], s["cache_len"],
                               s["count"], path=s["path"])
    kw = dict(history=s["history"], prompt_len=s["prompt_len"], hist_len=s["hist_len"], node_tok=s["node_tok"],
              parent=s["parent"], repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
              bias_tok=s["bias_tok"], bias_val=s["bias_val"], mask=s["mask"])
    if op == "process":
        return api.LogitsProcess(s["logits"], mask_value=-math.inf, argmax=True, **kw)
    return api.LogitsProcessGrad(s["dz"], s["logits"], **kw)


def run(state):
    if own:
        if "handle" not in state:
            state["handle"] = _handle(state)
        return state["handle"]().outputs()
    return {"attention": _attention, "process": _process, "grad": _grad, "verify": _verify,
            "append": _append}[state["case"]["op"]](state)


def work(case):
    c, B, n = case, case["B"], case["n"]
    if c["op"] == "attention":
        keys = B * (c["lo"] + c["hi"]) / 2
        row = c["Hkv"] * c["D"] * 2
        return dict(bytes=2 * row * (keys + B * n) + 2 * 2 * B * n * c["Hq"] * c["D"] + 4 * B * n * c["Hq"],
                    flops=4 * n * c["Hq"] * c["D"] * (keys + B * (n + 1) / 2))
    if c["op"] == "append":
        rows = B * (1 + 0.4 * (n - 1) if c["path"] else 0.75 * n)
        return dict(bytes=2 * 2 * 2 * rows * c["Hkv"] * c["D"], flops=0)
    logits = B * n * c["V"]
    if c["op"] == "verify":
        return dict(bytes=2 * logits, flops=logits)
    mask = {"none": 0, "row": logits / 8, "seq": logits / n / 8}[c["mask"]]
    lists = B * (4 * 0.75 * c["hist"] + 8 * c["bias"] + 8 * n)
    if c["op"] == "process":
        return dict(bytes=4 * logits + mask + lists, flops=logits)
    # the raw logits are needed where an id was seen: sparse, so not counted
    return dict(bytes=2 * logits * (2 if c["dtype"] == "bf16" else 4) + mask + lists, flops=logits)


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------------------------
def _up(parent, j):
    while j >= 0:
        yield j
        j = parent[j]


def exact(case, seed):
    s = prepare(case, seed)
    c, B, n = case, case["B"], case["n"]
    if c["op"] == "verify":
        return None
    if c["op"] == "append":
        k, v = s["cache_k"].double(), s["cache_v"].double()
        for b in range(B):
            m, at = int(s["count"][b]), int(s["cache_len"][b])
            node = torch.arange(m, device="cuda") if s["path"] is None else s["path"][b, :m].long()
            t = torch.arange(at, at + m, device="cuda")
            pg, off = s["page_table"][b][t // c["page"]].long(), t % c["page"]
            k[pg, off], v[pg, off] = s["k_new"][b, node].double(), s["v_new"][b, node].double()
        return dict(cache_k=k, cache_v=v, new_len=None)
    parents = s["parent"].tolist()
    if c["op"] == "attention":
        out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.empty(s["q"].shape[:3], dtype=torch.float64, device="cuda")
        G = c["Hq"] // c["Hkv"]
        for b in range(B):
            L = int(s["cache_len"][b])
            pages = s["page_table"][b, :-(-L // c["page"])].long()
            K, W = (torch.cat([s[x][pages].reshape(-1, c["Hkv"], c["D"])[:L], s[y][b]]).double()
                    for x, y in (("cache_k", "k_new"), ("cache_v", "v_new")))
            hide = torch.zeros((n, L + n), dtype=torch.bool, device="cuda")
            hide[:, L:] = True
            for j in range(n):
                hide[j, [L + i for i in _up(parents[b], j)]] = False
            for h in range(c["Hkv"]):
                z = torch.einsum("ngd,td->ngt", s["q"][b, :, h * G:(h + 1) * G].double(), K[:, h]) * c["D"] ** -0.5
                z = z.masked_fill(hide[:, None], -math.inf)
                lse[b, :, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
                out[b, :, h * G:(h + 1) * G] = torch.einsum("ngt,td->ngd", torch.softmax(z, -1), W[:, h])
        return dict(out=out, lse=lse)
    V = c["V"]
    got = []
    for b in range(B):
        pl, hl = int(s["prompt_len"][b]), int(s["hist_len"][b])
        h = s["history"][b].long()
        made = torch.bincount(h[pl:hl], minlength=V).double()
        given = torch.bincount(h[:pl], minlength=V) > 0
        rep, fr, pr = (s[x][b].double() for x in ("repetition", "frequency", "presence"))
        add = torch.zeros(V, dtype=torch.float64, device="cuda")
        if s["bias_tok"] is not None:
            add.index_add_(0, s["bias_tok"][b].long(), s["bias_val"][b].double())
        for j in range(n):
            cnt = made + torch.bincount(s["node_tok"][b, list(_up(parents[b], j))].long(), minlength=V)
            seen = given | (cnt > 0)
            x = s["logits"][b, j].double()
            factor = torch.where(seen, torch.where(x > 0, 1 / rep, rep), torch.ones_like(x))
            if c["op"] == "process":
                z = x * factor - fr * cnt - pr * (cnt > 0) + add
            else:
                z = s["dz"][b, j].double() * factor
            if s["mask"] is not None:
                words = s["mask"][b, j if c["mask"] == "row" else 0]
                ids = torch.arange(V, device="cuda")
                z = z.masked_fill(((words[ids // 32] >> (ids % 32)) & 1) == 0, -math.inf if c["op"] == "process" else 0.0)
            got.append(z)
    z = torch.stack(got).view(B, n, V)
    return dict(out=z, argmax=None) if c["op"] == "process" else dict(dlogits=z)
