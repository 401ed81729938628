"""The operators on a tree of drafts against their plain 64-bit forms (tests/tree_ref.py): sizes and
masks where they can go wrong, poisoned memory that must not matter, error words, streams, graphs,
and a step of all of them together."""
import math

import pytest
import torch

from speculative_decoding_verify_distill_b200 import api
from tests import tree_ref as R

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]
BF, FP = torch.bfloat16, torch.float16
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_verify_distill_b200 import build
    build.build()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(x):
    return torch.tensor(x, dtype=I32, device="cuda")


# ------------------------------------------------------------------------------------------
# attention
# ------------------------------------------------------------------------------------------
def attention_case(lens, n, Hq, Hkv, D, page, dtype=BF, kind="tree", seed=0, spare=3, poison=math.nan, extra_pages=0):
    """Random inputs whose unused memory (rows behind a length, spare pages) holds `poison`."""
    g, B = gen(seed), len(lens)
    per = max(-(-L // page) for L in lens) + extra_pages
    n_pages = B * per + spare
    table = torch.randperm(n_pages, generator=g, device="cuda")[:B * per].to(I32).view(B, per)
    cache = torch.full((2, n_pages, page, Hkv, D), poison, dtype=dtype, device="cuda")
    for b, L in enumerate(lens):
        if L:
            t = torch.arange(L, device="cuda")
            for x in (0, 1):
                cache[x, table[b].long()[t // page], t % page] = torch.randn((L, Hkv, D), generator=g, device="cuda").to(dtype)
    new = [torch.randn((B, n, Hkv, D), generator=g, device="cuda").to(dtype) for _ in range(2)]
    q = (1.5 * torch.randn((B, n, Hq, D), generator=g, device="cuda")).to(dtype)
    return dict(q=q, k_new=new[0], v_new=new[1], cache_k=cache[0], cache_v=cache[1], page_table=table,
                cache_len=ints(lens), parent=R.random_tree(B, n, seed, kind).cuda())


def check_attention(c, lse=True, scale=None, op=None, **kw):
    a = {**c, **kw}
    pos = [a.pop(x) for x in ("q", "k_new", "v_new", "cache_k", "cache_v", "page_table", "cache_len")]
    op = op or api.TreeAttention(*pos, lse=lse, scale=scale, **a)
    out = op().outputs()
    torch.cuda.synchronize()
    assert op.device_error() == 0
    ro, rl, to, tl = R.attention(*pos, scale=scale, **a)
    d = (out["out"].double() - ro).abs()
    assert not torch.isnan(out["out"]).any()
    assert (d <= to).all(), (d - to).max().item()
    if lse:
        same = (out["lse"] == rl) | ((out["lse"].double() - rl).abs() <= tl)
        assert same.all()
    return op


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n,Hq,Hkv,D,page,lens,kind", [
    (1, 8, 2, 128, 16, [0, 1, 15, 16, 17, 127, 128, 129, 300], "chain"),
    (1, 1, 1, 64, 8, [5], "chain"),
    (9, 8, 2, 64, 16, [0, 1, 500, 255, 256, 257], "tree"),
    (17, 32, 8, 128, 32, [700, 3, 64], "chain"),
    (33, 8, 2, 128, 64, [130, 65, 64, 63], "tree"),
    (64, 8, 1, 128, 128, [385, 0, 128], "tree"),
    (64, 3, 3, 96, 16, [40, 200], "star"),
    (5, 14, 2, 80, 256, [600, 256, 255, 1], "forest"),
    (3, 4, 4, 8, 8, [9, 17, 1], "tree"),
    (13, 24, 8, 72, 16, [77, 150], "tree"),
    (2, 40, 1, 128, 16, [1000], "chain"),
    (63, 6, 2, 120, 512, [513, 1], "forest"),
])
def test_attention(n, Hq, Hkv, D, page, lens, kind, dtype):
    check_attention(attention_case(lens, n, Hq, Hkv, D, page, dtype, kind, seed=n + D))


@pytest.mark.parametrize("poison", [math.inf, -math.inf, 0.0])
def test_attention_unused_memory_does_not_matter(poison):
    """Rows behind the length and pages of nobody hold NaN in every other test."""
    check_attention(attention_case([33, 0, 131], 7, 8, 2, 128, 16, seed=3, poison=poison, extra_pages=2))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("where", ["k_new", "v_new"])
def test_attention_of_other_branches_does_not_matter(where, bad):
    """A node whose key or value is not finite spoils the rows below it and no other."""
    c = attention_case([50, 0, 300], 12, 8, 2, 64, 16, seed=5)
    clean = check_attention(c).outputs()
    clean = {k: v.clone() for k, v in clean.items()}
    par = c["parent"].tolist()
    c[where] = c[where].clone()
    c[where][:, 4] = bad
    pos = [c[x] for x in ("q", "k_new", "v_new", "cache_k", "cache_v", "page_table", "cache_len")]
    out = api.svd_tree_attention(*pos, parent=c["parent"], lse=True)
    for b in range(3):
        for j in range(12):
            if 4 in R.ancestors(par[b], j):
                if where == "v_new":
                    got = out["out"][b, j].float()
                    assert (got == bad).all() if math.isinf(bad) else got.isnan().all()
                    assert torch.equal(out["lse"][b, j], clean["lse"][b, j])
                elif math.isnan(bad):
                    assert out["out"][b, j].isnan().all() and out["lse"][b, j].isnan().all()
            else:
                assert torch.equal(out["out"][b, j], clean["out"][b, j])
                assert torch.equal(out["lse"][b, j], clean["lse"][b, j])


def test_attention_padding_nodes():
    c = attention_case([50, 0, 300, 20], 12, 8, 2, 128, 16, seed=6)
    nn = ints([12, 5, 1, 0])
    for x in ("q", "k_new", "v_new"):
        for b, m in enumerate(nn.tolist()):
            c[x][b, m:] = math.nan
    out = check_attention(c, n_nodes=nn).outputs()
    for b, m in enumerate(nn.tolist()):
        assert (out["out"][b, m:] == 0).all() and (out["lse"][b, m:] == -math.inf).all()


def test_attention_default_chain_scales_and_shared_pages():
    c = attention_case([100, 40], 6, 4, 2, 64, 16, seed=8, kind="chain")
    c["parent"] = None
    c["page_table"][1, :2] = c["page_table"][0, :2]      # a shared prefix
    for x in ("cache_k", "cache_v"):
        t = torch.arange(40, device="cuda")
        c[x][c["page_table"][1].long()[t // 16], t % 16] = torch.randn((40, 2, 64), generator=gen(1), device="cuda").to(BF)
    for scale in (None, 0.0, -0.2, 1.0):
        check_attention(c, scale=scale)
    check_attention(c, lse=False)


def test_attention_large_scores():
    """Scores far apart: the running maximum moves by hundreds within a row, both ways."""
    c = attention_case([600, 600], 4, 4, 1, 128, 16, seed=9)
    ramp = torch.linspace(0.05, 3.0, 600, device="cuda").view(600, 1, 1)
    t = torch.arange(600, device="cuda")
    for b, r in ((0, ramp), (1, ramp.flip(0))):
        pg = c["page_table"][b].long()[t // 16]
        c["cache_k"][pg, t % 16] = (c["cache_k"][pg, t % 16].float() * r * 4).to(BF)
    check_attention(c)


def test_attention_interleaved_pages():
    c = attention_case([90, 33, 200], 5, 8, 2, 128, 32, seed=10)
    both = torch.stack([c["cache_k"], c["cache_v"]], 1).contiguous()
    check_attention({**c, "cache_k": both[:, 0], "cache_v": both[:, 1]})


def test_attention_offsets_past_32_bits():
    page, Hkv, D = 128, 8, 128
    n_pages = (1 << 32) // (page * Hkv * D) + 40
    cache = torch.empty((2, n_pages, page, Hkv, D), dtype=BF, device="cuda")
    pages = torch.tensor([n_pages - 1, 0, n_pages - 7, n_pages // 2 + 1], device="cuda")
    cache[:, pages] = torch.randn((2, 4, page, Hkv, D), generator=gen(2), device="cuda").to(BF)
    c = attention_case([1], 3, 16, Hkv, D, page, seed=11)
    c.update(cache_k=cache[0], cache_v=cache[1], page_table=pages.to(I32).view(1, 4), cache_len=ints([450]))
    check_attention(c)
    del cache
    torch.cuda.empty_cache()


def test_attention_many_sequences_and_long_one():
    lens = [int(x) for x in torch.randint(0, 400, (150,), generator=torch.Generator().manual_seed(3))]
    check_attention(attention_case(lens, 2, 4, 2, 64, 16, seed=12))
    lens[77] = 20000
    check_attention(attention_case(lens, 1, 4, 1, 128, 64, seed=13))


@pytest.mark.parametrize("n,Hq,Hkv,D,dtype", [(3, 8, 8, 128, BF), (40, 4, 2, 64, FP)])
def test_attention_items_of_one_tile(n, Hq, Hkv, D, dtype):
    """Many sequences with nothing in the cache, or next to nothing: every part holds many items."""
    lens = [0] * 300 + [1, 0, 128, 0, 5] * 30
    c = attention_case(lens, n, Hq, Hkv, D, 16, dtype, seed=18, extra_pages=0)
    op = check_attention(c, n_nodes=torch.arange(len(lens), device="cuda").remainder(n + 1).to(I32))
    first = {k: v.clone() for k, v in op.outputs().items()}
    for _ in range(20):
        op()
    assert all(torch.equal(v, first[k]) for k, v in op.outputs().items())


def test_attention_parts_of_many_sequences():
    """More sequences in a part than a part keeps lengths of; one key each, so out is v and lse is the score."""
    B, D = 12001, 64
    g = gen(20)
    q, k, v = (torch.randn((B, 1, 1, D), generator=g, device="cuda").to(BF) for _ in range(3))
    empty = torch.empty((0, 16, 1, D), dtype=BF, device="cuda")
    out = api.svd_tree_attention(q, k, v, empty, empty, torch.empty((B, 0), dtype=I32, device="cuda"),
                                 torch.zeros(B, dtype=I32, device="cuda"), lse=True)
    assert torch.equal(out["out"], v)
    s = (q.double() * k.double()).sum(-1) / 8
    mag = (q.double() * k.double()).abs().sum(-1) / 8
    assert ((out["lse"].double() - s).abs() <= 2.0 ** -23 * D * mag + 2.0 ** -21 * s.abs() + 2.0 ** -21).all()


def test_attention_more_row_groups_than_sms():
    """One key head for 1024 query heads of 20 nodes: 160 groups of 128 rows."""
    check_attention(attention_case([300, 7], 20, 1024, 1, 64, 32, seed=19))


def test_attention_no_cache_at_all():
    c = attention_case([0, 0], 6, 4, 2, 64, 16, seed=14)
    empty = torch.empty((0, 16, 2, 64), dtype=BF, device="cuda")
    check_attention({**c, "cache_k": empty, "cache_v": empty, "page_table": torch.empty((2, 0), dtype=I32, device="cuda")})


def test_attention_errors_are_reported_and_bounded():
    c = attention_case([40, 20], 4, 4, 2, 64, 16, seed=15)
    pos = [c[x] for x in ("q", "k_new", "v_new", "cache_k", "cache_v", "page_table", "cache_len")]
    for bad_table in (-1, 1 << 20):
        t = c["page_table"].clone()
        t[0, 1] = bad_table
        op = api.TreeAttention(*pos[:5], t, pos[6], parent=c["parent"])
        op()
        assert op.device_error() == 8
        assert op.device_error() == 0
    for bad_len in (-5, 10 ** 6):
        op = api.TreeAttention(*pos[:6], ints([bad_len, 20]), parent=c["parent"])
        op()
        assert op.device_error() == 8
    par = c["parent"].clone()
    par[1, 2] = 3
    op = api.TreeAttention(*pos, parent=par)
    op()
    assert op.device_error() == 9


def test_attention_repeats_bit_for_bit_on_streams_and_in_graphs():
    c1, c2 = attention_case([900, 10, 333], 9, 16, 4, 128, 16, seed=16), attention_case([64, 2000], 17, 8, 1, 64, 32, FP, seed=17)
    ops = [api.TreeAttention(*[c[x] for x in ("q", "k_new", "v_new", "cache_k", "cache_v", "page_table", "cache_len")],
                             parent=c["parent"], lse=True) for c in (c1, c2)]
    want = []
    for op in ops:
        op()
        want.append({k: v.clone() for k, v in op.outputs().items()})
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for op, s in zip(ops, streams):
            op(s)
    torch.cuda.synchronize()
    for op, w in zip(ops, want):
        assert all(torch.equal(v, w[k]) for k, v in op.outputs().items())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for op in ops:
            op()
    for op in ops:
        for v in op.outputs().values():
            v.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for op, w in zip(ops, want):
        assert all(torch.equal(v, w[k]) for k, v in op.outputs().items())
        assert op.device_error() == 0


# ------------------------------------------------------------------------------------------
# logits processing and its gradient
# ------------------------------------------------------------------------------------------
def process_case(B, n, V, S, nb, mask, seed, kind="tree"):
    g = gen(seed)
    ri = lambda hi, *s: torch.randint(0, hi, s, generator=g, device="cuda", dtype=I32)  # noqa: E731
    few = max(1, min(V, 40))     # ids that repeat
    c = dict(node_tok=ri(few, B, n), parent=R.random_tree(B, n, seed, kind).cuda(),
             repetition=1.0 + 0.5 * torch.rand(B, generator=g, device="cuda"),
             frequency=0.7 * torch.rand(B, generator=g, device="cuda"),
             presence=0.7 * torch.rand(B, generator=g, device="cuda"))
    if S:
        c["history"] = torch.where(torch.rand((B, S), generator=g, device="cuda") < 0.5, ri(few, B, S), ri(V, B, S))
        c["hist_len"] = ri(S + 1, B)
        c["prompt_len"] = torch.minimum(ri(S + 1, B), c["hist_len"])
    if nb:
        c["bias_tok"], c["bias_val"] = ri(V, B, nb), 3 * torch.randn((B, nb), generator=g, device="cuda")
    if mask:
        W = (V + 31) // 32
        c["mask"] = torch.randint(-2 ** 31, 2 ** 31, (B, n if mask == "row" else 1, W), generator=g, device="cuda",
                                  dtype=torch.int64).to(I32)
    logits = (2 * torch.randn((B, n, V), generator=g, device="cuda")).to(BF)
    return logits, c


def first_argmax(x):
    x = torch.where(x.isnan(), -math.inf, x.float())
    hit = x == x.amax(-1, keepdim=True)
    return torch.where(hit, torch.arange(x.shape[-1], device=x.device), x.shape[-1]).amin(-1).to(I32)


def check_process(logits, c, **kw):
    op = api.LogitsProcess(logits, argmax=True, **{**c, **kw})
    raw = logits.clone()
    out = op().outputs()
    torch.cuda.synchronize()
    assert op.device_error() == 0
    kw.pop("out", None)
    z, tol = R.process(raw, **{**c, **kw})
    got = out["out"].double()
    ok = (got == z) | ((got - z).abs() <= tol)
    assert ok.all(), (got - z).abs().max().item()
    assert torch.equal(out["argmax"], first_argmax(out["out"]))
    return out


@pytest.mark.parametrize("B,n,V,S,nb,mask", [
    (3, 5, 1024, 50, 6, "row"), (2, 9, 1000, 0, 0, None), (1, 1, 1, 3, 1, "row"), (2, 3, 7, 20, 2, "seq"), (2, 2, 8, 1, 0, "row"),
    (1, 4, 31, 9, 3, "row"), (1, 4, 33, 9, 0, "seq"), (3, 64, 2049, 300, 40, "row"), (2, 17, 4104, 1000, 9, "seq"),
    (1, 33, 40960, 5000, 100, "row"), (130, 2, 512, 30, 2, "row"), (2, 6, 9001, 64, 11, None), (1, 2, 151936, 2048, 300, "row"),
    (1, 1, 327680, 10, 0, "row")])
def test_process(B, n, V, S, nb, mask):
    logits, c = process_case(B, n, V, S, nb, mask, seed=B + n + V)
    out = check_process(logits, c)
    # in place, and the argmax alone, give the same
    same = logits.clone()
    api.svd_logits_process(same, out=same, **c)
    assert torch.equal(same.view(torch.int16), out["out"].view(torch.int16))
    assert torch.equal(api.svd_logits_process(logits, values=False, argmax=True, **c)["argmax"], out["argmax"])


@pytest.mark.parametrize("mask_value", [-32768.0, -math.inf, torch.finfo(BF).min, 0.0])
def test_process_masks(mask_value):
    logits, c = process_case(2, 4, 1031, 30, 5, "row", seed=7)
    c["mask"][0, 1] = 0            # leaves nothing
    c["mask"][0, 2] = -1           # leaves everything
    logits[1, 0, 100:120] = math.nan
    logits[1, 1, 100:110] = math.inf
    logits[1, 1, 110:120] = -math.inf
    c["mask"][1, :2, 3] = 0        # NaN and infinities of ids 96..127 are masked
    out = check_process(logits, c, mask_value=mask_value)
    assert (out["out"][0, 1].float() == torch.tensor(mask_value).to(BF).float().item()).all()
    assert out["argmax"][0, 1].item() == 0


def test_process_single_parts_and_nothing():
    logits, c = process_case(2, 5, 2000, 60, 4, "row", seed=8)
    hist = {k: c[k] for k in ("history", "hist_len", "prompt_len")}
    for part in ({}, hist, dict(hist, repetition=c["repetition"]), dict(hist, frequency=c["frequency"]),
                 dict(hist, presence=c["presence"]), dict(history=c["history"], presence=c["presence"]),
                 dict(node_tok=c["node_tok"], repetition=c["repetition"]),
                 dict(node_tok=c["node_tok"], parent=c["parent"], frequency=c["frequency"]),
                 dict(bias_tok=c["bias_tok"], bias_val=c["bias_val"]), dict(mask=c["mask"])):
        out = check_process(logits, part)
        if not part:
            assert torch.equal(out["out"], logits)


def test_process_padding_and_repeated_ids():
    logits, c = process_case(2, 4, 100, 12, 6, None, seed=9)
    c["history"][0, :] = -1
    c["history"][1, :] = 7
    c["node_tok"][:, 1] = -1
    c["node_tok"][:, 2:] = 7
    c["bias_tok"][0] = 7           # six biases on one id, added in order
    c["bias_tok"][1, :3] = -1
    check_process(logits, c)


def test_process_values_that_are_not_numbers():
    logits, _ = process_case(1, 3, 300, 0, 0, None, seed=10)
    logits[0, 0] = math.nan
    logits[0, 1, :200] = math.nan
    logits[0, 2] = -math.inf
    out = api.svd_logits_process(logits, argmax=True)
    assert torch.equal(out["out"].view(torch.int16), logits.view(torch.int16))
    assert out["argmax"].tolist()[0][0] == 0 and out["argmax"].tolist()[0][2] == 0
    assert out["argmax"][0, 1].item() == first_argmax(logits[0, 1]).item()
    zeros = torch.zeros((1, 1, 64), dtype=BF, device="cuda")
    zeros[0, 0, 5:] = -0.0
    assert api.svd_logits_process(zeros, argmax=True)["argmax"].item() == 0
    zeros[0, 0, :5] = -0.0
    zeros[0, 0, 9] = 0.0
    assert api.svd_logits_process(zeros, argmax=True)["argmax"].item() == 0


def shifted(t, by=1):
    """The same values at an address that is not 16-byte aligned."""
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    return buf[by:].view(t.shape).copy_(t)


def test_tensors_that_are_not_aligned():
    logits, c = process_case(3, 5, 2056, 40, 6, "row", seed=13)
    want = check_process(logits, c)
    got = check_process(shifted(logits), c, out=shifted(torch.empty_like(logits)))
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["argmax"], want["argmax"])
    dz = torch.randn((3, 5, 2056), generator=gen(3), device="cuda")
    g = {k: v for k, v in c.items() if k not in ("frequency", "presence")}
    a = api.svd_logits_process_grad(dz, logits, **g)["dlogits"]
    assert torch.equal(api.svd_logits_process_grad(shifted(dz), shifted(logits), **g)["dlogits"], a)
    tok = c["node_tok"]
    a, b = (api.svd_tree_verify(tok, logits=x, parent=c["parent"]) for x in (logits, shifted(logits)))
    assert all(torch.equal(a[k], b[k]) for k in a)
    t = attention_case([20], 2, 4, 2, 64, 16, seed=1)
    for name in ("q", "k_new", "cache_v"):
        x = {**t, name: shifted(t[name])}
        with pytest.raises(api.SvdError) as e:
            api.svd_tree_attention(*[x[k] for k in ("q", "k_new", "v_new", "cache_k", "cache_v", "page_table", "cache_len")])
        assert e.value.code == 2


def test_refused_tensors():
    """Types, shapes and strides that the entry points do not take."""
    t = attention_case([20, 30], 2, 4, 2, 64, 16, seed=1)
    names = ("q", "k_new", "v_new", "cache_k", "cache_v", "page_table", "cache_len")
    for name, bad in (("k_new", t["k_new"].half()), ("cache_k", t["cache_k"].float()), ("page_table", t["page_table"].long()),
                      ("cache_len", t["cache_len"][:1]), ("q", t["q"].transpose(1, 2)), ("v_new", t["v_new"][:, :1]),
                      ("cache_v", t["cache_v"].transpose(1, 2)), ("cache_v", t["cache_v"][:3]), ("cache_len", t["cache_len"].cpu())):
        with pytest.raises((TypeError, ValueError)):
            api.TreeAttention(*[{**t, name: bad}[k] for k in names])
    with pytest.raises(ValueError):
        api.TreeAttention(*[t[k] for k in names], parent=t["parent"][:1])
    for kw, code in ((dict(scale=math.inf), 1),):
        with pytest.raises(api.SvdError) as e:
            api.svd_tree_attention(*[t[k] for k in names], **kw)
        assert e.value.code == code
    wide = attention_case([20], 2, 2, 1, 136, 16, seed=1)
    with pytest.raises(api.SvdError) as e:
        api.svd_tree_attention(*[wide[k] for k in names])
    assert e.value.code == 6


def test_process_errors():
    logits, c = process_case(2, 4, 100, 12, 3, None, seed=11)
    for name, bad, code in (("history", 100, 7), ("history", -2, 7), ("node_tok", 100, 7), ("bias_tok", 100, 7), ("parent", 9, 9)):
        d = dict(c)
        d[name] = c[name].clone()
        d[name][1, 0] = bad
        d["hist_len"], d["prompt_len"] = ints([12, 12]), ints([6, 6])
        op = api.LogitsProcess(logits, **d)
        op()
        assert op.device_error() == code, name
    with pytest.raises(ValueError):
        api.LogitsProcess(logits, bias_tok=c["bias_tok"])
    with pytest.raises(ValueError):
        api.LogitsProcess(logits, mask=torch.zeros((2, 3, 4), dtype=I32, device="cuda"))
    with pytest.raises(ValueError):
        api.LogitsProcess(logits, values=False)
    with pytest.raises(ValueError):
        api.LogitsProcess(logits, prompt_len=c["prompt_len"])


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("B,n,V,S,mask", [(3, 5, 1024, 50, "row"), (1, 1, 1, 3, None), (2, 3, 7, 20, "seq"), (2, 64, 2049, 300, "row"),
                                          (2, 17, 4104, 0, "seq"), (1, 2, 151936, 2048, "row")])
def test_process_gradient(B, n, V, S, mask, dtype):
    logits, c = process_case(B, n, V, S, 0, mask, seed=B + n + V)
    logits[..., ::7] = 0           # the border of the repetition rule
    dz = torch.randn((B, n, V), generator=gen(1), device="cuda").to(dtype)
    c = {k: v for k, v in c.items() if k not in ("frequency", "presence")}
    op = api.LogitsProcessGrad(dz, logits, **c)
    got = op().outputs()["dlogits"]
    assert op.device_error() == 0
    want = R.process_grad(dz, logits, **c)
    # one fp32 operation and the rounding of the type
    tol = (2.0 ** -24 + torch.finfo(dtype).eps / 2) * want.abs()
    assert ((got.double() - want).abs() <= tol).all()
    same = dz.clone()
    api.svd_logits_process_grad(same, logits, out=same, **c)
    assert torch.equal(same, got)


def test_process_gradient_against_differences():
    """dL/dx of L = sum(w z(x)) against central differences of the 64-bit form, and the kernel's."""
    logits, c = process_case(2, 5, 100, 20, 0, "row", seed=12)
    logits = torch.where(logits.abs() < 0.1, torch.tensor(0.5, device="cuda", dtype=BF), logits)   # away from the border
    w = torch.randn((2, 5, 100), generator=gen(2), device="cuda")
    h = 2.0 ** -10
    zp, _ = R.process(logits.double() + h, **c)
    zm, _ = R.process(logits.double() - h, **c)
    diff = (zp - zm) / (2 * h) * w.double()
    g = {k: v for k, v in c.items() if k not in ("frequency", "presence")}
    got = api.svd_logits_process_grad(w, logits, **g)["dlogits"].double()
    # z is linear on either side of zero, so the differences are exact up to fp64 rounding / h
    assert ((got - diff).abs() <= 2.0 ** -22 * diff.abs() + 1e-10).all()


def test_process_streams_and_graph():
    cases = [process_case(4, 9, 5000, 200, 10, "row", seed=s) for s in (20, 21)]
    ops = [api.LogitsProcess(x, argmax=True, **c) for x, c in cases]
    want = [{k: v.clone() for k, v in op().outputs().items()} for op in ops]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for op, s in zip(ops, streams):
            op(s)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for op in ops:
            op()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for op, w in zip(ops, want):
        assert all(torch.equal(v, w[k]) for k, v in op.outputs().items())


# ------------------------------------------------------------------------------------------
# acceptance
# ------------------------------------------------------------------------------------------
def check_walk(out, y, node_tok, parent, n_nodes, n):
    paths, toks = R.verify(y, node_tok, parent, n_nodes)
    for b, (p, e) in enumerate(zip(paths, toks)):
        assert out["path"][b].tolist() == p + [-1] * (n - len(p))
        assert out["emitted"][b].tolist() == e + [-1] * (n - len(e))
        assert out["n_path"][b].item() == out["n_emitted"][b].item() == len(p)
        assert out["accept_len"][b].item() == max(0, len(p) - 1)


@pytest.mark.parametrize("B,n,V,kind", [(1, 1, 1, "chain"), (4, 9, 1024, "tree"), (7, 64, 333, "tree"), (3, 33, 8193, "star"),
                                        (40, 17, 1000, "chain"), (5, 40, 7, "tree"), (2, 12, 151936, "tree"), (9, 30, 64, "forest")])
def test_verify(B, n, V, kind):
    g = gen(B + n + V)
    T = torch.randn((B, n, V), generator=g, device="cuda").to(BF)
    T[..., V // 2:] = T[..., :V - V // 2]           # ties
    parent = R.random_tree(B, n, V, kind).cuda()
    y = first_argmax(T)
    rnd = torch.rand((B, n), generator=g, device="cuda")
    node_tok = torch.where(rnd < 0.8, y.gather(1, parent.clamp(min=0).long()),
                           torch.randint(0, V, (B, n), generator=g, device="cuda", dtype=I32)).to(I32)
    node_tok[rnd > 0.95] = -1
    nn = torch.randint(0, n + 1, (B,), generator=g, device="cuda", dtype=I32)
    for n_nodes in (None, nn):
        op = api.TreeVerify(node_tok, logits=T, parent=parent, n_nodes=n_nodes)
        for _ in range(2):
            out = op().outputs()
        assert op.device_error() == 0
        check_walk(out, y, node_tok, parent, n_nodes, n)
        used = torch.arange(n, device="cuda") < (n if n_nodes is None else n_nodes.view(B, 1))
        assert torch.equal(out["target_argmax"], torch.where(used, y, -1).to(I32))
        given = api.svd_tree_verify(node_tok, target_tok=y.contiguous(), parent=parent, n_nodes=n_nodes)
        assert all(torch.equal(given[k], out[k]) for k in out)


def test_verify_of_a_chain_is_svd_verify():
    B, k, V = 6, 8, 1024
    g = gen(3)
    T = torch.randn((B, k + 1, V), generator=g, device="cuda").to(BF)
    D = (T[:, :k].float() + 0.3 * torch.randn((B, k, V), generator=g, device="cuda")).to(BF)
    draft = first_argmax(D)
    ref = api.svd_verify(D, T, draft, ints([k] * B))
    tok = torch.cat([torch.zeros((B, 1), dtype=I32, device="cuda"), draft], 1)
    out = api.svd_tree_verify(tok, logits=T)
    assert torch.equal(out["accept_len"], ref["accept_len"])
    assert torch.equal(out["emitted"], ref["emitted"])
    assert torch.equal(out["n_emitted"], ref["n_emitted"])


def test_verify_errors():
    T = torch.randn((2, 6, 50), generator=gen(4), device="cuda").to(BF)
    tok = ints([[0, 1, 2, 3, 4, 5]] * 2)
    bad = tok.clone()
    bad[1, 3] = 50
    op = api.TreeVerify(bad, logits=T)
    op()
    assert op.device_error() == 7
    op = api.TreeVerify(tok, logits=T, parent=ints([[-1, 0, 2, 1, 0, -7]] * 2))
    op()
    assert op.device_error() == 9
    with pytest.raises(ValueError):
        api.TreeVerify(tok, logits=T, target_tok=tok)
    with pytest.raises(TypeError):
        api.TreeVerify(tok, logits=T.float())


# ------------------------------------------------------------------------------------------
# append
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("B,n,Hkv,D,page,use_path,inter", [(3, 17, 2, 64, 16, True, False), (1, 1, 1, 8, 1, False, False),
                                                           (5, 9, 8, 128, 5, True, True), (2, 300, 2, 96, 64, False, False),
                                                           (129, 4, 1, 72, 8, True, False)])
def test_append(B, n, Hkv, D, page, use_path, inter, dtype):
    g = gen(B + n)
    per = -(-(40 + n) // page)
    n_pages = B * per + 2
    buf = torch.randn((n_pages, 2, page, Hkv, D), generator=g, device="cuda").to(dtype)
    cache = [buf[:, 0], buf[:, 1]] if inter else [buf[:, 0].contiguous(), buf[:, 1].contiguous()]
    table = torch.randperm(n_pages, generator=g, device="cuda")[:B * per].to(I32).view(B, per)
    k, v = (torch.randn((B, n, Hkv, D), generator=g, device="cuda").to(dtype) for _ in range(2))
    k[0, 0], v[0, 0] = math.nan, math.inf                     # moved as they are
    lens = torch.randint(0, 41, (B,), generator=g, device="cuda", dtype=I32)
    count = torch.randint(0, n + 1, (B,), generator=g, device="cuda", dtype=I32)
    path = None
    if use_path:
        path = torch.argsort(torch.rand((B, n), generator=g, device="cuda"), 1).to(I32)
        path[torch.arange(n, device="cuda") >= count.view(B, 1)] = -1
    want = [c.clone() for c in cache]
    for b in range(B):
        for i in range(int(count[b])):
            node, pos = (i if path is None else int(path[b, i])), int(lens[b]) + i
            for w, x in zip(want, (k, v)):
                w[int(table[b, pos // page]), pos % page] = x[b, node]
    new = lens + count
    op = api.CacheAppend(k, v, *cache, table, lens, count, path=path, new_len=lens)   # the length in place
    op()
    assert op.device_error() == 0
    assert torch.equal(lens, new)
    for got, w in zip(cache, want):
        assert torch.equal(got.contiguous().view(torch.int16), w.contiguous().view(torch.int16))


def test_append_errors_skip_and_report():
    B, n, page = 2, 4, 4
    table = ints([[0, 1], [2, 3]])
    k = torch.ones((B, n, 1, 8), dtype=BF, device="cuda")

    def run(code, new_len=None, lens=(1, 2), count=(3, 4), path=None, table=table, written=None):
        c = [torch.zeros((4, page, 1, 8), dtype=BF, device="cuda") for _ in range(2)]
        op = api.CacheAppend(k, k, *c, table, ints(lens), ints(count), path=path)
        op()
        assert op.device_error() == code
        assert [int(x) for x in c[0].view(16, 8)[:, 0].nonzero()] == written
        assert torch.equal(c[0], c[1])
        if new_len:
            assert op.outputs()["new_len"].tolist() == new_len

    run(0, [4, 6], written=[1, 2, 3, 10, 11, 12, 13])
    run(8, [8, 6], lens=(7, 2), written=[7, 10, 11, 12, 13])                 # past the capacity
    run(8, [3, 6], lens=(-4, 2), written=[0, 1, 2, 10, 11, 12, 13])
    run(8, [4, 6], table=ints([[9, 1], [2, -1]]), written=[10, 11])          # bad pages
    run(9, [4, 6], path=ints([[0, 4, -1, 2], [0, 1, 2, 3]]), written=[1, 10, 11, 12, 13])
    run(9, [5, 2], count=(9, -1), written=[1, 2, 3, 4])


# ------------------------------------------------------------------------------------------
# together
# ------------------------------------------------------------------------------------------
def test_steps_of_tree_decoding():
    """Three steps as a server makes them: attention of the drafted tree, logits, grammar and penalties
    with the argmax, acceptance, append of the accepted path.  The cache must hold exactly the accepted
    tokens' keys and values, and a request's tokens must be those of decoding one token at a time."""
    B, n, Hq, Hkv, D, V, page, steps = 3, 13, 4, 2, 64, 160, 8, 3
    g = gen(77)
    f64 = torch.float64
    emb = torch.randn((V, Hkv * D * 2 + Hq * D), generator=g, device="cuda").to(BF)      # token -> q, k, v
    head = (torch.randn((Hq * D, V), generator=g, device="cuda") * 0.3).to(BF)
    mask = torch.full((B, 1, V // 32), -1, dtype=I32, device="cuda")
    mask[1, 0, 2] = 0x0f0f0f0f
    pen = dict(repetition=torch.tensor([1.0, 1.2, 1.1], device="cuda"), frequency=torch.tensor([0.0, 0.1, 0.5], device="cuda"),
               presence=torch.tensor([0.0, 0.3, 0.0], device="cuda"), mask=mask)
    kv = lambda tok: [x.contiguous() for x in (emb[tok][..., :Hkv * D].view(*tok.shape, Hkv, D),  # noqa: E731
                                               emb[tok][..., Hkv * D:2 * Hkv * D].view(*tok.shape, Hkv, D))]
    query = lambda tok: emb[tok][..., 2 * Hkv * D:].view(*tok.shape, Hq, D).contiguous()  # noqa: E731
    prompts = torch.randint(0, V, (B, 11), generator=g, device="cuda")
    cache = [torch.full((40, page, Hkv, D), math.nan, dtype=BF, device="cuda") for _ in range(2)]
    table = torch.randperm(40, generator=g, device="cuda")[:B * 10].to(I32).view(B, 10).contiguous()
    lens = torch.zeros(B, dtype=I32, device="cuda")
    # the prompt without its last token goes into the cache; that one is the root of the first tree
    pk, pv = kv(prompts[:, :10])
    api.svd_cache_append(pk, pv, *cache, table, lens, ints([10] * B), new_len=lens)
    said = prompts.tolist()
    for step in range(steps):
        parent = R.random_tree(B, n, 50 + step).cuda()
        tok = torch.randint(0, V, (B, n), generator=g, device="cuda")
        tok[:, 0] = torch.tensor([s[-1] for s in said], device="cuda")

        def target(tok):
            k, v = kv(tok)
            o = api.svd_tree_attention(query(tok), k, v, *cache, table, lens, parent=parent)["out"]
            logits = (o.view(B, n, Hq * D).float() @ head.float()).to(BF)
            hist = torch.full((B, 64), -1, dtype=I32, device="cuda")
            for b, s in enumerate(said):
                hist[b, :len(s) - 1] = torch.tensor(s[:-1], device="cuda")
            r = api.svd_logits_process(logits, history=hist, prompt_len=ints([11] * B), hist_len=ints([len(s) - 1 for s in said]),
                                       node_tok=tok.to(I32), parent=parent, argmax=True, **pen)
            return k, v, r, logits, hist

        # draft well: two rounds of setting half of the nodes to the target's choice at their parent
        for rnd in range(4):
            _, _, r, _, _ = target(tok)
            better = r["argmax"].gather(1, parent.clamp(min=0).long()).long()
            keep = torch.rand((B, n), generator=g, device="cuda") < 0.6
            keep[:, 0] = False
            tok = torch.where(keep, better, tok)
        k, v, r, logits, hist = target(tok)
        out = api.svd_tree_verify(tok.to(I32), target_tok=r["argmax"], parent=parent)
        whole = api.svd_tree_verify(tok.to(I32), logits=r["out"], parent=parent)
        assert all(torch.equal(out[x], whole[x]) for x in out)
        check_walk(out, r["argmax"], tok.to(I32), parent, None, n)
        api.svd_cache_append(k, v, *cache, table, lens, out["n_path"], path=out["path"], new_len=lens)
        for b in range(B):
            m = int(out["n_emitted"][b])
            # one token at a time, in 64 bits, over all that was said so far
            for i in range(m):
                seq = torch.tensor(said[b], device="cuda")
                sk, sv = kv(seq)
                qq = query(seq[-1:])[0].to(f64)
                o = torch.empty((Hq, D), dtype=f64, device="cuda")
                for h in range(Hq):
                    s = sk[:, h // 2].to(f64) @ qq[h] / 8.0
                    o[h] = torch.softmax(s, 0) @ sv[:, h // 2].to(f64)
                raw = o.to(BF).view(1, 1, -1).float() @ head.float()
                z, _ = R.process(raw.to(BF), history=seq.view(1, -1).to(I32), prompt_len=ints([11]),
                                 **{x: y[b:b + 1] for x, y in pen.items()})
                z = z.view(V)
                said_tok = int(out["emitted"][b, i])
                # the kernel's attention is within a bf16 step of this one, so is the logit: a choice within
                # the rounding of sum|o||head| of the best is the best
                slack = 2 * 2.0 ** -7 * (o.abs().view(-1) @ head.double().abs())[said_tok].item()
                assert z[said_tok] >= z.max() - slack
                said[b].append(said_tok)
    assert lens.tolist() == [len(s) - 1 for s in said]
    for b, s in enumerate(said):
        t = torch.arange(len(s) - 1, device="cuda")
        pg = table[b].long()[t // page]
        for c, x in zip(cache, kv(torch.tensor(s[:-1], device="cuda"))):
            assert torch.equal(c[pg, t % page], x)


def test_processed_logits_through_verify_and_distill():
    """A chain under a grammar: both rows processed, verified and distilled, and the gradient carried back
    to the drafter's raw logits; against autograd in 64 bits."""
    B, k, V = 2, 4, 512
    g = gen(5)
    T = (2 * torch.randn((B, k, V), generator=g, device="cuda")).to(BF)
    D = (T.float() + torch.randn((B, k, V), generator=g, device="cuda")).to(BF)
    c = dict(history=torch.randint(0, 60, (B, 30), generator=g, device="cuda", dtype=I32),
             node_tok=torch.randint(0, 60, (B, k), generator=g, device="cuda", dtype=I32),
             repetition=torch.tensor([1.3, 1.1], device="cuda"),
             mask=torch.randint(-2 ** 31, 2 ** 31, (B, k, V // 32), generator=g, device="cuda", dtype=torch.int64).to(I32))
    zd, zt = api.svd_logits_process(D, **c)["out"], api.svd_logits_process(T, **c)["out"]
    out = api.svd_verify_distill(zd, zt, bk_in=ints([k] * B), lam=0.5, clip_c=math.inf, dlogits_fp32=True)
    got = api.svd_logits_process_grad(out["dlogits"], D, **c)["dlogits"]
    _, seen = R.counts(B, k, V, c["history"], None, None, c["node_tok"], None, "cuda")
    ok = R.allowed(c["mask"], k, V)
    r = c["repetition"].double().view(B, 1, 1)
    x = D.double().requires_grad_(True)
    f = torch.where(seen, torch.where(x > 0, 1 / r, r), torch.ones_like(x))
    # the value that the distillation saw (rounded to bf16), the slope of the map
    z = torch.where(ok, zd.double() + (x * f - (x * f).detach()), torch.full_like(x, api.MASK_VALUE))
    lq, lp = torch.log_softmax(z, -1), torch.log_softmax(zt.double(), -1)
    y = first_argmax(zt).long().unsqueeze(-1)
    loss = (0.5 * -lq.gather(-1, y).squeeze(-1) + 0.5 * (lq.exp() * (lq - lp)).sum(-1)).sum()
    loss.backward()
    assert abs(out["loss_total"].item() - loss.item()) <= 1e-3 * abs(loss.item())
    assert ((got.double() - x.grad).abs() <= torch.clamp(1e-3 * x.grad.abs(), min=1e-5)).all()
    assert (got[~ok] == 0).all()
