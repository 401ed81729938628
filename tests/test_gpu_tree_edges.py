"""Edges of the operators on a tree of drafts: very small softmax weights, values that are not finite
across parts, padding, streams, captured calls, and workspaces between calls."""
import math

import pytest
import torch

from speculative_decoding_verify_distill_b200 import api
from tests import tree_ref as R
from tests.test_gpu_tree_ops import (BF, FP, I32, attention_case, check_attention, first_argmax, gen, ints,
                                     process_case)

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]
ATT = ("q", "k_new", "v_new", "cache_k", "cache_v", "page_table", "cache_len")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_verify_distill_b200 import build
    build.build()


def copies(op):
    return {k: v.clone() for k, v in op.outputs().items()}


def same_bits(a, b):
    view = {2: torch.int16, 4: torch.int32}
    return all(torch.equal(v.view(view[v.element_size()]), b[k].view(view[v.element_size()])) for k, v in a.items())


# ------------------------------------------------------------------------------------------
# attention
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("B", [148, 1])
@pytest.mark.parametrize("gap", [8.0, 12.0, 14.0, 16.0, 17.5, 19.0])
def test_attention_one_large_weight_and_a_long_tail(gap, B, dtype):
    """One key takes nearly all of the weight and 32767 others share e^-gap each: what they add up to must not
    be lost where a weight is rounded to 16 bits.  All sequences read the same pages, so that with 148 of
    them a whole sequence is one part.

    A weight 2^z, relative to the row's largest, goes into the product as 2^(z + 7) in fp16: it is off by half a step
    (2^-11 of itself), or by half of the smallest step, 2^-25, which is 2^-32 of the largest weight; in bf16 by
    half a step alone (2^-8).  Scores are exact here; exp2 and the scaling to base 2 are off by
    e = 2^-21 + 2^-22 gap, the sum over T keys by T 2^-24 of itself, and the result is rounded once."""
    L, D, page = 32768, 64, 128
    dev = "cuda"
    k, v = torch.zeros((L, D), device=dev), torch.randn((L, D), generator=gen(31), device=dev).abs() + 0.25
    k[1:, 0] = -gap
    v[0] = 0
    q = torch.zeros((B, 1, 1, D), device=dev)
    q[..., 0] = 1
    k_new, v_new = torch.zeros((B, 1, 1, D), device=dev), torch.ones((B, 1, 1, D), device=dev)
    k_new[..., 0] = -gap
    k, v, q, k_new, v_new = (x.to(dtype) for x in (k, v, q, k_new, v_new))
    table = torch.arange(L // page, device=dev, dtype=I32).expand(B, -1).contiguous()
    op = api.TreeAttention(q, k_new, v_new, k.view(-1, page, 1, D), v.view(-1, page, 1, D), table,
                           torch.full((B,), L, dtype=I32, device=dev), scale=1.0, lse=True)
    out = op().outputs()
    assert op.device_error() == 0
    w = torch.exp(torch.cat([k[:, 0], k_new[0, 0, 0, :1]]).double())
    vv = torch.cat([v, v_new[0, 0]]).double()
    l, T = w.sum(), L + 1
    want, mag = w @ vv / l, w @ vv.abs() / l
    u, e = torch.finfo(dtype).eps / 2, 2.0 ** -21 + 2.0 ** -22 * gap
    small = 2.0 ** -32 if dtype == FP else 0.0
    out_step = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    tol = u * want + mag * (u + 2 * e + T * 2.0 ** -24) + small * vv.abs().sum(0) / l + out_step
    got = out["out"].double().view(B, D)
    assert ((got - want).abs() <= tol).all(), ((got - want).abs() / want).max().item()
    assert ((out["lse"].double() - l.log()).abs() <= 2 * e + T * 2.0 ** -24 + 2.0 ** -22 * l.log().abs()).all()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("L,B", [(100, 1), (100, 148), (700, 1), (20000, 1)])
def test_attention_infinite_drafted_value_far_below_the_maximum(L, B, bad, dtype):
    """A drafted value that is not finite reaches the rows that see its node, however small the node's weight is and
    however the sequence was cut into parts (148 short ones are a part each): the scores of all cached keys but the
    last 300 lie 200 above."""
    c = attention_case([L] * B, 3, 2, 1, 64, 16, dtype, seed=32, kind="chain")
    c["page_table"][:] = c["page_table"][0].clone()
    t = torch.arange(L, device="cuda")
    c["q"], c["k_new"] = torch.zeros_like(c["q"]), torch.zeros_like(c["k_new"])
    c["q"][..., 0] = 20
    k = torch.zeros((L, 1, 64), device="cuda")
    k[:max(1, L - 300), 0, 0] = 10
    c["cache_k"][c["page_table"][0].long()[t // 16], t % 16] = k.to(dtype)
    clean = copies(check_attention(c, scale=1.0))
    assert (clean["lse"] >= 199).all()
    c["v_new"] = c["v_new"].clone()
    c["v_new"][:, 1, 0, 5:40] = bad
    op = api.TreeAttention(*[c[x] for x in ATT], parent=c["parent"], scale=1.0, lse=True)
    out = op().outputs()
    assert op.device_error() == 0
    assert torch.equal(out["lse"], clean["lse"])
    hit = torch.zeros((B, 3, 2, 64), dtype=torch.bool, device="cuda")
    hit[:, 1:, :, 5:40] = True
    assert torch.equal(out["out"][~hit], clean["out"][~hit])
    got = out["out"][hit].float()
    assert got.isnan().all() if math.isnan(bad) else (got == bad).all()


def test_attention_parents_of_padding_nodes_are_not_read():
    """What lies behind n_nodes may be anything, the parents too; a parent out of range of a node in use is recorded."""
    c = attention_case([50, 0, 300, 20], 40, 8, 2, 64, 16, seed=33)
    nn = ints([40, 33, 5, 0])
    want = copies(check_attention(c, n_nodes=nn))
    for b, m in enumerate(nn.tolist()):
        c["parent"][b, m:] = 1 << 20
        c["parent"][b, m + 1:] = -7
    assert same_bits(check_attention(c, n_nodes=nn).outputs(), want)
    c["parent"][1, 32] = 33
    op = api.TreeAttention(*[c[x] for x in ATT], parent=c["parent"], n_nodes=nn)
    op()
    assert op.device_error() == 9


@pytest.mark.parametrize("n,Hq,Hkv,D,page,dtype", [(1, 4, 1, 128, 16, BF), (33, 8, 2, 64, 64, FP), (64, 16, 2, 128, 32, BF)])
def test_attention_of_parts_that_end_on_either_warpgroup(n, Hq, Hkv, D, page, dtype):
    """Lengths at which parts hold one, two, three or more tiles, an odd or an even number: the results are right and the
    same in every repeat."""
    for lens in ([148 * 128 * k + d for k, d in ((1, 0), (1, -128), (2, 100), (3, 1))],
                 [128 * i + 5 for i in range(9)] * 4, [4096] * 37):
        if n > 1:
            lens = [x // 4 for x in lens]
        c = attention_case(lens[:2] if n > 1 and max(lens) > 5000 else lens, n, Hq, Hkv, D, page, dtype, seed=34)
        if n > 1 and len(c["cache_len"]) > 4:
            op = api.TreeAttention(*[c[x] for x in ATT], parent=c["parent"], lse=True)()
        else:
            op = check_attention(c)
        first = copies(op)
        for _ in range(30):
            op()
        assert same_bits(op.outputs(), first)
        assert op.device_error() == 0


# ------------------------------------------------------------------------------------------
# workspaces, streams and graphs
# ------------------------------------------------------------------------------------------
def handles():
    """An object of every operator whose workspace holds keys or tickets between its blocks."""
    logits, c = process_case(4, 9, 5000, 200, 10, "row", seed=40)
    g = gen(41)
    T = torch.randn((3, 12, 20000), generator=g, device="cuda").to(BF)
    parent = R.random_tree(3, 12, 41).cuda()
    y = first_argmax(T)
    tok = torch.where(torch.rand((3, 12), generator=g, device="cuda") < 0.8, y.gather(1, parent.clamp(min=0).long()), 0).to(I32)
    k, v = (torch.randn((5, 21, 2, 64), generator=g, device="cuda").to(BF) for _ in range(2))
    cache = [torch.zeros((5 * 8, 8, 2, 64), dtype=BF, device="cuda") for _ in range(2)]
    table = torch.randperm(40, generator=g, device="cuda").to(I32).view(5, 8)
    return [api.LogitsProcess(logits, argmax=True, **c), api.LogitsProcess(logits, argmax=True, values=False, **c),
            api.TreeVerify(tok, logits=T, parent=parent),
            api.CacheAppend(k, v, *cache, table, ints([0, 3, 17, 8, 43]), ints([21, 0, 13, 5, 1]))]


def wipe(op):
    for t in op.outputs().values():
        t.view(torch.int16 if t.element_size() == 2 else torch.int32).fill_(0x55)


def wiped_cache(op):
    """The cache keeps what a call does not write."""
    if isinstance(op, api.CacheAppend):
        op.cache_k.zero_()
        op.cache_v.zero_()


@pytest.mark.parametrize("which", range(4))
def test_workspace_is_ready_after_every_call_and_after_a_reset(which):
    """Behind the header everything is zero again after a call.  Keys and tickets that were left by a call that did not end
    spoil the next one, until the workspace is reset."""
    op = handles()[which]
    want = copies(op())
    assert op.device_error() == 0 and not op.ws[256:].any()
    op.ws[:4] = 5                      # a recorded time-out
    op.ws[256:] = 1                    # ... and counts of blocks that had already run
    assert op.reset() is op
    assert not op.ws.any() and op.device_error() == 0
    for _ in range(3):
        wipe(op)
        wiped_cache(op)
        op()
        assert same_bits(op.outputs(), want)
    assert op.device_error() == 0 and not op.ws[256:].any()


@pytest.mark.parametrize("which", range(4))
def test_streams_and_captured_calls(which):
    """Two objects on two streams at once, then both captured into a graph and replayed: every output is written
    again, with the bits of the first call."""
    ops = [handles()[which] for _ in range(2)]
    want = [copies(op()) for op in ops]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for op in ops:
        wipe(op)
        wiped_cache(op)
    torch.cuda.synchronize()
    for _ in range(5):
        for op, s in zip(ops, streams):
            op(s)
    torch.cuda.synchronize()
    for op, w in zip(ops, want):
        assert same_bits(op.outputs(), w) and op.device_error() == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for op in ops:
            op()
    for _ in range(3):
        for op in ops:
            wipe(op)
            wiped_cache(op)
        graph.replay()
        torch.cuda.synchronize()
        for op, w in zip(ops, want):
            assert same_bits(op.outputs(), w)
    for op in ops:
        assert op.device_error(torch.cuda.current_stream()) == 0 and not op.ws[256:].any()


def test_gradient_streams_and_captured_calls():
    logits, c = process_case(4, 9, 5000, 200, 0, "row", seed=42)
    c = {k: v for k, v in c.items() if k not in ("frequency", "presence")}
    for dtype in (BF, torch.float32):
        dz = torch.randn(logits.shape, generator=gen(43), device="cuda").to(dtype)
        op = api.LogitsProcessGrad(dz, logits, **c)
        want = copies(op())
        wipe(op)
        torch.cuda.synchronize()
        op(torch.cuda.Stream())
        torch.cuda.synchronize()
        assert same_bits(op.outputs(), want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            op()
        wipe(op)
        graph.replay()
        torch.cuda.synchronize()
        assert same_bits(op.outputs(), want) and op.device_error() == 0


def test_one_call_on_a_stream_keeps_its_inputs():
    """Tensors that nobody else holds are not handed out again before the call on the side stream has read them."""
    logits, c = process_case(2, 8, 100000, 50, 4, "row", seed=44)
    want = copies(api.LogitsProcess(logits, argmax=True, **c)())
    t = attention_case([500, 90], 4, 8, 2, 128, 16, seed=45)
    att = copies(api.TreeAttention(*[t[x] for x in ATT], parent=t["parent"])())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        a, b = logits.clone(), {k: t[k].clone() for k in ATT[:5]}
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(50_000_000)
        got = api.svd_logits_process(a, stream=side, argmax=True, **c)
        out = api.svd_tree_attention(*b.values(), t["page_table"], t["cache_len"], parent=t["parent"], stream=side)
        del a, b
        # as large as what was let go, and filled before the side stream gets to its calls
        spoil = [torch.full_like(logits, 77.0)] + [torch.full_like(t[k], 1) for k in ATT[:5]]
        torch.cuda.synchronize()
        assert same_bits(got, want) and same_bits(out, att)
        del spoil


def test_attention_infinite_keys():
    """A drafted key with an infinite element: a row that sees it with the score -inf is as if the node were not
    there, one with the score +inf is not a number (inf - inf in every softmax)."""
    c = attention_case([50, 0, 300], 12, 8, 2, 64, 16, seed=35)
    c["q"][..., 0] = 1.0
    par = c["parent"].tolist()
    k_new = c["k_new"].clone()
    k_new[:, 4, :, 0] = -math.inf
    run = lambda k: api.svd_tree_attention(c["q"], k, *[c[x] for x in ATT[2:]], parent=c["parent"], lse=True)  # noqa: E731
    clean, low = run(c["k_new"]), run(k_new)
    k_new[:, 4, :, 0] = math.inf
    high = run(k_new)
    for b in range(3):
        for j in range(12):
            anc = R.ancestors(par[b], j)
            if 4 not in anc:
                for got in (low, high):
                    assert torch.equal(got["out"][b, j], clean["out"][b, j]) and torch.equal(got["lse"][b, j], clean["lse"][b, j])
                continue
            assert high["out"][b, j].isnan().all() and high["lse"][b, j].isnan().all()
            # the row alone, over the cache and a chain of the other nodes it sees
            rest = [i for i in anc if i != 4]
            one = lambda t: t[b:b + 1, rest].contiguous()  # noqa: E731
            o, l, to, tl = R.attention(c["q"][b:b + 1, [j] * len(rest)], one(c["k_new"]), one(c["v_new"]), c["cache_k"], c["cache_v"],
                                       c["page_table"][b:b + 1], c["cache_len"][b:b + 1])
            assert ((low["out"][b, j].double() - o[0, -1]).abs() <= to[0, -1]).all()
            assert ((low["lse"][b, j].double() - l[0, -1]).abs() <= tl[0, -1]).all()


@pytest.mark.parametrize("dtype", [BF, FP])
def test_attention_parts_of_many_sequences_of_differing_lengths(dtype):
    """More sequences in a part than a part keeps lengths of, each of its own length (n = 1, one head, so the plain form
    is one batched product)."""
    B, D, page, per = 12011, 64, 8, 20
    g = gen(36)
    lens = torch.randint(0, per * page + 1, (B,), generator=g, device="cuda", dtype=I32)
    cache = torch.randn((2, 4096, page, 1, D), generator=g, device="cuda").to(dtype)
    table = torch.randint(0, 4096, (B, per), generator=g, device="cuda", dtype=I32)
    q, k, v = (torch.randn((B, 1, 1, D), generator=g, device="cuda").to(dtype) for _ in range(3))
    op = api.TreeAttention(q, k, v, cache[0], cache[1], table, lens, lse=True)
    out = op().outputs()
    assert op.device_error() == 0
    u, tiny = torch.finfo(dtype).eps / 2, torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    for at in range(0, B, 1001):
        s = slice(at, at + 1001)
        kk, vv = (torch.cat([cache[x][table[s].long()].view(-1, per * page, D), y[s, 0]], 1).double() for x, y in ((0, k), (1, v)))
        hide = torch.arange(per * page, device="cuda") >= lens[s].view(-1, 1)
        hide = torch.cat([hide, torch.zeros_like(hide[:, :1])], 1)
        z = (kk @ q[s, 0].double().transpose(1, 2)).squeeze(2) / 8
        mag = ((kk.abs() @ q[s, 0].double().abs().transpose(1, 2)).squeeze(2) / 8).masked_fill(hide, 0).amax(1, keepdim=True)
        big = z.masked_fill(hide, 0).abs().amax(1, keepdim=True)
        p = torch.softmax(z.masked_fill(hide, -math.inf), 1)
        want, spread = ((p.unsqueeze(1) @ x).squeeze(1) for x in (vv, vv.abs()))
        lse = torch.logsumexp(z.masked_fill(hide, -math.inf), 1, keepdim=True)
        e = 2.0 ** -23 * D * mag + 2.0 ** -22 * big + 2.0 ** -21
        T = per * page + 1
        tol = u * want.abs() + spread * (u + 2 * e + T * 2.0 ** -24) + tiny * (1 + T * vv.abs().amax(1))
        assert ((out["out"][s].view(-1, D).double() - want).abs() <= tol).all()
        assert ((out["lse"][s].view(-1, 1).double() - lse).abs() <= 2 * e + T * 2.0 ** -24 + 2.0 ** -22 * lse.abs()).all()


# ------------------------------------------------------------------------------------------
# together
# ------------------------------------------------------------------------------------------
def test_a_captured_step_of_tree_decoding():
    """Attention, logits, processing, acceptance and append as one graph, with the lengths updated in place, replayed over four
    steps of new drafts: the tokens, lengths and cache of eager calls, bit for bit."""
    B, n, Hq, Hkv, D, V, page, steps = 4, 12, 4, 2, 64, 512, 8, 4
    g = gen(50)
    emb = torch.randn((V, (2 * Hkv + Hq) * D), generator=g, device="cuda").to(BF)
    head = (torch.randn((Hq * D, V), generator=g, device="cuda") * 0.3).to(BF)
    parent = R.random_tree(B, n, 50).cuda()
    drafts = torch.randint(0, 40, (steps, B, n), generator=g, device="cuda", dtype=I32)
    prompt = torch.randn((2, B, 30, Hkv, D), generator=g, device="cuda").to(BF)
    nn = ints([12, 7, 1, 12])

    class Server:
        def __init__(self):
            self.cache = [torch.zeros((B * 16, page, Hkv, D), dtype=BF, device="cuda") for _ in range(2)]
            self.table = torch.arange(B * 16, device="cuda", dtype=I32).flip(0).view(B, 16).contiguous()
            self.lens = torch.zeros(B, dtype=I32, device="cuda")
            api.svd_cache_append(*prompt, *self.cache, self.table, self.lens, ints([30, 9, 0, 24]), new_len=self.lens)
            self.tok = torch.zeros((B, n), dtype=I32, device="cuda")

        def step(self):
            x = emb[self.tok.long()].view(B, n, 2 * Hkv + Hq, D)
            q, k, v = (y.contiguous() for y in (x[:, :, 2 * Hkv:], x[:, :, :Hkv], x[:, :, Hkv:2 * Hkv]))
            o = api.svd_tree_attention(q, k, v, *self.cache, self.table, self.lens, parent=parent, n_nodes=nn)["out"]
            z = api.svd_logits_process(o.view(B, n, -1) @ head, node_tok=self.tok, parent=parent, argmax=True,
                                       frequency=torch.full((B,), 0.5, device="cuda"))
            walk = api.svd_tree_verify(self.tok, target_tok=z["argmax"], parent=parent, n_nodes=nn)
            api.svd_cache_append(k, v, *self.cache, self.table, self.lens, walk["n_path"], path=walk["path"], new_len=self.lens)
            return dict(walk, z=z["out"], o=o)

    def draft(s, i, choice):
        """Half of the nodes carry what the target said a step before at their parent."""
        s.tok.copy_(drafts[i])
        if choice is not None:
            s.tok[:, ::2] = choice.gather(1, parent.clamp(min=0).long())[:, ::2]

    eager, seen = Server(), []
    for i in range(steps):
        draft(eager, i, seen[-1]["target_argmax"].clamp(min=0) if seen else None)
        seen.append({k: v.clone() for k, v in eager.step().items()})
    server = Server()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = server.step()
    choice = None
    for i in range(steps):
        draft(server, i, choice)
        graph.replay()
        assert same_bits(out, seen[i])
        choice = out["target_argmax"].clamp(min=0)
    assert torch.equal(server.lens, eager.lens)
    assert all(torch.equal(a, b) for a, b in zip(server.cache, eager.cache))
    assert eager.lens.tolist()[2] == steps          # a root alone is accepted in every step
