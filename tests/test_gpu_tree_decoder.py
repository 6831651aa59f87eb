"""Steps of a decoder that checks drafted trees (GPU only): its launches one after the
other, each against the oracle on the library's own inputs of that stage, and
captured steps against eager ones.
"""

import numpy as np
import pytest
import torch

import bit_ptq_vla_amd as q
import oracle
from bit_ptq_vla_amd.workload import TreeDecoder
from test_gpu_kv_attention import Cache, f64, i32
from test_gpu_layer import check_norm, pull
from test_gpu_tree import check, make_sees, mask_words, random_parents

pytestmark = pytest.mark.gpu
DEV = "cuda"


def build(dtype="f16", **kw):
    args = dict(layers=2, batch=3, nodes=7, tokens=60, vocab=1000, dtype=dtype)
    args.update(kw)
    d = TreeDecoder(torch.device(DEV), **args)
    for c in d.stack.caches:                          # (a page needs no clearing: whatever it held)
        c.k.fill_(77)
        c.v.fill_(-77)
        c.k_scale.fill_(float("nan"))
        c.v_scale.fill_(float("nan"))
    g = np.random.default_rng(4)
    lengths = [9, 30, 1][:args["batch"]]
    d.prompt(i32(g.integers(0, args["vocab"], sum(lengths))), lengths)
    d.last.copy_(i32(g.integers(0, args["vocab"], args["batch"])))
    return d, lengths, g


def inputs(d, g):
    parents = np.concatenate([random_parents(d.nodes, g, wide=3) for _ in range(d.batch)])
    draft = g.integers(0, d.vocab, len(parents))
    draft[::d.nodes] = d.last.cpu().numpy()
    return parents, draft, g.random(len(parents)).astype(np.float32)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_steps_against_the_oracle(dtype):
    d, lengths, g = build(dtype)
    page, cols = 16, d.table.shape[1]
    pool = oracle.Pool(len(d.pool.refs), d.batch, cols, page)
    lens, _ = pool.resize([0] * d.batch, lengths)
    start = np.arange(0, d.batch * d.nodes + 1, d.nodes)
    sampling = dict(temperature=np.full(d.batch * d.nodes, 0.8, np.float32), top_p=np.full(d.batch * d.nodes, 0.9, np.float32))
    took = 0
    for t in range(5):
        parents, draft, u = inputs(d, g)
        if t >= 2:
            # drafts that come true: the step is run once to learn what is sampled behind each node
            keep = [x.clone() for x in [d.table, d.pool.refs, d.pool.free_bits, d.len, d.last]]
            held = [[x.clone() for x in (c.k, c.v, c.k_scale, c.v_scale)] for c in d.stack.caches]
            for _ in range(2):
                d.step(i32(parents), i32(draft), torch.from_numpy(u).to(DEV), **{n: torch.from_numpy(x).to(DEV) for n, x in sampling.items()})
                token = d.token.cpu().numpy()
                for b in range(d.batch):
                    s = slice(start[b], start[b + 1])
                    for i in range(1, d.nodes):
                        p = parents[s][i]
                        if 0 <= p < i and g.random() < 0.9:
                            draft[s][i] = token[s][p]
                for x, y in zip([d.table, d.pool.refs, d.pool.free_bits, d.len, d.last], keep):
                    x.copy_(y)
                for c, h in zip(d.stack.caches, held):
                    for x, y in zip((c.k, c.v, c.k_scale, c.v_scale), h):
                        x.copy_(y)
        grown, _ = pool.resize(lens, [n + d.nodes for n in lens])
        table = pool.table.copy()
        before = [pull(c) for c in d.stack.caches]
        compact = q.qlin_kv_compact
        seen = {}

        def spy(stack, batch, path, count, kv_len_out=None):
            torch.cuda.synchronize()
            seen["caches"] = [pull(c) for c in stack.caches]
            return compact(stack, batch, path, count, kv_len_out=kv_len_out)

        q.qlin_kv_compact = spy
        try:
            path, count, last = d.step(i32(parents), i32(draft), torch.from_numpy(u).to(DEV),
                                       **{n: torch.from_numpy(x).to(DEV) for n, x in sampling.items()})
        finally:
            q.qlin_kv_compact = compact
        torch.cuda.synchronize()
        sees = make_sees(parents, start, d.nodes)
        assert np.array_equal(d.mask.cpu().numpy(), mask_words(sees, 1))
        seq = np.repeat(np.arange(d.batch), d.nodes)
        positions = np.array(lens)[seq] + sees.sum(1) - 1
        assert np.array_equal(d.positions.cpu().numpy(), positions)
        # every layer's append at the nodes' places, turned by their depth, and attention by the mask
        for layer, was, now in zip(d.layers, before, seen["caches"]):
            m = d.batch * d.nodes
            oracle.rope_append_kv(f64(layer.qkv[:m]), was, table, start, grown, layer.heads, layer.rope.cpu().numpy(), 64, False,
                                  positions=positions)
            for name in ("k_scale", "v_scale", "k", "v"):
                assert np.array_equal(now[name], was[name], equal_nan=name.endswith("scale")), name
            c = Cache.__new__(Cache)
            c.host, c.cache = {n: np.nan_to_num(x) for n, x in now.items()}, layer.cache
            check(layer.ctx[:m], layer.qr[:m], c, table, start, np.array(grown), layer.heads, sees, 64 ** -0.5, 0.0, dtype)
        x = d.layers[-1].y[:m]
        check_norm(d.codes, *[torch.from_numpy(oracle.add_rmsnorm(f64(x), f64(d.residual), d.gamma.cpu().numpy(), 1e-6, dtype)[0]).to(x.dtype), x],
                   d.residual, d.gamma, dtype)
        logits, token = f64(d.logits), d.token.cpu().numpy()
        for r in range(m):
            want, lp, near = oracle.sample(logits[r], float(u[r]), temperature=float(np.float32(0.8)), top_p=float(np.float32(0.9)))
            assert near > 2.0 ** -38 and token[r] == want
        nodes = []
        for b in range(d.batch):
            s = slice(start[b], start[b + 1])
            want, new = oracle.tree_accept(parents[s], draft[s], token[s])
            assert path[b].tolist() == want + [-1] * (d.nodes - len(want)) and int(count[b]) == len(want) and int(last[b]) == new
            nodes.append(want)
            took += len(want)
        kept = oracle.kv_compact(seen["caches"], table, start, grown, nodes, [len(n) for n in nodes])
        for c, want in zip(d.stack.caches, seen["caches"]):
            now = pull(c)
            for name in ("k_scale", "v_scale", "k", "v"):
                assert np.array_equal(now[name], want[name], equal_nan=name.endswith("scale")), name
        lens, _ = pool.resize(grown, kept)
        assert d.len.tolist() == lens
        assert np.array_equal(d.table.cpu().numpy(), pool.table) and np.array_equal(d.pool.refs.cpu().numpy(), pool.refs)
    assert took > 5 * d.batch                       # (some drafts were taken)


def test_captured_steps():
    a, _, ga = build()
    b, _, gb = build()
    n = a.batch * a.nodes
    parents, draft, u = (torch.zeros(n, dtype=torch.int32, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV),
                         torch.zeros(n, device=DEV))
    a.layers[0].workspace(n), a.layers[1].workspace(n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(parents, draft, u)
    for t in range(6):
        p, d, r = inputs(b, gb)
        want = [x.clone() for x in b.step(i32(p), i32(d), torch.from_numpy(r).to(DEV))]
        parents.copy_(i32(p))
        draft.copy_(i32(d))
        u.copy_(torch.from_numpy(r))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a.path, want))
        assert torch.equal(a.len, b.len) and torch.equal(a.table, b.table) and torch.equal(a.pool.free_bits, b.pool.free_bits)
        for x, y in zip(a.stack.caches, b.stack.caches):
            for i in range(a.batch):
                held = a.table[i, :-(-int(a.len[i]) // 16)].long()
                assert torch.equal(x.k_scale[held], y.k_scale[held]) and torch.equal(x.k[held], y.k[held])


def test_layer_with_a_chain_is_the_layer_without_a_tree():
    """A tree that is a chain, against the same tokens without one: the same codes in the
    cache, and attention within two roundings of its output."""
    a, _, _ = build(layers=1)
    b, _, _ = build(layers=1)
    n = a.batch * a.nodes
    x = torch.randn((n, a.hidden), device=DEV).to(a.embed.dtype)
    chain = i32(np.tile(np.arange(a.nodes) - 1, a.batch))
    for d in (a, b):
        d.want.copy_(d.len + d.nodes)
        q.qlin_kv_resize(d.pool, d.stack, d.table, d.len, d.want, len_out=d.grown)
    mask, positions = q.qlin_tree_plan(chain, a.kv)
    a.layers[0].step(x, torch.zeros_like(x), a.kv, tree=(mask, positions))
    b.layers[0].step(x, torch.zeros_like(x), b.kv)
    torch.cuda.synchronize()
    assert torch.equal(a.stack.caches[0].k, b.stack.caches[0].k) and torch.equal(a.layers[0].qr[:n], b.layers[0].qr[:n])
    assert torch.allclose(a.layers[0].ctx[:n].float(), b.layers[0].ctx[:n].float(), rtol=2.0 ** -10, atol=1e-3)


def held_tokens(d, b):
    """What the caches hold of sequence b's tokens: codes times scales, exactly as stored."""
    n, out = int(d.len[b]), []
    pages = d.table[b, :-(-n // 16)].long()
    for c in d.stack.caches:
        out += [c.k[pages].transpose(1, 2).flatten(0, 1)[:n].clone(), c.k_scale[pages].clone(),
                c.v[pages].permute(0, 3, 1, 2).flatten(0, 1)[:n].clone(), c.v_scale[pages].clone()]
    return out


@pytest.mark.parametrize("captured", [False, True])
def test_sequences_without_room_stay_as_they_are(captured):
    """Steps up to and past the end of the first row's pages, and without free pages: the
    sequences that do not get them take no token and keep what they hold, the others go on."""
    d = TreeDecoder(torch.device(DEV), layers=2, batch=3, nodes=7, tokens=60, vocab=1000, dtype="f16")
    g = np.random.default_rng(12)
    d.prompt(i32(g.integers(0, d.vocab, 93)), [60, 32, 1])
    d.last.copy_(i32(g.integers(0, d.vocab, 3)))
    n = d.batch * d.nodes
    args = (torch.zeros(n, dtype=torch.int32, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV), torch.zeros(n, device=DEV))
    step = lambda: d.step(*args)  # noqa: E731
    if captured:
        for layer in d.layers:
            layer.workspace(n)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            d.step(*args)
        step = lambda: graph.replay() or d.path  # noqa: E731
    room = d.table.shape[1] * 16
    stayed = went = 0
    for t in range(30):
        parents, draft, u = inputs(d, g)
        for x, y in zip(args, (i32(parents), i32(draft), torch.from_numpy(u).to(DEV))):
            x.copy_(y)
        none_free = t >= 26
        if none_free:                                  # (as if other rows held them)
            d.pool.free_bits.zero_()
        lens, last, table = d.len.tolist(), d.last.tolist(), d.table.clone()
        before = [held_tokens(d, b) for b in range(d.batch)]
        path, count, token = step()
        torch.cuda.synchronize()
        for b in range(d.batch):
            fits = lens[b] + d.nodes <= room and not (none_free and -(-(lens[b] + d.nodes) // 16) > -(-lens[b] // 16))
            took = int(count[b])
            assert (took > 0) == fits, (t, b)
            assert int(d.len[b]) == lens[b] + took
            pages = -(-lens[b] // 16)
            if fits:
                went += 1
                assert path[b, :1].tolist() == [0] and torch.all(path[b, took:] == -1)
            else:
                stayed += 1
                assert torch.all(path[b] == -1) and int(token[b]) == last[b]
                assert torch.equal(d.table[b], table[b])
                assert all(torch.equal(x, y) for x, y in zip(held_tokens(d, b), before[b])), (t, b)
            assert torch.equal(d.table[b, :pages], table[b, :pages]) and torch.all(d.table[b, -(-int(d.len[b]) // 16):] == -1)
    assert stayed > 8 and went > 40


def test_prompts_past_the_room_are_refused():
    d = TreeDecoder(torch.device(DEV), layers=1, batch=2, nodes=3, tokens=20, vocab=1000)
    tokens = i32(np.arange(30))
    for lengths in ([21, 9], [30], [10, 10], [31, -1], [10, 10, 10]):
        with pytest.raises(ValueError, match="prompt"):
            d.prompt(tokens, lengths)
    d.prompt(tokens, [20, 10])
    assert d.len.tolist() == [20, 10]
