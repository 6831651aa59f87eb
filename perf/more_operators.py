"""Decoding with drafted tokens over the paged int8 cache, as measured cases.

One step of a decoder that checks a tree of drafted tokens in each sequence,
and the parallel continuations of one prompt, take five operators:

  tree     attention of a tree of drafted tokens over the cache: each sees the
           cached tokens, its ancestors among the new ones, and itself;
  sample   a token from each row of logits: temperature, min-p, top-k, top-p,
           and a given random number;
  verify   the tree's masks and rotary positions from its parents, and the path
           of drafted tokens that the sampled ones confirm;
  compact  the keys and values of that path moved to the end of the sequence,
           under page scales, in every layer's cache;
  fork     rows of the page table that share their pages, the growth of a row
           (new pages; a last page shared with others is copied), and the
           return of its pages.

A plain form in elementary torch operations stands beside the library's own
calls (own).  Cache layout: k [layers][pages][heads][page][d], v
[layers][pages][heads][d][page] int8, k_scale, v_scale [layers][pages][heads]
float32.  Sequence b's token j lies in page page_table[b][j // page] at
j % page; its new tokens are its last ones.  A node's parent is the index of an
earlier node of its sequence, or -1; node 0 is the last token already taken.
"""

import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}

# the largest amounts of work any case has, listed or drawn
TREE_CACHE = 64 * 4096 * 8 * 128           # padded values of the keys
TREE_PAIRS = 4 * 256 * 16384 * 32          # padded (node, key, head) triples
SAMPLE_VALUES = 256 * 257152
COMPACT_VALUES = 64 * 8 * 16 * 8 * 128     # (moved tokens x layers) x heads x d
FORK_VALUES = 128 * 16 * 64 * 8 * 128      # (children x layers) x page x heads x d
VERIFY_NODES = 64 * 256


def listed():
    return [
        # 16 drafted tokens of one request of a 7B decoder behind 816 cached ones: latency
        {"name": "tree_one", "op": "tree", "dtype": "f16", "batch": 1, "nodes": 16, "ctx": 816, "ragged": False,
         "hq": 32, "hkv": 32, "d": 128, "page": 16, "cap": 0.0},
        # 64 requests at different lengths, up to 16 nodes each, four query heads to a key head: bandwidth
        {"name": "tree_batch", "op": "tree", "dtype": "bf16", "batch": 64, "nodes": 16, "ctx": 4080, "ragged": True,
         "hq": 32, "hkv": 8, "d": 128, "page": 32, "cap": 0.0},
        # wide trees over long caches, capped: the matrix units
        {"name": "tree_wide", "op": "tree", "dtype": "bf16", "batch": 4, "nodes": 256, "ctx": 16100, "ragged": True,
         "hq": 32, "hkv": 8, "d": 128, "page": 64, "cap": 30.0},
        # the next token of one request: latency
        {"name": "sample_one", "op": "sample", "dtype": "f16", "rows": 1, "vocab": 32000, "filters": "p"},
        # the nodes of 64 trees, each request with its own settings
        {"name": "sample_trees", "op": "sample", "dtype": "bf16", "rows": 1024, "vocab": 32003, "filters": "all"},
        # a large vocabulary in fp32, 256 requests that set a temperature only: bandwidth
        {"name": "sample_large", "op": "sample", "dtype": "f32", "rows": 256, "vocab": 257152, "filters": "none"},
        # one tree, and 64 wide ones
        {"name": "verify_one", "op": "verify", "batch": 1, "nodes": 16, "ragged": False},
        {"name": "verify_batch", "op": "verify", "batch": 64, "nodes": 256, "ragged": True},
        # one request, 32 layers of 32 heads: five nodes of sixteen taken
        {"name": "compact_one", "op": "compact", "layers": 32, "batch": 1, "nodes": 16, "taken": 5, "ctx": 100,
         "ragged": False, "hkv": 32, "d": 128, "page": 16},
        # 64 requests
        {"name": "compact_batch", "op": "compact", "layers": 16, "batch": 64, "nodes": 32, "taken": 8, "ctx": 120,
         "ragged": True, "hkv": 8, "d": 128, "page": 32},
        # four continuations of one prompt: a page of each layer copied for each
        {"name": "fork_one", "op": "fork", "layers": 8, "parents": 1, "children": 4, "ctx": 820, "grow": 16,
         "hkv": 32, "d": 128, "page": 16},
        # eight continuations of sixteen prompts: bandwidth
        {"name": "fork_batch", "op": "fork", "layers": 16, "parents": 16, "children": 8, "ctx": 1000, "grow": 16,
         "hkv": 8, "d": 128, "page": 64},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["tree", "tree", "sample", "sample", "verify", "compact", "fork"])
    d = rng.choice([64, 128, 256])
    page = rng.choice([16, 32, 64])
    hkv = rng.choice([1, 2, 4, 8, 16, 32])
    batch = _log_int(rng, 1, 64)
    nodes = _log_int(rng, 1, 256)
    ragged = rng.random() < 0.7
    if op == "tree":
        hkv = min(hkv, 16)
        hq = hkv * rng.choice([g for g in (1, 2, 4, 8) if g * hkv <= 32])
        ctx = rng.choice([0, _log_int(rng, 1, 16384), _log_int(rng, 64, 16384)])
        while batch > 1 and (batch * nodes * (nodes + ctx) * hq > TREE_PAIRS or batch * (nodes + ctx) * hkv * d > TREE_CACHE):
            batch //= 2
        return {"op": "tree", "dtype": rng.choice(["f16", "bf16"]), "batch": batch, "nodes": nodes, "ctx": ctx,
                "ragged": ragged, "hq": hq, "hkv": hkv, "d": d, "page": page, "cap": rng.choice([0.0, 0.0, 30.0])}
    if op == "sample":
        vocab = _log_int(rng, 300, 257152)
        rows = _log_int(rng, 1, min(1024, SAMPLE_VALUES // vocab))
        return {"op": "sample", "dtype": rng.choice(["f16", "bf16", "f32"]), "rows": rows, "vocab": vocab,
                "filters": rng.choice(["none", "p", "k", "min", "all"])}
    if op == "verify":
        return {"op": "verify", "batch": min(batch, VERIFY_NODES // nodes), "nodes": nodes, "ragged": ragged}
    layers = _log_int(rng, 1, 32)
    if op == "compact":
        taken = _log_int(rng, 1, min(nodes, 16))
        while batch > 1 and batch * taken * layers * hkv * d > COMPACT_VALUES:
            batch //= 2
        return {"op": "compact", "layers": layers, "batch": batch, "nodes": min(nodes, 64), "taken": taken,
                "ctx": rng.randrange(0, 150), "ragged": ragged, "hkv": min(hkv, 16), "d": min(d, 128), "page": page}
    parents, children = _log_int(rng, 1, 16), _log_int(rng, 1, 8)
    while layers > 1 and parents * children * layers * page * hkv * d > FORK_VALUES // 4:
        layers //= 2
    hkv = min(hkv, 16)
    return {"op": "fork", "layers": layers, "parents": parents, "children": children, "ctx": rng.randrange(1, 1000),
            "grow": rng.randrange(1, 64), "hkv": hkv, "d": d, "page": page}


def _lengths(case):
    """New and cached tokens of each sequence: the largest ones, or spread over their upper half."""
    n = [case["nodes"] - (b * 7919 % (case["nodes"] // 2 + 1) if case["ragged"] else 0) for b in range(case["batch"])]
    ctx = case.get("ctx", 0)
    c = [ctx - (b * 10473 % (ctx // 2 + 1) if case["ragged"] else 0) for b in range(case["batch"])]
    return n, c


# ---- inputs -------------------------------------------------------------------------------------------------


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"case": case, "dev": dev}
    if own:
        import bit_ptq_vla_amd
        s["lib"] = bit_ptq_vla_amd
    {"tree": _make_tree, "sample": _make_sample, "verify": _make_verify, "compact": _make_compact,
     "fork": _make_fork}[case["op"]](s, case, g, seed)
    return s


def _make_cache(s, g, layers, pool, hkv, page, d):
    dev = s["dev"]

    def codes(shape):
        return torch.randint(-127, 128, shape, generator=g, device=dev, dtype=torch.int8)

    def scales():
        return 0.025 * torch.exp(0.3 * torch.randn((layers, pool, hkv), generator=g, device=dev))

    s["k"], s["v"] = codes((layers, pool, hkv, page, d)), codes((layers, pool, hkv, d, page))
    s["ks"], s["vs"] = scales(), scales()
    if own:
        s["caches"] = [s["lib"].KvCache(s["k"][i], s["ks"][i], s["v"][i], s["vs"][i]) for i in range(layers)]


def _make_batch(s, case, g):
    """Sequences whose last tokens are the nodes: lengths, page table and index tensors."""
    dev = s["dev"]
    new, ctx = _lengths(case)
    page = case.get("page", 16)
    kv = [a + b for a, b in zip(new, ctx)]
    width = -(-max(kv) // page)
    pool = case["batch"] * width + 3
    order = torch.randperm(pool, generator=g, device=dev)[:case["batch"] * width]
    s["table"] = order.reshape(case["batch"], width).to(torch.int32)
    s["q_start"] = torch.tensor([0] + new, device=dev).cumsum(0).to(torch.int32)
    s["kv_len"] = torch.tensor(kv, device=dev, dtype=torch.int32)
    s["max_q"], s["max_kv"] = max(new), max(kv)
    s["seq"] = torch.repeat_interleave(torch.arange(case["batch"], device=dev), torch.tensor(new, device=dev))
    s["node"] = torch.arange(sum(new), device=dev) - s["q_start"][:-1].long()[s["seq"]]
    if own:
        s["batch"] = s["lib"].KvBatch(s["table"], s["q_start"], s["kv_len"], max_q=s["max_q"], max_kv=s["max_kv"])
    return pool


def _make_parents(s, g):
    """Trees: a node hangs from one of the eight nodes before it, the nearest ones more often."""
    i = s["node"]
    r = torch.rand(i.shape, generator=g, device=i.device)
    back = (r * r * i.clamp(max=8)).long()
    s["parents"] = (i - 1 - back).clamp(min=0).to(torch.int32)
    s["parents"][i == 0] = -1


def _make_tree(s, case, g, seed):
    pool = _make_batch(s, case, g)
    _make_cache(s, g, 1, pool, case["hkv"], case["page"], case["d"])
    _make_parents(s, g)
    tokens = s["node"].numel()
    dt = DTYPES[case["dtype"]]
    s["q"] = torch.randn((tokens, case["hq"] * case["d"]), generator=g, device=s["dev"]).to(dt)
    s["out"] = torch.empty_like(s["q"])
    if own:
        # one plan and one workspace serve every layer of a step
        s["mask"], s["positions"] = s["lib"].qlin_tree_plan(s["parents"], s["batch"])
        s["work"] = s["lib"].kv_attention_tree_workspace(s["caches"][0], s["batch"], case["hq"])
    else:
        s["sees"] = _ancestors(s)


def _make_sample(s, case, g, seed):
    dev, rows, vocab = s["dev"], case["rows"], case["vocab"]
    pitch = -(-vocab // 8) * 8
    x = torch.randn((rows, pitch), generator=g, device=dev)
    x = x.mul_(2.5).add_(4.0 * (torch.rand((rows, pitch), generator=g, device=dev) < 4.0 / vocab))
    s["logits"] = x.to(DTYPES[case["dtype"]])[:, :vocab]

    def uniform(lo, hi):
        return lo + (hi - lo) * torch.rand(rows, generator=g, device=dev)

    f = case["filters"]
    s["u"] = torch.rand(rows, generator=g, device=dev)
    s["temperature"] = uniform(0.5, 1.2)
    s["top_p"] = uniform(0.8, 0.98) if f in ("p", "all") else None
    s["top_k"] = (torch.randint(5, 200, (rows,), generator=g, device=dev, dtype=torch.int32) if f in ("k", "all") else None)
    s["min_p"] = uniform(0.01, 0.1) if f in ("min", "all") else None
    if f == "all":                                       # requests without a filter among the others, and greedy ones
        off = torch.rand((4, rows), generator=g, device=dev) < 0.15
        s["top_p"][off[0]] = 1.0
        s["top_k"][off[1]] = 0
        s["min_p"][off[2]] = 0.0
        s["temperature"][off[3]] = 0.0
    s["token"] = torch.empty(rows, dtype=torch.int32, device=dev)
    s["logprob"] = torch.empty(rows, dtype=torch.float32, device=dev)
    if own:
        s["work"] = s["lib"].sample_workspace(rows, vocab, dev)


def _make_verify(s, case, g, seed):
    _make_batch(s, dict(case, ctx=500, page=16), g)
    _make_parents(s, g)
    tokens, dev = s["node"].numel(), s["dev"]
    s["draft"] = torch.randint(0, 32000, (tokens,), generator=g, device=dev, dtype=torch.int32)
    s["sampled"] = torch.randint(0, 32000, (tokens,), generator=g, device=dev, dtype=torch.int32)
    # four nodes of five find one of their children confirmed
    row0 = s["q_start"].long()[s["seq"]]
    child = torch.full((tokens,), -1, dtype=torch.int64, device=dev)
    inner = s["node"] > 0
    at = torch.arange(tokens, device=dev)[inner]
    child.scatter_reduce_(0, (row0 + s["parents"].long())[inner], at, "amax")
    hit = (child >= 0) & (torch.rand(tokens, generator=g, device=dev) < 0.8)
    s["sampled"][hit] = s["draft"][child[hit]]
    if own:
        words = -(-s["max_q"] // 32)
        s["mask"] = torch.empty((tokens, words), dtype=torch.int32, device=dev)
        s["positions"] = torch.empty(tokens, dtype=torch.int32, device=dev)
        s["path"] = (torch.empty((case["batch"], s["max_q"]), dtype=torch.int32, device=dev),
                     torch.empty(case["batch"], dtype=torch.int32, device=dev),
                     torch.empty(case["batch"], dtype=torch.int32, device=dev))


def _make_compact(s, case, g, seed):
    pool = _make_batch(s, case, g)
    _make_cache(s, g, case["layers"], pool, case["hkv"], case["page"], case["d"])
    rng = random.Random(seed)
    new, _ = _lengths(case)
    path, count = [], []
    for n in new:
        m = min(case["taken"], n)
        # node 0, then nodes of a path: often the first ones of a level
        rest = sorted(rng.sample(range(1, min(n, 3 * m + 1)), m - 1)) if m > 1 else []
        path.append([0] + rest + [-1] * (s["max_q"] - m))
        count.append(m)
    s["accepted"] = torch.tensor(path, device=s["dev"], dtype=torch.int32)
    s["count"] = torch.tensor(count, device=s["dev"], dtype=torch.int32)
    s["kv_out"] = torch.empty_like(s["kv_len"])
    if own:
        s["stack"] = s["lib"].KvStack(s["caches"])


def _make_fork(s, case, g, seed):
    dev, p, c, page = s["dev"], case["parents"], case["children"], case["page"]
    ctx = [case["ctx"] - b * 7919 % (case["ctx"] // 2 + 1) for b in range(p)]
    width = -(-(case["ctx"] + case["grow"]) // page)
    rows = p + p * c
    used = [-(-n // page) for n in ctx]
    pool = p * width + p * c * (-(-case["grow"] // page) + 1) + 5
    _make_cache(s, g, case["layers"], pool, case["hkv"], page, case["d"])
    order = torch.randperm(pool, generator=g, device=dev)[:sum(used)].to(torch.int32)
    s["table"] = torch.full((rows, width), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(used):
        s["table"][b, :n] = order[at:at + n]
        at += n
    parent = [b for b in range(p) for _ in range(c)]
    i32 = {"dtype": torch.int32, "device": dev}
    s["src"], s["dst"] = torch.tensor(parent, **i32), torch.arange(p, rows, **i32)
    s["src_len"] = torch.tensor([ctx[b] for b in parent], **i32)
    s["empty"] = torch.tensor(ctx + [0] * (p * c), **i32)
    s["full"] = torch.tensor(ctx + [ctx[b] for b in parent], **i32)
    s["grown"] = torch.tensor(ctx + [ctx[b] + case["grow"] for b in parent], **i32)
    s["len"] = s["empty"].clone()                        # what the rows hold between the passes
    s["refs"] = torch.zeros(pool, **i32)
    s["refs"][order.long()] = 1
    if own:
        s["stack"] = s["lib"].KvStack(s["caches"])
        s["pool"] = s["lib"].KvPool(s["refs"], _bits(s["refs"] == 0))
        s["held"] = torch.empty_like(s["len"])
        s["moved"] = torch.empty((rows, 2), **i32)


def run(s):
    return {"tree": _tree, "sample": _sample, "verify": _verify, "compact": _compact, "fork": _fork}[s["case"]["op"]](s)


def _bits(flags):
    """Truth values of the last axis as the bits of int32 words, the lowest bit first."""
    n = flags.shape[-1]
    words = -(-n // 32)
    full = torch.zeros(flags.shape[:-1] + (words * 32,), dtype=torch.int64, device=flags.device)
    full[..., :n] = flags
    w = (full.reshape(flags.shape[:-1] + (words, 32)) << torch.arange(32, device=flags.device)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


# ---- trees --------------------------------------------------------------------------------------------------


def _ancestors(s):
    """[tokens][max_q]: whether a node is the token itself or an ancestor of it."""
    row0 = s["q_start"].long()[s["seq"]]
    sees = torch.zeros((s["node"].numel(), s["max_q"]), dtype=torch.bool, device=s["dev"])
    at = s["node"].clone()
    up = s["parents"].long()
    rows = torch.arange(at.numel(), device=s["dev"])
    while rows.numel():
        sees[rows, at] = True
        at = up[row0[rows] + at]
        rows, at = rows[at >= 0], at[at >= 0]
    return sees


def _tree(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    if own:
        return {"out": s["lib"].qlin_kv_attention_tree(s["q"], s["caches"][0], s["batch"], hq, s["mask"], sm_scale=d ** -0.5,
                                                       softcap=c["cap"], out=s["out"], workspace=s["work"])}
    table = s["table"].long()
    batch, group = table.shape[0], hq // hkv
    k = s["k"][0][table].float() * s["ks"][0][table][..., None, None]          # [b][pages][h][page][d]
    k = k.permute(0, 2, 1, 3, 4).reshape(batch, hkv, -1, d)
    v = s["v"][0][table].float() * s["vs"][0][table][..., None, None]          # [b][pages][h][d][page]
    v = v.permute(0, 2, 1, 4, 3).reshape(batch, hkv, -1, d)
    keys, mq = k.shape[2], s["max_q"]
    q_pad = torch.zeros((batch, mq, hq * d), device=k.device)
    q_pad[s["seq"], s["node"]] = s["q"].float()
    qh = q_pad.reshape(batch, mq, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, d)
    sc = torch.matmul(qh, k.transpose(2, 3).contiguous()).mul_(d ** -0.5)
    if c["cap"]:
        sc = torch.tanh(sc.div_(c["cap"])).mul_(c["cap"])
    first = s["kv_len"].long() - s["q_start"].long().diff()
    j = torch.arange(keys, device=k.device)
    seen = (j < first[:, None])[:, None, :].repeat(1, mq, 1)                   # [b][node][keys]
    t, n = torch.nonzero(s["sees"], as_tuple=True)
    seen[s["seq"][t], s["node"][t], first[s["seq"][t]] + n] = True
    sc = sc.reshape(batch, hkv, group, mq, keys)
    sc.masked_fill_(~seen[:, None, None], float("-inf"))
    top = sc.amax(-1, keepdim=True)
    p = torch.exp_(sc.sub_(torch.where(top > float("-inf"), top, torch.zeros_like(top))))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(batch, hkv, -1, keys), v).reshape(batch, hkv, group, mq, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.permute(0, 3, 1, 2, 4).reshape(batch, mq, hq * d)
    return {"out": o[s["seq"], s["node"]].to(s["q"].dtype)}


def _verify(s):
    if own:
        lib = s["lib"]
        mask, positions = lib.qlin_tree_plan(s["parents"], s["batch"], mask=s["mask"], positions=s["positions"])
        path, count, token = lib.qlin_tree_accept(s["parents"], s["draft"], s["sampled"], s["batch"], out=s["path"])
        return {"mask": mask, "positions": positions, "path": path, "count": count, "token": token}
    sees = _ancestors(s)
    first = s["kv_len"].long() - s["q_start"].long().diff()
    positions = first[s["seq"]] + sees.sum(1) - 1
    # every node's confirmed child: the first of its children that holds the token sampled at it
    row0 = s["q_start"].long()[s["seq"]]
    tokens = s["node"].numel()
    up = row0 + s["parents"].long()
    good = (s["node"] > 0) & (s["draft"] == s["sampled"][up.clamp(min=0)])
    follow = torch.full((tokens,), tokens, dtype=torch.int64, device=s["dev"])
    follow.scatter_reduce_(0, up[good], torch.arange(tokens, device=s["dev"])[good], "amin")
    batch = s["kv_len"].numel()
    path = torch.full((batch, s["max_q"]), -1, dtype=torch.int32, device=s["dev"])
    count = torch.zeros(batch, dtype=torch.int64, device=s["dev"])
    at = s["q_start"].long()[:-1].clone()
    end = at.clone()
    live = torch.arange(batch, device=s["dev"])
    while live.numel():
        end[live] = at[live]
        path[live, count[live]] = s["node"][at[live]].to(torch.int32)
        count[live] += 1
        at[live] = follow[at[live]]
        live = live[at[live] < tokens]
    return {"mask": _bits(sees), "positions": positions.to(torch.int32), "path": path, "count": count.to(torch.int32),
            "token": s["sampled"][end]}


# ---- sampling -----------------------------------------------------------------------------------------------


def _sample(s):
    if own:
        token, logprob = s["lib"].qlin_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                                              top_p=s["top_p"], min_p=s["min_p"], out=(s["token"], s["logprob"]),
                                              workspace=s["work"])
        return {"token": token, "logprob": logprob}
    # in 64 bits: a token is decided next to a border
    x, order = torch.sort(s["logits"].double(), dim=1, descending=True, stable=True)
    t = s["temperature"].double()[:, None]
    w = torch.exp((x - x[:, :1]) / torch.where(t > 0, t, 1.0))
    place = torch.arange(x.shape[1], device=x.device)
    keep = torch.where(t > 0, place >= 0, place == 0)
    if s["min_p"] is not None:
        keep = keep & (w >= s["min_p"].double()[:, None])
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        keep = keep & ((k <= 0) | (place < k))
    w = torch.where(keep, w, 0.0)
    total = w.cumsum(1)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        before = torch.cat([torch.zeros_like(total[:, :1]), total[:, :-1]], 1)
        w = torch.where((p >= 1) | (before < p * total[:, -1:]), w, 0.0)
        total = w.cumsum(1)
    at = (total > s["u"].double()[:, None] * total[:, -1:]).to(torch.int8).argmax(1)[:, None]
    s["token"].copy_(order.gather(1, at)[:, 0])
    s["logprob"].copy_(torch.log(w.gather(1, at) / total[:, -1:])[:, 0])
    return {"token": s["token"], "logprob": s["logprob"]}


# ---- pages --------------------------------------------------------------------------------------------------


def _compact(s):
    out = {"k": s["k"], "v": s["v"], "k_scale": s["ks"], "v_scale": s["vs"], "kv_len": s["kv_out"]}
    if own:
        s["lib"].qlin_kv_compact(s["stack"], s["batch"], s["accepted"], s["count"], kv_len_out=s["kv_out"])
        return out
    page = s["case"]["page"]
    first = s["kv_len"].long() - s["q_start"].long().diff()
    m = s["count"].long()
    b, i = torch.nonzero(torch.arange(s["max_q"], device=s["dev"])[None] < m[:, None], as_tuple=True)
    src, dst = first[b] + s["accepted"].long()[b, i], first[b] + i
    table = s["table"].long()
    ps, pd = table[b, src // page], table[b, dst // page]
    held = (first % page > 0) & (m > 0)                  # first pages that keep earlier tokens
    page0 = table.gather(1, (first // page).clamp(max=table.shape[1] - 1)[:, None])[:, 0][held]
    upto = (first % page)[held]
    for codes, scale, by_token in ((s["k"], s["ks"], True), (s["v"], s["vs"], False)):
        layers, pool, heads = scale.shape
        grown = torch.zeros_like(scale)
        grown[:, page0] = scale[:, page0]
        grown.index_reduce_(1, pd, scale[:, ps], "amax")
        some = torch.where(grown > 0, grown, torch.ones_like(grown)).double()
        was = codes[:, ps, :, src % page] if by_token else codes[:, ps, :, :, src % page]       # [moved][layers][h][d]
        now = torch.round(was.double() * scale[:, ps].double().permute(1, 0, 2)[..., None]
                          / some[:, pd].permute(1, 0, 2)[..., None])
        slots = torch.arange(page, device=s["dev"])[None] < upto[:, None]
        slots = slots[None, :, None, :, None] if by_token else slots[None, :, None, None, :]
        kept = codes[:, page0]
        moved = torch.round(kept.double() * scale[:, page0].double()[..., None, None] / some[:, page0][..., None, None])
        codes[:, page0] = torch.where(slots, moved.to(torch.int8), kept)
        if by_token:
            codes[:, pd, :, dst % page] = now.to(torch.int8)
        else:
            codes[:, pd, :, :, dst % page] = now.to(torch.int8)
        scale[:, pd] = grown[:, pd]
    s["kv_out"].copy_(first + m)
    return out


def _fork(s):
    """The continuations of the pass before are given back; then a row of each, and the growth of all."""
    out = {"table": s["table"], "refs": s["refs"], "len": s["len"], "k": s["k"], "v": s["v"], "k_scale": s["ks"],
           "v_scale": s["vs"]}
    if own:
        lib, page = s["lib"], s["case"]["page"]
        args = (s["pool"], s["stack"], s["table"])
        lib.qlin_kv_resize(*args, s["len"], s["empty"], len_out=s["held"], moved=s["moved"])
        lib.qlin_kv_fork(s["pool"], s["table"], s["src"], s["dst"], s["src_len"], page)
        lib.qlin_kv_resize(*args, s["full"], s["grown"], len_out=s["len"], moved=s["moved"])
        return dict(out, free=s["pool"].free_bits)
    _plain_resize(s, s["len"], s["empty"])
    page, table, refs = s["case"]["page"], s["table"], s["refs"]
    j = torch.arange(table.shape[1], device=s["dev"])
    share = j[None] < (s["src_len"].long() + page - 1)[:, None] // page
    rows = torch.where(share, table[s["src"].long()], table[s["dst"].long()])
    table[s["dst"].long()] = rows
    refs.index_add_(0, rows[share].long(), torch.ones_like(rows[share]))
    s["len"].copy_(_plain_resize(s, s["full"], s["grown"]))
    return dict(out, free=_bits(refs == 0))


def _plain_resize(s, old, new):
    page, table, refs = s["case"]["page"], s["table"], s["refs"]
    old, new = old.long(), new.long()
    have, want = (old + page - 1) // page, (new + page - 1) // page
    j = torch.arange(table.shape[1], device=s["dev"])[None]
    drop = (j >= want[:, None]) & (j < have[:, None])
    gone = table[drop]
    refs.index_add_(0, gone.long(), -torch.ones_like(gone))
    table[drop] = -1
    # the last page of a growing row, where others hold it too: each but the last of its holders takes a copy
    part = (new > old) & (old % page > 0)
    last = table.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0].long()
    same = (last[:, None] == last[None]) & part[:, None] & part[None]
    copy = part & (refs[last.clamp(min=0)] - torch.tril(same, -1).sum(1) > 1)
    need = torch.where(new > old, want - have, 0) + copy
    free = torch.nonzero(refs == 0)[:, 0]
    ok = (need == 0) | (need.cumsum(0) <= free.numel())
    copy = copy & ok
    take = ((j >= have[:, None]) & (j < want[:, None]) & ok[:, None]) | (copy[:, None] & (j == have[:, None] - 1))
    fresh = free[:int(take.sum())]
    table[take] = fresh.to(torch.int32)
    refs[fresh] = 1
    a, b = last[copy], table.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0].long()[copy]
    refs.index_add_(0, a, -torch.ones_like(a, dtype=torch.int32))
    for t in (s["k"], s["v"], s["ks"], s["vs"]):
        t[:, b] = t[:, a]
    return torch.where(ok, new, old).to(torch.int32)


# ---- work and definition ------------------------------------------------------------------------------------


def work(case):
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (4 if case["dtype"] == "f32" else 2) + case["rows"] * 28, "flops": 4 * n}
    if case["op"] == "fork":
        rows = case["parents"] * case["children"]
        partial = sum(case["children"] for b in range(case["parents"])
                      if (case["ctx"] - b * 7919 % (case["ctx"] // 2 + 1)) % case["page"])
        page = case["layers"] * case["hkv"] * (2 * case["page"] * case["d"] + 8)
        return {"bytes": 2 * partial * page + rows * -(-case["ctx"] // case["page"]) * 16, "flops": rows}
    new, ctx = _lengths(case)
    if case["op"] == "verify":
        return {"bytes": sum(new) * (16 + 4 * -(-max(new) // 32)) + case["batch"] * (8 + 4 * max(new)), "flops": sum(new)}
    hkv, d, page = case["hkv"], case["d"], case["page"]
    if case["op"] == "compact":
        moved = sum(min(case["taken"], n) - 1 for n in new)
        rows = case["layers"] * hkv
        return {"bytes": rows * (moved * 4 * d + case["batch"] * 16) + case["batch"] * 16, "flops": 4 * rows * moved * d}
    size = pairs = 0
    for n, c in zip(new, ctx):
        pairs += n * (c + 1)
        size += hkv * ((c + n) * 2 * d + -(-(c + n) // page) * 8)
    return {"bytes": size + sum(new) * (case["hq"] * d * 4 + 4 * -(-max(new) // 32)), "flops": 4 * d * case["hq"] * pairs}


def exact(case, seed):
    if case["op"] in ("verify", "fork"):
        return None                                      # whole numbers and copies
    if case["op"] == "sample":
        return _exact_sample(prepare(case, seed))
    if case["op"] == "compact":
        return _exact_compact(prepare(case, seed))
    s = prepare(case, seed)
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    new, ctx = _lengths(case)
    group, at = hq // hkv, 0
    up = s["parents"].tolist()
    out = torch.zeros((sum(new), hq, d), dtype=torch.float64, device=s["dev"])
    for i, (n, c) in enumerate(zip(new, ctx)):
        pages = s["table"][i, :-(-(c + n) // page)].long()
        sees = [[False] * n for _ in range(n)]
        for t in range(n):
            if up[at + t] >= 0:
                sees[t] = list(sees[up[at + t]])
            sees[t][t] = True
        hidden = torch.zeros((n, c + n), dtype=torch.bool, device=s["dev"])
        hidden[:, c:] = ~torch.tensor(sees, device=s["dev"])
        x = s["q"][at:at + n].double().reshape(n, hkv, group, d)
        for h in range(hkv):
            k = (s["k"][0, pages, h].double() * s["ks"][0, pages, h].double()[:, None, None]).reshape(-1, d)[:c + n]
            v = (s["v"][0, pages, h].double() * s["vs"][0, pages, h].double()[:, None, None]).transpose(1, 2)
            v = v.reshape(-1, d)[:c + n]
            w = torch.einsum("nd,kd->nk", x[:, h].reshape(-1, d), k).reshape(n, group, -1) / math.sqrt(d)
            if case["cap"]:
                w = case["cap"] * torch.tanh(w / case["cap"])
            w = torch.softmax(w.masked_fill_(hidden[:, None], float("-inf")), -1)
            out[at:at + n, h * group:(h + 1) * group] = torch.matmul(w, v)
        at += n
    return {"out": out.reshape(-1, hq * d)}


def _exact_sample(s):
    """Row by row: the kept set as a threshold, then the token by running mass."""
    rows = s["logits"].shape[0]
    token = torch.empty(rows, dtype=torch.int32, device=s["dev"])
    logprob = torch.empty(rows, dtype=torch.float64, device=s["dev"])
    get = {n: (s[n].tolist() if s[n] is not None else None) for n in ("u", "temperature", "top_k", "top_p", "min_p")}
    for r in range(rows):
        x = s["logits"][r].double()
        t = get["temperature"][r]
        if t <= 0:
            token[r], logprob[r] = torch.nonzero(x == x.max())[0, 0], 0.0
            continue
        lw = (x - x.max()) / t
        floor = math.log(get["min_p"][r]) if get["min_p"] and get["min_p"][r] > 0 else -math.inf
        index = torch.nonzero(lw >= floor)[:, 0]
        index = index[torch.sort(-x[index], stable=True).indices]
        if get["top_k"] and get["top_k"][r] > 0:
            index = index[:get["top_k"][r]]
        run_mass = torch.exp(lw[index]).cumsum(0)
        if get["top_p"] and get["top_p"][r] < 1:
            run_mass = run_mass[:int((run_mass < get["top_p"][r] * run_mass[-1]).sum()) + 1]
        at = min(int((run_mass <= get["u"][r] * run_mass[-1]).sum()), run_mass.numel() - 1)
        token[r] = index[at]
        logprob[r] = lw[index[at]] - torch.log(run_mass[-1])
    return {"token": token, "logprob": logprob}


def _exact_compact(s):
    """The page scales, a sequence at a time; codes are whole numbers."""
    page = s["case"]["page"]
    ks, vs = s["ks"].double(), s["vs"].double()
    kv, start, table = s["kv_len"].tolist(), s["q_start"].tolist(), s["table"].tolist()
    for b, (path, m) in enumerate(zip(s["accepted"].tolist(), s["count"].tolist())):
        first = kv[b] - (start[b + 1] - start[b])
        for scale, was in ((ks, s["ks"].double()), (vs, s["vs"].double())):
            for p in range(first // page, (first + m - 1) // page + 1 if m else 0):
                from_pages = [table[b][(first + path[i]) // page] for i in range(m) if (first + i) // page == p]
                if first % page and p == first // page:
                    from_pages.append(table[b][p])
                scale[:, table[b][p]] = was[:, from_pages].amax(1)
    return {"k": None, "v": None, "k_scale": ks, "v_scale": vs, "kv_len": None}
