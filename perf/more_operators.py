"""Cases that measure a speculative step on the 4-bit key/value cache.

Drafted tokens form a tree: node 0 is the token that the last step decided, every
other node continues its parent. ``tree`` lays a step's nodes out (which see
which, positions, slots), ``attend`` with a tree mask attends over cache and
ancestors, ``verify`` walks the tree against the target's probabilities, and
``commit`` moves the accepted tokens to their places in every layer's cache.

The plain forms are elementary torch operations on the documented page layout
(include/kvcache.h): a page holds, for each kv head, blocks of 32 tokens; a
block holds the tokens' key nibbles row by row, their value nibbles in groups
of 8 tokens, and a binary16 pair (s, b) a token for keys and for values. A
nibble n stands for the binary16 nearest to (16 + n) s + b.
"""
import math
import random

import torch

own = False

LOWEST = torch.finfo(torch.float32).min  # lse of a row that sees no key


# ---------------------------------------------------------------- cases

def listed():
    return [
        # A chat's step: one small tree, all latency.
        dict(name="tree of 8", op="tree", batch=1, nodes=8, words=1, ragged=False, len_max=777, hq=64, hkv=8, d=128,
             page=64),
        # A server's step with large trees of many sizes.
        dict(name="trees up to 200", op="tree", batch=128, nodes=200, words=4, ragged=True, len_max=8192, hq=64, hkv=8,
             d=128, page=64),
        # A chat early on: a small tree on one short sequence, latency again.
        dict(name="attend short", op="attend", batch=1, nodes=13, queries=13, words=1, len_max=777, ragged=False, hq=64,
             hkv=8, d=128, page=64, out="f16"),
        # A serving batch of ragged sequences with trees of an odd size, small heads.
        dict(name="attend ragged d64", op="attend", batch=24, nodes=25, queries=25, words=1, len_max=4099, ragged=True,
             hq=32, hkv=4, d=64, page=32, out="f16"),
        # A serving batch with full 64-node trees: matrix products count.
        dict(name="attend batch", op="attend", batch=16, nodes=64, queries=64, words=1, len_max=8192, ragged=False, hq=64,
             hkv=8, d=128, page=64, out="f16"),
        # One long context, 96 heads, binary32 partials for the Flash-Decode combine.
        dict(name="attend long", op="attend", batch=1, nodes=48, queries=48, words=1, len_max=131072, ragged=False, hq=96,
             hkv=8, d=128, page=256, out="f32"),
        # A chat's drafts, one after another, with the draft's probabilities.
        dict(name="verify chain", op="verify", batch=1, nodes=6, shape="chain", vocab=32768, drawn=True),
        # The same for a serving batch with a large vocabulary.
        dict(name="verify chains", op="verify", batch=64, nodes=6, shape="chain", vocab=131072, drawn=True),
        # Trees of the draft's most likely tokens (no probabilities of the draft), odd vocabulary.
        dict(name="verify certain trees", op="verify", batch=32, nodes=60, shape="tree", vocab=65537, drawn=False),
        # Trees whose siblings were drawn one after another: a rejection changes what the next one is held against.
        dict(name="verify drawn trees", op="verify", batch=16, nodes=25, shape="tree", vocab=131072, drawn=True),
        # The accepted tokens of one sequence, one layer.
        dict(name="commit one", op="commit", batch=1, nodes=13, layers=1, len_max=777, hq=64, hkv=8, d=128, page=64),
        # The accepted tokens of a serving batch, several layers.
        dict(name="commit batch", op="commit", batch=64, nodes=64, layers=6, len_max=8192, hq=64, hkv=8, d=128, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hq, hkv, d = rng.choice([(64, 8, 128), (32, 8, 128), (96, 8, 128), (16, 16, 64), (32, 4, 64), (16, 2, 256),
                             (20, 20, 128), (40, 8, 128), (12, 1, 128)])
    page = rng.choice([32, 64, 128, 256])
    kind = rng.choice(["tree", "attend", "attend", "attend", "verify", "verify", "commit"])
    if kind == "tree":
        nodes = _log(rng, 1, 256)
        return dict(op="tree", batch=_log(rng, 1, 128), nodes=nodes, words=-(-nodes // 64), ragged=rng.random() < 0.6,
                    len_max=_log(rng, 1, 8192), hq=hq, hkv=hkv, d=d, page=page)
    if kind == "attend":
        batch = _log(rng, 1, 32)
        nodes = _log(rng, 2, 128)
        queries = nodes if rng.random() < 0.7 else rng.randint(1, nodes)  # or only the tree's last level
        most = min(131072, (1 << 27) // (batch * hkv * d), int(6e10) // (batch * queries * hq * d))
        return dict(op="attend", batch=batch, nodes=nodes, queries=queries, words=-(-nodes // 64),
                    len_max=_log(rng, nodes, max(nodes + 1, most)), ragged=rng.random() < 0.6, hq=hq, hkv=hkv, d=d,
                    page=page, out=rng.choice(["f16", "f32"]))
    if kind == "verify":
        shape = rng.choice(["chain", "tree"])
        vocab = _log(rng, 1000, 200000)
        nodes = _log(rng, 1, 12 if shape == "chain" else 64)
        most = max(1, min(96, (1 << 26) // (nodes * vocab)))
        return dict(op="verify", batch=_log(rng, 1, most), nodes=nodes, shape=shape, vocab=vocab,
                    drawn=shape == "chain" or rng.random() < 0.5)
    return dict(op="commit", batch=_log(rng, 1, 64), nodes=_log(rng, 1, 128), layers=rng.randint(1, 6),
                len_max=_log(rng, 1, 8192), hq=hq, hkv=hkv, d=d, page=page)


def _lengths(case):
    """Tokens of each sequence before this step (tree, commit) or with it (attend), from the case alone."""
    b, top = case["batch"], case["len_max"]
    low = case["nodes"] if case["op"] == "attend" else 0
    rng = random.Random(b * 1000003 + top * 31 + case["nodes"])
    if not case.get("ragged", True):
        return [top] * b
    return [top] + [_log(rng, max(1, low, top // 64), top) if rng.random() < 0.95 else low for _ in range(b - 1)]


def _sizes(case):
    """Nodes of each sequence's tree, from the case alone."""
    if not case.get("ragged", False) or case["op"] != "tree":
        return [case["nodes"]] * case["batch"]
    rng = random.Random(case["batch"] * 7919 + case["nodes"])
    return [case["nodes"]] + [rng.randint(0, case["nodes"]) for _ in range(case["batch"] - 1)]


def work(case):
    if case["op"] == "tree":
        t = sum(_sizes(case))
        return {"bytes": t * (4 + 8 * case["words"] + 16) + case["batch"] * 20, "flops": 0}
    if case["op"] == "verify":
        # at the least, the row that the last token is drawn from
        return {"bytes": case["batch"] * (case["vocab"] * (8 if case["drawn"] else 4) + 28 * case["nodes"]),
                "flops": case["batch"] * case["vocab"] * (4 if case["drawn"] else 1)}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "commit":
        kept = sum(len(p) for p in _paths(case, 0))
        moved = sum(sum(i != j for i, j in enumerate(p)) for p in _paths(case, 0))
        back = kept * case["layers"] * hkv * (d + 8 + 4 * d)  # the kept tokens read back as binary16
        return {"bytes": 2 * moved * case["layers"] * hkv * (d + 8) + back, "flops": 0}
    lens, rows = _lengths(case), case["batch"] * case["queries"] * hq
    pairs = sum(case["queries"] * (n - case["nodes"] + 1) for n in lens)  # and a node's ancestors, of which few are certain
    return {"bytes": sum(lens) * hkv * (d + 8) + rows * (d * (2 + (4 if case["out"] == "f32" else 2)) + 4),
            "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------- the 4-bit form, in elementary operations

def _quantise(x):
    """(nibbles uint8, s, b) of the last axis of x, in 64 bits."""
    x = x.double()
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s = ((hi - lo) / 15).half()
    b = (lo - 16 * s.double()).half()
    sd = s.double()
    n = torch.where(sd > 0, torch.round((x - b.double()) / torch.where(sd > 0, sd, 1.0)) - 16, 0.0)
    return n.clamp(0, 15).to(torch.uint8), s, b


def _value(n, s, b):
    """The binary16 values that nibbles stand for."""
    return torch.addcmul(b.float(), n.float() + 16, s.float()).half()


def _pack(kn, ks, kb, vn, vs, vb):
    """Blocks of 32 tokens in their stored bytes. Nibbles (..., 32, D), s and b (..., 32, 1) -> (..., 32 (D + 8))."""
    d, lead = kn.shape[-1], kn.shape[:-2]
    k = (kn[..., 0::2] | (kn[..., 1::2] << 4)).reshape(*lead, 16 * d)
    v = vn.reshape(*lead, 2, 4, 4, 16, d // 64, 4)  # token = (half, quarter, i), channel = (c, group, j)
    n = len(lead)
    v = v.permute(*range(n), n + 4, n + 1, n + 3, n, n + 2, n + 5).contiguous()
    v = (v[..., 0::2] | (v[..., 1::2] << 4)).reshape(*lead, 16 * d)
    kp = torch.cat([ks, kb], -1).reshape(*lead, 64).contiguous().view(torch.uint8)
    order = lambda p: p.reshape(*lead, 2, 4, 4).transpose(-3, -2).reshape(*lead, 32)  # noqa: E731
    vp = torch.cat([order(vs), order(vb)], -1).contiguous().view(torch.uint8)
    return torch.cat([k, v, kp, vp], -1)


def _unpack(block, d):
    """The binary16 keys and values (..., 32, D) of stored blocks (..., 32 (D + 8))."""
    lead = block.shape[:-1]
    k, v, kp, vp = block.split([16 * d, 16 * d, 128, 128], -1)
    kn = torch.stack([k & 15, k >> 4], -1).reshape(*lead, 32, d)
    kp = kp.contiguous().view(torch.float16).reshape(*lead, 32, 2)
    v = torch.stack([v & 15, v >> 4], -1).reshape(*lead, d // 64, 4, 16, 2, 4, 4)
    n = len(lead)
    vn = v.permute(*range(n), n + 3, n + 1, n + 4, n + 2, n, n + 5).reshape(*lead, 32, d)
    vp = vp.contiguous().view(torch.float16).reshape(*lead, 2, 4, 2, 4).transpose(-3, -2).reshape(*lead, 2, 32, 1)
    return _value(kn, kp[..., :1], kp[..., 1:]), _value(vn, vp[..., 0, :, :], vp[..., 1, :, :])


def _token_bytes(slot, hkv, d, page):
    """Bytes of tokens in the flat pages: (len(slot), hkv, D + 8), key row, value words, key pair, value pairs."""
    token = slot % 32
    head = torch.arange(hkv, device="cuda")
    block = ((slot // page)[:, None] * hkv + head) * (page // 32) + (slot % page // 32)[:, None]
    base = (block * (32 * (d + 8)))[..., None]
    half, quarter, i = token // 16, token // 4 % 4, token % 4
    e = (half * 4 + i)[:, None, None]
    key = (token * (d // 2))[:, None, None] + torch.arange(d // 2, device="cuda")
    j = torch.arange(d // 2, device="cuda")  # byte pair (j % 2) of group (j // 2) % (d / 64) of channel run j // (d / 32)
    value = 16 * d + ((j // 2 % (d // 64) * 4 + quarter[:, None]) * 16 + j // (d // 32))[:, None] * 16 + e * 2 + j % 2
    kpair = 32 * d + (token * 4)[:, None, None] + torch.arange(4, device="cuda")
    vs = 32 * d + 128 + ((quarter * 8)[:, None, None] + e) * 2 + torch.arange(2, device="cuda")
    return torch.cat([base + key, base + value, base + kpair, base + vs, base + vs + 64], -1)


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _starts(sizes):
    start = [0]
    for n in sizes:
        start.append(start[-1] + n)
    return start


def _parents(rng, n, shape="tree"):
    """A tree as drafting leaves it: nodes in the order of their making, some runs and some spread."""
    return [-1] + [i - 1 if shape == "chain" or rng.random() < 0.3 else int(i * rng.random() ** 1.5) for i in range(1, n)] \
        if n else []


def _paths(case, seed):
    """Accepted nodes of each sequence, how many and how many in place already from the case alone. A destination is
    no other node's source, so that a pass can be repeated."""
    sizes, rng = random.Random(case["batch"] * 31 + case["nodes"]), random.Random(seed * 31 + case["nodes"])
    out = []
    for _ in range(case["batch"]):
        n = case["nodes"]
        count = sizes.randint(1, min(9, n))
        stay = max(sizes.randint(1, count), 2 * count - n)
        out.append(list(range(stay)) + sorted(rng.sample(range(count, n), count - stay)))
    return out


def _table(case, need, g):
    """Page table of sequences that need so many pages each, in a random order, and the number of pages."""
    width = max(1, max(need))
    pages = sum(need) + 2
    order = torch.randperm(pages, device="cuda", generator=g).int()
    table = torch.zeros(case["batch"], width, device="cuda", dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, pages


def _filled(case, pages, g):
    """Pages as earlier appends left them."""
    hkv, d, page = case["hkv"], case["d"], case["page"]
    store = torch.empty(pages, hkv * page * (d + 8), device="cuda", dtype=torch.uint8)
    gain = torch.exp(0.5 * torch.randn(2, hkv, 1, 1, d, device="cuda", generator=g))
    step = max(1, (1 << 27) // (hkv * page * d))
    for p in range(0, pages, step):
        x = torch.randn(2, min(step, pages - p), hkv, page // 32, 32, d, device="cuda", generator=g) * gain[:, None]
        (kn, ks, kb), (vn, vs, vb) = _quantise(x[0]), _quantise(x[1])
        store[p:p + step] = _pack(kn, ks, kb, vn, vs, vb).reshape(-1, hkv * page * (d + 8))
    return store


def _handle(case, pages):
    from shard_decomposed_gemm_amd import KvCache
    if case["op"] == "verify":
        return KvCache(1, 1, 128)
    return KvCache(case["hq"], case["hkv"], case["d"], page_tokens=case["page"], num_pages=pages)


def _prepare_tree(case, seed):
    sizes, lens, rng = _sizes(case), _lengths(case), random.Random(seed)
    table, pages = _table(case, [-(-(n + m) // case["page"]) for n, m in zip(lens, sizes)], _gen(seed))
    t = sum(sizes)
    st = dict(case=case, parent=_int(sum((_parents(rng, n) for n in sizes), [])), start=_int(_starts(sizes)),
              lens=_int(lens), table=table, mask=torch.empty(t, case["words"], device="cuda", dtype=torch.int64),
              positions=torch.empty(t, device="cuda", dtype=torch.int64),
              slots=torch.empty(t, device="cuda", dtype=torch.int64),
              total=torch.empty(case["batch"], device="cuda", dtype=torch.int32))
    if own:
        st["kv"] = _handle(case, pages)
    return st


def _prepare_attend(case, seed):
    hq, d, page, nq, n, b = (case[k] for k in ("hq", "d", "page", "queries", "nodes", "batch"))
    g, rng, lens = _gen(seed), random.Random(seed), _lengths(case)
    table, pages = _table(case, [-(-m // page) for m in lens], g)
    store = _filled(case, pages, g)
    rows = []  # masks of the tree's last nq nodes
    for _ in range(b):
        seen = []
        for i, p in enumerate(_parents(rng, n)):
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
        for m in seen[n - nq:]:
            words = [m >> 64 * w & (1 << 64) - 1 for w in range(case["words"])]
            rows.append([w - (1 << 64) if w >> 63 else w for w in words])
    t = b * nq
    st = dict(case=case, pages=store, table=table, lens=_int(lens), start=_int(_starts([nq] * b)),
              off=_int([m - n for m in lens]), mask=torch.tensor(rows, dtype=torch.int64, device="cuda"),
              q=torch.randn(t, hq, d, device="cuda", generator=g).half(),
              out=torch.empty(t, hq, d, device="cuda", dtype=torch.float32 if case["out"] == "f32" else torch.float16),
              lse=torch.empty(t, hq, device="cuda"))
    if own:
        st["kv"] = _handle(case, pages)
        st["workspace"] = st["kv"].workspace(b, nq, case["len_max"])
    return st


def _prepare_verify(case, seed):
    b, n, v = case["batch"], case["nodes"], case["vocab"]
    g, rng, t = _gen(seed), random.Random(seed), b * n
    parent, row, rank = [], [], []  # of each node, its parent's row and its place among the siblings
    for s in range(b):
        own_parents, children = _parents(rng, n, case["shape"]), [0] * n
        for p in own_parents:
            row.append(s * n + max(p, 0))
            rank.append(children[max(p, 0)] if p >= 0 else 0)
            if p >= 0:
                children[p] += 1
        parent += own_parents
    most = max(rank) + 1
    p = torch.empty(t, v, device="cuda")
    q = torch.empty(t, v, device="cuda")
    top = torch.empty(t, most, device="cuda", dtype=torch.int64)
    step = max(1, (1 << 26) // v)
    for i in range(0, t, step):
        # a target's peaked distributions, and a draft's that come near them
        x = 4 * torch.randn(min(step, t - i), v, device="cuda", generator=g)
        y = x + 0.7 * torch.randn(x.shape, device="cuda", generator=g)
        p[i:i + step], q[i:i + step] = torch.softmax(x, -1), torch.softmax(y, -1)
        if case["drawn"]:  # the largest of perturbed logits, in order, are draws without replacement
            y = y - (-torch.rand(y.shape, device="cuda", generator=g).clamp(min=1e-30).log()).log()
        top[i:i + step] = y.topk(most, -1).indices
    st = dict(case=case, tokens=top[torch.tensor(row, device="cuda"), torch.tensor(rank, device="cuda")].contiguous(),
              parent=_int(parent), start=_int(_starts([n] * b)), p=p, q=q if case["drawn"] else None,
              u=torch.rand(t, device="cuda", generator=g), path=torch.empty(t, device="cuda", dtype=torch.int32),
              count=torch.empty(b, device="cuda", dtype=torch.int32),
              next=torch.empty(b, device="cuda", dtype=torch.int64), children=most)
    if own:
        st["kv"] = _handle(case, 1)
        st["workspace"] = st["kv"].verify_workspace(b, v)
    return st


def _prepare_commit(case, seed):
    g, lens, n, page = _gen(seed), _lengths(case), case["nodes"], case["page"]
    # only the pages that the trees lie on hold anything of interest: the rest of every table names a page that is shared
    first = [m // page for m in lens]
    need = [(m + n - 1) // page - f + 1 for m, f in zip(lens, first)]
    near, pages = _table(case, need, g)
    table = torch.full((case["batch"], max(f + k for f, k in zip(first, need))), pages, device="cuda", dtype=torch.int32)
    for i, (f, k) in enumerate(zip(first, need)):
        table[i, f:f + k] = near[i, :k]
    pages += 1
    paths = _paths(case, seed)
    path, slots = [], []
    host = table.tolist()
    for s, accepted in enumerate(paths):
        path += accepted + [-1] * (n - len(accepted))
        at = [lens[s] + i for i in range(len(accepted))]
        slots += [host[s][x // page] * page + x % page for x in at]
    shape = (len(slots), case["hkv"], case["d"])
    st = dict(case=case, pages=[_filled(case, pages, g) for _ in range(case["layers"])], table=table, lens=_int(lens),
              start=_int(_starts([n] * case["batch"])), path=_int(path), count=_int([len(x) for x in paths]),
              slots=torch.tensor(slots, dtype=torch.int64, device="cuda"),
              new=torch.empty(case["batch"], device="cuda", dtype=torch.int32),
              k_out=[torch.empty(shape, device="cuda", dtype=torch.float16) for _ in range(case["layers"])],
              v_out=[torch.empty(shape, device="cuda", dtype=torch.float16) for _ in range(case["layers"])])
    if own:
        st["kv"] = _handle(case, pages)
    return st


def prepare(case, seed):
    return {"tree": _prepare_tree, "attend": _prepare_attend, "verify": _prepare_verify,
            "commit": _prepare_commit}[case["op"]](case, seed)


# ---------------------------------------------------------------- one pass

def _tree_plain(st):
    c = st["case"]
    start, parent, lens = st["start"].long(), st["parent"].long(), st["lens"].long()
    t = parent.shape[0]
    row = torch.arange(t, device="cuda")
    seq = torch.searchsorted(start[1:].contiguous(), row, right=True)
    first = start[seq]
    node = row - first
    up = torch.where(parent >= 0, first + parent, -1)
    one = torch.ones((), device="cuda", dtype=torch.int64)
    mask = torch.where(torch.arange(c["words"], device="cuda") == (node // 64)[:, None], (one << node % 64)[:, None], 0)
    depth = (parent >= 0).long()
    for _ in range(max(1, (c["nodes"] - 1).bit_length())):  # what the ancestor so far has seen, and its ancestor next
        has = up >= 0
        at = up.clamp(min=0)
        mask = torch.where(has[:, None], mask | mask[at], mask)
        depth = torch.where(has, depth + depth[at], depth)
        up = torch.where(has, up[at], -1)
    at = lens[seq] + node
    page = st["table"][seq, at // c["page"]].long()
    st["mask"].copy_(mask)
    st["positions"].copy_(lens[seq] + depth)
    st["slots"].copy_(page * c["page"] + at % c["page"])
    st["total"].copy_(lens + start[1:] - start[:-1])
    return st["mask"], st["positions"], st["slots"], st["total"]


def _attend_plain(st):
    c = st["case"]
    hq, hkv, d, page, nq, words = (c[k] for k in ("hq", "hkv", "d", "page", "queries", "words"))
    b, width = st["table"].shape
    size = width * page
    block = st["pages"][st["table"].long()].reshape(b, width, hkv, page // 32, 32 * (d + 8))
    k, v = (x.permute(0, 2, 1, 3, 4, 5).reshape(b * hkv, size, d).float() for x in _unpack(block, d))
    lens, off = st["lens"].long(), st["off"].long()
    q = st["q"].reshape(b, nq, hkv, hq // hkv, d).transpose(1, 2).reshape(b * hkv, -1, d).float()
    s = torch.matmul(q, k.transpose(1, 2).contiguous()).reshape(b, hkv, nq, hq // hkv, -1) * (1 / math.sqrt(d))
    token = torch.arange(size, device="cuda")
    bits = (st["mask"].reshape(b, nq, words, 1) >> torch.arange(64, device="cuda") & 1).reshape(b, nq, 64 * words).bool()
    node = token - off[:, None]
    inside = (node >= 0) & (node < 64 * words) & (token < lens[:, None])
    seen = torch.gather(bits, 2, node.clamp(0, 64 * words - 1)[:, None].expand(b, nq, size)) & inside[:, None]
    seen |= (node < 0)[:, None]
    s = s.masked_fill(~seen[:, None, :, None, :], -math.inf)
    top = s.amax(-1, keepdim=True).clamp(min=LOWEST)
    p = (s - top).exp()
    del s
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(b * hkv, -1, size), v).reshape(b, hkv, nq, hq // hkv, d)
    o = torch.where(total > 0, o / total, 0.0).transpose(1, 2).reshape(b * nq, hq, d)
    lse = torch.where(total > 0, total.log() + top, LOWEST)[..., 0].transpose(1, 2).reshape(b * nq, hq)
    st["out"].copy_(o)
    st["lse"].copy_(lse)
    return st["out"], st["lse"]


def _verify_plain(st):
    c = st["case"]
    b, n, v, drawn = c["batch"], c["nodes"], c["vocab"], c["drawn"]
    first = st["start"][:-1].long()
    tokens, parent, u = st["tokens"].reshape(b, n), st["parent"].long().reshape(b, n), st["u"].double().reshape(b, n)
    seq = torch.arange(b, device="cuda")
    cur = torch.zeros(b, device="cuda", dtype=torch.int64)
    accepted = torch.zeros(b, n, device="cuda", dtype=torch.bool)
    accepted[:, 0] = True
    zero, one = torch.zeros(b, device="cuda", dtype=torch.float64), torch.ones(b, device="cuda", dtype=torch.float64)
    a, s, z = zero, zero, one  # of the current node: share of q taken off p, mass of rejected drafts, mass that is left
    out = torch.zeros(b, v, device="cuda", dtype=torch.bool)  # rejected tokens of the current node
    for i in range(1, n):  # a node's children come after it, siblings in their order
        mine = parent[:, i] == cur
        x = tokens[:, i]
        px = st["p"][first + cur, x].double()
        fresh = mine & ~out[seq, x]
        if drawn:
            qx = st["q"][first + cur, x].double()
            take = fresh & (u[:, i] * qx * z < (px - a * qx).clamp(min=0) * (1 - s))
            drop = fresh & ~take
            a = torch.where(drop, a + z / (1 - s), a)
            s = torch.where(drop, s + qx, s)
            if c["shape"] != "chain":
                left = (st["p"][first + cur].double() - a[:, None] * st["q"][first + cur].double()).clamp(min=0).sum(-1)
                z = torch.where(drop, left, z)
        else:
            take = fresh & (u[:, i] * z < px)
            drop = fresh & ~take
            z = torch.where(drop, z - px, z)
        out[seq, x] |= drop
        accepted[:, i] = take
        cur = torch.where(take, i, cur)
        a, s, z = torch.where(take, zero, a), torch.where(take, zero, s), torch.where(take, one, z)
        out &= ~take[:, None]
    w = st["p"][first + cur].double()
    w = (w - a[:, None] * st["q"][first + cur].double()).clamp(min=0) if drawn else w.masked_fill(out, 0.0)
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, st["p"][first + cur].double())
    sums = w.cumsum(-1)
    st["next"].copy_((sums <= u[:, :1] * sums[:, -1:]).sum(-1))
    st["count"].copy_(accepted.sum(-1))
    order = torch.where(accepted, torch.arange(n, device="cuda"), n).sort(-1).values
    st["path"].copy_(torch.where(order < n, order, -1).reshape(-1))
    return st["path"], st["count"], st["next"]


def _commit_plain(st):
    c = st["case"]
    n, page, hkv, d = c["nodes"], c["page"], c["hkv"], c["d"]
    start, lens = st["start"].long(), st["lens"].long()
    kept = torch.nonzero(st["path"] >= 0)[:, 0]
    seq = torch.div(kept, n, rounding_mode="floor")

    def slot(place):
        at = lens[seq] + place
        return st["table"][seq, at // page].long() * page + at % page

    source = _token_bytes(slot(st["path"][kept].long()), hkv, d, page)
    target = _token_bytes(slot(kept - start[seq]), hkv, d, page)
    for pages, k_out, v_out in zip(st["pages"], st["k_out"], st["v_out"]):
        flat = pages.view(-1)
        row = flat[source]
        flat[target] = row
        kb, vb, kp, vp = row.split([d // 2, d // 2, 4, 4], -1)
        kp, vp = (x.contiguous().view(torch.float16) for x in (kp, vp))
        for out, x, pair in ((k_out, kb, kp), (v_out, vb, vp)):
            out.copy_(_value(torch.stack([x & 15, x >> 4], -1).flatten(-2), pair[..., :1], pair[..., 1:]))
    st["new"].copy_(lens + st["count"])
    return (st["new"], *st["k_out"], *st["v_out"])


def run(st):
    c = st["case"]
    if not own:
        return {"tree": _tree_plain, "attend": _attend_plain, "verify": _verify_plain, "commit": _commit_plain}[c["op"]](st)
    kv = st["kv"]
    if c["op"] == "tree":
        kv.tree(st["parent"], st["start"], st["lens"], st["table"], c["nodes"], st["mask"], positions=st["positions"],
                slots=st["slots"], total_len=st["total"])
        return st["mask"], st["positions"], st["slots"], st["total"]
    if c["op"] == "attend":
        kv.attend(st["pages"], st["q"], st["lens"], st["table"], st["out"], lse=st["lse"], q_start=st["start"],
                  max_q=c["queries"], q_off=st["off"], max_kv=c["len_max"], workspace=st["workspace"], tree=st["mask"])
        return st["out"], st["lse"]
    if c["op"] == "verify":
        kv.verify(st["tokens"], st["parent"], st["start"], st["p"], st["u"], st["path"], st["count"], st["next"],
                  max_q=c["nodes"], q=st["q"], max_children=st["children"], workspace=st["workspace"])
        return st["path"], st["count"], st["next"]
    kv.commit(st["pages"], st["start"], st["lens"], st["path"], st["count"], st["table"], c["nodes"], new_len=st["new"])
    for pages, k_out, v_out in zip(st["pages"], st["k_out"], st["v_out"]):
        kv.read(pages, st["slots"], k_out, v_out)
    return (st["new"], *st["k_out"], *st["v_out"])


# ---------------------------------------------------------------- the definition, in 64 bits

def _exact_tree(st):
    c = st["case"]
    parent, start, lens, table = (st[k].tolist() for k in ("parent", "start", "lens", "table"))
    mask, positions, slots, total = [], [], [], []
    for b, n in enumerate(lens):
        for i in range(start[b + 1] - start[b]):
            chain, at = [], i
            while at >= 0:
                chain.append(at)
                at = parent[start[b] + at]
            words = [0] * c["words"]
            for a in chain:
                words[a // 64] += 1 << a % 64
            mask.append([w - (1 << 64) if w >= 1 << 63 else w for w in words])
            positions.append(n + len(chain) - 1)
            slots.append(table[b][(n + i) // c["page"]] * c["page"] + (n + i) % c["page"])
        total.append(n + start[b + 1] - start[b])
    as_long = lambda x: torch.tensor(x, dtype=torch.int64, device="cuda")  # noqa: E731
    return as_long(mask).reshape(-1, c["words"]), as_long(positions), as_long(slots), _int(total)


def _held(blk, d):
    """Keys and values (tokens, D) in 64 bits of blocks (n, 32 (D + 8)), nibble by nibble."""
    ch, tok = torch.arange(d, device="cuda"), torch.arange(32, device="cuda")
    kbyte, kshift = tok[:, None] * (d // 2) + ch // 2, ch % 2 * 4
    run_, rest = ch // (d // 16), ch % (d // 16)
    e = tok // 16 * 4 + tok % 4
    vhalf = ((rest // 4 * 4 + (tok // 4 % 4)[:, None]) * 16 + run_) * 8 + e[:, None]
    vbyte, vshift = 16 * d + vhalf * 2 + rest % 4 // 2, rest % 2 * 4
    vat = (tok // 4 % 4) * 8 + e
    par = blk[:, 32 * d:].contiguous().view(torch.float16).double()
    out = []
    for byte, shift, s, o in ((kbyte, kshift, par[:, 0:64:2], par[:, 1:64:2]),
                              (vbyte, vshift, par[:, 64 + vat], par[:, 96 + vat])):
        nib = (blk[:, byte.reshape(-1)].reshape(-1, 32, d) >> shift.to(torch.uint8)) & 15
        out.append(((nib.double() + 16) * s[..., None] + o[..., None]).half().double().reshape(-1, d))
    return out


def _exact_attend(st):
    c = st["case"]
    hq, hkv, d, page, nq = (c[k] for k in ("hq", "hkv", "d", "page", "queries"))
    grp = hq // hkv
    out = torch.zeros(st["q"].shape, device="cuda", dtype=torch.float64)
    lse = torch.full(st["lse"].shape, LOWEST, device="cuda", dtype=torch.float64)
    masks, off = st["mask"].tolist(), st["off"].tolist()
    for b, n in enumerate(st["lens"].tolist()):
        first = b * nq
        hidden = torch.ones(nq, n, dtype=torch.bool)
        for i in range(nq):
            hidden[i, :max(0, off[b])] = False
            m = sum((w & (1 << 64) - 1) << 64 * k for k, w in enumerate(masks[first + i]))
            for j in range(off[b], n):
                if m >> j - off[b] & 1:
                    hidden[i, j] = False
        hidden = hidden.cuda().repeat_interleave(grp, 0)
        ids = st["table"][b, :-(-n // page)].long()
        for h in range(hkv):
            blk = st["pages"].view(-1, hkv, page // 32, 32 * (d + 8))[ids, h].reshape(-1, 32 * (d + 8))
            key, value = (x[:n] for x in _held(blk, d))
            q = st["q"][first:first + nq, h * grp:(h + 1) * grp].double().reshape(nq * grp, d)
            step = max(1, (1 << 28) // n)
            for at in range(0, nq * grp, step):
                part = slice(at, min(nq * grp, at + step))
                s = (q[part] @ key.t().contiguous() / math.sqrt(d)).masked_fill_(hidden[part], -math.inf)
                z = torch.logsumexp(s, -1)
                r = torch.arange(nq * grp, device="cuda")[part]
                out[first + r // grp, h * grp + r % grp] = torch.nan_to_num((s - z[:, None]).exp_(), nan=0.0) @ value
                lse[first + r // grp, h * grp + r % grp] = z.clamp(min=LOWEST)
    return out, lse


def _exact_verify(st):
    c = st["case"]
    n, b = c["nodes"], c["batch"]
    tokens, parent, u = st["tokens"].tolist(), st["parent"].tolist(), st["u"].tolist()
    path, count, drawn_tokens = [], [], []
    for s in range(b):
        cur, taken = 0, [0]
        while True:
            target = st["p"][s * n + cur].double()
            draft = st["q"][s * n + cur].double() if c["drawn"] else None
            nxt = None
            for i in range(cur + 1, n):
                if parent[s * n + i] != cur:
                    continue
                x = tokens[s * n + i]
                proposal = draft if c["drawn"] else torch.zeros_like(target).index_fill_(0, torch.tensor([x], device="cuda"), 1.0)
                if proposal[x].item() <= 0 and target[x].item() <= 0:
                    continue  # a sibling's token again
                if u[s * n + i] * proposal[x].item() < target[x].item():
                    nxt = i
                    break
                rest = (target - proposal).clamp(min=0)
                if rest.sum().item() <= 0:  # nothing left: the target's own
                    target = st["p"][s * n + cur].double()
                    break
                target = rest / rest.sum()
                if c["drawn"]:  # the next one was drawn from what was left of the draft
                    draft = draft.clone()
                    draft[x] = 0
                    draft = draft / draft.sum()
            if nxt is None:
                break
            cur = nxt
            taken.append(cur)
        sums = target.cumsum(0)
        drawn_tokens.append(int((sums <= u[s * n] * sums[-1]).sum().item()))
        count.append(len(taken))
        path += taken + [-1] * (n - len(taken))
    return _int(path), _int(count), torch.tensor(drawn_tokens, dtype=torch.int64, device="cuda")


def _exact_commit(st):
    c = st["case"]
    n, page, hkv, d = c["nodes"], c["page"], c["hkv"], c["d"]
    path, lens, table = (st[k].tolist() for k in ("path", "lens", "table"))
    source = []
    for s, m in enumerate(lens):
        for x in path[s * n:(s + 1) * n]:
            if x >= 0:
                source.append(table[s][(m + x) // page] * page + (m + x) % page)
    source = torch.tensor(source, device="cuda")
    keys, values = [], []
    for pages in st["pages"]:
        blk = pages.view(-1, hkv, page // 32, 32 * (d + 8))[source // page, :, source % page // 32]  # (kept, hkv, bytes)
        k, v = (x.reshape(-1, hkv, 32, d) for x in _held(blk.reshape(-1, 32 * (d + 8)), d))
        at = torch.arange(source.shape[0], device="cuda")
        keys.append(k[at, :, source % 32])
        values.append(v[at, :, source % 32])
    kept = [sum(x >= 0 for x in path[s * n:(s + 1) * n]) for s in range(c["batch"])]
    return (_int([m + k for m, k in zip(lens, kept)]), *keys, *values)


def exact(case, seed):
    st = prepare(case, seed)
    return {"tree": _exact_tree, "attend": _exact_attend, "verify": _exact_verify, "commit": _exact_commit}[case["op"]](st)
