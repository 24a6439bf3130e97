"""Latent attention over a paged cache, and the cache's pages: workloads and plain forms.

Five operators of the library, each with the calls a serving program makes
(``own``) and the same result in elementary torch operations:

decode    absorbed latent attention of the newest tokens of a batch of sequences
prefix    the same for a batch whose sequences share a long prefix
prefill   expanded latent attention of a block of prompt tokens
fork      sequences become copies of others (full pages shared, the last page copied)
turnover  sequences leave, the pages are compacted, new sequences are admitted and stored

A cache row is one token's latent vector (``rank`` values) and its rotary key
(``rope`` values) in bf16.  The sizes are the ones the library's workloads use
(hidden 4096 = 32 heads of 128, batches of 32, blocks of 8192 and 16384
tokens, stacks of 4 layers) or generic.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
HEAD_DIM = 128     # dimensions a head has without its rotary part, and of its values


def listed():
    return [
        # one user, a short conversation: latency
        dict(name="decode one short", kind="decode", batch=1, queries=1, heads=32, rank=512, rope=64, page=16,
             shortest=333, longest=333),
        # a batch of agents in mid-conversation, ragged
        dict(name="decode batch", kind="decode", batch=32, queries=1, heads=64, rank=512, rope=64, page=64,
             shortest=250, longest=6001),
        # few long documents, two tokens verified at once, many heads
        dict(name="decode long", kind="decode", batch=4, queries=2, heads=128, rank=512, rope=64, page=128,
             shortest=40001, longest=65537),
        # a small fan-out of one system prompt
        dict(name="prefix small", kind="prefix", batch=8, queries=1, heads=16, rank=512, rope=64, page=32,
             shared=1024, shortest=1, longest=200),
        # a large fan-out of one long document
        dict(name="prefix large", kind="prefix", batch=64, queries=1, heads=32, rank=512, rope=64, page=64,
             shared=16384, shortest=17, longest=1500),
        # a few short prompts in one call, a single token among them
        dict(name="prefill ragged", kind="prefill", batch=5, heads=32, rank=512, rope=64, page=16,
             new_shortest=1, new_longest=300, context=0),
        # a chunk of a long prompt over what is cached already
        dict(name="prefill chunk", kind="prefill", batch=1, heads=16, rank=512, rope=64, page=64,
             new_shortest=1000, new_longest=1000, context=15001),
        # one prompt block
        dict(name="prefill block", kind="prefill", batch=1, heads=32, rank=512, rope=64, page=64,
             new_shortest=8192, new_longest=8192, context=0),
        # beams of a search change their parents in place
        dict(name="fork beams", kind="fork", batch=16, parents=0, layers=1, rank=512, rope=64, page=16,
             shortest=100, longest=500),
        # agents branch off long contexts, all layers of a stack at once
        dict(name="fork agents", kind="fork", batch=64, parents=8, layers=4, rank=512, rope=64, page=64,
             shortest=2000, longest=16384),
        # short requests come and go
        dict(name="turnover small", kind="turnover", batch=32, groups=8, layers=1, rank=512, rope=64, page=16,
             shortest=20, longest=300),
        # long requests come and go, all layers of a stack
        dict(name="turnover large", kind="turnover", batch=64, groups=4, layers=4, rank=512, rope=64, page=64,
             shortest=500, longest=6000),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["decode", "prefix", "prefill", "fork", "turnover"])
    c = dict(kind=kind, rank=rng.choice([256, 512, 512]), rope=rng.choice([32, 64, 64]), page=rng.choice([16, 32, 64, 128]))
    if kind == "decode":
        c["batch"] = _log_int(rng, 1, 64)
        c["queries"] = rng.choice([1, 1, 1, 2, 3])
        c["heads"] = rng.choice([8, 16, 20, 32, 64, 128])
        c["longest"] = _log_int(rng, 100, min(65537, 250000 // c["batch"])) | 1
        c["shortest"] = rng.randint(1, c["longest"])
    elif kind == "prefix":
        c["batch"] = _log_int(rng, 2, 64)
        c["queries"] = rng.choice([1, 1, 2])
        c["heads"] = rng.choice([8, 16, 20, 32])
        c["shared"] = 128 * (_log_int(rng, 4, 126 // c["queries"]) | 1)
        c["longest"] = _log_int(rng, 4, 1500) | 1
        c["shortest"] = rng.randint(c["queries"], c["longest"])
    elif kind == "prefill":
        c["batch"] = rng.choice([1, 1, 2, 3, 6])
        c["heads"] = rng.choice([8, 16, 20, 32])
        c["context"] = rng.choice([0, 0, _log_int(rng, 10, 4000)])
        c["new_longest"] = _log_int(rng, 16, (4096 if c["context"] else 8192) // c["batch"])
        c["new_shortest"] = rng.randint(1, c["new_longest"])
    elif kind == "fork":
        c["batch"] = _log_int(rng, 4, 64)
        c["parents"] = rng.choice([0, 1, 3, 8])
        c["layers"] = rng.choice([1, 2, 4])
        c["longest"] = _log_int(rng, 50, 16384 if c["parents"] else 4000) | 1
        c["shortest"] = rng.randint(1, c["longest"])
    else:
        c["batch"] = _log_int(rng, 8, 64)
        c["groups"] = rng.choice([2, 4, 8])
        c["layers"] = rng.choice([1, 2, 4])
        c["longest"] = _log_int(rng, 50, 5999) | 1
        c["shortest"] = rng.randint(1, c["longest"])
    return c


# ------------------------------------------------------------------ inputs
def _lengths(seed, lo, hi, n):
    """n lengths from lo to hi, the same ones for every seed and in an order that the seed gives."""
    v = np.random.RandomState(n).randint(lo, hi + 1, n)
    v[0] = hi
    if n > 1:
        v[-1] = lo
    return np.random.RandomState(seed % (1 << 31)).permutation(v)


def _sizes(case, seed):
    """Tokens held by each sequence."""
    k = case["kind"]
    if k == "decode":
        return _lengths(seed, max(case["shortest"], case["queries"]), max(case["longest"], case["queries"]),
                        case["batch"])
    if k == "prefix":
        return case["shared"] + _lengths(seed, case["shortest"], case["longest"], case["batch"])
    if k == "prefill":
        return case["context"] + _lengths(seed, case["new_shortest"], case["new_longest"], case["batch"])
    if k == "fork" and case["parents"]:
        return np.concatenate([_lengths(seed, case["shortest"], case["longest"], case["parents"]),
                               np.zeros(case["batch"], np.int64)])
    return _lengths(seed, case["shortest"], case["longest"], case["batch"])


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = np.random.RandomState((seed * 7 + 1) % (1 << 31))
    k, page, row = case["kind"], case["page"], case["rank"] + case["rope"]
    lens = _sizes(case, seed)
    blocks = -(-lens // page)
    shared = case.get("shared", 0) // page
    held = int(blocks.sum()) - shared * (len(lens) - 1)
    layers = case.get("layers", 1)
    in_order = k == "turnover"                     # a turnover starts from a compact pool
    spare = 3 * case["batch"] + 8 if k == "fork" else 8 + held // 8
    n_pages = held + spare
    order = np.arange(n_pages) if in_order else r.permutation(n_pages)   # elsewhere pages lie anywhere
    max_blocks = int(blocks.max()) + 1
    table = np.full((len(lens), max_blocks), -1, np.int32)
    refs = np.zeros(n_pages, np.int32)
    at = 0
    for i, n in enumerate(blocks):
        first = shared if i else 0
        table[i, :first] = table[0, :first]
        table[i, first:n] = order[at:at + n - first]
        at += n - first
    np.add.at(refs, table[table >= 0], 1)
    s = dict(case=case,
             pages=torch.empty(layers, n_pages, page, row, device=DEV, dtype=torch.bfloat16).normal_(generator=g),
             table=torch.from_numpy(table).to(DEV), lens=torch.from_numpy(lens.astype(np.int32)).to(DEV),
             refs=torch.from_numpy(refs).to(DEV))
    ids = torch.arange(len(lens), dtype=torch.int32, device=DEV)
    if k in ("decode", "prefix"):
        s["seqs"] = ids.flip(0).contiguous() if k == "decode" else ids
        s["q"] = torch.empty(case["batch"] * case["queries"], case["heads"], row, device=DEV,
                             dtype=torch.bfloat16).normal_(generator=g)
        s["scale"] = (HEAD_DIM + case["rope"]) ** -0.5
    elif k == "prefill":
        new = lens - case["context"]
        off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        s["seqs"] = ids
        s["q_offsets"] = torch.from_numpy(off).to(DEV)
        s["total"], s["held"] = int(off[-1]), int(lens.sum())
        s["q"] = torch.empty(s["total"], case["heads"], HEAD_DIM + case["rope"], device=DEV,
                             dtype=torch.bfloat16).normal_(generator=g)
        s["w_kv"] = torch.empty(case["heads"], 2 * HEAD_DIM, case["rank"], device=DEV,
                                dtype=torch.bfloat16).normal_(std=case["rank"] ** -0.5, generator=g)
        s["scale"] = (HEAD_DIM + case["rope"]) ** -0.5
    elif k == "fork":
        n = case["batch"]
        if case["parents"]:
            src, dst = r.randint(0, case["parents"], n), case["parents"] + np.arange(n)
        else:
            src, dst = r.randint(0, n, n), np.arange(n)      # beams: some survive in place, some are replaced
        s["src"] = torch.from_numpy(src.astype(np.int32)).to(DEV)
        s["dst"] = torch.from_numpy(dst.astype(np.int32)).to(DEV)
    else:
        # groups of sequences leave in turn and others of the same lengths are admitted in their place
        groups = [np.arange(i, case["batch"], case["groups"]) for i in range(case["groups"])]
        s["turn"], s["groups"] = 0, []
        for ids_g in groups:
            n_new = lens[ids_g]
            s["groups"].append(dict(
                seqs=torch.from_numpy(ids_g.astype(np.int32)).to(DEV), n_new=torch.from_numpy(n_new.astype(np.int32)).to(DEV),
                tok_seq=torch.from_numpy(np.repeat(ids_g, n_new).astype(np.int32)).to(DEV),
                tok_pos=torch.from_numpy(np.concatenate([np.arange(n) for n in n_new]).astype(np.int32)).to(DEV)))
        most = max(len(x["tok_seq"]) for x in s["groups"])
        s["rows"] = torch.empty(layers, most, row, device=DEV, dtype=torch.bfloat16).normal_(generator=g)
    return s


def run(state):
    k = state["case"]["kind"]
    if own:
        return {"decode": _own_decode, "prefix": _own_decode, "prefill": _own_prefill, "fork": _own_fork,
                "turnover": _own_turnover}[k](state)
    return {"decode": _decode, "prefix": _decode, "prefill": _prefill, "fork": _fork, "turnover": _turnover}[k](state)


# ------------------------------------------------------------------ the library's calls
def _handle(s):
    """The cache handle, status word and workspace that a serving program makes once."""
    if "handle" not in s:
        import edge_moe_serving_gb300 as moe
        c = s["case"]
        h = moe.moe_kv_cache(s["pages"].data_ptr(), s["table"].data_ptr(), s["lens"].data_ptr(), s["refs"].data_ptr(),
                             s["pages"].shape[0], s["pages"].shape[1], c["page"], c["rank"], c["rope"],
                             s["table"].shape[0], s["table"].shape[1], 0)
        if c["kind"] in ("decode", "prefix"):
            n = moe.moe_latent_decode_workspace_size(h, c["batch"], c["queries"], c["heads"], c.get("shared", 0))
            s["out"] = torch.empty(c["batch"] * c["queries"], c["heads"], c["rank"], device=DEV, dtype=torch.bfloat16)
        elif c["kind"] == "prefill":
            n = moe.moe_latent_prefill_workspace_size(h, c["batch"], s["total"], c["heads"], HEAD_DIM, HEAD_DIM, s["held"])
            s["out"] = torch.empty(s["total"], c["heads"], HEAD_DIM, device=DEV, dtype=torch.bfloat16)
        else:
            n = moe.moe_kv_workspace_size(h, c["batch"])
        s["ws"] = torch.empty(max(n, 256), device=DEV, dtype=torch.uint8)
        s["status"] = torch.zeros(1, device=DEV, dtype=torch.int32)
        s["handle"] = (moe, h)
    return s["handle"]


def _own_decode(s):
    moe, h = _handle(s)
    c = s["case"]
    moe.moe_latent_decode(h, 0, s["q"], s["seqs"], c["batch"], c["queries"], c["heads"], s["scale"], c.get("shared", 0),
                          s["out"], None, s["ws"], s["ws"].numel(), s["status"])
    return s["out"]


def _own_prefill(s):
    moe, h = _handle(s)
    c = s["case"]
    moe.moe_latent_prefill(h, 0, s["q"], s["seqs"], s["q_offsets"], c["batch"], s["total"], c["heads"], HEAD_DIM, HEAD_DIM,
                           s["w_kv"], s["scale"], s["held"], s["out"], s["ws"], s["ws"].numel(), s["status"])
    return s["out"]


def _own_fork(s):
    moe, h = _handle(s)
    moe.moe_kv_fork(h, s["src"], s["dst"], s["src"].numel(), s["ws"], s["ws"].numel(), s["status"])
    return dict(pages=s["pages"], table=s["table"], lens=s["lens"], refs=s["refs"])


def _own_turnover(s):
    moe, h = _handle(s)
    x = s["groups"][s["turn"]]
    s["turn"] = (s["turn"] + 1) % len(s["groups"])
    n = x["seqs"].numel()
    moe.moe_kv_free(h, x["seqs"], n, s["status"])
    moe.moe_kv_compact(h, None, s["ws"], s["ws"].numel(), s["status"])
    moe.moe_kv_reserve(h, x["seqs"], x["n_new"], n, s["ws"], s["ws"].numel(), s["status"])
    for layer in range(s["pages"].shape[0]):
        moe.moe_kv_append(h, layer, s["rows"][layer], x["tok_seq"], x["tok_pos"], x["tok_seq"].numel(), s["status"])
    return dict(pages=s["pages"], table=s["table"], lens=s["lens"], refs=s["refs"])


# ------------------------------------------------------------------ plain forms
def _gather(s, rows, first, last):
    """Cache rows of blocks [first, last) of the given sequences, in 32 bits: [n, tokens, rank + rope]."""
    ids = s["table"][rows, first:last].long().clamp(min=0)
    x = s["pages"][0][ids]
    return x.reshape(x.shape[0], -1, x.shape[-1]).float()


def _softmax_parts(scores, mask):
    """exp(scores - m), its sum and m, with masked places at zero and rows that have none left at m = 0."""
    scores = scores.masked_fill(~mask, -math.inf)
    m = scores.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(scores - m)
    return p, p.sum(-1, keepdim=True), m


def _decode(s):
    c = s["case"]
    seqs, rank, page = s["seqs"].long(), c["rank"], c["page"]
    n, nq, heads = c["batch"], c["queries"], c["heads"]
    lens = s["lens"][seqs].long()
    limit = lens[:, None] - nq + torch.arange(1, nq + 1, device=DEV)           # tokens each query sees
    limit = limit[:, :, None].expand(n, nq, heads).reshape(n, nq * heads, 1)
    q = s["q"].float().view(n, nq * heads, -1)
    shared = c.get("shared", 0)
    kv = _gather(s, seqs, shared // page, s["table"].shape[1])
    pos = shared + torch.arange(kv.shape[1], device=DEV)
    p, l, m = _softmax_parts(torch.bmm(q, kv.transpose(1, 2)) * s["scale"], pos < limit)
    o = torch.bmm(p, kv[:, :, :rank])
    if shared:                                                                 # the prefix, once for all rows
        kv = _gather(s, seqs[:1], 0, shared // page)[0]
        pos = torch.arange(shared, device=DEV)
        p, l2, m2 = _softmax_parts(torch.matmul(q, kv.T) * s["scale"], pos < limit)
        o2 = torch.matmul(p, kv[:, :rank])
        top = torch.maximum(m, m2)
        a, b = torch.exp(m - top), torch.exp(m2 - top)
        o, l = o * a + o2 * b, l * a + l2 * b
    o = o / torch.where(l == 0, torch.ones_like(l), l)
    return o.to(torch.bfloat16).view(n * nq, heads, rank)


def _prefill(s):
    c = s["case"]
    seqs, off = s["seqs"].long(), s["q_offsets"].long()
    n, heads, rank = c["batch"], c["heads"], c["rank"]
    kv = _gather(s, seqs, 0, s["table"].shape[1])                              # [n, S, row]
    lens, new = s["lens"][seqs].long(), off[1:] - off[:-1]
    both = torch.einsum("nsr,hdr->nhsd", kv[:, :, :rank], s["w_kv"].float())
    rope = kv[:, None, :, rank:].expand(n, heads, kv.shape[1], c["rope"])
    k, v = torch.cat([both[..., :HEAD_DIM], rope], -1), both[..., HEAD_DIM:]
    most = c["new_longest"]
    at = torch.arange(most, device=DEV)
    there = at < new[:, None]                                                  # [n, most]
    rows = (off[:-1, None] + at).clamp(max=s["total"] - 1)
    q = s["q"].float()[rows].transpose(1, 2)                                   # [n, heads, most, dim]
    limit = (lens - new)[:, None] + at + 1
    mask = torch.arange(kv.shape[1], device=DEV) < limit[:, None, :, None]
    p, l, _ = _softmax_parts(torch.matmul(q, k.transpose(2, 3)) * s["scale"], mask)
    o = (torch.matmul(p, v) / l).transpose(1, 2)                               # [n, most, heads, dim]
    return o[there].to(torch.bfloat16)


def _plain_fork(s, src, dst):
    page = s["case"]["page"]
    src, dst = src.long(), dst.long()
    moved = src != dst
    src, dst = src[moved], dst[moved]
    lens, new = s["lens"][src].clone(), s["table"][src].clone()
    old = s["table"][dst]
    free = torch.nonzero(s["refs"] == 0)[:, 0]                                 # ascending
    part = torch.nonzero(lens % page)[:, 0]
    last = (lens[part] // page).long()
    to, frm = free[:part.numel()], new[part, last].long()
    valid = torch.arange(page, device=DEV) < (lens[part] % page)[:, None]
    s["pages"][:, to] = torch.where(valid[..., None], s["pages"][:, frm], s["pages"][:, to])
    new[part, last] = to.int()
    one = torch.ones((), dtype=torch.int32, device=DEV)
    s["refs"].index_put_((old[old >= 0].long(),), -one, accumulate=True)
    s["refs"].index_put_((new[new >= 0].long(),), one, accumulate=True)
    s["table"][dst] = new
    s["lens"][dst] = lens


def _fork(s):
    _plain_fork(s, s["src"], s["dst"])
    return dict(pages=s["pages"], table=s["table"], lens=s["lens"], refs=s["refs"])


def _turnover(s):
    x = s["groups"][s["turn"]]
    s["turn"] = (s["turn"] + 1) % len(s["groups"])
    page, seqs = s["case"]["page"], x["seqs"].long()
    one = torch.ones((), dtype=torch.int32, device=DEV)
    # free
    old = s["table"][seqs]
    s["refs"].index_put_((old[old >= 0].long(),), -one, accumulate=True)
    s["table"][seqs] = -1
    s["lens"][seqs] = 0
    # compact
    live = s["refs"] > 0
    at = torch.arange(live.numel(), device=DEV)
    n_live = live.sum()
    movers, holes = torch.nonzero(live & (at >= n_live))[:, 0], torch.nonzero(~live & (at < n_live))[:, 0]
    s["pages"][:, holes] = s["pages"][:, movers]
    s["refs"][holes] = s["refs"][movers]
    s["refs"][movers] = 0
    at[movers] = holes
    s["table"].copy_(torch.where(s["table"] >= 0, at[s["table"].long().clamp(min=0)].int(), s["table"]))
    # reserve
    need = (x["n_new"].long() + page - 1) // page
    free = torch.nonzero(s["refs"] == 0)[:, 0]
    who = torch.repeat_interleave(torch.arange(need.numel(), device=DEV), need)
    block = torch.arange(who.numel(), device=DEV) - (need.cumsum(0) - need)[who]
    s["table"][seqs[who], block] = free[:who.numel()].int()
    s["refs"][free[:who.numel()]] = 1
    s["lens"][seqs] = x["n_new"]
    # append
    pos = x["tok_pos"].long()
    pages = s["table"][x["tok_seq"].long(), pos // page].long()
    s["pages"][:, pages, pos % page] = s["rows"][:, :pos.numel()]
    return dict(pages=s["pages"], table=s["table"], lens=s["lens"], refs=s["refs"])


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    k, rank, page = case["kind"], case["rank"], case["page"]
    row = rank + case["rope"]
    lens = _sizes(case, 1)
    if k in ("decode", "prefix"):
        shared, rows = case.get("shared", 0), case["batch"] * case["queries"] * case["heads"]
        tokens = int(lens.sum()) - shared * (case["batch"] - 1)
        pairs = int(lens.sum()) * case["queries"] * case["heads"]
        return {"bytes": tokens * row * 2 + rows * (row + rank) * 2, "flops": 2 * pairs * (row + rank)}
    if k == "prefill":
        new = lens - case["context"]
        pairs = sum(int(a) * case["context"] + int(a) * (int(a) + 1) // 2 for a in new) * case["heads"]
        dim = 2 * HEAD_DIM + case["rope"]
        total, held = int(new.sum()), int(lens.sum())
        return {"bytes": held * row * 2 + case["heads"] * (2 * HEAD_DIM * rank + total * dim) * 2,
                "flops": 2 * pairs * dim + 2 * held * rank * 2 * HEAD_DIM * case["heads"]}
    if k == "fork":
        parents = case["parents"] or case["batch"]
        mean = float(lens[:parents].mean())
        moved = case["batch"] if case["parents"] else case["batch"] - 1
        part = float((lens[:parents] % page).mean())
        return {"bytes": moved * (2 * case["layers"] * part * row * 2 + 4 * 4 * mean / page), "flops": 0}
    gone, tokens = int((-(-lens // page)).sum()) // case["groups"], int(lens.sum()) // case["groups"]
    return {"bytes": case["layers"] * row * 2 * (2 * gone * page + 2 * tokens) + 4 * (8 * gone + 2 * tokens), "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    k = case["kind"]
    s = prepare(case, seed)
    return {"decode": _exact_decode, "prefix": _exact_decode, "prefill": _exact_prefill, "fork": _exact_fork,
            "turnover": _exact_turnover}[k](s)


def _tokens_of(s, seq):
    """The rows of one sequence in 64 bits, page after page."""
    n, page = int(s["lens"][seq]), s["case"]["page"]
    ids = s["table"][seq].tolist()[:-(-n // page)]
    return torch.cat([s["pages"][0, i] for i in ids])[:n].double()


def _attend(q, k, v, scale, hidden):
    """One head group: q [r, d], k [t, d], v [t, e]; hidden [r] = how many of the last tokens a row does not see."""
    t = torch.arange(k.shape[0], device=DEV)
    z = (q @ k.T) * scale
    z[t[None] >= (k.shape[0] - hidden)[:, None]] = -math.inf
    return torch.softmax(z, -1) @ v


def _exact_decode(s):
    c = s["case"]
    out = []
    for b, seq in enumerate(s["seqs"].tolist()):
        x = _tokens_of(s, seq)
        q = s["q"][b * c["queries"]:(b + 1) * c["queries"]].double()
        for i in range(c["queries"]):
            hidden = torch.full((c["heads"],), c["queries"] - 1 - i, device=DEV)
            out.append(_attend(q[i], x, x[:, :c["rank"]], s["scale"], hidden))
    return torch.stack(out)


def _exact_prefill(s):
    c = s["case"]
    off = s["q_offsets"].tolist()
    out = torch.empty(s["total"], c["heads"], HEAD_DIM, dtype=torch.float64, device=DEV)
    for b, seq in enumerate(s["seqs"].tolist()):
        x = _tokens_of(s, seq)
        n = off[b + 1] - off[b]
        hidden = n - 1 - torch.arange(n, device=DEV)
        for h in range(c["heads"]):
            w = s["w_kv"][h].double()
            k = torch.cat([x[:, :c["rank"]] @ w[:HEAD_DIM].T, x[:, c["rank"]:]], 1)
            v = x[:, :c["rank"]] @ w[HEAD_DIM:].T
            for a in range(0, n, 2048):
                z = min(n, a + 2048)
                out[off[b] + a:off[b] + z, h] = _attend(s["q"][off[b] + a:off[b] + z, h].double(), k, v, s["scale"], hidden[a:z])
    return out


def _state_of(pages, table, lens, refs):
    return dict(pages=pages.double(), table=torch.from_numpy(table), lens=torch.from_numpy(lens), refs=torch.from_numpy(refs))


def _exact_fork(s):
    """Sequence after sequence, on lists, from copies of what was there before."""
    page, pages = s["case"]["page"], s["pages"]
    table, lens, refs = (s[x].cpu().numpy().copy() for x in ("table", "lens", "refs"))
    table0, lens0, before = table.copy(), lens.copy(), pages.clone()
    free = [i for i in range(len(refs)) if refs[i] == 0]
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        if a == b:
            continue
        n = int(lens0[a])
        for i in table0[b]:
            if i >= 0:
                refs[i] -= 1
        new = [int(i) for i in table0[a]]
        if n % page:
            p = free.pop(0)
            pages[:, p, :n % page] = before[:, new[n // page], :n % page]
            new[n // page] = p
        for i in new:
            if i >= 0:
                refs[i] += 1
        table[b], lens[b] = new, n
    return _state_of(pages, table, lens, refs)


def _exact_turnover(s):
    page, pages, x = s["case"]["page"], s["pages"], s["groups"][0]
    table, lens, refs = (s[k].cpu().numpy().copy() for k in ("table", "lens", "refs"))
    for q in x["seqs"].tolist():
        for i in table[q]:
            if i >= 0:
                refs[i] -= 1
        table[q], lens[q] = -1, 0
    live = [i for i in range(len(refs)) if refs[i] > 0]
    holes = [i for i in range(len(live)) if refs[i] == 0]
    to = {}
    for i, h in zip([i for i in live if i >= len(live)], holes):
        pages[:, h] = pages[:, i]
        refs[h], refs[i], to[i] = refs[i], 0, h
    for q in range(len(lens)):
        table[q] = [to.get(int(i), int(i)) for i in table[q]]
    at = 0
    for q, n in zip(x["seqs"].tolist(), x["n_new"].tolist()):
        free = [i for i in range(len(refs)) if refs[i] == 0]
        for b in range(-(-n // page)):
            table[q, b], refs[free[b]] = free[b], 1
            rows = min(page, n - b * page)
            pages[:, free[b], :rows] = s["rows"][:, at:at + rows]
            at += rows
        lens[q] = n
    return _state_of(pages, table, lens, refs)
