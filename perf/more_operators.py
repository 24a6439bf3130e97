"""The latent cache held in 4 bits, and its eviction by attention weight: workloads and plain forms.

Five operators of the library, each with the calls a serving program makes
(``own``) and the same result in elementary torch operations:

store     rows of new tokens become 4-bit rows of the cache and are read back
decode    absorbed latent attention of the newest tokens over 4-bit pages, with or without a shared prefix
prefill   expanded latent attention of prompt tokens over 4-bit pages
weights   the attention weight that each cached token got, added to what it had before
evict     long sequences keep their heaviest tokens, and get room for their next chunk

A token's row is its latent vector (``rank`` values) and its rotary key
(``rope`` values, bf16).  In 4 bits, 16 neighbouring latent values share a
scale of 5 exponent and 3 significand bits, and each value is a number of
{0, 0.5, 1, 1.5, 2, 3, 4, 6} with a sign: rank / 2 bytes of values, the rotary
key, rank / 16 bytes of scales, filled up to a multiple of 16 bytes.  The sizes are
the ones the library's workloads use (32 heads of 128, batches of 32, stacks
of 4 layers) or generic.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
HEAD_DIM = 128     # dimensions a head has without its rotary part, and of its values
BLOCK = 16         # latent values that share a scale


def listed():
    return [
        # one step of a batch of agents: a token each, latency
        dict(name="store step", kind="store", batch=32, shortest=1, longest=1, context=700, rank=512, rope=64, page=16),
        # prompts of a batch, ragged
        dict(name="store prompts", kind="store", batch=8, shortest=250, longest=4001, context=0, rank=512, rope=64, page=64),
        # one user, a short conversation: latency
        dict(name="decode one short", kind="decode", batch=1, queries=1, heads=32, rank=512, rope=64, page=16,
             shortest=333, longest=333, shared=0),
        # a batch of agents in mid-conversation, a share of a model's heads, ragged
        dict(name="decode batch", kind="decode", batch=32, queries=1, heads=16, rank=512, rope=64, page=64,
             shortest=250, longest=6001, shared=0),
        # few long documents, which a cache in 4 bits has room for, two tokens verified at once
        dict(name="decode long", kind="decode", batch=4, queries=2, heads=32, rank=512, rope=64, page=128,
             shortest=40001, longest=65537, shared=0),
        # a fan-out of one long document
        dict(name="decode prefix", kind="decode", batch=64, queries=1, heads=32, rank=512, rope=64, page=64,
             shortest=17, longest=1500, shared=16384),
        # a few short prompts in one call, over a little context
        dict(name="prefill ragged", kind="prefill", batch=5, heads=32, rank=512, rope=64, page=16,
             new_shortest=1, new_longest=300, context=100),
        # a chunk of a long prompt over what is cached already
        dict(name="prefill chunk", kind="prefill", batch=1, heads=16, rank=512, rope=64, page=64,
             new_shortest=1000, new_longest=1000, context=15001),
        # after a decode step of a batch: what its queries looked at, old weight fading
        dict(name="weights batch", kind="weights", batch=32, queries=1, heads=64, rank=512, rope=64, page=64,
             shortest=250, longest=6001, bits=16, decay=0.98),
        # the last tokens of a long prompt vote on what is kept of it
        dict(name="weights window", kind="weights", batch=1, queries=32, heads=32, rank=512, rope=64, page=64,
             shortest=16001, longest=16001, bits=4, decay=1.0),
        # short conversations pass their budget
        dict(name="evict small", kind="evict", batch=8, layers=1, rank=512, rope=64, page=16,
             shortest=520, longest=700, budget=512, first=4, recent=64, shared=0),
        # long conversations off one system prompt, all layers of a stack
        dict(name="evict large", kind="evict", batch=32, layers=4, rank=512, rope=64, page=64,
             shortest=2500, longest=8192, budget=4096, first=4, recent=512, shared=1024),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["store", "decode", "prefill", "weights", "evict"])
    c = dict(kind=kind, rank=rng.choice([256, 512, 512]), rope=rng.choice([32, 64, 64]), page=rng.choice([16, 32, 64, 128]))
    if kind == "store":
        c["batch"] = _log_int(rng, 1, 64)
        c["context"] = rng.choice([0, rng.randint(1, 1000)])
        c["longest"] = _log_int(rng, 1, 16000 // c["batch"])
        c["shortest"] = rng.randint(1, c["longest"])
    elif kind == "decode":
        c["queries"] = rng.choice([1, 1, 1, 2, 3])
        c["heads"] = rng.choice([8, 16, 16, 20, 32])
        if rng.random() < 0.3:
            c["batch"] = _log_int(rng, 2, 64)
            c["shared"] = 128 * (_log_int(rng, 4, 126 // c["queries"]) | 1)
            c["longest"] = _log_int(rng, 4, 1500) | 1
        else:
            c["batch"] = _log_int(rng, 1, 64)
            c["shared"] = 0
            c["longest"] = _log_int(rng, 100, min(65537, 200000 // c["batch"])) | 1
        c["shortest"] = rng.randint(1, c["longest"])
    elif kind == "prefill":
        c["batch"] = rng.choice([1, 1, 2, 3, 6])
        c["heads"] = rng.choice([8, 16, 20])
        c["context"] = rng.choice([0, _log_int(rng, 10, 4000)])
        c["new_longest"] = _log_int(rng, 16, 3000 // c["batch"])
        c["new_shortest"] = rng.randint(1, c["new_longest"])
    elif kind == "weights":
        c["queries"] = rng.choice([1, 1, 2, 16])
        c["heads"] = rng.choice([8, 16, 20, 32, 64])
        c["batch"] = _log_int(rng, 1, 64 if c["queries"] < 16 else 4)
        c["longest"] = _log_int(rng, 100, min(30001, 100000 // c["batch"]) if c["queries"] < 16 else 8001) | 1
        c["shortest"] = rng.randint(1, c["longest"])
        c["bits"] = rng.choice([4, 16])
        c["decay"] = rng.choice([0.0, 0.9, 1.0])
    else:
        c["batch"] = _log_int(rng, 1, 32)
        c["layers"] = rng.choice([1, 2, 4])
        c["longest"] = _log_int(rng, 200, 8191) | 1
        c["shortest"] = rng.randint(c["longest"] // 4, c["longest"])
        c["first"] = rng.choice([0, 1, 4])
        c["shared"] = 128 * rng.choice([0, 0, 1, 3]) if c["shortest"] > 600 else 0
        c["budget"] = rng.randint(c["longest"] // 4, c["longest"] - 1)
        c["recent"] = rng.randint(0, c["budget"] // 4)
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
    if k == "store":
        return case["context"] + _lengths(seed, case["shortest"], case["longest"], case["batch"])
    if k == "prefill":
        return case["context"] + _lengths(seed, case["new_shortest"], case["new_longest"], case["batch"])
    if k == "decode":
        return case["shared"] + _lengths(seed, max(case["shortest"], case["queries"]),
                                         max(case["longest"], case["queries"]), case["batch"])
    return _lengths(seed, case["shortest"], case["longest"], case["batch"])


def _row_bytes(case):
    """Bytes of a row in 4 bits."""
    n = case["rank"] // 2 + 2 * case["rope"] + case["rank"] // BLOCK
    return -(-n // 16) * 16


def _bits(case):
    return {"weights": case.get("bits"), "evict": 16}.get(case["kind"], 4)


def _kept(case, n):
    """Tokens that a sequence of n keeps: the budget, or what may not go where that is more."""
    if n <= case["budget"]:
        return n
    head = min(n, max(case["first"], case["shared"]))
    return max(case["budget"], min(n, head + case["recent"]))


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
    n_pages = held + 8 + held // 8
    order = r.permutation(n_pages)                       # pages lie anywhere
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
    pages = torch.empty(layers, n_pages, page, row, device=DEV, dtype=torch.bfloat16).normal_(generator=g)
    if _bits(case) == 4:
        pages = torch.cat([_pack(case, p) for p in pages.view(-1, page, row).split(4096)])
        pages = pages.view(layers, n_pages, page, _row_bytes(case))
    s = dict(case=case, host_lens=lens, pages=pages, table=torch.from_numpy(table).to(DEV),
             lens=torch.from_numpy(lens.astype(np.int32)).to(DEV), refs=torch.from_numpy(refs).to(DEV))
    ids = torch.arange(len(lens), dtype=torch.int32, device=DEV)
    s["seqs"] = ids
    if k == "store":
        n_new = lens - case["context"]
        s["tok_seq"] = torch.from_numpy(np.repeat(np.arange(len(lens)), n_new).astype(np.int32)).to(DEV)
        s["tok_pos"] = torch.from_numpy(np.concatenate([case["context"] + np.arange(n) for n in n_new]).astype(np.int32)).to(DEV)
        # normalised latents: about one in size, a few dimensions larger than the others
        gain = torch.empty(row, device=DEV).normal_(generator=g).mul_(0.7).exp_()
        s["rows"] = torch.empty(int(n_new.sum()), row, device=DEV).normal_(generator=g).mul_(gain).to(torch.bfloat16)
    elif k in ("decode", "weights"):
        s["q"] = torch.empty(case["batch"] * case["queries"], case["heads"], row, device=DEV,
                             dtype=torch.bfloat16).normal_(generator=g)
        s["scale"] = (HEAD_DIM + case["rope"]) ** -0.5
        if k == "weights":
            # what the decode step left: log-sum-exp of every query, and the weights of earlier steps
            s["lse"] = torch.cat([_lse(s, b) for b in range(case["batch"])]).contiguous()
            s["weights"] = torch.empty(len(lens), max_blocks * page, device=DEV).normal_(generator=g).exp_()
    elif k == "prefill":
        new = lens - case["context"]
        off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        s["q_offsets"] = torch.from_numpy(off).to(DEV)
        s["total"], s["held"] = int(off[-1]), int(lens.sum())
        s["q"] = torch.empty(s["total"], case["heads"], HEAD_DIM + case["rope"], device=DEV,
                             dtype=torch.bfloat16).normal_(generator=g)
        s["w_kv"] = torch.empty(case["heads"], 2 * HEAD_DIM, case["rank"], device=DEV,
                                dtype=torch.bfloat16).normal_(std=case["rank"] ** -0.5, generator=g)
        s["scale"] = (HEAD_DIM + case["rope"]) ** -0.5
    else:
        # accumulated weights span orders of magnitude; the newest tokens have none yet
        w = torch.empty(layers, len(lens), max_blocks * page, device=DEV).normal_(generator=g).mul_(2).exp_()
        for i, n in enumerate(lens):
            w[:, i, max(0, int(n) - case["budget"] // 8):] = 0
        s["weights"] = w
        s["kept"] = torch.zeros(layers, len(lens), max_blocks * page, dtype=torch.int32, device=DEV)
        s["host_new"] = np.array([_kept(case, int(n)) for n in lens])
        s["n_new"] = torch.from_numpy((lens - s["host_new"]).astype(np.int32)).to(DEV)   # the next chunk's tokens
    return s


def run(state):
    k = state["case"]["kind"]
    if own:
        return {"store": _own_store, "decode": _own_decode, "prefill": _own_prefill, "weights": _own_weights,
                "evict": _own_evict}[k](state)
    return {"store": _store, "decode": _decode, "prefill": _prefill, "weights": _weights, "evict": _evict}[k](state)


# ------------------------------------------------------------------ the library's calls
def _handle(s):
    """The cache handle, status word and workspace that a serving program makes once."""
    if "handle" not in s:
        import edge_moe_serving_gb300 as moe
        c = s["case"]
        h = moe.moe_kv_cache(s["pages"].data_ptr(), s["table"].data_ptr(), s["lens"].data_ptr(), s["refs"].data_ptr(),
                             s["pages"].shape[0], s["pages"].shape[1], c["page"], c["rank"], c["rope"],
                             s["table"].shape[0], s["table"].shape[1],
                             moe.MOE_KV_FP4 if _bits(c) == 4 else moe.MOE_KV_BF16)
        n = 0
        if c["kind"] == "store":
            s["back"] = torch.empty_like(s["rows"])
        elif c["kind"] == "decode":
            n = moe.moe_latent_decode_workspace_size(h, c["batch"], c["queries"], c["heads"], c["shared"])
            s["out"] = torch.empty(c["batch"] * c["queries"], c["heads"], c["rank"], device=DEV, dtype=torch.bfloat16)
        elif c["kind"] == "prefill":
            n = moe.moe_latent_prefill_workspace_size(h, c["batch"], s["total"], c["heads"], HEAD_DIM, HEAD_DIM, s["held"])
            s["out"] = torch.empty(s["total"], c["heads"], HEAD_DIM, device=DEV, dtype=torch.bfloat16)
        elif c["kind"] == "weights":
            n = moe.moe_latent_weights_workspace_size(h, c["batch"], c["queries"], c["heads"])
        else:
            n = max(moe.moe_kv_evict_workspace_size(h, c["batch"]), moe.moe_kv_workspace_size(h, c["batch"]))
        s["ws"] = torch.empty(max(n, 256), device=DEV, dtype=torch.uint8)
        s["status"] = torch.zeros(1, device=DEV, dtype=torch.int32)
        s["handle"] = (moe, h)
    return s["handle"]


def _own_store(s):
    moe, h = _handle(s)
    n = s["tok_seq"].numel()
    moe.moe_kv_append(h, 0, s["rows"], s["tok_seq"], s["tok_pos"], n, s["status"])
    moe.moe_kv_read(h, 0, s["tok_seq"], s["tok_pos"], n, s["back"], s["status"])
    return s["back"]


def _own_decode(s):
    moe, h = _handle(s)
    c = s["case"]
    moe.moe_latent_decode(h, 0, s["q"], s["seqs"], c["batch"], c["queries"], c["heads"], s["scale"], c["shared"],
                          s["out"], None, s["ws"], s["ws"].numel(), s["status"])
    return s["out"]


def _own_prefill(s):
    moe, h = _handle(s)
    c = s["case"]
    moe.moe_latent_prefill(h, 0, s["q"], s["seqs"], s["q_offsets"], c["batch"], s["total"], c["heads"], HEAD_DIM, HEAD_DIM,
                           s["w_kv"], s["scale"], s["held"], s["out"], s["ws"], s["ws"].numel(), s["status"])
    return s["out"]


def _own_weights(s):
    moe, h = _handle(s)
    c = s["case"]
    moe.moe_latent_weights(h, 0, s["q"], s["seqs"], c["batch"], c["queries"], c["heads"], s["scale"], s["lse"],
                           c["decay"], s["weights"], s["ws"], s["ws"].numel(), s["status"])
    return s["weights"]


def _own_evict(s):
    moe, h = _handle(s)
    c = s["case"]
    # the system prompt stays whether or not another sequence holds its pages too
    first = max(c["first"], c["shared"])
    moe.moe_kv_evict(h, s["seqs"], c["batch"], s["weights"], max(c["budget"], first + c["recent"]), first, c["recent"],
                     s["kept"], s["ws"], s["ws"].numel(), s["status"])
    moe.moe_kv_reserve(h, s["seqs"], s["n_new"], c["batch"], s["ws"], s["ws"].numel(), s["status"])
    return _evict_state(s)


def _evict_state(s):
    return dict(pages=s["pages"], table=s["table"], lens=s["lens"], refs=s["refs"], weights=s["weights"], kept=s["kept"])


# ------------------------------------------------------------------ plain forms
def _quantise(x):
    """bf16 [..., rank] -> codes 0..15 and scales as bytes: the scale is the block's largest / 6 in 5 exponent and 3
    significand bits (nearest, ties to even), a code the nearest multiple of it."""
    x = x.float().unflatten(-1, (-1, BLOCK))
    a = x.abs()
    want = a.amax(-1, keepdim=True) / 6
    exponent = torch.frexp(want).exponent - 1
    step = torch.exp2(exponent.clamp(min=-14).float() - 3)
    scale = (torch.round(want / step) * step).clamp(max=61440.0)
    code = torch.zeros_like(a, dtype=torch.uint8)
    for border, at in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= border * scale) if at else (a > border * scale)
    code += 8 * (x < 0).to(torch.uint8)
    code = torch.where(scale > 0, code, torch.zeros_like(code))
    byte = (scale[..., 0].half().view(torch.int16) >> 7).to(torch.uint8)     # f16 has the same exponents
    return code.flatten(-2), byte


def _pack(case, rows):
    """bf16 rows [..., rank + rope] -> their 4-bit rows, bytes."""
    rank, rope = case["rank"], case["rope"]
    code, scale = _quantise(rows[..., :rank])
    out = torch.zeros(*rows.shape[:-1], _row_bytes(case), dtype=torch.uint8, device=rows.device)
    out[..., :rank // 2] = code[..., 0::2] + 16 * code[..., 1::2]
    out[..., rank // 2:rank // 2 + 2 * rope] = rows[..., rank:].contiguous().view(torch.uint8)
    out[..., rank // 2 + 2 * rope:rank // 2 + 2 * rope + rank // BLOCK] = scale
    return out


def _values(case, x):
    """4-bit rows [..., bytes] -> the values they stand for, [..., rank + rope] in 32 bits."""
    rank, rope = case["rank"], case["rope"]
    code = torch.stack([x[..., :rank // 2] & 15, x[..., :rank // 2] >> 4], -1).flatten(-2)
    size = code & 7
    e, m = (size >> 1).float(), (size & 1).float()
    v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e - 1)) * (1 - 2 * (code >> 3).float())
    at = rank // 2 + 2 * rope
    scale = (x[..., at:at + rank // BLOCK].to(torch.int16) << 7).view(torch.float16).float()
    v = (v.unflatten(-1, (-1, BLOCK)) * scale[..., None]).flatten(-2)
    return torch.cat([v, x[..., rank // 2:at].contiguous().view(torch.bfloat16).float()], -1)


def _rows(case, x):
    return _values(case, x) if x.dtype == torch.uint8 else x.float()


def _gather(s, rows, first, last):
    """Cache rows of blocks [first, last) of the given sequences, in 32 bits: [n, tokens, rank + rope]."""
    ids = s["table"][rows, first:last].long().clamp(min=0)
    x = s["pages"][0][ids]
    return _rows(s["case"], x.reshape(x.shape[0], -1, x.shape[-1]))


def _softmax_parts(scores, mask):
    """exp(scores - m), its sum and m, with masked places at zero and rows that have none left at m = 0."""
    scores = scores.masked_fill(~mask, -math.inf)
    m = scores.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(scores - m)
    return p, p.sum(-1, keepdim=True), m


def _store(s):
    page, seq, pos = s["case"]["page"], s["tok_seq"].long(), s["tok_pos"].long()
    at = s["table"][seq, pos // page].long()
    s["pages"][0, at, pos % page] = _pack(s["case"], s["rows"])
    return _values(s["case"], s["pages"][0, at, pos % page]).to(torch.bfloat16)


def _limits(s):
    """Tokens each query row of each sequence sees: [n, queries * heads, 1]."""
    c = s["case"]
    n, nq, heads = c["batch"], c["queries"], c["heads"]
    limit = s["lens"][s["seqs"].long()].long()[:, None] - nq + torch.arange(1, nq + 1, device=DEV)
    return limit[:, :, None].expand(n, nq, heads).reshape(n, nq * heads, 1)


def _decode(s):
    c = s["case"]
    seqs, rank, page = s["seqs"].long(), c["rank"], c["page"]
    n, nq, heads = c["batch"], c["queries"], c["heads"]
    limit = _limits(s)
    q = s["q"].float().view(n, nq * heads, -1)
    shared = c["shared"]
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


def _weights(s):
    c = s["case"]
    seqs = s["seqs"].long()
    n, nq, heads = c["batch"], c["queries"], c["heads"]
    kv = _gather(s, seqs, 0, s["table"].shape[1])
    q = s["q"].float().view(n, nq * heads, -1)
    pos = torch.arange(kv.shape[1], device=DEV)
    z = torch.bmm(q, kv.transpose(1, 2)) * s["scale"] - s["lse"].view(n, nq * heads, 1)
    p = torch.exp(z.masked_fill(pos >= _limits(s), -math.inf)).sum(1)
    old = s["weights"][seqs]
    new = p + (c["decay"] * old if c["decay"] else 0)
    s["weights"][seqs] = torch.where(pos < s["lens"][seqs].long()[:, None], new, old)
    return s["weights"]


def _evict(s):
    c = s["case"]
    page, layers = c["page"], s["pages"].shape[0]
    for i, (n, new) in enumerate(zip(s["host_lens"].tolist(), s["host_new"].tolist())):
        at = torch.arange(n, device=DEV)
        if n > c["budget"]:
            w = s["weights"][:, i, :n].clone()
            stays = (at < max(c["first"], c["shared"])) | (at >= n - c["recent"])
            order = torch.sort(w.masked_fill(stays, math.inf), dim=-1, descending=True, stable=True).indices
            keep = torch.sort(order[:, :new], dim=-1).values                                     # [layers, new]
            ids = s["table"][i].long()
            layer = torch.arange(layers, device=DEV)[:, None]
            moved = s["pages"][layer, ids[keep // page], keep % page]
            to = torch.arange(new, device=DEV)
            s["pages"][layer, ids[to // page], to % page] = moved
            s["weights"][:, i, :new] = torch.gather(w, 1, keep)
            s["weights"][:, i, new:n] = 0
            s["kept"][:, i, :new] = keep.int()
            first, last = -(-new // page), -(-n // page)
            s["refs"][ids[first:last]] -= 1
            s["table"][i, first:last] = -1
            s["lens"][i] = new
        else:
            s["kept"][:, i, :n] = at.int()
    # room for the next chunk: the lowest free pages, in the sequences' order
    was, now = -(-s["host_new"] // page), -(-s["host_lens"] // page)
    need = torch.from_numpy(now - was).to(DEV)
    free = torch.nonzero(s["refs"] == 0)[:, 0]
    who = torch.repeat_interleave(torch.arange(need.numel(), device=DEV), need)
    block = torch.from_numpy(was).to(DEV)[who] + torch.arange(who.numel(), device=DEV) - (need.cumsum(0) - need)[who]
    s["table"][who, block] = free[:who.numel()].int()
    s["refs"][free[:who.numel()]] = 1
    s["lens"] += s["n_new"]
    return _evict_state(s)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    k, rank = case["kind"], case["rank"]
    row = rank + case["rope"]
    held = _row_bytes(case) if _bits(case) == 4 else 2 * row
    lens = _sizes(case, 1)
    if k == "store":
        n = int((lens - case["context"]).sum())
        return {"bytes": n * 2 * (2 * row + held), "flops": 0}
    if k in ("decode", "weights"):
        shared, rows = case.get("shared", 0), case["batch"] * case["queries"] * case["heads"]
        tokens = int(lens.sum()) - shared * (case["batch"] - 1)
        pairs = int(lens.sum()) * case["queries"] * case["heads"]
        if k == "decode":
            return {"bytes": tokens * held + rows * (row + rank) * 2, "flops": 2 * pairs * (row + rank)}
        return {"bytes": tokens * (held + 8) + rows * (2 * row + 4), "flops": 2 * pairs * row}
    if k == "prefill":
        new = lens - case["context"]
        pairs = sum(int(a) * case["context"] + int(a) * (int(a) + 1) // 2 for a in new) * case["heads"]
        dim = 2 * HEAD_DIM + case["rope"]
        total, tokens = int(new.sum()), int(lens.sum())
        return {"bytes": tokens * held + case["heads"] * (2 * HEAD_DIM * rank + total * dim) * 2,
                "flops": 2 * pairs * dim + 2 * tokens * rank * 2 * HEAD_DIM * case["heads"]}
    # tokens behind the protected head move where something before them goes
    head = max(case["first"], case["shared"])
    gone = [(int(n), _kept(case, int(n))) for n in lens if n > case["budget"]]
    moved, seen = sum(new - min(head, new) for _, new in gone), sum(n for n, _ in gone)
    return {"bytes": case["layers"] * (moved * 2 * held + 8 * seen + 4 * sum(new for _, new in gone)), "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits
SIZES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def exact(case, seed):
    s = prepare(case, seed)
    return {"store": _exact_store, "decode": _exact_decode, "prefill": _exact_prefill, "weights": _exact_weights,
            "evict": _exact_evict}[case["kind"]](s)


def _scale_values():
    """All scales, ascending; byte i is the i-th."""
    return [m * 2.0 ** -17 for m in range(8)] + [(8 + m) * 2.0 ** (e - 18) for e in range(1, 31) for m in range(8)]


def _stands_for(case, x):
    """4-bit rows [n, bytes] by look-up, in 64 bits."""
    rank, at = case["rank"], case["rank"] // 2 + 2 * case["rope"]
    sizes = torch.tensor(SIZES + [-v for v in SIZES], dtype=torch.float64, device=DEV)
    scales = torch.tensor(_scale_values() + [math.nan] * 8, dtype=torch.float64, device=DEV)
    out = torch.empty(x.shape[0], rank + case["rope"], dtype=torch.float64, device=DEV)
    scale = scales[x[:, at:at + rank // BLOCK].int()].repeat_interleave(BLOCK, 1)
    out[:, 0:rank:2] = sizes[(x[:, :rank // 2] % 16).int()] * scale[:, 0::2]
    out[:, 1:rank:2] = sizes[(x[:, :rank // 2] // 16).int()] * scale[:, 1::2]
    out[:, rank:] = x[:, rank // 2:at].contiguous().view(torch.bfloat16).double()
    return out


def _tokens_of(s, seq):
    """The rows of one sequence in 64 bits, page after page."""
    n, page = int(s["lens"][seq]), s["case"]["page"]
    ids = s["table"][seq].tolist()[:-(-n // page)]
    x = torch.cat([s["pages"][0, i] for i in ids])[:n]
    return _stands_for(s["case"], x) if x.dtype == torch.uint8 else x.double()


def _nearest(x, values):
    """Index of the value nearest to each x >= 0, the even one of two equally near."""
    v = torch.tensor(values, dtype=torch.float64, device=DEV)
    hi = torch.searchsorted(v, x.contiguous()).clamp(max=len(values) - 1)
    lo = (hi - 1).clamp(min=0)
    a, b = x - v[lo], v[hi] - x
    return torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)


def _exact_store(s):
    rank = s["case"]["rank"]
    x = s["rows"].double()
    lat = x[:, :rank].unflatten(-1, (-1, BLOCK))
    scales = torch.tensor(_scale_values(), dtype=torch.float64, device=DEV)
    scale = scales[_nearest(lat.abs().amax(-1) / 6, _scale_values())][..., None]
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    size = torch.tensor(SIZES, dtype=torch.float64, device=DEV)[_nearest(lat.abs() / safe, SIZES)]
    return torch.cat([(size * scale * torch.sign(lat)).flatten(-2), x[:, rank:]], -1)


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


def _scores64(s, b):
    """Scores of sequence b's queries, [queries * heads, tokens] in 64 bits, and which tokens each sees."""
    c = s["case"]
    x = _tokens_of(s, b)
    q = s["q"][b * c["queries"]:(b + 1) * c["queries"]].double().flatten(0, 1)
    query = torch.arange(q.shape[0], device=DEV) // c["heads"]
    sees = torch.arange(x.shape[0], device=DEV)[None] <= (x.shape[0] - c["queries"] + query)[:, None]
    return (q @ x.T) * s["scale"], sees


def _lse(s, b):
    z, sees = _scores64(s, b)
    return torch.logsumexp(z.masked_fill(~sees, -math.inf), -1).float().view(s["case"]["queries"], -1)


def _exact_weights(s):
    c = s["case"]
    out = s["weights"].double()
    lse = s["lse"].double().view(c["batch"], -1)
    for b in range(c["batch"]):
        z, sees = _scores64(s, b)
        n = z.shape[1]
        out[b, :n] = c["decay"] * out[b, :n] + torch.exp(z - lse[b][:, None]).masked_fill(~sees, 0.0).sum(0)
    return out


def _exact_evict(s):
    """Sequence after sequence, on lists."""
    c, pages = s["case"], s["pages"]
    page, before = c["page"], s["pages"].clone()
    table, lens, refs = (s[x].cpu().numpy().copy() for x in ("table", "lens", "refs"))
    weights, kept = s["weights"].cpu().double().numpy().copy(), s["kept"].cpu().numpy().copy()
    new_lens = []
    for b, n in enumerate(lens.tolist()):
        head, new = max(c["first"], c["shared"]), n
        if n > c["budget"]:
            tail = max(head, n - c["recent"])
            middle = np.arange(head, tail)
            new = max(c["budget"], head + n - tail)
        for layer in range(pages.shape[0]):
            if n > c["budget"]:
                order = sorted(middle.tolist(), key=lambda t: (-weights[layer, b, t], t))[:new - head - (n - tail)]
                keep = list(range(head)) + sorted(order) + list(range(tail, n))
            else:
                keep = list(range(n))
            src, to = np.array(keep), np.arange(new)
            pages[layer, table[b][to // page], to % page] = before[layer, table[b][src // page], src % page]
            weights[layer, b, :n] = np.concatenate([weights[layer, b][src], np.zeros(n - new)])
            kept[layer, b, :new] = src
        for i in range(-(-new // page), -(-n // page)):
            refs[table[b, i]] -= 1
            table[b, i] = -1
        new_lens.append(new)
    for b, n in enumerate(lens.tolist()):
        for i in range(-(-new_lens[b] // page), -(-n // page)):
            table[b, i] = int(np.nonzero(refs == 0)[0][0])
            refs[table[b, i]] = 1
    return dict(pages=pages.double(), table=torch.from_numpy(table), lens=torch.from_numpy(lens), refs=torch.from_numpy(refs),
                weights=torch.from_numpy(weights), kept=torch.from_numpy(kept))
