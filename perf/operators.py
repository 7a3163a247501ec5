"""The serving operators around the packed matvec, as measured cases.

Four kinds of call, each a step of decoding a batch of sequences over the
paged Group-32 4-bit KV cache:

  append     quantise new tokens' K and V into cache slots, and read them back;
  attention  attention of each sequence's newest tokens over its pages (score
             cap, distance bias, window, accumulated weights);
  evict      keep the entries with the largest accumulated weight and the
             newest ones, moved to fresh pages, and read them back;
  sample     temperature, top-k, top-p and min-p over the LM head's logits,
             from given uniform numbers.

`run` computes them with elementary torch operations where `own` is false and
with the package's operators where it is true, on the same state.

Cache layout (one pool, G = head_dim / 32, slot = (page * heads + head) *
page_size + r): a K or V vector of one head is G groups of 32 channels, each
with a 4-bit code per channel, an FP16 scale and a 4-bit zero point, value =
(code - zero) * scale.  K codes: 32-bit word slot*4G + w*G + g holds channels
32g + 8w .. +7 of group g, lowest nibble first; V codes: 16-bit word
slot*8G + e*G + g holds channels 32g + 4e .. +3; scales: FP16 slot*G + g;
zero points: 32-bit word slot, nibble g.
"""
import random

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases

def _attn(name, n_seq, q_heads, kv_heads, head_dim, page, min_len, max_len, q_tokens=1, softcap=0.0,
          slopes=False, window=0, out="bf16", mass=False):
    c = {"op": "attention", "n_seq": n_seq, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim,
         "page": page, "min_len": min_len, "max_len": max_len, "q_tokens": q_tokens, "softcap": softcap,
         "slopes": slopes, "window": window, "out": out, "mass": mass}
    return {"name": name, **c} if name else c


def _append(name, n_tok, kv_heads, head_dim, page):
    c = {"op": "append", "n_tok": n_tok, "kv_heads": kv_heads, "head_dim": head_dim, "page": page}
    return {"name": name, **c} if name else c


def _evict(name, n_seq, kv_heads, head_dim, page, min_len, max_len, budget, recent):
    c = {"op": "evict", "n_seq": n_seq, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
         "min_len": min_len, "max_len": max_len, "budget": budget, "recent": recent}
    return {"name": name, **c} if name else c


def _sample(name, rows, vocab, top_k, top_p, min_p):
    c = {"op": "sample", "rows": rows, "vocab": vocab, "top_k": top_k, "top_p": top_p, "min_p": min_p}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one conversation early in its answer, the 1.5B-class heads: the smallest call, where latency counts
        _attn("attn_one_short", 1, 12, 2, 128, 16, 300, 300, out="fp32"),
        # one conversation at the cache's full 8192 positions
        _attn("attn_one_8192", 1, 12, 2, 128, 64, 8192, 8192),
        # a serving batch of the 4B-class heads, ragged lengths, accumulating weights for a later eviction
        _attn("attn_batch_mass", 48, 32, 8, 128, 32, 1, 6000, mass=True),
        # the same with capped scores, a distance bias and a window, on small heads
        _attn("attn_capped_window", 33, 24, 6, 64, 16, 17, 5003, softcap=30.0, slopes=True, window=2048),
        # a few tokens per sequence at once: a draft being checked, or a short prompt chunk
        _attn("attn_chunk_16", 12, 32, 8, 128, 64, 40, 7001, q_tokens=16, out="fp32"),
        # the largest: long documents of a batch
        _attn("attn_long_batch", 16, 32, 8, 128, 64, 20000, 65536),
        # one new token of one sequence, and a prompt's worth of them
        _append("append_one", 1, 2, 128, 16),
        _append("append_prompt", 8192, 8, 128, 64),
        # a full cache cut to a quarter, for one sequence and for a ragged batch
        _evict("evict_one_8192", 1, 2, 128, 64, 8192, 8192, 2048, 256),
        _evict("evict_batch", 24, 8, 128, 32, 100, 6007, 1500, 128),
        # the LM head's rows: one conversation, and a serving batch with an odd vocabulary
        _sample("sample_one", 1, 131072, 50, 0.95, 0.0),
        _sample("sample_batch", 64, 131071, 0, 0.9, 0.02),
    ]


def _span(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "evict", "sample"])
    head_dim = rng.choice([64, 96, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 6, 8])
    if op == "attention":
        q_tokens = rng.choice([1, 1, 1, 2, 5, 16, 32])
        q_heads = kv_heads * rng.choice([1, 2, 3, 4, 6, 8])
        # at most the longest listed case's cache, and a twentieth of a tera-operation
        most = min(640000 * 1024 // (kv_heads * head_dim), 40 * 10 ** 9 // (4 * q_tokens * q_heads * head_dim))
        max_len = _span(rng, 1, min(40000, most))
        n_seq = _span(rng, 1, max(1, min(96, most // max_len)))
        return _attn(None, n_seq, q_heads, kv_heads, head_dim, page, rng.randint(0, max_len), max_len,
                     q_tokens, rng.choice([0.0, 0.0, 20.0, 50.0]), rng.random() < 0.3,
                     rng.choice([0, 0, 0, 129, 1024]), rng.choice(["bf16", "bf16", "fp32"]), rng.random() < 0.3)
    if op == "append":
        return _append(None, _span(rng, 1, 8192), kv_heads, head_dim, page)
    if op == "evict":
        max_len = _span(rng, 8, 16384)
        budget = rng.randint(max(1, max_len // 8), max(1, 3 * max_len // 4))
        return _evict(None, _span(rng, 1, max(1, min(32, 150000 // max_len))), kv_heads, min(head_dim, 128), page,
                      rng.randint(1, max_len), max_len, budget, rng.randint(0, budget))
    return _sample(None, _span(rng, 1, 64), _span(rng, 1000, 150000), rng.choice([0, 1, 20, 50, 400]),
                   rng.choice([1.0, 0.95, 0.8, 0.3]), rng.choice([0.0, 0.0, 0.02, 0.1]))


def _lengths(case):
    """The sequences' lengths: part of the case, whatever the seed."""
    r = random.Random("%d %d %d" % (case["n_seq"], case["min_len"], case["max_len"]))
    got = [r.randint(case["min_len"], case["max_len"]) for _ in range(case["n_seq"])]
    got[0] = case["max_len"]
    return got


def _queries(case):
    """The number of new tokens of each sequence; where it has fewer positions, the first of them see nothing."""
    r = random.Random("%d %d" % (case["n_seq"], case["q_tokens"]))
    got = [r.randint(1, case["q_tokens"]) for _ in range(case["n_seq"])]
    got[0] = case["q_tokens"]
    return got


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _tokens(gen, n, heads, dim):
    """K or V projections: normal values, some channels of a head larger than the others."""
    gain = 0.5 + 2.0 * torch.rand((heads, dim), generator=gen, device=DEV) ** 4
    return torch.randn((n, heads, dim), generator=gen, device=DEV) * gain


def _pool(gen, heads, dim, page, n_pages):
    """A pool whose every slot holds a quantised token: buffers as the package lays them out."""
    G = dim // 32
    out = {}
    for which in ("k", "v"):
        x = _tokens(gen, n_pages * page, heads, dim).reshape(n_pages, page, heads, G, 32).transpose(1, 2)
        lo, hi = x.amin(-1), x.amax(-1)
        s = ((hi - lo) / 15).half().float()
        z = torch.round(-lo / s).clamp_(0, 15)
        c = (torch.round(x / s.unsqueeze(-1)) + z.unsqueeze(-1)).clamp_(0, 15).to(torch.uint8)
        del x
        b = c[..., 0::2] | (c[..., 1::2] << 4)  # [pages, heads, page, G, 16]
        cut = 4 if which == "k" else 2          # bytes of one code word
        b = b.reshape(n_pages, heads, page, G, 16 // cut, cut).transpose(3, 4)
        out[which + "_codes"] = b.reshape(-1).contiguous()
        out[which + "_scales"] = s.half().reshape(-1).view(torch.int16)
        nib = (z.to(torch.int64) << (4 * torch.arange(G, device=DEV))).sum(-1)
        out[which + "_zeros"] = (nib - ((nib >> 31) << 32)).to(torch.int32).reshape(-1)
        del b, c
    return out


def _geometry(case, n_pages):
    return {"heads": case["kv_heads"], "dim": case["head_dim"], "page": case["page"], "n_pages": n_pages}


def _tables(gen, lengths, page, spare):
    """A page table [n_seq][max pages] of distinct pages in shuffled order, and the pool's page count."""
    need = [-(-n // page) for n in lengths]
    width = max(1, max(need))
    n_pages = sum(need) + spare + 1
    order = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros((len(need), width), dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, n_pages, order[at:]


def prepare(case, seed):
    gen = _gen(seed)
    op = case["op"]
    if op == "sample":
        m, v = case["rows"], case["vocab"]
        f32 = {"dtype": torch.float32, "device": DEV}
        return {"op": op, "logits": 2.5 * torch.randn((m, v), generator=gen, device=DEV),
                "u": torch.rand(m, generator=gen, device=DEV),
                "temperature": 0.6 + 0.6 * torch.rand(m, generator=gen, device=DEV),
                "top_k": torch.full((m,), case["top_k"], dtype=torch.int32, device=DEV),
                "top_p": torch.full((m,), case["top_p"], **f32), "min_p": torch.full((m,), case["min_p"], **f32)}
    heads, dim, page = case["kv_heads"], case["head_dim"], case["page"]
    if op == "append":
        n = case["n_tok"]
        n_pages = -(-n // page) + 3
        st = {"op": op, **_geometry(case, n_pages), **_pool(gen, heads, dim, page, n_pages)}
        st["k"] = _tokens(gen, n, heads, dim).bfloat16()
        st["v"] = _tokens(gen, n, heads, dim).bfloat16()
        pages = torch.randperm(n_pages, generator=gen, device=DEV)
        i = torch.arange(n, device=DEV) + page // 2  # the prompt goes on in a page begun earlier
        st["slots"] = (pages[i // page] * page + i % page).to(torch.int32)
    else:
        lengths = _lengths(case)
        kept = -(-case["budget"] // page) if op == "evict" else 0
        table, n_pages, free = _tables(gen, lengths, page, kept * case["n_seq"])
        st = {"op": op, **_geometry(case, n_pages), **_pool(gen, heads, dim, page, n_pages), "pages": table,
              "lengths": torch.tensor(lengths, dtype=torch.int32, device=DEV)}
        if op == "evict":
            # accumulated weights are far from even: a few entries hold most, many hold hardly any
            st["mass"] = torch.exp(2.0 * torch.randn(n_pages * heads * page, generator=gen, device=DEV) - 6.0)
            st["dst_pages"] = free[: kept * case["n_seq"]].reshape(case["n_seq"], kept).contiguous()
            st["budget"], st["recent"] = case["budget"], case["recent"]
            i = torch.arange(case["budget"], device=DEV)
            dst = st["dst_pages"][:, i // page] * page + (i % page).to(torch.int32)
            there = i < torch.tensor(lengths, device=DEV).unsqueeze(1)
            st["dst_slots"] = torch.where(there, dst, -1).to(torch.int32).reshape(-1)
        else:
            n_q = _queries(case)
            st["mass"] = torch.zeros(n_pages * heads * page, device=DEV) if case["mass"] else None
            st["q"] = torch.randn((sum(n_q), case["q_heads"], dim), generator=gen, device=DEV).bfloat16()
            start = torch.tensor([0] + n_q, dtype=torch.int32, device=DEV).cumsum(0).to(torch.int32)
            st["q_start"] = None if case["q_tokens"] == 1 else start
            st["max_q"] = case["q_tokens"]
            st["scale"], st["softcap"], st["window"] = dim ** -0.5, case["softcap"], case["window"]
            h = torch.arange(1, case["q_heads"] + 1, device=DEV, dtype=torch.float32)
            st["slopes"] = torch.exp2(-8.0 * h / case["q_heads"]) if case["slopes"] else None
            st["out"] = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    return st


# ---------------------------------------------------------------- plain forms

def _words(codes, bits, slots, n):
    """The code words of the slots (one row each) as whole numbers, [slots][n]."""
    return codes.view(torch.int32 if bits == 32 else torch.int16).view(-1, n)[slots].to(torch.int32)


def _values(st, which, slots):
    """Slots (any shape) of the pool, dequantised: FP32 [..., head_dim]."""
    G = st["dim"] // 32
    bits, per = (32, 4) if which == "k" else (16, 8)
    w = _words(st[which + "_codes"], bits, slots, per * G).unflatten(-1, (per, G)).transpose(-1, -2)
    c = (w.unsqueeze(-1) >> (4 * torch.arange(bits // 4, device=DEV, dtype=torch.int32))) & 15
    c = c.flatten(-2)  # [..., G, 32]
    z = (st[which + "_zeros"][slots].unsqueeze(-1) >> (4 * torch.arange(G, device=DEV, dtype=torch.int32))) & 15
    s = st[which + "_scales"].view(torch.float16).view(-1, G)[slots].float()
    return ((c - z.unsqueeze(-1)).float() * s.unsqueeze(-1)).flatten(-2)


def _head_slots(st, token_slots):
    """Slots of every head, [..., heads], from token slots page * page_size + r."""
    h = torch.arange(st["heads"], device=DEV)
    t = token_slots.long().unsqueeze(-1)
    return (t // st["page"] * st["heads"] + h) * st["page"] + t % st["page"]


def _plain_read(st, slots):
    """K and V of the token slots, BF16 [n][heads][head_dim]; zeros for a negative slot."""
    at = _head_slots(st, slots.clamp(min=0))
    there = (slots >= 0)[:, None, None]
    return [torch.where(there, _values(st, w, at), 0.0).bfloat16() for w in ("k", "v")]


def _to_fp16(x):
    """FP64 values rounded once, half to even, to FP16's numbers."""
    step = torch.exp2(torch.floor(torch.log2(x.clamp(min=2.0 ** -14))) - 10)
    return torch.round(x / step) * step


def _plain_append(st):
    G = st["dim"] // 32
    at = _head_slots(st, st["slots"])
    for which, x in (("k", st["k"]), ("v", st["v"])):
        x = x.double().unflatten(-1, (G, 32))
        lo, hi = x.amin(-1), x.amax(-1)
        s = _to_fp16((hi - lo) / 15)
        by = torch.where(s == 0, 1.0, s)
        z = torch.where(s == 0, 0.0, torch.round(-lo / by).clamp(0, 15))
        c = torch.where(s.unsqueeze(-1) == 0, 0.0, torch.round(x / by.unsqueeze(-1)) + z.unsqueeze(-1)).clamp(0, 15)
        n = 8 if which == "k" else 4  # codes of a word
        w = (c.long().unflatten(-1, (-1, n)) << (4 * torch.arange(n, device=DEV))).sum(-1).transpose(-1, -2)
        kind = torch.int32 if which == "k" else torch.int16
        st[which + "_codes"].view(kind).view(-1, w.shape[-2] * G)[at] = w.flatten(-2).to(kind)
        st[which + "_scales"].view(torch.float16).view(-1, G)[at] = s.half()
        zw = (z.long() << (4 * torch.arange(G, device=DEV))).sum(-1)
        st[which + "_zeros"][at] = zw.to(torch.int32)
    return _plain_read(st, st["slots"])


def _plain_attention(st):
    page, heads, dim = st["page"], st["heads"], st["dim"]
    q = st["q"].float()
    n_seq, grp = len(st["lengths"]), q.shape[1] // heads
    length = st["lengths"].long()
    L = st["pages"].shape[1] * page
    t = torch.arange(L, device=DEV)
    at = _head_slots(st, st["pages"][:, t // page] * page + t % page).transpose(1, 2)  # [seq][head][position]
    start = st["q_start"].long() if st["q_start"] is not None else torch.arange(n_seq + 1, device=DEV)
    # the sequences' queries side by side: [seq][token][q head][dim], tokens beyond a sequence's own repeated
    n_q = start[1:] - start[:-1]
    j = torch.arange(st["max_q"], device=DEV)
    row = (start[:-1, None] + torch.minimum(j, n_q[:, None] - 1))  # [seq][token]
    qs = q[row].unflatten(2, (heads, grp)).permute(0, 2, 1, 3, 4)  # [seq][head][token][grp][dim]
    s = torch.matmul(qs.flatten(2, 3), _values(st, "k", at).transpose(2, 3)).unflatten(2, (-1, grp)) * st["scale"]
    if st["softcap"]:
        s = st["softcap"] * torch.tanh(s / st["softcap"])
    pos = length[:, None] - n_q[:, None] + j  # [seq][token]
    gap = pos[:, None, :, None, None] - t     # [seq][1][token][1][position]
    if st["slopes"] is not None:
        s = s - st["slopes"].view(heads, 1, grp, 1) * gap
    seen = gap >= 0
    if st["window"]:
        seen = seen & (gap < st["window"])
    s = torch.where(seen, s, float("-inf"))
    top = s.amax(-1, keepdim=True)
    e = torch.where(seen, torch.exp(s - torch.where(top > float("-inf"), top, 0.0)), 0.0)
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total > 0, total, 1.0)
    o = torch.matmul(p.flatten(2, 3), _values(st, "v", at)).unflatten(2, (-1, grp))  # [seq][head][token][grp][dim]
    mine = (j < n_q[:, None])
    out = torch.empty((q.shape[0], heads * grp, dim), dtype=st["out"], device=DEV)
    out[row[mine]] = o.permute(0, 2, 1, 3, 4).flatten(2, 3)[mine].to(st["out"])
    lse = torch.empty((q.shape[0], heads * grp), device=DEV)
    lse[row[mine]] = (top + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).flatten(2)[mine]
    if st["mass"] is None:
        return [out, lse]
    got = (p.sum(3) * mine[:, None, :, None]).sum(2)  # [seq][head][position]
    there = (t < length[:, None])[:, None, :].expand(-1, heads, -1)
    st["mass"][at[there]] += got[there]
    return [out, lse, st["mass"]]


def _plain_evict(st):
    page, heads, budget = st["page"], st["heads"], st["budget"]
    length = st["lengths"].long()
    L = st["pages"].shape[1] * page
    t = torch.arange(L, device=DEV)
    at = _head_slots(st, st["pages"][:, t // page] * page + t % page).transpose(1, 2)  # [seq][head][position]
    rank = torch.where(t >= length[:, None] - st["recent"], float("inf"), 0.0)
    rank = torch.where(t < length[:, None], rank, float("-inf"))[:, None, :]
    m = torch.where(rank == 0, st["mass"][at], rank)
    best = torch.sort(m, dim=-1, descending=True, stable=True).indices[..., :budget]
    n = torch.minimum(length, torch.tensor(budget, device=DEV))
    i = torch.arange(budget, device=DEV)
    there = (i < n[:, None])[:, None, :].expand(-1, heads, -1)
    best = torch.sort(torch.where(there, best, L), dim=-1).values.clamp(max=L - 1)
    src = at.gather(2, best)
    dst = _head_slots(st, st["dst_pages"][:, i // page] * page + i % page).transpose(1, 2)
    src, dst = src[there], dst[there]
    G = st["dim"] // 32
    moved = [(st[w + "_codes"].view(-1, 16 * G), st[w + "_scales"].view(-1, G), st[w + "_zeros"]) for w in ("k", "v")]
    for buf in (*moved[0], *moved[1], st["mass"]):
        buf[dst] = buf[src]
    return [n.to(torch.int32), *_plain_read(st, st["dst_slots"]), st["mass"]]


def _plain_sample(st):
    x = st["logits"].double()
    w = torch.exp((x - x.amax(-1, keepdim=True)) / st["temperature"].double()[:, None])
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    best = w.gather(1, order)
    k = st["top_k"].long()[:, None]
    keep = (torch.arange(x.shape[1], device=DEV) < k) | (k <= 0)
    best = torch.where(keep, best, 0.0)
    p = st["top_p"].double()[:, None]
    before = best.cumsum(-1) - best
    keep = keep & ((before < p * best.sum(-1, keepdim=True)) | (p >= 1))
    keep = keep & (best >= st["min_p"].double()[:, None] * best[:, :1])
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, best, 0.0))
    cum = w.cumsum(-1)
    total = cum[:, -1:]
    # the first token whose sum passes u of the whole; never one that was filtered out
    pick = (cum <= st["u"].double()[:, None] * total).sum(-1)
    last = x.shape[1] - 1 - (w.flip(-1) > 0).to(torch.int32).argmax(-1)
    pick = torch.minimum(pick, last)
    logp = torch.log(w.gather(1, pick[:, None]) / total).squeeze(1)
    return [pick.to(torch.int32), logp.float()]


_PLAIN = {"append": _plain_append, "attention": _plain_attention, "evict": _plain_evict, "sample": _plain_sample}


# ---------------------------------------------------------------- the package's calls

def _own(st):
    import outlier_split_bit_b200 as sp
    op = st["op"]
    if op != "sample" and "pool" not in st:  # the object that a program keeps over its cache's buffers
        st["pool"] = sp.KVPool.from_buffers(st["heads"], st["dim"], st["page"], st["n_pages"], st["k_codes"],
                                            st["k_scales"], st["k_zeros"], st["v_codes"], st["v_scales"],
                                            st["v_zeros"], st.get("mass"))
    if op == "append":
        st["pool"].append(st["k"], st["v"], st["slots"])
        return list(st["pool"].read(st["slots"]))
    if op == "attention":
        out, lse = sp.spectra_attention_paged(st["pool"], st["pages"], st["lengths"], st["q"], st["q_start"],
                                              max_q=st["max_q"], scale=st["scale"], softcap=st["softcap"],
                                              slopes=st["slopes"], window=st["window"], out_dtype=st["out"],
                                              want_lse=True, update_mass=st["mass"] is not None)
        return [out, lse] if st["mass"] is None else [out, lse, st["mass"]]
    if op == "evict":
        n = sp.spectra_kv_evict(st["pool"], st["pages"], st["lengths"], st["dst_pages"], st["budget"], st["recent"])
        k, v = st["pool"].read(st["dst_slots"])
        return [n, k, v, st["mass"]]
    ids, logp = sp.spectra_sample(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"],
                                  top_p=st["top_p"], min_p=st["min_p"])
    return [ids, logp]


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["op"]](state)


# ---------------------------------------------------------------- what a pass needs

def _vector(dim):
    """Bytes of one quantised K or V vector of a head."""
    return dim // 2 + dim // 16 + 4


def work(case):
    op = case["op"]
    if op == "sample":
        # each logit read once; its weight once
        return {"bytes": case["rows"] * (4 * case["vocab"] + 28), "flops": 3 * case["rows"] * case["vocab"]}
    heads, dim = case["kv_heads"], case["head_dim"]
    if op == "append":
        n = case["n_tok"] * heads
        # BF16 K and V in, quantised; read back as BF16
        return {"bytes": n * 2 * (2 * dim + 2 * _vector(dim) + 2 * dim) + 8 * case["n_tok"], "flops": 8 * n * dim}
    lengths = _lengths(case)
    if op == "evict":
        kept = heads * sum(min(n, case["budget"]) for n in lengths)
        rows = heads * case["n_seq"] * case["budget"]
        # every entry's weight; the kept entries moved (K, V, weight); read back as BF16, weights as FP32
        return {"bytes": 4 * heads * sum(lengths) + kept * (2 * 3 * _vector(dim) + 8) + rows * (4 * dim + 4),
                "flops": 2 * rows * dim}
    n_q = _queries(case)
    seen, pairs = 0, 0
    for n, m in zip(lengths, n_q):
        first = max(0, n - m - case["window"] + 1) if case["window"] else 0
        seen += max(0, n - first)
        for j in range(m):
            pos = n - m + j
            pairs += max(0, min(pos + 1, case["window"] or pos + 1))
    item = 2 if case["out"] == "bf16" else 4
    rows = sum(n_q) * case["q_heads"]
    mass = 8 * heads * seen if case["mass"] else 0
    return {"bytes": 2 * heads * seen * _vector(dim) + rows * (dim * (2 + item) + 4) + mass,
            "flops": 4 * pairs * case["q_heads"] * dim}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_values(st, which, pages, head):
    """The positions of some pages of one head, dequantised from their bytes: FP64 [positions][head_dim]."""
    dim, P = st["dim"], st["page"]
    G, cut = dim // 32, 4 if which == "k" else 2
    raw = st[which + "_codes"].reshape(-1, st["heads"], P * dim // 2)[pages, head]
    raw = raw.reshape(len(pages) * P, 16 // cut, G, cut).transpose(1, 2).reshape(-1, G, 16)
    code = torch.stack([raw % 16, raw // 16], -1).reshape(-1, G, 32).double()
    zero = st[which + "_zeros"].reshape(-1, st["heads"], P)[pages, head].reshape(-1).long() % (1 << 32)
    zero = torch.stack([(zero // 16 ** g) % 16 for g in range(G)], -1).double()
    scale = st[which + "_scales"].view(torch.float16).reshape(-1, st["heads"], P * G)[pages, head]
    return ((code - zero[..., None]) * scale.double().reshape(-1, G)[..., None]).reshape(-1, dim)


def _exact_attention(st, case):
    P, heads = st["page"], st["heads"]
    grp = st["q"].shape[1] // heads
    q = st["q"].double()
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.full(q.shape[:2], float("-inf"), dtype=torch.float64, device=DEV)
    mass = None if st["mass"] is None else st["mass"].double()
    at = 0
    for b, (n, m) in enumerate(zip(_lengths(case), _queries(case))):
        pages = st["pages"][b, :-(-n // P)].long()
        for h in range(heads if n else 0):
            k, v = (_exact_values(st, which, pages, h)[:n] for which in ("k", "v"))
            gap = (n - m + torch.arange(m, device=DEV))[:, None] - torch.arange(n, device=DEV)
            hidden = gap < 0
            if st["window"]:
                hidden = hidden | (gap >= st["window"])
            weight = torch.zeros(len(pages) * P, dtype=torch.float64, device=DEV)
            for i in range(grp):
                s = q[at:at + m, h * grp + i] @ k.T * st["scale"]
                if st["softcap"]:
                    s = torch.tanh(s / st["softcap"]) * st["softcap"]
                if st["slopes"] is not None:
                    s = s - st["slopes"][h * grp + i].double() * gap
                s = s.masked_fill(hidden, float("-inf"))
                lse[at:at + m, h * grp + i] = torch.logsumexp(s, -1)
                w = torch.nan_to_num(torch.softmax(s, -1))
                out[at:at + m, h * grp + i] = w @ v
                weight[:n] += w.sum(0)
            if mass is not None:
                mass.view(-1, heads, P)[pages, h] += weight.view(-1, P)
        at += m
    return [out, lse] if mass is None else [out, lse, mass]


def _exact_append(st):
    got = []
    for x in (st["k"], st["v"]):
        x = x.double().reshape(-1, 32)
        spread = (x.max(1).values - x.min(1).values) / 15
        # FP16: 11 significant bits, a step of 2^-24 at the least
        mant, expo = torch.frexp(spread)
        step = torch.ldexp(torch.ones_like(mant), (expo - 11).clamp(min=-24))
        scale = torch.round(spread / step) * step
        ok = scale > 0
        zero = torch.round(-x.min(1).values / scale).clamp(0, 15)
        code = (torch.round(x / scale[:, None]) + zero[:, None]).clamp(0, 15)
        value = (code - zero[:, None]) * scale[:, None]
        got.append(torch.where(ok[:, None], value, 0.0).reshape(st["k"].shape))
    return got


def _exact_evict(st, case):
    P, heads, dim, budget = st["page"], st["heads"], st["dim"], st["budget"]
    lengths = _lengths(case)
    n_new = [min(n, budget) for n in lengths]
    k = torch.zeros((len(lengths), budget, heads, dim), dtype=torch.float64, device=DEV)
    v = torch.zeros_like(k)
    mass = st["mass"].double().reshape(-1, heads, P)
    moved = mass.clone()
    for b, n in enumerate(lengths):
        pages = st["pages"][b, :-(-n // P)].long()
        for h in range(heads):
            m = mass[pages, h].reshape(-1)[:n]
            host = m.tolist()
            old = max(0, n - case["recent"])
            keep = sorted(range(old), key=lambda i: (-host[i], i))[:max(0, n_new[b] - (n - old))]
            keep = sorted(keep) + list(range(old, n))
            keep = torch.tensor(keep[len(keep) - n_new[b]:], device=DEV)
            k[b, :len(keep), h] = _exact_values(st, "k", pages, h)[keep]
            v[b, :len(keep), h] = _exact_values(st, "v", pages, h)[keep]
            i = torch.arange(len(keep), device=DEV)
            moved[st["dst_pages"][b].long()[i // P], h, i % P] = m[keep]
    return [torch.tensor(n_new, dtype=torch.int32, device=DEV), k.reshape(-1, heads, dim), v.reshape(-1, heads, dim),
            moved.reshape(-1)]


def _exact_sample(st):
    import numpy as np
    ids, logp = [], []
    for r in range(len(st["u"])):
        x = st["logits"][r].double().cpu().numpy()
        w = np.exp((x - x.max()) / float(st["temperature"][r]))
        order = np.lexsort((np.arange(len(x)), -x))  # by value, then by index
        k, p, least = int(st["top_k"][r]), float(st["top_p"][r]), float(st["min_p"][r])
        kept = order[:k] if k > 0 else order
        if p < 1:
            ahead = np.concatenate([[0.0], np.cumsum(w[kept])])
            kept = kept[ahead[:-1] < p * ahead[-1]]
        kept = np.sort(kept[w[kept] >= least])
        sums = np.cumsum(w[kept])
        i = min(int(np.searchsorted(sums, float(st["u"][r]) * sums[-1], side="right")), len(kept) - 1)
        ids.append(int(kept[i]))
        logp.append(float(np.log(w[kept[i]] / sums[-1])))
    return [torch.tensor(ids, dtype=torch.int32, device=DEV), torch.tensor(logp, dtype=torch.float64, device=DEV)]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "append":
        return _exact_append(st)
    if op == "attention":
        return _exact_attention(st, case)
    if op == "evict":
        return _exact_evict(st, case)
    return _exact_sample(st)
