"""Measured cases of the operators around a paged key/value cache.

Four operators of a serving step of one attention layer (head size 128, bf16):

  rope     RMS norm of every query and key head and the position rotation in
           one pass, from the rows of a fused projection to the layout that
           the attention reads;
  append   the new tokens' keys (normed and rotated on the way) and values
           into the pages of the cache, the queries beside them, and the
           per-page minima and maxima of the keys that a selection reads;
  attn     causal attention of each sequence's new tokens (one, or a chunk)
           over its pages;
  select   the pages that a cheap upper bound of the logits selects for each
           new token, and the attention over them.

``run`` computes the plain form with elementary torch operations, or, where
``own`` is true, calls the library's entry points.
"""

import math
import random

import torch

own = False

D = 128
EPS = 1e-6

# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # one step of 16 chat sequences of the 64/8-head layer: the rows of the fused projection,
        # normed and rotated in token order
        dict(name="rope_step_16", op="rope", batch=1, tokens=16, hq=64, hkv=8, rot=128, pairs=0,
             norm=1, head_major=0, far=131072),
        # four 16K prompts of the 32/8-head layer, written head by head for the prefill
        dict(name="rope_prompts_4x16384", op="rope", batch=4, tokens=16384, hq=32, hkv=8, rot=128,
             pairs=0, norm=1, head_major=1, far=0),
        # one step of 64 sequences: one token each into its page, with its queries
        dict(name="append_step_64", op="append", seqs=64, q_len=1, mix=0, kv=4096, hq=32, hkv=8,
             page=16, rot=128, pairs=0, norm=1, queries=1, summary=1),
        # ragged prompt chunks of five sequences into pages of 64, odd lengths, some at odd places
        dict(name="append_chunks_5", op="append", seqs=5, q_len=2047, mix=1, kv=16384, hq=64,
             hkv=8, page=64, rot=128, pairs=0, norm=1, queries=0, summary=1),
        # one chat sequence early in its answer: the smallest call, all latency
        dict(name="attn_token_1000", op="attn", seqs=1, q_len=1, mix=0, kv=1000, hq=32, hkv=8,
             page=16),
        # a batch of 32 sequences of very different lengths, one token each
        dict(name="attn_tokens_32x16384", op="attn", seqs=32, q_len=1, mix=1, kv=16384, hq=32,
             hkv=8, page=64),
        # one token at the end of a 128K context of the 64/8-head layer
        dict(name="attn_token_131071", op="attn", seqs=1, q_len=1, mix=0, kv=131071, hq=64, hkv=8,
             page=128),
        # a 2048-token prompt chunk at the end of a 32K context: the most work
        dict(name="attn_chunk_2048_at_32768", op="attn", seqs=1, q_len=2048, mix=0, kv=32768,
             hq=32, hkv=8, page=64),
        # a mixed step: chunks of up to 509 tokens beside single tokens, five query heads a kv head
        dict(name="attn_mixed_12", op="attn", seqs=12, q_len=509, mix=2, kv=8191, hq=20, hkv=4,
             page=32),
        # one token over 32 pages of a 128K context
        dict(name="select_token_131072", op="select", seqs=1, q_len=1, mix=0, kv=131072, hq=32,
             hkv=8, page=64, sink=2, local=4, top=26),
        # a batch of 16 sequences over small pages, eight query heads a kv head
        dict(name="select_tokens_16x32768", op="select", seqs=16, q_len=1, mix=1, kv=32768, hq=64,
             hkv=8, page=16, sink=4, local=16, top=108),
        # short chunks, every token with pages of its own
        dict(name="select_chunk_2x125", op="select", seqs=2, q_len=125, mix=0, kv=16381, hq=32,
             hkv=8, page=32, sink=2, local=4, top=26),
    ]


HEADS = [(32, 8), (64, 8), (20, 4), (8, 2), (6, 6), (28, 4), (16, 1)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn", "select", "select"])
    hq, hkv = rng.choice(HEADS)
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        batch = rng.choice([1, 1, 2, 3])
        tokens = min(_log(rng, 1, 65536), 65536 * 40 // ((hq + hkv) * batch))
        return dict(op=op, batch=batch, tokens=tokens, hq=hq, hkv=hkv,
                    rot=rng.choice([128, 128, 64, 32]), pairs=rng.randint(0, 1),
                    norm=rng.randint(0, 1), head_major=rng.randint(0, 1),
                    far=rng.choice([0, 131072]))
    seqs = _log(rng, 1, 96)
    if op == "append":
        kv = _log(rng, 1, 16384)
        q_len = 1 if rng.random() < 0.4 else _log(rng, 1, max(1, min(kv, 10000 // seqs)))
        return dict(op=op, seqs=seqs, q_len=q_len, mix=rng.randint(0, 2), kv=kv, hq=hq, hkv=hkv,
                    page=page, rot=rng.choice([128, 128, 64]), pairs=rng.randint(0, 1),
                    norm=rng.randint(0, 1), queries=rng.randint(0, 1), summary=rng.randint(0, 1))
    if op == "attn":
        kv = _log(rng, 1, max(1, min(131072, 500000 // seqs)))
        # query rows times keys of the padded batch, below those of the largest listed case
        room = 2048 * 32768 * 32 // (2 * seqs * kv * hq)
        q_len = 1 if rng.random() < 0.4 else _log(rng, 1, max(1, min(kv, 2048, room)))
        return dict(op=op, seqs=seqs, q_len=q_len, mix=rng.randint(0, 2), kv=kv, hq=hq, hkv=hkv,
                    page=page)
    kv = _log(rng, 1, max(1, min(131072, 500000 // seqs)))
    keys = _log(rng, page, 4096)
    pages = max(2, keys // page)
    local = max(1, pages // 8)
    sink = rng.randint(0, max(0, pages // 8))
    # gathered rows of keys, below 256 tokens x 8 heads x 1024 keys
    room = 256 * 8 * 1024 // (seqs * hkv * pages * page)
    q_len = 1 if rng.random() < 0.5 else _log(rng, 1, max(1, min(kv, 128, room)))
    return dict(op=op, seqs=seqs, q_len=q_len, mix=rng.randint(0, 2), kv=kv, hq=hq, hkv=hkv,
                page=page, sink=sink, local=local, top=pages - local - sink)


def _lengths(case):
    """New tokens and cache lengths (after them) of every sequence, by the case alone.

    mix 0: all sequences alike; 1: both lengths spread below the case's; 2: a
    third of the sequences with chunks, the others with one token.
    """
    rng = random.Random("%d %d %d %d" % (case["seqs"], case["q_len"], case["kv"], case["mix"]))
    n, kv = [], []
    for s in range(case["seqs"]):
        if case["mix"] == 0:
            a, b = case["q_len"], case["kv"]
        else:
            b = case["kv"] if s == 0 else _log(rng, max(1, case["kv"] // 64), case["kv"])
            a = case["q_len"] if s == 0 else rng.randint((case["q_len"] + 1) // 2, case["q_len"])
            if case["mix"] == 2 and s % 3:
                a = 1
        b = max(b, 1)
        n.append(min(a, b))
        kv.append(b)
    return n, kv


# ---------------------------------------------------------------------------
# what a program has in hand
# ---------------------------------------------------------------------------


def _randn(gen, *shape):
    return torch.randn(*shape, device="cuda", dtype=torch.float32, generator=gen)


def _table(rows, rot):
    """cos and sin of position x frequency (base 500000), fp32 [rows, rot]."""
    inv = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    ang = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * inv[None]
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


def _weight(gen):
    return (1.0 + 0.2 * _randn(gen, D)).to(torch.bfloat16)


def _pages(case, gen):
    """Lengths, offsets and a block table over shuffled pages, some of them free."""
    n, kv = _lengths(case)
    page, seqs = case["page"], case["seqs"]
    need = [(x + page - 1) // page for x in kv]
    per_seq = max(need)
    num = sum(need) + 3
    perm = torch.randperm(num, device="cuda", generator=gen).to(torch.int32)
    cu, first = [0], [0]
    for a, b in zip(n, need):
        cu.append(cu[-1] + a)
        first.append(first[-1] + b)
    col = torch.arange(per_seq, device="cuda")[None]
    at = torch.tensor(first[:-1], device="cuda")[:, None] + col
    used = col < torch.tensor(need, device="cuda")[:, None]
    table = torch.where(used, perm[at.clamp(max=num - 1)], torch.zeros_like(perm[:1]))
    return dict(n=n, kv=kv, max_n=max(n), max_kv=max(kv), tokens=cu[-1], per_seq=per_seq,
                num_pages=num, seqs=seqs,
                cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                kv_lens=torch.tensor(kv, dtype=torch.int32, device="cuda"),
                block_table=table.contiguous())


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    st = dict(case=case)
    hq, hkv = case["hq"], case["hkv"]
    if case["op"] == "rope":
        b, t = case["batch"], case["tokens"]
        rows = max(case["far"], t)
        qkv = torch.empty(b, t, hq + 2 * hkv, D, device="cuda", dtype=torch.bfloat16)
        for x in qkv:
            x.copy_(_randn(gen, t, hq + 2 * hkv, D))
        pos = torch.arange(t, device="cuda", dtype=torch.int32).expand(b, t)
        if case["far"]:
            pos = torch.randint(0, rows, (b, t), device="cuda", generator=gen, dtype=torch.int32)
        st.update(qkv=qkv, positions=pos.contiguous(), table=_table(rows, case["rot"]),
                  q_weight=_weight(gen) if case["norm"] else None,
                  k_weight=_weight(gen) if case["norm"] else None)
        shape = (lambda h: (b, h, t, D)) if case["head_major"] else (lambda h: (b, t, h, D))
        st.update(q_out=torch.empty(shape(hq), device="cuda", dtype=torch.bfloat16),
                  k_out=torch.empty(shape(hkv), device="cuda", dtype=torch.bfloat16))
    else:
        st.update(_pages(case, gen))
        t, page, num = st["tokens"], case["page"], st["num_pages"]
        # keys around a mean of their page, so that pages differ; a shared part in the queries
        cache = torch.empty(2, num, hkv, page, D, device="cuda", dtype=torch.bfloat16)
        step = max(1, 1 << 26 >> (hkv * page * D).bit_length())
        for i in range(0, num, step):
            m = min(step, num - i)
            cache[0, i:i + m] = _randn(gen, m, hkv, page, D) + 0.5 * _randn(gen, m, hkv, 1, D)
            cache[1, i:i + m] = _randn(gen, m, hkv, page, D)
        qkv = _randn(gen, t, hq + 2 * hkv, D)
        qkv += _randn(gen, 1, hq + 2 * hkv, D)
        st.update(qkv=qkv.to(torch.bfloat16), k_cache=cache[0], v_cache=cache[1])
        if case["op"] == "append":
            st.update(table=_table(st["max_kv"], case["rot"]),
                      q_weight=_weight(gen) if case["norm"] else None,
                      k_weight=_weight(gen) if case["norm"] else None,
                      q_out=torch.empty(t, hq, D, device="cuda", dtype=torch.bfloat16),
                      summary=torch.stack([st["k_cache"].amin(2), st["k_cache"].amax(2)], 2))
        else:
            st.update(q=st["qkv"][:, :hq],
                      o=torch.empty(t, hq, D, device="cuda", dtype=torch.bfloat16),
                      lse=torch.empty(t, hq, device="cuda", dtype=torch.float32))
        if case["op"] == "select":
            width = case["sink"] + case["top"] + case["local"]
            st.update(summary=torch.stack([st["k_cache"].amin(2), st["k_cache"].amax(2)], 2),
                      lists=torch.empty(t, hkv, width, device="cuda", dtype=torch.int32),
                      counts=torch.empty(t, hkv, device="cuda", dtype=torch.int32))
    st["error"] = torch.zeros(1, device="cuda", dtype=torch.int32)
    st["handle"] = {}
    return st


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------


def _handles(st):
    """Parameters and workspace, made once for a state as a program does."""
    import block_sparse_long_sm_b200 as spa
    case, h = st["case"], st["handle"]
    if case["op"] in ("rope", "append"):
        h["rope"] = spa.make_rope_params(
            case.get("batch", 1), case["tokens"] if case["op"] == "rope" else st["tokens"],
            case["hq"], case["hkv"], table_rows=st["table"].shape[0], rotary_dim=case["rot"],
            interleaved=case["pairs"], eps=EPS)
    if case["op"] != "rope":
        h["paged"] = spa.make_paged_params(
            case["hq"], case["hkv"], page_size=case["page"], num_pages=st["num_pages"],
            seqs=st["seqs"], tokens=st["tokens"], pages_per_seq=st["per_seq"],
            sink_pages=case.get("sink", 0), local_pages=case.get("local", 1),
            top_pages=case.get("top", 0))
        if case["op"] != "append":
            h["ws"] = torch.empty(spa.sparse_paged_workspace_bytes(h["paged"]),
                                  dtype=torch.uint8, device="cuda")
    h["spa"] = spa
    return h


def _run_own(st):
    h = st["handle"] or _handles(st)
    spa, case = h["spa"], st["case"]
    hq, hkv = case["hq"], case["hkv"]
    qkv = st.get("qkv")
    if case["op"] == "rope":
        q_out, k_out = st["q_out"], st["k_out"]
        hm = case["head_major"]
        spa.check(spa.sparse_qk_norm_rope(
            h["rope"], qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], st["q_weight"], st["k_weight"],
            st["positions"], st["table"], q_out.transpose(1, 2) if hm else q_out,
            k_out.transpose(1, 2) if hm else k_out, st["error"]), "rope")
        return q_out, k_out
    if case["op"] == "append":
        queries = case["queries"]
        spa.check(spa.sparse_paged_append(
            h["paged"], h["rope"], qkv[:, :hq] if queries else None, qkv[:, hq:hq + hkv],
            qkv[:, hq + hkv:], st["q_weight"] if queries else None, st["k_weight"], st["table"],
            st["cu_q"], st["kv_lens"], st["block_table"], st["q_out"] if queries else None,
            st["k_cache"], st["v_cache"], st["summary"] if case["summary"] else None,
            st["error"]), "append")
        out = [st["k_cache"], st["v_cache"]]
        out += [st["q_out"]] if queries else []
        return out + ([st["summary"]] if case["summary"] else [])
    lists = counts = None
    if case["op"] == "select":
        lists, counts = st["lists"], st["counts"]
        spa.check(spa.sparse_paged_select(
            h["paged"], st["q"], st["summary"], st["cu_q"], st["kv_lens"], st["block_table"],
            lists, counts, h["ws"], st["error"]), "select")
    spa.check(spa.sparse_paged_attn(
        h["paged"], st["q"], st["k_cache"], st["v_cache"], st["cu_q"], st["kv_lens"],
        st["block_table"], lists, counts, st["o"], st["lse"], h["ws"], st["error"]), "attn")
    out = [st["o"], st["lse"]]
    return out + [lists, counts] if case["op"] == "select" else out


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------


def _norm_rotate(x, weight, cos, sin, rot, pairs):
    """x fp32 [..., heads, 128]; cos, sin [..., 1, rot / 2]."""
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    half = rot // 2
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., :half], x[..., half:rot])
    y = torch.empty_like(x)
    y[..., rot:] = x[..., rot:]
    if pairs:
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        y[..., :half], y[..., half:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _tokens(st):
    """Sequence, index in it, and cache position of every token."""
    cu, t = st["cu_q"].long(), st["tokens"]
    at = torch.arange(t, device="cuda")
    seq = torch.bucketize(at, cu[1:], right=True)
    loc = at - cu[seq]
    n = cu[1:] - cu[:-1]
    return seq, loc, st["kv_lens"].long()[seq] - n[seq] + loc


def _plain_rope(st):
    case = st["case"]
    hq, hkv, rot = case["hq"], case["hkv"], case["rot"]
    cs = st["table"][st["positions"].long()].unsqueeze(-2)
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    out = []
    for x, w, buf in ((st["qkv"][:, :, :hq], st["q_weight"], st["q_out"]),
                      (st["qkv"][:, :, hq:hq + hkv], st["k_weight"], st["k_out"])):
        y = _norm_rotate(x.float(), w, cos, sin, rot, case["pairs"])
        buf.copy_(y.transpose(1, 2) if case["head_major"] else y)
        out.append(buf)
    return tuple(out)


def _plain_append(st):
    case = st["case"]
    hq, hkv, rot, page = case["hq"], case["hkv"], case["rot"], case["page"]
    seq, _, pos = _tokens(st)
    cs = st["table"][pos].unsqueeze(-2)
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    k = _norm_rotate(st["qkv"][:, hq:hq + hkv].float(), st["k_weight"], cos, sin, rot,
                     case["pairs"])
    where = st["block_table"].long()[seq, pos // page]
    st["k_cache"][where, :, pos % page] = k.to(torch.bfloat16)
    st["v_cache"][where, :, pos % page] = st["qkv"][:, hq + hkv:]
    out = [st["k_cache"], st["v_cache"]]
    if case["queries"]:
        q = _norm_rotate(st["qkv"][:, :hq].float(), st["q_weight"], cos, sin, rot, case["pairs"])
        st["q_out"].copy_(q)
        out.append(st["q_out"])
    if case["summary"]:
        # rows of the touched pages that the sequence has filled; a page may come several times
        rows = torch.arange(page, device="cuda")
        filled = (pos // page * page)[:, None] + rows < st["kv_lens"].long()[seq][:, None]
        kk = st["k_cache"][where].float()
        lo = torch.where(filled[:, None, :, None], kk, math.inf).amin(2)
        hi = torch.where(filled[:, None, :, None], kk, -math.inf).amax(2)
        st["summary"][where] = torch.stack([lo, hi], 2).to(torch.bfloat16)
        out.append(st["summary"])
    return out


def _gathered(st, cache):
    """fp32 [seqs, hkv, keys, 128] of every sequence's pages."""
    x = cache[st["block_table"].long()].float()
    return x.transpose(1, 2).flatten(2, 3)[:, :, :st["max_kv"]]


def _softmax_rows(s, v):
    """Attention and LSE of masked scores s [..., rows, keys] (no row is empty)."""
    m = s.amax(-1, keepdim=True)
    s.sub_(m).exp_()
    l = s.sum(-1, keepdim=True)
    return torch.matmul(s, v) / l, (m + l.log()).squeeze(-1)


def _plain_attn(st):
    case = st["case"]
    hq, hkv = case["hq"], case["hkv"]
    seqs, n = st["seqs"], st["max_n"]
    seq, loc, pos = _tokens(st)
    q = torch.zeros(seqs, n, hq, D, device="cuda")
    q[seq, loc] = st["q"].float()
    last = torch.zeros(seqs, n, dtype=torch.long, device="cuda")
    last[seq, loc] = pos
    q = q.view(seqs, n, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4).reshape(seqs, hkv, -1, D)
    s = torch.matmul(q, _gathered(st, st["k_cache"]).transpose(2, 3)).mul_(1.0 / math.sqrt(D))
    keys = torch.arange(st["max_kv"], device="cuda")
    hidden = keys[None, None] > last[:, :, None]
    s.view(seqs, hkv, hq // hkv, n, -1).masked_fill_(hidden[:, None, None], -math.inf)
    o, lse = _softmax_rows(s, _gathered(st, st["v_cache"]))
    o = o.view(seqs, hkv, -1, n, D).permute(0, 3, 1, 2, 4).reshape(seqs, n, hq, D)
    lse = lse.view(seqs, hkv, -1, n).permute(0, 3, 1, 2).reshape(seqs, n, hq)
    return [o[seq, loc].to(torch.bfloat16), lse[seq, loc]]


def _plain_select(st):
    case = st["case"]
    hq, hkv, page = case["hq"], case["hkv"], case["page"]
    sink, top, local = case["sink"], case["top"], case["local"]
    group, t, per_seq = hq // hkv, st["tokens"], st["per_seq"]
    seq, _, pos = _tokens(st)
    table = st["block_table"].long()[seq]
    # the score in 64 bits, rounded once: values next to the border of the selection
    q = st["q"].double().view(t, hkv, group, D)
    bound = torch.empty(t, hkv, per_seq, device="cuda")
    step = max(1, (1 << 30) // (per_seq * hkv * 2 * D * 8))
    for i in range(0, t, step):  # in pieces that fit in memory
        sm = st["summary"][table[i:i + step]].double()  # [., pages, hkv, 2, D]
        lo, hi = (sm[:, :, :, j].permute(0, 2, 3, 1) for j in (0, 1))
        a = q[i:i + step]
        u = torch.matmul(a.clamp(min=0), hi) + torch.matmul(a.clamp(max=0), lo)
        bound[i:i + step] = u.amax(2).float()
    idx = torch.arange(per_seq, device="cuda")
    seen = (pos // page + 1)[:, None]
    always = ((idx < sink) | (idx >= seen - local)) & (idx < seen)
    open_ = (idx >= sink) & (idx < seen - local)
    rank = torch.where(open_[:, None], bound, -math.inf).sort(dim=-1, descending=True, stable=True)[1]
    keep = torch.zeros(t, hkv, per_seq, dtype=torch.bool, device="cuda")
    keep.scatter_(2, rank[:, :, :top], True)
    keep = (keep & open_[:, None]) | always[:, None]
    counts = keep.sum(-1).to(torch.int32)
    width = sink + top + local
    order = torch.where(keep, idx, per_seq).sort(dim=-1)[0]
    order = torch.nn.functional.pad(order, (0, width), value=per_seq)[:, :, :width]
    lists = torch.where(order < per_seq, order, -1).to(torch.int32)
    # attention over the listed pages
    at = torch.where(order < per_seq, order, 0)
    where = table[:, None].expand(t, hkv, per_seq).gather(2, at)
    head = torch.arange(hkv, device="cuda")[None, :, None]
    key = (order[..., None] * page + torch.arange(page, device="cuda")).flatten(2)
    hidden = (key > pos[:, None, None]) | (key >= per_seq * page)
    k = st["k_cache"][where, head].flatten(2, 3).float()
    s = torch.matmul(st["q"].float().view(t, hkv, group, D), k.transpose(2, 3))
    s = s.mul_(1.0 / math.sqrt(D)).masked_fill_(hidden[:, :, None], -math.inf)
    del k
    o, lse = _softmax_rows(s, st["v_cache"][where, head].flatten(2, 3).float())
    return [o.reshape(t, hq, D).to(torch.bfloat16), lse.reshape(t, hq), lists, counts]


def run(state):
    if own:
        return _run_own(state)
    plain = dict(rope=_plain_rope, append=_plain_append, attn=_plain_attn, select=_plain_select)
    return plain[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    hq, hkv = case["hq"], case["hkv"]
    row = 2 * D
    if case["op"] == "rope":
        t = case["batch"] * case["tokens"]
        return dict(bytes=t * (hq + hkv) * row * 2 + t * (4 * case["rot"] + 4),
                    flops=t * (hq + hkv) * D * 7)
    n, kv = _lengths(case)
    page, t = case["page"], sum(n)
    if case["op"] == "append":
        rows = t * (2 * hkv + (hq if case["queries"] else 0))
        touched = sum((b - 1) // page - (b - a) // page + 1 for a, b in zip(n, kv))
        old = sum((b - a) % page for a, b in zip(n, kv))
        more = (touched * hkv * 2 * row + old * hkv * row) if case["summary"] else 0
        return dict(bytes=rows * row * 2 + t * 4 * case["rot"] + more, flops=rows * D * 7)
    if case["op"] == "attn":
        pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(n, kv))
        return dict(bytes=sum(kv) * hkv * row * 2 + t * hq * (2 * row + 4),
                    flops=4 * D * hq * pairs)
    width = case["sink"] + case["top"] + case["local"]
    pages = pairs = loads = scored = 0
    for a, b in zip(n, kv):
        own_keys = 0
        for i in range(a):
            p = b - a + i
            seen = p // page + 1
            kept = min(seen, width)
            keys = (kept - 1) * page + p % page + 1
            own_keys += keys
            scored += max(0, seen - case["sink"] - case["local"])
        pairs += own_keys
        pages += max(0, (b - 1) // page + 1 - case["sink"] - case["local"])
        loads += min(own_keys, b)
    return dict(bytes=pages * hkv * 2 * row + loads * hkv * row * 2 + t * hq * (2 * row + 4) +
                t * hkv * (width + 1) * 4,
                flops=4 * D * hq * pairs + 2 * D * hq * scored)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------


def _exact_rows(x, weight, angles, rot, pairs):
    """One token's heads x [heads, 128] as complex numbers turned by its angles' cos and sin."""
    x = x.double()
    if weight is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * weight.double()
    turn = torch.complex(angles[..., :rot // 2].double(), angles[..., rot // 2:].double())
    part = x[..., :rot]
    part = part.unflatten(-1, (rot // 2, 2)) if pairs else part.unflatten(-1, (2, -1)).mT
    z = torch.complex(part[..., 0].contiguous(), part[..., 1].contiguous()) * turn[..., None, :]
    y = torch.stack([z.real, z.imag], -1)
    y = y.flatten(-2) if pairs else y.mT.flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _exact_attend(q, k, v, hidden):
    s = (q @ k.T) / D ** 0.5
    s = s.masked_fill(hidden, -math.inf)
    return s.softmax(-1) @ v, s.logsumexp(-1)


def exact(case, seed):
    st = prepare(case, seed)
    hq, hkv = case["hq"], case["hkv"]
    group = hq // hkv
    if case["op"] == "rope":
        outs = []
        for lo, hi, w in ((0, hq, st["q_weight"]), (hq, hq + hkv, st["k_weight"])):
            y = torch.empty(case["batch"], case["tokens"], hi - lo, D, device="cuda",
                            dtype=torch.float64)
            for b in range(case["batch"]):
                for i in range(0, case["tokens"], 4096):
                    ang = st["table"][st["positions"][b, i:i + 4096].long()]
                    y[b, i:i + 4096] = _exact_rows(st["qkv"][b, i:i + 4096, lo:hi], w, ang,
                                                   case["rot"], case["pairs"])
            outs.append(y.transpose(1, 2) if case["head_major"] else y)
        return tuple(outs)
    page, t = case["page"], st["tokens"]
    if case["op"] == "append":
        kc, vc = st["k_cache"].double(), st["v_cache"].double()
        sm = st["summary"].double()
        qo = torch.empty(t, hq, D, device="cuda", dtype=torch.float64)
        at = 0
        for s, (a, b) in enumerate(zip(st["n"], st["kv"])):
            x = st["qkv"][at:at + a]
            ang = st["table"][b - a:b]
            new = _exact_rows(x[:, hq:hq + hkv], st["k_weight"], ang, case["rot"], case["pairs"])
            qo[at:at + a] = _exact_rows(x[:, :hq], st["q_weight"], ang, case["rot"],
                                        case["pairs"])
            for j in range((b - a) // page, (b - 1) // page + 1):
                phys = int(st["block_table"][s, j])
                lo, hi = max(b - a, j * page), min(b, (j + 1) * page)
                rows = slice(lo - j * page, hi - j * page)
                kc[phys, :, rows] = new[lo - b + a:hi - b + a].transpose(0, 1)
                vc[phys, :, rows] = x[lo - b + a:hi - b + a, hq + hkv:].double().transpose(0, 1)
                full = kc[phys, :, :hi - j * page]
                sm[phys, :, 0], sm[phys, :, 1] = full.amin(1), full.amax(1)
            at += a
        out = [kc, vc] + ([qo] if case["queries"] else [])
        return out + ([sm] if case["summary"] else [])
    o = torch.empty(t, hq, D, device="cuda", dtype=torch.float64)
    lse = torch.empty(t, hq, device="cuda", dtype=torch.float64)
    if case["op"] == "attn":
        at = 0
        for s, (a, b) in enumerate(zip(st["n"], st["kv"])):
            pages = st["block_table"][s, :(b + page - 1) // page].long()
            future = (torch.arange(b, device="cuda")[None] >
                      torch.arange(b - a, b, device="cuda")[:, None])
            for g in range(hkv):
                k = st["k_cache"][pages, g].reshape(-1, D)[:b].double()
                v = st["v_cache"][pages, g].reshape(-1, D)[:b].double()
                for h in range(g * group, (g + 1) * group):
                    o[at:at + a, h], lse[at:at + a, h] = _exact_attend(
                        st["q"][at:at + a, h].double(), k, v, future)
            at += a
        return [o, lse]
    if t * hkv > 4096:
        return None
    at = 0
    for s, (a, b) in enumerate(zip(st["n"], st["kv"])):
        pages = st["block_table"][s].long()
        lo = st["summary"][pages, :, 0].double()
        hi = st["summary"][pages, :, 1].double()
        for i in range(a):
            p = b - a + i
            seen = p // page + 1
            first, last = min(case["sink"], seen), max(seen - case["local"], 0)
            for g in range(hkv):
                qg = st["q"][at + i, g * group:(g + 1) * group].double()
                if last - first > case["top"]:
                    u = torch.maximum(qg[:, None] * lo[None, first:last, g],
                                      qg[:, None] * hi[None, first:last, g])
                    u = u.sum(-1).amax(0).float()
                    best = u.argsort(descending=True, stable=True)[:case["top"]] + first
                else:
                    best = torch.arange(first, max(first, last), device="cuda")
                sel = torch.cat([torch.arange(first, device="cuda"), best,
                                 torch.arange(max(first, last), seen, device="cuda")])
                key = (sel[:, None] * page + torch.arange(page, device="cuda")).flatten()
                ph = pages[sel]
                o[at + i, g * group:(g + 1) * group], lse[at + i, g * group:(g + 1) * group] = \
                    _exact_attend(qg, st["k_cache"][ph, g].reshape(-1, D).double(),
                                  st["v_cache"][ph, g].reshape(-1, D).double(), (key > p)[None])
        at += a
    return [o, lse, None, None]
