"""Measured cases of the paged latent cache: the append with the position rotation on the way, attention of
new tokens over the pages, the choice of pages by a cheap score, and attention over the chosen pages.

The cache is a pool of pages, [num_pages, page_size, d_c + d_r]; block_table[b, i] is the page that holds rows
i * page_size .. of sequence b; kv_lens[b] counts its cached rows, the new tokens included, and cu_q packs the
new tokens, the last ones of each sequence. Every query head attends over the one latent row of each token.
"""
import functools
import random

import torch

own = False

DEVICE = "cuda"
#: heads, latent width, rotary width, type of the cache and the queries (the sizes of this repository's
#: bf16 and fp32 configurations)
DIMS = {
    "v3": {"n_h": 128, "d_h": 128, "d_c": 512, "d_r": 64, "dtype": torch.bfloat16},
    "tiny": {"n_h": 4, "d_h": 32, "d_c": 64, "d_r": 16, "dtype": torch.float32},
}
ROPE_BASE = 10000.0


def _case(name, op, dims, batch, tq, len_lo, len_hi, page, ragged=0, top_k=0, first=0, last=0):
    """batch sequences of len_lo .. len_hi cached rows, the last tq of them new (ragged: 1 .. tq)."""
    return {"name": name, "op": op, "dims": dims, "batch": batch, "tq": tq, "len_lo": len_lo, "len_hi": len_hi,
            "page": page, "ragged": ragged, "top_k": top_k, "first": first, "last": last}


def listed():
    return [
        # one decode step's new rows, a batch of 16 sequences (launch latency counts)
        _case("append_decode_b16", "append", "v3", 16, 1, 4096, 4096, 64),
        # the rows of a chunked prompt, ragged chunks, pages that end inside a chunk
        _case("append_chunk_ragged", "append", "v3", 5, 2047, 2048, 9001, 64, ragged=1),
        # one short sequence on small pages: the smallest call
        _case("attn_b1_l77", "attn", "v3", 1, 1, 77, 77, 16),
        # a decode step of the usual batch
        _case("attn_decode_b16_l4096", "attn", "v3", 16, 1, 4096, 4096, 64),
        # draft-and-verify decode: two tokens a sequence, ragged lengths
        _case("attn_mtp_b64_ragged", "attn", "v3", 64, 2, 1024, 32768, 64),
        # a few long sequences: the cache's bytes count
        _case("attn_long_b4_l131072", "attn", "v3", 4, 1, 131072, 131072, 64),
        # short chunks of new tokens behind long prefixes: the products count
        _case("attn_chunk_b8_t64_l16384", "attn", "v3", 8, 64, 15001, 16384, 64, ragged=1),
        # the exact fp32 configuration, ragged chunks on odd lengths
        _case("attn_fp32_ragged", "attn", "tiny", 9, 5, 33, 700, 32, ragged=1),
        # the choice of pages for a decode step over long sequences
        _case("select_decode_b4_l131072", "select", "v3", 4, 1, 131072, 131072, 64, top_k=64, first=1, last=2),
        # the choice of pages for every token of a chunk
        _case("select_chunk_t512_l32768", "select", "v3", 1, 512, 32768, 32768, 64, top_k=32, first=1, last=2),
        # a decode step over the chosen pages, ragged lengths
        _case("sparse_decode_b16", "sparse", "v3", 16, 1, 8001, 65536, 64, top_k=32, first=1, last=2),
        # a chunk over the chosen pages, each token its own
        _case("sparse_chunk_t512_l32768", "sparse", "v3", 1, 512, 32768, 32768, 64, top_k=32, first=1, last=2),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "select", "sparse"])
    page = rng.choice([16, 32, 64, 64, 128])
    if op == "append":
        batch = _log(rng, 1, 64)
        tq = _log(rng, 1, max(1, 8192 // batch))
        lo = tq + _log(rng, 1, 8000) - 1
        return _case("", op, rng.choice(["v3", "v3", "tiny"]), batch, tq, lo, lo + rng.randrange(500), page,
                     ragged=rng.randrange(2))
    if op == "attn" and rng.random() < 0.2:
        lo = _log(rng, 8, 700)
        return _case("", op, "tiny", _log(rng, 1, 32), rng.randint(1, 8), lo, lo + rng.randrange(300), page, ragged=1)
    if op == "attn":
        batch, tq = _log(rng, 1, 64), _log(rng, 1, 64)
        most = min(131072, 6_000_000 // (batch * tq), 2_000_000 // batch)
        hi = _log(rng, tq, max(tq + 1, most))
        return _case("", op, "v3", batch, tq, max(tq, rng.randint(hi // 4, hi)), hi, page, ragged=rng.randrange(2))
    page = max(page, 32)
    first, last = rng.randrange(3), rng.randint(1, 4)
    top_k = max(first + last, _log(rng, 4, 64))
    batch = _log(rng, 1, 16)
    tq = _log(rng, 1, max(1, 512 // batch))
    lo = tq + _log(rng, 1, 60000)
    if op == "sparse":
        top_k = max(first + last, min(top_k, 1_000_000 // (batch * tq * page)))
    return _case("", op, "v3", batch, tq, lo, lo + rng.randrange(3000), page, ragged=rng.randrange(2), top_k=top_k,
                 first=first, last=last)


def _lengths(case):
    """(new tokens, cached rows) of each sequence: a function of the case alone."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    tq = [r.randint(1, case["tq"]) if case["ragged"] else case["tq"] for _ in range(case["batch"])]
    lens = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["batch"])]
    return tq, [max(n, t) for n, t in zip(lens, tq)]


def work(case):
    d = DIMS[case["dims"]]
    es = torch.finfo(d["dtype"]).bits // 8
    row, heads, page = (d["d_c"] + d["d_r"]) * es, d["n_h"], case["page"]
    tq, lens = _lengths(case)
    T = sum(tq)
    if case["op"] == "append":
        done = sum(n // page - (n - t) // page for t, n in zip(tq, lens))      # pages that these rows complete
        held = sum((n - t) % page if n // page > (n - t) // page else 0 for t, n in zip(tq, lens))
        nbytes = T * (2 * row + 2 * heads * d["d_r"] * es) + held * row + done * (d["d_c"] + d["d_r"] + 16)
        return {"bytes": nbytes, "flops": T * (heads + 1) * d["d_r"] * 3}
    q = T * heads * (d["d_c"] + d["d_r"]) * es
    out = T * heads * (d["d_c"] * es + 4)
    per = 2 * heads * (2 * d["d_c"] + d["d_r"])                                  # one token over one cached row
    if case["op"] == "attn":
        return {"bytes": sum(lens) * row + q + out, "flops": per * sum(t * n - t * (t - 1) // 2 for t, n in zip(tq, lens))}
    blocks = [-(-n // page) for n in lens]
    if case["op"] == "select":
        return {"bytes": sum(blocks) * (d["d_c"] + d["d_r"] + 4) + q + T * case["top_k"] * 4,
                "flops": 2 * heads * (d["d_c"] + d["d_r"]) * sum(t * n for t, n in zip(tq, blocks))}
    rows = [min(case["top_k"] * page, n) for n in lens]
    return {"bytes": sum(rows) * row + q + out, "flops": per * sum(t * n for t, n in zip(tq, rows))}


def prepare(case, seed):
    d = DIMS[case["dims"]]
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    tq, lens = _lengths(case)
    page, B, T = case["page"], case["batch"], sum(tq)
    blocks = [-(-n // page) for n in lens]
    spare = 3                                                                    # pages of nobody
    num_pages, width = sum(blocks) + spare, max(blocks) + 1
    order = torch.randperm(num_pages, generator=g, device=DEVICE).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEVICE)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[at:at + n]
        at += n

    def normal(*shape, std=1.0, dtype=d["dtype"]):
        return (torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32) * std).to(dtype)

    cache = torch.empty(num_pages, page, d["d_c"] + d["d_r"], dtype=d["dtype"], device=DEVICE)
    step = max(1, (1 << 26) // (page * (d["d_c"] + d["d_r"])))
    for p in range(0, num_pages, step):                                          # rows near their page's own mean
        n = min(step, num_pages - p)
        cache[p:p + n] = normal(n, page, d["d_c"] + d["d_r"], dtype=torch.float32) \
            + normal(n, 1, d["d_c"] + d["d_r"], std=0.3, dtype=torch.float32)
    s = {"case": case, "cache": cache, "table": table,
         "cu_q": torch.tensor([0] + tq, dtype=torch.int64, device=DEVICE).cumsum(0),
         "kv_lens": torch.tensor(lens, dtype=torch.int64, device=DEVICE), "T": T, "max_tq": max(tq), "max_len": max(lens)}
    if case["op"] == "append":
        s["kv"] = normal(T, d["d_c"] + d["d_r"])
        s["q_rope"] = normal(T, d["n_h"], d["d_r"])
        s["q_out"] = torch.empty_like(s["q_rope"])
        s["summaries"] = torch.zeros(num_pages, d["d_c"] + d["d_r"] + 16, dtype=torch.uint8, device=DEVICE)
        return s
    s["q_abs"] = normal(T, d["n_h"], d["d_c"], std=0.5)
    s["q_rope"] = normal(T, d["n_h"], d["d_r"])
    if case["op"] in ("select", "sparse"):
        s["summaries"] = torch.cat([_summarise(cache[p:p + step]) for p in range(0, num_pages, step)])
    if case["op"] == "sparse":
        s["blocks"] = _select(s)
    return s


# ---- the plain forms --------------------------------------------------------------------------------------
def _quantise(x):
    """Codes in -127 .. 127 and the scale of each row of x (fp32): code = x / scale to the nearest, ties to even."""
    scale = x.abs().amax(-1, keepdim=True) / torch.tensor(127.0, device=x.device)
    codes = torch.where(scale > 0, x / torch.where(scale > 0, scale, 1.0), 0.0).round().clamp(-127, 127)
    return codes, scale


def _summarise(pages):
    """Summary rows of whole pages: the codes of the mean row, its scale, 12 zero bytes."""
    codes, scale = _quantise((pages.double().sum(1) / pages.shape[1]).float())
    pad = torch.zeros(pages.shape[0], 12, dtype=torch.uint8, device=pages.device)
    return torch.cat([codes.to(torch.int8).view(torch.uint8), scale.contiguous().view(torch.uint8), pad], 1)


def _tokens(s):
    """Sequence and position of each new token."""
    t = torch.arange(s["T"], device=DEVICE)
    seq = torch.searchsorted(s["cu_q"], t, right=True) - 1
    new = s["cu_q"][1:] - s["cu_q"][:-1]
    return seq, s["kv_lens"][seq] - new[seq] + t - s["cu_q"][seq]


def _rotate(x, pos):
    """Pairs (2m, 2m + 1) of the last axis turned by pos * base^(-2m / d_r); x: [T, ..., d_r]."""
    n = x.shape[-1]
    angle = pos.double()[:, None] * ROPE_BASE ** (-torch.arange(0, n, 2, device=x.device, dtype=torch.float64) / n)
    angle = angle.reshape([x.shape[0]] + [1] * (x.dim() - 2) + [n // 2])
    a, b = x[..., 0::2].double(), x[..., 1::2].double()
    return torch.stack([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1).flatten(-2)


def _append(s):
    d, page = DIMS[s["case"]["dims"]], s["case"]["page"]
    seq, pos = _tokens(s)
    where = s["table"][seq, pos // page].long(), pos % page
    rows = torch.cat([s["kv"][:, :d["d_c"]], _rotate(s["kv"][:, d["d_c"]:], pos).to(d["dtype"])], 1)
    s["cache"].index_put_(where, rows)
    s["q_out"].copy_(_rotate(s["q_rope"], pos))
    fresh = s["table"][seq, pos // page].long()[pos % page == page - 1]          # pages that are whole now
    s["summaries"].index_put_((fresh,), _summarise(s["cache"][fresh]))


def _padded(s, q):
    """[B, max_tq, heads, width] fp32 of packed queries, and each packed token's place in it."""
    seq, _ = _tokens(s)
    at = torch.arange(s["T"], device=DEVICE) - s["cu_q"][seq]
    full = torch.zeros(s["case"]["batch"], s["max_tq"], *q.shape[1:], device=DEVICE)
    full[seq, at] = q.float()
    return full, seq, at


def _attend(q, rows, seen, d):
    """q [N, Q, H, d_c + d_r], rows [N, L, d_c + d_r], seen [N, Q, L]: outputs and log-sum-exp, in fp32."""
    n, width, heads = q.shape[0], q.shape[1], q.shape[2]
    x = torch.bmm(q.reshape(n, width * heads, -1), rows.transpose(1, 2)).mul_((d["d_h"] + d["d_r"]) ** -0.5)
    x = x.view(n, width, heads, -1).masked_fill_(~seen[:, :, None], float("-inf"))
    top = x.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.bmm(x.view(n, width * heads, -1), rows[..., :d["d_c"]]).view(n, width, heads, -1)
    return torch.where(total > 0, o / total, 0.0), (top + total.log())[..., 0]


def _attn(s):
    d, page = DIMS[s["case"]["dims"]], s["case"]["page"]
    q, seq, at = _padded(s, torch.cat([s["q_abs"], s["q_rope"]], -1))
    most = -(-s["max_len"] // page)
    rows = s["cache"][s["table"][:, :most].long().clamp_min(0)].flatten(1, 2).float()
    place = torch.arange(most * page, device=DEVICE)
    rows = rows.masked_fill_((place >= s["kv_lens"][:, None])[..., None], 0.0)
    new = s["cu_q"][1:] - s["cu_q"][:-1]
    pos = (s["kv_lens"] - new)[:, None] + torch.arange(s["max_tq"], device=DEVICE)
    o, lse = _attend(q, rows, place <= pos[..., None], d)
    return [o[seq, at].to(d["dtype"]), lse[seq, at].contiguous()]


def _select(s):
    """The blocks that each token attends to, ascending, -1 behind the last: the first and the last ones, then
    those of the largest score, max over the heads of (codes of q) . (codes of the block) * scales."""
    c, page = s["case"], s["case"]["page"]
    width = s["q_abs"].shape[-1] + s["q_rope"].shape[-1]
    q, seq, at = _padded(s, torch.cat([s["q_abs"], s["q_rope"]], -1))
    codes, scale = _quantise(q)
    most = -(-s["max_len"] // page)
    sums = s["summaries"][s["table"][:, :most].long().clamp_min(0)]
    block_codes = sums[..., :width].contiguous().view(torch.int8).float()
    block_scale = sums[..., width:width + 4].contiguous().view(torch.float32)[..., 0]
    n = codes.shape[0]
    x = torch.bmm(codes.reshape(n, -1, width), block_codes.transpose(1, 2))      # whole numbers below 2^24: exact
    x = (x.view(n, codes.shape[1], -1, most) * scale).amax(2)[seq, at] * block_scale[seq]
    _, pos = _tokens(s)
    seen = (pos // page + 1)[:, None]
    g = torch.arange(most, device=DEVICE)[None]
    x = x.masked_fill_((g < c["first"]) | (g >= seen - c["last"]), float("inf")).masked_fill_(g >= seen, float("-inf"))
    best = x.sort(dim=-1, descending=True, stable=True).indices[:, :c["top_k"]]
    best = torch.where(best < seen, best, most).sort(-1).values
    out = torch.full((s["T"], c["top_k"]), -1, dtype=torch.int32, device=DEVICE)
    out[:, :best.shape[1]] = torch.where(best < most, best, -1)
    return out


def _sparse(s):
    d, page = DIMS[s["case"]["dims"]], s["case"]["page"]
    seq, pos = _tokens(s)
    chosen = s["blocks"].long()
    pages = s["table"][seq[:, None], chosen.clamp_min(0)].long()
    place = (chosen[..., None] * page + torch.arange(page, device=DEVICE)).flatten(1)
    seen = (place <= pos[:, None]) & (chosen >= 0).repeat_interleave(page, 1)
    rows = s["cache"][pages].flatten(1, 2).float().masked_fill_(~seen[..., None], 0.0)
    q = torch.cat([s["q_abs"], s["q_rope"]], -1).float()[:, None]
    o, lse = _attend(q, rows, seen[:, None], d)
    return [o[:, 0].to(d["dtype"]), lse[:, 0]]


# ---- the framework's operators ------------------------------------------------------------------------------
@functools.lru_cache(maxsize=None)
def _module(dims):
    from mla_latent_kv_31_b200 import mla, synth
    return mla.MLA(synth.V3 if dims == "v3" else synth.TINY, None, mla.MLA_BF16 if dims == "v3" else mla.MLA_FP32)


def _own(s):
    from mla_latent_kv_31_b200 import mla
    m, c = _module(s["case"]["dims"]), s["case"]
    batch = mla.PagedBatch(s["cache"], s["table"], s["cu_q"], s["kv_lens"], s["T"])
    if c["op"] == "append":
        m.paged_append(batch, s["kv"], q_rope=s["q_rope"], q_out=s["q_out"], summaries=s["summaries"])
    elif c["op"] == "attn":
        return m.attn_paged(batch, s["q_abs"], s["q_rope"])
    elif c["op"] == "select":
        return m.paged_select(batch, s["q_abs"], s["q_rope"], s["summaries"], c["top_k"], n_first=c["first"], n_last=c["last"])
    else:
        return m.attn_paged_sparse(batch, s["q_abs"], s["q_rope"], s["blocks"])


def _appended(s):
    """The whole state after an append. The summaries' codes are whole numbers, each the exact rounding of a sum
    in 64 bits, so they are returned as such, with their scales."""
    width = s["kv"].shape[1]
    return {"cache": s["cache"], "q": s["q_out"], "codes": s["summaries"][:, :width].view(torch.int8),
            "scales": s["summaries"][:, width:width + 4].view(torch.float32)}


def run(state):
    op = state["case"]["op"]
    if own:
        out = _own(state)
    else:
        out = {"append": _append, "attn": _attn, "select": _select, "sparse": _sparse}[op](state)
    return _appended(state) if op == "append" else out


# ---- the definition in 64 bits, sequence by sequence --------------------------------------------------------
def exact(case, seed):
    if case["op"] == "select":
        return None                                                              # whole numbers: compared as they are
    d = DIMS[case["dims"]]
    s = prepare(case, seed)
    page, dc, dr = case["page"], d["d_c"], d["d_r"]
    tq, lens = _lengths(case)
    flat = s["cache"].view(-1, dc + dr)
    theta = torch.tensor([ROPE_BASE ** (-2.0 * m / dr) for m in range(dr // 2)], dtype=torch.float64, device=DEVICE)

    def turn(x, pos):
        z = torch.view_as_complex(x.double().reshape(*x.shape[:-1], dr // 2, 2).contiguous())
        w = torch.polar(torch.ones(1, dtype=torch.float64, device=DEVICE), pos[:, None] * theta)
        return torch.view_as_real(z * (w if x.dim() == 2 else w[:, None])).reshape(x.shape)

    def rows_of(b, j):
        return s["table"][b].long()[j // page] * page + j % page

    if case["op"] == "append":
        cache, q, at = flat.double(), torch.empty(s["q_rope"].shape, dtype=torch.float64, device=DEVICE), 0
        scales = torch.zeros(s["cache"].shape[0], 1, dtype=torch.float64, device=DEVICE)
        for b, (t, n) in enumerate(zip(tq, lens)):
            pos = torch.arange(n - t, n, device=DEVICE)
            cache[rows_of(b, pos), :dc] = s["kv"][at:at + t, :dc].double()
            cache[rows_of(b, pos), dc:] = turn(s["kv"][at:at + t, dc:], pos.double())
            q[at:at + t] = turn(s["q_rope"][at:at + t], pos.double())
            whole = s["table"][b, (n - t) // page:n // page].long()
            if whole.numel():
                scales[whole] = cache.view(-1, page, dc + dr)[whole].to(d["dtype"]).double().mean(1).abs().amax(-1, keepdim=True) / 127
            at += t
        return {"cache": cache.view(s["cache"].shape), "q": q, "codes": None, "scales": scales}
    o = torch.zeros(s["T"], d["n_h"], dc, dtype=torch.float64, device=DEVICE)
    lse = torch.zeros(s["T"], d["n_h"], dtype=torch.float64, device=DEVICE)
    at = 0
    for b, (t, n) in enumerate(zip(tq, lens)):
        every = flat[rows_of(b, torch.arange(n, device=DEVICE))].double() if case["op"] == "attn" else None
        for k in range(t):
            p = n - t + k
            if case["op"] == "attn":
                keys = every[:p + 1]
            else:
                g = s["blocks"][at + k].long()
                j = (g[g >= 0][:, None] * page + torch.arange(page, device=DEVICE)).flatten()
                keys = flat[rows_of(b, j[j <= p])].double()
            q = torch.cat([s["q_abs"][at + k], s["q_rope"][at + k]], -1).double()
            score = q @ keys.T / (d["d_h"] + dr) ** 0.5
            lse[at + k] = torch.logsumexp(score, -1)
            o[at + k] = torch.softmax(score, -1) @ keys[:, :dc]
        at += t
    return [o, lse]
