"""The paged-cache operators, as cases to measure: appending latent rows to a paged cache with the
position rotation applied on the way, and the attention of one new token per sequence over that
cache, dense (every entry) or sparse (selected entries).

A latent row is key and value for all query heads: keys use all d_k dims, values the first d_v.
The cache is a pool of pages [n_pages, page, d_k]; entry e of sequence b is row e % page of page
table[b, e // page].  Page 0 of the pools made here belongs to no sequence.

``own = False`` computes each operator in elementary torch operations, ``own = True`` calls the
framework.  A case is a dict of plain values:

  op       "append", "dense" or "sparse"
  dtype    "bf16" or "f32" (storage; both sides compute in 32 bits or more)
  B, H     sequences and query heads;  dk, dv  row and value widths
  page     rows per page;  cap  entries per sequence that the table has room for
  append:  T rows (T == B: one new token per sequence), pad of them padding, dr rotated dims,
           pairs "near" (2i, 2i+1) or "far" (i, i + dr/2), stride = tokens per entry
  dense:   low = smallest length as a share of cap (0: some sequences are empty), W window rows
  sparse:  k selected entries, W window rows, empty = share of unused index slots
"""
import math

import torch

own = False

F32 = {"f32": torch.float32, "bf16": torch.bfloat16}


def _append(name, dtype, T, B, H, dk, dr, page, cap, pad, pairs, stride):
    return dict(name=name, op="append", dtype=dtype, T=T, B=B, H=H, dk=dk, dv=dk, dr=dr, page=page, cap=cap, pad=pad,
                pairs=pairs, stride=stride)


def _dense(name, dtype, B, H, dk, dv, page, cap, low, W):
    return dict(name=name, op="dense", dtype=dtype, B=B, H=H, dk=dk, dv=dv, page=page, cap=cap, low=low, W=W)


def _sparse(name, dtype, B, H, dk, dv, page, cap, k, W, empty):
    return dict(name=name, op="sparse", dtype=dtype, B=B, H=H, dk=dk, dv=dv, page=page, cap=cap, k=k, W=W, empty=empty)


def listed():
    return [
        # one user's next token: the latency of a call
        _append("append one token", "bf16", 1, 1, 128, 576, 64, 64, 4096, 0, "near", 128),
        # the decode step of a full serving batch, a few slots of it unused
        _append("append decode batch", "bf16", 96, 96, 128, 576, 64, 64, 4096, 5, "near", 4),
        # a prefill chunk of three prompts, padded to its bucket
        _append("append prefill chunk", "bf16", 4096, 3, 128, 576, 64, 64, 4096, 97, "near", 1),
        # single precision, the other pairing, small pages: a small model or a check run
        _append("append f32 small", "f32", 301, 7, 4, 64, 32, 16, 160, 3, "far", 1),
        # a short prompt's decode: the latency of a call
        _dense("dense one short", "bf16", 1, 128, 576, 512, 64, 100, 0.5, 0),
        # one-million-token contexts compressed 128x, with the raw window
        _dense("dense 1m compressed", "bf16", 4, 128, 576, 512, 64, 8192, 1.0, 128),
        # a serving batch with ragged contexts, empty slots among them
        _dense("dense ragged batch", "bf16", 32, 128, 576, 512, 32, 16384, 0.0, 0),
        # two very long uncompressed contexts, 64 heads
        _dense("dense 64 heads long", "bf16", 2, 64, 576, 512, 64, 131072, 0.9, 0),
        # single precision, pages that no tile size divides
        _dense("dense f32 small", "f32", 5, 4, 64, 64, 24, 3001, 0.0, 16),
        # 64K-token contexts compressed 4x, top-512 entries and the raw window
        _sparse("sparse 64k top-512", "bf16", 16, 128, 576, 512, 64, 16384, 512, 128, 0.0),
        # a larger batch, top-1024, small pages
        _sparse("sparse batch top-1024", "bf16", 48, 128, 576, 512, 16, 16384, 1024, 128, 0.0),
        # a young context: fewer eligible entries than index slots, odd pages
        _sparse("sparse f32 young", "f32", 2, 4, 64, 64, 7, 600, 77, 16, 0.3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "dense", "dense", "sparse"])
    small = rng.random() < 0.25
    dtype = rng.choice(["f32", "f32", "bf16"]) if small else "bf16"
    dk, dv, dr = (64, 64, 32) if small else (576, 512, 64)
    page = rng.choice([1, 7, 16, 24, 32, 48, 64, 64, 100, 128, 256])
    H = _log(rng, 1, 16) if small else rng.choice([128, 128, 64, _log(rng, 1, 128)])
    W = rng.choice([0, 16, 128, rng.randint(1, 200)])
    if op == "append":
        T = _log(rng, 1, 4096)
        B = T if T <= 256 and rng.random() < 0.6 else rng.randint(1, min(T, 9))
        per = -(-T // B)
        return {k: v for k, v in _append("", dtype, T, B, H, dk, dr, page, per + _log(rng, 1, 512), rng.randint(0, T // 8),
                                         rng.choice(["near", "far"]), rng.choice([1, 4, 128])).items() if k != "name"}
    if op == "dense":
        B = _log(rng, 1, 48)
        cap = _log(rng, 1, min(131072, 240000 // B) if not small else 4000)
        low = rng.choice([0.0, 0.0, 0.3, 1.0])
        return {k: v for k, v in _dense("", dtype, B, H, dk, dv, page, cap, low, W).items() if k != "name"}
    B = _log(rng, 1, 48)
    cap = _log(rng, 8, 16384 if not small else 2000)
    k = min(_log(rng, 1, 1500), cap) if not small else min(_log(rng, 1, 200), cap)
    return {k_: v for k_, v in _sparse("", dtype, B, H, dk, dv, page, cap, k, W, rng.choice([0.0, 0.0, 0.2])).items() if k_ != "name"}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"
    c, dt = case, F32[case["dtype"]]
    B, H, dk, page, cap = c["B"], c["H"], c["dk"], c["page"], c["cap"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev).mul_(std).to(dt)

    def ints(lo, hi, *shape):            # lo .. hi - 1
        return torch.randint(lo, hi, shape, generator=g, device=dev, dtype=torch.int32)

    width = -(-cap // page)
    n_pages = B * width + 1
    pages = torch.empty(n_pages, page, dk, device=dev, dtype=dt)
    for i in range(0, n_pages, 4096):    # a bounded fp32 temporary
        pages[i:i + 4096] = normal(min(4096, n_pages - i), page, dk)
    order = torch.randperm(n_pages - 1, generator=g, device=dev)
    table = (order + 1).reshape(B, width).to(torch.int32)
    s = {"case": c, "pages": pages, "table": table}

    if c["op"] == "append":
        T, dr = c["T"], c["dr"]
        if T == B:                                    # one new token per sequence
            seq = torch.arange(B, device=dev, dtype=torch.int32)
            entry = ints(0, cap, B)
        else:                                         # a run of new tokens per sequence
            per = -(-T // B)
            t = torch.arange(T, device=dev)
            seq = (t // per).to(torch.int32)
            entry = (ints(0, cap - per + 1, B)[seq.long()] + (t % per)).to(torch.int32)
        if c["pad"]:
            entry[T - c["pad"]:] = -1                 # padding rows of the bucket
        s["seq"], s["entry"] = seq, entry
        # the entry's first token; far positions are those of long contexts
        s["pos"] = (entry.clamp(min=0) * c["stride"] + ints(0, 400000, B)[seq.long()]).to(torch.int32)
        s["inv_freq"] = 10000.0 ** (-torch.arange(0, dr, 2, device=dev, dtype=torch.float32) / dr)
        s["rows"] = normal(T, dk)
        s["q_pe"] = normal(T, H, dr)
        s["q"] = normal(T, H, dk) if T * H <= 65536 else normal(1, 1, dk).expand(T, H, dk).contiguous()
        return s

    s["q"] = normal(B, H, dk, std=2.0)
    s["sink"] = torch.randn(H, generator=g, device=dev)
    s["scale"] = dk ** -0.5
    W = c["W"]
    s["win"] = normal(B, W, dk) if W else None
    s["win_len"] = ints(W // 2, W + 1, B) if W else None
    if c["op"] == "dense":
        lo = int(c["low"] * cap)
        n = ints(lo, cap + 1, B)
        if c["low"] == 0.0 and B > 2:
            n[1] = 0                                  # an empty slot of the batch
        s["n"] = n
    else:
        # ascending distinct entries, the unused slots (-1) behind them
        k = c["k"]
        keys = torch.rand(B, cap, generator=g, device=dev)
        idx = keys.topk(k, dim=1).indices.sort(dim=1).values.to(torch.int32)
        used = k - int(c["empty"] * k)
        idx[:, used:] = -1
        s["idx"] = idx.contiguous()
    s["out"] = torch.empty(B, H, c["dv"], device=dev, dtype=dt)
    s["lse"] = torch.empty(B, H, device=dev, dtype=torch.float32)
    return s


# ---------------------------------------------------------------- plain forms

def _rotate_plain(x, pos, inv_freq, pairs):
    """x [T, ..., dr] fp32, pos [T]: each pair turned by pos * inv_freq (angles in 64 bits)."""
    ang = pos.double()[:, None] * inv_freq.double()
    shape = (x.shape[0],) + (1,) * (x.dim() - 2) + (ang.shape[1],)
    cos, sin = ang.cos().float().reshape(shape), ang.sin().float().reshape(shape)
    if pairs == "near":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    a, b = x.chunk(2, dim=-1)
    return torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)


def _append_plain(s):
    c, pages, page, dr = s["case"], s["pages"], s["case"]["page"], s["case"]["dr"]
    flat = pages.view(-1, c["dk"])
    used = s["entry"] >= 0
    e = s["entry"].clamp(min=0).long()
    slot = s["table"][s["seq"].long(), e // page].long() * page + e % page
    slot = torch.where(used, slot, torch.zeros_like(slot))       # row 0 belongs to no sequence
    x = s["rows"].float()
    x = torch.cat((x[:, :-dr], _rotate_plain(x[:, -dr:], s["pos"], s["inv_freq"], c["pairs"])), dim=1)
    flat[slot] = torch.where(used[:, None], x.to(flat.dtype), flat[0])
    turned = _rotate_plain(s["q_pe"].float(), s["pos"], s["inv_freq"], c["pairs"]).to(s["q"].dtype)
    s["q"][..., -dr:] = torch.where(used[:, None, None], turned, s["q"][..., -dr:])
    return {"pages": pages, "q": s["q"]}


def _attend_plain(s):
    c, page = s["case"], s["case"]["page"]
    B, dk, dv = c["B"], c["dk"], c["dv"]
    if c["op"] == "dense":
        e = torch.arange(c["cap"], device="cuda").expand(B, -1)
        ok = e < s["n"][:, None]
    else:
        e = s["idx"].long()
        ok = e >= 0
        e = e.clamp(min=0)
    slot = s["table"].long().gather(1, e // page) * page + e % page
    rows = s["pages"].view(-1, dk)[slot].float()                 # [B, N, dk]
    if s["win"] is not None:
        ok = torch.cat((ok, torch.arange(c["W"], device="cuda") < s["win_len"][:, None]), dim=1)
        rows = torch.cat((rows, s["win"].float()), dim=1)
    rows = rows.masked_fill_(~ok[..., None], 0.0)
    logits = torch.matmul(s["q"].float(), rows.transpose(1, 2)).mul_(s["scale"])
    logits = logits.masked_fill_(~ok[:, None, :], -math.inf)
    sink = s["sink"][None, :]
    top = torch.maximum(logits.amax(dim=-1), sink)
    p = logits.sub_(top[..., None]).exp_()
    den = p.sum(dim=-1) + torch.exp(sink - top)
    out = torch.matmul(p, rows[..., :dv]) / den[..., None]
    return {"out": out.to(s["out"].dtype), "lse": top + torch.log(den)}


# ---------------------------------------------------------------- the framework's calls

def _run_own(s):
    import compressed_sparse_long_csa_b200 as csa
    c = s["case"]
    if c["op"] == "append":
        csa.latent_append_paged(s["rows"], s["entry"], s["pages"], s["table"], seq=s["seq"], pos=s["pos"],
                                inv_freq=s["inv_freq"], interleaved=c["pairs"] == "near", q_pe=s["q_pe"], q=s["q"])
        return {"pages": s["pages"], "q": s["q"]}
    if "ws" not in s:                                            # the program's workspace, kept between steps
        rows = (s["table"].shape[1] * c["page"] if c["op"] == "dense" else c["k"]) + c["W"]
        s["ws"] = torch.empty(max(1, csa.attn_decode_paged_workspace_size(c["B"], c["H"], c["dv"], rows)),
                              dtype=torch.uint8, device="cuda")
    if c["op"] == "dense":
        csa.hca_attn_decode_paged(s["q"], s["pages"], s["table"], s["n"], s["win"], s["win_len"], s["sink"], s["scale"],
                                  c["dv"], s["out"], s["lse"], s["ws"])
    else:
        csa.sparse_attn_decode_paged(s["q"], s["pages"], s["table"], s["idx"], s["win"], s["win_len"], s["sink"],
                                     s["scale"], c["dv"], s["out"], s["lse"], s["ws"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _run_own(state)
    return _append_plain(state) if state["case"]["op"] == "append" else _attend_plain(state)


# ---------------------------------------------------------------- what a pass cannot do without

def _mean_rows(case):
    """Expected attended rows per sequence."""
    w = 0.75 * case["W"]
    if case["op"] == "sparse":
        return case["k"] - int(case["empty"] * case["k"]) + w
    n = 0.5 * (case["low"] + 1.0) * case["cap"]
    if case["low"] == 0.0 and case["B"] > 2:
        n *= (case["B"] - 1) / case["B"]
    return n + w


def work(case):
    c, es = case, 4 if case["dtype"] == "f32" else 2
    if c["op"] == "append":
        rows = c["T"] - c["pad"]
        per_row = 2 * c["dk"] * es + 2 * c["H"] * c["dr"] * es + 16
        # a turned pair: two products and a sum for each of its two values
        return {"bytes": rows * per_row + c["T"] * 4, "flops": rows * (c["H"] + 1) * c["dr"] * 3}
    n = c["B"] * _mean_rows(c)
    per_seq = c["H"] * (c["dk"] + c["dv"]) * es + c["H"] * 4
    idx = 4 * c["B"] * (c["k"] if c["op"] == "sparse" else -(-c["cap"] // c["page"]))
    return {"bytes": n * c["dk"] * es + c["B"] * per_seq + idx, "flops": 2 * n * c["H"] * (c["dk"] + c["dv"])}


# ---------------------------------------------------------------- the definition, in 64 bits

def _exact_append(c, s):
    pages, q = s["pages"].double(), s["q"].double()
    used = (s["entry"] >= 0).nonzero()[:, 0]
    half = c["dr"] // 2
    first = torch.arange(half, device="cuda")
    lo, hi = (2 * first, 2 * first + 1) if c["pairs"] == "near" else (first, first + half)
    # e^{i * angle} times the pair read as a complex number
    turn = torch.polar(torch.ones(len(used), half, dtype=torch.float64, device="cuda"),
                       s["pos"][used].double()[:, None] * s["inv_freq"].double())
    base = c["dk"] - c["dr"]
    x = s["rows"][used].double()
    z = torch.complex(x[:, base + lo], x[:, base + hi]) * turn
    x[:, base + lo], x[:, base + hi] = z.real, z.imag
    e = s["entry"][used].long()
    where = s["table"][s["seq"][used].long(), torch.div(e, c["page"], rounding_mode="floor")].long()
    pages[where, e % c["page"]] = x
    y = s["q_pe"][used].double()
    z = torch.complex(y[..., lo], y[..., hi]) * turn[:, None, :]
    turned = torch.empty_like(y)
    turned[..., lo], turned[..., hi] = z.real, z.imag
    q[used, :, base:] = turned
    return {"pages": pages, "q": q}


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "append":
        return _exact_append(c, s)
    outs, lses = [], []
    for b in range(c["B"]):
        ids = torch.arange(int(s["n"][b]), device="cuda") if c["op"] == "dense" else s["idx"][b][s["idx"][b] >= 0].long()
        row = s["pages"][s["table"][b].long()[ids // c["page"]], ids % c["page"]].double()
        if s["win"] is not None:
            row = torch.cat((row, s["win"][b, :int(s["win_len"][b])].double()))
        score = s["q"][b].double() @ row.T * s["scale"]
        # the sink: one more logit whose value is the zero vector
        score = torch.cat((score, s["sink"].double()[:, None]), dim=1)
        lse = torch.logsumexp(score, dim=1)
        outs.append(torch.exp(score[:, :-1] - lse[:, None]) @ row[:, :c["dv"]])
        lses.append(lse)
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
