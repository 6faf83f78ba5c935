"""Measured cases of the 4-bit cache (turbo4) and of the cache's page operations.

Every case names one operator and the sizes of one call of it:

  codec    token rows written into 4-bit K and V caches and read back as fp32 rows
  attend   single-token attention over 4-bit caches, one step of a decoder's layer;
           with "append", the step's new token is written first
  chunk    causal attention of a prompt chunk over 4-bit caches
  fork     sequences of a paged cache dropped and forked again from their parents: pages
           shared by count, the last, partly filled page of each parent copied
  compact  the pages in use moved to the lowest page numbers, tables and counts renumbered

With ``own`` false, run() computes them in their plain form: elementary torch operations
in fp32.  With ``own`` true it makes the library's calls on the same inputs.

The 4-bit block (128 values): norm = fp16(min(|x|, 65504)); y = W x / (sqrt(128) |x|) with W
the 128-point Walsh-Hadamard matrix in natural order; every y becomes the nearer of 16
levels +-LEVELS[m], a value on a border going to the level nearer zero.  A token's row holds
the codes of all its blocks, 64 bytes each, then their norms, 2 bytes each.
"""
import math

import torch

own = False

DEV = "cuda"
B = 128                                    # values of a block
STEP = 2619.0 / 131072.0 / 16.0            # the levels are whole multiples of this
MAGS = (9, 26, 44, 64, 88, 112, 144, 192)
INV_SQRT_B = float.fromhex("0x1.6a09e6p-4")     # the fp32 value nearest to 1 / sqrt(128)

LLAMA = {"hkv": 8, "hq": 32, "d": 128}     # the shape of an 8B model with 8 KV heads
QWEN = {"hkv": 8, "hq": 40, "d": 128}      # the shape of a 14B model, five queries per KV head
HD256 = {"hkv": 4, "hq": 16, "d": 256}     # head_dim 256
TINY = {"hkv": 2, "hq": 8, "d": 128}       # rows that are no multiple of 16 bytes


def listed():
    return [
        # one token of each of 37 running sequences written to scattered positions
        {"name": "codec-append-37", "op": "codec", "n": 37, "hkv": 8, "d": 128, "signs": True,
         "correct": False, "scatter": True},
        # the prompt of one layer: K and V rows of 32,768 tokens
        {"name": "codec-prompt-32k", "op": "codec", "n": 32768, "hkv": 8, "d": 128,
         "signs": False, "correct": False, "scatter": False},
        # a short chat turn of a small model: one sequence, 257 positions
        {"name": "attend-tiny-257", "op": "attend", "seqs": 1, "lo": 257, "hi": 257, "page": 0,
         "append": False, "signs": False, **TINY},
        # one decode step of a layer at the benchmark's context
        {"name": "attend-step-32k", "op": "attend", "seqs": 1, "lo": 32768, "hi": 32768,
         "page": 0, "append": True, "signs": False, **LLAMA},
        # one long sequence, head_dim 256
        {"name": "attend-hd256-128k", "op": "attend", "seqs": 1, "lo": 131072, "hi": 131072,
         "page": 0, "append": False, "signs": False, **HD256},
        # a serving batch on a paged cache: ragged lengths, one of them empty
        {"name": "attend-paged-33", "op": "attend", "seqs": 33, "lo": 0, "hi": 8191,
         "page": 256, "append": True, "signs": True, **QWEN},
        # the last, short chunk of a prompt
        {"name": "chunk-49-at-1000", "op": "chunk", "nq": 49, "pos0": 1000, "page": 32,
         "signs": True, **QWEN},
        # a full prompt chunk in the middle of a long prompt
        {"name": "chunk-1024-at-15k", "op": "chunk", "nq": 1024, "pos0": 15360, "page": 0,
         "signs": False, **LLAMA},
        # four continuations of one prompt, one layer
        {"name": "fork-4", "op": "fork", "caches": 2, "page": 256, "parents": 1, "per": 4,
         "lo": 700, "hi": 701, "hkv": 8, "d": 128},
        # a beam step of a batch over all layers of a 32-layer model
        {"name": "fork-48", "op": "fork", "caches": 64, "page": 256, "parents": 12, "per": 4,
         "lo": 500, "hi": 1900, "hkv": 8, "d": 128},
        # a small pool after a few sequences ended, one layer
        {"name": "compact-61", "op": "compact", "caches": 2, "page": 64, "pages": 61,
         "used": 0.5, "hkv": 8, "d": 128},
        # a large pool of eight layers, a third of it holes
        {"name": "compact-509", "op": "compact", "caches": 16, "page": 256, "pages": 509,
         "used": 0.66, "hkv": 8, "d": 128},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["codec", "attend", "attend", "chunk", "fork", "compact"])
    shape = rng.choice([LLAMA, QWEN, HD256, {"hkv": 4, "hq": 16, "d": 128},
                        {"hkv": 8, "hq": 8, "d": 128}, {"hkv": 3, "hq": 6, "d": 128},
                        {"hkv": 2, "hq": 16, "d": 128}])
    if op == "codec":
        return {"op": op, "n": _log(rng, 1, 32000), "hkv": rng.choice([1, 2, 3, 5, 8]), "d": 128,
                "signs": rng.random() < 0.5, "correct": rng.random() < 0.5,
                "scatter": rng.random() < 0.5}
    if op == "attend":
        if rng.random() < 0.5:
            n = _log(rng, 1, 131000)
            return {"op": op, "seqs": 1, "lo": n, "hi": n, "page": rng.choice([0, 0, 32, 256]),
                    "append": rng.random() < 0.5, "signs": rng.random() < 0.5, **shape}
        hi = _log(rng, 40, 8000)
        return {"op": op, "seqs": rng.randint(2, 32), "lo": rng.choice([0, 1, hi // 8]), "hi": hi,
                "page": rng.choice([0, 32, 64, 256]), "append": rng.random() < 0.5,
                "signs": rng.random() < 0.5, **shape}
    if op == "chunk":
        nq = _log(rng, 1, 1000)
        return {"op": op, "nq": nq, "pos0": _log(rng, 1, 15000) - 1, "page": rng.choice([0, 32, 256]),
                "signs": rng.random() < 0.5, **shape}
    if op == "fork":
        lo = _log(rng, 1, 900)
        return {"op": op, "caches": rng.choice([1, 2, 8, 32]), "page": rng.choice([32, 64, 256]),
                "parents": rng.randint(1, 12), "per": rng.randint(1, 5), "lo": lo,
                "hi": lo + _log(rng, 1, 900), "hkv": rng.choice([1, 2, 4, 8]), "d": 128}
    return {"op": op, "caches": rng.choice([1, 2, 8, 12]), "page": rng.choice([32, 64, 256]),
            "pages": _log(rng, 3, 500), "used": rng.uniform(0.05, 0.95),
            "hkv": rng.choice([1, 2, 4, 8]), "d": 128}


# ------------------------------------------------------------------ the plain form
def _tree_sum(x):
    """Sum over the last axis (128): element i with element i + half, level by level."""
    while x.shape[-1] > 1:
        h = x.shape[-1] // 2
        x = x[..., :h] + x[..., h:]
    return x[..., 0]


def _butterflies(x):
    """W x over the last axis (128), natural order, stages 1, 2, 4 .. 64."""
    shape, h = x.shape, 1
    while h < B:
        x = x.reshape(-1, B // (2 * h), 2, h)
        x = torch.stack((x[:, :, 0] + x[:, :, 1], x[:, :, 0] - x[:, :, 1]), 2)
        h *= 2
    return x.reshape(shape)


def _levels(device):
    return torch.tensor([m * STEP for m in MAGS], dtype=torch.float32, device=device)


def _encode_plain(x16, signs, correct):
    """fp16 [..., 128] -> (magnitude indexes, sign bits, fp16 norms); every fp32 operation
    in the order that the format fixes, so that the codes are the same bits."""
    x = x16.float() * signs
    n = torch.sqrt(_tree_sum(x * x))
    k = torch.where(n > 0, torch.div(torch.full_like(n, INV_SQRT_B), n), torch.zeros_like(n))
    y = _butterflies(x) * k[..., None]
    lev = _levels(x.device)
    border = (lev[1:] + lev[:-1]) * 0.5
    mag = torch.bucketize(y.abs(), border)          # borders strictly below |y|
    if correct:
        c = lev[mag]
        n = n / torch.sqrt(_tree_sum(c * c))
    return mag, torch.signbit(y), torch.clamp(n, max=65504.0).half()


def _pack(mag, neg, norm):
    """[tokens, blocks, 128] codes -> uint8 rows [tokens, blocks * 66]."""
    t, nb = mag.shape[:2]
    m = mag.reshape(t, nb, 16, 8).int()
    s = neg.reshape(t, nb, 16, 2, 4).int()
    k = torch.arange(8, device=mag.device, dtype=torch.int32)
    j = torch.arange(4, device=mag.device, dtype=torch.int32)
    w = (m.long() << (4 * k)).sum(-1)
    w += (s[..., 0, :].long() << (8 * j + 7)).sum(-1) + (s[..., 1, :].long() << (8 * j + 3)).sum(-1)
    byte = torch.arange(4, device=mag.device) * 8
    codes = ((w[..., None] >> byte) & 255).to(torch.uint8).reshape(t, nb * 64)
    return torch.cat((codes, norm.contiguous().view(torch.uint8).reshape(t, nb * 2)), 1)


def _unpack(rows, nb):
    """uint8 rows [..., nb * 66] -> (fp32 levels [..., nb, 128], fp32 norms [..., nb])."""
    lead = rows.shape[:-1]
    b = rows[..., : nb * 64].reshape(*lead, nb, 16, 4).long()
    w = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16) | (b[..., 3] << 24)
    k = torch.arange(8, device=rows.device)
    at = torch.cat((8 * k[:4] + 7, 8 * k[:4] + 3))
    mag = (w[..., None] >> (4 * k)) & 7
    neg = (w[..., None] >> at) & 1
    c = _levels(rows.device)[mag] * (1 - 2 * neg).float()
    norm = rows[..., nb * 64:].contiguous().view(torch.float16).float()
    return c.reshape(*lead, nb, B), norm.reshape(*lead, nb)


def _dequant(rows, nb, signs):
    c, norm = _unpack(rows, nb)
    return _butterflies(c) * (norm * INV_SQRT_B)[..., None] * signs


def _sign_row(signs):
    return 1.0 if signs is None else signs


def _gather(pool, table, page, n):
    """Rows 0 .. n-1 of every sequence of a cache: [seqs, n, row_bytes]."""
    if not page:
        return pool[:, :n]
    t = table.long()[:, : (n + page - 1) // page]
    return pool[t].reshape(t.shape[0], -1, pool.shape[-1])[:, :n]


def _attend_plain(q, krows, vrows, hkv, d, keep, sk, sv):
    """softmax(q K^T / sqrt(d)) V in the rotated domain.  q fp16 [S, nq, hq, d]; rows
    [S, T, bytes]; keep [S, nq, T] true where a query sees a key.  fp16 [S, nq, hq, d]."""
    S, nq, hq = q.shape[:3]
    nb, G, T = d // B, hq // hkv, krows.shape[1]
    qr = _butterflies((q.float().reshape(S, nq, hq, nb, B) * sk)) * INV_SQRT_B
    kc, kn = _unpack(krows, hkv * nb)
    kc = (kc * kn[..., None]).reshape(S, T, hkv, d)
    qr = qr.reshape(S, nq, hkv, G, d).permute(0, 2, 3, 1, 4).reshape(S, hkv, G * nq, d)
    s = torch.matmul(qr, kc.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(d))
    s = s.reshape(S, hkv, G, nq, T)
    see = keep[:, None, None]
    s = torch.where(see, s, torch.full_like(s, -math.inf))
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    vc, vn = _unpack(vrows, hkv * nb)
    vc = (vc * vn[..., None]).reshape(S, T, hkv, d).permute(0, 2, 1, 3)
    o = torch.matmul(p.reshape(S, hkv, G * nq, T), vc).reshape(S, hkv, G, nq, nb, B)
    o = _butterflies(o) * INV_SQRT_B * sv
    o = o.reshape(S, hkv, G, nq, d) / torch.where(total > 0, total, torch.ones_like(total))
    return o.permute(0, 3, 1, 2, 4).reshape(S, nq, hq, d).half()


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _kv(g, n, hkv, d, outliers):
    """fp16 [n, hkv, d] as attention layers make them: normal values; for keys every channel
    with a gain of its own and four channels of each head ten times larger."""
    x = torch.randn(n, hkv, d, generator=g, device=DEV)
    if outliers:
        gain = torch.exp(0.5 * torch.randn(hkv, d, generator=g, device=DEV))
        gain[:, torch.randperm(d, generator=g, device=DEV)[:4]] *= 10.0
        x = x * gain
    return x.half()


def _sign_bits(g, on):
    if not on:
        return None, None
    bits = torch.randint(0, 2, (B,), generator=g, device=DEV)
    return 1.0 - 2.0 * bits.float(), bits


def _rows(x16, signs):
    """The packed rows of fp16 [n, hkv, d] tokens, made 8,192 tokens at a time."""
    out = []
    for part in x16.split(8192):
        mag, neg, norm = _encode_plain(part.reshape(part.shape[0], -1, B), _sign_row(signs), False)
        out.append(_pack(mag, neg, norm))
    return torch.cat(out)


def _handles(st, case, pools):
    """The library's cache objects over the same bytes (what a program makes once)."""
    import rotated_bit_kv_tq_gb300 as tq
    tq.codebook_init(tq.TQ_TURBO4, torch.cuda.current_device())
    made = []
    for pool, bits in pools:
        sg = None if bits is None else bits.tolist()
        kw = dict(buffer=pool.reshape(-1), rotation_signs=sg,
                  norm_correction=bool(case.get("correct", False)))
        if case.get("page"):
            made.append(tq.KVCache(tq.TQ_TURBO4, case["hkv"], case["d"], n_seqs=st["table"].shape[0],
                                   page_tokens=case["page"], page_table=st["table"],
                                   n_pages=pool.shape[0], **kw))
        else:
            made.append(tq.KVCache(tq.TQ_TURBO4, case["hkv"], case["d"], n_seqs=pool.shape[0],
                                   capacity_tokens=pool.shape[1], **kw))
    st["tq"] = tq
    st["caches"] = made
    return tq


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": case, "table": None}
    if op == "codec":
        n, hkv, d = case["n"], case["hkv"], case["d"]
        cap = n + 5
        st["x"] = [_kv(g, n, hkv, d, k) for k in (True, False)]
        st["sg"], bits = zip(*[_sign_bits(g, case["signs"]) for _ in range(2)])
        st["pos0"] = 3
        st["pos"] = torch.randperm(cap, generator=g, device=DEV)[:n].int() if case["scatter"] else None
        st["pool"] = [torch.zeros(1, cap, hkv * (d // B) * 66, dtype=torch.uint8, device=DEV) for _ in range(2)]
        if own:
            _handles(st, case, list(zip(st["pool"], bits)))
            st["out"] = [torch.empty(cap, hkv, d, device=DEV) for _ in range(2)]
        return st
    if op in ("attend", "chunk"):
        hkv, hq, d, page = case["hkv"], case["hq"], case["d"], case["page"]
        if op == "attend":
            S = case["seqs"]
            lens = torch.randint(case["lo"], case["hi"] + 1, (S,), generator=g, device=DEV, dtype=torch.int32)
            if S > 1:
                lens[-1], lens[0] = case["lo"], case["hi"]
            most = case["hi"]
            st["q"] = torch.randn(S, hq, d, generator=g, device=DEV).half()
        else:
            S, most = 1, case["pos0"] + case["nq"]
            lens = torch.full((1,), most, device=DEV, dtype=torch.int32)
            st["q"] = torch.randn(case["nq"], hq, d, generator=g, device=DEV).half()
        st["lens"], st["most"] = lens, most
        st["sg"], bits = zip(*[_sign_bits(g, case["signs"]) for _ in range(2)])
        if page:
            cols = (most + page - 1) // page
            st["table"] = torch.randperm(S * cols, generator=g, device=DEV).int().reshape(S, cols)
        st["pool"] = []
        for kind in range(2):
            cap = (most + page - 1) // page * page if page else most
            r = _rows(_kv(g, S * cap, hkv, d, kind == 0), st["sg"][kind])
            if page:
                pool = torch.empty(S * cols, page, r.shape[1], dtype=torch.uint8, device=DEV)
                pool[st["table"].long().reshape(-1)] = r.reshape(S * cols, page, -1)
                st["pool"].append(pool)
            else:
                st["pool"].append(r.reshape(S, cap, -1))
        if op == "attend" and case["append"]:
            st["new"] = [_kv(g, S, hkv, d, k) for k in (True, False)]
        if own:
            tq = _handles(st, case, list(zip(st["pool"], bits)))
            st["out"] = torch.empty(st["q"].shape, dtype=torch.float16, device=DEV)
            if op == "attend":
                st["ws"] = torch.empty(max(16, tq.attn_workspace_bytes(S, hq, d, most)), dtype=torch.uint8, device=DEV)
        return st
    page, row = case["page"], case["hkv"] * (case["d"] // B) * 66
    if op == "fork":
        P, per = case["parents"], case["per"]
        lens = torch.randint(case["lo"], case["hi"], (P,), generator=g, device=DEV, dtype=torch.int32)
        cols = (case["hi"] + page - 1) // page
        n_pages = P * cols + P * per + 3
        S = P * (1 + per)
        table = torch.full((S, cols), -1, dtype=torch.int32, device=DEV)
        perm = torch.randperm(n_pages, generator=g, device=DEV).int()
        have = (lens + page - 1) // page
        held = torch.arange(cols, device=DEV)[None] < have[:, None]
        table[:P] = torch.where(held, perm[: P * cols].reshape(P, cols), table[:P])
        st["parents"] = torch.arange(P, device=DEV, dtype=torch.int32).repeat_interleave(per)
        st["children"] = P + torch.randperm(P * per, generator=g, device=DEV).int()
        seq_lens = torch.zeros(S, dtype=torch.int32, device=DEV)
        seq_lens[:P] = lens
        refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
        refs[table[table >= 0].long()] = 1
    else:
        n_pages = case["pages"]
        count = min(n_pages, max(1, round(n_pages * case["used"])))
        ids = torch.randperm(n_pages, generator=g, device=DEV)[:count]
        cols = max(2, math.isqrt(count))
        S = -(-count // cols) + 1
        table = torch.full((S * cols,), -1, dtype=torch.int32, device=DEV)
        table[: ids.numel()] = ids.int()
        table = table.reshape(S, cols)
        table[S - 1] = table[0]                 # the last sequence shares the first one's pages
        refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
        held = table[table >= 0].long()
        refs.index_add_(0, held, torch.ones_like(held, dtype=torch.int32))
        seq_lens = (table >= 0).sum(1).int() * page
    st["table"], st["lens"], st["refs"] = table, seq_lens, refs
    bits = torch.randint(-2 ** 31, 2 ** 31, (case["caches"], n_pages, page * row // 4), generator=g,
                         device=DEV, dtype=torch.int32)
    st["bits"] = bits
    st["pool"] = bits.view(torch.uint8).reshape(case["caches"], n_pages, page, row)
    if own:
        import rotated_bit_kv_tq_gb300 as tq
        _handles(st, case, [(p, None) for p in st["pool"]])
        st["group"] = tq.CacheGroup(st["caches"])
        st["pages"] = tq.PagePool(n_pages, page, S, cols, device=DEV, page_table=table,
                                  seq_lens=seq_lens, refcounts=refs)
        if op == "compact":
            st["after"] = tq.PagePool(n_pages, page, S, cols, device=DEV)
    return st


# ------------------------------------------------------------------ one pass
def _run_own(st):
    tq, case = st["tq"], st["case"]
    if case["op"] == "codec":
        kc, vc = st["caches"]
        n = case["n"]
        if case["scatter"]:
            tq.encode_kv(kc, vc, st["x"][0].reshape(n, -1), st["x"][1].reshape(n, -1), positions=st["pos"])
        else:
            tq.encode_kv(kc, vc, st["x"][0].reshape(n, -1), st["x"][1].reshape(n, -1), pos0=st["pos0"])
        tq.decode(kc, 0, 0, n + 5, st["out"][0])
        tq.decode(vc, 0, 0, n + 5, st["out"][1])
        return st["out"]
    if case["op"] == "attend":
        kc, vc = st["caches"]
        if case["append"]:
            tq.attn_decode_append(kc, vc, st["new"][0], st["new"][1], st["q"], st["lens"], st["most"],
                                  st["out"], st["ws"])
            return [st["out"], *st["pool"]]      # the caches with the new rows in them
        else:
            tq.attn_decode(kc, vc, st["q"], st["lens"], st["most"], st["out"], st["ws"])
            return st["out"]
    if case["op"] == "chunk":
        kc, vc = st["caches"]
        tq.attn_prefill(kc, vc, st["q"], st["out"], pos0=case["pos0"])
        return st["out"]
    if case["op"] == "fork":
        pool = st["pages"]
        tq.pages_free(pool, st["children"])
        tq.pages_fork(pool, st["group"], st["parents"], st["children"])
        return [pool.page_table, pool.seq_lens, pool.refcounts, st["bits"]]
    after = st["after"]
    tq.pages_compact(st["pages"], st["group"], out=after)
    return [after.page_table, after.seq_lens, after.refcounts, st["bits"]]


def run(st):
    if own:
        return _run_own(st)
    case, op = st["case"], st["case"]["op"]
    if op == "codec":
        n, nb = case["n"], case["hkv"] * (case["d"] // B)
        at = st["pos"].long() if case["scatter"] else slice(st["pos0"], st["pos0"] + n)

        def both(x, pool, sg):
            mag, neg, norm = _encode_plain(x.reshape(n, nb, B), sg, case["correct"])
            pool[0, at] = _pack(mag, neg, norm)
            return _dequant(pool[0], nb, sg).reshape(n + 5, case["hkv"], case["d"])

        return [both(st["x"][0], st["pool"][0], _sign_row(st["sg"][0])),
                both(st["x"][1], st["pool"][1], _sign_row(st["sg"][1]))]
    if op in ("attend", "chunk"):
        hkv, d, page, n = case["hkv"], case["d"], case["page"], st["most"]
        sk, sv = (_sign_row(s) for s in st["sg"])
        lens = st["lens"].long()
        T = torch.arange(n, device=DEV)
        if op == "attend" and case["append"]:
            S = lens.numel()
            live = torch.nonzero(lens > 0)[:, 0]
            last = lens[live] - 1
            at = (st["table"].long()[live, last // page], last % page) if page else (live, last)

            def write(x, pool, sg):
                mag, neg, norm = _encode_plain(x.reshape(S, -1, B), sg, False)
                pool[at] = _pack(mag, neg, norm)[live]

            write(st["new"][0], st["pool"][0], sk)
            write(st["new"][1], st["pool"][1], sv)
        krows, vrows = (_gather(p, st["table"], page, n) for p in st["pool"])
        if op == "attend":
            keep = (T[None] < lens[:, None])[:, None]
            o = _attend_plain(st["q"][:, None], krows, vrows, hkv, d, keep, sk, sv)[:, 0]
            return [o, *st["pool"]] if case["append"] else o
        keep = (T[None] <= (case["pos0"] + torch.arange(case["nq"], device=DEV))[:, None])[None]
        return _attend_plain(st["q"][None], krows, vrows, hkv, d, keep, sk, sv)[0]
    table, lens, refs, page = st["table"], st["lens"], st["refs"], case["page"]
    pool = st["pool"].reshape(case["caches"], refs.numel(), -1)       # bytes of a page
    if op == "fork":
        par, ch = st["parents"].long(), st["children"].long()
        row = pool.shape[-1] // page
        old = table[ch]
        gone = old[old >= 0].long()
        refs.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
        table[ch] = -1
        lens[ch] = 0
        rows = lens[par].long() % page
        part = rows > 0
        free = torch.nonzero(refs == 0)[:, 0]
        fresh = free[: int(part.sum())]
        whole = lens[par].long() // page
        copy = table[par]
        held = torch.arange(table.shape[1], device=DEV)[None] < whole[:, None]
        kept = torch.where(held, copy, torch.full_like(copy, -1))
        kept[part, whole[part]] = fresh.int()
        table[ch] = kept
        lens[ch] = lens[par]
        shared = copy[held].long()
        refs.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
        refs[fresh] = 1
        src = copy[part, whole[part]].long()
        mine = torch.arange(page * row, device=DEV)[None] < (rows[part] * row)[:, None]
        pool[:, fresh] = torch.where(mine[None], pool[:, src], pool[:, fresh])
        return [table, lens, refs, st["bits"]]
    used = refs > 0
    count = int(used.sum())
    holes = torch.nonzero(~used[:count])[:, 0]
    movers = torch.nonzero(used[count:])[:, 0] + count
    new = torch.arange(refs.numel(), device=DEV)
    new[movers] = holes
    after = torch.where(table >= 0, new[table.clamp(min=0).long()].int(), table)
    counts = torch.zeros_like(refs)
    counts[new[used]] = refs[used]
    pool[:, holes] = pool[:, movers]
    return [after, lens.clone(), counts, st["bits"]]


# ------------------------------------------------------------------ what a pass needs
def _lens_mean(case):
    return case["hi"] if case["seqs"] == 1 else 0.5 * (case["lo"] + case["hi"])


def work(case):
    op = case["op"]
    row = case["hkv"] * (case["d"] // B) * 66
    if op == "codec":
        n, vals = case["n"], case["hkv"] * case["d"]
        back = (n + 5) * (row + 4 * vals)        # rows read back whole
        return {"bytes": 2 * (n * (2 * vals + row) + back), "flops": 2 * 2 * (2 * n + 5) * vals * 8}
    if op == "attend":
        toks = case["seqs"] * _lens_mean(case)
        qo = 4 * case["seqs"] * case["hq"] * case["d"]
        new = 2 * case["seqs"] * (2 * case["hkv"] * case["d"] + row) if case["append"] else 0
        return {"bytes": 2 * toks * row + qo + new, "flops": 4 * case["hq"] * case["d"] * toks}
    if op == "chunk":
        nq, pos0 = case["nq"], case["pos0"]
        pairs = nq * pos0 + nq * (nq + 1) // 2
        return {"bytes": 2 * (pos0 + nq) * row + 4 * nq * case["hq"] * case["d"],
                "flops": 4 * case["hq"] * case["d"] * pairs}
    page_bytes = case["page"] * row
    if op == "fork":
        lo, hi, page = case["lo"], case["hi"], case["page"]
        part = sum(n % page for n in range(lo, hi)) / (hi - lo)
        n = case["parents"] * case["per"]
        cols = (hi + page - 1) // page
        return {"bytes": 2 * case["caches"] * n * part * row + 3 * 4 * n * cols, "flops": 0}
    p, u = case["pages"], case["used"]
    return {"bytes": 2 * case["caches"] * page_bytes * max(0.5, p * u * (1 - u)) + 4 * 4 * p, "flops": 0}


# ------------------------------------------------------------------ the definition in 64 bits
def _hadamard():
    h = torch.ones(1, 1, dtype=torch.float64, device=DEV)
    pair = torch.tensor([[1.0, 1.0], [1.0, -1.0]], dtype=torch.float64, device=DEV)
    for _ in range(7):
        h = torch.kron(h, pair)
    return h


def _f32(x):
    return x.to(torch.float32).to(torch.float64)


def _exact_codes(x16, signs, correct):
    """Levels (as whole multiples of STEP) and norms of fp16 [n, 128] blocks.  The format
    fixes the fp32 rounding of every sum, so that writers agree on each code: here each
    64-bit operation is rounded to fp32 where the format says so."""
    x = x16.double() * signs
    q = _f32(x * x)
    for half in (64, 32, 16, 8, 4, 2, 1):
        q = _f32(q[:, :half] + q[:, half:2 * half])
    n = _f32(torch.sqrt(q[:, 0]))
    k = torch.where(n > 0, _f32(INV_SQRT_B / n.clamp(min=1e-300)), torch.zeros_like(n))
    z = x
    for bit in range(7):
        idx = torch.arange(B, device=x.device)
        up = (idx >> bit) & 1
        other = z[:, idx ^ (1 << bit)]
        z = _f32(torch.where(up.bool(), other - z, z + other))
    y = _f32(z * k[:, None])
    lev = torch.full_like(y, MAGS[0])
    for a, b in zip(MAGS[:-1], MAGS[1:]):
        lev = torch.where(y.abs() > (a + b) * 0.5 * STEP, torch.full_like(y, b), lev)
    if correct:
        c = _f32(_f32(lev * STEP) ** 2)
        for half in (64, 32, 16, 8, 4, 2, 1):
            c = _f32(c[:, :half] + c[:, half:2 * half])
        n = _f32(n / _f32(torch.sqrt(c[:, 0])))
    neg = (z < 0) | ((z == 0) & torch.signbit(z * k[:, None]))
    return torch.where(neg, -lev, lev), n.clamp(max=65504.0).to(torch.float16).double()


def _exact_rows(rows, nb):
    """uint8 rows [n, nb * 66] -> 64-bit values in the rotated domain [n, nb, 128]."""
    n = rows.shape[0]
    byte = rows[:, : nb * 64].reshape(n, nb, 16, 4)
    low, high = (byte & 15).double(), (byte >> 4).double()
    nib = torch.stack((low, high), -1).reshape(n, nb, 16, 8)       # nibble k: bits 4k .. 4k+3
    top = (nib >= 8)
    idx = (nib - 8.0 * top).long()
    order = torch.tensor([1, 3, 5, 7, 0, 2, 4, 6], device=rows.device)   # sign of value k
    sign = 1.0 - 2.0 * top[..., order].double()
    lev = torch.tensor(MAGS, dtype=torch.float64, device=rows.device)[idx] * sign * STEP
    raw = rows[:, nb * 64:].reshape(n, nb, 2).long()
    bits = raw[..., 0] | (raw[..., 1] << 8)
    norm = torch.where(bits >= 32768, bits - 65536, bits).to(torch.int16).view(torch.float16).double()
    return lev.reshape(n, nb, B) * norm[..., None]


def exact(case, seed):
    global own
    if case["op"] in ("fork", "compact"):
        return None
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    H = _hadamard() / math.sqrt(B)
    hkv, d = case["hkv"], case["d"]
    nb = d // B
    sg = [torch.ones(B, dtype=torch.float64, device=DEV) if s is None else s.double() for s in st["sg"]]
    if case["op"] == "codec":
        out = []
        for x, s in zip(st["x"], sg):
            n = case["n"]
            o = torch.zeros(n + 5, hkv * nb, B, dtype=torch.float64, device=DEV)
            back = []
            for part in x.reshape(n, hkv * nb, B).split(4096):
                lev, norm = _exact_codes(part.reshape(-1, B), s, case["correct"])
                back.append(((lev * STEP * norm[:, None]) @ H * s).reshape(-1, hkv * nb, B))
            back = torch.cat(back)
            if case["scatter"]:
                o[st["pos"].long()] = back
            else:
                o[st["pos0"]: st["pos0"] + n] = back
            out.append(o.reshape(n + 5, hkv, d))
        return out
    hq, page = case["hq"], case["page"]
    G = hq // hkv
    lens = st["lens"].tolist()
    outs = []
    for s_i, L in enumerate(lens):
        def rows_of(pool):
            if not page:
                return pool[s_i, :L]
            ids = st["table"][s_i, : (L + page - 1) // page].long()
            return pool[ids].reshape(-1, pool.shape[-1])[:L]
        q = st["q"][s_i: s_i + 1] if case["op"] == "attend" else st["q"]
        o = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
        if L:
            kv = [_exact_rows(rows_of(p), hkv * nb) for p in st["pool"]]
            if case.get("append"):
                for r, x, s in zip(kv, st["new"], sg):
                    lev, norm = _exact_codes(x[s_i].reshape(-1, B), s, False)
                    r[L - 1] = lev * STEP * norm[:, None]
            k, v = (((r @ H) * s).reshape(L, hkv, d) for r, s in zip(kv, sg))
            first = L - q.shape[0] + 1
            see = torch.arange(L, device=DEV)[None] < (first + torch.arange(q.shape[0], device=DEV))[:, None]
            for h in range(hq):
                t = q[:, h].double() @ k[:, h // G].T / math.sqrt(d)
                p = torch.softmax(t.masked_fill(~see, -math.inf), -1)
                o[:, h] = p @ v[:, h // G]
        outs.append(o)
    return [torch.cat(outs), None, None] if case.get("append") else torch.cat(outs)
