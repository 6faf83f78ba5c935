"""turbo4 on the GPU against the 64-bit reference (turbo4_ref): codec bit for bit, attention
within the bound that its docstring derives."""
import numpy as np
import pytest

import turbo4_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import rotated_bit_kv_tq_gb300 as m
    from rotated_bit_kv_tq_gb300 import build
    build.build()
    torch.cuda.set_device(0)
    for t in (m.TQ_TURBO2, m.TQ_TURBO3, m.TQ_TURBO4):
        m.codebook_init(t, 0)
    return m


def rng(*seed):
    return np.random.default_rng(list(seed))


def kv16(r, n, hkv, d, outliers=False):
    x = r.standard_normal((n, hkv, d)).astype(np.float32)
    if outliers:
        g = np.exp(0.5 * r.standard_normal((hkv, d))).astype(np.float32)
        g[:, r.permutation(d)[:4]] *= 10
        x *= g
    return x.astype(np.float16)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def sign_bits(r, on):
    return r.integers(0, 2, 128) if on else None


def make_cache(tq, kind, hkv, d, rows_by_seq, page=0, signs=None, r=None, cols=None):
    """A cache holding the given packed rows of every sequence; pages in shuffled order."""
    S = len(rows_by_seq)
    rb = tq.row_bytes(kind, hkv, d)
    sg = None if signs is None else [int(b) for b in signs]
    if not page:
        cap = max(1, max(len(x) for x in rows_by_seq))
        pool = np.full((S, cap, rb), 0xA5, np.uint8)
        for s, x in enumerate(rows_by_seq):
            pool[s, : len(x)] = x
        return tq.KVCache(kind, hkv, d, n_seqs=S, capacity_tokens=cap, buffer=dev(pool.reshape(-1)), rotation_signs=sg)
    cols = cols or max(1, max(-(-len(x) // page) for x in rows_by_seq))
    n_pages = S * cols + 2
    ids = r.permutation(n_pages)[: S * cols].reshape(S, cols).astype(np.int32)
    pool = np.full((n_pages, page, rb), 0xA5, np.uint8)
    for s, x in enumerate(rows_by_seq):
        for i in range(0, len(x), page):
            part = x[i:i + page]
            pool[ids[s, i // page], : len(part)] = part
    c = tq.KVCache(kind, hkv, d, n_seqs=S, page_tokens=page, page_table=dev(ids), n_pages=n_pages,
                   buffer=dev(pool.reshape(-1)), rotation_signs=sg)
    return c


# ------------------------------------------------------------------ codec
@pytest.mark.parametrize("n,hkv,d", [(1, 1, 128), (3, 2, 128), (7, 3, 128), (41, 8, 128), (130, 4, 256),
                                     (700, 8, 128), (1500, 3, 128), (4200, 1, 128), (33, 5, 256)])
@pytest.mark.parametrize("signs,correct", [(False, False), (True, True)])
def test_encode_bits_and_decode(tq, n, hkv, d, signs, correct):
    r = rng(1, n, hkv, d, signs)
    blocks = hkv * d // 128
    x = kv16(r, n, hkv, d, outliers=True).reshape(n, -1)
    edge = min(n, 6)
    x[:edge, :128] = np.array([0.0, 65504.0, -65504.0, 6e-8, -0.0, 1.0], np.float16)[:edge, None]
    sg = sign_bits(r, signs)
    cache = tq.KVCache(tq.TQ_TURBO4, hkv, d, capacity_tokens=n + 9,
                       rotation_signs=None if sg is None else [int(b) for b in sg], norm_correction=correct)
    cache.buffer.fill_(0x5A)
    tq.encode(cache, dev(x), pos0=4)
    out = torch.full((n + 9, hkv, d), 7.0, device=DEV)
    tq.decode(cache, 0, 4, n, out[4:])
    torch.cuda.synchronize()
    assert tq.device_status() == 0
    rows = cache.buffer.cpu().numpy().reshape(n + 9, -1)
    want = ref.encode_rows(x, blocks, sg, correct)
    assert np.array_equal(rows[4:4 + n], want)
    assert (rows[:4] == 0x5A).all() and (rows[4 + n:] == 0x5A).all()     # other rows untouched
    got = out[4:4 + n].cpu().numpy().reshape(n, blocks, 128).astype(np.float64)
    exact = ref.dequant(want, blocks, sg)
    norms = ref.unpack(want, blocks)[1]
    # 7 butterfly levels of fp32 sums of |c| <= 0.24 (128 of them: at most 2.72 |norm| after
    # the 1/sqrt(128)) and three more roundings: 10 half-steps
    assert (np.abs(got - exact) <= 10 * 2.0 ** -24 * 2.72 * np.abs(norms)[..., None] + 1e-45).all()
    assert (out[:4] == 7).all() and (out[4 + n:] == 7).all()


@pytest.mark.parametrize("hkv,off", [(8, 4), (3, 4), (8, 0)])
def test_decode_offset_output_and_missing_rows(tq, hkv, off):
    """An output on an odd 16-byte boundary; rows past the capacity read as zeros and are reported."""
    r = rng(6, hkv, off)
    n, over = 37, 5
    x = kv16(r, n, hkv, 128).reshape(n, -1)
    cache = tq.KVCache(tq.TQ_TURBO4, hkv, 128, capacity_tokens=n)
    tq.encode(cache, dev(x))
    flat = torch.full((off + (n - 2 + over) * hkv * 128 + 8,), 7.0, device=DEV)
    out = flat[off:off + (n - 2 + over) * hkv * 128].view(-1, hkv, 128)
    tq.decode(cache, 0, 2, n - 2 + over, out)
    torch.cuda.synchronize()
    assert tq.device_status() == 7
    rows = ref.encode_rows(x, hkv)
    got = out.cpu().numpy().astype(np.float64)
    norms = ref.unpack(rows, hkv)[1][2:]
    assert (np.abs(got[: n - 2] - ref.dequant(rows, hkv)[2:]) <= 10 * 2.0 ** -24 * 2.72 * norms[..., None]).all()
    assert (got[n - 2:] == 0).all()
    assert (flat[:off] == 7).all() and (flat[off + (n - 2 + over) * hkv * 128:] == 7).all()


@pytest.mark.parametrize("n", [5, 900])
def test_encode_kv_scattered_strided_paged(tq, n):
    """K and V of one call, token rows wider than the heads, positions in random order over
    shuffled pages; out-of-range rows are reported and leave the pool alone."""
    r = rng(2, n)
    hkv, d, page, S = 8, 128, 64, 3
    cols = -(-n // page) + 1
    wide = kv16(r, n, 2 * hkv, d).reshape(n, -1)
    caches, tables = [], []
    for _ in range(2):
        t = r.permutation(S * cols).reshape(S, cols).astype(np.int32)
        tables.append(t)
        c = tq.KVCache(tq.TQ_TURBO4, hkv, d, n_seqs=S, page_tokens=page, page_table=dev(t), n_pages=S * cols)
        c.buffer.fill_(0x33)
        caches.append(c)
    pos = r.permutation(cols * page)[:n].astype(np.int32)
    seq = r.integers(0, S, n).astype(np.int32)
    pos[-1] = cols * page                     # one row past the last page
    src = dev(wide)
    tq.encode_kv(*caches, src[:, : hkv * d], src[:, hkv * d:], seq_ids=dev(seq), positions=dev(pos))
    torch.cuda.synchronize()
    assert tq.device_status() == 7
    for i, (c, t) in enumerate(zip(caches, tables)):
        want = np.full((S * cols, page, 528), 0x33, np.uint8)
        rows = ref.encode_rows(wide[:, i * hkv * d:(i + 1) * hkv * d], hkv)
        for j in range(n - 1):
            want[t[seq[j], pos[j] // page], pos[j] % page] = rows[j]
        assert np.array_equal(c.buffer.cpu().numpy().reshape(want.shape), want)


# ------------------------------------------------------------------ attention
def check(got, want, bound, f16):
    got = got.cpu().numpy().astype(np.float64)
    err = np.linalg.norm(got - want, axis=-1)
    assert np.isfinite(got).all()
    assert (err <= bound + 1e-30).all(), (float((err / np.maximum(bound, 1e-30)).max()))


SHAPES = [(8, 32, 128), (8, 40, 128), (4, 16, 256), (8, 8, 128), (8, 64, 128), (4, 16, 128), (2, 8, 128),
          (3, 6, 128), (1, 4, 128), (16, 32, 128), (2, 12, 256), (4, 28, 128), (1, 1, 256), (8, 48, 128)]


@pytest.mark.parametrize("hkv,hq,d", SHAPES)
@pytest.mark.parametrize("lens,page", [((1,), 0), ((31,), 32), ((33,), 0), ((700,), 0), ((1301,), 64),
                                       ((0, 5, 64, 300), 0), ((129, 0, 1, 65, 512, 33), 32)])
@pytest.mark.parametrize("append", [False, True])
def test_decode_attention(tq, hkv, hq, d, lens, page, append):
    r = rng(3, hkv, hq, d, len(lens), page, append)
    signs = (hq + page) % 3 == 1
    sk, sv = sign_bits(r, signs), sign_bits(r, signs)
    f16 = (hq // hkv) % 2 == 0
    blocks = hkv * d // 128
    S = len(lens)
    ks = [ref.encode_rows(kv16(r, L, hkv, d, True).reshape(L, hkv * d), blocks, sk) for L in lens]
    vs = [ref.encode_rows(kv16(r, L, hkv, d).reshape(L, hkv * d), blocks, sv) for L in lens]
    kc = make_cache(tq, tq.TQ_TURBO4, hkv, d, ks, page, sk, r)
    vc = make_cache(tq, tq.TQ_TURBO4, hkv, d, vs, page, sv, r)
    q = r.standard_normal((S, hq, d)).astype(np.float16)
    most = max(lens)
    out = torch.full((S, hq, d), 9.0, dtype=torch.float16 if f16 else torch.float32, device=DEV)
    ws = torch.empty(max(16, tq.attn_workspace_bytes(S, hq, d, most)), dtype=torch.uint8, device=DEV)
    ws.random_(0, 256)
    lens_d = dev(np.array(lens, np.int32))
    if append:
        kn, vn = kv16(r, S, hkv, d, True), kv16(r, S, hkv, d)
        before = [c.buffer.clone() for c in (kc, vc)]
        tq.attn_decode_append(kc, vc, dev(kn), dev(vn), dev(q), lens_d, most, out, ws)
        for s, L in enumerate(lens):
            if L:
                ks[s][L - 1] = ref.encode_rows(kn[s].reshape(1, -1), blocks, sk)
                vs[s][L - 1] = ref.encode_rows(vn[s].reshape(1, -1), blocks, sv)
        for c, b, rows in ((kc, before[0], ks), (vc, before[1], vs)):
            want = b.cpu().numpy().reshape(-1, blocks * 66).copy()
            table = c.page_table.cpu().numpy() if page else None
            for s, L in enumerate(lens):
                if L:
                    at = table[s, (L - 1) // page] * page + (L - 1) % page if page else s * max(1, most) + L - 1
                    want[at] = rows[s][L - 1]
            assert np.array_equal(c.buffer.cpu().numpy().reshape(want.shape), want)
    else:
        tq.attn_decode(kc, vc, dev(q), lens_d, most, out, ws)
    torch.cuda.synchronize()
    assert tq.device_status() == 0
    scale = 1 / np.sqrt(d)
    for s, L in enumerate(lens):
        see = np.ones((1, L), bool)
        want = ref.attention(ref.dequant(ks[s], blocks, sk), ref.dequant(vs[s], blocks, sv), q[s:s + 1], see, scale, hkv)
        bound = ref.attention_bound(ks[s], vs[s], q[s:s + 1], see, scale, hkv, f16, False, sk)
        check(out[s:s + 1], want, bound, f16)


@pytest.mark.parametrize("tk,tv", [(36, 3), (36, 2), (3, 36), (2, 36)])
@pytest.mark.parametrize("hkv,hq,d", [(8, 32, 128), (8, 40, 128), (4, 16, 256), (3, 6, 128)])
def test_mixed_types(tq, tk, tv, hkv, hq, d):
    """A turbo4 cache beside one of the other types: decode step and prompt chunk against a
    dense product with the library's own dequantised rows, within the library's bar of 2e-3
    per head vector (the other types' levels are rounded operands)."""
    r = rng(4, tk, tv, hkv, hq)
    n, nq = 333, 21
    kc = tq.KVCache(tk, hkv, d, capacity_tokens=n)
    vc = tq.KVCache(tv, hkv, d, capacity_tokens=n)
    tq.encode_kv(kc, vc, dev(kv16(r, n, hkv, d, True).reshape(n, -1)), dev(kv16(r, n, hkv, d).reshape(n, -1)))
    kd, vd = (torch.empty(n, hkv, d, device=DEV) for _ in range(2))
    tq.decode(kc, 0, 0, n, kd)
    tq.decode(vc, 0, 0, n, vd)
    q = r.standard_normal((nq, hq, d)).astype(np.float16)
    out = torch.empty(nq, hq, d, device=DEV)
    tq.attn_prefill(kc, vc, dev(q), out, pos0=n - nq)
    one = torch.empty(1, hq, d, device=DEV)
    ws = torch.empty(tq.attn_workspace_bytes(1, hq, d, n), dtype=torch.uint8, device=DEV)
    tq.attn_decode(kc, vc, dev(q[-1:]), dev(np.array([n], np.int32)), n, one, ws)
    torch.cuda.synchronize()
    assert tq.device_status() == 0
    see = np.arange(n)[None] <= (n - nq + np.arange(nq))[:, None]
    blocks = hkv * d // 128
    want = ref.attention(kd.cpu().numpy().astype(np.float64).reshape(n, blocks, 128),
                         vd.cpu().numpy().astype(np.float64).reshape(n, blocks, 128), q, see, 1 / np.sqrt(d), hkv)
    for got, w in ((out, want), (one, want[-1:])):
        g = got.cpu().numpy().astype(np.float64)
        assert (np.linalg.norm(g - w, axis=-1) < 2e-3 * np.linalg.norm(w, axis=-1)).all()


@pytest.mark.parametrize("hkv,hq,d", [(8, 32, 128), (8, 40, 128), (4, 16, 256), (8, 8, 128), (3, 6, 128),
                                      (2, 16, 128), (1, 5, 256)])
@pytest.mark.parametrize("pos0,nq,page", [(0, 1, 0), (0, 33, 32), (126, 3, 0), (127, 130, 64), (700, 49, 0),
                                          (1, 300, 256)])
def test_prompt_chunk(tq, hkv, hq, d, pos0, nq, page):
    r = rng(5, hkv, hq, d, pos0, nq)
    signs = nq % 2 == 1
    sk, sv = sign_bits(r, signs), sign_bits(r, signs)
    f16 = pos0 % 2 == 0
    blocks, n = hkv * d // 128, pos0 + nq
    ks = ref.encode_rows(kv16(r, n, hkv, d, True).reshape(n, -1), blocks, sk)
    vs = ref.encode_rows(kv16(r, n, hkv, d).reshape(n, -1), blocks, sv)
    other = np.full((5, blocks * 66), 0xFF, np.uint8)
    kc = make_cache(tq, tq.TQ_TURBO4, hkv, d, [other, ks], page, sk, r)
    vc = make_cache(tq, tq.TQ_TURBO4, hkv, d, [other, vs], page, sv, r)
    q = r.standard_normal((nq, hq, d)).astype(np.float16)
    out = torch.full((nq + 1, hq, d), 9.0, dtype=torch.float16 if f16 else torch.float32, device=DEV)
    tq.attn_prefill(kc, vc, dev(q), out[:nq], pos0=pos0, seq_id=1)
    torch.cuda.synchronize()
    assert tq.device_status() == 0
    assert (out[nq] == 9).all()
    see = np.arange(n)[None] <= (pos0 + np.arange(nq))[:, None]
    scale = 1 / np.sqrt(d)
    want = ref.attention(ref.dequant(ks, blocks, sk), ref.dequant(vs, blocks, sv), q, see, scale, hkv)
    bound = ref.attention_bound(ks, vs, q, see, scale, hkv, f16, True, sk)
    check(out[:nq], want, bound, f16)
