"""turbo4 attention as programs use it: one workspace for calls of every shape, captured graphs,
streams, rows that are missing, masked or far into a pool, and a run of the operators together."""
import ctypes

import numpy as np
import pytest
import torch

import turbo4_ref as ref
from test_gpu_turbo4 import DEV, check, dev, kv16, make_cache, rng, sign_bits, tq  # noqa: F401

pytestmark = pytest.mark.gpu


def caches(tq, r, lens, hkv, d, page=0):
    blocks = hkv * d // 128
    ks = [ref.encode_rows(kv16(r, L, hkv, d, True).reshape(L, hkv * d), blocks, None) for L in lens]
    vs = [ref.encode_rows(kv16(r, L, hkv, d).reshape(L, hkv * d), blocks, None) for L in lens]
    return (make_cache(tq, tq.TQ_TURBO4, hkv, d, ks, page, None, r), make_cache(tq, tq.TQ_TURBO4, hkv, d, vs, page, None, r),
            ks, vs)


def expect(got, ks, vs, q, hkv, see=None, f16=False, v_rounded=False):
    """got, q: [n, hq, d] of one sequence whose rows are ks, vs."""
    n, d = q.shape[0], q.shape[2]
    blocks, scale = hkv * d // 128, 1 / np.sqrt(d)
    see = np.ones((n, len(ks)), bool) if see is None else see
    want = ref.attention(ref.dequant(ks, blocks), ref.dequant(vs, blocks), q, see, scale, hkv)
    check(got, want, ref.attention_bound(ks, vs, q, see, scale, hkv, f16, v_rounded, None), f16)


def test_one_workspace_for_every_shape(tq):
    """Calls that merge in their own grid and calls with a merge kernel, of changing sizes, in one
    workspace that starts as noise; each is checked."""
    r = rng(21)
    calls = (((700,), 8, 32, 128), ((33, 900, 1), 8, 32, 128), ((5000,), 8, 32, 128), ((12,), 4, 16, 256),
             ((64, 0, 3000, 2, 2, 2, 2), 2, 8, 128), ((1,), 8, 40, 128), ((700,), 8, 32, 128))
    ws = torch.empty(max(tq.attn_workspace_bytes(len(c[0]), c[2], c[3], max(c[0])) for c in calls), dtype=torch.uint8,
                     device=DEV).random_(0, 256)
    for lens, hkv, hq, d in calls:
        kc, vc, ks, vs = caches(tq, r, lens, hkv, d)
        q = r.standard_normal((len(lens), hq, d)).astype(np.float16)
        out = torch.empty(len(lens), hq, d, device=DEV)
        for _ in range(2):
            tq.attn_decode(kc, vc, dev(q), dev(np.array(lens, np.int32)), max(lens), out, ws)
        assert tq.device_status() == 0
        for s in range(len(lens)):
            expect(out[s:s + 1], ks[s], vs[s], q[s:s + 1], hkv)


@pytest.mark.parametrize("lens", [(40,), (40, 0, 7)])
def test_captured_steps_that_share_a_workspace(tq, lens):
    """Two captured steps over two pairs of caches, one workspace, replayed in turn while the lengths
    in device memory grow: every replay appends its row and attends to it."""
    r = rng(22, len(lens))
    S, hkv, hq, d, room = len(lens), 8, 32, 128, 64
    full = [room] * S
    sets = [caches(tq, r, full, hkv, d) for _ in range(2)]
    ws = torch.empty(tq.attn_workspace_bytes(S, hq, d, room), dtype=torch.uint8, device=DEV).random_(0, 256)
    lens_d = [dev(np.array(lens, np.int32)) for _ in sets]
    new = [[torch.zeros(S, hkv, d, dtype=torch.float16, device=DEV) for _ in range(2)] for _ in sets]
    q = [torch.zeros(S, hq, d, dtype=torch.float16, device=DEV) for _ in sets]
    out = [torch.empty(S, hq, d, device=DEV) for _ in sets]

    def step(i):
        tq.attn_decode_append(sets[i][0], sets[i][1], new[i][0], new[i][1], q[i], lens_d[i], room, out[i], ws)

    graphs = []
    keep = [(c[0].buffer.clone(), c[1].buffer.clone()) for c in sets]
    for i in range(2):
        step(i)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(i)
        graphs.append(g)
    for c, b in zip(sets, keep):
        c[0].buffer.copy_(b[0])
        c[1].buffer.copy_(b[1])
    now = np.array(lens)
    for t in range(6):
        now = np.where(now > 0, now + 1, 0) if t else now
        for i in (0, 1) if t % 2 else (1, 0):
            kn, vn, qn = kv16(r, S, hkv, d, True), kv16(r, S, hkv, d), r.standard_normal((S, hq, d)).astype(np.float16)
            new[i][0].copy_(dev(kn))
            new[i][1].copy_(dev(vn))
            q[i].copy_(dev(qn))
            lens_d[i].copy_(dev(now.astype(np.int32)))
            graphs[i].replay()
            ks, vs = sets[i][2], sets[i][3]
            for s in range(S):
                if now[s]:
                    ks[s][now[s] - 1] = ref.encode_rows(kn[s].reshape(1, -1), hkv, None)
                    vs[s][now[s] - 1] = ref.encode_rows(vn[s].reshape(1, -1), hkv, None)
                expect(out[i][s:s + 1], ks[s][:now[s]], vs[s][:now[s]], qn[s:s + 1], hkv)
    assert tq.device_status() == 0


def test_two_streams_with_a_workspace_each(tq):
    r = rng(23)
    hkv, hq, d, n = 8, 32, 128, 3000
    kc, vc, ks, vs = caches(tq, r, (n,), hkv, d)
    q = [r.standard_normal((1, hq, d)).astype(np.float16) for _ in range(2)]
    lens = dev(np.array([n], np.int32))
    ws = [torch.empty(tq.attn_workspace_bytes(1, hq, d, n), dtype=torch.uint8, device=DEV).random_(0, 256) for _ in range(2)]
    out = [torch.empty(1, hq, d, device=DEV) for _ in range(2)]
    qd = [dev(x) for x in q]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                tq.attn_decode(kc, vc, qd[i], lens, n, out[i], ws[i])
    torch.cuda.synchronize()
    assert tq.device_status() == 0
    for i in range(2):
        expect(out[i], ks[0], vs[0], q[i], hkv)


def test_lengths_past_the_bound(tq):
    """Lengths beyond max_seq_len count as max_seq_len, negative ones as 0; both are reported."""
    r = rng(24)
    hkv, hq, d = 8, 32, 128
    kc, vc, ks, vs = caches(tq, r, (80, 80, 80), hkv, d)
    q = r.standard_normal((3, hq, d)).astype(np.float16)
    out = torch.empty(3, hq, d, device=DEV)
    ws = torch.empty(tq.attn_workspace_bytes(3, hq, d, 50), dtype=torch.uint8, device=DEV).random_(0, 256)
    tq.attn_decode(kc, vc, dev(q), dev(np.array([60, -3, 20], np.int32)), 50, out, ws)
    assert tq.device_status() == 7
    for s, n in enumerate((50, 0, 20)):
        expect(out[s:s + 1], ks[s][:n], vs[s][:n], q[s:s + 1], hkv)
    tq.attn_decode(kc, vc, dev(q), dev(np.array([60, 3, 20], np.int32)), 0, out, ws)
    assert tq.device_status() == 7
    assert (out == 0).all()
    # one sequence: the grid that merges itself
    tq.attn_decode(kc, vc, dev(q[:1]), dev(np.array([60], np.int32)), 50, out[:1], ws)
    assert tq.device_status() == 7
    expect(out[:1], ks[0][:50], vs[0][:50], q[:1], hkv)


@pytest.mark.parametrize("S", [1, 3])
def test_missing_pages_are_masked(tq, S):
    """Page ids outside the pool, in the K table or the V table only: their rows are reported and take
    no part in a decode step."""
    r = rng(25, S)
    hkv, hq, d, n, page = 8, 32, 128, 300, 32
    kc, vc, ks, vs = caches(tq, r, (n,) * S, hkv, d, page)
    kt, vt = kc.page_table.clone(), vc.page_table.clone()
    kt[S - 1, 2], kt[S - 1, 5], vt[S - 1, 7] = -1, 10 ** 6, -7
    kc.page_table.copy_(kt)
    vc.page_table.copy_(vt)
    q = r.standard_normal((S, hq, d)).astype(np.float16)
    out = torch.empty(S, hq, d, device=DEV)
    ws = torch.empty(tq.attn_workspace_bytes(S, hq, d, n), dtype=torch.uint8, device=DEV).random_(0, 256)
    tq.attn_decode(kc, vc, dev(q), dev(np.array([n] * S, np.int32)), n, out, ws)
    assert tq.device_status() == 7
    for s in range(S):
        see = np.ones((1, n), bool)
        if s == S - 1:
            for p in (2, 5, 7):
                see[:, p * page:(p + 1) * page] = False
        expect(out[s:s + 1], ks[s], vs[s], q[s:s + 1], hkv, see)


@pytest.mark.parametrize("bad", [0x7C00, 0x7E00, 0xFC00])
def test_later_rows_that_are_not_finite(tq, bad):
    """Rows behind a query's position, and rows behind a sequence's length, whose norms are infinite or
    no numbers: what does not see them does not depend on them."""
    r = rng(26, bad)
    hkv, hq, d, n, nq = 2, 8, 128, 90, 40
    kc, vc, ks, vs = caches(tq, r, (n,), hkv, d)
    for c in (kc, vc):
        rows = c.buffer.view(n, hkv * 66)
        rows[70:, hkv * 64:].view(torch.int16).copy_(torch.tensor(np.array(bad, np.uint16).view(np.int16).item(), device=DEV))
    q = r.standard_normal((nq, hq, d)).astype(np.float16)
    out = torch.empty(nq, hq, d, device=DEV)
    tq.attn_prefill(kc, vc, dev(q), out, pos0=n - nq)       # queries 0 .. 19 see rows 0 .. 69
    ws = torch.empty(tq.attn_workspace_bytes(1, hq, d, n), dtype=torch.uint8, device=DEV).random_(0, 256)
    one = torch.empty(1, hq, d, device=DEV)
    tq.attn_decode(kc, vc, dev(q[:1]), dev(np.array([70], np.int32)), n, one, ws)
    torch.cuda.synchronize()
    assert tq.device_status() == 0
    see = np.arange(70)[None] <= (n - nq + np.arange(20))[:, None]
    expect(out[:20], ks[0][:70], vs[0][:70], q[:20], hkv, see)
    expect(one, ks[0][:70], vs[0][:70], q[:1], hkv)


@pytest.mark.parametrize("bad", [0x7C00, 0x7E00])
@pytest.mark.parametrize("page", [0, 32])
def test_later_rows_that_are_not_finite_head_dim_256(tq, bad, page):
    r = rng(32, bad, page)
    hkv, hq, d, n, nq = 2, 8, 256, 90, 40
    blocks = hkv * 2
    kc, vc, ks, vs = caches(tq, r, (n,), hkv, d, page)
    for c in (kc, vc):
        rows = c.buffer.view(-1, blocks * 66)
        for t in range(70, n):
            at = int(c.page_table[0, t // page]) * page + t % page if page else t
            rows[at, blocks * 64:].view(torch.int16).copy_(torch.tensor(bad, dtype=torch.int16))
    q = r.standard_normal((nq, hq, d)).astype(np.float16)
    out = torch.empty(nq, hq, d, dtype=torch.float16, device=DEV)
    tq.attn_prefill(kc, vc, dev(q), out, pos0=n - nq)       # queries 0 .. 19 see rows 0 .. 69
    torch.cuda.synchronize()
    assert tq.device_status() == 0
    see = np.arange(70)[None] <= (n - nq + np.arange(20))[:, None]
    expect(out[:20], ks[0][:70], vs[0][:70], q[:20], hkv, see, True)


@pytest.mark.parametrize("power", [-4, 0, 4])
def test_prompt_chunk_value_sizes_head_dim_256(tq, power):
    """One rounding per product at every size of the values (test_prompt_chunk allows two)."""
    r = rng(33, 9 + power)
    hkv, hq, d, n, nq = 2, 8, 256, 200, 30
    blocks = hkv * 2
    ks = ref.encode_rows(kv16(r, n, hkv, d, True).reshape(n, -1), blocks, None)
    vs = ref.encode_rows((kv16(r, n, hkv, d).astype(np.float32) * 10.0 ** power).astype(np.float16).reshape(n, -1), blocks, None)
    kc, vc = (make_cache(tq, tq.TQ_TURBO4, hkv, d, [x]) for x in (ks, vs))
    q = r.standard_normal((nq, hq, d)).astype(np.float16)
    out = torch.empty(nq, hq, d, device=DEV)
    tq.attn_prefill(kc, vc, dev(q), out, pos0=n - nq)
    torch.cuda.synchronize()
    assert tq.device_status() == 0
    expect(out, ks, vs, q, hkv, np.arange(n)[None] <= (n - nq + np.arange(nq))[:, None])


@pytest.mark.parametrize("page", [0, 256])
def test_rows_past_four_gigabytes(tq, page):
    """A sequence whose rows start 4.4 GB into the pool: written, read back, attended to."""
    r = rng(27, page)
    hkv, hq, d, n, nq = 8, 32, 128, 300, 30
    rb = tq.row_bytes(tq.TQ_TURBO4, hkv, d)
    cap = (1 << 23) + 512                                   # 4.43 GB
    x = [kv16(r, n, hkv, d, k).reshape(n, -1) for k in (True, False)]
    want = [ref.encode_rows(a, hkv, None) for a in x]
    pool = torch.empty(2 * cap * rb if not page else (cap + 1024) * rb, dtype=torch.uint8, device=DEV)
    cs = []
    for i in range(2):                                      # K and V share the pool, apart by n rows' worth
        if not page:
            cs.append(tq.KVCache(tq.TQ_TURBO4, hkv, d, n_seqs=2, capacity_tokens=cap, buffer=pool))
        else:
            pages = cap // page
            t = torch.tensor([[0, 0], [pages + 2 * i, pages + 2 * i + 1]], dtype=torch.int32, device=DEV)
            cs.append(tq.KVCache(tq.TQ_TURBO4, hkv, d, n_seqs=2, page_tokens=page, page_table=t, n_pages=pages + 4,
                                 buffer=pool))
    p0 = [0, 0]
    if not page:
        p0 = [cap - n, 0]                                   # K's rows at the end; V's cache is its own pool below
        cs[1] = tq.KVCache(tq.TQ_TURBO4, hkv, d, n_seqs=2, capacity_tokens=n)
    ids = torch.ones(n, dtype=torch.int32, device=DEV)
    for c, a, at, w in zip(cs, x, p0, want):
        tq.encode(c, dev(a), pos0=at, seq_ids=ids)
        start = (cap + at if not page and c is cs[0] else n if not page else int(c.page_table[1, 0]) * page) * rb
        assert np.array_equal(c.buffer[start:start + n * rb].cpu().numpy().reshape(n, rb), w)
        back = torch.empty(n, hkv, d, device=DEV)
        tq.decode(c, 1, at, n, back)
        exact = ref.dequant(w, hkv)
        assert (np.abs(back.cpu().numpy() - exact) <= 10 * 2.0 ** -24 * 2.72 * ref.unpack(w, hkv)[1][..., None]).all()
    assert tq.device_status() == 0
    if page:
        q = r.standard_normal((nq, hq, d)).astype(np.float16)
        out = torch.empty(nq, hq, d, device=DEV)
        tq.attn_prefill(*cs, dev(q), out, pos0=n - nq, seq_id=1)
        expect(out, *want, q, hkv, np.arange(n)[None] <= (n - nq + np.arange(nq))[:, None])
        ws = torch.empty(tq.attn_workspace_bytes(2, hq, d, n), dtype=torch.uint8, device=DEV).random_(0, 256)
        one = torch.empty(2, hq, d, device=DEV)
        tq.attn_decode(*cs, dev(q[:2]), dev(np.array([0, n], np.int32)), n, one, ws)
        assert (one[0] == 0).all()
        expect(one[1:], *want, q[1:2], hkv)
    assert tq.device_status() == 0


@pytest.mark.parametrize("hkv,hq,d", [(8, 32, 128), (3, 6, 128), (4, 16, 256)])
@pytest.mark.parametrize("lens", [(500,), (500, 90)])
def test_injected_wait_timeout(tq, hkv, hq, d, lens):
    """Waits that run out are reported, the context stays usable and the next call is right."""
    r = rng(28, hkv, len(lens))
    kc, vc, ks, vs = caches(tq, r, lens, hkv, d)
    S = len(lens)
    q = r.standard_normal((S, hq, d)).astype(np.float16)
    lens_d = dev(np.array(lens, np.int32))
    ws = torch.empty(tq.attn_workspace_bytes(S, hq, d, max(lens)), dtype=torch.uint8, device=DEV).random_(0, 256)
    out = torch.full((S, hq, d), float("nan"), device=DEV)
    tq.inject_wait_timeout(1)
    tq.attn_decode(kc, vc, dev(q), lens_d, max(lens), out, ws)
    torch.cuda.synchronize()
    assert tq.device_status() == 6
    tq.attn_decode(kc, vc, dev(q), lens_d, max(lens), out, ws)
    torch.cuda.synchronize()
    assert tq.device_status() == 0
    for s in range(S):
        expect(out[s:s + 1], ks[s], vs[s], q[s:s + 1], hkv)


@pytest.mark.parametrize("lens,hkv,hq,d", [((2500,), 8, 32, 128), ((777, 64), 4, 16, 256)])
def test_allocation_free_call(tq, lens, hkv, hq, d):
    r = rng(29, hkv)
    kc, vc, ks, vs = caches(tq, r, lens, hkv, d)
    S = len(lens)
    q = r.standard_normal((S, hq, d)).astype(np.float16)
    qd, lens_d = dev(q), dev(np.array(lens, np.int32))
    out = torch.full((S, hq, d), float("nan"), device=DEV)
    for _ in range(2):
        st = tq.load().tq_attn_decode_noalloc(ctypes.byref(kc.view), ctypes.byref(vc.view), ctypes.c_void_p(qd.data_ptr()),
                                              S, hq, ctypes.c_void_p(lens_d.data_ptr()), max(lens), 0.0,
                                              ctypes.c_void_p(out.data_ptr()),
                                              ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert st in (0, 4)
        if st == 4:                                          # more than its fixed scratch holds
            assert tq.attn_workspace_bytes(S, hq, d, max(lens)) > 0
            return
    torch.cuda.synchronize()
    assert tq.device_status() == 0
    for s in range(S):
        expect(out[s:s + 1], ks[s], vs[s], q[s:s + 1], hkv)


@pytest.mark.parametrize("hkv,hq", [(8, 32), (4, 28), (2, 2)])
def test_short_prompts_over_a_cluster(tq, hkv, hq):
    """Prompt chunks whose query blocks see fewer key tiles than the CTAs that share them."""
    r = rng(30, hkv, hq)
    d = 128
    for pos0, nq in ((0, 150), (100, 60), (500, 1), (380, 140)):
        n = pos0 + nq
        kc, vc, ks, vs = caches(tq, r, (n,), hkv, d)
        q = r.standard_normal((nq, hq, d)).astype(np.float16)
        out = torch.empty(nq, hq, d, dtype=torch.float16, device=DEV)
        tq.attn_prefill(kc, vc, dev(q), out, pos0=pos0)
        torch.cuda.synchronize()
        assert tq.device_status() == 0
        expect(out, ks[0], vs[0], q, hkv, np.arange(n)[None] <= (pos0 + np.arange(nq))[:, None], True, True)


@pytest.mark.parametrize("d,power", [(128, -4), (128, 0), (128, 4), (256, -2), (256, 4)])
def test_prompt_chunk_value_sizes(tq, d, power):
    """Value norms from 1e-3 (head_dim 256: 0.1) to the largest: the outputs keep their relative accuracy."""
    r = rng(31, d, 9 + power)
    scale = 10.0 ** power
    hkv, hq, n, nq = 2, 8, 200, 30
    blocks = hkv * d // 128
    ks = ref.encode_rows(kv16(r, n, hkv, d, True).reshape(n, -1), blocks, None)
    vs = ref.encode_rows((kv16(r, n, hkv, d).astype(np.float32) * scale).astype(np.float16).reshape(n, -1), blocks, None)
    kc, vc = (make_cache(tq, tq.TQ_TURBO4, hkv, d, [x]) for x in (ks, vs))
    q = r.standard_normal((nq, hq, d)).astype(np.float16)
    out = torch.empty(nq, hq, d, device=DEV)
    tq.attn_prefill(kc, vc, dev(q), out, pos0=n - nq)
    torch.cuda.synchronize()
    assert tq.device_status() == 0
    expect(out, ks, vs, q, hkv, np.arange(n)[None] <= (n - nq + np.arange(nq))[:, None], False, d == 256)


@pytest.mark.parametrize("d", [128, 256])
def test_captured_prompt_chunks_and_a_missing_page(tq, d):
    """Two prompt chunks of different lengths captured into one graph and replayed with other queries;
    then a page id outside the pool: reported, and what lies before it is not affected."""
    r = rng(34, d)
    hkv, hq, n, page = 4, 16, 700, 64
    kc, vc, ks, vs = caches(tq, r, (n,), hkv, d, page)
    spans = ((n - 130, 130), (100, 17))
    qd = [torch.zeros(nq, hq, d, dtype=torch.float16, device=DEV) for _, nq in spans]
    out = [torch.empty(nq, hq, d, device=DEV) for _, nq in spans]

    def run():
        for (pos0, _), a, b in zip(spans, qd, out):
            tq.attn_prefill(kc, vc, a, b, pos0=pos0)

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for turn in range(2):
        q = [r.standard_normal((nq, hq, d)).astype(np.float16) for _, nq in spans]
        for a, b in zip(qd, q):
            a.copy_(dev(b))
        if turn:
            kc.page_table[0, 8] = 10 ** 7          # rows 512 .. 575
        g.replay()
        torch.cuda.synchronize()
        assert tq.device_status() == (7 if turn else 0)
        for (pos0, nq), a, b in list(zip(spans, q, out))[turn:]:
            m = pos0 + nq
            expect(b, ks[0][:m], vs[0][:m], a, hkv, np.arange(m)[None] <= (pos0 + np.arange(nq))[:, None], False, True)
        assert torch.isfinite(out[0]).all()
