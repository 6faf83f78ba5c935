"""Page calls on the GPU against a plain Python model (pages_ref), and together with the
cache and attention calls that they serve."""
import numpy as np
import pytest

import pages_ref
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


def ints(x):
    return torch.tensor(list(x), dtype=torch.int32, device=DEV)


class Pair:
    """The pool on the GPU and its model, with caches of several types and head counts."""

    def __init__(self, tq, n_pages, pt, n_seqs, cols, kinds, seed):
        self.tq, self.r = tq, np.random.default_rng(seed)
        self.model = pages_ref.Pool(n_pages, pt, n_seqs, cols)
        self.pool = tq.PagePool(n_pages, pt, n_seqs, cols, device=DEV)
        self.caches = [tq.KVCache(t, hkv, 128, n_seqs=n_seqs, page_tokens=pt, page_table=self.pool.page_table,
                                  n_pages=n_pages) for t, hkv in kinds]
        self.data = []
        for c in self.caches:
            x = self.r.integers(0, 256, (n_pages, pt, c.row_bytes), dtype=np.uint8)
            c.buffer.copy_(torch.from_numpy(x.reshape(-1)))
            self.data.append(x)
        self.group = tq.CacheGroup(self.caches)

    def same(self, ok=True):
        torch.cuda.synchronize()
        assert (self.tq.device_status() == 0) == ok
        m = self.model
        assert np.array_equal(self.pool.page_table.cpu().numpy(), m.table)
        assert np.array_equal(self.pool.seq_lens.cpu().numpy(), m.lens)
        assert np.array_equal(self.pool.refcounts.cpu().numpy(), m.refs)
        for c, x in zip(self.caches, self.data):
            assert np.array_equal(c.buffer.cpu().numpy().reshape(x.shape), x)

    def extend(self, seqs, n):
        ok = self.model.extend(seqs, n)
        self.tq.pages_extend(self.pool, ints(seqs), ints(n))
        self.same(ok)

    def free(self, seqs):
        ok = self.model.free(seqs)
        self.tq.pages_free(self.pool, ints(seqs))
        self.same(ok)

    def fork(self, parents, children):
        ok = self.model.fork(self.data, parents, children)
        self.tq.pages_fork(self.pool, self.group, ints(parents), ints(children))
        self.same(ok)

    def compact(self):
        U = self.model.compact(self.data)
        used = ints([-5])
        self.tq.pages_compact(self.pool, self.group, n_used=used)
        self.same()
        assert int(used) == U


KINDS = [(36, 8), (3, 8), (36, 1), (2, 3)]


def test_refusals_and_repeats(tq):
    p = Pair(tq, 9, 32, 6, 4, KINDS[:2], 0)
    p.extend([0, 1], [70, 32])                     # 3 + 1 pages
    p.extend([2, 2, 9, -1, 3], [1, 40, 1, 1, -2])  # repeated, out of range, negative
    p.extend([1, 0], [97, 0])                      # more than a table row holds; nothing to add
    p.extend([3, 4, 5, 0], [100, 33, 0, 1])        # 4 pages, then 2 that are not there, none, one within a page
    p.fork([0, 0, 1, 7, 5], [4, 4, 0, 5, 5])       # repeated child, non-empty child, bad parent, empty parent
    p.free([3, 3, 8, 5])
    p.fork([0, 0, 0, 2, 1], [3, 5, 9, 3, 1])
    p.free(list(range(6)))
    p.compact()                                    # an empty pool


def test_exhausted_fork(tq):
    p = Pair(tq, 5, 32, 8, 3, KINDS[2:], 1)
    p.extend([0, 1], [33, 32])                     # 3 pages, 2 left
    p.fork([0, 1, 0, 0, 1], [2, 3, 4, 5, 6])       # the third copy of a part page finds none
    p.free([0, 2])
    p.compact()


@pytest.mark.parametrize("n_pages,pt,n_seqs,cols,seed", [(7, 32, 5, 3, 2), (64, 32, 24, 6, 3), (40, 256, 12, 5, 4),
                                                         (5000, 32, 40, 9, 5), (9000, 32, 300, 40, 6)])
def test_random_runs(tq, n_pages, pt, n_seqs, cols, seed):
    kinds = KINDS if n_pages < 100 else [(36, 1)]
    p = Pair(tq, n_pages, pt, n_seqs, cols, kinds, seed)
    r = p.r
    for step in range(25):
        op = step % 5 if step < 5 else r.integers(0, 5)
        k = int(r.integers(1, n_seqs + 1))
        seqs = r.permutation(n_seqs)[:k].tolist()
        if op in (0, 1):
            p.extend(seqs, r.integers(0, cols * pt // 2 + 2, k).tolist())
        elif op == 2:
            empty = [s for s in range(n_seqs) if p.model.lens[s] == 0]
            ch = r.permutation(empty)[:k].tolist()
            if ch:
                p.fork(r.integers(0, n_seqs, len(ch)).tolist(), [int(c) for c in ch])
        elif op == 3:
            p.free(seqs[: max(1, k // 2)])
        else:
            p.compact()


def test_compact_out_of_place(tq):
    """The old table and its pages stay readable beside the new one."""
    p = Pair(tq, 30, 32, 8, 4, [(36, 8)], 7)
    p.extend(range(8), [100, 20, 64, 1, 128, 33, 5, 90])
    p.free([0, 2, 5])
    before = p.model.copy()
    old = p.data[0].copy()
    out = tq.PagePool(30, 32, 8, 4, device=DEV)
    tq.pages_compact(p.pool, p.group, out=out)
    torch.cuda.synchronize()
    U = p.model.compact(p.data)
    assert tq.device_status() == 0
    assert np.array_equal(out.page_table.cpu().numpy(), p.model.table)
    assert np.array_equal(out.refcounts.cpu().numpy(), p.model.refs) and (p.model.refs[U:] == 0).all()
    assert np.array_equal(out.seq_lens.cpu().numpy(), p.model.lens)
    assert np.array_equal(p.pool.page_table.cpu().numpy(), before.table)
    now = p.caches[0].buffer.cpu().numpy().reshape(old.shape)
    for q in np.nonzero(before.refs)[0]:
        assert np.array_equal(now[q], old[q])


def test_copy(tq):
    p = Pair(tq, 20, 64, 2, 2, KINDS, 8)
    src, dst, rows = [0, 5, 0, 3, 7, 25, 2, 6], [10, 11, 12, 10, 5, 1, -1, 13], [64, 1, 0, 9, 3, 1, 1, 65]
    ws = torch.empty(tq.pages_workspace_bytes(20, 0, len(src)), dtype=torch.uint8, device=DEV)
    tq.pages_copy(p.group, ints(src), ints(dst), ints(rows), workspace=ws)
    for x in p.data:
        x[10] = x[0]
        x[11, :1] = x[5, :1]
    p.same(ok=False)      # a repeated destination, one that is a source, three bad numbers
    tq.pages_copy(p.group, ints([1, 1, 2]), ints([3, 4, 19]), workspace=ws)
    for x in p.data:
        x[3], x[4], x[19] = x[1], x[1], x[2]
    p.same()


def test_graph_and_stream(tq):
    """A beam step (free, fork, extend, compact) captured once and replayed on another stream:
    every replay gives what the model gives."""
    p = Pair(tq, 40, 32, 9, 4, KINDS[:2], 9)
    p.extend([0, 1], [75, 40])
    p.fork([0, 0, 1], [2, 3, 4])
    ch, par, seqs, add = ints([2, 3, 4]), ints([0, 1, 1]), ints([2, 4]), ints([30, 1])
    side = torch.cuda.Stream()

    def step():
        tq.pages_free(p.pool, ch)
        tq.pages_fork(p.pool, p.group, par, ch)
        tq.pages_extend(p.pool, seqs, add)
        tq.pages_compact(p.pool, p.group)

    def model():
        p.model.free([2, 3, 4])
        p.model.fork(p.data, [0, 1, 1], [2, 3, 4])
        p.model.extend([2, 4], [30, 1])
        p.model.compact(p.data)

    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    model()
    p.same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    for _ in range(3):
        g.replay()
        model()
        p.same()


def test_serving_run(tq):
    """Prompt, parallel continuations, decode steps, release, compaction: the caches' rows and
    the attention of every live sequence stay what contiguous references give."""
    r = np.random.default_rng(10)
    hkv, hq, d, pt, S, cols, n_pages = 8, 32, 128, 32, 6, 8, 40
    pool = tq.PagePool(n_pages, pt, S, cols, device=DEV)
    kc, vc = (tq.KVCache(tq.TQ_TURBO4, hkv, d, n_seqs=S, page_tokens=pt, page_table=pool.page_table,
                         n_pages=n_pages) for _ in range(2))
    group = tq.CacheGroup([kc, vc])
    rows = {s: [np.zeros((0, 528), np.uint8)] * 2 for s in range(S)}

    def draw(n):
        return r.standard_normal((n, hkv, d)).astype(np.float16)

    def prompt(s, n):
        x = [draw(n), draw(n)]
        pool_n = ints([n])
        tq.pages_extend(pool, ints([s]), pool_n)
        tq.encode_kv(kc, vc, *[torch.from_numpy(a.reshape(n, -1)).to(DEV) for a in x], seq_id=s)
        rows[s] = [ref.encode_rows(a.reshape(n, -1), hkv) for a in x]

    def step(live):
        tq.pages_extend(pool, ints(live), ints([1] * len(live)))
        new = [draw(S), draw(S)]
        q = r.standard_normal((S, hq, d)).astype(np.float16)
        out = torch.full((S, hq, d), 5.0, dtype=torch.float16, device=DEV)
        most = max(len(rows[s][0]) for s in range(S)) + 1
        ws = torch.empty(tq.attn_workspace_bytes(S, hq, d, most), dtype=torch.uint8, device=DEV)
        lens = torch.zeros(S, dtype=torch.int32, device=DEV)
        lens[live] = pool.seq_lens[live]
        tq.attn_decode_append(kc, vc, *[torch.from_numpy(a).to(DEV) for a in new],
                              torch.from_numpy(q).to(DEV), lens, most, out, ws)
        for s in live:
            rows[s] = [np.concatenate([x, ref.encode_rows(a[s].reshape(1, -1), hkv)]) for x, a in zip(rows[s], new)]
        torch.cuda.synchronize()
        assert tq.device_status() == 0
        got = out.cpu().numpy().astype(np.float64)
        for s in range(S):
            if s not in live:
                assert (got[s] == 0).all()
                continue
            n = len(rows[s][0])
            see = np.ones((1, n), bool)
            want = ref.attention(*[ref.dequant(x, hkv) for x in rows[s]], q[s:s + 1], see, d ** -0.5, hkv)
            bound = ref.attention_bound(*rows[s], q[s:s + 1], see, d ** -0.5, hkv, True, False)
            assert (np.linalg.norm(got[s:s + 1] - want, axis=-1) <= bound).all()

    def stored():
        t, lens = pool.page_table.cpu().numpy(), pool.seq_lens.cpu().numpy()
        for c, i in ((kc, 0), (vc, 1)):
            x = c.buffer.cpu().numpy().reshape(n_pages, pt, 528)
            for s in range(S):
                n = lens[s]
                assert n == len(rows[s][0])
                have = x[t[s, : -(-n // pt)]].reshape(-1, 528)[:n] if n else rows[s][i]
                assert np.array_equal(have, rows[s][i])

    prompt(0, 70)
    prompt(1, 64)
    tq.pages_fork(pool, group, ints([0, 0, 1]), ints([2, 3, 4]))
    rows[2], rows[3], rows[4] = list(rows[0]), list(rows[0]), list(rows[1])
    for _ in range(3):
        step([0, 2, 3, 4])
    stored()
    tq.pages_free(pool, ints([0, 3]))
    rows[0] = rows[3] = [np.zeros((0, 528), np.uint8)] * 2
    tq.pages_compact(pool, group)
    stored()
    prompt(5, 33)
    step([1, 2, 4, 5])
    stored()
    tq.pages_free(pool, ints(range(S)))
    torch.cuda.synchronize()
    assert (pool.refcounts == 0).all() and (pool.page_table == -1).all()
