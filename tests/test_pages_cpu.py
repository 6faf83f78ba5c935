"""Page calls without a GPU: workspace sizes and what the host refuses before a launch."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from rotated_bit_kv_tq_gb300 import build, _lib
    build.build()
    return _lib.load()


def pool(**kw):
    from rotated_bit_kv_tq_gb300._lib import TqPagePool
    a = dict(n_pages=8, page_tokens=64, n_seqs=4, max_pages_per_seq=3, page_table=16, seq_lens=16, refcounts=16)
    a.update(kw)
    return TqPagePool(*[a[k] for k, _ in TqPagePool._fields_])


def group(*caches):
    from rotated_bit_kv_tq_gb300._lib import TqCache
    return (ctypes.POINTER(TqCache) * len(caches))(*[ctypes.pointer(c) for c in caches])


def test_workspace_bytes(lib):
    assert lib.tq_pages_workspace_bytes(0, 1, 1) == 0
    assert lib.tq_pages_workspace_bytes(8, -1, 1) == 0
    small, large = lib.tq_pages_workspace_bytes(8, 4, 2), lib.tq_pages_workspace_bytes(8, 4, 20)
    assert 0 < small < large and small % 4 == 0
    # head, three list words and two page words per page, two words per item, one per sequence
    assert small == 4 * (64 + 3 * 8 + 2 * 2 + 4 + 2 * 8)


@pytest.mark.parametrize("bad,status", [(dict(n_pages=0), 1), (dict(page_tokens=0), 1), (dict(n_seqs=0), 1),
                                        (dict(max_pages_per_seq=0), 1), (dict(page_table=None), 1),
                                        (dict(seq_lens=None), 1), (dict(refcounts=None), 1),
                                        (dict(page_tokens=48), 2), (dict(max_pages_per_seq=1 << 26), 2),
                                        (dict(page_tokens=32, max_pages_per_seq=1 << 25, n_seqs=64), 2)])
def test_bad_pools(lib, bad, status):
    p = ctypes.byref(pool(**bad))
    assert lib.tq_pages_extend(p, 16, 16, 1, 16, 1 << 40, None) == status
    assert lib.tq_pages_free(p, 16, 1, None) == status
    assert lib.tq_pages_fork(p, None, 0, 16, 16, 1, 16, 1 << 40, None) == status
    assert lib.tq_pages_compact(p, p, None, 0, None, 16, 1 << 40, None) == status


def test_bad_calls(lib):
    from rotated_bit_kv_tq_gb300._lib import TqCache
    p = ctypes.byref(pool())
    need = lib.tq_pages_workspace_bytes(8, 4, 1)
    assert lib.tq_pages_extend(p, 16, 16, -1, 16, need, None) == 1
    assert lib.tq_pages_extend(p, None, 16, 1, 16, need, None) == 1
    assert lib.tq_pages_extend(p, 16, 16, 1, 16, need - 1, None) == 4
    assert lib.tq_pages_extend(p, 16, 16, 1, None, need, None) == 4
    assert lib.tq_pages_extend(p, 16, 16, 1, 8, need, None) == 1          # misaligned workspace
    assert lib.tq_pages_extend(p, None, None, 0, None, 0, None) == 0      # empty list
    assert lib.tq_pages_free(p, None, 1, None) == 1
    assert lib.tq_pages_free(p, 16, -1, None) == 1
    assert lib.tq_pages_free(p, None, 0, None) == 0
    assert lib.tq_pages_fork(p, None, 0, 16, 16, 1, 16, need, None) == 1
    assert lib.tq_pages_fork(p, group(TqCache()), 300, 16, 16, 1, 16, need, None) == 2
    assert lib.tq_pages_fork(p, group(TqCache()), 1, 16, 16, 1, 16, need, None) == 1
    assert lib.tq_pages_compact(p, ctypes.byref(pool(n_seqs=5)), group(TqCache()), 1, None, 16, need, None) == 1
    flat = TqCache(3, 2, 128, 0, 16, 10, 1, 0, None, 0)
    assert lib.tq_pages_copy(group(flat), 1, 16, 16, None, 1, 16, need, None) == 1   # no pages
    assert lib.tq_pages_copy(None, 1, 16, 16, None, 1, 16, need, None) == 1


def test_python_lists_are_checked():
    import torch
    import rotated_bit_kv_tq_gb300 as tq
    with pytest.raises(tq.TQError):
        tq._list(torch.zeros(3, dtype=torch.int64))
    with pytest.raises(tq.TQError):
        tq._list(torch.zeros(6, dtype=torch.int32)[::2])
    with pytest.raises(tq.TQError):
        tq._list(torch.zeros(3, dtype=torch.int32), 4)
    with pytest.raises(tq.TQError):
        tq.PagePool(8, 64, 4, 3, device="cpu", page_table=torch.zeros(4, 2, dtype=torch.int32))


def test_model_keeps_its_invariants():
    """The Python model that the GPU tests compare with: counts, tables and rows stay
    consistent over random calls."""
    import numpy as np
    import pages_ref
    r = np.random.default_rng(0)
    m = pages_ref.Pool(20, 32, 9, 5)
    data = np.arange(20 * 32).reshape(20, 32, 1).astype(np.int64)
    own = {s: [] for s in range(9)}      # every sequence's rows as it wrote them
    for step in range(300):
        op = r.integers(0, 4)
        if op == 0:
            s, add = int(r.integers(0, 9)), int(r.integers(0, 70))
            before = int(m.lens[s])
            if m.extend([s], [add]):
                for i in range(before, before + add):
                    v = 10000 + step * 100 + i
                    data[m.table[s, i // 32], i % 32] = v
                    own[s].append(v)
        elif op == 1:
            s = int(r.integers(0, 9))
            m.free([s])
            own[s] = []
        elif op == 2:
            p, c = (int(x) for x in r.integers(0, 9, 2))
            if m.lens[c] == 0 and m.fork([data], [p], [c]):
                own[c] = list(own[p])
        else:
            m.compact([data])
        counts = np.zeros(20, int)
        for s in range(9):
            n = m.held(m.lens[s])
            assert (m.table[s, n:] == -1).all() and (m.table[s, :n] >= 0).all()
            np.add.at(counts, m.table[s, :n], 1)
            rows = [int(data[m.table[s, i // 32], i % 32, 0]) for i in range(m.lens[s])]
            assert rows == own[s]
        assert np.array_equal(counts, m.refs)
