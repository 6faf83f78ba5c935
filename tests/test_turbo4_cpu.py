"""turbo4 without a GPU: the codebook, the sizes, the layout of the reference and every
refusal that the host makes before it launches anything."""
import ctypes

import numpy as np
import pytest

import turbo4_ref as ref


@pytest.fixture(scope="module")
def lib():
    from rotated_bit_kv_tq_gb300 import build, _lib
    build.build()
    return _lib.load()


def test_sizes(lib):
    import rotated_bit_kv_tq_gb300 as tq
    assert tq.TQ_TURBO4 == 36
    assert lib.tq_block_bytes(36) == 66
    assert lib.tq_row_bytes(36, 8, 128) == 528 and lib.tq_row_bytes(36, 4, 256) == 528
    assert lib.tq_row_bytes(36, 3, 100) == 0


def test_codebook(lib):
    import rotated_bit_kv_tq_gb300 as tq
    c, t = tq.codebook_get(tq.TQ_TURBO4)
    assert c.shape == (16,) and t.shape == (15,)
    assert np.array_equal(c.astype(np.float64), ref.CENT)          # exact in fp32
    assert np.array_equal(t.astype(np.float64), (ref.CENT[1:] + ref.CENT[:-1]) / 2)


def test_levels_are_e4m3_numbers():
    for v in ref.LEVELS / 16:
        m, e = np.frexp(v)                    # v = m 2^e, m in [0.5, 1)
        assert (m * 16) == int(m * 16) and -6 <= e - 1 <= 8        # four significant bits


def test_levels_are_close_to_lloyd_max():
    """Normalised MSE of one coordinate of a unit vector in R^128, by quadrature: within 1 % of
    the unconstrained 16-level optimum, and no neighbouring e4m3 level improves it."""
    y = np.linspace(0, 0.8, 80001)
    f = (1 - y * y) ** 62.5
    f /= f.sum()

    def mse(levels):
        t = (levels[1:] + levels[:-1]) / 2
        return 128 * (f * (y - levels[np.searchsorted(t, y)]) ** 2).sum()

    lm = np.linspace(0.01, 0.25, 8)
    for _ in range(2000):
        i = np.searchsorted((lm[1:] + lm[:-1]) / 2, y)
        lm = np.array([(f * y)[i == k].sum() / f[i == k].sum() for k in range(8)])
    ours = mse(ref.LEVELS * ref.STEP)
    assert ours < 1.01 * mse(lm)
    for k in range(8):
        m, e = np.frexp(ref.LEVELS[k])
        for d in (-1, 1):
            other = ref.LEVELS.copy()
            other[k] = (m * 16 + d) / 16 * 2.0 ** e
            assert mse(other * ref.STEP) > ours


def test_layout_by_hand():
    """One value in one place: nibble and sign bit of every value of a block."""
    for i in range(128):
        mag = np.zeros((2, 128), int)
        neg = np.zeros((2, 128), bool)
        mag[1, i], neg[1, i] = 5, True
        row = ref.pack(mag, neg, np.array([1.0, 2.0], np.float16), 2)
        assert row.shape == (1, 132)
        words = row[0, 64:128].view("<u4")
        k = i % 8
        assert words[i // 8] == (5 << (4 * k)) | (1 << (8 * k + 7 if k < 4 else 8 * (k - 4) + 3))
        assert not row[0, :64].any() and words.astype(bool).sum() == 1
        assert list(row[0, 128:132].view(np.float16)) == [1.0, 2.0]


def test_refusals(lib):
    from rotated_bit_kv_tq_gb300._lib import TqCache
    ok = TqCache(36, 2, 128, 0, 16, 10, 1, 0, None, 0)
    assert lib.tq_codebook_get(4, None, None) == 1
    plain4 = TqCache(4, 2, 128, 0, 16, 10, 1, 0, None, 0)
    assert lib.tq_encode(ctypes.byref(plain4), 16, 1, 256, None, None, 0, 0, None) == 1
    odd = TqCache(36, 2, 96, 0, 16, 10, 1, 0, None, 0)
    assert lib.tq_encode(ctypes.byref(odd), 16, 1, 256, None, None, 0, 0, None) == 2
    for name in ("tq_attn_decode_f16", "tq_attn_decode_append_f16"):
        lead = (16, 16) if "append" in name else ()
        args = (ctypes.byref(ok), None, *lead, 16, 1, 4, 16, 64, 0.0, 16, None, 0, None)
        assert getattr(lib, name)(*args) != 0
    assert lib.tq_attn_decode_append_f16(ctypes.byref(ok), ctypes.byref(ok), 8, 16, 16, 1, 4, 16, 64,
                                         0.0, 16, None, 0, None) == 1     # misaligned new row
    assert lib.tq_attn_prefill_f16(None, None, 16, 0, 0, 1, 4, 0.0, 16, None) == 1
    assert lib.tq_attn_decode_f16(None, None, 16, 1, 4, 16, 64, 0.0, 16, None, 0, None) == 1


def test_output_type_is_checked():
    import torch
    import rotated_bit_kv_tq_gb300 as tq
    with pytest.raises(tq.TQError):
        tq._fn("tq_attn_decode", torch.empty(1, dtype=torch.float64))
