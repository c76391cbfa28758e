"""The serving and norm operators without a GPU: argument checks of the C ABI (every call fails validation, nothing
reaches CUDA), and the tests' own plain forms against closed forms, brute force and differences."""
import ctypes
import math

import numpy as np
import pytest

import serving_ref as ref
import ternary_gemm_b200 as hbl
from ternary_gemm_b200 import build as hbl_build

A, ODD, NULL, S0 = (ctypes.c_void_p(v) for v in (0x10000, 0x10001, 0, 0))
A2, A3 = ctypes.c_void_p(0x20000), ctypes.c_void_p(0x30000)
E_ARG, E_UNS, E_WS = hbl.HBL_ERR_INVALID_ARG, hbl.HBL_ERR_UNSUPPORTED, hbl.HBL_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    hbl_build.build()
    return hbl.lib()


def _refuses(fn, good, changes):
    """fn(*good) with one argument replaced at a time answers the named status."""
    for i, value, want in changes:
        args = list(good)
        args[i] = value
        assert fn(*args) == want, (i, value, want)
    assert hbl.lib().hbl_last_cuda_error() == 0


def test_kv_plan_refusals(L):
    #        cached added B  block free n  taken table width T  total row_start slots positions taken_out
    good = [A, A, 8, 64, A, 16, A, A, 32, 8, A2, A2, A2, A2, A2, S0]
    _refuses(L.hbl_kv_plan, good, [(i, NULL, E_ARG) for i in (0, 1, 4, 6, 7, 10, 11, 12, 13, 14)])
    _refuses(L.hbl_kv_plan, good, [(i, ODD, E_ARG) for i in (0, 1, 4, 6, 7, 10, 11, 12, 13, 14)])
    _refuses(L.hbl_kv_plan, good, [(2, 0, E_ARG), (2, 4097, E_UNS), (3, 0, E_ARG), (3, 48, E_UNS), (3, 256, E_UNS),
                                   (5, -1, E_ARG), (8, 0, E_ARG), (8, 1 << 31, E_UNS), (9, 0, E_ARG),
                                   (9, (1 << 26) + 1, E_UNS),
                                   (10, A, E_ARG),      # total over cached
                                   (14, A, E_ARG)])     # taken_out over taken


def test_kv_append_refusals(L):
    #       k  v  t  T  H  D    ks    vs    slots bits n  block kc ks vc vs
    good = [A, A, 1, 8, 4, 128, 1024, 1024, A, 8, 100, 64, A, A, A2, A2, S0]
    f = L.hbl_kv_append
    _refuses(f, good, [(i, NULL, E_ARG) for i in (0, 1, 8, 12, 13, 14, 15)] + [(i, ODD, E_ARG) for i in (0, 1, 8, 12, 13, 14, 15)])
    _refuses(f, good, [(2, 2, E_ARG), (3, 0, E_ARG), (3, (1 << 26) + 1, E_UNS), (4, 0, E_ARG), (4, 1025, E_UNS),
                       (5, 0, E_ARG), (5, 96, E_UNS), (6, 511, E_ARG), (6, 504, E_ARG), (6, 1028, E_ARG),
                       (7, 500, E_ARG), (7, (1 << 32) + 8, E_UNS), (9, 0, E_ARG), (9, 1, E_UNS), (9, 9, E_UNS),
                       (10, 0, E_ARG), (10, 1 << 25, E_UNS), (11, 0, E_ARG), (11, 8, E_UNS),
                       (14, A, E_ARG), (15, A, E_ARG)])   # K and V in one buffer


def test_kv_attention_refusals(L):
    ws = hbl.hbl_kv_attention_workspace_bytes(8, 32, 8, 128, 4)
    assert ws > 0
    #       q  t  T  stride Hq  Hkv D   rows tot B table w  n    block bits kc ks vc vs scale o  ot ws
    good = [A, 1, 8, 4096, 32, 8, 128, A, A, 4, A, 32, 100, 64, 8, A, A, A, A, NULL, A2, 1, A3, ws, S0]
    f = L.hbl_kv_attention
    _refuses(f, good, [(i, NULL, E_ARG) for i in (0, 7, 8, 10, 15, 16, 17, 18, 20)])
    _refuses(f, good, [(i, ODD, E_ARG) for i in (0, 7, 8, 10, 15, 16, 17, 18, 19, 20)])
    _refuses(f, good, [(1, 2, E_ARG), (21, 2, E_ARG), (2, 0, E_ARG), (3, 4095, E_ARG), (3, 4100, E_ARG), (4, 0, E_ARG),
                       (4, 30, E_UNS), (4, 2048, E_UNS), (5, 0, E_ARG), (6, 0, E_ARG), (6, 80, E_UNS), (9, 0, E_ARG),
                       (9, 4097, E_UNS), (11, 0, E_ARG), (11, 1 << 25, E_UNS), (2, 1 << 26, E_UNS), (12, 0, E_ARG), (12, 1 << 25, E_UNS), (13, 0, E_ARG),
                       (13, 24, E_UNS), (14, 0, E_ARG), (14, 1, E_UNS), (14, 9, E_UNS), (20, A, E_ARG),
                       (22, NULL, E_WS), (22, ctypes.c_void_p(0x30010), E_WS), (23, ws - 1, E_WS)])
    for bad in ((0, 32, 8, 128, 4), (8, 32, 5, 128, 4), (8, 32, 8, 100, 4), (8, 32, 8, 128, 0), (8, 32, 8, 128, 5000)):
        assert hbl.hbl_kv_attention_workspace_bytes(*bad) == 0


def test_add_rms_quant_refusals(L):
    #       x  r  t  M  K     gain bits h  codes scales
    good = [A, A, 1, 8, 1040, A, 8, A, A, A, S0]
    _refuses(L.hbl_add_rms_quant, good, [(0, NULL, E_ARG), (8, NULL, E_ARG), (9, NULL, E_ARG), (2, 3, E_ARG), (3, 0, E_ARG),
                                         (3, (1 << 26) + 1, E_UNS), (4, 0, E_ARG), (4, 1000, E_UNS), (4, 32784, E_UNS),
                                         (6, 5, E_ARG)] + [(i, ODD, E_ARG) for i in (0, 1, 5, 7, 8, 9)])
    ws = hbl.hbl_add_rms_quant_backward_workspace_bytes(8, 1040)
    assert ws > 0 and hbl.hbl_add_rms_quant_backward_workspace_bytes(8, 1000) == 0
    assert hbl.hbl_add_rms_quant_backward_workspace_bytes(0, 1040) == 0
    #       h  t  M  K     gain g_t gt g_h g_x g_gain ws
    good = [A, 1, 8, 1040, A, A, 1, A, A2, A, A, ws, S0]
    _refuses(L.hbl_add_rms_quant_backward, good,
             [(0, NULL, E_ARG), (5, NULL, E_ARG), (8, NULL, E_ARG), (1, 3, E_ARG), (6, 3, E_ARG), (2, 0, E_ARG),
              (3, 24, E_UNS), (3, 32784, E_UNS), (8, A, E_ARG), (10, NULL, E_WS), (11, ws - 1, E_WS),
              (10, ctypes.c_void_p(0x10010), E_WS)] + [(i, ODD, E_ARG) for i in (0, 4, 5, 7, 8, 9)])


# ------------------------------------------------------------------ the plain forms themselves

def test_plan_by_hand():
    table = np.full((3, 3), -1)
    table[0, 0] = 7
    t, total, rows, slots, pos, out = ref.plan([3, 0, -5], [2, 5, 1], [9, 8, 4], 1, table, 4, 9)
    assert t.tolist() == [[7, 8, -1], [4, -1, -1], [-1, -1, -1]]   # the free list ran out after 8 and 4
    assert total.tolist() == [5, 5, 1] and rows.tolist() == [0, 2, 7, 8] and out == 5
    assert slots.tolist() == [31, 32, 16, 17, 18, 19, -1, -1, -1]
    assert pos.tolist() == [3, 4, 0, 1, 2, 3, 4, 0, -1]


def test_a_plan_that_cuts_a_request_shows():
    """T at or above the sum of `added`: the sum of total - cached is row_start[B], and positions are what the attention
    takes them to be, total - n + i.  Below it the sums differ, which is how a caller sees that rows were cut."""
    cached, added, free = [3, 10, 0], [2, 5, 4], list(range(20, 40))
    for T in (11, 14, 9, 6, 1):
        _, total, rows, _, pos, _ = ref.plan(cached, added, free, 0, np.full((3, 8), -1), 4, T)
        whole = (total - cached).sum() == rows[-1]
        assert whole == (T >= 11)
        as_attended = [total[b] - (rows[b + 1] - rows[b]) + i for b in range(3) for i in range(rows[b + 1] - rows[b])]
        assert (as_attended == pos[:rows[-1]].tolist()) == whole


def test_plan_lays_the_rows_of_a_block_out_as_one_run():
    """What the write asks of its slots: each block's rows are neighbours, at consecutive slots, with nothing between."""
    rng = np.random.default_rng(8)
    for block in (16, 64):
        cached, added = rng.integers(0, 100, 30), rng.integers(0, 150, 30)
        _, _, _, slots, _, _ = ref.plan(cached, added, rng.permutation(900)[:300], 0, _owned(rng, cached, block, 17), block, int(added.sum()) + 9)
        rows = np.flatnonzero(slots >= 0)
        for page in set((slots[rows] // block).tolist()):
            own = rows[slots[rows] // block == page]
            assert (np.diff(own) == 1).all() and (np.diff(slots[own]) == 1).all()


def _owned(rng, cached, block, width):
    """A table whose requests own blocks that no free list names."""
    table, at = np.full((len(cached), width), -1), 1000
    for b, c in enumerate(cached):
        n = min(-(-int(c) // block), width)
        table[b, :n] = np.arange(at, at + n)
        at += n
    return table


@pytest.mark.parametrize("bits", [2, 3, 8])
def test_cache_values_are_within_half_a_step(bits):
    """A value is held to half a step of its block's gamma, gamma / L, and a requantized one to half a step more for
    each growth of gamma; the float32 arithmetic of the codes and eps / gamma add 2^-20 of gamma."""
    rng = np.random.default_rng(bits)
    x = rng.standard_normal((40, 2, 32)).astype(np.float32)
    x[20] *= 3.0                                            # gamma of the second block grows inside it
    codes, scales = np.full((4, 2, 16, 32), 99, np.uint8), np.full((4, 2), np.nan, np.float32)
    slots = np.r_[48:64, 0:16, 16:24]
    grown = np.zeros(40)
    for i in range(40):                                     # token by token
        before = scales.copy()
        codes, scales = ref.append(x[i:i + 1], slots[i:i + 1], codes, scales, bits)
        if slots[i] % 16 and (scales[slots[i] // 16] > before[slots[i] // 16]).any():
            grown[[j for j in range(i) if slots[j] // 16 == slots[i] // 16]] += 1
    assert grown.max() >= 1
    got = ref.values(codes, scales, bits)
    for i, s in enumerate(slots):
        gamma = scales[s // 16].astype(np.float64)[:, None]
        bound = gamma / (2 ** bits - 1) * (1 + grown[i]) + 2.0 ** -16 * gamma + 2e-5
        assert np.all(np.abs(got[s // 16, :, s % 16] - x[i]) <= bound)


def test_attention_reference_closed_forms():
    """Equal keys give the mean of the values, one dominating key gives its value; a row sees its own token and none
    behind it; absent pages are not seen; no page gives 0."""
    rng = np.random.default_rng(1)
    v = rng.standard_normal((3, 1, 16, 32))
    k = np.ones((3, 1, 16, 32))
    q = rng.standard_normal((2, 1, 32))
    table = np.array([[2, 0]])
    o, *_ = ref.attention(q, [0, 2], [20], table, k, v, 0.3)
    line = np.concatenate([v[2, 0], v[0, 0]])
    assert np.allclose(o[0, 0], line[:19].mean(0)) and np.allclose(o[1, 0], line[:20].mean(0))
    k[2, 0, 5] = 400.0 * np.sign(q[0, 0])
    o, *_ = ref.attention(q, [0, 1], [20], table, k, v, 0.3)
    assert np.allclose(o[0, 0], v[2, 0, 5]) and np.isnan(o[1]).all()
    o, *_ = ref.attention(q, [0, 2], [20], np.array([[-1, 0]]), np.ones_like(k), v, 0.3)
    assert np.allclose(o[1, 0], v[0, 0, :4].mean(0))
    assert np.all(ref.attention(q, [0, 2], [20], np.array([[9, 3]]), k, v, 0.3)[0] == 0)


@pytest.mark.parametrize("with_gain", [False, True])
def test_rms_gradient_against_differences(with_gain):
    rng = np.random.default_rng(4)
    M, K, d = 3, 48, 1e-6
    h, g_t, g_h = rng.standard_normal((3, M, K))
    gain = 1.0 + 0.3 * rng.standard_normal(K) if with_gain else None
    g_x, g_gain, _ = ref.add_rms_backward(h, gain, g_t, g_h)
    loss = lambda hh, gg: (ref.rms_value(hh, gg) * g_t).sum() + (hh * g_h).sum()  # noqa: E731
    for m, k in [(0, 0), (1, 17), (2, 47)]:
        e = np.zeros((M, K))
        e[m, k] = d
        # central differences: an error of order d^2 and rounding of 1e-16 * |loss| / d
        assert math.isclose((loss(h + e, gain) - loss(h - e, gain)) / (2 * d), g_x[m, k], rel_tol=1e-6, abs_tol=1e-7)
    if with_gain:
        e = np.zeros(K)
        e[9] = d
        assert math.isclose((loss(h, gain + e) - loss(h, gain - e)) / (2 * d), g_gain[9], rel_tol=1e-6, abs_tol=1e-7)


def test_quantizer_of_the_plain_form_matches_the_oracle(orc):
    rng = np.random.default_rng(6)
    x, r = rng.standard_normal((2, 5, 256)).astype(np.float32)
    for bits in (4, 8):
        _, t, q, s = ref.add_rms_quant(x, r, None, bits, False)
        qo, so = orc.quant(t.astype(np.float32), bits)
        assert np.array_equal(q, qo) and np.array_equal(s, so)
