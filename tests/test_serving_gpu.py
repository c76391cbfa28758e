"""GPU tests of the serving and norm operators against their plain forms (serving_ref): the cache's plan and codes
exactly, the attention within the error that its contract counts, the norm's codes exactly from its h, the gradient
within counted float errors; at ragged sizes, strides, pages and masks, on other streams and in captured graphs."""
import numpy as np
import pytest

import serving_ref as ref
from helpers import to_device, to_host

pytestmark = pytest.mark.gpu

GUARD, FILL = 4096, 0xA5


@pytest.fixture(scope="module")
def H():
    import torch
    from ternary_gemm_b200 import build
    assert torch.cuda.is_available()
    build.build()
    import ternary_gemm_b200 as hbl
    return hbl


def _dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def _i32(a):
    return _dev(np.asarray(a, np.int32))


def _values(x, bf16):
    return ref.bf16_round(np.asarray(x, np.float32)) if bf16 else np.asarray(x, np.float32)


def _as(x, bf16):
    import torch
    return _dev(x, torch.bfloat16 if bf16 else torch.float32)


def _np(t):
    return t.float().cpu().numpy()


def _guarded(shape, dtype):
    """A tensor inside a canary-filled buffer, and a check that the canaries are whole."""
    import torch
    n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
    buf = torch.full((2 * GUARD + n,), FILL, dtype=torch.uint8, device="cuda")

    def check(what):
        torch.cuda.synchronize()
        assert bool((buf[:GUARD] == FILL).all()) and bool((buf[GUARD + n:] == FILL).all()), what

    return buf[GUARD:GUARD + n].view(dtype).view(*shape), check


# ------------------------------------------------------------------ plan

def _plan_case(rng, B, block, width, longest, new):
    cached = rng.integers(0, longest + 1, B)
    added = rng.integers(0, new + 1, B)
    had = np.minimum(-(-cached // block), width)
    ids = rng.permutation(2 * B * width + 40)
    table = np.full((B, width), -1)
    for b in range(B):
        table[b, :had[b]], ids = ids[:had[b]], ids[had[b]:]
    return cached, added, table, ids


@pytest.mark.parametrize("B,block,width,longest,new,pad", [
    (1, 16, 1, 0, 1, 0), (1, 128, 3, 200, 300, 5), (7, 16, 40, 500, 3, 0), (33, 64, 20, 1200, 1, 31),
    (300, 32, 12, 250, 40, 9), (4096, 16, 4, 40, 2, 100)])
def test_plan(H, B, block, width, longest, new, pad):
    rng = np.random.default_rng(B + block)
    cached, added, table, free = _plan_case(rng, B, block, width, longest, new)
    added[0] = max(1, added[0])
    T = int(added.sum()) + pad
    want = ref.plan(cached, added, free, 2, table, block, T)
    dev = _i32(table)
    for _ in range(2):          # a repeated call gives the same
        got = H.hbl_kv_plan(_i32(cached), _i32(added), _i32(free), _i32([2]), dev, block, T)
        for name, g, w in zip(("table", "total", "row_start", "slots", "positions", "taken"), (dev,) + got, want):
            assert np.array_equal(to_host(g).reshape(-1), np.asarray(w).reshape(-1)), name


def test_plan_short_of_rows_blocks_and_width(H):
    rng = np.random.default_rng(3)
    cached, added, table, free = _plan_case(rng, 40, 16, 6, 110, 60)
    cached[3], added[4], added[5] = -7, -2, 2 ** 31 - 1        # negative lengths, one past every width
    for T, n in ((300, 20), (50, len(free)), (2000, 1)):
        want = ref.plan(cached, added, free[:n], 0, table, 16, T)
        dev = _i32(table)
        got = H.hbl_kv_plan(_i32(cached), _i32(added), _i32(free[:n]), _i32([0]), dev, 16, T)
        for g, w in zip((dev,) + got, want):
            assert np.array_equal(to_host(g).reshape(-1), np.asarray(w).reshape(-1))


def test_plan_without_free_blocks(H):
    """Steps that need no block take an empty free list; one that needs some gets -1."""
    import torch
    table = _i32([[5, -1], [2, 3]])
    none = torch.empty((0,), dtype=torch.int32, device="cuda")
    for cached, added in (([3, 17], [2, 15]), ([16, 20], [1, 1])):
        want = ref.plan(cached, added, [], 0, to_host(table), 16, 20)
        got = H.hbl_kv_plan(_i32(cached), _i32(added), none, _i32([0]), table, 16, 20)
        for g, w in zip((table,) + got, want):
            assert np.array_equal(to_host(g).reshape(-1), np.asarray(w).reshape(-1))


# ------------------------------------------------------------------ append

def _cache(rng, n, H, block, D, bits):
    codes = rng.integers(0, 2 ** bits, (n, H, block, D)).astype(np.uint8)
    scales = np.exp(rng.uniform(-3, 1.5, (n, H))).astype(np.float32)
    return codes, scales


def _slots(rng, lengths, new, block, spare=3):
    """Slots of `new[b]` rows behind lengths[b] cached tokens, pages in random order: (slots, table, pages)."""
    total = np.asarray(lengths) + np.asarray(new)
    pages = -(-total // block)
    ids = rng.permutation(int(pages.sum()) + spare)
    table, slots = np.full((len(total), int(pages.max()) + 1), -1), []
    for b, n in enumerate(pages):
        table[b, :n], ids = ids[:n], ids[n:]
        p = np.arange(lengths[b], total[b])
        slots.append(table[b, p // block] * block + p % block)
    return np.concatenate(slots), table, int(pages.sum()) + spare


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("heads,D,block,bits,lengths,new", [
    (1, 32, 16, 8, [0], [1]),
    (3, 128, 64, 8, [0, 63, 64, 5, 129], [1, 1, 1, 1, 1]),
    (2, 64, 32, 3, [0, 31, 7], [70, 2, 25]),
    (5, 256, 16, 4, [15, 0, 3], [3, 16, 13]),
    (8, 128, 128, 8, [100, 0, 0, 255], [200, 128, 1, 130]),
    (1, 128, 16, 2, [1], [300])])
def test_append(H, heads, D, block, bits, lengths, new, bf16):
    rng = np.random.default_rng(D + block + bits)
    slots, _, n = _slots(rng, lengths, new, block)
    T = len(slots)
    wide = _values(rng.standard_normal((T, 2 * heads * D + 24)) * np.exp(rng.uniform(-2, 2, (T, 1))), bf16)
    wide[0, :heads * D] = 0.0                                   # a row of zeros
    k, v = wide[:, :heads * D].reshape(T, heads, D), wide[:, heads * D + 16:2 * heads * D + 16].reshape(T, heads, D)
    (kc, ks), (vc, vs) = _cache(rng, n, heads, block, D, bits), _cache(rng, n, heads, block, D, bits)
    for page in set((slots // block).tolist()):                 # what a fresh block's scale holds does not matter
        if (slots[slots // block == page] % block).min() == 0:
            ks[page] = np.nan
    wk, wv = ref.append(k, slots, kc, ks, bits), ref.append(v, slots, vc, vs, bits)
    d = _as(wide, bf16)
    dk, dv = d[:, :heads * D].unflatten(1, (heads, D)), d[:, heads * D + 16:2 * heads * D + 16].unflatten(1, (heads, D))
    state = [_dev(a) for a in (kc, ks, vc, vs)]
    for _ in range(2):                                          # the same rows again change nothing
        H.hbl_kv_append(dk, dv, _i32(slots), *state, bits)
        for name, g, w in zip(("k codes", "k scales", "v codes", "v scales"), state, wk + wv):
            assert np.array_equal(to_host(g), w, equal_nan=True), name


def test_append_passes_over_rows_without_a_place(H):
    """Slots below 0 and past the cache, NaN in their rows: the other rows' blocks are as without them."""
    rng = np.random.default_rng(8)
    heads, D, block, bits, n = 2, 64, 16, 8, 9
    slots = np.array([-1, 30, 31, -1, 32, 33, n * block, 2 ** 31 - 1, 64, -2 ** 31, 5])
    x = _values(rng.standard_normal((len(slots), heads, D)), True)
    x[(slots < 0) | (slots >= n * block)] = np.nan
    kc, ks = _cache(rng, n, heads, block, D, bits)
    want = ref.append(x, slots, kc, ks, bits)
    codes, check_c = _guarded((n, heads, block, D), _dev(kc).dtype)
    scales, check_s = _guarded((n, heads), _dev(ks).dtype)
    codes.copy_(_dev(kc))
    scales.copy_(_dev(ks))
    vc, vs = _dev(kc), _dev(ks)
    H.hbl_kv_append(_as(x, True), _as(x, True), _i32(slots), codes, scales, vc, vs, bits)
    check_c("codes")
    check_s("scales")
    for g in ((codes, scales), (vc, vs)):
        assert np.array_equal(to_host(g[0]), want[0]) and np.array_equal(to_host(g[1]), want[1])


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("new", [[1, 1], [90, 64]])
def test_append_of_nan(H, new, bf16):
    """A NaN takes no part in its block's gamma, its code is one of the levels, and all other codes are as with 0 in its
    place; the other heads and blocks know nothing of it."""
    rng = np.random.default_rng(sum(new))
    heads, D, block, bits = 3, 128, 32, 3
    slots, _, n = _slots(rng, [10, 0], new, block)
    x = _values(rng.standard_normal((len(slots), heads, D)), bf16)
    x[0, 1, 5], x[-1, 2, 127] = 0.0, 0.0
    kc, ks = _cache(rng, n, heads, block, D, bits)
    want = ref.append(x, slots, kc, ks, bits)
    x[0, 1, 5], x[-1, 2, 127] = np.nan, -np.nan
    state = [_dev(a) for a in (kc, ks, kc, ks)]
    H.hbl_kv_append(_as(x, bf16), _as(x, bf16), _i32(slots), *state, bits)
    for codes, scales in (state[:2], state[2:]):
        codes, same = to_host(codes), want[0].copy()
        for row, h, d in ((0, 1, 5), (-1, 2, 127)):
            at = slots[row] // block, h, slots[row] % block, d
            assert codes[at] < 2 ** bits
            same[at] = codes[at]
        assert np.array_equal(codes, same) and np.array_equal(to_host(scales), want[1])


def test_append_many_rows(H):
    """A prompt batch long enough that every CTA works: sampled pages against the plain form."""
    rng = np.random.default_rng(12)
    heads, D, block = 8, 128, 64
    lengths, new = [0, 40, 1000, 3], [1500, 900, 1, 1211]
    slots, _, n = _slots(rng, lengths, new, block)
    x = _values(rng.standard_normal((len(slots), heads, D)), True)
    kc, ks = _cache(rng, n, heads, block, D, 8)
    want = ref.append(x, slots, kc, ks, 8)
    state = [_dev(a) for a in (kc, ks, kc, ks)]
    H.hbl_kv_append(_as(x, True), _as(x, True), _i32(slots), *state)
    assert np.array_equal(to_host(state[0]), want[0]) and np.array_equal(to_host(state[1]), want[1])
    assert np.array_equal(to_host(state[2]), want[0]) and np.array_equal(to_host(state[3]), want[1])


def _grown_blocks(seed, bits, bf16):
    """One row into each of thousands of blocks that hold earlier tokens under smaller scales, and the plain form."""
    rng = np.random.default_rng(seed)
    n, heads, block, D = 5000, 8, 16, 32
    codes, _ = _cache(rng, n, heads, block, D, bits)
    scales = np.exp(rng.uniform(-3, 1, (n, heads))).astype(np.float32)
    slots = rng.permutation(n) * block + rng.integers(1, block, n)
    x = _values(rng.standard_normal((n, heads, D)) * 4.0, bf16)
    want = ref.append(x, slots, codes, scales, bits)
    assert (want[1] > scales).mean() > 0.95
    return x, slots, codes, scales, want


@pytest.mark.parametrize("bits,bf16", [(8, True), (8, False), (3, True)])
def test_append_into_thousands_of_growing_blocks(H, bits, bf16):
    """Enough requantized codes that one reading of gamma / L beside the rule's (a product with the rounded reciprocal)
    would show: bit for bit the plain form."""
    x, slots, codes, scales, want = _grown_blocks(40 + bits, bits, bf16)
    state = [_dev(a) for a in (codes, scales, codes, scales)]
    H.hbl_kv_append(_as(x, bf16), _as(x, bf16), _i32(slots), *state, bits)
    for g, w in zip(state, want + want):
        assert np.array_equal(to_host(g), w)


@pytest.mark.parametrize("bits", [8, 4])
def test_the_workloads_plain_write_follows_the_rule(bits):
    """The plain form that the measured write is compared with, on the same blocks."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "operators.py")
    spec = importlib.util.spec_from_file_location("operators", path)
    ops = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ops)
    x, slots, codes, scales, want = _grown_blocks(50 + bits, bits, True)
    dc, ds = _dev(codes), _dev(scales)
    ops._plain_append_one(_as(x, True), _i32(slots), dc, ds, bits)
    assert np.array_equal(to_host(dc), want[0]) and np.array_equal(to_host(ds), want[1])


# ------------------------------------------------------------------ attention

def _attend(H, rng, new, total, Hq, Hkv, D, block, bits, bf16, o_bf16=None, pad=0, first=0, scale=None, mend=None,
            spare=4, k_gain=1.0):
    """One attention call on random pages against the plain form; `mend` may change (table, codes, scales) first."""
    import torch
    o_bf16 = bf16 if o_bf16 is None else o_bf16
    B = len(new)
    pages = -(-np.maximum(total, 0) // block)
    ids = rng.permutation(int(pages.sum()) + spare)
    table = np.full((B, max(1, int(pages.max())) + 2), -1)
    for b in range(B):
        table[b, :pages[b]], ids = ids[:pages[b]], ids[pages[b]:]
    n = int(pages.sum()) + spare
    (kc, ks), (vc, vs) = _cache(rng, n, Hkv, block, D, bits), _cache(rng, n, Hkv, block, D, bits)
    ks *= np.float32(k_gain)
    rows = first + np.concatenate([[0], np.cumsum(new)])
    T = int(rows[-1]) + pad
    q = _values(rng.standard_normal((T, Hq * D + 16)), bf16)
    if mend:
        mend(table, kc, ks, vc, vs, q)
    s64 = D ** -0.5 if scale is None else float(np.float32(scale))
    q3 = q[:, :Hq * D].reshape(T, Hq, D)
    want, *sizes = ref.attention(q3, rows, total, table, ref.values(kc, ks, bits), ref.values(vc, vs, bits), s64, vs)
    dt = torch.bfloat16 if o_bf16 else torch.float32
    o, check = _guarded((T, Hq, D), dt)
    o.fill_(7.0)
    ws, check_ws = _guarded((H.hbl_kv_attention_workspace_bytes(T, Hq, Hkv, D, B),), torch.uint8)
    got = H.hbl_kv_attention(_as(q, bf16)[:, :Hq * D].unflatten(1, (Hq, D)), _i32(rows), _i32(total), _i32(table), _dev(kc),
                             _dev(ks), _dev(vc), _dev(vs), bits, scale=None if scale is None else _dev(np.float32([scale])),
                             o=o, workspace=ws)
    check("o")
    check_ws("workspace")
    assert H.hbl_last_device_error() == H.HBL_OK
    got = _np(got).astype(np.float64)
    mine = ~np.isnan(want[:, 0, 0])
    assert np.all(got[~mine] == 7.0), "rows outside the requests were written"
    tol = ref.attention_tolerance(want, *sizes, int(max(1, max(total))), not bf16, not o_bf16)
    off = np.abs(got - want)[mine]
    assert np.isfinite(got[mine]).all()
    assert np.all(off <= tol[mine]), (off - tol[mine]).max()
    return got, want


HEADS = [(1, 1), (4, 4), (8, 2), (16, 1), (20, 5), (6, 2), (40, 1)]


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("D,block", [(32, 16), (64, 32), (128, 64), (256, 128), (128, 16), (64, 128)])
def test_attention_single_rows(H, D, block, bf16):
    rng = np.random.default_rng(D + block)
    total = np.array([1, 2, block - 1, block, block + 1, 3 * block + 5, 700])
    _attend(H, rng, [1] * 7, total, 8, 2, D, block, 8, bf16)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_attention_head_layouts(H, Hq, Hkv, bf16):
    rng = np.random.default_rng(Hq * 100 + Hkv)
    _attend(H, rng, [1, 3, 1, 18], np.array([333, 40, 1, 150]), Hq, Hkv, 64, 32, 8, bf16)


@pytest.mark.parametrize("bits", [2, 3, 4, 8])
def test_attention_bits(H, bits):
    _attend(H, np.random.default_rng(bits), [1, 20], np.array([100, 77]), 4, 2, 128, 16, bits, True)


@pytest.mark.parametrize("bf16,o_bf16", [(True, True), (False, False), (True, False), (False, True)])
@pytest.mark.parametrize("new,total", [([300], [300]), ([129, 1, 64], [129, 500, 700]), ([17, 200], [300, 200])])
def test_attention_prompts(H, new, total, bf16, o_bf16):
    """Prompts, chunks over a cached prefix, and single rows in one batch."""
    _attend(H, np.random.default_rng(len(new)), new, np.array(total), 8, 2, 128, 64, 8, bf16, o_bf16)


@pytest.mark.parametrize("D,block", [(32, 16), (64, 16), (64, 128), (128, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("Hq,Hkv", [(3, 3), (10, 2), (16, 1)])
def test_attention_prompt_shapes(H, D, block, Hq, Hkv):
    _attend(H, np.random.default_rng(D + Hq), [150, 37, 260], np.array([150, 137, 400]), Hq, Hkv, D, block, 8, True)


@pytest.mark.parametrize("o_bf16", [True, False])
@pytest.mark.parametrize("D,Hq,Hkv,new,total", [(128, 8, 2, [64], [2100]), (128, 8, 2, [130, 2], [1500, 3700]),
                                                (64, 6, 1, [700], [700]), (64, 4, 4, [300, 0, 90], [4200, 0, 90]),
                                                (128, 16, 4, [257], [2000])])
def test_attention_prompts_over_many_ctas(H, D, Hq, Hkv, new, total, o_bf16):
    """Few row tiles over long contexts, which several CTAs share: rows that see nothing of a CTA's tokens, requests
    too short to be shared beside long ones."""
    _attend(H, np.random.default_rng(D + sum(new)), new, np.array(total), Hq, Hkv, D, 64, 8, True, o_bf16, pad=3)


def test_attention_rows_without_tokens_and_padding(H):
    """Requests of no rows, lengths of 0, more rows than tokens, rows before and behind the requests."""
    rng = np.random.default_rng(5)
    got, want = _attend(H, rng, [0, 2, 5, 0, 1, 3], np.array([50, 0, 3, 0, 64, -4]), 4, 2, 64, 16, 8, True, pad=9, first=3)
    assert np.all(want[3:5] == 0) and np.all(got[3:7] == 0) and np.any(got[7] != 0)


def test_attention_pages_outside_the_cache(H):
    """Absent pages (any index outside the cache) are not seen, wherever they stand; a request of none gives 0."""
    def mend(table, kc, ks, vc, vs, q):
        n = len(kc)
        table[0, [0, 3]] = -1, n
        table[1, 1] = 2 ** 31 - 1
        table[2, :] = -2 ** 31
        table[3, 5] = n + 17
    rng = np.random.default_rng(6)
    for new in ([1] * 4, [40, 1, 100, 30]):
        got, want = _attend(H, rng, new, np.array([100, 48, 200, 150]), 4, 2, 128, 16, 8, True, mend=mend)
        lo = sum(new[:2])
        assert np.all(got[lo:lo + new[2]] == 0)


@pytest.mark.parametrize("o_bf16", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_rows_that_see_no_token(H, D, o_bf16):
    """Hundreds of rows over no token, or over far fewer than there are rows, beside a whole prompt: whole row tiles see
    nothing and give exactly 0, in every one of many runs."""
    import torch
    rng = np.random.default_rng(63 + D)
    new, total = [300, 400, 350], np.array([0, 60, 350])
    got, want = _attend(H, rng, new, total, 8, 2, D, 64, 8, True, o_bf16)
    assert np.all(want[:640] == 0) and np.all(got[:640] == 0) and np.any(got[640:] != 0)
    cache = [_dev(a) for a in _cache(rng, 20, 2, 64, D, 8) + _cache(rng, 20, 2, 64, D, 8)]
    q = _as(rng.standard_normal((1050, 8, D)), True)
    o = torch.empty((1050, 8, D), dtype=torch.bfloat16 if o_bf16 else torch.float32, device="cuda")
    ws = torch.empty((H.hbl_kv_attention_workspace_bytes(1050, 8, 2, D, 3),), dtype=torch.uint8, device="cuda")
    rows, table = _i32([0, 300, 700, 1050]), _i32(np.arange(18).reshape(3, 6))
    first = None
    for i in range(60):
        o.fill_(3.0)
        H.hbl_kv_attention(q, rows, _i32(total), table, *cache, o=o, workspace=ws)
        first = o.clone() if first is None else first
        assert bool((o[:640] == 0).all()) and torch.equal(o, first), i


def test_attention_longer_than_its_table(H):
    """A length past the table: the tokens that the table has are seen."""
    rng = np.random.default_rng(7)
    n, block, D = 6, 16, 64
    (kc, ks), (vc, vs) = _cache(rng, n, 1, block, D, 8), _cache(rng, n, 1, block, D, 8)
    table, total, rows = np.array([[4, 1]]), np.array([100]), np.array([0, 2])
    q = _values(rng.standard_normal((2, 1, D)), True)
    want, *sizes = ref.attention(q, rows, total, table, ref.values(kc, ks, 8), ref.values(vc, vs, 8), D ** -0.5)
    got = H.hbl_kv_attention(_as(q, True), _i32(rows), _i32(total), _i32(table), _dev(kc), _dev(ks), _dev(vc), _dev(vs))
    assert np.all(np.abs(_np(got) - want) <= ref.attention_tolerance(want, *sizes, 32, False, False))


def test_attention_ignores_what_is_masked(H):
    """What lies behind a request's tokens (codes, and the scales of blocks it does not reach) does not matter: the
    outputs are bit for bit those of a cache that holds NaN scales and other codes there."""
    import torch
    rng = np.random.default_rng(9)
    Hq, Hkv, D, block = 8, 2, 128, 16
    total, new = np.array([5, 130, 48]), [1, 40, 1]
    rows = np.concatenate([[0], np.cumsum(new)])
    table = np.arange(3 * 12).reshape(3, 12)
    (kc, ks), (vc, vs) = _cache(rng, 36, Hkv, block, D, 8), _cache(rng, 36, Hkv, block, D, 8)
    q = _as(rng.standard_normal((int(rows[-1]), Hq, D)), True)
    outs = []
    for spoil in (False, True):
        if spoil:
            for b in range(3):
                last = -(-total[b] // block)
                ks[table[b, last:]] = np.nan
                vs[table[b, last:]] = np.inf
                kc[table[b, last:]] ^= 0xFF
                if total[b] % block:
                    kc[table[b, last - 1], :, total[b] % block:] ^= 0x5A
                    vc[table[b, last - 1], :, total[b] % block:] ^= 0x77
        outs.append(H.hbl_kv_attention(q, _i32(rows), _i32(total), _i32(table), *(_dev(a) for a in (kc, ks, vc, vs))))
    assert torch.equal(outs[0], outs[1]) and bool(torch.isfinite(outs[0]).all())


@pytest.mark.parametrize("bf16", [True, False])
def test_attention_behind_a_long_run_of_zeros(H, bf16):
    """More than ten thousand tokens of zero keys and values in one warp's share, then blocks with values: the sum of
    the zeros' weights stays finite, and the few values are not lost."""
    rng = np.random.default_rng(64)
    B, heads, D, block, pages = 64, 8, 256, 128, 128
    (kc, ks), (vc, vs) = _cache(rng, 10, heads, block, D, 8), _cache(rng, 10, heads, block, D, 8)
    ks[0], vs[0] = 0.0, 0.0
    table = np.zeros((B, pages), np.int64)
    table[:, -2:] = rng.integers(1, 10, (B, 2))
    total = pages * block - rng.integers(0, 100, B)
    q = _values(rng.standard_normal((B, heads, D)), bf16)
    got = _np(H.hbl_kv_attention(_as(q, bf16), _i32(range(B + 1)), _i32(total), _i32(table), *(_dev(a) for a in (kc, ks, vc, vs))))
    k, v = ref.values(kc, ks, 8), ref.values(vc, vs, 8)
    for b in (0, 1, 17, 40, 63):
        want, *sizes = ref.attention(q[b:b + 1], [0, 1], total[b:b + 1], table[b:b + 1], k, v, D ** -0.5, vs)
        assert np.all(np.abs(got[b] - want[0]) <= ref.attention_tolerance(want, *sizes, pages * block, not bf16, not bf16)[0])


@pytest.mark.parametrize("new", [1, 90])
@pytest.mark.parametrize("bf16", [True, False])
def test_attention_of_zeros_beside_large_values(H, new, bf16):
    """Blocks of zeros keep their share of the sum beside values of 2^48, and values of 2^-40 are not zeros."""
    def mend(table, kc, ks, vc, vs, q):
        vs[table[0, :5]] = 0.0
        vs[table[0, 5:]] *= np.float32(2.0 ** 48)
        vs[table[1]] *= np.float32(2.0 ** -40)
    _attend(H, np.random.default_rng(65 + new), [new, new], np.array([150, 130]), 8, 2, 64, 16, 8, bf16, mend=mend)


@pytest.mark.parametrize("new", [1, 90])
@pytest.mark.parametrize("bf16", [True, False])
def test_attention_of_the_largest_values(H, new, bf16):
    """Values up to 2^118, alone and beside blocks of zeros."""
    def mend(table, kc, ks, vc, vs, q):
        vs *= np.float32(2.0 ** 115)
        vs[table[0, ::2]] = 0.0
    _attend(H, np.random.default_rng(68 + new), [new, new], np.array([150, 130]), 8, 2, 64, 16, 8, bf16, mend=mend)


@pytest.mark.parametrize("new", [1, 70])
def test_attention_of_uneven_scales(H, new):
    """Blocks of zero, tiny and large gamma, and scores far apart (a key that takes nearly all the weight while its
    value block is zero): the small weights that make the output keep their precision."""
    def mend(table, kc, ks, vc, vs, q):
        ks[table[0, 2]], vs[table[0, 2]] = 0.0, 0.0
        vs[table[0, 1]] = 1e-6
        vs[table[0, 4]] = 3e4
        vs[table[0, 0]] = 0.0
        ks[table[0, 0]] *= 8.0
        vs[table[1, :2]] = 0.0
    _attend(H, np.random.default_rng(new), [new, new], np.array([120, 100]), 4, 2, 64, 16, 8, True, mend=mend, k_gain=2.0)


def test_attention_one_bad_row_stays_alone(H):
    """NaN and infinity in one row of q: that row's outputs are not finite, all others are as without it."""
    import torch
    rng = np.random.default_rng(10)
    table, total, rows = np.arange(20).reshape(2, 10), np.array([150, 160]), np.array([0, 30, 60])
    cache = [_dev(a) for a in _cache(rng, 20, 2, 16, 64, 8) + _cache(rng, 20, 2, 16, 64, 8)]
    q = _as(rng.standard_normal((60, 4, 64)), True)
    clean = H.hbl_kv_attention(q, _i32(rows), _i32(total), _i32(table), *cache)
    bad = q.clone()
    bad[7, 1, 3] = float("nan")
    bad[40, 2, 9] = float("inf")
    got = H.hbl_kv_attention(bad, _i32(rows), _i32(total), _i32(table), *cache)
    hit = torch.zeros((60, 4), dtype=torch.bool, device="cuda")
    hit[7, 1] = hit[40, 2] = True
    assert torch.equal(got[~hit], clean[~hit])
    assert not bool(torch.isfinite(got[7, 1]).any())


def test_attention_scale(H):
    rng = np.random.default_rng(11)
    for s in (0.02, 1.0, 0.0, -0.1):
        _attend(H, rng, [1, 33], np.array([90, 60]), 4, 4, 64, 16, 8, True, scale=s)


def test_attention_long(H):
    """Enough tokens that a request is split over many CTAs, and offsets that pass 32 bits in the cache: a request's
    pages at both ends of a cache of more than 4 GiB."""
    import torch
    rng = np.random.default_rng(13)
    Hkv, D, block = 8, 128, 128
    n = 33000                                                    # x 128 KiB = 4.3 GB each for K and V
    kc = torch.empty((n, Hkv, block, D), dtype=torch.uint8, device="cuda")
    vc = torch.empty_like(kc)
    ks, vs = (torch.ones((n, Hkv), device="cuda") for _ in range(2))
    total = np.array([9000, 20000])
    table = np.full((2, 160), -1)
    pages = np.unique(np.r_[rng.integers(0, 300, 400), rng.integers(n - 300, n, 400)])
    pages = rng.permutation(pages)[:71 + 157]
    table[0, :71], table[1, :157] = pages[:71], pages[71:]
    small_k, small_ks = _cache(rng, len(pages), Hkv, block, D, 8)
    small_v, small_vs = _cache(rng, len(pages), Hkv, block, D, 8)
    at = _dev(pages)
    kc[at], vc[at], ks[at], vs[at] = _dev(small_k), _dev(small_v), _dev(small_ks), _dev(small_vs)
    q = _values(rng.standard_normal((2, 16, D)), True)
    got = _np(H.hbl_kv_attention(_as(q, True), _i32([0, 1, 2]), _i32(total), _i32(table), kc, ks, vc, vs))
    small = np.full_like(table, -1)
    small[0, :71], small[1, :157] = np.arange(71), np.arange(71, 228)
    want, *sizes = ref.attention(q, [0, 1, 2], total, small, ref.values(small_k, small_ks, 8),
                                      ref.values(small_v, small_vs, 8), D ** -0.5)
    tol = ref.attention_tolerance(want, *sizes, 20000, False, False)
    assert np.all(np.abs(got - want) <= tol)


@pytest.mark.parametrize("new,total,Hq,Hkv", [([900, 900], [2448, 2400], 16, 2), ([1] * 4, [32768, 30000, 32000, 31111], 8, 1)])
def test_attention_of_float_rows_over_many_tokens(H, new, total, Hq, Hkv):
    """Long sums keep float's bits.  With values of either sign an output is a random sum, as its errors are: a score
    of less than 16 in log2 units rounds twice (half steps of 2^-21, rms 2^-21 / sqrt(3) each, times ln 2: 2.7e-7 of a
    weight), the exponential and the two-part weights 2^-22 each, about eighty additions of 2^-24 / sqrt(3) each
    3.1e-7: together 5.3e-7 of the whole's norm, and 2^-20 is above it."""
    got, want = _attend(H, np.random.default_rng(17), new, np.array(total), Hq, Hkv, 64, 32, 8, False)
    assert np.linalg.norm(got - want) <= 2.0 ** -20 * np.linalg.norm(want)


@pytest.mark.parametrize("B,new", [(1500, 1), (4096, 1), (600, 9)])
def test_attention_many_requests(H, B, new):
    rng = np.random.default_rng(B)
    total = rng.integers(0, 70, B)
    rows = rng.integers(0, new + 1, B)
    rows[0] = new
    _attend(H, rng, rows.tolist(), total, 2, 1, 64, 16, 8, True)


def test_attention_over_shared_and_repeated_blocks(H):
    """One block in several requests' tables, and twice in one: a shared prefix, read by all."""
    def mend(table, kc, ks, vc, vs, q):
        table[1, :4] = table[0, :4]
        table[2, 1] = table[2, 0]
    for new in ([1, 1, 1], [90, 120, 64]):
        _attend(H, np.random.default_rng(sum(new)), new, np.array([130, 150, 140]), 8, 2, 128, 16, 8, True, mend=mend)


def test_prompt_attention_in_a_graph(H):
    """Chunks of prompts, captured once and replayed with other lengths, rows and pages (the same batch size)."""
    import torch
    rng = np.random.default_rng(31)
    Hq, Hkv, D, block, n, T = 16, 4, 128, 32, 400, 700
    cache = [_dev(a) for a in _cache(rng, n, Hkv, block, D, 8) + _cache(rng, n, Hkv, block, D, 8)]
    q, o = _as(rng.standard_normal((T, Hq, D)), True), torch.zeros((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    rows, total, table = _i32([0, 300, 700]), _i32([2000, 900]), _i32(rng.integers(0, n, (2, 90)))
    ws = torch.empty((H.hbl_kv_attention_workspace_bytes(T, Hq, Hkv, D, 2),), dtype=torch.uint8, device="cuda")
    call = lambda out, w: H.hbl_kv_attention(q, rows, total, table, *cache, o=out, workspace=w)  # noqa: E731
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        call(o, ws)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call(o, ws)
    other = torch.empty_like(ws)
    for r, t in (([0, 300, 700], [2000, 900]), ([0, 64, 65], [64, 2500]), ([0, 0, 690], [5, 2800]), ([10, 500, 700], [490, 200])):
        rows.copy_(_i32(r))
        total.copy_(_i32(t))
        table.copy_(_i32(rng.integers(-3, n + 3, (2, 90))))
        q.copy_(_as(rng.standard_normal((T, Hq, D)), True))
        want = torch.full_like(o, 3.0)
        o.fill_(3.0)
        call(want, other)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)
        ref_o, *sizes = ref.attention(_np(q), r, t, to_host(table), ref.values(to_host(cache[0]), to_host(cache[1]), 8),
                                      ref.values(to_host(cache[2]), to_host(cache[3]), 8), D ** -0.5, to_host(cache[3]))
        mine = ~np.isnan(ref_o[:, 0, 0])
        tol = ref.attention_tolerance(ref_o, *sizes, max(t), False, False)
        assert np.all(np.abs(_np(o) - ref_o)[mine] <= tol[mine]) and np.all(_np(o)[~mine] == 3.0)
    assert H.hbl_last_device_error() == H.HBL_OK


def test_prompt_attention_on_two_streams(H):
    """Two prompts at once (each wants all of an SM's tensor memory) with workspaces of their own, beside a product
    that uses tensor memory too."""
    import torch
    rng = np.random.default_rng(32)
    Hq, Hkv, D, n = 16, 4, 128, 300
    cache = [_dev(a) for a in _cache(rng, n, Hkv, 64, D, 8) + _cache(rng, n, Hkv, 64, D, 8)]
    args = (_i32([0, 900]), _i32([4000]), _i32(rng.permutation(n)[:64].reshape(1, 64)), *cache)
    qs = [_as(rng.standard_normal((900, Hq, D)), True) for _ in range(2)]
    want = [H.hbl_kv_attention(q, *args) for q in qs]
    A, W = (torch.randint(-8, 8, s, device="cuda", dtype=torch.int8) for s in ((512, 2048), (1024, 2048)))
    acc = H.hbl_gemm_i8_i32(A, W)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    size = H.hbl_kv_attention_workspace_bytes(900, Hq, Hkv, D, 1)
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [[torch.zeros_like(want[0]) for _ in range(4)] for _ in range(2)]
    accs = [torch.zeros_like(acc) for _ in range(4)]
    torch.cuda.synchronize()
    for i in range(4):
        for j in (0, 1):
            with torch.cuda.stream(streams[j]):
                H.hbl_kv_attention(qs[j], *args, o=outs[j][i], workspace=ws[j])
        with torch.cuda.stream(streams[2]):
            H.hbl_gemm_i8_i32(A, W, acc=accs[i])
    torch.cuda.synchronize()
    for i in range(4):
        assert torch.equal(outs[0][i], want[0]) and torch.equal(outs[1][i], want[1]) and torch.equal(accs[i], acc)
    assert H.hbl_last_device_error() == H.HBL_OK


def test_attention_is_reproducible(H):
    import torch
    rng = np.random.default_rng(14)
    total, new = rng.integers(1, 3000, 40), [1] * 40
    table = rng.permutation(40 * 50).reshape(40, 50)
    cache = [_dev(a) for a in _cache(rng, 2000, 2, 64, 128, 8) + _cache(rng, 2000, 2, 64, 128, 8)]
    q = _as(rng.standard_normal((40, 8, 128)), True)
    first = H.hbl_kv_attention(q, _i32(range(41)), _i32(total), _i32(table), *cache)
    for _ in range(3):
        assert torch.equal(first, H.hbl_kv_attention(q, _i32(range(41)), _i32(total), _i32(table), *cache))


# ------------------------------------------------------------------ residual, RMSNorm, quantizer

@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (5, 256), (9, 1040), (2, 2560), (4, 4096), (150, 2064), (3, 16400),
                                 (2, 32768)])
def test_add_rms_quant(H, M, K, bits, bf16):
    import torch
    rng = np.random.default_rng(M * K + bits)
    x, r = _values(rng.standard_normal((M, K)) * 3.0, bf16), _values(rng.standard_normal((M, K)), bf16)
    x[0, K // 2] = 200.0
    gain = (1.0 + 0.2 * rng.standard_normal(K)).astype(np.float32)
    if M > 2:
        x[1] = 0.0
        r[1] = 0.0                       # a row of zeros
    for use_r, use_gain in ((True, True), (False, False)):
        h, t, q, s = ref.add_rms_quant(x, r if use_r else None, gain if use_gain else None, bits, bf16)
        dh, check_h = _guarded((M, K), torch.bfloat16 if bf16 else torch.float32)
        dq, check_q = _guarded((M, K), torch.int8)
        H.hbl_add_rms_quant(_as(x, bf16), bits, residual=_as(r, bf16) if use_r else None,
                            gain=_dev(gain) if use_gain else None, h=dh, codes=dq, scales=(ds := torch.empty(M, device="cuda")))
        check_h("h")
        check_q("codes")
        assert np.array_equal(_np(dh), h)
        assert np.array_equal(to_host(ds), s) and np.array_equal(to_host(dq), q)


def test_add_rms_quant_in_place(H):
    """h over the residual (a residual stream updated in place), and over x."""
    import torch
    rng = np.random.default_rng(2)
    x, r = (_as(rng.standard_normal((70, 2560)), True) for _ in range(2))
    gain = _dev(rng.standard_normal(2560).astype(np.float32))
    h, q, s = H.hbl_add_rms_quant(x, 8, residual=r, gain=gain)
    for over in (0, 1):
        a, b = x.clone(), r.clone()
        h2, q2, s2 = H.hbl_add_rms_quant(a, 8, residual=b, gain=gain, h=(a, b)[over])
        assert h2 is (a, b)[over] and torch.equal(h2, h) and torch.equal(q2, q) and torch.equal(s2, s)
        assert torch.equal((b, a)[over], (r, x)[over])


def test_add_rms_quant_against_norm_quant(H):
    """Without residual and gain it is hbl_norm_quant's RMSNorm: the same values up to its float sum."""
    rng = np.random.default_rng(3)
    x = _as(rng.standard_normal((64, 1024)), True)
    _, q, s = H.hbl_add_rms_quant(x, 8)
    q0, s0 = H.hbl_norm_quant(x, 8, H.HBL_NORM_RMS)
    # K = 1024 squares in a float sum: at most 2^-14 relative (1024 half steps), half of it in the root
    assert np.all(np.abs(_np(s) - _np(s0)) <= 2.0 ** -15 * _np(s) * 1.001)
    assert np.mean(to_host(q) != to_host(q0)) <= 0.01 and np.abs(_np(q) - _np(q0)).max() <= 1


def _grad_tolerance(size, K, M, g_x, out_bf16):
    """Counted float errors of g_x: two row sums of K terms (K half steps of 2^-24 at the worst order, in fact taken in
    partial sums of at most K / 256 + 40 terms), ten more operations, then the output's rounding."""
    return (K / 256 + 50) * 2.0 ** -24 * size + (2.0 ** -8 if out_bf16 else 2.0 ** -24) * np.abs(g_x)


@pytest.mark.parametrize("bf16,gt_bf16", [(True, True), (False, False), (True, False), (False, True)])
@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (7, 1040), (130, 256), (33, 2560), (1000, 4096), (5, 16400), (2, 32768)])
def test_add_rms_backward(H, M, K, bf16, gt_bf16):
    import torch
    rng = np.random.default_rng(M + K)
    h, g_h = _values(rng.standard_normal((M, K)) * 2.0, bf16), _values(rng.standard_normal((M, K)), bf16)
    g_t = _values(rng.standard_normal((M, K)), gt_bf16)
    if M > 2:
        h[1] = 0.0
    gain = (1.0 + 0.2 * rng.standard_normal(K)).astype(np.float32)
    for with_gain, with_h in ((True, True), (False, False), (True, False)):
        wx, wg, size = ref.add_rms_backward(h, gain if with_gain else None, g_t, g_h if with_h else None)
        g_x, check = _guarded((M, K), torch.bfloat16 if bf16 else torch.float32)
        g_gain, check_g = _guarded((K,), torch.float32)
        ws, check_ws = _guarded((H.hbl_add_rms_quant_backward_workspace_bytes(M, K),), torch.uint8)
        H.hbl_add_rms_quant_backward(_as(h, bf16), _as(g_t, gt_bf16), gain=_dev(gain) if with_gain else None,
                                     g_h=_as(g_h, bf16) if with_h else None, g_x=g_x, g_gain=g_gain if with_gain else None,
                                     workspace=ws)
        check("g_x")
        check_g("g_gain")
        check_ws("workspace")
        assert np.all(np.abs(_np(g_x) - wx) <= _grad_tolerance(size, K, M, wx, bf16))
        if with_gain:
            # M terms in partial sums of at most M / 128 + 300 terms, each with the error of its n
            n = np.abs(h / np.sqrt((h.astype(np.float64) ** 2).mean(1, keepdims=True) + 1e-5) * g_t).sum(0)
            assert np.all(np.abs(_np(g_gain) - wg) <= (K / 256 + M / 128 + 350) * 2.0 ** -24 * n)


MANY = [(9600, 48), (7300, 1040), (3600, 1536), (2500, 4080), (1300, 8176), (500, 16368)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("M,K", MANY)
def test_add_rms_quant_of_many_rows(H, M, K, bf16, bits):
    """Batches long enough for the grid that stays: the bits of the same rows in short batches; in place too."""
    import torch
    rng = np.random.default_rng(M)
    x, r = (_as(_values(rng.standard_normal((M, K)), bf16), bf16) for _ in range(2))
    gain = _dev((1.0 + 0.2 * rng.standard_normal(K)).astype(np.float32))
    h, q, s = H.hbl_add_rms_quant(x, bits, residual=r, gain=gain)
    for i in list(range(0, M, max(1, M // 7))) + [M - 30]:
        j = min(i + 30, M)
        h1, q1, s1 = H.hbl_add_rms_quant(x[i:j], bits, residual=r[i:j], gain=gain)
        assert torch.equal(h[i:j], h1) and torch.equal(q[i:j], q1) and torch.equal(s[i:j], s1)
    h2, q2, s2 = H.hbl_add_rms_quant(x, bits, residual=r, gain=gain, h=r)
    assert h2 is r and torch.equal(h2, h) and torch.equal(q2, q) and torch.equal(s2, s)


@pytest.mark.parametrize("bf16,gt_bf16", [(True, True), (False, False), (True, False), (False, True)])
@pytest.mark.parametrize("M,K", MANY)
def test_add_rms_backward_of_many_rows(H, M, K, bf16, gt_bf16):
    """The wide blocks: a row's gradient has the bits that it has in a short batch, whatever block it falls to, in place
    too; the gain's is the sum over all rows."""
    import torch
    rng = np.random.default_rng(M + 1)
    h, g_h = (_as(_values(rng.standard_normal((M, K)), bf16), bf16) for _ in range(2))
    g_t = _as(_values(rng.standard_normal((M, K)), gt_bf16), gt_bf16)
    gain = _dev((1.0 + 0.2 * rng.standard_normal(K)).astype(np.float32))
    ws, check = _guarded((H.hbl_add_rms_quant_backward_workspace_bytes(M, K),), torch.uint8)
    g_x, g_gain = H.hbl_add_rms_quant_backward(h, g_t, gain=gain, g_h=g_h, workspace=ws)
    check("workspace")
    for i in list(range(0, M, max(1, M // 7))) + [M - 30]:
        j = min(i + 30, M)
        assert torch.equal(g_x[i:j], H.hbl_add_rms_quant_backward(h[i:j], g_t[i:j], gain=gain, g_h=g_h[i:j])[0])
    n = h.double() / torch.sqrt(h.double().square().mean(1, keepdim=True) + 1e-5)
    terms = n * g_t.double()
    # M terms in partial sums of at most M / 128 + 300 terms, each with the error of its n
    off = (g_gain.double() - terms.sum(0)).abs()
    assert bool((off <= (K / 256 + M / 128 + 350) * 2.0 ** -24 * terms.abs().sum(0)).all())
    got, _ = H.hbl_add_rms_quant_backward(h, g_t, gain=gain, g_h=g_h, g_x=g_h)
    assert got is g_h and torch.equal(got, g_x)


def test_add_rms_backward_gain_over_ctas(H):
    """The partial sums of CTAs are added in double: large ones of either sign that cancel leave the small ones whole.
    With h of +-1 the normalised values of all rows are equal in size, so +-2^30 cancel exactly; what remains is off by
    the roundings of rstd (three operations), of a product and of the result, each half a step."""
    import torch
    M, K = 128, 1024                                            # at most a row a CTA
    rng = np.random.default_rng(66)
    h = np.sign(rng.standard_normal((M, K))).astype(np.float32)
    h[96] = h[0]
    g_t = rng.uniform(0.5, 1.5, (M, K)).astype(np.float32)
    g_t[0], g_t[96] = 2.0 ** 30, -2.0 ** 30
    _, got = H.hbl_add_rms_quant_backward(_dev(h), _dev(g_t), g_gain=torch.empty(K, device="cuda"))
    small = np.delete(h.astype(np.float64) * g_t, (0, 96), 0) / np.sqrt(1.0 + 1e-5)
    tol = 5 * 2.0 ** -24 * np.abs(small).sum(0) + 2.0 ** -52 * 2.0 ** 31 * 8     # and a few double additions of 2^30
    assert np.all(np.abs(_np(got) - small.sum(0)) <= tol)


def test_add_rms_backward_in_place_and_alone(H):
    """g_x over g_h; without a gain no gain gradient; a gain gradient without a gain is the sum all the same."""
    import torch
    rng = np.random.default_rng(4)
    h, g_t, g_h = (_as(rng.standard_normal((300, 1040)), True) for _ in range(3))
    gain = _dev(rng.standard_normal(1040).astype(np.float32))
    want, want_gain = H.hbl_add_rms_quant_backward(h, g_t, gain=gain, g_h=g_h)
    over = g_h.clone()
    got, got_gain = H.hbl_add_rms_quant_backward(h, g_t, gain=gain, g_h=over, g_x=over)
    assert got is over and torch.equal(got, want) and torch.equal(got_gain, want_gain)
    assert H.hbl_add_rms_quant_backward(h, g_t)[1] is None
    _, alone = H.hbl_add_rms_quant_backward(h, g_t, g_gain=torch.empty(1040, device="cuda"))
    assert torch.equal(alone, want_gain)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("M,K,size", [(9, 4096, 2e18), (700, 2560, 2e18), (5, 32768, 2e18), (9, 1040, 1e-30)])
def test_add_rms_backward_of_large_and_small_rows(H, M, K, size, bf16):
    """Rows whose squares add up past float's range while their mean, and so the forward's rstd, does not; and tiny ones.
    The forward's codes and the gradient are those of the definition all the same."""
    rng = np.random.default_rng(K)
    h, g_t = _values(rng.standard_normal((M, K)) * size, bf16), _values(rng.standard_normal((M, K)), bf16)
    gain = (1.0 + 0.2 * rng.standard_normal(K)).astype(np.float32)
    _, _, q, s = ref.add_rms_quant(h, None, gain, 8, bf16)
    _, got_q, got_s = H.hbl_add_rms_quant(_as(h, bf16), 8, gain=_dev(gain))
    assert np.array_equal(to_host(got_q), q) and np.array_equal(to_host(got_s), s)
    wx, wg, terms = ref.add_rms_backward(h, gain, g_t, None)
    g_x, g_gain = H.hbl_add_rms_quant_backward(_as(h, bf16), _as(g_t, bf16), gain=_dev(gain))
    assert np.all(np.abs(_np(g_x) - wx) <= _grad_tolerance(terms, K, M, wx, bf16))
    n = np.abs(h / np.sqrt((h.astype(np.float64) ** 2).mean(1, keepdims=True) + 1e-5) * g_t).sum(0)
    assert np.all(np.abs(_np(g_gain) - wg) <= (K / 256 + M / 128 + 350) * 2.0 ** -24 * n)


def test_add_rms_backward_against_differences(H):
    """g_x of the kernel (float) against central differences of the 64-bit value."""
    rng = np.random.default_rng(5)
    M, K, d = 4, 256, 1e-6
    h, g_t = rng.standard_normal((2, M, K)).astype(np.float32)
    gain = (1.0 + 0.2 * rng.standard_normal(K)).astype(np.float32)
    g_x, g_gain = H.hbl_add_rms_quant_backward(_dev(h), _dev(g_t), gain=_dev(gain))
    _, _, size = ref.add_rms_backward(h, gain, g_t, None)
    for m, k in ((0, 0), (1, 100), (2, 255), (3, 31)):
        e = np.zeros((M, K))
        e[m, k] = d
        slope = ((ref.rms_value(h + e, gain) - ref.rms_value(h - e, gain)) * g_t).sum() / (2 * d)
        assert abs(_np(g_x)[m, k] - slope) <= 52 * 2.0 ** -24 * size[m, k] + 1e-8


# ------------------------------------------------------------------ together

def _layer_state(rng, B, block, width, hidden, heads, kv_heads, D):
    import torch
    return dict(
        table=torch.full((B, width), -1, dtype=torch.int32, device="cuda"),
        free=_i32(rng.permutation(B * width)), taken=_i32([0]), cached=torch.zeros(B, dtype=torch.int32, device="cuda"),
        cache=[torch.zeros((B * width, kv_heads, block, D), dtype=torch.uint8, device="cuda"),
               torch.zeros((B * width, kv_heads), device="cuda"),
               torch.zeros((B * width, kv_heads, block, D), dtype=torch.uint8, device="cuda"),
               torch.zeros((B * width, kv_heads), device="cuda")])


def test_a_layer_step_by_step(H):
    """One attention sublayer as it is served: a prompt step and decode steps of residual + norm + quantizer, ternary
    QKV product, plan, cache write, attention, and the H-BitLinear output product, against the plain forms at every
    hand-over (each operator's inputs are the framework's own outputs so far)."""
    import torch
    rng = np.random.default_rng(21)
    B, block, width, hidden, heads, kv_heads, D = 3, 16, 8, 512, 8, 2, 64
    N = (heads + 2 * kv_heads) * D
    s = _layer_state(rng, B, block, width, hidden, heads, kv_heads, D)
    packed, alpha = H.hbl_pack_ternary(_as(rng.standard_normal((N, hidden)) * 0.02, True))
    w8 = H.hbl_widen_ternary(packed, hidden)
    wo, wo_alpha = H.hbl_pack_ternary(_as(rng.standard_normal((hidden, heads * D)) * 0.02, True))
    gain = _dev((1.0 + 0.1 * rng.standard_normal(hidden)).astype(np.float32))
    for added in ([37, 5, 20], [1, 1, 1], [1, 0, 3], [1, 1, 1]):
        T = sum(added) + 2
        x, stream = (_as(rng.standard_normal((T, hidden)), True) for _ in range(2))
        before = [to_host(t).copy() for t in (s["cached"], s["table"], s["taken"])] + [to_host(t).copy() for t in s["cache"]]
        total, rows, slots, pos, taken = H.hbl_kv_plan(s["cached"], _i32(added), s["free"], s["taken"], s["table"], block, T)
        h, codes, scales = H.hbl_add_rms_quant(x, 8, residual=stream, gain=gain)
        qkv = H.hbl_gemm_dequant(codes, w8, scales, alpha)
        cut = lambda i, n: qkv[:, i * D:(i + n) * D].unflatten(1, (n, D))  # noqa: E731
        q, k, v = cut(0, heads), cut(heads, kv_heads), cut(heads + kv_heads, kv_heads)
        H.hbl_kv_append(k, v, slots, *s["cache"])
        o = H.hbl_kv_attention(q, rows, total, s["table"], *s["cache"])
        y = H.hbl_forward(o.view(T, heads * D), wo, wo_alpha, hidden, 4)
        # the plain forms at each hand-over
        p = ref.plan(before[0], added, to_host(s["free"]), before[2][0], before[1], block, T)
        for g, w in zip((s["table"], total, rows, slots, pos, taken), p):
            assert np.array_equal(to_host(g).reshape(-1), np.asarray(w).reshape(-1))
        wk = ref.append(_np(k), p[3], before[3], before[4], 8)
        wv = ref.append(_np(v), p[3], before[5], before[6], 8)
        for g, w in zip(s["cache"], wk + wv):
            assert np.array_equal(to_host(g), w)
        want, *sizes = ref.attention(_np(q), p[2], p[1], p[0], ref.values(*wk, 8), ref.values(*wv, 8), D ** -0.5)
        want[np.isnan(want)] = 0.0
        assert np.all(np.abs(_np(o) - want) <= ref.attention_tolerance(want, *sizes, int(max(p[1])), False, False))
        assert bool(torch.isfinite(y).all()) and y.shape == (T, hidden)
        s["cached"], s["taken"] = total, taken


def test_decode_step_in_a_graph(H):
    """A decode step (plan, norm, append, attention) captured once and replayed as lengths grow gives what the calls
    give outside a graph."""
    import torch
    rng = np.random.default_rng(22)
    B, block, width, hidden, heads, kv_heads, D = 5, 16, 12, 256, 8, 2, 64

    def state():
        g = np.random.default_rng(23)
        s = _layer_state(g, B, block, width, hidden, heads, kv_heads, D)
        s["cached"].copy_(_i32([0, 15, 16, 40, 7]))
        ids = to_host(s["free"])
        at = 0
        for b, n in enumerate([0, 1, 1, 3, 1]):
            s["table"][b, :n] = _i32(ids[at:at + n])
            at += n
        s["taken"].fill_(at)
        for i in (1, 3):
            s["cache"][i].fill_(0.5)
        s["one"] = torch.ones(B, dtype=torch.int32, device="cuda")
        s["x"] = torch.zeros((B, hidden), dtype=torch.bfloat16, device="cuda")
        s["qkv"] = torch.zeros((B, heads + 2 * kv_heads, D), dtype=torch.bfloat16, device="cuda")
        s["total"], s["rows"] = torch.empty_like(s["one"]), torch.empty(B + 1, dtype=torch.int32, device="cuda")
        s["slots"], s["pos"], s["out"] = torch.empty_like(s["one"]), torch.empty_like(s["one"]), torch.empty_like(s["taken"])
        s["o"] = torch.zeros((B, heads, D), dtype=torch.bfloat16, device="cuda")
        s["ws"] = torch.empty((H.hbl_kv_attention_workspace_bytes(B, heads, kv_heads, D, B),), dtype=torch.uint8, device="cuda")
        s["nq"] = H.hbl_add_rms_quant(s["x"], 8)
        return s

    def step(s):
        H.hbl_kv_plan(s["cached"], s["one"], s["free"], s["taken"], s["table"], block, B, s["total"], s["rows"], s["slots"],
                      s["pos"], s["out"])
        H.hbl_add_rms_quant(s["x"], 8, residual=s["x"], h=s["nq"][0], codes=s["nq"][1], scales=s["nq"][2])
        q, k, v = s["qkv"][:, :heads], s["qkv"][:, heads:heads + kv_heads], s["qkv"][:, heads + kv_heads:]
        H.hbl_kv_append(k, v, s["slots"], *s["cache"])
        H.hbl_kv_attention(q, s["rows"], s["total"], s["table"], *s["cache"], o=s["o"], workspace=s["ws"])
        s["cached"].copy_(s["total"])
        s["taken"].copy_(s["out"])

    eager, graphed = state(), state()
    stream = torch.cuda.Stream()
    spare = state()
    with torch.cuda.stream(stream):
        step(spare)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step(graphed)
    for i in range(20):
        x, qkv = _as(rng.standard_normal((B, hidden)), True), _as(rng.standard_normal((B, heads + 2 * kv_heads, D)), True)
        for s in (eager, graphed):
            s["x"].copy_(x)
            s["qkv"].copy_(qkv)
        step(eager)
        graph.replay()
        torch.cuda.synchronize()
        for name in ("total", "slots", "pos", "o", "table"):
            assert torch.equal(eager[name], graphed[name]), (i, name)
        for a, b in zip(eager["cache"] + list(eager["nq"]), graphed["cache"] + list(graphed["nq"])):
            assert torch.equal(a, b)
    assert H.hbl_last_device_error() == H.HBL_OK


def test_two_streams_at_once(H):
    """Calls on two streams with workspaces of their own, and calls in a row on one stream with one workspace."""
    import torch
    rng = np.random.default_rng(24)
    total, table = rng.integers(1, 1500, 24), rng.permutation(24 * 24).reshape(24, 24)
    cache = [_dev(a) for a in _cache(rng, 576, 2, 64, 64, 8) + _cache(rng, 576, 2, 64, 64, 8)]
    qs = [_as(rng.standard_normal((24, 8, 64)), True) for _ in range(2)]
    args = (_i32(range(25)), _i32(total), _i32(table), *cache)
    want = [H.hbl_kv_attention(q, *args) for q in qs]
    gx = [H.hbl_add_rms_quant_backward(q.view(24, 512), q.view(24, 512) * 2, gain=torch.ones(512, device="cuda")) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    n = H.hbl_kv_attention_workspace_bytes(24, 8, 2, 64, 24)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [[torch.empty_like(want[0]) for _ in range(6)] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(6):
        for j in (0, 1):
            with torch.cuda.stream(streams[j]):
                H.hbl_kv_attention(qs[(i + j) % 2], *args, o=outs[j][i], workspace=ws[j])
    torch.cuda.synchronize()
    for i in range(6):
        for j in (0, 1):
            assert torch.equal(outs[j][i], want[(i + j) % 2])
    for j in (0, 1):
        with torch.cuda.stream(streams[j]):
            again = H.hbl_add_rms_quant_backward(qs[j].view(24, 512), qs[j].view(24, 512) * 2,
                                                 gain=torch.ones(512, device="cuda"))
        torch.cuda.synchronize()
        assert torch.equal(again[0], gx[j][0]) and torch.equal(again[1], gx[j][1])


def _busy(stream, cycles=40_000_000):
    """Some 20 ms of nothing on a stream."""
    import torch
    with torch.cuda.stream(stream):
        torch.cuda._sleep(cycles)


def test_results_on_a_stream_that_is_not_the_current_one(H):
    """stream= with buffers that the call makes itself: what it fills and what it computes is in one order, however far
    behind the current stream is."""
    import torch
    rng = np.random.default_rng(61)
    total, table = rng.integers(1, 300, 6), rng.permutation(60).reshape(6, 10)
    cache = [_dev(a) for a in _cache(rng, 60, 2, 32, 64, 8) + _cache(rng, 60, 2, 32, 64, 8)]
    q = _as(rng.standard_normal((9, 8, 64)), True)              # three rows behind the last request
    args = (q, _i32(range(7)), _i32(total), _i32(table), *cache)
    want = H.hbl_kv_attention(*args)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    _busy(torch.cuda.current_stream())
    got = H.hbl_kv_attention(*args, stream=other)
    torch.cuda.synchronize()
    assert bool((want[:6] != 0).any()) and torch.equal(got, want)


def test_memory_of_a_call_on_another_stream_is_its_own(H):
    """While a call with stream= has yet to run, allocations on the current stream do not get its scratch or a result
    that was dropped."""
    import torch
    rng = np.random.default_rng(62)
    total, table = rng.integers(1, 300, 6), rng.permutation(60).reshape(6, 10)
    cache = [_dev(a) for a in _cache(rng, 60, 2, 32, 64, 8) + _cache(rng, 60, 2, 32, 64, 8)]
    q = _as(rng.standard_normal((6, 8, 64)), True)
    args = (q, _i32(range(7)), _i32(total), _i32(table), *cache)
    x, gain = _as(rng.standard_normal((500, 2048)), True), torch.ones(2048, device="cuda")
    packed, alpha = H.hbl_pack_ternary(_as(rng.standard_normal((1024, 2048)), True))
    calls = [(lambda s: H.hbl_kv_attention(*args, stream=s), H.hbl_kv_attention_workspace_bytes(6, 8, 2, 64, 6)),
             (lambda s: H.hbl_add_rms_quant_backward(x, x, gain=gain, stream=s),
              H.hbl_add_rms_quant_backward_workspace_bytes(500, 2048)),
             (lambda s: H.hbl_add_rms_quant(x, 8, gain=gain, stream=s), 2 * 500 * 2048),      # h
             (lambda s: H.hbl_forward(x, packed, alpha, 1024, 8, stream=s), H.hbl_forward_workspace_bytes(500, 2048, 1024, 8))]
    other = torch.cuda.Stream()
    for call, size in calls:
        call(None)
        torch.cuda.synchronize()
        _busy(other)
        call(other)
        mine = [torch.full((size,), 7, dtype=torch.uint8, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        assert all(bool((m == 7).all()) for m in mine)


def test_calls_on_a_forked_stream_of_a_capture(H):
    """stream= with buffers of the calls' own, on a stream that a captured one forked off and joins again."""
    import torch
    rng = np.random.default_rng(67)
    total, table = rng.integers(1, 900, 6), rng.permutation(180).reshape(6, 30)
    cache = [_dev(a) for a in _cache(rng, 180, 2, 32, 64, 8) + _cache(rng, 180, 2, 32, 64, 8)]
    q, x = _as(rng.standard_normal((8, 8, 64)), True), _as(rng.standard_normal((70, 1040)), True)
    args = (_i32(range(7)), _i32(total), _i32(table), *cache)
    gain = torch.ones(1040, device="cuda")

    def step(stream):
        o = H.hbl_kv_attention(q, *args, stream=stream)
        h, codes, scales = H.hbl_add_rms_quant(x, 8, gain=gain, stream=stream)
        return (o, h, codes, scales) + H.hbl_add_rms_quant_backward(h, x, gain=gain, stream=stream)

    main, fork = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(main):
        step(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        fork.wait_stream(main)
        outs = step(fork)
        main.wait_stream(fork)
    for _ in range(3):
        q.copy_(_as(rng.standard_normal((8, 8, 64)), True))
        x.copy_(_as(rng.standard_normal((70, 1040)), True))
        want = step(None)
        for t in outs:
            t.view(torch.uint8).fill_(0x55)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_the_binding_refuses(H):
    """Wrong types, shapes, strides, devices: nothing is launched on tensors that do not fit."""
    import torch
    cache = [torch.zeros((4, 2, 16, 64), dtype=torch.uint8, device="cuda"), torch.zeros((4, 2), device="cuda"),
             torch.zeros((4, 2, 16, 64), dtype=torch.uint8, device="cuda"), torch.zeros((4, 2), device="cuda")]
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16, device="cuda")
    rows, total, table = _i32([0, 3]), _i32([3]), _i32([[0, 1]])
    ok = lambda **k: H.hbl_kv_attention(*[k.get(n, d) for n, d in (  # noqa: E731
        ("q", q), ("rows", rows), ("total", total), ("table", table), ("kc", cache[0]), ("ks", cache[1]), ("vc", cache[2]),
        ("vs", cache[3]))], **{n: v for n, v in k.items() if n in ("o", "scale", "workspace")})
    ok()
    for bad in (dict(q=q.half()), dict(rows=rows.long()), dict(table=table.cpu()), dict(ks=cache[1].double()),
                dict(total=_i32([3, 4])), dict(rows=_i32([0, 1, 3])), dict(q=q.transpose(0, 1)), dict(vc=cache[2][:3]),
                dict(kc=cache[0].transpose(1, 2)), dict(o=q[:2].clone()), dict(scale=torch.ones(1)), dict(o=q)):
        with pytest.raises((TypeError, ValueError, H.HBLError)):
            ok(**bad)
    with pytest.raises(H.HBLError):
        ok(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    k = torch.zeros((3, 2, 64), device="cuda")
    with pytest.raises(TypeError):
        H.hbl_kv_append(k, k.bfloat16(), _i32([0, 1, 2]), *cache)
    with pytest.raises(ValueError):
        H.hbl_kv_append(k, k, _i32([0, 1]), *cache)
    with pytest.raises(ValueError):
        H.hbl_kv_plan(_i32([0]), _i32([1, 2]), _i32([1]), _i32([0]), table, 16, 4)
    with pytest.raises(TypeError):
        H.hbl_kv_plan(_i32([0]), _i32([1]).long(), _i32([1]), _i32([0]), table, 16, 4)
    x = torch.zeros((2, 64), device="cuda")
    with pytest.raises(TypeError):
        H.hbl_add_rms_quant(x, 8, residual=x.bfloat16())
    with pytest.raises(ValueError):
        H.hbl_add_rms_quant(x, 8, gain=torch.ones(32, device="cuda"))
    with pytest.raises(H.HBLError):
        H.hbl_add_rms_quant_backward(x, x.clone(), g_x=x)
