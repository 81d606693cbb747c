"""The operators over 8-bit pages on the GPU against the fp64 oracle
(oracle/paged_q8.py decodes the pages, oracle/paged_cache.py attends).

Tolerances, from the arithmetic, u = half a step of the tokens' type (bf16
2^-8, fp16 2^-11):
 - write: a rotated key is off by at most 2^-20 (|x| + |y|), as in 16 bits; so
   is a row's largest, whose quotients by 127 are rounded once more (2^-23).
   A code is the nearest whole number to a quotient that is off by 127 times
   that, so what it stands for is within half a step of the rotated row, and
   2^-19 of the row's largest pair. Values are not rotated: their codes are the
   oracle's but where x (127 / m) lies within 2^-15 of a half (two fp32
   roundings of numbers up to 127).
 - read: code * scale in fp32 (2^-24) and one rounding: (u + 2^-24) |ref|, and
   half a step of the smallest fp16 values.
 - attention, A = sum of w |v|, S = scale sum |q||k|. The products are of fp16:
   in batches of more than 32 rows of a kv head for each sequence (the kernel for
   128 rows) what a key or value stands for is rounded to its 11 bits, twice (bf16
   tokens: the scale, then its product with the code) or once (fp16 tokens: the scale
   is taken in two parts of 11). The sharp check is against the definition
   over keys and values that are rounded so, for fewer rows over those that are not
   (codes are exact, scales stay in fp32); its tolerance is that for
   16-bit pages with these differences. Weights are rounded to fp16, whatever
   the tokens' type: 2^-11 A. Rounded keys and values are off by 127 times half a
   step of the smallest fp16 values more, where the step's largest scale is put at
   2^7 at least: 2^-25 / 2^7 of the largest row, 2^-32, for each of the two
   roundings. The queries are taken to fp16 behind a power of two that puts a row's
   largest between 2^-1 and 1, in steps of 2^-24 at least: off by 2^-24 max |q|
   each. Three more factors are multiplied in in fp32: four more roundings of a score
   of size S. A weight, in the unit of the largest value exponent so far (4 times
   what the visible ones reach, at most: two powers of two), is scaled to 2^7 for
   the largest before it is rounded in steps of 2^-24 at least: of each of n terms at
   most 2^-25 2^-7 4 max |v| = 2^-30 max |v|.
   Against the definition itself the roundings of keys and values count in full:
   a score is off by 2 2^-11 S more (fp16 tokens 2^-11 S), a weight by twice that,
   and the sum of the values by 2 2^-11 A (2^-11 A). (That is what all of them on one
   side would give; found is 0.0020 of the output's norm for bf16 and 0.0005 for fp16.)
"""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle import paged_cache as pc  # noqa: E402
from oracle import paged_q8 as p8  # noqa: E402
from tests.test_gpu_paged import BF, DEV, HF, TINY, U, Batch, dfl, f64  # noqa: E402, F401

HEADS = [(8, 2, 128, BF), (4, 4, 64, HF), (28, 4, 64, BF), (8, 1, 128, HF)]


class Batch8(Batch):
    """A batch whose pool has 8-bit pages, with values whose norms vary by token."""

    def __init__(self, lens, heads, n_kv, d, dtype=BF, spread=0.5, **kw):
        super().__init__(lens, heads, n_kv, d, dtype, **kw)
        rng = np.random.default_rng(kw.get("seed", 0) + 100)
        n = self.pool.shape[0]
        keys, values = (f64(x) for x in (self.pool[:, 0].reshape(n, n_kv, 64, d), self.pool[:, 1].reshape(n, n_kv, 64, d)))
        values = values * np.exp(spread * rng.standard_normal((n, n_kv, 64, 1)))
        self.pool = torch.from_numpy(p8.encode(keys, values)).to(DEV)

    def decoded(self, bits=None):
        return p8.decode(self.pool.cpu().numpy(), self.d, bits, whole=self.dtype == HF)

    def oracle(self, bits="as run", **kw):
        mixed = False
        if bits == "as run":
            group, n_seq = self.heads // self.n_kv, len(self.kv_len)
            few = [group <= 32 and self.T * group <= 32 * n for n in (1, n_seq)]
            mixed = "prefix_len" in kw and not few[0] and few[1] and n_seq >= 64 and n_seq * self.table.shape[1] > 1024
            bits = None if few[0 if "prefix_len" in kw else 1] or mixed else 11
        scale = kw.pop("scale", self.d ** -0.5)
        ints = [t.cpu().numpy() for t in (self.q_start, self.kv_len, self.table)]
        pool = self.decoded(bits)
        if mixed:   # the own caches by the kernel for few rows, the prefix by the other
            pages = np.unique(kw["prefix_table"])
            pages = pages[(pages >= 0) & (pages < len(pool))]
            pool[pages] = self.decoded(11)[pages]
        return pc.attention(f64(self.q), pool, *ints, scale, **kw)


def check(b, got, ref, keys, scale=None, whole=False):
    """`got` against the oracle over rounded keys and values, or (whole) over what they stand for."""
    out, mass, size, owned = ref
    got = f64(got)[owned]
    out, mass, size = out[owned], mass[owned], size[owned][..., None]
    u, d = U[b.dtype], b.d
    pool = np.nan_to_num(b.decoded(), nan=0.0, posinf=0.0, neginf=0.0)
    vmax, kmax = np.abs(pool[:, 1]).max(), np.abs(pool[:, 0]).max()
    q = f64(b.q)[owned]
    lost = (2.0 ** -24 + 2.0 ** -31) * np.abs(q).max(axis=-1, keepdims=True) * d * kmax * (d ** -0.5 if scale is None else scale)
    score = 2 * (d / 16 + 8) * 2.0 ** -23 * size + 2 * lost + 2.0 ** -21
    tol = u * np.abs(out) + (2.0 ** -11 + score + (keys / 16 + 64) * 2.0 ** -23) * mass + (keys * 2.0 ** -30 + 2.0 ** -31) * vmax
    if whole:
        once = 2.0 ** -11 * (2 if b.dtype == BF else 1)
        tol = tol + (2 * once * size + once) * mass
    tol = tol + TINY[b.dtype]
    bad = np.abs(got - out) - tol
    bad[np.isnan(got) | np.isnan(out)] = np.inf
    at = np.unravel_index(np.argmax(bad), bad.shape) if bad.size else None
    assert bad.size == 0 or bad.max() <= 0, f"row/head/dim {at}: {got[at]} for {out[at]}, tolerance {tol[at]}"


def check_attn(dfl, b, shared=False, **kw):  # noqa: F811
    got = (b.attend_shared if shared else b.attend)(dfl, **kw)
    okw = {k: v for k, v in kw.items() if k not in ("out", "status", "stream")}
    if shared:
        okw.update(prefix_table=b.prefix_np, prefix_len=b.prefix)
    keys = int(b.kv_len.max()) + b.prefix if len(b.kv_len) else 0
    check(b, got, b.oracle(**okw), keys, kw.get("scale"))
    check(b, got, b.oracle(bits=None, **okw), keys, kw.get("scale"), whole=True)
    return got


# --- write ---------------------------------------------------------------------

def check_write(dfl, b, base, positions=None, with_q=True):  # noqa: F811
    d, before = b.d, b.pool.cpu().numpy()
    ints = [t.cpu().numpy() for t in (b.q_start, b.kv_len, b.table)]
    q0, k0, v0 = f64(b.q), f64(b.k), f64(b.v)
    pos_np = None if positions is None else positions.cpu().numpy()
    out = torch.full((b.T, b.heads, d), 7.0, dtype=b.dtype, device=DEV) if with_q else None
    got = dfl.dflash_kv_append(b.pool, b.k, b.v, b.q_start, b.kv_len, b.table, q=b.q if with_q else None, q_out=out,
                               positions=positions, rope_base=base)
    after = b.pool.cpu().numpy()
    kc, vc, ks, vs = p8.parts(after, d)
    want = p8.parts(before, d)
    for x in want:
        x[:] = x.copy()
    wk, wv, wks, wvs = (x.copy() for x in want)
    owned = np.zeros(b.T, dtype=bool)
    for t, i, pos in pc.places(ints[0], ints[1]):
        if pos < 0:
            continue
        owned[t] = True
        page, s = int(ints[2][i][pos // 64]), pos % 64
        if not 0 <= page < len(after):
            continue
        rot = pc.rotate(k0[t:t + 1], [pos if pos_np is None else int(pos_np[t])], base)[0]
        pair = np.abs(k0[t]) + np.abs(np.roll(k0[t], d // 2, axis=-1))
        assert np.abs(ks[page, :, s] - np.abs(rot).max(-1) / 127).max() <= 2.0 ** -20 * pair.max() / 127
        tol = 0.5 * ks[page, :, s][:, None] + 2.0 ** -19 * pair.max()
        assert (np.abs(kc[page, :, s] * ks[page, :, s][:, None] - rot) <= tol).all()
        assert (np.abs(kc[page, :, s]).max(-1) == 127).all()
        codes, scales = p8.quantise(v0[t])
        assert np.abs(vs[page, :, s] - scales).max() <= 2.0 ** -24 * scales.max()
        exact = v0[t] * (127.0 / np.abs(v0[t]).max(-1, keepdims=True))
        sure = np.abs(exact - np.floor(exact) - 0.5) > 2.0 ** -15
        assert (vc[page, :, s] == codes)[sure].all() and np.abs(vc[page, :, s] - codes).max() <= 1
        wk[page, :, s], wv[page, :, s], wks[page, :, s], wvs[page, :, s] = (x[page, :, s] for x in (kc, vc, ks, vs))
    for x, y in zip((kc, vc, ks, vs), (wk, wv, wks, wvs)):   # nothing else was touched
        np.testing.assert_array_equal(x, y)
    if with_q:
        g, q = f64(got), q0.copy()
        for t, i, pos in pc.places(ints[0], ints[1]):
            if pos >= 0:
                q[t] = pc.rotate(q0[t:t + 1], [pos if pos_np is None else int(pos_np[t])], base)[0]
        size = np.abs(q0) + np.abs(np.roll(q0, d // 2, axis=-1))
        assert (np.abs(g - q)[owned] <= (U[b.dtype] * np.abs(q) + 2.0 ** -20 * size + TINY[b.dtype])[owned]).all()
        assert (g[~owned] == 7.0).all()
    else:
        assert got is None


WRITE_LENS = [
    [(1, 1)],
    [(1, 64), (1, 65), (1, 128), (1, 1)],
    [(16, 100)],
    [(0, 10), (3, 66), (0, 0), (64, 64), (65, 65), (1, 63)],
    [(130, 200), (5, 5), (129, 129)],
]


@pytest.mark.parametrize("lens", WRITE_LENS, ids=str)
@pytest.mark.parametrize("heads,n_kv,d,dtype", [(8, 2, 128, BF), (4, 4, 64, HF), (7, 1, 64, BF), (15, 3, 128, HF)])
def test_write(dfl, lens, heads, n_kv, d, dtype):  # noqa: F811
    check_write(dfl, Batch8(lens, heads, n_kv, d, dtype), 1e4)
    check_write(dfl, Batch8(lens, heads, n_kv, d, dtype, pad=(3, 2), wide=8), 0.0)
    check_write(dfl, Batch8(lens, heads, n_kv, d, dtype), 1e6, with_q=False)


def test_write_in_place_at_given_positions(dfl):  # noqa: F811
    b = Batch8([(5, 70), (2, 2)], 8, 2, 64, BF)
    pos = torch.tensor([0, 262143, 2 ** 24 + 1, 2 ** 30, 2 ** 31 - 1, -5, 3], dtype=torch.int32, device=DEV)
    check_write(dfl, b, 1e4, positions=pos)
    c = Batch8([(5, 70), (2, 2)], 8, 2, 64, BF)
    q = c.q.clone()
    one = dfl.dflash_kv_append(c.pool, c.k, c.v, c.q_start, c.kv_len, c.table, q=q, positions=pos, rope_base=1e4)
    two = dfl.dflash_kv_append(c.pool, c.k, c.v, c.q_start, c.kv_len, c.table, q=q, q_out=q, positions=pos, rope_base=1e4)
    assert two is q and torch.equal(one, two)


def test_a_large_write(dfl):  # noqa: F811
    """As many tokens as whole blocks of the kernel take, and heads in groups."""
    check_write(dfl, Batch8([(700, 800), (1, 3000), (333, 333)], 32, 8, 128, BF), 1e6)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_special_values(dfl, d, dtype):  # noqa: F811
    """Zeros, one value, the smallest and largest of the type, infinities and NaN; each row alone."""
    big, small = torch.finfo(dtype).max, torch.finfo(dtype).tiny
    rows = torch.zeros(10, 1, d)
    rows[1, 0, 5] = -3.0
    rows[2] = big
    rows[3, 0, ::2], rows[3, 0, 1::2] = small, -small
    rows[4, 0, 7], rows[4, 0, 8] = float("inf"), 1.0
    rows[5] = float("nan")
    rows[6, 0, 0], rows[6, 0, 1:] = 1.0, float("-inf")
    rows[7] = torch.arange(d) - d / 2
    rows[8, 0, 3], rows[8, 0, 4] = float("nan"), 2.0
    rows[9] = -0.0
    x = rows.to(dtype).to(DEV)
    pool = dfl.kv_pool_q8(1, 1, d)
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    dfl.dflash_kv_append(pool, x, x, i(0, 10), i(10), i(0)[None])
    kc, vc, ks, vs = p8.parts(pool.cpu().numpy(), d)
    codes, scales = p8.quantise(f64(x)[:, 0])
    for c, s in ((kc, ks), (vc, vs)):
        np.testing.assert_allclose(s[0, 0, :10], scales, rtol=2.0 ** -23, equal_nan=True)
        exact = np.nan_to_num(f64(x)[:, 0], nan=0, posinf=0, neginf=0)
        ratio = np.where(np.abs(exact).max(-1, keepdims=True) > 0, np.abs(exact).max(-1, keepdims=True), 1)
        sure = np.abs(exact * 127 / ratio - np.floor(exact * 127 / ratio) - 0.5) > 2.0 ** -15
        assert (c[0, 0, :10] == codes)[sure | ~np.isfinite(scales)[:, None]].all()
    k, v = dfl.dflash_kv_read(pool, 10, i(0, 10), i(10), i(0)[None], dtype=dtype)
    for y in (k, v):
        assert y[4:7].isnan().all() and y[8].isnan().all()
        keep = [0, 1, 2, 3, 7, 9]
        ref = f64(x)[keep]
        half = np.abs(ref).max(-1, keepdims=True) / 254
        # rows below 2^-100 (the smallest bf16 values) are held as zeros, by definition: off by less than that
        assert (np.abs(f64(y)[keep] - ref) <= half + 2 * U[dtype] * np.abs(ref) + TINY[dtype] + p8.LEAST).all()


# --- read ----------------------------------------------------------------------

def rows_of(b, pool):
    """(keys, values [T, n_kv, d] in fp64 and which rows have a page) of a pool in the 16-bit oracle's form."""
    q_start, kv_len, table = (t.cpu().numpy() for t in (b.q_start, b.kv_len, b.table))
    out, there = np.zeros((2, b.T, b.n_kv, b.d)), np.zeros(b.T, dtype=bool)
    for t, i, pos in pc.places(q_start, kv_len):
        if pos < 0 or not 0 <= table[i][pos // 64] < len(pool):
            continue
        page = pool[table[i][pos // 64]]
        out[0, t] = page[0].reshape(b.n_kv, 64, b.d)[:, pos % 64]
        out[1, t] = page[1].reshape(b.n_kv, b.d, 64)[:, :, pos % 64]
        there[t] = True
    return out[0], out[1], there


READ_LENS = [[(1, 1)], [(1, 64), (1, 65), (0, 9), (1, 128)], [(300, 300)], [(64, 64), (65, 65), (130, 200), (0, 0), (7, 1000)]]


@pytest.mark.parametrize("lens", READ_LENS, ids=str)
@pytest.mark.parametrize("heads,n_kv,d,dtype", [(8, 2, 128, BF), (4, 4, 64, HF), (7, 1, 64, BF), (15, 3, 128, HF)])
def test_read(dfl, lens, heads, n_kv, d, dtype):  # noqa: F811
    b = Batch8(lens, heads, n_kv, d, dtype, pad=(2, 3))
    ref = rows_of(b, b.decoded())
    wide = torch.full((b.T, 2 * n_kv * d + 8), 7.0, dtype=dtype, device=DEV)   # both as columns of one matrix
    k, v = (wide.as_strided((b.T, n_kv, d), (wide.shape[1], d, 1), at) for at in (0, n_kv * d))
    got = dfl.dflash_kv_read(b.pool, b.T, b.q_start, b.kv_len, b.table, k_out=k, v_out=v)
    assert got[0] is k and got[1] is v
    for g, r in zip((k, v), ref):
        assert (np.abs(f64(g) - r) <= (U[dtype] + 2.0 ** -24) * np.abs(r) + TINY[dtype])[ref[2]].all()
        assert (f64(g)[~ref[2]] == 7.0).all()
    assert (wide[:, 2 * n_kv * d:] == 7.0).all()
    fresh = dfl.dflash_kv_read(b.pool, b.T, b.q_start, b.kv_len, b.table, dtype=dtype)
    own = torch.from_numpy(ref[2]).to(DEV)
    assert all(torch.equal(x[own], y[own]) for x, y in zip(fresh, (k, v)))


@pytest.mark.parametrize("lens", READ_LENS, ids=str)
@pytest.mark.parametrize("heads,n_kv,d,dtype", [(8, 2, 128, BF), (4, 4, 64, HF)])
def test_read_of_16_bit_pages_is_a_copy(dfl, lens, heads, n_kv, d, dtype):  # noqa: F811
    b = Batch(lens, heads, n_kv, d, dtype, pad=(1, 2))
    ref = rows_of(b, f64(b.pool))
    k, v = (torch.full((b.T, n_kv, d), 7.0, dtype=dtype, device=DEV) for _ in range(2))
    dfl.dflash_kv_read(b.pool, b.T, b.q_start, b.kv_len, b.table, k_out=k, v_out=v)
    for g, r in zip((k, v), ref):
        np.testing.assert_array_equal(f64(g), np.where(ref[2][:, None, None], r, 7.0))


@pytest.mark.parametrize("q8", [False, True])
def test_rows_without_a_page_are_left(dfl, q8):  # noqa: F811
    b = (Batch8 if q8 else Batch)([(100, 300), (5, 3), (2, 100)], 4, 2, 64, BF)
    b.table[0, 4] = -7                 # tokens 256 .. 299
    b.table[2, 1] = b.pool.shape[0]    # tokens 64 ..
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    k, v = (torch.full((b.T, 2, 64), 7.0, dtype=BF, device=DEV) for _ in range(2))
    dfl.dflash_kv_read(b.pool, b.T, b.q_start, b.kv_len, b.table, k_out=k, v_out=v, status=status)
    assert int(status) == 2
    ref = rows_of(b, b.decoded() if q8 else f64(b.pool))
    assert ref[2].sum() == 56 + 3
    for g, r in zip((k, v), ref):
        assert (f64(g)[~ref[2]] == 7.0).all() and (np.abs(f64(g) - r) <= 2.0 ** -8 * np.abs(r))[ref[2]].all()
    status.zero_()
    before = b.pool.clone()
    dfl.dflash_kv_append(b.pool, b.k, b.v, b.q_start, b.kv_len, b.table, status=status)
    assert int(status) == 2
    assert (b.pool != before).flatten(1).any(1).sum() <= 3   # pages of sequence 0 (2) and of sequence 1


def test_an_append_is_read_back(dfl):  # noqa: F811
    """Keys that were read and written again without a rotation are the same codes."""
    b = Batch8([(90, 200), (3, 64)], 8, 2, 128, HF)
    dfl.dflash_kv_append(b.pool, b.k, b.v, b.q_start, b.kv_len, b.table, rope_base=1e4)
    codes = [x.clone() for x in dfl.kv_pool_q8_views(b.pool, 128)[:2]]
    k, v = dfl.dflash_kv_read(b.pool, b.T, b.q_start, b.kv_len, b.table, dtype=HF)
    dfl.dflash_kv_append(b.pool, k, v, b.q_start, b.kv_len, b.table)
    for x, y in zip(codes, dfl.kv_pool_q8_views(b.pool, 128)[:2]):
        assert torch.equal(x, y)


# --- attention -----------------------------------------------------------------

LENS = [
    [(1, 1)],
    [(1, 64), (1, 65), (1, 127), (1, 129), (1, 1)],
    [(16, 700)],
    [(3, 66), (0, 10), (64, 64), (65, 65), (1, 63), (0, 0)],
    [(130, 200), (5, 5), (129, 129), (2, 1500)],
]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("heads,n_kv,d,dtype", HEADS)
def test_attention(dfl, lens, heads, n_kv, d, dtype):  # noqa: F811
    b = Batch8(lens, heads, n_kv, d, dtype)
    check_attn(dfl, b)
    check_attn(dfl, b, causal=False)
    check_attn(dfl, b, window=33, sinks=5)
    check_attn(dfl, b, window=1)


@pytest.mark.parametrize("window,sinks", [(1, 0), (64, 0), (65, 1), (127, 64), (128, 129), (500, 70), (2 ** 31 - 1, 0)])
def test_windows(dfl, window, sinks):  # noqa: F811
    b = Batch8([(40, 900), (1, 300), (200, 200), (3, 64)], 8, 2, 64, BF)
    check_attn(dfl, b, window=window, sinks=sinks)
    check_attn(dfl, b, window=window, sinks=sinks, causal=False)


def test_long_prefill_with_a_window(dfl):  # noqa: F811
    for d, dtype in ((64, HF), (128, BF)):
        b = Batch8([(700, 900), (513, 513)], 4, 1, d, dtype)
        check_attn(dfl, b, window=256, sinks=10)
        check_attn(dfl, b)


@pytest.mark.parametrize("heads,n_kv,d,dtype", [(5, 1, 128, BF), (7, 7, 64, HF), (128, 1, 64, BF), (96, 2, 128, HF), (12, 4, 64, BF)])
def test_groups(dfl, heads, n_kv, d, dtype):  # noqa: F811
    b = Batch8([(3, 200), (20, 90), (1, 5)], heads, n_kv, d, dtype, prefix=70)
    check_attn(dfl, b, window=50, sinks=3)
    check_attn(dfl, b, shared=True)


@pytest.mark.parametrize("prefix", [1, 64, 100, 128, 129, 900])
@pytest.mark.parametrize("heads,n_kv,d,dtype", [(8, 2, 128, BF), (28, 4, 64, HF)])
def test_shared_prefix(dfl, prefix, heads, n_kv, d, dtype):  # noqa: F811
    for lens in ([(1, 1 + 9 * i) for i in range(20)], [(16, 40), (0, 9), (3, 3), (90, 300)], [(10, 4), (3, 0), (5, 5), (200, 20)]):
        check_attn(dfl, Batch8(lens, heads, n_kv, d, dtype, prefix=prefix), shared=True)


MANY = [(1, int(n)) for n in np.random.default_rng(5).integers(1, 1500, 64)]


@pytest.mark.parametrize("prefix", [0, 1, 300, 1500])
@pytest.mark.parametrize("heads,n_kv,d,dtype", [(8, 2, 128, BF), (4, 4, 64, HF), (28, 4, 64, BF), (32, 1, 128, HF)])
def test_many_short_blocks_behind_a_prefix(dfl, prefix, heads, n_kv, d, dtype):  # noqa: F811
    """(Where the own caches are taken apart from the prefix; with 63 sequences they are not.)"""
    check_attn(dfl, Batch8(MANY, heads, n_kv, d, dtype, prefix=prefix), shared=True)
    check_attn(dfl, Batch8(MANY[:63], heads, n_kv, d, dtype, prefix=prefix), shared=True)
    lens = MANY[:40] + [(0, 40), (0, 0), (3, 5), (2, 2), (1, 1), (1, 64), (1, 65), (0, 0), (1, 9000)] + MANY[40:]
    b = Batch8(lens, heads, n_kv, d, dtype, prefix=prefix, pad=(2, 3))
    out = torch.full((b.T, b.heads, d), 7.0, dtype=dtype, device=DEV)
    got = f64(check_attn(dfl, b, shared=True, causal=False, out=out))
    owned = np.zeros(b.T, dtype=bool)
    for t, _, pos in pc.places(b.q_start.cpu().numpy(), b.kv_len.cpu().numpy()):
        owned[t] = pos >= 0
    assert (got[~owned] == 7.0).all() and (~owned).sum() == 5


def test_strides_and_rows_of_no_sequence(dfl):  # noqa: F811
    b = Batch8([(5, 90), (130, 400)], 8, 2, 128, BF, pad=(3, 4), wide=8, prefix=65, extra_cols=5)
    whole = torch.full((b.T, 8 * 128 + 16), 9.0, dtype=BF, device=DEV)
    out = whole.as_strided((b.T, 8, 128), (8 * 128 + 16, 128, 1))
    for shared in (False, True):
        whole.fill_(9.0)
        check_attn(dfl, b, shared=shared, out=out)
        assert (whole[:3] == 9.0).all() and (whole[-4:] == 9.0).all() and (whole[:, 8 * 128:] == 9.0).all()


def test_long_caches(dfl):  # noqa: F811
    """Rows split over CTAs."""
    check_attn(dfl, Batch8([(16, 20013)], 8, 1, 128, BF))
    check_attn(dfl, Batch8([(1, 30001), (2, 77)], 8, 2, 64, HF), window=20000, sinks=65)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [-30, -12, 12, 30])
def test_queries_of_any_size(dfl, d, power):  # noqa: F811
    """bf16 queries far outside what fp16 holds, with a scale that brings the scores back."""
    b = Batch8([(3, 200), (17, 150)], 8, 2, d, BF)
    b.q = (b.q.float() * 2.0 ** power).to(BF)
    check_attn(dfl, b, scale=2.0 ** -power * d ** -0.5)


def test_queries_with_values_of_very_different_size(dfl):  # noqa: F811
    b = Batch8([(3, 200), (17, 150)], 8, 2, 64, BF)
    b.q = (b.q.float() * torch.exp2(torch.randint(-20, 4, b.q.shape, device=DEV).float())).to(BF)
    check_attn(dfl, b)


@pytest.mark.parametrize("spread", [0.0, 3.0])
@pytest.mark.parametrize("power", [-40, 0, 40])
def test_scales_of_any_size(dfl, spread, power):  # noqa: F811
    """Values whose norms differ by powers of ten between tokens, and far from 1 (bf16 holds them)."""
    b = Batch8([(3, 200), (17, 1500), (1, 70)], 8, 2, 128, BF, spread=spread, prefix=200)
    _, _, ks, vs = dfl.kv_pool_q8_views(b.pool, 128)
    vs *= 2.0 ** power
    check_attn(dfl, b)
    check_attn(dfl, b, shared=True)
    ks *= 2.0 ** power
    check_attn(dfl, b, scale=2.0 ** -power * 128 ** -0.5)


def test_values_that_grow_along_the_cache(dfl):  # noqa: F811
    """Every step of keys has larger values than the one before, then smaller ones."""
    for order in (1, -1):
        b = Batch8([(16, 1500), (200, 1500)], 8, 2, 128, BF)
        _, _, _, vs = dfl.kv_pool_q8_views(b.pool, 128)
        for i in range(2):
            for n, p in enumerate(b.table[i].tolist()[::order]):
                vs[p] *= 2.0 ** n
        check_attn(dfl, b)


def test_zero_values_count_as_keys(dfl):  # noqa: F811
    b = Batch8([(2, 300), (1, 64)], 8, 2, 64, BF)
    kc, vc, ks, vs = dfl.kv_pool_q8_views(b.pool, 64)
    vs[b.table[0, 0].item()], vc[b.table[0, 0].item()] = 0.0, 128
    check_attn(dfl, b)
    vs.zero_()
    got = check_attn(dfl, b)
    assert (got == 0).all()


# --- what must not matter ------------------------------------------------------

def poison(b, dfl, value):  # noqa: F811
    """Scales of `value` and codes of any kind in every slot that no row of the batch may see."""
    kc, vc, ks, vs = dfl.kv_pool_q8_views(b.pool, b.d)
    places = [(int(p), 0) for p in b.spare]
    places += [(int(b.table[i, n // 64]), n % 64) for i, n in enumerate(b.kv_len.tolist()) if n % 64]
    if b.prefix % 64:
        places.append((int(b.prefix_table[b.prefix // 64]), b.prefix % 64))
    for p, s in places:
        ks[p][:, s:], vs[p][:, s:] = value, -value
        kc[p][:, s:], vc[p][:, s:] = 255, 0


@pytest.mark.parametrize("heads,n_kv,d,dtype", HEADS)
def test_slots_past_a_length_change_no_bit(dfl, heads, n_kv, d, dtype):  # noqa: F811
    for lens, prefix in (([(1, 1), (1, 70), (16, 100), (3, 129), (40, 40), (1, 900), (7, 64)], 77), ([(200, 1101), (1, 13)], 127),
                         ([(16, 9013)], 8), ([(1, 1 + 11 * i) for i in range(40)], 1077)):
        b = Batch8(lens, heads, n_kv, d, dtype, prefix=prefix)
        calls = lambda: [b.attend(dfl), b.attend(dfl, window=200, sinks=70), b.attend_shared(dfl)]
        clean = calls()
        for value in (float("nan"), float("inf"), 1e30):
            poison(b, dfl, value)
            for x, y in zip(clean, calls()):
                assert x.isfinite().all() and torch.equal(x, y)


@pytest.mark.parametrize("lens,at", [(((64, 300),), 280), (((200, 3000),), 2900), (((16, 9000),), 8990)])
def test_hidden_keys_may_hold_anything(dfl, lens, at):  # noqa: F811
    """Keys that only some rows of a tile see: a later token's, and those before the window."""
    b = Batch8(lens, 8, 2, 128, BF)
    _, _, ks, vs = dfl.kv_pool_q8_views(b.pool, 128)
    first = at - (lens[0][1] - lens[0][0])        # the first new token that sees it
    p, s = int(b.table[0, at // 64]), at % 64
    for array in (ks, vs):
        for value in (float("nan"), float("inf"), float("-inf")):
            kept, clean = array[p][:, s].clone(), b.attend(dfl)
            array[p][:, s] = value
            got = b.attend(dfl)
            assert torch.equal(got[:first], clean[:first])
            if array is vs or value != value:
                assert not got[first:].isfinite().any()
            windowed = b.attend(dfl, window=8, sinks=2)
            array[p][:, s] = kept
            assert torch.equal(windowed[first + 8:], b.attend(dfl, window=8, sinks=2)[first + 8:])


def test_a_broken_neighbour_behind_the_same_prefix(dfl):  # noqa: F811
    b = Batch8([(1, 60), (2, 100), (1, 33)], 8, 2, 64, HF, prefix=200)
    clean = b.attend_shared(dfl)
    _, _, ks, _ = dfl.kv_pool_q8_views(b.pool, 64)
    for p in b.table[1, :2].tolist():
        ks[p] = float("nan")
    got = b.attend_shared(dfl)
    assert got[1:3].isnan().all() and torch.equal(got[0], clean[0]) and torch.equal(got[3], clean[3])


def test_broken_queries_harm_themselves_only(dfl):  # noqa: F811
    b = Batch8([(20, 300), (3, 90)], 8, 2, 128, BF, prefix=130)
    clean = b.attend(dfl), b.attend_shared(dfl)
    b.q = b.q.clone()
    b.q[4, 3, 7] = float("nan")
    b.q[6, 1] = float("inf")
    for x, y in zip(clean, (b.attend(dfl), b.attend_shared(dfl))):
        away = torch.ones(23, 8, dtype=torch.bool, device=DEV)
        away[4, 3] = away[6, 1] = False
        assert torch.equal(x[away], y[away]) and y[4, 3].isnan().all()


def test_missing_pages_are_not_seen(dfl):  # noqa: F811
    b = Batch8([(4, 300), (2, 100)], 4, 2, 64, BF, prefix=130)
    b.table[0, 1] = -7
    b.table[1, 0] = b.pool.shape[0]
    b.prefix_table[1] = 2 ** 30
    b.prefix_np = b.prefix_table.cpu().numpy()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for shared in (False, True):
        status.zero_()
        check_attn(dfl, b, shared=shared, status=status)
        assert int(status) == 2
    status.zero_()
    b.attend(dfl, window=20, status=status)    # sequence 1 sees 80 .., page 1; sequence 0 does not reach page 1
    assert int(status) == 0


def test_broken_lengths_stay_inside_the_buffers(dfl):  # noqa: F811
    b = Batch8([(4, 100), (4, 100), (4, 100)], 4, 2, 64, BF)
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    for q_start, kv_len in ((i(0, 8, 4, 12), i(100, 100, 100)), (i(-5, 4, 8, 1000), i(100, 100, 100)),
                            (i(0, 4, 8, 12), i(-3, 2 ** 31 - 1, 100)), (i(9, 3, 2, 1), i(5, 5, 5))):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        for call in (lambda: dfl.dflash_paged_attn(b.q, b.pool, q_start, kv_len, b.table, status=status),
                     lambda: dfl.dflash_shared_prefix_attn(b.q, b.pool, q_start, kv_len, b.table, i(0, 1), 100, status=status),
                     lambda: dfl.dflash_kv_append(b.pool, b.k, b.v, q_start, kv_len, b.table, rope_base=1e4, status=status),
                     lambda: dfl.dflash_kv_read(b.pool, b.T, q_start, kv_len, b.table, status=status)):
            status.zero_()
            call()
            assert int(status) == 2
    torch.cuda.synchronize()


@pytest.mark.parametrize("heads,tokens", [(8, 3), (64, 200)])
def test_a_cache_of_millions_of_tokens(dfl, heads, tokens):  # noqa: F811
    """A few pages over and over: the softmax over many copies of the same keys is the softmax over one of them."""
    b = Batch8([(tokens, 1024)], heads, 1, 128, BF, prefix=1024)
    copies = 4096 if tokens < 10 else 256
    own, pre = b.table.repeat(1, copies), b.prefix_table.repeat(copies)
    one = dfl.dflash_paged_attn(b.q, b.pool, b.q_start, b.kv_len * copies, own, causal=False)
    check(b, one, b.oracle(causal=False), 1024 * copies)
    two = dfl.dflash_shared_prefix_attn(b.q, b.pool, b.q_start, b.kv_len * copies, own, pre, 1024 * copies, causal=False)
    check(b, two, b.oracle(causal=False, prefix_table=b.prefix_np, prefix_len=1024), 2048 * copies)


def test_pages_far_into_a_large_pool(dfl):  # noqa: F811
    """Offsets above 2^32 bytes."""
    n_kv, d = 8, 128
    pages = (1 << 32) // (n_kv * 64 * (2 * d + 8)) + 70
    pool = dfl.kv_pool_q8(pages, n_kv, d)
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    k, v = (torch.randn(100, n_kv, d, generator=g, device=DEV).to(BF) for _ in range(2))
    q = torch.randn(100, n_kv, d, generator=g, device=DEV).to(BF)
    near, far = i(1, 0)[None], i(pages - 1, pages - 3)[None]
    outs = []
    for table in (near, far):
        dfl.dflash_kv_append(pool, k, v, i(0, 100), i(100), table)
        outs.append((*dfl.dflash_kv_read(pool, 100, i(0, 100), i(100), table),
                     dfl.dflash_paged_attn(q, pool, i(0, 100), i(100), table)))
    assert all(torch.equal(x, y) for x, y in zip(*outs)) and outs[0][0].abs().max() > 1


# --- refusals on the device ----------------------------------------------------

def test_wrong_tensors_are_refused(dfl):  # noqa: F811
    b = Batch8([(4, 100)], 8, 2, 64, BF)
    E = dfl.DFlashError
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)
    bad = [dict(q=b.q.float()), dict(pool=b.pool.view(torch.int8)), dict(pool=b.pool[:, :, :-8]), dict(pool=b.pool[:, :1]),
           dict(pool=b.pool.cpu()), dict(kv_len=b.kv_len.long()), dict(table=b.table[0]), dict(q_start=i(5))]
    for kw in bad:
        f = dict(q=b.q, pool=b.pool, q_start=b.q_start, kv_len=b.kv_len, table=b.table)
        f.update(kw)
        with pytest.raises(E):
            dfl.dflash_paged_attn(f["q"], f["pool"], f["q_start"], f["kv_len"], f["table"])
    with pytest.raises(E):   # k and v of two types
        dfl.dflash_kv_append(b.pool, b.k, b.v.half(), b.q_start, b.kv_len, b.table)
    with pytest.raises(E):   # heads that are not the pool's
        dfl.dflash_kv_append(b.pool, b.k[:, :1], b.v[:, :1], b.q_start, b.kv_len, b.table)
    with pytest.raises(E):   # buffers inside the pool
        inside = b.pool.view(-1)[:4 * 2 * 64 * 2].view(BF).view(4, 2, 64)
        dfl.dflash_kv_read(b.pool, 4, b.q_start, b.kv_len, b.table, k_out=inside)
    with pytest.raises(E):
        dfl.dflash_kv_read(b.pool, 4, b.q_start, b.kv_len, b.table, k_out=b.k, dtype=HF)
    with pytest.raises(E):
        dfl.dflash_kv_read(b.pool, 4, b.q_start, b.kv_len, b.table, k_out=b.k, v_out=b.k)
    with pytest.raises(E):
        dfl.dflash_kv_read(b.pool, 4, b.q_start, b.kv_len, b.table, dtype=torch.float32)


# --- a run of them together ----------------------------------------------------

def test_a_serving_step(dfl):  # noqa: F811
    """A decoding loop over 8-bit pages: each step appends one token per sequence,
    attends through a windowed layer and behind the shared prefix, and at the
    end the cache is read back and continues in 16 bits."""
    b = Batch8([(1, 60), (1, 1), (1, 127)], 8, 2, 64, BF, prefix=100)
    g = torch.Generator(device=DEV).manual_seed(9)
    for step in range(5):
        b.k, b.v, b.q = (torch.randn(3, h, 64, generator=g, device=DEV).to(BF) for h in (2, 2, 8))
        at = (b.kv_len - 1 + 100).contiguous()
        q = b.q
        check_write(dfl, b, 1e4, positions=at)
        b.q = dfl.dflash_kv_append(b.pool, b.k, b.v, b.q_start, b.kv_len, b.table, q=q, positions=at, rope_base=1e4)
        check_attn(dfl, b, window=50, sinks=4)
        check_attn(dfl, b, shared=True)
        if step < 4:
            b.kv_len += torch.tensor([1, 1, 1 if step == 0 else 0], dtype=torch.int32, device=DEV)
    whole = torch.cat([torch.zeros_like(b.kv_len[:1]), b.kv_len.cumsum(0).to(torch.int32)])
    T = int(whole[-1])
    k, v = dfl.dflash_kv_read(b.pool, T, whole, b.kv_len, b.table)
    pool = dfl.kv_pool(b.pool.shape[0], 2, 64)
    dfl.dflash_kv_append(pool, k, v, whole, b.kv_len, b.table)
    one, two = b.attend(dfl, window=50, sinks=4), dfl.dflash_paged_attn(b.q, pool, b.q_start, b.kv_len, b.table, window=50, sinks=4)
    # every key is rounded to bf16: scores move by 2^-8 of their size (below 8 here), values by 2^-8
    assert (one.float() - two.float()).abs().max() < 0.1


def test_the_workspace_depends_on_the_tokens_only(dfl):  # noqa: F811
    """One buffer for all batches of so many tokens or fewer: for one sequence, many, with wide tables or narrow ones."""
    lib = dfl.load_library()

    def need(T, n_seq, table_pages, dtype=16):
        pb = dfl.dflash_paged_batch(dtype, 32, 8, 128, n_seq, T, 1, table_pages, table_pages, *([1 << 20] * 4), None)
        n = ctypes.c_size_t()
        assert lib.dflash_paged_attn_workspace(ctypes.byref(pb), ctypes.byref(n)) == dfl.DFLASH_OK
        return n.value

    last = 0
    for T in (1, 2, 8, 32, 33, 64, 128, 129, 1000, 1024, 1025, 100000):
        sizes = {need(T, n_seq, pages) for n_seq in (1, 8, 64, 1024) for pages in (1, 16, 4096)}
        assert len(sizes) == 1 and min(sizes) >= last and need(T, 8, 1, 0) == need(min(T, 129), 64, 16, 0)
        last = min(sizes)
    assert need(1024, 1, 1) == last


def test_repeats_are_bit_identical(dfl):  # noqa: F811
    b = Batch8([(16, 2000), (1, 700), (300, 900)], 32, 8, 128, BF, prefix=1500)
    for kw in (dict(), dict(window=300, sinks=8)):
        x = b.attend(dfl, **kw)
        assert all(torch.equal(x, b.attend(dfl, **kw)) for _ in range(5))
    x = b.attend_shared(dfl)
    assert all(torch.equal(x, b.attend_shared(dfl)) for _ in range(5))


def test_streams_and_threads(dfl):  # noqa: F811
    """Four host threads at once, each with a stream, a pool and shapes of its own."""
    import threading
    bs = [Batch8([(1 + 5 * i, 400 + 300 * i), (i, 50)], 8, 2, d, dt, prefix=100 * i, seed=i)
          for i, (d, dt) in enumerate(((64, BF), (64, HF), (128, BF), (128, HF)))]
    run = lambda b, **kw: (b.attend(dfl, window=90, sinks=3, **kw), b.attend_shared(dfl, **kw),
                           *dfl.dflash_kv_read(b.pool, b.T, b.q_start, b.kv_len, b.table, **kw))
    ref = [run(b) for b in bs]
    torch.cuda.synchronize()
    wrong = []

    def work(b, r):
        try:
            s = torch.cuda.Stream()
            for _ in range(50):
                got = run(b, stream=s)
                s.synchronize()
                if not all(torch.equal(x, y) for x, y in zip(got, r)):
                    wrong.append(b.d)
        except BaseException as e:   # shown by the assertion below
            wrong.append(e)
    threads = [threading.Thread(target=work, args=a) for a in zip(bs, ref)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong


def test_captured_calls_follow_the_lengths(dfl):  # noqa: F811
    """One captured step replayed over growing caches, and two graphs with their own workspaces."""
    b = Batch8([(1, 300), (1, 120), (1, 5)], 8, 2, 128, BF, prefix=64)
    k, v, q = b.k.contiguous(), b.v.contiguous(), b.q.contiguous()
    b.attend(dfl)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        qr = dfl.dflash_kv_append(b.pool, k, v, b.q_start, b.kv_len, b.table, q=q, rope_base=1e4)
        o1 = dfl.dflash_paged_attn(qr, b.pool, b.q_start, b.kv_len, b.table, window=100, sinks=4)
        rk, rv = dfl.dflash_kv_read(b.pool, 3, b.q_start, b.kv_len, b.table)
    with torch.cuda.graph(g2):
        o2 = dfl.dflash_shared_prefix_attn(qr, b.pool, b.q_start, b.kv_len, b.table, b.prefix_table, 64)
    for lens in ((300, 120, 5), (301, 121, 6), (310, 65, 1)):
        b.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        b.q = qr
        check(b, o1, b.oracle(window=100, sinks=4), 400)
        check(b, o2, b.oracle(prefix_table=b.prefix_np, prefix_len=64), 400)
        ref = rows_of(b, b.decoded())
        assert np.abs(f64(rk) - ref[0]).max() < 0.05 and np.abs(f64(rv) - ref[1]).max() < 0.05
    kept = o1.clone(), o2.clone()
    side = torch.cuda.Stream()
    for _ in range(10):   # both at once: g2 only reads what g1 has written before
        with torch.cuda.stream(side):
            g2.replay()
        o3 = b.attend(dfl, window=100, sinks=4)
    torch.cuda.synchronize()
    assert torch.equal(o3, kept[0]) and torch.equal(o2, kept[1])
