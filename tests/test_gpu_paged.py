"""Paged-cache operators on the GPU against the fp64 oracle
(oracle/paged_cache.py).

Tolerances, from the arithmetic, u = half a step of the stored type (bf16
2^-8, fp16 2^-11):
 - append: x cos - y sin in fp32 with cos and sin off by at most 2^-22, one
   rounding: u |ref| + 2^-20 (|x| + |y|), and for fp16 results below 2^-14, whose
   steps are 2^-24, half of such a step; values are copied, so they are equal.
 - attention, A = sum of w |v|: the weights may be rounded to the stored type
   (u A) and the output is (u |o|). A score of size S = scale sum |q||k| is an
   fp32 sum over d in steps of 16, so it is off by at most (d/16 + 4) 2^-23 S,
   and a weight by twice that (its own, and the sum's); the exponential by
   2^-21. The product with the values is an fp32 sum of n terms in steps of 16:
   (n/16 + 64) 2^-23 A. fp16 weights below 2^-14 are rounded in absolute steps:
   a weight is scaled by at least 2^7 over the row's largest, or by 2^-1 when a
   stale maximum is up to 2^8 low, so each of the n is off by at most 2^-31
   of the largest, which is at most 1: n 2^-31 max |v|.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle import paged_cache as pc  # noqa: E402

DEV = "cuda:0"
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}   # half a step of the smallest values
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dfl():
    import __graft_entry__
    __graft_entry__.build()
    import block_diffusion_drafter_pass_gb300 as m
    return m


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


class Batch:
    """Sequences of (new tokens, cached tokens) with their pages scattered in
    a pool of random values, a prefix, and `pad` token rows of no sequence on
    both sides."""

    def __init__(self, lens, heads, n_kv, d, dtype=BF, prefix=0, seed=0, pad=(0, 0), wide=0, spare=3, q_scale=1.5,
                 extra_cols=0):
        rng = np.random.default_rng(seed)
        need = [(n + 63) // 64 for _, n in lens]
        pn = (prefix + 63) // 64
        total = sum(need) + pn + spare
        order = rng.permutation(total).astype(np.int32)
        cols = max(need + [1])
        full = np.full((len(lens), cols + extra_cols), 2 ** 30, dtype=np.int32)   # unused entries are no page at all
        at = 0
        for i, n in enumerate(need):
            full[i, :n] = order[at:at + n]
            at += n
        self.full = torch.from_numpy(full).to(DEV)
        self.table = self.full[:, :cols]
        self.prefix, self.prefix_np = prefix, order[at:at + pn]
        self.spare = order[at + pn:]
        self.prefix_table = torch.from_numpy(self.prefix_np.copy()).to(DEV)
        starts = pad[0] + np.concatenate([[0], np.cumsum([a for a, _ in lens])])
        self.T = int(starts[-1]) + pad[1]
        self.q_start = torch.from_numpy(starts.astype(np.int32)).to(DEV)
        self.kv_len = torch.tensor([n for _, n in lens], dtype=torch.int32, device=DEV)
        self.heads, self.n_kv, self.d, self.dtype = heads, n_kv, d, dtype
        g = torch.Generator(device=DEV).manual_seed(seed)
        normal = lambda *s: torch.randn(s, generator=g, device=DEV).to(dtype)
        self.pool = normal(total, 2, n_kv, 64 * d)
        row = (heads + 2 * n_kv) * d + wide
        self.qkv = normal(self.T, row)
        cut = lambda a, h: self.qkv[:, a * d:(a + h) * d].view(self.T, h, d) if wide == 0 else \
            self.qkv.as_strided((self.T, h, d), (row, d, 1), a * d)
        self.q = cut(0, heads)
        if q_scale != 1:
            self.q.mul_(q_scale)
        self.k, self.v = cut(heads, n_kv), cut(heads + n_kv, n_kv)

    def attend(self, dfl, **kw):
        return dfl.dflash_paged_attn(self.q, self.pool, self.q_start, self.kv_len, self.table, **kw)

    def attend_shared(self, dfl, **kw):
        return dfl.dflash_shared_prefix_attn(self.q, self.pool, self.q_start, self.kv_len, self.table,
                                             self.prefix_table, self.prefix, **kw)

    def oracle(self, **kw):
        scale = kw.pop("scale", self.d ** -0.5)
        return pc.attention(f64(self.q), f64(self.pool), self.q_start.cpu().numpy(), self.kv_len.cpu().numpy(),
                            self.table.cpu().numpy(), scale, **kw)


def check(got, ref, dtype, d, keys, vmax, what=""):
    out, mass, size, owned = ref
    got = f64(got)[owned]
    out, mass, size = out[owned], mass[owned], size[owned][..., None]
    u = U[dtype]
    score = 2 * (d / 16 + 4) * 2.0 ** -23 * size + 2.0 ** -21
    tol = u * (mass + np.abs(out)) + (score + (keys / 16 + 64) * 2.0 ** -23) * mass
    if dtype == HF:
        tol = tol + keys * 2.0 ** -31 * vmax + 2.0 ** -25
    bad = np.abs(got - out) - tol
    bad[np.isnan(got) | np.isnan(out)] = np.inf
    at = np.unravel_index(np.argmax(bad), bad.shape) if bad.size else None
    assert bad.size == 0 or bad.max() <= 0, f"{what}: row/head/dim {at}: {got[at]} for {out[at]}, tolerance {tol[at]}"


def check_attn(dfl, b, shared=False, **kw):
    got = (b.attend_shared if shared else b.attend)(dfl, **kw)
    okw = dict(kw)
    for name in ("out", "status", "stream"):
        okw.pop(name, None)
    if shared:
        okw.update(prefix_table=b.prefix_np, prefix_len=b.prefix)
    keys = int(b.kv_len.max()) + b.prefix if len(b.kv_len) else 0
    check(got, b.oracle(**okw), b.dtype, b.d, keys, float(b.pool.float().nan_to_num(0, 0, 0).abs().max()))
    return got


# --- append --------------------------------------------------------------------

def check_append(dfl, b, base, positions=None, with_q=True, in_place=False):
    before, q0 = f64(b.pool), f64(b.q)
    k0, v0 = f64(b.k), f64(b.v)
    pos_np = None if positions is None else positions.cpu().numpy()
    pool, q = pc.append(before, k0, v0, b.q_start.cpu().numpy(), b.kv_len.cpu().numpy(), b.table.cpu().numpy(), base,
                        positions=pos_np, q=q0)
    owned = np.zeros(b.T, dtype=bool)
    for t, _, p in pc.places(b.q_start.cpu().numpy(), b.kv_len.cpu().numpy()):
        owned[t] = p >= 0
    sentinel = torch.full((b.T, b.heads, b.d), 7.0, dtype=b.dtype, device=DEV)
    out = b.q if in_place else sentinel
    got = dfl.dflash_kv_append(b.pool, b.k, b.v, b.q_start, b.kv_len, b.table, q=b.q if with_q else None,
                               q_out=out if with_q else None, positions=positions, rope_base=base)
    u = U[b.dtype]
    if with_q:
        g = f64(got)
        size = np.abs(q0) + np.abs(np.roll(q0, b.d // 2, axis=-1))
        assert (np.abs(g - q)[owned] <= (u * np.abs(q) + 2.0 ** -20 * size + TINY[b.dtype])[owned]).all()
        if in_place:
            np.testing.assert_array_equal(g[~owned], q0[~owned])
        else:
            assert (g[~owned] == 7.0).all()
    else:
        assert got is None
    after = f64(b.pool)
    np.testing.assert_array_equal(after[:, 1], pool[:, 1])          # values: copied, nothing else touched
    touched = pool[:, 0] != before[:, 0]
    np.testing.assert_array_equal(after[:, 0][~touched], before[:, 0][~touched])
    tol = u * np.abs(pool[:, 0]) + 2.0 ** -20 * 2 * np.abs(k0).max() + TINY[b.dtype]
    assert (np.abs(after[:, 0] - pool[:, 0]) <= np.where(touched, tol, 0.0)).all()


APPEND_LENS = [
    [(1, 1)],
    [(1, 64), (1, 65), (1, 128), (1, 1)],
    [(16, 100)],
    [(0, 10), (3, 66), (0, 0), (64, 64), (65, 65), (1, 63)],
    [(130, 200), (5, 5), (129, 129)],
]


@pytest.mark.parametrize("lens", APPEND_LENS, ids=str)
@pytest.mark.parametrize("heads,n_kv,d,dtype", [(8, 2, 128, BF), (4, 4, 64, HF), (7, 1, 64, BF), (15, 3, 128, HF)])
def test_append(dfl, lens, heads, n_kv, d, dtype):
    check_append(dfl, Batch(lens, heads, n_kv, d, dtype), 1e4)


def test_append_without_rotation_is_a_copy(dfl):
    b = Batch([(5, 70), (64, 64)], 4, 2, 64, HF)
    q0 = f64(b.q)
    check_append(dfl, b, 0.0)
    got = dfl.dflash_kv_append(b.pool, b.k, b.v, b.q_start, b.kv_len, b.table, q=b.q)
    np.testing.assert_array_equal(f64(got), q0)


@pytest.mark.parametrize("base", [1e4, 1e6, 1.5])
def test_append_at_far_positions(dfl, base):
    """Positions where a float product has no fraction of a turn left."""
    b = Batch([(6, 6)], 8, 2, 128, HF, q_scale=1)
    far = torch.tensor([0, 262143, 2 ** 24 + 1, 2 ** 30, 2 ** 31 - 1, -5], dtype=torch.int32, device=DEV)
    check_append(dfl, b, base, positions=far)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_append_at_given_positions(dfl, dtype):
    """Positions of the caller's (also negative ones), results of every size down to fp16's smallest steps."""
    b = Batch([(33, 90), (5, 5), (200, 200)], 24, 2, 64, dtype)
    at = np.random.default_rng(5).integers(-100, 1 << 20, b.T).astype(np.int32)
    check_append(dfl, b, 1e4, positions=torch.from_numpy(at).to(DEV))


def test_append_strided_padded_and_in_place(dfl):
    lens = [(3, 60), (9, 70)]
    check_append(dfl, Batch(lens, 8, 2, 64, BF, pad=(2, 5), wide=24), 1e4, in_place=True)
    check_append(dfl, Batch(lens, 8, 2, 128, BF, pad=(1, 1), wide=8, extra_cols=3), 1e6)
    check_append(dfl, Batch(lens, 8, 2, 128, BF), 1e6, with_q=False)


def test_append_skips_tokens_without_a_place(dfl):
    """A bad page id, and more new tokens than the cache is said to hold."""
    b = Batch([(4, 66), (3, 2), (2, 130)], 4, 2, 64, BF)
    b.table[0, 1] = -1
    b.table[2, 2] = b.pool.shape[0]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    before = b.pool.clone()
    check_append(dfl, b, 1e4)
    b.pool.copy_(before)
    dfl.dflash_kv_append(b.pool, b.k, b.v, b.q_start, b.kv_len, b.table, rope_base=1e4, status=status)
    assert int(status) == 2


def test_append_at_a_page_beyond_32_bits_of_elements(dfl):
    """The last pages of a pool of more than 2^31 elements."""
    n_kv, d = 8, 128
    per = 2 * n_kv * 64 * d
    pages = 2 ** 31 // per + 40
    pool = torch.zeros(pages, 2, n_kv, 64 * d, dtype=BF, device=DEV)
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device=DEV)
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    k, v = torch.randn(70, n_kv, d, device=DEV).to(BF), torch.randn(70, n_kv, d, device=DEV).to(BF)
    dfl.dflash_kv_append(pool, k, v, i(0, 70), i(70), table)
    keys, values = dfl.kv_pool_views(pool, d)
    assert torch.equal(keys[pages - 1], k[:64].transpose(0, 1)) and torch.equal(keys[pages - 3][:, :6], k[64:].transpose(0, 1))
    assert torch.equal(values[pages - 1], v[:64].permute(1, 2, 0))
    assert int(pool[:pages - 3].abs().max() != 0) == 0
    q = torch.randn(70, 16, d, device=DEV).to(BF)
    out = dfl.dflash_paged_attn(q, pool, i(0, 70), i(70), table)
    small = torch.stack([pool[pages - 1], pool[pages - 3]])
    assert torch.equal(out, dfl.dflash_paged_attn(q, small, i(0, 70), i(70), i(0, 1)[None]))


# --- attention over a sequence's own cache ---------------------------------------

LENS = [
    [(1, 1)],
    [(1, 64), (1, 65), (1, 127), (1, 128), (1, 129)],
    [(1, 1000)],
    [(16, 300), (16, 16), (16, 777)],
    [(0, 100), (5, 5), (1, 0), (3, 1), (0, 0), (31, 200)],
    [(130, 130), (33, 500)],
    [(1, 3000), (2, 90)],
]
HEADS = [(32, 8, 128, BF), (4, 4, 64, HF), (28, 4, 64, BF), (10, 2, 128, HF), (6, 1, 64, BF)]


@pytest.mark.parametrize("heads,n_kv,d,dtype", HEADS)
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_full_attention(dfl, lens, heads, n_kv, d, dtype):
    b = Batch(lens, heads, n_kv, d, dtype)
    check_attn(dfl, b)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 4), (64, 64), (100, 0), (128, 130), (300, 5), (4096, 1),
                                          (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_window_and_sinks(dfl, window, sinks, causal):
    b = Batch([(1, 900), (16, 640), (40, 200), (3, 5), (70, 70)], 8, 2, 64, BF)
    check_attn(dfl, b, window=window, sinks=sinks, causal=causal)


@pytest.mark.parametrize("d,dtype", [(64, HF), (128, BF)])
def test_long_prefill_with_a_window(dfl, d, dtype):
    b = Batch([(700, 900), (513, 513)], 4, 1, d, dtype)
    check_attn(dfl, b, window=200, sinks=10)
    check_attn(dfl, b)


def test_one_query_head_and_the_widest_group(dfl):
    check_attn(dfl, Batch([(3, 200), (1, 70)], 128, 1, 64, BF))
    check_attn(dfl, Batch([(3, 200), (1, 70)], 1, 1, 128, BF))
    check_attn(dfl, Batch([(3, 200), (150, 170)], 65, 1, 128, BF))


@pytest.mark.parametrize("scale", [1e-6, 0.5, 30.0])
def test_scales(dfl, scale):
    """Flat rows, and rows whose largest score leaves nothing of the others
    (running maxima that jump by hundreds)."""
    check_attn(dfl, Batch([(16, 700), (5, 300)], 8, 2, 64, BF), scale=scale)
    check_attn(dfl, Batch([(16, 700), (5, 300)], 8, 2, 128, HF), scale=scale)


def test_rising_scores(dfl):
    """Every key's score above the one before it, so that the running maximum
    moves in every tile; the first of them far below."""
    b = Batch([(4, 1500)], 4, 1, 64, BF, q_scale=1)
    b.q.fill_(1.0)
    keys, _ = dfl.kv_pool_views(b.pool, 64)
    for p in range(24):
        keys[int(b.table[0, p])] = torch.linspace(p * 0.3 - 4, p * 0.3 - 3.7, 64, device=DEV).to(BF)[None, :, None]
    check_attn(dfl, b, scale=0.5)


def test_many_sequences(dfl):
    rng = np.random.default_rng(5)
    lens = [(int(a), int(a + n)) for a, n in zip(rng.integers(0, 3, 1024), rng.integers(0, 90, 1024))]
    check_attn(dfl, Batch(lens, 2, 1, 64, BF))
    check_attn(dfl, Batch(lens, 2, 1, 64, BF, prefix=70), shared=True)


def test_no_sequences_and_no_tokens(dfl):
    b = Batch([(0, 10), (0, 70)], 4, 2, 64)
    assert check_attn(dfl, b).shape == (0, 4, 64)
    e = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)
    out = torch.full((3, 4, 64), 5.0, dtype=BF, device=DEV)
    dfl.dflash_paged_attn(torch.zeros_like(out), b.pool, e(1), e(0), e(0, 1), out=out)
    assert (out == 5).all()


# --- behind a shared prefix -------------------------------------------------------

@pytest.mark.parametrize("prefix", [0, 1, 63, 64, 65, 128, 1000])
@pytest.mark.parametrize("heads,n_kv,d,dtype", [(8, 2, 128, BF), (28, 4, 64, HF)])
def test_shared_prefix(dfl, prefix, heads, n_kv, d, dtype):
    for lens in ([(1, 1)], [(1, 30), (1, 64), (1, 200), (1, 1)], [(16, 40), (0, 9), (3, 3), (16, 300)]):
        check_attn(dfl, Batch(lens, heads, n_kv, d, dtype, prefix=prefix), shared=True)


def test_shared_prefix_long_blocks_and_no_mask(dfl):
    b = Batch([(100, 150), (1, 400), (300, 300), (2, 2)], 8, 2, 64, BF, prefix=500)
    check_attn(dfl, b, shared=True)
    check_attn(dfl, b, shared=True, causal=False)


def test_shared_prefix_wide_batches(dfl):
    """More rows than one tile holds, from many sequences."""
    check_attn(dfl, Batch([(1, 1 + 7 * i) for i in range(40)], 32, 4, 64, BF, prefix=900), shared=True)
    check_attn(dfl, Batch([(5, 5 + 13 * i) for i in range(20)], 10, 2, 128, HF, prefix=333), shared=True)


def test_shared_prefix_of_tokens_before_their_cache(dfl):
    """More new tokens than cached ones: the first rows see a part of the prefix."""
    check_attn(dfl, Batch([(10, 4), (3, 0), (5, 5), (200, 20)], 4, 2, 64, BF, prefix=150), shared=True)


def test_shared_prefix_equals_the_joined_cache(dfl):
    b = Batch([(4, 50), (2, 200)], 8, 2, 128, BF, prefix=256)
    one = check_attn(dfl, b, shared=True)
    joined = torch.cat([b.prefix_table[None].expand(2, -1), b.table], dim=1).contiguous()
    two = dfl.dflash_paged_attn(b.q, b.pool, b.q_start, b.kv_len + 256, joined)
    ref = b.oracle(prefix_table=b.prefix_np, prefix_len=256)
    check(two, ref, BF, 128, 500, 6.0)
    assert (one.float() - two.float()).abs().max() < 0.1


# --- what must not matter ----------------------------------------------------------

def poison(b, dfl, value):
    """`value` in every slot that no row of the batch may see: spare pages, and
    slots past the lengths."""
    keys, values = dfl.kv_pool_views(b.pool, b.d)
    for p in b.spare:
        b.pool[int(p)] = value
    for i, n in enumerate(b.kv_len.tolist()):
        if n % 64:
            p = int(b.table[i, n // 64])
            keys[p][:, n % 64:] = value
            values[p][:, :, n % 64:] = value
    if b.prefix % 64:
        p = int(b.prefix_table[b.prefix // 64])
        keys[p][:, b.prefix % 64:] = value
        values[p][:, :, b.prefix % 64:] = value


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_slots_past_a_length_may_hold_anything(dfl, value, dtype):
    lens = [(1, 70), (16, 100), (3, 129), (40, 40), (1, 900)]
    for d in (64, 128):
        b = Batch(lens, 8, 2, d, dtype, prefix=77)
        clean = b.attend(dfl), b.attend_shared(dfl), b.attend(dfl, window=20, sinks=3)
        poison(b, dfl, value)
        for x, y in zip(clean, (check_attn(dfl, b), check_attn(dfl, b, shared=True),
                                check_attn(dfl, b, window=20, sinks=3))):
            assert (x.float() - y.float()).abs().max() < 0.05


def test_hidden_keys_may_hold_anything(dfl):
    """Keys a row does not see, in tiles it reads: a later token's (causal), and
    those before the window. Rows that do see them are not compared."""
    b = Batch([(64, 300)], 4, 2, 128, BF)
    keys, values = dfl.kv_pool_views(b.pool, 128)
    clean = b.attend(dfl)
    at = 280                                # seen by new tokens 44 ..
    p, s = int(b.table[0, at // 64]), at % 64
    kept = keys[p][:, s].clone(), values[p][:, :, s].clone()
    values[p][:, :, s] = float("nan")
    got = b.attend(dfl)
    assert (got[:44].float() - clean[:44].float()).abs().max() < 0.05 and got[44:].isnan().all()
    keys[p][:, s] = float("inf")
    got = b.attend(dfl)
    assert (got[:44].float() - clean[:44].float()).abs().max() < 0.05 and got[44:].isnan().all()
    keys[p][:, s], values[p][:, :, s] = kept
    clean = b.attend(dfl, window=30, sinks=2)
    p, s = int(b.table[0, 250 // 64]), 250 % 64   # in the window of tokens 14 .. 43
    values[p][:, :, s] = float("inf")
    got = b.attend(dfl, window=30, sinks=2)
    away = torch.ones(64, dtype=torch.bool)
    away[14:44] = False
    assert (got[away].float() - clean[away].float()).abs().max() < 0.05
    assert not got[14:44].isfinite().any()


def test_hidden_values_in_long_blocks(dfl):
    """As above where each stream of a CTA has 128 rows, and where a block's keys are split between CTAs."""
    for lens, at in (((200, 9000),), 8900), (((600, 700),), 400), (((16, 30000),), 29990):
        b = Batch(lens, 8, 2, 128, BF)
        _, values = dfl.kv_pool_views(b.pool, 128)
        clean = b.attend(dfl)
        first = at - (lens[0][1] - lens[0][0])        # the first new token that sees it
        p, s = int(b.table[0, at // 64]), at % 64
        for value in (float("nan"), float("inf")):
            values[p][:, :, s] = value
            got = b.attend(dfl)
            assert (got[:first].float() - clean[:first].float()).abs().max() < 0.05
            assert not got[first:].isfinite().any()


def test_slots_past_the_lengths_of_a_wide_batch(dfl):
    b = Batch([(8, 30 + 13 * i) for i in range(24)], 16, 1, 128, HF, prefix=1000)
    poison(b, dfl, float("nan"))
    check_attn(dfl, b)
    check_attn(dfl, b, shared=True)


@pytest.mark.parametrize("heads,tokens", [(8, 3), (64, 200)])
def test_a_cache_of_millions_of_tokens(dfl, heads, tokens):
    """A few pages over and over: the softmax over many copies of the same keys
    is the softmax over one of them."""
    b = Batch([(tokens, 1024)], heads, 1, 128, BF, prefix=1024)
    copies = 4096 if tokens < 10 else 256
    own, pre = b.table.repeat(1, copies), b.prefix_table.repeat(copies)
    ref = b.oracle(causal=False)
    one = dfl.dflash_paged_attn(b.q, b.pool, b.q_start, b.kv_len * copies, own, causal=False)
    check(one, ref, BF, 128, 1024 * copies, 6.0)
    ref = b.oracle(causal=False, prefix_table=b.prefix_np, prefix_len=1024)
    two = dfl.dflash_shared_prefix_attn(b.q, b.pool, b.q_start, b.kv_len * copies, own, pre, 1024 * copies, causal=False)
    check(two, ref, BF, 128, 2048 * copies, 6.0)


def test_a_page_in_two_places(dfl):
    """Tables that name a page twice, of one sequence and of two, and of the prefix and a sequence."""
    b = Batch([(3, 300), (20, 200)], 8, 2, 64, BF, prefix=130)
    b.table[0, 2] = b.table[0, 0]
    b.table[1, 1] = b.table[0, 1]
    b.prefix_table[0] = b.table[1, 0]
    b.prefix_np = b.prefix_table.cpu().numpy()
    check_attn(dfl, b)
    check_attn(dfl, b, window=100, sinks=70)
    check_attn(dfl, b, shared=True)


def test_a_broken_neighbour_behind_the_same_prefix(dfl):
    """One sequence's cache is full of NaN: the others are unharmed, itself NaN."""
    b = Batch([(1, 60), (2, 100), (1, 33)], 8, 2, 64, HF, prefix=200)
    clean = b.attend_shared(dfl)
    for p in b.table[1, :2].tolist():
        b.pool[p] = float("nan")
    got = b.attend_shared(dfl)
    assert got[1:3].isnan().all()
    for r in (0, 3):
        assert (got[r].float() - clean[r].float()).abs().max() < 0.01


def test_pages_outside_the_pool_are_not_seen(dfl):
    b = Batch([(4, 300), (2, 100)], 4, 2, 64, BF, prefix=130)
    b.table[0, 1] = -7
    b.table[1, 0] = b.pool.shape[0]
    b.prefix_table[1] = 2 ** 30
    b.prefix_np = b.prefix_table.cpu().numpy()
    for shared in (False, True):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        check_attn(dfl, b, shared=shared, status=status)
        assert int(status) == 2
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    Batch([(4, 300)], 4, 2, 64, BF).attend(dfl, status=status)
    assert int(status) == 0


def test_broken_lengths_stay_inside_the_buffers(dfl):
    b = Batch([(4, 100), (4, 100), (4, 100)], 4, 2, 64, BF)
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    for q_start, kv_len in ((i(0, 8, 4, 12), i(100, 100, 100)), (i(-5, 4, 8, 1000), i(100, 100, 100)),
                            (i(0, 4, 8, 12), i(-3, 2 ** 31 - 1, 100)), (i(9, 3, 2, 1), i(5, 5, 5))):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        dfl.dflash_paged_attn(b.q, b.pool, q_start, kv_len, b.table, status=status)
        assert int(status) == 2
        status.zero_()
        dfl.dflash_kv_append(b.pool, b.k, b.v, q_start, kv_len, b.table, rope_base=1e4, status=status)
        assert int(status) == 2
        status.zero_()
        dfl.dflash_shared_prefix_attn(b.q, b.pool, q_start, kv_len, b.table, i(0, 1), 100, status=status)
        assert int(status) == 2
    torch.cuda.synchronize()


def test_strides_and_rows_of_no_sequence(dfl):
    b = Batch([(5, 70), (20, 300)], 8, 2, 128, BF, pad=(3, 6), wide=40, extra_cols=5, prefix=100)
    whole = torch.full((b.T, 8 * 128 + 16), 9.0, dtype=BF, device=DEV)
    out = whole.as_strided((b.T, 8, 128), (1040, 128, 1), 8)
    for shared in (False, True):
        whole.fill_(9.0)
        check_attn(dfl, b, shared=shared, out=out)
        assert (whole[:, :8] == 9).all() and (whole[:, 1032:] == 9).all()
        assert (whole[:3] == 9).all() and (whole[-6:] == 9).all()


def test_refused_tensors(dfl):
    b = Batch([(5, 70)], 8, 2, 64, BF, prefix=64)
    E = dfl.DFlashError
    bad = [dict(q=b.q.half()), dict(q=b.q[..., :32]), dict(q=b.q.float()), dict(pool=b.pool[:, :, :1]),
           dict(pool=b.pool.half()), dict(q_start=b.q_start.long()), dict(q_start=b.q_start[:1]),
           dict(kv_len=b.kv_len.cpu()), dict(table=b.table.long()), dict(table=b.table[:, :0]),
           dict(q=b.q.transpose(0, 1).contiguous().transpose(0, 1)), dict(q=b.q[:, :7])]
    for kw in bad:
        f = dict(q=b.q, pool=b.pool, q_start=b.q_start, kv_len=b.kv_len, table=b.table)
        f.update(kw)
        with pytest.raises(E):
            dfl.dflash_paged_attn(f["q"], f["pool"], f["q_start"], f["kv_len"], f["table"])
    with pytest.raises(E):
        b.attend(dfl, window=-1)
    with pytest.raises(E):
        b.attend(dfl, out=b.q)
    with pytest.raises(E):
        b.attend_shared(dfl, out=b.q)
    with pytest.raises(E):
        dfl.dflash_kv_append(b.pool, b.k, b.v, b.q_start, b.kv_len, b.table, q=b.q,
                             q_out=b.qkv.as_strided(b.q.shape, b.q.stride(), 64))
    with pytest.raises(E):
        b.attend(dfl, out=torch.empty(4, 8, 64, dtype=BF, device=DEV))
    with pytest.raises(E):
        dfl.dflash_shared_prefix_attn(b.q, b.pool, b.q_start, b.kv_len, b.table, b.prefix_table, 65)
    with pytest.raises(E):
        dfl.dflash_kv_append(b.pool, b.k, b.v[:, :1], b.q_start, b.kv_len, b.table)
    with pytest.raises(E):
        dfl.dflash_kv_append(b.pool, b.k, b.v, b.q_start, b.kv_len, b.table, q_out=b.q)
    lib = dfl.load_library()
    import ctypes
    pb = dfl.dflash_paged_batch(0, 8, 2, 64, 1, b.T, b.pool.shape[0], b.table.shape[1], b.table.stride(0), b.pool.data_ptr(),
                                b.table.data_ptr(), b.q_start.data_ptr(), b.kv_len.data_ptr(), None)
    need = ctypes.c_size_t()
    assert lib.dflash_paged_attn_workspace(ctypes.byref(pb), ctypes.byref(need)) == dfl.DFLASH_OK
    if need.value:
        ws = torch.empty(need.value, dtype=torch.uint8, device=DEV)
        out = torch.empty(b.T, 8, 64, dtype=BF, device=DEV)
        args = (b.q.data_ptr(), b.q.stride(0), out.data_ptr(), 512, 0, 0, 1, 0.1)
        assert lib.dflash_paged_attn(ctypes.byref(pb), *args, ws.data_ptr(), need.value - 1, None) == dfl.DFLASH_EINVAL
        assert lib.dflash_paged_attn(ctypes.byref(pb), *args, None, need.value, None) == dfl.DFLASH_EINVAL
        assert lib.dflash_paged_attn(ctypes.byref(pb), *args, ws.data_ptr() + 4, need.value, None) == dfl.DFLASH_EINVAL


# --- a run of them together --------------------------------------------------------

def test_append_then_attend_as_a_serving_step(dfl):
    """A decoding loop: each step appends one token per sequence and attends
    through a windowed layer and behind the shared prefix; the cache the loop
    built is the oracle's."""
    b = Batch([(1, 60), (1, 1), (1, 127)], 8, 2, 64, BF, prefix=100)
    g = torch.Generator(device=DEV).manual_seed(9)
    for step in range(5):
        k, v, q = (torch.randn(3, h, 64, generator=g, device=DEV).to(BF) for h in (2, 2, 8))
        at = (b.kv_len - 1 + 100).contiguous()
        want_pool, want_q = pc.append(f64(b.pool), f64(k), f64(v), b.q_start.cpu().numpy(), b.kv_len.cpu().numpy(),
                                      b.table.cpu().numpy(), 1e4, positions=at.cpu().numpy(), q=f64(q))
        qr = dfl.dflash_kv_append(b.pool, k, v, b.q_start, b.kv_len, b.table, q=q, positions=at, rope_base=1e4)
        assert np.abs(f64(b.pool) - want_pool).max() <= 2.0 ** -8 * np.abs(want_pool).max()
        b.q = qr
        check_attn(dfl, b, window=50, sinks=4)
        check_attn(dfl, b, shared=True)
        b.kv_len += torch.tensor([1 if step < 4 else 0, 1, 1 if step == 0 else 0], dtype=torch.int32, device=DEV)


def test_repeats_are_bit_identical(dfl):
    b = Batch([(16, 2000), (1, 700), (300, 900)], 32, 8, 128, BF, prefix=1500)
    for kw in (dict(), dict(window=300, sinks=8)):
        x = b.attend(dfl, **kw)
        assert all(torch.equal(x, b.attend(dfl, **kw)) for _ in range(5))
    x = b.attend_shared(dfl)
    assert all(torch.equal(x, b.attend_shared(dfl)) for _ in range(5))


def test_streams(dfl):
    """Calls on two streams at once, each its own result and workspace."""
    a, b = Batch([(16, 3000)], 32, 8, 128, BF, seed=1), Batch([(1, 2500)] * 8, 32, 8, 128, BF, seed=2, prefix=600)
    ra, rb = a.attend(dfl), b.attend_shared(dfl)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        got.append((a.attend(dfl, stream=s1), b.attend_shared(dfl, stream=s2.cuda_stream)))
    torch.cuda.synchronize()
    assert all(torch.equal(x, ra) and torch.equal(y, rb) for x, y in got)


def test_threads(dfl):
    """Four host threads at once, each with a stream, a pool and shapes of its own."""
    import threading
    bs = [Batch([(1 + 5 * i, 400 + 300 * i), (i, 50)], 8, 2, d, dt, prefix=100 * i, seed=i)
          for i, (d, dt) in enumerate(((64, BF), (64, HF), (128, BF), (128, HF)))]
    ref = [(b.attend(dfl, window=90, sinks=3), b.attend_shared(dfl)) for b in bs]
    torch.cuda.synchronize()
    wrong = []

    def work(b, r):
        try:
            s = torch.cuda.Stream()
            for _ in range(50):
                x, y = b.attend(dfl, window=90, sinks=3, stream=s), b.attend_shared(dfl, stream=s)
                with pytest.raises(dfl.DFlashError):
                    b.attend(dfl, scale=-1.0, stream=s)
                s.synchronize()
                if not (torch.equal(x, r[0]) and torch.equal(y, r[1])):
                    wrong.append(b.d)
        except BaseException as e:   # shown by the assertion below
            wrong.append(e)
    threads = [threading.Thread(target=work, args=a) for a in zip(bs, ref)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong


def test_captured_calls_follow_the_lengths(dfl):
    """One captured step replayed over growing caches, and two graphs with
    their own workspaces replayed in turn and at once."""
    b = Batch([(1, 300), (1, 120), (1, 5)], 8, 2, 128, BF, prefix=64, q_scale=1)
    k, v = b.k.contiguous(), b.v.contiguous()
    q = b.q.contiguous()
    warm = b.attend(dfl)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        qr = dfl.dflash_kv_append(b.pool, k, v, b.q_start, b.kv_len, b.table, q=q, rope_base=1e4)
        o1 = dfl.dflash_paged_attn(qr, b.pool, b.q_start, b.kv_len, b.table, window=100, sinks=4)
    with torch.cuda.graph(g2):
        o2 = dfl.dflash_shared_prefix_attn(qr, b.pool, b.q_start, b.kv_len, b.table, b.prefix_table, 64)
    for lens in ((300, 120, 5), (301, 121, 6), (310, 65, 1)):
        b.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        b.q = qr
        check(o1, b.oracle(window=100, sinks=4), BF, 128, 400, 6.0)
        check(o2, b.oracle(prefix_table=b.prefix_np, prefix_len=64), BF, 128, 400, 6.0)
    k1, k2 = o1.clone(), o2.clone()
    side = torch.cuda.Stream()
    g1.replay()
    torch.cuda.synchronize()
    for _ in range(10):   # both at once: g2 only reads what g1 has written before
        with torch.cuda.stream(side):
            g2.replay()
        o3 = b.attend(dfl, window=100, sinks=4)
    torch.cuda.synchronize()
    check(o3, b.oracle(window=100, sinks=4), BF, 128, 400, 6.0)
    g1.replay()
    torch.cuda.synchronize()
    assert torch.equal(o1, k1) and torch.equal(o2, k2)
    assert warm.shape == o1.shape
