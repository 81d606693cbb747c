"""Edges of the attention over 8-bit pages on the GPU: which of its kernels takes
a batch, waits that run out, streams by number, captured calls, pages in two tables.

Tolerances are those of tests/test_gpu_paged_q8.py.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_gpu_paged import BF, DEV, HF, dfl  # noqa: E402, F401
from tests.test_gpu_paged_q8 import MANY, Batch8, check, check_attn  # noqa: E402


# --- around the bounds between the kernels ---------------------------------------

@pytest.mark.parametrize("d,dtype", [(64, HF), (128, BF)])
@pytest.mark.parametrize("heads,n_kv", [(4, 4), (8, 2), (14, 2), (16, 1), (17, 1), (32, 1), (33, 1), (128, 1)])
def test_rows_around_16_and_32(dfl, heads, n_kv, d, dtype):  # noqa: F811
    """As many rows as the kernels for few rows take on average, one token less and
    one more, in even and in uneven blocks."""
    group = heads // n_kv
    for rows in (16, 32):
        for tokens in (rows // group - 1, rows // group, rows // group + 1):
            if tokens < 1:
                continue
            check_attn(dfl, Batch8([(tokens, 70 + tokens)], heads, n_kv, d, dtype, prefix=90), shared=True)
            check_attn(dfl, Batch8([(tokens, 300), (tokens, tokens)], heads, n_kv, d, dtype), window=100, sinks=3)
            if tokens > 1:
                check_attn(dfl, Batch8([(2 * tokens - 1, 200), (1, 129)], heads, n_kv, d, dtype))


@pytest.mark.parametrize("heads,n_kv,d,dtype", [(32, 8, 128, BF), (14, 2, 64, HF)])
def test_a_prompt_among_single_tokens(dfl, heads, n_kv, d, dtype):  # noqa: F811
    """By its average the batch is one of few rows; the prompt is cut into many tiles."""
    check_attn(dfl, Batch8([(1, 40 + 3 * i) for i in range(30)] + [(150, 700)] + [(1, 513)], heads, n_kv, d, dtype))


@pytest.mark.parametrize("d,dtype", [(64, HF), (128, BF)])
def test_single_tokens_over_many_units(dfl, d, dtype):  # noqa: F811
    """More than 32 units of 32 keys a warp (page numbers are looked up that many at a time), and runs that end inside a tile."""
    check_attn(dfl, Batch8([(1, 100000)], 4, 1, d, dtype))
    check_attn(dfl, Batch8([(8, 66000), (1, 31), (7, 5000)], 4, 1, d, dtype), window=60001, sinks=1000)


@pytest.mark.parametrize("heads,n_kv,d,dtype", [(8, 2, 128, BF), (4, 4, 64, HF)])
def test_masks_of_few_rows(dfl, heads, n_kv, d, dtype):  # noqa: F811
    """Windows and first tokens that begin and end around units of 32 keys and steps of 128."""
    lens = [(1, 1000), (3, 161), (8, 129), (2, 2), (5, 4), (0, 7)]
    b = Batch8(lens, heads, n_kv, d, dtype)
    for window, sinks in ((1, 0), (1, 1), (31, 32), (32, 33), (33, 31), (128, 127), (129, 128), (1000, 5), (2 ** 31 - 1, 0)):
        check_attn(dfl, b, window=window, sinks=sinks)
        check_attn(dfl, b, window=window, sinks=sinks, causal=False)


def test_as_many_sequences_as_a_call_takes(dfl):  # noqa: F811
    rng = np.random.default_rng(3)
    lens = [(int(rng.integers(0, 3)), int(rng.integers(2, 150))) for _ in range(1024)]
    check_attn(dfl, Batch8(lens, 4, 2, 64, HF))
    check_attn(dfl, Batch8(lens, 4, 2, 64, HF, prefix=70), shared=True)


# --- what must not matter to few rows ------------------------------------------

@pytest.mark.parametrize("d,dtype", [(64, HF), (128, BF)])
def test_hidden_keys_may_hold_anything(dfl, d, dtype):  # noqa: F811
    """Keys that only some of the rows see: a later token's, and those before the window."""
    b = Batch8([(6, 300)], 8, 2, d, dtype)
    _, _, ks, vs = dfl.kv_pool_q8_views(b.pool, d)
    first = 297 - 294     # the first new token that sees key 297
    p, s = int(b.table[0, 297 // 64]), 297 % 64
    for array in (ks, vs):
        for value in (float("nan"), float("inf"), float("-inf")):
            kept, clean = array[p][:, s].clone(), b.attend(dfl)
            array[p][:, s] = value
            got = b.attend(dfl)
            assert torch.equal(got[:first], clean[:first])
            if array is vs or value != value:
                assert not got[first:].isfinite().any()
            array[p][:, s] = kept
    clean = b.attend(dfl, window=3, sinks=2)
    p, s = int(b.table[0, 4]), 290 - 256
    vs[p][:, s] = float("nan")
    ks[p][:, s + 1] = float("inf")
    assert torch.equal(b.attend(dfl, window=3, sinks=2), clean)


def test_broken_rows_harm_themselves_only(dfl):  # noqa: F811
    """A query of NaN or infinity, and a neighbour's cache of NaN, behind a prefix and alone."""
    b = Batch8([(3, 300), (2, 90), (1, 33)], 8, 2, 128, BF, prefix=130)
    clean = b.attend(dfl), b.attend_shared(dfl)
    b.q = b.q.clone()
    b.q[1, 3, 7], b.q[2, 1] = float("nan"), float("inf")
    _, _, ks, _ = dfl.kv_pool_q8_views(b.pool, 128)
    for p in b.table[1, :2].tolist():
        ks[p] = float("nan")
    for x, y in zip(clean, (b.attend(dfl), b.attend_shared(dfl))):
        away = torch.ones(6, 8, dtype=torch.bool, device=DEV)
        away[1, 3] = away[2, 1] = away[3:5] = False
        assert torch.equal(x[away], y[away]) and y[1, 3].isnan().all() and y[3:5].isnan().all()


def test_single_tokens_far_into_a_large_pool(dfl):  # noqa: F811
    """Pages beyond 2^32 bytes, of which a batch of single tokens sees a few."""
    b = Batch8([(1, 500), (1, 70), (1, 1), (4, 200)], 8, 2, 128, BF)
    ref, n = b.attend(dfl), b.pool.shape[0]
    big = torch.empty(160000, *b.pool.shape[1:], dtype=torch.uint8, device=DEV)
    assert big.numel() > 5 * 2 ** 30
    at = torch.linspace(123457, 159999, n, device=DEV).long()
    big[at] = b.pool
    table = torch.where(b.table < n, at.int()[b.table.clamp(max=n - 1).long()], b.table)
    got = dfl.dflash_paged_attn(b.q, big, b.q_start, b.kv_len, table.contiguous())
    assert torch.equal(got, ref)
    q = b.q.clone()
    dfl.dflash_kv_append(b.pool, b.k, b.v, b.q_start, b.kv_len, b.table, q=q, rope_base=1e4)
    dfl.dflash_kv_append(big, b.k, b.v, b.q_start, b.kv_len, table.contiguous(), q=q, rope_base=1e4)
    assert torch.equal(big[at], b.pool)


@pytest.mark.parametrize("heads,n_kv,d,dtype", [(8, 2, 128, BF), (4, 4, 64, HF), (8, 1, 128, HF)])
def test_rows_of_very_different_size(dfl, heads, n_kv, d, dtype):  # noqa: F811
    """Query rows far from 1 beside ordinary ones (of many rows, a row is scaled only where fp16 asks for it), and rows of zeros."""
    for lens in ([(2, 200), (1, 90)], [(40, 200), (17, 150)]):
        b = Batch8(lens, heads, n_kv, d, dtype, prefix=70)
        power = torch.tensor([-30 if dtype == BF else -9, -12, -1, 0, 0, 0, 2, 3], device=DEV).float()
        pick = torch.randint(0, 8, (b.T, heads, 1), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
        b.q = (b.q.float() * torch.exp2(power[pick])).to(dtype)
        b.q[1, 0] = 0.0
        clean = check_attn(dfl, b), check_attn(dfl, b, shared=True)
        big = b.q.clone()
        b.q[0, 1] = torch.finfo(dtype).max / 2    # nothing can be said of this row but that the others stay
        away = torch.ones(b.T, heads, dtype=torch.bool, device=DEV)
        away[0, 1] = False
        for x, y in zip(clean, (b.attend(dfl), b.attend_shared(dfl))):
            assert torch.equal(x[away], y[away])
        b.q = big


# --- waits that run out --------------------------------------------------------

@pytest.mark.parametrize("lens,prefix,waits", [([(40, 3000)], 0, True), ([(300, 900), (2, 70)], 0, True),
                                               ([(1, 90)] * 40, 700, True), (MANY, 700, True), ([(1, 3000)], 0, False)],
                         ids=["block", "prompt", "shared", "apart", "few"])
@pytest.mark.parametrize("d,dtype", [(64, HF), (128, BF)])
def test_any_call_that_is_given_up_ends_and_says_so(dfl, lens, prefix, waits, d, dtype):  # noqa: F811
    """(The kernel for few rows has no waits that could.)"""
    b = Batch8(lens, 8, 2, d, dtype, prefix=prefix)
    call = b.attend_shared if prefix else b.attend
    clean = call(dfl)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    dfl.dflash_debug_paged_wait_tries(0)
    try:
        call(dfl, status=status)
        torch.cuda.synchronize()
    finally:
        dfl.dflash_debug_paged_wait_tries()
    assert int(status) == int(waits)
    status.zero_()
    assert torch.equal(call(dfl, status=status), clean) and int(status) == 0


# --- streams and graphs --------------------------------------------------------

@pytest.mark.parametrize("handle", [0, 1])
def test_the_default_stream_by_its_number(dfl, handle):  # noqa: F811
    """The calls are ordered behind what that stream does before, also a slow fill."""
    lens = [(1, 300), (5, 90), (64, 64)]
    b, other = Batch8(lens, 8, 2, 64, BF, prefix=70), Batch8(lens, 8, 2, 64, BF, prefix=70, seed=1)
    calls = lambda b, **kw: (b.attend(dfl, **kw), b.attend_shared(dfl, **kw),
                             *dfl.dflash_kv_read(b.pool, b.T, b.q_start, b.kv_len, b.table, **kw))
    ref = calls(other)
    torch.cuda.synchronize()
    slow = torch.empty(1 << 28, device=DEV)
    for _ in range(10):
        slow.fill_(1.0)
    for x, y in ((b.pool, other.pool), (b.qkv, other.qkv), (b.table, other.table), (b.prefix_table, other.prefix_table)):
        x.copy_(y)
    got = calls(b, stream=handle)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, ref))


def test_a_captured_decode_behind_a_prefix(dfl):  # noqa: F811
    """64 growing caches, taken apart from their prefix: replays follow the lengths, and two graphs over one batch may run at once."""
    b = Batch8(MANY, 8, 2, 128, BF, prefix=300)
    b.attend_shared(dfl)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(b.attend_shared(dfl))
    full = b.kv_len.clone()
    for less in (0, 1, 700):
        b.kv_len.copy_((full - less).clamp(min=1))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        check(b, outs[0], b.oracle(prefix_table=b.prefix_np, prefix_len=300), 2000)
        assert torch.equal(*outs)
    kept, side = outs[0].clone(), torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(side):
            graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], kept) and torch.equal(outs[1], kept)


# --- pages -------------------------------------------------------------------------

@pytest.mark.parametrize("q", [1, 20])
def test_pages_in_two_tables(dfl, q):  # noqa: F811
    """Sequences that hold the same pages get the same results, also where a page comes up twice in one table."""
    b = Batch8([(q, 500), (q, 500), (q, 900)], 8, 2, 128, BF)
    b.table[1] = b.table[0]
    b.table[2, 9] = b.table[2, 3]
    b.q[q:2 * q] = b.q[:q]
    got = check_attn(dfl, b)
    assert torch.equal(got[:q], got[q:2 * q])


@pytest.mark.parametrize("q", [1, 3, 20])
def test_hidden_keys_that_are_larger(dfl, q):  # noqa: F811
    """Keys that a row does not see share an exponent with those it does. Of finite
    ones that is all they do: the tolerance counts the largest of the pool."""
    b = Batch8([(q, 200)], 8, 2, 128, BF)
    _, _, ks, vs = dfl.kv_pool_q8_views(b.pool, 128)
    for s in (150, 170):      # before the window
        p = int(b.table[0, s // 64])
        ks[p][:, s % 64] *= 2.0 ** 10
        vs[p][:, s % 64] *= 2.0 ** 10
    check_attn(dfl, b, window=200 - 171 - q)


# --- many rows ---------------------------------------------------------------------

@pytest.mark.parametrize("d,dtype", [(64, HF), (64, BF), (128, HF), (128, BF)])
def test_missing_pages_and_broken_rows_of_longer_blocks(dfl, d, dtype):  # noqa: F811
    """As for few rows: pages that are not there are not seen and are told of, rows of NaN and infinity harm themselves only."""
    b = Batch8([(40, 300), (50, 100)], 4, 2, d, dtype, prefix=130)
    b.table[0, 1] = -7
    b.table[1, 0] = b.pool.shape[0]
    b.prefix_table[1] = 2 ** 30
    b.prefix_np = b.prefix_table.cpu().numpy()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    clean = []
    for shared in (False, True):
        status.zero_()
        clean.append(check_attn(dfl, b, shared=shared, status=status))
        assert int(status) == 2
    b.q = b.q.clone()
    b.q[4, 3, 7], b.q[60, 1] = float("nan"), float("inf")
    away = torch.ones(90, 4, dtype=torch.bool, device=DEV)
    away[4, 3] = away[60, 1] = False
    for x, y in zip(clean, (b.attend(dfl), b.attend_shared(dfl))):
        assert torch.equal(x[away], y[away]) and y[4, 3].isnan().all()
