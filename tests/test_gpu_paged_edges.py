"""Paged-cache operators at edges of the page pool and the lengths."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_gpu_paged import BF, HF, Batch, dfl, poison  # noqa: E402, F401


# Lengths that end in either page of a step of 128 keys, at its slots 1, 8, 13 and 63, and at its end.
TAILS = [
    ("own", dict(lens=[(1, 1), (1, 70), (16, 100), (3, 129), (40, 40), (1, 900), (5, 136), (2, 191), (7, 64), (9, 128)])),
    ("own", dict(lens=[(200, 1101), (130, 141), (1, 13)])),       # rows of both streams of a CTA
    ("own", dict(lens=[(16, 20013)])),                            # split between CTAs
    ("window", dict(lens=[(300, 1103), (1, 513), (20, 77)])),
    ("shared", dict(lens=[(1, 1 + 11 * i) for i in range(40)], prefix=1077)),
    ("shared", dict(lens=[(16, 40), (0, 9), (3, 3), (90, 301)], prefix=8)),
    ("shared", dict(lens=[(2, 63), (1, 65)], prefix=127)),
]


@pytest.mark.parametrize("heads,n_kv,d,dtype", [(8, 2, 128, BF), (28, 4, 64, HF), (4, 4, 64, BF), (8, 1, 128, HF)])
@pytest.mark.parametrize("kind,shape", TAILS, ids=lambda x: str(x)[:40])
def test_slots_past_a_length_change_no_bit(dfl, kind, shape, heads, n_kv, d, dtype):
    """Not even by another way through the kernel: NaN or infinity there costs nothing."""
    b = Batch(heads=heads, n_kv=n_kv, d=d, dtype=dtype, **shape)
    call = {"own": lambda: b.attend(dfl), "window": lambda: b.attend(dfl, window=200, sinks=70),
            "shared": lambda: b.attend_shared(dfl)}[kind]
    clean = call()
    assert clean.isfinite().all()
    for value in (float("nan"), float("-inf")):
        poison(b, dfl, value)
        assert torch.equal(call(), clean)


# --- streams given as numbers --------------------------------------------------

@pytest.mark.parametrize("handle", [0, 1])
def test_the_default_stream_by_its_number(dfl, handle):
    """0 is what `torch.cuda.current_stream().cuda_stream` says by default: the
    calls are ordered behind what that stream does before, also a slow fill."""
    b = Batch([(1, 300), (5, 90)], 8, 2, 64, BF, prefix=70)
    other = Batch([(1, 300), (5, 90)], 8, 2, 64, BF, prefix=70, seed=1)
    ref = other.attend(dfl), other.attend_shared(dfl)
    torch.cuda.synchronize()
    slow = torch.empty(1 << 28, device=b.pool.device)
    for _ in range(10):
        slow.fill_(1.0)                          # about 2 ms of work ahead of the copies
    b.pool.copy_(other.pool)
    b.qkv.copy_(other.qkv)
    b.table.copy_(other.table)
    b.prefix_table.copy_(other.prefix_table)
    results = b.attend(dfl, stream=handle), b.attend_shared(dfl, stream=handle)
    assert dfl._run_on(torch, 0, handle, lambda s: s) == 0
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(results, ref))
    with pytest.raises(dfl.DFlashError, match="per-thread"):
        b.attend(dfl, stream=2)


# --- waits that run out --------------------------------------------------------

def broken_neighbour(dfl):
    """32 sequences behind a prefix, the fourth with a cache of NaN: the rows of
    the others in its tiles are done again, key by key, while the kernel's other
    roles wait for milliseconds."""
    b = Batch([(16, 40 + 7 * i) for i in range(32)], 32, 8, 128, BF, prefix=16000)
    clean = b.attend_shared(dfl)
    for p in b.table[3, :1].tolist():
        b.pool[p] = float("nan")
    return b, clean


def check_broken(b, clean, got):
    mine = torch.zeros(b.T, dtype=torch.bool, device=got.device)
    mine[48:64] = True
    assert got[mine].isnan().all() and (got[~mine].float() - clean[~mine].float()).abs().max() < 0.05


def test_rows_that_are_done_again_keep_the_waits_going(dfl):
    """They take longer than a wait may (about 70 ms), but each of their pages counts."""
    b, clean = broken_neighbour(dfl)
    status = torch.zeros(1, dtype=torch.int32, device=b.pool.device)
    dfl.dflash_debug_paged_wait_tries(20000)   # 20 ms at most
    try:
        check_broken(b, clean, b.attend_shared(dfl, status=status))
    finally:
        dfl.dflash_debug_paged_wait_tries()
    assert int(status) == 0


def test_a_wait_that_runs_out_says_so(dfl):
    """With no time at all the same call is given up: the status says so, nothing
    hangs, and the next calls are right."""
    b, clean = broken_neighbour(dfl)
    status = torch.zeros(1, dtype=torch.int32, device=b.pool.device)
    dfl.dflash_debug_paged_wait_tries(0)
    try:
        b.attend_shared(dfl, status=status)
        torch.cuda.synchronize()
    finally:
        dfl.dflash_debug_paged_wait_tries()
    assert int(status) == 1
    status.zero_()
    check_broken(b, clean, b.attend_shared(dfl, status=status))
    assert int(status) == 0
    with pytest.raises(dfl.DFlashError):
        dfl.dflash_debug_paged_wait_tries(-1)
    with pytest.raises(dfl.DFlashError):
        dfl.dflash_debug_paged_wait_tries((1 << 23) + 1)


# --- pages given back ----------------------------------------------------------

@pytest.mark.parametrize("window,sinks,free", [(30, 0, 15), (41, 0, 14), (30, 4, 15), (30, 70, 15)])
@pytest.mark.parametrize("new", [1, 3])
def test_pages_before_the_window_may_be_given_back(dfl, window, sinks, free, new):
    """Also the one that shares a step with the window's first; those of the first tokens stay."""
    b = Batch([(new, 1000), (new, 70)], 8, 2, 128, BF)
    status = torch.zeros(1, dtype=torch.int32, device=b.pool.device)
    whole = b.attend(dfl, window=window, sinks=sinks)
    b.table[0, (sinks + 63) // 64:free] = -1
    assert torch.equal(b.attend(dfl, window=window, sinks=sinks, status=status), whole)
    assert int(status) == 0
    b.table[0, 15] = -1                                      # the window's own
    b.attend(dfl, window=window, sinks=sinks, status=status)
    assert int(status) == 2
