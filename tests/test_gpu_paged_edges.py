"""Paged-cache operators at edges of the page pool and the lengths."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle import paged_cache as pc  # noqa: E402
from tests.test_gpu_paged import BF, DEV, HF, Batch, dfl, f64, poison  # noqa: E402, F401


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


@pytest.mark.parametrize("lens,prefix", [([(1, 3000)], 0), ([(300, 900), (2, 70)], 0), ([(1, 90)] * 40, 700)], ids=str)
@pytest.mark.parametrize("d,dtype", [(64, HF), (128, BF)])
def test_any_call_that_is_given_up_ends_and_says_so(dfl, lens, prefix, d, dtype):
    b = Batch(lens, 8, 2, d, dtype, prefix=prefix)
    call = b.attend_shared if prefix else b.attend
    clean = call(dfl)
    status = torch.zeros(1, dtype=torch.int32, device=b.pool.device)
    dfl.dflash_debug_paged_wait_tries(0)
    try:
        call(dfl, status=status)
        torch.cuda.synchronize()
    finally:
        dfl.dflash_debug_paged_wait_tries()
    assert int(status) == 1
    status.zero_()
    assert torch.equal(call(dfl, status=status), clean) and int(status) == 0


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


def misses(b, shared, window=0, sinks=0, causal=True):
    """Whether some new token sees a key whose page is outside the pool."""
    away = lambda ids: (ids < 0) | (ids >= b.pool.shape[0])
    table, pre = b.table.cpu().numpy(), b.prefix_table.cpu().numpy()
    for _, i, pos in pc.places(b.q_start.tolist(), b.kv_len.tolist()):
        key = np.arange(int(b.kv_len[i]))
        see = key <= (pos if causal else len(key))
        if window:
            see &= (key > pos - window) | (key < sinks)
        if (see & away(table[i][key // 64])).any():
            return True
        key = np.arange(b.prefix if shared else 0)
        if ((key <= (b.prefix + pos if causal else b.prefix)) & away(pre[key // 64])).any():
            return True
    return False


@pytest.mark.parametrize("seed", range(16))
def test_the_status_says_when_a_page_that_is_seen_is_missing(dfl, seed):
    """And only then: pages past what the tokens see, or before their windows, may be missing."""
    rng = np.random.default_rng(seed)
    lens = [(int(a), int(a + n)) for a, n in zip(rng.integers(0, 40, 3), rng.integers(0, 500, 3))] + [(1, 1)]
    b = Batch(lens, 8, 2, (64, 128)[seed % 2], BF, prefix=int(rng.integers(1, 400)), seed=seed)
    for _ in range(rng.integers(1, 4)):
        b.table[int(rng.integers(0, 4)), int(rng.integers(0, b.table.shape[1]))] = -1
    if seed % 4 == 3:
        b.prefix_table[int(rng.integers(0, len(b.prefix_table)))] = 2 ** 31 - 1
    status = torch.zeros(1, dtype=torch.int32, device=b.pool.device)
    for window, sinks, causal in ((0, 0, True), (0, 0, False), (60, 0, True), (130, 70, False), (3, 1, True)):
        status.zero_()
        b.attend(dfl, window=window, sinks=sinks, causal=causal, status=status)
        assert int(status) == (2 if misses(b, False, window, sinks, causal) else 0), (window, sinks, causal)
    for causal in (True, False):
        status.zero_()
        b.attend_shared(dfl, causal=causal, status=status)
        assert int(status) == (2 if misses(b, True, causal=causal) else 0), causal


# --- single pages far into a cache ---------------------------------------------

class FarCache:
    """One sequence of about 2^22 cached tokens (behind a prefix of about 2^21),
    nearly all in 16 pages over and over whose keys count for 2% together. Single
    places far apart have pages of their own, each with one key that has its share
    of the rest and a value of its own, so a page that is lost, read twice or taken
    from elsewhere moves the output by far more than the tolerance: the first
    page, one near 2^21 keys, the last, and those on both sides of places where
    one CTA's run of steps ends and the next one's begins."""

    def __init__(self, tokens, d, dtype, prefix, window=0, sinks=0, seed=3):
        rng = np.random.default_rng(seed)
        self.heads, self.d, self.dtype, self.tokens = 8, d, dtype, tokens
        self.window, self.sinks = window, sinks
        n_own, self.len = 65536, 65536 * 64 - 5
        self.prefix = 32768 * 64 - 43 if prefix else 0
        n_pre = (self.prefix + 63) // 64
        own, pre = rng.integers(0, 16, n_own), rng.integers(0, 16, n_pre)
        # the line of steps that is dealt to the CTAs: 4 places, then a tile's steps (2 pages each)
        ctas = torch.cuda.get_device_properties(0).multi_processor_count
        first = (self.len - tokens - window + 1) // 128 if window else 0
        lead = (sinks + 127) // 128 if window else n_pre // 2
        steps, tiles = lead + n_own // 2 - first, -(-tokens // 32)
        run = -(-tiles * (steps + 4) // ctas)
        self.run, self.pieces = run, -(-steps // run) + 1
        at = {("own", n_own - 1), ("own", n_own - 40)}
        if window:
            at |= {("own", 0), ("own", (self.len - window) // 64 + 1), ("own", 1)}   # a first token's, the window's, one hidden
        else:
            at |= {("own", 0), ("own", 32768), ("own", 32767)}
        if prefix:
            at |= {("pre", 0), ("pre", n_pre - 1), ("pre", n_pre // 2)}
        for tile in range(tiles):
            for c in (1, ctas // tiles // 3, ctas // tiles - 1):
                edge = (-(-tile * (steps + 4) // run) + c) * run - tile * (steps + 4) - 4
                for step, page in ((edge - 1, 1), (edge, 0)):
                    if lead <= step < steps:
                        at.add(("own", (step - lead + first) * 2 + page))
                    elif prefix and 0 <= step < lead:
                        at.add(("pre", step * 2 + page))
        at = sorted(at)
        for i, (where, p) in enumerate(at):
            (own if where == "own" else pre)[p] = 16 + i
        self.own, self.pre, self.places = own, pre, at
        pages = 16 + len(at)
        g = torch.Generator(device=DEV).manual_seed(seed)
        normal = lambda *s: torch.randn(s, generator=g, device=DEV)
        self.pool = normal(pages, 2, 1, 64 * d).to(dtype)
        keys, values = self.pool[:, 0].view(pages, 64, d), self.pool[:, 1].view(pages, d, 64)
        keys[:, :, :8] = 0
        self.q = normal(tokens, 8, d).to(dtype)
        self.q[:, :, :8] = 4
        self.slots = []
        for i, (where, p) in enumerate(at):
            slot = 18 if p in (n_own - 1, n_pre - 1) else int(rng.integers(0, 64))   # the last pages are not full
            score = 16.5 + 0.1 * (i % 12)
            self.slots.append(slot)
            keys[16 + i, slot] = 0
            keys[16 + i, slot, :8] = score / (32 * d ** -0.5)
        i32 = lambda x: torch.from_numpy(np.asarray(x, dtype=np.int32)).to(DEV)
        self.table, self.prefix_table = i32(own)[None], i32(pre)
        self.q_start, self.kv_len = i32([0, tokens]), i32([self.len])

    def call(self, dfl):
        if self.prefix:
            return dfl.dflash_shared_prefix_attn(self.q, self.pool, self.q_start, self.kv_len, self.table,
                                                 self.prefix_table, self.prefix)
        return dfl.dflash_paged_attn(self.q, self.pool, self.q_start, self.kv_len, self.table, window=self.window,
                                     sinks=self.sinks)

    def counts(self, table, lo, hi):
        """How often each slot of each page lies in the positions [lo, hi) of a table."""
        n = np.zeros((self.pool.shape[0], 64))
        if hi <= lo:
            return n
        a, b = lo // 64, (hi - 1) // 64
        n += np.bincount(table[a:b + 1], minlength=len(n))[:, None]
        n[table[a], :lo % 64] -= 1
        n[table[b], (hi - 1) % 64 + 1:] -= 1
        return n

    def seen(self, token):
        pos = self.len - self.tokens + token
        lo = max(0, pos - self.window + 1) if self.window else 0
        return (self.counts(self.own, lo, pos + 1) + self.counts(self.own, 0, min(self.sinks, lo)) +
                self.counts(self.pre, 0, self.prefix))

    def reference(self, without=None):
        """(out, sum of w |v|, largest score size, largest weight), each [tokens, heads, ...], in 64 bits."""
        pool, q = f64(self.pool), f64(self.q)
        k = pool[:, 0].reshape(-1, self.d)
        v = pool[:, 1].reshape(-1, self.d, 64).transpose(0, 2, 1).reshape(-1, self.d)
        n = np.stack([self.seen(t) for t in range(self.tokens)])
        if without is not None:
            n[:, without] = np.maximum(n[:, without] - 1, 0)
        n = n.reshape(self.tokens, 1, -1)
        s = np.einsum("thd,kd->thk", q, k) * self.d ** -0.5
        size = (np.einsum("thd,kd->thk", np.abs(q), np.abs(k)) * self.d ** -0.5).max(-1)
        w = n * np.exp(s - s.max(-1, keepdims=True))
        total = w.sum(-1, keepdims=True)
        w /= total
        return w @ v, w @ np.abs(v), size[..., None], w.max(-1, keepdims=True)


FAR = [dict(tokens=3, prefix=False), dict(tokens=40, prefix=False), dict(tokens=3, prefix=True),
       dict(tokens=40, prefix=True), dict(tokens=1, prefix=False, window=(1 << 20) + 33, sinks=40)]


@pytest.mark.parametrize("d,dtype", [(128, BF), (64, HF), (64, BF), (128, HF)])
@pytest.mark.parametrize("shape", FAR, ids=str)
def test_single_pages_far_into_a_cache(dfl, shape, d, dtype):
    """Tolerance as in the tests of short caches, with the sums as they are made:
    a product adds 16 keys at a time, 8 times a step, a CTA's run of steps after
    each other, then the pieces; fp16 weights below 2^-14 are off by up to 2^-31
    of the largest."""
    c = FarCache(d=d, dtype=dtype, **shape)
    out, mass, size, top = c.reference()
    u = 2.0 ** -8 if dtype == BF else 2.0 ** -11
    sums = (8 * c.run + c.run + c.pieces + 104) * 2.0 ** -23
    tol = u * (mass + np.abs(out)) + (2 * (d / 16 + 4) * 2.0 ** -23 * size + 2.0 ** -21 + sums) * mass
    if dtype == HF:
        tol += (c.len + c.prefix) * 2.0 ** -31 * top * float(c.pool.abs().max()) + 2.0 ** -25
    seen = c.seen(0)
    for i, place in enumerate(c.places):   # what is looked for is not below the tolerance
        if seen[16 + i, c.slots[i]]:
            assert (np.abs(c.reference(without=16 + i)[0] - out) / tol).max() > 3, place
    got = f64(c.call(dfl))
    bad = np.abs(got - out) / tol
    assert np.isfinite(got).all() and bad.max() <= 1, bad.max()
