"""The paged-cache oracle (oracle/paged_cache.py) against brute force, and the
host-side refusals of the operators (no GPU: every refused call returns before
any CUDA call)."""
import ctypes
import math

import numpy as np
import pytest

import block_diffusion_drafter_pass_gb300 as dfl
from block_diffusion_drafter_pass_gb300 import _build
from oracle import paged_cache as pc


def make(rng, lens, n_kv, d, spare=2):
    """Pool of random pages with each sequence's pages scattered in it."""
    need = [(n + 63) // 64 for _, n in lens]
    total = sum(need) + spare
    order = rng.permutation(total)
    width = max(need + [1])
    table, at = np.zeros((len(lens), width), dtype=np.int32), 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    q_start = np.concatenate([[0], np.cumsum([a for a, _ in lens])]).astype(np.int32)
    return rng.standard_normal((total, 2, n_kv, 64 * d)), table, q_start, np.array([n for _, n in lens], np.int32), order[at:]


def test_rotation_is_a_complex_rotation_and_keeps_norms():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 64))
    pos = np.array([0, 1, 63, 262143, 2 ** 30])
    y = pc.rotate(x, pos, 1e6)
    z = (x[..., :32] + 1j * x[..., 32:]) * np.exp(1j * pos[:, None] * 1e6 ** (-np.arange(32) / 32.0))[:, None]
    np.testing.assert_allclose(y, np.concatenate([z.real, z.imag], -1), atol=1e-6)
    np.testing.assert_allclose(y[0], x[0])
    np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    np.testing.assert_array_equal(pc.rotate(x, pos, 0), x)


@pytest.mark.parametrize("window,sinks,causal", [(0, 0, True), (5, 0, True), (5, 3, True), (70, 2, True), (0, 0, False),
                                                 (4, 1, False), (1, 0, True)])
def test_attention_is_the_scalar_loop(window, sinks, causal):
    rng = np.random.default_rng(1)
    lens = [(1, 1), (3, 70), (0, 5), (2, 130)]
    n_kv, d, heads = 2, 8, 4
    pool, table, q_start, kv_len, _ = make(rng, lens, n_kv, d)
    q = rng.standard_normal((6, heads, d))
    got, mass, _, owned = pc.attention(q, pool, q_start, kv_len, table, 0.3, window, sinks, causal)
    assert owned.all()
    t = 0
    for i, (a, n) in enumerate(lens):
        for j in range(a):
            p = n - a + j
            for h in range(heads):
                num, den, absn = np.zeros(d), 0.0, np.zeros(d)
                for key in range(n):
                    if causal and key > p:
                        continue
                    if window and not (key > p - window or key < sinks):
                        continue
                    page = pool[table[i, key // 64]]
                    kk = [page[0, h // 2, (key % 64) * d + e] for e in range(d)]
                    vv = np.array([page[1, h // 2, e * 64 + key % 64] for e in range(d)])
                    w = math.exp(0.3 * sum(q[t, h, e] * kk[e] for e in range(d)))
                    num, den, absn = num + w * vv, den + w, absn + w * np.abs(vv)
                np.testing.assert_allclose(got[t, h], num / den, rtol=1e-9, atol=1e-12)
                np.testing.assert_allclose(mass[t, h], absn / den, rtol=1e-9)
            t += 1


def test_a_shared_prefix_is_the_concatenated_cache():
    rng = np.random.default_rng(2)
    P, n_kv, d = 128, 1, 8                                  # whole pages, so one table can hold both
    lens = [(2, 9), (1, 64), (3, 65)]
    pool, table, q_start, kv_len, spare = make(rng, lens, n_kv, d, spare=2)
    q = rng.standard_normal((6, 3, d))
    a = pc.attention(q, pool, q_start, kv_len, table, 1.0, prefix_table=spare, prefix_len=P)[0]
    joined = np.concatenate([np.tile(spare[None], (3, 1)), table], axis=1)
    b = pc.attention(q, pool, q_start, kv_len + P, joined, 1.0)[0]
    np.testing.assert_allclose(a, b, rtol=1e-12)
    np.testing.assert_array_equal(pc.attention(q, pool, q_start, kv_len, table, 1.0)[0],
                                  pc.attention(q, pool, q_start, kv_len, table, 1.0, prefix_table=spare, prefix_len=0)[0])


def test_rows_that_see_nothing_are_zero():
    rng = np.random.default_rng(3)
    pool, table, q_start, kv_len, _ = make(rng, [(3, 2)], 1, 8)   # the first token lies before its cache
    out, _, _, _ = pc.attention(rng.standard_normal((3, 1, 8)), pool, q_start, kv_len, table, 1.0)
    assert (out[0] == 0).all() and (out[1:] != 0).any()


def test_append_then_attend_equals_a_dense_cache():
    rng = np.random.default_rng(4)
    lens = [(4, 66), (1, 1)]
    pool, table, q_start, kv_len, _ = make(rng, lens, 1, 8)
    k, v, q = (rng.standard_normal((5, 1, 8)) for _ in range(3))
    new, qr = pc.append(pool, k, v, q_start, kv_len, table, 1e4, q=q)
    kk, vv, _ = pc.cached(new, table[0], 66, 8)
    np.testing.assert_allclose(kk[62:], pc.rotate(k[:4], np.arange(62, 66), 1e4))
    np.testing.assert_allclose(vv[62:], v[:4])
    np.testing.assert_allclose(qr[4], q[4])                   # position 0
    np.testing.assert_allclose(kk[:62], pc.cached(pool, table[0], 62, 8)[0])
    assert (np.abs(new - pool) > 0).sum() == 2 * 5 * 8


# --- refusals ----------------------------------------------------------------

@pytest.fixture(scope="module")
def lib():
    _build.build()
    return dfl.load_library()


FAKE = 1 << 20   # a non-null, aligned address that no refused call reads


def batch(**kw):
    f = dict(dtype=0, n_heads=8, n_kv_heads=2, head_dim=64, n_seq=2, n_tokens=4, n_pages=3, table_pages=2,
             table_stride=2, pool=FAKE, page_table=FAKE, q_start=FAKE, kv_len=FAKE, status=None)
    f.update(kw)
    b = dfl.dflash_paged_batch()
    for name, value in f.items():
        setattr(b, name, value)
    return b


BAD_BATCH = [dict(dtype=2), dict(dtype=-1), dict(head_dim=32), dict(head_dim=256), dict(n_heads=0), dict(n_kv_heads=0),
             dict(n_kv_heads=3), dict(n_heads=258, n_kv_heads=2), dict(n_seq=-1), dict(n_seq=1025), dict(n_tokens=-1),
             dict(n_tokens=(1 << 24) + 1), dict(pool=None), dict(page_table=None), dict(q_start=None), dict(kv_len=None),
             dict(pool=FAKE + 2), dict(n_pages=0), dict(table_pages=0), dict(table_stride=1),
             dict(table_pages=(1 << 24) + 1, table_stride=1 << 25),
             dict(table_pages=(1 << 20) + 1, table_stride=1 << 25), dict(n_heads=129, n_kv_heads=129)]


def append_call(lib, b, **kw):
    f = dict(k=FAKE, ks=128, v=2 * FAKE, vs=128, q=3 * FAKE, qs=512, qo=3 * FAKE, qos=512, pos=None, base=1e4)
    f.update(kw)
    return lib.dflash_kv_append(b, f["k"], f["ks"], f["v"], f["vs"], f["q"], f["qs"], f["qo"], f["qos"], f["pos"],
                                f["base"], None)


def attn_call(lib, b, shared=False, **kw):
    f = dict(q=FAKE, qs=512, out=2 * FAKE, os=512, window=0, sinks=0, causal=1, scale=0.1, ws=FAKE, wb=1 << 40,
             pt=FAKE, pl=100)
    f.update(kw)
    if shared:
        return lib.dflash_shared_prefix_attn(b, f["pt"], f["pl"], f["q"], f["qs"], f["out"], f["os"], f["causal"],
                                             f["scale"], f["ws"], f["wb"], None)
    return lib.dflash_paged_attn(b, f["q"], f["qs"], f["out"], f["os"], f["window"], f["sinks"], f["causal"],
                                 f["scale"], f["ws"], f["wb"], None)


@pytest.mark.parametrize("bad", BAD_BATCH, ids=lambda b: ",".join(f"{k}={v}" for k, v in b.items()))
def test_broken_batches_are_refused(lib, bad):
    b = ctypes.byref(batch(**bad))
    assert append_call(lib, b) == dfl.DFLASH_EINVAL
    assert attn_call(lib, b) == dfl.DFLASH_EINVAL
    assert attn_call(lib, b, shared=True) == dfl.DFLASH_EINVAL
    assert lib.dflash_last_error(None)
    n = ctypes.c_size_t(7)
    assert lib.dflash_paged_attn_workspace(b, ctypes.byref(n)) == dfl.DFLASH_EINVAL and n.value == 0


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(v=FAKE + 4), dict(ks=64),
                                 dict(vs=132), dict(q=None), dict(qo=None), dict(q=FAKE + 2), dict(qs=516),
                                 dict(qos=0), dict(base=1.0), dict(base=-5.0), dict(base=float("nan")),
                                 dict(base=float("inf")),
                                 dict(qo=FAKE + 3 * 256 + 128), dict(qo=2 * FAKE - 3 * 1024), dict(qo=3 * FAKE + 16),
                                 dict(qo=3 * FAKE, qos=1024)])
def test_append_refusals(lib, bad):
    assert append_call(lib, ctypes.byref(batch()), **bad) == dfl.DFLASH_EINVAL


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("bad", [dict(q=None), dict(out=None), dict(q=FAKE + 2), dict(out=FAKE + 8), dict(qs=504),
                                 dict(os=513), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                                 dict(scale=float("inf")),
                                 dict(out=FAKE), dict(out=FAKE + 3 * 1024 + 1008), dict(out=FAKE - 3 * 1024 - 16),
                                 dict(qs=1024, os=1024, out=FAKE + 1008), dict(qs=1024, os=512, out=FAKE + 1024)])
def test_attention_refusals(lib, bad, shared):
    assert attn_call(lib, ctypes.byref(batch()), shared=shared, **bad) == dfl.DFLASH_EINVAL


def test_window_and_prefix_refusals(lib):
    b = ctypes.byref(batch())
    assert attn_call(lib, b, window=-1) == dfl.DFLASH_EINVAL
    assert attn_call(lib, b, window=5, sinks=-1) == dfl.DFLASH_EINVAL
    assert attn_call(lib, b, shared=True, pl=-1) == dfl.DFLASH_EINVAL
    assert attn_call(lib, b, shared=True, pl=(1 << 30) + 1) == dfl.DFLASH_EINVAL
    assert attn_call(lib, b, shared=True, pl=(1 << 26) + 1) == dfl.DFLASH_EINVAL
    assert attn_call(lib, b, shared=True, pt=None) == dfl.DFLASH_EINVAL
    assert lib.dflash_paged_attn_workspace(b, None) == dfl.DFLASH_EINVAL
    assert lib.dflash_kv_append(None, FAKE, 128, FAKE, 128, None, 0, None, 0, None, 0.0, None) == dfl.DFLASH_EINVAL


@pytest.mark.parametrize("kw", [dict(out=FAKE + 4 * 1024), dict(out=FAKE - 4 * 1024),
                                dict(qs=1024, os=1024, out=FAKE + 1024), dict(qs=1536, os=1536, out=FAKE - 1536)])
def test_rows_that_share_nothing_pass_the_overlap_check(lib, kw):
    """Neighbouring buffers, and column ranges of one wider matrix: refused for the workspace only."""
    assert attn_call(lib, ctypes.byref(batch()), ws=None, **kw) in (dfl.DFLASH_EINVAL, dfl.DFLASH_ECUDA)
    assert b"overlap" not in lib.dflash_last_error(None)


def test_an_empty_batch_is_no_work(lib):
    for b in (batch(n_seq=0), batch(n_tokens=0), batch(n_seq=0, pool=None, page_table=None, q_start=None, kv_len=None)):
        b = ctypes.byref(b)
        assert append_call(lib, b) == dfl.DFLASH_OK
        assert attn_call(lib, b) == dfl.DFLASH_OK
        assert attn_call(lib, b, shared=True) == dfl.DFLASH_OK


def test_tensors_of_the_wrong_kind_are_refused_before_the_library():
    torch = pytest.importorskip("torch")
    pool = torch.zeros(3, 2, 2, 64 * 64, dtype=torch.bfloat16)   # not on a GPU
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    q = torch.zeros(4, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(dfl.DFlashError):
        dfl.dflash_kv_append(pool, k, k, i(3), i(2), i(2, 2))
    with pytest.raises(dfl.DFlashError):
        dfl.dflash_paged_attn(q, pool, i(3), i(2), i(2, 2))
    with pytest.raises(dfl.DFlashError):
        dfl.dflash_shared_prefix_attn(q, pool, i(3), i(2), i(2, 2), i(1), 100)
    # numbers that a C int would wrap
    for kw in (dict(window=(1 << 32) + 100), dict(window=-1), dict(window=5, sinks=1 << 31)):
        with pytest.raises(dfl.DFlashError, match="window and sinks"):
            dfl.dflash_paged_attn(q, pool, i(3), i(2), i(2, 2), **kw)
    for n in (-1, (1 << 26) + 1, (1 << 32) + 64):
        with pytest.raises(dfl.DFlashError, match="prefix_len"):
            dfl.dflash_shared_prefix_attn(q, pool, i(3), i(2), i(2, 2), i(1), n)
