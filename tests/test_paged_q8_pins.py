"""The oracle of 8-bit pages (oracle/paged_q8.py) against loops, and the
host-side refusals of the operators over them (no GPU: every refused call
returns before any CUDA call)."""
import ctypes

import numpy as np
import pytest

import block_diffusion_drafter_pass_gb300 as dfl
from oracle import paged_cache as pc
from oracle import paged_q8 as p8
from tests.test_paged_pins import FAKE, append_call, attn_call, batch, lib  # noqa: F401

Q8 = dfl.DFLASH_POOL_Q8


def test_codes_are_the_scalar_loop():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 16)) * np.exp(rng.standard_normal((5, 1)) * 3)
    codes, scales = p8.quantise(x)
    for r in range(5):
        m = max(abs(v) for v in x[r])
        assert scales[r] == m / 127
        for c, v in zip(codes[r], x[r]):
            assert c == round(v * (127 / m)) and -127 <= c <= 127
            assert abs(c * scales[r] - v) <= scales[r] * (0.5 + 1e-9)
    assert (np.abs(codes).max(axis=-1) == 127).all()


def test_rows_without_a_scale():
    x = np.array([[0.0, 0.0], [2.0 ** -101, 0.0], [2.0 ** -100, -(2.0 ** -101)], [np.inf, 1.0], [np.nan, 1.0]])
    codes, scales = p8.quantise(x)
    assert scales[0] == 0 and scales[1] == 0 and scales[2] == 2.0 ** -100 / 127 and np.isnan(scales[3:]).all()
    np.testing.assert_array_equal(codes, [[0, 0], [0, 0], [127, -64], [0, 0], [0, 0]])


def test_the_bytes_stand_for_the_rows():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((2, 3, 2, 64, 64))
    pool = p8.encode(k, v)
    assert pool.shape == (3, 2, 64 * (2 * 64 + 8))
    d = p8.decode(pool, 64)
    assert d.shape == (3, 2, 2, 64 * 64)
    for x, y in ((k, d[:, 0].reshape(3, 2, 64, 64)), (v, d[:, 1].reshape(3, 2, 64, 64).transpose(0, 1, 3, 2))):
        half = np.abs(x).max(axis=-1, keepdims=True) / 254
        assert (np.abs(x - y) <= half * (1 + 1e-6)).all() and np.abs(x - y).max() > 0.5 * half.min()
    # what cached() of the 16-bit oracle reads from it is a row of the original, within half a step
    got, _, there = pc.cached(d, np.array([2, 0]), 70, 64)
    assert there.all() and np.abs(got[69] - k[0, :, 5]).max() < 0.02


def test_rounding_to_bits_is_fp16s():
    rng = np.random.default_rng(3)
    x = rng.standard_normal(2000) * np.exp(rng.standard_normal(2000))
    x = x[np.abs(x) > 2.0 ** -13]
    np.testing.assert_array_equal(p8.rounded(x, 11), x.astype(np.float16).astype(np.float64))
    assert p8.rounded(np.array([0.0, 3.0, 2049.0, 2051.0]), 11).tolist() == [0.0, 3.0, 2048.0, 2052.0]


def test_the_views_of_a_pool_are_its_parts():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(2)
    pool = p8.encode(*rng.standard_normal((2, 3, 2, 64, 128)))
    views = dfl.kv_pool_q8_views(torch.from_numpy(pool), 128)
    for got, want, off in zip(views, p8.parts(pool, 128), (128, 128, 0, 0)):
        np.testing.assert_array_equal(got.double().numpy() - off, want)
    assert dfl.kv_pool_q8(2, 3, 64, device="cpu").shape == (2, 3, 64 * 136)


# --- refusals ------------------------------------------------------------------

def read_call(lib, b, **kw):
    f = dict(k=2 * FAKE, ks=128, v=3 * FAKE, vs=128)
    f.update(kw)
    return lib.dflash_kv_read(b, f["k"], f["ks"], f["v"], f["vs"], None)


BAD = [dict(dtype=Q8 + 2), dict(dtype=2 * Q8), dict(dtype=-Q8), dict(head_dim=32), dict(head_dim=256), dict(n_heads=0),
       dict(n_kv_heads=3), dict(n_seq=-1), dict(n_seq=1025), dict(n_tokens=(1 << 24) + 1), dict(pool=None),
       dict(page_table=None), dict(q_start=None), dict(kv_len=None), dict(pool=FAKE + 8), dict(n_pages=0),
       dict(table_pages=0), dict(table_stride=1), dict(table_pages=(1 << 20) + 1, table_stride=1 << 25)]


@pytest.mark.parametrize("bad", BAD, ids=lambda b: ",".join(f"{k}={v}" for k, v in b.items()))
def test_broken_batches_are_refused(lib, bad):  # noqa: F811
    b = ctypes.byref(batch(**dict(dict(dtype=Q8), **bad)))
    assert append_call(lib, b) == dfl.DFLASH_EINVAL
    assert read_call(lib, b) == dfl.DFLASH_EINVAL
    assert attn_call(lib, b) == dfl.DFLASH_EINVAL
    assert attn_call(lib, b, shared=True) == dfl.DFLASH_EINVAL
    n = ctypes.c_size_t(7)
    assert lib.dflash_paged_attn_workspace(b, ctypes.byref(n)) == dfl.DFLASH_EINVAL and n.value == 0


@pytest.mark.parametrize("dtype", [0, 1, Q8, Q8 + 1])
@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(v=FAKE + 2), dict(ks=120), dict(vs=132),
                                 dict(v=2 * FAKE), dict(v=2 * FAKE + 3 * 256 + 16), dict(k=3 * FAKE - 512)])
def test_read_refusals(lib, bad, dtype):  # noqa: F811
    assert read_call(lib, ctypes.byref(batch(dtype=dtype)), **bad) == dfl.DFLASH_EINVAL
    assert lib.dflash_last_error(None)


def test_buffers_in_the_pool_are_refused(lib):  # noqa: F811
    """The pool's size is counted by its format: 3 pages of 2 heads of 64 * 136 bytes."""
    size = 3 * 2 * 64 * 136
    b = ctypes.byref(batch(dtype=Q8, pool=FAKE))
    for at in (FAKE, FAKE + size - 16):
        assert read_call(lib, b, k=at, v=8 * FAKE) == dfl.DFLASH_EINVAL and b"pool" in lib.dflash_last_error(None)
        assert read_call(lib, b, v=at, k=8 * FAKE) == dfl.DFLASH_EINVAL and b"pool" in lib.dflash_last_error(None)
        assert append_call(lib, b, k=at, v=8 * FAKE, q=9 * FAKE, qo=9 * FAKE) == dfl.DFLASH_EINVAL
        assert attn_call(lib, b, q=8 * FAKE, out=at) == dfl.DFLASH_EINVAL
    # right behind it: only the workspace is missing
    assert attn_call(lib, b, q=8 * FAKE, out=FAKE + size, ws=None) in (dfl.DFLASH_EINVAL, dfl.DFLASH_ECUDA)
    assert b"pool" not in lib.dflash_last_error(None)


def test_an_empty_batch_is_no_work(lib):  # noqa: F811
    for b in (batch(dtype=Q8, n_seq=0), batch(dtype=Q8, n_tokens=0), batch(n_tokens=0)):
        b = ctypes.byref(b)
        assert append_call(lib, b) == dfl.DFLASH_OK
        assert read_call(lib, b, k=None, v=None) == dfl.DFLASH_OK
        assert attn_call(lib, b) == dfl.DFLASH_OK
        assert attn_call(lib, b, shared=True) == dfl.DFLASH_OK


def test_tensors_of_the_wrong_kind_are_refused_before_the_library():
    torch = pytest.importorskip("torch")
    pool = dfl.kv_pool_q8(3, 2, 64, device="cpu")   # not on a GPU
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    q = torch.zeros(4, 8, 64, dtype=torch.bfloat16)
    for call in (lambda: dfl.dflash_kv_append(pool, k, k, i(3), i(2), i(2, 2)),
                 lambda: dfl.dflash_kv_read(pool, 4, i(3), i(2), i(2, 2)),
                 lambda: dfl.dflash_kv_read(pool, -1, i(3), i(2), i(2, 2)),
                 lambda: dfl.dflash_kv_read(pool, (1 << 32) + 4, i(3), i(2), i(2, 2)),
                 lambda: dfl.dflash_kv_read(pool.view(-1), 4, i(3), i(2), i(2, 2)),
                 lambda: dfl.dflash_kv_read(dfl.kv_pool(3, 2, 64, device="cpu"), 4, i(3), i(2), i(2, 2), dtype=torch.float16),
                 lambda: dfl.dflash_paged_attn(q, pool, i(3), i(2), i(2, 2)),
                 lambda: dfl.dflash_shared_prefix_attn(q, pool, i(3), i(2), i(2, 2), i(2), 100)):
        with pytest.raises(dfl.DFlashError):
            call()
