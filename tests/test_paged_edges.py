"""Host-side checks of the paged-cache operators at edges (no GPU)."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

import block_diffusion_drafter_pass_gb300 as dfl
from block_diffusion_drafter_pass_gb300 import _build


# --- how places are dealt to the CTAs ------------------------------------------

@pytest.fixture(scope="module")
def deal(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("deal")
    src, lib = os.path.join(d, "deal.cpp"), os.path.join(d, "deal.so")
    with open(src, "w") as f:
        f.write('#include "paged_deal.h"\nextern "C" int run_of(long long all, int ctas) {\n'
                '  return dfl::deal_fits(all, ctas) ? dfl::deal_run(all, ctas) : -1;\n}\n')
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    "-static-libubsan", "-I", _build.CSRC, src, "-o", lib], check=True)
    fn = ctypes.CDLL(lib).run_of
    fn.argtypes, fn.restype = [ctypes.c_longlong, ctypes.c_int], ctypes.c_int
    return fn


def test_runs_hold_every_place(deal):
    """All places are dealt, in runs no longer than they need to be (but for the
    rounding of very long ones) whose halves of the ring an int counts; what is
    longer than that does not fit."""
    rng = random.Random(1)
    for ctas in (1, 2, 7, 148, 152, 1024):
        most = ctas * 2 ** 29
        edges = [most + d for d in (-ctas, -1, 0, 1)] + [2 ** 31 + d for d in (-1, 0, 1)] + [4 * most, 2 ** 31 * ctas - 1]
        for places in [0, 1, ctas, ctas + 1] + edges + [int(2 ** rng.uniform(0, 50)) for _ in range(300)]:
            run = deal(places, ctas)
            if places >= most:
                assert run == -1
            else:
                up = 2 ** max(0, places.bit_length() - 31)
                spare = 1 if up == 1 else 2 * up
                assert run * ctas >= places and (run - spare) * ctas < max(places, 1) and 2 * run < 2 ** 31


# --- streams -------------------------------------------------------------------

def test_a_stream_of_another_device_is_refused():
    """Its work would run on the pool's device's current stream instead."""
    torch = pytest.importorskip("torch")

    class Stream:
        cuda_stream, device_index = 12345, 1

    with pytest.raises(dfl.DFlashError, match="another device"):
        dfl._run_on(torch, 0, Stream(), lambda s: pytest.fail("the call ran"))


# --- refusals ------------------------------------------------------------------

FAKE = 1 << 20   # a non-null, aligned address that no refused call reads


def batch(**kw):
    f = dict(dtype=0, n_heads=8, n_kv_heads=2, head_dim=64, n_seq=2, n_tokens=4, n_pages=3, table_pages=2,
             table_stride=2, pool=FAKE, page_table=FAKE, q_start=FAKE, kv_len=FAKE, status=None)
    f.update(kw)
    return ctypes.byref(dfl.dflash_paged_batch(*[f[n] for n, _ in dfl.dflash_paged_batch._fields_]))


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return dfl.load_library()


@pytest.mark.parametrize("scale,refused", [(1.8e38, True), (3.4e38, True), (2.0 ** 127, False), (1e-45, False)])
def test_scales_whose_product_with_log2_e_is_infinite_are_refused(lib, scale, refused):
    """(Others are refused for their workspace, or fail without a GPU.)"""
    for shared in (False, True):
        args = (2 * FAKE, 512, 3 * FAKE, 512)
        if shared:
            r = lib.dflash_shared_prefix_attn(batch(), FAKE, 100, *args, 1, scale, None, 0, None)
        else:
            r = lib.dflash_paged_attn(batch(), *args, 0, 0, 1, scale, None, 0, None)
        assert r != dfl.DFLASH_OK and (b"scale" in lib.dflash_last_error(None)) == refused


POOL = 3 * 2 * 2 * 64 * 64 * 2   # bytes of the pool of `batch`
ROWS = (4 - 1) * 1024 + 1024     # and of four tokens' queries


@pytest.mark.parametrize("at,refused", [(0, True), (POOL - 16, True), (16 - ROWS, True), (POOL, False), (-ROWS, False)])
def test_outputs_in_the_pool_are_refused(lib, at, refused):
    """(Others are refused for their workspace, or fail without a GPU.)"""
    out = 8 * FAKE + at
    pool = batch(pool=8 * FAKE)
    for shared in (False, True):
        args = (2 * FAKE, 512, out, 512)
        if shared:
            r = lib.dflash_shared_prefix_attn(pool, FAKE, 100, *args, 1, 0.1, None, 0, None)
        else:
            r = lib.dflash_paged_attn(pool, *args, 0, 0, 1, 0.1, None, 0, None)
        assert r != dfl.DFLASH_OK and (b"in the pool" in lib.dflash_last_error(None)) == refused


@pytest.mark.parametrize("name", ["k", "v", "q", "q_out"])
def test_appended_rows_in_the_pool_are_refused(lib, name):
    f = dict(k=FAKE, v=2 * FAKE, q=3 * FAKE, q_out=4 * FAKE)
    f[name] = 8 * FAKE + 1024
    r = lib.dflash_kv_append(batch(pool=8 * FAKE), f["k"], 128, f["v"], 128, f["q"], 512, f["q_out"], 512, None, 0.0, None)
    assert r == dfl.DFLASH_EINVAL and b"in the pool" in lib.dflash_last_error(None)
