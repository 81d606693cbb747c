"""What the scales of other keys may do to a row of the attention over 8-bit pages on
the GPU: those of keys whose values are zero.

Tolerances: those of tests/test_gpu_paged_q8.py.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_gpu_paged import BF, DEV, dfl  # noqa: E402, F401
from tests.test_gpu_paged_q8 import Batch8, check_attn  # noqa: E402


@pytest.mark.parametrize("power", [0, 30, 50, 60, 100])
@pytest.mark.parametrize("lens,heads,n_kv", [([(2, 1024)], 8, 2), ([(8, 1024)], 8, 2), ([(40, 1024), (3, 700)], 8, 2), ([(200, 1500)], 4, 2),
                                             ([(1, 20013)], 8, 1), ([(16, 20013)], 8, 1), ([(64, 20013)], 8, 1)])
def test_zero_values_behind_larger_ones(dfl, power, lens, heads, n_kv):  # noqa: F811
    """Keys count in the sum whatever their values are, also when the sum's parts
    lie in other warps and CTAs; the larger values come first, or last."""
    for d in (64, 128):
        b = Batch8(lens, heads, n_kv, d, BF)
        _, _, _, vs = dfl.kv_pool_q8_views(b.pool, d)
        kept = vs.clone()
        for first in (True, False):
            vs.copy_(kept)
            for i, n in enumerate(b.kv_len.tolist()):
                pages = b.table[i, :(n + 63) // 64].tolist()
                half = len(pages) // 2
                for p in pages[:half]:
                    vs[p] *= 2.0 ** power if first else 0.0
                for p in pages[half:]:
                    vs[p] *= 0.0 if first else 2.0 ** power
            check_attn(dfl, b)


@pytest.mark.parametrize("power", [0, 50, 60, 100])
@pytest.mark.parametrize("lens", [[(1, 300)] * 5, [(40, 300), (1, 70)], [(1, 1 + 23 * i) for i in range(64)]], ids=["few", "many", "apart"])
def test_zero_values_behind_a_prefix_of_larger_ones(dfl, power, lens):  # noqa: F811
    for d in (64, 128):
        b = Batch8(lens, 8, 2, d, BF, prefix=500)
        _, _, _, vs = dfl.kv_pool_q8_views(b.pool, d)
        kept, own = vs.clone(), torch.ones(b.pool.shape[0], dtype=torch.bool, device=DEV)
        own[b.prefix_table.long()] = False
        for zero in (own, ~own):
            vs.copy_(kept)
            vs[zero] = 0.0
            vs[~zero] *= 2.0 ** power
            check_attn(dfl, b, shared=True)
