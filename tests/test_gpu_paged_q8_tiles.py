"""Batches in whose CTAs tiles of one stream and of two follow each other, in the
attention over 8-bit pages on the GPU. Tolerances: tests/test_gpu_paged_q8.py.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_gpu_paged import BF, HF, dfl  # noqa: E402, F401
from tests.test_gpu_paged_q8 import Batch8, check_attn  # noqa: E402


@pytest.mark.parametrize("heads,n_kv,d,dtype", [(4, 1, 128, BF), (4, 1, 64, HF), (8, 2, 128, HF)])
def test_many_short_prompts(dfl, heads, n_kv, d, dtype):  # noqa: F811
    """Tiles of one stream, of two and of one again, of a step or a few, many in each CTA."""
    rng = np.random.default_rng(11)
    lens = []
    for i in range(600):
        q = int(rng.integers(17, 33)) if i % 2 else int(rng.integers(33, 65))
        lens.append((q, q + int(rng.choice([0, 0, 60, 120, 300]))))
    b = Batch8(lens, heads, n_kv, d, dtype)
    got = check_attn(dfl, b)
    assert all(torch.equal(got, b.attend(dfl)) for _ in range(20))
    windowed = check_attn(dfl, b, window=40, sinks=3)
    assert all(torch.equal(windowed, b.attend(dfl, window=40, sinks=3)) for _ in range(20))
