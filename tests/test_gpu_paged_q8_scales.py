"""What the scales of other keys may do to a row of the attention over 8-bit pages on
the GPU: those of keys that it does not see or that have no weight in it, and
those of keys whose values are zero.

Tolerances: those of tests/test_gpu_paged_q8.py against the definition, with the
largest value that has a weight in the row (max |v| there) in place of the pool's, and the
size of the scores of such keys. The weights' rounding counts for values 2^10 larger:
scales that lie closer together than that count as the largest of their step of 128
keys (of few rows, of their 32), whichever key has it; of others each is its key's alone.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_gpu_paged import BF, DEV, HF, dfl  # noqa: E402, F401
from tests.test_gpu_paged_q8 import Batch8, check, check_attn  # noqa: E402

KINDS = [(1, 8, 2, 128, BF), (3, 8, 2, 64, HF), (8, 8, 2, 128, BF), (20, 8, 2, 128, BF), (40, 4, 2, 64, HF), (90, 8, 2, 128, HF)]
POWERS = (9, 14, 31, 60)   # an outlier's scale beside ordinary ones


def compare(b, got, ref, keys):
    """`check` against the definition, the term of the weights' rounding 2^10 times as large (by way of the
    mass, which 2^-11 is multiplied to)."""
    out, mass, size, owned = ref
    more = keys * 2.0 ** -30 * np.abs(b.decoded()[:, 1]).max() * 2.0 ** 10
    check(b, got, (out, mass + 2.0 ** 11 * more, size, owned), keys, whole=True)


def put(b, dfl, seq, at, keys=None, values=None):  # noqa: F811
    """Multiplies the scales of the key at a position of a sequence."""
    _, _, ks, vs = dfl.kv_pool_q8_views(b.pool, b.d)
    p = int(b.table[seq, at // 64])
    if keys is not None:
        ks[p][:, at % 64] *= keys
    if values is not None:
        vs[p][:, at % 64] *= values


@pytest.mark.parametrize("q,heads,n_kv,d,dtype", KINDS)
def test_scales_in_front_of_the_window(dfl, q, heads, n_kv, d, dtype):  # noqa: F811
    """Keys that no row sees, in steps that rows see: the definition over an ordinary cache."""
    b = Batch8([(q, 300)], heads, n_kv, d, dtype)
    window = 300 - q - 170
    ref = b.oracle(bits=None, window=window)
    for at in (150, 100, 169):      # in the window's first units of 32 and steps of 128
        for power in POWERS:
            for kw in (dict(values=2.0 ** power), dict(keys=2.0 ** power), dict(keys=2.0 ** power, values=2.0 ** power)):
                clean = b.pool.clone()
                put(b, dfl, 0, at, **kw)
                got = b.attend(dfl, window=window)
                b.pool.copy_(clean)
                compare(b, got, ref, 300)


@pytest.mark.parametrize("q,heads,n_kv,d,dtype", KINDS[1:])
def test_scales_of_later_tokens(dfl, q, heads, n_kv, d, dtype):  # noqa: F811
    """Rows before a token do not see its key, which other rows of their tile do."""
    b = Batch8([(q, 300), (q, 129)], heads, n_kv, d, dtype, prefix=70)
    refs = b.oracle(bits=None), b.oracle(bits=None, prefix_table=b.prefix_np, prefix_len=70)
    sees = q - 1                    # only the last token of sequence 0
    rows = np.ones(2 * q, dtype=bool)
    rows[sees] = False
    for power in POWERS:
        for kw in (dict(values=2.0 ** power), dict(keys=2.0 ** power)):
            clean = b.pool.clone()
            put(b, dfl, 0, 299, **kw)
            got = b.attend(dfl), b.attend_shared(dfl)
            b.pool.copy_(clean)
            for g, (out, mass, size, owned) in zip(got, refs):
                compare(b, g, (out, mass, size, owned & rows), 370)


@pytest.mark.parametrize("q,heads,n_kv,d,dtype", KINDS)
def test_scales_of_keys_without_weight(dfl, q, heads, n_kv, d, dtype):  # noqa: F811
    """A key far below the others in every row (by 70 or more, so that its weight is below 2^-90)
    with larger values: it has no part in the output, and takes none from the others."""
    b = Batch8([(q, 300)], heads, n_kv, d, dtype)
    b.q = b.q.abs() + 0.5
    kc, _, ks, _ = dfl.kv_pool_q8_views(b.pool, d)
    _, mass, size, owned = b.oracle(bits=None)
    lowest = float((b.q.double().sum(dim=-1) * d ** -0.5 * 127).min())
    for at in (0, 130, 200):
        for power in POWERS:
            clean = b.pool.clone()
            p = int(b.table[0, at // 64])
            kc[p][:, at % 64], ks[p][:, at % 64] = 1, 75.0 / lowest     # code -126
            put(b, dfl, 0, at, values=2.0 ** power)
            got, out = b.attend(dfl), b.oracle(bits=None)[0]
            b.pool.copy_(clean)
            compare(b, got, (out, mass, size, owned), 300)


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


@pytest.mark.parametrize("q", [1, 8, 20, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_keys_as_large_as_the_type_holds(dfl, q, d):  # noqa: F811
    """bf16 keys near 2^127 and queries near 2^-106, and the other way round: the scores are ordinary."""
    for power in (-106, -60, 60, 100):
        b = Batch8([(q, 200)], 8, 2, d, BF)
        _, _, ks, _ = dfl.kv_pool_q8_views(b.pool, d)
        ks *= 2.0 ** min(-power + 20, 125)
        b.q = (b.q.float() * 2.0 ** power).to(BF)
        back = 2.0 ** (-power - min(-power + 20, 125))
        check_attn(dfl, b, scale=back * d ** -0.5)


@pytest.mark.parametrize("q,heads,n_kv,d", [(1, 8, 2, 128), (3, 8, 2, 64), (8, 8, 2, 128), (20, 8, 2, 128), (40, 4, 2, 64), (90, 8, 2, 128)])
def test_a_key_of_all_the_weight_without_values(dfl, q, heads, n_kv, d):  # noqa: F811
    """A key 20 or more above the others (in units of e) whose values are zeros: what is left of the
    others is small, and as precise as without it. Compared behind the factor between the two, by
    which the score's own error counts (its size is that key's)."""
    b = Batch8([(q, 300)], heads, n_kv, d, BF)
    b.q = b.q.abs() + 0.5
    kc, _, ks, vs = dfl.kv_pool_q8_views(b.pool, d)
    lowest = float((b.q.double().sum(dim=-1) * d ** -0.5 * 127).min())
    for at in (0, 130, 200):
        clean = b.pool.clone()
        p = int(b.table[0, at // 64])
        kc[p][:, at % 64], ks[p][:, at % 64], vs[p][:, at % 64] = 1, 75.0 / lowest, 0.0   # out of it all
        out, mass, _, owned = b.oracle(bits=None)
        kc[p][:, at % 64], ks[p][:, at % 64] = 255, 25.0 / lowest
        got, (_, less, size, _) = b.attend(dfl), b.oracle(bits=None)
        b.pool.copy_(clean)
        back = (mass.max(axis=-1) / less.max(axis=-1))[..., None]
        assert back.min() > 2.0 ** 20
        compare(b, got.double() * torch.from_numpy(back).to(DEV), (out, mass, size, owned), 300)
