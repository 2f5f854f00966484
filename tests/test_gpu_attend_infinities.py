"""GPU tests of the attention over a binary16 cache with infinities and NaN in places that rows see: what the
definition gives, wherever in a sequence they lie."""
import numpy as np
import pytest

import moe_expert_amd as M
from tests import kv_refs as R
from tests.gpu_util import dev, host
from tests.test_gpu_attend import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vkind", ["f16", "q8_0", "iq4_nl"])
@pytest.mark.parametrize("dim,heads", [(64, 20), (128, 5), (192, 5), (256, 1)])
def test_infinite_keys(dim, heads, vkind):
    """A key of an infinity gives a score of one: at -inf the position has the weight 0, at +inf the row is NaN, and where
    the query's value there is 0 too.  Beside it, a key whose score is 120 below the rest has no weight either,
    and gives the bits that a row is to have."""
    n, found = 260, False
    for sign in (1.0, -1.0):
        for where in (0, 3, 100, n - 1):
            print(f"infinite key {dim} {heads} {vkind} {sign} {where}", flush=True)
            c = Case([n], kinds=("f16", vkind), heads=heads, kv=1, dim=dim, page=16, seed=where)
            q = host(c.q).reshape(heads, dim)
            q[:, 7] += np.copysign(0.1, q[:, 7])
            if heads > 1:
                q[0, 7] = 0.0
            c.q = dev(q.reshape(1, -1))
            pg, at = c.pages[0, where // 16], where % 16
            c.raw[0][pg, 0, at, 7] = sign * np.inf
            got, lse = (host(t) for t in c.run())
            got = got.reshape(heads, dim)
            low = sign * q[:, 7] < 0
            found |= low.any()
            assert np.isnan(got[~low]).all() and np.isnan(lse[0, ~low]).all()
            # the same with a finite key far below
            for h in np.flatnonzero(low):
                key = c.raw[0][pg, 0, at].copy()
                rest = c.scale * (q[h].astype(np.float64) @ np.where(np.isinf(key), 0, key.astype(np.float64)))
                key[7] = (-120.0 - rest) / (c.scale * q[h, 7])
                c.val[0][pg, 0, at] = key.astype(np.float64)
                o, l, bound, lbound, _ = c.want()
                assert (np.abs(got[h] - o[0, h * dim:(h + 1) * dim]) <= (bound + np.abs(o) * R.U)[0, h * dim:(h + 1) * dim]).all()
                assert abs(lse[0, h] - l[0, h]) <= lbound[0, h]
                saved = c.raw[0][pg, 0, at].copy()
                c.raw[0][pg, 0, at] = key
                finite, _ = c.run()
                c.raw[0][pg, 0, at] = saved
                assert np.array_equal(host(finite).reshape(heads, dim)[h], got[h])
    assert found


def test_keys_of_both_infinities():
    """Opposite infinities in one key, and NaN: the score is NaN, and so is the row."""
    for value in ((np.inf, np.inf), (np.inf, -np.inf), (-np.inf, np.inf), (np.nan, 1.0), (-np.inf, np.nan)):
        c = Case([150], kinds=("f16", "f16"), heads=4, kv=1, dim=64, page=16)
        q = np.abs(host(c.q)) + 0.1
        q[0, 3::2] *= -1
        c.q = dev(q)
        for where in (5, 149):
            raw = c.raw[0].copy()
            c.raw[0][c.pages[0, where // 16], 0, where % 16, 2:4] = value
            got, lse = (host(t) for t in c.run())
            c.raw[0][:] = raw
            s = q.reshape(4, 64)[:, 2].astype(np.float64) * value[0] + q.reshape(4, 64)[:, 3] * value[1]
            if (s == -np.inf).all():
                assert np.isfinite(got).all() and np.isfinite(lse).all()
            else:
                assert not (s == -np.inf).any() and np.isnan(got).all() and np.isnan(lse).all()


@pytest.mark.parametrize("dim,heads,kv", [(64, 40, 2), (96, 5, 1), (128, 10, 2), (192, 3, 1), (256, 2, 2)])
def test_infinite_values(dim, heads, kv):
    """An infinite value gives its infinity to the rows that see it, two opposite ones and NaN give NaN, wherever they
    lie; other dims keep every bit."""
    n = 260
    for where in (0, 3, 100, 131, n - 1):
        for first, second, want in ((np.inf, None, np.inf), (-np.inf, None, -np.inf), (np.inf, np.inf, np.inf), (np.inf, -np.inf, np.nan),
                                    (np.nan, None, np.nan), (-np.inf, np.nan, np.nan)):
            print(f"infinite value {dim} {heads} {where} {first} {second}", flush=True)
            c = Case([n, 20], new=[2, 1], kinds=("f16", "f16"), heads=heads, kv=kv, dim=dim, page=16, seed=where)
            clean, lse = (host(t) for t in c.run())
            put = [(where, first)] + ([] if second is None else [((where + 37) % (n - 1), second)])
            for j, value in put:
                c.raw[1][c.pages[0, j // 16], :, j % 16, 9] = value
            got, lse2 = (host(t) for t in c.run())
            assert np.array_equal(lse, lse2)
            got, clean = got.reshape(3, heads, dim), clean.reshape(3, heads, dim)
            other = np.arange(dim) != 9
            assert np.array_equal(got[:, :, other], clean[:, :, other]) and np.array_equal(got[2], clean[2])
            for t in range(2):
                seen = [value for j, value in put if j <= n - 2 + t]
                if len(seen) == len(put):
                    assert np.array_equal(got[t, :, 9], np.full(heads, want), equal_nan=True)
                elif not seen:
                    assert np.array_equal(got[t], clean[t])
                else:
                    assert np.array_equal(got[t, :, 9], np.full(heads, seen[0]), equal_nan=True)


@pytest.mark.parametrize("window", [0, 50])
def test_written_infinities(window):
    """Values beyond binary16 that a write makes infinities of, keys and values of one position, a long sequence."""
    c = Case([900], kinds=("f16", "f16"), heads=4, kv=1, dim=64, page=16)
    q = host(c.q).reshape(4, 64)
    q[:, 4] = np.abs(q[:, 4]) + 0.1
    c.q = dev(q.reshape(1, -1))
    clean, lse = (host(t) for t in c.run(window))
    j = 860
    x = np.zeros((2, 1, 64), np.float32)
    x[0, 0, 4], x[1, 0, 6] = -70000.0, 80000.0
    cache = c.cache()
    pages, lens, _ = c.args()
    M.qmm_kv_write(cache, pages, lens - (900 - 1 - j), dev(x[0]), dev(x[1]))
    got, lse2 = (host(t) for t in c.run(window, cache=cache))
    # weight 0 and an infinite value: NaN in that dim, the other dims without the position
    val = c.val[0][c.pages[0, j // 16], 0, j % 16]
    val[:] = 0
    val[4] = -120.0 / c.scale / q[:, 4].min()
    o, l, bound, lbound, _ = c.want(window)
    got, o, bound = got.reshape(4, 64), o.reshape(4, 64), bound.reshape(4, 64)
    other = np.arange(64) != 6
    assert np.isnan(got[:, 6]).all()
    assert (np.abs(got - o)[:, other] <= (bound + np.abs(o) * R.U)[:, other]).all()
    assert (np.abs(lse2 - l) <= lbound).all()


def test_nothing_but_infinities():
    """Every score of a row -inf: as a row that sees no position."""
    for n in (1, 70, 300):
        c = Case([n], kinds=("f16", "f16"), heads=2, kv=1, dim=64, page=16)
        q = host(c.q)
        q[0, 5], q[0, 64 + 5] = 1.0, -1.0
        c.q = dev(q)
        c.raw[0][:, :, :, 5] = -np.inf
        got, lse = (host(t) for t in c.run())
        assert (got[0, :64] == 0).all() and np.isneginf(lse[0, 0])
        assert np.isnan(got[0, 64:]).all() and np.isnan(lse[0, 1])
