"""GPU tests of the attention over values whose blocks' scales lie far apart, or are not finite, against its
definition in 64 bits."""
import numpy as np
import pytest

from tests import kv_refs as R
from tests.gpu_util import host
from tests.test_gpu_attend import Case

pytestmark = pytest.mark.gpu

BLOCK_VALUES = [("f16", "q8_0"), ("f16", "iq4_nl"), ("q8_0", "q8_0"), ("q8_0", "iq4_nl"), ("iq4_nl", "iq4_nl")]


def scales_of(c, side=1):
    """The scales [page, head, place, block] of a block format's side, a view of its bytes."""
    kind = c.kinds[side]
    raw = c.raw[side].reshape(c.npages, c.kv, -1)
    return raw[:, :, c.page * (c.dim // 32) * R.FACTOR[kind]:].view(np.float16).reshape(c.npages, c.kv, c.page, c.dim // 32)


def value_again(c, side=1):
    """What the side's bytes stand for."""
    for p in range(c.npages):
        for h in range(c.kv):
            c.val[side][p, h] = R.chunk_values(c.raw[side][p, h], c.kinds[side], c.page, c.dim)


def put_key(c, position, row):
    """A row of binary32 values as the key of head 0 at a position of the first sequence."""
    pg, at, kind = c.pages[0, position // c.page], position % c.page, c.kinds[0]
    if kind == "f16":
        c.raw[0][pg, 0, at] = row
    else:
        code, d = R.quantize(row[None].astype(np.float32), kind)
        one = R.chunk_bytes(code, d, kind)
        fb = c.dim // 32 * R.FACTOR[kind]
        flat = c.raw[0][pg, 0].reshape(-1)
        flat[at * fb:(at + 1) * fb] = one[:fb]
        scales_of(c, 0)[pg, 0, at] = d[0]
    c.val[0][pg, 0, at] = R.stored(row[None].astype(np.float32), kind)[0]


def led(n, kinds, dim, lead, at, **kw):
    """A sequence of n positions whose scores are near zero but for one, `lead` above them."""
    c = Case([n], kinds=kinds, heads=1, kv=1, dim=dim, page=16, kscale=0.01, **kw)
    q = host(c.q)[0]
    put_key(c, at, q / np.square(q).sum() / c.scale * lead)
    return c


def spread(c, factor):
    """Scales of the values times factor (broadcast to [page, head, place, block]), in binary16."""
    s = scales_of(c)
    s[:] = (s.astype(np.float64) * factor).astype(np.float16)


def nothing_at(c, position, blocks):
    """Values of zero at a position: factors of zero beside their scale, or, where no level is zero, a scale of zero."""
    pg, at, nb = c.pages[0, position // c.page], position % c.page, c.dim // 32
    if c.kinds[1] == "q8_0":
        f = c.raw[1][pg, 0].reshape(-1)[:c.page * nb * 32].reshape(c.page, 16, nb, 2)
        f[at][:, blocks] = 0
    else:
        scales_of(c)[pg, 0, at, blocks] = 0


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("kinds", BLOCK_VALUES)
@pytest.mark.parametrize("n,lead,down", [(4096, 14.0, 10), (300, 12.0, 13), (300, 8.0, 16), (20, 8.0, 8)])
def test_blocks_apart(dim, kinds, n, lead, down):
    """Blocks of a head whose scales are a power of two below their neighbours', with one position of nearly all the weight
    whose values there are zero: what the others give is as exact as beside blocks of one scale."""
    print(f"blocks apart {dim} {kinds} {n} {lead} {down}", flush=True)
    for at in (1, n - 1):
        c = led(n, kinds, dim, lead, at, seed=dim + n)
        nb = dim // 32
        factor = np.where(np.arange(nb) % 2, 2.0 ** -down, 1.0) if down < 16 else 2.0 ** (6 - np.arange(nb) * 16.0 / (nb - 1))
        spread(c, factor)
        nothing_at(c, at, np.arange(1, nb))
        value_again(c)
        c.check()


@pytest.mark.parametrize("kinds", BLOCK_VALUES)
@pytest.mark.parametrize("dim", [64, 96, 256])
def test_blocks_and_positions_apart(dim, kinds):
    """Scales that differ from block to block and from position to position, many heads, several tokens of a sequence.

    Weights times scales enter the products in two binary16 parts after a power of two that puts the row's largest weight
    times its block's largest scale D in [2^13, 2^15): each is off by up to 2^-25 there beside 2^-21 of itself, which
    over the positions is 2^-38 D sum |factor| of what the largest weight is 1 in; the sum of all weights is at least 1."""
    rng = np.random.default_rng(dim)
    c = Case([700, 90, 33], new=[3, 1, 2], kinds=kinds, heads=10, kv=2, dim=dim, page=16, qscale=2.0, seed=dim)
    nb = dim // 32
    spread(c, 2.0 ** rng.uniform(-14, 0, (c.npages, c.kv, 1, nb)) * 2.0 ** rng.uniform(-8, 8, (c.npages, c.kv, c.page, nb)))
    value_again(c)
    got, lse = c.run()
    o, l, bound, lbound, live = c.want()
    d = np.abs(scales_of(c).astype(np.float64))
    seq, pos = R.positions(c.off, c.lens, c.ntok, 3)
    for t in range(c.ntok):
        n = int(pos[t]) + 1
        pg, at = c.pages[seq[t], np.arange(n) // 16], np.arange(n) % 16
        for h in range(c.heads):
            top = d[pg, h // 5, at].max(axis=0)  # of each block
            v = np.abs(c.val[1][pg, h // 5, at]).reshape(n, nb, 32)
            factors = (v / np.maximum(d[pg, h // 5, at], 1e-30)[..., None]).sum(axis=0)
            bound[t, h * dim:(h + 1) * dim] += (2.0 ** -38 * top[:, None] * factors).reshape(-1)
    c.compare(got, lse, (o, l, bound, lbound, live), "f32")


@pytest.mark.parametrize("odd", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("kinds", BLOCK_VALUES)
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_scale_that_is_not_finite(dim, kinds, odd):
    """One block with such a scale at one position, in the first steps, the middle and the last: NaN in that block of the
    rows that see it, and no digit less anywhere else."""
    n, nb = 500, dim // 32
    for where in (0, 40, 255, n - 1):
        print(f"not finite {dim} {kinds} {odd} {where}", flush=True)
        c = led(n, kinds, dim, 8.0, 77, seed=where)
        spread(c, np.where(np.arange(nb) % 2, 0.05, 1.0))
        value_again(c)
        o, l, bound, lbound, _ = c.want()
        scales_of(c)[c.pages[0, where // 16], 0, where % 16, 0] = odd
        got, lse = (host(t) for t in c.run())
        assert np.isnan(got[0, :32]).all()
        assert (np.abs(got - o)[0, 32:] <= (bound + np.abs(o) * R.U)[0, 32:]).all()
        assert (np.abs(lse - l) <= lbound).all()


@pytest.mark.parametrize("kinds", BLOCK_VALUES)
def test_scales_that_a_row_does_not_see(kinds):
    """The largest scales there are, and ones that are not finite, at the last token's position alone: the tokens before
    it keep every bit, and so does everything behind a window."""
    import torch
    for lens, window in (([45], 0), ([300], 0), ([300], 40)):
        c = Case(lens, new=[4], kinds=kinds, heads=6, kv=2, dim=128, page=16)
        clean, lse = c.run(window)
        for value in (65504.0, -65504.0, np.inf, np.nan):
            last = lens[0] - 1
            s = scales_of(c)
            old = s.copy()
            s[c.pages[0, last // 16], :, last % 16, 1] = value
            if window:
                s[c.pages[0, 16], :, 0, 2] = value  # position 256, in a step that is read, before every row's window
            got, lse2 = c.run(window)
            s[:] = old
            assert torch.equal(got[:3], clean[:3]) and torch.equal(lse, lse2)
            other = got[3].view(6, 4, 32)[:, [0, 2, 3]]
            assert torch.isfinite(other).all() and torch.equal(other, clean[3].view(6, 4, 32)[:, [0, 2, 3]])


@pytest.mark.parametrize("odd", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("kinds", [("q8_0", "q8_0"), ("q8_0", "iq4_nl"), ("iq4_nl", "iq4_nl")])
def test_key_scale_that_is_not_finite(kinds, odd):
    """It counts times the sum of its block's products: a score of -inf, without weight, or a row of NaN."""
    for n, where in ((40, 39), (300, 0), (300, 140)):
        c = Case([n], kinds=kinds, heads=8, kv=1, dim=96, page=16, seed=where)
        q = host(c.q).reshape(8, 96).astype(np.float64)
        pg, at = c.pages[0, where // 16], where % 16
        s = scales_of(c, 0)
        sums = q[:, 32:64] @ (c.val[0][pg, 0, at, 32:64] / float(s[pg, 0, at, 1]))
        assert (np.abs(sums) > 1).all()
        s[pg, 0, at, 1] = odd
        got, lse = (host(t) for t in c.run())
        got = got.reshape(8, 96)
        gone = sums * odd < 0
        assert np.isnan(got[~gone]).all() and np.isnan(lse[0, ~gone]).all()
        key = c.val[0][pg, 0, at]
        for h in np.flatnonzero(gone):
            key[:] = -120.0 / c.scale * q[h] / np.square(q[h]).sum()
            o, l, bound, lbound, _ = c.want()
            rows = slice(96 * h, 96 * h + 96)
            assert (np.abs(got[h] - o[0, rows]) <= (bound + np.abs(o) * R.U)[0, rows]).all()
            assert abs(lse[0, h] - l[0, h]) <= lbound[0, h]


@pytest.mark.parametrize("kinds", [("f16", "f16"), ("q8_0", "iq4_nl")])
def test_largest_scale(kinds):
    """The largest factors that are finite, against queries of zero and ones so small that scores are ordinary."""
    for scale, q in ((3.3e38, 0.0), (-3.3e38, 0.0), (3.0e38, 1e-38), (2.0 ** 127, 2.0 ** -126)):
        c = Case([90], kinds=kinds, heads=4, kv=2, dim=64, page=16, qscale=q)
        c.scale = scale
        c.check()
