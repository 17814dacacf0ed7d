"""GPU: the softmax weights of the paged attention where they lie far apart: one key far above a long tail, tiles
that go up and down, block scales far apart beside a flat tail.  Every share is one whole row, so that nothing but
the kernel's own running reference separates the keys.

A value weight W enters the product as e4m3(W) + e5m2(W - e4m3(W)), by way of fp16.  Per weight:
  W >= 2^-6   e4m3's half step is 2^-4 of W, so the rest is at most 2^-4 of it and e5m2's half step of that 2^-8 of
              W; fp16's rounding adds 2^-12:                                  at most 1.09 * 2^-8 of W
  W < 2^-6    e4m3's step is 2^-9, the rest at most 2^-10 and e5m2's half step of that 2^-14; fp16 adds
              2^-18 at most:                                                   at most 1.07 * 2^-14
and a row of up to t tiles of 128 keys has a weight of t or more (references go down as t grows), so that its small
weights lose at most 128 t * 1.07 * 2^-14 against t: 1.07 * 2^-7, however long the row.
All values here are positive, so that this is relative to the output itself, whose bf16 rounding is 2^-8 more.
The scores have few products that are not zero: 16 roundings of a number up to |s| + 64 (as in paged_ref.attend,
whose 1032 are for 1024 products)."""

import math

import numpy as np
import pytest

import paged_ref as ref

pytestmark = pytest.mark.gpu

D, P, SHARES = 512, 64, 152
SCALE = 0.0625
LOG2E = 1.4426950408889634
BIG = 1.09 * 2.0 ** -8                 # a weight's own error
SMALL = 1.07 * 2.0 ** -7               # what all small weights of a row add up to
# One weight of t and a flat tail of 128 t weights W lose 128 e / (1 + 128 W) of their sum, e the error of W: for W
# below 2^-11 (e half as large: its rest is below 2^-11) at most 0.0040, from there to 2^-6 at most
# 128 * 1.07 * 2^-14 / (1 + 2^-4) = 0.0079, above it BIG = 0.0043.  A tail that is not flat loses less.
TAIL = 0.0079
BF16 = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    import torch
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)


def _values(rng, n):
    """Codes of n keys: columns 0 to 2 (which the scores are made of) zero, positive values in the others."""
    codes = ref.encode(60.0 * rng.uniform(0.1, 1.9, (n, D)))
    codes[:, :3] = 0
    return codes


def _run(codes, scales, q, sink=None, selection=False):
    """All rows of q [R, H, 512] over the same n keys (codes [n, 512], n a multiple of 64, scales [n / S]); returns
    (out, want, rel) with rel the scores' error bound, all in 64 bits."""
    import torch
    from deepseek_v4_top_gb300 import dsa
    n, R, H = codes.shape[0], q.shape[0], q.shape[1]
    S = n // scales.shape[0]
    cache = torch.from_numpy(codes.reshape(n // P, P, D)).cuda()
    cs = torch.from_numpy(scales.reshape(n // P, P // S).astype(np.float32)).cuda()
    pages = torch.arange(n // P, dtype=torch.int32, device="cuda").repeat(R, 1).contiguous()
    lens = torch.full((R,), n, dtype=torch.int32, device="cuda")
    qt = torch.from_numpy(q.astype(np.float32)).cuda().to(torch.bfloat16)
    ts = None if sink is None else torch.from_numpy(sink.astype(np.float32)).cuda()
    out = torch.empty((R, H, D), dtype=torch.bfloat16, device="cuda")
    if selection:
        idx = torch.arange(n, dtype=torch.int32, device="cuda").repeat(R, 1).contiguous()
        dsa.dsa_paged_sparse_attn(qt, cache, cs, pages, lens, idx, lens, ts, SCALE, out)
    else:
        dsa.dsa_paged_attn(qt, cache, cs, pages, lens, ts, SCALE, out)
    assert dsa.dsa_get_device_error() == 0
    kv = torch.from_numpy(ref.decode(codes) * np.repeat(scales, S)[:, None]).cuda()
    want = torch.empty((R, H, D), dtype=torch.float64, device="cuda")
    rel = 0.0
    for r in range(0, R, 8):
        s = torch.einsum("rhd,nd->rhn", qt[r:r + 8].double(), kv) * SCALE
        rel = max(rel, (s.abs().max().item() + 64) * 16 * 2.0 ** -24)
        top = s.amax(2, keepdim=True)
        if ts is not None:
            top = torch.maximum(top, ts.double()[None, :, None])
        e = torch.exp(s - top)
        den = e.sum(2)
        if ts is not None:
            den = den + torch.exp(ts.double()[None] - top[..., 0])
        want[r:r + 8] = torch.einsum("rhn,nd->rhd", e, kv) / den[..., None]
    return out.double(), want, rel


def _check(out, want, tol):
    """The error of each row and head against its norm; all weights' errors might have one sign."""
    import torch
    assert torch.isfinite(out).all()
    err = (out - want).norm(dim=2) / want.norm(dim=2)
    worst = int(err.argmax())
    assert err.max().item() <= tol, "row and head %d: %g of the norm, %g allowed" % (worst, err.max().item(), tol)


def _one_key(rng, n, at, spread, sigma):
    """(codes, q): a key `at` that is 0 to 40 octaves above the others by (row, head), the others `spread`
    octaves apart."""
    H = 16
    codes = _values(rng, n)
    codes[:, 1] = ref.encode(np.clip(rng.standard_normal(n), -3.5, 3.5) * 64)
    codes[at, 0], codes[at, 1] = ref.encode(np.array([256.0, 0.0]))
    d = np.linspace(0.0, 40.0, SHARES * H).reshape(SHARES, H)
    octave = 1.0 / (SCALE * LOG2E * sigma)
    q = np.zeros((SHARES, H, D))
    q[..., 0] = d * octave / 256.0
    q[..., 1] = spread * octave / 64.0
    return codes, q


@pytest.mark.parametrize("n", [640, 8192, 32768])
@pytest.mark.parametrize("spread", [0.0, 0.3, 1.6])
@pytest.mark.parametrize("selection", [False, True])
def test_one_key_far_above_a_long_tail(n, spread, selection):
    rng = np.random.default_rng(n + int(10 * spread))
    sigma = 2.0 ** -6
    for at in (0, n // 2 + 3, n - 1):
        codes, q = _one_key(rng, n, at, spread, sigma)
        out, want, rel = _run(codes, np.full(n // P, sigma), q, selection=selection)
        _check(out, want, TAIL + BF16 + 2.2 * rel)


def test_one_key_with_a_sink_and_padded_heads():
    rng = np.random.default_rng(7)
    n, H = 8192, 5
    codes, q = _one_key(rng, n, 1, 0.5, 2.0 ** -6)
    out, want, rel = _run(codes, np.full(n // P, 2.0 ** -6), q[:, 3:3 + H], sink=np.linspace(-6.0, 12.0, H))
    _check(out, want, TAIL + BF16 + 2.2 * rel)


@pytest.mark.parametrize("drop", [3.0, 9.5, 16.3, 23.0, 70.0])
@pytest.mark.parametrize("pattern", ["alternate", "stairs", "one high in each"])
def test_tiles_that_go_up_and_down(drop, pattern):
    """Tiles of 128 keys whose levels are `drop` octaves apart: every other one, or falling and rising again, or one
    key of each tile above the rest of it."""
    rng = np.random.default_rng(11)
    n, H, sigma = 8192, 8, 2.0 ** -5
    codes = _values(rng, n)
    tile = np.arange(n) // 128
    if pattern == "alternate":
        level = tile % 2
    elif pattern == "stairs":
        level = np.abs(tile - 31) / 32.0
    else:
        level = 1.0 - (np.arange(n) % 128 == 77)
    codes[:, 0] = ref.encode(-256.0 * level)
    codes[:, 1] = ref.encode(rng.standard_normal(n) * 16)
    octave = 1.0 / (SCALE * LOG2E * sigma)
    q = np.zeros((SHARES, H, D))
    q[..., 0] = (drop + np.linspace(0.0, 1.0, SHARES * H).reshape(SHARES, H)) * octave / 256.0
    q[..., 1] = octave / 64.0
    out, want, rel = _run(codes, np.full(n // P, sigma), q)
    _check(out, want, BIG + SMALL + BF16 + 2.2 * rel)


@pytest.mark.parametrize("S", [1, 16, 64])
def test_block_scales_far_apart_beside_a_flat_tail(S):
    """One block in 40 has a scale 2^8 above the others (a token with an outlier); the scores are flat, but for one
    key far above."""
    rng = np.random.default_rng(13 + S)
    n, H = 8192, 16
    codes = _values(rng, n)
    scales = np.full(n // S, 2.0 ** -9)
    scales[rng.permutation(n // S)[:max(2, n // S // 40)]] = 2.0 ** -1
    # the outlier's column (3) is the one whose code is large in those blocks
    wide = np.repeat(scales, S) > 2.0 ** -5
    codes[wide] = ref.encode(ref.decode(codes[wide]) / 2.0 ** 7)
    codes[wide, 3] = ref.encode(np.array([300.0]))[0]
    codes[5, 0] = ref.encode(np.array([256.0]))[0]
    q = np.zeros((SHARES, H, D))
    q[..., 0] = np.linspace(0.0, 30.0, SHARES * H).reshape(SHARES, H) / (SCALE * LOG2E * np.repeat(scales, S)[5] * 256.0)
    out, want, rel = _run(codes, scales, q)
    # (the other columns hold every key alike: the outlier's would hide what the small scales lose)
    _check(out[..., 4:], want[..., 4:], BIG + SMALL + BF16 + 2.2 * rel)


@pytest.mark.parametrize("low,high", [(-64, 26), (29, 119)])
@pytest.mark.parametrize("sink", [False, True])
def test_scales_at_their_limits(low, high, sink):
    """Blocks of the least and the greatest scales, 2^90 apart: q has nothing in their columns, so that all keys count
    alike in the denominator, whatever their scale."""
    rng = np.random.default_rng(19)
    n, H = 1024, 8
    codes = _values(rng, n)
    scales = np.where(rng.random(n // 16) < 0.5, 2.0 ** low, 2.0 ** high)
    q = np.zeros((SHARES, H, D))
    q[..., 1] = rng.standard_normal((SHARES, H))
    out, want, rel = _run(codes, scales, q, sink=np.linspace(0.0, 8.0, H) if sink else None)
    _check(out, want, BIG + SMALL + BF16 + 2.2 * rel)


@pytest.mark.parametrize("n,R", [(64, SHARES), (640, SHARES), (8192, SHARES), (32768, 3)])
def test_heads_far_below_their_sink(n, R):
    """Sinks of 0 to 98 above all scores: the outputs shrink with them, down to 1e-38, and no further off; whole rows
    and cut ones."""
    rng = np.random.default_rng(23)
    H, sigma = 64, 2.0 ** -8
    codes = _values(rng, n)
    codes[:, 1] = ref.encode(np.clip(rng.standard_normal(n), -3.5, 3.5) * 64)
    q = np.zeros((R, H, D))
    q[..., 1] = 0.3 / (SCALE * LOG2E * sigma * 64.0)
    out, want, rel = _run(codes, np.full(n // P, sigma), q, sink=np.linspace(0.0, 98.0, H))
    # bf16 and float32 have numbers of 1.2e-38 and above to their full precision: heads of smaller outputs are left out
    full = (want[..., 4:].amin(dim=(0, 2)) > 2.0 ** -125).nonzero()[:, 0]
    assert 40 < len(full) < H
    _check(out[:, full], want[:, full], TAIL + BF16 + 2.2 * rel)


def test_a_long_tail_in_every_head_of_a_cut_row():
    """Three rows of 32768 keys, so that some fifty shares cut each: the parts' references differ by the dominant key
    (which one part holds) and the merge weighs them."""
    rng = np.random.default_rng(17)
    n, H, sigma = 32768, 64, 2.0 ** -6
    codes = _values(rng, n)
    codes[:, 1] = ref.encode(np.clip(rng.standard_normal(n), -3.5, 3.5) * 64)
    codes[0, 0], codes[0, 1] = ref.encode(np.array([256.0, 0.0]))
    octave = 1.0 / (SCALE * LOG2E * sigma)
    q = np.zeros((3, H, D))
    q[..., 0] = np.linspace(0.0, 40.0, 3 * H).reshape(3, H) * octave / 256.0
    q[..., 1] = 0.5 * octave / 64.0
    out, want, rel = _run(codes, np.full(n // P, sigma), q)
    _check(out, want, TAIL + BF16 + 2.2 * rel)
    assert math.isfinite(rel)
