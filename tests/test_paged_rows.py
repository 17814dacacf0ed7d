"""GPU: rows of the norm and of the append whose squares underflow in float32, the append's default for eps, and
offsets with a bad entry among good sequences."""

import numpy as np
import pytest

import paged_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    import torch
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)


def _dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# magnitudes whose squares are normal, subnormal or zero in float32, subnormal elements, the least one
MAGNITUDES = [1.0, 1e-12, 1e-15, 1e-18, 1e-19, 1e-20, 1e-22, 1e-24, 1e-30, 1e-37, 1e-39, 1e-42, 2.0 ** -149]


def _tiny(rng, f32):
    """(tensor, its values in 64 bits): a row of each magnitude, one row of a single element, one of mixed ones."""
    import torch
    x = rng.standard_normal((len(MAGNITUDES) + 2, 512))
    x[:len(MAGNITUDES)] *= np.array(MAGNITUDES)[:, None]
    x[-2] = 0.0
    x[-2, 300] = -1e-30
    x[-1] *= 10.0 ** rng.uniform(-44, -20, 512)
    x[:, 17] = np.where(np.abs(x[:, 17]) < 2.0 ** -133, 2.0 ** -130, x[:, 17])      # (no row of zeros alone)
    t = torch.from_numpy(x.astype(np.float32)).cuda()
    if not f32:
        t = t.to(torch.bfloat16)
    return t, t.double().cpu().numpy()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("eps", [0.0, 1e-42, 1e-36, 1e-31, 1e-6])
@pytest.mark.parametrize("rope,style", [(0, 0), (64, 1)])
def test_norm_of_rows_whose_squares_underflow(f32, eps, rope, style):
    import torch
    from deepseek_v4_top_gb300 import dsa
    rng = np.random.default_rng(21)
    x, x64 = _tiny(rng, f32)
    w = (1 + rng.standard_normal(512) * 0.3).astype(np.float32)
    R = x.shape[0]
    pos = np.arange(R, dtype=np.int32)
    table = ref.table64(R, rope) if rope else None
    out = torch.empty((R, 1, 512), dtype=x.dtype, device="cuda")
    dsa.dsa_qk_norm_rope(x.view(R, 1, 512), _dev(pos), out, q_weight=_dev(w), eps=eps, rope=_dev(table) if rope else None,
                         rope_style=style)
    assert dsa.dsa_get_device_error() == 0
    y, room = ref.rows(x64, w, float(np.float32(eps)), table[pos] if rope else None, rope, style)
    # (results below float32's least normal number are off by half a step of it a rounding: 4 of them)
    bound = room * ref.ROW_EPS + 4 * 2.0 ** -150
    if not f32:
        bound = bound * (1 + 2.0 ** -8) + np.abs(y) * 2.0 ** -8 + 2.0 ** -134
    err = np.abs(out[:, 0].double().cpu().numpy() - y)
    assert (err <= bound).all(), float(np.nanmax(err / bound))


@pytest.mark.parametrize("S", [1, 16, 64])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("eps", [0.0, 1e-42, 1e-36])
def test_append_of_rows_whose_squares_underflow(S, f32, eps):
    """The codes and scales of the 64-bit rows, as for any other row."""
    from deepseek_v4_top_gb300 import dsa
    rng = np.random.default_rng(23 + S)
    x, x64 = _tiny(rng, f32)
    w = (1 + rng.standard_normal(512) * 0.3).astype(np.float32)
    R, P = x.shape[0], 64
    table = ref.table64(64, 64)
    offsets, starts, pages = np.array([0, R], np.int32), np.array([3], np.int32), np.array([[1]], np.int32)
    codes0, scales0 = np.zeros((2, P, 512), np.uint8), np.full((2, P // S), 2.0 ** -7, np.float32)
    cache, scale = _dev(codes0), _dev(scales0)
    dsa.dsa_paged_append(x, _dev(offsets), _dev(starts), _dev(pages), cache, scale, norm_weight=_dev(w), eps=eps,
                         rope=_dev(table))
    assert dsa.dsa_get_device_error() == 0
    want, wscale, _ = ref.append(x64, offsets, starts, pages, codes0, scales0, w, float(np.float32(eps)), table, 64, 0)
    assert np.array_equal(scale.cpu().numpy().astype(np.float64), wscale)
    assert np.array_equal(cache.cpu().numpy(), want)


def test_append_takes_the_norm_with_its_weight():
    """norm_weight without eps norms as dsa_qk_norm_rope does by default; neither leaves the rows as they are."""
    import torch
    from deepseek_v4_top_gb300 import dsa
    g = torch.Generator(device="cuda").manual_seed(3)
    kv = torch.randn((5, 512), generator=g, device="cuda") * 3
    w = 1 + 0.2 * torch.randn(512, generator=g, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def stored(**kw):
        cache, scale = torch.zeros((1, 16, 512), dtype=torch.uint8, device="cuda"), torch.ones((1, 16), device="cuda")
        dsa.dsa_paged_append(kv, i32(0, 5), i32(0), i32(0).view(1, 1), cache, scale, **kw)
        return torch.cat((cache.view(-1).float(), scale.view(-1)))

    assert torch.equal(stored(norm_weight=w), stored(norm_weight=w, eps=1e-6))
    assert not torch.equal(stored(norm_weight=w), stored())
    assert torch.equal(stored(), stored(eps=-1.0)) and torch.equal(stored(eps=-1.0), stored(norm_weight=w, eps=-1.0))
    assert torch.equal(stored(eps=1e-6), stored(norm_weight=torch.ones_like(w)))
    assert dsa.dsa_get_device_error() == 0


@pytest.mark.parametrize("offsets,bad,good", [
    ([0, 1000, 8, 24], [1], [0, 1000, 1008, 1024]), ([0, 40, 5000, 60], [1, 2], [0, 40, 50, 60]),
    ([0, -7, 90, 200], [0, 1], [0, 50, 90, 200])])
def test_append_with_a_bad_offset_among_good_sequences(offsets, bad, good):
    """Tokens of the good sequences may be missing, whole scale blocks of them; what is stored is right, nothing else
    is touched, and the call with the right offsets then stores everything."""
    from deepseek_v4_top_gb300 import dsa
    rng = np.random.default_rng(29)
    P, S, R, most = 32, 16, 1024, 40
    B = len(offsets) - 1
    kv = rng.standard_normal((R, 512)).astype(np.float32)
    starts = np.array([3, 5, 0], np.int32)
    pages = rng.permutation(B * most).reshape(B, most).astype(np.int32)
    codes0 = ref.encode(rng.standard_normal((B * most, P, 512)) * 50)
    scales0 = np.full((B * most, P // S), 2.0 ** -7, np.float32)
    cache, scale = _dev(codes0), _dev(scales0)

    def call(offs):
        dsa.dsa_paged_append(_dev(kv), _dev(np.array(offs, np.int32)), _dev(starts), _dev(pages), cache, scale)
        return dsa.dsa_get_device_error(), cache.cpu().numpy(), scale.cpu().numpy().astype(np.float64)

    code, codes, scales = call(offsets)
    assert code == dsa.DSA_DEVERR_SEQ_RANGE
    left = codes0.copy(), scales0.astype(np.float64)
    for b in range(B):
        if b in bad:
            assert np.array_equal(codes[pages[b]], left[0][pages[b]]) and np.array_equal(scales[pages[b]], left[1][pages[b]])
            continue
        n = offsets[b + 1] - offsets[b]
        one = ref.append(kv.astype(np.float64)[offsets[b]:offsets[b + 1]], [0, n], starts[b:b + 1], pages[b:b + 1], codes0, scales0,
                         None, -1.0, None, 0, 0)
        for at in range(0, P * most, S):
            page, place = pages[b, at // P], at % P
            got = codes[page, place:place + S], scales[page, place // S]
            new = one[0][page, place:place + S], one[1][page, place // S]
            old = left[0][page, place:place + S], left[1][page, place // S]
            assert any(np.array_equal(got[0], w[0]) and got[1] == w[1] for w in (new, old)), (b, at)
    code, codes, scales = call(good)
    assert code == 0
    want, wscale, _ = ref.append(kv.astype(np.float64), good, starts, pages, codes0, scales0, None, -1.0, None, 0, 0)
    assert np.array_equal(codes, want) and np.array_equal(scales, wscale)
