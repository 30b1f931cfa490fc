"""Every variant of the block8 row kernels, and of the products, by the rules that choose
them: rows on 32 bytes (d a multiple of 16), on 16 (of 8), on 8, and on single elements;
by slots and in order; short calls and those that settle their slots first.

Rows are compared bit for bit with the oracle. Products are of whole numbers whose sums are
exact in fp32, or are compared with one another bit for bit: no tolerance."""

import numpy as np
import pytest
import torch

from oracle import block8_oracle as B

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def em():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import mini_ema_means_b200

    return mini_ema_means_b200


def _rows(n, d, seed, kind):
    g = np.random.default_rng(seed)
    x = g.standard_normal((n, d)) * np.exp2(g.integers(-8, 9, (n, 1)).astype(float))
    x[g.random((n, d)) < 0.05] = 0
    x[n // 2, : min(d, 128)] = 0
    return torch.from_numpy(x).to(TYPES[kind])


def _f64(t):
    return t.detach().cpu().double().numpy()


def _check_rows(m, rows, x):
    codes, exps = B.quantise(_f64(x))
    got = m.codes.cpu().numpy()[rows]
    assert np.array_equal(got[:, :m.d], codes) and not got[:, m.d:].any()
    assert np.array_equal(B.exponents_of(m.scales.cpu().numpy(), rows, m.d), exps)


# wide (96, 768: also one and six blocks), 16 bytes, 8 bytes, single elements
WIDTHS = [96, 768, 136, 140, 141]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("n", [1, 200, 512, 513, 1500])
@pytest.mark.parametrize("order", ["rows", "columns"])
def test_rows_by_slot(em, n, d, kind, order):
    """Padding, repeated slots (the last stays) and slots outside the matrix, written from
    each type and read back to each, into rows that every vector store can reach and into
    rows that none can."""
    rows = 900
    g = np.random.default_rng(n + d)
    x = _rows(n, d, n + d, kind)
    slots = g.integers(0, rows, n)
    slots[g.random(n) < 0.1] = -1
    slots[n // 2:] = np.where(g.random(n - n // 2) < 0.5, slots[:n - n // 2], slots[n // 2:])
    outside = g.random(n) < 0.05
    slots[outside] = g.choice([rows, -2, 2 ** 40], int(outside.sum()))
    m = em.Block8(rows, d)
    m.codes.fill_(0x55)
    m.scales.fill_(0x60)
    m.claims.copy_(torch.from_numpy(g.integers(-5, n + 5, rows).astype(np.int32)))  # any content
    before, sbefore = m.codes.cpu(), m.scales.cpu().numpy()
    s = torch.from_numpy(slots).cuda()
    xin = x.cuda()
    m.write(xin.t().contiguous().t() if order == "columns" else xin, slots=s)
    if outside.any():
        with pytest.raises(em.EmeansError) as e:
            m.check()
        assert e.value.code == em.EM_E_BOUNDS
    m.check()
    last = {int(v): i for i, v in enumerate(slots) if 0 <= v < rows}
    if last:
        named = np.array(sorted(last))
        _check_rows(m, named, x[[last[v] for v in named]])
    rest = np.setdiff1d(np.arange(rows), np.array(list(last), dtype=int))
    assert torch.equal(m.codes.cpu()[rest], before[rest])
    at = B.scale_at(rest[:, None], np.arange(B.blocks(d))[None, :], d)
    assert np.array_equal(m.scales.cpu().numpy()[at], sbefore[at])
    held = B.held(_f64(x))
    want = np.stack([held[last[int(v)]] if int(v) in last else np.zeros(d) for v in slots])
    for dt in TYPES.values():
        ref = torch.from_numpy(want).to(dt)
        for pad in (0, 1, 4):
            wide = torch.full((n + 1, d + pad), 9.0, dtype=dt, device="cuda")
            m.read(wide[:n, :d], slots=s)
            assert torch.equal(wide[:n, :d].cpu(), ref), (dt, pad)
            assert (wide[n] == 9).all() and (wide[:, d:] == 9).all()
    if outside.any():
        with pytest.raises(em.EmeansError):
            m.check()


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("n", [1, 33, 700])
def test_rows_in_order(em, n, d, kind):
    x = _rows(n, d, n + d, kind)
    m = em.Block8(n + 3, d)
    m.codes.fill_(0x55)
    m.write(x.cuda(), first=2)
    m.check()
    _check_rows(m, np.arange(2, n + 2), x)
    assert (m.codes[:2] == 0x55).all() and (m.codes[n + 2:] == 0x55).all()
    held = B.held(_f64(x))
    for dt in TYPES.values():
        out = torch.full((n + 1, d), 9.0, dtype=dt, device="cuda")
        m.read(out[:n], first=2)
        assert torch.equal(out[:n].cpu(), torch.from_numpy(held).to(dt)), dt
        assert (out[n] == 9).all()


# ---------------------------------------------------------------- products without a tolerance

# a result's few rows, few columns, one tile, several, and pairs of CTAs
RESULTS = [(1, 64), (16, 500), (300, 20), (150, 140), (2000, 1700)]


def _product(em, x, y, dtype=torch.float32):
    A, Bm = em.Block8(*x.shape), em.Block8(*y.shape)
    A.write(x.cuda())
    Bm.write(y.cuda())
    out = torch.empty(len(x), len(y), dtype=dtype, device="cuda")
    A.matmul(Bm, out)
    A.check()
    return out


@pytest.mark.parametrize("d", [640, 768, 2049, 5000, 8192, 9000])
@pytest.mark.parametrize("na,nb", RESULTS)
def test_whole_numbers_are_multiplied_exactly(em, na, nb, d):
    """Numbers of -4 .. 4 are held exactly, and all partial sums are below 2^24: every
    value of a row counts once."""
    g = np.random.default_rng(d + na)
    x, y = (g.integers(-4, 5, s).astype(np.float32) for s in ((na, d), (nb, d)))
    assert 16 * d < 2 ** 24
    out = _product(em, torch.from_numpy(x), torch.from_numpy(y))
    want = x.astype(np.float64) @ y.astype(np.float64).T
    assert np.array_equal(_f64(out), want)


@pytest.mark.parametrize("d", [2048, 4096, 8192, 9216, 16384])
@pytest.mark.parametrize("na,nb", RESULTS)
def test_small_terms_behind_large_ones_are_kept(em, na, nb, d):
    """The first 1,024 products of a result are 2^14, which makes 2^24 (times a power of two
    for each row), and of each 32 after them one is 1 and the others are 0. Added up by 1,024
    they are whole multiples of fp32's last place there; added to 2^24 one MMA step at a
    time each would be lost."""
    x, y = np.zeros((na, d)), np.ones((nb, d))
    x[:, :1024] = y[:, :1024] = 128
    x[:, 1024::32] = 1
    x *= np.exp2(np.arange(na) % 5)[:, None]
    y *= np.exp2(-(np.arange(nb) % 3))[:, None]
    out = _product(em, torch.from_numpy(x).float(), torch.from_numpy(y).float())
    want = x @ y.T
    assert want[0, 0] == 2 ** 24 + (d - 1024) // 32
    assert np.array_equal(_f64(out), want)


@pytest.mark.parametrize("d", [300, 400, 640, 700, 768])
def test_pairs_that_keep_their_rows_make_the_same_sums(em, d):
    """Rows of 3 to 6 blocks, which the pair kernel keeps in shared memory for 16-bit results
    (of 6 blocks for 32-bit ones): the sums of the single-CTA kernels, rounded once."""
    g = np.random.default_rng(d)
    x, y = (torch.from_numpy(g.standard_normal((n, d))).float() for n in (2000, 1700))
    full = _product(em, x, y)
    assert torch.equal(_product(em, x[:128], y), full[:128]) and torch.equal(_product(em, x, y[:32]), full[:, :32])
    assert torch.equal(_product(em, x[300:301], y[:90]), full[300:301, :90])
    for dt in (torch.bfloat16, torch.float16):
        assert torch.equal(_product(em, x, y, dt), full.to(dt)), dt
