"""Block-scaled FP8 matrices on the GPU, through the public entry points, against the
fp64 oracle (oracle/block8_oracle.py).

Writing and reading are compared bit for bit. A product of held values is exact in
fp32 (4 + 4 significant bits), so only its d - 1 additions round: each by at most one
unit in the last place of a partial sum, 2^-23 of sum |a_t b_t|, and a result in a
16-bit type by half a step more (2^-8 bf16, 2^-11 fp16, relative; fp16 results below
2^-14 by at most 2^-25).
"""

import numpy as np
import pytest
import torch

from oracle import block8_oracle as B

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {"f32": 0.0, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(scope="module")
def em():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import mini_ema_means_b200

    return mini_ema_means_b200


def _rows(n, d, seed, kind="f32"):
    """Rows of mixed sizes: exact zeros, zero blocks, outliers, 60 binary orders."""
    g = np.random.default_rng(seed)
    x = g.standard_normal((n, d)) * np.exp2(g.integers(-3, 4, (1, d)).astype(float))
    scale = np.exp2(g.integers(-30, 31, (n, 1)).astype(float)) if kind != "f16" else np.exp2(g.integers(-8, 9, (n, 1)).astype(float))
    x = x * scale
    x[g.random((n, d)) < 0.05] = 0
    if n > 2:
        x[g.integers(0, n), :128] = 0
    return torch.from_numpy(x).to(TYPES[kind])


def _f64(t):
    return t.detach().cpu().double().numpy()


def _check_rows(m, rows, x):
    """Rows of the matrix hold what the oracle makes of x: codes, zero padding, exponents."""
    codes, exps = B.quantise(_f64(x))
    got = m.codes.cpu().numpy()[rows]
    nan = codes == 127
    assert np.array_equal(np.where(nan, got[:, :m.d] & 127, got[:, :m.d]), codes)
    assert not got[:, m.d:].any()
    assert np.array_equal(B.exponents_of(m.scales.cpu().numpy(), rows, m.d), exps)


# ---------------------------------------------------------------- write and read


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("order", ["rows", "columns"])
@pytest.mark.parametrize("n,d", [(1, 1), (1, 128), (2, 129), (3, 16), (65, 127), (64, 512), (130, 513), (7, 1500),
                                 (1, 30001), (300, 96)])
def test_write_and_read_are_the_oracles(em, n, d, order, kind):
    x = _rows(n, d, n * 1000 + d, kind).cuda()
    xin = x.t().contiguous().t() if order == "columns" else x
    m = em.Block8(n + 9, d)
    m.codes.fill_(0x55)
    before = m.codes.clone()
    m.write(xin, first=4)
    m.check()
    rows = np.arange(4, 4 + n)
    _check_rows(m, rows, x)
    assert torch.equal(m.codes[:4], before[:4]) and torch.equal(m.codes[4 + n:], before[4 + n:])
    want = B.held(_f64(x))
    for out_kind, dt in TYPES.items():
        wide = torch.full((n + 2, d + 5), 3.0, dtype=dt, device="cuda")
        m.read(wide[1:n + 1, :d], first=4)
        ref = torch.from_numpy(want).to(dt)  # exact but in fp16, where it rounds once
        assert torch.equal(wide[1:n + 1, :d].cpu(), ref), out_kind
        assert (wide[0] == 3).all() and (wide[n + 1] == 3).all() and (wide[:, d:] == 3).all()


def test_special_values(em):
    """Zeros of both signs, the block border 448 * 2^e and its neighbours, fp32's
    smallest and largest values, NaN and infinities among finite values."""
    inf, nan = float("inf"), float("nan")
    top = 448.0
    up, down = float(np.nextafter(np.float32(top), np.float32(inf))), float(np.nextafter(np.float32(top), np.float32(0)))
    rows = [
        [0.0, -0.0], [1e-45, -1e-45], [1.1754944e-38, -3e-39], [3.4028235e38, 1.0], [top, 1.0], [up, 1.0], [down, -1.0],
        [top * 2.0 ** -100, 2.0 ** -109], [nan, 1.0], [inf, 5.0], [-inf, nan], [nan, nan], [inf, 0.0], [240.0, -17.0],
        [2.0 ** -126, 2.0 ** -127], [448.0 * 2.0 ** -117, 2.0 ** -127], [1.5 * 2.0 ** -127, 2.0 ** -140],
    ]
    x = torch.zeros(len(rows), 150)
    x[:, 3], x[:, 140] = torch.tensor([r[0] for r in rows]), torch.tensor([r[1] for r in rows])
    x[:, 5] = torch.tensor([r[1] for r in rows])
    for order in (x.cuda(), x.cuda().t().contiguous().t()):
        m = em.Block8(len(rows), 150)
        m.write(order)
        _check_rows(m, np.arange(len(rows)), x)
        out = torch.empty(len(rows), 150, device="cuda")
        m.read(out)
        np.testing.assert_array_equal(_f64(out), B.held(_f64(x)))
        bad = ~torch.isfinite(x)
        assert torch.isnan(out.cpu()[bad]).all() and torch.isfinite(out.cpu()[~bad]).all()


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("d", [136, 141])
def test_non_finite_values_leave_their_neighbours_alone(em, kind, d):
    """NaN and infinities of both signs in every place of a row's two blocks, whole blocks
    of them, and rows without any in between."""
    x = _rows(2 * d + 3, d, 17, kind)
    inf, nan = float("inf"), float("nan")
    for i in range(d):
        x[2 * i, i] = (inf, -inf, nan)[i % 3]
    x[2 * d] = nan
    x[2 * d + 1, :128], x[2 * d + 1, 128:] = inf, 1.0
    x[2 * d + 2, 128:] = -inf
    for xin in (x.cuda(), x.cuda().t().contiguous().t()):
        m = em.Block8(len(x), d)
        m.write(xin)
        _check_rows(m, np.arange(len(x)), x)
        for out_kind, dt in TYPES.items():
            out = torch.empty(len(x), d, dtype=dt, device="cuda")
            m.read(out)
            ref = torch.from_numpy(B.held(_f64(x))).to(dt)
            assert torch.equal(torch.isnan(out.cpu()), ~torch.isfinite(x))
            assert torch.equal(out.cpu().nan_to_num(0.0), ref.nan_to_num(0.0)), out_kind


@pytest.mark.parametrize("kind", list(TYPES))
def test_strides_and_alignments(em, kind):
    """Pitched, offset, repeated and transposed inputs, and outputs off every vector width."""
    big = _rows(40, 300, 5, kind).cuda()
    views = [big[:, :200], big[:, 1:201], big[:, 3:203], big[::2, 2:202], big[3:4, :200].expand(11, 200),
             big[:, :37].t(), big[1:, 1:38].t(), big[:39, 3:40].t(), big[::3, :30].t()]
    for v in views:
        m = em.Block8(v.shape[0], v.shape[1])
        m.write(v)
        m.check()
        _check_rows(m, np.arange(v.shape[0]), v)
    m = em.Block8(40, 200)
    m.write(big[:, :200])
    want = torch.from_numpy(B.held(_f64(big[:, :200]))).to(TYPES[kind])
    for off in range(4):
        wide = torch.zeros(40, 210 + off, dtype=TYPES[kind], device="cuda")
        m.read(wide[:, off:off + 200])
        assert torch.equal(wide[:, off:off + 200].cpu(), want)
    with pytest.raises(em.EmeansError):
        m.write(_rows(40, 400, 6, kind).cuda()[:, ::2])


@pytest.mark.parametrize("n", [1, 33, 512, 513, 5000])
@pytest.mark.parametrize("order", ["rows", "columns"])
def test_slots(em, n, order):
    """Rows by slot: padding, the last of equal slots, unnamed rows as they were, slots
    outside the matrix refused by the kernel without touching memory; read back the same way."""
    d, rows = 140, 2000
    g = np.random.default_rng(n)
    x = _rows(n, d, n)
    for trial in range(2):  # the second trial meets the claims that the first left
        slots = g.integers(0, rows, n)
        slots[g.random(n) < 0.1] = -1
        slots[n // 2:] = np.where(g.random(n - n // 2) < 0.5, slots[:n - n // 2], slots[n // 2:])
        m = em.Block8(rows, d) if trial == 0 else m
        before, sbefore = m.codes.clone(), m.scales.clone()
        xin = x.cuda()
        m.write(xin.t().contiguous().t() if order == "columns" else xin, slots=torch.from_numpy(slots).cuda())
        m.check()
        last = {int(s): i for i, s in enumerate(slots) if s >= 0}
        if last:
            named = np.array(sorted(last))
            _check_rows(m, named, x[[last[s] for s in named]])
        rest = torch.from_numpy(np.setdiff1d(np.arange(rows), np.array(list(last), dtype=int)))
        assert torch.equal(m.codes.cpu()[rest], before.cpu()[rest])
        at = B.scale_at(rest.numpy()[:, None], np.arange(2)[None, :], d)
        assert np.array_equal(m.scales.cpu().numpy()[at], sbefore.cpu().numpy()[at])
        out = torch.full((n, d), 9.0, device="cuda")
        m.read(out, slots=torch.from_numpy(slots).cuda())
        held = B.held(_f64(x))
        want = np.stack([held[last[int(s)]] if s >= 0 else np.zeros(d) for s in slots])
        assert np.array_equal(_f64(out), want)
        x = -2 * x


@pytest.mark.parametrize("n", [40, 700])
def test_a_slot_outside_is_left_out_and_reported(em, n):
    d = 70
    m = em.Block8(100, d)
    x = _rows(n, d, 3).cuda()
    slots = torch.arange(n, device="cuda") % 90
    slots[5], slots[6], slots[7] = 100, -2, 2 ** 62
    guard = m.codes.clone()
    m.write(x, slots=slots)
    with pytest.raises(em.EmeansError) as e:
        m.check()
    assert e.value.code == em.EM_E_BOUNDS
    m.check()  # cleared
    assert torch.equal(m.codes[90:], guard[90:])
    out = torch.full((n, d), 9.0, device="cuda")
    m.read(out, slots=slots)
    with pytest.raises(em.EmeansError) as e:
        m.check()
    assert e.value.code == em.EM_E_BOUNDS
    assert (out[5:8] == 0).all()
    # an unread error does not stop a product
    m.read(out, slots=slots)
    s = torch.empty(100, 100, device="cuda")
    m.matmul(m, s)
    ref = torch.empty(100, d, device="cuda")
    m.read(ref)
    _assert_product(s, _f64(ref), _f64(ref), "f32")
    with pytest.raises(em.EmeansError):
        m.check()


# ---------------------------------------------------------------- products


def _assert_product(out, a, b, kind):
    ref, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = a.shape[1] * 2.0 ** -23 * mag
    tol += HALF_STEP[kind] * (np.abs(ref) + tol) + (2.0 ** -25 if kind == "f16" else 0.0)
    got = _f64(out)
    assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) / np.maximum(tol, 1e-300)))


def _plain(n, d, seed):
    """Rows whose products fit every result type."""
    g = np.random.default_rng(seed)
    return torch.from_numpy(g.standard_normal((n, d)) * np.exp2(g.integers(-4, 3, (n, 1)).astype(float))).float()


SHAPES = [(1, 1, 1), (1, 1, 4096), (1, 300, 768), (3, 129, 128), (16, 1000, 96), (33, 40, 33), (128, 129, 640),
          (129, 128, 130), (127, 1, 700), (200, 16, 513), (300, 257, 512), (513, 770, 200), (260, 300, 1100),
          (1000, 1, 64), (2, 5, 9000), (150, 140, 5000), (40, 300, 2049),
          (17, 500, 8192), (300, 20, 3000), (140, 129, 1025)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("na,nb,d", SHAPES)
def test_product(em, na, nb, d, kind):
    """Products of leading rows of larger matrices whose other rows hold NaN codes and
    NaN scales, into a strided result whose surroundings stay as they were."""
    x, y = _plain(na, d, na + d), _plain(nb, d, 7 * nb + d)
    A, Bm = em.Block8(na + 70, d), em.Block8(nb + 3, d)
    for m, v in ((A, x), (Bm, y)):
        m.codes.fill_(0x7F)
        m.scales.fill_(0xFF)
        m.write(v.cuda())
    for pad in (0, 3, 8):
        wide = torch.full((na + 2, nb + pad), 5.0, dtype=TYPES[kind], device="cuda")
        A.matmul(Bm, wide[1:na + 1, :nb])
        A.check()
        _assert_product(wide[1:na + 1, :nb], B.held(_f64(x)), B.held(_f64(y)), kind)
        assert (wide[0] == 5).all() and (wide[na + 1] == 5).all() and (wide[:, nb:] == 5).all()


# More than a wave of 128 x 128 tiles: pairs of CTAs. Rows of 3 to 6 blocks (A kept),
# more and fewer, ragged in both directions, one span and several.
LARGE = [(2500, 1500, 300), (1500, 3001, 700), (20000, 777, 96), (2100, 2000, 1300), (1300, 2050, 2100), (1921, 1729, 640),
         (3000, 1, 900), (4000, 32, 128), (3777, 24, 70), (2500, 33, 260)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("na,nb,d", LARGE)
def test_large_product(em, na, nb, d, kind):
    x, y = _plain(na, d, 1), _plain(nb, d, 2)
    A, Bm = em.Block8(na + 5, d), em.Block8(nb + 200, d)
    for m, v in ((A, x), (Bm, y)):
        m.codes.fill_(0x7F)
        m.scales.fill_(0xFF)
        m.write(v.cuda())
    a, b = B.held(_f64(x)), B.held(_f64(y))
    for pad in (0, 1, 8):
        wide = torch.full((na + 2, nb + pad), 5.0, dtype=TYPES[kind], device="cuda")
        A.matmul(Bm, wide[1:na + 1, :nb])
        A.check()
        _assert_product(wide[1:na + 1, :nb], a, b, kind)
        assert (wide[0] == 5).all() and (wide[na + 1] == 5).all() and (wide[:, nb:] == 5).all()


@pytest.mark.parametrize("d", [900, 1100, 5000, 8192])
def test_one_row_of_results_is_the_same_whoever_computes_it(em, d):
    """Few rows, some and many take different kernels, long rows with few tiles several
    CTAs to a tile; the sums of a result are the same in each, bit for bit."""
    x, y = _plain(2000, d, 1), _plain(1700, d, 2)
    A, Bm = em.Block8(2000, d), em.Block8(1700, d)
    A.write(x.cuda())
    Bm.write(y.cuda())
    all_rows = torch.empty(2000, 1700, device="cuda")
    A.matmul(Bm, all_rows)
    for n, k in ((1, 1700), (20, 300), (32, 1700), (33, 90), (128, 1700), (129, 130), (300, 257), (300, 1700), (200, 3)):
        out = torch.empty(n, k, device="cuda")
        A.matmul(Bm, out)
        assert torch.equal(out, all_rows[:n, :k]), (n, k)
    A.check()


def test_product_of_a_matrix_with_itself_and_repeats(em):
    x = _plain(300, 384, 1)
    m = em.Block8(300, 384)
    m.write(x.cuda())
    out = torch.empty(300, 300, device="cuda")
    m.matmul(m, out)
    h = B.held(_f64(x))
    _assert_product(out, h, h, "f32")
    assert torch.equal(out, out.t())  # the same sums in the same order
    again = torch.empty_like(out)
    m.matmul(m, again)
    assert torch.equal(out, again)


def test_a_nan_row_stays_alone(em):
    x, y = _plain(140, 300, 2), _plain(270, 300, 3)
    x[17, 250] = float("nan")
    y[200, 3] = float("inf")
    A, Bm = em.Block8(140, 300), em.Block8(270, 300)
    A.write(x.cuda())
    Bm.write(y.cuda())
    out = torch.empty(140, 270, device="cuda")
    A.matmul(Bm, out)
    hit = torch.zeros(140, 270, dtype=torch.bool)
    hit[17], hit[:, 200] = True, True
    assert torch.equal(torch.isnan(out.cpu()), hit)
    hx, hy = B.held(_f64(x)), B.held(_f64(y))
    keep = np.setdiff1d(np.arange(140), 17), np.setdiff1d(np.arange(270), 200)
    _assert_product(out.cpu()[keep[0]][:, keep[1]], hx[keep[0]], hy[keep[1]], "f32")


def test_scales_of_every_block_enter(em):
    """One non-zero block at a time, with scales 2^-40 .. 2^40: a byte taken from the
    wrong row, block or group would be off by a power of two."""
    d, n = 1300, 256
    g = np.random.default_rng(8)
    x = np.zeros((n, d))
    y = g.standard_normal((n, d))
    for i in range(n):
        b = i % B.blocks(d)
        x[i, b * 128:(b + 1) * 128] = g.standard_normal(x[i, b * 128:(b + 1) * 128].shape) * 2.0 ** g.integers(-40, 41)
    y *= np.exp2(g.integers(-20, 21, (n, B.blocks(d))).astype(float)).repeat(128, axis=1)[:, :d]
    x, y = torch.from_numpy(x).float(), torch.from_numpy(y).float()
    A, Bm = em.Block8(n, d), em.Block8(n, d)
    A.write(x.cuda())
    Bm.write(y.cuda())
    out = torch.empty(n, n, device="cuda")
    A.matmul(Bm, out)
    _assert_product(out, B.held(_f64(x)), B.held(_f64(y)), "f32")


def test_scales_at_the_ends_of_the_range(em):
    """Sums of 128 equal powers of two are exact: subnormal results, scales that cancel,
    and results beyond fp32."""
    m, out = em.Block8(2, 128), torch.empty(2, 2, device="cuda")
    for p, q in ((-70, -70), (-126, -10), (-64, -62), (100, -100), (119, -126), (60, 59), (100, 100)):
        m.write(torch.tensor([[2.0 ** p], [2.0 ** q]], device="cuda").expand(2, 128).contiguous())
        m.matmul(m, out)
        want = torch.tensor([[2.0 * p + 7, p + q + 7.0], [p + q + 7.0, 2.0 * q + 7]], dtype=torch.float64).exp2().float()
        assert torch.equal(out.cpu(), want), (p, q, out, want)


# ---------------------------------------------------------------- gradients


def _gradients(em, g, a, b):
    """dA and dB of out = A B^T as a training step makes them."""
    n, k = g.shape
    d = a.shape[1]
    G, Gt, Bt, At = em.Block8(n, k), em.Block8(k, n), em.Block8(d, k), em.Block8(d, n)
    G.write(g)
    Gt.write(g.t())
    Bt.write(b.t())
    At.write(a.t())
    da, db = torch.empty(n, d, device="cuda"), torch.empty(k, d, device="cuda")
    G.matmul(Bt, da)
    Gt.matmul(At, db)
    G.check()
    Gt.check()
    return da, db


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("n,k,d", [(5, 3, 7), (200, 130, 96), (333, 257, 200), (1, 400, 64), (1500, 2, 129)])
def test_gradients_follow_the_formula(em, n, k, d, kind):
    """Against the formula on the held values (the accumulation's bound) and on the given
    ones: a held value is off by at most 2^-4 of itself or half the smallest code,
    2^-10 * 2^e <= 2^-18 * (2 / 1.75) of its block's largest."""
    g, a, b = (t.to(TYPES[kind]).cuda() for t in (_plain(n, k, 1) / 16, _plain(n, d, 2), _plain(k, d, 3)))
    da, db = _gradients(em, g, a, b)
    hg, ha, hb = _f64(g), _f64(a), _f64(b)
    _assert_product(da, B.held(hg), B.held(hb.T), "f32")
    _assert_product(db, B.held(hg.T), B.held(ha.T), "f32")

    def off(x):  # bound of |held - given|, blocks along the rows
        v = np.abs(x)
        pad = np.pad(v, ((0, 0), (0, -v.shape[1] % 128)))
        top = pad.reshape(len(v), -1, 128).max(axis=2).repeat(128, axis=1)[:, :v.shape[1]]
        return np.maximum(2.0 ** -4 * v, 2.0 ** -17 * top)

    for got, p, q in ((da, hg, hb.T), (db, hg.T, ha.T)):
        ep, eq = off(p), off(q)
        tol = ep @ np.abs(q).T + np.abs(p) @ eq.T + ep @ eq.T + p.shape[1] * 2.0 ** -22 * (np.abs(p) @ np.abs(q).T)
        assert np.all(np.abs(_f64(got) - p @ q.T) <= tol)


def test_gradients_are_the_differences(em):
    """Small whole numbers are held exactly and their products summed without rounding,
    so the gradient of L = sum W * (A B^T) equals L's central differences exactly."""
    g = np.random.default_rng(4)
    n, k, d = 140, 70, 90
    w, a, b = (torch.from_numpy(g.integers(-4, 5, s)).float() for s in ((n, k), (n, d), (k, d)))
    da, db = _gradients(em, w.cuda(), a.cuda(), b.cuda())
    A, Bm, out = em.Block8(n, d), em.Block8(k, d), torch.empty(n, k, device="cuda")

    def loss(a, b):
        A.write(a.cuda())
        Bm.write(b.cuda())
        A.matmul(Bm, out)
        return float((out.cpu().double() * w.double()).sum())

    for _ in range(12):
        i, j, t = g.integers(0, n), g.integers(0, k), g.integers(0, d)
        for x, other, at, grad in ((a, b, (i, t), da), (b, a, (j, t), db)):
            hi, lo = x.clone(), x.clone()
            hi[at] += 1
            lo[at] -= 1
            up, down = (loss(hi, other), loss(lo, other)) if x is a else (loss(other, hi), loss(other, lo))
            assert (up - down) / 2 == float(grad[at])


# ---------------------------------------------------------------- streams, graphs, size


def test_a_captured_run_is_replayed_on_new_inputs(em):
    """Write by slots, read back and score, captured once; replays see new values, new
    slots (with repeats) and an eager call of the same matrices in between."""
    d, n, rows = 200, 600, 900
    store, queries = em.Block8(rows, d), em.Block8(20, d)
    x, q = torch.zeros(n, d, device="cuda"), torch.zeros(20, d, device="cuda")
    slots = torch.arange(n, device="cuda")
    back, scores = torch.empty(n, d, device="cuda"), torch.empty(20, rows, device="cuda")

    def step():
        store.write(x, slots=slots)
        store.read(back, slots=slots)
        queries.write(q)
        queries.matmul(store, scores)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = np.random.default_rng(0)
    for t in range(3):
        xs, qs = _plain(n, d, 10 + t), _plain(20, d, 20 + t)
        s = torch.from_numpy(g.integers(0, rows, n))
        if t == 1:  # an eager call with other slots between two replays
            store.write(_plain(n, d, 99).cuda(), slots=torch.from_numpy(g.permutation(rows)[:n].copy()).cuda())
        x.copy_(xs)
        q.copy_(qs)
        slots.copy_(s)
        graph.replay()
        store.check()
        queries.check()
        last = {int(v): i for i, v in enumerate(s)}
        held = B.held(_f64(xs))
        assert np.array_equal(_f64(back), np.stack([held[last[int(v)]] for v in s]))
        every = torch.empty(rows, d, device="cuda")
        store.read(every)
        _assert_product(scores, B.held(_f64(qs)), _f64(every), "f32")


def test_check_is_refused_while_the_stream_is_captured(em):
    m = em.Block8(10, 20)
    x = torch.ones(10, 20, device="cuda")
    m.write(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.write(x)
        with pytest.raises(em.EmeansError) as e:
            m.check()
        m.write(x)
    assert e.value.code == em.EM_E_STATE
    graph.replay()
    m.check()
    _check_rows(m, np.arange(10), x)


def test_two_streams_at_once(em):
    """Calls of different matrices run side by side on two streams, in rounds, with the
    results of each alone."""
    d = 384
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    work = []
    for s in range(2):
        x, y = _plain(700, d, s).cuda(), _plain(900, d, 5 + s).cuda()
        A, Bm = em.Block8(700, d), em.Block8(900, d)
        out, few = torch.empty(700, 900, device="cuda"), torch.empty(9, 900, device="cuda")
        work.append((x, y, A, Bm, out, few))
    torch.cuda.synchronize()
    for _ in range(10):
        for st, (x, y, A, Bm, out, few) in zip(sides, work):
            A.write(x, stream=st)
            Bm.write(y, stream=st)
            A.matmul(Bm, out, stream=st)
            A.matmul(Bm, few, stream=st)
    torch.cuda.synchronize()
    for x, y, A, Bm, out, few in work:
        A.check()
        hx, hy = B.held(_f64(x)), B.held(_f64(y))
        _assert_product(out, hx, hy, "f32")
        _assert_product(few, hx[:9], hy, "f32")


def test_offsets_past_32_bits(em):
    """A matrix of 4.7 GB: rows behind 2^32 bytes written, gathered and scored."""
    rows, d = 6_200_000, 760
    m = em.Block8(rows, d)
    assert m.codes.numel() > 2 ** 32
    x = _plain(300, d, 1)
    slots = torch.cat([torch.arange(rows - 200, rows), torch.arange(0, 100)])
    m.write(x.cuda(), slots=slots.cuda())
    out = torch.empty(300, d, device="cuda", dtype=torch.bfloat16)
    m.read(out, slots=slots.cuda())
    held = B.held(_f64(x))
    assert np.array_equal(_f64(out), held)
    m.read(out[:200], first=rows - 200)
    assert np.array_equal(_f64(out[:200]), held[:200])
    q = em.Block8(2, d)
    q.write(x[:2].cuda())
    s = torch.empty(2, rows, device="cuda")
    q.matmul(m, s)
    q.check()
    _assert_product(s[:, -200:], held[:2], held[:200], "f32")
    _assert_product(s[:, :100], held[:2], held[200:], "f32")
    assert (s[:, 100:-200] == 0).all()
    wide = torch.empty(rows, 3, device="cuda", dtype=torch.float16)  # the other orientation
    m.matmul(em.Block8(3, d), wide)
    m.check()
    assert (wide == 0).all()


def test_a_wait_that_runs_out_is_reported(em):
    """The bounded wait of the products: gives up within its limit, leaves the context
    usable, and one warp's giving up ends the other's wait."""
    import time

    m = em.Model(8, 4, seed=1)
    t0 = time.monotonic()
    assert m.selftest(3, wait_ms=200.0) == em.EM_E_TIMEOUT
    assert time.monotonic() - t0 < 5.0  # the second warp alone would wait 12.8 s
    m.close()
    a = em.Block8(200, 64)
    out = torch.ones(200, 200, device="cuda")
    a.matmul(a, out)
    a.check()
    assert (out == 0).all()


# ---------------------------------------------------------------- with the model


def test_a_model_takes_a_block8_matrix(em):
    """Training, assignment, MSE and Lloyd on a block8 matrix are those on the bf16 rows
    it reads back, bit for bit; its checks and refusals; a raw pointer afterwards."""
    d, k, n = 90, 24, 3000
    x = _plain(n + 50, d, 3)
    m8 = em.Block8(n + 50, d)
    m8.write(x.cuda())
    rows = torch.empty(n + 50, d, dtype=torch.bfloat16, device="cuda")
    m8.read(rows)
    torch.cuda.synchronize()
    got = []
    for X in (m8, rows):
        m = em.Model(d, k, seed=5, check_finite=1)
        m.train(X, n=n, epochs=2.0)
        c, lab, dist = torch.empty(k, d), torch.empty(n, dtype=torch.int64), torch.empty(n)
        m.centroids(c)
        m.assign(X, labels=lab, dists=dist, n=n)
        mse = m.mse(X, n=n)
        m.lloyd(X, 3, n=n)
        c2 = torch.empty(k, d)
        m.centroids(c2)
        got.append((c, lab, dist, torch.tensor(mse), c2))
        if X is m8:  # a raw pointer is again what the model's dtype says
            f = x.cuda()
            m.set_option("input_dtype", 0)
            m.mse(m8)
            torch.cuda.synchronize()
            assert m.mse(f.data_ptr(), n=n) == m.mse(f, n=n)
        m.close()
    assert all(torch.equal(a, b) for a, b in zip(*got))
    m = em.Model(d, k, seed=5, check_finite=1)
    with pytest.raises(em.EmeansError) as e:
        m.train(m8, n=n + 51)
    assert e.value.code == em.EM_E_INVAL
    with pytest.raises(em.EmeansError):
        m.train(em.Block8(n, d + 1))
    x[7, 3] = float("nan")
    m8.write(x.cuda())
    torch.cuda.synchronize()
    with pytest.raises(em.EmeansError) as e:
        m.train(m8)
    assert e.value.code == em.EM_E_NONFINITE
    m.close()


def test_a_model_waits_for_the_writes_of_the_current_stream(em):
    """A matrix written on the current stream, behind a long queue, and handed to a model
    at once; then what set_option says of raw pointers."""
    n, d, k = 200_000, 256, 8
    x = _plain(n, d, 7).cuda()
    m8, ref = em.Block8(n, d), em.Block8(n, d)
    ref.write(x)
    m = em.Model(d, k, seed=2)
    m.train(ref, epochs=0.05)
    want = m.mse(ref)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(200):
            m8.write(x * -1.0)
        m8.write(x)
        assert m.mse(m8) == want
    m.set_option("input_dtype", "block8")
    assert m.mse(int(__import__("ctypes").addressof(m8.view)), n=n) == want
    with pytest.raises(em.EmeansError):
        m.set_option("input_dtype", 2)
    m.close()


def test_memory_dropped_after_a_call_on_another_stream(em):
    """Inputs freed by the caller while a call on a given stream is still queued are not
    handed out again before it is done."""
    st = torch.cuda.Stream()
    m = em.Block8(4096, 512)
    x = _plain(4096, 512, 3)
    xg = x.cuda()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        torch.cuda._sleep(50_000_000)
    m.write(xg, stream=st)
    del xg
    for _ in range(4):
        torch.full((4096, 512), 9.0, device="cuda")
    st.synchronize()
    _check_rows(m, np.arange(0, 4096, 97), x[::97])


def test_the_operators_together(em):
    """As a service uses them: a store filled in pieces, centroids trained on it, and
    queries scored against the nearest cluster's stored rows, gathered by number."""
    d, n, k = 96, 4000, 16
    g = np.random.default_rng(2)
    centers = g.standard_normal((k, d)) * 3
    x = torch.from_numpy(centers[g.integers(0, k, n)] + g.standard_normal((n, d))).float()
    store = em.Block8(n, d)
    for i in range(0, n, 700):
        store.write(x[i:i + 700].cuda(), first=i)
    torch.cuda.synchronize()
    m = em.Model(d, k, seed=1)
    m.train(store, epochs=3.0)
    lab = torch.empty(n, dtype=torch.int64, device="cuda")
    m.assign(store, labels=lab)
    q = x[:1] + 0.01
    qlab = torch.empty(1, dtype=torch.int64, device="cuda")
    m.assign(q.cuda(), labels=qlab)
    members = torch.nonzero(lab == qlab).flatten()
    rows = torch.empty(len(members), d, dtype=torch.bfloat16, device="cuda")
    store.read(rows, slots=members)
    part = em.Block8(len(members), d)
    part.write(rows)  # held values are held again as they are
    back = torch.empty_like(rows)
    part.read(back)
    assert torch.equal(back, rows)
    Q, s = em.Block8(1, d), torch.empty(1, len(members), device="cuda")
    Q.write(q.cuda())
    Q.matmul(part, s)
    Q.check()
    _assert_product(s, B.held(_f64(q)), _f64(rows), "f32")
    m.close()
