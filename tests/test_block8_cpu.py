"""Block-scaled FP8 matrices without a GPU: the oracle's own definition, the layout
that the library reports, and every refusal that comes before device work."""

import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import block8_oracle as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def em():
    import importlib.util

    spec = importlib.util.spec_from_file_location("_b", os.path.join(ROOT, "mini_ema_means_b200", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    b.build()
    import mini_ema_means_b200

    return mini_ema_means_b200


# ---------------------------------------------------------------- the definition


def test_oracle_rounds_to_the_nearest_code_with_ties_to_even():
    """The vectorised rounding against a search of the grid, on every midpoint, its
    neighbours and random values; and against torch's E4M3 conversion."""
    grid = B._GRID
    mid = (grid[:-1] + grid[1:]) / 2
    v = np.concatenate([mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9), grid,
                        np.random.default_rng(0).uniform(0, 448, 2000)])
    v = np.concatenate([v, -v, [448.0]])
    for x in (v[i:i + 127] for i in range(0, len(v), 127)):
        row = np.concatenate([x, [448.0]])[None, :]  # 448 fixes the exponent at 0
        codes, exps = B.quantise(row)
        assert exps[0, 0] == 0
        assert np.array_equal(codes[0], [B.nearest_code(t) for t in row[0]])
    f = v.astype(np.float32)
    want = torch.from_numpy(f).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(want, [B.nearest_code(t) for t in f.astype(np.float64)])


@pytest.mark.parametrize("k", [-100, -3, 0, 5, 110])
def test_oracle_exponent_at_its_border(k):
    top = 448.0 * 2.0 ** k
    assert B.exponent(top) == k and B.exponent(float(np.nextafter(top, np.inf))) == k + 1
    assert B.exponent(top / 2) == k - 1 and B.exponent(0.0) == 0 and B.exponent(1e-45) == B.MIN_EXP
    assert B.exponent(3.4028235e38) == B.MAX_EXP and B.held([[3.4028235e38]])[0, 0] == 448.0 * 2.0 ** 119


def test_held_values_are_exact_in_bf16():
    """Every code at the smallest and largest exponents is a normal bf16 number."""
    for e in (B.MIN_EXP, -50, 0, 50, 119):
        v = B._GRID * 2.0 ** e
        assert np.array_equal(torch.from_numpy(v).to(torch.bfloat16).double().numpy(), v)
    assert B._GRID[1] * 2.0 ** B.MIN_EXP == 2.0 ** -126


# ---------------------------------------------------------------- layout


@pytest.mark.parametrize("rows,d", [(1, 1), (128, 128), (129, 129), (1000, 512), (1000, 513), (70000, 768), (5, 30001)])
def test_layout(em, rows, d):
    pitch, code_bytes, scale_bytes = em.block8_layout(rows, d)
    assert pitch == -(-d // 16) * 16 and code_bytes == rows * pitch
    assert scale_bytes == -(-rows // 128) * -(-B.blocks(d) // 4) * 512
    r = np.unique(np.concatenate([np.arange(min(rows, 300)), [rows - 1]]))
    at = B.scale_at(r[:, None], np.arange(B.blocks(d))[None, :], d)
    assert len(np.unique(at)) == at.size and at.min() >= 0 and at.max() < scale_bytes


@pytest.mark.parametrize("rows,d", [(0, 8), (-1, 8), (1 << 31, 8), (8, 0), (8, (1 << 24) + 1)])
def test_layout_refuses_sizes(em, rows, d):
    with pytest.raises(em.EmeansError) as e:
        em.block8_layout(rows, d)
    assert e.value.code == em.EM_E_INVAL


# ---------------------------------------------------------------- refusals of the C entry points


def _view(em, rows=200, d=130, **over):
    f = dict(codes=1 << 20, scales=1 << 21, claims=1 << 22, status=1 << 23, rows=rows, d=d)
    f.update(over)
    return em.em_block8_t(**f)


X = 1 << 24  # an address that is never read: each call below is refused first


def _write(em, v=None, X=X, dtype=0, n=10, rs=130, cs=1, first=0, slots=None):
    return em.em_block8_write(ctypes.byref(v or _view(em)), X, dtype, n, rs, cs, first, slots, None)


def _read(em, v=None, out=X, dtype=0, n=10, rs=130, first=0, slots=None):
    return em.em_block8_read(ctypes.byref(v or _view(em)), first, slots, n, out, dtype, rs, None)


def _matmul(em, a=None, b=None, na=10, nb=20, out=X, dtype=0, rs=20):
    return em.em_block8_matmul(ctypes.byref(a or _view(em)), na, ctypes.byref(b or _view(em)), nb, out, dtype, rs, None)


def _cases(em):
    v = lambda **o: _view(em, **o)  # noqa: E731
    return [
        (_write, dict(v=v(codes=None))), (_write, dict(v=v(scales=None))), (_write, dict(v=v(status=None))),
        (_write, dict(v=v(codes=(1 << 20) + 8))), (_write, dict(v=v(scales=(1 << 21) + 4))),
        (_write, dict(v=v(status=(1 << 23) + 2))), (_write, dict(v=v(rows=0))), (_write, dict(v=v(d=0))),
        (_write, dict(dtype=3)), (_write, dict(dtype=-1)), (_write, dict(X=X + 2)), (_write, dict(X=X + 1, dtype=1)),
        (_write, dict(X=None)), (_write, dict(n=-1)), (_write, dict(n=1 << 31)), (_write, dict(first=-1)),
        (_write, dict(v=v(rows=1 << 20, d=1 << 24), n=1 << 14)), (_read, dict(v=v(rows=1 << 20, d=1 << 24), n=1 << 14, rs=1 << 24)),
        (_write, dict(first=191)), (_write, dict(n=201)), (_write, dict(rs=130, cs=2)), (_write, dict(rs=-1, cs=1)),
        (_write, dict(first=1, slots=1 << 25)), (_write, dict(slots=(1 << 25) + 4)),
        (_write, dict(v=v(claims=None), n=600, slots=1 << 25)),
        (_read, dict(rs=129)), (_read, dict(out=None)), (_read, dict(first=195)), (_read, dict(n=-5)),
        (_read, dict(dtype=7)), (_read, dict(first=2, slots=1 << 25)), (_read, dict(out=X + 2)),
        (_matmul, dict(b=v(d=131))), (_matmul, dict(na=201)), (_matmul, dict(nb=201, rs=300)), (_matmul, dict(na=-1)),
        (_matmul, dict(rs=19)), (_matmul, dict(out=None)), (_matmul, dict(dtype=3)), (_matmul, dict(out=X + 1, dtype=2)),
        (_matmul, dict(b=v(scales=None))),
    ]


def test_c_entry_points_refuse_bad_arguments(em):
    for call, over in _cases(em):
        rc = call(em, **over)
        assert rc == em.EM_E_INVAL, (call.__name__, over, rc)
        assert em.em_last_error(), over
    for call, args in ((em.em_block8_write, (None, X, 0, 1, 1, 1, 0, None, None)),
                       (em.em_block8_read, (None, 0, None, 1, X, 0, 1, None)),
                       (em.em_block8_matmul, (None, 1, None, 1, X, 0, 1, None)), (em.em_block8_check, (None, None))):
        assert call(*args) == em.EM_E_INVAL


def test_empty_calls_do_nothing(em):
    assert _write(em, n=0) == em.EM_OK and _write(em, n=0, X=None) == em.EM_OK
    assert _read(em, n=0, out=None) == em.EM_OK
    assert _matmul(em, na=0) == em.EM_OK and _matmul(em, nb=0) == em.EM_OK


def test_host_memory_is_refused(em):
    m = em.Block8(4, 8, device="cpu")
    want = em.EM_E_INVAL if em.em_device_count() else em.EM_E_NODEVICE
    for call in (lambda: m.write(torch.zeros(2, 8), stream=0), lambda: m.read(torch.zeros(2, 8), stream=0),
                 lambda: m.matmul(m, torch.zeros(4, 4), stream=0), lambda: m.check(stream=0)):
        with pytest.raises(em.EmeansError) as e:
            call()
        assert e.value.code == want


# ---------------------------------------------------------------- refusals of the binding


def test_binding_refuses_bad_tensors(em):
    m = em.Block8(16, 40, device="cpu")
    f = torch.float32
    idx = torch.arange(3)
    bad = [
        (TypeError, lambda: m.write(torch.zeros(3, 40, dtype=torch.float64), stream=0)),
        (TypeError, lambda: m.write(torch.zeros(3, 40, dtype=torch.int32), stream=0)),
        (ValueError, lambda: m.write(torch.zeros(3, 41), stream=0)),
        (ValueError, lambda: m.write(torch.zeros(40), stream=0)),
        (ValueError, lambda: m.write(torch.zeros(3, 40, device="meta"), stream=0)),
        (ValueError, lambda: m.write(torch.zeros(3, 40), slots=idx[:2], stream=0)),
        (ValueError, lambda: m.write(torch.zeros(3, 40), slots=idx.int(), stream=0)),
        (ValueError, lambda: m.write(torch.zeros(3, 40), slots=torch.arange(6)[::2], stream=0)),
        (ValueError, lambda: m.write(torch.zeros(3, 40), slots=idx, first=1, stream=0)),
        (em.EmeansError, lambda: m.write(torch.zeros(3, 80)[:, ::2], stream=0)),
        (em.EmeansError, lambda: m.write(torch.zeros(3, 40), first=14, stream=0)),
        (ValueError, lambda: m.read(torch.zeros(40, 3).t(), stream=0)),
        (TypeError, lambda: m.read(torch.zeros(3, 40, dtype=torch.int8), stream=0)),
        (ValueError, lambda: m.matmul(m, torch.zeros(8, 4).t(), stream=0)),
        (ValueError, lambda: em.Block8(16, 40, codes=torch.zeros(16, 40, dtype=torch.uint8), device="cpu")),
        (ValueError, lambda: em.Block8(16, 40, scales=torch.zeros(512, dtype=torch.int8), device="cpu")),
        (em.EmeansError, lambda: em.Block8(0, 40, device="cpu")),
        (em.EmeansError, lambda: m.matmul(em.Block8(16, 41, device="cpu"), torch.zeros(2, 2), stream=0)),
        (em.EmeansError, lambda: m.matmul(m, torch.zeros(17, 2), stream=0)),
    ]
    for err, call in bad:
        with pytest.raises(err):
            call()
    assert m.write(torch.zeros(0, 40, dtype=f), stream=0) is None
    assert m.read(torch.zeros(0, 40), stream=0).shape == (0, 40)
    assert m.matmul(m, torch.zeros(0, 3), stream=0).shape == (0, 3)


def test_a_model_refuses_data_of_other_types(em):
    """float16 rows, which a Block8 can be written from, are no input of a model: they would
    be read as float32, past their end."""
    class Options:
        was = 0

        def get_option(self, name):
            return self.was

        def set_option(self, name, value):
            self.was = value

    m = Options()
    m._raw_dtype = None
    for X, want in ((torch.zeros(3, 4), 0), (torch.zeros(3, 4, dtype=torch.bfloat16), 1), (np.zeros((3, 4), np.float32), 0)):
        m.was = 7
        em.Model._dtype_of(m, X)
        assert m.was == want
    for X in (torch.zeros(3, 4).half(), torch.zeros(3, 4).double(), torch.zeros(3, 4).long(), np.zeros((3, 4)), np.zeros((3, 4), np.float16)):
        with pytest.raises(TypeError):
            em.Model._dtype_of(m, X)
