"""A block8 matrix as a model's data: what a refused call leaves behind."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def em():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import mini_ema_means_b200

    return mini_ema_means_b200


D, K, N = 90, 24, 3000


def _store(em, n=N, d=D, seed=3):
    g = np.random.default_rng(seed)
    x = torch.from_numpy(g.standard_normal((n, d)) + 3 * g.integers(0, 4, (n, 1))).float()
    m8 = em.Block8(n, d)
    m8.write(x.cuda())
    m8.check()
    return m8


def _centroids(m):
    c = torch.empty(m.k, m.d)
    m.centroids(c)
    return c


def _refused(em):
    """(matrix, rows asked for) that no model of D values can take."""
    host = em.Block8(N, D, device="cpu")
    torn = _store(em)
    torn.view.scales = None
    return [(_store(em), (1 << 31) - 1), (_store(em), N + 1), (_store(em, d=D + 1), N), (torn, N), (host, N)]


def test_a_matrix_is_refused_before_anything_is_allocated(em):
    """Each model call with a matrix that it cannot take is EM_E_INVAL, whatever the number
    of rows, and makes no allocation."""
    m8 = _store(em)
    m = em.Model(D, K, seed=5)
    m.train(m8, epochs=2.0)
    calls = {"train": lambda X, n: em.em_train(m.h, em._ptr(X), n, 1.0), "begin": lambda X, n: em.em_begin(m.h, em._ptr(X), n, 1.0),
             "lloyd": lambda X, n: em.em_lloyd(m.h, em._ptr(X), n, 1),
             "assign": lambda X, n: em.em_assign(m.h, em._ptr(X), n, None, None),
             "mse": lambda X, n: em.em_mse(m.h, em._ptr(X), n, em.ctypes.byref(em.ctypes.c_double()))}
    for X, n in _refused(em):
        for name, call in calls.items():
            em.fail_allocation(0)
            assert call(X, n) == em.EM_E_INVAL, (name, X.shape, n, em.em_last_error())
            assert em.fail_allocation(0) == 0, (name, X.shape, n)
    m.close()


def test_a_refused_matrix_leaves_the_run_as_it_was(em):
    """A run in progress goes on after the refusal of another matrix, and a finished one
    keeps its labels, recipe and error history."""
    m8 = _store(em)
    got = []
    for refuse in (False, True):
        m = em.Model(D, K, seed=5)
        recipe = m.begin(m8, epochs=2.0)
        m.step(3)
        if refuse:
            for X, n in _refused(em):
                assert em.em_begin(m.h, em._ptr(X), n, 1.0) == em.EM_E_INVAL
        m.step(10 ** 6)
        m.finalize()
        if refuse:
            for X, n in _refused(em):
                assert em.em_lloyd(m.h, em._ptr(X), n, 1) == em.EM_E_INVAL
                assert em.em_train(m.h, em._ptr(X), n, 1.0) == em.EM_E_INVAL
        assert m.recipe() == recipe
        lab = torch.full((N + 5,), -7, dtype=torch.int64)
        m.labels(lab)
        assert (lab[N:] == -7).all() and (lab[:N] >= 0).all()
        got.append((_centroids(m), lab, torch.from_numpy(m.obj())))
        m.close()
    assert all(torch.equal(a, b) for a, b in zip(*got))


def _finished(em):
    """A finished run on N rows that checks its data, and what it reports."""
    m = em.Model(D, K, seed=5, check_finite=1)
    m.train(_store(em), epochs=2.0)
    lab = torch.full((2 * N,), -7, dtype=torch.int64)
    m.labels(lab)
    return m, (lab, m.recipe(), m.obj().tolist(), m.stats()["steps_done"])


@pytest.mark.parametrize("kind", ["block8", "float32", "bfloat16"])
def test_data_that_are_not_finite_leave_the_last_run_readable(em, kind):
    """More rows than the last run had, one of them NaN: em_begin, em_train and em_lloyd
    refuse them, and the last run's labels, recipe and error history stay, with its number
    of rows; then the same model trains as a new one does."""
    x = torch.randn(2 * N - 1, D, generator=torch.Generator().manual_seed(1))
    good = x.cuda()
    x[N + 7, 3] = float("nan")
    X = x.cuda()
    if kind == "block8":
        X = em.Block8(2 * N - 1, D)
        X.write(x.cuda())
        X.check()
    elif kind == "bfloat16":
        X = X.bfloat16()
    m, want = _finished(em)
    for call in (lambda: m.begin(X), lambda: m.train(X), lambda: m.lloyd(X, 2)):
        with pytest.raises(em.EmeansError) as e:
            call()
        assert e.value.code == em.EM_E_NONFINITE
        lab = torch.full((2 * N,), -7, dtype=torch.int64)
        m.labels(lab)
        assert torch.equal(lab, want[0]) and (lab[N:] == -7).all()
        assert (m.recipe(), m.obj().tolist(), m.stats()["steps_done"]) == want[1:]
        with pytest.raises(em.EmeansError) as e:
            m.step(1)
        assert e.value.code == em.EM_E_STATE
    fresh = em.Model(D, K, seed=5)
    for t in (m, fresh):
        t.train(good, epochs=1.0)
    assert torch.equal(_centroids(m), _centroids(fresh))
    m.close()
    fresh.close()


def test_labels_kept_from_the_middle_of_a_run_on_are_refused(em):
    """A run begun without keeping labels has none, also where the option is set later."""
    m = em.Model(D, K, seed=5)
    m.train(_store(em, n=500), epochs=1.0)
    m.set_option("capture_labels", 0)
    store = _store(em)
    m.begin(store, epochs=2.0)
    m.set_option("capture_labels", 1)
    m.step(10 ** 6)
    m.finalize()
    with pytest.raises(em.EmeansError) as e:
        m.labels(torch.empty(N, dtype=torch.int64))
    assert e.value.code == em.EM_E_STATE
    m.train(store, epochs=2.0)
    lab = torch.empty(N, dtype=torch.int64)
    m.labels(lab)
    assert (lab >= 0).all() and (lab < K).all()
    m.close()
