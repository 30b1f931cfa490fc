"""Block8 calls next to autograd: results that require gradients are refused, and what a
call writes counts as modified in place."""

import os

import pytest
import torch

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


def test_results_that_require_gradients_are_refused(em):
    m = em.Block8(16, 40, device="cpu")
    leaf = torch.zeros(0, 40, requires_grad=True)
    for call in (lambda o: m.read(o, stream=0), lambda o: m.matmul(em.Block8(40, 40, device="cpu"), o, stream=0)):
        for out in (leaf, leaf * 2):
            with pytest.raises(ValueError):
                call(out)
            with torch.no_grad():
                assert call(out) is out
    assert m.write(leaf, stream=0) is None  # the values alone


def test_what_a_call_writes_counts_as_modified(em):
    m = em.Block8(16, 40, device="cpu")
    base = torch.zeros(4, 44)
    out = base[:0, :40]
    was = base._version
    m.read(out, stream=0)
    assert base._version > was
    was = base._version
    m.matmul(em.Block8(40, 40, device="cpu"), out, stream=0)
    assert base._version > was
    was = m.codes._version, m.scales._version
    m.write(torch.zeros(0, 40), stream=0)
    assert m.codes._version > was[0] and m.scales._version > was[1]
    with torch.inference_mode():  # tensors without versions
        k = em.Block8(16, 40, device="cpu")
        k.write(torch.zeros(0, 40), stream=0)
        k.read(torch.zeros(0, 40), stream=0)
    k.write(torch.zeros(0, 40), stream=0)
    k.read(torch.zeros(0, 40), stream=0)


@pytest.mark.gpu
def test_a_backward_pass_refuses_what_a_call_has_overwritten(em):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    m = em.Block8(64, 40)
    x = torch.randn(64, 40, device="cuda")
    m.write(x)
    w = torch.ones(64, 40, device="cuda", requires_grad=True)
    v = torch.ones(64, 64, device="cuda", requires_grad=True)
    out, scores = torch.empty(64, 40, device="cuda"), torch.empty(64, 64, device="cuda")
    m.read(out)
    m.matmul(m, scores)
    (w * out).sum().backward()
    assert torch.equal(w.grad, out)
    for loss, again in (((w * out).sum(), lambda: m.read(out)), ((v * scores).sum(), lambda: m.matmul(m, scores))):
        again()
        with pytest.raises(RuntimeError, match="inplace"):
            loss.backward()


@pytest.mark.gpu
def test_values_that_require_gradients_are_written_as_they_are(em):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    x = torch.randn(64, 40, device="cuda", requires_grad=True)
    a, b = em.Block8(64, 40), em.Block8(64, 40)
    a.write(x)
    b.write(x.detach())
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
