"""W4Weight has no backward pass: a call that would lose a gradient is refused, before anything else of it is looked at."""
import pytest
import torch


@pytest.fixture(scope="module")
def w():
    from graph_replay_gb300 import W4Weight, build
    build.build()
    return object.__new__(W4Weight)   # needs no device: the check comes first


def grad(*shape):
    return torch.zeros(*shape, requires_grad=True)


@pytest.mark.parametrize("kw", [dict(x=grad(2, 64)), dict(norm=grad(64)), dict(residual=grad(2, 32)), dict(out=grad(2, 32)),
                                dict(x=grad(2, 64) * 2.0)])
def test_refused(w, kw):
    x = kw.pop("x", torch.zeros(2, 64))
    with pytest.raises(ValueError, match="gradient"):
        w.linear(x, **kw)
    if "residual" not in kw:
        with pytest.raises(ValueError, match="gradient"):
            w.glu(w, x, **kw)


@pytest.mark.parametrize("off", [torch.no_grad, torch.inference_mode])
def test_passes_without_gradients(w, off):
    """Where none is recorded, the call goes on to what it needs next (this one has no device)."""
    with off(), pytest.raises(AttributeError):
        w.linear(grad(2, 64), norm=grad(64))
    with pytest.raises(AttributeError):
        w.linear(torch.zeros(2, 64), norm=torch.zeros(64))
