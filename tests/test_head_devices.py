"""Tensors of a GPU that is not the current one: the binding refuses them
before anything is launched. (A launch goes to the current device, whatever
device its stream was asked for: a default stream's handle is 0 everywhere.)
No GPU is needed: the tensors are stand-ins and the library is never reached.
"""
import pytest

import token_perturbation_estimator_gb300 as dust

torch = pytest.importorskip("torch")


class OnGpu:
    """What the binding reads of a contiguous CUDA tensor."""

    is_cuda = True

    def __init__(self, shape, index, dtype=None):
        self.like = torch.empty(shape, dtype=dtype or torch.float32, device="meta")
        self.index = index
        self.shape, self.dtype = self.like.shape, self.like.dtype
        self.device = torch.device("cuda", index)

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 1 << 20

    def as_strided(self, shape, stride):
        return OnGpu(shape, self.index, self.dtype)

    def __getattr__(self, name):  # dim, stride, is_contiguous, numel
        return getattr(self.like, name)


class Reached(Exception):
    pass


def _calls(i):
    T, d, V, K = 4, 16, 32, 3
    f = lambda *shape: OnGpu(shape, i)  # noqa: E731
    ids = lambda *shape: OnGpu(shape, i, torch.int32)  # noqa: E731
    x, E, row, st, ws = f(T, d), f(V, d), f(T), f(T, K), OnGpu((1 << 20,), i, torch.uint8)
    loss = dict(loss=row, lse=row, workspace=ws)
    grad = dict(gH=x, gE=E, workspace=ws)
    return {
        "dust_layer_norm": lambda: dust.dust_layer_norm(x, y=x, mean=row, rstd=row),
        "dust_layer_norm_grad": lambda: dust.dust_layer_norm_grad(
            x, x, row, row, gx=x, gweight=f(d), gbias=f(d), workspace=ws),
        "dust_head_loss": lambda: dust.dust_head_loss(x, E, ids(T), **loss),
        "dust_head_loss_grad": lambda: dust.dust_head_loss_grad(x, E, ids(T), row, row, **grad),
        "dust_distill_loss": lambda: dust.dust_distill_loss(x, E, ids(T, K), st, student=st,
                                                            **loss),
        "dust_distill_loss_grad": lambda: dust.dust_distill_loss_grad(
            x, E, ids(T, K), st, row, st, row, **grad),
    }


@pytest.mark.parametrize("name", sorted(_calls(0)))
@pytest.mark.parametrize("tensors,current", [(1, 0), (0, 1), (0, 0), (1, 1)])
def test_tensors_have_to_be_on_the_current_device(name, tensors, current, monkeypatch):
    def reached():
        raise Reached

    monkeypatch.setattr(dust, "lib", reached)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
    monkeypatch.setattr(dust, "_types_cache", None)  # made anew, with this current device
    # (monkeypatch puts the cache back afterwards)
    call = _calls(tensors)[name]
    if tensors == current:
        with pytest.raises(Reached):
            call()
    else:
        with pytest.raises(ValueError, match="cuda:%d.*current.*cuda:%d" % (tensors, current)):
            call()
