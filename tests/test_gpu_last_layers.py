"""The example of the operators used together: finite everywhere, and the
estimate of the layer's weight gradient from the head's loss changes points
where the exact gradient does, as far as K draws of a d-wide jitter can (the
cosine law sqrt(K / (K + d)) of a per-token search of d dimensions; the sums
over tokens average its noise, so the cosine is at least about that)."""
import importlib.util
import os

import pytest

from helpers import cuda

pytestmark = pytest.mark.gpu


def test_example_runs_and_the_estimate_points_the_right_way():
    import torch
    cuda()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "last_layers.py")
    spec = importlib.util.spec_from_file_location("last_layers", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    out = m.step(T=2048, d=128, V=1000, K=64, sigma=0.02)
    assert 4.0 < out["loss"] < 12.0 and out["distillation"] > 0.0
    for k in ("gE", "gweight", "gbias", "dH", "dE"):
        assert torch.isfinite(out[k].float()).all(), k
    assert out["cosine"] > 0.5 * out["expected_cosine"]
