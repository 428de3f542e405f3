"""Orthogonalised updates of long thin matrices, and of matrices that are zero or
next to it, with an eps as small as fp32 has one.  Bounds: those of
test_gpu_orthogonalize.py."""
import numpy as np
import pytest
import torch

from tests.test_gpu_orthogonalize import check, run, values

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

# of a cluster, and of the general kernels
SHAPES = [(3, 64, 80), (2, 128, 300), (3, 300, 280), (2, 140, 600)]


@pytest.mark.parametrize("eps", [np.float32(1.2e-38), np.float32(1e-45)])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("momentum", [0.0, 0.9])
def test_zero_matrices_stay_zero_with_any_eps(shape, dtype, eps, momentum):
    g = values(shape, "full", 1)
    g[1] = 0
    kw = dict(eps=float(eps), momentum=momentum, nesterov=True)
    got = run(g, dtype=dtype, mom=np.zeros(shape) if momentum else None, **kw)
    assert not got[2][1].any()
    check(*got, **kw)


@pytest.mark.parametrize("eps", [np.float32(1e-36), np.float32(1.2e-38), np.float32(1e-45)])
@pytest.mark.parametrize("size", [1e-36, 1e-38, 1e-40])
@pytest.mark.parametrize("shape", SHAPES)
def test_matrices_of_the_smallest_numbers(shape, size, eps):
    """The factor that makes the norm one is past fp32's range."""
    g = values(shape, "full", 2) * size
    check(*run(g, dtype=torch.float32, eps=float(eps)), eps=float(eps))


@pytest.mark.parametrize("shape", SHAPES)
def test_matrices_of_the_largest_numbers(shape):
    g = np.clip(values(shape, "full", 3), -3, 3) * 1.1e38
    check(*run(g, dtype=torch.float32))


@pytest.mark.parametrize("shape", [(1, 64, 4104), (3, 64, 7168), (2, 1, 5000), (1, 9, 16384),
                                   (2, 33, 4500), (1, 128, 2056), (2, 100, 7168), (1, 256, 7168)])
@pytest.mark.parametrize("tall", [False, True])
def test_long_thin_matrices_that_no_cluster_holds(shape, tall):
    b, m, n = shape
    check(*run(values((b, n, m) if tall else shape, "full", 4)))
