"""GPU: the FP64 exponential and reciprocal of the expert selection against extended precision on the host and CUDA's own.

Bounds, relative, in half units of the last place (2^-53): the exponential rounds three times (table, polynomial,
product) and loses 0.06 more to the polynomial's remainder and inner roundings: 3.1. The reciprocal's last step rounds
once: 1.001. CUDA's exp is off by at most one unit (2 halves), its division rounds once."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

HALF_ULP = 2.0 ** -53

SOURCE = """
#include "fp64.cuh"
__global__ void k(const double* x, double* y, double* cuda, int n, int which)
{
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) {
        y[i] = which ? moe::rcp64(x[i]) : moe::exp64(x[i]);
        cuda[i] = which ? 1.0 / x[i] : exp(x[i]);
    }
}
extern "C" int run(const double* x, double* y, double* cuda, int n, int which)
{
    k<<<256, 128>>>(x, y, cuda, n, which);
    return static_cast<int>(cudaDeviceSynchronize());
}
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_w4a4_mixture_gb300 import build as b

    folder = tmp_path_factory.mktemp("fp64")
    src, lib = str(folder / "fp64.cu"), str(folder / "fp64.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([b._nvcc()] + b.ARCH + b.FLAGS + ["-I" + b.SRC_DIR, "-shared", src, "-o", lib], check=True)
    L = ctypes.CDLL(os.path.abspath(lib))

    def call(x, which):
        x = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float64)).cuda()
        y, cuda = torch.empty_like(x), torch.empty_like(x)
        torch.cuda.synchronize()
        p = [ctypes.c_void_p(t.data_ptr()) for t in (x, y, cuda)]
        assert L.run(*p, x.numel(), which) == 0
        return y.cpu().numpy(), cuda.cpu().numpy()

    return call


def relative(got, want):
    return float(np.max(np.abs((got.astype(np.longdouble) - want) / want)))


def test_exponential(run):
    assert np.finfo(np.longdouble).eps < 1e-18
    rng = np.random.default_rng(0)
    ns = np.arange(-32300, 32300)
    border = (ns + 0.5) * (np.log(2.0) / 32)  # between two entries of the table
    x = np.concatenate([rng.uniform(-40, 40, 200000), rng.uniform(-700, 700, 100000), rng.uniform(-0.02, 0.02, 50000),
                        border, np.nextafter(border, 1e9), np.nextafter(border, -1e9), ns * (np.log(2.0) / 32),
                        np.ldexp(1.0, -np.arange(1, 1000)), -np.ldexp(1.0, -np.arange(1, 1000)),
                        [0.0, -0.0, 1.0, -1.0, np.nextafter(700.0, 0), np.nextafter(-700.0, 0)]])
    x = x[np.abs(x) < 700]
    got, cuda = run(x, 0)
    assert relative(got, np.exp(x.astype(np.longdouble))) <= 3.1 * HALF_ULP
    assert relative(got, cuda.astype(np.longdouble)) <= (3.1 + 2.0) * HALF_ULP * 1.001
    assert np.all(got[x == 0] == 1.0)


def test_exponential_past_its_range(run):
    x = np.array([700.0, -700.0, 709.0, 710.0, -740.0, -750.0, 1e300, -1e300, np.inf, -np.inf, np.nan])
    got, cuda = run(x, 0)
    np.testing.assert_array_equal(got, cuda)
    assert got[8] == np.inf and got[9] == 0.0 and np.isnan(got[10])


def test_reciprocal(run):
    rng = np.random.default_rng(1)
    p = np.ldexp(1.0, np.arange(0, 99))
    d = np.concatenate([np.exp(rng.uniform(0, np.log(9e29), 200000)), rng.uniform(1, 2, 100000), rng.uniform(1, 1024, 100000),
                        p, np.nextafter(p, 1e300), np.nextafter(p[1:], 0), np.arange(1.0, 2000.0)])
    got, cuda = run(d, 1)
    assert relative(got, 1 / d.astype(np.longdouble)) <= 1.001 * HALF_ULP
    assert relative(got, cuda.astype(np.longdouble)) <= 2.002 * HALF_ULP
    past = np.array([1e30, 1e40, 1e300, np.inf, np.nan])
    got, cuda = run(past, 1)
    np.testing.assert_array_equal(got, cuda)
