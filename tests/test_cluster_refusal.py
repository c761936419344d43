"""What the windowed prefill's launcher does where clusters are refused (SMs partitioned or shared
with other work), on the CPU: its own source against stand-ins for the few runtime calls it makes."""
import ctypes
import os
import shutil
import subprocess

import pytest

from paged_gqa_attention_gb300 import build as pa_build

HARNESS = r"""
#include <cuda_runtime.h>

// stand-ins: what the launcher asks of the runtime, and what the test lets it answer
static int f_device, f_refusal, f_query_error, f_clusters, f_launches, f_cluster_of[8], f_cleared, f_queries;

template <typename... A>
static cudaError_t fake_launch(const cudaLaunchConfig_t *cfg, A...) {
    int ctas = 1;
    for (unsigned i = 0; i < cfg->numAttrs; ++i)
        if (cfg->attrs[i].id == cudaLaunchAttributeClusterDimension) ctas = (int)cfg->attrs[i].val.clusterDim.x;
    if (f_launches < 8) f_cluster_of[f_launches] = ctas;
    ++f_launches;
    return ctas > 1 ? (cudaError_t)f_refusal : cudaSuccess;
}
template <typename K>
static cudaError_t fake_clusters(int *n, K, const cudaLaunchConfig_t *) {
    ++f_queries;
    *n = f_query_error ? 0 : f_clusters;
    return (cudaError_t)f_query_error;
}
template <typename K>
static cudaError_t fake_attribute(K, cudaFuncAttribute, int) { return cudaSuccess; }
static cudaError_t fake_device(int *dev) { *dev = f_device; return cudaSuccess; }
static cudaError_t fake_last_error() { ++f_cleared; return cudaSuccess; }

#define cudaLaunchKernelEx fake_launch
#define cudaOccupancyMaxActiveClusters fake_clusters
#define cudaFuncSetAttribute fake_attribute
#define cudaGetDevice fake_device
#define cudaGetLastError fake_last_error
#include "prefill.cu"

// in: device, refusal, query_error, clusters, max_q_len, tiles; out: launches, their clusters, cleared, queries
extern "C" int window_launch(const int *in, int *out) {
    f_device = in[0], f_refusal = in[1], f_query_error = in[2], f_clusters = in[3];
    f_launches = f_cleared = f_queries = 0;
    pa::PrefillArgs a = {};
    a.num_seqs = 1, a.max_q_len = in[4], a.total_tokens = in[4], a.max_blocks_per_seq = 64, a.window = 4096;
    const CUtensorMap m = {};
    const int e = (int)pa::launch_prefill_window(a, in[5], m, m, m, m, m, 152, 0);
    out[0] = f_launches, out[1] = f_cluster_of[0], out[2] = f_cluster_of[1], out[3] = f_cleared, out[4] = f_queries;
    return e;
}
"""


@pytest.fixture(scope="module")
def launch(tmp_path_factory):
    if not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")):
        pytest.skip("no nvcc")
    d = tmp_path_factory.mktemp("launcher")
    src, lib = d / "harness.cu", d / "harness.so"
    src.write_text(HARNESS)
    cmd = [pa_build._nvcc(), "-gencode", "arch=compute_103a,code=compute_103a", "-O1", "-std=c++17", "-shared",
           "-Xcompiler", "-fPIC", "-I", pa_build.INCLUDE, "-I", pa_build.CSRC, "-o", str(lib), str(src)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    fn = ctypes.CDLL(str(lib)).window_launch

    def call(device, refusal=0, query_error=0, clusters=18, max_q_len=64, tiles=34):
        out = (ctypes.c_int * 5)()
        status = fn((ctypes.c_int * 6)(device, refusal, query_error, clusters, max_q_len, tiles), out)
        return status, list(out[1:1 + min(out[0], 2)]), out[3], out[4]

    return call


def test_few_units_run_as_clusters(launch):
    status, ctas, cleared, queries = launch(0)
    assert status == 0 and len(ctas) == 1 and ctas[0] > 1 and cleared == 0 and queries == 7
    assert launch(0)[3] == 0                                    # the answer is kept
    assert launch(0, max_q_len=64 * 12)[1] == [1]               # many units: no clusters


@pytest.mark.parametrize("refusal", [701, 720, 801, 912])
def test_a_refused_cluster_runs_unclustered(launch, refusal):
    """Launch out of resources, cooperative launch too large, not supported, invalid cluster size:
    the launch error is cleared and the same work launched without clusters."""
    status, ctas, cleared, _ = launch(1, refusal=refusal)
    assert status == 0 and len(ctas) == 2 and ctas[0] > 1 and ctas[1] == 1 and cleared == 1


def test_another_error_is_returned(launch):
    status, ctas, cleared, _ = launch(2, refusal=719)           # launch failure
    assert status == 719 and len(ctas) == 1 and cleared == 0


def test_a_failed_query_is_asked_again(launch):
    """The number of clusters that fit could not be had: no clusters this time, but the next call asks
    again."""
    status, ctas, cleared, queries = launch(3, query_error=46)  # devices unavailable
    assert status == 0 and ctas == [1] and cleared == queries == 7
    status, ctas, _, queries = launch(3)
    assert status == 0 and ctas[0] > 1 and queries == 7


def test_no_clusters_that_fit_is_an_answer(launch):
    assert launch(4, clusters=0)[:2] == (0, [1])
    assert launch(4, clusters=18)[1::2] == ([1], 0)
