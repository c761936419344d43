"""What the low-bit prefill's launcher does where clusters are refused (SMs partitioned or shared with other work), on
the CPU: its own source against stand-ins for the few runtime calls it makes."""
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
#include "prefill_quant.cu"

// in: device, refusal, query_error, clusters, max_q_len, tiles, sequences, bits; out: launches, the clusters of the first
// eight, cleared errors
extern "C" int quant_launch(const int *in, int *out) {
    f_device = in[0], f_refusal = in[1], f_query_error = in[2], f_clusters = in[3];
    f_launches = f_cleared = f_queries = 0;
    static int32_t order;
    static uint8_t exps;
    pa::PrefillArgs a = {};
    a.num_seqs = in[6], a.max_q_len = in[4], a.total_tokens = in[4] * in[6], a.max_blocks_per_seq = 64, a.window = 1 << 30;
    a.order = &order;
    if (in[7] == 4) a.k_exp = a.v_exp = &exps;
    const CUtensorMap m = {};
    const int e = (int)pa::launch_prefill_quant(a, in[5], m, m, m, m, m, 152, 0);
    out[0] = f_launches;
    for (int i = 0; i < 8; ++i) out[1 + i] = f_cluster_of[i];
    out[9] = f_cleared;
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
    fn = ctypes.CDLL(str(lib)).quant_launch

    def call(device, bits, max_q_len, seqs, refusal=0, clusters=18, tiles=34, query_error=0):
        out = (ctypes.c_int * 10)()
        status = fn((ctypes.c_int * 8)(device, refusal, query_error, clusters, max_q_len, tiles, seqs, bits), out)
        return status, list(out[1:1 + out[0]]), out[9]

    return call


BITS = pytest.mark.parametrize("bits", [8, 4])


@BITS
def test_the_forms_by_size(launch, bits):
    status, ctas, cleared = launch(0, bits, 64, 1)
    assert status == 0 and len(ctas) == 1 and ctas[0] > 1 and cleared == 0        # few units: their keys are split
    assert launch(0, bits, 64 * 20, 1) == (0, [1, 2], 0)                          # more pairs than fit: planned, in pairs
    assert launch(0, bits, 65, 5) == (0, [2], 0)                                  # pairs that all start at once
    assert launch(0, bits, 64, 30) == (0, [1, 1], 0)                              # nobody to share with: planned, one CTA each
    assert launch(0, bits, 64, 18) == (0, [1], 0)                                 # all units start at once: no planning


@BITS
@pytest.mark.parametrize("refusal", [701, 720, 801, 912])
def test_a_refused_cluster_runs_without(launch, refusal, bits):
    """Launch out of resources, cooperative launch too large, not supported, invalid cluster size: the
    launch error is cleared and the same work launched in the next form, in the end one CTA a unit."""
    status, ctas, cleared = launch(1, bits, 64, 1, refusal)
    assert status == 0 and len(ctas) == 2 and ctas[0] > 1 and ctas[1] == 1 and cleared == 1
    status, ctas, cleared = launch(6, bits, 129, 1, refusal, clusters=24)   # (24 units, on a device of its own)
    assert status == 0 and len(ctas) == 3 and ctas[0] > 1 and ctas[1:] == [2, 1] and cleared == 2
    status, ctas, cleared = launch(1, bits, 64 * 20, 1, refusal)
    assert status == 0 and ctas == [1, 2, 1, 1] and cleared == 1                  # (each form plans for itself)


@BITS
def test_another_error_is_returned(launch, bits):
    assert launch(2, bits, 64 * 20, 1, refusal=719)[::2] == (719, 0)              # launch failure
    assert launch(2, bits, 64, 1, refusal=719)[::2] == (719, 0)


@BITS
def test_no_clusters_that_fit_is_an_answer(launch, bits):
    assert launch(4, bits, 64, 1, clusters=0) == (0, [1], 0)
    assert launch(5, bits, 64, 1, query_error=46)[:2] == (0, [1])                 # could not be had: asked again next time
    assert launch(5, bits, 64, 1)[1][0] > 1
