"""The 4-bit decode's choice of splits and of their merge, and what its launcher does where a cluster is refused, on the CPU:
the sources themselves against stand-ins for the runtime calls that they make."""
import ctypes
import os
import shutil
import subprocess

import pytest

from paged_gqa_attention_gb300 import build as pa_build
from paged_gqa_attention_gb300 import ops

LAUNCHER = r"""
#include <cuda_runtime.h>

static int f_device, f_refusal, f_query_error, f_lone, f_fit, f_launches, f_cluster_of[4], f_cleared, f_queries, f_set;

template <typename... A>
static cudaError_t fake_launch(const cudaLaunchConfig_t *cfg, A...) {
    int ctas = 1;
    for (unsigned i = 0; i < cfg->numAttrs; ++i)
        if (cfg->attrs[i].id == cudaLaunchAttributeClusterDimension) ctas = (int)cfg->attrs[i].val.clusterDim.y;
    if (f_launches < 4) f_cluster_of[f_launches] = ctas;
    ++f_launches;
    return ctas > 1 ? (cudaError_t)f_refusal : cudaSuccess;
}
template <typename K>
static cudaError_t fake_clusters(int *n, K, const cudaLaunchConfig_t *cfg) {
    ++f_queries;
    // (with more than half of an SM's shared memory a CTA has an SM to itself)
    *n = f_query_error ? 0 : 2 * cfg->dynamicSmemBytes > 233472 ? f_lone : f_fit;
    return (cudaError_t)f_query_error;
}
template <typename K>
static cudaError_t fake_attribute(K, cudaFuncAttribute, int) { ++f_set; return cudaSuccess; }
static cudaError_t fake_device(int *dev) { *dev = f_device; return cudaSuccess; }
static cudaError_t fake_last_error() { ++f_cleared; return cudaSuccess; }

#define cudaLaunchKernelEx fake_launch
#define cudaOccupancyMaxActiveClusters fake_clusters
#define cudaFuncSetAttribute fake_attribute
#define cudaGetDevice fake_device
#define cudaGetLastError fake_last_error
#include "decode_fp4.cu"

// in: device, refusal, batch, nsplit, cluster_merge; out: launches, clusters of the first four, cleared errors, kernels configured
extern "C" int launch4(const int *in, int *out) {
    f_device = in[0], f_refusal = in[1];
    f_launches = f_cleared = f_set = 0;
    pa::DecodeArgs a = {};
    a.batch = in[2], a.nsplit = in[3], a.cluster_merge = in[4];
    const CUtensorMap m = {};
    const int e = (int)pa::launch_decode_fp4(a, m, m, m, m, 0);
    out[0] = f_launches;
    for (int i = 0; i < 4; ++i) out[1 + i] = f_cluster_of[i];
    out[5] = f_cleared, out[6] = f_set;
    return e;
}
// in: device, query error, lone, fit; out: lone[9], fit[9], queries, cleared
extern "C" int room4(const int *in, int *out) {
    f_device = in[0], f_query_error = in[1], f_lone = in[2], f_fit = in[3];
    f_queries = f_cleared = 0;
    pa::ClusterRoom r;
    const int e = (int)pa::decode_fp4_clusters(r);
    for (int c = 0; c < 9; ++c) out[c] = r.lone[c], out[9 + c] = r.fit[c];
    out[18] = f_queries, out[19] = f_cleared;
    return e;
}
"""

CHOICE = r"""
#include <cuda_runtime.h>
#include <cuda.h>

static cudaError_t fake_device(int *dev) { *dev = 0; return cudaSuccess; }
static cudaError_t fake_sms(int *n, cudaDeviceAttr, int) { *n = 152; return cudaSuccess; }
static CUresult fake_encode(...) { return CUDA_SUCCESS; }
template <typename Q>
static cudaError_t fake_entry(const char *, void **fn, unsigned, unsigned long long, Q *q) {
    *fn = (void *)fake_encode;
    *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
#define cudaGetDevice fake_device
#define cudaDeviceGetAttribute fake_sms
#define cudaGetDriverEntryPointByVersion fake_entry
#include "api.cu"

static ClusterRoom f_room;
static int f_launched[4];
namespace pa {
cudaError_t decode_fp4_clusters(ClusterRoom &room) { room = f_room; return cudaSuccess; }
cudaError_t launch_decode_fp4(const DecodeArgs &a, const CUtensorMap &, const CUtensorMap &, const CUtensorMap &,
                              const CUtensorMap &, cudaStream_t) {
    f_launched[0] = 1, f_launched[1] = a.nsplit, f_launched[2] = a.split_tokens, f_launched[3] = a.cluster_merge;
    return cudaSuccess;
}
}  // namespace pa

// lone, fit: of every size of cluster; out: launched, nsplit, split_tokens, cluster_merge
extern "C" int decode4(int batch, int width, int window, int split, const int *lone, const int *fit, int *out) {
    for (int c = 0; c < 9; ++c) f_room.lone[c] = lone[c], f_room.fit[c] = fit[c];
    f_launched[0] = 0;
    char *p = (char *)256;     // (never read: the launch is a stand-in)
    const pa_shape shape = {32, 8, 128, 256};
    const int e = (int)paged_attn_decode_fp4(shape, p, nullptr, p, p, p, p, p, p, p, (int *)p, width, 1, (int *)p, batch, window, 0,
                                             0.1f, split, p, (size_t)1 << 40, nullptr);
    for (int i = 0; i < 4; ++i) out[i] = f_launched[i];
    return e;
}
extern "C" int merges4(long long pairs, long long splits, int sms, const int *lone, const int *fit) {
    for (int c = 0; c < 9; ++c) f_room.lone[c] = lone[c], f_room.fit[c] = fit[c];
    return merges_as_cluster(pairs, splits, sms, &f_room);
}
"""


def compiled(d, name, source, *link):
    if not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")):
        pytest.skip("no nvcc")
    src, lib = d / f"{name}.cu", d / f"{name}.so"
    src.write_text(source)
    cmd = [pa_build._nvcc(), "-gencode", "arch=compute_103a,code=compute_103a", "-O1", "-std=c++17", "-shared",
           "-Xcompiler", "-fPIC", "-I", pa_build.INCLUDE, "-I", pa_build.CSRC, "-o", str(lib), str(src), *link]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    return ctypes.CDLL(str(lib))


def ints(*x):
    return (ctypes.c_int * len(x))(*x)


@pytest.fixture(scope="module")
def launcher(tmp_path_factory):
    return compiled(tmp_path_factory.mktemp("launcher4"), "launcher", LAUNCHER)


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    pa_build.build()
    ops.load()
    return compiled(tmp_path_factory.mktemp("choice4"), "choice", CHOICE, pa_build.LIB_PATH, "-Xlinker", "-rpath", "-Xlinker",
                    os.path.dirname(pa_build.LIB_PATH))


def launch(lib, device, nsplit, cluster, refusal=0):
    out = ints(*[0] * 7)
    status = lib.launch4(ints(device, refusal, 1, nsplit, cluster), out)
    return status, list(out[1:1 + out[0]]), out[5], out[6]


def test_the_merge_asked_for_is_launched(launcher):
    assert launch(launcher, 0, 8, 1) == (0, [8], 0, 2)       # (and both kernels configured, once a device)
    assert launch(launcher, 0, 8, 0) == (0, [1], 0, 0)       # through the workspace
    assert launch(launcher, 0, 12, 0) == (0, [1], 0, 0)
    assert launch(launcher, 0, 9, 1) == (1, [], 0, 0)        # no such cluster


@pytest.mark.parametrize("refusal", [701, 720, 801, 912])
def test_a_refused_cluster_merges_through_the_workspace(launcher, refusal):
    """Launch out of resources, cooperative launch too large, not supported, invalid cluster size."""
    assert launch(launcher, 1, 6, 1, refusal)[:3] == (0, [6, 1], 1)


def test_another_error_is_returned(launcher):
    assert launch(launcher, 2, 6, 1, 719)[:3] == (719, [6], 0)


def room(lib, device, query_error=0, lone=18, fit=36):
    out = ints(*[0] * 20)
    assert lib.room4(ints(device, query_error, lone, fit), out) == 0
    return list(out[2:9]), list(out[11:18]), out[18], out[19]


def test_the_room_for_clusters_is_looked_up_once(launcher):
    assert room(launcher, 3) == ([18] * 7, [36] * 7, 14, 0)
    assert room(launcher, 3, lone=1, fit=1) == ([18] * 7, [36] * 7, 0, 0)
    assert room(launcher, 4, lone=0, fit=0) == ([-1] * 7, [-1] * 7, 14, 0)      # none fits: an answer
    assert room(launcher, 4) == ([-1] * 7, [-1] * 7, 0, 0)
    assert room(launcher, 5, query_error=46) == ([0] * 7, [0] * 7, 14, 14)      # could not be had: cleared, asked again
    assert room(launcher, 5) == ([18] * 7, [36] * 7, 14, 0)
    assert launcher.room4(ints(64, 0, 1, 1), ints(*[0] * 20)) == 101            # no such device


def test_clusters_only_where_all_of_them_are_there_at_once(choice):
    def merges(pairs, splits, lone, fit, sms=152):
        return choice.merges4(ctypes.c_longlong(pairs), ctypes.c_longlong(splits), sms, ints(*[lone] * 9), ints(*[fit] * 9))
    assert not merges(8, 1, 99, 99) and not merges(8, 9, 99, 99)
    assert merges(8, 2, 99, 99) and merges(8, 8, 99, 99)
    # up to an SM for each CTA the clusters of lone CTAs count, beyond that those of two CTAs an SM
    assert merges(19, 8, 19, 0) and not merges(19, 8, 18, 99)                   # 152 CTAs
    assert merges(20, 8, 0, 20) and not merges(20, 8, 99, 19)                   # 160
    assert not merges(8, 4, -1, -1) and not merges(8, 4, 0, 0)                  # none fits, or it is not known


@pytest.mark.parametrize("window", [2 ** 31 - 1, 700])
def test_the_decode_launches_the_merge_that_its_splits_were_chosen_for(choice, window):
    seen = set()
    for lone, fit in ((18, 36), (4, 36), (18, 4), (-1, -1), (0, 0)):
        for batch in (1, 2, 3, 5, 6, 10, 16, 19, 32, 38, 39, 64, 200):
            for width in (1, 2, 6, 16, 36, 160):
                out = ints(0, 0, 0, 0)
                assert choice.decode4(batch, width, window, 0, ints(*[lone] * 9), ints(*[fit] * 9), out) == 0
                launched, nsplit, tokens, cluster = out
                tiles = min(width, 700 // 256 + 2) if window == 700 else width
                assert launched and tokens % 256 == 0 and (nsplit - 1) * tokens < tiles * 256 <= nsplit * tokens
                there = lone if batch * 8 * nsplit <= 152 else fit
                assert bool(cluster) == (2 <= nsplit <= 8 and batch * 8 <= there)
                seen.add((nsplit > 1, bool(cluster)))
    assert seen == {(False, False), (True, False), (True, True)}


def test_a_split_length_of_the_caller(choice):
    room = ints(*[18] * 9), ints(*[36] * 9)
    out = ints(0, 0, 0, 0)
    for split, want in ((256, (36, 0)), (1280, (8, 1)), (9216, (1, 0))):
        assert choice.decode4(1, 36, 2 ** 31 - 1, split, *room, out) == 0
        assert (out[1], out[3], out[2]) == (*want, split)
