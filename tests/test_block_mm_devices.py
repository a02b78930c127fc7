"""The product's host side on several devices and from several threads, against a fake CUDA runtime: what a kernel has to be
granted (more than 48 KB of shared memory) is granted on every device that it is launched on, and what is asked of one
device is not taken for another's. The object of csrc/wq4_block_mm.cu is linked with the fake; runs without a GPU."""
import os
import shutil
import subprocess

import pytest

import weight_only_quantized_wq4_gb300 as wq4
from weight_only_quantized_wq4_gb300 import builder

OUT = os.path.join(builder.BUILD, "fake_cuda")

FAKE = r"""
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <mutex>
#include <thread>
#include <utility>
#include <vector>
#include "wq4_runtime.h"

namespace {
thread_local int g_device = 0;
std::mutex g_mu;
std::map<std::pair<int, const void*>, int> g_granted;     // (device, kernel) -> bytes of shared memory
int g_clusters[8] = {30, 10, 30, 30, 30, 30, 30, 30};     // clusters that each device holds
int g_fail_attribute = 0;
unsigned g_last_cluster = 0;
int g_launches = 0, g_refused = 0;

template <typename R> auto set_device(R& r, int d, int) -> decltype(r.device = d, void()) { r.device = d; }
template <typename R> void set_device(R&, int, long) {}

CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
    return CUDA_SUCCESS;
}
}  // namespace

namespace wq4 {
int runtime(Runtime* out) {
    std::memset(out, 0, sizeof *out);
    out->sm_count = 152;
    out->timeout_cycles = 1;
    out->encode = encode;
    set_device(*out, g_device, 0);
    return WQ4_OK;
}
}  // namespace wq4

extern "C" {
void** __cudaRegisterFatBinary(void*) { static void* p; return &p; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, uint3*, uint3*, dim3*, dim3*, int*) {}
cudaError_t __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return cudaErrorUnknown; }
cudaError_t __cudaGetKernel(cudaKernel_t*, const void*) { return cudaErrorUnknown; }
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void**, size_t, cudaStream_t) { return cudaErrorUnknown; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) {
    std::memset(a, 0, sizeof *a);
    a->numRegs = 168;
    return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute, int v) {
    std::lock_guard<std::mutex> lk(g_mu);
    if (g_fail_attribute) return cudaErrorUnknown;
    g_granted[{g_device, f}] = v;
    return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t*) {
    *n = g_clusters[g_device];
    return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
    std::lock_guard<std::mutex> lk(g_mu);
    auto it = g_granted.find({g_device, f});
    const size_t most = it == g_granted.end() ? 48 * 1024 : it->second;
    if (c->dynamicSmemBytes > most) { ++g_refused; return cudaErrorInvalidValue; }
    ++g_launches;
    g_last_cluster = 1;
    for (unsigned i = 0; i < c->numAttrs; ++i)
        if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) g_last_cluster = c->attrs[i].val.clusterDim.x;
    return cudaSuccess;
}
}

static int call(int M, int N, int K) {
    return wq4_block_mm(reinterpret_cast<void*>(0x10000), 8192, reinterpret_cast<float*>(0x20000), 8192, reinterpret_cast<void*>(0x30000),
                        8192, reinterpret_cast<float*>(0x40000), 64, reinterpret_cast<void*>(0x50000), 8192, M, N, K, WQ4_BF16, nullptr);
}

int main(int, char** v) {
    const char* what = v[1];
    const int sizes[][3] = {{4, 2560, 1024}, {20, 2560, 1024}, {60, 2560, 1024}, {100, 2560, 1024}, {3000, 8000, 1024}};
    if (!std::strcmp(what, "devices")) {                   // every form on one device, then on the next, then back
        for (int d : {0, 1, 0, 7, 1})
            for (auto& s : sizes) {
                g_device = d;
                const int rc = call(s[0], s[1], s[2]);
                if (rc != WQ4_OK) std::printf("device %d M %d: status %d\n", d, s[0], rc);
            }
    } else if (!std::strcmp(what, "occupancy")) {          // 20 tiles: clusters where the device holds 20 of them
        for (int d : {0, 1, 0}) {
            g_device = d;
            if (call(4, 2560, 1024) != WQ4_OK) std::printf("device %d: failed\n", d);
            if ((g_last_cluster > 1) != (g_clusters[d] >= 20)) std::printf("device %d: clusters of %u\n", d, g_last_cluster);
        }
    } else if (!std::strcmp(what, "failure")) {            // a refused attribute is an error, and asked for again next time
        g_fail_attribute = 1;
        if (call(100, 2560, 1024) != WQ4_ERR_CUDA) std::printf("no error\n");
        g_fail_attribute = 0;
        if (call(100, 2560, 1024) != WQ4_OK) std::printf("the failure was kept\n");
    } else {                                               // eight host threads, a device each
        std::vector<std::thread> t;
        int bad[8] = {};
        for (int d = 0; d < 8; ++d)
            t.emplace_back([&, d] {
                g_device = d;
                for (int i = 0; i < 50; ++i)
                    for (auto& s : sizes) bad[d] += call(s[0], s[1], s[2]) != WQ4_OK;
            });
        for (auto& x : t) x.join();
        for (int d = 0; d < 8; ++d)
            if (bad[d]) std::printf("device %d: %d of 250 calls failed\n", d, bad[d]);
    }
    std::printf("launches %d refused %d\n", g_launches, g_refused);
    return 0;
}
"""


@pytest.fixture(scope="module")
def exe():
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    wq4.build()
    os.makedirs(OUT, exist_ok=True)
    src, out = os.path.join(OUT, "fake.cpp"), os.path.join(OUT, "fake")
    with open(src, "w") as f:
        f.write(FAKE)
    cuda = os.path.join(os.path.dirname(os.path.dirname(builder._nvcc())), "include")
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-w", "-pthread", "-I", builder.CSRC, "-I", builder.INCLUDE, "-isystem", cuda, src,
                        os.path.join(builder.BUILD, "wq4_block_mm.o"), "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return out


@pytest.mark.parametrize("what,launches", [("devices", 25), ("occupancy", 3), ("failure", 1), ("threads", 2000)])
def test_every_device(exe, what, launches):
    r = subprocess.run([exe, what], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "launches %d refused 0\n" % launches, r.stdout + r.stderr
