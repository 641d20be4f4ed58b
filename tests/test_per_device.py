"""What the library sets once per device, against a stand-in of the CUDA
runtime with several devices (no GPU; a host compiler)."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from speculative_decoding_markov_gb300 import build

MAIN = r"""
#include <cassert>
#include <cstdio>
#include <map>
#include <thread>
#include <utility>
#include <vector>
#include "per_device.h"

static thread_local int device = 0;
static int fail = 0, calls = 0, queries = 0;
static std::map<std::pair<int, const void*>, int> limits;
extern "C" {
cudaError_t cudaGetDevice(int* d) { return *d = device, device < 0 ? cudaErrorNoDevice : cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
    assert(a == cudaFuncAttributeMaxDynamicSharedMemorySize);
    ++calls;
    if (fail > 0) return --fail, cudaErrorMemoryAllocation;
    limits[{device, f}] = v;
    return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int d) {
    assert(a == cudaDevAttrMultiProcessorCount);
    ++queries;
    if (fail > 0) return --fail, cudaErrorInitializationError;
    *v = 100 + d;
    return cudaSuccess;
}
}
static void kernel(int) {}
static const void* key = reinterpret_cast<const void*>(kernel);

int main() {
    using namespace sdm;
    static SmemLimit limit;
    // raised once on each device
    for (int turn = 0; turn < 3; ++turn)
        for (device = 0; device < 3; ++device) assert(limit.raise(kernel, 1000) == cudaSuccess);
    assert(calls == 3);
    for (int d = 0; d < 3; ++d) assert((limits[{d, key}] == 1000));
    // raised further where more is wanted, and lowered nowhere
    device = 1;
    assert(limit.raise(kernel, 3000) == cudaSuccess && limit.raise(kernel, 2000) == cudaSuccess);
    assert((limits[{1, key}] == 3000) && (limits[{2, key}] == 1000) && calls == 4);
    // a failure is returned, and not kept
    device = 5, fail = 1;
    assert(limit.raise(kernel, 1000) == cudaErrorMemoryAllocation && limit.raise(kernel, 1000) == cudaSuccess);
    device = -1;
    assert(limit.raise(kernel, 1000) == cudaErrorNoDevice);
    device = kMaxDevices;   // beyond those that are remembered
    calls = 0;
    assert(limit.raise(kernel, 10) == cudaSuccess && limit.raise(kernel, 10) == cudaSuccess && calls == 2);
    // several threads, several sizes: the largest stays
    for (int round = 0; round < 50; ++round) {
        SmemLimit one;
        limits.clear();
        std::vector<std::thread> all;
        for (int t = 0; t < 8; ++t)
            all.emplace_back([&one, t] { device = 0; assert(one.raise(kernel, 1000 + 100 * (t ^ 5)) == cudaSuccess); });
        for (auto& t : all) t.join();
        assert((limits[{0, key}] == 1700));
    }
    // the SMs of each device, asked for once
    for (int turn = 0; turn < 3; ++turn)
        for (device = 0; device < 4; ++device) assert(sms_of_device() == 100 + device);
    assert(queries == 4);
    device = 6, fail = 1;
    assert(sms_of_device() == 148 && sms_of_device() == 106);
    device = -1;
    assert(sms_of_device() == 148);
    puts("ok");
}
"""


def test_limits_and_sms_are_each_devices_own(tmp_path):
    cc = shutil.which("g++") or shutil.which("c++")
    if cc is None:
        pytest.skip("no host compiler")
    include = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    (tmp_path / "main.cpp").write_text(MAIN)
    exe = str(tmp_path / "main")
    r = subprocess.run([cc, "-std=c++17", "-O1", "-pthread", "-I", include, "-I", build.CSRC, str(tmp_path / "main.cpp"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stderr
    for name in build.SOURCES:                                     # no launch keeps a flag of its own
        with open(os.path.join(build.CSRC, name)) as f:
            assert "cudaFuncSetAttribute" not in f.read(), name
