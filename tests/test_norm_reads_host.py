"""What the group norm's kernels read (no GPU): the kernels of csrc/group_norm.h are compiled for
the CPU and run thread after thread on tensors whose rows behind the lengths lie on pages that
cannot be read, so that a read of one ends the program.  Lanes and barriers play no part in what
is read: exchanges between lanes give a lane its own value."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "convolution_forward_implicit_amd", "csrc")
CLANG = os.environ.get("CLANGXX", "/opt/rocm/llvm/bin/clang++")

RUNTIME = r"""
#pragma once
#include <math.h>
#include <stdint.h>
#define __device__
#define __global__
#define __shared__ static
#define __launch_bounds__(...)
#define __forceinline__ inline __attribute__((always_inline))
#define __builtin_amdgcn_exp2f exp2f
#define __builtin_amdgcn_rcpf(v) (1.0f / (v))
struct At { unsigned x; };
inline At threadIdx, blockIdx;
inline void __syncthreads() {}
template <typename T> T __shfl_xor(T v, int) { return v; }
template <typename T> T min(T a, T b) { return a < b ? a : b; }
"""

DRIVER = r"""
#include <signal.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <sys/mman.h>
#include <unistd.h>
#include <type_traits>
#include "group_norm.h"
using namespace convfwd;

constexpr int N = 3, L = 5, W = 1024, PAGE = W * 4;       // a row is a page
static const int32_t lengths[N] = {0, 3, 5};
static char doing[64];

static float *rows(bool hidden)
{
    float *p = (float *)mmap(nullptr, (size_t)N * L * PAGE, PROT_READ | PROT_WRITE, MAP_PRIVATE | MAP_ANONYMOUS, -1, 0);
    for (int i = 0; i < N * L * W; ++i) p[i] = (float)(i % 97) - 48.0f;
    for (int r = 0; hidden && r < N * L; ++r)
        if (r % L >= lengths[r / L]) mprotect((char *)p + (size_t)r * PAGE, PAGE, PROT_NONE);
    return p;
}
static void caught(int)
{
    (void)!write(2, doing, strlen(doing));
    _exit(3);
}
template <typename F> void run(const char *what, int64_t blocks, F kernel)
{
    snprintf(doing, sizeof(doing), "%s read a row behind a length\n", what);
    for (blockIdx.x = 0; blockIdx.x < blocks; ++blockIdx.x)
        for (threadIdx.x = 0; threadIdx.x < 256; ++threadIdx.x) kernel();
}
static int zeros(const char *what, const float *y)
{
    for (int r = 0; r < N * L; ++r)
        for (int i = 0; i < W && r % L >= lengths[r / L]; ++i)
            if (y[r * W + i] != 0.0f) return printf("%s left row %d as it was\n", what, r), 1;
    return 0;
}

int main(int argc, char **argv)
{
    const int G = atoi(argv[1]);
    const bool tokens = atoi(argv[2]) != 0;             // a token is a sample
    if (sysconf(_SC_PAGESIZE) != PAGE) return 77;
    signal(SIGSEGV, caught);
    signal(SIGBUS, caught);
    static float w[W], ones[N * L * W * 2], sums[N * L * W * 2 * 2], group[N * L * W * 2];
    for (float &v : w) v = 1.0f;
    for (float &v : ones) v = 1.0f;
    NormParams p{};
    p.x = rows(true), p.gate = rows(true), p.dy = rows(true), p.w = w, p.bias = w, p.lengths = lengths;
    float *y = rows(false), *dx = rows(false), *dz = rows(false);
    p.y = y, p.dx = dx, p.dgate = dz;
    p.x_ld = p.gate_ld = p.y_ld = p.dy_ld = p.dx_ld = p.dgate_ld = W;
    p.samples = tokens ? N * L : N, p.rows = tokens ? 1 : L, p.L = L, p.tokens = N * L;
    p.G = G, p.C = W / G, p.act = NORM_SILU, p.center = 1, p.eps = 1e-5f;
    p.stats = ones, p.moments = ones, p.pulls = ones, p.sums = sums, p.group = group;
    int bad = 0;
    for (int slab = 1; slab <= p.rows; ++slab) {
        p.slab = slab, p.slabs = (p.rows + slab - 1) / slab;
        auto form = [&](auto v) {
            constexpr int V = decltype(v)::value;
            p.groups = p.C / V >= 256 ? 1 : 256 / (p.C / V);
            if (p.groups > G) p.groups = G;
            p.blocks = (G + p.groups - 1) / p.groups;
            const int64_t grid = p.samples * p.slabs * p.blocks;
            run("stats", grid, [&] { gnorm_stats_kernel<float, V>(p); });
            run("apply", grid, [&] { gnorm_apply_kernel<float, V>(p); });
            run("sums", grid, [&] { gnorm_sums_kernel<float, V>(p); });
            run("gradient", grid, [&] { gnorm_grad_kernel<float, V>(p); });
            bad += zeros("apply", y) + zeros("gradient", dx) + zeros("gradient of the gate", dz);
        };
        form(std::integral_constant<int, 4>()), form(std::integral_constant<int, 1>());
    }
    if (G >= 4) {                                       // a token's group in registers
        p.lanes = 64, p.groups = 4, p.blocks = G / 4, p.slab = 2;
        const int64_t grid = (p.tokens + 1) / 2 * p.blocks;
        run("tokens", grid, [&] { gnorm_token_kernel<float, 4, 1>(p); });
        run("tokens' gradient", grid, [&] { gnorm_token_grad_kernel<float, 4, 1>(p); });
        bad += zeros("tokens", y) + zeros("tokens' gradient", dx) + zeros("tokens' gradient of the gate", dz);
    }
    return bad != 0;
}
"""


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    if not os.path.exists(CLANG):
        pytest.skip("clang++ not found")
    d = tmp_path_factory.mktemp("reads")
    (d / "hip").mkdir()
    (d / "hip" / "hip_runtime.h").write_text(RUNTIME)
    (d / "driver.cpp").write_text(DRIVER)
    exe = str(d / "driver")
    r = subprocess.run([CLANG, "-std=c++17", "-O1", "-I" + str(d), "-I" + CSRC, str(d / "driver.cpp"), "-o", exe],
                       stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-3000:]
    return exe


# groups of 1024, 256 and 16 channels: rows wider than a workgroup's threads and narrower
@pytest.mark.parametrize("tokens", [0, 1], ids=["samples", "tokens"])
@pytest.mark.parametrize("groups", [1, 4, 64])
def test_rows_behind_a_length_are_not_read(driver, groups, tokens):
    r = subprocess.run([driver, str(groups), str(tokens)], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=120)
    if r.returncode == 77:
        pytest.skip("pages are not 4096 bytes")
    assert r.returncode == 0, r.stdout
