"""Host-side checks of the grouped products, the MXFP4 pack and the norm (CPU):
each call refuses what its header text excludes, with the documented status, before
anything is launched; sizes at the ends of int64_t under AddressSanitizer and
UndefinedBehaviorSanitizer."""

import ctypes
import os
import subprocess

import pytest
import torch

from test_abi_sanitize import _toolchain

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from moe_token_block_amd import build as b
    if not os.path.exists(b.LIB):
        b.build()
    import moe_token_block_amd as m
    return m.lib()


@pytest.mark.skipif(torch.cuda.is_available(), reason="passes fake pointers: only where no GPU exists")
def test_validation_before_launch(lib):
    P, N = ctypes.c_void_p(0x1000), None  # never dereferenced: every call below fails validation or does nothing
    for f in (lib.ep_bf16_grouped_gemm, lib.ep_bf16_grouped_dgrad):
        assert f(P, -1, 8, P, 2, 8, P, P, 4, P, N) == -2
        assert f(P, 32, 0, P, 2, 8, P, P, 4, P, N) == -2
        assert f(P, 32, 8, P, 0, 8, P, P, 4, P, N) == -2
        assert f(P, 32, 8, P, 1025, 8, P, P, 4, P, N) == -2
        assert f(P, 32, 8, P, 2, 0, P, P, 4, P, N) == -2
        assert f(P, 32, 8, P, 2, 8, N, P, 4, P, N) == -2      # counts and offsets come together
        assert f(P, 32, 8, P, 2, 8, P, N, 4, P, N) == -2
        assert f(P, 32, 8, P, 2, 8, N, N, 4, P, N) == -2      # one matrix: one expert
        assert f(P, 32, 8, P, 2, 8, P, P, -1, P, N) == -2
        assert f(P, 1 << 25, 8, P, 2, 8, P, P, 4, P, N) == -8
        assert f(P, 32, (1 << 20) + 1, P, 2, 8, P, P, 4, P, N) == -8
        assert f(P, 32, 8, P, 2, (1 << 20) + 1, P, P, 4, P, N) == -8
        assert f(N, 32, 8, P, 2, 8, P, P, 4, P, N) == -1
        assert f(P, 32, 8, N, 2, 8, P, P, 4, P, N) == -1
        assert f(P, 32, 8, P, 2, 8, P, P, 4, N, N) == -1
        assert f(N, 0, 8, P, 2, 8, P, P, 0, N, N) == 0
    w = lib.ep_bf16_grouped_wgrad
    assert w(P, P, -1, 8, 8, 2, P, P, 4, P, 0, N, 0, N) == -2
    assert w(P, P, 32, 0, 8, 2, P, P, 4, P, 0, N, 0, N) == -2
    assert w(P, P, 32, 8, 8, 2, P, N, 4, P, 0, N, 0, N) == -2
    assert w(P, P, 1 << 25, 8, 8, 2, P, P, 4, P, 0, N, 0, N) == -8
    assert w(N, P, 32, 8, 8, 2, P, P, 4, P, 0, N, 0, N) == -1
    assert w(P, N, 32, 8, 8, 2, P, P, 4, P, 0, N, 0, N) == -1
    assert w(P, P, 32, 8, 8, 2, P, P, 4, N, 0, N, 0, N) == -1
    p = lib.ep_mxfp4_pack
    assert p(P, -1, 64, P, P, N) == -2
    assert p(P, 4, 48, P, P, N) == -2
    assert p(P, 4, 0, P, P, N) == -2
    assert p(P, 1 << 40, 64, P, P, N) == -8
    assert p(P, 4, 64, P, N, N) == -1
    assert p(N, 0, 64, N, N, N) == 0
    assert lib.ep_mxfp4_unpack(P, P, 4, 33, P, N) == -2
    assert lib.ep_mxfp4_unpack(P, N, 4, 64, P, N) == -1
    assert lib.ep_mxfp4_unpack(N, N, 0, 64, N, N) == 0
    g = lib.ep_mxfp4_grouped_gemm
    assert g(P, P, 0, -1, 64, P, P, 2, 8, P, P, 4, P, N) == -2
    assert g(P, P, 0, 32, 48, P, P, 2, 8, P, P, 4, P, N) == -2
    assert g(P, P, 0, 32, 0, P, P, 2, 8, P, P, 4, P, N) == -2
    assert g(P, P, 0, 32, 64, P, P, 2, 8, N, P, 4, P, N) == -2
    assert g(P, P, 2, 32, 64, P, P, 2, 8, P, P, 4, P, N) == -5
    assert g(P, P, 0, 1 << 25, 64, P, P, 2, 8, P, P, 4, P, N) == -8
    assert g(P, N, 0, 32, 64, P, P, 2, 8, P, P, 4, P, N) == -1
    assert g(P, P, 1, 32, 64, P, N, 2, 8, P, P, 4, P, N) == -1
    assert g(N, N, 0, 0, 64, P, P, 2, 8, P, P, 0, N, N) == 0
    n = lib.rmsnorm_mxfp8
    assert n(P, P, P, 4, 48, 1e-6, P, P, P, P, N) == -2
    assert n(P, P, P, -1, 64, 1e-6, P, P, P, P, N) == -2
    assert n(P, P, P, 4, 16416, 1e-6, P, P, P, P, N) == -2
    assert n(P, P, P, 4, 64, -1.0, P, P, P, P, N) == -2
    assert n(P, P, P, 4, 64, float("nan"), P, P, P, P, N) == -2
    assert n(P, P, P, 4, 64, 0.0, P, P, P, P, N) == -2
    assert n(P, P, P, 4, 64, float("inf"), P, P, P, P, N) == -2
    assert n(P, P, P, 1 << 30, 64, 1e-6, P, P, P, P, N) == -8
    assert n(P, P, P, 4, 64, 1e-6, N, P, P, P, N) == -1      # a residual needs h
    assert n(N, N, P, 4, 64, 1e-6, N, P, P, P, N) == -1
    assert n(N, N, N, 0, 64, 1e-6, N, N, N, N, N) == 0
    d = lib.drmsnorm
    ws = lib.drmsnorm_workspace_bytes(40, 64)
    assert ws > 0 and lib.drmsnorm_workspace_bytes(4, 64) == 0 and lib.drmsnorm_workspace_bytes(0, 64) == 0 and lib.drmsnorm_workspace_bytes(4, 33) == 0
    assert d(P, P, P, P, N, 4, 48, P, P, P, ws, N) == -2
    assert d(P, P, P, N, N, 4, 64, P, P, P, ws, N) == -1
    assert d(P, P, P, P, N, 4, 64, P, N, P, ws, N) == -1
    assert d(P, P, P, P, N, 40, 64, P, P, P, ws - 1, N) == -7
    assert d(P, P, P, P, N, 40, 64, P, P, N, ws, N) == -7
    assert d(P, P, P, P, N, 40, 64, P, P, ctypes.c_void_p(0x1004), ws, N) == -7


@pytest.mark.skipif(torch.cuda.is_available(), reason="passes fake pointers: only where no GPU exists")
def test_grids_that_do_not_fit(lib):
    """Sizes within every other limit whose output tiles would need 2^32 threads."""
    P, N, wide, e = ctypes.c_void_p(0x1000), None, 1 << 20, 1024
    assert lib.ep_bf16_grouped_dgrad(P, 32, 1, P, e, wide, P, P, 32, P, N) == -8
    assert lib.ep_bf16_grouped_gemm(P, 192 * e, 32, P, e, wide, P, P, 192 * e, P, N) == -8
    assert lib.ep_bf16_grouped_wgrad(P, P, 32, 257, wide, e, P, P, 32, P, 0, N, 0, N) == -8
    for fmt in (0, 1):
        assert lib.ep_mxfp4_grouped_gemm(P, P, fmt, 192 * e, 32, P, P, e, wide, P, P, 192 * e, P, N) == -8


@pytest.mark.skipif(torch.cuda.is_available(), reason="passes fake pointers: only where no GPU exists")
def test_rows_past_one_grid(lib):
    P, N = ctypes.c_void_p(0x1000), None
    assert lib.ep_mxfp4_pack(P, 1 << 29, 32, P, P, N) == -8
    assert lib.ep_mxfp4_unpack(P, P, 1 << 29, 32, P, N) == -8
    assert lib.rmsnorm_mxfp8(P, P, P, 1 << 23, 16384, 1e-6, P, P, P, P, N) == -8
    assert lib.drmsnorm(P, P, P, P, N, 1 << 23, 64, P, P, P, 1 << 40, N) == -8


def test_binding_refuses_cpu_tensors(lib):
    import moe_token_block_amd as m
    bf = torch.zeros((2, 64), dtype=torch.bfloat16)
    u8 = torch.zeros((2, 64), dtype=torch.uint8)
    for call in (lambda: m.ep_bf16_grouped_gemm(bf, bf), lambda: m.ep_bf16_grouped_dgrad(bf, bf),
                 lambda: m.ep_bf16_grouped_wgrad(bf, bf), lambda: m.ep_mxfp4_pack(bf), lambda: m.ep_mxfp4_unpack(u8, u8),
                 lambda: m.ep_mxfp4_grouped_gemm(u8, u8, u8, u8), lambda: m.rmsnorm_mxfp8(bf, bf[0]),
                 lambda: m.drmsnorm(bf, bf, bf[0], bf[:, 0])):
        with pytest.raises((ValueError, TypeError)):
            call()


DRIVER = r"""
#include <stdio.h>
#include "moe_token_block.h"
static int failures = 0;
#define REFUSED(expr) do { long long g_ = (long long)(expr); \
  if (g_ >= 0) { fprintf(stderr, "%s = %lld\n", #expr, g_); ++failures; } } while (0)
#define P ((void*)0x1000)
int main(void) {
  const int64_t big[] = {INT64_MAX, INT64_MAX & ~(int64_t)63, INT64_MIN, -1, (int64_t)1 << 62, (int64_t)1 << 32};
  for (int i = 0; i < 6; ++i) {
    const int64_t b = big[i];
    REFUSED(ep_bf16_grouped_gemm(P, b, 8, P, 2, 8, P, P, 4, P, 0));
    REFUSED(ep_bf16_grouped_gemm(P, 32, b, P, 2, 8, P, P, 4, P, 0));
    REFUSED(ep_bf16_grouped_gemm(P, 32, 8, P, b, 8, P, P, 4, P, 0));
    REFUSED(ep_bf16_grouped_gemm(P, 32, 8, P, 2, b, P, P, 4, P, 0));
    REFUSED(ep_bf16_grouped_dgrad(P, b, 8, P, 2, 8, P, P, 4, P, 0));
    REFUSED(ep_bf16_grouped_dgrad(P, 32, b, P, 2, 8, P, P, 4, P, 0));
    REFUSED(ep_bf16_grouped_dgrad(P, 32, 8, P, 2, b, P, P, 4, P, 0));
    REFUSED(ep_bf16_grouped_wgrad(P, P, b, 8, 8, 2, P, P, 4, P, 0, 0, 0, 0));
    REFUSED(ep_bf16_grouped_wgrad(P, P, 32, b, 8, 2, P, P, 4, P, 0, 0, 0, 0));
    REFUSED(ep_bf16_grouped_wgrad(P, P, 32, 8, b, 2, P, P, 4, P, 0, 0, 0, 0));
    REFUSED(ep_bf16_grouped_wgrad(P, P, 32, 8, 8, b, P, P, 4, P, 0, 0, 0, 0));
    if (ep_bf16_grouped_wgrad_workspace_bytes(b, b, b, b) != 0) ++failures;
    if (ep_bf16_grouped_wgrad_workspace_bytes(8, 8, 2, b) != 0) ++failures;
    REFUSED(ep_mxfp4_pack(P, 4, b, P, P, 0));
    REFUSED(ep_mxfp4_unpack(P, P, 4, b, P, 0));
    REFUSED(ep_mxfp4_grouped_gemm(P, P, 0, b, 64, P, P, 2, 8, P, P, 4, P, 0));
    REFUSED(ep_mxfp4_grouped_gemm(P, P, 0, 32, b, P, P, 2, 8, P, P, 4, P, 0));
    REFUSED(ep_mxfp4_grouped_gemm(P, P, 1, 32, 64, P, P, b, 8, P, P, 4, P, 0));
    REFUSED(ep_mxfp4_grouped_gemm(P, P, 1, 32, 64, P, P, 2, b, P, P, 4, P, 0));
    REFUSED(rmsnorm_mxfp8(P, P, P, b, 64, 1e-6f, P, P, P, P, 0));
    REFUSED(rmsnorm_mxfp8(P, P, P, 4, b, 1e-6f, P, P, P, P, 0));
    if (drmsnorm_workspace_bytes(b, 64) != 0 || drmsnorm_workspace_bytes(4, b) != 0) ++failures;
    REFUSED(drmsnorm(P, P, P, P, 0, b, 64, P, P, P, 1, 0));
    REFUSED(drmsnorm(P, P, P, P, 0, 4, b, P, P, P, 1, 0));
    if (b != (int64_t)1 << 32) {
      REFUSED(ep_mxfp4_pack(P, b, 64, P, P, 0));
      REFUSED(ep_mxfp4_unpack(P, P, b, 64, P, 0));
    }
    if (b < 0) {
      REFUSED(ep_bf16_grouped_gemm(P, 32, 8, P, 2, 8, P, P, b, P, 0));
      REFUSED(ep_bf16_grouped_wgrad(P, P, 32, 8, 8, 2, P, P, b, P, 0, 0, 0, 0));
      REFUSED(ep_mxfp4_grouped_gemm(P, P, 0, 32, 64, P, P, 2, 8, P, P, b, P, 0));
    }
  }
  if (failures) return 1;
  printf("all checks passed\n");
  return 0;
}
"""


def test_validation_under_sanitizers(tmp_path):
    tc = _toolchain()
    if tc is None:
        pytest.skip("hipcc or ROCm's clang++ not found")
    b, cc, cxx, rocm = tc
    flags = ["-O0", "-Xarch_host", "-O1", "-g", "-std=c++17", f"--offload-arch={b.ARCH}", "-fPIC",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-Wno-unused-command-line-argument",
             "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=all"]
    procs, objs = [], []
    for src in ("grouped.hip", "mxgemm.hip", "mxfp4.hip", "norm.hip"):
        objs.append(str(tmp_path / (src + ".o")))
        procs.append(subprocess.Popen([cc] + flags + ["-c", os.path.join(b.CSRC, src), "-o", objs[-1]],
                                      stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
    for p in procs:
        out, _ = p.communicate(timeout=900)
        assert p.returncode == 0, out[-4000:]
    driver = tmp_path / "driver.c"
    driver.write_text(DRIVER)
    exe = str(tmp_path / "driver")
    lib_dir = os.path.join(rocm, "lib")
    r = subprocess.run([cxx, "-I", os.path.join(ROOT, "include"), "-x", "c", str(driver), "-x", "none", "-g",
                        "-fsanitize=address,undefined", "-fno-sanitize-recover=all"] + objs +
                       ["-L" + lib_dir, "-lamdhip64", "-Wl,-rpath," + lib_dir, "-o", exe],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:halt_on_error=1", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=env)
    assert r.returncode == 0 and "all checks passed" in r.stdout, r.stdout + r.stderr
