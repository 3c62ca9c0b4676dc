"""Host-side checks of the expert layer's entry points (CPU): each refuses what
its header text excludes, with the documented status, before anything is
launched; sizes at the ends of int64_t under AddressSanitizer and
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
    P, N = ctypes.c_void_p(0x1000), None         # never dereferenced: every call below fails validation or does nothing
    assert lib.ep_bf16_dispatch(P, 4, 0, 2, 8, P, P, P, N) == -2
    assert lib.ep_bf16_dispatch(P, -1, 8, 2, 8, P, P, P, N) == -2
    assert lib.ep_bf16_dispatch(P, 4, 8, 0, 8, P, P, P, N) == -2
    assert lib.ep_bf16_dispatch(P, 4, 8, 2, 1 << 25, P, P, P, N) == -8
    assert lib.ep_bf16_dispatch(P, 1 << 23, 8, 2, 8, P, P, P, N) == -8
    assert lib.ep_bf16_dispatch(P, 4, (1 << 20) + 1, 2, 8, P, P, P, N) == -8
    assert lib.ep_bf16_dispatch(P, 4, 8, 2, 8, P, N, P, N) == -1
    assert lib.ep_bf16_dispatch(P, 4, 8, 2, 8, N, P, P, N) == -1
    assert lib.ep_bf16_dispatch(N, 4, 8, 2, 8, P, P, P, N) == -1
    assert lib.ep_bf16_dispatch(N, 0, 8, 2, 0, N, N, N, N) == 0
    assert lib.ep_bf16_combine(P, 8, 8, 4, 0, P, P, P, N) == -2
    assert lib.ep_bf16_combine(P, 8, 8, 4, 1025, P, P, P, N) == -8
    assert lib.ep_bf16_combine(P, 8, 8, 1 << 23, 2, P, P, P, N) == -8
    assert lib.ep_bf16_combine(P, 8, 8, 4, 2, N, P, P, N) == -1
    assert lib.ep_bf16_combine(N, 8, 8, 4, 2, P, P, P, N) == -1
    assert lib.ep_bf16_combine(N, 0, 8, 0, 2, N, N, N, N) == 0
    assert lib.ep_bf16_combine_bwd(P, P, 4, 8, 2, -1, P, P, P, P, P, N) == -2
    assert lib.ep_bf16_combine_bwd(P, P, 4, 8, 2, 8, P, P, N, P, P, N) == -1
    assert lib.ep_bf16_combine_bwd(P, P, 4, 8, 2, 8, P, N, P, P, P, N) == -1
    assert lib.ep_bf16_combine_bwd(P, P, 4, 8, 2, 8, P, P, P, P, N, N) == -1
    assert lib.ep_bf16_combine_bwd(N, N, 0, 8, 2, 0, N, N, N, N, N, N) == 0
    mv = lib.ep_nvfp4_expert_matvec
    assert mv(P, 4, 100, 0, P, 2, 8, P, 0, 2, 0, P, N, N) == -2          # hidden % 64
    assert mv(P, 4, 64, 0, P, 2, 9, P, 0, 2, 1, P, N, N) == -2           # odd width with swiglu
    assert mv(P, 4, 64, 0, P, 2, 8, N, 0, 1, 0, P, N, N) == -2           # dense, two experts
    assert mv(P, 4, 64, 0, P, 1, 8, N, 0, 2, 0, P, N, N) == -2           # dense, two slots
    assert mv(P, 4, 64, 0, P, 1025, 8, P, 0, 2, 0, P, N, N) == -2
    assert mv(P, 4, 64, 0, P, 2, 8, P, 3, 2, 0, P, N, N) == -5           # index dtype
    assert mv(P, 2049, 64, 0, P, 2, 8, P, 0, 2, 0, P, N, N) == -8        # more than 4096 entries
    assert mv(P, 4, 64, 0, P, 2, (1 << 24) + 1, P, 0, 2, 0, P, N, N) == -8
    assert mv(N, 4, 64, 0, P, 2, 8, P, 0, 2, 0, P, N, N) == -1
    assert mv(P, 4, 64, 0, P, 2, 8, P, 0, 2, 0, N, N, N) == -1
    assert mv(N, 0, 64, 0, N, 2, 8, P, 0, 2, 0, N, N, N) == 0
    assert lib.swiglu_mxfp8_checkpoint(P, 4, 48, P, P, P, N) == -2
    assert lib.swiglu_mxfp8_checkpoint(P, 4, 64, P, P, N, N) == -1
    assert lib.swiglu_mxfp8_checkpoint(P, 1 << 30, 64, P, P, P, N) == -8
    assert lib.swiglu_mxfp8_checkpoint(N, 0, 64, N, N, N, N) == 0
    assert lib.dswiglu_mxfp8_checkpoint(P, P, P, 4, 16, P, P, N) == -2
    assert lib.dswiglu_mxfp8_checkpoint(P, P, P, 4, 64, N, P, N) == -1
    assert lib.dswiglu_mxfp8_checkpoint(N, N, N, 0, 64, N, N, N) == 0
    assert lib.ep_mxfp8_unpack(P, P, 4, 33, P, N) == -2
    assert lib.ep_mxfp8_unpack(P, N, 4, 64, P, N) == -1
    assert lib.ep_mxfp8_unpack(P, P, 1 << 40, 64, P, N) == -8


def test_binding_refuses_cpu_tensors(lib):
    import moe_token_block_amd as m
    bf = torch.zeros((2, 64), dtype=torch.bfloat16)
    u8 = torch.zeros((2, 64), dtype=torch.uint8)
    plan = dict(r_cap=16, num_experts=1, counts=u8, offsets=u8, src_row=u8, dst_row=u8)
    for call in (lambda: m.ep_bf16_dispatch(bf, plan), lambda: m.ep_bf16_combine(bf, plan),
                 lambda: m.ep_bf16_combine_bwd(bf, bf, plan, bf), lambda: m.ep_nvfp4_expert_matvec(bf, u8),
                 lambda: m.swiglu_mxfp8_checkpoint(bf), lambda: m.dswiglu_mxfp8_checkpoint(u8, u8, bf),
                 lambda: m.ep_mxfp8_unpack(u8, u8)):
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
    REFUSED(ep_bf16_dispatch(P, b, 8, 2, 8, P, P, P, 0));
    REFUSED(ep_bf16_dispatch(P, 4, b, 2, 8, P, P, P, 0));
    REFUSED(ep_bf16_dispatch(P, 4, 8, b, 8, P, P, P, 0));
    REFUSED(ep_bf16_dispatch(P, 4, 8, 2, b, P, P, P, 0));
    REFUSED(ep_bf16_combine(P, b, 8, 4, 2, P, P, P, 0));
    REFUSED(ep_bf16_combine(P, 8, 8, b, 2, P, P, P, 0));
    REFUSED(ep_bf16_combine(P, 8, 8, 4, b, P, P, P, 0));
    REFUSED(ep_bf16_combine(P, 8, b, 4, 2, P, P, P, 0));
    REFUSED(ep_bf16_combine_bwd(P, P, b, 8, 2, 8, P, P, P, P, P, 0));
    REFUSED(ep_bf16_combine_bwd(P, P, 4, b, 2, 8, P, P, P, P, P, 0));
    REFUSED(ep_bf16_combine_bwd(P, P, 4, 8, b, 8, P, P, P, P, P, 0));
    REFUSED(ep_bf16_combine_bwd(P, P, 4, 8, 2, b, P, P, P, P, P, 0));
    REFUSED(ep_nvfp4_expert_matvec(P, b, 64, 0, P, 2, 8, P, 0, 2, 0, P, 0, 0));
    REFUSED(ep_nvfp4_expert_matvec(P, 4, b, 0, P, 2, 8, P, 0, 2, 0, P, 0, 0));
    REFUSED(ep_nvfp4_expert_matvec(P, 4, 64, 0, P, b, 8, P, 0, 2, 0, P, 0, 0));
    REFUSED(ep_nvfp4_expert_matvec(P, 4, 64, 0, P, 2, b, P, 0, 2, 0, P, 0, 0));
    REFUSED(ep_nvfp4_expert_matvec(P, 4, 64, 0, P, 2, 8, P, 0, b, 0, P, 0, 0));
    REFUSED(swiglu_mxfp8_checkpoint(P, b, 64, P, P, P, 0));
    REFUSED(swiglu_mxfp8_checkpoint(P, 4, b, P, P, P, 0));
    REFUSED(dswiglu_mxfp8_checkpoint(P, P, P, 4, b, P, P, 0));
    REFUSED(ep_mxfp8_unpack(P, P, 4, b, P, 0));
    if (b != (int64_t)1 << 32) {
      REFUSED(dswiglu_mxfp8_checkpoint(P, P, P, b, 64, P, P, 0));
      REFUSED(ep_mxfp8_unpack(P, P, b, 64, P, 0));
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
    for src in ("combine.hip", "matvec.hip", "swiglu.hip"):
        objs.append(str(tmp_path / (src + ".o")))
        procs.append(subprocess.Popen([cc] + flags + ["-c", os.path.join(b.CSRC, src), "-o", objs[-1]],
                                      stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
    for p in procs:
        out, _ = p.communicate(timeout=600)
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
