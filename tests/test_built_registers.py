"""The check of a kernel's registers in front of a launch that moves them between warps, with stand-ins for the runtime's
query and the library's error record (no GPU): a query that fails once is an error of that call and is asked again by the next."""
import subprocess

from mixture_experts_routing_token_gb300.build import ARCH, CSRC, INCLUDE, nvcc

SOURCE = r"""
#include <stdarg.h>
#include <stdio.h>
#include <string.h>
#include "common.cuh"

static char said[256];
static cudaError_t answer;
static int registers, asked;
namespace moe {
int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(said, sizeof(said), fmt, ap);
  va_end(ap);
  return code;
}
}  // namespace moe
extern "C" cudaError_t __wrap_cudaFuncGetAttributes(cudaFuncAttributes* at, const void*) {
  ++asked;
  memset(at, 0, sizeof(*at));
  at->numRegs = registers;
  return answer;
}
#define EXPECT(c) if (!(c)) { printf("line %d: %s (said: %s)\n", __LINE__, #c, said); return 1; }

int main() {
  const void* kernel = &answer;
  moe::BuiltRegisters a, b;
  answer = cudaErrorMemoryAllocation;
  registers = 0;
  EXPECT(a.check(kernel, 12, 2016, "product") == MOE_ERR_CUDA && asked == 1);
  EXPECT(strstr(said, "product") && strstr(said, cudaGetErrorString(cudaErrorMemoryAllocation)) && !strstr(said, "too few"));
  answer = cudaSuccess;
  registers = 168;
  EXPECT(a.check(kernel, 12, 2016, "product") == MOE_OK && asked == 2);
  EXPECT(a.check(kernel, 12, 2016, "product") == MOE_OK && asked == 2);
  registers = 167;
  EXPECT(b.check(kernel, 12, 2016, "product") == MOE_ERR_CUDA && strstr(said, "too few registers"));
  EXPECT(b.check(kernel, 12, 2016, "product") == MOE_ERR_CUDA && asked == 3);
  return 0;
}
"""


def test_a_failed_query_is_asked_again(tmp_path):
    src, exe = tmp_path / "registers.cu", tmp_path / "registers"
    src.write_text(SOURCE)
    made = subprocess.run([nvcc(), *ARCH, "-std=c++17", "-I", INCLUDE, "-I", CSRC, str(src), "-o", str(exe),
                           "-Xlinker", "--wrap=cudaFuncGetAttributes"], capture_output=True, text=True)
    assert made.returncode == 0, made.stderr
    ran = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert ran.returncode == 0, ran.stdout
