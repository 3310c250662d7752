// Says which kernels the launchers of the feed-forward block, the FP8 product and
// the orthogonalised update start for given sizes (no GPU): their host code is
// compiled as it is, and the runtime's entry points below take the launches down
// instead of making them.  Pointers handed in are never dereferenced.
//
// Reads lines "ffn M E H I", "ffn_backward M E H I", "fp8 M E N K" and
// "orthogonalize E N K steps" and answers each with "kernel<arguments> groups
// threads" for each launch, separated by semicolons.
#include <cxxabi.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <map>
#include <string>
#include <vector>

#include "ffn.h"
#include "fp8.h"
#include "ortho.h"

static std::map<const void*, std::string>& names() {
  static std::map<const void*, std::string> m;
  return m;
}
static dim3 groups, threads;

extern "C" {
void** __hipRegisterFatBinary(const void*) { return nullptr; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
void __hipRegisterFunction(void**, const void* f, char*, const char* name, unsigned, void*, void*, void*, void*, int*) {
  names()[f] = name;
}
hipError_t __hipPushCallConfiguration(dim3 g, dim3 t, size_t, hipStream_t) {
  groups = g;
  threads = t;
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* g, dim3* t, size_t* shared, hipStream_t* s) {
  *g = groups;
  *t = threads;
  *shared = 0;
  *s = nullptr;
  return hipSuccess;
}
hipError_t hipGetLastError(void) { return hipSuccess; }
hipError_t hipLaunchKernel(const void* f, dim3 g, dim3 t, void**, size_t, hipStream_t) {
  int status = 0;
  char* full = abi::__cxa_demangle(names()[f].c_str(), nullptr, nullptr, &status);
  std::string name = full ? full : names()[f];
  free(full);
  // "void moeq::(anonymous namespace)::kernel<arguments>(parameters)"
  const size_t scope = name.find("namespace)::");
  if (scope != std::string::npos) name = name.substr(scope + 12);
  int depth = 0;
  for (size_t i = 0; i < name.size(); ++i) {
    depth += name[i] == '<' ? 1 : name[i] == '>' ? -1 : 0;
    if (name[i] == '(' && depth == 0) name.resize(i);
  }
  printf("%s %llu %u;", name.c_str(), (unsigned long long)g.x * g.y * g.z, t.x * t.y * t.z);
  return hipSuccess;
}
}  // extern "C"

using namespace moeq;

int main() {
  char line[256], op[32];
  char* at = reinterpret_cast<char*>(uintptr_t(1) << 40);
  while (fgets(line, sizeof line, stdin)) {
    int a, b, c, d;
    if (sscanf(line, "%31s %d %d %d %d", op, &a, &b, &c, &d) != 5) return 2;
    hipError_t e;
    if (!strcmp(op, "ffn")) {
      e = launch_glu({at, at, nullptr, nullptr, nullptr, at, a, b, d, c}, nullptr, nullptr);
    } else if (!strcmp(op, "ffn_backward")) {
      e = launch_glu_backward({at, at, nullptr, nullptr, nullptr, at, a, b, d, c}, nullptr, nullptr, nullptr);
    } else if (!strcmp(op, "fp8")) {
      e = launch_grouped_mm_fp8({at, at, nullptr, nullptr, nullptr, at, a, b, c, d}, nullptr, nullptr, nullptr);
    } else if (!strcmp(op, "orthogonalize")) {
      const std::vector<float> table(3 * d, 1.0f);
      e = launch_orthogonalize(at, true, ortho_plan(a, b, c), table.data(), d, nullptr, at, nullptr);
    } else {
      return 2;
    }
    if (e != hipSuccess) return 3;
    printf("\n");
  }
  return 0;
}
