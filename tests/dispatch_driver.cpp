// What libengram.so launches for a call, without a GPU: this program defines
// the HIP runtime calls that the library makes (they take precedence over the
// runtime's own), reads calls from stdin and prints every launch with its grid,
// block, dynamic LDS and the kernel's LDS limit at that moment.
//
//   cus N                              compute units from here on (256)
//   wkv T K N F | mx T K N F           F: 0 bf16, 1 MXFP8, 2 MXFP4
//   partials T K HC DIM F
//   forward T HC DIM C HD F OPTIONS
//   norm T HC DIM OUTPUTS              OUTPUTS: 1 bf16, 2 MXFP8, 3 both
//   kernels                            every kernel of the library
//
// Answers: "= STATUS NAME GRID_X GRID_Y GRID_Z BLOCK LDS LIMIT; NAME ...".
#include <cxxabi.h>
#include <stdint.h>

#include <cstdio>
#include <cstdlib>
#include <iostream>
#include <map>
#include <sstream>
#include <string>
#include <vector>

#include <hip/hip_runtime_api.h>

#include "../include/engram.h"

namespace {

struct State {
  std::map<const void*, std::string> names;
  std::map<const void*, int> limits;   // hipFuncSetAttribute
  std::string launches;
  dim3 grid, block;
  size_t lds = 0;
  hipStream_t stream = nullptr;
  int cus = 256;
};
State& st() {
  static State s;   // filled by the library's initializers, before main
  return s;
}

std::string plain_name(const char* mangled) {
  int status = 0;
  char* d = abi::__cxa_demangle(mangled, nullptr, nullptr, &status);
  std::string s = status == 0 && d ? d : mangled;
  free(d);
  const std::string head = "engram::(anonymous namespace)::";
  const size_t at = s.find(head);
  if (at != std::string::npos) s = s.substr(at + head.size());
  s = s.substr(0, s.find('('));
  for (size_t i; (i = s.find(", ")) != std::string::npos;) s.erase(i + 1, 1);
  for (char& c : s) c = c == ' ' ? '_' : c;
  return s;
}

}  // namespace

extern "C" {

void** __hipRegisterFatBinary(const void*) {
  static void* module = nullptr;
  return &module;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* fn, char*, const char* name, unsigned, void*, void*, dim3*, dim3*, int*) {
  st().names[fn] = plain_name(name);
}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t s) {
  st().grid = grid;
  st().block = block;
  st().lds = lds;
  st().stream = s;
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* s) {
  *grid = st().grid;
  *block = st().block;
  *lds = st().lds;
  *s = st().stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* fn, dim3 grid, dim3 block, void**, size_t lds, hipStream_t) {
  const auto lim = st().limits.find(fn);
  std::ostringstream o;
  o << st().names[fn] << ' ' << grid.x << ' ' << grid.y << ' ' << grid.z << ' ' << block.x << ' ' << lds << ' '
    << (lim == st().limits.end() ? 0 : lim->second) << ';';
  st().launches += o.str();
  return hipSuccess;
}
hipError_t hipFuncSetAttribute(const void* fn, hipFuncAttribute attr, int value) {
  if (attr == hipFuncAttributeMaxDynamicSharedMemorySize) st().limits[fn] = value;
  return hipSuccess;
}
hipError_t hipGetLastError(void) { return hipSuccess; }
hipError_t hipGetDevice(int* d) {
  *d = 0;
  return hipSuccess;
}
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) {
  *v = st().cus;
  return hipSuccess;
}

}  // extern "C"

int main() {
  // tensors far apart, never read
  uint8_t* at[12];
  for (int i = 0; i < 12; ++i) at[i] = (uint8_t*)((uintptr_t)(i + 1) << 48);
  void *x = at[0], *w = at[2], *kv = at[4], *ws = at[5];
  uint8_t *xs = at[1], *s = at[3];
  const size_t room = (size_t)1 << 60;
  std::string line;
  while (std::getline(std::cin, line)) {
    std::istringstream in(line);
    std::string op;
    in >> op;
    long long v[7] = {0};
    for (auto& a : v) in >> a;
    st().launches.clear();
    int r = -1;
    if (op == "cus") {
      st().cus = (int)v[0];
      r = 0;
    } else if (op == "kernels") {
      for (const auto& n : st().names) st().launches += n.second + ';';
      r = 0;
    } else if (op == "wkv") {
      r = engram_wkv(x, v[0], (int)v[1], w, v[3] ? s : nullptr, (int)v[3], (int)v[2], kv, ws, room, nullptr);
    } else if (op == "mx") {
      r = engram_wkv_mx((uint8_t*)x, xs, v[0], (int)v[1], w, s, (int)v[3], (int)v[2], kv, nullptr);
    } else if (op == "partials") {
      r = engram_wkv_gate_partials(x, v[0], (int)v[1], w, v[4] ? s : nullptr, (int)v[4], (int)v[2], (int)v[3], at[6],
                                   at[7], at[8], kv, (float*)at[9], ws, room, nullptr);
    } else if (op == "forward") {
      engram_forward_args a = {};
      a.table = at[6];
      a.num_rows = 1000;
      a.hash_ids = (const int32_t*)at[7];
      a.ids_stride_t = v[3];
      a.ids_stride_c = 1;
      a.w = w;
      a.w_scales = v[5] ? s : nullptr;
      a.w_format = (int)v[5];
      a.hidden = at[8];
      a.q_weight = at[9];
      a.k_weight = at[10];
      a.T = v[0];
      a.hc = (int)v[1];
      a.dim = (int)v[2];
      a.n_cols = (int)v[3];
      a.head_dim = (int)v[4];
      a.eps = a.clamp = 1e-6f;
      a.out = at[11];
      a.options = (int)v[6];
      r = engram_forward(&a, ws, room, nullptr);
    } else if (op == "norm") {
      const bool b = v[3] & 1, q = v[3] & 2;
      r = engram_add_rms_norm(x, v[1] * v[2], v[2], nullptr, 0, 0, nullptr, 1, v[0], (int)v[1], (int)v[2], 1e-6f,
                              nullptr, b ? kv : nullptr, q ? at[6] : nullptr, q ? at[7] : nullptr, nullptr);
    }
    std::cout << "= " << r << ' ' << st().launches << std::endl;
  }
  return 0;
}
