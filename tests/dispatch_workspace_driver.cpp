// tests/dispatch_driver.cpp with a workspace of the caller's choice for the int8
// projection from bf16 rows.
//
//   wkvat T K N P OFS BYTES    engram_wkv, int8 weights; the workspace at OFS bytes into
//                              tensor P (0 x, 2 w, 3 scales, 4 kv, 5 one of its own), of BYTES
//   fwdsize T HC DIM C HD F    engram_forward_workspace_size in KiB, rounded up
//   noalloc T HC DIM C HD F    engram_forward_noalloc
#define main other_main
#include "dispatch_driver.cpp"
#undef main

extern "C" hipError_t hipGetSymbolAddress(void** p, const void*) {
  *p = (void*)((uintptr_t)13 << 48);
  return hipSuccess;
}

int main() {
  uint8_t* at[12];
  for (int i = 0; i < 12; ++i) at[i] = (uint8_t*)((uintptr_t)(i + 1) << 48);
  std::string line;
  while (std::getline(std::cin, line)) {
    std::istringstream in(line);
    std::string op;
    long long v[6] = {0};
    in >> op;
    for (auto& a : v) in >> a;
    st().launches.clear();
    long long r = -1;
    if (op == "wkvat") {
      r = engram_wkv(at[0], v[0], (int)v[1], at[2], at[3], ENGRAM_W_INT8, (int)v[2], at[4], at[v[3]] + v[4], (size_t)v[5],
                     nullptr);
    } else {
      engram_forward_args a = {};
      a.table = at[6];
      a.num_rows = 1000;
      a.hash_ids = (const int32_t*)at[7];
      a.ids_stride_t = v[3];
      a.ids_stride_c = 1;
      a.w = at[2];
      a.w_scales = v[5] ? at[3] : nullptr;
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
      r = op == "fwdsize" ? (long long)((engram_forward_workspace_size(&a) + 1023) / 1024) : engram_forward_noalloc(&a, nullptr);
    }
    std::cout << "= " << r << ' ' << st().launches << std::endl;
  }
  return 0;
}
