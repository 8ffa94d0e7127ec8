// tests/dispatch_driver.cpp with the int8 entry points and the norms around a block.
//
//   i8 T K N            engram_wkv_int8
//   i8q T K             engram_int8_quantize
//   ppn T HC DIM Q      engram_post_pre_norm, Q: 0 bf16, 1 MXFP8, 2 int8
//   every other line of that driver's
#define main other_main
#include "dispatch_driver.cpp"
#undef main

int main() {
  uint8_t* at[12];
  for (int i = 0; i < 12; ++i) at[i] = (uint8_t*)((uintptr_t)(i + 1) << 48);
  std::string line;
  std::stringbuf one;
  while (std::getline(std::cin, line)) {
    std::istringstream in(line);
    std::string op;
    long long v[4] = {0};
    in >> op;
    for (auto& a : v) in >> a;
    if (op != "i8" && op != "i8q" && op != "ppn") {
      std::istringstream rest(line + "\n");
      std::streambuf* was = std::cin.rdbuf(rest.rdbuf());
      other_main();
      std::cin.rdbuf(was);
      std::cin.clear();
      continue;
    }
    st().launches.clear();
    int r;
    if (op == "i8") {
      r = engram_wkv_int8((int8_t*)at[0], (float*)at[1], v[0], (int)v[1], (int8_t*)at[2], (float*)at[3], (int)v[2], at[4], nullptr);
    } else if (op == "i8q") {
      r = engram_int8_quantize(at[0], v[0], (int)v[1], (int8_t*)at[1], (float*)at[2], nullptr);
    } else {
      engram_post_pre_norm_args a = {};
      a.x = at[0];
      a.x_stride_t = v[1] * v[2];
      a.x_stride_h = v[2];
      a.T = v[0];
      a.hc = (int)v[1];
      a.dim = (int)v[2];
      a.post_norm = 1;
      a.residual_out = at[1];
      a.out = at[2];
      a.q_format = (int)v[3];
      if (a.q_format) {
        a.xq = at[3];
        a.xs = at[4];
      }
      r = engram_post_pre_norm(&a, nullptr);
    }
    std::cout << "= " << r << ' ' << st().launches << std::endl;
  }
  return 0;
}
