// tests/dispatch_driver.cpp with a workspace of the caller's choice for the int8
// projection from bf16 rows.
//
//   wkvat T K N P OFS BYTES    engram_wkv, int8 weights; the workspace at OFS bytes into
//                              tensor P (0 x, 2 w, 3 scales, 4 kv, 5 one of its own), of BYTES
#define main other_main
#include "dispatch_driver.cpp"
#undef main

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
    int r = -1;
    if (op == "wkvat")
      r = engram_wkv(at[0], v[0], (int)v[1], at[2], at[3], ENGRAM_W_INT8, (int)v[2], at[4], at[v[3]] + v[4], (size_t)v[5],
                     nullptr);
    std::cout << "= " << r << ' ' << st().launches << std::endl;
  }
  return 0;
}
