/*
 * Host-side driver for the address-sanitized build of the ABI layer, the int8
 * products' and the norms' around a block part (tests/test_abi_asan_int8.py). Every
 * call is answered by the checks before any HIP launch.
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "../include/engram.h"

static int g_fail = 0, g_checks = 0;

static void expect(int got, int want, const char* what) {
  ++g_checks;
  if (got != want) {
    printf("FAIL %s: got %d want %d\n", what, got, want);
    ++g_fail;
  }
}

int main(void) {
  char* base = (char*)aligned_alloc(256, 1 << 20);
  char *x = base, *w = base + 0x20000, *s = base + 0x60000, *kv = base + 0x80000, *h = base + 0xa0000;
  float *xs = (float*)(base + 0xc0000), *part = (float*)(base + 0xe0000), *ws = (float*)s;
  char* stage = base + 0xf0000;
  int8_t *q = (int8_t*)x, *wq = (int8_t*)w;
  const uint8_t* sc = (const uint8_t*)s;
  const int OK = ENGRAM_OK, INV = ENGRAM_EINVAL, UNS = ENGRAM_EUNSUPPORTED, I8 = ENGRAM_W_INT8;

  /* K 256, N 64 */
  expect(engram_int8_quantize(NULL, 0, 256, NULL, NULL, NULL), OK, "quantize T=0");
  expect(engram_int8_quantize(x, INT64_MAX, 256, (int8_t*)kv, xs, NULL), UNS, "quantize T too large");
  expect(engram_int8_quantize(x, 4, 264, (int8_t*)kv, xs, NULL), UNS, "quantize K%16");
  expect(engram_int8_quantize(x, 4, 256, q + 1024, xs, NULL), INV, "quantize onto x");
  expect(engram_wkv_int8(NULL, NULL, 0, 256, NULL, NULL, 64, NULL, NULL), OK, "i8 T=0");
  expect(engram_wkv_int8(q, NULL, 4, 256, wq, ws, 64, kv, NULL), INV, "i8 NULL x scales");
  expect(engram_wkv_int8(q, xs, 4, 256, wq, NULL, 64, kv, NULL), INV, "i8 NULL scales");
  expect(engram_wkv_int8(q, xs, 4, 256, wq, ws + 1, 64, kv, NULL), INV, "i8 misaligned scales");
  expect(engram_wkv_int8(q, xs, -1, 256, wq, ws, 64, kv, NULL), INV, "i8 T<0");
  expect(engram_wkv_int8(q, xs, 4, 1 << 17, wq, ws, 64, kv, NULL), UNS, "i8 K too large");
  expect(engram_wkv_int8(q, xs, INT64_MAX, 131056, wq, ws, 1 << 28, kv, NULL), UNS, "i8 T too large");
  expect(engram_wkv_int8(q, xs, 4, 256, wq, ws, 64, xs, NULL), INV, "i8 kv on x scales");
  expect(engram_wkv_int8(q, xs, 4, 256, wq, ws, 64, s, NULL), INV, "i8 kv on scales");
  expect(engram_wkv(x, 20, 256, w, sc, I8, 64, kv, NULL, 0, NULL), INV, "wkv i8 without its workspace");
  expect(engram_wkv(x, 20, 256, w, sc, I8, 64, kv, kv, 4096, NULL), INV, "wkv i8 workspace on kv");
  expect(engram_wkv(x, 20, 256, w, NULL, I8, 64, kv, stage, 4096, NULL), INV, "wkv i8 NULL scales");
  expect(engram_wkv(x, 4, 256, w, sc, I8, 64, x, NULL, 0, NULL), INV, "wkv i8 kv on x");
  expect(engram_wkv(NULL, 0, 256, NULL, NULL, I8, 64, NULL, NULL, 0, NULL), OK, "wkv i8 T=0");
  expect((int)engram_wkv_workspace_size(4, 256, 64, I8), 0, "no workspace for few tokens");
  expect(engram_wkv_workspace_size(INT64_MAX, 131056, 64, I8) != 1, 1, "any T has a size");

  /* gate partials: hc 2, dim 256 */
  const size_t need = engram_wkv_gate_partials_workspace_size(4, 256, 2, 256, I8);
  expect(engram_wkv_gate_partials(x, 4, 256, w, sc, I8, 2, 256, h, h + 8192, h + 16384, kv, part, stage, need - 1, NULL), INV,
         "partials short workspace");
  expect(engram_wkv_gate_partials(x, 4, 256, w, sc, I8, 2, 256, h, h + 8192, h + 16384, kv, part, part, need, NULL), INV,
         "partials on the workspace");
  expect(engram_wkv_gate_partials(x, 4, 256, w, sc, I8, 2, 256, h, h + 8192, h + 16384, x, part, stage, need, NULL), INV,
         "value on x");

  /* norms: 4 tokens of 2 rows of 64 */
  engram_post_pre_norm_args n;
  memset(&n, 0, sizeof(n));
  expect(engram_post_pre_norm(NULL, NULL), INV, "norms NULL");
  expect(engram_post_pre_norm(&n, NULL), INV, "norms zeroed");
  n.x = x; n.x_stride_t = 128; n.x_stride_h = 64;
  n.residual = w; n.residual_stride_t = 128; n.residual_stride_h = 64;
  n.gate = h; n.gate_stride_t = 128; n.gate_stride_h = 64; n.gate_format = ENGRAM_GATE_CHANNEL;
  n.post_weight = s; n.pre_weight = s; n.post_weight_hc = 1; n.pre_weight_hc = 2;
  n.T = 4; n.hc = 2; n.dim = 64; n.post_norm = 1; n.post_eps = n.eps = 1e-6f;
  n.residual_scale = n.branch_scale = 1.f;
  n.residual_out = w;   /* in place */
  n.q_format = ENGRAM_Q_INT8; n.xq = (uint8_t*)kv; n.xs = xs;
  engram_post_pre_norm_args a = n;
#define TRY(change, want, what) a = n; change; expect(engram_post_pre_norm(&a, NULL), want, what)
  TRY(a.T = 0, OK, "norms T=0");
  TRY(a.T = INT64_MAX, UNS, "norms too many rows");
  TRY(a.T = 1 << 30, UNS, "norms rows past 2^31");
  TRY(a.dim = 72 - 4, UNS, "norms dim%8");
  TRY((a.dim = 40, a.q_format = ENGRAM_Q_MXFP8), UNS, "norms dim%32");
  TRY(a.post_eps = -1.f, INV, "norms post eps");
  TRY(a.eps = NAN, INV, "norms eps NaN");
  TRY(a.gate_format = 7, INV, "norms gate format");
  TRY(a.gate = NULL, INV, "norms gate missing");
  TRY(a.xs = NULL, INV, "norms codes without scales");
  TRY(a.xq = (uint8_t*)x, INV, "norms codes on x");
  TRY(a.xs = h + 512, INV, "norms scales on the gate");
  TRY(a.residual_out = x, INV, "norms stream on x");
  TRY(a.out = x + 64, INV, "norms out inside x");
  TRY((a.residual_out = w, a.residual_stride_t = 192), INV, "norms in place on strided rows");
  TRY(a.x_stride_t = INT64_MAX / 4 * 4, UNS, "norms stride%8");

  /* forward */
  engram_forward_args f;
  memset(&f, 0, sizeof(f));
  f.table = x; f.num_rows = 10; f.hash_ids = (int32_t*)h; f.ids_stride_t = 4; f.ids_stride_c = 1;
  f.w = w; f.w_scales = NULL; f.w_format = I8;
  f.hidden = h; f.q_weight = s; f.k_weight = s; f.out = kv;
  f.T = 4; f.hc = 2; f.dim = 64; f.n_cols = 4; f.head_dim = 64; f.eps = f.clamp = 1e-6f;
  const size_t fw = engram_forward_workspace_size(&f);
  expect(engram_forward(&f, base, fw, NULL), INV, "forward NULL scales");
  f.w_scales = sc;
  expect(engram_forward(&f, base, fw - 1, NULL), INV, "forward short workspace");
  expect(engram_forward_single_launch(&f, base, fw, NULL), UNS, "single launch");
  f.n_cols = 1; f.head_dim = 8;
  expect(engram_forward(&f, base, fw, NULL), UNS, "forward K%16");

  free(base);
  printf("int8 and norms abi checks under ASan: %d checks, %d failures\n", g_checks, g_fail);
  return g_fail ? 1 : 0;
}
