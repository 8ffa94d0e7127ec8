/*
 * Host-side driver for the address-sanitized build of the ABI layer, the norm's
 * and the 4-bit and 8-bit products' part (tests/test_abi_asan_norm_4bit.py; the
 * rest: tests/abi_asan_driver.c). Every call is answered by the checks before
 * any HIP launch.
 */
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
  uint8_t* xs = (uint8_t*)base + 0xc0000;
  float* part = (float*)(base + 0xe0000);
  const int OK = ENGRAM_OK, INV = ENGRAM_EINVAL, UNS = ENGRAM_EUNSUPPORTED;
  const int F4 = ENGRAM_W_MXFP4, F8 = ENGRAM_W_MXFP8;
  const uint8_t* sc = (const uint8_t*)s;

  /* products: K 256, N 64, 4 tokens */
  expect(engram_wkv(NULL, 0, 256, NULL, NULL, F4, 64, NULL, NULL, 0, NULL), OK, "w4 T=0");
  expect(engram_wkv(x, 4, 256, w, NULL, F4, 64, kv, NULL, 0, NULL), INV, "w4 NULL scales");
  expect(engram_wkv(x, 4, 256, w, sc + 4, F4, 64, kv, NULL, 0, NULL), INV, "w4 misaligned scales");
  expect(engram_wkv(x, 4, 192, w, sc, F4, 64, kv, NULL, 0, NULL), UNS, "w4 K%128");
  expect(engram_wkv(x, 4, 256, w, sc, F4, 66, kv, NULL, 0, NULL), UNS, "w4 N%4");
  expect(engram_wkv(x, 4, 256, w, sc, F4, (1 << 28) + 4, kv, NULL, 0, NULL), UNS, "w4 N too large");
  expect(engram_wkv(x, INT64_MAX, 1 << 20, w, sc, F4, 1 << 28, kv, NULL, 0, NULL), UNS, "w4 T too large");
  expect(engram_wkv(x, 4, 256, w, sc, F4, 64, x, NULL, 0, NULL), INV, "w4 kv on x");
  expect(engram_wkv(x, 4, 256, w, sc, F4, 64, w + 8176, NULL, 0, NULL), INV, "w4 kv on w");
  for (int f = F8; f <= F4; ++f) {
    expect(engram_wkv_mx(NULL, NULL, 0, 256, NULL, NULL, f, 64, NULL, NULL), OK, "mx T=0");
    expect(engram_wkv_mx((uint8_t*)x, NULL, 4, 256, w, sc, f, 64, kv, NULL), INV, "mx NULL x scales");
    expect(engram_wkv_mx((uint8_t*)x, xs + 8, 4, 256, w, sc, f, 64, kv, NULL), INV, "mx misaligned x scales");
    expect(engram_wkv_mx((uint8_t*)x, xs, 4, 256, w, NULL, f, 64, kv, NULL), INV, "mx NULL scales");
    expect(engram_wkv_mx((uint8_t*)x, xs, -1, 256, w, sc, f, 64, kv, NULL), INV, "mx T<0");
    expect(engram_wkv_mx((uint8_t*)x, xs, 4, 200, w, sc, f, 64, kv, NULL), UNS, "mx K%128");
    expect(engram_wkv_mx((uint8_t*)x, xs, INT64_MAX, 1 << 20, w, sc, f, 64, kv, NULL), UNS, "mx T too large");
    expect(engram_wkv_mx((uint8_t*)x, xs, 4, 256, w, sc, f, 64, xs, NULL), INV, "mx kv on x scales");
  }
  expect(engram_wkv_mx((uint8_t*)x, xs, 4, 256, w, NULL, ENGRAM_W_BF16, 64, kv, NULL), UNS, "mx bf16 weights");
  expect(engram_wkv_mx((uint8_t*)x, xs, 4, 256, w, sc, 9, 64, kv, NULL), INV, "mx unknown format");

  /* gate partials on MXFP4: hc 2, dim 256 */
  expect(engram_wkv_gate_partials(NULL, 0, 256, NULL, NULL, F4, 2, 256, NULL, NULL, NULL, NULL, NULL, NULL, 0, NULL), OK,
         "partials T=0");
  expect(engram_wkv_gate_partials(x, 4, 256, w, sc, F4, 2, 256, h, h + 8192, h + 16384, x, part, NULL, 0, NULL), INV,
         "value on x");
  expect(engram_wkv_gate_partials(x, 4, 256, w, sc, F4, 2, 256, h, h + 8192, h + 16384, kv, (float*)h, NULL, 0, NULL), INV,
         "partials on hidden");
  expect(engram_wkv_gate_partials(x, 4, 256, w, sc, F4, 2, 256, h, h + 8192, h + 16384, kv, (float*)kv, NULL, 0, NULL), INV,
         "partials on value");
  expect(engram_wkv_gate_partials(x, 4, 256, w, NULL, F4, 2, 256, h, h, h, kv, part, NULL, 0, NULL), INV,
         "partials NULL scales");

  /* norm: 4 tokens of 2 rows of 64 */
#define NORM(X, XT, XH, R, RT, RH, W, WH, T, HC, DIM, EPS, RO, O, Q, S) \
  engram_add_rms_norm(X, XT, XH, R, RT, RH, W, WH, T, HC, DIM, EPS, RO, O, (uint8_t*)(Q), (uint8_t*)(S), NULL)
  expect(NORM(NULL, 0, 0, NULL, 0, 0, NULL, 1, 0, 2, 64, 1e-6f, NULL, NULL, NULL, NULL), OK, "norm T=0");
  expect(NORM(NULL, 128, 64, NULL, 0, 0, NULL, 1, 4, 2, 64, 1e-6f, NULL, kv, NULL, NULL), INV, "norm NULL x");
  expect(NORM(x, 128, 64, NULL, 0, 0, NULL, 1, 4, 2, 64, 1e-6f, NULL, NULL, NULL, NULL), INV, "norm no output");
  expect(NORM(x, 128, 64, NULL, 0, 0, NULL, 1, 4, 2, 64, 1e-6f, NULL, kv, h, NULL), INV, "norm codes without scales");
  expect(NORM(x, 128, 64, NULL, 0, 0, NULL, 3, 4, 2, 64, 1e-6f, NULL, x + 64, NULL, NULL), INV, "norm out inside x");
  expect(NORM(x, 128, 64, NULL, 0, 0, s, 3, 4, 2, 64, 1e-6f, NULL, kv, NULL, NULL), INV, "norm weight rows");
  expect(NORM(x, -8, 64, NULL, 0, 0, NULL, 1, 4, 2, 64, 1e-6f, NULL, kv, NULL, NULL), INV, "norm stride < 0");
  expect(NORM(x, 128, 64, NULL, 0, 0, NULL, 1, 4, 2, 64, -1.f, NULL, kv, NULL, NULL), INV, "norm eps < 0");
  expect(NORM(x, 128, 64, NULL, 0, 0, NULL, 1, INT64_MAX, 2, 64, 1e-6f, NULL, kv, NULL, NULL), UNS, "norm too many rows");
  expect(NORM(x, 128, 64, NULL, 0, 0, NULL, 1, 4, 2, 72, 1e-6f, NULL, kv, h, xs), UNS, "norm dim%32");
  expect(NORM(x, 128, 64, w, 128, 64, NULL, 1, 4, 2, 64, 1e-6f, x, kv, NULL, NULL), INV, "norm residual_out on x");

  /* forward */
  engram_forward_args a;
  memset(&a, 0, sizeof(a));
  a.table = x; a.num_rows = 10; a.hash_ids = (int32_t*)h; a.ids_stride_t = 4; a.ids_stride_c = 1;
  a.w = w; a.w_scales = NULL; a.w_format = F4;
  a.hidden = h; a.q_weight = s; a.k_weight = s; a.out = kv;
  a.T = 4; a.hc = 2; a.dim = 64; a.n_cols = 4; a.head_dim = 64; a.eps = a.clamp = 1e-6f;
  const size_t ws = engram_forward_workspace_size(&a);
  expect(engram_forward(&a, base, ws, NULL), INV, "forward NULL scales");
  a.w_scales = sc + 4;
  expect(engram_forward(&a, base, ws, NULL), INV, "forward misaligned scales");
  a.w_scales = sc;
  expect(engram_forward(&a, base, ws - 1, NULL), INV, "forward short workspace");
  a.n_cols = 3;
  expect(engram_forward(&a, base, ws, NULL), UNS, "forward K%128");
  a.n_cols = 4;
  expect(engram_forward_single_launch(&a, base, ws, NULL), UNS, "single launch");

  free(base);
  printf("norm and 4-bit abi checks under ASan: %d checks, %d failures\n", g_checks, g_fail);
  return g_fail ? 1 : 0;
}
