// Calls every host-side check of the router and the 8-bit operators on valid
// and invalid arguments; built with sanitizers by tests/test_layer8_sanitizers.py.
#include <climits>
#include <cmath>
#include <cstdio>
#include <cstdlib>

#include "validate_layer8.hpp"

using namespace mc2;

static int failures = 0;
static void expect(mc2_status got, mc2_status want, const char* what) {
  if (got != want) {
    std::printf("%s: got %d, want %d (%s)\n", what, (int)got, (int)want, last_error_text());
    failures++;
  }
  clear_error();
}

int main() {
  void* a = reinterpret_cast<void*>(0x1000);
  void* odd = reinterpret_cast<void*>(0x1002);
  const int64_t big = INT64_MAX;
  const mc2_score soft = MC2_SCORE_SOFTMAX;

  expect(check_moe_route(a, a, 4, 64, 4, MC2_F32, soft, 1, 1, 1, 1.f, a, a), MC2_OK, "route");
  expect(check_moe_route(a, nullptr, 4, 256, 8, MC2_BF16, MC2_SCORE_SIGMOID, 8, 4, 2, 1.f, a, a), MC2_OK, "groups");
  expect(check_moe_route(a, a, big, 64, 4, MC2_F32, soft, 1, 1, 1, 1.f, a, a), MC2_ERR_SHAPE, "tokens");
  expect(check_moe_route(a, a, 4, big, 4, MC2_F32, soft, 1, 1, 1, 1.f, a, a), MC2_ERR_SHAPE, "experts");
  expect(check_moe_route(a, a, 4, 64, big, MC2_F32, soft, 1, 1, 1, 1.f, a, a), MC2_ERR_SHAPE, "top");
  expect(check_moe_route(a, a, 4, 64, 4, MC2_F32, soft, big, 1, 1, 1.f, a, a), MC2_ERR_SHAPE, "groups big");
  expect(check_moe_route(a, a, 4, 64, 4, MC2_F32, soft, 0, 1, 1, 1.f, a, a), MC2_ERR_SHAPE, "no groups");
  expect(check_moe_route(a, a, 4, 64, 4, MC2_F32, soft, 8, big, 1, 1.f, a, a), MC2_ERR_SHAPE, "top_groups");
  expect(check_moe_route(a, a, 4, 64, 4, MC2_F32, soft, 8, 2, big, 1.f, a, a), MC2_ERR_SHAPE, "group_top");
  expect(check_moe_route(a, a, 4, 64, 4, MC2_F32, soft, 1, 1, 1, NAN, a, a), MC2_ERR_SHAPE, "scale");
  expect(check_moe_route(a, a, 4, 64, 4, MC2_I8, soft, 1, 1, 1, 1.f, a, a), MC2_ERR_DTYPE, "dtype");
  expect(check_moe_route(a, a, 4, 64, 4, MC2_F32, (mc2_score)2, 1, 1, 1, 1.f, a, a), MC2_ERR_UNSUPPORTED, "score");
  expect(check_moe_route(nullptr, nullptr, 0, 64, 4, MC2_F32, soft, 1, 1, 1, 1.f, nullptr, nullptr), MC2_OK, "no tokens");
  expect(check_moe_route(odd, a, 4, 64, 4, MC2_F32, soft, 1, 1, 1, 1.f, a, a), MC2_ERR_ALIGN, "align");
  expect(check_moe_route_grad(a, a, a, 4, 64, 4, MC2_F16, soft, 1.f, a), MC2_OK, "route grad");
  expect(check_moe_route_grad(a, a, nullptr, 4, 64, 4, MC2_F16, soft, 1.f, a), MC2_ERR_NULL, "ids");

  expect(check_code_rows("t", a, a, a, 4, 256, MC2_BF16, 128, MC2_ACT_NONE), MC2_OK, "codes");
  expect(check_code_rows("t", a, a, a, big, 256, MC2_BF16, 0, MC2_ACT_NONE), MC2_ERR_SHAPE, "rows");
  expect(check_code_rows("t", a, a, a, 4, big, MC2_BF16, 0, MC2_ACT_NONE), MC2_ERR_SHAPE, "cols");
  expect(check_code_rows("t", a, a, a, 4, 256, MC2_BF16, big, MC2_ACT_NONE), MC2_ERR_SHAPE, "group");
  expect(check_code_rows("t", a, a, nullptr, 4, 256, MC2_BF16, 0, MC2_ACT_NONE), MC2_ERR_NULL, "scale");
  expect(check_code_rows("t", a, a, a, 4, 256, MC2_BF16, 0, (mc2_act)9), MC2_ERR_UNSUPPORTED, "act");

  expect(check_linear_i8_sizes("t", 1, (1 << 17) - 1, 1, 0), MC2_OK, "linear sizes");
  expect(check_linear_i8_sizes("t", 1, 1 << 17, 1, 0), MC2_ERR_SHAPE, "k");
  expect(check_linear_i8_sizes("t", 1, 1, big, 0), MC2_ERR_SHAPE, "n");
  expect(check_linear_i8_sizes("t", 1, 1, 1, big), MC2_ERR_SHAPE, "groups");
  expect(check_linear_i8(a, a, a, a, a, a, 4, 16, 8, nullptr, 0, MC2_BF16, MC2_ACT_SILU, a, nullptr, 0, 0), MC2_OK, "i8");
  expect(check_linear_i8(a, a, a, nullptr, a, a, 4, 16, 8, nullptr, 0, MC2_BF16, MC2_ACT_SILU, a, nullptr, 0, 0),
         MC2_ERR_NULL, "w_scale");
  expect(check_linear_i8(a, a, a, a, a, a, 4, 16, 8, a, 3, MC2_BF16, MC2_ACT_SILU, a, a, 63, 64), MC2_ERR_WORKSPACE, "ws");
  expect(check_linear_act_grad_i8(a, a, a, a, a, MC2_ACT_GELU, a, 4, 8, 8, nullptr, 0, MC2_BF16, MC2_ACT_GELU, a, a, a, a,
                                  64, 64), MC2_OK, "grad");
  expect(check_linear_act_grad_i8(a, nullptr, nullptr, nullptr, nullptr, MC2_ACT_NONE, a, 4, 8, 8, nullptr, 0, MC2_BF16,
                                  MC2_ACT_NONE, a, nullptr, a, a, 64, 64), MC2_OK, "dx alone");
  expect(check_linear_act_grad_i8(a, a, nullptr, a, a, MC2_ACT_NONE, a, 4, 8, 8, nullptr, 0, MC2_BF16, MC2_ACT_GELU, a, a,
                                  a, a, 64, 64), MC2_ERR_NULL, "z_scale");
  expect(check_linear_act_grad_i8(a, a, a, a, a, (mc2_act)-1, a, 4, 8, 8, nullptr, 0, MC2_BF16, MC2_ACT_GELU, a, a, a, a,
                                  64, 64), MC2_ERR_UNSUPPORTED, "x_act");
  if (failures) return 1;
  std::printf("clean\n");
  return 0;
}
