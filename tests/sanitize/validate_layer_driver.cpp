// Calls every host-side check of the feed-forward operators on valid and
// invalid arguments; built with sanitizers by tests/test_layer_sanitizers.py.
#include <climits>
#include <cmath>
#include <cstdio>
#include <cstdlib>

#include "validate_layer.hpp"

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

  expect(check_norm_sizes("t", 0, 1), MC2_OK, "norm sizes");
  expect(check_norm_sizes("t", big, 1), MC2_ERR_SHAPE, "norm rows");
  expect(check_norm_sizes("t", -1, 1), MC2_ERR_SHAPE, "norm rows below 0");
  expect(check_norm_sizes("t", 1, big), MC2_ERR_SHAPE, "norm h");
  expect(check_add_rms_norm(a, a, a, 4, 256, MC2_BF16, 0.f, a, MC2_BF16, nullptr, 0, a, a), MC2_OK, "norm");
  expect(check_add_rms_norm(a, a, a, 4, 256, MC2_F16, 1.f, a, MC2_I8, a, 128, a, a), MC2_OK, "norm int8");
  expect(check_add_rms_norm(a, a, a, 4, 256, MC2_F16, NAN, a, MC2_F16, nullptr, 0, a, a), MC2_ERR_SHAPE, "eps");
  expect(check_add_rms_norm(a, a, a, 4, 256, MC2_F16, 1.f, a, MC2_I8, nullptr, 0, a, a), MC2_ERR_NULL, "scale");
  expect(check_add_rms_norm(a, a, a, 4, 256, MC2_F16, 1.f, a, MC2_F16, nullptr, big, a, a), MC2_ERR_SHAPE, "group");
  expect(check_add_rms_norm(a, odd, a, 4, 256, MC2_F16, 1.f, a, MC2_F16, nullptr, 0, a, a), MC2_ERR_ALIGN, "align");
  expect(check_add_rms_norm(nullptr, nullptr, nullptr, 0, 256, MC2_F16, 1.f, nullptr, MC2_F16, nullptr, 0, nullptr,
                            nullptr), MC2_OK, "no rows");
  expect(check_add_rms_norm_grad(a, nullptr, a, a, a, 4, 256, MC2_BF16, a, a, a, 64, 64), MC2_OK, "norm grad");
  expect(check_add_rms_norm_grad(a, nullptr, a, a, a, 4, 256, MC2_BF16, a, a, a, 63, 64), MC2_ERR_WORKSPACE, "ws");
  expect(check_add_rms_norm_grad(a, nullptr, a, a, a, 4, 256, MC2_BF16, a, a, odd, 64, 64), MC2_ERR_ALIGN, "ws align");

  expect(check_linear_sizes("t", 0, 1, 1, 0), MC2_OK, "linear sizes");
  expect(check_linear_sizes("t", big, 1, 1, 0), MC2_ERR_SHAPE, "m");
  expect(check_linear_sizes("t", 1, big, 1, 0), MC2_ERR_SHAPE, "k");
  expect(check_linear_sizes("t", 1, 1, big, 0), MC2_ERR_SHAPE, "n");
  expect(check_linear_sizes("t", 1, 1, 1, big), MC2_ERR_SHAPE, "groups");
  expect(check_linear_sizes("t", 1, 1 << 21, 1, 4096), MC2_ERR_SHAPE, "groups * k");
  expect(check_linear_act(a, a, a, a, 4, 8, 8, nullptr, 0, MC2_BF16, MC2_ACT_SILU, a, a, nullptr, 0, 0), MC2_OK,
         "linear");
  expect(check_linear_act(a, a, a, a, 4, 8, 8, a, 3, MC2_BF16, MC2_ACT_SILU, a, a, nullptr, 0, 0), MC2_OK, "groups");
  expect(check_linear_act(a, a, a, a, 4, 8, 8, nullptr, 3, MC2_BF16, MC2_ACT_SILU, a, a, nullptr, 0, 0), MC2_ERR_NULL,
         "offsets");
  expect(check_linear_act(a, a, a, a, 4, 8, 8, nullptr, 0, MC2_BF16, (mc2_act)7, a, a, nullptr, 0, 0),
         MC2_ERR_UNSUPPORTED, "act");
  expect(check_linear_act_grad(a, nullptr, a, a, 4, 8, 8, nullptr, 0, MC2_BF16, MC2_ACT_NONE, a, a, a, a, 16, 16),
         MC2_OK, "linear grad");
  expect(check_linear_act_grad(a, nullptr, a, a, 4, 8, 8, nullptr, 0, MC2_BF16, MC2_ACT_GELU, a, a, a, a, 16, 16),
         MC2_ERR_NULL, "z");

  expect(check_permute_sizes("t", 0, 1, 1), MC2_OK, "permute sizes");
  expect(check_permute_sizes("t", 1 << 20, big, 1), MC2_ERR_SHAPE, "top");
  expect(check_permute_sizes("t", 1 << 23, 256, 1), MC2_ERR_SHAPE, "choices");
  expect(check_permute_sizes("t", big, 1, 1), MC2_ERR_SHAPE, "tokens");
  expect(check_permute_sizes("t", 1, 1, big), MC2_ERR_SHAPE, "experts");
  expect(check_moe_permute(a, a, 4, 2, 8, 4, MC2_F16, a, a, a, nullptr, 0, 0), MC2_OK, "permute");
  expect(check_moe_permute(a, a, 4, 2, 8, 4, MC2_F16, a, a, nullptr, nullptr, 0, 0), MC2_ERR_NULL, "offsets");
  expect(check_moe_unpermute(a, a, nullptr, 4, 2, 8, 8, MC2_F16, a), MC2_OK, "unpermute");
  expect(check_moe_unpermute(nullptr, a, nullptr, 4, 2, 8, 0, MC2_F16, a), MC2_OK, "no rows of y");
  expect(check_moe_unpermute(a, a, nullptr, 4, 2, 8, big, MC2_F16, a), MC2_ERR_SHAPE, "rows");
  expect(check_moe_unpermute_grad(a, a, a, nullptr, 4, 2, 8, 8, MC2_F16, a, a), MC2_OK, "unpermute grad");
  expect(check_moe_unpermute_grad(a, a, a, nullptr, 4, 2, 8, 8, MC2_F16, nullptr, nullptr), MC2_ERR_NULL, "nothing");
  if (failures) return 1;
  std::printf("clean\n");
  return 0;
}
