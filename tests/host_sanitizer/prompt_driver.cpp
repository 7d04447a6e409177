// Host-side validation of the rotary, prompt attention, slot and page entry
// points, for a build of their host code with AddressSanitizer and
// UndefinedBehaviorSanitizer: every size in turn takes values at and past its
// limits, and every call either fails validation or is an empty batch.  Pointers
// are made-up addresses that are never dereferenced on the host.  The driver
// refuses to run when a GPU is visible: it is a test of host code only.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "qlin.h"

namespace {

int g_failures = 0, g_calls = 0;

template <class T>
T* at(uintptr_t a) {
  return reinterpret_cast<T*>(a);
}

void refused(const char* what, int64_t x, qlin_status st) {
  ++g_calls;
  if (st == QLIN_OK || st == QLIN_ERR_HIP || strlen(qlin_last_error()) == 0) {
    ++g_failures;
    printf("FAIL %s = %lld: %s\n", what, (long long)x, qlin_status_string(st));
  }
}

struct Rope {
  int64_t ld_q = 512, ld_k = 256, T = 3, ld_qo = 512, ld_ko = 256;
  int32_t heads = 4, kv_heads = 2, head_dim = 128, rot_dim = 64;
  qlin_status call() const {
    return qlin_rope(at<uint16_t>(0x10000), ld_q, heads, at<uint16_t>(0x20000), ld_k, kv_heads, T, head_dim, rot_dim, 0,
                     at<int32_t>(0x30000), at<double>(0x40000), 1.0f, 0, at<uint16_t>(0x50000), ld_qo,
                     at<uint16_t>(0x60000), ld_ko, nullptr);
  }
};

struct Prompt {
  int64_t ld_q = 512, ld_k = 256, ld_v = 256, ld_do = 512, ld_dq = 512, ld_dk = 256, ld_dv = 256, B = 2, Tq = 40, Tk = 50;
  int32_t heads = 4, kv_heads = 2, head_dim = 128, causal = 1, window = 0;
  qlin_status forward() const {
    return qlin_attn_prompt(at<uint16_t>(0x10000), ld_q, heads, at<uint16_t>(0x20000), ld_k, at<uint16_t>(0x30000), ld_v,
                            kv_heads, head_dim, at<int32_t>(0x40000), at<int32_t>(0x50000), B, Tq, Tk, 1.0f, causal,
                            window, at<uint16_t>(0x60000), nullptr, at<void>(0x70000), nullptr);
  }
  qlin_status backward() const {
    return qlin_attn_prompt_backward(at<uint16_t>(0x10000), ld_do, at<uint16_t>(0x20000), ld_q, heads,
                                     at<uint16_t>(0x30000), ld_k, at<uint16_t>(0x40000), ld_v, kv_heads, head_dim,
                                     at<uint16_t>(0x50000), at<float>(0x60000), at<int32_t>(0x70000),
                                     at<int32_t>(0x80000), B, Tq, Tk, 1.0f, causal, window, at<uint16_t>(0x90000), ld_dq,
                                     at<uint16_t>(0xa0000), ld_dk, at<uint16_t>(0xb0000), ld_dv, at<void>(0xc0000),
                                     nullptr);
  }
  void both(const char* what, int64_t x) const {
    refused(what, x, forward());
    refused(what, x, backward());
    g_calls += 1;
    (void)qlin_attn_prompt_work_bytes(heads, kv_heads, head_dim, B, Tq, Tk, causal, window);
    (void)qlin_attn_prompt_backward_work_bytes(heads, kv_heads, head_dim, B, Tq, Tk, causal, window);
  }
};

qlin_status slots(int64_t B, int64_t T) {
  return qlin_kv_slots(at<int32_t>(0x10000), at<int32_t>(0x20000), nullptr, B, T, at<int32_t>(0x30000),
                       at<int32_t>(0x40000), at<int32_t>(0x50000), at<int32_t>(0x60000), at<int32_t>(0x70000), nullptr);
}

qlin_status pages(int64_t B, int64_t max_pages, int32_t page, int64_t n) {
  return qlin_kv_pages(at<int32_t>(0x10000), B, max_pages, page, at<int32_t>(0x20000), at<int32_t>(0x30000),
                       at<int32_t>(0x40000), n, at<int32_t>(0x50000), at<int32_t>(0x60000), at<int32_t>(0x70000),
                       at<int32_t>(0x80000), at<int32_t>(0x90000), nullptr);
}

const int64_t kOdd[] = {INT64_MIN, INT64_MIN + 1, -(int64_t(1) << 40), -1, int64_t(1) << 31, (int64_t(1) << 31) + 8,
                        int64_t(1) << 40, int64_t(1) << 62, INT64_MAX - 7, INT64_MAX};
const int32_t kOdd32[] = {INT32_MIN, INT32_MIN + 1, -1, 3, 7, INT32_MAX};

}  // namespace

int main() {
  int gpus = 0;
  if (hipGetDeviceCount(&gpus) == hipSuccess && gpus > 0) return 77;

#define EACH(T, field, values, CALL)   \
  for (auto x : values) {              \
    T a;                               \
    a.field = x;                       \
    CALL;                              \
  }
  EACH(Rope, ld_q, kOdd, refused("rope ld_q", x, a.call()))
  EACH(Rope, ld_k, kOdd, refused("rope ld_k", x, a.call()))
  EACH(Rope, ld_qo, kOdd, refused("rope ld_qo", x, a.call()))
  EACH(Rope, ld_ko, kOdd, refused("rope ld_ko", x, a.call()))
  EACH(Rope, T, kOdd, refused("rope T", x, a.call()))
  EACH(Rope, head_dim, kOdd32, refused("rope head_dim", x, a.call()))
  EACH(Rope, rot_dim, kOdd32, refused("rope rot_dim", x, a.call()))
  for (int32_t x : {INT32_MIN, -1, 0, 65536, INT32_MAX}) {
    Rope a;
    a.heads = x;
    a.ld_q = a.ld_qo = int64_t(1) << 30;
    refused("rope heads", x, a.call());
    a.heads = 4;
    a.kv_heads = x;
    refused("rope kv_heads", x, a.call());
  }
  EACH(Prompt, ld_q, kOdd, a.both("ld_q", x))
  EACH(Prompt, ld_k, kOdd, a.both("ld_k", x))
  EACH(Prompt, ld_v, kOdd, a.both("ld_v", x))
  EACH(Prompt, ld_do, kOdd, refused("ld_dout", x, a.backward()))
  EACH(Prompt, ld_dq, kOdd, refused("ld_dq", x, a.backward()))
  EACH(Prompt, ld_dk, kOdd, refused("ld_dk", x, a.backward()))
  EACH(Prompt, ld_dv, kOdd, refused("ld_dv", x, a.backward()))
  EACH(Prompt, B, kOdd, a.both("B", x))
  EACH(Prompt, Tq, kOdd, a.both("Tq", x))
  EACH(Prompt, Tk, kOdd, a.both("Tk", x))
  EACH(Prompt, heads, kOdd32, a.both("heads", x))
  EACH(Prompt, kv_heads, kOdd32, a.both("kv_heads", x))
  EACH(Prompt, head_dim, kOdd32, a.both("head_dim", x))
  for (int32_t x : {INT32_MIN, -1}) {
    Prompt a;
    a.window = x;
    a.both("window", x);
  }
  {
    Prompt a;  // the most workgroups, and one too many
    a.heads = a.kv_heads = 65535;
    a.ld_q = a.ld_k = a.ld_v = a.ld_do = a.ld_dq = a.ld_dk = a.ld_dv = int64_t(1) << 22;
    a.head_dim = 64;
    a.B = 65535;
    a.both("workgroups", a.B);
  }
  for (int64_t x : kOdd) {
    refused("slots B", x, slots(x, 5));
    refused("slots T", x, slots(2, x));
    refused("pages B", x, pages(x, 4, 16, 8));
    refused("pages max_pages", x, pages(2, x, 16, 8));
    refused("pages of the ring", x, pages(2, 4, 16, x));
  }
  for (int32_t x : {INT32_MIN, -16, 0, 8, 24, 2048, INT32_MAX}) refused("page", x, pages(2, 4, x, 8));
  double freq[128];
  float amplitude;
  for (int32_t x : kOdd32) refused("rot_dim", x, qlin_rope_freqs(x, 1e4, 0, 1.0, 0, 32.0, 1.0, freq, &amplitude));
  for (int64_t x : kOdd)
    refused("original_len", x, qlin_rope_freqs(256, 1e4, QLIN_ROPE_RAMP, 2.0, x, 32.0, 1.0, freq, &amplitude));
  for (int32_t s = 0; s < 4; ++s) {
    ++g_calls;
    if (qlin_rope_freqs(256, 1e4, s, 2.0, 100, 32.0, 1.0, freq, &amplitude) != QLIN_OK) {
      ++g_failures;
      printf("FAIL frequencies %d: %s\n", s, qlin_last_error());
    }
  }
  g_calls += 3;
  Prompt none;
  none.B = 0;
  Rope still;
  still.T = 0;
  if (none.forward() != QLIN_OK || none.backward() != QLIN_OK || still.call() != QLIN_OK) {
    ++g_failures;
    printf("FAIL empty calls: %s\n", qlin_last_error());
  }
  printf("%d calls, %d failures\n", g_calls, g_failures);
  return g_failures ? 1 : 0;
}
