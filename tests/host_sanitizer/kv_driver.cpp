// Host-side validation of the key/value cache's entry points, for a build of
// their host code with AddressSanitizer and UndefinedBehaviorSanitizer: every
// argument in turn takes values at and past its limits, and every call either
// fails validation or is an empty batch.  Pointers are made-up addresses that
// are never dereferenced on the host.  The driver refuses to run when a GPU is
// visible: it is a test of host code only.
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

void refused(const char* what, qlin_status st) {
  ++g_calls;
  if (st == QLIN_OK || st == QLIN_ERR_HIP || strlen(qlin_last_error()) == 0) {
    ++g_failures;
    printf("FAIL %s: %s\n", what, qlin_status_string(st));
  }
}

void accepted(const char* what, qlin_status st) {
  ++g_calls;
  if (st != QLIN_OK) {
    ++g_failures;
    printf("FAIL %s: %s (%s)\n", what, qlin_status_string(st), qlin_last_error());
  }
}

qlin_kv_cache good() {
  qlin_kv_cache c{};
  c.k = at<void>(0x10000);
  c.v = at<void>(0x20000);
  c.kmeta = at<uint16_t>(0x30000);
  c.vmeta = at<uint16_t>(0x40000);
  c.pages = 8;
  c.page = 16;
  c.kv_heads = 2;
  c.head_dim = 128;
  c.bits = 4;
  return c;
}

const int64_t kOdd[] = {INT64_MIN, INT64_MIN + 1, -(int64_t(1) << 40), -1, int64_t(1) << 31, (int64_t(1) << 31) + 8,
                        int64_t(1) << 40, int64_t(1) << 62, INT64_MAX - 7, INT64_MAX};

qlin_status append(const qlin_kv_cache* c, int64_t ld_k, int64_t ld_v, int64_t T, int64_t B, int64_t max_pages,
                   int64_t ld, bool track) {
  return qlin_kv_append(c, at<uint16_t>(0x50000), ld_k, at<uint16_t>(0x60000), ld_v, T, at<int32_t>(0x70000),
                        at<int32_t>(0x80000), at<int32_t>(0x90000), B, max_pages,
                        track ? at<int32_t>(0xa0000) : nullptr, track ? at<float>(0xb0000) : nullptr,
                        track ? at<int32_t>(0xc0000) : nullptr, ld, nullptr);
}

qlin_status attend(const qlin_kv_cache* c, int64_t ld_q, int32_t heads, int64_t B, int64_t max_pages, int64_t max_len,
                   int64_t ld, bool mass) {
  return qlin_attn_decode(c, at<uint16_t>(0x50000), ld_q, heads, at<int32_t>(0x60000), at<int32_t>(0x70000), B,
                          max_pages, max_len, 1.0f, 0, at<uint16_t>(0x80000), nullptr,
                          mass ? at<float>(0x90000) : nullptr, ld, at<void>(0xa0000), nullptr);
}

qlin_status evict(const qlin_kv_cache* c, int64_t B, int64_t max_pages, int64_t max_len, int32_t budget,
                  int32_t recent, int64_t ld) {
  return qlin_kv_evict(c, at<int32_t>(0x50000), at<int32_t>(0x60000), B, max_pages, max_len, budget, recent,
                       at<float>(0x70000), at<int32_t>(0x80000), ld, at<float>(0x90000), at<int32_t>(0xa0000),
                       at<int32_t>(0xb0000), at<int32_t>(0xc0000), at<void>(0xd0000), nullptr);
}

}  // namespace

int main() {
  int gpus = 0;
  if (hipGetDeviceCount(&gpus) == hipSuccess && gpus > 0) return 77;

  const qlin_kv_cache c = good();
  for (int64_t x : kOdd) {
    refused("append ld_k", append(&c, x, 256, 4, 2, 4, 64, false));
    refused("append ld_v", append(&c, 256, x, 4, 2, 4, 64, false));
    refused("append T", append(&c, 256, 256, x, 2, 4, 64, false));
    refused("append B", append(&c, 256, 256, 4, x, 4, 64, false));
    refused("append max_pages", append(&c, 256, 256, 4, 2, x, 64, false));
    refused("append ld", append(&c, 256, 256, 4, 2, 4, x, true));
    refused("attend ld_q", attend(&c, x, 4, 2, 4, 64, 64, false));
    refused("attend B", attend(&c, 512, 4, x, 4, 64, 64, false));
    refused("attend max_pages", attend(&c, 512, 4, 2, x, 64, 64, false));
    refused("attend max_len", attend(&c, 512, 4, 2, 4, x, 64, false));
    refused("attend ld", attend(&c, 512, 4, 2, 4, 64, x, true));
    refused("evict B", evict(&c, x, 4, 64, 16, 4, 64));
    refused("evict max_pages", evict(&c, 2, x, 64, 16, 4, 64));
    refused("evict max_len", evict(&c, 2, 4, x, 16, 4, 64));
    refused("evict ld", evict(&c, 2, 4, 64, 16, 4, x));
    qlin_kv_cache d = good();
    d.pages = x;
    refused("pages", append(&d, 256, 256, 4, 2, 4, 64, false));
    g_calls += 4;
    if (qlin_attn_decode_work_bytes(&c, 4, x, 64, 0, 1) != 0 || qlin_attn_decode_work_bytes(&c, 4, 2, x, 0, 1) != 0 ||
        qlin_kv_evict_work_bytes(&c, x, 64, 16) != 0 || qlin_kv_evict_work_bytes(&c, 2, x, 16) != 0) {
      ++g_failures;
      printf("FAIL workspace bytes of %lld\n", (long long)x);
    }
  }
  const int32_t odd32[] = {INT32_MIN, -1, 0, 3, INT32_MAX};
  for (int32_t x : odd32) {
    refused("attend heads", attend(&c, int64_t(1) << 30, x, 2, 4, 64, 64, false));
    if (x != 3 && x != INT32_MAX) refused("evict budget", evict(&c, 2, 4, 64, x, 0, 64));
    if (x != 3 && x != 0) refused("evict recent", evict(&c, 2, 4, 64, 16, x, 64));
    qlin_kv_cache d = good();
    d.page = x;
    refused("page", evict(&d, 2, 4, 64, 16, 4, 64));
    d = good();
    d.bits = x;
    refused("bits", attend(&d, 512, 4, 2, 4, 64, 64, false));
    d = good();
    d.head_dim = x;
    refused("head_dim", append(&d, 256, 256, 4, 2, 4, 64, false));
    d = good();
    d.kv_heads = x;
    refused("kv_heads", attend(&d, 512, 4, 2, 4, 64, 64, false));
    g_calls += 2;
    (void)qlin_attn_decode_work_bytes(&c, x, 2, 64, x, 1);
    (void)qlin_kv_evict_work_bytes(&c, 2, 64, x);
  }
  refused("no cache", append(nullptr, 256, 256, 4, 2, 4, 64, false));
  refused("no cache", attend(nullptr, 512, 4, 2, 4, 64, 64, false));
  refused("no cache", evict(nullptr, 2, 4, 64, 16, 4, 64));
  accepted("append no tokens", append(&c, 256, 256, 0, 2, 4, 64, true));
  accepted("append no rows", append(&c, 256, 256, 0, 0, 4, 64, true));
  accepted("attend no rows", attend(&c, 512, 4, 0, 4, 64, 64, true));
  accepted("evict no rows", evict(&c, 0, 4, 64, 16, 4, 64));
  printf("%d calls, %d failures\n", g_calls, g_failures);
  return g_failures ? 1 : 0;
}
