// Host-side pieces shared by the files that implement the C ABI: the context,
// error reporting, launch timing and workspace carving.
#pragma once

#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <string>

#include "qi.h"
#include "qi_common.cuh"
#include "qi_internal.h"

// Optional per-launch timing: when enabled, every kernel launch of the library
// is bracketed by a pair of CUDA events on its stream; durations are summed per
// kernel class when read back.  Launches are counted per class either way.
constexpr int QI_PROF_CLASSES = 8;
constexpr int QI_PROF_MAX_PAIRS = 16384;

struct qi_ctx {
  int device;
  int num_sms;
  int* status;   // device status word
  bool prof_on;
  int prof_used;
  cudaEvent_t* prof_ev;          // [2 * QI_PROF_MAX_PAIRS]
  int* prof_cls;                 // [QI_PROF_MAX_PAIRS]
  long long launches[QI_PROF_CLASSES];
  int attn_fp8;                  // steps run e4m3 attention (qi_ctx_set_attention_fp8)
  bool taps_on;                  // copy the quantizers' inputs and outputs (qi_ctx_set_block_taps)
  qi_block_taps taps;
  void* attn_scratch;            // key-range split scratch of qi_attn_block_causal(_fp8)
  size_t attn_scratch_bytes;
};

// Error text of the calling thread, and helpers that set it.
namespace qi_host {

inline thread_local std::string g_last_error;

inline int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return code;
}

inline int cuda_fail(const char* what) {
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) {   // already read by the launcher
    e = qi::last_launch_error();
    qi::last_launch_error() = cudaSuccess;
  }
  return fail(QI_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline cudaStream_t S(void* s) { return static_cast<cudaStream_t>(s); }

struct Prof {
  qi_ctx* c;
  int slot;
  cudaStream_t st;
  Prof(qi_ctx* ctx, int cls, cudaStream_t s) : c(ctx), slot(-1), st(s) {
    if (!c) return;
    c->launches[cls] += 1;
    if (c->prof_on && c->prof_used < QI_PROF_MAX_PAIRS) {
      slot = c->prof_used++;
      c->prof_cls[slot] = cls;
      cudaEventRecord(c->prof_ev[2 * slot], st);
    }
  }
  ~Prof() {
    if (slot >= 0) cudaEventRecord(c->prof_ev[2 * slot + 1], st);
  }
};

// Bump allocator over the caller's workspace (256-byte aligned pieces).
struct Carve {
  uint8_t* base;
  size_t cap, off;
  template <class T>
  T* take(size_t count) {
    off = (off + 255) & ~static_cast<size_t>(255);
    T* p = reinterpret_cast<T*>(base ? base + off : nullptr);
    off += count * sizeof(T);
    return p;
  }
};

}  // namespace qi_host
