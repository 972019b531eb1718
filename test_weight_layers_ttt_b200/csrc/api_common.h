// Host-side plumbing shared by the C ABI's translation units (ttt_api.cu, mixer_api.cu):
// error messages, kernel tracing, workspace carving, the debug checks around a call. The
// state behind it is defined in ttt_api.cu.
#pragma once

#include <atomic>
#include <initializer_list>
#include <mutex>
#include <vector>

#include "ops.h"

namespace ttt {

void set_error_message(const char* fmt, ...);
unsigned* device_error_word();

// Records a formatted message for the calling thread and returns `st`.
ttt_status fail(ttt_status st, const char* fmt, ...);

// ------------------------------------------------------------------ kernel tracing
struct TraceState {
  std::mutex mu;
  bool on = false;
  int dev = -1;
  int n = 0;
  int cap = 0;
  std::vector<cudaEvent_t> ev;  // 2 per record
  std::vector<const char*> names;
};
extern TraceState g_trace;

// Brackets one kernel launch with two events on its stream while tracing is enabled.
struct TraceScope {
  int idx = -1;
  cudaStream_t s;
  TraceScope(const char* name, cudaStream_t st) : s(st) {
    if (!g_trace.on) return;
    std::lock_guard<std::mutex> lk(g_trace.mu);
    int d = -1;
    if (!g_trace.on || cudaGetDevice(&d) != cudaSuccess || d != g_trace.dev ||
        g_trace.n >= g_trace.cap)
      return;
    idx = g_trace.n++;
    g_trace.names[idx] = name;
    cudaEventRecord(g_trace.ev[2 * idx], s);
  }
  ~TraceScope() {
    if (idx >= 0) cudaEventRecord(g_trace.ev[2 * idx + 1], s);
  }
};

#define TTT_TRY(expr)                        \
  do {                                       \
    ttt_status st__ = (expr);                \
    if (st__ != TTT_OK) return st__;         \
  } while (0)

#define TTT_CUDA(expr)                                                                    \
  do {                                                                                    \
    cudaError_t e__ = (expr);                                                             \
    if (e__ != cudaSuccess) {                                                             \
      set_error_message("%s failed: %s", #expr, cudaGetErrorString(e__));                 \
      return TTT_ERR_CUDA;                                                                \
    }                                                                                     \
  } while (0)

// One traced kernel launch of ops.h.
#define TTT_OP(name, expr)         \
  do {                             \
    TraceScope ts__((name), s);    \
    TTT_CUDA(expr);                \
  } while (0)

inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// ------------------------------------------------------------------ debug checks
// Process-wide TTT_CHECK_* flags (ttt_set_debug_checks), and the guards the calling thread's
// current call carved from its workspace.
extern std::atomic<int> g_checks;
extern thread_local std::vector<unsigned*> t_guards;

// Bump allocator over the caller's workspace (or a size counter when base is null). With
// TTT_CHECK_GUARDS on, a kGuardBytes guard sits in front of the first region and right
// after the end of every region (16-byte aligned); the guards of a real workspace are
// listed in t_guards.
struct Carve {
  char* base;
  size_t off = 0;
  bool guards;
  explicit Carve(void* b)
      : base(static_cast<char*>(b)), guards((g_checks.load() & TTT_CHECK_GUARDS) != 0) {
    if (guards) guard();
  }
  void guard() {
    off = (off + 15) & ~static_cast<size_t>(15);
    if (base) t_guards.push_back(reinterpret_cast<unsigned*>(base + off));
    off += kGuardBytes;
  }
  void* take(size_t bytes) {
    off = (off + 255) & ~static_cast<size_t>(255);
    void* p = base ? base + off : nullptr;
    off += bytes;
    if (guards) guard();
    return p;
  }
  template <typename T> T* take_n(long long n) { return static_cast<T*>(take(sizeof(T) * (size_t)n)); }
};

// Fills (check = false) or compares (check = true) every guard in t_guards.
ttt_status run_guards(bool check, cudaStream_t s);

// One output of a call, for the non-finite scan.
struct OutBuf {
  const void* p;
  long long n;
  int dt;
};

// Start of a call's work on `s`: writes the guards of the workspace just planned.
ttt_status checks_begin(cudaStream_t s);

// End of a call's work on `s`: compares the guards and scans the outputs.
ttt_status checks_end(cudaStream_t s, std::initializer_list<OutBuf> outs);

// A call's body between checks_begin and checks_end; the end runs after a successful body.
template <typename F>
ttt_status with_checks(cudaStream_t s, std::initializer_list<OutBuf> outs, F&& body) {
  TTT_TRY(checks_begin(s));
  TTT_TRY(body());
  return checks_end(s, outs);
}

// A caller workspace of at least `need` bytes, 256-byte aligned (TTT_ERR_WORKSPACE otherwise).
ttt_status check_ws(void* ws, size_t have, size_t need);

}  // namespace ttt
