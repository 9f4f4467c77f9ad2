// qmv_attn.cuh -- what the attention kernels over the paged cache share: sequence geometry
// read on the device, barrier and copy primitives, 16-bit operand decoding.
#pragma once
#include "qmv_internal.h"
#include "qmv_attn_geom.h"

namespace qmv {

constexpr unsigned long long kAttnTimeoutNs = 1000000000ull;
constexpr float kLog2e = 1.4426950408889634f;

// Probabilities are formed against a reference per row, in base 2: p = 2^(s - m). m is raised only
// when a logit passes it by more than kHead + kLazy, and then to kHead below the largest. f16
// probabilities use f16's range for the small ones: with kHead = 7 the largest is between 2^7
// and 2^15, so one that f16's smallest step, 2^-24, rounds off is below 2^-32 of it (2^18 keys
// beside one that outweighs them by e^18 still count; at kHead = 0 they were lost). bf16 has
// fp32's range. m stands for the reference wherever parts are joined.
constexpr int kLazy = 8;               // log2 of the growth of a maximum that O tolerates
template <bool BF>
constexpr int kHead = BF ? 0 : 7;

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ unsigned long long attn_timer() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ void bar_init(uint32_t b, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(b), "r"(count) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t b, uint32_t parity) {
  uint32_t ok;
  asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
               : "=r"(ok) : "r"(b), "r"(parity) : "memory");
  return ok != 0;
}
// ... without waiting
__device__ __forceinline__ bool bar_test(uint32_t b, uint32_t parity) {
  uint32_t ok;
  asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
               : "=r"(ok) : "r"(b), "r"(parity) : "memory");
  return ok != 0;
}
// every wait ends: false after a second
__device__ __forceinline__ bool bar_wait_slow(uint32_t b, uint32_t parity) {
  const unsigned long long t0 = attn_timer();
  for (uint32_t it = 1;; ++it) {
    if (bar_try(b, parity)) return true;
    if ((it & 63u) == 0 && attn_timer() - t0 > kAttnTimeoutNs) return false;
  }
}
__device__ __forceinline__ bool bar_wait(uint32_t b, uint32_t parity) {
  return bar_try(b, parity) || bar_wait_slow(b, parity);
}
__device__ __forceinline__ void bar_arrive(uint32_t b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(b) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(b), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// The two attention kernels of one call run beside each other: either may start on the SMs that
// the one before it leaves (let_next_start), and neither ends before it (wait_for_previous,
// by one thread of every CTA). Both do nothing where a kernel is launched by itself.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---- 16-bit operands ------------------------------------------------------------
__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t h2_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// E4M3 codes of a word (bytes 0..3) -> two f16x2, exact (NaN kept)
__device__ __forceinline__ void e4m3_word(uint32_t w, uint32_t* o) {
  asm("{ .reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(o[0]), "=r"(o[1]) : "r"(w));
}
__device__ __forceinline__ uint32_t e4m3_half(uint32_t two) {
  uint32_t r;
  const unsigned short v = (unsigned short)two;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
// E2M1 codes of a word (bytes 0..3, low nibble first) -> four f16x2, exact. The conversion
// picks its byte by itself when it is handed the word's bytes (10.3 cycles a word per warp
// with the products behind it; taken out by shifts, 14.1)
__device__ __forceinline__ void e2m1_word(uint32_t w, uint32_t* o) {
  asm("{ .reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]) : "r"(w));
}
// Q8_0 codes q + 128 of a word -> two f16x2 of q, exact: the byte under f16's 1024
__device__ __forceinline__ void q8_word(uint32_t w, uint32_t* o) {
  o[0] = h2_sub(__byte_perm(w, 0x64646464u, 0x4140), 0x64806480u);
  o[1] = h2_sub(__byte_perm(w, 0x64646464u, 0x4342), 0x64806480u);
}
__device__ __forceinline__ uint32_t dup_lo(uint32_t h) { return __byte_perm(h, h, 0x1010); }
__device__ __forceinline__ uint32_t dup_hi(uint32_t h) { return __byte_perm(h, h, 0x3232); }
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// power of two that brings a row of queries to 2^14 .. 2^15 (f16 operands: values down to
// 2^-28 of the row's largest stay exact), and its inverse
__device__ __forceinline__ void row_scale(float amax, float* mul, float* inv) {
  const int e = (int)(__float_as_uint(amax) >> 23);
  if (e == 255) {
    *mul = *inv = 1.0f;
    return;
  }
  const int f = 268 - e < 253 ? 268 - e : 253;
  *mul = __uint_as_float((uint32_t)f << 23);
  *inv = __uint_as_float((uint32_t)(254 - f) << 23);
}

// A CTA's places among the numbered tiles are 32-bit integers from the start of its range; a
// batch that gives one more than this many (half a minute of work at least) latches QMV_ERANGE instead
constexpr int64_t kMostPlaces = (int64_t)1 << 30;
// places among the numbered tiles nearly always fit 32 bits, where a division is a fifth as long
__device__ __forceinline__ int64_t place_div(int64_t a, int64_t b) {
  return ((a | b) >> 31) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// ---- sequence geometry ------------------------------------------------------------
struct SeqInfo {
  int n, c, s0;        // cached tokens, new tokens, first query row
};
// false (and a latched QMV_ERANGE from the reporting thread): nothing of it is computed
__device__ __forceinline__ bool seq_info(const AttnArgs& a, int b, SeqInfo* s, bool report) {
  s->n = __ldg(a.kv_len + b);
  s->s0 = __ldg(a.q_start + b);
  const int s1 = __ldg(a.q_start + b + 1);
  s->c = s1 - s->s0;
  const bool ok = s->s0 >= 0 && s1 >= s->s0 && s1 <= a.T && s->c <= a.max_q && s->n >= 0 &&
                  s->n <= (a.max_pages << a.c.page_shift);
  if (!ok) {
    if (report) atomicOr(a.status, kStatRange);
    s->c = 0;
    s->n = 0;
  }
  return ok;
}
// first key that any query of the sequence sees
__device__ __forceinline__ int seq_first(const AttnArgs& a, const SeqInfo& s) {
  return window_first(s.n - s.c, a.window);
}
__device__ __forceinline__ int checked_page(const AttnArgs& a, int page) {
  if (page < 0 || page >= a.c.pages) {
    atomicOr(a.status, kStatRange);
    return 0;
  }
  return page;
}

// Queries that see no key (an empty cache, or positions before the first token): zeros.
// The sequences are dealt to the CTAs; `threads` threads of each call this.
__device__ __forceinline__ void zero_unseeing(const AttnArgs& a, int tid, int threads) {
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    SeqInfo s;
    if (!seq_info(a, b, &s, false)) continue;
    const int cnt = a.causal ? s.c - s.n : (s.n == 0 ? s.c : 0);      // the chunk's first tokens
    const int vecs = a.q_heads * a.c.dim / 8;
    for (int64_t i = tid; i < (int64_t)cnt * vecs; i += threads)
      *reinterpret_cast<uint4*>(a.out + (s.s0 + i / vecs) * a.out_stride + 8 * (i % vecs)) = make_uint4(0u, 0u, 0u, 0u);
    if (a.lse)
      for (int64_t i = tid; i < (int64_t)cnt * a.q_heads; i += threads) a.lse[(int64_t)s.s0 * a.q_heads + i] = -INFINITY;
  }
}

// A CTA per SM; `second`: it may start before the launch in front of it has ended
template <typename Params>
cudaError_t launch_beside(void (*kernel)(Params), const Params& p, int sms, int threads, int smem, bool second,
                          cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = second ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}
// second: right behind the other one, whose CTAs it may run beside (they share nothing)
cudaError_t launch_attn_rows(const AttnArgs& a, int sms, bool second, cudaStream_t s);
int64_t attn_rows_workspace(const KvCache& c, int sms);
cudaError_t launch_attn_chunk(const AttnArgs& a, int sms, bool second, cudaStream_t s);
int64_t attn_chunk_workspace(const KvCache& c, int sms);

}  // namespace qmv
