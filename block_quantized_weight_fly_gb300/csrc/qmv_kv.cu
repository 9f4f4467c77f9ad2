// qmv_kv.cu -- writing rows into a paged KV cache with quantization, and reading rows back.
//
// Write, per K or V row x of D values (fp32 arithmetic, every operation rounded on its own):
//   BF16 : x rounded to nearest even
//   Q8_0 : per 32 values d = min(fp16(amax / 127), 515.5), q = clamp(rint(x / d), -127, 127)
//   FP8  : e4m3(x / s), saturating; s = the cache's static k_scale or v_scale
//   NVFP4: per 16 values b = e4m3(amax / (6 s)), saturating; e2m1(x / (b s)), saturating
// A zero divisor gives zero codes. Infinities saturate; a NaN makes its block (FP8: its
// value) NaN. Read back: q d, e4m3 s, (e2m1 b) s.
//
// Both are bound by memory traffic (2 or 4 bytes and the code bytes per value). A thread
// takes 16 consecutive values: 32 bytes of bf16 are one whole sector per lane, 16 values are
// an NVFP4 block and half a Q8_0 block (one warp shuffle), and the place in the cache is
// worked out once for them. The codes of a warp are whole rows of a group record, so the
// swizzled 8- and 16-byte stores still fill every 32-byte sector they touch.
//
// Quotients: x times the divisor's reciprocal is within 2^-22 of x / divisor, so both round
// to the same code unless a rounding boundary lies between; only a thread with a value that
// close to one divides. That keeps 16 IEEE divisions per thread off the path.
//
// 40001 tokens of 8 heads of 128 bf16 values, us and TB/s: write BF16 61 (5.3), FP8 74 (3.3), Q8_0
// 76 (3.3), NVFP4 84 (2.5); read 57 (5.7), 47 (5.2), 49 (5.1), 43 (4.9). 262144 NVFP4 tokens are
// read in 231 us (5.96), of DRAM's 1.32 GB moved. The quantizing writes are 2.0 to 2.7 times
// their floors and no unit is full: the Q8_0 one issues in 64 % of its cycles (integer pipe 60 %,
// DRAM 3.2 TB/s) from 22 warps an SM, all that its 71 registers leave room for, and a third of
// what passes through L1 is local memory: the parameter arrays indexed by K or V are copied to
// each thread's stack first (128 bytes in the writes, 96 in the reads).
#include "qmv_internal.h"
#include "qmv_attn.cuh"

namespace qmv {

namespace {

constexpr int kKvThreads = 256;

__device__ __forceinline__ uint32_t e4m3_sat(float f) {
  unsigned short v;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(0.0f), "f"(f));
  return v & 0xFFu;
}
// 32 bytes: one access if the place is 32-byte aligned
__device__ __forceinline__ void load32(const void* p, uint32_t* w, bool wide) {
  if (wide) {
    asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4 a = __ldg(static_cast<const uint4*>(p)), b = __ldg(static_cast<const uint4*>(p) + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
}
__device__ __forceinline__ void store32(void* p, const uint32_t* w, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// maximum of |x| over the block a lane's 16 values belong to (LANES neighbouring lanes);
// fmaxf passes NaN over, so `nan` reports one
template <int LANES>
__device__ __forceinline__ float block_amax(const float (&x)[16], bool* nan) {
  float a = 0.0f;
  bool n = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    a = fmaxf(a, fabsf(x[i]));
    n |= x[i] != x[i];
  }
  uint32_t f = n ? 1u : 0u;
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) {
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    f |= __shfl_xor_sync(0xffffffffu, f, o);
  }
  *nan = f != 0u;
  return a;
}

constexpr float kFar = 9.5367431640625e-07f;      // 2^-20: a product with the reciprocal is nearer than that

// reciprocals are used for divisors in a range where neither they nor the products leave fp32
__device__ __forceinline__ bool plain_divisor(float d) { return d > 7.9e-31f && d < 1.2e30f; }

// codes clamp(rint(x / d), +-127) + 128 of 16 values, inv = 1 / d (or 0): the sum with
// 1.5 2^23 rounds to an integer and holds it in its low bits. One value near a half sends
// all 16 through the division.
__device__ __forceinline__ void q8_codes(const float (&x)[16], float d, float inv, uint32_t (&o)[4]) {
  constexpr float kMagic = 12582912.0f;
  float t[16], far = 0.0f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float r = fminf(fmaxf(x[j] * inv, -127.0f), 127.0f);
    t[j] = r + kMagic;
    far = fmaxf(far, fabsf(r - (t[j] - kMagic)));
  }
  if (far > 0.4999f) {
#pragma unroll
    for (int j = 0; j < 16; ++j) t[j] = fminf(fmaxf(rintf(__fdiv_rn(x[j], d)), -127.0f), 127.0f) + kMagic;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t a = __byte_perm(__float_as_uint(t[4 * j]), __float_as_uint(t[4 * j + 1]), 0x0040);
    const uint32_t b = __byte_perm(__float_as_uint(t[4 * j + 2]), __float_as_uint(t[4 * j + 3]), 0x0040);
    o[j] = __byte_perm(a, b, 0x5410) ^ 0x80808080u;
  }
}
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  unsigned short v;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
  return v;
}
__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi) {
  uint32_t v;
  asm("{ .reg .b8 t; cvt.rn.satfinite.e2m1x2.f32 t, %1, %2; cvt.u32.u8 %0, t; }" : "=r"(v) : "f"(hi), "f"(lo));
  return v & 0xFFu;
}
// codes of 16 values over d, a byte (E4M3) or a nibble (E2M1) each, from the low end of o;
// quick: d is a plain divisor. One value near a rounding boundary sends all through the division.
template <bool E4M3>
__device__ __forceinline__ void fp_codes(const float (&x)[16], float d, float inv, bool quick,
                                         uint32_t (&o)[E4M3 ? 4 : 2]) {
  auto pair = [](float a, float b) { return E4M3 ? e4m3_pair(a, b) : e2m1_pair(a, b); };
  uint32_t c[8], differ = quick ? 0u : 1u;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float r0 = x[2 * j] * inv, r1 = x[2 * j + 1] * inv;
    c[j] = pair(fmaf(r0, -kFar, r0), fmaf(r1, -kFar, r1));
    differ |= c[j] ^ pair(fmaf(r0, kFar, r0), fmaf(r1, kFar, r1));
  }
  if (differ) {
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = pair(__fdiv_rn(x[2 * j], d), __fdiv_rn(x[2 * j + 1], d));
  }
  constexpr int B = E4M3 ? 2 : 4;             // pairs per word
#pragma unroll
  for (int j = 0; j < 8 / B; ++j) {
    o[j] = 0u;
#pragma unroll
    for (int q = 0; q < B; ++q) o[j] |= c[B * j + q] << (32 / B * q);
  }
}

// x / d for 0 <= x < 2^31 by a multiplication (Granlund and Montgomery's invariant
// division): m = ceil(2^(31 + L) / d), L = ceil(log2 d)
struct FastDiv {
  uint32_t m, s, d;
};
FastDiv fast_div(uint32_t d) {                // d >= 2
  uint32_t L = 0;
  while ((1ull << L) < d) ++L;
  FastDiv f;
  f.m = (uint32_t)(((1ull << (31 + L)) + d - 1) / d);
  f.s = L - 1;
  f.d = d;
  return f;
}
__device__ __forceinline__ int quotient(int x, const FastDiv& f) { return (int)(__umulhi((uint32_t)x, f.m) >> f.s); }

struct KvWriteParams {
  KvCache c;
  const void* src[2];
  int64_t token_stride[2], head_stride[2];    // in values
  const int64_t* slots;
  int rows;                                   // tokens * 2 * heads
  FastDiv h2;                                 // by 2 * heads
  int chunk_shift;                            // log2(D / 16)
  int wide;                                   // rows start on 32-byte boundaries
  unsigned* status;
};

// the place of row r = (token * 2 + part) * heads + head: its record, or null (skipped)
__device__ __forceinline__ uint8_t* row_part(const KvCache& c, int64_t slot, int part, int head, unsigned* status,
                                             int* tok) {
  if (slot < 0) return nullptr;
  const int64_t page = slot >> c.page_shift;
  if (page >= c.pages) {
    atomicOr(status, kStatRange);
    return nullptr;
  }
  const int t = (int)(slot & ((1 << c.page_shift) - 1));
  *tok = t & 7;
  const int gb = kv_group_bytes(c.fmt, c.dim);
  return c.data + kv_record_off(c, page, head, t, gb) + (part ? gb / 2 : 0);
}

template <int FMT, bool F32, int U>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(const KvWriteParams p) {
  const KvCache& c = p.c;
  uint32_t raw[U][F32 ? 16 : 8];
  int64_t slot[U];
  int part[U], head[U], chunk[U];
  bool in[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = ((int64_t)blockIdx.x * U + u) * kKvThreads + threadIdx.x;
    const int64_t r64 = i >> p.chunk_shift;
    in[u] = r64 < p.rows;
    const int r = in[u] ? (int)r64 : 0;
    const int t = quotient(r, p.h2), hp = r - t * (int)p.h2.d;
    part[u] = hp >= c.heads ? 1 : 0;
    head[u] = hp - part[u] * c.heads;
    chunk[u] = (int)(i & ((1 << p.chunk_shift) - 1));
    slot[u] = __ldg(p.slots + t);
    const int64_t off = (int64_t)t * p.token_stride[part[u]] + (int64_t)head[u] * p.head_stride[part[u]] + 16 * chunk[u];
    if constexpr (F32) {
      load32(static_cast<const float*>(p.src[part[u]]) + off, raw[u], p.wide);
      load32(static_cast<const float*>(p.src[part[u]]) + off + 8, raw[u] + 8, p.wide);
    } else {
      load32(static_cast<const uint16_t*>(p.src[part[u]]) + off, raw[u], p.wide);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float x[16];
#pragma unroll
    for (int j = 0; j < 16; ++j)
      x[j] = F32 ? __uint_as_float(raw[u][F32 ? j : 0])
                 : __uint_as_float((j & 1) ? raw[u][j >> 1] & 0xFFFF0000u : raw[u][j >> 1] << 16);
    int tok = 0;
    uint8_t* dst = in[u] ? row_part(c, slot[u], part[u], head[u], p.status, &tok) : nullptr;
    const int rb = kv_row_bytes(FMT, c.dim), sb = kv_scale_bytes(FMT, c.dim);
    uint8_t* scales = dst + 8 * rb + tok * sb;
    const int ch = chunk[u];
    const float s = part[u] ? c.v_scale : c.k_scale;
    if constexpr (FMT == KV_BF16) {
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = F32 ? bf16_pair(x[2 * j], x[2 * j + 1]) : raw[u][j];
      if (dst) {
        *reinterpret_cast<uint4*>(dst + kv_piece_off(rb, tok, 2 * ch)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(dst + kv_piece_off(rb, tok, 2 * ch + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
      }
    } else if constexpr (FMT == KV_FP8) {
      const float inv = __frcp_rn(s);
      const bool quick = plain_divisor(s);
      uint32_t o[4];
      fp_codes<true>(x, s, inv, quick, o);
      if (dst) *reinterpret_cast<uint4*>(dst + kv_piece_off(rb, tok, ch)) = make_uint4(o[0], o[1], o[2], o[3]);
    } else if constexpr (FMT == KV_Q8_0) {
      bool nan;
      const float amax = block_amax<2>(x, &nan);
      const __half dh = __float2half_rn(fminf(__fdiv_rn(amax, 127.0f), kKvQ8MaxScale));
      const float d = __half2float(dh);
      const float inv = d == 0.0f ? 0.0f : __frcp_rn(d);      // d = 0 or at least 2^-24
      uint32_t o[4];
      q8_codes(x, d, inv, o);
      if (dst) {
        *reinterpret_cast<uint4*>(dst + kv_piece_off(rb, tok, ch)) = make_uint4(o[0], o[1], o[2], o[3]);
        if ((ch & 1) == 0) *reinterpret_cast<unsigned short*>(scales + ch) = nan ? 0x7FFFu : __half_as_ushort(dh);
      }
    } else {
      bool nan;
      const float amax = block_amax<1>(x, &nan);
      const float t6 = __fmul_rn(6.0f, s);
      const uint32_t b = t6 > 0.0f ? e4m3_sat(__fdiv_rn(amax, t6)) : 0u;
      const float den = __fmul_rn(e4m3f(b), s);
      const float inv = __frcp_rn(den);
      const bool quick = plain_divisor(den);
      uint32_t o[2] = {0u, 0u};
      if (den != 0.0f) fp_codes<false>(x, den, inv, quick, o);
      if (dst) {
        *reinterpret_cast<uint2*>(dst + kv_piece_off(rb, tok, ch >> 1) + 8 * (ch & 1)) = make_uint2(o[0], o[1]);
        scales[ch] = (uint8_t)(nan ? 0x7Fu : b);
      }
    }
  }
}

struct KvReadParams {
  KvCache c;
  void* dst[2];
  const int64_t* slots;
  int rows;
  FastDiv h2;
  int chunk_shift;
  int wide;
  unsigned* status;
};

__device__ __forceinline__ float2 half2_floats(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2*>(&h)); }

template <int FMT, bool F32, int U>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const KvReadParams p) {
  const KvCache& c = p.c;
  const int rb = kv_row_bytes(FMT, c.dim), sb = kv_scale_bytes(FMT, c.dim);
  uint32_t code[U][FMT == KV_BF16 ? 8 : FMT == KV_NVFP4 ? 2 : 4];
  uint32_t scale[U];
  int row[U], t[U], hp[U], chunk[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = ((int64_t)blockIdx.x * U + u) * kKvThreads + threadIdx.x;
    const int64_t r64 = i >> p.chunk_shift;
    row[u] = r64 < p.rows ? (int)r64 : -1;
    const int ch = chunk[u] = (int)(i & ((1 << p.chunk_shift) - 1));
    // a skipped slot reads as zeros: code 128 is Q8_0's zero
#pragma unroll
    for (int j = 0; j < (FMT == KV_BF16 ? 8 : FMT == KV_NVFP4 ? 2 : 4); ++j) code[u][j] = FMT == KV_Q8_0 ? 0x80808080u : 0u;
    scale[u] = 0u;
    if (row[u] < 0) continue;
    t[u] = quotient(row[u], p.h2);
    hp[u] = row[u] - t[u] * (int)p.h2.d;
    const int part = hp[u] >= c.heads ? 1 : 0;
    int tok = 0;
    const uint8_t* src = row_part(c, __ldg(p.slots + t[u]), part, hp[u] - part * c.heads, p.status, &tok);
    if (!src) continue;
    const uint8_t* scales = src + 8 * rb + tok * sb;
    if constexpr (FMT == KV_BF16) {
      const uint4 a = *reinterpret_cast<const uint4*>(src + kv_piece_off(rb, tok, 2 * ch));
      const uint4 b = *reinterpret_cast<const uint4*>(src + kv_piece_off(rb, tok, 2 * ch + 1));
      code[u][0] = a.x; code[u][1] = a.y; code[u][2] = a.z; code[u][3] = a.w;
      code[u][4] = b.x; code[u][5] = b.y; code[u][6] = b.z; code[u][7] = b.w;
    } else if constexpr (FMT == KV_NVFP4) {
      const uint2 v = *reinterpret_cast<const uint2*>(src + kv_piece_off(rb, tok, ch >> 1) + 8 * (ch & 1));
      code[u][0] = v.x;
      code[u][1] = v.y;
      scale[u] = scales[ch];
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(src + kv_piece_off(rb, tok, ch));
      code[u][0] = v.x; code[u][1] = v.y; code[u][2] = v.z; code[u][3] = v.w;
      if constexpr (FMT == KV_Q8_0) scale[u] = *reinterpret_cast<const unsigned short*>(scales + (ch & ~1));
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (row[u] < 0) continue;
    const int part = hp[u] >= c.heads ? 1 : 0, head = hp[u] - part * c.heads;
    const float s = part ? c.v_scale : c.k_scale;
    float x[16];
    if constexpr (FMT == KV_BF16) {
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = __uint_as_float((j & 1) ? code[u][j >> 1] & 0xFFFF0000u : code[u][j >> 1] << 16);
    } else if constexpr (FMT == KV_FP8) {
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        const float2 v = half2_floats(e4m3_half(code[u][j >> 2] >> (8 * (j & 2))));
        x[j] = __fmul_rn(v.x, s);
        x[j + 1] = __fmul_rn(v.y, s);
      }
    } else if constexpr (FMT == KV_Q8_0) {
      const float d = h2f(scale[u]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t h[2];
        q8_word(code[u][j], h);
        const float2 a = half2_floats(h[0]), b = half2_floats(h[1]);
        x[4 * j] = __fmul_rn(a.x, d);
        x[4 * j + 1] = __fmul_rn(a.y, d);
        x[4 * j + 2] = __fmul_rn(b.x, d);
        x[4 * j + 3] = __fmul_rn(b.y, d);
      }
    } else {
      // code times block scale is exact in f16
      const uint32_t b = dup_lo(e4m3_half(scale[u]));
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t h[4];
        e2m1_word(code[u][j], h);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 v = half2_floats(h2_mul(h[q], b));
          x[8 * j + 2 * q] = __fmul_rn(v.x, s);
          x[8 * j + 2 * q + 1] = __fmul_rn(v.y, s);
        }
      }
    }
    const int64_t off = ((int64_t)t[u] * c.heads + head) * c.dim + 16 * chunk[u];
    if constexpr (F32) {
      float* o = static_cast<float*>(p.dst[part]) + off;
      store32(o, reinterpret_cast<const uint32_t*>(x), p.wide);
      store32(o + 8, reinterpret_cast<const uint32_t*>(x) + 8, p.wide);
    } else {
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = FMT == KV_BF16 ? code[u][FMT == KV_BF16 ? j : 0] : bf16_pair(x[2 * j], x[2 * j + 1]);
      store32(static_cast<uint16_t*>(p.dst[part]) + off, o, p.wide);
    }
  }
}

int aligned32(const void* p) { return reinterpret_cast<uintptr_t>(p) % 32 == 0 ? 1 : 0; }
int chunk_shift_of(int dim) { return dim == 64 ? 2 : dim == 128 ? 3 : 4; }

// blocks of `items` 16-value items at U per thread
unsigned kv_blocks(int64_t items, int U) { return (unsigned)((items + (int64_t)U * kKvThreads - 1) / (U * kKvThreads)); }

template <template <int, bool, int> class Launch, typename P>
cudaError_t kv_dispatch(const P& p, bool f32, cudaStream_t s) {
  const int sms = num_sms_current_device();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int64_t items = (int64_t)p.rows << p.chunk_shift;
  // two items per thread once that still leaves several blocks per SM: more loads in
  // flight; below it one item per thread, for the shortest path
  const bool two = items >= (int64_t)sms * 8 * 2 * kKvThreads;
  switch (p.c.fmt * 4 + (f32 ? 2 : 0) + (two ? 1 : 0)) {
#define QMV_KV_CASE(F)                                                                   \
  case F * 4 + 0: Launch<F, false, 1>::go(p, kv_blocks(items, 1), s); break;             \
  case F * 4 + 1: Launch<F, false, 2>::go(p, kv_blocks(items, 2), s); break;             \
  case F * 4 + 2: Launch<F, true, 1>::go(p, kv_blocks(items, 1), s); break;              \
  case F * 4 + 3: Launch<F, true, 2>::go(p, kv_blocks(items, 2), s); break;
    QMV_KV_CASE(KV_BF16)
    QMV_KV_CASE(KV_Q8_0)
    QMV_KV_CASE(KV_FP8)
    QMV_KV_CASE(KV_NVFP4)
#undef QMV_KV_CASE
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}
template <int FMT, bool F32, int U>
struct WriteLaunch {
  static void go(const KvWriteParams& p, unsigned blocks, cudaStream_t s) {
    kv_write_kernel<FMT, F32, U><<<blocks, kKvThreads, 0, s>>>(p);
  }
};
template <int FMT, bool F32, int U>
struct ReadLaunch {
  static void go(const KvReadParams& p, unsigned blocks, cudaStream_t s) {
    kv_read_kernel<FMT, F32, U><<<blocks, kKvThreads, 0, s>>>(p);
  }
};

}  // namespace

cudaError_t launch_kv_write(const KvCache& c, const void* k, const void* v, bool f32, const int64_t* strides,
                            const int64_t* slots, int64_t tokens, unsigned* status, cudaStream_t s) {
  KvWriteParams p;
  p.c = c;
  p.src[0] = k;
  p.src[1] = v;
  p.token_stride[0] = strides[0];
  p.head_stride[0] = strides[1];
  p.token_stride[1] = strides[2];
  p.head_stride[1] = strides[3];
  p.slots = slots;
  p.rows = (int)(tokens * 2 * c.heads);
  p.h2 = fast_div((uint32_t)(2 * c.heads));
  p.chunk_shift = chunk_shift_of(c.dim);
  const int64_t size = f32 ? 4 : 2;
  p.wide = aligned32(k) && aligned32(v);
  for (int i = 0; i < 4; ++i) p.wide = p.wide && strides[i] * size % 32 == 0;
  p.status = status;
  return kv_dispatch<WriteLaunch>(p, f32, s);
}

cudaError_t launch_kv_read(const KvCache& c, const int64_t* slots, int64_t tokens, void* k, void* v, bool f32,
                           unsigned* status, cudaStream_t s) {
  KvReadParams p;
  p.c = c;
  p.dst[0] = k;
  p.dst[1] = v;
  p.slots = slots;
  p.rows = (int)(tokens * 2 * c.heads);
  p.h2 = fast_div((uint32_t)(2 * c.heads));
  p.chunk_shift = chunk_shift_of(c.dim);
  p.wide = aligned32(k) && aligned32(v);
  p.status = status;
  return kv_dispatch<ReadLaunch>(p, f32, s);
}

}  // namespace qmv
