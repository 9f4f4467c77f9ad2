// qmv_attn_chunk.cu -- attention of many new tokens over the paged KV cache, on the
// 5th-generation tensor cores. A row is one query head of one new token; the G query heads
// of a KV head share its keys, so a block of rows is QB / G tokens with all their heads.
//
// Work: units (sequence, KV head, block of QB rows), each with its visible key tiles of KT
// tokens, numbered through; each CTA takes one contiguous range of tiles (lengths are
// read on the device), so every SM gets the same number of tiles whatever the batch. A
// unit cut between CTAs leaves its parts (O, maximum, sum) in the workspace; the last CTA
// to arrive adds them in order.
// Roles (one CTA of 512 threads per SM):
//  * producer warp: copies K and V parts of 8-token records with cp.async.bulk;
//  * four converter warps, or eight (D = 256) (quantized caches): codes -> f16 operand tiles in the 128-byte
//    swizzled layout; a BF16 cache's records are such tiles already and are copied
//    straight into the operand ring. In tiles that the mask cuts they also take out values
//    that are not finite (0 x NaN would reach rows that do not see them) and mark their tokens;
//  * MMA warp: S = Q K^T (shared x shared -> tensor memory), O += P V (P from tensor memory);
//  * two softmax warpgroups, a thread per row: S from tensor memory into registers, running
//    maximum and sum in fp32 (base 2), P as 16-bit back over S, O rescaled in tensor memory
//    only when a row's maximum grows by more than 2^8.
// S is formed 64 keys at a time in two buffers per row tile, so the product for the next keys
// runs under the softmax of these; two row tiles of 128 (D <= 128; O of D = 256 fills
// half of tensor memory) share each key and value tile. P takes the place of its S.
// Bound by the tensor cores and, behind them, by the softmax's latency per 64 keys: 2048
// tokens of 64 heads after 28001 FP8 ones (D = 128) take 1363 to 1387 us, 1.42 PFLOP/s; fresh BF16
// prompts of 700 to 6001 tokens 800 us, 1.06 PFLOP/s (half of the last tiles is masked); 8 new
// tokens of 24 heads (D = 256, 48 of 128 rows used) over 15000 Q8_0 ones, five times, 96 us.
// All twelve instances spill 336 to 548 bytes of stores at the launch's 128 registers (the roles'
// shares, which setmaxnreg gives them, change nothing in the code).
#include <type_traits>
#include "qmv_attn.cuh"

namespace qmv {

namespace {

constexpr int kThreads = 512;
constexpr int kSub = 64;               // keys per S tile
// A unit counts as its key tiles plus this many: its queries, its last product and its
// output take about as long, and ranges are cut to be equal in time
constexpr int kUnitCost = 3;           // for key tiles of 128
constexpr int kUnitCostHalf = 8;       // for key tiles of 64
__host__ __device__ constexpr int unit_overhead(int KT) { return KT == 64 ? kUnitCostHalf : kUnitCost; }

template <int FMT, int D>
struct ChunkCfg {
  static constexpr bool BF = FMT == KV_BF16;
  static constexpr int KT = D == 256 ? 64 : 128;             // tokens per key tile
  static constexpr int NQ = D == 256 ? 1 : 2;                // row tiles per block
  static constexpr int QB = 128 * NQ;
  static constexpr int NCW = NQ == 1 ? 8 : 4;                // converter warps: with one row tile, the second warpgroup too
  static constexpr int RB = kv_row_bytes(FMT, D), SB = kv_scale_bytes(FMT, D);
  static constexpr int PART = kv_part_bytes(FMT, D), GB = kv_group_bytes(FMT, D);
  static constexpr int TEAM = NCW / 2;                       // one half of them for keys, one for values
  static constexpr int GROUPS = KT / 8;
  static constexpr int RAW = GROUPS * PART;                  // one part of a tile as stored
  static constexpr int OP = KT * D * 2;                      // ... as operand
  static constexpr int QT = 128 * D * 2;                     // one row tile of queries
  static constexpr int CTRL = 1024;
  static constexpr int ROOM = 232448 - 512 - 1024 - CTRL - NQ * QT;   // 512: static, 1024: alignment
  static constexpr int NOP = BF ? (ROOM / OP > 6 ? 6 : ROOM / OP) : (D == 64 ? 4 : 3);
  static constexpr int RAWPAD = (RAW + 127) / 128 * 128;
  static constexpr int NRAW0 = (ROOM - NOP * OP) / RAWPAD;
  static constexpr int NRAW = BF ? 1 : (NRAW0 > 4 ? 4 : NRAW0);
  static constexpr int SMEM = CTRL + NQ * QT + NOP * OP + (BF ? 0 : NRAW * RAWPAD) + 1024;
  static constexpr int GRP = 16 * D;                         // bytes of 8 operand rows
};

// Operand descriptors (128-byte swizzle, version 1) as two words: the low one holds the
// address and the leading byte offset, so a step is one 32-bit addition; the high one (stride
// between groups of 8 rows) is a constant. `on` predicates the instruction: the whole warp
// runs the issuing code, which keeps its operands in uniform registers (in a branch that one
// lane takes, moving five operands over per instruction held the tensor cores at 40 %).
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
  return ((addr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}
constexpr uint32_t desc_hi(uint32_t sbo) { return (sbo >> 4) | (1u << 14) | (2u << 29); }
template <uint32_t HA, uint32_t HB, uint32_t ID, bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t on) {
  asm volatile(
      "{ .reg .pred q, c; .reg .b64 x, y; setp.ne.b32 q, %3, 0; setp.ne.b32 c, %7, 0;\n"
      "mov.b64 x, {%1, %4}; mov.b64 y, {%2, %5};\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %6, c; }" ::"r"(d), "r"(a), "r"(b), "r"(on), "n"(HA), "n"(HB),
      "n"(ID), "n"(ACC ? 1 : 0)
      : "memory");
}
template <uint32_t HB, uint32_t ID>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t acc, uint32_t on) {
  asm volatile(
      "{ .reg .pred q, c; .reg .b64 y; setp.ne.b32 q, %3, 0; setp.ne.b32 c, %6, 0;\n"
      "mov.b64 y, {%2, %4};\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %5, c; }" ::"r"(d), "r"(a), "r"(b), "r"(on), "n"(HB),
      "n"(ID), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar, uint32_t on) {
  asm volatile(
      "{ .reg .pred q; setp.ne.b32 q, %1, 0;\n"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(bar), "r"(on)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
  return r;
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
#define QMV_R32(r, o)                                                                                              \
  "=r"(r[o + 0]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), "=r"(r[o + 6]),  \
      "=r"(r[o + 7]), "=r"(r[o + 8]), "=r"(r[o + 9]), "=r"(r[o + 10]), "=r"(r[o + 11]), "=r"(r[o + 12]),           \
      "=r"(r[o + 13]), "=r"(r[o + 14]), "=r"(r[o + 15]), "=r"(r[o + 16]), "=r"(r[o + 17]), "=r"(r[o + 18]),        \
      "=r"(r[o + 19]), "=r"(r[o + 20]), "=r"(r[o + 21]), "=r"(r[o + 22]), "=r"(r[o + 23]), "=r"(r[o + 24]),        \
      "=r"(r[o + 25]), "=r"(r[o + 26]), "=r"(r[o + 27]), "=r"(r[o + 28]), "=r"(r[o + 29]), "=r"(r[o + 30]),        \
      "=r"(r[o + 31])
template <int O, int N>
__device__ __forceinline__ void tm_load32(uint32_t (&r)[N], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : QMV_R32(r, O)
      : "r"(addr));
}
__device__ __forceinline__ void tm_load16(uint32_t (&r)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tm_store16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tm_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void to_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 32 bytes of a row: one whole sector per lane if the place is 32-byte aligned
__device__ __forceinline__ void store_pair(uint8_t* dst, const uint4 (&x)[2], bool wide) {
  if (wide)
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(x[0].x), "r"(x[0].y), "r"(x[0].z),
                 "r"(x[0].w), "r"(x[1].x), "r"(x[1].y), "r"(x[1].z), "r"(x[1].w)
                 : "memory");
  else {
    reinterpret_cast<uint4*>(dst)[0] = x[0];
    reinterpret_cast<uint4*>(dst)[1] = x[1];
  }
}

// two fp32 operations in one instruction; the larger of three
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{ .reg .b64 x, y, z, w; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%6, %7};\n"
      "fma.rn.f32x2 w, x, y, z; mov.b64 {%0, %1}, w; }"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{ .reg .b64 x, y, w; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5};\n"
      "add.rn.f32x2 w, x, y; mov.b64 {%0, %1}, w; }"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

struct ChunkParams {
  AttnArgs a;
  unsigned* counters;        // [grid][2]: parts arrived of the row tiles that CTA i leaves unfinished
  float* parts;              // [2 grid][QB (D + 2)]
};

// One unit, and where its key tiles lie.
struct Unit {
  int b, h, qb, nqb;         // sequence, head, block of rows and their number
  SeqInfo s;
  int tile0, nt, hi;         // first key tile, key tiles, last key that a row sees
  int org;                   // place of its first key tile in the CTA's range (may be negative)
  int k;                     // first tile of the CTA's part
};
template <int KT, int QB>
__device__ __forceinline__ void unit_range(const AttnArgs& a, const SeqInfo& s, int G, int qb, int* tile0, int* nt,
                                           int* last) {
  const BlockRange r = block_range<KT, QB>(s.n, s.c, G, qb, a.causal, a.window);
  *tile0 = r.tile0;
  *nt = r.nt;
  *last = r.last;
}
// the numbered tiles of one head's blocks, in every lane of the warp
template <int KT, int QB>
__device__ __forceinline__ int64_t head_cost(const AttnArgs& a, const SeqInfo& s, int G, int nqb, int lane) {
  int64_t sum = blocks_cost<KT, QB>(s.n, s.c, G, nqb, lane, a.causal, a.window, unit_overhead(KT));
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}
template <int KT, int QB>
__device__ __forceinline__ void unit_seq(const AttnArgs& a, Unit& u, int G) {
  seq_info(a, u.b, &u.s, false);
  u.nqb = u.s.c * G > a.few_rows ? (u.s.c * G + QB - 1) / QB : 0;
}
// a part of this unit is in the range, and so is one of the next
__device__ __forceinline__ bool unit_here(const Unit& u, int len) { return u.org + u.k < len; }
template <int KT>
__device__ __forceinline__ bool unit_after(const Unit& u, int len) { return u.org + u.nt + unit_overhead(KT) < len; }
// one past the last tile of the CTA's part
__device__ __forceinline__ int unit_end(const Unit& u, int len) { return u.nt < len - u.org ? u.nt : len - u.org; }
// S tiles of the part: the last key tile's second half may hold no key that is seen
template <int KT>
__device__ __forceinline__ int unit_subs(const Unit& u, int kend) {
  if (KT == kSub) return kend - u.k;
  return 2 * (kend - u.k) - (kend == u.nt && ((u.hi / kSub) & 1) == 0 ? 1 : 0);
}
// the next unit with a tile. The caller knows that there is one (unit_after)
template <int KT, int QB>
__device__ __forceinline__ void unit_next(const AttnArgs& a, Unit& u, int G) {
  u.org += u.nt + unit_overhead(KT);
  do {
    if (++u.qb >= u.nqb) {
      u.qb = 0;
      if (++u.h >= a.c.heads) {
        u.h = 0;
        do {
          ++u.b;
          unit_seq<KT, QB>(a, u, G);
        } while (u.nqb == 0 && u.b + 1 < a.B);
      }
    }
    u.nt = 0;
    if (u.nqb > 0) unit_range<KT, QB>(a, u.s, G, u.qb, &u.tile0, &u.nt, &u.hi);
  } while (u.nt == 0 && (u.b + 1 < a.B || u.h + 1 < a.c.heads || u.qb + 1 < u.nqb));
  u.k = 0;
}
// Keys lo .. hi are seen by every row of the block: a key tile is cut by the mask (an edge)
// if it reaches outside.
struct Full {
  int lo, hi;
  __device__ bool edge(int j0, int tokens) const { return j0 + tokens - 1 > hi || j0 < lo; }
};
template <int QB>
__device__ __forceinline__ Full unit_full(const AttnArgs& a, const Unit& u, int G) {
  const BlockRange r = block_range<kSub, QB>(u.s.n, u.s.c, G, u.qb, a.causal, a.window);
  Full f;
  f.hi = a.causal ? r.first_pos : u.s.n - 1;
  f.lo = window_first(r.last_pos, a.window);
  return f;
}

// 16 bytes of codes -> f16 operands, VPP / 8 pieces of 8 values
template <int FMT>
__device__ __forceinline__ void convert_piece(uint4 code, uint32_t scale, uint32_t (&o)[16]) {
  const uint32_t w[4] = {code.x, code.y, code.z, code.w};
  if constexpr (FMT == KV_FP8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) e4m3_word(w[i], o + 2 * i);
  } else if constexpr (FMT == KV_Q8_0) {
    const uint32_t d = dup_lo(scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q8_word(w[i], o + 2 * i);
      o[2 * i] = h2_mul(o[2 * i], d);
      o[2 * i + 1] = h2_mul(o[2 * i + 1], d);
    }
  } else {
    const uint32_t s = e4m3_half(scale);
    const uint32_t d[2] = {dup_lo(s), dup_hi(s)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      e2m1_word(w[i], o + 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[4 * i + e] = h2_mul(o[4 * i + e], d[i >> 1]);
    }
  }
}
// zero the values of 8 (four words) that are not finite; true if there was one
template <bool BF>
__device__ __forceinline__ bool clean8(uint32_t* o) {
  constexpr uint32_t E = BF ? 0x7F80u : 0x7C00u;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = o[i];
    if ((x & E) == E) {
      o[i] &= 0xFFFF0000u;
      bad = true;
    }
    if ((x & (E << 16)) == (E << 16)) {
      o[i] &= 0x0000FFFFu;
      bad = true;
    }
  }
  return bad;
}

// One part (keys or values) of a tile, codes -> operand rows; warp cw of TEAM. The loads of
// a batch come before its stores: the two may alias as far as the compiler knows, and
// piece by piece each load waited for the stores before it (1500 cycles per part, against
// 620). EDGE: values that are not finite are taken out, their tokens marked.
template <int FMT, int D, bool EDGE>
__device__ __forceinline__ void convert_part(const uint8_t* raw, uint8_t* op, uint32_t* poison, int cw, int lane) {
  using C = ChunkCfg<FMT, D>;
  constexpr int NP = C::RB / 16;                               // pieces per token
  constexpr int NO = FMT == KV_NVFP4 ? 4 : 2;                  // operand pieces per piece
  constexpr int STEPS = C::KT * NP / (32 * C::TEAM);           // pieces per thread
  constexpr int BATCH = STEPS < 8 ? STEPS : 8;
#pragma unroll
  for (int i0 = 0; i0 < STEPS; i0 += BATCH) {
    uint4 code[BATCH];
    uint32_t sc[BATCH];
    int grp[BATCH], t[BATCH], pc[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int x = ((i0 + i) * C::TEAM + cw) * 32 + lane;     // piece of the tile
      if constexpr (NP >= 8) {
        t[i] = x & 7;
        pc[i] = (x >> 3) % NP;
        grp[i] = (x >> 3) / NP;
      } else {
        pc[i] = x % NP;
        t[i] = (x / NP) & 7;
        grp[i] = x / (8 * NP);
      }
      const uint8_t* rec = raw + grp[i] * C::PART;
      code[i] = *reinterpret_cast<const uint4*>(rec + kv_piece_off(C::RB, t[i], pc[i]));
      sc[i] = 0u;
      if constexpr (FMT == KV_Q8_0)
        sc[i] = *reinterpret_cast<const unsigned short*>(rec + 8 * C::RB + t[i] * C::SB + 2 * (pc[i] >> 1));
      if constexpr (FMT == KV_NVFP4)
        sc[i] = *reinterpret_cast<const unsigned short*>(rec + 8 * C::RB + t[i] * C::SB + 2 * pc[i]);
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      uint32_t o[16];
      convert_piece<FMT>(code[i], sc[i], o);
      if constexpr (EDGE) {
        bool bad = false;
#pragma unroll
        for (int e = 0; e < NO; ++e) bad |= clean8<false>(o + 4 * e);
        if (bad) atomicOr(poison + ((grp[i] * 8 + t[i]) >> 5), 1u << ((grp[i] * 8 + t[i]) & 31));
      }
#pragma unroll
      for (int e = 0; e < NO; ++e)
        *reinterpret_cast<uint4*>(op + grp[i] * C::GRP + kv_piece_off(2 * D, t[i], pc[i] * NO + e)) =
            make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
    }
  }
}

template <int FMT, int D>
__global__ void __launch_bounds__(kThreads, 1) attn_chunk_kernel(const ChunkParams p) {
  using C = ChunkCfg<FMT, D>;
  constexpr int KT = C::KT, QB = C::QB, NQ = C::NQ;
  constexpr bool BF = C::BF;
  const AttnArgs& a = p.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* const qtile = smem;                               // [NQ][QT]
  uint8_t* const ops = qtile + NQ * C::QT;                   // [NOP][OP]
  uint8_t* const raws = ops + C::NOP * C::OP;                // [NRAW][RAWPAD]
  uint8_t* const ctrl = raws + (BF ? 0 : C::NRAW * C::RAWPAD);
  __shared__ int64_t s_first[2];
  __shared__ int64_t s_wsum[kThreads / 32];
  __shared__ uint32_t s_poison[8][4];                        // per tile (mod 8): its tokens with a non-finite value
  __shared__ uint32_t s_tmem;
  __shared__ int s_last[2];
  int64_t* const s_sum = reinterpret_cast<int64_t*>(qtile);  // [kThreads], while the work is laid out
  // barriers
  const uint32_t bar = smem_u32(ctrl);
  const uint32_t raw_full = bar, raw_empty = raw_full + 8 * C::NRAW, op_full = raw_empty + 8 * C::NRAW,
                 op_done = op_full + 8 * C::NOP, op_fix = op_done + 64, q_ready = op_fix + 32,
                 s_full = q_ready + 16, p_ready = s_full + 32, o_done = p_ready + 32, joined = o_done + 16,
                 all_done = joined + 16, marked = all_done + 8;
  // s_full, p_ready: [row tile][S buffer]. op_done: [keys, values][tile % 4], the products of
  // a tile are complete: a slot's last occupant may be of the other kind, so its release is
  // told by tile, and no waiter is four tiles from a barrier's phase
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.q_heads / a.c.heads;
  let_next_start();
  // the barrier, and its phase, that frees the slot of use m (K0 V0 K1 V1 ...)
  auto op_free = [&](int m) { return op_done + 32u * (m & 1) + 8u * ((m >> 1) & 3); };
  auto op_free_parity = [](int m) { return (uint32_t)((m >> 3) & 1); };
  if (tid == 0) {
    for (int i = 0; i < C::NRAW; ++i) {
      bar_init(raw_full + 8 * i, 1);
      bar_init(raw_empty + 8 * i, C::TEAM);
    }
    for (int i = 0; i < C::NOP; ++i) {
      bar_init(op_full + 8 * i, BF ? 1 : C::TEAM);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(q_ready + 8 * i, 4);
      bar_init(o_done + 8 * i, 1);
      bar_init(joined + 8 * i, 4);
    }
    for (int i = 0; i < 4; ++i) {
      bar_init(s_full + 8 * i, 1);
      bar_init(p_ready + 8 * i, 4);
      bar_init(op_fix + 8 * i, C::NCW);
      bar_init(op_done + 8 * i, 1);
      bar_init(op_done + 32 + 8 * i, 1);
    }
    bar_init(all_done, 1);
    bar_init(marked, 4);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid < 32) s_poison[tid >> 2][tid & 3] = 0u;
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }

  // ---- the numbered tiles: a warp sums a sequence's blocks, two passes over windows of
  // sequences find the total and this CTA's first unit --------------------------------------
  int64_t total = 0, w0 = 0, w1 = 0, per = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int64_t base = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
      const int cnt = a.B - b0 < kThreads ? a.B - b0 : kThreads;
      for (int i = warp; i < kThreads; i += kThreads / 32) {
        int64_t sum = 0;
        if (i < cnt) {
          SeqInfo s;
          seq_info(a, b0 + i, &s, pass == 0 && blockIdx.x == 0 && lane == 0);
          const int nqb = s.c * G > a.few_rows ? (s.c * G + QB - 1) / QB : 0;
          sum = head_cost<KT, QB>(a, s, G, nqb, lane);
        }
        if (lane == 0) s_sum[i] = sum;
      }
      __syncthreads();
      const int64_t mine = s_sum[tid] * a.c.heads;
      int64_t scan = mine;
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += v;
      }
      if (lane == 31) s_wsum[warp] = scan;
      __syncthreads();
      int64_t before = 0, all = 0;
      for (int i = 0; i < kThreads / 32; ++i) {
        if (i < warp) before += s_wsum[i];
        all += s_wsum[i];
      }
      if (pass == 1) {
        const int64_t lo = base + before + scan - mine;
        if (w0 >= lo && w0 < lo + mine) {
          s_first[0] = b0 + tid;
          s_first[1] = w0 - lo;
        }
      }
      base += all;
      __syncthreads();
    }
    if (pass == 0) {
      total = base;
      per = place_div(total + gridDim.x - 1, gridDim.x);
      if (per < unit_overhead(KT) + 2) per = unit_overhead(KT) + 2;
      if (per > kMostPlaces) {
        if (blockIdx.x == 0 && tid == 0) atomicOr(a.status, kStatRange);
        total = 0;
      }
      w0 = (int64_t)blockIdx.x * per;
      w1 = w0 + per < total ? w0 + per : total;
    }
  }
  zero_unseeing(a, tid, kThreads);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = s_tmem;
  const int len = (int)(w1 > w0 ? w1 - w0 : 0);
  bool work = len > 0;
  Unit first;
  if (work) {
    first.b = (int)s_first[0];
    unit_seq<KT, QB>(a, first, G);
    // head and block: tiles of one head's blocks, in turn
    const int64_t per_head = head_cost<KT, QB>(a, first.s, G, first.nqb, lane);
    first.h = (int)place_div(s_first[1], per_head);
    int64_t rest = s_first[1] - first.h * per_head;
    first.qb = 0;
    for (int qb = 0; qb < first.nqb; qb += 32) {
      const int cost = qb + lane < first.nqb ? block_cost<KT, QB>(first.s.n, first.s.c, G, qb + lane, a.causal, a.window,
                                                                  unit_overhead(KT)) : 0;
      int scan = cost;                                           // of 32 blocks: below 2^31
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += v;
      }
      const int all = __shfl_sync(0xffffffffu, scan, 31);
      if (rest < all) {
        const uint32_t hit = __ballot_sync(0xffffffffu, scan > rest);
        const int l = __ffs(hit) - 1;
        first.qb = qb + l;
        rest -= __shfl_sync(0xffffffffu, scan - cost, l);
        break;
      }
      rest -= all;
    }
    unit_range<KT, QB>(a, first.s, G, first.qb, &first.tile0, &first.nt, &first.hi);
    first.org = unit_overhead(KT) - (int)rest;
    first.k = first.org < 0 ? -first.org : 0;
    work = unit_here(first, len);
  }

  // Registers by warpgroup, within the launch's 4 x 128: softmax 160 + 160 (one row tile:
  // 208, and 104 more for converters), converters 104, MMA and producer 88
  if (warp >= 12) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  if (work && warp == 13) {
    // ------------------------------ producer ----------------------------------------------
    Unit u = first;
    int st = 0, issued = 0;
    uint32_t ph = 0;
    bool ok = true;
    const int page_mask = (1 << a.c.page_shift) - 1;
    const int64_t page_bytes = (int64_t)C::GB << (a.c.page_shift - 3);   // of one head
    // lane i < GROUPS: token group i of the tile; its page is looked up a tile ahead
    // (groups that no query of the sequence sees are not copied: their pages may be gone)
    int tok = 0, page = 0;
    bool wanted = false;
    auto look = [&](const Unit& v, int k) {
      tok = (v.tile0 + k) * KT + 8 * lane;
      wanted = lane < C::GROUPS && tok < v.s.n && tok + 8 > seq_first(a, v.s);
      if (wanted)
        page = __ldg(a.table + (int64_t)v.b * a.max_pages + (tok >> a.c.page_shift));
    };
    look(u, u.k);
    for (;;) {
      const int kend = unit_end(u, len), head = u.h;
      const bool after = unit_after<KT>(u, len);
      for (int k = u.k; k < kend && ok; ++k) {
        const bool have = wanted;
        const uint8_t* src = a.c.data;
        if (have)
          src += ((int64_t)checked_page(a, page) * a.c.heads + head) * page_bytes + (int64_t)((tok & page_mask) >> 3) * C::GB;
        const int groups = __popc(__ballot_sync(0xffffffffu, have));
        if (k + 1 < kend) look(u, k + 1);
        for (int part = 0; part < 2 && ok; ++part) {
          const int N = BF ? C::NOP : C::NRAW;
          const uint32_t full = (BF ? op_full : raw_full) + 8 * st;
          if (issued >= N) ok = BF ? bar_wait(op_free(issued - N), op_free_parity(issued - N)) : bar_wait(raw_empty + 8 * st, ph ^ 1u);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) bar_expect(full, groups * C::PART);
          __syncwarp();
          if (have)
            bulk_copy(smem_u32(BF ? ops + st * C::OP : raws + st * C::RAWPAD) + lane * C::PART, src + part * C::PART,
                      C::PART, full);
          ++issued;
          if (++st == N) {
            st = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok || !after) break;
      unit_next<KT, QB>(a, u, G);
      look(u, 0);
    }
    if (!ok && lane == 0) atomicOr(a.status, kStatTimeout);
    // copies in flight land before the CTA can leave
    const int N = BF ? C::NOP : C::NRAW;
    for (int i = issued > N ? issued - N : 0; i < issued; ++i)
      (void)bar_wait((BF ? op_full : raw_full) + 8 * (i % N), (uint32_t)((i / N) & 1));
  } else if (work && warp == 12) {
    // ------------------------------ MMA warp: all lanes run, one issues ------------------------
    constexpr uint32_t fm = BF ? ((1u << 7) | (1u << 10)) : 0u;
    constexpr uint32_t id_s = (1u << 4) | fm | ((uint32_t)(kSub >> 3) << 17) | (8u << 24);
    constexpr uint32_t id_o = (1u << 4) | fm | (1u << 16) | ((uint32_t)(D >> 3) << 17) | (8u << 24);
    constexpr uint32_t hi = desc_hi(C::GRP);
    const uint32_t on = elect_one();
    const uint32_t tm = (uint32_t)uniform((int)tmem);
    const uint32_t qa = desc_lo(smem_u32(qtile), 16), ka = desc_lo(smem_u32(ops), 16),
                   va = desc_lo(smem_u32(ops), 1024);
    Unit u = first;
    // the operand ring: slots in the order K0 V0 K1 V1 ...; kslot, vslot: of the next K and V
    int kslot = 0, vslot = 1;
    uint32_t kph = 0, vph = 0, ktile = 0, vtile = 0, fixes = 0;
    uint32_t nq0 = 0, nq1 = 0, p0[2] = {0, 0}, p1[2] = {0, 0};         // phases of the Q and P barriers
    bool ok = true;
    auto next2 = [](int& slot, uint32_t& phase, uint32_t& tile) {
      ++tile;
      slot += 2;
      if (slot >= C::NOP) {
        slot -= C::NOP;
        phase ^= 1u;
      }
    };
    auto wait_k = [&]() { ok = ok && bar_wait(op_full + 8 * kslot, kph); };
    auto wait_v = [&]() {
      ok = ok && bar_wait(op_full + 8 * vslot, vph);
      // a BF16 values tile passes the converters, which clean it where the mask cuts
      if (BF) {
        ok = ok && bar_wait(op_fix + 8 * (fixes & 3u), (fixes >> 2) & 1u);
        ++fixes;
      }
    };
    auto scores = [&](int w, int buf, int sub) {               // S[w][buf] = Q[w] K^T, 64 keys
      const uint32_t kb = ka + (uint32_t)(kslot * (C::OP >> 4) + sub * (8 * C::GRP >> 4));
      const uint32_t qb = qa + (uint32_t)(w * (C::QT >> 4)), d = tm + (uint32_t)(128 * w + 64 * buf);
      mma_ss<hi, hi, id_s, false>(d, qb, kb, on);
#pragma unroll
      for (int e = 1; e < D / 16; ++e) {
        const uint32_t off = (uint32_t)((e >> 2) * 64 + (e & 3) * 2);
        mma_ss<hi, hi, id_s, true>(d, qb + off, kb + off, on);
      }
      mma_commit(s_full + 16 * w + 8 * buf, on);
    };
    auto values = [&](int w, int buf, int sub, uint32_t acc) {           // O[w] += P[w][buf] V, 64 keys
      const uint32_t vb = va + (uint32_t)(vslot * (C::OP >> 4) + sub * (8 * C::GRP >> 4));
      const uint32_t d = tm + 256u + (uint32_t)(w * D), pa = tm + (uint32_t)(128 * w + 64 * buf);
#pragma unroll
      for (int e = 0; e < kSub / 16; ++e)
        mma_ts<hi, id_o>(d, pa + 8u * e, vb + (uint32_t)(e * (2 * C::GRP >> 4)), e ? 1u : acc, on);
      mma_commit(o_done + 8 * w, on);
    };
    auto wait_on = [&](uint32_t bar, uint32_t& phase) {
      ok = ok && bar_wait(bar, phase & 1u);
      ++phase;
    };
    auto settle = [&]() {
      ok = __all_sync(0xffffffffu, ok);
      if (ok) tc_after();
      return ok;
    };
    for (;;) {
      // S tiles j of the part: S of tile j + 1 is formed while the softmax works on tile j
      const int n = uniform(unit_subs<KT>(u, unit_end(u, len)));
      const bool pair = NQ == 2 && uniform(u.s.c * G - u.qb * QB) > 128;
      wait_on(q_ready, nq0);
      if (pair) wait_on(q_ready + 8, nq1);
      wait_k();
      if (!settle()) break;
      scores(0, 0, 0);
      if (pair) scores(1, 0, 0);
      if (KT == kSub || n == 1) {
        mma_commit(op_done + 8 * (ktile & 3u), on);
        next2(kslot, kph, ktile);
      }
      for (int j = 0; j < n; j += 2) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {          // tile j + x: S buffer x, half x of a 128-key tile
          if (x == 1 && j + 1 >= n) break;
          const bool next = j + x + 1 < n;
          auto form_next = [&]() -> bool {     // S of tile j + x + 1
            if (KT == kSub || x == 1) wait_k();
            if (!settle()) return false;
            scores(0, x ^ 1, KT == kSub ? 0 : x ^ 1);
            if (pair) scores(1, x ^ 1, KT == kSub ? 0 : x ^ 1);
            if (KT == kSub || x == 0 || j + x + 2 == n) {
              mma_commit(op_done + 8 * (ktile & 3u), on);
              next2(kslot, kph, ktile);
            }
            return true;
          };
          // With three slots of one S tile each, the next keys wait for the slot of the values
          // before these: if P is there first, its product goes first
          bool late = false;
          if (next && KT == kSub && C::NOP == 3) {
            for (uint32_t it = 0; it < 100000u; ++it) {
              const bool kk = bar_test(op_full + 8 * kslot, kph);
              const bool pv = bar_test(op_full + 8 * vslot, vph) && bar_test(p_ready + 8 * x, p0[x] & 1u);
              if (uniform(kk)) break;
              if (uniform(pv)) {
                late = true;
                break;
              }
            }
          }
          if (next && !late && !form_next()) break;
          if (KT == kSub || x == 0) wait_v();
          wait_on(p_ready + 8 * x, p0[x]);
          if (!settle()) break;
          values(0, x, KT == kSub ? 0 : x, j + x ? 1u : 0u);
          if (pair) {
            wait_on(p_ready + 16 + 8 * x, p1[x]);
            if (!settle()) break;
            values(1, x, KT == kSub ? 0 : x, j + x ? 1u : 0u);
          }
          if (KT == kSub || x == 1 || !next) {
            mma_commit(op_done + 32 + 8 * (vtile & 3u), on);
            next2(vslot, vph, vtile);
          }
          if (late && !form_next()) break;
        }
        if (!ok) break;
      }
      if (!ok || !uniform(unit_after<KT>(u, len))) break;
      unit_next<KT, QB>(a, u, G);
    }
    if (!ok && lane == 0) atomicOr(a.status, kStatTimeout);
    mma_commit(all_done, on);                                  // when every MMA issued above has completed
    (void)bar_wait(all_done, 0u);
    __syncwarp();
  }
  } else if (warp >= 12 - C::NCW) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
  if (work) {
    // ------------------------------ converters ----------------------------------------------
    const int cw = warp - (12 - C::NCW);
    Unit u = first;
    int use = 0;
    uint32_t tileno = 0;
    bool ok = true;
    for (;;) {
      const int kend = unit_end(u, len);
      const Full full = unit_full<QB>(a, u, G);
      for (int k = u.k; k < kend && ok; ++k, ++tileno) {
        const bool edge = full.edge((u.tile0 + k) * KT, KT);
        uint32_t* poison = s_poison[tileno & 7];
        if constexpr (BF) {
          const int vu = use + 1;
          // The slot's release first, as the producer waits for it. With five slots its last
          // occupant was a keys tile, whose arrival no converter has seen: while that copy is under
          // way, the parity of the phase after it looks like a completed one, and a warp would
          // run ahead of its tiles, past a phase of op_fix that others have yet to arrive at
          if (vu >= C::NOP) ok = bar_wait(op_free(vu - C::NOP), op_free_parity(vu - C::NOP));
          ok = ok && bar_wait(op_full + 8 * (vu % C::NOP), (uint32_t)((vu / C::NOP) & 1));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (edge) {
            // warp cw: tokens 32 cw .. 32 cw + 31 (KT = 64: warps 0, 1)
            if (32 * cw < KT) {
              uint32_t bad = 0u;
              uint8_t* tile = ops + (vu % C::NOP) * C::OP;
              const int t = 32 * cw + lane;
#pragma unroll 4
              for (int pc = 0; pc < D / 8; ++pc) {
                uint4* q = reinterpret_cast<uint4*>(tile + (t >> 3) * C::GRP + kv_piece_off(2 * D, t & 7, pc));
                uint4 v = *q;
                uint32_t o[4] = {v.x, v.y, v.z, v.w};
                if (clean8<true>(o)) {
                  *q = make_uint4(o[0], o[1], o[2], o[3]);
                  bad = 1u;
                }
              }
              const uint32_t word = __ballot_sync(0xffffffffu, bad != 0u);
              if (lane == 0) poison[cw] = word;
            }
            to_async_proxy();
            __syncwarp();
          }
          if (lane == 0) bar_arrive(op_fix + 8 * ((vu >> 1) & 3));
          use += 2;
        } else {
          // the marks of the tile after the next start clean (their last use is six tiles back)
          if (cw == 0 && lane == 0) {
#pragma unroll
            for (int q = 0; q < 4; ++q) s_poison[(tileno + 2) & 7][q] = 0u;
          }
          // keys and values are converted side by side: a part's waits and fences take as long
          // as its conversion
          const int part = cw / C::TEAM, mine = use + part, rs = mine % C::NRAW, os = mine % C::NOP;
          // the slot first: with three slots and three raw stages, its last occupant's release
          // also shows that the stage's last phase, the other team's, is over
          static_assert(C::NRAW % 2 == 0 || (C::NRAW == 3 && C::NOP == 3), "a team's raw stages");
          if (mine >= C::NOP) ok = bar_wait(op_free(mine - C::NOP), op_free_parity(mine - C::NOP));
          ok = ok && bar_wait(raw_full + 8 * rs, (uint32_t)((mine / C::NRAW) & 1));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (part == 1 && edge)
            convert_part<FMT, D, true>(raws + rs * C::RAWPAD, ops + os * C::OP, poison, cw % C::TEAM, lane);
          else
            convert_part<FMT, D, false>(raws + rs * C::RAWPAD, ops + os * C::OP, poison, cw % C::TEAM, lane);
          to_async_proxy();
          __syncwarp();
          if (lane == 0) {
            bar_arrive(op_full + 8 * os);
            bar_arrive(raw_empty + 8 * rs);
          }
          use += 2;
        }
      }
      if (!ok || !unit_after<KT>(u, len)) break;
      unit_next<KT, QB>(a, u, G);
    }
    if (!ok && lane == 0) atomicOr(a.status, kStatTimeout);
  }
  } else {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(NQ == 1 ? 208 : 160));
  if (work && warp < 4 * NQ) {
    // ------------------------------ softmax: a thread per row ----------------------------------
    const int w = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t oT = tmem + 256u + (uint32_t)(w * D) + lanes;
    constexpr int PP = D / 8, RPI = 32 / PP == 0 ? 1 : 32 / PP;          // pieces per row, rows per instruction
    uint8_t* const wtile = qtile + w * C::QT + (warp & 3) * 4 * C::GRP;  // this warp's 32 rows of the query tile
    Unit u = first;
    uint32_t n_even = 0, n_odd = 0, nd = 0, nj = 0, nm = 0;   // phases of the two S barriers, O, joins, marks
    bool marks_due = false;
    uint32_t tileno = 0;
    bool ok = true;
    // The queries of a unit's 32 rows into the operand tile (free once the last S of the unit
    // before is there), a row (or two, four) per load, four loads under way beside four in work: unrolled
    // further, code that runs once per unit would cost more in instruction fetches than
    // the loads' latency. f16 operands are scaled by a power of two per row; the sign of the
    // softmax scale goes in here, so that rf, which takes S to base-2 logits, is positive
    float rf_next = 0.0f;
    auto queries = [&](const Unit& v) {
      const int r = v.qb * QB + 128 * w + row;
      const uint64_t mine = (uint64_t)(r < v.s.c * G ? a.q + (int64_t)(v.s.s0 + r / G) * a.q_stride +
                                                           (int64_t)(v.h * G + r % G) * D
                                                     : nullptr);
      const float sgn = a.scale > 0.f ? 1.f : a.scale < 0.f ? -1.f : 0.f;
      float inv = 1.0f;
      uint4 nx[4];
      auto load = [&](int i0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t src = __shfl_sync(0xffffffffu, mine, ((i0 + i) * RPI + lane / PP) & 31);
          nx[i] = make_uint4(0u, 0u, 0u, 0u);
          if (src) nx[i] = __ldg(reinterpret_cast<const uint4*>(src) + lane % PP);
        }
      };
      load(0);
#pragma unroll 1
      for (int i0 = 0; i0 < PP; i0 += 4) {
        uint4 qv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) qv[i] = nx[i];
        if (i0 + 4 < PP) load(i0 + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t x[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
          float mul = sgn;
          if constexpr (!BF) {
            float amax = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              amax = max3(amax, fabsf(bf2f(x[e])), fabsf(__uint_as_float(x[e] & 0xFFFF0000u)));
#pragma unroll
            for (int o = 1; o < PP; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            float back;
            row_scale(amax, &mul, &back);
            mul *= sgn;
            // the lane whose row this is keeps the inverse
#pragma unroll
            for (int q = 0; q < RPI; ++q) {
              const float b = __shfl_sync(0xffffffffu, back, q * PP);
              if (lane == (i0 + i) * RPI + q) inv = b;
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float lo = bf2f(x[e]) * mul, hi = __uint_as_float(x[e] & 0xFFFF0000u) * mul;
            x[e] = BF ? bf16x2(lo, hi) : f16_pair(lo, hi);
          }
          const int rr = (i0 + i) * RPI + lane / PP;
          *reinterpret_cast<uint4*>(wtile + (rr >> 3) * C::GRP + kv_piece_off(2 * D, rr & 7, lane % PP)) =
              make_uint4(x[0], x[1], x[2], x[3]);
        }
      }
      rf_next = fmaxf(fabsf(a.scale) * kLog2e * a.c.k_scale * inv, 1.2e-38f);
      to_async_proxy();
      tc_before();
      __syncwarp();
      if (lane == 0) bar_arrive(q_ready + 8 * w);
    };
    // their lines into L2 a unit earlier, each row by its thread
    auto prefetch = [&](const Unit& v) {
      const int r = v.qb * QB + 128 * w + row;
      if (r >= v.s.c * G) return;
      const uint16_t* src = a.q + (int64_t)(v.s.s0 + r / G) * a.q_stride + (int64_t)(v.h * G + r % G) * D;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + 64 * i));
    };
    auto active = [&](const Unit& v) { return w == 0 || (NQ == 2 && v.s.c * G - v.qb * QB > 128); };
    if (active(u)) queries(u);
    for (;;) {
      const int kend = unit_end(u, len), ns = unit_subs<KT>(u, kend);
      const bool after = unit_after<KT>(u, len);
      const int r0 = u.qb * QB, R = u.s.c * G;
      const bool pair = NQ == 2 && R - r0 > 128;
      Unit un = u;
      if (after) {
        unit_next<KT, QB>(a, un, G);
        if (active(un)) prefetch(un);
      }
      // Behind a unit with two row tiles, one with a single tile goes on without the second tile's
      // warps: its first probabilities wait until those have read the marks of their last
      // tiles, which later tiles would write over
      const bool leaves = pair && after && !(un.s.c * G - un.qb * QB > 128);
      if (w == 0 && marks_due) {
        ok = bar_wait(marked, nm & 1u);
        ++nm;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      marks_due = leaves;
      if (w == 0 || pair) {
        const int r = r0 + 128 * w + row;
        const bool real = r < R;
        const int tok = real ? r / G : 0;
        const float rf = rf_next;
        const int pos = u.s.n - u.s.c + tok;
        const int see_hi = a.causal ? pos : u.s.n - 1;          // first and last key that this row sees
        const int see_lo = window_first(pos, a.window);
        const Full full = unit_full<QB>(a, u, G);
        float m = -INFINITY, l = 0.0f;
        bool bad_row = false;
        // S tiles e0 .. e1-1 are seen whole by every row and run the short form; the
        // others, the two behind a cut key tile (whose marks they look at, those of a half that
        // is not cut itself among them: values are cleaned by key tiles) and the last one run
        // the long one
        const int key0 = (u.tile0 + u.k) * KT;                  // first key of the part
        int e0 = full.lo > key0 ? (full.lo - key0 + KT - 1) / KT * (KT / kSub) + 2 : 0;
        if (e0 > ns) e0 = ns;
        int e1 = full.hi + 1 - key0 >= 0 ? (full.hi + 1 - key0) / kSub : 0;
        if (e1 > ns - 1) e1 = ns - 1;
        // Tokens with a value that is not finite: rows that see one show it. The marks of tile j
        // are there once its product is complete, which the arrival of S of tile j + 2 shows; the
        // last two at the end.
        auto marks = [&](int j) {
          const int j0 = key0 + j * kSub;
          if (!full.edge(j0 / KT * KT, KT)) return;
          const uint32_t* bits = KT == kSub ? s_poison[(tileno + j) & 7] : &s_poison[(tileno + (j >> 1)) & 7][2 * (j & 1)];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t x = *reinterpret_cast<const volatile uint32_t*>(bits + q);
            while (x) {
              const int e = 32 * q + __ffs(x) - 1;
              x &= x - 1;
              bad_row |= j0 + e >= see_lo && j0 + e <= see_hi;
            }
          }
        };
        // one S tile in buffer `buf`: its maximum, then P over it. False: a wait ran out
        auto step = [&](auto edge, int j, int buf, uint32_t phase) -> bool {
          constexpr bool EDGE = decltype(edge)::value;
          const uint32_t sT = tmem + (uint32_t)(128 * w + 64 * buf) + lanes;
          const uint32_t sbar = 16 * w + 8 * buf;
          bool good = bar_wait(s_full + sbar, phase & 1u);
          if (!__all_sync(0xffffffffu, good)) return false;
          tc_after();
          uint32_t s[kSub];
          tm_load32<0>(s, sT);
          tm_load32<32>(s, sT + 32);
          if constexpr (EDGE) {
            if (j >= 2) marks(j - 2);
          }
          tm_wait_load();
          if constexpr (EDGE) {
            const int lo = see_lo - (key0 + j * kSub), hi = see_hi - (key0 + j * kSub);
#pragma unroll
            for (int e = 0; e < kSub; ++e)
              if (e < lo || e > hi) s[e] = 0xFF800000u;
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < kSub; e += 8)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              mx[q] = max3(mx[q], __uint_as_float(s[e + 2 * q]), __uint_as_float(s[e + 2 * q + 1]));
          const float mt = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * rf;
          if (__builtin_expect(__any_sync(0xffffffffu, mt > m + (kHead<BF> + kLazy)), 0)) {
            const float mn = fmaxf(m, mt - kHead<BF>);
            const float fac = mn == -INFINITY ? 1.0f : ex2(m - mn);
            m = mn;
            l *= fac;
            if (j > 0) {
              // O of the tiles before is complete (all but the last of them are known to
              // be, from this S) and this tile's product waits for P
              good = bar_wait(o_done + 8 * w, (nd - 1) & 1u);
              if (!__all_sync(0xffffffffu, good)) return false;
              tc_after();
#pragma unroll 1
              for (int e = 0; e < D; e += 16) {
                uint32_t o[16];
                tm_load16(o, oT + e);
                tm_wait_load();
#pragma unroll
                for (int q = 0; q < 16; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * fac);
                tm_store16(oT + e, o);
              }
            }
          }
          if constexpr (EDGE) {
            if (j > 0 && j == ns - 1) {
              // the wait for the last product, below, needs the one before it to be known complete
              good = bar_wait(o_done + 8 * w, (nd - 1) & 1u);
              if (!__all_sync(0xffffffffu, good)) return false;
            }
          }
          const float base = m == -INFINITY ? 0.0f : m;
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          const float2 rf2 = make_float2(rf, rf), nb2 = make_float2(-base, -base);
#pragma unroll
          for (int h = 0; h < kSub / 32; ++h) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float2 x = fma2(make_float2(__uint_as_float(s[32 * h + 2 * e]), __uint_as_float(s[32 * h + 2 * e + 1])),
                              rf2, nb2);
              x = make_float2(ex2(x.x), ex2(x.y));
              sum[e & 1] = add2(sum[e & 1], x);
              // rounding to 16 bits: P is the second product's operand; its sum stays fp32
              pk[e] = BF ? bf16x2(x.x, x.y) : f16_pair(x.x, x.y);
            }
            tm_store16(sT + 16 * h, pk);
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          tm_wait_store();
          tc_before();
          __syncwarp();
          if (lane == 0) bar_arrive(p_ready + sbar);
          ++nd;
          return true;
        };
        // one call site of each form: the loop's code should fit the instruction caches
        for (int j = 0; j < ns && ok; ++j) {
#pragma unroll 1
          for (; j < e1 && j >= e0 && ok; ++j) {
            const int buf = j & 1;
            ok = step(std::false_type{}, j, buf, buf ? n_odd : n_even);
            n_odd += buf;
            n_even += buf ^ 1;
          }
          if (!ok || j >= ns) break;
          const int buf = j & 1;
          ok = step(std::true_type{}, j, buf, buf ? n_odd : n_even);
          n_odd += buf;
          n_even += buf ^ 1;
        }
        if (!ok) break;
        // ---- the unit's, or this part's, output ------------------------------------------------
        // the next unit's queries first: its S is formed while this output is written
        if (after && active(un)) queries(un);
        ok = bar_wait(o_done + 8 * w, (nd - 1) & 1u);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_after();
        for (int j = ns > 2 ? ns - 2 : 0; j < ns; ++j) marks(j);
        if (w == 1 && leaves) {
          __syncwarp();
          if (lane == 0) bar_arrive(marked);
        }
        const int64_t ustart = w0 + u.org;
        const int i0 = (int)place_div(ustart, per), i1 = (int)place_div(ustart + u.nt - 1, per);
        const bool whole = i0 == i1;
        float* const part = p.parts + (int64_t)(2 * (int)blockIdx.x + ((int)blockIdx.x == i0 ? 1 : 0)) * (QB * (D + 2));
        const int hq = real ? u.h * G + r % G : 0;
        const float mult = bad_row ? __int_as_float(0x7FFFFFFF) : whole ? (l == 0.0f ? 0.0f : a.c.v_scale / l) : 1.0f;
        uint8_t* const mine =
            whole ? reinterpret_cast<uint8_t*>(a.out + (int64_t)(u.s.s0 + tok) * a.out_stride + (int64_t)hq * D)
                  : reinterpret_cast<uint8_t*>(part + (int64_t)(128 * w + row) * D);
#pragma unroll 1
        for (int e = 0; e < D; e += 16) {
          uint32_t o[16];
          tm_load16(o, oT + e);
          tm_wait_load();
          float v[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) v[q] = __uint_as_float(o[q]) * mult;
          if (real) {
            if (whole) {
              uint4 x[2];
#pragma unroll
              for (int q = 0; q < 2; ++q)
                x[q] = make_uint4(bf16x2(v[8 * q], v[8 * q + 1]), bf16x2(v[8 * q + 2], v[8 * q + 3]),
                                  bf16x2(v[8 * q + 4], v[8 * q + 5]), bf16x2(v[8 * q + 6], v[8 * q + 7]));
              store_pair(mine + 2 * e, x, a.out_wide);
            } else {
#pragma unroll
              for (int q = 0; q < 16; q += 8) {
                const uint4 x[2] = {make_uint4(__float_as_uint(v[q]), __float_as_uint(v[q + 1]),
                                               __float_as_uint(v[q + 2]), __float_as_uint(v[q + 3])),
                                    make_uint4(__float_as_uint(v[q + 4]), __float_as_uint(v[q + 5]),
                                               __float_as_uint(v[q + 6]), __float_as_uint(v[q + 7]))};
                store_pair(mine + 4 * (e + q), x, true);
              }
            }
          }
        }
        tc_before();
        if (whole) {
          if (real && a.lse)
            a.lse[(int64_t)(u.s.s0 + tok) * a.q_heads + hq] =
                l == 0.0f ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
        } else {
          if (real) {
            __stcg(part + QB * D + 128 * w + row, m);
            __stcg(part + QB * (D + 1) + 128 * w + row, l);
          }
          // the row tile's warps meet (bounded), then count this part in
          __threadfence();
          __syncwarp();
          if (lane == 0) bar_arrive(joined + 8 * w);
          ok = bar_wait(joined + 8 * w, nj & 1u);
          ++nj;
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if ((tid & 127) == 0) s_last[w] = atomicAdd(p.counters + 2 * i0 + w, 1u) == (unsigned)(i1 - i0);
          __threadfence();
          __syncwarp();
          if (lane == 0) bar_arrive(joined + 8 * w);
          ok = bar_wait(joined + 8 * w, nj & 1u);
          ++nj;
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const bool last = *reinterpret_cast<volatile int*>(&s_last[w]) != 0;
          if (last) {
            __threadfence();
            auto slot = [&](int i) { return p.parts + (int64_t)(2 * i + (i == i0 ? 1 : 0)) * (QB * (D + 2)); };
            // Warp q joins rows q, q + 4, ... (few rows still occupy all warps). Lane: the
            // maximum and sum of one of them first, then a row's values over the lanes, four
            // parts' loads at a time
            const int jrow = 128 * w + 4 * lane + (warp & 3), jr = r0 + jrow;
            const bool jreal = jr < R;
            const int jtok = jreal ? jr / G : 0, jh = jreal ? u.h * G + jr % G : 0;
            float M = -INFINITY, L = 0.0f;
            for (int i = i0; i <= i1; i += 4) {
              float mi[4], li[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const bool in = jreal && i + y <= i1;
                const float* q = slot(in ? i + y : i0) + QB * D + jrow;
                mi[y] = in ? __ldcg(q) : -INFINITY;
                li[y] = in ? __ldcg(q + QB) : 0.0f;
              }
              const float mn = fmaxf(M, fmaxf(fmaxf(mi[0], mi[1]), fmaxf(mi[2], mi[3])));
              const float b = mn == -INFINITY ? 0.0f : mn;
              L *= ex2(M - b);
#pragma unroll
              for (int y = 0; y < 4; ++y) L += ex2(mi[y] - b) * li[y];
              M = mn;
            }
            const float bs = M == -INFINITY ? 0.0f : M;
            const float inv = L == 0.0f ? 0.0f : a.c.v_scale / L;
            if (jreal && a.lse)
              a.lse[(int64_t)(u.s.s0 + jtok) * a.q_heads + jh] =
                  L == 0.0f ? -INFINITY : (M + __log2f(L)) * 0.6931471805599453f;
            const uint64_t outp =
                jreal ? (uint64_t)(a.out + (int64_t)(u.s.s0 + jtok) * a.out_stride + (int64_t)jh * D) : 0ull;
            constexpr int PF = D / 4;                           // 16-byte pieces of an fp32 row
            const int items = (R - r0 - 128 * w - (warp & 3) + 3) / 4 * PF < 32 * PF
                                  ? (R - r0 - 128 * w - (warp & 3) + 3) / 4 * PF : 32 * PF;
            for (int x0 = 0; x0 < items; x0 += 128) {           // four pieces per lane
              float4 v[4];
              float mr[4], ir[4];
              uint64_t dst[4];
              int off[4], pr[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const int x = x0 + 32 * y + lane, rr = (x / PF) & 31;
                dst[y] = __shfl_sync(0xffffffffu, outp, rr);
                mr[y] = __shfl_sync(0xffffffffu, bs, rr);
                ir[y] = __shfl_sync(0xffffffffu, inv, rr);
                if (x >= items) dst[y] = 0ull;
                pr[y] = 128 * w + 4 * rr + (warp & 3);
                off[y] = x % PF;
                v[y] = make_float4(0.f, 0.f, 0.f, 0.f);
              }
#pragma unroll 2
              for (int i = i0; i <= i1; ++i) {
                const float* q = slot(i);
                float4 o[4];
                float mi[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  o[y] = __ldcg(reinterpret_cast<const float4*>(q + (int64_t)pr[y] * D) + off[y]);
                  mi[y] = __ldcg(q + QB * D + pr[y]);
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  const float fw = ex2(mi[y] - mr[y]);
                  v[y].x += fw * o[y].x; v[y].y += fw * o[y].y; v[y].z += fw * o[y].z; v[y].w += fw * o[y].w;
                }
              }
#pragma unroll
              for (int y = 0; y < 4; ++y)
                if (dst[y])
                  *(reinterpret_cast<uint2*>(dst[y]) + off[y]) =
                      make_uint2(bf16x2(v[y].x * ir[y], v[y].y * ir[y]), bf16x2(v[y].z * ir[y], v[y].w * ir[y]));
            }
            if ((tid & 127) == 0) p.counters[2 * i0 + w] = 0u;
          }
        }
      } else {
        if (after && active(un)) queries(un);
      }
      tileno += kend - u.k;
      if (!after) break;
      u = un;
    }
    if (!ok && lane == 0) atomicOr(a.status, kStatTimeout);
  }
  }
  tc_before();
  __syncthreads();
  if (tid == 0) wait_for_previous();
  if (warp == 12) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

template <int FMT, int D>
cudaError_t chunk_go(const ChunkParams& p, int sms, bool second, cudaStream_t s) {
  using C = ChunkCfg<FMT, D>;
  static_assert(C::NOP >= 3 && (C::BF || C::NRAW >= 2), "rings");
  static_assert(C::SMEM <= 232448 - 512, "shared memory");
  static int opted[64] = {0};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!opted[dev]) {
    // the register split above needs the launch to hold 128 per thread
    cudaFuncAttributes fa;
    err = cudaFuncGetAttributes(&fa, attn_chunk_kernel<FMT, D>);
    if (err != cudaSuccess) return err;
    if (fa.numRegs != 128) return cudaErrorInvalidConfiguration;
    err = cudaFuncSetAttribute(attn_chunk_kernel<FMT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (err != cudaSuccess) return err;
    opted[dev] = 1;
  }
  return launch_beside(attn_chunk_kernel<FMT, D>, p, sms, kThreads, C::SMEM, second, s);
}
template <int FMT>
cudaError_t chunk_dim(const ChunkParams& p, int sms, bool second, cudaStream_t s) {
  return p.a.c.dim == 64    ? chunk_go<FMT, 64>(p, sms, second, s)
         : p.a.c.dim == 128 ? chunk_go<FMT, 128>(p, sms, second, s)
                            : chunk_go<FMT, 256>(p, sms, second, s);
}

}  // namespace

// counters, then two parts of a block of rows per CTA
int64_t attn_chunk_workspace(const KvCache& c, int sms) {
  const int64_t rows = c.dim == 256 ? 128 : 256;
  return align_up((int64_t)sms * 8, 256) + (int64_t)sms * 2 * rows * (c.dim + 2) * 4;
}

cudaError_t launch_attn_chunk(const AttnArgs& a, int sms, bool second, cudaStream_t s) {
  ChunkParams p;
  p.a = a;
  p.a.out_wide = (reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && a.out_stride % 16 == 0) ? 1 : 0;
  uint8_t* const ws = a.ws + attn_rows_workspace(a.c, sms);
  p.counters = reinterpret_cast<unsigned*>(ws);
  p.parts = reinterpret_cast<float*>(ws + align_up((int64_t)sms * 8, 256));
  switch (a.c.fmt) {
    case KV_BF16: return chunk_dim<KV_BF16>(p, sms, second, s);
    case KV_Q8_0: return chunk_dim<KV_Q8_0>(p, sms, second, s);
    case KV_FP8: return chunk_dim<KV_FP8>(p, sms, second, s);
    default: return chunk_dim<KV_NVFP4>(p, sms, second, s);
  }
}

}  // namespace qmv
