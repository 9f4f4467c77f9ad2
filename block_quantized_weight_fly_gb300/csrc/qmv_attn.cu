// qmv_attn.cu -- attention of few new tokens over the paged KV cache: at most 16 query rows
// per (sequence, KV head), 32 where registers allow (most_rows), a row being one query head
// of one new token. Bound by the cache's bytes, each read once: 64 sequences of 200 to 16000
// FP8 tokens (8 heads of 128) take 180 to 183 us, 6.2 TB/s; one of 262144 NVFP4 tokens 75 us, 4.0
// TB/s, with no unit full: DRAM at half its rate, issue slots 51 % (59 % of the active cycles), tensor
// pipe 17 %. Its 16 warps are held to 128 registers each, spill 106 bytes of stores and 132 of
// loads, and stall on fixed latencies, on one another and on the math pipe before memory.
//
// Work: the cached tokens of every (sequence, KV head) in tiles of 32 (wide rows: 16),
// numbered through; each CTA takes one contiguous range of tiles, whatever the lengths are
// (read on the device), and inside it warp w every NW-th tile. A warp is its own pipeline:
// a lane copies 16 tokens of K, V and scales (one contiguous span, qmv_kv.cuh) into the
// warp's ring with cp.async.bulk, the warp decodes them in registers straight into mma.sync
// fragments:
//   S^T[16 tokens][rows]  = K[16 x D] Q^T        (A = keys)
//   O^T[D][rows]         += V^T[D x 16] P^T      (A = values, pairs of tokens interleaved)
// with 16-bit operands and fp32 sums. Dimensions are permuted so that a lane's 16-byte
// loads feed its own fragments: lane (g = lane / 4, c = lane % 4) holds of token g the
// pieces 2c, 2c+1 (keys) and of tokens 2c, 2c+1, 2c+8, 2c+9 the piece g (values); O's rows
// are permuted the same way. P^T comes out of S^T's accumulators by an 8x8 transpose
// (movmatrix). Running maximum and sum per row (softmax in base 2); O is rescaled only
// when a maximum grows by more than 2^8.
// The warps' parts join in shared memory, CTAs' parts of a row in the workspace: the last
// CTA to arrive adds them in order, so results do not depend on timing.
#include "qmv_attn.cuh"

namespace qmv {

namespace {

// A unit (one KV head of one sequence) counts as its tiles plus this many: its queries and
// the join of its parts take about as long, and shares are cut to be equal in time
constexpr int kUnitCost = 16;

template <int FMT, int D, int NT>
struct RowsCfg {
  static constexpr int RB = kv_row_bytes(FMT, D), SB = kv_scale_bytes(FMT, D);
  static constexpr int PART = kv_part_bytes(FMT, D), GB = kv_group_bytes(FMT, D);
  // tokens of a tile: 32, or 16 where those are 8 KB and where O of 32 rows of 128
  // dimensions leaves no registers for more (64 x 4001 NVFP4 tokens, 8 heads: 246 us, 332 with 32)
  static constexpr int HALVES = 2 * GB <= 4608 && NT * D < 512 ? 2 : 1;
  static constexpr int TILE = 16 * HALVES;
  static constexpr int STAGE = HALVES * 2 * GB;
  // warps: as many as registers (O, queries) and two ring stages each allow
  static constexpr int NW = FMT == KV_BF16 ? (D < 256 ? 8 : NT == 1 ? 6 : 5)
                            : NT >= 2 || D == 256 ? 8
                            : D == 64 || FMT == KV_NVFP4 ? 16
                            : FMT == KV_Q8_0             ? 10
                                                         : 12;
  static constexpr bool QSMEM = NT * D >= 512;               // queries in shared memory, not registers
  static constexpr int ROWS = 8 * NT;
  static constexpr int PITCH = D + 4;                        // floats per row of the join buffer
  static constexpr int CTRL = 1024 + (QSMEM ? NT * D * 16 : 0);
  static constexpr int JOIN = NW * 4 * PITCH * 4;            // 4 rows at a time
  static constexpr int BUDGET = 232448 - 2048 - CTRL - JOIN;      // 2048: static shared memory
  static constexpr int NS0 = BUDGET / (NW * STAGE);
  static constexpr int NS = NS0 > 6 ? 6 : NS0;
  static constexpr int SMEM = CTRL + JOIN + NW * NS * STAGE;
  static constexpr int VPP = FMT == KV_BF16 ? 8 : FMT == KV_NVFP4 ? 32 : 16;   // values per 16 bytes
  static constexpr int KB = RB / 4, VB = RB / 8;             // bytes per lane and token: keys, values
  static constexpr int KW = KB / 4 < 4 ? KB / 4 : 4, KCH = KB / 4 / KW;   // words per load, loads
  static constexpr int VW = VB / 4 < 4 ? VB / 4 : 4, VCH = VB / 4 / VW;
};

template <int W>
__device__ __forceinline__ void lds_words(const uint8_t* p, uint32_t* o) {
  if constexpr (W == 1) {
    o[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (W == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    o[0] = v.x; o[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w;
  }
}
template <bool BF>
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, const uint32_t* b) {
  if constexpr (BF)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// dimension of entry e of lane c's key list, of lane g's value list
template <class C>
__device__ __forceinline__ int kdim(int c, int e) {
  if constexpr (C::KB <= 16) return c * (C::KB * C::VPP / 16) + e;
  const int i = e / C::VPP;
  return ((i >> 1) * 8 + 2 * c + (i & 1)) * C::VPP + e % C::VPP;
}
template <class C>
__device__ __forceinline__ int vdim(int g, int e) {
  if constexpr (C::VB <= 16) return g * (C::VB * C::VPP / 16) + e;
  return ((e / C::VPP) * 8 + g) * C::VPP + e % C::VPP;
}

// One load of keys (KW words of tokens g and g + 8) -> the A fragments of its MMA steps.
// Steps per load: BF16 KW / 2, 8 bits KW, NVFP4 2 KW; entries 4s .. 4s+3 each.
template <int FMT, class C>
__device__ __forceinline__ void key_frags(const uint8_t* st, int g, int c, int i, uint32_t (&f)[8][4]) {
  int off;
  int dim0;                                   // first dimension of the load
  if constexpr (C::KB >= 16) {
    const int p = C::KB == 16 ? c : (i >> 1) * 8 + 2 * c + (i & 1);
    off = kv_piece_off(C::RB, g, p);
    dim0 = p * C::VPP;
  } else {                                    // 8 bytes: half a piece
    off = kv_piece_off(C::RB, g, c >> 1) + 8 * (c & 1);
    dim0 = c * (C::VPP / 2);
  }
  uint32_t lo[4], hi[4];
  lds_words<C::KW>(st + off, lo);
  lds_words<C::KW>(st + C::GB + off, hi);
  const uint8_t* sc = st + 8 * C::RB + g * C::SB;
  if constexpr (FMT == KV_BF16) {
#pragma unroll
    for (int w = 0; w < C::KW; w += 2) {
      f[w >> 1][0] = lo[w]; f[w >> 1][1] = hi[w]; f[w >> 1][2] = lo[w + 1]; f[w >> 1][3] = hi[w + 1];
    }
  } else if constexpr (FMT == KV_FP8) {
#pragma unroll
    for (int w = 0; w < C::KW; ++w) {
      uint32_t x[2], y[2];
      e4m3_word(lo[w], x);
      e4m3_word(hi[w], y);
      f[w][0] = x[0]; f[w][1] = y[0]; f[w][2] = x[1]; f[w][3] = y[1];
    }
  } else if constexpr (FMT == KV_Q8_0) {
    const uint32_t d = *reinterpret_cast<const unsigned short*>(sc + 2 * (dim0 >> 5));
    const uint32_t e = *reinterpret_cast<const unsigned short*>(sc + C::GB + 2 * (dim0 >> 5));
    const uint32_t d2 = dup_lo(d), e2 = dup_lo(e);
#pragma unroll
    for (int w = 0; w < C::KW; ++w) {
      uint32_t x[2], y[2];
      q8_word(lo[w], x);
      q8_word(hi[w], y);
      f[w][0] = h2_mul(x[0], d2); f[w][1] = h2_mul(y[0], e2); f[w][2] = h2_mul(x[1], d2); f[w][3] = h2_mul(y[1], e2);
    }
  } else {
    uint32_t d, e;                            // E4M3 scales of the load's one or two 16-value blocks
    if constexpr (C::KW == 4) {
      d = *reinterpret_cast<const unsigned short*>(sc + (dim0 >> 4));
      e = *reinterpret_cast<const unsigned short*>(sc + C::GB + (dim0 >> 4));
    } else {
      d = sc[dim0 >> 4];
      e = sc[C::GB + (dim0 >> 4)];
    }
    const uint32_t dh = e4m3_half(d), eh = e4m3_half(e);
#pragma unroll
    for (int w = 0; w < C::KW; ++w) {
      uint32_t x[4], y[4];
      e2m1_word(lo[w], x);
      e2m1_word(hi[w], y);
      const uint32_t d2 = w < 2 ? dup_lo(dh) : dup_hi(dh), e2 = w < 2 ? dup_lo(eh) : dup_hi(eh);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t* o = f[2 * w + h];
        o[0] = h2_mul(x[2 * h], d2); o[1] = h2_mul(y[2 * h], e2);
        o[2] = h2_mul(x[2 * h + 1], d2); o[3] = h2_mul(y[2 * h + 1], e2);
      }
    }
  }
}

// One load of values (VW words of tokens 2c, 2c+1, 2c+8, 2c+9) -> A fragments of the tiles
// of 16 dimensions it feeds: entries 2j, 2j+1 in rows g, g + 8. Tiles per load: VW * VPW / 2.
template <int FMT, class C>
__device__ __forceinline__ void value_frags(const uint8_t* st, int g, int c, int i, uint32_t (&f)[16][4]) {
  int p, sub, dim0;
  if constexpr (C::VB >= 16) {
    p = i * 8 + g;
    sub = 0;
    dim0 = p * C::VPP;
  } else {
    p = g * C::VB / 16;
    sub = (g * C::VB) & 15;
    dim0 = g * (C::VB * C::VPP / 16);
  }
  uint32_t w[4][4];
#pragma unroll
  for (int t = 0; t < 4; ++t)
    lds_words<C::VW>(st + C::PART + (t >> 1) * C::GB + kv_piece_off(C::RB, 2 * c + (t & 1), p) + sub, w[t]);
  const uint8_t* sc = st + C::PART + 8 * C::RB + 2 * c * C::SB;
#pragma unroll
  for (int h = 0; h < 2; ++h) {               // token pairs (2c, 2c+1), (2c+8, 2c+9): fragments 2h, 2h + 1
    const uint32_t* A = w[2 * h];
    const uint32_t* B = w[2 * h + 1];
    const uint8_t* s = sc + h * C::GB;
    if constexpr (FMT == KV_BF16) {
#pragma unroll
      for (int k = 0; k < C::VW; ++k) {
        f[k][2 * h] = __byte_perm(A[k], B[k], 0x5410);
        f[k][2 * h + 1] = __byte_perm(A[k], B[k], 0x7632);
      }
    } else if constexpr (FMT == KV_NVFP4) {
      uint32_t s0, s1 = 0u;                   // (token 2c, token 2c+1) scales of the one or two blocks
      if constexpr (C::VW == 4) {
        const uint32_t a = *reinterpret_cast<const unsigned short*>(s + (dim0 >> 4));
        const uint32_t b = *reinterpret_cast<const unsigned short*>(s + C::SB + (dim0 >> 4));
        s0 = e4m3_half(__byte_perm(a, b, 0x0040));
        s1 = e4m3_half(__byte_perm(a, b, 0x0051));
      } else {
        s0 = e4m3_half((uint32_t)s[dim0 >> 4] | ((uint32_t)s[C::SB + (dim0 >> 4)] << 8));
      }
#pragma unroll
      for (int k = 0; k < C::VW; ++k) {
        const uint32_t even = (A[k] & 0x0F0F0F0Fu) | ((B[k] << 4) & 0xF0F0F0F0u);
        const uint32_t odd = ((A[k] >> 4) & 0x0F0F0F0Fu) | (B[k] & 0xF0F0F0F0u);
        uint32_t x[4], y[4];
        e2m1_word(even, x);
        e2m1_word(odd, y);
        const uint32_t s2 = k < 2 ? s0 : s1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f[4 * k + e][2 * h] = h2_mul(x[e], s2);
          f[4 * k + e][2 * h + 1] = h2_mul(y[e], s2);
        }
      }
    } else {
      uint32_t s2 = 0u;
      if constexpr (FMT == KV_Q8_0)
        s2 = (uint32_t)*reinterpret_cast<const unsigned short*>(s + 2 * (dim0 >> 5)) |
             ((uint32_t)*reinterpret_cast<const unsigned short*>(s + C::SB + 2 * (dim0 >> 5)) << 16);
#pragma unroll
      for (int k = 0; k < C::VW; ++k) {
        const uint32_t u = __byte_perm(A[k], B[k], 0x5140), v = __byte_perm(A[k], B[k], 0x7362);
        uint32_t x[2], y[2];
        if constexpr (FMT == KV_FP8) {
          e4m3_word(u, x);
          e4m3_word(v, y);
        } else {
          q8_word(u, x);
          q8_word(v, y);
          x[0] = h2_mul(x[0], s2); x[1] = h2_mul(x[1], s2); y[0] = h2_mul(y[0], s2); y[1] = h2_mul(y[1], s2);
        }
        f[2 * k][2 * h] = x[0]; f[2 * k][2 * h + 1] = x[1];
        f[2 * k + 1][2 * h] = y[0]; f[2 * k + 1][2 * h + 1] = y[1];
      }
    }
  }
}

// a place in the numbered tiles: (sequence, head, tile of the unit)
struct Cursor {
  int b, h, k, nt;
  SeqInfo s;
};
template <int TILE>
__device__ __forceinline__ int unit_tiles(const AttnArgs& a, const SeqInfo& s) {
  if (s.c * (a.q_heads / a.c.heads) > a.few_rows) return 0;
  return s.n == 0 || s.c == 0 ? 0 : tiles_of<TILE>(s.n, seq_first(a, s));
}
// move on by `step` tiles; false past the last sequence
template <int TILE>
__device__ __forceinline__ bool advance(const AttnArgs& a, Cursor& u, int step) {
  u.k += step;
  while (u.k >= u.nt) {
    u.k -= u.nt;
    if (++u.h == a.c.heads) {
      u.h = 0;
      do {
        if (++u.b >= a.B) return false;
        seq_info(a, u.b, &u.s, false);
        u.nt = unit_tiles<TILE>(a, u.s);
      } while (u.nt == 0);
    }
  }
  return true;
}

struct RowsParams {
  AttnArgs a;
  unsigned* counters;        // [grid]: parts arrived of the row that CTA i leaves unfinished
  float* parts;              // [2 grid][ROWS (D + 2)]
};

template <int FMT, int D, int NT>
__global__ void __launch_bounds__(RowsCfg<FMT, D, NT>::NW * 32, 1) attn_rows_kernel(const RowsParams p) {
  using C = RowsCfg<FMT, D, NT>;
  constexpr bool BF = FMT == KV_BF16;
  constexpr int THREADS = C::NW * 32, TILE = C::TILE, HV = C::HALVES;
  const AttnArgs& a = p.a;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint2* const qsm = reinterpret_cast<uint2*>(smem + 1024);            // [NT][D / 16][32] if QSMEM
  uint8_t* const rings = smem + C::CTRL;
  float* const join = reinterpret_cast<float*>(smem + C::CTRL + C::NW * C::NS * C::STAGE);
  __shared__ int64_t s_first[4];              // first sequence, place in it, tiles before start and end
  __shared__ int64_t s_sum[C::NW], s_real[C::NW];
  __shared__ int s_max[C::NW];
  __shared__ float s_m[C::NW][8], s_l[C::NW][8];
  __shared__ int s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  let_next_start();
  const int G = a.q_heads / a.c.heads;
  const uint32_t bars = smem_u32(smem) + (uint32_t)(warp * C::NS * 8);
  const uint32_t ring = smem_u32(rings) + (uint32_t)(warp * C::NS * C::STAGE);
  const uint8_t* const ring_p = rings + warp * C::NS * C::STAGE;
  if (lane == 0) {
    for (int i = 0; i < C::NS; ++i) bar_init(bars + 8 * i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();

  // ---- the numbered tiles (kUnitCost, then its tiles, for each unit): total, where this
  // CTA's range starts, and how many tiles lie before its start and its end
  int64_t total = 0, tiles = 0, w0 = 0, w1 = 0, per = 0;
  int64_t before0 = 0, before1 = 0;
  int longest = 0, first_b = 0, first_off = 0;
  // Shares: equal, but no smaller than one tile per warp; units of up to three tiles per
  // warp go whole, since joining parts across CTAs costs more than those rounds
  auto share = [&]() {
    per = place_div(total + gridDim.x - 1, gridDim.x);
    const int least = kUnitCost + (longest <= 3 * C::NW ? longest : C::NW);
    if (per < least) per = least;
    if (per > kMostPlaces) {
      if (blockIdx.x == 0 && tid == 0) atomicOr(a.status, kStatRange);
      total = 0;
    }
    w0 = (int64_t)blockIdx.x * per;
    w1 = w0 + per < total ? w0 + per : total;
  };
  // tiles before place `off` of a sequence whose units have nt tiles
  auto tiles_to = [&](int off, int nt) {
    const int h = (int)((uint32_t)off / (uint32_t)(nt + kUnitCost)), rest = off - h * (nt + kUnitCost) - kUnitCost;
    return h * nt + (rest < 0 ? 0 : rest);
  };
  if (a.B <= 32) {                            // a warp's lanes hold them all: no meeting of warps
    SeqInfo s;
    int nt = 0;
    if (lane < a.B) {
      seq_info(a, lane, &s, blockIdx.x == 0 && warp == 0);
      nt = unit_tiles<TILE>(a, s);
    }
    const int64_t cost = nt ? (int64_t)a.c.heads * (nt + kUnitCost) : 0, real = (int64_t)a.c.heads * nt;
    int64_t scan = cost, rscan = real;
    longest = nt;
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, scan, o), r = __shfl_up_sync(0xffffffffu, rscan, o);
      if (lane >= o) {
        scan += v;
        rscan += r;
      }
      longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
    }
    total = __shfl_sync(0xffffffffu, scan, 31);
    tiles = __shfl_sync(0xffffffffu, rscan, 31);
    share();
    const bool in0 = w0 >= scan - cost && w0 < scan, in1 = w1 >= scan - cost && w1 < scan;
    const int at0 = in0 ? (int)(w0 - (scan - cost)) : 0;
    const int64_t b0 = in0 ? rscan - real + tiles_to(at0, nt) : 0;
    const int64_t b1 = in1 ? rscan - real + tiles_to((int)(w1 - (scan - cost)), nt) : 0;
    const uint32_t hit0 = __ballot_sync(0xffffffffu, in0), hit1 = __ballot_sync(0xffffffffu, in1);
    first_b = hit0 ? __ffs(hit0) - 1 : 0;
    first_off = __shfl_sync(0xffffffffu, at0, first_b);
    before0 = __shfl_sync(0xffffffffu, b0, first_b);
    before1 = __shfl_sync(0xffffffffu, b1, hit1 ? __ffs(hit1) - 1 : 0);
    if (!hit1) before1 = tiles;
  }
  // sums over windows of THREADS sequences; a second pass finds the windows of start and end
  for (int pass = 0; pass < 2 && a.B > 32; ++pass) {
    int64_t base = 0, rbase = 0;
    for (int win = 0; win < a.B; win += THREADS) {
      const int b = win + tid;
      SeqInfo s;
      int nt = 0;
      if (b < a.B) {
        seq_info(a, b, &s, pass == 0 && blockIdx.x == 0);
        nt = unit_tiles<TILE>(a, s);
      }
      const int64_t cost = nt ? (int64_t)a.c.heads * (nt + kUnitCost) : 0, real = (int64_t)a.c.heads * nt;
      int64_t scan = cost, rscan = real;
      int big = nt;
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, scan, o), r = __shfl_up_sync(0xffffffffu, rscan, o);
        if (lane >= o) {
          scan += v;
          rscan += r;
        }
        big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
      }
      if (lane == 31) {
        s_sum[warp] = scan;
        s_real[warp] = rscan;
        s_max[warp] = big;
      }
      __syncthreads();
      int64_t lo = base + scan - cost, rlo = rbase + rscan - real;
      for (int i = 0; i < C::NW; ++i) {
        if (i < warp) {
          lo += s_sum[i];
          rlo += s_real[i];
        }
        base += s_sum[i];
        rbase += s_real[i];
        longest = max(longest, s_max[i]);
      }
      if (pass == 1) {
        if (w0 >= lo && w0 < lo + cost) {
          s_first[0] = b;
          s_first[1] = w0 - lo;
          s_first[2] = rlo + tiles_to((int)(w0 - lo), nt);
        }
        if (w1 >= lo && w1 < lo + cost) s_first[3] = rlo + tiles_to((int)(w1 - lo), nt);
      }
      __syncthreads();
    }
    if (pass == 0) {
      total = base;
      tiles = rbase;
      share();
    } else {
      first_b = (int)s_first[0];
      first_off = (int)s_first[1];
      before0 = s_first[2];
      before1 = w1 < total ? s_first[3] : tiles;
    }
  }
  zero_unseeing(a, tid, THREADS);
  if (w0 >= w1 || before0 == before1) {
    if (tid == 0) wait_for_previous();
    return;
  }

  Cursor unit;                                // the unit being computed; k: its tile at the segment's start
  unit.b = first_b;
  seq_info(a, unit.b, &unit.s, false);
  unit.nt = unit_tiles<TILE>(a, unit.s);
  unit.h = (int)((uint32_t)first_off / (uint32_t)(unit.nt + kUnitCost));
  int org = kUnitCost - (first_off - unit.h * (unit.nt + kUnitCost));      // place of its first tile in the range
  unit.k = org < 0 ? -org : 0;
  const int len = (int)(before1 - before0), span = (int)(w1 - w0);         // tiles, places

  // A unit's queries as they are stored, in B fragment order: fetched before the copies are
  // issued, or before the last unit's parts are joined (with QSMEM, when they are needed)
  uint2 qf[NT][D / 16];
  auto fetch = [&](const Cursor& v) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = 8 * nt + g;
      const bool real = r < v.s.c * G;
      const uint16_t* src = a.q + (int64_t)(v.s.s0 + (real ? r / G : 0)) * a.q_stride +
                            (int64_t)(v.h * G + (real ? r % G : 0)) * D;
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        qf[nt][s] = make_uint2(0u, 0u);
        if (real) qf[nt][s] = __ldg(reinterpret_cast<const uint2*>(src + kdim<C>(c, 4 * s)));
      }
    }
  };
  if constexpr (!C::QSMEM) fetch(unit);

  // ---- the warp's copies: lane i < HALVES copies 16 tokens of the tile --------------------
  const int64_t page_bytes = (int64_t)C::GB << (a.c.page_shift - 3);   // of one head
  const int page_mask = (1 << a.c.page_shift) - 1;
  int to_issue = len > warp ? (len - warp + C::NW - 1) / C::NW : 0;    // tiles of this warp not yet copied
  int outstanding = 0, ist = 0;               // copies not yet waited for; the ring stage of the next one
  Cursor next = unit;
  if (to_issue && warp) advance<TILE>(a, next, warp);
  int page = 0, ntok = 0;                     // the next copy's page, looked up one tile ahead, and first token
  bool nhave = false;                         // this lane has 16 tokens to copy: one of them is cached and in a window
  auto look = [&]() {
    const int first = seq_first(a, next.s);
    ntok = (first / TILE + next.k) * TILE + 16 * (lane & (HV - 1));
    nhave = lane < HV && ntok < next.s.n && ntok + 16 > first;
    if (nhave) page = __ldg(a.table + (int64_t)next.b * a.max_pages + (ntok >> a.c.page_shift));
  };
  auto issue = [&]() {
    if (to_issue) {
      const bool have = nhave;
      const uint32_t bar = bars + 8 * ist;
      const int cnt = __popc(__ballot_sync(0xffffffffu, have));
      if (lane == 0) bar_expect(bar, cnt * 2 * C::GB);
      __syncwarp();
      if (have) {
        const int pg = checked_page(a, page);
        const uint8_t* src = a.c.data + ((int64_t)pg * a.c.heads + next.h) * page_bytes +
                             (int64_t)((ntok & page_mask) >> 3) * C::GB;
        bulk_copy(ring + ist * C::STAGE + (lane & (HV - 1)) * (2 * C::GB), src, 2 * C::GB, bar);
      }
      ++outstanding;
      if (++ist == C::NS) ist = 0;
      if (--to_issue) {
        advance<TILE>(a, next, C::NW);
        look();
      }
    }
  };
  // the first NS tiles in one go, a lane per 16 tokens
  {
    const int cnt = to_issue < C::NS ? to_issue : C::NS;
    const int mine = lane / HV;
    const uint8_t* src = nullptr;
    if (mine < cnt) {
      Cursor v = next;
      if (mine) advance<TILE>(a, v, mine * C::NW);
      const int first = seq_first(a, v.s), tok = (first / TILE + v.k) * TILE + 16 * (lane % HV);
      if (tok < v.s.n && tok + 16 > first) {
        const int pg = checked_page(a, __ldg(a.table + (int64_t)v.b * a.max_pages + (tok >> a.c.page_shift)));
        src = a.c.data + ((int64_t)pg * a.c.heads + v.h) * page_bytes + (int64_t)((tok & page_mask) >> 3) * C::GB;
      }
    }
    const uint32_t had = __ballot_sync(0xffffffffu, src != nullptr);
    const uint32_t bar = bars + 8 * mine;
    if (mine < cnt && lane % HV == 0) bar_expect(bar, __popc((had >> lane) & (HV == 2 ? 3u : 1u)) * 2 * C::GB);
    __syncwarp();
    if (src) bulk_copy(ring + mine * C::STAGE + (lane % HV) * (2 * C::GB), src, 2 * C::GB, bar);
    outstanding = cnt;
    ist = cnt == C::NS ? 0 : cnt;
    to_issue -= cnt;
    if (to_issue) {
      advance<TILE>(a, next, cnt * C::NW);
      look();
    }
  }

  // ---- segments: this CTA's part of one unit each ---------------------------------------
  int st = 0;                                 // ring stage and parity of the next tile
  uint32_t ph = 0;
  bool dead = false;
  int f0 = 0, f = warp;                       // the segment's first tile; this warp's next one, counted from w0
  while (f0 < len) {
    const int kend = unit.nt < span - org ? unit.nt : span - org;
    const int n = unit.s.n, cn = unit.s.c, R = cn * G;
    const int tok0 = (seq_first(a, unit.s) / TILE + unit.k) * TILE;      // first token of the segment

    // queries: B fragments, scaled to f16's range by a power of two per row
    float rf[NT][2];
    if constexpr (C::QSMEM) fetch(unit);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float inv = 1.0f;
      if constexpr (!BF) {
        float amax = 0.0f;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint2 v = qf[nt][s];
          amax = fmaxf(amax, fmaxf(fabsf(bf2f(v.x)), fabsf(__uint_as_float(v.x & 0xFFFF0000u))));
          amax = fmaxf(amax, fmaxf(fabsf(bf2f(v.y)), fabsf(__uint_as_float(v.y & 0xFFFF0000u))));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        float mul;
        row_scale(amax, &mul, &inv);
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint2 v = qf[nt][s];
          qf[nt][s].x = f16_pair(bf2f(v.x) * mul, __uint_as_float(v.x & 0xFFFF0000u) * mul);
          qf[nt][s].y = f16_pair(bf2f(v.y) * mul, __uint_as_float(v.y & 0xFFFF0000u) * mul);
        }
      }
      if constexpr (C::QSMEM) {
        if (warp == 0)
#pragma unroll
          for (int s = 0; s < D / 16; ++s) qsm[(nt * (D / 16) + s) * 32 + lane] = qf[nt][s];
      }
      const float fq = a.scale * kLog2e * a.c.k_scale * inv;
      rf[nt][0] = __shfl_sync(0xffffffffu, fq, 8 * c);
      rf[nt][1] = __shfl_sync(0xffffffffu, fq, 8 * c + 4);
    }
    if constexpr (C::QSMEM) __syncthreads();
    // visibility: key j of row r = token i is seen if lo(i) <= j <= hi(i)
    const int first_pos = n - cn;
    const int full_hi = a.causal ? first_pos : n - 1;                    // seen by every row up to here
    const int full_lo = a.window ? n - a.window : 0;                     // ... from here

    float m[NT][2], l[NT][2], o[NT][D / 16][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) o[nt][j][0] = o[nt][j][1] = o[nt][j][2] = o[nt][j][3] = 0.0f;
    }
    const int f1 = f0 + (kend - unit.k);
    for (; f < f1; f += C::NW) {
      const int tok = tok0 + (f - f0) * TILE;
      if (!dead) {
        if (!bar_wait(bars + 8 * st, ph)) {
          dead = true;
          if (lane == 0) atomicOr(a.status, kStatTimeout);
        }
        dead = __any_sync(0xffffffffu, dead);
        --outstanding;
      }
      if (dead) continue;
      const uint8_t* stage = ring_p + st * C::STAGE;

      float s[HV][NT][4];
#pragma unroll
      for (int hv = 0; hv < HV; ++hv)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[hv][nt][0] = s[hv][nt][1] = s[hv][nt][2] = s[hv][nt][3] = 0.0f;
      constexpr int SPL = D / 16 / C::KCH;                               // MMA steps per load
#pragma unroll
      for (int i = 0; i < C::KCH; ++i)
#pragma unroll
        for (int hv = 0; hv < HV; ++hv) {
          uint32_t kf[8][4];
          key_frags<FMT, C>(stage + hv * 2 * C::GB, g, c, i, kf);
#pragma unroll
          for (int e = 0; e < SPL; ++e)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint2 qv;
              if constexpr (C::QSMEM) qv = qsm[(nt * (D / 16) + i * SPL + e) * 32 + lane];
              else qv = qf[nt][i * SPL + e];
              const uint32_t bq[2] = {qv.x, qv.y};
              mma16816<BF>(s[hv][nt], kf[e], bq);
            }
        }
      const bool edge = tok + TILE - 1 > full_hi || tok < full_lo;
      auto seen = [&](int j, int r) {
        const int pos = first_pos + r / G;
        return j < n && (!a.causal || j <= pos) && (!a.window || j > pos - a.window);
      };
      float mt[NT][2];
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int hv = 0; hv < HV; ++hv) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[hv][nt][e] *= rf[nt][e & 1];
          if (edge) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!seen(tok + 16 * hv + g + 8 * (e >> 1), 8 * nt + 2 * c + (e & 1))) s[hv][nt][e] = -INFINITY;
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float v = fmaxf(s[0][nt][i], s[0][nt][2 + i]);
          if constexpr (HV == 2) v = fmaxf(v, fmaxf(s[1][nt][i], s[1][nt][2 + i]));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
          mt[nt][i] = v;
          grow |= v > m[nt][i] + (kHead<BF> + kLazy);
        }
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float mn = fmaxf(m[nt][i], mt[nt][i] - kHead<BF>);
            const float fac = mn == -INFINITY ? 1.0f : ex2(m[nt][i] - mn);
            m[nt][i] = mn;
            l[nt][i] *= fac;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              o[nt][j][i] *= fac;
              o[nt][j][2 + i] *= fac;
            }
          }
      }
      uint32_t pf[HV][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float base[2] = {m[nt][0] == -INFINITY ? 0.0f : m[nt][0], m[nt][1] == -INFINITY ? 0.0f : m[nt][1]};
#pragma unroll
        for (int hv = 0; hv < HV; ++hv) {
          float pr[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            pr[e] = ex2(s[hv][nt][e] - base[e & 1]);
            l[nt][e & 1] += pr[e];
          }
          // rounding to 16 bits: P enters the second product; its sum stays in fp32
          pf[hv][nt][0] = transpose8x8(BF ? bf16x2(pr[0], pr[1]) : f16_pair(pr[0], pr[1]));
          pf[hv][nt][1] = transpose8x8(BF ? bf16x2(pr[2], pr[3]) : f16_pair(pr[2], pr[3]));
        }
      }
      constexpr int TPL = D / 16 / C::VCH;                               // dimension tiles per load
#pragma unroll
      for (int hv = 0; hv < HV; ++hv) {
        uint32_t poison = 0u;
#pragma unroll
        for (int i = 0; i < C::VCH; ++i) {
          uint32_t vf[16][4];
          value_frags<FMT, C>(stage + hv * 2 * C::GB, g, c, i, vf);
          if (edge) {
            // a value that is not finite would spoil rows that do not see it (0 x NaN): take
            // it out here, mark its token
            constexpr uint32_t E = BF ? 0x7F80u : 0x7C00u;
#pragma unroll
            for (int e = 0; e < TPL; ++e)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t x = vf[e][k];
                if ((x & E) == E) {
                  vf[e][k] &= 0xFFFF0000u;
                  poison |= 1u << (2 * (k >> 1));
                }
                if ((x & (E << 16)) == (E << 16)) {
                  vf[e][k] &= 0x0000FFFFu;
                  poison |= 2u << (2 * (k >> 1));
                }
              }
          }
#pragma unroll
          for (int e = 0; e < TPL; ++e)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<BF>(o[nt][i * TPL + e], vf[e], pf[hv][nt]);
        }
        if (edge) {
          poison |= __shfl_xor_sync(0xffffffffu, poison, 4);
          poison |= __shfl_xor_sync(0xffffffffu, poison, 8);
          poison |= __shfl_xor_sync(0xffffffffu, poison, 16);
          if (__any_sync(0xffffffffu, poison != 0u)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              bool hit = false;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                hit |= ((poison >> k) & 1u) && seen(tok + 16 * hv + 2 * c + (k & 1) + 8 * (k >> 1), 8 * nt + g);
              const uint32_t rows = __ballot_sync(0xffffffffu, hit);
#pragma unroll
              for (int i = 0; i < 2; ++i)
                if ((rows >> (4 * (2 * c + i))) & 15u) {
#pragma unroll
                  for (int j = 0; j < D / 16; ++j) o[nt][j][i] = o[nt][j][2 + i] = __int_as_float(0x7FFFFFFF);
                }
            }
          }
        }
      }
      __syncwarp();
      if (++st == C::NS) {
        st = 0;
        ph ^= 1u;
      }
      issue();
    }

    Cursor after = unit;
    int next_org = org;
    if (f1 < len) {
      after.k = after.nt - 1;
      advance<TILE>(a, after, 1);
      next_org = org + unit.nt + kUnitCost;
      if constexpr (!C::QSMEM) fetch(after);
    }
    // ---- join the warps' parts: 4 rows (one of each lane column) at a time ----------------------------------------
    // the CTAs that share the unit
    const int i0 = (int)place_div(w0 + org, per), i1 = (int)place_div(w0 + org + unit.nt - 1, per);
    const bool whole = i0 == i1;
    // parts that begin with their unit in odd slots, continued ones in even slots
    const int slot = 2 * (int)blockIdx.x + ((int)blockIdx.x == i0 ? 1 : 0);
    float* const part = p.parts + (int64_t)slot * (C::ROWS * (D + 2));
    auto store_row = [&](int r, int d4, float4 v, float inv) {
      uint2 w = make_uint2(bf16x2(v.x * inv, v.y * inv), bf16x2(v.z * inv, v.w * inv));
      *reinterpret_cast<uint2*>(a.out + (int64_t)(unit.s.s0 + r / G) * a.out_stride +
                                (int64_t)(unit.h * G + r % G) * D + 4 * d4) = w;
    };
    auto store_lse = [&](int r, float mm, float ll) {
      if (a.lse)
        a.lse[(int64_t)(unit.s.s0 + r / G) * a.q_heads + unit.h * G + r % G] =
            ll == 0.0f ? -INFINITY : (mm + __log2f(ll)) * 0.6931471805599453f;
    };
#pragma unroll
    for (int x = 0; x < 2 * NT; ++x) {
      const int nt = x >> 1, i = x & 1;
      if (8 * nt + i >= R) break;
      float v = l[nt][i];
      v += __shfl_xor_sync(0xffffffffu, v, 4);
      v += __shfl_xor_sync(0xffffffffu, v, 8);
      v += __shfl_xor_sync(0xffffffffu, v, 16);
      if (g == 0) {
        s_m[warp][c] = m[nt][i];
        s_l[warp][c] = v;
      }
      float* dst = join + (warp * 4 + c) * C::PITCH;
#pragma unroll
      for (int j = 0; j < D / 16; j += 2)
        *reinterpret_cast<float4*>(dst + vdim<C>(g, 2 * j)) =
            make_float4(o[nt][j][i], o[nt][j][2 + i], o[nt][j + 1][i], o[nt][j + 1][2 + i]);
      __syncthreads();
      for (int y = tid; y < D; y += THREADS) {                            // (row, 4 dimensions)
        const int cr = y / (D / 4), d4 = y % (D / 4), r = 8 * nt + 2 * cr + i;
        if (r < R) {
          float M = -INFINITY;
#pragma unroll
          for (int w = 0; w < C::NW; ++w) M = fmaxf(M, s_m[w][cr]);
          const float base = M == -INFINITY ? 0.0f : M;
          float L = 0.0f;
          float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < C::NW; ++w) {
            const float fw = ex2(s_m[w][cr] - base);
            L += fw * s_l[w][cr];
            const float4 z = *reinterpret_cast<const float4*>(join + (w * 4 + cr) * C::PITCH + 4 * d4);
            u.x += fw * z.x; u.y += fw * z.y; u.z += fw * z.z; u.w += fw * z.w;
          }
          if (whole) {
            store_row(r, d4, u, L == 0.0f ? 0.0f : a.c.v_scale / L);
            if (d4 == 0) store_lse(r, M, L);
          } else {
            __stcg(reinterpret_cast<float4*>(part + r * D + 4 * d4), u);
            if (d4 == 0) {
              __stcg(part + C::ROWS * D + r, M);
              __stcg(part + C::ROWS * (D + 1) + r, L);
            }
          }
        }
      }
      __syncthreads();
    }
    if (!whole) {
      __threadfence();
      __syncthreads();
      if (tid == 0) s_last = atomicAdd(p.counters + i0, 1u) == (unsigned)(i1 - i0);
      __syncthreads();
      if (s_last) {
        __threadfence();
        constexpr int PART = C::ROWS * (D + 2), IN = 8;         // parts in flight
        const float* const q0 = p.parts + (int64_t)(2 * i0) * PART;         // part i0 + i at 2 i PART, the first at PART
        const int n_parts = i1 - i0 + 1;
        for (int x = tid; x < R * (D / 4); x += THREADS) {
          const int r = x / (D / 4), d4 = x % (D / 4);
          float M = -INFINITY, L = 0.0f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int i = 0; i < n_parts; i += IN) {
            float mi[IN], li[IN];
            float4 ui[IN];
#pragma unroll
            for (int y = 0; y < IN; ++y) {
              const int z = i + y < n_parts ? i + y : 0;
              const float* q = q0 + (int64_t)(z ? 2 * z : 1) * PART;
              mi[y] = i + y < n_parts ? __ldcg(q + C::ROWS * D + r) : -INFINITY;
              li[y] = __ldcg(q + C::ROWS * (D + 1) + r);
              ui[y] = __ldcg(reinterpret_cast<const float4*>(q + r * D + 4 * d4));
            }
            float mn = M;
#pragma unroll
            for (int y = 0; y < IN; ++y) mn = fmaxf(mn, mi[y]);
            const float base = mn == -INFINITY ? 0.0f : mn, f = ex2(M - base);
            M = mn;
            L *= f;
            v.x *= f; v.y *= f; v.z *= f; v.w *= f;
#pragma unroll
            for (int y = 0; y < IN; ++y) {
              if (i + y < n_parts) {
                const float fw = ex2(mi[y] - base);
                L += fw * li[y];
                v.x += fw * ui[y].x; v.y += fw * ui[y].y; v.z += fw * ui[y].z; v.w += fw * ui[y].w;
              }
            }
          }
          store_row(r, d4, v, L == 0.0f ? 0.0f : a.c.v_scale / L);
          if (d4 == 0) store_lse(r, M, L);
        }
        __syncthreads();
        if (tid == 0) p.counters[i0] = 0u;
      }
    }
    f0 = f1;
    unit = after;
    org = next_org;
  }
  // after a wait that ran out: copies still in flight land before the CTA leaves
  if (dead) {
    for (int i = 0; i <= outstanding; ++i) {  // from the one that was waited for
      (void)bar_wait(bars + 8 * st, ph);
      if (++st == C::NS) {
        st = 0;
        ph ^= 1u;
      }
    }
  }
  if (tid == 0) wait_for_previous();
}

template <int FMT, int D, int NT>
cudaError_t rows_go(const RowsParams& p, int sms, bool second, cudaStream_t s) {
  using C = RowsCfg<FMT, D, NT>;
  static_assert(C::NS >= 2, "ring");
  static int opted[64] = {0};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!opted[dev]) {
    err = cudaFuncSetAttribute(attn_rows_kernel<FMT, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (err != cudaSuccess) return err;
    opted[dev] = 1;
  }
  return launch_beside(attn_rows_kernel<FMT, D, NT>, p, sms, C::NW * 32, C::SMEM, second, s);
}
template <int FMT, int NT>
cudaError_t rows_dim(const RowsParams& p, int sms, bool second, cudaStream_t s) {
  if (p.a.c.dim == 64) return rows_go<FMT, 64, NT>(p, sms, second, s);
  if constexpr (NT <= 2 || FMT == KV_NVFP4)
    if (p.a.c.dim == 128) return rows_go<FMT, 128, NT>(p, sms, second, s);
  if constexpr (NT <= 2)
    if (p.a.c.dim == 256) return rows_go<FMT, 256, NT>(p, sms, second, s);
  return cudaErrorInvalidValue;
}
template <int NT>
cudaError_t rows_fmt(const RowsParams& p, int sms, bool second, cudaStream_t s) {
  switch (p.a.c.fmt) {
    case KV_BF16: return rows_dim<KV_BF16, NT>(p, sms, second, s);
    case KV_Q8_0: return rows_dim<KV_Q8_0, NT>(p, sms, second, s);
    case KV_FP8: return rows_dim<KV_FP8, NT>(p, sms, second, s);
    default: return rows_dim<KV_NVFP4, NT>(p, sms, second, s);
  }
}

}  // namespace

// The most query rows of a KV head that stream the cache; the chunk kernel, whose time is
// the same up to 128 rows, takes more. us of 64 sequences x 4001 tokens x 8 heads, streaming
// 16 and 32 rows | chunk kernel: D = 64: FP8 98, 147 | 195, BF16 111, 155 | 194, NVFP4 102, 154
// | 201, Q8_0 109, 163 | 202. D = 128: NVFP4 137, 247 | 353; FP8 125, 238 | 230, BF16 195, 281 |
// 226, Q8_0 141, 272 | 268. D = 256, where O of 32 rows does not fit a warp's registers: Q8_0
// 249 | 360. The 32-row form wins at every other shape tried too, 32 rows of it against 33 of the
// chunk kernel: one sequence of 131072 tokens, 8 heads and 1: FP8 D = 64 78, 68 | 121, 134, NVFP4
// D = 128 126, 111 | 195, 179; 32 of 16000, 1 head: 52 | 81, 76 | 117; 128 of 500, 4 heads: 58 |
// 85, 78 | 115; 4 of 333, 8 heads: 19 | 46, 21 | 56. The 16-row form is ahead of or even with
// the chunk kernel's 17 rows at all of these in every format and width (BF16 D = 256, one of 131072: 207 |
// 207). Not tried at them: a 32-row form of the other three formats with D = 128.
static int most_rows(const KvCache& c) { return c.dim == 64 || (c.dim == 128 && c.fmt == KV_NVFP4) ? 32 : 16; }

// counters, then two parts of most_rows rows per CTA
int64_t attn_rows_workspace(const KvCache& c, int sms) {
  return align_up((int64_t)sms * 8, 256) + align_up((int64_t)sms * 2 * most_rows(c) * (c.dim + 2) * 4, 256);
}

cudaError_t launch_attn_rows(const AttnArgs& a, int sms, bool second, cudaStream_t s) {
  RowsParams p;
  p.a = a;
  p.counters = reinterpret_cast<unsigned*>(a.ws);
  p.parts = reinterpret_cast<float*>(a.ws + align_up((int64_t)sms * 8, 256));
  return a.few_rows <= 8    ? rows_fmt<1>(p, sms, second, s)
         : a.few_rows <= 16 ? rows_fmt<2>(p, sms, second, s)
                            : rows_fmt<4>(p, sms, second, s);
}

// Sequences with few query rows per KV head are bound by the cache's bytes and go to the
// streaming kernel, the others to the tensor-core kernel with its tiles of 128 rows. A batch
// of single tokens and one chunk takes both: 47 single tokens and a chunk of 777 took 407 us
// in 128-row tiles alone, 171 to 173 us split.
cudaError_t launch_attn(AttnArgs a, cudaStream_t s) {
  const int sms = num_sms_current_device();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int G = a.q_heads / a.c.heads;
  const int most = most_rows(a.c);
  if ((int64_t)a.max_q * G <= most) {
    a.few_rows = a.max_q * G;
    return launch_attn_rows(a, sms, false, s);
  }
  // The new tokens of each sequence are known on the device alone: T may count rows of no
  // sequence, so a batch padded to B max_q rows can be single tokens all the same. With T below
  // that some sequence is shorter, and the streaming kernel goes first; else probably none
  // is, and it goes second, in the chunks' shadow: five blocks of 8 tokens (Q8_0, D = 256) 96 us,
  // 99 with it first, 92 without it; 31 single tokens and a chunk of 512 (FP8, D = 128) 122 us
  // padded to B max_q rows, 120 not padded
  a.few_rows = 0;
  if (G > most || (a.B == 1 && a.T >= a.max_q)) return launch_attn_chunk(a, sms, false, s);
  a.few_rows = G <= 8 ? 8 : G <= 16 ? 16 : 32;
  const bool rows_first = a.T < (int64_t)a.B * a.max_q;
  const cudaError_t err = rows_first ? launch_attn_rows(a, sms, false, s) : launch_attn_chunk(a, sms, false, s);
  if (err != cudaSuccess) return err;
  return rows_first ? launch_attn_chunk(a, sms, true, s) : launch_attn_rows(a, sms, true, s);
}

// the two kernels' areas lie apart: in a mixed batch they overlap in time
int64_t attn_workspace_bytes(const KvCache& c, int, int sms) {
  return attn_rows_workspace(c, sms) + align_up(attn_chunk_workspace(c, sms), 256);
}

}  // namespace qmv
