// decode_paged.cu -- one query per sequence over a paged cache held in 16 bits
// or in 4 (E2M1 codes with one E4M3 factor for each 16).
//
// Work.  The key axis of every (sequence, KV head, group of query heads) is cut
// into units of kUnitKeys keys; a grid of resident CTAs takes equal runs of the
// list of all units (order: sequence, head, key), whatever the sequences'
// lengths are.  A run covers whole (sequence, head) segments, which the CTA
// finishes itself, and at its two ends parts of segments, whose states (m, l, o)
// it leaves in the workspace; a second kernel folds those.  The division of the
// list follows from the lengths alone, so results repeat bitwise.  Where a page
// table has room for few units (short_cluster), a cluster of 1 to 8 CTAs takes each
// segment instead and folds its states through shared memory.
//
// Inside a CTA each warp takes every fourth piece of a segment (16 keys, or 32 of
// a 4-bit cache) and keeps its own online-softmax state.  It computes S^T = K Q^T
// and O^T = V^T P^T with m16n8k16 tensor-core products: the keys (or head
// elements) fill the 16 rows and up to 8 query heads the 8 columns; tcgen05's 128
// rows would find nothing to fill them with.  The order of the head's elements
// inside a product is free as long as Q follows it, so a lane's 16-byte piece of
// a row of K is its operand for several products, and V, whose operand pairs two
// keys, takes one byte permute for two elements.
//
// "The large batch", here and below: 64 sequences whose lengths lie evenly between
// 1024 and 32768 tokens (16896 on average), in random order, 32 query heads on 8
// (128 for 16 heads a unit), bf16, pages of 64.
//
// 16 bits: rows go from global memory straight into operand registers, requested
// as an earlier piece's are consumed (kDepth).  Bound by HBM: the large batch at
// d = 128 takes 630 us, 7.0 TB/s.
// 4 bits: rows go through a ring in shared memory that asynchronous copies fill.
// A pair of codes becomes an fp16 pair in one conversion, one product applies the
// factor (exact, 2 by 4 significant bits), and the bytes of two keys' codes are
// interleaved for V before the conversion.  That is 275 instructions for 16 keys
// of one KV head (72 conversions at half rate, 64 products), against 390 issue
// slots in the time that HBM takes for their 2304 bytes: bound by issue and by
// the conversions' pipe (62 % and 53 % busy, 16 warps an SM).  The same batch
// takes 205 us, 6.1 TB/s.
//
// The scores' reference m follows the maximum lazily (it moves when a score is
// more than 8 above it in base-2 units), so P <= 256; l sums P before it is
// rounded for P V (kTerms).
#include <cuda_runtime.h>

#include <type_traits>

#include "gbattn_copy.cuh"
#include "gbattn_internal.h"
#include "gbattn_ptx.cuh"

namespace gbattn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCtas = 1024;        // bound of the grid, for the workspace's size
constexpr int kMaxGroup = 16;         // query heads of one unit
constexpr float kRescaleThreshold = 8.f;
// The reference before any key: finite, so that a masked score minus it is -inf,
// and below every score that does not overflow.
constexpr float kNoReference = -3e38f;

enum Format : int { kF16 = 0, kBf16 = 1, kFp4 = 2 };

struct Params {
  const uint16_t* q;
  const uint8_t* data[2];
  const uint8_t* factor[2];
  const float* descale[2];
  const int* page_table;
  const int* seqlens;
  uint16_t* o;
  float* lse;
  float* part_o;   // [ctas][2][rows][D]
  float* part_ml;  // [ctas][2][rows][2]: m in base-2 units, l
  int2* parts;     // [B][heads of units]: first CTA * 2 + its slot, number of parts (0: finished)
  int B, Hq, Hkv, g, groups, rows;
  int page_shift, n_pages, max_pages;
  float scale_log2;
  int out_bf16;
  int most_ctas;   // states that the workspace has room for
  int* status;
};

__device__ __forceinline__ int seq_len(const Params& p, int b) {
  const int cap = p.max_pages << p.page_shift;
  return max(0, min(p.seqlens[b], cap));
}

// Not a read-only load: the previous kernel may write the cache while this one has
// already started (and waits).
__device__ __forceinline__ uint4 ld16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void lds(uint32_t (&v)[4], uint32_t a) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void lds(uint32_t (&v)[2], uint32_t a) {
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(a) : "memory");
}
__device__ __forceinline__ void lds(uint32_t (&v)[1], uint32_t a) {
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[0]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (BF16) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}

// The same with accumulators of zero.
template <bool BF16>
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  if constexpr (BF16) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  }
}

// The 8 x 8 transpose of 16-bit elements held as two to a lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Four codes' bytes of E2M1 pairs to fp16 pairs (exact).
__device__ __forceinline__ void e2m1_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <int NT>
__device__ __forceinline__ void add(float (&s)[NT][4], const float (&s2)[NT][4]) {
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int c = 0; c < 4; ++c) s[t][c] += s2[t][c];
}

// Both halves of a times one half of b.
__device__ __forceinline__ uint32_t hmul2_half(uint32_t a, uint32_t b, bool high) {
  uint32_t r;
  if (high)
    asm("{\n\t.reg .b16 l, h;\n\t.reg .b32 t;\n\tmov.b32 {l, h}, %2;\n\tmov.b32 t, {h, h};\n\tmul.rn.f16x2 %0, %1, t;\n\t}"
        : "=r"(r)
        : "r"(a), "r"(b));
  else
    asm("{\n\t.reg .b16 l, h;\n\t.reg .b32 t;\n\tmov.b32 {l, h}, %2;\n\tmov.b32 t, {l, l};\n\tmul.rn.f16x2 %0, %1, t;\n\t}"
        : "=r"(r)
        : "r"(a), "r"(b));
  return r;
}

// Where a lane's pieces of the pool's first 16 rows lie.
struct LanePtrs {
  const uint8_t* data[2];
  const uint8_t* factor;  // 4 bits: the piece of K's or V's factors that the lane copies
};

// Terms that P is held in for P V.  Over a 16-bit cache the rounding's remainder
// is a second one: a single bf16 (or fp16) P shows in O next to O's own rounding
// (relative error 2.3e-3 against 1.7e-3 in bf16 at 64 sequences of 17 thousand
// tokens), and the loop, bound by memory, has room for the products (the large
// batch 630 us with and without them; with 16 heads a unit 689 and 674).  Over a
// 4-bit cache P is one fp16, off by 2^-11 at most: the loop is bound by issue there,
// and the cache's own error is larger (O in bf16 1.7e-3 off, as with P in fp32; in
// fp16 2.5e-4, with P in fp32 2.1e-4).
template <int FMT>
constexpr int kTerms = FMT == kFp4 ? 1 : 2;

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// What one lane holds of 16 keys: for K rows r and r + 8 (r = lane / 4), for V
// keys 2 q, 2 q + 1, 2 q + 8, 2 q + 9 (q = lane % 4).  Keys from n_keys on are
// not read (zeros): a unit's last rows may lie behind the sequence.
template <int D, int FMT>
struct Tile {
  // 16 bits: K pieces q, q + 4, .. of a row (8 elements each); V pieces r, r + 8.
  uint4 k[2][D / 32];
  uint4 v[4][D / 64];

  __device__ static __forceinline__ LanePtrs ptrs(const Params& p, int lane) {
    LanePtrs a{};
    a.data[0] = p.data[0] + (lane >> 2) * (2 * D) + (lane & 3) * 16;
    a.data[1] = p.data[1] + (2 * (lane & 3)) * (2 * D) + (lane >> 2) * 16;
    return a;
  }
  __device__ __forceinline__ void load_k(const LanePtrs& a, int block, int lane, int n_keys) {
    const uint8_t* src = a.data[0] + static_cast<long long>(block) * (16 * 2 * D);
    if (n_keys >= 16) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < D / 32; ++c) k[i][c] = ld16(src + 8 * i * (2 * D) + c * 64);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
          k[i][c] = (lane >> 2) + 8 * i < n_keys ? ld16(src + 8 * i * (2 * D) + c * 64) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  __device__ __forceinline__ void load_v(const LanePtrs& a, int block, int lane, int n_keys) {
    const uint8_t* src = a.data[1] + static_cast<long long>(block) * (16 * 2 * D);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = (i & 1) + 8 * (i >> 1);
      if (n_keys >= 16 || 2 * (lane & 3) + key < n_keys) {
#pragma unroll
        for (int c = 0; c < D / 64; ++c) v[i][c] = ld16(src + key * (2 * D) + c * 128);
      } else {
#pragma unroll
        for (int c = 0; c < D / 64; ++c) v[i][c] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
  // s[t] = K Q^T for the 8 query heads of each tile t, in two chains of products.
  template <int NT>
  __device__ __forceinline__ void scores(float (&s)[NT][4], const uint32_t (&qf)[NT][D / 16][2]) const {
    float s2[NT][4];
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint32_t(&q0)[2] = qf[t][2 * c], (&q1)[2] = qf[t][2 * c + 1];
        if (c == 0) {
          mma16816_first<FMT == kBf16>(s[t], k[0][c].x, k[1][c].x, k[0][c].y, k[1][c].y, q0[0], q0[1]);
          mma16816_first<FMT == kBf16>(s2[t], k[0][c].z, k[1][c].z, k[0][c].w, k[1][c].w, q1[0], q1[1]);
        } else {
          mma16816<FMT == kBf16>(s[t], k[0][c].x, k[1][c].x, k[0][c].y, k[1][c].y, q0[0], q0[1]);
          mma16816<FMT == kBf16>(s2[t], k[0][c].z, k[1][c].z, k[0][c].w, k[1][c].w, q1[0], q1[1]);
        }
      }
    add(s, s2);
  }
  // o += V^T P^T; product j = 4 c + w holds elements 64 c + 8 r + 2 w (rows r)
  // and the next one (rows r + 8).
  template <int NT>
  __device__ __forceinline__ void values(float (&o)[NT][D / 16][4], const uint32_t (&pf)[NT][kTerms<FMT>][2]) const {
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const uint32_t w[4][4] = {{v[0][c].x, v[0][c].y, v[0][c].z, v[0][c].w},
                                {v[1][c].x, v[1][c].y, v[1][c].z, v[1][c].w},
                                {v[2][c].x, v[2][c].y, v[2][c].z, v[2][c].w},
                                {v[3][c].x, v[3][c].y, v[3][c].z, v[3][c].w}};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a0 = __byte_perm(w[0][j], w[1][j], 0x5410), a1 = __byte_perm(w[0][j], w[1][j], 0x7632);
        const uint32_t a2 = __byte_perm(w[2][j], w[3][j], 0x5410), a3 = __byte_perm(w[2][j], w[3][j], 0x7632);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < kTerms<FMT>; ++i)
            mma16816<FMT == kBf16>(o[t][4 * c + j], a0, a1, a2, a3, pf[t][i][0], pf[t][i][1]);
      }
    }
  }
  // First of the 8 elements of Q that steps 2 i and 2 i + 1 take from a lane.
  __device__ static __forceinline__ int k_element(int i, int lane) { return 32 * i + 8 * (lane & 3); }
  __device__ static __forceinline__ int o_element(int j, int lane, int half) {
    return 64 * (j / 4) + 8 * (lane >> 2) + 2 * (j & 3) + half;
  }
};

// 16 keys of a 4-bit cache in shared memory, one stage of a warp's own ring,
// which asynchronous copies of 16 bytes fill.  Rows of V of 64 bytes are stored
// in pairs of 128 bytes with their 16-byte pieces permuted, so that the four
// keys that 16 lanes read at a time lie in different banks.
template <int D>
struct Stage {
  static constexpr int kRow = D / 2, kFactors = D / 16;  // bytes of a row
  static constexpr int kV = 16 * kRow, kKf = 2 * kV, kVf = kKf + 16 * kFactors;
  static constexpr int kBytes = kVf + 16 * kFactors;

  __device__ static __forceinline__ int v_offset(int key, int byte) {
    if constexpr (D == 64) return key * kRow + byte;
    return (key >> 1) * 128 + ((((key & 1) << 2 | byte >> 4) ^ ((key >> 1 & 3) << 1)) << 4) + (byte & 15);
  }
  static constexpr int kPieces = 2 * kFactors;  // 16-byte pieces of a block's factors, K's and then V's
  // A unit's two blocks of 16 rows each (a page holds whole blocks).  Every lane
  // copies in every instruction: 2 kPieces lanes have the factors of both blocks,
  // and at D = 64 the other half copies the same pieces once more.
  __device__ static __forceinline__ void fill(const LanePtrs& a, uint32_t stage, const int (&block)[2], int lane) {
    const int byte = lane * 16;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint8_t* ks = a.data[0] + static_cast<long long>(block[k]) * kV;
      const uint8_t* vs = a.data[1] + static_cast<long long>(block[k]) * kV;
      const uint32_t to_k = stage + k * kBytes + byte;
      const uint32_t to_v = stage + k * kBytes + kV + v_offset(byte / kRow, byte % kRow);
#pragma unroll
      for (int i = 0; i < kV / 512; ++i) {  // 512 bytes on: 8 or 16 keys on, where the pieces lie alike
        copy16(to_k + i * 512, ks + i * 512);
        copy16(to_v + i * 512, vs + i * 512);
      }
    }
    const int which = lane / kPieces & 1;
    copy16(stage + which * kBytes + kKf + lane % kPieces * 16,
           a.factor + static_cast<long long>(which ? block[1] : block[0]) * (16 * kFactors));
  }
};

template <int D>
struct Tile<D, kFp4> {
  // 4 bits: K piece q of a row (D / 4 elements, D / 64 groups); V piece r (D / 8).
  static constexpr int kW = D / 32;  // 32-bit words of a K piece
  static constexpr int kU = D / 64;  // of a V piece
  uint32_t k[2][kW];
  uint32_t kf[2];      // factors of the piece's groups, one to a byte
  uint32_t v[4][kU];
  uint32_t vf[4];

  __device__ static __forceinline__ LanePtrs ptrs(const Params& p, int lane) {
    LanePtrs a;
    a.data[0] = p.data[0] + lane * 16;
    a.data[1] = p.data[1] + lane * 16;
    const int piece = lane % Stage<D>::kPieces;  // of a block's factors, as Stage::fill copies them
    a.factor = p.factor[piece / Stage<D>::kFactors] + piece % Stage<D>::kFactors * 16;
    return a;
  }
  __device__ __forceinline__ void load_k(uint32_t stage, int lane) {
    const int r = lane >> 2, q = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      lds(k[i], stage + (r + 8 * i) * (D / 2) + q * (D / 8));
      const uint32_t f = stage + Stage<D>::kKf + (r + 8 * i) * (D / 16) + q * (D / 64);
      kf[i] = D == 128 ? lds_u16(f) : lds_u8(f);
    }
  }
  // Keys from n_keys on get factor 0: whatever their slots hold does not count.
  template <bool WHOLE>
  __device__ __forceinline__ void load_v(uint32_t stage, int lane, int n_keys) {
    const int r = lane >> 2, q = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = 2 * q + (i & 1) + 8 * (i >> 1);
      lds(v[i], stage + Stage<D>::kV + Stage<D>::v_offset(key, r * (D / 16)));
      vf[i] = lds_u8(stage + Stage<D>::kVf + key * (D / 16) + r * (D / 8) / 16);
      if (!WHOLE && key >= n_keys) vf[i] = 0u;
    }
  }
  template <int NT>
  __device__ __forceinline__ void scores(float (&s)[NT][4], const uint32_t (&qf)[NT][D / 16][2]) const {
    const uint32_t f2[2] = {e4m3x2_to_f16(kf[0]), e4m3x2_to_f16(kf[1])};  // factors of the piece's groups
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      uint32_t a[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        e2m1_to_f16(k[i][w], a[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) a[i][e] = hmul2_half(a[i][e], f2[i], w >= 2);  // exact: 2 by 4 significant bits
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint32_t(&q0)[2] = qf[t][2 * w], (&q1)[2] = qf[t][2 * w + 1];
        if (w == 0) {
          mma16816_first<false>(s[t], a[0][0], a[1][0], a[0][1], a[1][1], q0[0], q0[1]);
        } else {
          mma16816<false>(s[t], a[0][0], a[1][0], a[0][1], a[1][1], q0[0], q0[1]);
        }
        mma16816<false>(s[t], a[0][2], a[1][2], a[0][3], a[1][3], q1[0], q1[1]);
      }
    }
  }
  // Product j holds elements (D / 8) r + 2 j (rows r) and the next (rows r + 8).
  template <int NT>
  __device__ __forceinline__ void values(float (&o)[NT][D / 16][4], const uint32_t (&pf)[NT][1][2]) const {
    const uint32_t f01 = e4m3x2_to_f16(vf[0] + vf[1] * 256u), f23 = e4m3x2_to_f16(vf[2] + vf[3] * 256u);
#pragma unroll
    for (int w = 0; w < kU; ++w) {
      // Bytes (key a, key b) for the even elements, then for the odd ones.
      uint32_t lo0[4], lo1[4], hi0[4], hi1[4];
      e2m1_to_f16((v[0][w] & 0x0F0F0F0Fu) | ((v[1][w] * 16u) & 0xF0F0F0F0u), lo0);
      e2m1_to_f16(((v[0][w] >> 4) & 0x0F0F0F0Fu) | (v[1][w] & 0xF0F0F0F0u), lo1);
      e2m1_to_f16((v[2][w] & 0x0F0F0F0Fu) | ((v[3][w] * 16u) & 0xF0F0F0F0u), hi0);
      e2m1_to_f16(((v[2][w] >> 4) & 0x0F0F0F0Fu) | (v[3][w] & 0xF0F0F0F0u), hi1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a0 = hmul2(lo0[j], f01), a1 = hmul2(lo1[j], f01);
        const uint32_t a2 = hmul2(hi0[j], f23), a3 = hmul2(hi1[j], f23);
#pragma unroll
        for (int t = 0; t < NT; ++t) mma16816<false>(o[t][4 * w + j], a0, a1, a2, a3, pf[t][0][0], pf[t][0][1]);
      }
    }
  }
  __device__ static __forceinline__ int k_element(int i, int lane) { return (D / 4) * (lane & 3) + 8 * i; }
  __device__ static __forceinline__ int o_element(int j, int lane, int half) {
    return (D / 8) * (lane >> 2) + 2 * j + half;
  }
};

// Stages of a warp's ring (4-bit caches), each of 32 keys: 4608 bytes at D = 128,
// where two take 205 us at the large batch and three 209; at D = 64, half the bytes,
// three take 127 and two 129.
template <int D>
constexpr int kStages = D == 128 ? 2 : 3;

// Units whose rows of a 16-bit cache a warp holds or has on their way.  At d = 128 two
// take the registers of a third CTA on an SM (four sequences of 4000 tokens in
// clusters: 15.4 -> 17.4 us, one of 8000 19.7 -> 16.0, where the list takes 12); at
// d = 64 24 sequences of 2000 tokens, 64 heads on 8, take 21.2 us with one and 18.6
// with two, and the list with 16 heads a unit 341 and 336 at the large batch, but
// with 8 heads 325 and 333.
template <int D, int NT, bool SHORT>
constexpr int kDepth = D == 64 && (SHORT || NT == 2) ? 2 : 1;

// Blocks of 16 keys that a warp works on at a time.
template <int FMT>
constexpr int kBlocks = FMT == kFp4 ? 2 : 1;
template <int FMT>
constexpr int kUnitKeys = 16 * kBlocks<FMT> * kWarps;
// Units of work that a segment's fixed part (its first pages and rows, Q, the
// merge of the warps) counts as when the list is divided; without it the CTAs
// whose run holds many short sequences end last.  The large batch, us, with 0, with
// 1, with this and with 2 more (d = 128; d = 64):
//   4 bits, 8 heads a unit   212, 206, 205, 208; 131, 127, 127, 128
//   4 bits, 16 heads         309, 299, 277, 277; 183, 178, 165, 166
//   16 bits, 8 heads         631, -, 630, 628; 325, -, 325, 325
//   16 bits, 16 heads        714, 705, 689, 690; 353, 348, 336, 337
template <int FMT, int NT>
constexpr int kSegmentCost = (FMT == kFp4 ? 3 : 1) + 2 * (NT - 1);

// Scores s of KB blocks of 16 keys (in units of the products) to P as the operand
// of P V, and the state (m, l, o) brought up to them.  A block's keys from
// n_keys on do not count (WHOLE: there are none).
template <int D, int FMT, bool WHOLE, int KB, int NT>
__device__ __forceinline__ void softmax_step(float (&s)[KB][NT][4], const float (&lam)[NT][2], int r, const int (&n_keys)[KB],
                                             float (&m)[NT][2], float (&l)[NT][2], float (&o)[NT][D / 16][4],
                                             uint32_t (&pf)[KB][NT][kTerms<FMT>][2]) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    // Exponents relative to the reference; it moves (for the whole warp) only
    // where one of them is above the threshold.
    float x[KB][4];
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < KB; ++k)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        x[k][c] = fmaf(s[k][t][c], lam[t][c & 1], -m[t][c & 1]);
        if (!WHOLE && r + 8 * (c >> 1) >= n_keys[k]) x[k][c] = -INFINITY;
        top = fmaxf(top, x[k][c]);
      }
    if (__any_sync(0xffffffffu, top > kRescaleThreshold)) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float mx = kNoReference;
#pragma unroll
        for (int k = 0; k < KB; ++k) {
          // The score itself, or for a key that does not count: no reference.
#pragma unroll
          for (int e = c; e < 4; e += 2)
            if (WHOLE || r + 8 * (e >> 1) < n_keys[k]) mx = fmaxf(mx, s[k][t][e] * lam[t][c]);
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        if (mx > m[t][c]) {
          const float gamma = ex2_approx(m[t][c] - mx);  // 0 for the first keys (m = kNoReference)
          m[t][c] = mx;
          l[t][c] *= gamma;
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            o[t][j][c] *= gamma;
            o[t][j][2 + c] *= gamma;
          }
        }
#pragma unroll
        for (int k = 0; k < KB; ++k)
#pragma unroll
          for (int e = c; e < 4; e += 2)
            if (WHOLE || r + 8 * (e >> 1) < n_keys[k]) x[k][e] = fmaf(s[k][t][e], lam[t][c], -m[t][c]);
      }
    }
#pragma unroll
    for (int k = 0; k < KB; ++k) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        x[k][c] = ex2_approx(x[k][c]);
        l[t][c & 1] += x[k][c];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t w = pack2<FMT == kBf16>(x[k][2 * i], x[k][2 * i + 1]);
        pf[k][t][0][i] = transpose8x8(w);
        if constexpr (kTerms<FMT> == 2) {
          const float2 v = unpack2<FMT == kBf16>(w);
          pf[k][t][1][i] = transpose8x8(pack2<FMT == kBf16>(x[k][2 * i] - v.x, x[k][2 * i + 1] - v.y));
        }
      }
    }
  }
}

// Writes elements e, e + 1 of a row of o from their weighted sum, and its lse.
__device__ __forceinline__ void finish(const Params& p, long long row_g, int d, int e, float a0, float a1, float M,
                                       float ls) {
  const float inv = ls > 0.f ? 1.f / ls : (ls == 0.f ? 0.f : ls);
  *reinterpret_cast<uint32_t*>(p.o + row_g * d + e) =
      p.out_bf16 ? pack2<true>(a0 * inv, a1 * inv) : pack2<false>(a0 * inv, a1 * inv);
  if (e == 0 && p.lse != nullptr) p.lse[row_g] = ls == 0.f ? -INFINITY : (M + log2f(ls)) * 0.69314718055994531f;
}

constexpr int kMaxCluster = 8;

__device__ __forceinline__ uint32_t cluster_ctas() {
  uint32_t n;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}
__device__ __forceinline__ float2 ld_cluster(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}

// Dynamic shared memory of a CTA.
template <int D, int FMT, int NT>
struct Smem {
  static constexpr int kRing = FMT == kFp4 ? kStages<D> * kBlocks<FMT> * Stage<D>::kBytes : 0;
  static constexpr int kStates = 8 * NT * (D + 4) * 4;  // of a warp
  static constexpr int kBytes = kWarps * (kRing > kStates ? kRing : kStates);
};

// CTAs of four warps that an SM holds at least, which bounds the registers.  The
// large batch, us, with 8 and with 16 query heads a unit (in brackets: CTAs; *: some
// registers spill, bytes stored):
//   d = 64, 16 bits: 326 (4), 325 (5, *28), 344 (6, *136) and 375 (2), 336 (3), 505 (4, *380)
//   d = 64, 4 bits: 128 (3), 127 (4), 132 (5) and 187 (2), 165 (3), 176 (4)
//   d = 128, 16 bits: 655 (2), 630 (3), 731 (4, *200) and 689 (2), 915 (3, *312)
//   d = 128, 4 bits: 201 (3), 205 (4), 217 (5, *108) and 277 (2), 288 (3, *40)
// Kept although it spills: d = 64, 16 bits, the list with 8 heads (28 bytes, even
// with 4 CTAs that do not) and clusters with 16 (12 bytes).
// d = 128 over 4 bits: three CTAs gain 2 % here and up to 13 % on one sequence
// (32000 tokens 16.5 -> 14.3), and lose 3 % on 64 short ones of 80 heads on 16.
template <int D, int FMT, int NT, bool SHORT>
constexpr int kResident = D == 64 ? (FMT != kFp4 && kDepth<D, NT, SHORT> == 1 ? 6 : 5) - NT
                                  : FMT == kFp4 && NT == 1 ? 4 : 4 - NT;

// SHORT: a cluster for each segment, its CTAs take equal runs of the segment's
// units and fold their states through shared memory.
template <int D, int FMT, int NT, bool SHORT>
__global__ void __launch_bounds__(kThreads, kResident<D, FMT, NT, SHORT>)
    decode_paged_kernel(const __grid_constant__ Params p) {
  using C = Smem<D, FMT, NT>;
  constexpr int KB = kBlocks<FMT>, UK = kUnitKeys<FMT>;
  // The warps' rings (4 bits), and at a segment's end their states.
  extern __shared__ __align__(128) uint8_t sm_raw[];
  auto sm_o = reinterpret_cast<float (*)[8 * NT][D + 4]>(sm_raw);
  __shared__ float sm_ml[kWarps][8 * NT][2];
  [[maybe_unused]] __shared__ float2 sm_fold[8 * NT];
  __shared__ long long sm_scan[kWarps + 1];
  __shared__ int sm_b;
  __shared__ long long sm_before;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const int r = lane >> 2, q4 = lane & 3;
  wait_for_previous_kernel();
  if constexpr (!SHORT) let_next_kernel_start();
  const int HG = p.Hkv * p.groups;
  [[maybe_unused]] const uint32_t ring = smem_u32(sm_raw) + warp * C::kRing;
  const LanePtrs src = Tile<D, FMT>::ptrs(p, lane);

  // ---- this CTA's run of units, [u0, u1) of U, and the sequence that holds u0
  long long U = 0, N = 0, u0 = 0, u1 = 1, rem = 0;
  int b, cost = 0, hg = 0, at = 0, n_units = 0;
  [[maybe_unused]] int rank = 0, ranks = 1;
  if constexpr (SHORT) {
    rank = static_cast<int>(cluster_ctarank());
    ranks = static_cast<int>(cluster_ctas());
    const int segment = blockIdx.x / ranks;
    b = segment / HG;
    hg = segment % HG;
  } else {
    // Tiles of a sequence and, in the upper bits, whether it has any: summed up,
    // tiles and sequences with keys.
    constexpr int kShift = 44;
    auto tiles_of = [&](int i) {
      const int n = i < p.B ? (seq_len(p, i) + UK - 1) / UK : 0;
      return n > 0 ? (1ll << kShift) + n : 0ll;
    };
    auto units_of = [&](long long x) { return (x & ((1ll << kShift) - 1)) + cost * (x >> kShift); };
    auto scan = [&](long long n, long long before, long long& all) {
      long long incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) sm_scan[warp] = incl;
      __syncthreads();
      incl += before;
      all = before;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) incl += sm_scan[w];
        all += sm_scan[w];
      }
      return incl;
    };
    // The first kThreads sequences are scanned, the others summed.
    int i = threadIdx.x;
    long long n = tiles_of(i), upto;
    const long long first = scan(n, 0, upto);
    long long total = upto;
    if (p.B > kThreads) {
      long long mine = 0;
      for (int j = i + kThreads; j < p.B; j += kThreads) mine += tiles_of(j);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
      __syncthreads();
      if (lane == 0) sm_scan[warp] = mine;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) total += sm_scan[w];
      __syncthreads();
    }
    cost = 0;
    if (units_of(total) * HG > gridDim.x) cost = kSegmentCost<FMT, NT>;
    U = units_of(total) * HG;
    N = min(static_cast<long long>(gridDim.x), U);
    if (blockIdx.x >= N) return;
    u0 = U * blockIdx.x / N;
    u1 = U * (blockIdx.x + 1) / N;
    const long long t0 = u0 / HG;  // < units_of(total), so the search ends
    long long incl = first, all = upto;
    for (;;) {
      const long long before = units_of(incl - n);
      if (t0 >= before && t0 < units_of(incl)) {
        sm_b = i;
        sm_before = before;
      }
      if (t0 < units_of(all)) break;
      i += kThreads;
      n = tiles_of(i);
      __syncthreads();
      incl = scan(n, all, all);
    }
    __syncthreads();
    b = sm_b;
    rem = u0 - sm_before * HG;
  }
  // Position in the segment: `cost` units that stand for its fixed work, then its tiles.
  if constexpr (!SHORT) {
    n_units = (seq_len(p, b) + UK - 1) / UK + cost;
    hg = static_cast<int>(rem / n_units);
    at = static_cast<int>(rem % n_units);
  }

  for (long long u = u0; u < u1;) {
    const int L = seq_len(p, b);
    const int n_tiles = (L + UK - 1) / UK;
    n_units = n_tiles + cost;
    int at_end = 0, tile, tile_end;
    if constexpr (SHORT) {
      tile = static_cast<int>(static_cast<long long>(n_tiles) * rank / ranks);
      tile_end = static_cast<int>(static_cast<long long>(n_tiles) * (rank + 1) / ranks);
    } else {
      at_end = static_cast<int>(min(static_cast<long long>(n_units), at + (u1 - u)));
      tile = max(0, at - cost), tile_end = at_end - cost;
      if (tile_end <= tile) break;  // the run ends before the segment's first tile
    }
    const int kvh = hg / p.groups, grp = hg % p.groups;
    const int head0 = kvh * p.g + grp * kMaxGroup;
    const int n_heads = min(kMaxGroup, p.g - grp * kMaxGroup);
    if constexpr (SHORT) {
      if (L == 0) {  // for all CTAs of the cluster alike
        const long long row0 = static_cast<long long>(b) * p.Hq + head0;
        if (rank == 0) {
          for (int i = threadIdx.x; i < n_heads * (D / 2); i += kThreads)
            *reinterpret_cast<uint32_t*>(p.o + row0 * D + 2 * i) = 0u;
          if (p.lse != nullptr && static_cast<int>(threadIdx.x) < n_heads) p.lse[row0 + threadIdx.x] = -INFINITY;
        }
        return;
      }
    }

    // ---- Q as the products' B operand, in the element order of K; read once the
    // first keys are on their way
    uint32_t qf[NT][D / 16][2];
    float lam[NT][2];  // base-2 units of a score, for the lane's two query columns
    auto load_q = [&] {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int row = 8 * t + r;
        const uint16_t* qrow = p.q + (static_cast<long long>(b) * p.Hq + head0 + row) * D;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint4 w = row < n_heads ? *reinterpret_cast<const uint4*>(qrow + Tile<D, FMT>::k_element(i, lane))
                                        : make_uint4(0u, 0u, 0u, 0u);
          qf[t][2 * i][0] = w.x;
          qf[t][2 * i][1] = w.y;
          qf[t][2 * i + 1][0] = w.z;
          qf[t][2 * i + 1][1] = w.w;
        }
        lam[t][0] = lam[t][1] = p.scale_log2;
        if constexpr (FMT == kFp4) {
          // The products are in fp16: scale the row by a power of two that brings
          // its largest element to [1, 2).  Exact for bf16 too, but for elements
          // under 2^-14 of the largest, which keep an error of 2^-25 of it.
          float2 f[D / 16][2];
          float top = 0.f;
#pragma unroll
          for (int st = 0; st < D / 16; ++st)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              f[st][h] = p.out_bf16 ? unpack2<true>(qf[t][st][h]) : unpack2<false>(qf[t][st][h]);
              top = fmaxf(top, fmaxf(fabsf(f[st][h].x), fabsf(f[st][h].y)));
            }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          // Exponent field in [2, 252]: both the factor and its inverse are normal.
          const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23), 2), 252);
          const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
          const float up = __uint_as_float(static_cast<uint32_t>(e) << 23);
#pragma unroll
          for (int st = 0; st < D / 16; ++st)
#pragma unroll
            for (int h = 0; h < 2; ++h) qf[t][st][h] = pack2<false>(f[st][h].x * down, f[st][h].y * down);
          const float kd = p.descale[0] != nullptr ? p.descale[0][kvh] : 1.f;
          const float row_lam = p.scale_log2 * kd * up;
          lam[t][0] = __shfl_sync(0xffffffffu, row_lam, 8 * q4);
          lam[t][1] = __shfl_sync(0xffffffffu, row_lam, 8 * q4 + 4);
        }
      }
    };

    float o[NT][D / 16][4];
    float m[NT][2], l[NT][2];  // per query column; l is this lane's share of the sum
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j) o[t][j][0] = o[t][j][1] = o[t][j][2] = o[t][j][3] = 0.f;
      m[t][0] = m[t][1] = kNoReference;
      l[t][0] = l[t][1] = 0.f;
    }

    // ---- the keys: piece 4 i + warp, of KB blocks of 16 keys, of every unit i
    const int* pages = p.page_table + static_cast<long long>(b) * p.max_pages;
    const int warp_keys = L - warp * (16 * KB);  // keys from this warp's first one on
    const int end = min(tile_end, (warp_keys + UK - 1) / UK);
    const int whole_end = (warp_keys + UK - 16 * KB) / UK;  // units before it have all of the warp's keys
    const int block_shift = p.page_shift - 4;               // log2 of a page's blocks
    const int head_block = kvh << block_shift, page_blocks = p.Hkv << block_shift;
    const int last_block = (L - 1) >> 4;
    // Page of a block of the sequence (behind the last: the last one's), and the
    // pool's block, or -1 for a page that does not exist: its keys are left out.
    auto page_of = [&](int blk) { return pages[min(blk, last_block) >> block_shift]; };
    auto exists = [&](int page) { return static_cast<unsigned>(page) < static_cast<unsigned>(p.n_pages); };
    auto block_at = [&](int blk, int page) {
      return page * page_blocks + head_block + (blk & ((1 << block_shift) - 1));
    };
    auto block_of = [&](int blk, int page) {
      if (exists(page)) return block_at(blk, page);
      if (lane == 0) report_index(p.status);
      return -1;
    };
    if constexpr (FMT == kFp4) {
      Tile<D, FMT> tl;
      // kStages<D> - 1 units are on their way while one is worked on.
      int page0 = page_of((tile * kWarps + warp) * KB), page1 = page_of((tile * kWarps + warp) * KB + 1);
      unsigned absent = 0;  // two bits a request, the newest lowest: block k has no page
      auto request = [&](int i, uint32_t stage) {
        absent <<= 2;
        if (i < end) {
          const int blk = (i * kWarps + warp) * KB;
          int block[KB] = {block_at(blk, page0), block_at(blk + 1, page1)};
          if (!exists(page0) || !exists(page1)) {
            if (lane == 0) report_index(p.status);
            absent |= (exists(page0) ? 0u : 1u) | (exists(page1) ? 0u : 2u);
            // What is copied instead does not matter.
            if (!exists(page0)) block[0] = 0;
            if (!exists(page1)) block[1] = 0;
          }
          page0 = page_of(blk + kWarps * KB);
          page1 = block_shift > 0 ? page0 : page_of(blk + kWarps * KB + 1);
          Stage<D>::fill(src, stage, block, lane);
        }
        copy_commit();
      };
      constexpr uint32_t kUnitBytes = KB * Stage<D>::kBytes;
#pragma unroll
      for (int i = 0; i < kStages<D> - 1; ++i) request(tile + i, ring + i * kUnitBytes);
      load_q();
      uint32_t stage = ring, free_stage = ring + (kStages<D> - 1) * kUnitBytes;
      for (int i = tile; i < end; ++i) {
        copy_wait<kStages<D> - 2>();
        __syncwarp();  // every lane's copies of unit i, and every lane done with unit i - 1
        request(i + kStages<D> - 1, free_stage);
        auto step = [&](auto whole, int n0, int n1) {
          const int n_keys[KB] = {n0, n1};
          float s[KB][NT][4];
          uint32_t pf[KB][NT][1][2];
#pragma unroll
          for (int k = 0; k < KB; ++k) {
            tl.load_k(stage + k * Stage<D>::kBytes, lane);
            tl.template scores<NT>(s[k], qf);
          }
          softmax_step<D, FMT, decltype(whole)::value, KB, NT>(s, lam, r, n_keys, m, l, o, pf);
#pragma unroll
          for (int k = 0; k < KB; ++k) {
            tl.template load_v<decltype(whole)::value>(stage + k * Stage<D>::kBytes, lane, n_keys[k]);
            tl.template values<NT>(o, pf[k]);
          }
        };
        const unsigned gone = absent >> (2 * (kStages<D> - 1)) & 3;
        const int left = warp_keys - i * UK;
        if (i < whole_end && gone == 0)
          step(std::true_type(), 16, 16);
        else
          step(std::false_type(), gone & 1 ? 0 : left, gone & 2 ? 0 : left - 16);
        free_stage = stage;
        stage = stage == ring + (kStages<D> - 1) * kUnitBytes ? ring : stage + kUnitBytes;
      }
      copy_wait<0>();
    } else {
      // A unit's K is requested right after the scores of the unit whose registers it
      // takes, and its V right after that one's P V.
      constexpr int kAhead = kDepth<D, NT, SHORT>;
      Tile<D, FMT> tl[kAhead];
      int n_keys[kAhead][1], page[kAhead] = {};  // page: of the unit kAhead further
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (tile + k < end) page[k] = page_of((tile + k) * kWarps + warp);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        n_keys[k][0] = 0;
        if (tile + k < end) {
          const int blk = (tile + k) * kWarps + warp, block = block_of(blk, page[k]);
          n_keys[k][0] = block < 0 ? 0 : L - 16 * blk;
          page[k] = page_of(blk + kAhead * kWarps);
          tl[k].load_k(src, block, lane, n_keys[k][0]);
          tl[k].load_v(src, block, lane, n_keys[k][0]);
        }
      }
      load_q();
      for (int i0 = tile; i0 < end; i0 += kAhead) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int i = i0 + k;
          if (k > 0 && i >= end) break;
          float s[1][NT][4];
          uint32_t pf[1][NT][kTerms<FMT>][2];
          tl[k].template scores<NT>(s[0], qf);
          int n_next = 0, block = 0;
          if (i + kAhead < end) {
            const int blk = (i + kAhead) * kWarps + warp;
            block = block_of(blk, page[k]);
            n_next = block < 0 ? 0 : L - 16 * blk;
            page[k] = page_of(blk + kAhead * kWarps);
            tl[k].load_k(src, block, lane, n_next);
          }
          softmax_step<D, FMT, false, 1, NT>(s, lam, r, n_keys[k], m, l, o, pf);
          tl[k].template values<NT>(o, pf[0]);
          if (i + kAhead < end) tl[k].load_v(src, block, lane, n_next);
          n_keys[k][0] = n_next;
        }
      }
    }

    // ---- the four warps' states into one
    if constexpr (FMT == kFp4) __syncthreads();  // the states take the rings' place
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float v = l[t][c];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        const int row = 8 * t + 2 * q4 + c;
        if (r == 0) {
          sm_ml[warp][row][0] = m[t][c];
          sm_ml[warp][row][1] = v;
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          sm_o[warp][row][Tile<D, FMT>::o_element(j, lane, 0)] = o[t][j][c];
          sm_o[warp][row][Tile<D, FMT>::o_element(j, lane, 1)] = o[t][j][2 + c];
        }
      }
    __syncthreads();
    const bool whole = tile == 0 && tile_end == n_tiles;
    const int slot = u == u0 ? 0 : 1;
    const float vd = FMT == kFp4 && p.descale[1] != nullptr ? p.descale[1][kvh] : 1.f;
    for (int idx = threadIdx.x; idx < n_heads * (D / 2); idx += kThreads) {
      const int row = idx / (D / 2), e = 2 * (idx % (D / 2));
      float M = kNoReference;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_ml[w][row][0]);
      float a0 = 0.f, a1 = 0.f, ls = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2_approx(sm_ml[w][row][0] - M);  // NaN stays NaN where f is 0
        a0 = fmaf(f, sm_o[w][row][e], a0);
        a1 = fmaf(f, sm_o[w][row][e + 1], a1);
        ls = fmaf(f, sm_ml[w][row][1], ls);
      }
      a0 *= vd;
      a1 *= vd;
      if (SHORT && ranks > 1) {  // in the place of the first warp's state
        *reinterpret_cast<float2*>(&sm_o[0][row][e]) = make_float2(a0, a1);
        if (e == 0) sm_fold[row] = make_float2(M, ls);
      } else if (whole) {
        finish(p, static_cast<long long>(b) * p.Hq + head0 + row, D, e, a0, a1, M, ls);
      } else {
        const long long st = (static_cast<long long>(blockIdx.x) * 2 + slot) * p.rows + row;
        *reinterpret_cast<float2*>(p.part_o + st * D + e) = make_float2(a0, a1);
        if (e == 0) *reinterpret_cast<float2*>(p.part_ml + st * 2) = make_float2(M, ls);
      }
    }
    if constexpr (SHORT) {
      if (ranks == 1) return;
      cluster_sync_all();
      // Every CTA folds a share of the elements, in the order of the ranks.
      for (int idx = rank * kThreads + threadIdx.x; idx < n_heads * (D / 2); idx += ranks * kThreads) {
        const int row = idx / (D / 2), e = 2 * (idx % (D / 2));
        float2 ml[kMaxCluster], v[kMaxCluster];
        float M = kNoReference;
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k)
          if (k < ranks) {
            ml[k] = ld_cluster(mapa_shared(&sm_fold[row], k));
            v[k] = ld_cluster(mapa_shared(&sm_o[0][row][e], k));
            M = fmaxf(M, ml[k].x);
          }
        float a0 = 0.f, a1 = 0.f, ls = 0.f;
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k)
          if (k < ranks) {
            const float f = ex2_approx(ml[k].x - M);
            a0 = fmaf(f, v[k].x, a0);
            a1 = fmaf(f, v[k].y, a1);
            ls = fmaf(f, ml[k].y, ls);
          }
        finish(p, static_cast<long long>(b) * p.Hq + head0 + row, D, e, a0, a1, M, ls);
      }
      cluster_sync_all();  // no CTA leaves before the others have read its state
      return;
    }
    if (threadIdx.x == 0 && tile == 0) {
      const long long last = u - at + n_units - 1;  // the segment's last unit
      const int n_parts = whole ? 0 : static_cast<int>(((last + 1) * N - 1) / U) - static_cast<int>(blockIdx.x) + 1;
      p.parts[static_cast<long long>(b) * HG + hg] = make_int2(static_cast<int>(blockIdx.x) * 2 + slot, n_parts);
    }
    __syncthreads();

    u += at_end - at;
    at = 0;
    if (u < u1) {
      if (++hg == HG) {
        hg = 0;
        do ++b;
        while (seq_len(p, b) == 0);  // a unit is left, so a sequence with keys follows
      }
    }
  }
}

constexpr int kMergeThreads = 256;

// Where a (sequence, query head)'s parts lie.
struct Parts {
  int first, n, rows, row;  // first CTA * 2 + slot; number of parts (0: finished, or an empty sequence)
  bool empty;
  // Part 0 is in the first CTA's slot; the others in slot 0 of the next CTAs.
  __device__ __forceinline__ long long state(int i) const {
    return (i == 0 ? first : (first / 2 + i) * 2) * static_cast<long long>(rows) + row;
  }
};
__device__ __forceinline__ Parts parts_of(const Params& p, int row_g) {
  const int b = row_g / p.Hq, hq = row_g % p.Hq, kvh = hq / p.g, in_g = hq % p.g;
  const int hg = kvh * p.groups + in_g / kMaxGroup;
  Parts a;
  const int2 part = p.parts[static_cast<long long>(b) * p.Hkv * p.groups + hg];  // anything for an empty sequence
  a.empty = seq_len(p, b) == 0;
  a.first = part.x;
  a.n = a.empty ? 0 : part.y;
  a.rows = p.rows;
  a.row = in_g % kMaxGroup;
  return a;
}

// N consecutive elements of a part's values, and of the output.
template <int N>
struct Piece {
  float x[N];
  __device__ __forceinline__ void load(const float* src) {
    if constexpr (N == 4) {
      const float4 v = *reinterpret_cast<const float4*>(src);
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(src);
      x[0] = v.x, x[1] = v.y;
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = 0.f;
  }
  __device__ __forceinline__ void add(float f, const Piece& v) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = fmaf(f, v.x[i], x[i]);
  }
  __device__ __forceinline__ void store(const Params& p, long long row_g, int d, int e, float M, float ls) const {
#pragma unroll
    for (int i = 0; i < N; i += 2) finish(p, row_g, d, e + i, x[i], x[i + 1], M, ls);
  }
};

// Fold the parts of segments that were split, in the order of the parts, and write
// the zeros of empty sequences (a part's NaN counts whatever its weight is, as it
// does in the formula); launched while the decode kernel runs, they wait
// for its end.  Bound by latency (place, then states and values, then their sum).
// With few rows there may be many parts to each: a CTA a row, its teams of D / 4
// threads taking parts in turn (57 parts of each of 32 rows: 3 us).
template <int D>
__global__ void __launch_bounds__(kMergeThreads) decode_paged_merge_cta_kernel(const __grid_constant__ Params p) {
  constexpr int kLanes = D / 4;                  // threads of a part's row
  constexpr int kTeams = kMergeThreads / kLanes; // parts read at a time
  constexpr int kMergeWarps = kMergeThreads / 32;
  constexpr int kAhead = 8;                      // parts of a thread requested before their weights are known
  __shared__ float weight[kMaxCtas];
  __shared__ float red[2][kMergeWarps];
  __shared__ Piece<4> sum[kTeams][kLanes];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int team = threadIdx.x / kLanes, e = threadIdx.x % kLanes * 4;
  wait_for_previous_kernel();
  const Parts a = parts_of(p, blockIdx.x);
  if (a.n == 0 && !a.empty) return;  // finished by one CTA
  Piece<4> v[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    v[u].clear();
    if (team + u * kTeams < a.n) v[u].load(p.part_o + a.state(team + u * kTeams) * D + e);
  }
  float M = kNoReference, ls = 0.f;
  for (int i = threadIdx.x; i < a.n; i += kMergeThreads) M = fmaxf(M, p.part_ml[a.state(i) * 2]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) red[0][warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) M = fmaxf(M, red[0][w]);
  for (int i = threadIdx.x; i < a.n; i += kMergeThreads) {
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + a.state(i) * 2);
    const float f = ex2_approx(ml.x - M);
    weight[i] = f;
    ls = fmaf(f, ml.y, ls);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
  if (lane == 0) red[1][warp] = ls;
  __syncthreads();
  ls = 0.f;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) ls += red[1][w];
  Piece<4> acc;
  acc.clear();
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (team + u * kTeams < a.n) acc.add(weight[team + u * kTeams], v[u]);
#pragma unroll 4
  for (int i = team + kAhead * kTeams; i < a.n; i += kTeams) {
    v[0].load(p.part_o + a.state(i) * D + e);
    acc.add(weight[i], v[0]);
  }
  sum[team][threadIdx.x % kLanes] = acc;
  __syncthreads();
  if (team != 0) return;
#pragma unroll
  for (int i = 1; i < kTeams; ++i) acc.add(1.f, sum[i][threadIdx.x]);
  acc.store(p, blockIdx.x, D, e, M, ls);
}

// With many rows most are finished, and the split ones have few parts: a warp a row.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) decode_paged_merge_warp_kernel(const __grid_constant__ Params p) {
  constexpr int kAhead = 4;
  const int row_g = blockIdx.x * (kMergeThreads / 32) + threadIdx.x / 32, lane = threadIdx.x % 32;
  wait_for_previous_kernel();
  if (row_g >= p.B * p.Hq) return;
  const Parts a = parts_of(p, row_g);
  if (a.n == 0 && !a.empty) return;
  const int e = lane * (D / 32);
  Piece<D / 32> v[kAhead], acc;
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (u < a.n) v[u].load(p.part_o + a.state(u) * D + e);
  float M = kNoReference, ls = 0.f;
  for (int i = lane; i < a.n; i += 32) M = fmaxf(M, p.part_ml[a.state(i) * 2]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  acc.clear();
  for (int base = 0; base < a.n; base += 32) {
    float f = 0.f;
    if (base + lane < a.n) {
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + a.state(base + lane) * 2);
      f = ex2_approx(ml.x - M);
      ls = fmaf(f, ml.y, ls);
    }
    const int m = min(32, a.n - base);
#pragma unroll 8
    for (int i = 0; i < m; ++i) {
      const float fi = __shfl_sync(0xffffffffu, f, i);
      if (base == 0 && i < kAhead) continue;  // below, from what was requested ahead
      Piece<D / 32> x;
      x.load(p.part_o + a.state(base + i) * D + e);
      acc.add(fi, x);
    }
    if (base == 0) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const float fu = __shfl_sync(0xffffffffu, f, u);
        if (u < a.n) acc.add(fu, v[u]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
  acc.store(p, row_g, D, e, M, ls);
}

int group_rows(int Hq, int Hkv) {
  const int g = Hq / Hkv;
  return g < kMaxGroup ? g : kMaxGroup;
}

int unit_groups(int Hq, int Hkv) { return (Hq / Hkv + kMaxGroup - 1) / kMaxGroup; }

// CTAs that can have work: one for each unit at most (the smallest unit is 64 keys).
int max_ctas(int B, size_t heads, int max_len) {
  const size_t units = B * heads * ((static_cast<size_t>(max_len) + 63) / 64);
  return units < kMaxCtas ? static_cast<int>(units) : kMaxCtas;
}

// CTAs of a cluster that takes a whole segment, or 0 where the list of all units is
// divided instead.  The host knows what the pages of a sequence can hold, not the
// lengths, so a cluster is for tables of few units: it saves the division and the
// second kernel (6.4 -> 4.7 us for one sequence of 4 units, 10.4 -> 7 us of host
// time), and loses where one cluster has much more to do than a CTA's even share,
// half of which is taken off for ragged batches.  Measured with 32 heads on 8,
// d = 128, 16 bits, us (list against clusters), lengths of 0 up to what the table
// holds:
//   8 sequences, 4 CTAs each: 16 units 10.0 / 8.6, 24 10.6 / 10.0, 32 12.8 / 13.1
//   24 sequences, 2 CTAs each: 8 units 12.3 / 10.4, 16 15.3 / 15.4, 24 17.7 / 19.6
//   48 sequences, a CTA each: 8 units 16.0 / 14.4, 12 about even, 24 28 / 32
// one sequence, 8 CTAs, equal lengths: 16 units 6.7 / 5.8, 32 7.3 / 7.2, 48 8.1 / 8.6.
// The same thresholds serve the other forms, where clusters would win further up.
// Of 42 batches of each form (1 to 96 sequences of up to 2 to 48 units, rows in L2)
// the choice is within 5 % of the best division in 33 (this form), 32 (16 heads a
// unit; 4 bits with 8), 31 (4 bits with 16) and 26 to 28 (d = 64); at worst, list
// against clusters of 8: d = 64, 8 sequences of up to 24 units in 16 bits 9.4 / 6.5,
// of 48 in 4 bits 9.7 / 7.0; d = 128, 4 sequences of up to 48 in 4 bits 11.2 / 8.8.
// Tables of two units get clusters of two where one CTA is faster by 0.4 to 1.5 us.
// With more segments than resident CTAs they take turns, and the last turn's
// idle places cost what the list does not lose: from four turns on clusters of
// one win at all 16 units tried (512 sequences 313 / 302, 4 bits 215 / 197); at
// 1.1 turns 16 bits win up to 4 units (17.8 / 16.9) and lose at 6 (22.1 / 23.2),
// 4 bits win up to 8 (1.7 turns: 39.1 / 32.2).
template <int FMT>
int short_cluster(const Params& p, int ctas) {
  const long long segments = static_cast<long long>(p.B) * p.Hkv * p.groups;
  const long long units = ((p.max_pages << p.page_shift) + kUnitKeys<FMT> - 1) / kUnitKeys<FMT>;
  if (segments > ctas) return units <= (segments >= 4LL * ctas ? 16 : FMT == kFp4 ? 8 : 4) ? 1 : 0;
  // Clusters of eight leave places of an SM group idle: 54 of them do not fit
  // where 432 CTAs would (15.6 us against 11.9 with four).
  int cluster = kMaxCluster;
  while (cluster > 1 && (segments * cluster > (cluster == kMaxCluster ? ctas * 3 / 4 : ctas) || cluster / 2 >= units))
    cluster /= 2;
  // units / cluster - units segments / (2 ctas) <= 4 (a cluster of one: 8)
  return units * (2 * ctas - segments * cluster) <= (cluster == 1 ? 16LL : 8LL) * ctas * cluster ? cluster : 0;
}

// CTAs of a kernel that fit on an SM; the same on every GPU this library runs on.
template <int D, int FMT, int NT, bool SHORT>
int resident() {
  constexpr int kBytes = Smem<D, FMT, NT>::kBytes;
  static std::atomic<unsigned long long> attr_done{0};  // per instantiation
  static std::atomic<int> fit{0};
  auto kern = decode_paged_kernel<D, FMT, NT, SHORT>;
  if (!set_smem_limit_once(kern, kBytes, attr_done)) return 0;
  int n = fit.load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kThreads, kBytes) != cudaSuccess || n < 1) {
      cudaGetLastError();
      return 0;
    }
    fit.store(n, std::memory_order_relaxed);
  }
  return n;
}

template <int D, int FMT, int NT>
int launch_t(const Params& p, const PagedDecodeArgs& a) {
  const int short_fit = resident<D, FMT, NT, true>();
  if (short_fit == 0) return -1;
  if (const int cluster = short_cluster<FMT>(p, short_fit * a.num_sms))
    return launch_after(decode_paged_kernel<D, FMT, NT, true>,
                        dim3(static_cast<unsigned>(p.B * p.Hkv * p.groups * cluster)), kThreads, a.stream, p,
                        Smem<D, FMT, NT>::kBytes, cluster);
  const int fit = resident<D, FMT, NT, false>();
  if (fit == 0) return -1;
  const int ctas = fit * a.num_sms < p.most_ctas ? fit * a.num_sms : p.most_ctas;
  if (launch_after(decode_paged_kernel<D, FMT, NT, false>, dim3(static_cast<unsigned>(ctas)), kThreads, a.stream, p,
                   Smem<D, FMT, NT>::kBytes) != 0)
    return -1;
  // A CTA a row while that is at most four CTAs for each SM.
  const int rows = a.B * a.Hq;
  if (rows <= 4 * a.num_sms)
    return launch_after(decode_paged_merge_cta_kernel<D>, dim3(static_cast<unsigned>(rows)), kMergeThreads, a.stream, p);
  constexpr int kRows = kMergeThreads / 32;
  return launch_after(decode_paged_merge_warp_kernel<D>, dim3(static_cast<unsigned>((rows + kRows - 1) / kRows)),
                      kMergeThreads, a.stream, p);
}

template <int D, int FMT>
int launch_d(const Params& p, const PagedDecodeArgs& a) {
  return p.rows > 8 ? launch_t<D, FMT, 2>(p, a) : launch_t<D, FMT, 1>(p, a);
}

}  // namespace

size_t paged_decode_workspace_bytes(int B, int Hq, int Hkv, int d, int max_len) {
  const size_t rows = group_rows(Hq, Hkv), heads = static_cast<size_t>(Hkv) * unit_groups(Hq, Hkv);
  return static_cast<size_t>(max_ctas(B, heads, max_len)) * 2 * rows * (static_cast<size_t>(d) + 2) * sizeof(float) +
         B * heads * sizeof(int2);
}

int launch_decode_paged(const PagedDecodeArgs& a) {
  Params p{};
  const CacheArgs& c = a.cache;
  p.q = static_cast<const uint16_t*>(a.q);
  for (int i = 0; i < 2; ++i) {
    p.data[i] = static_cast<const uint8_t*>(c.data[i]);
    p.factor[i] = static_cast<const uint8_t*>(c.scale[i]);
    p.descale[i] = c.descale[i];
  }
  p.page_table = c.page_table;
  p.seqlens = c.seqlens;
  p.o = static_cast<uint16_t*>(a.o);
  p.lse = a.lse;
  p.B = a.B;
  p.Hq = a.Hq;
  p.Hkv = c.Hkv;
  p.g = a.Hq / c.Hkv;
  p.groups = unit_groups(a.Hq, c.Hkv);
  p.most_ctas = max_ctas(a.B, static_cast<size_t>(c.Hkv) * p.groups, c.max_pages << c.page_shift);
  p.rows = group_rows(a.Hq, c.Hkv);
  p.page_shift = c.page_shift;
  p.n_pages = c.n_pages;
  p.max_pages = c.max_pages;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.out_bf16 = a.bf16 ? 1 : 0;
  p.status = a.status;
  float* ws = static_cast<float*>(a.workspace);
  const size_t states = static_cast<size_t>(p.most_ctas) * 2 * p.rows;
  p.part_o = ws;
  p.part_ml = ws + states * c.d;
  p.parts = reinterpret_cast<int2*>(ws + states * (c.d + 2));
  if (c.d == 128) {
    if (c.fp4()) return launch_d<128, kFp4>(p, a);
    return a.bf16 ? launch_d<128, kBf16>(p, a) : launch_d<128, kF16>(p, a);
  }
  if (c.fp4()) return launch_d<64, kFp4>(p, a);
  return a.bf16 ? launch_d<64, kBf16>(p, a) : launch_d<64, kF16>(p, a);
}

}  // namespace gbattn
