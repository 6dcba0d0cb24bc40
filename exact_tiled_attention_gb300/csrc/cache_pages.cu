// cache_pages.cu -- writing new keys and values into a paged cache, with the
// position rotation on the way, and reading a cache's sequences back as
// contiguous 16-bit tensors; for a cache held in 16 bits and one held in 4.
//
// Append: token i of sequence b stands at position p = seqlens[b] - new[b] + i
// and goes to slot p % page of page page_table[b][p / page]; keys (and queries,
// which go to q_out) are rotated by the table's row p in fp32 and rounded once.
// 4 bits: for each group of 16 elements, f = E4M3(min(448, max |x| / (6 descale)))
// and code = E2M1(x * (1 / (f descale))), both rounded to nearest even; f = 0
// gives codes of magnitude 0 with the elements' signs.  Division and reciprocal are
// the IEEE ones, so the codes are those of the same formula evaluated anywhere in
// fp32.
//
// Both are bound by HBM, or, for one token a sequence, by the launch (64 tokens of
// 32 + 16 heads: 1.7 us one behind another, 4.1 alone from memory).  A row is read
// once and written once; a thread keeps one token's angles and place and walks over
// heads.  Eight ragged prompts of up to 4096 tokens into 16 bits, 526 MB in all, take
// 88 us, 6.0 TB/s; chunks of 2048 tokens of four sequences into 4 bits 31 us, 5.7
// TB/s.  Reading contexts of up to 16384 tokens of four sequences back is nearly all
// writes: 50 us, 5.4 TB/s written (a fill of the same memory reaches 4.0); from 16
// bits [4, 8192] tokens of 16 heads take 79.5 us, 6.8 TB/s.  A partial rotation by
// halves reads each turning piece's partner again, when it is needed: [2, 4096]
// tokens of 32 + 16 heads 45 us into 16 bits and 48 into 4, where the other
// rotations take 33 and 31.
#include <cuda_runtime.h>

#include "gbattn_rows.cuh"

namespace gbattn {
namespace {

constexpr int kThreads = 128;

struct AppendParams {
  const uint16_t* x[3];  // q, k, v
  RowStrides xs[3];
  uint16_t* q_out;
  uint8_t* data[2];
  uint8_t* scale[2];
  const float* descale[2];
  const int* page_table;
  const int* seqlens;
  const int* new_lens;
  const float* table;
  int table_rows, rot;
  int B, S, heads[3], chunks[3], per_chunk;
  int page_shift, n_pages, max_pages;
  int* status;
};

__device__ __forceinline__ uint32_t e2m1x8(const float (&y)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return r;
}

__device__ __forceinline__ __half e4m3_half(uint32_t code) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(code & 0xFF)));
  return __ushort_as_half(static_cast<uint16_t>(h2 & 0xFFFF));
}

// The two E2M1 codes in the lowest byte, the low half first.
__device__ __forceinline__ __half2 e2m1x2_half2(uint32_t codes) {
  uint32_t h2;
  asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(h2) : "r"(codes));
  return *reinterpret_cast<const __half2*>(&h2);
}

// One chunk of 8 elements to 4 bits; the other half of its group of 16 is the
// neighbouring lane's.  Magnitudes are compared as integers, where a NaN is above
// infinity, so it goes through the maximum; the factor's bound then gives 448 and
// the conversion 6, as for infinity.
__device__ __forceinline__ uint32_t quantise8(const float (&z)[8], float descale, uint8_t& factor) {
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(z[i]) & 0x7FFFFFFFu);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  const float f = fminf(__fdiv_rn(__uint_as_float(top), __fmul_rn(6.f, descale)), 448.f);  // NaN: 448
  factor = static_cast<uint8_t>(pack4_e4m3(f, 0.f, 0.f, 0.f) & 0xFF);
  const float fv = __half2float(e4m3_half(factor));
  const float inv = fv > 0.f ? __frcp_rn(__fmul_rn(fv, descale)) : 0.f;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(z[i], inv);
  return e2m1x8(y);
}

// CTAs that an SM holds at least, which bounds the registers (64 and 72).  Without
// it and with one more each, us: [1, 2094] tokens of 64 + 8 heads in 16 bits 11.7, here
// 10.5, more 13.0 (spills); [4, 2048] of 32 + 16 in 4 bits 34.0, 31.2, 31.7.  A
// partial rotation holds its partners too and would spill.
template <int MODE, bool FP4>
constexpr int kResident = MODE == kRopePart ? 1 : FP4 ? 7 : 8;

template <int D, bool BF16, int MODE, bool FP4>
__global__ void __launch_bounds__(kThreads, kResident<MODE, FP4>) cache_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kLanes = RowCfg<D>::kLanes;
  constexpr int kRowsCta = kThreads / kLanes;
  const int lane_in_row = threadIdx.x % kLanes;
  const int e0 = 8 * lane_in_row;
  const int tokens = p.B * p.S;
  const int at = blockIdx.x * kRowsCta + static_cast<int>(threadIdx.x) / kLanes;
  const bool in_grid = at < tokens;
  const int t = min(at, tokens - 1);  // the whole warp stays for the shuffles
  const int b = t / p.S, i = t % p.S;
  // 0: queries, 1: keys, 2: values.  The CTAs that quantise take longest and start
  // first ([5, 1434] tokens of 40 + 16 heads, d = 64: 19.9 -> 17.4 us); in 16 bits that order costs (33.3 -> 35.9).
  int which = 0, chunk = blockIdx.y;
  if constexpr (FP4) {
    const int kv = p.chunks[1] + p.chunks[2];
    which = chunk < p.chunks[1] ? 1 : chunk < kv ? 2 : 0;
    chunk -= which == 1 ? 0 : which == 2 ? p.chunks[1] : kv;
  } else {
    while (which < 2 && chunk >= p.chunks[which]) chunk -= p.chunks[which++];
  }
  const int h0 = chunk * p.per_chunk;
  const int h1 = min(h0 + p.per_chunk, p.heads[which]);

  wait_for_previous_kernel();
  const int n_new = p.new_lens != nullptr ? min(p.new_lens[b], p.S) : p.S;
  const long long pos = static_cast<long long>(p.seqlens[b]) - n_new + i;
  const bool real = in_grid && i < n_new && pos >= 0;  // else padding
  if (which != 0 && __all_sync(0xffffffffu, !real)) return;  // nothing to store
  const RowStrides xs = p.xs[which];
  const uint16_t* xrow = p.x[which] + b * xs.b + i * xs.s + h0 * xs.h;
  // Rows are requested two heads ahead, the first ones before the page and the
  // angles are looked up; padding is not read.
  uint4 raw[2][2] = {};
  auto request = [&](int k, const uint16_t* row) {
    if (real) {
      raw[k][0] = *reinterpret_cast<const uint4*>(row + e0);
      raw[k][1] = *reinterpret_cast<const uint4*>(row + D / 2 + e0);
    }
  };
  request(0, xrow);
  if (h0 + 1 < h1) request(1, xrow + xs.h);
  bool stored = real;
  long long slot = 0;  // row of head 0 of the token's page
  if (real && which != 0) {
    const long long pg = pos >> p.page_shift;
    const int page = pg < p.max_pages ? p.page_table[static_cast<long long>(b) * p.max_pages + pg] : -1;
    if (page < 0 || page >= p.n_pages) {
      stored = false;
      report_index(p.status);
    } else {
      slot = ((static_cast<long long>(page) * p.heads[1]) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
    }
  }
  LaneRope rope;
  int pc[2] = {e0, D / 2 + e0};
  if constexpr (MODE != kRopeNone) {
    if (which != 2) {
      long long row = real ? pos : 0;
      if (row >= p.table_rows) {
        report_index(p.status);
        row = p.table_rows - 1;
      }
      load_rope<D, MODE>(rope, p.table + row * p.rot, p.rot, lane_in_row);
      if constexpr (MODE == kRopePart)
        for (int c = 0; c < 2; ++c) pc[c] = partner_chunk(c * (D / 2) + e0, p.rot);
    }
  }
  for (int h = h0; h < h1; ++h, xrow += xs.h) {
    float z[2][8], part[2][8];
    unpack8<BF16>(raw[0][0], z[0]);
    unpack8<BF16>(raw[0][1], z[1]);
    raw[0][0] = raw[1][0];
    raw[0][1] = raw[1][1];
    if (h + 2 < h1) request(1, xrow + 2 * xs.h);
    if constexpr (MODE != kRopeNone) {
      if (which != 2) {
        if constexpr (MODE == kRopePart) {
          uint4 other[2] = {};
          if (real && rope.turns[0]) other[0] = *reinterpret_cast<const uint4*>(xrow + pc[0]);
          if (real && rope.turns[1]) other[1] = *reinterpret_cast<const uint4*>(xrow + pc[1]);
          unpack8<BF16>(other[0], part[0]);
          unpack8<BF16>(other[1], part[1]);
          __syncwarp();  // q_out may be q: the row's other lanes write what this one has just read
        }
        rotate<MODE, false>(z, part, rope);
      }
    }
    if (which == 0) {
      if (in_grid) {
        uint16_t* y = p.q_out + ((static_cast<long long>(b) * p.heads[0] + h) * p.S + i) * D;
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(y + e0) = real ? pack8<BF16>(z[0]) : zero;
        *reinterpret_cast<uint4*>(y + D / 2 + e0) = real ? pack8<BF16>(z[1]) : zero;
      }
      continue;
    }
    const long long row = slot + (static_cast<long long>(h) << p.page_shift);
    if constexpr (FP4) {
      const float ds = p.descale[which - 1] != nullptr ? p.descale[which - 1][h] : 1.f;
      uint8_t f0, f1;
      const uint32_t c0 = quantise8(z[0], ds, f0), c1 = quantise8(z[1], ds, f1);
      if (stored) {
        uint8_t* y = p.data[which - 1] + row * (D / 2);
        *reinterpret_cast<uint32_t*>(y + e0 / 2) = c0;
        *reinterpret_cast<uint32_t*>(y + D / 4 + e0 / 2) = c1;
        if (lane_in_row % 2 == 0) {
          uint8_t* f = p.scale[which - 1] + row * (D / 16);
          f[e0 / 16] = f0;
          f[D / 32 + e0 / 16] = f1;
        }
      }
    } else if (stored) {
      uint16_t* y = reinterpret_cast<uint16_t*>(p.data[which - 1]) + row * D;
      *reinterpret_cast<uint4*>(y + e0) = pack8<BF16>(z[0]);
      *reinterpret_cast<uint4*>(y + D / 2 + e0) = pack8<BF16>(z[1]);
    }
  }
}

struct GatherParams {
  const uint8_t* data[2];
  const uint8_t* scale[2];
  const float* descale[2];
  uint16_t* out[2];
  const int* page_table;
  const int* seqlens;
  int B, Hkv, S;
  int page_shift, n_pages, max_pages;
  int* status;
};

constexpr int kGatherPasses = 8;  // rows of a thread, all requested before the first is written

// Grid (row blocks of one (batch, head), B * Hkv, 2).  A thread writes 8
// elements (16 bytes) of each of its rows, so that a warp's store is 512
// consecutive bytes.
template <int D, bool BF16, bool FP4>
__global__ void __launch_bounds__(kThreads) cache_gather_kernel(const __grid_constant__ GatherParams p) {
  constexpr int kParts = D / 8, kRowsPass = kThreads / kParts;
  const int which = blockIdx.z;
  const int b = blockIdx.y / p.Hkv, h = blockIdx.y % p.Hkv;
  const int s0 = blockIdx.x * (kRowsPass * kGatherPasses) + threadIdx.x / kParts;
  const int part = threadIdx.x % kParts;
  wait_for_previous_kernel();
  const int n = min(min(p.seqlens[b], p.max_pages << p.page_shift), p.S);
  int page[kGatherPasses];
#pragma unroll
  for (int u = 0; u < kGatherPasses; ++u) {
    const int s = s0 + u * kRowsPass, pg = s >> p.page_shift;
    page[u] = s < n ? p.page_table[static_cast<long long>(b) * p.max_pages + pg] : -1;
  }
  // Bytes of a row, and from one page's head to the next page's.
  constexpr int kRow = FP4 ? D / 2 : 2 * D;
  const long long head = static_cast<long long>(h) << p.page_shift, page_rows = static_cast<long long>(p.Hkv) << p.page_shift;
  const int in_page = (1 << p.page_shift) - 1;
  const uint8_t* data = p.data[which] + head * kRow + part * (kRow / kParts);
  [[maybe_unused]] const uint8_t* factors = FP4 ? p.scale[which] + head * (D / 16) + part / 2 : nullptr;
  uint4 y[kGatherPasses];
  uint32_t f[kGatherPasses];
#pragma unroll
  for (int u = 0; u < kGatherPasses; ++u) {
    const int s = s0 + u * kRowsPass;
    y[u] = make_uint4(0u, 0u, 0u, 0u);
    f[u] = 0u;  // a row behind the sequence: factor 0
    if (static_cast<unsigned>(page[u]) < static_cast<unsigned>(p.n_pages)) {
      const long long row = page[u] * page_rows + (s & in_page);
      if constexpr (FP4) {
        y[u].x = *reinterpret_cast<const uint32_t*>(data + row * kRow);
        f[u] = factors[row * (D / 16)];
      } else {
        y[u] = *reinterpret_cast<const uint4*>(data + row * kRow);
      }
    } else if (s < n) {
      report_index(p.status);
    }
  }
  const float ds = FP4 && p.descale[which] != nullptr ? p.descale[which][h] : 1.f;
  uint16_t* out = p.out[which] + (static_cast<long long>(blockIdx.y) * p.S + s0) * D + part * 8;
#pragma unroll
  for (int u = 0; u < kGatherPasses; ++u, out += kRowsPass * D) {
    if (s0 + u * kRowsPass >= p.S) break;
    if constexpr (FP4) {
      if (f[u] != 0) {
        // code * factor is exact in fp16 (2 by 4 significant bits, at most 2688).
        const __half2 f2 = __half2half2(e4m3_half(f[u]));
        float z[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 t = __half22float2(__hmul2(e2m1x2_half2(y[u].x >> (8 * k)), f2));
          z[2 * k] = __fmul_rn(t.x, ds);
          z[2 * k + 1] = __fmul_rn(t.y, ds);
        }
        y[u] = pack8<BF16>(z);
      } else {
        y[u] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    *reinterpret_cast<uint4*>(out) = y[u];
  }
}

template <int D, bool BF16, bool FP4>
int launch_append_t(const AppendArgs& a) {
  AppendParams p{};
  for (int i = 0; i < 3; ++i) {
    p.x[i] = static_cast<const uint16_t*>(a.x[i]);
    p.xs[i] = a.xs[i];
    p.heads[i] = i == 0 ? (a.x[0] != nullptr ? a.H : 0) : a.cache.Hkv;
  }
  for (int i = 0; i < 2; ++i) {
    p.data[i] = static_cast<uint8_t*>(a.cache.data[i]);
    p.scale[i] = static_cast<uint8_t*>(a.cache.scale[i]);
    p.descale[i] = a.cache.descale[i];
  }
  p.q_out = static_cast<uint16_t*>(a.q_out);
  p.page_table = a.cache.page_table;
  p.seqlens = a.cache.seqlens;
  p.new_lens = a.new_lens;
  p.table = a.rope.table;
  p.table_rows = a.rope.rows;
  p.rot = a.rope.rot_dim;
  p.B = a.B;
  p.S = a.S;
  p.page_shift = a.cache.page_shift;
  p.n_pages = a.cache.n_pages;
  p.max_pages = a.cache.max_pages;
  p.status = a.status;
  const long long tokens = static_cast<long long>(a.B) * a.S;
  const long long token_ctas = (tokens + kThreads / RowCfg<D>::kLanes - 1) / (kThreads / RowCfg<D>::kLanes);
  // As many heads a thread as leave four CTAs for each SM, at most 8.  Four CTAs
  // against 32: 4.6 and 6.1 us at [2, 911] tokens of 24 + 6 heads, 12.5 and 16.3 at
  // [1, 2094] of 64 + 8; the other way round 19.4 and 18.2 at [5, 1434] of 40 + 16.
  int per = 8;
  const int heads = p.heads[0] + p.heads[1] + p.heads[2];
  while (per > 1 && token_ctas * (heads / per) < 4LL * a.num_sms) per /= 2;
  p.per_chunk = per;
  int chunks = 0;
  for (int i = 0; i < 3; ++i) chunks += p.chunks[i] = (p.heads[i] + per - 1) / per;
  if (token_ctas > 0x7FFFFFFFLL || chunks > 65535) return -1;
  const dim3 grid(static_cast<unsigned>(token_ctas), chunks);
  switch (rope_mode(a.rope, D)) {
    case kRopeNone: return launch_after(cache_append_kernel<D, BF16, kRopeNone, FP4>, grid, kThreads, a.stream, p);
    case kRopePairs: return launch_after(cache_append_kernel<D, BF16, kRopePairs, FP4>, grid, kThreads, a.stream, p);
    case kRopeHalves: return launch_after(cache_append_kernel<D, BF16, kRopeHalves, FP4>, grid, kThreads, a.stream, p);
    default: return launch_after(cache_append_kernel<D, BF16, kRopePart, FP4>, grid, kThreads, a.stream, p);
  }
}

template <int D, bool BF16, bool FP4>
int launch_gather_t(const GatherArgs& a) {
  GatherParams p{};
  for (int i = 0; i < 2; ++i) {
    p.data[i] = static_cast<const uint8_t*>(a.cache.data[i]);
    p.scale[i] = static_cast<const uint8_t*>(a.cache.scale[i]);
    p.descale[i] = a.cache.descale[i];
    p.out[i] = static_cast<uint16_t*>(a.out[i]);
  }
  p.page_table = a.cache.page_table;
  p.seqlens = a.cache.seqlens;
  p.B = a.B;
  p.Hkv = a.cache.Hkv;
  p.S = a.S;
  p.page_shift = a.cache.page_shift;
  p.n_pages = a.cache.n_pages;
  p.max_pages = a.cache.max_pages;
  p.status = a.status;
  constexpr int kRowsCta = kThreads / (D / 8) * kGatherPasses;
  const long long bh = static_cast<long long>(a.B) * a.cache.Hkv;
  if (bh > 65535) return -1;
  const dim3 grid(static_cast<unsigned>((static_cast<long long>(a.S) + kRowsCta - 1) / kRowsCta), static_cast<unsigned>(bh), 2);
  return launch_after(cache_gather_kernel<D, BF16, FP4>, grid, kThreads, a.stream, p);
}

}  // namespace

int launch_cache_append(const AppendArgs& a) {
  if (a.cache.d == 128) {
    if (a.cache.fp4()) return a.bf16 ? launch_append_t<128, true, true>(a) : launch_append_t<128, false, true>(a);
    return a.bf16 ? launch_append_t<128, true, false>(a) : launch_append_t<128, false, false>(a);
  }
  if (a.cache.fp4()) return a.bf16 ? launch_append_t<64, true, true>(a) : launch_append_t<64, false, true>(a);
  return a.bf16 ? launch_append_t<64, true, false>(a) : launch_append_t<64, false, false>(a);
}

int launch_cache_gather(const GatherArgs& a) {
  if (a.cache.d == 128) {
    if (a.cache.fp4()) return a.bf16 ? launch_gather_t<128, true, true>(a) : launch_gather_t<128, false, true>(a);
    return launch_gather_t<128, true, false>(a);  // a copy: the type does not matter
  }
  if (a.cache.fp4()) return a.bf16 ? launch_gather_t<64, true, true>(a) : launch_gather_t<64, false, true>(a);
  return launch_gather_t<64, true, false>(a);
}

}  // namespace gbattn
