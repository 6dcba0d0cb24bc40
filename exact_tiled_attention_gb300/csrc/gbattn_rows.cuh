// gbattn_rows.cuh -- how the row operators (norm and rotation, cache append)
// hold one head's row of d 16-bit elements: D / 16 lanes of a warp share a row,
// and each holds two chunks of 8 consecutive elements, [8 L, 8 L + 8) and
// [D / 2 + 8 L, ...).  A full rotation pairs element i with i + D / 2, which is
// then the same lane's; each of the two loads of a row is a contiguous D bytes.
#pragma once

#include <stdint.h>

#include "gbattn_copy.cuh"
#include "gbattn_internal.h"
#include "gbattn_ptx.cuh"

namespace gbattn {

template <int D>
struct RowCfg {
  static constexpr int kLanes = D / 16;       // lanes of a row
  static constexpr int kRows = 32 / kLanes;   // rows of a warp
};

// How a kernel rotates: not at all, adjacent pairs, pairs half a head apart
// (rot_dim = d), or pairs rot_dim / 2 apart in the first rot_dim elements.
enum RopeMode : int { kRopeNone = 0, kRopePairs = 1, kRopeHalves = 2, kRopePart = 3 };

inline RopeMode rope_mode(const RopeArgs& r, int d) {
  if (r.rot_dim == 0) return kRopeNone;
  if (r.interleaved) return kRopePairs;
  return r.rot_dim == d ? kRopeHalves : kRopePart;
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2<BF16>(f[0], f[1]), pack2<BF16>(f[2], f[3]), pack2<BF16>(f[4], f[5]),
                    pack2<BF16>(f[6], f[7]));
}

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// The rotation of one token, held by the lane for its own elements: for element
// e of chunk c, y = x * cos + partner * sin, with sin already negative for the
// first element of a pair.  Chunks behind the rotated part do not turn: an angle of
// zero would make NaN of an infinity there (x + inf * 0) and of its neighbour.
struct LaneRope {
  float cos[2][8];
  float sin[2][8];
  bool turns[2];  // (a full rotation by halves turns both chunks and does not ask)
};

// First of the pairs that the chunk at e0 (< rot) takes part in.
template <int MODE>
__device__ __forceinline__ int first_pair(int e0, int rot) {
  return MODE == kRopePairs ? e0 / 2 : e0 < rot / 2 ? e0 : e0 - rot / 2;
}
// Pairs of a chunk.
template <int MODE>
constexpr int kPairs = MODE == kRopePairs ? 4 : 8;

// Places the cosines and sines of chunk c's pairs at its elements.
template <int MODE>
__device__ __forceinline__ void set_chunk(LaneRope& r, int c, const float* cs, const float* ss, bool first_half) {
  if constexpr (MODE == kRopePairs) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.cos[c][2 * i] = r.cos[c][2 * i + 1] = cs[i];
      r.sin[c][2 * i] = -ss[i];
      r.sin[c][2 * i + 1] = ss[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      r.cos[c][i] = cs[i];
      r.sin[c][i] = MODE == kRopePart && first_half ? -ss[i] : ss[i];
    }
  }
}

// Loads the cosines and sines of chunk c's pairs from one table row.
template <int MODE>
__device__ __forceinline__ void load_chunk(LaneRope& r, int c, const float* row, int e0, int rot) {
  const int i0 = first_pair<MODE>(e0, rot);
  float cs[8], ss[8];
  if constexpr (MODE == kRopePairs) {
    const float4 co = *reinterpret_cast<const float4*>(row + i0);
    const float4 si = *reinterpret_cast<const float4*>(row + rot / 2 + i0);
    cs[0] = co.x, cs[1] = co.y, cs[2] = co.z, cs[3] = co.w;
    ss[0] = si.x, ss[1] = si.y, ss[2] = si.z, ss[3] = si.w;
  } else {
    load8(row + i0, cs);
    load8(row + rot / 2 + i0, ss);
  }
  set_chunk<MODE>(r, c, cs, ss, e0 < rot / 2);
}

// Loads the lane's cosines and sines of a table row.
template <int D, int MODE>
__device__ __forceinline__ void load_rope(LaneRope& r, const float* row, int rot, int lane_in_row) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int e0 = c * (D / 2) + 8 * lane_in_row;
    r.turns[c] = e0 < rot;
    if (MODE == kRopeHalves ? c == 0 : e0 < rot) load_chunk<MODE>(r, c, row, e0, rot);
  }
}

// Positions of several axes: the axes of the pairs of a lane's chunks, two bits
// each; they stay the same for all tokens.
template <int D, int MODE>
struct LaneAxes {
  uint32_t of[2];
  bool same[2];  // one axis for all of the chunk's pairs
  __device__ __forceinline__ LaneAxes(const uint32_t* pair_axes, int rot, int lane_in_row) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int e0 = c * (D / 2) + 8 * lane_in_row;
      const int i0 = e0 < rot ? first_pair<MODE>(e0, rot) : 0;
      constexpr uint32_t kMask = (1u << 2 * kPairs<MODE>) - 1;
      of[c] = pair_axes[i0 / 16] >> (2 * (i0 % 16)) & kMask;
      same[c] = of[c] == (of[c] & 3u) * (0x5555u & kMask);
    }
  }
};

// load_rope from the table rows of a token's positions; row_of(a) is that of axis a.
template <int D, int MODE, typename RowOf>
__device__ __forceinline__ void load_rope_axes(LaneRope& r, const LaneAxes<D, MODE>& axes, RowOf&& row_of, int rot,
                                               int lane_in_row) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int e0 = c * (D / 2) + 8 * lane_in_row;
    r.turns[c] = e0 < rot;
    if (!(MODE == kRopeHalves ? c == 0 : e0 < rot)) continue;
    if (axes.same[c]) {
      load_chunk<MODE>(r, c, row_of(axes.of[c] & 3u), e0, rot);
    } else {
      const int i0 = first_pair<MODE>(e0, rot);
      float cs[8], ss[8];
#pragma unroll
      for (int i = 0; i < kPairs<MODE>; ++i) {
        const float* row = row_of(axes.of[c] >> 2 * i & 3u);
        cs[i] = row[i0 + i];
        ss[i] = row[rot / 2 + i0 + i];
      }
      set_chunk<MODE>(r, c, cs, ss, e0 < rot / 2);
    }
  }
}

// The table rows of a token's positions, [n_axes] of them `step` apart; positions
// outside the table are clamped into it and reported.
struct AxisRows {
  const float* row[4];
  __device__ __forceinline__ AxisRows(const int* positions, long long step, int n_axes, const float* table, int rows,
                                      int rot, int* status) {
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      int pos = a < n_axes ? positions[a * step] : 0;
      if (pos < 0 || pos >= rows) {
        report_index(status);
        pos = min(max(pos, 0), rows - 1);
      }
      row[a] = table + static_cast<long long>(pos) * rot;
    }
  }
  __device__ __forceinline__ const float* operator()(uint32_t a) const {
    return a & 2u ? (a & 1u ? row[3] : row[2]) : (a & 1u ? row[1] : row[0]);
  }
};

// The rows that a thread works on, of N tensors at once, on their way through
// shared memory: for tokens t0, t0 + step, .. (t0 a CTA's first, a row's lanes
// one token each) the heads [h0, h1).  Each lane copies its own pieces, STAGES - 1
// rows ahead over heads and tokens alike, and waits for nobody else's; what it
// has on its way would not fit in its registers.
template <int D, int N, int THREADS, int STAGES>
struct RowRing {
  using Smem = uint4[STAGES][2 * N][THREADS];
  Smem* smem;
  const uint16_t* base[N];
  RowStrides strides[N];
  int S, tokens, step, h0, h1;
  const uint16_t* row[N];  // of the next request
  int t, h, in, out;       // its token block and head; stages to fill and to read next

  __device__ __forceinline__ void at_token() {
    const int i = min(t + static_cast<int>(threadIdx.x) / RowCfg<D>::kLanes, tokens - 1);
    const int b = i / S, s = i % S;
#pragma unroll
    for (int k = 0; k < N; ++k) row[k] = base[k] + b * strides[k].b + s * strides[k].s + h0 * strides[k].h;
  }
  // The first requests; base and strides are set.
  __device__ __forceinline__ void start(Smem* smem_, int S_, int tokens_, int t0, int step_, int h0_, int h1_) {
    smem = smem_, S = S_, tokens = tokens_, t = t0, step = step_, h0 = h = h0_, h1 = h1_, in = out = 0;
    at_token();
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) request();
  }
  __device__ __forceinline__ void request() {
    if (t < tokens) {
      const int e0 = 8 * (threadIdx.x % RowCfg<D>::kLanes);
#pragma unroll
      for (int k = 0; k < N; ++k) {
#pragma unroll
        for (int c = 0; c < 2; ++c) copy16(smem_u32(&(*smem)[in][2 * k + c][threadIdx.x]), row[k] + c * (D / 2) + e0);
        row[k] += strides[k].h;
      }
      in = in + 1 == STAGES ? 0 : in + 1;
      if (++h == h1) {
        h = h0;
        t += step;
        at_token();
      }
    }
    copy_commit();
  }
  // Waits for the next row; piece(k, c) is then its chunk c of tensor k, until pop().
  __device__ __forceinline__ void wait() const { copy_wait<STAGES - 2>(); }
  __device__ __forceinline__ uint4 piece(int k, int c) const { return (*smem)[out][2 * k + c][threadIdx.x]; }
  // The chunk of tensor k that starts at element e of the row, copied by another
  // of the row's lanes: between wait(), __syncwarp() and pop().  (The stage that
  // pop() fills again is the previous row's, which every lane has left by then.)
  __device__ __forceinline__ uint4 chunk_at(int k, int e) const {
    const int c = e >= D / 2;
    return (*smem)[out][2 * k + c][threadIdx.x - threadIdx.x % RowCfg<D>::kLanes + (e - c * (D / 2)) / 8];
  }
  __device__ __forceinline__ void pop() {
    out = out + 1 == STAGES ? 0 : out + 1;
    request();  // into the stage that the row before this one has left
  }
};

// Offset of the chunk that holds the partners of the chunk at e0 when pairs
// are rot / 2 apart in a part of the head (kRopePart); e0 itself outside it.
__device__ __forceinline__ int partner_chunk(int e0, int rot) {
  const int half = rot / 2;
  return e0 < half ? e0 + half : (e0 < rot ? e0 - half : e0);
}

// Rotates the lane's two chunks z; `part` holds the partners' chunks when MODE
// is kRopePart.  Products and sum are rounded one by one (no contraction into
// a fused multiply-add): the 4-bit codes made from the result then do not
// depend on how an expression is compiled.  BACK turns by the negative angle.
template <int MODE, bool BACK>
__device__ __forceinline__ void rotate(float (&z)[2][8], const float (&part)[2][8], const LaneRope& r) {
  if constexpr (MODE == kRopeHalves) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = z[0][i], b = z[1][i], c = r.cos[0][i], s = BACK ? -r.sin[0][i] : r.sin[0][i];
      z[0][i] = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
      z[1][i] = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    }
  } else if constexpr (MODE == kRopePairs) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (!r.turns[c]) continue;
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float a = z[c][i], b = z[c][i + 1], co = r.cos[c][i], s = BACK ? r.sin[c][i] : r.sin[c][i + 1];
        z[c][i] = __fsub_rn(__fmul_rn(a, co), __fmul_rn(b, s));
        z[c][i + 1] = __fadd_rn(__fmul_rn(b, co), __fmul_rn(a, s));
      }
    }
  } else if constexpr (MODE == kRopePart) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (!r.turns[c]) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float s = BACK ? -r.sin[c][i] : r.sin[c][i];
        z[c][i] = __fadd_rn(__fmul_rn(z[c][i], r.cos[c][i]), __fmul_rn(part[c][i], s));
      }
    }
  }
}

}  // namespace gbattn
