// qk_norm_rope.cu -- RMS norm of every query and key head with the position
// rotation in the same pass, and its backward.
//
// Forward, for one row x of d elements:  r = (mean x^2 + eps)^-1/2,  n = x r,
// z = n o w,  y = R(position) z.  Backward, from dy:  dz = R^T dy,
// dw += dz o n,  g = dz o w,  dx = r (g - n mean(g o n));  r and n are formed
// again from x, which the backward reads anyway, so the forward saves nothing.
//
// Both are bound by HBM: a forward reads and writes each row once (2 bytes an
// element each way), a backward reads two rows and writes one.  A thread keeps
// one token's cosines and sines in registers and walks over heads, so the
// 4-byte table is read once for several heads, and the rows come through a ring
// of asynchronous copies (RowRing).  At [4, 8192] tokens of 16 + 16 heads of 128
// the forward takes 83 us (6.5 TB/s) and the backward 127 us (6.4 TB/s); when the
// ring came in they fell from 84 to 80 and from 137 to 121 against the next row alone
// requested ahead, in registers.  The rotation without norms takes 83 and 82 us.
#include <cuda_runtime.h>

#include <type_traits>

#include "gbattn_rows.cuh"

namespace gbattn {
namespace {

constexpr int kThreads = 128;
constexpr int kStages = 4;         // of the rings of rows
constexpr int kFwdCtas = 64;       // of the forward for each SM, at most
constexpr int kMaxBwdCtas = 1024;  // partial weight gradients kept for each of q and k

struct NormRopeParams {
  const uint16_t* x[2];
  const float* w[2];
  uint16_t* y[2];
  const uint16_t* dy[2];
  uint16_t* dx[2];
  RowStrides xs[2], dxs[2];
  int heads[2];
  int chunks[2];        // head chunks of q and of k
  const int* positions;
  const float* table;
  int table_rows, rot;
  float eps;
  int B, S, per_chunk;  // heads that a thread walks over
  float* partial;       // backward: [2][kMaxBwdCtas][D]
  int* status;
};

// The table row of token (b, s); a position outside the table is clamped into
// it and reported.
__device__ __forceinline__ const float* table_row(const NormRopeParams& p, int b, int s) {
  int pos = p.positions != nullptr ? p.positions[static_cast<long long>(b) * p.S + s] : s;
  if (pos < 0 || pos >= p.table_rows) {
    report_index(p.status);
    pos = min(max(pos, 0), p.table_rows - 1);
  }
  return p.table + static_cast<long long>(pos) * p.rot;
}

template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = RowCfg<D>::kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Grid: (CTAs that walk over tokens, head chunks of q then k).
template <int D, bool BF16, int MODE, bool NORM>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int kLanes = RowCfg<D>::kLanes;
  constexpr int kRowsCta = kThreads / kLanes;
  using Ring = RowRing<D, 1, kThreads, kStages>;
  __shared__ typename Ring::Smem ring_smem;
  const int lane_in_row = threadIdx.x % kLanes;
  const int tokens = p.B * p.S;
  const int which = blockIdx.y < p.chunks[0] ? 0 : 1;
  const int h0 = (blockIdx.y - (which ? p.chunks[0] : 0)) * p.per_chunk;
  const int h1 = min(h0 + p.per_chunk, p.heads[which]);
  const int e0 = 8 * lane_in_row;

  wait_for_previous_kernel();
  Ring ring;
  ring.base[0] = p.x[which];
  ring.strides[0] = p.xs[which];
  ring.start(&ring_smem, p.S, tokens, blockIdx.x * kRowsCta, gridDim.x * kRowsCta, h0, h1);
  float w[2][8], wp[2][8];
  int pc[2] = {0, 0};
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    if constexpr (MODE == kRopePart) pc[c] = partner_chunk(c * (D / 2) + e0, p.rot);
    if constexpr (NORM) {
      load8(p.w[which] + c * (D / 2) + e0, w[c]);
      if constexpr (MODE == kRopePart) load8(p.w[which] + pc[c], wp[c]);
    }
  }
  for (int t0 = blockIdx.x * kRowsCta; t0 < tokens; t0 += gridDim.x * kRowsCta) {
    const int at = t0 + static_cast<int>(threadIdx.x) / kLanes;
    const bool real = at < tokens;
    const int t = min(at, tokens - 1);  // the whole warp stays for the shuffles
    const int b = t / p.S, s = t % p.S;
    LaneRope rope;
    if constexpr (MODE != kRopeNone) load_rope<D, MODE>(rope, table_row(p, b, s), p.rot, lane_in_row);
    uint16_t* yrow = p.y[which] + ((static_cast<long long>(b) * p.heads[which] + h0) * p.S + s) * D;
    for (int h = h0; h < h1; ++h, yrow += static_cast<long long>(p.S) * D) {
      ring.wait();
      if constexpr (MODE == kRopePart) __syncwarp();
      float z[2][8], part[2][8];
      float sq = 0.f;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        unpack8<BF16>(ring.piece(0, c), z[c]);
        if constexpr (MODE == kRopePart) unpack8<BF16>(ring.chunk_at(0, pc[c]), part[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) sq = fmaf(z[c][i], z[c][i], sq);
      }
      ring.pop();
      if constexpr (NORM) {
        const float r = rsqrtf(row_sum<D>(sq) * (1.f / D) + p.eps);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            z[c][i] *= r * w[c][i];
            if constexpr (MODE == kRopePart) part[c][i] *= r * wp[c][i];
          }
      }
      rotate<MODE, false>(z, part, rope);
      if (real) {
        *reinterpret_cast<uint4*>(yrow + e0) = pack8<BF16>(z[0]);
        *reinterpret_cast<uint4*>(yrow + D / 2 + e0) = pack8<BF16>(z[1]);
      }
    }
  }
}

// Grid: (CTAs that walk over tokens, head chunks of q then k).  With NORM each
// CTA leaves the sum of its rows' weight gradients in `partial`.
template <int D, bool BF16, int MODE, bool NORM>
__global__ void __launch_bounds__(kThreads, 4) norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int kLanes = RowCfg<D>::kLanes;
  constexpr int kRowsCta = kThreads / kLanes;
  const int lane_in_row = threadIdx.x % kLanes;
  const int tokens = p.B * p.S;
  const int which = blockIdx.y < p.chunks[0] ? 0 : 1;
  const int chunk = blockIdx.y - (which ? p.chunks[0] : 0);
  const int h0 = chunk * p.per_chunk;
  const int h1 = min(h0 + p.per_chunk, p.heads[which]);
  const int e0 = 8 * lane_in_row;
  wait_for_previous_kernel();
  if constexpr (NORM) let_next_kernel_start();  // norm_dw_kernel; without weights none of this call follows
  int pc[2] = {0, 0};
  float w[2][8], dw[2][8];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    if constexpr (MODE == kRopePart) pc[c] = partner_chunk(c * (D / 2) + e0, p.rot);
    if constexpr (NORM) load8(p.w[which] + c * (D / 2) + e0, w[c]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = 0.f;
  }
  const RowStrides dxs = p.dxs[which];
  const long long dy_head = static_cast<long long>(p.S) * D;
  using Ring = RowRing<D, NORM ? 2 : 1, kThreads, kStages>;
  __shared__ typename Ring::Smem ring_smem;
  const int step = gridDim.x * kRowsCta;
  Ring ring;
  ring.base[0] = p.dy[which];
  ring.strides[0] = {p.heads[which] * dy_head, dy_head, D};
  if constexpr (NORM) {
    ring.base[1] = p.x[which];
    ring.strides[1] = p.xs[which];
  }
  ring.start(&ring_smem, p.S, tokens, blockIdx.x * kRowsCta, step, h0, h1);
  for (int t0 = blockIdx.x * kRowsCta; t0 < tokens; t0 += step) {
    const bool real = t0 + static_cast<int>(threadIdx.x) / kLanes < tokens;
    const int t = min(t0 + static_cast<int>(threadIdx.x) / kLanes, tokens - 1);
    const int b = t / p.S, s = t % p.S;
    LaneRope rope;
    if constexpr (MODE != kRopeNone) load_rope<D, MODE>(rope, table_row(p, b, s), p.rot, lane_in_row);
    uint16_t* dxrow = p.dx[which] + b * dxs.b + s * dxs.s + h0 * dxs.h;
    for (int h = h0; h < h1; ++h, dxrow += dxs.h) {
      ring.wait();
      if constexpr (MODE == kRopePart) __syncwarp();
      float g[2][8], part[2][8], n[2][8];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        unpack8<BF16>(ring.piece(0, c), g[c]);
        if constexpr (MODE == kRopePart) unpack8<BF16>(ring.chunk_at(0, pc[c]), part[c]);
        if constexpr (NORM) unpack8<BF16>(ring.piece(1, c), n[c]);
      }
      ring.pop();
      rotate<MODE, true>(g, part, rope);
      if constexpr (NORM) {
        float sq = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) sq = fmaf(n[c][i], n[c][i], sq);
        const float r = rsqrtf(row_sum<D>(sq) * (1.f / D) + p.eps);
        float dot = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            n[c][i] *= r;
            if (real) dw[c][i] = fmaf(g[c][i], n[c][i], dw[c][i]);
            g[c][i] *= w[c][i];
            dot = fmaf(g[c][i], n[c][i], dot);
          }
        dot = row_sum<D>(dot) * (1.f / D);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) g[c][i] = r * (g[c][i] - n[c][i] * dot);
      }
      if (real) {
        *reinterpret_cast<uint4*>(dxrow + e0) = pack8<BF16>(g[0]);
        *reinterpret_cast<uint4*>(dxrow + D / 2 + e0) = pack8<BF16>(g[1]);
      }
    }
  }
  if constexpr (NORM) {
    __shared__ float sum[kThreads / 32][D];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int o = kLanes; o < 32; o <<= 1) dw[c][i] += __shfl_xor_sync(0xffffffffu, dw[c][i], o);
        if (threadIdx.x % 32 < kLanes) sum[threadIdx.x / 32][c * (D / 2) + e0 + i] = dw[c][i];
      }
    __syncthreads();
    const int row = chunk * gridDim.x + blockIdx.x;  // < kMaxBwdCtas
    for (int i = threadIdx.x; i < D; i += kThreads) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < kThreads / 32; ++k) v += sum[k][i];
      p.partial[(static_cast<long long>(which) * kMaxBwdCtas + row) * D + i] = v;
    }
  }
}

struct DwParams {
  const float* partial;
  int rows[2];
  int d;
  float* dw[2];
};

// dw[which][i] = sum of the CTAs' partials, in a fixed order.  Grid (d / 16, 2):
// a CTA sums 16 columns, 64 rows at a time.  Launched while the backward kernel
// runs; it waits for that kernel's end.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const __grid_constant__ DwParams p) {
  __shared__ float sum[32][17];
  const int which = blockIdx.y, rows = p.rows[which];
  const int col = threadIdx.x % 16, r0 = threadIdx.x / 16;
  const float* base = p.partial + static_cast<long long>(which) * kMaxBwdCtas * p.d + blockIdx.x * 16 + col;
  wait_for_previous_kernel();
  float v = 0.f;
#pragma unroll 8
  for (int r = r0; r < rows; r += 64) v += base[static_cast<long long>(r) * p.d];
  v += __shfl_xor_sync(0xffffffffu, v, 16);
  if (threadIdx.x % 32 < 16) sum[threadIdx.x / 32][col] = v;
  __syncthreads();
  if (threadIdx.x >= 512) return;
  v = sum[threadIdx.x % 32][threadIdx.x / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (threadIdx.x % 32 == 0) p.dw[which][blockIdx.x * 16 + threadIdx.x / 32] = v;
}

NormRopeParams params(const NormRopeArgs& a) {
  NormRopeParams p{};
  for (int i = 0; i < 2; ++i) {
    p.x[i] = static_cast<const uint16_t*>(a.x[i]);
    p.w[i] = a.w[i];
    p.y[i] = static_cast<uint16_t*>(a.y[i]);
    p.dy[i] = static_cast<const uint16_t*>(a.dy[i]);
    p.dx[i] = static_cast<uint16_t*>(a.dx[i]);
    p.xs[i] = a.xs[i];
    p.dxs[i] = a.dxs[i];
    p.heads[i] = a.heads[i];
  }
  p.positions = a.positions;
  p.table = a.rope.table;
  p.table_rows = a.rope.rows;
  p.rot = a.rope.rot_dim;
  p.eps = a.eps;
  p.B = a.B;
  p.S = a.S;
  p.partial = a.workspace;
  p.status = a.status;
  return p;
}

void set_chunks(NormRopeParams& p, int per_chunk) {
  p.per_chunk = per_chunk;
  for (int i = 0; i < 2; ++i) p.chunks[i] = (p.heads[i] + per_chunk - 1) / per_chunk;
}

// Calls f with the rotation mode and the presence of a norm as constants.
template <typename F>
int with_mode(const NormRopeArgs& a, F&& f) {
  const bool norm = a.w[0] != nullptr;
  switch (rope_mode(a.rope, a.d)) {
    case kRopeNone: return f(std::integral_constant<int, kRopeNone>(), std::true_type());
    case kRopePairs:
      return norm ? f(std::integral_constant<int, kRopePairs>(), std::true_type())
                  : f(std::integral_constant<int, kRopePairs>(), std::false_type());
    case kRopeHalves:
      return norm ? f(std::integral_constant<int, kRopeHalves>(), std::true_type())
                  : f(std::integral_constant<int, kRopeHalves>(), std::false_type());
    default:
      return norm ? f(std::integral_constant<int, kRopePart>(), std::true_type())
                  : f(std::integral_constant<int, kRopePart>(), std::false_type());
  }
}

template <int D, bool BF16>
int launch_fwd(const NormRopeArgs& a) {
  NormRopeParams p = params(a);
  const long long tokens = static_cast<long long>(a.B) * a.S;
  const long long token_ctas = (tokens + kThreads / RowCfg<D>::kLanes - 1) / (kThreads / RowCfg<D>::kLanes);
  const int heads = a.heads[0] + a.heads[1];
  // As many heads a thread as leave four CTAs for each SM, at most 8: a thread
  // with few rows hardly uses its ring.  Four CTAs against 32: 10.5 and 16.1 us at
  // [1, 2094] tokens of 68 heads, 4.9 and 6.7 at [2, 911] of 27; the other way
  // round 28.1 and 27.5 at [2, 4096] of 40.
  int per = 8;
  while (per > 1 && token_ctas * (heads / per) < 4LL * a.num_sms) per /= 2;
  set_chunks(p, per);
  const int chunks = p.chunks[0] + p.chunks[1];
  if (chunks > 65535) return -1;
  long long x = (kFwdCtas * static_cast<long long>(a.num_sms) + chunks - 1) / chunks;
  if (x > token_ctas) x = token_ctas;
  const dim3 grid(static_cast<unsigned>(x), chunks);
  return with_mode(a, [&](auto mode, auto norm) {
    return launch_after(norm_rope_kernel<D, BF16, decltype(mode)::value, decltype(norm)::value>, grid, kThreads, a.stream, p);
  });
}

template <int D, bool BF16>
int launch_bwd(const NormRopeArgs& a) {
  NormRopeParams p = params(a);
  const long long tokens = static_cast<long long>(a.B) * a.S;
  const long long token_ctas = (tokens + kThreads / RowCfg<D>::kLanes - 1) / (kThreads / RowCfg<D>::kLanes);
  const int heads = a.heads[0] + a.heads[1];
  // Up to 16 heads a thread and two CTAs for each SM: each CTA ends with the sum of
  // its weight gradients.  16 and 8 heads: 17.9 and 21.3 us at [1, 2094] tokens of
  // 68 heads, 42.0 and 46.2 at [2, 4096] of 40, 61.7 and 60.5 at [1, 4777] of 96.
  int per = 16;
  while (per > 1 && token_ctas * (heads / per) < 2LL * a.num_sms) per /= 2;
  const int most = a.heads[0] > a.heads[1] ? a.heads[0] : a.heads[1];
  while ((most + per - 1) / per > kMaxBwdCtas) per *= 2;
  set_chunks(p, per);
  const int most_chunks = p.chunks[0] > p.chunks[1] ? p.chunks[0] : p.chunks[1];
  // CTAs over tokens: sixteen for each SM in all, and no more partials than fit.
  long long x = (16LL * a.num_sms + p.chunks[0] + p.chunks[1] - 1) / (p.chunks[0] + p.chunks[1]);
  if (x > kMaxBwdCtas / most_chunks) x = kMaxBwdCtas / most_chunks;
  if (x > token_ctas) x = token_ctas;
  const dim3 grid(static_cast<unsigned>(x), p.chunks[0] + p.chunks[1]);
  const int rc = with_mode(a, [&](auto mode, auto norm) {
    return launch_after(norm_rope_bwd_kernel<D, BF16, decltype(mode)::value, decltype(norm)::value>, grid, kThreads, a.stream, p);
  });
  if (rc != 0 || a.w[0] == nullptr) return rc;
  DwParams dp{};
  dp.partial = p.partial;
  dp.d = D;
  for (int i = 0; i < 2; ++i) {
    dp.rows[i] = static_cast<int>(x) * p.chunks[i];
    dp.dw[i] = a.dw[i];
  }
  return launch_after(norm_dw_kernel, dim3(D / 16, 2), 1024, a.stream, dp);
}

}  // namespace

size_t norm_rope_bwd_workspace_bytes(int d) {
  return 2 * static_cast<size_t>(kMaxBwdCtas) * static_cast<size_t>(d) * sizeof(float);
}

int launch_norm_rope(const NormRopeArgs& a) {
  if (a.d == 128) return a.bf16 ? launch_fwd<128, true>(a) : launch_fwd<128, false>(a);
  return a.bf16 ? launch_fwd<64, true>(a) : launch_fwd<64, false>(a);
}

int launch_norm_rope_bwd(const NormRopeArgs& a) {
  if (a.d == 128) return a.bf16 ? launch_bwd<128, true>(a) : launch_bwd<128, false>(a);
  return a.bf16 ? launch_bwd<64, true>(a) : launch_bwd<64, false>(a);
}

}  // namespace gbattn
