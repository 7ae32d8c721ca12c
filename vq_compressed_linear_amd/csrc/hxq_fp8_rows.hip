// Row operators of the 8-bit path: the root-mean-square norm with the
// residual's addition, its gradient, and the conversion of rows and weights to
// e4m3 with power-of-two block scales.
//
// norm:      h = x + residual (rounded to the residual's type, as it is kept),
//            r = 1 / sqrt(mean_k h^2 + eps), y = h r w.
// gradient:  g = dy w, dx = r (g - h r^2 mean_k(g h)) + dsum,
//            dw = sum over rows of dy h r.
// All sums and statistics are fp32.
//
// Bound: bytes (6 to 20 operations for 10 to 14 bytes).  A row is read once:
// a team of 64 or 256 threads keeps it in registers, 8 consecutive columns to
// a thread, from the sum of squares to the store.  A 128-column group is then
// held by 16 lanes of one DPP row, whose largest magnitude needs no LDS.
// Rows wider than 12288 columns are read a second time (from the caches).
//
// Measured, inputs from memory: the norm of 25600 rows of 2048 (float32 x, bf16
// residual, e4m3 out) 84 us, 5.6 TB/s; one row 2.3 us; the gradient of 2047
// rows of 4096 with the weight's 28 + 4.0 us (4.2 TB/s in the first launch);
// conversion of 25600 rows of 11008 from bf16 157 us, 5.4 TB/s (a large copy:
// 4.9 TB/s).  A weight of 22016 x 2048 from bf16 in 107 us (1.3 TB/s), with its
// transposed copy 114: a layer is laid out once, so its bytes leave LDS one at
// a time and nothing was made faster.

#include "hxq_fp8.h"
#include "hxq_fp8_device.h"

namespace hxq {

namespace {

// Sum over a team of TPR threads (64: a wave; 256: the workgroup), in a fixed
// order; every thread receives it.  `slot`: 4 floats of LDS of this use.
template <int TPR>
__device__ __forceinline__ float team_sum(float v, float* slot) {
  v = wave_sum_dpp(v);
  if constexpr (TPR == 64) return v;
  if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
  __syncthreads();
  return (slot[0] + slot[1]) + (slot[2] + slot[3]);
}

template <int RT>
__device__ __forceinline__ void add_residual(float (&v)[8], const float (&r)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] += r[i];
    if constexpr (RT == kBf16) v[i] = (float)(__bf16)v[i];
  }
}

// The output of 8 columns: y, or its e4m3 bytes and the group's scale.
template <int OT>
__device__ __forceinline__ void emit(const NormArgs& a, int64_t m, int col, const float (&v)[8], float r,
                                     const float (&w)[8]) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = v[i] * r * w[i];
  if constexpr (OT == kE4m3) {
    const int Kp = (a.K + 127) & ~127, Gs = (a.K + 511) / 512 * 4;
    int byte;
    const uint2 q = quant_group(y, byte);
    if (col < Kp) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + m * Kp + col) = q;
    // the scale row's padding (groups past the last) holds ones
    if ((threadIdx.x & 15) == 0 && (col >> 7) < Gs) a.scales[m * Gs + (col >> 7)] = (uint8_t)(col < a.K ? byte : 127);
  } else {
    if (col < a.K) store_row8<OT>(a.out, m * (int64_t)a.K, col, a.K, y);
  }
}

// NCH chunks of 8 TPR columns in registers; NCH == 0: any width, the row read
// twice.  XT, OT: types; RT: the residual's, or -1.
template <int TPR, int NCH, int XT, int RT, int OT>
__global__ __launch_bounds__(256) void rms_norm_rows(NormArgs a) {
  __shared__ float slot[4];
  const int t = threadIdx.x % TPR;
  const int64_t m = (int64_t)blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
  if (TPR == 64 && m >= a.M) return;  // (a whole wave; TPR == 256 has no barrier to miss either)
  const int K = a.K;
  const int64_t row0 = m * (int64_t)K;
  float ss = 0.f;
  if constexpr (NCH > 0) {
    float v[NCH][8], w[NCH][8];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = (c * TPR + t) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = 0.f, w[c][i] = 1.f;
      if (col < K) {
        load_row8<XT>(a.x, row0, col, K, v[c]);
        if constexpr (RT >= 0) {
          float r[8];
          load_row8<RT>(a.residual, row0, col, K, r);
          add_residual<RT>(v[c], r);
        }
        if (a.weight) load_row8<kF32>(a.weight, 0, col, K, w[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(v[c][i], v[c][i], ss);
    const float r = 1.f / sqrtf(team_sum<TPR>(ss, slot) / (float)K + a.eps);
    if (t == 0 && a.rstd) a.rstd[m] = r;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = (c * TPR + t) * 8;
      if constexpr (RT >= 0)
        if (col < K) store_row8<RT>(a.sum_out, row0, col, K, v[c]);
      emit<OT>(a, m, col, v[c], r, w[c]);
    }
  } else {
    const int wide = (K + 511) & ~511;  // whole groups of the scale row
    for (int col = t * 8; col < K; col += TPR * 8) {
      float v[8];
      load_row8<XT>(a.x, row0, col, K, v);
      if constexpr (RT >= 0) {
        float r[8];
        load_row8<RT>(a.residual, row0, col, K, r);
        add_residual<RT>(v, r);
        store_row8<RT>(a.sum_out, row0, col, K, v);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
    }
    const float r = 1.f / sqrtf(team_sum<TPR>(ss, slot) / (float)K + a.eps);
    if (t == 0 && a.rstd) a.rstd[m] = r;
    for (int c0 = 0; c0 < wide; c0 += TPR * 8) {  // (all lanes of a DPP row go round together)
      const int col = c0 + t * 8;
      float v[8], w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f, w[i] = 1.f;
      if (col < K) {
        // what this thread itself stored, where there is a residual
        if constexpr (RT >= 0)
          load_row8<RT>(a.sum_out, row0, col, K, v);
        else
          load_row8<XT>(a.x, row0, col, K, v);
        if (a.weight) load_row8<kF32>(a.weight, 0, col, K, w);
      }
      emit<OT>(a, m, col, v, r, w);
    }
  }
}

template <int XT, int RT, int OT>
void norm_launch(const NormArgs& a, hipStream_t s) {
  const int K = a.K;
  // A wave to a short row (25600 x 512: 21 us, 32 with a workgroup), else a workgroup: a wave with four chunks of
  // a row of 2048 took 92 us against 84 at 25600 rows, 8.3 against 3.8 at 256.  As many chunks as the row has up to
  // two (20480 x 2560: 101 us, 125 with room for six; 12800 x 4096: 102, 104), then six (with fewer no faster:
  // 10240 x 5120 102 us, 104 with three; 6400 x 8192 99, 102 with four) rather than a second reading (105, 107;
  // 4266 x 12288: 103, 117).
  const unsigned rows = (unsigned)a.M, rows4 = (unsigned)((a.M + 3) / 4);
  if (K <= 512)
    hipLaunchKernelGGL((rms_norm_rows<64, 1, XT, RT, OT>), dim3(rows4), dim3(256), 0, s, a);
  else if (K <= 2048)
    hipLaunchKernelGGL((rms_norm_rows<256, 1, XT, RT, OT>), dim3(rows), dim3(256), 0, s, a);
  else if (K <= 4096)
    hipLaunchKernelGGL((rms_norm_rows<256, 2, XT, RT, OT>), dim3(rows), dim3(256), 0, s, a);
  else if (K <= 12288)
    hipLaunchKernelGGL((rms_norm_rows<256, 6, XT, RT, OT>), dim3(rows), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((rms_norm_rows<256, 0, XT, RT, OT>), dim3(rows), dim3(256), 0, s, a);
}

template <int XT, int RT>
void norm_launch_out(const NormArgs& a, hipStream_t s) {
  if (a.out_dtype == kF32)
    norm_launch<XT, RT, kF32>(a, s);
  else if (a.out_dtype == kBf16)
    norm_launch<XT, RT, kBf16>(a, s);
  else
    norm_launch<XT, RT, kE4m3>(a, s);
}

template <int XT>
void norm_launch_res(const NormArgs& a, hipStream_t s) {
  if (a.res_dtype < 0)
    norm_launch_out<XT, -1>(a, s);
  else if (a.res_dtype == kF32)
    norm_launch_out<XT, kF32>(a, s);
  else
    norm_launch_out<XT, kBf16>(a, s);
}

// ------------------------------------------------------------- the gradient

// Teams of TPR threads walk the rows team, team + teams, ...; a thread keeps
// its columns' part of the weight's gradient in registers over its team's rows
// (NCH > 0; the four waves of a workgroup then add theirs in LDS) or in its
// workgroup's partial row in memory (NCH == 0), and the second launch adds the
// workgroups' partial rows in order.
template <int TPR, int NCH, int DT, int HT>
__global__ __launch_bounds__(256) void rms_norm_bwd_rows(NormBwdArgs a) {
  __shared__ float slot[2][4];
  __shared__ float wave_dw[TPR == 64 ? 4 : 1][TPR == 64 ? 512 * NCH : 1];
  const int t = threadIdx.x % TPR;
  const int64_t team = (int64_t)blockIdx.x * (256 / TPR) + threadIdx.x / TPR, teams = (int64_t)gridDim.x * (256 / TPR);
  const int K = a.K;
  float* part = a.part ? a.part + blockIdx.x * (int64_t)K : nullptr;
  if constexpr (NCH > 0) {
    float w[NCH][8], dw[NCH][8];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = (c * TPR + t) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) w[c][i] = 1.f, dw[c][i] = 0.f;
      if (a.weight && col < K) load_row8<kF32>(a.weight, 0, col, K, w[c]);
    }
    int par = 0;
    for (int64_t m = team; m < a.M; m += teams, par ^= 1) {
      const int64_t row0 = m * (int64_t)K;
      float d[NCH][8], h[NCH][8];
      const float r = a.rstd[m];
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int col = (c * TPR + t) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) d[c][i] = h[c][i] = 0.f;
        if (col < K) {
          load_row8<DT>(a.dy, row0, col, K, d[c]);
          load_row8<HT>(a.h, row0, col, K, h[c]);
        }
      }
      float dot = 0.f;
#pragma unroll
      for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dw[c][i] = fmaf(d[c][i] * r, h[c][i], dw[c][i]);
          d[c][i] *= w[c][i];
          dot = fmaf(d[c][i], h[c][i], dot);
        }
      // (two LDS slots in turn: a row's barrier keeps the one before from being overwritten early)
      const float f = r * r * (team_sum<TPR>(dot, slot[par]) / (float)K);
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int col = (c * TPR + t) * 8;
        if (col < K) {
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = r * (d[c][i] - h[c][i] * f);
          if (a.dsum) {
            float s[8];
            load_row8<kF32>(a.dsum, row0, col, K, s);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] += s[i];
          }
          stream_row8(a.dx, row0, col, K, o);  // (20000 x 2048: 83 -> 69 us)
        }
      }
    }
    if (!part) return;
    if constexpr (TPR == 64) {
#pragma unroll
      for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) wave_dw[threadIdx.x >> 6][(c * 64 + t) * 8 + i] = dw[c][i];
      __syncthreads();
      for (int col = threadIdx.x; col < K; col += 256)
        part[col] = (wave_dw[0][col] + wave_dw[1][col]) + (wave_dw[2][col] + wave_dw[3][col]);
    } else {
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int col = (c * TPR + t) * 8;
        if (col < K) store_row8<kF32>(part, 0, col, K, dw[c]);
      }
    }
  } else {
    int par = 0;
    for (int64_t m = team; m < a.M; m += teams, par ^= 1) {
      const int64_t row0 = m * (int64_t)K;
      const float r = a.rstd[m];
      float dot = 0.f;
      for (int col = t * 8; col < K; col += TPR * 8) {
        float d[8], h[8], w[8], p[8];
        load_row8<DT>(a.dy, row0, col, K, d);
        load_row8<HT>(a.h, row0, col, K, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 1.f, p[i] = 0.f;
        if (a.weight) load_row8<kF32>(a.weight, 0, col, K, w);
        if (part) {
          if (m != team) load_row8<kF32>(part, 0, col, K, p);
#pragma unroll
          for (int i = 0; i < 8; ++i) p[i] = fmaf(d[i] * r, h[i], p[i]);
          store_row8<kF32>(part, 0, col, K, p);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) dot = fmaf(d[i] * w[i], h[i], dot);
      }
      const float f = r * r * (team_sum<TPR>(dot, slot[par]) / (float)K);
      for (int col = t * 8; col < K; col += TPR * 8) {
        float d[8], h[8], w[8], s[8];
        load_row8<DT>(a.dy, row0, col, K, d);
        load_row8<HT>(a.h, row0, col, K, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 1.f, s[i] = 0.f;
        if (a.weight) load_row8<kF32>(a.weight, 0, col, K, w);
        if (a.dsum) load_row8<kF32>(a.dsum, row0, col, K, s);
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = r * (d[i] * w[i] - h[i] * f) + s[i];
        stream_row8(a.dx, row0, col, K, o);
      }
    }
  }
}

// dw[k] = sum of the partial rows: 64 columns x 64 runs of rows to a
// workgroup (16 lanes of 4 columns: 256-byte pieces), each run summed in
// order, then the runs in order.
__global__ __launch_bounds__(1024) void norm_dw_sum(const float* part, float* dw, int64_t rows, int K) {
  __shared__ float s[64][64];
  const int c = 4 * (threadIdx.x & 15), run = threadIdx.x >> 4;
  const int col = blockIdx.x * 64 + c;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (col + 4 <= K) {
    struct __attribute__((packed, aligned(4))) P {
      float f[4];
    };
#pragma unroll 4
    for (int64_t p = run; p < rows; p += 64) {
      const P u = *reinterpret_cast<const P*>(part + p * (int64_t)K + col);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += u.f[i];
    }
  } else {
    for (int64_t p = run; p < rows; p += 64)
      for (int i = 0; i < 4; ++i)
        if (col + i < K) v[i] += part[p * (int64_t)K + col + i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) s[run][c + i] = v[i];
  __syncthreads();
  const int o = blockIdx.x * 64 + threadIdx.x;
  if (threadIdx.x >= 64 || o >= K) return;
  float sum = 0.f;
#pragma unroll 16
  for (int i = 0; i < 64; ++i) sum += s[i][threadIdx.x];
  dw[o] = sum;
}

// A wave to a short row, else a workgroup (20000 x 2048: 83 us, 96 with a wave to a row).  Two chunks up to 4096
// columns (20480 x 2560: 121 us, 229 with room for six; 12800 x 4096: 104, 168), then six rather than a second reading
// (10240 x 5120: 169 us, 279; 6400 x 8192: 146, 244; 4266 x 12288: 141, 251).  Six cost widths well below 12288 more
// than they need: with three chunks 10240 x 5120 took 112 us, with four 6400 x 8192 112.
bool bwd_waves(int64_t K) { return K <= 512; }

template <int DT, int HT>
void norm_bwd_launch(const NormBwdArgs& a, hipStream_t s) {
  const int K = a.K;
  const dim3 grid((unsigned)norm_bwd_parts(a.M, K));
  if (bwd_waves(K))
    hipLaunchKernelGGL((rms_norm_bwd_rows<64, 1, DT, HT>), grid, dim3(256), 0, s, a);
  else if (K <= 2048)
    hipLaunchKernelGGL((rms_norm_bwd_rows<256, 1, DT, HT>), grid, dim3(256), 0, s, a);
  else if (K <= 4096)
    hipLaunchKernelGGL((rms_norm_bwd_rows<256, 2, DT, HT>), grid, dim3(256), 0, s, a);
  else if (K <= 12288)
    hipLaunchKernelGGL((rms_norm_bwd_rows<256, 6, DT, HT>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((rms_norm_bwd_rows<256, 0, DT, HT>), grid, dim3(256), 0, s, a);
}

// ------------------------------------------------------------ conversion

// 16 lanes to a 128-column group, 16 groups to a workgroup; groups of all rows
// (padding groups of the scale rows included) numbered one after another.
template <int XT>
__global__ __launch_bounds__(256) void quant_rows(const void* x, uint8_t* q, uint8_t* scales, int64_t groups, int K,
                                                  int Gs) {
  const int64_t g = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  if (g >= groups) return;  // (whole DPP rows)
  const int64_t m = g / Gs;
  const int gi = (int)(g - m * Gs), col = gi * 128 + (threadIdx.x & 15) * 8;
  const int Kp = (K + 127) & ~127;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  if (col < K) load_row8<XT>(x, m * (int64_t)K, col, K, v);
  int byte;
  const uint2 b = quant_group(v, byte);
  if (col < Kp) *reinterpret_cast<uint2*>(q + m * Kp + col) = b;
  if ((threadIdx.x & 15) == 0) scales[g] = (uint8_t)(gi * 128 < K ? byte : 127);
}

// One 128 x 128 block of a weight to a workgroup: thread t holds half a row
// (64 columns).  The transposed copy goes through LDS (rows of 132 bytes).
template <int WT>
__global__ __launch_bounds__(256) void quant_weight(const void* w, uint8_t* q, uint8_t* scales, uint8_t* qt,
                                                    uint8_t* scales_t, int64_t N, int64_t K, int64_t blocks_k,
                                                    int64_t blocks_n) {
  __shared__ uint32_t tile[128 * 33];
  __shared__ uint32_t wmax[4];
  int64_t b = blockIdx.x;
  const int64_t kb = b % blocks_k;
  b /= blocks_k;
  const int64_t nb = b % blocks_n, e = b / blocks_n;
  const int r = threadIdx.x >> 1, half = threadIdx.x & 1;
  const int64_t n = nb * 128 + r, k0 = kb * 128 + half * 64;
  const int64_t Kp = blocks_k * 128, Np = blocks_n * 128;
  float v[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    const int64_t col = k0 + 8 * i;
    if (n < N && col < K) load_row8<WT>(w, (e * N + n) * K, (int)col, (int)K, v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, finite_bits(v[i][j]));
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
  if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = m;
  __syncthreads();
  const int byte = e8m0_of(max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3])));
  const float inv = __uint_as_float((uint32_t)(254 - byte) << 23);
  uint2 o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = to_e4m3x8(v[i], inv);
  if (n < N) {
    uint4* d = reinterpret_cast<uint4*>(q + (e * N + n) * Kp + k0);
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = make_uint4(o[2 * i].x, o[2 * i].y, o[2 * i + 1].x, o[2 * i + 1].y);
  }
  const int64_t Gs = (K + 511) / 512 * 4, Gt = (N + 511) / 512 * 4;
  if (threadIdx.x == 0) {
    uint8_t* s = scales + (e * blocks_n + nb) * Gs;
    s[kb] = (uint8_t)byte;
    if (kb == blocks_k - 1)
      for (int64_t g = blocks_k; g < Gs; ++g) s[g] = 127;
    if (scales_t) {
      uint8_t* st = scales_t + (e * blocks_k + kb) * Gt;
      st[nb] = (uint8_t)byte;
      if (nb == blocks_n - 1)
        for (int64_t g = blocks_n; g < Gt; ++g) st[g] = 127;
    }
  }
  if (!qt) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    tile[r * 33 + half * 16 + 2 * i] = o[i].x;
    tile[r * 33 + half * 16 + 2 * i + 1] = o[i].y;
  }
  __syncthreads();
  // column kc = thread / 2 of the block, its rows 64 half .. + 63
  const int64_t kc = kb * 128 + r;
  if (kc >= K) return;
  const uint8_t* tb = reinterpret_cast<const uint8_t*>(tile);
  uint4* d = reinterpret_cast<uint4*>(qt + (e * K + kc) * Np + nb * 128 + half * 64);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u[j] = 0;
#pragma unroll
      for (int z = 0; z < 4; ++z) u[j] |= (uint32_t)tb[(half * 64 + 16 * i + 4 * j + z) * 132 + r] << (8 * z);
    }
    d[i] = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s) {
  if (a.x_dtype == kF32)
    norm_launch_res<kF32>(a, s);
  else
    norm_launch_res<kBf16>(a, s);
  return hipGetLastError();
}

// Workgroups of the gradient, each with a partial row of dw: two to a CU, few
// enough that the partial rows stay a small part of the bytes.
int64_t norm_bwd_parts(int64_t M, int64_t K) {
  const int64_t need = bwd_waves(K) ? (M + 3) / 4 : M;
  return need < 512 ? need : 512;
}

hipError_t launch_rms_norm_bwd(const NormBwdArgs& a, hipStream_t s) {
  if (a.M > 0) {
    if (a.dy_dtype == kF32 && a.h_dtype == kF32)
      norm_bwd_launch<kF32, kF32>(a, s);
    else if (a.dy_dtype == kF32)
      norm_bwd_launch<kF32, kBf16>(a, s);
    else if (a.h_dtype == kF32)
      norm_bwd_launch<kBf16, kF32>(a, s);
    else
      norm_bwd_launch<kBf16, kBf16>(a, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.dweight) return hipSuccess;
  hipLaunchKernelGGL(norm_dw_sum, dim3((unsigned)((a.K + 63) / 64)), dim3(1024), 0, s, a.part, a.dweight,
                     norm_bwd_parts(a.M, a.K), a.K);
  return hipGetLastError();
}

hipError_t launch_quant_rows(const void* x, int x_dtype, uint8_t* q, uint8_t* scales, int64_t M, int K,
                             hipStream_t s) {
  const int Gs = (int)fp8_scale_row(K);
  const int64_t groups = M * Gs;
  const dim3 grid((unsigned)((groups + 15) / 16));
  if (x_dtype == kF32)
    hipLaunchKernelGGL((quant_rows<kF32>), grid, dim3(256), 0, s, x, q, scales, groups, K, Gs);
  else
    hipLaunchKernelGGL((quant_rows<kBf16>), grid, dim3(256), 0, s, x, q, scales, groups, K, Gs);
  return hipGetLastError();
}

hipError_t launch_quant_weight(const void* w, int w_dtype, uint8_t* q, uint8_t* scales, uint8_t* qt,
                               uint8_t* scales_t, int64_t E, int64_t N, int64_t K, hipStream_t s) {
  const int64_t bk = (K + 127) / 128, bn = (N + 127) / 128;
  const dim3 grid((unsigned)(E * bk * bn));
  if (w_dtype == kF32)
    hipLaunchKernelGGL((quant_weight<kF32>), grid, dim3(256), 0, s, w, q, scales, qt, scales_t, N, K, bk, bn);
  else
    hipLaunchKernelGGL((quant_weight<kBf16>), grid, dim3(256), 0, s, w, q, scales, qt, scales_t, N, K, bk, bn);
  return hipGetLastError();
}

}  // namespace hxq
