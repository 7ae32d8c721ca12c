// Block-scaled 8-bit product for few rows of x, one layer or one per expert.
//
//     y[m][n] = bias[n] + sum_k (qx[m][k] px[m][k / 128]) (qw[n][k] pw[n / 128][k / 128])
//
// Operands are widened to bf16 on their way to the matrix cores, with their
// power of two (v_cvt_scalef32_pk_bf16_fp8: 4 significant bits, so exactly),
// and multiplied by v_mfma_f32_16x16x32_bf16: the 8-bit matrix operations keep
// a product only down to 2^-13 of the largest of its group of 8 (measured:
// 1.5e-5 of the result against 5e-8 this way), and these calls do not wait for
// the matrix cores.  The weight is the A operand (its 16 rows are outputs), x
// is B (its 16 columns are tokens).  The order of k within an instruction is
// free as long as both operands agree, so lane (row, g) loads bytes 16 g .. + 15
// and 64 + 16 g .. + 15 of a 128-block: each load instruction reads 64
// consecutive bytes of each of its 16 rows, and the block's two instructions
// share their cache lines.
//
// Bound: the weight's bytes (each weight row is read once for up to 64 rows of
// x).  Operands go from memory straight to registers.  A workgroup owns
// 16 RW outputs and 16 NT rows of x; its waves share the sum (wave w takes
// blocks w, w + waves, ...) so that a layer with few outputs still has enough
// loads in flight, and add their parts in wave order through LDS.  A sum that
// is split over workgroups as well leaves its parts in the workspace for
// fp8_sum.

#include "hxq_fp8.h"
#include "hxq_fp8_device.h"
#include "hxq_fp8_tiles.h"

namespace hxq {

namespace {

template <int RW, int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void fp8_skinny(Fp8Args a, int tiles_n, int tiles_m) {
  constexpr int TN = 16 * RW, TM = 16 * NT;
  extern __shared__ float red[];  // [WAVES][TM][TN]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  int b = blockIdx.x;
  const int tn = b % tiles_n;
  b /= tiles_n;
  const int tm = b % tiles_m, split = b / tiles_m;
  const RowTile t = fp8_row_tile(a, tm, TM);
  if (t.rows <= 0) return;  // past the last expert's rows (uniform over the workgroup)
  const int n0 = tn * TN;
  const int nb = (a.N + 127) >> 7;
  const int kb1 = min((split + 1) * a.kbs, a.Kp >> 7);

  const uint8_t* wp[RW];
  const uint8_t* wsp[RW];
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    const int n = min(n0 + 16 * i + l16, a.N - 1);
    wp[i] = a.w + ((int64_t)t.expert * a.N + n) * a.Kp + 16 * g;
    wsp[i] = a.ws + ((int64_t)t.expert * nb + (n >> 7)) * a.Gs;
  }
  const uint8_t* xp[NT];
  const uint8_t* xsp[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t r = fp8_x_row(a, t.row0 + min(16 * j + l16, t.rows - 1));
    xp[j] = a.x + r * a.Kp + 16 * g;
    xsp[j] = a.xs + r * a.Gs;
  }
  f32x4 acc[RW][NT];
#pragma unroll
  for (int i = 0; i < RW; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

#pragma unroll 2
  for (int kb = split * a.kbs + wave; kb < kb1; kb += WAVES) {
    const int64_t k = (int64_t)kb << 7;
    i32x8 wa[RW], xb[NT];
    float sa[RW], sb[NT];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const i32x4 lo = *reinterpret_cast<const i32x4*>(wp[i] + k), hi = *reinterpret_cast<const i32x4*>(wp[i] + k + 64);
      wa[i] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      sa[i] = __uint_as_float((uint32_t)wsp[i][kb] << 23);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const i32x4 lo = *reinterpret_cast<const i32x4*>(xp[j] + k), hi = *reinterpret_cast<const i32x4*>(xp[j] + k + 64);
      xb[j] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      sb[j] = __uint_as_float((uint32_t)xsp[j][kb] << 23);
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) {  // 8 bytes of each lane: 32 of the block's k
      bf16x8 wv[RW], xv[NT];
#pragma unroll
      for (int i = 0; i < RW; ++i) wv[i] = widen8(wa[i][2 * p], wa[i][2 * p + 1], sa[i]);
#pragma unroll
      for (int j = 0; j < NT; ++j) xv[j] = widen8(xb[j][2 * p], xb[j][2 * p + 1], sb[j]);
#pragma unroll
      for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[i], xv[j], acc[i][j], 0, 0, 0);
    }
  }

  // lane (token l16, g) holds outputs 4 g .. + 3 of each 16 x 16 tile
#pragma unroll
  for (int i = 0; i < RW; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
      *reinterpret_cast<f32x4*>(red + ((wave * TM + 16 * j + l16) * TN + 16 * i + 4 * g)) = acc[i][j];
  __syncthreads();
  for (int o = threadIdx.x; o < TM * TN; o += 64 * WAVES) {
    const int m = o / TN, n = n0 + o % TN;
    if (m >= t.rows || n >= a.N) continue;
    float v = red[o];
    for (int w = 1; w < WAVES; ++w) v += red[w * TM * TN + o];
    const int64_t at = (int64_t)(t.row0 + m) * a.N + n;
    if (a.S > 1) {
      a.part[(int64_t)split * a.M * a.N + at] = v;
    } else {
      if (a.bias) v += a.bias[(int64_t)t.expert * a.N + n];
      fp8_store(a, at, v);
    }
  }
}

// y = bias + the splits' parts, in order.  Rows past the last expert's are
// left as they are.
__global__ __launch_bounds__(256) void fp8_sum(Fp8Args a) {
  const int64_t total = (int64_t)fp8_rows_end(a) * a.N, stride = (int64_t)a.M * a.N;
  for (int64_t o = (int64_t)blockIdx.x * 256 + threadIdx.x; o < total; o += (int64_t)gridDim.x * 256) {
    float v = 0.f;
    for (int s = 0; s < a.S; ++s) v += a.part[s * stride + o];
    if (a.bias) {
      const int m = (int)(o / a.N);
      const int e = a.offsets ? fp8_expert_of(a, m) : 0;
      v += a.bias[(int64_t)e * a.N + (o - (int64_t)m * a.N)];
    }
    fp8_store(a, o, v);
  }
}

template <int RW, int NT, int WAVES>
void skinny_launch(const Fp8Args& a, const Fp8Plan& p, hipStream_t s) {
  const int lds = WAVES * RW * NT * 256 * 4;
  hipLaunchKernelGGL((fp8_skinny<RW, NT, WAVES>), dim3((unsigned)(p.tiles_n * p.tiles_m * p.S)), dim3(64 * WAVES), lds,
                     s, a, (int)p.tiles_n, (int)p.tiles_m);
}

}  // namespace

hipError_t launch_fp8_skinny(const Fp8Args& a, const Fp8Plan& p, hipStream_t s) {
  if (p.kernel == kFp8Skinny16)
    p.waves == 4 ? skinny_launch<1, 1, 4>(a, p, s) : skinny_launch<1, 1, 8>(a, p, s);
  else if (p.kernel == kFp8Skinny32)
    skinny_launch<2, 2, 4>(a, p, s);
  else
    skinny_launch<4, 4, 4>(a, p, s);
  return hipGetLastError();
}

hipError_t launch_fp8_sum(const Fp8Args& a, hipStream_t s) {
  const int64_t wgs = ((int64_t)a.M * a.N + 1023) / 1024;
  hipLaunchKernelGGL(fp8_sum, dim3((unsigned)(wgs < 4096 ? wgs : 4096)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace hxq
