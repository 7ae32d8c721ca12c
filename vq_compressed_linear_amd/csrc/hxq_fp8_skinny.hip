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
// Bound: the weight's bytes (each weight row is read once for up to 16 rows of
// x).  Operands go from memory straight to registers.  A workgroup owns
// 16 outputs and 16 rows of x; its waves share the sum (wave w takes
// blocks w, w + waves, ...) so that a layer with few outputs still has enough
// loads in flight, and add their parts in wave order through LDS.  A sum that
// is split over workgroups as well leaves its parts in the workspace for
// fp8_sum.
//
// Measured, one row of x (bf16, converted in the kernel), the weights of enough
// layers in turn that they come from memory: 22016 x 2048 in 10.2 us (4.4 TB/s;
// a plain read of those bytes takes 8.8), 8512 x 2048 7.5, 2048 x 2048 5.2,
// 2048 x 11008 8.7 + 1.8 (two launches); 8 experts of 64, 2048 x 2048 each,
// 10.3 us.  (The figures that the plan's rules give are of weights that the
// last-level cache holds in part, the same for both sides of each.)

#include "hxq_fp8.h"
#include "hxq_fp8_device.h"
#include "hxq_fp8_tiles.h"

namespace hxq {

namespace {

// DEPTH: blocks of a wave in flight.  XT: -1 (x is e4m3), or the type of the values that the workgroup converts
// for itself (hxq_quant_fp8's arithmetic), into LDS: [16 rows][the split's
// bytes], then the scales.  That saves a launch where x is small (measured:
// one token through 22016 x 2048 and 2048 x 2048).
template <int WAVES, int XT, int DEPTH>
__global__ __launch_bounds__(64 * WAVES) void fp8_skinny(Fp8Args a, int tiles_n, int tiles_m) {
  __shared__ float red[WAVES][16][16];
  extern __shared__ __align__(16) uint8_t xlds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  int b = blockIdx.x;
  const int tn = b % tiles_n;
  b /= tiles_n;
  const int tm = b % tiles_m, split = b / tiles_m;
  const RowTile t = fp8_row_tile(a, tm, 16);
  if (t.rows <= 0) return;  // past the last expert's rows (uniform over the workgroup)
  const int n0 = tn * 16, n = min(n0 + l16, a.N - 1);
  const int nb = (a.N + 127) >> 7;
  const int kb0 = split * a.kbs, kb1 = min(kb0 + a.kbs, a.Kp >> 7), nk = kb1 - kb0;
  const uint8_t* wp = a.w + ((int64_t)t.expert * a.N + n) * a.Kp + 16 * g;
  const uint8_t* wsp = a.ws + ((int64_t)t.expert * nb + (n >> 7)) * a.Gs;
  const int row = min(l16, t.rows - 1);
  const uint8_t *xp, *xsp;  // of block kb0
  if constexpr (XT < 0) {
    const int64_t r = fp8_x_row(a, t.row0 + row);
    xp = a.x + r * a.Kp + 16 * g + ((int64_t)kb0 << 7);
    xsp = a.xs + r * a.Gs + kb0;
  }
  i32x4 w0[DEPTH], w1[DEPTH];
  float sw[DEPTH];
  auto load_w = [&](int kb, int d) {  // (past the end the last block again: read, not used)
    const int k = min(kb + d * WAVES, kb1 - 1);
    w0[d] = *reinterpret_cast<const i32x4*>(wp + ((int64_t)k << 7));
    w1[d] = *reinterpret_cast<const i32x4*>(wp + ((int64_t)k << 7) + 64);
    sw[d] = __uint_as_float((uint32_t)wsp[k] << 23);
  };
  if (nk > 0)
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load_w(kb0 + wave, d);
  if constexpr (XT >= 0) {
    uint8_t* scales = xlds + t.rows * (nk << 7);
    for (int q = threadIdx.x >> 4; q < t.rows * nk; q += 4 * WAVES) {  // 16 lanes to a group
      const int m = q / nk, kb = q - m * nk, col = ((kb0 + kb) << 7) + 8 * (threadIdx.x & 15);
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
      if (col < a.K) load_row8<XT>(a.xf, fp8_x_row(a, t.row0 + m) * a.K, col, a.K, v);
      int byte;
      const uint2 o = quant_group(v, byte);
      *reinterpret_cast<uint2*>(xlds + (m * nk + kb) * 128 + 8 * (threadIdx.x & 15)) = o;
      if ((threadIdx.x & 15) == 0) scales[m * nk + kb] = (uint8_t)byte;
    }
    __syncthreads();
    xp = xlds + row * (nk << 7) + 16 * g;
    xsp = scales + row * nk;
  }
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int kb = kb0 + wave; kb < kb1; kb += DEPTH * WAVES) {
    i32x4 x0[DEPTH], x1[DEPTH];
    float sx[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int k = min(kb + d * WAVES, kb1 - 1) - kb0;
      x0[d] = *reinterpret_cast<const i32x4*>(xp + (k << 7));
      x1[d] = *reinterpret_cast<const i32x4*>(xp + (k << 7) + 64);
      sx[d] = __uint_as_float((uint32_t)xsp[k] << 23);
    }
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      if (kb + d * WAVES >= kb1) break;
#pragma unroll
      for (int p = 0; p < 2; ++p) {  // 8 bytes of each lane: 32 of the block's k
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(w0[d][2 * p], w0[d][2 * p + 1], sw[d]),
                                                     widen8(x0[d][2 * p], x0[d][2 * p + 1], sx[d]), acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(w1[d][2 * p], w1[d][2 * p + 1], sw[d]),
                                                     widen8(x1[d][2 * p], x1[d][2 * p + 1], sx[d]), acc, 0, 0, 0);
      }
    }
    if (kb + DEPTH * WAVES < kb1)
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) load_w(kb + DEPTH * WAVES, d);
  }

  // lane (token l16, g) holds outputs 4 g .. + 3
  *reinterpret_cast<f32x4*>(&red[wave][l16][4 * g]) = acc;
  __syncthreads();
  if (threadIdx.x >= 256) return;
  const int m = threadIdx.x >> 4, c = threadIdx.x & 15;
  if (m >= t.rows || n0 + c >= a.N) return;
  float v = red[0][m][c];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) v += red[w][m][c];
  const int64_t at = (int64_t)(t.row0 + m) * a.N + n0 + c;
  if (a.S > 1) {
    a.part[(int64_t)split * a.M * a.N + at] = v;
  } else {
    if (a.bias) v += a.bias[(int64_t)t.expert * a.N + n0 + c];
    fp8_store(a, at, v);
  }
}

// y = bias + the splits' parts, in order: V consecutive outputs of a row to a
// thread, four splits' loads in flight.  Rows past the last expert's are left
// as they are.
template <int V>
__global__ __launch_bounds__(256) void fp8_sum(Fp8Args a) {
  typedef float vec __attribute__((ext_vector_type(V)));
  const int64_t total = (int64_t)fp8_rows_end(a) * a.N, stride = (int64_t)a.M * a.N;
  for (int64_t o = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V; o < total; o += (int64_t)gridDim.x * (256 * V)) {
    vec v = 0.f;
    const float* p = a.part + o;
    int s = 0;
    for (; s + 4 <= a.S; s += 4, p += 4 * stride) {
      vec u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = *reinterpret_cast<const vec*>(p + i * stride);
#pragma unroll
      for (int i = 0; i < 4; ++i) v += u[i];
    }
    for (; s < a.S; ++s, p += stride) v += *reinterpret_cast<const vec*>(p);
    if (a.bias) {
      const int m = (int)(o / a.N);
      const int e = a.offsets ? fp8_expert_of(a, m) : 0;
      const float* b = a.bias + (int64_t)e * a.N + (o - (int64_t)m * a.N);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] += b[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) fp8_store(a, o + i, v[i]);
  }
}

template <int WAVES, int DEPTH>
void skinny_launch(const Fp8Args& a, const Fp8Plan& p, hipStream_t s) {
  const dim3 grid((unsigned)(p.tiles_n * p.tiles_m * p.S)), block(64 * WAVES);
  const int lds = (a.M < 16 ? a.M : 16) * a.kbs * 129 + 15;
  if (a.x_dtype == kF32)
    hipLaunchKernelGGL((fp8_skinny<WAVES, kF32, DEPTH>), grid, block, lds, s, a, (int)p.tiles_n, (int)p.tiles_m);
  else if (a.x_dtype == kBf16)
    hipLaunchKernelGGL((fp8_skinny<WAVES, kBf16, DEPTH>), grid, block, lds, s, a, (int)p.tiles_n, (int)p.tiles_m);
  else
    hipLaunchKernelGGL((fp8_skinny<WAVES, -1, DEPTH>), grid, block, 0, s, a, (int)p.tiles_n, (int)p.tiles_m);
}

}  // namespace

hipError_t launch_fp8_skinny(const Fp8Args& a, const Fp8Plan& p, hipStream_t s) {
  if (p.depth == 2)  // (many workgroups: four waves each)
    skinny_launch<4, 2>(a, p, s);
  else if (p.waves == 4)
    skinny_launch<4, 1>(a, p, s);
  else if (p.waves == 8)
    skinny_launch<8, 1>(a, p, s);
  else
    skinny_launch<16, 1>(a, p, s);
  return hipGetLastError();
}

hipError_t launch_fp8_sum(const Fp8Args& a, hipStream_t s) {
  const bool vec = a.N % 4 == 0;  // (the workspace's parts are 256-byte aligned)
  const int64_t n = (int64_t)a.M * a.N / (vec ? 4 : 1), wgs = (n + 255) / 256;
  const dim3 grid((unsigned)(wgs < 8192 ? wgs : 8192));
  if (vec)
    hipLaunchKernelGGL(fp8_sum<4>, grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL(fp8_sum<1>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace hxq
