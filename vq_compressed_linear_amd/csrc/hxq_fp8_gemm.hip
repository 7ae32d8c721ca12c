// Block-scaled 8-bit product for many rows of x: 256 x 256 tiles of y, one
// layer or one per expert.
//
//     y[m][n] = bias[n] + sum_k (qx[m][k] px[m][k / 128]) (qw[n][k] pw[n / 128][k / 128])
//
// Eight waves, two to a SIMD, each own 128 rows of x by 64 outputs: eight
// accumulators of 32 x 32, the weight as the A operand (so a lane holds runs
// of four outputs of one row of y).  Two forms:
//   - bf16 y: v_mfma_scale_f32_32x32x64_f8f6f4 on the bytes as they are, which
//     takes both operands' powers of two;
//   - float32 y (WIDE): the bytes widened to bf16 with their power of two
//     (exact) for v_mfma_f32_32x32x16_bf16, because the 8-bit operation keeps
//     a product only down to 2^-13 of the largest in its group of 8.  Half the
//     matrix rate.
//
// A stage is 128 of k: one cache line of each of the tile's 512 operand rows,
// 64 KB of LDS, two stages in it.  Lines go from memory straight to LDS
// (global_load_lds_dwordx4, 8 lines to a wave instruction).  Piece c (16
// bytes) of row r is kept at position c ^ ((r >> 1) & 7) of the row: then any
// 16 lanes that read one piece of 16 consecutive rows touch every LDS bank
// once.  Per stage s and wave:
//   - the matrix ops of its first 64 of k, while the second half's operands
//     are read;
//   - wait until this wave's part of stage s + 1 has landed and its reads of
//     stage s are back; barrier (the one barrier of a stage: after it stage
//     s + 1 is whole and no wave reads stage s any more);
//   - the matrix ops of the second half, while stage s + 2 is requested into
//     the slot of stage s and the first operands of stage s + 1 are read.
// The requests are inline assembly: known to the compiler, every later read of
// LDS would wait for all of them.  They name no register that they write.

#include <type_traits>

#include "hxq_fp8.h"
#include "hxq_fp8_device.h"
#include "hxq_fp8_tiles.h"

namespace hxq {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int TILE = 256, ROW = 128, STAGE = 2 * TILE * ROW;

// 64 lanes x 16 bytes, from base + off (of each lane) to the 1024 bytes of LDS at `lds`.
__device__ __forceinline__ void request_lines(const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}

template <bool WIDE>
__global__ __launch_bounds__(512, 2) void fp8_tile256(Fp8Args a, int tiles_n, int tiles_m) {
  __shared__ __align__(1024) uint8_t lds[2 * STAGE];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave & 1, wn = wave >> 1;  // 2 x 4 over the tile
  const int r32 = lane & 31, half = lane >> 5;

  // tiles of eight row tiles (all of a column of them first) stay together on
  // one XCD, which then shares their lines in its L2
  const int total_m = a.offsets ? fp8_row_tiles(a, TILE) : tiles_m;
  const int64_t work = (int64_t)total_m * tiles_n;
  if ((int64_t)blockIdx.x >= work) return;
  const int per = (int)(work >> 3);
  const int bx = blockIdx.x;
  const int L = bx < 8 * per ? (bx & 7) * per + (bx >> 3) : bx;
  const int group = L / (8 * tiles_n), in = L - group * 8 * tiles_n;
  const int gm = min(8, total_m - 8 * group);
  const int tn = in / gm, tm = 8 * group + in - tn * gm;
  const RowTile t = fp8_row_tile(a, tm, TILE);
  if (t.rows <= 0) return;
  const int n0 = tn * TILE;
  const int nk = a.Kp >> 7, nb = (a.N + 127) >> 7;

  // this wave's lines of a stage: rows 32 wave .. + 31 of x and of the weight
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const uint8_t* wbase = a.w + ((int64_t)t.expert * a.N + n0) * a.Kp;
  const uint8_t* xbase = a.rows ? a.x : a.x + (int64_t)t.row0 * a.Kp;
  uint32_t xoff[4], woff[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = 32 * wave + 8 * j + (lane >> 3);
    const uint32_t piece = (uint32_t)((lane & 7) ^ ((r >> 1) & 7)) << 4;
    const int m = min(r, t.rows - 1);
    xoff[j] = (uint32_t)(a.rows ? fp8_x_row(a, t.row0 + m) : m) * (uint32_t)a.Kp + piece;
    woff[j] = (uint32_t)min(r, a.N - 1 - n0) * (uint32_t)a.Kp + piece;
  }
  auto request = [&](int s) {
    const uint32_t d = lds0 + (s & 1) * STAGE + wave * (32 * ROW);
#pragma unroll
    for (int j = 0; j < 4; ++j) request_lines(xbase + (int64_t)s * ROW, xoff[j], d + j * (8 * ROW));
#pragma unroll
    for (int j = 0; j < 4; ++j) request_lines(wbase + (int64_t)s * ROW, woff[j], d + TILE * ROW + j * (8 * ROW));
  };

  // scales: a word holds four stages' bytes
  const uint8_t* wsp = a.ws + ((int64_t)t.expert * nb + min((n0 + 64 * wn) >> 7, nb - 1)) * a.Gs;
  const uint8_t* xsp[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    xsp[j] = a.xs + fp8_x_row(a, t.row0 + min(128 * wm + 32 * j + r32, t.rows - 1)) * a.Gs;
  uint32_t sw, sx[4], sw_next, sx_next[4];
  auto load_scales = [&](int s) {  // of stages s .. s + 3 (s % 4 == 0)
    const int at = min(s, a.Gs - 4);
    sw_next = *reinterpret_cast<const uint32_t*>(wsp + at);
#pragma unroll
    for (int j = 0; j < 4; ++j) sx_next[j] = *reinterpret_cast<const uint32_t*>(xsp[j] + at);
  };

  // operand reads: piece 4 k64 + 2 half + q of row r32 (q = 0, 1), rows 32 apart 4096 bytes apart
  const int swz = (r32 >> 1) & 7;
  const uint32_t rd = lds0 + r32 * ROW + (((2 * half) ^ swz) << 4);
  const uint32_t rx = rd + 128 * wm * ROW, rw = rd + TILE * ROW + 64 * wn * ROW;
  // where the reads of (stage s, k64) start (piece q at + 16 q, flipped: the bit is never carried); kept
  // from being computed for all of a loop's stages ahead, which would not fit the registers
  auto at = [&](uint32_t base, int s, int k64) {
    uint32_t o = (base ^ (uint32_t)(k64 << 6)) + (s & 1) * STAGE;
    asm volatile("" : "+v"(o));
    return o;
  };
  auto read32 = [&](uint32_t o, int row) {
    typedef __attribute__((address_space(3))) const i32x4 lds_vec;
    const i32x4 lo = *(lds_vec*)(o + row * ROW), hi = *(lds_vec*)((o ^ 16) + row * ROW);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  i32x8 wcur[2], wnext[2], x[4];  // 32 bytes of a row each; x is read again as soon as its last matrix op is issued

  f32x16 acc[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
  // the matrix ops of one 64 of k, each x block's next bytes read behind them
  // (past the last stage what the slot holds, which nothing uses); SEL: the
  // stage's byte of the scale words
  auto step = [&](auto sel, int s, int k64) {
    constexpr int SEL = decltype(sel)::value;
    const float fw = __uint_as_float(((sw >> (8 * SEL)) & 255u) << 23);
#pragma unroll
    for (int i = 0; i < 2; ++i) wcur[i] = wnext[i];
    const uint32_t ow = at(rw, s, k64), ox = at(rx, s, k64);
#pragma unroll
    for (int i = 0; i < 2; ++i) wnext[i] = read32(ow, 32 * i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (!WIDE) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wcur[i], x[j], acc[i][j], 0, 0, SEL, (int)sw, SEL,
                                                                     (int)sx[j]);
      } else {
        const float fx = __uint_as_float(((sx[j] >> (8 * SEL)) & 255u) << 23);
#pragma unroll
        for (int p = 0; p < 4; ++p) {  // 8 bytes of each lane: 16 of the 64 k
          const bf16x8 xv = widen8(x[j][2 * p], x[j][2 * p + 1], fx);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen8(wcur[i][2 * p], wcur[i][2 * p + 1], fw), xv,
                                                               acc[i][j], 0, 0, 0);
        }
      }
      x[j] = read32(ox, 32 * j);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto landed = [&]() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory"); };

  auto take_scales = [&]() {
    sw = sw_next;
#pragma unroll
    for (int j = 0; j < 4; ++j) sx[j] = sx_next[j];
  };
  // a stage; REQ: stage s + 2 is there
  auto stage = [&](auto sel, auto req, int s) {
    step(sel, s, 1);
    landed();
    __builtin_amdgcn_s_barrier();
    // (the words requested in the group's first stage are here: looked at now, the compiler's wait for them is free)
    if constexpr (decltype(sel)::value == 1)
#pragma unroll
      for (int j = 0; j < 4; ++j) asm volatile("" : "+v"(sx_next[j]));
    if constexpr (decltype(req)::value) request(s + 2);
    step(sel, s + 1, 0);
  };
  using std::integral_constant;
  constexpr integral_constant<int, 0> s0{};
  constexpr integral_constant<int, 1> s1{};
  constexpr integral_constant<int, 2> s2{};
  constexpr integral_constant<int, 3> s3{};

  request(0);
  load_scales(0);
  landed();
  __builtin_amdgcn_s_barrier();
  if (nk > 1) request(1);
  take_scales();
#pragma unroll
  for (int i = 0; i < 2; ++i) wnext[i] = read32(rw, 32 * i);
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = read32(rx, 32 * j);
  // four stages to a scale word while there are two more behind them, then the rest
  int s = 0;
  for (; s + 6 <= nk; s += 4) {
    load_scales(s + 4);
    stage(s0, std::true_type{}, s);
    stage(s1, std::true_type{}, s + 1);
    stage(s2, std::true_type{}, s + 2);
    stage(s3, std::true_type{}, s + 3);
    take_scales();
  }
  load_scales(s + 4);
  const int turn = s + 3;
  auto shift_scales = [&]() {
    sw = s == turn ? sw_next : sw >> 8;
#pragma unroll
    for (int j = 0; j < 4; ++j) sx[j] = s == turn ? sx_next[j] : sx[j] >> 8;
  };
  for (; s + 2 < nk; ++s) {  // at most three
    stage(s0, std::true_type{}, s);
    shift_scales();
  }
  for (; s < nk; ++s) {
    stage(s0, std::false_type{}, s);
    shift_scales();
  }

  // lane: row of y 128 wm + 32 j + r32, outputs 64 wn + 32 i + 8 e + 4 half .. + 3
  const float* bias = a.bias ? a.bias + (int64_t)t.expert * a.N : nullptr;
  const bool vec = (a.N & 3) == 0 && ((uintptr_t)a.y & 15) == 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int m = 128 * wm + 32 * j + r32;
    if (m >= t.rows) continue;
    const int64_t row = (int64_t)(t.row0 + m) * a.N;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int n = n0 + 64 * wn + 32 * i + 8 * e + 4 * half;
        float v[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) v[z] = acc[i][j][4 * e + z];
        if (bias)
#pragma unroll
          for (int z = 0; z < 4; ++z) v[z] += n + z < a.N ? bias[n + z] : 0.f;
        if (vec && n + 4 <= a.N) {
          if (WIDE)
            *reinterpret_cast<float4*>(static_cast<float*>(a.y) + row + n) = make_float4(v[0], v[1], v[2], v[3]);
          else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + row + n) =
                make_uint2(f32_to_bf16_rne(v[0]) | (f32_to_bf16_rne(v[1]) << 16),
                           f32_to_bf16_rne(v[2]) | (f32_to_bf16_rne(v[3]) << 16));
        } else {
#pragma unroll
          for (int z = 0; z < 4; ++z)
            if (n + z < a.N) fp8_store(a, row + n + z, v[z]);
        }
      }
  }
}

}  // namespace

hipError_t launch_fp8_tile256(const Fp8Args& a, const Fp8Plan& p, hipStream_t s) {
  const dim3 grid((unsigned)(p.tiles_n * p.tiles_m));
  if (a.y_bf16)
    hipLaunchKernelGGL((fp8_tile256<false>), grid, dim3(512), 0, s, a, (int)p.tiles_n, (int)p.tiles_m);
  else
    hipLaunchKernelGGL((fp8_tile256<true>), grid, dim3(512), 0, s, a, (int)p.tiles_n, (int)p.tiles_m);
  return hipGetLastError();
}

}  // namespace hxq
