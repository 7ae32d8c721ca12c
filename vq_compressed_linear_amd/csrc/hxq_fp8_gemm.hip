// Block-scaled 8-bit product for more than a few rows of x: tiles of y staged
// through LDS, one layer or one per expert.
//
//     y[m][n] = bias[n] + sum_k (qx[m][k] px[m][k / 128]) (qw[n][k] pw[n / 128][k / 128])
//
// Shapes (rows of x x outputs): 32 x 64 (2 waves), 64 x 128 (8), 128 x 128 (4)
// and 256 x 256 (8).  A wave owns FJ x FI blocks of 32 x 32, the weight as the
// A operand (so a lane holds runs of four outputs of one row of y).  In two
// forms:
//   - bf16 y: v_mfma_scale_f32_32x32x64_f8f6f4 on the bytes as they are, which
//     takes both operands' powers of two;
//   - float32 y (WIDE): the bytes widened to bf16 with their power of two
//     (exact) for v_mfma_f32_32x32x16_bf16, because the 8-bit operation keeps
//     a product only down to 2^-13 of the largest in its group of 8.  Half the
//     matrix rate.
//
// Bound: the matrix cores for the large tiles, the weight's bytes for the small
// ones.  Measured: 8192^3 in 411-414 us with bf16 y (2.7 PFLOP/s), 745-761 us
// with float32 y (1.45-1.48); gate|up (22016 x 2048) at 2048 rows 88-90 us with
// bf16 y; 64 experts of 2048 x 2048 with 8 rows each 54 us from memory (5.0
// TB/s).  In the large tile the matrix cores are busy for 74% of the CUs' time
// at 8192^3 (64 stages; 82% with float32 y), 57% at gate|up's 16 stages and 45%
// with experts' ragged rows there: a stage takes 1.4 us, a tile's start and its
// output (every CU stores 128 KB at once) some 8 to 10 us.  No LDS bank conflicts
// in the loop.  Four waves of 128 x 128 instead of eight of 128 x 64
// read a third less LDS but leave nothing to run behind a wait (8192^3 485
// against 428 us); rings of four to seven stages gained nothing for the small
// tiles; s_setprio around the matrix ops cost 1-2%.
//
// A stage is 128 of k: one cache line of each of the tile's operand rows (64 KB
// of LDS for the largest tile), SLOTS stages in a ring.  Lines go from memory straight to LDS
// (global_load_lds_dwordx4, 8 lines to a wave instruction).  Piece c (16
// bytes) of row r is kept at position c ^ ((r >> 1) & 7) of the row: then any
// 16 lanes that read one piece of 16 consecutive rows touch every LDS bank
// once.  Per stage s and wave:
//   - the matrix ops of its first 64 of k, while the second half's operands
//     are read;
//   - wait until this wave's part of stage s + 1 has landed and its reads of
//     stage s are back; barrier (the one barrier of a stage: after it stage
//     s + 1 is whole and no wave reads stage s any more);
//   - the matrix ops of the second half, while stage s + SLOTS is requested
//     into the slot of stage s and the first operands of stage s + 1 are read.
// Scales travel the same way, as words of four stages' bytes, every fourth
// stage.
// The requests are inline assembly: known to the compiler, every later read of
// LDS would wait for all of them.  They name no register that they write.

#include <type_traits>

#include "hxq_fp8.h"
#include "hxq_fp8_device.h"
#include "hxq_fp8_tiles.h"

namespace hxq {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int ROW = 128;  // bytes of a row in a stage

// 64 lanes x 16 (4) bytes, from base + off (of each lane) to the 1024 (256) bytes of LDS at `lds`.
__device__ __forceinline__ void request_lines(const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}
__device__ __forceinline__ void request_words(const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
               :
               : "s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}

// WM x WN waves, each FJ blocks of 32 rows of x by FI blocks of 32 outputs; SLOTS stages in LDS.
template <int WM_, int WN_, int FJ_, int FI_, int SLOTS_>
struct TileShape {
  static constexpr int WM = WM_, WN = WN_, FJ = FJ_, FI = FI_, SLOTS = SLOTS_;
  static constexpr int WAVES = WM * WN, TM = 32 * WM * FJ, TN = 32 * WN * FI;
  static constexpr int STAGE = (TM + TN) * ROW;
  static constexpr int PER = (TM + TN) / 8 / WAVES;  // line requests of a wave and stage
  static constexpr int XWORDS = TM < 64 ? 64 : TM;   // a group's scale words: x's rows, then the weight's blocks
  static constexpr int WORDS = 4 * (XWORDS + 64);
  static constexpr int WPER = (XWORDS / 64 + WAVES) / WAVES;  // word requests of a wave and group
  static constexpr int LDS = SLOTS * STAGE + 2 * WORDS;
  static_assert(PER * 8 * WAVES == TM + TN && SLOTS <= 4 && LDS <= 160 * 1024, "tile shape");
};

template <bool WIDE, class T>
__device__ __forceinline__ void tile_body(const Fp8Args& a, uint8_t* lds, const RowTile t, const int n0, const int split) {
  constexpr int WM = T::WM, FJ = T::FJ, FI = T::FI, SLOTS = T::SLOTS, TM = T::TM, STAGE = T::STAGE, PER = T::PER;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int r32 = lane & 31, half = lane >> 5;
  const int nb = (a.N + 127) >> 7;
  const int kb0 = split * a.kbs, nk = min(a.kbs, (a.Kp >> 7) - kb0);  // the split's stages (kbs % 4 == 0 if split)

  // this wave's lines of a stage: of the tile's rows of x, then of the weight
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const uint8_t* wbase = a.w + ((int64_t)t.expert * a.N + n0) * a.Kp + (int64_t)kb0 * ROW;
  const uint8_t* xbase = (a.rows ? a.x : a.x + (int64_t)t.row0 * a.Kp) + (int64_t)kb0 * ROW;
  const uint8_t* line_base[PER];
  uint32_t line_off[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int r = 8 * (PER * wave + j) + (lane >> 3);
    const bool of_x = 8 * (PER * wave + j) < TM;
    const uint32_t piece = (uint32_t)((lane & 7) ^ ((r >> 1) & 7)) << 4;
    const int m = min(r, t.rows - 1);
    const uint32_t row = of_x ? (uint32_t)(a.rows ? fp8_x_row(a, t.row0 + m) : m) : (uint32_t)min(r - TM, a.N - 1 - n0);
    line_off[j] = row * (uint32_t)a.Kp + piece;
    line_base[j] = of_x ? xbase : wbase;
  }
  // and scale words (four stages' bytes), a wave's 64 of them: x's rows, then the weight's blocks (which the
  // waves left over request as well: a branch here would part the matrix ops around it)
  const uint8_t* word_base[T::WPER];
  uint32_t word_off[T::WPER], word_to[T::WPER];
#pragma unroll
  for (int j = 0; j < T::WPER; ++j) {
    const int w = min(wave + j * T::WAVES, T::XWORDS / 64);
    word_to[j] = lds0 + SLOTS * STAGE + 256 * w;
    if (w < T::XWORDS / 64) {
      const int m = min(64 * w + lane, t.rows - 1);
      word_base[j] = (a.rows ? a.xs : a.xs + (int64_t)t.row0 * a.Gs) + kb0;
      word_off[j] = (uint32_t)(a.rows ? fp8_x_row(a, t.row0 + m) : m) * (uint32_t)a.Gs;
    } else {
      word_base[j] = a.ws + ((int64_t)t.expert * nb + (n0 >> 7)) * a.Gs + kb0;
      word_off[j] = (uint32_t)min(lane, nb - 1 - (n0 >> 7)) * (uint32_t)a.Gs;
    }
  }
  const uint32_t words0 = lds0 + SLOTS * STAGE;
  auto request_scales = [&](int s) {
#pragma unroll
    for (int j = 0; j < T::WPER; ++j)
      request_words(word_base[j] + (s & ~3), word_off[j], word_to[j] + ((s >> 2) & 1) * T::WORDS);
  };
  auto request = [&](int s, uint32_t slot, int from, int to) {  // lines from .. to - 1 of stage s
    const uint32_t d = lds0 + slot * STAGE + wave * (PER * 1024);
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (j >= from && j < to) request_lines(line_base[j] + (int64_t)s * ROW, line_off[j], d + j * 1024);
  };

  uint32_t sw, sx[FJ], sw_next, sx_next[FJ];
  auto read_scales = [&](int s) {  // the words of the group of stage s
    typedef __attribute__((address_space(3))) const uint32_t lds_word;
    const uint32_t o = words0 + ((s >> 2) & 1) * T::WORDS;
    sw_next = *(lds_word*)(o + 4 * T::XWORDS + 4 * ((32 * FI * wn) >> 7));
#pragma unroll
    for (int j = 0; j < FJ; ++j) sx_next[j] = *(lds_word*)(o + 4 * (32 * (FJ * wm + j) + r32));
  };

  // operand reads: piece 4 k64 + 2 half + q of row r32 (q = 0, 1), rows 32 apart 4096 bytes apart
  const int swz = (r32 >> 1) & 7;
  const uint32_t rd = lds0 + r32 * ROW + (((2 * half) ^ swz) << 4);
  const uint32_t rx = rd + 32 * FJ * wm * ROW, rw = rd + TM * ROW + 32 * FI * wn * ROW;
  // where the reads of (slot, k64) start (piece q at + 16 q, flipped: the bit is never carried); kept
  // from being computed for all of a loop's stages ahead, which would not fit the registers
  auto at = [&](uint32_t base, uint32_t slot, int k64) {
    uint32_t o = (base ^ (uint32_t)(k64 << 6)) + slot * STAGE;
    asm volatile("" : "+v"(o));
    return o;
  };
  auto read32 = [&](uint32_t o, int row) {
    typedef __attribute__((address_space(3))) const i32x4 lds_vec;
    const i32x4 lo = *(lds_vec*)(o + row * ROW), hi = *(lds_vec*)((o ^ 16) + row * ROW);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  i32x8 wcur[FI], wnext[FI], x[FJ];  // 32 bytes of a row each; x is read again as soon as its last matrix op is issued

  f32x16 acc[FI][FJ];
#pragma unroll
  for (int i = 0; i < FI; ++i)
#pragma unroll
    for (int j = 0; j < FJ; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
  // the matrix ops of one 64 of k, each x block's next bytes (of slot, k64) read behind them
  // (past the last stage what the slot holds, which nothing uses), and after x block j's behind(j);
  // SEL: the stage's byte of the scale words
  auto step = [&](auto sel, uint32_t slot, int k64, auto behind) {
    constexpr int SEL = decltype(sel)::value;
    const float fw = __uint_as_float(((sw >> (8 * SEL)) & 255u) << 23);
#pragma unroll
    for (int i = 0; i < FI; ++i) wcur[i] = wnext[i];
    const uint32_t ow = at(rw, slot, k64), ox = at(rx, slot, k64);
#pragma unroll
    for (int i = 0; i < FI; ++i) wnext[i] = read32(ow, 32 * i);
#pragma unroll
    for (int j = 0; j < FJ; ++j) {
      if constexpr (!WIDE) {
#pragma unroll
        for (int i = 0; i < FI; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wcur[i], x[j], acc[i][j], 0, 0, SEL, (int)sw, SEL,
                                                                     (int)sx[j]);
      } else {
        const float fx = __uint_as_float(((sx[j] >> (8 * SEL)) & 255u) << 23);
#pragma unroll
        for (int p = 0; p < 4; ++p) {  // 8 bytes of each lane: 16 of the 64 k
          const bf16x8 xv = widen8(x[j][2 * p], x[j][2 * p + 1], fx);
#pragma unroll
          for (int i = 0; i < FI; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen8(wcur[i][2 * p], wcur[i][2 * p + 1], fw), xv,
                                                               acc[i][j], 0, 0, 0);
        }
      }
      x[j] = read32(ox, 32 * j);
      behind(j);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // all but the newest LEFT requests of this wave have landed, and its reads of LDS are back
  auto landed = [&](auto left) {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(decltype(left)::value) : "memory");
  };
  using std::integral_constant;
  constexpr integral_constant<int, 0> s0{};
  constexpr integral_constant<int, 1> s1{};
  constexpr integral_constant<int, 2> s2{};
  constexpr integral_constant<int, 3> s3{};
  constexpr integral_constant<int, (SLOTS - 2) * PER> in_flight{};
  auto next = [](uint32_t slot) { return slot + 1 == SLOTS ? 0u : slot + 1; };
  // stage s, in `slot`; req: stage s + SLOTS is there (and so are the ones before it); words: its scale words too
  auto stage = [&](auto sel, auto req, auto words, int s, uint32_t slot) {
    step(sel, slot, 1, [](int) {});
    if constexpr (decltype(req)::value)
      landed(in_flight);
    else
      landed(s0);
    __builtin_amdgcn_s_barrier();
    // The largest tile's requests go out between the matrix ops, whose operands are here already (8192^3 429 ->
    // 413 us); the others', which wait for memory rather than for the matrix cores, before them (128 x 128 tiles
    // 65 against 67 us at 2047 x 2048 x 8512).
    constexpr bool REQ = decltype(req)::value, BETWEEN = FJ >= 4;
    if constexpr (REQ && decltype(words)::value) request_scales(s + SLOTS);
    if constexpr (REQ && !BETWEEN) request(s + SLOTS, slot, 0, PER);
    step(sel, next(slot), 0, [&](int j) {
      if constexpr (REQ && BETWEEN) request(s + SLOTS, slot, PER * j / FJ, PER * (j + 1) / FJ);
    });
  };
  auto take_scales = [&]() {
    sw = sw_next;
#pragma unroll
    for (int j = 0; j < FJ; ++j) sx[j] = sx_next[j];
  };

  request_scales(0);
#pragma unroll
  for (int i = 0; i < SLOTS; ++i)
    if (nk > i) request(i, i, 0, PER);
  if (nk >= SLOTS)
    landed(integral_constant<int, (SLOTS - 1) * PER>{});  // stage 0 and its scales
  else
    landed(s0);
  __builtin_amdgcn_s_barrier();
  read_scales(0);
  take_scales();
#pragma unroll
  for (int i = 0; i < FI; ++i) wnext[i] = read32(rw, 32 * i);
#pragma unroll
  for (int j = 0; j < FJ; ++j) x[j] = read32(rx, 32 * j);
  // four stages to a scale word while all four have stage s + SLOTS, then the rest
  int s = 0;
  uint32_t slot = 0;
  for (; s + 4 + SLOTS <= nk; s += 4) {
    stage(s0, std::true_type{}, integral_constant<bool, (SLOTS + 0) % 4 == 0>{}, s, slot);
    slot = next(slot);
    stage(s1, std::true_type{}, integral_constant<bool, (SLOTS + 1) % 4 == 0>{}, s + 1, slot);
    slot = next(slot);
    stage(s2, std::true_type{}, integral_constant<bool, (SLOTS + 2) % 4 == 0>{}, s + 2, slot);
    slot = next(slot);
    stage(s3, std::true_type{}, integral_constant<bool, (SLOTS + 3) % 4 == 0>{}, s + 3, slot);
    slot = next(slot);
    read_scales(s + 4);  // they landed with stage s + 4, before the last barrier
    take_scales();
  }
  auto shift_scales = [&]() {  // to the bytes of stage s + 1
    read_scales(s + 1);
    sw = (s & 3) == 3 ? sw_next : sw >> 8;
#pragma unroll
    for (int j = 0; j < FJ; ++j) sx[j] = (s & 3) == 3 ? sx_next[j] : sx[j] >> 8;
  };
  for (; s + SLOTS < nk; ++s) {  // at most three
    stage(s0, std::true_type{}, std::true_type{}, s, slot);  // (scale words that are there already: the same again)
    slot = next(slot);
    shift_scales();
  }
  for (; s < nk; ++s) {
    stage(s0, std::false_type{}, std::false_type{}, s, slot);
    slot = next(slot);
    shift_scales();
  }

  // A lane holds row r32 of 32 (FJ wm + j), outputs 32 i + 8 e + 4 half .. + 3: turned through LDS (no longer
  // read by anyone), 32 rows at a time in the wave's own part, so that each row's stores are whole cache lines.
  // 16-byte piece c of row r is kept at c ^ key(r), as above.
  landed(s0);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  constexpr int RB = 128 * FI, PIECES = 8 * FI;  // bytes and pieces of a row
  static_assert(T::WAVES * 32 * RB <= T::LDS, "the waves' parts");
  auto key = [](int r) { return FI == 1 ? (r >> 1) & 7 : r & 15; };
  float* turn = reinterpret_cast<float*>(lds + wave * (32 * RB));
  const float* bias = a.bias && a.S == 1 ? a.bias + (int64_t)t.expert * a.N : nullptr;
  float* part = a.S > 1 ? a.part + (int64_t)split * a.M * a.N : nullptr;
  const bool out_f32 = part || !a.y_bf16;
  float* yf = part ? part : static_cast<float*>(a.y);
  const int nw = n0 + 32 * FI * wn;  // the wave's first output
  const bool vec = part ? (a.N & 3) == 0
                        : ((uintptr_t)a.y & 15) == 0 && (a.N & (out_f32 ? 3 : 7)) == 0;
#pragma unroll
  for (int j = 0; j < FJ; ++j) {
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = (8 * i + 2 * e + half) ^ key(r32);
        *reinterpret_cast<f32x4*>(turn + r32 * (RB / 4) + 4 * c) =
            f32x4{acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]};
      }
    __builtin_amdgcn_wave_barrier();
    const int m0 = 32 * (FJ * wm + j);
    if (vec && out_f32) {
#pragma unroll 2
      for (int it = 0; it < PIECES / 2; ++it) {
        const int r = it * (64 / PIECES) + lane / PIECES, c = lane % PIECES, n = nw + 4 * c;
        f32x4 v = *reinterpret_cast<const f32x4*>(turn + r * (RB / 4) + 4 * (c ^ key(r)));
        if (m0 + r < t.rows && n < a.N) {
          if (bias)
#pragma unroll
            for (int z = 0; z < 4; ++z) v[z] += bias[n + z];
          // stored past the caches, which hold the operands that the tiles still to come share (experts with 64 rows
          // each, float32 y, 77 -> 67 us; 512 rows of gate|up, bf16 y, 32.4 -> 29.6; split sums gain as well)
          __builtin_nontemporal_store(v, reinterpret_cast<f32x4*>(yf + (int64_t)(t.row0 + m0 + r) * a.N + n));
        }
      }
    } else if (vec) {
      constexpr int PAIRS = PIECES / 2;
#pragma unroll 2
      for (int it = 0; it < PAIRS / 2; ++it) {
        const int r = it * (64 / PAIRS) + lane / PAIRS, c = 2 * (lane % PAIRS), n = nw + 4 * c;
        f32x4 v = *reinterpret_cast<const f32x4*>(turn + r * (RB / 4) + 4 * (c ^ key(r)));
        f32x4 u = *reinterpret_cast<const f32x4*>(turn + r * (RB / 4) + 4 * ((c + 1) ^ key(r)));
        if (m0 + r < t.rows && n < a.N) {
          if (bias)
#pragma unroll
            for (int z = 0; z < 4; ++z) v[z] += bias[n + z], u[z] += bias[n + 4 + z];
          const u32x4 o = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                           pack_bf16(u[0], u[1]), pack_bf16(u[2], u[3])};
          __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.y) + (int64_t)(t.row0 + m0 + r) * a.N + n));
        }
      }
    } else {
      for (int it = 0; it < 32 * 32 * FI / 64; ++it) {
        const int o = it * 64 + lane, r = o / (32 * FI), q = o % (32 * FI), n = nw + q;
        float v = turn[r * (RB / 4) + 4 * ((q >> 2) ^ key(r)) + (q & 3)];
        if (m0 + r < t.rows && n < a.N) {
          if (bias) v += bias[n];
          const int64_t o64 = (int64_t)(t.row0 + m0 + r) * a.N + n;
          if (part)
            part[o64] = v;
          else
            fp8_store(a, o64, v);
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// Tiles of T; one whose rows fit S's height (an expert's last, mostly) is done in that shape, with the matrix ops
// of the rows it has.
template <bool WIDE, class T, class S>
__global__ __launch_bounds__(64 * T::WAVES, 2) void fp8_tile(Fp8Args a, int tiles_n, int tiles_m) {
  static_assert(T::WAVES == S::WAVES && T::TN == S::TN, "one grid for both");
  __shared__ __align__(1024) uint8_t lds[T::LDS > S::LDS ? T::LDS : S::LDS];
  // tiles of eight row tiles (all of a column of them first) stay together on
  // one XCD, which then shares their lines in its L2
  const int total_m = a.offsets ? fp8_row_tiles(a, T::TM, tiles_m) : tiles_m;
  const int64_t work = (int64_t)total_m * tiles_n * a.S;
  if ((int64_t)blockIdx.x >= work) return;
  const int per = (int)(work >> 3);
  const int bx = blockIdx.x;
  int L = bx < 8 * per ? (bx & 7) * per + (bx >> 3) : bx;
  const int split = L / (total_m * tiles_n);
  L -= split * (total_m * tiles_n);
  const int group = L / (8 * tiles_n), in = L - group * 8 * tiles_n;
  const int gm = min(8, total_m - 8 * group);
  const int tn = in / gm, tm = 8 * group + in - tn * gm;
  const RowTile t = fp8_row_tile(a, tm, T::TM);
  if (t.rows <= 0) return;
  if (T::TM != S::TM && t.rows <= S::TM)
    tile_body<WIDE, S>(a, lds, t, tn * T::TN, split);
  else
    tile_body<WIDE, T>(a, lds, t, tn * T::TN, split);
}

template <class T, class S = T>
void tile_launch(const Fp8Args& a, const Fp8Plan& p, hipStream_t s) {
  const dim3 grid((unsigned)(p.tiles_n * p.tiles_m * p.S)), block(64 * T::WAVES);
  if (p.wide)
    hipLaunchKernelGGL((fp8_tile<true, T, S>), grid, block, 0, s, a, (int)p.tiles_n, (int)p.tiles_m);
  else
    hipLaunchKernelGGL((fp8_tile<false, T, S>), grid, block, 0, s, a, (int)p.tiles_n, (int)p.tiles_m);
}

}  // namespace

hipError_t launch_fp8_tile(const Fp8Args& a, const Fp8Plan& p, hipStream_t s) {
  switch (p.kernel) {
    case kFp8Tile32: tile_launch<TileShape<1, 2, 1, 1, 3>>(a, p, s); break;
    case kFp8Tile64: tile_launch<TileShape<2, 4, 1, 1, 3>>(a, p, s); break;
    case kFp8Tile128: tile_launch<TileShape<2, 2, 2, 2, 2>, TileShape<1, 4, 2, 1, 3>>(a, p, s); break;
    default: tile_launch<TileShape<2, 4, 4, 2, 2>, TileShape<1, 8, 4, 1, 3>>(a, p, s); break;
  }
  return hipGetLastError();
}

}  // namespace hxq
