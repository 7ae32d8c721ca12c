// C entry points of the 8-bit path: argument validation and planning on the
// host, then the launches.  Nothing here touches device memory or allocates.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "../../include/hxq.h"
#include "hxq_fp8.h"
#include "hxq_launch.h"

namespace {

using hxq::fp8_padded;
using hxq::fp8_scale_row;

constexpr int64_t kMaxDim = (int64_t)INT32_MAX - 65536;  // room for tile rounding in int32
constexpr int64_t kMaxTiles = (int64_t)1 << 22;           // workgroups of one launch: their threads fit 32 bits
constexpr int64_t kRowsPerLaunch = (int64_t)1 << 22;      // rows of a row operator's launch, likewise
constexpr int64_t kMaxExperts = 65535;

bool misaligned(const void* p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) % a) != 0; }
bool bad_dim(int64_t d) { return d < 0 || d > kMaxDim; }
bool float_dtype(int d) { return d == HXQ_F32 || d == HXQ_BF16; }
uintptr_t size_of(int d) { return d == HXQ_F32 ? 4 : d == HXQ_BF16 ? 2 : 16; }  // e4m3: the alignment it needs
int status_of(hipError_t e) { return e == hipSuccess ? HXQ_OK : HXQ_ERR_HIP; }
int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }
template <typename T>
T* at(T* p, int64_t bytes) {
  return p ? reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(p) + bytes) : nullptr;
}
const void* at(const void* p, int64_t bytes) { return p ? static_cast<const char*>(p) + bytes : nullptr; }
void* at(void* p, int64_t bytes) { return p ? static_cast<char*>(p) + bytes : nullptr; }

// Rows of x and outputs of a workgroup's tile, by kernel.
constexpr int64_t kTileRows[] = {16, 32, 64, 128, 256};
constexpr int64_t kTileOutputs[] = {16, 64, 128, 128, 256};

// Which kernel runs a product over `M` rows of y (of `E` experts; `gather`:
// rows of x by index), and how its sum over k is split.
hxq::Fp8Plan plan(bool y_bf16, int64_t Mx, int64_t M, int64_t N, int64_t K, int64_t E, bool gather) {
  hxq::Fp8Plan p = {};
  const int64_t Kp = fp8_padded(K), blocks = Kp / 128, cus = hxq::device_cu_count();
  const int64_t each = (M + E - 1) / E;  // rows of an expert, if they were even
  p.wide = !y_bf16;
  auto tiles_m = [&](int k) {
    const int64_t tm = kTileRows[k];
    return E > 1 ? M / tm + std::min(E, M) : (M + tm - 1) / tm;
  };
  auto tiles = [&](int k) { return tiles_m(k) * ((N + kTileOutputs[k] - 1) / kTileOutputs[k]); };
  // workgroups that share a tile's sum: to fill the CUs, each with at least 12 blocks
  auto splits = [&](int k) {
    if (k > hxq::kFp8Tile64) return (int64_t)1;
    return std::max<int64_t>(1, std::min(cus / std::max<int64_t>(1, tiles(k)), blocks / 12));
  };
  auto fills = [&](int k) { return 10 * tiles(k) * splits(k) >= 6 * cus; };
  const bool near32 = K > 0 && (gather ? Mx : 256) * Kp < ((int64_t)1 << 32) && Kp < ((int64_t)1 << 24);
  if (!near32 || each <= (E > 1 ? 1 : 8) || (each <= 128 && tiles(hxq::kFp8Skinny) <= 32 * cus / std::max<int64_t>(1, blocks)))
    p.kernel = hxq::kFp8Skinny;
  else if (each >= 192 && fills(hxq::kFp8Tile256))
    p.kernel = hxq::kFp8Tile256;
  else if (p.wide && each >= 96 && fills(hxq::kFp8Tile128))
    p.kernel = hxq::kFp8Tile128;
  else if (each >= (E > 1 ? 6 : 33) && fills(hxq::kFp8Tile64))
    p.kernel = hxq::kFp8Tile64;
  else
    p.kernel = hxq::kFp8Tile32;
  const bool skinny = p.kernel == hxq::kFp8Skinny;
  p.tiles_n = (N + kTileOutputs[p.kernel] - 1) / kTileOutputs[p.kernel];
  p.tiles_m = tiles_m(p.kernel);
  const int64_t wgs = p.tiles_n * p.tiles_m;
  p.S = (int)splits(p.kernel);
  if (skinny) {
    // Few workgroups share the sum between more waves (2048 x 2048 at one row: 4.3 us in 8 waves, 6.3 in two
    // splits of 4 waves, whose parts take a second launch), and between workgroups as well where it is long
    // (2048 x 11008: 10.8 us in splits, 13.4 without; 2048 x 4096: 7.0, 5.7).
    p.S = wgs < cus && blocks >= 48 ? (int)std::min<int64_t>((2 * cus + wgs - 1) / wgs, blocks / 16) : 1;
    p.waves = wgs >= 2 * cus || blocks < 16 ? 4 : p.S > 1 || wgs >= cus || blocks < 32 ? 8 : 16;
    // many workgroups: two blocks of each wave in flight (22016 x 2048: 10.8 against 11.5 us), else one, which
    // leaves room for more waves (8512 x 2048: 6.4 against 7.0); at four to a CU (16384 x 2048) 10.7 us either way
    p.depth = wgs > 4 * cus ? 2 : 1;
  }
  p.kbs = (int)((blocks + p.S - 1) / p.S);
  if (p.S > 1 && !skinny) p.kbs = (p.kbs + 3) / 4 * 4;  // whole words of scales
  if (p.kbs > 0) p.S = (int)((blocks + p.kbs - 1) / p.kbs);
  if (p.S < 1) p.S = 1;
  // A small x is converted by every workgroup for itself instead of in a launch before: through 22016 x 2048
  // 11.4 against 13.5 us for one row, 13.9 against 14.6 for three, 15.3 against 15.0 for four; one row through
  // 2048 x 11008 (split) 10.8 against 12.3.  At most 16 rows of the split's bytes lie in LDS.
  p.converts = skinny && K > 0 && Mx * p.kbs * 128 <= 6144 && std::min<int64_t>(M, 16) * p.kbs * 129 <= 40 * 1024;
  p.ok = p.tiles_n <= kMaxTiles && p.tiles_m <= kMaxTiles && p.tiles_n * p.tiles_m * p.S <= kMaxTiles;
  p.part_bytes = p.ok && p.S > 1 ? p.S * M * N * 4 : 0;
  return p;
}

// A product as it is launched: rows [0, cut) of y by `p`, the rest by `rest`
// (cut == M: all by `p`).  A few tiles more than whole rounds of the largest
// tiles over the CUs would take a round of their own; where they are at most
// half a round, their rows go to smaller tiles in a second launch (2048 x
// 11008 at 25600 rows, 800 tiles on 256 CUs: 536 -> 471 us).
struct Plans {
  hxq::Fp8Plan p, rest;
  int64_t cut;
  bool ok;
  int64_t xq, xs, part, bytes;  // offsets in the workspace, its size
};
Plans plans(int x_dtype, int y_dtype, int64_t Mx, int64_t M, int64_t N, int64_t K, int64_t E, bool experts, bool gather) {
  const bool y_bf16 = y_dtype == HXQ_BF16;
  Plans l = {};
  l.p = plan(y_bf16, Mx, M, N, K, E, gather);
  l.cut = M;
  if (!experts && l.p.ok && l.p.kernel == hxq::kFp8Tile256) {
    const int64_t cus = hxq::device_cu_count(), tiles = l.p.tiles_m * l.p.tiles_n, over = tiles % cus;
    const int64_t main_m = tiles / cus * cus / l.p.tiles_n;
    if (main_m > 0 && over > 0 && 2 * over <= cus) {
      const hxq::Fp8Plan rest = plan(y_bf16, M - main_m * 256, M - main_m * 256, N, K, 1, false);
      if (rest.ok && rest.kernel != hxq::kFp8Tile256) {
        l.cut = main_m * 256;
        l.p.tiles_m = main_m;
        l.rest = rest;
      }
    }
  }
  l.ok = l.p.ok;
  const bool converts = l.p.converts && l.cut == M;
  if (x_dtype != HXQ_E4M3 && !converts) {
    l.xs = round256(Mx * fp8_padded(K));
    l.part = l.xs + round256(Mx * fp8_scale_row(K));
  }
  l.bytes = l.part + std::max(l.p.part_bytes, l.rest.part_bytes);
  return l;
}

hipError_t launch(hxq::Fp8Args a, const hxq::Fp8Plan& p, hipStream_t stream) {
  a.S = p.S;
  a.kbs = p.kbs;
  const hipError_t e = p.kernel == hxq::kFp8Skinny ? hxq::launch_fp8_skinny(a, p, stream) : hxq::launch_fp8_tile(a, p, stream);
  return e == hipSuccess && p.S > 1 ? hxq::launch_fp8_sum(a, stream) : e;
}

hipError_t quant_rows(const void* x, int x_dtype, uint8_t* q, uint8_t* scales, int64_t M, int64_t K,
                      hipStream_t stream) {
  // groups of a launch: 16 to a workgroup
  const int64_t step = std::max<int64_t>(1, kMaxTiles * 16 / fp8_scale_row(K));
  const int64_t sx = x_dtype == HXQ_F32 ? 4 : 2;
  for (int64_t m = 0; m < M; m += step) {
    const hipError_t e =
        hxq::launch_quant_rows(at(x, m * K * sx), x_dtype, at(q, m * fp8_padded(K)), at(scales, m * fp8_scale_row(K)),
                               std::min(step, M - m), (int)K, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// The product, for one layer (offsets NULL, E = 1) or experts.
int product(const void* x, int x_dtype, const uint8_t* x_scales, const int32_t* rows, const int32_t* offsets,
            const uint8_t* wq, const uint8_t* w_scales, const float* bias, void* y, int y_dtype, int64_t Mx,
            int64_t M, int64_t E, int64_t N, int64_t K, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  if ((!float_dtype(x_dtype) && x_dtype != HXQ_E4M3) || !float_dtype(y_dtype)) return HXQ_ERR_DTYPE;
  if (bad_dim(Mx) || bad_dim(M) || bad_dim(N) || bad_dim(K) || E < 1 || E > kMaxExperts || workspace_bytes < 0)
    return HXQ_ERR_SHAPE;
  if (M == 0 || N == 0) return HXQ_OK;
  if (Mx == 0) return HXQ_ERR_SHAPE;
  const Plans l = plans(x_dtype, y_dtype, Mx, M, N, K, E, offsets != nullptr, rows != nullptr);
  if (!l.ok) return HXQ_ERR_SHAPE;
  if (!y) return HXQ_ERR_NULL;
  if (K > 0 && (!x || !wq || !w_scales || (x_dtype == HXQ_E4M3 && !x_scales))) return HXQ_ERR_NULL;
  if (misaligned(x, size_of(x_dtype)) || misaligned(wq, 16) || misaligned(w_scales, 4) || misaligned(x_scales, 4) ||
      misaligned(rows, 4) || misaligned(offsets, 4) || misaligned(bias, 4) || misaligned(y, size_of(y_dtype)) ||
      misaligned(workspace, 16))
    return HXQ_ERR_ALIGN;
  if (l.bytes > 0 && (!workspace || workspace_bytes < l.bytes)) return HXQ_ERR_UNSUPPORTED;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  hxq::Fp8Args a = {};
  a.rows = rows;
  a.offsets = offsets;
  a.w = wq;
  a.ws = w_scales;
  a.bias = bias;
  a.y = y;
  a.y_bf16 = y_dtype == HXQ_BF16;
  a.part = reinterpret_cast<float*>(at(ws, l.part));
  a.Mx = Mx;
  a.M = (int)l.cut;
  a.N = (int)N;
  a.K = (int)K;
  a.Kp = (int)fp8_padded(K);
  a.Gs = (int)fp8_scale_row(K);
  a.E = (int)E;
  a.x_dtype = HXQ_E4M3;
  (void)hipGetLastError();  // start from a clean error state
  if (x_dtype == HXQ_E4M3) {
    a.x = static_cast<const uint8_t*>(x);
    a.xs = x_scales;
  } else if (l.p.converts) {
    a.xf = x;
    a.x_dtype = x_dtype;
  } else if (K > 0) {
    a.x = ws + l.xq;
    a.xs = ws + l.xs;
    if (quant_rows(x, x_dtype, ws + l.xq, ws + l.xs, Mx, K, stream) != hipSuccess) return HXQ_ERR_HIP;
  }
  hipError_t e = launch(a, l.p, stream);
  if (e == hipSuccess && l.cut < M) {
    a.x += l.cut * a.Kp;
    a.xs += l.cut * a.Gs;
    a.y = at(a.y, l.cut * N * (a.y_bf16 ? 2 : 4));
    a.Mx = a.M = (int)(M - l.cut);
    e = launch(a, l.rest, stream);
  }
  return status_of(e);
}

int64_t product_workspace(int x_dtype, int64_t Mx, int64_t M, int64_t E, int64_t N, int64_t K, bool experts) {
  if (!float_dtype(x_dtype) && x_dtype != HXQ_E4M3) return HXQ_ERR_DTYPE;
  if (bad_dim(Mx) || bad_dim(M) || bad_dim(N) || bad_dim(K) || E < 1 || E > kMaxExperts) return HXQ_ERR_SHAPE;
  if (M == 0 || N == 0) return 0;
  if (Mx == 0) return HXQ_ERR_SHAPE;
  // enough for either type of y, with and without a gather
  int64_t bytes = 0;
  for (int i = 0; i < (experts ? 4 : 2); ++i) {
    const Plans l = plans(x_dtype, i & 1 ? HXQ_BF16 : HXQ_F32, Mx, M, N, K, E, experts, i >= 2);
    if (!l.ok) return HXQ_ERR_SHAPE;
    bytes = std::max(bytes, l.bytes);
  }
  return bytes;
}

}  // namespace

extern "C" {

int hxq_quant_fp8(const void* x, int x_dtype, uint8_t* q, uint8_t* scales, int64_t M, int64_t K, hipStream_t stream) {
  if (!float_dtype(x_dtype)) return HXQ_ERR_DTYPE;
  if (bad_dim(M) || bad_dim(K)) return HXQ_ERR_SHAPE;
  if (M == 0 || K == 0) return HXQ_OK;
  if (!x || !q || !scales) return HXQ_ERR_NULL;
  if (misaligned(x, size_of(x_dtype)) || misaligned(q, 16) || misaligned(scales, 4)) return HXQ_ERR_ALIGN;
  (void)hipGetLastError();
  return status_of(quant_rows(x, x_dtype, q, scales, M, K, stream));
}

int hxq_quant_fp8_weight(const void* w, int w_dtype, uint8_t* q, uint8_t* scales, uint8_t* qt, uint8_t* scales_t,
                         int64_t E, int64_t N, int64_t K, hipStream_t stream) {
  if (!float_dtype(w_dtype)) return HXQ_ERR_DTYPE;
  if (bad_dim(N) || bad_dim(K) || E < 1 || E > kMaxExperts) return HXQ_ERR_SHAPE;
  if (N == 0 || K == 0) return HXQ_OK;
  const int64_t blocks = ((N + 127) / 128) * ((K + 127) / 128);
  if (blocks > kMaxTiles * 2 / E) return HXQ_ERR_SHAPE;
  if (!w || !q || !scales || (qt != nullptr) != (scales_t != nullptr)) return HXQ_ERR_NULL;
  if (misaligned(w, size_of(w_dtype)) || misaligned(q, 16) || misaligned(qt, 16) || misaligned(scales, 4) ||
      misaligned(scales_t, 4))
    return HXQ_ERR_ALIGN;
  (void)hipGetLastError();
  return status_of(hxq::launch_quant_weight(w, w_dtype, q, scales, qt, scales_t, E, N, K, stream));
}

int hxq_linear_fwd_fp8(const void* x, int x_dtype, const uint8_t* x_scales, const uint8_t* wq,
                       const uint8_t* w_scales, const float* bias, void* y, int y_dtype, int64_t M, int64_t N,
                       int64_t K, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  return product(x, x_dtype, x_scales, nullptr, nullptr, wq, w_scales, bias, y, y_dtype, M, M, 1, N, K, workspace,
                 workspace_bytes, stream);
}

int64_t hxq_linear_fwd_fp8_workspace(int x_dtype, int64_t M, int64_t N, int64_t K) {
  return product_workspace(x_dtype, M, M, 1, N, K, false);
}

int hxq_linear_fwd_fp8_experts(const void* x, int x_dtype, const uint8_t* x_scales, const int32_t* rows,
                               const int32_t* offsets, const uint8_t* wq, const uint8_t* w_scales, const float* bias,
                               void* y, int y_dtype, int64_t M_x, int64_t M, int64_t E, int64_t N, int64_t K,
                               void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  if (M > 0 && N > 0 && E >= 1 && !offsets) return HXQ_ERR_NULL;
  if (!rows && M_x != M) return HXQ_ERR_SHAPE;
  return product(x, x_dtype, x_scales, rows, offsets, wq, w_scales, bias, y, y_dtype, M_x, M, E, N, K, workspace,
                 workspace_bytes, stream);
}

int64_t hxq_linear_fwd_fp8_experts_workspace(int x_dtype, int64_t M_x, int64_t M, int64_t E, int64_t N, int64_t K) {
  return product_workspace(x_dtype, M_x, M, E, N, K, true);
}

int hxq_rms_norm(const void* x, int x_dtype, const void* residual, int residual_dtype, const float* weight, float eps,
                 void* residual_out, void* out, int out_dtype, uint8_t* scales, float* rstd, int64_t M, int64_t K,
                 hipStream_t stream) {
  if (!float_dtype(x_dtype) || (residual && !float_dtype(residual_dtype)) ||
      (!float_dtype(out_dtype) && out_dtype != HXQ_E4M3))
    return HXQ_ERR_DTYPE;
  if (bad_dim(M) || bad_dim(K)) return HXQ_ERR_SHAPE;
  if (!(eps >= 0.f)) return HXQ_ERR_UNSUPPORTED;
  if (M == 0 || K == 0) return HXQ_OK;
  if (!x || !out || (residual != nullptr) != (residual_out != nullptr) || (out_dtype == HXQ_E4M3 && !scales))
    return HXQ_ERR_NULL;
  const uintptr_t rs = size_of(residual_dtype);
  if (misaligned(x, size_of(x_dtype)) || misaligned(residual, rs) || misaligned(residual_out, rs) ||
      misaligned(weight, 4) || misaligned(out, size_of(out_dtype)) || misaligned(scales, 4) || misaligned(rstd, 4))
    return HXQ_ERR_ALIGN;
  (void)hipGetLastError();
  const int64_t Kp = fp8_padded(K), Gs = fp8_scale_row(K);
  const int64_t sx = x_dtype == HXQ_F32 ? 4 : 2, sr = residual_dtype == HXQ_F32 ? 4 : 2;
  for (int64_t m = 0; m < M; m += kRowsPerLaunch) {
    hxq::NormArgs a = {};
    a.x = at(x, m * K * sx);
    a.residual = at(residual, m * K * sr);
    a.weight = weight;
    a.sum_out = at(residual_out, m * K * sr);
    a.out = at(out, out_dtype == HXQ_E4M3 ? m * Kp : m * K * (out_dtype == HXQ_F32 ? 4 : 2));
    a.scales = out_dtype == HXQ_E4M3 ? at(scales, m * Gs) : nullptr;
    a.rstd = at(rstd, m * 4);
    a.eps = eps;
    a.M = std::min(kRowsPerLaunch, M - m);
    a.K = (int)K;
    a.x_dtype = x_dtype;
    a.res_dtype = residual ? residual_dtype : -1;
    a.out_dtype = out_dtype;
    const hipError_t e = hxq::launch_rms_norm(a, stream);
    if (e != hipSuccess) return HXQ_ERR_HIP;
  }
  return HXQ_OK;
}

int64_t hxq_rms_norm_bwd_workspace(int64_t M, int64_t K) {
  if (bad_dim(M) || bad_dim(K)) return HXQ_ERR_SHAPE;
  return hxq::norm_bwd_parts(M, K) * K * 4;
}

int hxq_rms_norm_bwd(const void* dy, int dy_dtype, const void* h, int h_dtype, const float* weight, const float* rstd,
                     const float* dresidual, float* dx, float* dweight, int64_t M, int64_t K, void* workspace,
                     int64_t workspace_bytes, hipStream_t stream) {
  if (!float_dtype(dy_dtype) || !float_dtype(h_dtype)) return HXQ_ERR_DTYPE;
  if (bad_dim(M) || bad_dim(K) || workspace_bytes < 0) return HXQ_ERR_SHAPE;
  if (K == 0 || (M == 0 && !dweight)) return HXQ_OK;
  if (M > 0 && (!dy || !h || !rstd || !dx)) return HXQ_ERR_NULL;
  if (misaligned(dy, size_of(dy_dtype)) || misaligned(h, size_of(h_dtype)) || misaligned(weight, 4) ||
      misaligned(rstd, 4) || misaligned(dresidual, 4) || misaligned(dx, 4) || misaligned(dweight, 4) ||
      misaligned(workspace, 4))
    return HXQ_ERR_ALIGN;
  if (dweight && M > 0 && (!workspace || workspace_bytes < hxq_rms_norm_bwd_workspace(M, K)))
    return HXQ_ERR_UNSUPPORTED;
  hxq::NormBwdArgs a = {};
  a.dy = dy;
  a.h = h;
  a.weight = weight;
  a.rstd = rstd;
  a.dsum = dresidual;
  a.dx = dx;
  a.dweight = dweight;
  a.part = dweight ? static_cast<float*>(workspace) : nullptr;
  a.M = M;
  a.K = (int)K;
  a.dy_dtype = dy_dtype;
  a.h_dtype = h_dtype;
  (void)hipGetLastError();
  return status_of(hxq::launch_rms_norm_bwd(a, stream));
}

}  // extern "C"
