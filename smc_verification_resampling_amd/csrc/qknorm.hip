// qknorm.hip - query/key norms, rotation and the write into the paged cache (gfx950).
//
// One pass over the new tokens' heads.  A head of D elements belongs to a group of lanes
// of 8 elements (16 bytes) each: the sum of squares is a butterfly over the group, and the
// rotation's partner elements lie in the same lane (interleaved pairs) or in the lane
// rot_dim/16 away (pairs i, i + rot_dim/2), so nothing goes through LDS.  Bound by memory:
// each head is read once and written once; the cos/sin row of a token is read by each of its
// heads, from the caches.
#include "../../include/smcsd.h"
#include "device.hpp"
#include "half.hpp"
#include "internal.hpp"

namespace smcsd {

namespace {

constexpr int kRopeBlock = 256;

// LPH: lanes of a head, the power of two that covers D/8 (8 for D <= 64, 16, 32 for D > 128).
template <int DT, int LPH>
__global__ __launch_bounds__(kRopeBlock) void k_qk_norm_rope(QkNormRopeArgs a, int64_t rows, int64_t blocks) {
  const int l = threadIdx.x % LPH;
  const int heads = a.Hq + 2 * a.Hkv;
  const int D = a.D, half = a.rot_dim / 2;
  const bool in = 8 * l < D;
  for (int64_t blk = blockIdx.x; blk < blocks; blk += gridDim.x) {
    const int64_t row = blk * (kRopeBlock / LPH) + threadIdx.x / LPH;
    if (row >= rows) continue;  // a whole group of lanes leaves together
    const int64_t t = row / heads;
    const int h = (int)(row - t * heads);
    const int s = (int)(t / a.R), j = (int)(t - (int64_t)s * a.R);
    if (a.num_nodes && j >= a.num_nodes[s]) continue;
    const int64_t at = (int64_t)a.ctx_lens[s] + j;
    const int64_t pos = a.positions ? a.positions[t] : at;
    int32_t page = -1;
    if (at >= 0 && at < (int64_t)a.cache.M_cap * a.cache.block_size)
      page = a.cache.tables[(int64_t)s * a.cache.M_cap + at / a.cache.block_size];
    if (page < 0 || page >= a.cache.P || (half > 0 && (pos < 0 || pos >= a.max_pos))) {
      if (h == 0 && l == 0) atomicOr(a.status, SMCSD_ST_BAD_INPUT);
      continue;
    }
    const int hk = h - a.Hq, hv = hk - a.Hkv;
    const uint16_t *src = hk < 0 ? a.q + t * a.q_stride + (int64_t)h * D
                          : hv < 0 ? a.k + t * a.k_stride + (int64_t)hk * D
                                   : a.v + t * a.v_stride + (int64_t)hv * D;
    uint16_t *dst;
    if (hk < 0) {
      dst = a.q_out + (t * a.Hq + h) * D;
    } else {
      uint16_t *c = hv < 0 ? a.k_cache : a.v_cache;
      dst = c + page * a.cache.page + (at % a.cache.block_size) * a.cache.token +
            (hv < 0 ? hk : hv) * a.cache.head;
    }
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (in) raw = *reinterpret_cast<const uint4 *>(src + 8 * l);
    const uint16_t *wt = hk < 0 ? a.q_weight : a.k_weight;
    if (hv < 0 && (wt || half > 0)) {
      f32x8 x = widen8<DT>(raw);
      if (wt) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int m = 1; m < LPH; m <<= 1) ss += __shfl_xor(ss, m, LPH);
        const float r = 1.0f / sqrtf(ss / (float)D + a.eps);
        f32x8 w = {};
        if (in) w = widen8<DT>(*reinterpret_cast<const uint4 *>(wt + 8 * l));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
      }
      if (half > 0) {
        const float *cs = a.cos_sin + pos * a.rot_dim;
        if (a.interleaved) {
          if (8 * l < a.rot_dim) {
            const float4 c = *reinterpret_cast<const float4 *>(cs + 4 * l);
            const float4 sn = *reinterpret_cast<const float4 *>(cs + half + 4 * l);
            const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float u = x[2 * i], v = x[2 * i + 1];
              x[2 * i] = fmaf(u, cc[i], -(v * ss[i]));
              x[2 * i + 1] = fmaf(v, cc[i], u * ss[i]);
            }
          }
        } else {
          const int away = half / 8;  // lanes between the halves of a pair
          const bool lo = l < away, rot = l < 2 * away;
          const int other = rot ? (lo ? l + away : l - away) : l;
          f32x8 y;
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = __shfl(x[i], other, LPH);
          if (rot) {
            const int i0 = 8 * (lo ? l : l - away);
            float c[8], sn[8];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              *reinterpret_cast<float4 *>(c + 4 * q) = *reinterpret_cast<const float4 *>(cs + i0 + 4 * q);
              *reinterpret_cast<float4 *>(sn + 4 * q) =
                  *reinterpret_cast<const float4 *>(cs + half + i0 + 4 * q);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], c[i], lo ? -(y[i] * sn[i]) : y[i] * sn[i]);
          }
        }
      }
      raw = narrow8<DT>(x);
    }
    if (in) *reinterpret_cast<uint4 *>(dst + 8 * l) = raw;
  }
}

template <int DT>
void launch_dt(const QkNormRopeArgs &a, hipStream_t stream) {
  const int64_t rows = (int64_t)a.S * a.R * (a.Hq + 2 * a.Hkv);
  const int lph = a.D <= 64 ? 8 : a.D <= 128 ? 16 : 32;
  const int64_t blocks = ceil_div(rows, kRopeBlock / lph);
  const dim3 grid(grid_blocks(blocks, kRopeBlock)), block(kRopeBlock);
  if (lph == 8) hipLaunchKernelGGL((k_qk_norm_rope<DT, 8>), grid, block, 0, stream, a, rows, blocks);
  else if (lph == 16) hipLaunchKernelGGL((k_qk_norm_rope<DT, 16>), grid, block, 0, stream, a, rows, blocks);
  else hipLaunchKernelGGL((k_qk_norm_rope<DT, 32>), grid, block, 0, stream, a, rows, blocks);
}

}  // namespace

hipError_t launch_qk_norm_rope(const QkNormRopeArgs &a, int dtype, hipStream_t stream) {
  if (dtype == SMCSD_DTYPE_BF16) launch_dt<SMCSD_DTYPE_BF16>(a, stream);
  else launch_dt<SMCSD_DTYPE_F16>(a, stream);
  return hipGetLastError();
}

}  // namespace smcsd
