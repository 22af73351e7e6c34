// qknorm.hip - query/key norms, rotation and the write into the paged cache (gfx950).
//
// A workgroup takes heads of one token, so that the token's place in the cache and its
// position are scalars, looked up while the loads of its heads are already on their way.  A
// head of D elements belongs to a group of lanes of 8 elements (16 bytes) each: the sum of
// squares is a butterfly over the group, and the rotation's partner elements lie in the same
// lane (interleaved pairs) or in the lane rot_dim/16 away (pairs i, i + rot_dim/2), so
// nothing goes through LDS.  Bound by memory: each head is read once and written once; 2560
// tokens of 32 + 2 x 8 heads of 128 (63 MB) take 20.5 us (3.1 TB/s, launch and first loads included),
// 12 tokens of 8 + 2 x 2 heads of 64 take 3.8 us.
#include "../../include/smcsd.h"
#include "device.hpp"
#include "half.hpp"
#include "internal.hpp"

namespace smcsd {

namespace {

constexpr int kRopeBlock = 256;  // most threads of a workgroup

// LPH: lanes of a head, the power of two that covers D/8 (8 for D <= 64, 16, 32 for D > 128).
// A token's heads are cut into `chunks` workgroups.
template <int DT, int LPH>
__global__ __launch_bounds__(kRopeBlock) void k_qk_norm_rope(QkNormRopeArgs a, uint32_t chunks, uint32_t items,
                                                             float inv_D) {
  const int l = threadIdx.x % LPH;
  const int heads = a.Hq + 2 * a.Hkv;
  const int D = a.D, half = a.rot_dim / 2;
  const bool in = 8 * l < D;
  for (uint32_t it = blockIdx.x; it < items; it += gridDim.x) {
    const uint32_t t = it / chunks;
    const int h = (int)(it - t * chunks) * (int)(blockDim.x / LPH) + (int)threadIdx.x / LPH;
    const uint32_t s = t / (uint32_t)a.R;
    const int j = (int)(t - s * a.R);
    const int hk = h - a.Hq, hv = hk - a.Hkv;
    const uint16_t *src = hk < 0 ? a.q + t * a.q_stride + h * D
                          : hv < 0 ? a.k + t * a.k_stride + hk * D
                                   : a.v + t * a.v_stride + hv * D;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (in && h < heads) raw = *reinterpret_cast<const uint4 *>(src + 8 * l);
    // the token's place and position, the same for the whole workgroup
    if (a.num_nodes && j >= a.num_nodes[s]) continue;
    const int64_t at = (int64_t)a.ctx_lens[s] + j;
    const int64_t pos = a.positions ? a.positions[t] : at;
    // the block id and the angles are both on their way before either is looked at
    const bool at_ok = at >= 0 && at < (int64_t)a.cache.M_cap * a.cache.block_size;
    const uint32_t slot = at_ok ? (uint32_t)at / (uint32_t)a.cache.block_size : 0;
    const int32_t page = a.cache.tables[(int64_t)s * a.cache.M_cap + slot];
    const bool pos_ok = pos >= 0 && pos < a.max_pos;
    const bool lo = l < half / 8;  // the lane of a pair's first half, if not interleaved
    const bool rot = a.interleaved ? 8 * l < a.rot_dim : l < a.rot_dim / 8;
    float c[8], sn[8];  // interleaved: of the lane's four pairs
    if (rot && pos_ok) {
      const float *cs = a.cos_sin + pos * a.rot_dim + (a.interleaved ? 4 * l : 8 * (lo ? l : l - half / 8));
      *reinterpret_cast<float4 *>(c) = *reinterpret_cast<const float4 *>(cs);
      *reinterpret_cast<float4 *>(sn) = *reinterpret_cast<const float4 *>(cs + half);
      if (!a.interleaved) {
        *reinterpret_cast<float4 *>(c + 4) = *reinterpret_cast<const float4 *>(cs + 4);
        *reinterpret_cast<float4 *>(sn + 4) = *reinterpret_cast<const float4 *>(cs + half + 4);
      }
    }
    const uint16_t *wt = hk < 0 ? a.q_weight : a.k_weight;
    if (hv < 0 && (wt || half > 0)) {
      f32x8 x = widen8<DT>(raw);
      if (wt) {
        f32x8 w = {};
        if (in) w = widen8<DT>(*reinterpret_cast<const uint4 *>(wt + 8 * l));
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int m = 1; m < LPH; m <<= 1) ss += __shfl_xor(ss, m, LPH);
        const float r = rsqrtf(fmaf(ss, inv_D, a.eps));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
      }
      if (half > 0 && a.interleaved) {
        if (rot) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float u = x[2 * i], v = x[2 * i + 1];
            x[2 * i] = fmaf(u, c[i], -(v * sn[i]));
            x[2 * i + 1] = fmaf(v, c[i], u * sn[i]);
          }
        }
      } else if (half > 0) {
        const int other = rot ? (lo ? l + half / 8 : l - half / 8) : l;
        const float sign = lo ? -1.0f : 1.0f;
        f32x8 y;
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __shfl(x[i], other, LPH);
        if (rot) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], c[i], sign * (y[i] * sn[i]));
        }
      }
      raw = narrow8<DT>(x);
    }
    if (!at_ok || page < 0 || page >= a.cache.P || (half > 0 && !pos_ok)) {
      if (h == 0 && l == 0) atomicOr(a.status, SMCSD_ST_BAD_INPUT);
      continue;
    }
    if (h >= heads) continue;
    const int64_t place = page * a.cache.page +
                          (int64_t)((uint32_t)at - slot * a.cache.block_size) * a.cache.token;
    uint16_t *dst = hk < 0 ? a.q_out + (int64_t)t * a.Hq * D + h * D
                    : hv < 0 ? a.k_cache + place + hk * a.cache.head
                             : a.v_cache + place + hv * a.cache.head;
    if (in) *reinterpret_cast<uint4 *>(dst + 8 * l) = raw;
  }
}

template <int DT>
void launch_dt(const QkNormRopeArgs &a, hipStream_t stream) {
  const int lph = a.D <= 64 ? 8 : a.D <= 128 ? 16 : 32;
  const int64_t lanes = (int64_t)(a.Hq + 2 * a.Hkv) * lph;
  const unsigned threads = (unsigned)std::min<int64_t>(kRopeBlock, ceil_div(lanes, kWave) * kWave);
  const int64_t chunks = ceil_div(lanes, threads), items = (int64_t)a.S * a.R * chunks;
  const dim3 grid(grid_blocks(items, kRopeBlock)), block(threads);
  const float inv = 1.0f / (float)a.D;
  const uint32_t c = (uint32_t)chunks, n = (uint32_t)items;
  if (lph == 8) hipLaunchKernelGGL((k_qk_norm_rope<DT, 8>), grid, block, 0, stream, a, c, n, inv);
  else if (lph == 16) hipLaunchKernelGGL((k_qk_norm_rope<DT, 16>), grid, block, 0, stream, a, c, n, inv);
  else hipLaunchKernelGGL((k_qk_norm_rope<DT, 32>), grid, block, 0, stream, a, c, n, inv);
}

}  // namespace

hipError_t launch_qk_norm_rope(const QkNormRopeArgs &a, int dtype, hipStream_t stream) {
  if (dtype == SMCSD_DTYPE_BF16) launch_dt<SMCSD_DTYPE_BF16>(a, stream);
  else launch_dt<SMCSD_DTYPE_F16>(a, stream);
  return hipGetLastError();
}

}  // namespace smcsd
