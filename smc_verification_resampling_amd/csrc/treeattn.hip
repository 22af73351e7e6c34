// treeattn.hip - attention of drafted trees over the paged cache (gfx950).
#include "../../include/smcsd.h"
#include "device.hpp"
#include "half.hpp"
#include "internal.hpp"

namespace smcsd {

namespace {

constexpr int kAttnBlock = 256;

// The nodes that node i of sequence s sees, as bits.
__device__ __forceinline__ uint64_t node_bits(const TreeAttnArgs &a, int s, int i, int nodes) {
  const uint64_t all = nodes >= 64 ? ~0ull : (1ull << nodes) - 1;
  const uint64_t m = a.tree_mask ? a.tree_mask[(int64_t)s * a.R + i] : (i >= 63 ? ~0ull : (2ull << i) - 1);
  return m & all;
}

// One wave per query row (sequence, node, head): 64 tokens at a time, one per lane for the
// scores, then D elements over the lanes for the values.
template <int DT>
__global__ __launch_bounds__(kAttnBlock) void k_attn_row(TreeAttnArgs a, int64_t rows) {
  typedef typename Half<DT>::T T;
  __shared__ float sq[kAttnBlock / kWave][256];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  for (int64_t r0 = (int64_t)blockIdx.x * (kAttnBlock / kWave); r0 < rows;
       r0 += (int64_t)gridDim.x * (kAttnBlock / kWave)) {
    const int64_t r = r0 + wave;
    if (r >= rows) continue;
    const int64_t t = r / a.Hq;
    const int hq = (int)(r - t * a.Hq), s = (int)(t / a.R), i = (int)(t - (int64_t)s * a.R);
    const int hk = hq / (a.Hq / a.Hkv);
    int nodes = a.R;
    bool bad = false;
    if (a.num_nodes) {
      nodes = a.num_nodes[s];
      bad = nodes < 0 || nodes > a.R;
      nodes = max(0, min(nodes, a.R));
    }
    int64_t ctx = a.ctx_lens[s];
    const bool none = ctx < 0 || ctx + nodes > (int64_t)a.cache.M_cap * a.cache.block_size;
    if (none) ctx = 0;
    if (lane == 0 && (none || bad)) atomicOr(a.status, SMCSD_ST_BAD_INPUT);
    if (i >= nodes) continue;
    const uint64_t bits = node_bits(a, s, i, nodes);
    const int len = none ? 0 : (int)ctx + nodes;
    const T *q = reinterpret_cast<const T *>(a.q) + t * a.q_stride + (int64_t)hq * a.D;
    for (int d = lane; d < a.D; d += kWave) sq[wave][d] = (float)q[d];
    __builtin_amdgcn_wave_barrier();
    float m = kNegInf, l = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int p0 = 0; p0 < len; p0 += kWave) {
      const int p = p0 + lane;
      bool see = p < len && (p < ctx || ((bits >> (p - ctx)) & 1));
      int64_t off = 0;
      if (see) {
        const int32_t page = a.cache.tables[(int64_t)s * a.cache.M_cap + p / a.cache.block_size];
        see = page >= 0 && page < a.cache.P;
        if (!see) atomicOr(a.status, SMCSD_ST_BAD_INPUT);
        off = page * a.cache.page + (p % a.cache.block_size) * a.cache.token + hk * a.cache.head;
      }
      float z = kNegInf;
      if (see) {
        const uint16_t *k = a.k_cache + off;
        float sum = 0.0f;
        for (int d = 0; d < a.D; d += 8) {
          const f32x8 x = widen8<DT>(*reinterpret_cast<const uint4 *>(k + d));
#pragma unroll
          for (int c = 0; c < 8; ++c) sum = fmaf(x[c], sq[wave][d + c], sum);
        }
        z = sum * a.scale;
      }
      float top = z;
#pragma unroll
      for (int x = 1; x < kWave; x <<= 1) top = fmaxf(top, __shfl_xor(top, x, kWave));
      const float mn = fmaxf(m, top);
      if (mn == kNegInf && !__any(see)) continue;
      const float f = m == kNegInf ? 0.0f : expf(m - mn);
      const float pr = see ? expf(z - mn) : 0.0f;
      m = mn;
      l = l * f + wave_sum_f32(pr);
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c] *= f;
      const uint64_t seen = __ballot(see);
      for (int x = 0; x < kWave; ++x) {
        if (!((seen >> x) & 1)) continue;
        const float w = __shfl(pr, x, kWave);
        const int64_t o = __shfl((long long)off, x, kWave);
        const T *v = reinterpret_cast<const T *>(a.v_cache) + o;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (lane + c * kWave < a.D) acc[c] = fmaf(w, (float)v[lane + c * kWave], acc[c]);
      }
    }
    T *out = reinterpret_cast<T *>(a.out) + r * a.D;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (lane + c * kWave < a.D) out[lane + c * kWave] = (T)(l == 0.0f ? 0.0f : acc[c] / l);
    if (a.lse && lane == 0) a.lse[r] = l == 0.0f ? kNegInf : m + logf(l);
  }
}

}  // namespace

size_t tree_attn_ws_bytes(int64_t S, int R, int64_t HqD, int64_t Hkv) {
  return align256(sizeof(float));
}

hipError_t launch_tree_attn(const TreeAttnArgs &a, int dtype, hipStream_t stream) {
  const int64_t rows = (int64_t)a.B * a.N * a.R * a.Hq;
  const dim3 grid(grid_blocks(ceil_div(rows, kAttnBlock / kWave), kAttnBlock)), block(kAttnBlock);
  if (dtype == SMCSD_DTYPE_BF16)
    hipLaunchKernelGGL(k_attn_row<SMCSD_DTYPE_BF16>, grid, block, 0, stream, a, rows);
  else
    hipLaunchKernelGGL(k_attn_row<SMCSD_DTYPE_F16>, grid, block, 0, stream, a, rows);
  return hipGetLastError();
}

}  // namespace smcsd
