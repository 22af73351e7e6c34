// kvappend.hip - packed tokens' norms, rotation and way into pages of 16 or 8 bits (gfx950).
//
// Two kinds of waves in one launch.  A wave of the first kind takes one head's keys or values
// of the tokens that one sequence puts into one block: an 8-bit block has one scale for them,
// so the wave forms its tokens' values (in registers, up to kHold rounds of them; those of
// longer blocks are formed twice), their largest magnitude, the scale, and only then the
// rounded elements.  Nothing goes through LDS and no wave waits for another.  A wave of the
// second kind takes the queries of one token, all heads, with one look at its position and
// angles.  A head of D elements belongs to a group of lanes of 8 elements each, as in
// k_qk_norm_rope: the sum of squares is a butterfly over the group.
// Blocks of all sequences are numbered with room to spare: sequence s's begin at
// floor(cu[s] / block_size) + 2 s, since its n tokens touch at most floor(n / block_size) + 2.
#include "../../include/smcsd.h"
#include "device.hpp"
#include "fp8.hpp"
#include "half.hpp"
#include "internal.hpp"
#include "packed.hpp"

namespace smcsd {

namespace {

constexpr int kAppendBlock = 256;
constexpr int kAppendWaves = kAppendBlock / kWave;
constexpr int kHold = 4;  // rounds of tokens whose values a wave keeps: 16 tokens of heads of 128

// A lane's eight elements of a head: the norm over the head's LPH lanes (no norm where `weight`
// is null) and the rotation by the angles at `angles` (null: none; read where `known`).
template <int DT, int LPH>
__device__ __forceinline__ f32x8 norm_rotate(f32x8 x, const uint16_t *weight, const float *angles, bool known,
                                             const KvAppendArgs &a, float inv_D) {
  const int l = threadIdx.x % LPH, half = a.rot_dim / 2;
  const bool lo = l < half / 8;  // the lane of a pair's first half, if not interleaved
  const bool rot = a.interleaved ? 8 * l < a.rot_dim : l < a.rot_dim / 8;
  float c[8] = {}, sn[8] = {};  // interleaved: of the lane's four pairs
  if (angles && rot && known) {
    const float *cs = angles + (a.interleaved ? 4 * l : 8 * (lo ? l : l - half / 8));
    *reinterpret_cast<float4 *>(c) = *reinterpret_cast<const float4 *>(cs);
    *reinterpret_cast<float4 *>(sn) = *reinterpret_cast<const float4 *>(cs + half);
    if (!a.interleaved) {
      *reinterpret_cast<float4 *>(c + 4) = *reinterpret_cast<const float4 *>(cs + 4);
      *reinterpret_cast<float4 *>(sn + 4) = *reinterpret_cast<const float4 *>(cs + half + 4);
    }
  }
  if (weight) {
    f32x8 w = {};
    if (8 * l < a.D) w = widen8<DT>(*reinterpret_cast<const uint4 *>(weight + 8 * l));
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int m = 1; m < LPH; m <<= 1) ss += __shfl_xor(ss, m, LPH);
    const float r = rsqrtf(fmaf(ss, inv_D, a.eps));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
  }
  if (angles && a.interleaved) {
    if (rot) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float u = x[2 * i], v = x[2 * i + 1];
        x[2 * i] = fmaf(u, c[i], -(v * sn[i]));
        x[2 * i + 1] = fmaf(v, c[i], u * sn[i]);
      }
    }
  } else if (angles) {
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
  return x;
}

// One head's keys or values of the tokens that sequence s puts into one block.
template <int DT, int LPH, bool E4>
__device__ __forceinline__ void append_block(const KvAppendArgs &a, int64_t item, int which, int h, float inv_D) {
  constexpr int TW = kWave / LPH;  // tokens of a round
  const int lane = threadIdx.x % kWave, l = lane % LPH, sub = lane / LPH;
  const int bs = a.cache.block_size;
  auto first = [&](int s) { return (int64_t)(held_cu(a.cu, s, a.T) / bs) + 2 * (int64_t)s; };
  const int s = find_sequence(a.S, item, first);
  const int64_t j = item - first(s);
  const int t0 = a.cu[s], t1 = a.cu[s + 1], ctx = a.ctx_lens ? a.ctx_lens[s] : 0;
  if (t0 < 0 || t1 <= t0 || t1 > a.T || j < 0) return;
  if (ctx < 0) {
    if (lane == 0) atomicOr(a.status, SMCSD_ST_BAD_INPUT);
    return;
  }
  const int64_t slot = ctx / bs + j;
  const int64_t p0 = max((int64_t)ctx, slot * bs), p1 = min((int64_t)ctx + (t1 - t0), (slot + 1) * bs);
  if (p0 >= p1) return;
  const int32_t page = slot < a.cache.M_cap ? a.cache.tables[(int64_t)s * a.cache.M_cap + slot] : -1;
  if (page < 0 || page >= a.cache.P) {
    if (lane == 0) atomicOr(a.status, SMCSD_ST_BAD_INPUT);
    return;
  }
  const int count = (int)(p1 - p0), held = (int)(p0 - slot * bs);  // new tokens; older ones of the block
  const int first_t = t0 + (int)(p0 - ctx);
  const uint16_t *src = which ? a.v : a.k;
  const int64_t stride = which ? a.v_stride : a.k_stride;
  src += (int64_t)h * a.D + 8 * l;
  const bool in = 8 * l < a.D;
  const uint16_t *weight = which ? nullptr : a.k_weight;
  const bool turn = !which && a.rot_dim > 0;
  const int64_t place = page * a.cache.page + held * a.cache.token + h * a.cache.head + 8 * l;
  uint8_t *const dst8 = static_cast<uint8_t *>(which ? a.v_cache : a.k_cache) + place;
  uint16_t *const dst16 = static_cast<uint16_t *>(which ? a.v_cache : a.k_cache) + place;

  auto load = [&](int i) {  // token i of the block's new ones, its lanes' part (0 past the last)
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (in && i < count) raw = *reinterpret_cast<const uint4 *>(src + (first_t + i) * stride);
    return raw;
  };
  bool any = false;
  // whether token i may be written, and its values
  auto form = [&](int i, uint4 raw, bool &ok, f32x8 &x) {
    ok = i < count;
    const float *angles = nullptr;
    if (a.rot_dim > 0) {
      const int64_t pos = !ok ? -1 : a.positions ? a.positions[first_t + i] : p0 + i;
      const bool good = pos >= 0 && pos < a.max_pos;
      if (ok && !good && l == 0) atomicOr(a.status, SMCSD_ST_BAD_INPUT);
      ok &= good;
      angles = a.cos_sin + (good ? pos * a.rot_dim : 0);
    }
    x = widen8<DT>(raw);
    if (weight || turn) x = norm_rotate<DT, LPH>(x, weight, turn ? angles : nullptr, ok, a, inv_D);
    any |= ok;
    ok &= in;
  };
  if (!E4) {
    for (int i0 = 0; i0 < count; i0 += TW * kHold) {
      uint4 raw[kHold];
#pragma unroll
      for (int u = 0; u < kHold; ++u) raw[u] = load(i0 + u * TW + sub);
#pragma unroll
      for (int u = 0; u < kHold; ++u) {
        const int i = i0 + u * TW + sub;
        if (i0 + u * TW >= count) break;
        bool ok;
        f32x8 x;
        form(i, raw[u], ok, x);
        if (weight || turn) raw[u] = narrow8<DT>(x);
        if (ok) *reinterpret_cast<uint4 *>(dst16 + i * a.cache.token) = raw[u];
      }
    }
    return;
  }
  float top = 0.0f;
  f32x8 x[kHold];
  bool ok[kHold];
  auto most = [&](const f32x8 &y, bool good) {
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, good && fabsf(y[i]) < INFINITY ? fabsf(y[i]) : 0.0f);
  };
  {
    uint4 raw[kHold];
#pragma unroll
    for (int u = 0; u < kHold; ++u) raw[u] = load(u * TW + sub);
#pragma unroll
    for (int u = 0; u < kHold; ++u) {
      ok[u] = false;
      if (u * TW < count) {
        form(u * TW + sub, raw[u], ok[u], x[u]);
        most(x[u], ok[u]);
      }
    }
  }
  for (int i0 = kHold * TW; i0 < count; i0 += TW) {
    bool good;
    f32x8 y;
    form(i0 + sub, load(i0 + sub), good, y);
    most(y, good);
  }
  if (!__any(any)) return;
  top = wave_max_f32(top);
  uint8_t *const code = (which ? a.v_scales : a.k_scales) + (int64_t)page * a.Hkv + h;
  int now = code_for(top);
  if (held > 0) {
    const int was = *code;
    now = max(now, was);
    if (now != was)  // the block's older tokens follow
      for (int i = sub; i < held; i += TW) {
        uint2 *at = reinterpret_cast<uint2 *>(dst8 + (i - held) * a.cache.token);
        if (!in) continue;
        f32x8 y = widen8_e4m3(*at);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = ldexpf(y[e], was - now);
        *at = narrow8_e4m3(y);
      }
  }
  auto store = [&](int i, f32x8 y) {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = ldexpf(y[e], 127 - now);
    *reinterpret_cast<uint2 *>(dst8 + i * a.cache.token) = narrow8_e4m3(y);
  };
#pragma unroll
  for (int u = 0; u < kHold; ++u)
    if (ok[u]) store(u * TW + sub, x[u]);
  for (int i0 = kHold * TW; i0 < count; i0 += TW) {
    bool good;
    f32x8 y;
    form(i0 + sub, load(i0 + sub), good, y);
    if (good) store(i0 + sub, y);
  }
  if (lane == 0) *code = (uint8_t)now;
}

// One token's queries.
template <int DT, int LPH>
__device__ __forceinline__ void append_queries(const KvAppendArgs &a, int t, float inv_D) {
  constexpr int HW = kWave / LPH;  // heads of a round
  const int lane = threadIdx.x % kWave, l = lane % LPH, sub = lane / LPH;
  const int s = find_sequence(a.S, t, [&](int i) { return (int64_t)held_cu(a.cu, i, a.T); });
  const int t0 = a.cu[s], t1 = a.cu[s + 1], ctx = a.ctx_lens ? a.ctx_lens[s] : 0;
  if (t0 < 0 || t1 > a.T || t < t0 || t >= t1) return;
  const float *angles = nullptr;
  bool good = ctx >= 0;
  if (a.rot_dim > 0) {
    const int64_t pos = a.positions ? a.positions[t] : (int64_t)ctx + (t - t0);
    good &= pos >= 0 && pos < a.max_pos;
    angles = a.cos_sin + pos * a.rot_dim;
  }
  if (!good) {
    if (lane == 0) atomicOr(a.status, SMCSD_ST_BAD_INPUT);
    return;
  }
  const bool in = 8 * l < a.D;
  const uint16_t *src = a.q + t * a.q_stride + 8 * l;
  uint16_t *dst = a.q_out + (int64_t)t * a.Hq * a.D + 8 * l;
  constexpr int kHeads = 4;  // rounds of heads in flight
  for (int h0 = 0; h0 < a.Hq; h0 += HW * kHeads) {
    uint4 raw[kHeads];
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
      const int h = h0 + u * HW + sub;
      raw[u] = make_uint4(0, 0, 0, 0);
      if (in && h < a.Hq) raw[u] = *reinterpret_cast<const uint4 *>(src + h * a.D);
    }
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
      const int h = h0 + u * HW + sub;
      if (a.q_weight || angles) raw[u] = narrow8<DT>(norm_rotate<DT, LPH>(widen8<DT>(raw[u]), a.q_weight, angles, true, a, inv_D));
      if (in && h < a.Hq) *reinterpret_cast<uint4 *>(dst + h * a.D) = raw[u];
    }
  }
}

// LPH: lanes of a head, the power of two that covers D/8 (8 for D <= 64, 16, 32 for D > 128).
// The first `groups` items are four waves of blocks' heads each, the others four tokens' queries.
template <int DT, int LPH, bool E4>
__global__ __launch_bounds__(kAppendBlock) void k_kv_append(KvAppendArgs a, int64_t groups, int64_t items, float inv_D) {
  if (!lengths_in_order(a.cu, a.S, a.T)) atomicOr(a.status, SMCSD_ST_BAD_INPUT);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    if (it < groups) {
      const int64_t w = it * kAppendWaves + wave, block = w / (2 * a.Hkv);
      const int hw = (int)(w - block * 2 * a.Hkv);
      append_block<DT, LPH, E4>(a, block, hw >= a.Hkv, hw >= a.Hkv ? hw - a.Hkv : hw, inv_D);
    } else {
      const int64_t t = (it - groups) * kAppendWaves + wave;
      if (t < a.T) append_queries<DT, LPH>(a, (int)t, inv_D);
    }
  }
}

template <int DT, bool E4>
void launch_dt(const KvAppendArgs &a, hipStream_t stream) {
  const int64_t blocks = a.T / a.cache.block_size + 2 * (int64_t)a.S;
  const int64_t groups = ceil_div(blocks * 2 * a.Hkv, kAppendWaves);
  const int64_t items = groups + (a.q ? ceil_div(a.T, kAppendWaves) : 0);
  const dim3 grid(grid_blocks(items, kAppendBlock)), block(kAppendBlock);
  const float inv = 1.0f / (float)a.D;
  if (a.D <= 64) hipLaunchKernelGGL((k_kv_append<DT, 8, E4>), grid, block, 0, stream, a, groups, items, inv);
  else if (a.D <= 128) hipLaunchKernelGGL((k_kv_append<DT, 16, E4>), grid, block, 0, stream, a, groups, items, inv);
  else hipLaunchKernelGGL((k_kv_append<DT, 32, E4>), grid, block, 0, stream, a, groups, items, inv);
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs &a, int dtype, bool e4m3, hipStream_t stream) {
  if (dtype == SMCSD_DTYPE_BF16) {
    if (e4m3) launch_dt<SMCSD_DTYPE_BF16, true>(a, stream);
    else launch_dt<SMCSD_DTYPE_BF16, false>(a, stream);
  } else {
    if (e4m3) launch_dt<SMCSD_DTYPE_F16, true>(a, stream);
    else launch_dt<SMCSD_DTYPE_F16, false>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace smcsd
