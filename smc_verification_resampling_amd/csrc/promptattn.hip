// promptattn.hip - causal attention of packed prompts over the paged cache (gfx950).
//
// The query rows of one key/value head of a sequence - its tokens x Hq/Hkv heads, a token's
// heads side by side - are cut into tiles of 4 waves x RT x 32 rows, each workgroup's going
// through the keys that the tile's last token sees.  Products are formed transposed, as in the
// tree attention: S^T = K Q^T, so that a lane holds one query row and 16 of a step's 32 keys,
// and O^T = V^T P^T with the probabilities straight from the registers.  A wave's RT row tiles
// share each read of a key or value from LDS.
// Keys and values come through registers: the next tile's loads are on their way while a tile
// is computed, and 8-bit pages are widened between the two.
#include <cmath>
#include <type_traits>

#include "../../include/smcsd.h"
#include "device.hpp"
#include "fp8.hpp"
#include "half.hpp"
#include "internal.hpp"
#include "packed.hpp"

namespace smcsd {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

template <int DT> struct Mma;
template <> struct Mma<SMCSD_DTYPE_BF16> {
  typedef Half<SMCSD_DTYPE_BF16>::V8 V8;
  __device__ __forceinline__ static f32x16 run(V8 a, V8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};
template <> struct Mma<SMCSD_DTYPE_F16> {
  typedef Half<SMCSD_DTYPE_F16>::V8 V8;
  __device__ __forceinline__ static f32x16 run(V8 a, V8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
};

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;
constexpr int kRowsWave = 32;
constexpr int KT = 64;       // keys of a tile in LDS
constexpr float kLag = 8.0f; // a running maximum may fall behind by a factor of 2^8
constexpr int kItems = 1024; // workgroups that the splits of a launch aim at

inline int row_tiles(int D) { return D <= 128 ? 2 : 1; }
inline int tile_rows(int D) { return kWaves * kRowsWave * row_tiles(D); }

// n / d for 0 <= n < 2^31 (see treeattn.hip).
struct FastDiv {
  uint32_t d, mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f{d, 0, 0};
  if (d < 2) return f;
  int s = 0;
  while ((1ull << s) < d) ++s;
  f.mul = (uint32_t)(((1ull << (31 + s)) + d - 1) / d);
  f.shift = s - 1;
  return f;
}
__device__ __forceinline__ uint32_t div_by(const FastDiv &f, uint32_t n) {
  return f.d < 2 ? n : __umulhi(n, f.mul) >> f.shift;
}

struct Plan {
  FastDiv page, group;
  int tiles, splits;  // row tiles of all sequences, with room to spare
  float *ml, *acc;    // parts: [splits][T * Hq] (max, sum) pairs, [splits][T * Hq][D]
  float c;            // |scale| * log2(e)
  int negate;
};

// Row tiles of all sequences are numbered with room to spare: sequence s's begin at
// floor(cu[s] * G / M) + s.
__device__ __forceinline__ int64_t first_tile(const PromptAttnArgs &a, int s, int M) {
  return (int64_t)held_cu(a.cu, s, a.T) * (a.Hq / a.Hkv) / M + s;
}

__device__ __forceinline__ float2 both_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return make_float2(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_halves(float x) {
  const float2 h = both_halves(x);
  return h.x + h.y;
}
__device__ __forceinline__ float max_halves(float x) {
  const float2 h = both_halves(x);
  return fmaxf(h.x, h.y);
}

// A row's 16-byte chunks are stored permuted, as in the tree attention's tiles.
template <int CH>
__device__ __forceinline__ int place_of(int r) {
  return CH < 16 ? ((r & 2) << 1) | ((r >> 2) & 3) : ((r & 3) << 2) | ((r >> 2) & 3);
}

__device__ const uint4 kNothing = {0, 0, 0, 0};  // loaded where there is nothing to load

template <class T>
__device__ __forceinline__ T lds_read(const char *p) {
  return *reinterpret_cast<const T *>(p);
}
// four keys of one column (of this lane's 16 x 4 block)
__device__ __forceinline__ s16x4 lds_read_column(const char *p) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
}

// DC: head size padded to a multiple of 32; a row of LDS has DP >= DC elements, a power of two.
template <int DT, int DC, int RT, bool E4>
__global__ __launch_bounds__(kThreads, 1) void k_prompt(PromptAttnArgs a, Plan p) {
  typedef typename Half<DT>::V8 V8;
  typedef typename Half<DT>::V4 V4;
  typedef typename std::conditional<E4, uint8_t, uint16_t>::type Elem;
  constexpr int DP = DC <= 64 ? 64 : DC <= 128 ? 128 : 256;
  constexpr int CH = DP / 8, RB = DP * 2, TB = KT * RB;
  constexpr int NS = DC / 16, NA = DC / 32;
  constexpr int M = kWaves * kRowsWave * RT;
  constexpr int EC = E4 ? 16 : 8;                 // elements of a 16-byte load
  constexpr int CL = DP / EC;                     // loads of a row
  constexpr int NL = KT * CL / kThreads;          // loads of keys (and as many of values) of a thread
  static_assert(KT * CL % kThreads == 0, "whole loads");
  __shared__ __attribute__((aligned(16))) char sKV[4 * TB];  // keys' two buffers, then values'
  __shared__ uint32_t sOdd[M / 32 + 1];  // tokens of the tile whose values are not all finite
  const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int hw = lane / 32, col = lane % 32;
  const int G = a.Hq / a.Hkv;

  if (!lengths_in_order(a.cu, a.S, a.T)) atomicOr(a.status, SMCSD_ST_BAD_INPUT);
  // item: key/value head fastest, then split, then row tile, the last tiles (of the most keys) first
  uint32_t it = blockIdx.x;
  const int hk = (int)(it % (uint32_t)a.Hkv);
  it /= (uint32_t)a.Hkv;
  const int split = (int)(it % (uint32_t)p.splits);
  it /= (uint32_t)p.splits;
  const int64_t item = p.tiles - 1 - (int64_t)it;
  const int s = find_sequence(a.S, item, [&](int i) { return first_tile(a, i, M); });
  const int64_t tile = item - first_tile(a, s, M);
  const int t0 = a.cu[s], t1 = a.cu[s + 1];
  if (t0 < 0 || t1 <= t0 || t1 > a.T || tile < 0) return;
  const int n = t1 - t0, rows = n * G;
  if (tile * M >= rows) return;
  const int r0 = (int)(tile * M);
  int ctx = a.ctx_lens ? a.ctx_lens[s] : 0;
  const bool none = ctx < 0 || (int64_t)ctx + n > (int64_t)a.cache.M_cap * a.cache.block_size;
  if (none) {
    if (tid == 0 && hk == 0) atomicOr(a.status, SMCSD_ST_BAD_INPUT);
    ctx = 0;
  }
  const int i0 = div_by(p.group, r0), i1 = div_by(p.group, min(r0 + M, rows) - 1);  // first and last token
  const int hi = none ? 0 : ctx + i1 + 1;
  // this split's keys: an equal share in whole tiles
  const int share = ((hi + p.splits - 1) / p.splits + KT - 1) / KT * KT;
  const int k0 = (int)min((int64_t)hi, (int64_t)split * share), k1 = (int)min((int64_t)hi, (int64_t)k0 + share);
  const int own = ctx + i0;  // keys from here on are not seen by all rows

  if (tid < M / 32 + 1) sOdd[tid] = 0;

  // ---- this lane's query rows
  int tok[RT], limit[RT];
  int64_t orow[RT];
  bool live[RT];
  V8 q[RT][NS];
#pragma unroll
  for (int x = 0; x < RT; ++x) {
    const int r = r0 + (wave * RT + x) * kRowsWave + col;
    live[x] = r < rows;
    tok[x] = div_by(p.group, min(r, rows - 1));
    const int g = min(r, rows - 1) - tok[x] * G;
    limit[x] = live[x] && !none ? ctx + tok[x] : -1;
    orow[x] = (int64_t)(t0 + tok[x]) * a.Hq + hk * G + g;
    const uint16_t *qp = a.q + (int64_t)(t0 + tok[x]) * a.q_stride + (int64_t)(hk * G + g) * a.D;
    const uint32_t flip = p.negate ? 0x80008000u : 0u;
#pragma unroll
    for (int st = 0; st < NS; ++st) {
      const int d = 16 * st + 8 * hw;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (live[x] && d < a.D) w = *reinterpret_cast<const uint4 *>(qp + d);
      w.x ^= flip;
      w.y ^= flip;
      w.z ^= flip;
      w.w ^= flip;
      q[x][st] = __builtin_bit_cast(V8, w);
    }
  }
  const int wr = r0 + wave * RT * kRowsWave;  // the wave's first row
  const int wfirst = ctx + div_by(p.group, min(wr, rows - 1));
  const int wlast = wr < rows && !none ? ctx + (int)div_by(p.group, min(wr + RT * kRowsWave, rows) - 1) : -1;

  f32x16 o[RT][NA];
  float m[RT], l[RT];
#pragma unroll
  for (int x = 0; x < RT; ++x) {
#pragma unroll
    for (int t = 0; t < NA; ++t) o[x][t] = f32x16{};
    m[x] = kNegInf;
    l[x] = 0.0f;
  }

  // ---- staging
  const int32_t *table = a.cache.tables + (int64_t)s * a.cache.M_cap;
  const Elem *const kbase = static_cast<const Elem *>(a.k_cache) + (int64_t)hk * a.cache.head;
  const Elem *const vbase = static_cast<const Elem *>(a.v_cache) + (int64_t)hk * a.cache.head;
  bool bad_page = false;
  struct Tile {
    u32x4 k[NL], v[NL];
    int ks, vs;     // 8-bit pages: codes of the scales of row `lane`
    uint64_t rows;  // which may be read
  } next;
  auto ask_tile = [&](int base) {
    const int pos = base + lane, block = div_by(p.page, pos);
    const int32_t pg = pos < k1 ? table[block] : -1;
    const bool ok = pg >= 0 && pg < a.cache.P;
    bad_page |= !ok && pos < k1;
    next.rows = __ballot(ok);
    const int64_t off = ok ? pg * a.cache.page + (pos - block * (int)p.page.d) * a.cache.token : -1;
    if (E4) {
      next.ks = next.vs = 127;
      if (ok) {
        next.ks = a.k_scales[(int64_t)pg * a.Hkv + hk];
        next.vs = a.v_scales[(int64_t)pg * a.Hkv + hk];
      }
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int64_t at = __shfl((long long)off, (i * kThreads + tid) / CL, kWave);
      const int chunk = tid % CL;
      const bool in = at >= 0 && chunk * EC < a.D;
      next.k[i] = *(in ? (const u32x4 *)(kbase + at + chunk * EC) : (const u32x4 *)&kNothing);
      next.v[i] = *(in ? (const u32x4 *)(vbase + at + chunk * EC) : (const u32x4 *)&kNothing);
    }
  };
  constexpr uint32_t kExp = DT == SMCSD_DTYPE_BF16 ? 0x7F80u : 0x7C00u;
  auto finite = [&](uint32_t &w) {
    const uint32_t lo16 = (w & kExp) == kExp ? 0xFFFF0000u : ~0u;
    const uint32_t hi16 = (w & (kExp << 16)) == kExp << 16 ? 0xFFFFu : ~0u;
    w &= lo16 & hi16;
    return lo16 & hi16;
  };
  // Values of tokens that not all rows see and that are not finite become 0: a probability of 0
  // then takes nothing from them, and the rows that do see them get them after the last tile.
  auto mend = [&](uint4 &w, int pos) {
    const bool odd = (finite(w.x) & finite(w.y) & finite(w.z) & finite(w.w)) != ~0u;
    if (odd) atomicOr(&sOdd[(pos - own) / 32], 1u << ((pos - own) % 32));
  };
  auto put_tile = [&](int buf, int base) {
    const bool edge = base + KT > own;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int row = (i * kThreads + tid) / CL, chunk = tid % CL;
      const int place = place_of<CH>(row);
      char *const kr = sKV + buf * TB + row * RB, *const vr = kr + 2 * TB;
      if (E4) {
        const int ks = __shfl(next.ks, row, kWave), vs = __shfl(next.vs, row, kWave);
        uint4 k[2] = {widen8_e4m3<DT>(make_uint2(next.k[i][0], next.k[i][1]), ks), widen8_e4m3<DT>(make_uint2(next.k[i][2], next.k[i][3]), ks)};
        uint4 v[2] = {widen8_e4m3<DT>(make_uint2(next.v[i][0], next.v[i][1]), vs), widen8_e4m3<DT>(make_uint2(next.v[i][2], next.v[i][3]), vs)};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (edge && base + row >= own) {
            uint4 w = v[c];
            mend(w, base + row);
            v[c] = w;
          }
          *reinterpret_cast<uint4 *>(kr + ((2 * chunk + c) ^ place) * 16) = k[c];
          *reinterpret_cast<uint4 *>(vr + ((2 * chunk + c) ^ place) * 16) = v[c];
        }
      } else {
        uint4 v = __builtin_bit_cast(uint4, next.v[i]);
        if (edge && base + row >= own) mend(v, base + row);
        *reinterpret_cast<u32x4 *>(kr + (chunk ^ place) * 16) = next.k[i];
        *reinterpret_cast<uint4 *>(vr + (chunk ^ place) * 16) = v;
      }
    }
  };

  // ---- LDS offsets of a step's operands: keys, chunk 2 st + hw of row col; values, row 16h +
  // 8x + 4hw + i16/4, chunk 4t + 2dh + (i16%4)/2
  constexpr int NKA = NS < 8 ? NS : 8;
  constexpr int NVT = NA < 4 ? NA : 4;
  const int i16 = lane % 16, dh = (lane / 16) & 1;
  int ka[NKA], va[NVT][2];
#pragma unroll
  for (int st = 0; st < NKA; ++st) ka[st] = col * RB + (((2 * st + hw) ^ place_of<CH>(col)) * 16);
#pragma unroll
  for (int t = 0; t < NVT; ++t)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int row = 8 * x + 4 * hw + i16 / 4;
      va[t][x] = 2 * TB + row * RB + ((4 * t + 2 * dh + (i16 % 4) / 2) ^ place_of<CH>(row)) * 16 + (i16 & 1) * 8;
    }

  // 32 keys from position `base` on, in LDS from row `at` of buffer `buf`; ok: which may be read
  auto step = [&](int base, int buf, int at, uint32_t ok) {
    const char *const tile_at = sKV + buf * TB + at * RB;
    f32x16 z[RT];
#pragma unroll
    for (int x = 0; x < RT; ++x) z[x] = f32x16{};
#pragma unroll
    for (int st = 0; st < NS; ++st) {
      const V8 kf = lds_read<V8>(tile_at + ka[st % NKA] + (st / NKA) * 256);
#pragma unroll
      for (int x = 0; x < RT; ++x) z[x] = Mma<DT>::run(kf, q[x][st], z[x]);
    }
    V8 pr[RT][2];
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      if (ok != ~0u || base + 31 > wfirst) {
        const int lim = limit[x] - base;  // the last key seen
        const uint32_t see = (lim >= 31 ? ~0u : lim >= 0 ? (2u << lim) - 1 : 0u) & ok;
        const uint32_t mine = see >> (4 * hw);
#pragma unroll
        for (int i = 0; i < 16; ++i) z[x][i] = (mine >> (8 * (i / 4) + i % 4)) & 1 ? z[x][i] : kNegInf;
      }
      float top = z[x][0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top = fmaxf(top, z[x][i]);
      top = max_halves(top) * p.c;
      if (__any(top > m[x] + kLag)) {
        const float mn = fmaxf(m[x], top);
        const float f = m[x] == kNegInf ? 0.0f : fast_exp2(m[x] - mn);
        m[x] = mn;
        l[x] *= f;
#pragma unroll
        for (int t = 0; t < NA; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[x][t][i] *= f;
      }
      const float ms = m[x] == kNegInf ? 0.0f : m[x];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f32x8 e;
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = fast_exp2(fmaf(z[x][8 * h + i], p.c, -ms));
        l[x] += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
        pr[x][h] = __builtin_convertvector(e, V8);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < NA; ++t) {
        struct { s16x4 v[2]; } two = {{lds_read_column(tile_at + va[t % NVT][0] + 16 * h * RB + (t / 4) * 256),
                                       lds_read_column(tile_at + va[t % NVT][1] + 16 * h * RB + (t / 4) * 256)}};
        const V8 vf = __builtin_bit_cast(V8, two);
#pragma unroll
        for (int x = 0; x < RT; ++x) o[x][t] = Mma<DT>::run(vf, pr[x][h], o[x][t]);
      }
  };

  if (k0 < k1) {
    ask_tile(k0);
    __syncthreads();  // sOdd is clear
    put_tile(0, k0);
    uint64_t ok = next.rows;
    int buf = 0;
    if (k0 + KT < k1) ask_tile(k0 + KT);
    for (int base = k0; base < k1; base += KT) {
      __syncthreads();
      const uint64_t now = ok;
      if (base + KT < k1) {
        put_tile(buf ^ 1, base + KT);
        ok = next.rows;
        if (base + 2 * KT < k1) ask_tile(base + 2 * KT);
      }
#pragma unroll
      for (int u = 0; u < KT / 32; ++u)
        if (base + 32 * u <= wlast) step(base + 32 * u, buf, 32 * u, (uint32_t)(now >> (32 * u)));
      buf ^= 1;
    }
    __syncthreads();
    // of a value that is not finite any share is not finite either
    for (int w = 0; w < M / 32 + 1; ++w)
      for (uint32_t odd = sOdd[w]; odd; odd &= odd - 1) {
        const int pos = own + 32 * w + __builtin_ctz(odd), block = div_by(p.page, pos);
        const Elem *vp = vbase + table[block] * a.cache.page + (pos - block * (int)p.page.d) * a.cache.token;
#pragma unroll
        for (int x = 0; x < RT; ++x)
#pragma unroll
          for (int t = 0; t < NA; ++t)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const int d = 32 * t + 8 * b + 4 * hw;
              if (pos > limit[x] || d >= a.D) continue;
              if constexpr (E4) {  // no number but NaN is not finite: by element, or by the block's scale
                const uint32_t e = a.v_scales[(int64_t)table[block] * a.Hkv + hk] == 255 ? ~0u : *reinterpret_cast<const uint32_t *>(vp + d);
#pragma unroll
                for (int c = 0; c < 4; ++c) o[x][t][4 * b + c] += ((e >> (8 * c)) & 0x7F) == 0x7F ? NAN : 0.0f;
              } else {
                uint16_t e[4];
                *reinterpret_cast<uint2 *>(e) = *reinterpret_cast<const uint2 *>(vp + d);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  o[x][t][4 * b + c] += (e[c] & kExp) == kExp ? (float)__builtin_bit_cast(typename Half<DT>::T, e[c]) : 0.0f;
              }
            }
      }
  }
  if (bad_page) atomicOr(a.status, SMCSD_ST_BAD_INPUT);

#pragma unroll
  for (int x = 0; x < RT; ++x) {
    const float sum = sum_halves(l[x]);
    if (!live[x]) continue;
    if (p.splits > 1) {
      const int64_t part = (int64_t)split * a.T * a.Hq + orow[x];
      if (hw == 0) *reinterpret_cast<float2 *>(p.ml + 2 * part) = make_float2(m[x], sum);
      if (sum == 0.0f) continue;
      float *acc = p.acc + part * a.D;
#pragma unroll
      for (int t = 0; t < NA; ++t)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int d = 32 * t + 8 * b + 4 * hw;
          if (d < a.D)
            *reinterpret_cast<float4 *>(acc + d) =
                make_float4(o[x][t][4 * b], o[x][t][4 * b + 1], o[x][t][4 * b + 2], o[x][t][4 * b + 3]);
        }
      continue;
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint16_t *out = a.out + orow[x] * a.D;
#pragma unroll
    for (int t = 0; t < NA; ++t)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int d = 32 * t + 8 * b + 4 * hw;
        const f32x4 y = {o[x][t][4 * b] * inv, o[x][t][4 * b + 1] * inv, o[x][t][4 * b + 2] * inv, o[x][t][4 * b + 3] * inv};
        if (d < a.D) *reinterpret_cast<uint2 *>(out + d) = __builtin_bit_cast(uint2, __builtin_convertvector(y, V4));
      }
    if (a.lse && hw == 0) a.lse[orow[x]] = sum == 0.0f ? kNegInf : (float)(((double)m[x] + (double)log2f(sum)) * kLn2);
  }
}

// The parts of a row joined, in a fixed order: D/4 lanes (rounded up to a power of two) to a row.
constexpr int kJoinBlock = 256;

template <int DT>
__global__ __launch_bounds__(kJoinBlock) void k_prompt_join(PromptAttnArgs a, Plan p, int64_t rows, int width) {
  typedef typename Half<DT>::V4 V4;
  const int per = kJoinBlock / width, wl = threadIdx.x % width, d = 4 * wl;
  const int first = max(0, a.cu[0]), last = min(a.T, a.cu[a.S]);
  for (int64_t r = (int64_t)blockIdx.x * per + threadIdx.x / width; r < rows; r += (int64_t)gridDim.x * per) {
    const int64_t t = r / a.Hq;
    if (t < first || t >= last) continue;
    auto stat = [&](int i) { return *reinterpret_cast<const float2 *>(p.ml + 2 * (i * rows + r)); };
    float m = kNegInf, l = 0.0f;
    for (int i = 0; i < p.splits; ++i) m = stat(i).y != 0.0f ? fmaxf(m, stat(i).x) : m;
    f32x4 acc = {};
    for (int i = 0; i < p.splits; ++i) {
      const float2 ml = stat(i);
      const float f = ml.y == 0.0f || ml.x == kNegInf ? 0.0f : fast_exp2(ml.x - m);
      l = fmaf(ml.y, f, l);
      // an empty part is not written: what lies there is not used
      const f32x4 x = *reinterpret_cast<const f32x4 *>(p.acc + (i * rows + r) * a.D + (d < a.D ? d : 0));
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c] = ml.y != 0.0f ? fmaf(x[c], f, acc[c]) : acc[c];
    }
    acc *= l == 0.0f ? 0.0f : 1.0f / l;
    if (d < a.D)
      *reinterpret_cast<uint2 *>(a.out + r * a.D + d) = __builtin_bit_cast(uint2, __builtin_convertvector(acc, V4));
    if (a.lse && wl == 0) a.lse[r] = l == 0.0f ? kNegInf : (float)(((double)m + (double)log2f(l)) * kLn2);
  }
}

inline int64_t tiles_of(int64_t S, int64_t T, int G, int D) { return T * G / tile_rows(D) + S; }
// The most splits: a launch's share of kItems.
inline int max_splits(int64_t S, int64_t T, int D, int Hq, int Hkv) {
  return (int)std::max<int64_t>(1, kItems / std::max<int64_t>(1, tiles_of(S, T, Hq / Hkv, D) * Hkv));
}

template <int DT, bool E4>
void launch_pages(const PromptAttnArgs &a, const Plan &p, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)p.tiles * p.splits * a.Hkv)), block(kThreads);
  if (a.D <= 64) hipLaunchKernelGGL((k_prompt<DT, 64, 2, E4>), grid, block, 0, stream, a, p);
  else if (a.D <= 96) hipLaunchKernelGGL((k_prompt<DT, 96, 2, E4>), grid, block, 0, stream, a, p);
  else if (a.D <= 128) hipLaunchKernelGGL((k_prompt<DT, 128, 2, E4>), grid, block, 0, stream, a, p);
  else if (a.D <= 192) hipLaunchKernelGGL((k_prompt<DT, 192, 1, E4>), grid, block, 0, stream, a, p);
  else hipLaunchKernelGGL((k_prompt<DT, 256, 1, E4>), grid, block, 0, stream, a, p);
}

template <int DT>
void launch_dt(const PromptAttnArgs &a, const Plan &p, hipStream_t stream) {
  if (a.k_scales) launch_pages<DT, true>(a, p, stream);
  else launch_pages<DT, false>(a, p, stream);
  if (p.splits == 1) return;
  const int64_t rows = (int64_t)a.T * a.Hq;
  const int width = a.D <= 64 ? 16 : a.D <= 128 ? 32 : 64;
  hipLaunchKernelGGL(k_prompt_join<DT>, dim3(grid_blocks(ceil_div(rows * width, kJoinBlock), kJoinBlock)), dim3(kJoinBlock), 0,
                     stream, a, p, rows, width);
}

}  // namespace

// Workspace: [(max, sum) x splits x rows][O fp32 x splits x rows x D], for any call of up to T tokens:
// t of them in `tiles` >= max(1, t G / M) row tiles leave at most t Hq kItems / (tiles Hkv) <= kItems
// min(t G, M) parts of rows.
size_t prompt_attn_ws_bytes(int64_t T, int D, int G) {
  const size_t rows = (size_t)kItems * (size_t)std::min<int64_t>(T * G, tile_rows(D));
  return align256(sizeof(float) * 2 * rows) + align256(sizeof(float) * rows * (size_t)D) + 256;
}

hipError_t launch_prompt_attn(const PromptAttnArgs &a, int dtype, hipStream_t stream) {
  const int64_t cap = (int64_t)a.cache.M_cap * a.cache.block_size;
  const int64_t longest = a.max_len > 0 ? std::min(a.max_len, cap) : cap;
  Plan p{};
  p.page = fast_div((uint32_t)a.cache.block_size);
  p.group = fast_div((uint32_t)(a.Hq / a.Hkv));
  p.tiles = (int)tiles_of(a.S, a.T, a.Hq / a.Hkv, a.D);
  // a split's keys outweigh the part it leaves
  p.splits = (int)std::min<int64_t>(max_splits(a.S, a.T, a.D, a.Hq, a.Hkv), std::max<int64_t>(1, longest / 1024));
  const size_t rows = (size_t)p.splits * (size_t)a.T * (size_t)a.Hq;
  p.ml = reinterpret_cast<float *>(a.ws);
  p.acc = reinterpret_cast<float *>(a.ws + align256(sizeof(float) * 2 * rows));
  p.c = std::max(std::fabs(a.scale) * 1.44269504088896340736f, 1e-30f);
  p.negate = a.scale < 0.0f;
  if (dtype == SMCSD_DTYPE_BF16) launch_dt<SMCSD_DTYPE_BF16>(a, p, stream);
  else launch_dt<SMCSD_DTYPE_F16>(a, p, stream);
  return hipGetLastError();
}

}  // namespace smcsd
