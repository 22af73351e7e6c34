// logprobs.hip - log-probabilities of given tokens, entropy and top alternatives (gfx950).
//
// Two kernels.  k_lp_stream reads every logit once and keeps, per tile, the running
// maximum m with S = sum e and U = sum e*t, where t = x*c - m*c (c = log2(e)/T) and
// e = 2^t; with them ln sum exp z = m/T + ln S and the entropy is ln S - ln2 * U/S, both
// terms positive, so nothing cancels.  For the alternatives it also writes the maximum of
// every segment (the 64 vectors of 16 bytes that a wave loads together).  k_lp_finalize
// joins a row's tiles in fp64, gathers the given tokens, and finds the k largest logits:
// they lie in the k segments with the largest maxima (ordered like the elements: by value,
// then by place), because each of those k segments holds an element that precedes all
// elements of any other segment; only they are read again.
// Bound by memory: V logits in, one float per 1 KiB of them out.  2560 rows of 128,256 bf16, k = 20:
// 114 us for the stream (5.8 TB/s) and 31 us for the rest, which is latency: a row's steps follow
// one another, and five workgroups of a unit hide little of it.  576 rows of 152,063 fp32 with
// masked logits: 62 us (5.6 TB/s) and 19 us.
#include "../../include/smcsd.h"
#include "device.hpp"
#include "internal.hpp"

namespace smcsd {

namespace {

constexpr int kLpBlock = 256;
constexpr int kLpUnroll = 8;                          // vectors of a thread in flight
constexpr int kLpTileVecsMax = kLpBlock * kLpUnroll * 2;  // 64 KiB of logits
constexpr int kLpTilesWanted = 2048;                  // 8 workgroups for each of 256 CUs
constexpr int kLpSupers = 1024;                       // segments (or runs of them) ranked per row
constexpr int kLpCands = 1024;
// More than half of that at or above the bound that the slots' maxima give (as where a row has
// hardly more slots than k): the bound is formed again from the maxima of vectors, kept where
// the candidates go.  One row of 11,788 bf16, k = 32: 31 us, and 429 by the count over all bits.
// If more still reach it they are its equals, and the first of those by id are taken: 2560 rows of
// 128,256 bf16, all but 3 at the lowest value, k = 20: 295 us, and 1716 by that count.
constexpr int kLpUnits = 2 * kLpCands;

struct LpGeom {
  int tiles, tile_vecs, segs;  // segs: body segments of a row; with the head and the tail, segs + 2
};

// A row's vectors in equal tiles of whole 256-vector steps: as few as 64 KiB tiles allow,
// more where n rows would leave compute units idle.
inline LpGeom lp_geom(int64_t n, int V, int per_vec) {
  LpGeom g;
  const int64_t nvec = std::max<int64_t>(1, V / per_vec);
  int64_t want = std::max<int64_t>(ceil_div(nvec, kLpTileVecsMax), ceil_div(kLpTilesWanted, n));
  want = std::min<int64_t>(want, ceil_div(nvec, kLpBlock));
  g.tile_vecs = (int)(ceil_div(ceil_div(nvec, want), kLpBlock) * kLpBlock);
  g.tiles = (int)ceil_div(nvec, g.tile_vecs);
  g.segs = (int)ceil_div(nvec, kWave);
  return g;
}

// What a row's address makes of it: `head` elements before the first aligned vector, then
// vectors up to element a1, then a tail.
template <int DT>
struct LpRow {
  const char *p;
  int head, nvec, a1;
  __device__ __forceinline__ LpRow(const char *row, int V) : p(row) {
    head = min(V, (int)((16 - ((uintptr_t)row & 15)) & 15) / Elt<DT>::kBytes);
    nvec = (V - head) / Elt<DT>::kPerVec;
    a1 = head + nvec * Elt<DT>::kPerVec;
  }
};

// Whole numbers in the floats' order, the two zeros alike.
__device__ __forceinline__ int ordered(float x) {
  const int b = __float_as_int(x + 0.0f);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float unordered(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7FFFFFFF)); }
constexpr int kKeyNegInf = (int)0x807FFFFFu;  // ordered(-inf)
constexpr int kKeyLeast = INT32_MIN;

// The maximum over the 64 lanes, in lane 63: DPP moves whose missing lanes read the least
// value, which the compiler folds into the maxima.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ int dpp_max(int v) {
  return max(v, __builtin_amdgcn_update_dpp(kKeyLeast, v, CTRL, ROW_MASK, 0xf, false));
}
// N of them, a step for all before the next: a DPP move has to wait for the lane before it.
template <int N>
__device__ __forceinline__ void wave_max_keys(int (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = dpp_max<0x111, 0xf>(v[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = dpp_max<0x112, 0xf>(v[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = dpp_max<0x114, 0xf>(v[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = dpp_max<0x118, 0xf>(v[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = dpp_max<0x142, 0xa>(v[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = dpp_max<0x143, 0xc>(v[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __builtin_amdgcn_readlane(v[i], kWave - 1);
}
__device__ __forceinline__ int wave_max_key(int v) {
  int k[1] = {v};
  wave_max_keys(k);
  return k[0];
}

struct LpState {
  float m, mc, s, u;
};

// Beside a maximum this large the rounding of m*c itself would drown the exponent: x - m is
// formed first there.  Below it that rounding (at most 2^-4) is the same in every term of a
// tile and the finalize takes it out exactly.
__device__ __forceinline__ bool lp_wide(float mc) { return !(fabsf(mc) < 0x1p20f); }

__device__ __forceinline__ void lp_raise(LpState &st, float to, float c) {
  const float mcn = __fmul_rn(to, c), d = lp_wide(st.mc) || lp_wide(mcn) ? (st.m - to) * c : st.mc - mcn;
  if (st.m == kNegInf || !(d > -1e4f)) {
    st.s *= 0.0f;  // nothing yet, or nothing left beside the new maximum (a NaN stays)
    st.u = 0.0f;
  } else {
    const float f = fast_exp2(d);
    st.u = (st.u + st.s * d) * f;
    st.s *= f;
  }
  st.m = to;
  st.mc = mcn;
}

// One element in the careful form: masked ones (-inf, or so low that x*c overflows) add
// nothing, where the plain form's 0 * -inf would be NaN.
template <bool WIDE>
__device__ __forceinline__ void lp_careful(LpState &st, float x, float c) {
  const float t = WIDE ? (x - st.m) * c : fmaf(x, c, -st.mc);
  const float e = fast_exp2(t);
  st.s += e;
  st.u = fmaf(e, fmaxf(t, -1e4f), st.u);
}
__device__ __forceinline__ void lp_one(LpState &st, float x, float c) {
  if (x > st.m) lp_raise(st, x, c);
  if (lp_wide(st.mc)) lp_careful<true>(st, x, c);
  else lp_careful<false>(st, x, c);
}

// The same words, which the compiler does not know to be the same: elements are widened again
// where they are used rather than all kept in registers, which would leave two waves to a
// SIMD instead of five.
__device__ __forceinline__ uint4 again(uint4 w) {
  asm("" : "+v"(w.x), "+v"(w.y), "+v"(w.z), "+v"(w.w));
  return w;
}

// NU raw vectors whose largest element is vmax.  `masked` (the same in the whole wave):
// earlier ones held elements that need the careful form, so it is taken at once.
template <int DT, int NU>
__device__ __forceinline__ void lp_update(LpState &st, const uint4 (&raw)[NU], float vmax, float c, bool &masked) {
  constexpr int EPV = Elt<DT>::kPerVec;
  if (vmax > st.m) lp_raise(st, vmax, c);
  const bool wide = __any(lp_wide(st.mc));
  if (!masked && !wide) {
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f}, u[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < NU; ++v) {
      float x[EPV];
      Elt<DT>::unpack(raw[v], x);
#pragma unroll
      for (int i = 0; i < EPV; ++i) {
        const float t = fmaf(x[i], c, -st.mc);
        const float e = fast_exp2(t);
        s[i & 3] += e;
        u[i & 3] = fmaf(e, t, u[i & 3]);
      }
    }
    const float us = (u[0] + u[1]) + (u[2] + u[3]);
    masked = __any(!(fabsf(us) < __builtin_huge_valf()));
    if (!masked) {
      st.s += (s[0] + s[1]) + (s[2] + s[3]);
      st.u += us;
      return;
    }
  }
#pragma unroll
  for (int v = 0; v < NU; ++v) {
    float x[EPV];
    Elt<DT>::unpack(again(raw[v]), x);
    if (wide) {
#pragma unroll
      for (int i = 0; i < EPV; ++i) {
        if (lp_wide(st.mc)) lp_careful<true>(st, x[i], c);
        else lp_careful<false>(st, x[i], c);
      }
    } else {
#pragma unroll
      for (int i = 0; i < EPV; ++i) lp_careful<false>(st, x[i], c);
    }
  }
}

// The largest element of a raw vector.
template <int DT>
__device__ __forceinline__ float max_of(const uint4 &w) {
  float x[Elt<DT>::kPerVec];
  Elt<DT>::unpack(w, x);
  float v = x[0];
#pragma unroll
  for (int i = 1; i < Elt<DT>::kPerVec; ++i) v = fmaxf(v, x[i]);
  return v;
}

template <int DT, bool TOP>
__global__ __launch_bounds__(kLpBlock) void k_lp_stream(const char *__restrict__ logits,
                                                        int64_t row_bytes, int V, float c, LpGeom g,
                                                        int64_t items, float4 *__restrict__ part,
                                                        int *__restrict__ segkey) {
  __shared__ float sm[kLpBlock / kWave], ssum[kLpBlock / kWave], su[kLpBlock / kWave];
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t r = it / g.tiles;
    const int ch = (int)(it - r * g.tiles);
    const LpRow<DT> row(logits + r * row_bytes, V);
    int *const seg = TOP ? segkey + r * (g.segs + 2) : nullptr;
    const int v0 = ch * g.tile_vecs, v1 = min(row.nvec, v0 + g.tile_vecs);
    LpState st{kNegInf, 0.0f, 0.0f, 0.0f};
    if (ch == 0) {
      const float x = tid < row.head ? Elt<DT>::load(row.p, tid) : kNegInf;
      if (tid < row.head) lp_one(st, x, c);
      if (TOP && wave == 0) {
        const int w = wave_max_key(ordered(x));
        if (lane == 0) seg[0] = w;
      }
    }
    if (ch == g.tiles - 1) {
      const float x = tid < V - row.a1 ? Elt<DT>::load(row.p, row.a1 + tid) : kNegInf;
      if (tid < V - row.a1) lp_one(st, x, c);
      if (TOP && wave == 0) {
        const int w = wave_max_key(ordered(x));
        if (lane == 0) seg[g.segs + 1] = w;
      }
    }
    const uint4 *vp = reinterpret_cast<const uint4 *>(row.p + row.head * Elt<DT>::kBytes);
    int v = v0;
    bool masked = false;
    // segments past the row's vectors get -inf
    const int vend = TOP ? min(g.segs * kWave, v0 + g.tile_vecs) : v1;
    for (; v + kLpBlock < vend; v += kLpBlock * kLpUnroll) {
      uint4 buf[kLpUnroll];
      if (v + kLpBlock * kLpUnroll <= v1) {
        const __amdgpu_buffer_rsrc_t rs = stream_rsrc(vp + v, kLpBlock * kLpUnroll * 16);
#pragma unroll
        for (int u = 0; u < kLpUnroll; ++u) buf[u] = load_stream(rs, tid * 16, u * kLpBlock * 16);
      } else {  // the row's end: -inf past it, which the careful form passes over
        masked = true;
#pragma unroll
        for (int u = 0; u < kLpUnroll; ++u) {
          const int at = v + u * kLpBlock + tid;
          buf[u] = at < v1 ? load_stream(vp + at) : NegInfVec<DT>::get();
        }
      }
      float top = kNegInf;
      int key[kLpUnroll];
#pragma unroll
      for (int u = 0; u < kLpUnroll; ++u) {
        const float mine = max_of<DT>(buf[u]);
        buf[u] = again(buf[u]);
        top = fmaxf(top, mine);
        key[u] = ordered(mine);
      }
      if (TOP) {
        wave_max_keys(key);
        int keys = key[0];  // lane u: the largest of the wave's vectors u
#pragma unroll
        for (int u = 1; u < kLpUnroll; ++u) keys = lane == u ? key[u] : keys;
        const int at = v / kWave + wave + lane * (kLpBlock / kWave);
        if (lane < kLpUnroll && at < min(g.segs, (v0 + g.tile_vecs) / kWave)) seg[1 + at] = keys;
      }
      lp_update<DT, kLpUnroll>(st, buf, top, c, masked);
    }
    if (v < vend) {  // one step, as in the smallest tiles
      const int at = v + tid;
      float top = kNegInf;
      if (at < v1) {
        const uint4 raw[1] = {load_stream(vp + at)};
        top = max_of<DT>(raw[0]);
        lp_update<DT, 1>(st, raw, top, c, masked);
      }
      if (TOP) {
        const int w = wave_max_key(ordered(top));
        if (lane == 0 && v / kWave + wave < g.segs) seg[1 + v / kWave + wave] = w;
      }
    }
    // the workgroup's sums, relative to its maximum
    const float wm = wave_max_f32(st.m);
    if (lane == 0) sm[wave] = wm;
    __syncthreads();
    float M = sm[0];
#pragma unroll
    for (int w = 1; w < kLpBlock / kWave; ++w) M = fmaxf(M, sm[w]);
    if (M > st.m) lp_raise(st, M, c);
    const float s = wave_sum_f32(st.s), u = wave_sum_f32(st.u);
    if (lane == 0) {
      ssum[wave] = s;
      su[wave] = u;
    }
    __syncthreads();
    if (tid == 0) {
      float S = ssum[0], U = su[0];
#pragma unroll
      for (int w = 1; w < kLpBlock / kWave; ++w) {
        S += ssum[w];
        U += su[w];
      }
      part[it] = make_float4(M, S, U, 0.0f);
    }
  }
}

// First element of slot j of a row: the head, then the body's segments, then the tail.
template <int DT>
__device__ __forceinline__ int slot_start(const LpRow<DT> &row, int segs, int j, int V) {
  if (j <= 0) return 0;
  if (j > segs + 1) return V;
  return min(row.a1, row.head + (j - 1) * kWave * Elt<DT>::kPerVec);
}

// Slots of a row that one wave ranks with 4 keys a lane; more take 16 keys a lane (as 252 slots
// would, in 63 us for 2560 rows instead of 32).
constexpr int kLpSmall = 256;

// KREGS: keys of a lane of the wave that ranks the slots (4 or kLpSupers / 64).  Registers for five
// workgroups of a unit: 32 us for 2560 rows of 128,256, k = 20, against 39 with four, 36 with six
// (which spill).
template <int DT, int KREGS>
__global__ __launch_bounds__(kLpBlock, KREGS == 4 ? 5 : 3) void k_lp_finalize(LogprobsArgs a, LpGeom g, int64_t rows,
                                                          const float4 *__restrict__ part,
                                                          const int *__restrict__ segkey) {
  constexpr int EPV = Elt<DT>::kPerVec;
  constexpr int W = kLpBlock / kWave;
  __shared__ int2 cand[kLpCands];
  __shared__ int sel[kMaxTop];
  __shared__ int s_nsel, s_ncand, s_count, s_key, s_bits[32];
  __shared__ double s_max, s_ln;  // a row's largest logit, and ln of the sum relative to it
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int k = a.k;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const LpRow<DT> row(a.logits + r * a.row_bytes, a.V);
    const int slots = g.segs + 2;
    const int run = (slots + KREGS * kWave - 1) / (KREGS * kWave);  // slots ranked as one
    const int nsup = (slots + run - 1) / run;
    if (tid == 0) s_ncand = 0;
    if (wave == 0) {
      // the tiles joined in fp64: each is relative to m*c as rounded there
      const float4 *const p = part + r * g.tiles;
      float M = kNegInf;
      for (int i = lane; i < g.tiles; i += kWave) M = fmaxf(M, p[i].x);
      M = wave_max_f32(M);
      double S = 0.0, U = 0.0;
      for (int i = lane; i < g.tiles; i += kWave) {
        const float4 q = p[i];
        if (q.x == kNegInf) {
          S += (double)q.y * 0.0;
          continue;
        }
        const float mc = __fmul_rn(q.x, a.c);
        const double off = lp_wide(mc) ? 0.0 : (double)q.x * a.c - mc;
        const double d = (q.x == M ? 0.0 : ((double)q.x - M) * a.c) - off;
        const double f = (double)fast_exp2((float)d);  // d is small where f matters
        S += f * q.y;
        if (f > 0.0) U += f * (q.z + d * q.y);
      }
      S = wave_sum(S);
      U = wave_sum(U);
      const double ln = log(S);
      const bool nan = !(S < __builtin_huge_val()) || M == __builtin_huge_valf(), empty = !nan && M == kNegInf;
      if (lane == 0) {
        s_max = empty ? 0.0 : (double)M;
        s_ln = nan ? __builtin_nan("") : ln;
        if (a.lse) a.lse[r] = nan ? __builtin_nanf("") : empty ? kNegInf : (float)((double)M * a.inv_T + ln);
        if (a.entropy) a.entropy[r] = nan ? __builtin_nanf("") : empty ? 0.0f : (float)fmax(0.0, ln - kLn2 * U / S);
        if (nan || empty) atomicOr(a.status, nan ? SMCSD_ST_NAN_INPUT : SMCSD_ST_EMPTY_ROW);
      }
    } else if (wave == 1 && k > 0) {
      const int *seg = segkey + r * slots;
      int key[KREGS];
#pragma unroll
      for (int i = 0; i < KREGS; ++i) {
        const int sup = i * kWave + lane;
        key[i] = kKeyLeast;
        for (int q = 0; q < run && sup < nsup && sup * run + q < slots; ++q) key[i] = max(key[i], seg[sup * run + q]);
      }
      // the k-th largest of the slots' maxima, bit by bit from the top (as unsigned numbers)
      uint32_t T = 0;
      for (int b = 31; b >= (DT == SMCSD_DTYPE_BF16 ? 16 : 0); --b) {
        const int t = (int)((T | (1u << b)) ^ 0x80000000u);
        int n = 0;
#pragma unroll
        for (int i = 0; i < KREGS; ++i) n += __popcll(__ballot(key[i] >= t));
        if (n >= k) T |= 1u << b;
      }
      // bf16 keys end in 16 equal bits: the bound stands for all of them
      const int least = (int)(T ^ 0x80000000u), most = DT == SMCSD_DTYPE_BF16 ? least | 0xFFFF : least;
      int above = 0;
#pragma unroll
      for (int i = 0; i < KREGS; ++i) above += __popcll(__ballot(key[i] > most));
      int ties = k - above, at = 0;  // of those at the bound, the first by place
#pragma unroll
      for (int i = 0; i < KREGS; ++i) {
        const bool live = key[i] > kKeyNegInf, gt = live && key[i] > most;
        const uint64_t eq = __ballot(live && !gt && key[i] >= least);
        const uint64_t before = lane == 0 ? 0 : ~0ull >> (64 - lane);
        const bool take = gt || (((eq >> lane) & 1) && __popcll(eq & before) < ties);
        const uint64_t tk = __ballot(take);
        if (take) sel[at + __popcll(tk & before)] = i * kWave + lane;
        at += __popcll(tk);
        ties = max(0, ties - (int)__popcll(eq));
      }
      if (lane == 0) {
        s_nsel = at;
        s_key = max(least, kKeyNegInf + 1);
      }
    }
    // the last two waves look up the given tokens' logits meanwhile, one to a thread
    constexpr int kGather = kLpBlock / 2;
    float zt = 0.0f;
    bool ok = false;
    auto gather = [&](int i) {
      const int32_t x = a.tokens[r * a.C + i];
      ok = x >= 0 && x < a.V;
      if (ok) zt = Elt<DT>::load(row.p, x);
    };
    const int g0 = tid - kGather;
    const bool gathers = a.logp && g0 >= 0;
    if (gathers && g0 < a.C) gather(g0);
    __syncthreads();
    if (k > 0) {
      int T = s_key;
      float bound = unordered(T);
      const int nsel = s_nsel;
      // Candidates' ids: a wave's lanes count theirs, one lane takes places for all.
      auto offer = [&](uint32_t mine, auto value) {
        if (!__any(mine)) return;
        const int n = __popc(mine), upto = wave_inclusive_scan(n);
        int at = 0;
        if (lane == kWave - 1) at = atomicAdd(&s_ncand, upto);
        at = __builtin_amdgcn_readlane(at, kWave - 1) + upto - n;
        while (mine) {
          const int b = __builtin_ctz(mine);
          mine &= mine - 1;
          if (at < kLpCands) cand[at].y = value(b);
          ++at;
        }
      };
      auto offer_one = [&](bool in, int id) {
        const float x = in ? Elt<DT>::load(row.p, id) : kNegInf;
        offer(in && ordered(x) >= T ? 1u : 0u, [&](int) { return id; });
      };
      auto vec_bits = [&](const uint4 &w) {
        float x[EPV];
        Elt<DT>::unpack(w, x);
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < EPV; ++i) m |= (x[i] >= bound ? 1u : 0u) << i;
        return m;
      };
      auto load_vec = [&](int e) { return *reinterpret_cast<const uint4 *>(row.p + (int64_t)e * Elt<DT>::kBytes); };
      // The k-th largest of the maxima of the selected slots' vectors (or of runs of them), as of
      // the slots above: at least k elements reach it, and without ties at most k vectors' can.
      auto refine = [&] {
        int *const key = reinterpret_cast<int *>(cand);
        const int each = run * kWave, vecs = nsel * each;
        const int per = (vecs + kLpUnits - 1) / kLpUnits, units = (vecs + per - 1) / per;
#pragma unroll 1
        for (int u = tid; u < units; u += kLpBlock) {
          int most = kKeyNegInf;
#pragma unroll 1
          for (int v = u * per; v < min(u * per + per, vecs); ++v) {
            const int slot = sel[v / each] * run;
            const int e = max(slot_start<DT>(row, g.segs, slot, a.V), row.head) + v % each * EPV;
            if (e >= min(slot_start<DT>(row, g.segs, slot + run, a.V), row.a1)) continue;
            float x[EPV];
            Elt<DT>::unpack(load_vec(e), x);
#pragma unroll
            for (int i = 0; i < EPV; ++i) most = max(most, ordered(x[i]));
          }
          key[u] = most;
        }
        if (tid < 32) s_bits[tid] = 0;
        __syncthreads();
        uint32_t K = 0;
        for (int b = 31; b >= (DT == SMCSD_DTYPE_BF16 ? 16 : 0); --b) {
          const int t = (int)((K | (1u << b)) ^ 0x80000000u);
          int n = 0;
          for (int u = tid; u < units; u += kLpBlock) n += key[u] >= t;
          n = wave_inclusive_scan(n);
          if (lane == kWave - 1) atomicAdd(&s_bits[b], n);
          __syncthreads();
          if (s_bits[b] >= k) K |= 1u << b;
        }
        T = max((int)(K ^ 0x80000000u), kKeyNegInf + 1);
        bound = unordered(T);
        if (tid == 0) s_ncand = 0;
        __syncthreads();
      };
      // Pass 0: what reaches the slots' bound; 1: what reaches the finer one (at once where nothing
      // is below the first, as in rows of fewer slots than k); 2, where many equal the finer one
      // (rows masked with a lowest value): what is above it.
      int nc, pass = T > kKeyNegInf + 1 || nsel * run * kWave * EPV <= kLpCands / 2 ? 0 : 1;
      for (;; ++pass) {
        if (pass == 1) refine();
        // each wave reads its share of the slots, several at a time where a slot is one vector
        // a lane
        constexpr int kBatch = 4;
        for (int q0 = wave; q0 < nsel; q0 += W * kBatch) {
          uint4 w[kBatch];
          int at[kBatch];
#pragma unroll
          for (int q = 0; q < kBatch; ++q) {
            const int i = q0 + q * W;
            at[q] = -1;
            if (i >= nsel) continue;
            const int b0 = max(slot_start<DT>(row, g.segs, sel[i] * run, a.V), row.head) + lane * EPV;
            const int b1 = min(slot_start<DT>(row, g.segs, sel[i] * run + run, a.V), row.a1);
            if (b0 < b1) {
              at[q] = b0;
              w[q] = load_vec(b0);
            }
          }
          uint32_t mine = 0;
#pragma unroll
          for (int q = 0; q < kBatch; ++q)
            if (at[q] >= 0) mine |= vec_bits(w[q]) << (EPV * q);
          offer(mine, [&](int b) {
            const int q = b / EPV;
            return (q == 0 ? at[0] : q == 1 ? at[1] : q == 2 ? at[2] : at[3]) + b % EPV;
          });
          for (int i = q0; i < min(nsel, q0 + W * kBatch); i += W) {
            const int e0 = slot_start<DT>(row, g.segs, sel[i] * run, a.V);
            const int e1 = slot_start<DT>(row, g.segs, sel[i] * run + run, a.V);
            if (e0 < row.head) offer_one(e0 + lane < min(e1, row.head), e0 + lane);
            if (e1 > row.a1) offer_one(max(e0, row.a1) + lane < e1, max(e0, row.a1) + lane);
            for (int e = max(e0, row.head) + kWave * EPV; e < min(e1, row.a1); e += kWave * EPV) {
              const int m0 = e + lane * EPV;
              const uint32_t m = m0 < min(e1, row.a1) ? vec_bits(load_vec(m0)) : 0;
              offer(m, [&](int b) { return m0 + b; });
            }
          }
        }
        __syncthreads();
        nc = s_ncand;
        if (pass == 2 || nc <= (pass == 0 ? kLpCands / 2 : kLpCands) || isnan(s_ln)) break;
        __syncthreads();
        if (pass == 1) {
          T = (DT == SMCSD_DTYPE_BF16 ? T | 0xFFFF : T) + 1;
          bound = unordered(T);
          if (tid == 0) s_ncand = 0;
          __syncthreads();
        }
      }
      for (int i = tid; i < min(nc, kLpCands); i += kLpBlock) cand[i].x = ordered(Elt<DT>::load(row.p, cand[i].y));
      __syncthreads();
      if (pass == 2 && !isnan(s_ln)) {
        // the equals of the smallest ids: the slots, and the elements in them, stand by id
        for (int q = 0; q < nsel && nc < k; ++q) {
          const int e1 = slot_start<DT>(row, g.segs, sel[q] * run + run, a.V);
          for (int e0 = slot_start<DT>(row, g.segs, sel[q] * run, a.V); e0 < e1 && nc < k; e0 += kLpBlock) {
            const int e = e0 + tid;
            const int key = e < e1 ? ordered(Elt<DT>::load(row.p, e)) : 0;
            const uint64_t eq = __ballot(e < e1 && key < T && key >= T - (DT == SMCSD_DTYPE_BF16 ? 0x10000 : 1));
            if (lane == 0) s_bits[wave] = (int)__popcll(eq);
            __syncthreads();
            int at = nc + (int)__popcll(eq & (lane == 0 ? 0 : ~0ull >> (64 - lane)));
#pragma unroll
            for (int w = 0; w < W; ++w) {
              at += w < wave ? s_bits[w] : 0;
              nc += s_bits[w];
            }
            if (((eq >> lane) & 1) && at < kLpCands) cand[at] = make_int2(key, e);
            __syncthreads();
          }
        }
      }
      if (nc > kLpCands && !isnan(s_ln)) {
        // Too many elements above the finer bound, as in sorted rows of millions: the k-th
        // largest element itself, then the smallest ids among its equals, each bit by bit.
        auto count = [&](auto pred) {
          __syncthreads();
          if (tid == 0) s_count = 0;
          __syncthreads();
          int n = 0;
          for (int q = 0; q < nsel; ++q) {
            const int e1 = slot_start<DT>(row, g.segs, sel[q] * run + run, a.V);
            for (int e = slot_start<DT>(row, g.segs, sel[q] * run, a.V) + tid; e < e1; e += kLpBlock)
              n += pred(ordered(Elt<DT>::load(row.p, e)), e);
          }
          if (n) atomicAdd(&s_count, n);
          __syncthreads();
          return s_count;
        };
        uint32_t K = 0;
#pragma unroll 1
        for (int b = 31; b >= 0; --b) {
          const int t = (int)((K | (1u << b)) ^ 0x80000000u);
          if (count([&](int key, int) { return (int)(key >= t); }) >= k) K |= 1u << b;
        }
        const int bound = (int)(K ^ 0x80000000u);
        const int need = k - count([&](int key, int) { return (int)(key > bound); });
        int X = 0;  // the largest id bound that still holds fewer than `need` equals below it
#pragma unroll 1
        for (int b = 24; b >= 0; --b) {
          const int t = X | (1 << b);
          if (count([&](int key, int id) { return (int)(key == bound && id < t); }) < need) X = t;
        }
        __syncthreads();
        if (tid == 0) s_ncand = 0;
        __syncthreads();
        for (int q = 0; q < nsel; ++q) {
          const int e1 = slot_start<DT>(row, g.segs, sel[q] * run + run, a.V);
          for (int e = slot_start<DT>(row, g.segs, sel[q] * run, a.V) + tid; e < e1; e += kLpBlock) {
            const int key = ordered(Elt<DT>::load(row.p, e));
            if (key > bound || (key == bound && e <= X)) {
              const int at = atomicAdd(&s_ncand, 1);
              if (at < kLpCands) cand[at] = make_int2(key, e);
            }
          }
        }
        __syncthreads();
        nc = min(s_ncand, kLpCands);
      }
      if (isnan(s_ln)) nc = 0;  // a row with a NaN or +inf names no alternatives
      const double rmax = s_max, ln = s_ln;
      for (int i = tid; i < nc; i += kLpBlock) {
        const int2 me = cand[i];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < nc; ++j) {
          const int2 o = cand[j];
          rank += o.x > me.x || (o.x == me.x && o.y < me.y);
        }
        if (rank < k) {
          if (a.top_ids) a.top_ids[r * k + rank] = me.y;
          // log p = (x - max) / T - ln: the two never differ by more than the result holds
          if (a.top_logp) a.top_logp[r * k + rank] = (float)((unordered(me.x) - rmax) * a.inv_T - ln);
        }
      }
      for (int i = nc + tid; i < k; i += kLpBlock) {
        if (a.top_ids) a.top_ids[r * k + i] = -1;
        if (a.top_logp) a.top_logp[r * k + i] = isnan(ln) ? __builtin_nanf("") : kNegInf;
      }
    } else {
      __syncthreads();
    }
    if (gathers) {
      const double rmax = s_max, ln = s_ln;
      for (int i = g0; i < a.C; i += kGather) {
        if (i != g0) gather(i);
        if (!ok) atomicOr(a.status, SMCSD_ST_BAD_INPUT);
        float lp = (float)((zt - rmax) * a.inv_T - ln);
        if (!isnan(ln) && (zt == kNegInf || ln == -__builtin_huge_val())) lp = kNegInf;
        a.logp[r * a.C + i] = ok ? lp : __builtin_nanf("");
      }
    }
    __syncthreads();
  }
}

template <int DT>
void launch_dt(const LogprobsArgs &a, hipStream_t stream) {
  const LpGeom g = lp_geom(a.n, a.V, Elt<DT>::kPerVec);
  const int64_t items = (int64_t)a.n * g.tiles;
  float4 *part = reinterpret_cast<float4 *>(a.ws);
  int *seg = reinterpret_cast<int *>(a.ws + align256(sizeof(float4) * (size_t)items));
  const dim3 grid(grid_blocks(items, kLpBlock)), rows(grid_blocks(a.n, kLpBlock)), block(kLpBlock);
  if (a.k > 0)
    hipLaunchKernelGGL((k_lp_stream<DT, true>), grid, block, 0, stream, a.logits, a.row_bytes, a.V, a.c, g,
                       items, part, seg);
  else
    hipLaunchKernelGGL((k_lp_stream<DT, false>), grid, block, 0, stream, a.logits, a.row_bytes, a.V, a.c, g,
                       items, part, seg);
  if (g.segs + 2 <= kLpSmall)
    hipLaunchKernelGGL((k_lp_finalize<DT, kLpSmall / kWave>), rows, block, 0, stream, a, g, (int64_t)a.n, part, seg);
  else
    hipLaunchKernelGGL((k_lp_finalize<DT, kLpSupers / kWave>), rows, block, 0, stream, a, g, (int64_t)a.n, part, seg);
}

}  // namespace

size_t logprobs_ws_bytes(int64_t n, int k, int V) {
  size_t most = 0;
  for (int per_vec : {Elt<SMCSD_DTYPE_BF16>::kPerVec, Elt<SMCSD_DTYPE_F32>::kPerVec}) {
    const LpGeom g = lp_geom(std::max<int64_t>(n, 1), V, per_vec);
    size_t b = align256(sizeof(float4) * (size_t)(n * g.tiles));
    if (k > 0) b += align256(sizeof(int) * (size_t)(n * (g.segs + 2)));
    most = std::max(most, b);
  }
  return std::max<size_t>(most, 256);
}

hipError_t launch_logprobs(const LogprobsArgs &a, int dtype, hipStream_t stream) {
  if (dtype == SMCSD_DTYPE_BF16) launch_dt<SMCSD_DTYPE_BF16>(a, stream);
  else launch_dt<SMCSD_DTYPE_F32>(a, stream);
  return hipGetLastError();
}

}  // namespace smcsd
