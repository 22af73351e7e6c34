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
// Bound by memory: V logits in, one float per 1 KiB of them out.
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

// The careful form: masked elements (-inf, or so low that x*c overflows) add nothing, where
// the plain form's 0 * -inf would be NaN.
template <int NV>
__device__ __forceinline__ void lp_careful(LpState &st, const float (&x)[NV], float c) {
  const bool wide = lp_wide(st.mc);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const float t = wide ? (x[i] - st.m) * c : fmaf(x[i], c, -st.mc);
    const float e = fast_exp2(t);
    st.s += e;
    st.u = fmaf(e, fmaxf(t, -1e4f), st.u);
  }
}

template <int NV>
__device__ __forceinline__ void lp_update(LpState &st, const float (&x)[NV], float vmax, float c) {
  if (vmax > st.m) lp_raise(st, vmax, c);
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f}, u[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const float t = fmaf(x[i], c, -st.mc);
    const float e = fast_exp2(t);
    s[i & 3] += e;
    u[i & 3] = fmaf(e, t, u[i & 3]);
  }
  // infinite or NaN sums, and maxima too large for the plain form, take the careful one
  const float us = (u[0] + u[1]) + (u[2] + u[3]);
  if (fabsf(us) < __builtin_huge_valf() && !lp_wide(st.mc)) {
    st.s += (s[0] + s[1]) + (s[2] + s[3]);
    st.u += us;
  } else {
    lp_careful<NV>(st, x, c);
  }
}

template <int NV>
__device__ __forceinline__ float max_of(const float (&x)[NV]) {
  float v = x[0];
#pragma unroll
  for (int i = 1; i < NV; ++i) v = fmaxf(v, x[i]);
  return v;
}

template <int DT, bool TOP>
__global__ __launch_bounds__(kLpBlock) void k_lp_stream(const char *__restrict__ logits,
                                                        int64_t row_bytes, int V, float c, LpGeom g,
                                                        int64_t items, float4 *__restrict__ part,
                                                        float *__restrict__ segmax) {
  constexpr int EPV = Elt<DT>::kPerVec;
  __shared__ float sm[kLpBlock / kWave], ssum[kLpBlock / kWave], su[kLpBlock / kWave];
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t r = it / g.tiles;
    const int ch = (int)(it - r * g.tiles);
    const LpRow<DT> row(logits + r * row_bytes, V);
    float *const seg = TOP ? segmax + r * (g.segs + 2) : nullptr;
    const int v0 = ch * g.tile_vecs, v1 = min(row.nvec, v0 + g.tile_vecs);
    LpState st{kNegInf, 0.0f, 0.0f, 0.0f};
    if (ch == 0) {
      const float x[1] = {tid < row.head ? Elt<DT>::load(row.p, tid) : kNegInf};
      if (tid < row.head) lp_update<1>(st, x, x[0], c);
      if (TOP && wave == 0) {
        const float w = wave_max_f32(x[0]);
        if (lane == 0) seg[0] = w;
      }
    }
    if (ch == g.tiles - 1) {
      const float x[1] = {tid < V - row.a1 ? Elt<DT>::load(row.p, row.a1 + tid) : kNegInf};
      if (tid < V - row.a1) lp_update<1>(st, x, x[0], c);
      if (TOP && wave == 0) {
        const float w = wave_max_f32(x[0]);
        if (lane == 0) seg[g.segs + 1] = w;
      }
    }
    const uint4 *vp = reinterpret_cast<const uint4 *>(row.p + row.head * Elt<DT>::kBytes);
    int v = v0;
    for (; v + kLpBlock * kLpUnroll <= v1; v += kLpBlock * kLpUnroll) {
      const __amdgpu_buffer_rsrc_t rs = stream_rsrc(vp + v, kLpBlock * kLpUnroll * 16);
      uint4 buf[kLpUnroll];
#pragma unroll
      for (int u = 0; u < kLpUnroll; ++u) buf[u] = load_stream(rs, tid * 16, u * kLpBlock * 16);
      float x[kLpUnroll * EPV], top = kNegInf, mine[kLpUnroll];
#pragma unroll
      for (int u = 0; u < kLpUnroll; ++u) {
        float y[EPV];
        Elt<DT>::unpack(buf[u], y);
        mine[u] = max_of<EPV>(y);
        top = fmaxf(top, mine[u]);
#pragma unroll
        for (int i = 0; i < EPV; ++i) x[u * EPV + i] = y[i];
      }
      if (TOP) {
#pragma unroll
        for (int u = 0; u < kLpUnroll; ++u) {
          const float w = wave_max_f32(mine[u]);
          if (lane == 0) seg[1 + (v + u * kLpBlock) / kWave + wave] = w;
        }
      }
      lp_update<kLpUnroll * EPV>(st, x, top, c);
    }
    // the tile's last steps: segments past the row's vectors get -inf
    const int vend = TOP ? min(g.segs * kWave, v0 + g.tile_vecs) : v1;
    for (; v < vend; v += kLpBlock) {
      const int mv = v + tid;
      float top = kNegInf;
      if (mv < v1) {
        float x[EPV];
        Elt<DT>::unpack(load_stream(vp + mv), x);
        top = max_of<EPV>(x);
        lp_update<EPV>(st, x, top, c);
      }
      if (TOP) {
        const float w = wave_max_f32(top);
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

// Whole numbers in the floats' order, the two zeros alike.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;  // ordered(-inf)

// First element of slot j of a row: the head, then the body's segments, then the tail.
template <int DT>
__device__ __forceinline__ int slot_start(const LpRow<DT> &row, int segs, int j, int V) {
  if (j <= 0) return 0;
  if (j > segs + 1) return V;
  return (int)min((int64_t)row.a1, row.head + (int64_t)(j - 1) * kWave * Elt<DT>::kPerVec);
}

template <int DT>
__global__ __launch_bounds__(kLpBlock) void k_lp_finalize(LogprobsArgs a, LpGeom g, int64_t rows,
                                                          const float4 *__restrict__ part,
                                                          const float *__restrict__ segmax) {
  constexpr int EPV = Elt<DT>::kPerVec;
  __shared__ float sup[kLpSupers];
  __shared__ uint2 cand[kLpCands];
  __shared__ int sel[kMaxTop];
  __shared__ int s_nsel, s_ncand, s_count;
  __shared__ uint32_t s_key;
  __shared__ double s_max, s_ln;  // a row's largest logit, and ln of the sum relative to it
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int k = a.k;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const LpRow<DT> row(a.logits + r * a.row_bytes, a.V);
    const int slots = g.segs + 2;
    const int run = (slots + kLpSupers - 1) / kLpSupers;  // slots ranked as one
    const int nsup = (slots + run - 1) / run;
    if (tid == 0) s_ncand = 0;
    if (k > 0) {
      const float *seg = segmax + r * slots;
      for (int i = tid; i < nsup; i += kLpBlock) {
        float v = seg[i * run];
        for (int q = 1; q < run && i * run + q < slots; ++q) v = fmaxf(v, seg[i * run + q]);
        sup[i] = v;
      }
    }
    __syncthreads();
    if (wave == 0) {
      // the tiles joined in fp64: each is relative to m*c as rounded there
      const float4 *p = part + r * g.tiles;
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
        const double d = q.x == M ? 0.0 : ((double)q.x - M) * a.c;
        const double f = exp2(d - off);
        S += f * q.y;
        if (f > 0.0) U += f * (q.z + (d - off) * q.y);
      }
      S = wave_sum(S);
      U = wave_sum(U);
      if (lane == 0) {
        const double ln = log(S);
        const bool nan = isnan(S) || M == __builtin_huge_valf(), empty = !nan && M == kNegInf;
        const double lse = nan ? __builtin_nan("") : empty ? -__builtin_huge_val() : (double)M / a.T + ln;
        s_max = empty ? 0.0 : (double)M;
        s_ln = nan ? __builtin_nan("") : ln;
        if (a.lse) a.lse[r] = (float)lse;
        if (a.entropy) a.entropy[r] = nan ? __builtin_nanf("") : empty ? 0.0f : (float)fmax(0.0, ln - kLn2 * U / S);
        if (nan || empty) atomicOr(a.status, nan ? SMCSD_ST_NAN_INPUT : SMCSD_ST_EMPTY_ROW);
      }
    } else if (wave == 1 && k > 0) {
      // the k-th largest of the slots' maxima, bit by bit from the top
      constexpr int kRegs = kLpSupers / kWave;
      uint32_t key[kRegs];
#pragma unroll
      for (int i = 0; i < kRegs; ++i) key[i] = i * kWave + lane < nsup ? ordered(sup[i * kWave + lane]) : 0;
      const int regs = (nsup + kWave - 1) / kWave;
      uint32_t T = 0;
      for (int b = 31; b >= (DT == SMCSD_DTYPE_BF16 ? 16 : 0); --b) {
        const uint32_t t = T | (1u << b);
        int n = 0;
#pragma unroll
        for (int i = 0; i < kRegs; ++i)
          if (i < regs) n += __popcll(__ballot(key[i] >= t));
        if (n >= k) T = t;
      }
      // bf16 keys end in 16 equal bits: the bound stands for all of them
      const uint32_t hi = DT == SMCSD_DTYPE_BF16 ? T | 0xFFFFu : T;
      int above = 0;
#pragma unroll
      for (int i = 0; i < kRegs; ++i)
        if (i < regs) above += __popcll(__ballot(key[i] > hi));
      int ties = k - above, at = 0;  // of those at the bound, the first by place
#pragma unroll
      for (int i = 0; i < kRegs; ++i) {
        if (i >= regs) continue;
        const bool live = key[i] > kKeyNegInf, gt = live && key[i] > hi;
        const uint64_t eq = __ballot(live && !gt && key[i] >= T);
        const uint64_t before = lane == 0 ? 0 : ~0ull >> (64 - lane);
        const bool take = gt || (((eq >> lane) & 1) && __popcll(eq & before) < ties);
        const uint64_t tk = __ballot(take);
        if (take) sel[at + __popcll(tk & before)] = i * kWave + lane;
        at += __popcll(tk);
        ties = max(0, ties - (int)__popcll(eq));
      }
      if (lane == 0) {
        s_nsel = at;
        s_key = T;
      }
    }
    __syncthreads();
    // log p = (x - max) / T - ln: the two never differ by more than the result holds
    const double rmax = s_max, ln = s_ln, invT = 1.0 / a.T;
    const bool none = isnan(ln), empty = ln == -__builtin_huge_val();
    if (a.logp)
      for (int i = tid; i < a.C; i += kLpBlock) {
        const int32_t x = a.tokens[r * a.C + i];
        const bool ok = x >= 0 && x < a.V;
        if (!ok) atomicOr(a.status, SMCSD_ST_BAD_INPUT);
        const float z = ok ? Elt<DT>::load(row.p, x) : 0.0f;
        float lp = (float)((z - rmax) * invT - ln);
        if (!none && (z == kNegInf || empty)) lp = kNegInf;
        a.logp[r * a.C + i] = ok ? lp : __builtin_nanf("");
      }
    if (k > 0) {
      const uint32_t T = max(s_key, kKeyNegInf + 1);
      const int nsel = none ? 0 : s_nsel;  // a row with a NaN or +inf names no alternatives
      auto offer = [&](float x, int id) {
        const uint32_t key = ordered(x);
        if (key >= T) {
          const int at = atomicAdd(&s_ncand, 1);
          if (at < kLpCands) cand[at] = make_uint2(key, (uint32_t)id);
        }
      };
      for (int q = wave; q < nsel; q += kLpBlock / kWave) {
        const int e0 = slot_start<DT>(row, g.segs, sel[q] * run, a.V);
        const int e1 = slot_start<DT>(row, g.segs, sel[q] * run + run, a.V);
        if (e0 + lane < min(e1, row.head)) offer(Elt<DT>::load(row.p, e0 + lane), e0 + lane);
        const int b0 = max(e0, row.head), b1 = min(e1, row.a1);
        for (int e = b0 + lane * EPV; e < b1; e += kWave * EPV) {
          float x[EPV];
          Elt<DT>::unpack(*reinterpret_cast<const uint4 *>(row.p + (int64_t)e * Elt<DT>::kBytes), x);
#pragma unroll
          for (int i = 0; i < EPV; ++i) offer(x[i], e + i);
        }
        const int t0 = max(e0, row.a1);
        if (t0 + lane < e1) offer(Elt<DT>::load(row.p, t0 + lane), t0 + lane);
      }
      __syncthreads();
      int nc = s_ncand;
      if (nc > kLpCands) {
        // Too many elements at or above the bound (long runs of equal logits): the k-th
        // largest element itself, then the smallest ids among its equals, each bit by bit.
        auto count = [&](auto pred) {
          __syncthreads();
          if (tid == 0) s_count = 0;
          __syncthreads();
          int n = 0;
          for (int q = 0; q < nsel; ++q) {
            const int e1 = slot_start<DT>(row, g.segs, sel[q] * run + run, a.V);
            for (int e = slot_start<DT>(row, g.segs, sel[q] * run, a.V) + tid; e < e1; e += kLpBlock)
              n += pred(ordered(Elt<DT>::load(row.p, e)), (uint32_t)e);
          }
          if (n) atomicAdd(&s_count, n);
          __syncthreads();
          return s_count;
        };
        uint32_t K = 0;
        for (int b = 31; b >= 0; --b) {
          const uint32_t t = K | (1u << b);
          if (count([&](uint32_t key, uint32_t) { return (int)(key >= t); }) >= k) K = t;
        }
        const int need = k - count([&](uint32_t key, uint32_t) { return (int)(key > K); });
        uint32_t X = 0;  // the largest id bound that still holds fewer than `need` equals below it
        for (int b = 24; b >= 0; --b) {
          const uint32_t t = X | (1u << b);
          if (count([&](uint32_t key, uint32_t id) { return (int)(key == K && id < t); }) < need) X = t;
        }
        __syncthreads();
        if (tid == 0) s_ncand = 0;
        __syncthreads();
        for (int q = 0; q < nsel; ++q) {
          const int e1 = slot_start<DT>(row, g.segs, sel[q] * run + run, a.V);
          for (int e = slot_start<DT>(row, g.segs, sel[q] * run, a.V) + tid; e < e1; e += kLpBlock) {
            const uint32_t key = ordered(Elt<DT>::load(row.p, e));
            if (key > K || (key == K && (uint32_t)e <= X)) {
              const int at = atomicAdd(&s_ncand, 1);
              if (at < kLpCands) cand[at] = make_uint2(key, (uint32_t)e);
            }
          }
        }
        __syncthreads();
        nc = min(s_ncand, kLpCands);
      }
      for (int i = tid; i < nc; i += kLpBlock) {
        const uint2 me = cand[i];
        int rank = 0;
        for (int j = 0; j < nc; ++j) {
          const uint2 o = cand[j];
          rank += o.x > me.x || (o.x == me.x && o.y < me.y);
        }
        if (rank < k) {
          if (a.top_ids) a.top_ids[r * k + rank] = (int32_t)me.y;
          if (a.top_logp) a.top_logp[r * k + rank] = (float)((unordered(me.x) - rmax) * invT - ln);
        }
      }
      for (int i = nc + tid; i < k; i += kLpBlock) {
        if (a.top_ids) a.top_ids[r * k + i] = -1;
        if (a.top_logp) a.top_logp[r * k + i] = none ? __builtin_nanf("") : kNegInf;
      }
      __syncthreads();
    }
  }
}

template <int DT>
void launch_dt(const LogprobsArgs &a, hipStream_t stream) {
  const LpGeom g = lp_geom(a.n, a.V, Elt<DT>::kPerVec);
  const int64_t items = (int64_t)a.n * g.tiles;
  float4 *part = reinterpret_cast<float4 *>(a.ws);
  float *seg = reinterpret_cast<float *>(a.ws + align256(sizeof(float4) * (size_t)items));
  const dim3 grid(grid_blocks(items, kLpBlock)), rows(grid_blocks(a.n, kLpBlock)), block(kLpBlock);
  if (a.k > 0)
    hipLaunchKernelGGL((k_lp_stream<DT, true>), grid, block, 0, stream, a.logits, a.row_bytes, a.V, a.c, g,
                       items, part, seg);
  else
    hipLaunchKernelGGL((k_lp_stream<DT, false>), grid, block, 0, stream, a.logits, a.row_bytes, a.V, a.c, g,
                       items, part, seg);
  hipLaunchKernelGGL(k_lp_finalize<DT>, rows, block, 0, stream, a, g, (int64_t)a.n, part, seg);
}

}  // namespace

size_t logprobs_ws_bytes(int64_t n, int k, int V) {
  size_t most = 0;
  for (int per_vec : {Elt<SMCSD_DTYPE_BF16>::kPerVec, Elt<SMCSD_DTYPE_F32>::kPerVec}) {
    const LpGeom g = lp_geom(std::max<int64_t>(n, 1), V, per_vec);
    size_t b = align256(sizeof(float4) * (size_t)(n * g.tiles));
    if (k > 0) b += align256(sizeof(float) * (size_t)(n * (g.segs + 2)));
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
