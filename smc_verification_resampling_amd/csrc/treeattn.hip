// treeattn.hip - attention of drafted trees over the paged cache (gfx950).
//
// The query rows of one key/value head - R nodes x Hq/Hkv heads of a sequence, or those of
// all N particles of a prompt over the blocks that their tables share - go through the keys
// together, 32 rows to a wave.  Scores are formed transposed, S^T = K Q^T, with
// mfma 32x32x16: a lane then holds one query row and 16 of a step's 32 keys, so that the
// running maximum and sum need one exchange between the wave's halves, and its 16
// probabilities, rounded to 16 bits, are at once the second operand of O^T = V^T P^T: that
// product's order of keys is free, so the first operand takes the same order, four keys at
// a time, with the transposing LDS read.  Probabilities never leave the registers, and the
// rescaling of O is one factor per lane.
// Keys and values go through LDS in tiles of 32 tokens, shared by a workgroup's waves, with
// loads that write to LDS directly: the next tile is on its way while the present one is
// computed.  Rows of a tile are stored with their 16-byte chunks permuted by the row number,
// so that reads of one chunk over many rows fall on different banks.
// Long contexts are split over workgroups (each a range of keys of equal length) and the
// parts (m, l, O) joined in fp32.
#include <cmath>

#include "../../include/smcsd.h"
#include "device.hpp"
#include "half.hpp"
#include "internal.hpp"

namespace smcsd {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

// Reads of a tile.  In assembly, each with its wait: the compiler, which knows no buffers,
// would let a read of one wait for all loads to LDS, those of the next tiles too.
// four rows' 16 bytes each
template <class V8>
__device__ __forceinline__ void read_rows(V8 (&x)[4], uint32_t a, uint32_t b, uint32_t c, uint32_t d, int offset) {
  asm volatile(
      "ds_read_b128 %0, %4 offset:%8\n\tds_read_b128 %1, %5 offset:%8\n\t"
      "ds_read_b128 %2, %6 offset:%8\n\tds_read_b128 %3, %7 offset:%8\n\ts_waitcnt lgkmcnt(0)"
      : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3])
      : "v"(a), "v"(b), "v"(c), "v"(d), "i"(offset));
}
// two times 4 + 4 keys of one column
template <class V8>
__device__ __forceinline__ void read_columns(V8 (&x)[2], uint32_t a, uint32_t b, uint32_t c, uint32_t d, int offset) {
  s16x4 y[4];
  asm volatile(
      "ds_read_b64_tr_b16 %0, %4 offset:%8\n\tds_read_b64_tr_b16 %1, %5 offset:%8\n\t"
      "ds_read_b64_tr_b16 %2, %6 offset:%8\n\tds_read_b64_tr_b16 %3, %7 offset:%8\n\ts_waitcnt lgkmcnt(0)"
      : "=&v"(y[0]), "=&v"(y[1]), "=&v"(y[2]), "=&v"(y[3])
      : "v"(a), "v"(b), "v"(c), "v"(d), "i"(offset));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    struct { s16x4 v[2]; } two = {{y[2 * i], y[2 * i + 1]}};
    x[i] = __builtin_bit_cast(V8, two);
  }
}

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

// ---------------------------------------------------------------------------------
// Launch plan
// ---------------------------------------------------------------------------------
constexpr int kRowsWave = 32;
// Keys of a tile, and two buffers for them.  Heads of 128: 64 keys for four waves gave 110 us
// against 118 for 64 rows of 16 heads over 131,071 keys, but 154 against 147 for 32 prompts'
// 2048 shared keys and 320 x 8 rows each; three buffers 123 and 149 there, and for two waves
// (256 sequences of 8 heads, 3.2 GB) 687 us against 661, four buffers 802: what the loads gain
// in flight, the workgroups lose that no longer fit beside each other.
constexpr int KT = 32, NB = 2;
constexpr int kWavesMax = 4;
// Workgroups of one wave of rows that the splits of a launch aim at (half as many where two row tiles
// of four waves share a head's keys): 64 rows x 16 heads over 131,071 keys take 120 us and 12 to join
// the parts with 1024, 161 + 8 with 512, 136 + 22 with 2048.
constexpr int kPartItems = 1024;
// Shorter shared prefixes are read by every particle (the caches hold them): 512 sequences of 5 x
// 32 heads with 128 shared keys take 67 us so and 85 to 89 with a pass of their own, with 256 keys
// 94 against 93 to 107, and from there on the pass wins (2048 keys: 240 us against 482).
constexpr int kMinShared = 256;

// How the rows of one key/value head and the keys are cut: `tiles` workgroups of `waves`
// waves over the rows, `splits` over the keys.
struct Cut {
  int rows, tiles, tile_rows, waves, splits;
};
inline int pad_dim(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }
// The most splits for `heads` heads of `rows` rows each: a head's share of kPartItems, divided by the
// waves of its rows or, beyond four tiles, by its tiles.  Fewer for more rows.  Divided by four for
// any number of tiles, 64 particles x 9 nodes x 32 / 8 heads over 8192 shared keys (18 tiles) took 190 us
// and 1.5 GB of workspace for 160 us and 0.3 GB, over 32,768 keys 586 us for 439.
inline int max_splits(int64_t heads, int64_t rows) {
  const int64_t tiles = ceil_div(rows, kWavesMax * kRowsWave), waves = std::min<int64_t>(ceil_div(rows, kRowsWave), kWavesMax);
  return (int)std::max<int64_t>(1, ceil_div(kPartItems, std::max<int64_t>(heads, 1)) / std::max<int64_t>({waves, tiles, 1}));
}
inline Cut cut_of(int rows, int64_t heads, int64_t max_len) {
  Cut c;
  c.rows = rows;
  const int most = kWavesMax * kRowsWave;
  c.tiles = (int)ceil_div(rows, most);
  c.tile_rows = (int)ceil_div(ceil_div(rows, c.tiles), kRowsWave) * kRowsWave;  // whole waves
  // Two waves for up to 32 rows too, where the second one only loads: 66 us against 75 with one (512
  // sequences of 20 rows x 8 heads, 80 keys each), 250 against 261 (16 of 30,000 keys), 359 against
  // 396 (heads of 192), 5.6 against 6.1 (one token); four took 92, 469, 699 and 5.5.  36 rows of 256
  // sequences: 606 us with two, 684 with four; 107 to 128 rows: 150 with four, 208 with twice as
  // many tiles of two.
  c.waves = c.tile_rows <= 2 * kRowsWave ? 2 : kWavesMax;
  // enough workgroups to fill the chip, but a split's keys outweigh the part it leaves
  const int64_t most_splits = ceil_div(max_len, std::max(256, 4 * std::min(rows, most)));
  c.splits = (int)std::max<int64_t>(1, std::min<int64_t>(max_splits(heads, rows), most_splits));
  return c;
}

// n / d for 0 <= n < 2^31: the high half of n * ceil(2^(31+s) / d), s = ceil(log2 d),
// shifted by s - 1 (exact: the error n * (M*d - 2^(31+s)) < 2^31 * 2^s).
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
  FastDiv page;
  Cut prefix, suffix;          // prefix.splits = 0: no shared-prefix pass
  const int32_t *shared_len;   // [B] (null: none shared)
  float *ml;                   // [parts][rows of out] (max, sum) pairs; prefix parts first
  float *acc;                  // [parts][rows of out][D]
  float c;                     // |scale| * log2(e)
  int negate;                  // a negative scale turns the queries' signs
};

// What a sequence's arrays say, within bounds: `none` if it sees nothing at all.
struct Seq {
  int ctx, nodes;
  bool none, bad;
};
__device__ __forceinline__ Seq seq_of(const TreeAttnArgs &a, int s) {
  Seq q;
  q.nodes = a.R;
  q.bad = false;
  if (a.num_nodes) {
    const int n = a.num_nodes[s];
    q.bad = n < 0 || n > a.R;
    q.nodes = max(0, min(n, a.R));
  }
  const int c = a.ctx_lens[s];
  q.none = c < 0 || (int64_t)c + q.nodes > (int64_t)a.cache.M_cap * a.cache.block_size;
  q.bad |= q.none;
  q.ctx = q.none ? 0 : c;
  return q;
}

// ---------------------------------------------------------------------------------
// Shared prefix: per prompt, the length in whole blocks that all N tables name alike and
// that every particle has as context.  A thread per block of the table, 16 particles' entries
// in flight: bound by the latency of those loads (32 prompts of 16 x 133 entries 5.1 us, 4 of
// 31 x 4665 entries 15 us).
// ---------------------------------------------------------------------------------
constexpr int kShareBlock = 1024;
constexpr int kShareLoads = 16;

__global__ __launch_bounds__(kShareBlock) void k_shared_len(TreeAttnArgs a, int32_t *__restrict__ out) {
  __shared__ int s_first, s_ctx;
  const int tid = threadIdx.x;
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    __syncthreads();
    if (tid == 0) {
      s_first = INT32_MAX;
      s_ctx = INT32_MAX;
    }
    __syncthreads();
    int least = INT32_MAX;
    for (int n = tid; n < a.N; n += kShareBlock) least = min(least, seq_of(a, b * a.N + n).ctx);
    if (least != INT32_MAX) atomicMin(&s_ctx, least);
    __syncthreads();
    const int slots = s_ctx / a.cache.block_size;
    const int32_t *T = a.cache.tables + (int64_t)b * a.N * a.cache.M_cap;
    int done = slots;
    for (int c0 = 0; c0 < slots; c0 += kShareBlock) {
      const int c = c0 + tid;
      if (c < slots) {
        const int32_t id = T[c];
        bool same = id >= 0 && id < a.cache.P;
        for (int n = 1; n < a.N && same; n += kShareLoads) {
#pragma unroll
          for (int u = 0; u < kShareLoads; ++u) same &= T[(int64_t)min(n + u, a.N - 1) * a.cache.M_cap + c] == id;
        }
        if (!same) atomicMin(&s_first, c);
      }
      __syncthreads();
      const int first = s_first;
      __syncthreads();  // read by every wave before the next blocks' mismatches are noted
      if (first != INT32_MAX) {
        done = first;
        break;
      }
    }
    if (tid == 0) {
      const int len = done * a.cache.block_size;
      out[b] = len >= kMinShared ? len : 0;
    }
  }
}

// ---------------------------------------------------------------------------------
// The main kernel
// ---------------------------------------------------------------------------------
// The sum and the maximum of a lane and the lane 32 away.
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

// A row's chunks are stored permuted: chunk c of row r in place c ^ place_of(r).  The row's
// two low bits move the place furthest, since the transposing read takes two chunks of four
// neighbouring rows, and any 16 rows (8 of 128 bytes) get different places, since a score
// reads one chunk of every row.
template <int CH>
__device__ __forceinline__ int place_of(int r) {
  return CH < 16 ? ((r & 2) << 1) | ((r >> 2) & 3) : ((r & 3) << 2) | ((r >> 2) & 3);
}

// A running maximum may fall behind by this much (a factor of 2^8) before O and l are
// rescaled: probabilities up to 256 lose nothing in either type, and most steps then
// rescale nothing.
constexpr float kLag = 8.0f;

__device__ const uint4 kNothing = {0, 0, 0, 0};  // loaded where there is nothing to load

// DP: head size padded to 64, 128 or 256.  NW: waves.
// Measured, bf16, heads of 128: 32 prompts of 16 x 5 rows x 32 heads over 2048 shared keys, the
// shared pass 143 us (600 TFLOP/s: bound by a wave's chain of product, exponentials and product;
// with idle waves in it, 150 us, its arithmetic alone took 112 and its loads alone 71) and the
// particles' own keys 66 us; 64 rows x 16 heads over 131,071 keys 111 us (620 TFLOP/s); 256 sequences of 9 x 32 heads over up
// to 4093 keys, 3.2 GB of pages, 608 us (5.4 TB/s: bound by the loads, which took as long without
// any arithmetic, whatever the pages' order and the bytes in flight); f16, heads of 64,
// one token of 4 sequences of 16 keys 5.6 us, all of it latency.
template <int DT, int DP, int NW, bool PREFIX>
__global__ __launch_bounds__(NW * kWave, DP == 256 ? 1 : NW == 4 && PREFIX ? 3 : 2) void k_attn(TreeAttnArgs a, Plan p) {
  typedef typename Half<DT>::V8 V8;
  typedef typename Half<DT>::V4 V4;
  constexpr int CH = DP / 8;       // 16-byte chunks of a row
  constexpr int RB = DP * 2;       // bytes of a row
  constexpr int NS = DP / 16;      // product steps of a score
  constexpr int NA = DP / 32;      // accumulator tiles of an output row
  constexpr int TB = KT * RB;      // bytes of a tile
  constexpr int RW = kWave / CH;             // rows of a wave's load
  constexpr int NLD = KT / (RW * NW);        // loads of keys (and as many of values) of a wave for a tile
  __shared__ __attribute__((aligned(16))) char sKV[2 * NB * TB];  // keys' buffers, then values'
  __shared__ uint32_t sOdd[PREFIX ? 1 : KT];  // a new token whose values are not all finite
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int hw = lane / 32, col = lane % 32;
  const Cut &cut = PREFIX ? p.prefix : p.suffix;

  // item: key/value head fastest (a page's heads lie together), then row tile, split, and
  // sequence (or prompt)
  uint32_t it = blockIdx.x;
  const int hk = (int)(it % (uint32_t)a.Hkv);
  it /= (uint32_t)a.Hkv;
  const int tile = (int)(it % (uint32_t)cut.tiles);
  it /= (uint32_t)cut.tiles;
  const int split = (int)(it % (uint32_t)cut.splits);
  const int unit = (int)(it / (uint32_t)cut.splits);
  const int s0 = PREFIX ? unit * a.N : unit;
  const int G = a.Hq / a.Hkv;

  Seq sq{0, 0, false, false};
  int lo = 0, hi, ctx;
  if (PREFIX) {
    hi = p.shared_len[unit];
    ctx = INT32_MAX;
    if (hi == 0) return;
  } else {
    sq = seq_of(a, s0);
    if (sq.bad && tid == 0 && hk == 0 && tile == 0 && split == 0) atomicOr(a.status, SMCSD_ST_BAD_INPUT);
    if (sq.nodes == 0) return;
    ctx = sq.ctx;
    hi = sq.none ? 0 : ctx + sq.nodes;
    lo = p.shared_len ? min(hi, p.shared_len[s0 / a.N]) : 0;
  }
  // this split's keys: an equal share in whole tiles
  const int per = (hi - lo + cut.splits - 1) / cut.splits;
  const int64_t share = (int64_t)((per + KT - 1) / KT) * KT;
  const int k0 = (int)min((int64_t)hi, lo + split * share), k1 = (int)min((int64_t)hi, k0 + share);

  // Staging, by loads that go straight to LDS, 64 chunks of 16 bytes in a row for a wave's
  // instruction: instruction i of a wave fills rows (i * NW + wave) * RW + lane / CH, place
  // lane % CH, which asks for chunk (lane % CH) ^ place_of(row).  Every wave looks up a tile's
  // rows itself, one to a lane (row lane % KT), and its lanes take their rows' places from
  // there.
  const int32_t *table = a.cache.tables + (int64_t)s0 * a.cache.M_cap;
  const uint16_t *const kbase = a.k_cache + (int64_t)hk * a.cache.head;
  const uint16_t *const vbase = a.v_cache + (int64_t)hk * a.cache.head;
  typedef __attribute__((address_space(3))) char lds_char;
  typedef __attribute__((address_space(3))) void lds_void;
  typedef __attribute__((address_space(1))) const void glb_void;
  lds_char *const lds = (lds_char *)sKV;
  // Block ids: lane i holds that of block id0 + i of the table, loaded again when a tile ends
  // past them, once in 64 blocks.  A load for each tile would be waited for together with the
  // tile that was asked for before it.
  int32_t ids = 0;
  int id0 = -kWave;
  bool bad_page = false;
  // Starts a tile's loads into buffer `buf`; which of its rows may be read.  Rows that may not
  // be, and the padding of a head, become 0, as what such a lane loads is (0 * NaN is no 0).
  auto fetch_tile = [&](int buf, int base) {
    if ((int)div_by(p.page, min(base + KT, k1) - 1) >= id0 + kWave) {
      id0 = div_by(p.page, base);
      ids = table[min(id0 + lane, (int)div_by(p.page, k1 - 1))];
      asm volatile("" : "+v"(ids));  // waited for here, not by every tile
    }
    const int pos = base + lane % KT, block = div_by(p.page, pos);
    const int32_t pg = __shfl(ids, min(block - id0, kWave - 1), kWave);
    const bool page_ok = pg >= 0 && pg < a.cache.P, ok = page_ok && pos < k1;
    bad_page |= !page_ok && pos < k1;
    const uint64_t rows = __ballot(ok);
    const int64_t off = ok ? pg * a.cache.page + (pos - block * (int)p.page.d) * a.cache.token : -1;
    constexpr int NAT = NLD < 4 ? NLD : 4;  // looked up together
    // Up to 64 rows are one workgroup's, and it alone reads its keys: past the caches (nt).  256
    // sequences of 9 x 32 heads, 3.2 GB, 608 us against 660, of one x 32 heads 577 against 628 (both
    // then with a wave to 32 rows), 16 of 30,000 keys 264 against 297; where particles share fewer than
    // kMinShared keys it costs (128 keys, 512 sequences: 70 against 67).  Four waves' rows may be
    // several workgroups', of the same keys: 64 x 16 heads over 131,071 keys took 134 us with it, 130
    // without.  From 65 to 128 rows four waves are one workgroup too, and lose 1 to 3 % by that (256
    // sequences of 17 x 32 heads 711 us, 690 past the caches).
    constexpr int kPolicy = NW < 4 ? 2 : 0;
#pragma unroll
    for (int i0 = 0; i0 < NLD; i0 += NAT) {
      int64_t at[NAT];
#pragma unroll
      for (int i = 0; i < NAT; ++i) at[i] = __shfl((long long)off, ((i0 + i) * NW + wave) * RW + lane / CH, kWave);
#pragma unroll
      for (int i = 0; i < NAT; ++i) {
        const int first = ((i0 + i) * NW + wave) * RW;
        const int chunk = (lane % CH) ^ place_of<CH>(first + lane / CH);
        const bool in = at[i] >= 0 && chunk * 8 < a.D;
        const uint16_t *const k = in ? kbase + at[i] + chunk * 8 : (const uint16_t *)&kNothing;
        const uint16_t *const v = in ? vbase + at[i] + chunk * 8 : (const uint16_t *)&kNothing;
        __builtin_amdgcn_global_load_lds((glb_void *)k, (lds_void *)(lds + buf * TB + first * RB), 16, 0, kPolicy);
        __builtin_amdgcn_global_load_lds((glb_void *)v, (lds_void *)(lds + (NB + buf) * TB + first * RB), 16, 0, kPolicy);
      }
    }
    return rows;
  };

  // this lane's query row
  const int r = tile * cut.tile_rows + wave * kRowsWave + col;
  const bool row_in = wave * kRowsWave + col < cut.tile_rows && r < cut.rows;
  int n = 0, j = 0, g = 0;
  if (row_in) {
    n = PREFIX ? r / (a.R * G) : 0;
    const int rest = r - n * a.R * G;
    j = rest / G;
    g = rest - j * G;
  }
  const int s = s0 + n;
  const int64_t orow = ((int64_t)s * a.R + j) * a.Hq + hk * G + g;  // row of out
  const bool live = row_in && (PREFIX || j < sq.nodes);
  uint64_t bits = 0;
  if (!PREFIX && live) {
    bits = a.tree_mask ? a.tree_mask[(int64_t)s * a.R + j] : (j >= 63 ? ~0ull : (2ull << j) - 1);
    if (sq.nodes < 64) bits &= (1ull << sq.nodes) - 1;
  }
  V8 q[NS];
  {
    const uint16_t *qp = a.q + ((int64_t)s * a.R + j) * a.q_stride + (int64_t)(hk * G + g) * a.D;
    const uint32_t flip = p.negate ? 0x80008000u : 0u;
#pragma unroll
    for (int st = 0; st < NS; ++st) {
      const int d = 16 * st + 8 * hw;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (live && d < a.D) w = *reinterpret_cast<const uint4 *>(qp + d);
      w.x ^= flip;
      w.y ^= flip;
      w.z ^= flip;
      w.w ^= flip;
      q[st] = __builtin_bit_cast(V8, w);
    }
  }
  f32x16 o[NA];
#pragma unroll
  for (int t = 0; t < NA; ++t) o[t] = f32x16{};
  float m = kNegInf, l = 0.0f;

  // What a tile in LDS needs where new tokens are among its rows: their values that are not
  // finite become 0: a probability of 0 then takes nothing from them, and the rows that do see
  // them get them after the last tile.
  constexpr uint32_t kExp = DT == SMCSD_DTYPE_BF16 ? 0x7F80u : 0x7C00u;
  auto finite = [&](uint32_t &w) {
    const uint32_t lo16 = (w & kExp) == kExp ? 0xFFFF0000u : ~0u;
    const uint32_t hi16 = (w & (kExp << 16)) == kExp << 16 ? 0xFFFFu : ~0u;
    w &= lo16 & hi16;
    return lo16 & hi16;
  };
  auto mend = [&](int buf, int base) {
#pragma unroll 1
    for (int i = 0; i < NLD; ++i) {
      const int row = (i * NW + wave) * RW + lane / CH;
      char *const v = sKV + (NB + buf) * TB + row * RB + lane % CH * 16;
      uint4 w = *reinterpret_cast<uint4 *>(v);
      const bool odd = (finite(w.x) & finite(w.y) & finite(w.z) & finite(w.w)) != ~0u && base + row >= ctx;
      const uint64_t any = __ballot(odd);
      if (odd) *reinterpret_cast<uint4 *>(v) = w;
      if (lane % CH == 0) sOdd[row] = (any >> lane) & ((1ull << CH) - 1) ? 1 : 0;
    }
  };

  // LDS offsets of a step's operands.  Keys: chunk 2 st + hw of row col.  Values: row 16h +
  // 8x + 4hw + i16/4, chunk 4t + 2dh + (i16%4)/2.  The permuted places depend on the low bits
  // of st, and of t and x; the rest are constants.
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
      va[t][x] = NB * TB + row * RB + ((4 * t + 2 * dh + (i16 % 4) / 2) ^ place_of<CH>(row)) * 16 + (i16 & 1) * 8;
    }

  // The scores of a tile's keys.
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
  auto scores = [&] {
    f32x16 z = f32x16{};
#pragma unroll
    for (int st = 0; st < NS; st += 4) {
      V8 kf[4];
      read_rows(kf, lds0 + ka[st % NKA], lds0 + ka[st % NKA + 1], lds0 + ka[st % NKA + 2], lds0 + ka[st % NKA + 3],
                (st / NKA) * 256);
#pragma unroll
      for (int i = 0; i < 4; ++i) z = Mma<DT>::run(kf[i], q[st + i], z);
    }
    return z;
  };
  // A tile's keys, from position `base` on; ok: which may be read.
  auto step = [&](int base, uint64_t ok) {
    auto sees = [&] {  // the tile's keys that this lane's row sees
      const int nb = ctx - base;  // so many of them are context
      uint32_t see = nb >= 32 ? 0xFFFFFFFFu : nb > 0 ? (1u << nb) - 1 : 0u;
      if (nb < 32) see |= nb >= 0 ? (uint32_t)(bits << nb) : (nb > -64 ? (uint32_t)(bits >> -nb) : 0u);
      return see & (uint32_t)ok;
    };
    f32x16 z = scores();
    if (ok != ~0ull || (!PREFIX && base + KT > ctx)) {
      asm volatile("");  // a branch, taken by few tiles: not to be computed by all
      const uint32_t mine = sees() >> (4 * hw);
#pragma unroll
      for (int i = 0; i < 16; ++i) z[i] = (mine >> (8 * (i / 4) + i % 4)) & 1 ? z[i] : kNegInf;
    }
    float top = z[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, z[i]);
    top = max_halves(top) * p.c;
    if (__any(top > m + kLag)) {
      const float mn = fmaxf(m, top);
      const float f = m == kNegInf ? 0.0f : fast_exp2(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int t = 0; t < NA; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[t][i] *= f;
    }
    const float ms = m == kNegInf ? 0.0f : m;
    V8 pr[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f32x8 e;
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = fast_exp2(fmaf(z[8 * h + i], p.c, -ms));
      l += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
      // rounded for the product, as the matrix instruction takes them; l sums them unrounded.  Against 64
      // bits that makes 0.0023 of relative error in bf16 where fp32 probabilities leave 0.0017
      pr[h] = __builtin_convertvector(e, V8);
      // values: keys 16h + 8x + 4hw + 0..3 for operand element 4x + 0..3 of product h
#pragma unroll
      for (int t = 0; t < NA; t += 2) {
        V8 vf[2];
        read_columns(vf, lds0 + va[t % NVT][0], lds0 + va[t % NVT][1], lds0 + va[t % NVT + 1][0], lds0 + va[t % NVT + 1][1],
                     16 * h * RB + (t / 4) * 256);
        o[t] = Mma<DT>::run(vf[0], pr[h], o[t]);
        o[t + 1] = Mma<DT>::run(vf[1], pr[h], o[t + 1]);
      }
    }
  };

  // Tile n is computed from buffer n % 2 while the next one is on its way.  A wave waits for
  // its own loads of tile n, then for the other waves, which are then also done with the buffer
  // that is filled next.
  uint64_t odd = 0;  // new tokens, by node, whose values are not all finite
  // a wave without rows only loads (of four, the last one of a tile of 96 rows among them)
  const bool busy = wave * kRowsWave < cut.tile_rows && tile * cut.tile_rows + wave * kRowsWave < cut.rows;
  if (k0 < k1) {
    uint64_t next_ok = fetch_tile(0, k0);
    int buf = 0;
    for (int base = k0; base < k1; base += KT) {
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      const uint64_t ok = next_ok;
      if (base + KT < k1) next_ok = fetch_tile(buf ^ 1, base + KT);
      __builtin_amdgcn_sched_barrier(0);  // the loads go out before, and nothing below moves up
      if (!PREFIX && base + KT > ctx) {
        mend(buf, base);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        const uint64_t rows = __ballot(lane < KT && sOdd[lane % KT]);
        odd |= base >= ctx ? rows << (base - ctx) : rows >> (ctx - base);
      }
      if (busy) step(base, ok);
      // the next buffer's offsets
      const int d = buf ? -TB : TB;
      buf ^= 1;
#pragma unroll
      for (int st = 0; st < NKA; ++st) ka[st] += d;
#pragma unroll
      for (int t = 0; t < NVT; ++t) {
        va[t][0] += d;
        va[t][1] += d;
      }
    }
  }
  while (!PREFIX && odd) {
    // of a value that is not finite any share is not finite either
    const int node = __builtin_ctzll(odd), pos = ctx + node;
    odd &= odd - 1;
    const int block = div_by(p.page, pos);
    const uint16_t *vp = vbase + table[block] * a.cache.page + (pos - block * (int)p.page.d) * a.cache.token;
    const bool seen = (bits >> node) & 1;
#pragma unroll
    for (int t = 0; t < NA; ++t)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int d = 32 * t + 8 * b + 4 * hw;
        uint16_t x[4] = {0, 0, 0, 0};
        if (d < a.D) *reinterpret_cast<uint2 *>(x) = *reinterpret_cast<const uint2 *>(vp + d);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          o[t][4 * b + c] += seen && (x[c] & kExp) == kExp ? (float)__builtin_bit_cast(typename Half<DT>::T, x[c]) : 0.0f;
      }
  }
  if (bad_page) atomicOr(a.status, SMCSD_ST_BAD_INPUT);
  l = sum_halves(l);

  // the row's part, or the row itself
  const int64_t rows = (int64_t)a.B * a.N * a.R * a.Hq;
  const int part = PREFIX ? split : p.prefix.splits + split;
  if (PREFIX || cut.splits > 1) {
    if (!live) return;
    float *ml = p.ml + 2 * (part * rows + orow);
    if (hw == 0) {
      ml[0] = m;
      ml[1] = l;
    }
    if (l == 0.0f) return;
    float *acc = p.acc + (part * rows + orow) * a.D;
#pragma unroll
    for (int t = 0; t < NA; ++t)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int d = 32 * t + 8 * b + 4 * hw;
        if (d < a.D)
          *reinterpret_cast<float4 *>(acc + d) =
              make_float4(o[t][4 * b], o[t][4 * b + 1], o[t][4 * b + 2], o[t][4 * b + 3]);
      }
    return;
  }
  if (!live) return;
  if (p.prefix.splits > 0 && lo > 0) {  // the prompt's shared part of this row
    for (int i = 0; i < p.prefix.splits; ++i) {
      const float mp = p.ml[2 * (i * rows + orow)], lp = p.ml[2 * (i * rows + orow) + 1];
      if (lp == 0.0f) continue;
      const float mn = fmaxf(m, mp);
      const float f = m == kNegInf ? 0.0f : fast_exp2(m - mn), fp = mp == kNegInf ? 0.0f : fast_exp2(mp - mn);
      const float *acc = p.acc + (i * rows + orow) * a.D;
      m = mn;
      l = l * f + lp * fp;
#pragma unroll
      for (int t = 0; t < NA; ++t)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int d = 32 * t + 8 * b + 4 * hw;
          if (d >= a.D) continue;
          const float4 x = *reinterpret_cast<const float4 *>(acc + d);
          o[t][4 * b] = o[t][4 * b] * f + x.x * fp;
          o[t][4 * b + 1] = o[t][4 * b + 1] * f + x.y * fp;
          o[t][4 * b + 2] = o[t][4 * b + 2] * f + x.z * fp;
          o[t][4 * b + 3] = o[t][4 * b + 3] * f + x.w * fp;
        }
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint16_t *out = a.out + orow * a.D;
#pragma unroll
  for (int t = 0; t < NA; ++t)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int d = 32 * t + 8 * b + 4 * hw;
      typedef float f32x4 __attribute__((ext_vector_type(4)));
      const f32x4 x = {o[t][4 * b] * inv, o[t][4 * b + 1] * inv, o[t][4 * b + 2] * inv, o[t][4 * b + 3] * inv};
      if (d < a.D)
        *reinterpret_cast<uint2 *>(out + d) = __builtin_bit_cast(uint2, __builtin_convertvector(x, V4));
    }
  if (a.lse && hw == 0)
    a.lse[orow] = l == 0.0f ? kNegInf : (float)(((double)m + (double)log2f(l)) * kLn2);
}

// ---------------------------------------------------------------------------------
// The parts of a row joined.  Groups of D/4 lanes (rounded up to a power of two) take a row's
// parts, `per` groups to a row, each every per-th of them, four loads in flight; their sums
// meet in LDS, in a fixed order.  Bound by reading the parts: 1024 rows x 64 parts of 128
// (34 MB) 12 us with 8 groups to a row; a wave per row, part after part, took 49.
// 21,168 rows x 4 parts of 96 took 13 us with one group to a row, 42 with 8.
// ---------------------------------------------------------------------------------
constexpr int kJoinBlock = 256;
inline int join_width(int D) { return D <= 64 ? 16 : D <= 128 ? 32 : 64; }

template <int DT>
__global__ __launch_bounds__(kJoinBlock) void k_attn_join(TreeAttnArgs a, Plan p, int64_t rows, int width, int per) {
  typedef typename Half<DT>::V4 V4;
  typedef float f32x4 __attribute__((ext_vector_type(4)));
  __shared__ f32x4 sums[kJoinBlock];
  const int tid = threadIdx.x, group = tid / width, wl = tid % width, d = 4 * wl;
  const int sub = group % per, some = kJoinBlock / width / per;  // this group's place, rows of a workgroup
  for (int64_t r0 = (int64_t)blockIdx.x * some; r0 < rows; r0 += (int64_t)gridDim.x * some) {
    const int64_t r = min(r0 + group / per, rows - 1);
    const int64_t t = r / a.Hq;
    const int s = (int)(t / a.R), j = (int)(t - (int64_t)s * a.R);
    const bool live = r0 + group / per < rows && j < seq_of(a, s).nodes;
    const int first = p.prefix.splits > 0 && p.shared_len[s / a.N] > 0 ? 0 : p.prefix.splits;
    const int parts = live ? p.prefix.splits + p.suffix.splits : 0;
    auto stat = [&](int i) { return *reinterpret_cast<const float2 *>(p.ml + 2 * (i * rows + r)); };
    float m = kNegInf;
    for (int i = first + wl; i < parts; i += width) {
      const float2 ml = stat(i);
      m = ml.y != 0.0f ? fmaxf(m, ml.x) : m;
    }
    for (int o = width / 2; o > 0; o /= 2) m = fmaxf(m, __shfl_xor(m, o, kWave));
    auto factor = [&](float2 ml) { return ml.y == 0.0f || ml.x == kNegInf ? 0.0f : fast_exp2(ml.x - m); };
    float l = 0.0f;
    for (int i = first + wl; i < parts; i += width) {
      const float2 ml = stat(i);
      l = fmaf(ml.y, factor(ml), l);
    }
    for (int o = width / 2; o > 0; o /= 2) l += __shfl_xor(l, o, kWave);
    f32x4 acc = {};
#pragma unroll 4
    for (int i = first + sub; i < parts; i += per) {
      const float2 ml = stat(i);
      const float f = factor(ml);
      // an empty part is not written: what lies there is not used
      const f32x4 x = *reinterpret_cast<const f32x4 *>(p.acc + (i * rows + r) * a.D + (d < a.D ? d : 0));
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c] = ml.y != 0.0f ? fmaf(x[c], f, acc[c]) : acc[c];
    }
    if (per > 1) {
      sums[tid] = acc;
      __syncthreads();
      if (sub == 0)
        for (int g = 1; g < per; ++g) acc += sums[g * width + tid];
      __syncthreads();
    }
    if (sub > 0 || !live) continue;
    acc *= l == 0.0f ? 0.0f : 1.0f / l;
    if (d < a.D)
      *reinterpret_cast<uint2 *>(a.out + r * a.D + d) = __builtin_bit_cast(uint2, __builtin_convertvector(acc, V4));
    if (a.lse && wl == 0) a.lse[r] = l == 0.0f ? kNegInf : (float)(((double)m + (double)log2f(l)) * kLn2);
  }
}

template <int DT, int DP, bool PREFIX>
void launch_part(const TreeAttnArgs &a, const Plan &p, hipStream_t stream) {
  const Cut &c = PREFIX ? p.prefix : p.suffix;
  const int64_t units = PREFIX ? a.B : (int64_t)a.B * a.N;
  const dim3 grid((unsigned)(units * c.splits * c.tiles * a.Hkv)), block(c.waves * kWave);
  if (c.waves == 2)
    hipLaunchKernelGGL((k_attn<DT, DP, 2, PREFIX>), grid, block, 0, stream, a, p);
  else
    hipLaunchKernelGGL((k_attn<DT, DP, 4, PREFIX>), grid, block, 0, stream, a, p);
}

template <int DT, int DP>
void launch_dp(const TreeAttnArgs &a, const Plan &p, int32_t *shared_len, hipStream_t stream) {
  const int64_t rows = (int64_t)a.B * a.N * a.R * a.Hq;
  if (p.prefix.splits > 0) {
    hipLaunchKernelGGL(k_shared_len, dim3(grid_blocks(a.B, kShareBlock)), dim3(kShareBlock), 0, stream, a, shared_len);
    launch_part<DT, DP, true>(a, p, stream);
  }
  launch_part<DT, DP, false>(a, p, stream);
  if (p.suffix.splits > 1) {
    // four parts or more to a group
    const int width = join_width(a.D), parts = p.prefix.splits + p.suffix.splits;
    int per = 1;
    while (per < kJoinBlock / width && 8 * per <= parts) per *= 2;
    hipLaunchKernelGGL(k_attn_join<DT>, dim3(grid_blocks(ceil_div(rows * per * width, kJoinBlock), kJoinBlock)),
                       dim3(kJoinBlock), 0, stream, a, p, rows, width, per);
  }
}

}  // namespace

// Workspace: [shared lengths int32 x B][(max, sum) x parts x rows][O fp32 x parts x rows x D], with
// parts bounded by the splits that S*Hkv heads of R rows or more (B*Hkv heads of N*R or more) can ask
// for; N > 1 particles may share a prefix, which only the tables tell.  rows*2 <= rows*D / 4.
size_t tree_attn_ws_bytes(int64_t B, int64_t N, int R, int64_t HqD, int64_t Hkv) {
  const int64_t S = B * N;
  const int ss = max_splits(S * Hkv, R), sp = N > 1 ? max_splits(B * Hkv, N * R) : 0;
  const size_t floats = (size_t)((ss > 1 ? ss : 0) + sp) * (size_t)(S * R) * (size_t)HqD;
  return align256(sizeof(int32_t) * (size_t)std::max<int64_t>(B, 1)) + align256(sizeof(float) * (floats / 4)) +
         align256(sizeof(float) * floats);
}

hipError_t launch_tree_attn(const TreeAttnArgs &a, int dtype, hipStream_t stream) {
  const int DP = pad_dim(a.D);
  const int64_t S = (int64_t)a.B * a.N, cap = (int64_t)a.cache.M_cap * a.cache.block_size;
  const int64_t longest = a.max_len > 0 ? std::min(a.max_len, cap) : cap;
  const int G = a.Hq / a.Hkv;
  Plan p{};
  p.page = fast_div((uint32_t)a.cache.block_size);
  p.suffix = cut_of(a.R * G, S * a.Hkv, longest);
  if (a.N > 1 && longest > kMinShared) p.prefix = cut_of(a.N * a.R * G, (int64_t)a.B * a.Hkv, longest);
  const int parts = p.prefix.splits + (p.suffix.splits > 1 ? p.suffix.splits : 0);
  const int64_t rows = S * a.R * a.Hq;
  int32_t *shared_len = reinterpret_cast<int32_t *>(a.ws);
  char *at = a.ws + align256(sizeof(int32_t) * (size_t)a.B);
  if (p.prefix.splits > 0) p.shared_len = shared_len;
  p.ml = reinterpret_cast<float *>(at);
  p.acc = reinterpret_cast<float *>(at + align256(sizeof(float) * 2 * (size_t)(parts * rows)));
  p.c = std::max(std::fabs(a.scale) * 1.44269504088896340736f, 1e-30f);
  p.negate = a.scale < 0.0f;
  if (dtype == SMCSD_DTYPE_BF16) {
    if (DP == 64) launch_dp<SMCSD_DTYPE_BF16, 64>(a, p, shared_len, stream);
    else if (DP == 128) launch_dp<SMCSD_DTYPE_BF16, 128>(a, p, shared_len, stream);
    else launch_dp<SMCSD_DTYPE_BF16, 256>(a, p, shared_len, stream);
  } else {
    if (DP == 64) launch_dp<SMCSD_DTYPE_F16, 64>(a, p, shared_len, stream);
    else if (DP == 128) launch_dp<SMCSD_DTYPE_F16, 128>(a, p, shared_len, stream);
    else launch_dp<SMCSD_DTYPE_F16, 256>(a, p, shared_len, stream);
  }
  return hipGetLastError();
}

}  // namespace smcsd
