// Attention over the 8-bit key/value cache.
//
// A row is one query token and head; the g = heads / kv_heads heads that share a key/value head
// are rows of one product, row r = i g + (head mod g). With codes c, block scales s_k, s_v and
// the exponent in base 2,
//   e_rt = (scale log2 e) s_k (q_r . c_k,t),   out_r = sum_t 2^e_rt s_v c_v,t / sum_t 2^e_rt.
// One pass over the tokens keeps, for each row, the running maximum m of e_rt + log2 s_v, the
// sum of weights w_rt = 2^(e_rt + log2 s_v - m) times the codes, and the sum of w_rt / s_v: the
// value scale rides in the exponent, so every weight is in [0, 1] and no product is scaled.
//
// Precision: the products run on float16 MFMA with float32 sums. A code is exact in float16. A
// row of q is first multiplied by the power of two that takes its largest entry to [2^14, 2^15):
// a bf16 entry is then exact (entries 2^-38 of the row's largest are dropped), a float32 entry is
// a sum of two float16 pieces, off by 2^-22 of itself, a float32 sum's own error over 64 terms or
// more. Weights are held times 2^14 and rounded to float16 (2^-11, against the 2^-8 of a bf16
// output), for float32 outputs to two pieces; in bf16 prompts m may lag by 2^4 and they are held
// times 2^11. Maxima, sums and accumulators are float32.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "cache_internal.h"

namespace kq {
namespace {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));

constexpr int kTokenWaves = 8;          // waves that share a workgroup's range of the context
constexpr float kNoToken = -3.0e38f;   // running maximum before the first token (finite: no inf - inf)
constexpr float kZeroScale = -48.0f;   // log2 taken for a value scale of 0: any finite one (its codes are 0)
constexpr float kWeightExp = 14.0f;    // weights are held times 2^14, so that float16 keeps small ones
// Exponents are one fused multiply-add from the scores, e f + (log2 s_v - m), exact but for the rounding of m. Where
// m is larger than this, that rounding counts (2^-2 here, and a weight of 2^2 would pass float16's range): the
// exponent is then rounded as m is, before m is taken off, so that the largest is 0.
constexpr float kFarMax = 4194304.0f;

struct AttnArgs {
  SeqArgs seq;
  const int8_t* k;
  const int8_t* v;
  const float* k_scale;
  const float* v_scale;
  const void* q;
  int64_t ldq;
  void* out;
  int64_t ldo;
  int heads, kvh, g;
  float scale_log2e;
  int window;
  int batch, tiles, tile_rows, splits;
  int longest_first;  // take the sequences by length (batch <= 64)
  float* part_o;    // [rows * heads][splits][D], sum of weights (times 2^14) times codes
  float* part_ml;   // [rows * heads][splits][2]: m, sum of weights (times 2^14) / s_v
};

// Four signed bytes to two pairs of float16: bytes b + 128 become the low byte of float16 1024 + b + 128.
__device__ __forceinline__ void unpack4(uint32_t w, half2v& lo, half2v& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const half2v bias = {_Float16(-1152.0f), _Float16(-1152.0f)};
  lo = __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) + bias;
  hi = __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) + bias;
}

__device__ __forceinline__ half8 unpack8(uint32_t w0, uint32_t w1) {
  half2v a, b, c, d;
  unpack4(w0, a, b);
  unpack4(w1, c, d);
  return half8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

template <bool BF16>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&f)[8]) {
  if (BF16) {
    const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + at);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float4 a = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + at)[0];
    const float4 b = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + at)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
}

template <bool BF16>
__device__ __forceinline__ void store4(void* p, int64_t at, float a, float b, float c, float d) {
  if (BF16) {
    uint2 u;
    u.x = pack_bf16(a, b);
    u.y = pack_bf16(c, d);
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p) + at) = u;
  } else {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + at) = make_float4(a, b, c, d);
  }
}

// Power of two that takes amax to [2^14, 2^15) (1 for a row of zeros), and its inverse; a row
// with a NaN or an infinity is multiplied by NaN, which reaches all of its scores.
__device__ __forceinline__ void row_scale(float amax, float& up, float& down) {
  int e;
  (void)frexpf(amax, &e);  // amax = f 2^e, f in [0.5, 1)
  e = amax > 0.0f ? min(max(15 - e, -126), 126) : 0;
  up = amax < INFINITY ? ldexpf(1.0f, e) : NAN;
  down = ldexpf(1.0f, -e);
}

__device__ __forceinline__ float exp2_raw(float x) { return __builtin_amdgcn_exp2f(x); }

// Maximum over the lanes l and l + 32, in both.
__device__ __forceinline__ float across_halves_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// The sequence that is k-th longest (ties: the lower one first). A prompt's workgroups start in order, and the last
// to start should not be the longest: four pieces of prompts of 325 to 1000 tokens on 4682 to 16001, float32,
// 1335 us in the batch's order, 895 by length (228 tiles a CU on average). Single tokens gained nothing (475 us
// against 469).
__device__ __forceinline__ int by_length(const AttnArgs& a, int k) {
  if (!a.longest_first) return k;
  const int lane = threadIdx.x & 63;
  const int len = lane < a.batch ? a.seq.seq_lens[lane] : 0;
  int rank = lane < a.batch ? 0 : 64;
  for (int i = 0; i < a.batch; ++i) {
    const int other = __builtin_amdgcn_readlane(len, i);
    rank += other > len || (other == len && i < lane);
  }
  return __builtin_ctzll(__ballot(rank == k));
}

// This split's share [c0, c1) of the 64-token chunks that a tile of rows sees, the first and last 16-token
// groups of the whole tile (what lies outside is never looked up), and in how many parts the tile is split: a
// tile of one part is written by its workgroup, the others' parts are joined.
struct Range {
  int c0, c1, g0, g1, parts;
};

__device__ __forceinline__ Range chunk_range(const AttnArgs& a, const Seq& s, int i_first, int i_last, int split) {
  const int p_last = s.len - s.n + i_last, p_first = s.len - s.n + i_first;
  if (p_last < 0) return Range{0, 0, 0, 0, 1};
  const int low = a.window > 0 ? int(max(int64_t(0), int64_t(p_first) - a.window + 1)) : 0;
  const int c = low >> 6, n = (p_last >> 6) + 1 - c;
  const int per = max((n + a.splits - 1) / a.splits, 8);   // single tokens: a chunk for each wave
  const int c0 = min(c + split * per, c + n);
  return Range{c0, min(c0 + per, c + n), low >> 4, p_last >> 4, (n + per - 1) / per};
}

// ---------------------------------------------------------------------------
// A few rows a sequence: single tokens, drafts
//
// A workgroup takes 16 rows of one sequence and head and a range of the context; its waves
// take the range's 64-token chunks in turn and never share data before the end, where their
// partial sums are joined in LDS. Nothing is staged: each operand comes from the cache in the
// order its MFMA wants it. S^T = K Q^T has tokens as rows: lane (lk = lane / 16, li = lane mod 16)
// gets rows 4 lk + j of each 16-token product. Which token a row is, is free: row 4 lk + j of
// product i is token 16 lk + 4 i + j, so a lane ends up with 16 consecutive tokens, all of one
// cache block, and they are its operand of O^T = V^T P^T, whose other operand is 16 codes of one
// channel: one 16-byte load. Channels are permuted likewise so that a key row's loads are 16
// bytes a lane.
//
// Bound by HBM where the context is long: 64 tokens over up to 8191, 32 heads each (2.6 GB of
// codes), 461 us, 5.7 TB/s; one token over 131070, 64 over 8 heads (268 MB), 51 us, and 4 to join
// its parts. Short ones are latency: 300 tokens, 7.9 us. Eight waves a workgroup, joined in LDS,
// and one workgroup a CU leave half the parts to join from memory that four waves and two
// workgroups do (131070 tokens 54.9 us and 61.5, 300 tokens 8.2 and 8.7).
// ---------------------------------------------------------------------------
template <bool BF16, int D>
__global__ __launch_bounds__(kTokenWaves * 64, 2) void cache_token_kernel(AttnArgs a) {
  constexpr int W = kTokenWaves;
  constexpr int U = D / 64;       // 16-byte key loads a lane and token row
  constexpr int DT = D / 16;      // 16-channel tiles of the output
  constexpr int PITCH = D + 4;
  __shared__ float sh_o[W][16 * PITCH];
  __shared__ float sh_m[W][16], sh_l[W][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int li = lane & 15, lk = lane >> 4;
  int64_t id = blockIdx.x;
  const int nbh = a.batch * a.kvh;
  const int bh = id % nbh;
  id /= nbh;
  const int tile = id % a.tiles, split = id / a.tiles;
  const int b = bh / a.kvh, kh = bh - b * a.kvh;
  const Seq s = sequence(a.seq, b, kh == 0 && tile == 0 && split == 0 && threadIdx.x == 0);
  const int nrows = s.n * a.g;
  if (tile * 16 >= nrows) return;
  const int first = s.len - s.n;
  const int r = min(tile * 16 + li, nrows - 1);   // this lane's row (repeats past the last)
  const int i = r / a.g, hd = kh * a.g + (r - i * a.g);
  const int p = first + i;                         // its position
  const int i_first = tile * 16 / a.g, i_last = (min(tile * 16 + 16, nrows) - 1) / a.g;
  const Range rg = chunk_range(a, s, i_first, i_last, split);
  if (split >= rg.parts) return;
  // every token of a chunk is seen by every row if it lies in (p_last - window, p_first]
  const int p_first = first + i_first, p_last = first + i_last;

  const int page = 1 << a.seq.page_log2, pmask = page - 1;

  // Codes are loaded into the registers of the chunk before as soon as its products have used them, their pages
  // looked up a chunk earlier still.
  int idk = 0, idv = 0, offk = 0, offv = 0;
  uint4 kc[4][U], vc[DT];
  float ks = 0.0f, vs = 0.0f;
  bool lost = false;
  auto look = [&](int c) {
    // 16-token groups of this lane: of its key rows, and of its weights and values
    const int gk = min(max(4 * c + (li >> 2), rg.g0), rg.g1), gv = min(max(4 * c + lk, rg.g0), rg.g1);
    idk = table_entry(a.seq, b, gk << 4);
    idv = table_entry(a.seq, b, gv << 4);
    offk = (gk << 4) & pmask;
    offv = (gv << 4) & pmask;
  };
  auto load_keys = [&] {
    const int64_t blk = int64_t(is_page(a.seq, idk) ? idk : 0) * a.kvh + kh;
    const int8_t* const kp = a.k + (blk * page + offk) * D + (li & 3) * D + 16 * lk;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int u = 0; u < U; ++u) kc[t][u] = *reinterpret_cast<const uint4*>(kp + 4 * t * D + 64 * u);
  };
  auto load_values = [&] {
    const int64_t blk = int64_t(is_page(a.seq, idv) ? idv : 0) * a.kvh + kh;
    const int8_t* const vp = a.v + (blk * page + offv) * D + 16 * li;
    ks = a.k_scale[blk];
    vs = a.v_scale[blk];
#pragma unroll
    for (int t = 0; t < DT; ++t) vc[t] = *reinterpret_cast<const uint4*>(vp + 256 * t);
  };
  // The first chunk's table entries, the queries and the chunk's codes are under way before the queries are waited for.
  // A wave without a chunk loads what the others do.
  int c = rg.c0 + wave;
  look(c);
  // the row of q; its float16 pieces are in the channel order of the key loads
  float qx[2 * U][8];
  {
    const int64_t at = (int64_t(s.row0) + i) * a.ldq + int64_t(hd) * D;
#pragma unroll
    for (int t = 0; t < 2 * U; ++t) load8<BF16>(a.q, at + 64 * (t >> 1) + 16 * lk + 8 * (t & 1), qx[t]);
  }
  load_keys();
  load_values();
  bool known = is_page(a.seq, idv);              // whether this lane's block is a page, for the chunk in registers
  look(c + W);
  half8 qh[2 * U], ql[BF16 ? 1 : 2 * U];
  float down;
  {
    float amax = 0.0f, odd = 0.0f;
#pragma unroll
    for (int t = 0; t < 2 * U; ++t)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        amax = fmaxf(amax, fabsf(qx[t][j]));
        odd = fmaf(qx[t][j], 0.0f, odd);         // NaN once an entry is not finite
      }
    amax = odd == odd ? amax : INFINITY;
    amax = fmaxf(amax, __shfl_xor(amax, 16));
    amax = fmaxf(amax, __shfl_xor(amax, 32));
    float up;
    row_scale(amax, up, down);
#pragma unroll
    for (int t = 0; t < 2 * U; ++t)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float y = qx[t][j] * up;
        const _Float16 h = _Float16(y);
        qh[t][j] = h;
        if (!BF16) ql[t][j] = _Float16(y - float(h));
      }
  }
  const float qf = a.scale_log2e * down;

  floatx4 o[DT];
#pragma unroll
  for (int t = 0; t < DT; ++t) o[t] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  float m = kNoToken, l = 0.0f;
  // one chunk; every load is unconditional, so that the waits count those that are still out
  auto chunk = [&](int c, auto more) {
    floatx4 e[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      e[t] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const half8 k0 = unpack8(kc[t][u].x, kc[t][u].y), k1 = unpack8(kc[t][u].z, kc[t][u].w);
        e[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, qh[2 * u], e[t], 0, 0, 0);
        e[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, qh[2 * u + 1], e[t], 0, 0, 0);
        if (!BF16) {
          e[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, ql[2 * u], e[t], 0, 0, 0);
          e[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, ql[2 * u + 1], e[t], 0, 0, 0);
        }
      }
    }
    if constexpr (more) load_keys();
    lost |= !known;
    const float kscale = known ? ks : NAN, vscale = known ? vs : NAN;
    float f = kscale * qf;                                     // scores to base-2 exponents
    const float lv = vscale > 0.0f ? __log2f(vscale) : vscale == 0.0f ? kZeroScale : NAN;
    const float iv = vscale == 0.0f ? 0x1p48f : __builtin_amdgcn_rcpf(vscale);   // a unit of float32 off
    const int t0 = 64 * c + 16 * lk;                           // this lane's first token
    const bool cut = 64 * c + 63 > p_first || (a.window > 0 && 64 * c <= p_last - a.window);
    const int hi = p - t0, lo = a.window > 0 && hi >= 0 ? hi - a.window : -1;  // tokens x in (lo, hi] are seen
    if (cut) {
#pragma unroll
      for (int x = 0; x < 16; ++x) e[x >> 2][x & 3] = (x <= hi && x > lo) ? e[x >> 2][x & 3] : -INFINITY;
    }
    float mx = fmaxf(fmaxf(e[0][0], e[0][1]), fmaxf(e[0][2], e[0][3]));
#pragma unroll
    for (int t = 1; t < 4; ++t) mx = fmaxf(mx, fmaxf(fmaxf(e[t][0], e[t][1]), fmaxf(e[t][2], e[t][3])));
    mx = fmaf(mx, f, lv);   // f >= 0; a NaN (f NaN, or 0 with nothing seen) is dropped by the next maximum
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const float mn = fmaxf(m, mx);
    const float fall = exp2_raw(m - mn);
    m = mn;
    l *= fall;
#pragma unroll
    for (int t = 0; t < DT; ++t) o[t] *= fall;
    float shift = lv - m + kWeightExp;
    if (__any(fabsf(m) > kFarMax)) {
#pragma unroll
      for (int x = 0; x < 16; ++x) e[x >> 2][x & 3] = fmaf(e[x >> 2][x & 3], f, lv) - m;
      f = 1.0f;
      shift = kWeightExp;
    }
    float sum = 0.0f;
    float w[16];
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      w[x] = exp2_raw(fmaf(e[x >> 2][x & 3], f, shift));
      if (cut) w[x] = (x <= hi && x > lo) ? w[x] : 0.0f;       // also where a block's scale is NaN
      sum += w[x];
    }
    l += sum == 0.0f ? 0.0f : sum * iv;
    half8 ph[2], pl[2];
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      const _Float16 h = _Float16(w[x]);
      ph[x >> 3][x & 7] = h;
      if (!BF16) pl[x >> 3][x & 7] = _Float16(w[x] - float(h));
    }
#pragma unroll
    for (int t = 0; t < DT; ++t) {
      const half8 v0 = unpack8(vc[t].x, vc[t].y), v1 = unpack8(vc[t].z, vc[t].w);
      o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, ph[0], o[t], 0, 0, 0);
      o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, ph[1], o[t], 0, 0, 0);
      if (!BF16) {
        o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pl[0], o[t], 0, 0, 0);
        o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pl[1], o[t], 0, 0, 0);
      }
    }
    if constexpr (more) {
      load_values();
      known = is_page(a.seq, idv);
      look(c + 2 * W);
    }
  };
  if (c < rg.c1) {
    for (; c + W < rg.c1; c += W) chunk(c, std::true_type{});
    chunk(c, std::false_type{});
  }
  if (lost) report(a.seq.info, KQ_INFO_PAGE);
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
#pragma unroll
  for (int t = 0; t < DT; ++t) *reinterpret_cast<floatx4*>(&sh_o[wave][li * PITCH + 16 * t + 4 * lk]) = o[t];
  if (lk == 0) {
    sh_m[wave][li] = m;
    sh_l[wave][li] = l;
  }
  __syncthreads();
  // join the waves: D / 4 threads a row
  const int q = threadIdx.x / (D / 4), d = (threadIdx.x % (D / 4)) * 4;
  if (q >= 16 || tile * 16 + q >= nrows) return;
  float mj = sh_m[0][q];
#pragma unroll
  for (int w = 1; w < W; ++w) mj = fmaxf(mj, sh_m[w][q]);
  floatx4 x = {0.0f, 0.0f, 0.0f, 0.0f};
  float lj = 0.0f;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const float fw = exp2_raw(sh_m[w][q] - mj);
    lj += fw * sh_l[w][q];
    x += fw * *reinterpret_cast<const floatx4*>(&sh_o[w][q * PITCH + d]);
  }
  const int rq = tile * 16 + q, iq = rq / a.g;
  const int64_t row = int64_t(s.row0) + iq;
  const int head = kh * a.g + (rq - iq * a.g);
  if (rg.parts == 1) {
    const float inv = lj == 0.0f ? 0.0f : 1.0f / lj;
    store4<BF16>(a.out, row * a.ldo + int64_t(head) * D + d, x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
  } else {
    const int64_t at = (row * a.heads + head) * a.splits + split;
    *reinterpret_cast<floatx4*>(a.part_o + at * D + d) = x;
    if (d == 0) *reinterpret_cast<float2*>(a.part_ml + at * 2) = make_float2(mj, lj);
  }
}

// ---------------------------------------------------------------------------
// Prompts
//
// A workgroup takes 256 rows of one sequence and head, eight waves of 32, and walks the context in tiles of 64
// tokens. The codes of a tile are loaded and unpacked to float16 once a workgroup, into LDS, three tiles deep:
// unpacking takes five vector instructions for four codes and is the cost that many rows have to share. Where 256 rows
// a workgroup would leave CUs idle it takes 128, and two waves share 32 rows by halves of each tile.
//
// What bounds it is the SIMDs' vector issue, not the matrix pipe (measured on an 8192-token prompt over 32 heads):
// a 32 x 32 x 16 MFMA keeps the matrix pipe busy for 32 cycles and the issue port for about 12 of them, an
// exponential takes the port for 16, the others for 4. Removing the unpacking alone, or the exponentials alone,
// saved a sixth of the time each. So the instructions around a score are few: one fused multiply-add (the block's
// scales and the maximum are its operands), the exponential, an addition and half a conversion; the maximum is
// taken by threes; the accumulators are rescaled only when the maximum has grown by 2^4; one wave in turn prepares
// a tile's scales. MFMAs and vector instructions of one wave alternate (half a tile's weights with the other
// half's scores).
// ---------------------------------------------------------------------------

// A block's scales as the weights use them, finite where they multiply scores. A NaN (a poisoned block, a bad
// page) becomes a weight of 2^100 for whoever sees a token of it, and a NaN in their sum.
struct alignas(16) BlockScale {
  float ks, lv, iv;
};

__device__ __forceinline__ BlockScale block_scale(float ks, float vs) {
  const bool bad = !(ks == ks && vs == vs);
  BlockScale r;
  r.ks = bad ? 0x1p-100f : ks > 0.0f ? ks : 1.0f;            // 0: the codes are 0, so any factor will do
  r.lv = bad ? 100.0f : vs > 0.0f ? __log2f(vs) : kZeroScale;
  r.iv = bad ? NAN : vs > 0.0f ? __builtin_amdgcn_rcpf(vs) : 0x1p48f;   // the reciprocal a unit of float32 off
  return r;
}

template <bool BF16, int D, int ROWS>
__global__ __launch_bounds__(512, 2) void cache_prompt_kernel(AttnArgs a) {
  constexpr int NT = 512, GROUPS = ROWS / 32;    // groups of rows
  constexpr bool PAIRS = GROUPS < 8;             // two waves share a group's rows, each takes half of a tile's tokens
  constexpr int KS = D / 16, DT = D / 32;        // MFMA steps over channels, 32-channel output tiles
  // LDS rows in 16-byte units, of an odd number of them so that lanes reading one unit of consecutive rows meet
  // different banks, and every step's address is a constant away from the lane's first. Keys: the token of the
  // product's row r in place r, values: by channel.
  constexpr int KP = D / 8 + 1, VP = 9;
  constexpr int KB = 64 * KP, VB = D * VP;       // units of a tile
  constexpr int CH = 8 * D / NT;                 // 16-byte chunks of codes a thread stages (keys, then values)
  constexpr int P = BF16 ? 1 : 2;                // float16 pieces of a query and a weight
  // The running maximum of a bf16 row may lag by 2^4, so that accumulators are seldom rescaled; weights, held
  // times 2^11, then stay below 2^15. A float32 row's never lags.
  constexpr float kLag = BF16 ? 4.0f : 0.0f, kExp = BF16 ? 11.0f : 14.0f;
  __shared__ half8 sk[3 * KB];
  __shared__ half8 sv[3 * VB];
  __shared__ BlockScale sc[4][4];                // of a tile's four 16-token groups
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6) & 7;
  const int lq = lane & 31, lh = lane >> 5;
  int64_t id = blockIdx.x;
  const int kh = id % a.kvh;                     // a head's workgroups run on one XCD and share its tiles in L2
  id /= a.kvh;
  const int tile = a.tiles - 1 - int(id % a.tiles);   // the longest first
  id /= a.tiles;
  const int b = by_length(a, id % a.batch), split = id / a.batch;
  const Seq s = sequence(a.seq, b, kh == 0 && tile == 0 && split == 0 && tid == 0);
  const int nrows = s.n * a.g;
  if (tile * ROWS >= nrows) return;
  const int first = s.len - s.n;
  const Range rg = chunk_range(a, s, tile * ROWS / a.g, (min(tile * ROWS + ROWS, nrows) - 1) / a.g, split);
  if (split >= rg.parts) return;

  // this wave's rows, a lane's row and its position
  const int wh = PAIRS ? wave / GROUPS : 0;      // this wave's half of the tokens
  const int w0 = tile * ROWS + (wave & (GROUPS - 1)) * 32;
  const int p_hi = w0 < nrows ? first + (min(w0 + 32, nrows) - 1) / a.g : -1, p_lo = first + min(w0, nrows - 1) / a.g;
  const int r = min(w0 + lq, nrows - 1);
  const int i = r / a.g, head = kh * a.g + (r - i * a.g);
  const int pos = first + i;
  half8 qf[P][KS];
  float fq;
  {
    const int64_t at = (int64_t(s.row0) + i) * a.ldq + int64_t(head) * D + 8 * lh;
    float amax = 0.0f, odd = 0.0f;
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      float x[8];
      load8<BF16>(a.q, at + 16 * t, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        amax = fmaxf(amax, fabsf(x[j]));
        odd = fmaf(x[j], 0.0f, odd);             // NaN once an entry is not finite
      }
    }
    amax = odd == odd ? amax : INFINITY;
    amax = fmaxf(amax, __shfl_xor(amax, 32));
    float up, down;
    row_scale(amax, up, down);
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      float x[8];
      load8<BF16>(a.q, at + 16 * t, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float y = x[j] * up;
        const _Float16 h = _Float16(y);
        qf[0][t][j] = h;
        if (!BF16) qf[P - 1][t][j] = _Float16(y - float(h));
      }
    }
    fq = a.scale_log2e * down;
  }

  // Staging: chunk x < 4 D of keys (token x / (D / 16), 16 channels), then of values (group, channel); a wave's
  // chunks are all of one 16-token group, D chunks of either side. The table's entries are loaded a tile before
  // the codes and scales that they lead to, those a tile before they are unpacked.
  uint4 raw[CH];
  int entry[CH];
  bool lost = false;                             // an entry of the table that is no page (told at the end)
  const int page = 1 << a.seq.page_log2;
  auto group = [&](int c, int x) { return min(max(4 * c + x, rg.g0), rg.g1); };
  auto of_keys = [&](int n) { return NT * (n + 1) <= 4 * D || (NT * n < 4 * D && wave * 64 + NT * n < 4 * D); };
  auto chunk_group = [&](int n) { return ((wave * 64 + NT * n) & (4 * D - 1)) / D; };
  auto look = [&](int c) {
#pragma unroll
    for (int n = 0; n < CH; ++n) entry[n] = table_entry(a.seq, b, group(c, chunk_group(n)) << 4);
  };
  auto fetch = [&](int c) {
#pragma unroll
    for (int n = 0; n < CH; ++n) {
      const int pg = __builtin_amdgcn_readfirstlane(entry[n]);
      const int64_t at = (int64_t(is_page(a.seq, pg) ? pg : 0) * a.kvh + kh) * (int64_t(page) * D) +
                         ((group(c, chunk_group(n)) << 4) & (page - 1)) * D;
      raw[n] = *reinterpret_cast<const uint4*>((of_keys(n) ? a.k : a.v) + at + 16 * ((tid + NT * n) & (D - 1)));
    }
  };
  // The scales of a tile are one wave's work, in turn: four groups in its lanes, the same three steps.
  int entry_s = 0;
  float2 rscale = make_float2(1.0f, 1.0f);
  auto look_s = [&](int c) { entry_s = table_entry(a.seq, b, group(c, lane & 3) << 4); };
  auto fetch_s = [&] {
    const bool ok = is_page(a.seq, entry_s);
    const int64_t at = int64_t(ok ? entry_s : 0) * a.kvh + kh;
    rscale = make_float2(a.k_scale[at], a.v_scale[at]);
  };
  auto stage_s = [&](int slot) {
    const bool ok = is_page(a.seq, entry_s);
    lost |= !ok;
    if (lane < 4) sc[slot][lane] = block_scale(ok ? rscale.x : NAN, rscale.y);
  };
  // token 16 x + 4 y + z of a 32-token block is row 8 y + 4 x + z of its product: half x of the lanes gets the
  // scores of tokens 16 x .. 16 x + 15, all of one cache block
  auto key_row = [](int tok) { return (tok & 35) | ((tok & 12) << 1) | ((tok >> 2) & 4); };
  int put[CH];                                   // this thread's places in a tile
#pragma unroll
  for (int n = 0; n < CH; ++n) {
    const int y = (tid + NT * n) & (4 * D - 1);
    const int tok = y / (D / 16);
    put[n] = of_keys(n) ? key_row(tok) * KP + 2 * (y % (D / 16)) : (y % D) * VP + 2 * (y / D);
  }
  auto stage = [&](int slot, int n0, int n1) {   // chunks n0 .. n1 - 1
#pragma unroll
    for (int n = n0; n < n1; ++n) {
      const half8 h0 = unpack8(raw[n].x, raw[n].y), h1 = unpack8(raw[n].z, raw[n].w);
      half8* const to = of_keys(n) ? sk + slot * KB + put[n] : sv + slot * VB + put[n];
      to[0] = h0;
      to[1] = h1;
    }
  };

  floatx16 o[DT];
  float m = kNoToken, l = 0.0f;
#pragma unroll
  for (int t = 0; t < DT; ++t) o[t] = floatx16{};
  const int kat = (lq + 32 * wh) * KP + lh, vat = lq * VP + 2 * lh + 4 * wh;
  // Scores of half h of the tile in a slot: e[x] of this lane belongs to token 64 c + 32 h + 16 lh + x.
  auto key_step = [&](int slot, int h, int t, floatx16& e) {
    const half8 kf = (sk + slot * KB + kat)[h * 32 * KP + 2 * t];
#pragma unroll
    for (int q = 0; q < P; ++q) e = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, qf[q][t], t + q ? e : floatx16{}, 0, 0, 0);
  };
  auto hide = [&](int c, int h, floatx16& e) {                 // scores that the row must not see
    const int z = 64 * c + 32 * h;
    if (z + 31 <= p_lo && !(a.window > 0 && z <= p_hi - a.window)) return;
    const int hi = pos - (z + 16 * lh), lo = a.window > 0 && hi >= 0 ? hi - a.window : -1;
#pragma unroll
    for (int x = 0; x < 16; ++x) e[x] = (x <= hi && x > lo) ? e[x] : -INFINITY;
  };
  // The running maximum takes the scores of a half in; f and the shift it returns turn them into weights' exponents.
  auto raise = [&](floatx16& e, float& f, float lv) {
    float x0 = e[0], x1 = e[1];
#pragma unroll
    for (int x = 2; x < 16; x += 2) {
      x0 = fmaxf(x0, e[x]);
      x1 = fmaxf(x1, e[x + 1]);
    }
    const float mx = across_halves_max(fmaf(fmaxf(x0, x1), f, lv));
    if (__any(mx > m + kLag)) {
      const float mn = fmaxf(m, mx), fall = exp2_raw(m - mn);
      m = mn;
      l *= fall;
#pragma unroll
      for (int t = 0; t < DT; ++t) o[t] *= fall;
    }
    float shift = lv - m + kExp;
    if (__any(fabsf(m) > kFarMax)) {             // no farther above 0 than the maximum may lag, whatever m + kLag was
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const float t = fmaf(e[x], f, lv) - m;
        e[x] = t > kLag ? kLag : t;              // a NaN stays
      }
      f = 1.0f;
      shift = kExp;
    }
    return shift;
  };
  auto factor = [&](const BlockScale& bs) {
    return fmaxf(bs.ks * fq, 1e-37f);            // above 0, so that a hidden score stays -inf
  };
  // Half h of a tile from its scores e on: the weights alternate with the products of the queries and half hn's
  // keys, the next (to en), then the products with the values with the unpacking of chunk `part` of a later tile.
  // A wave's MFMAs and vector instructions overlap only where they alternate.
  auto half_body = [&](int h, float iv, float f, float shift, const floatx16& e, int slot, int kslot, int hn, floatx16& en,
                       auto&& unpack) {
    float sum = 0.0f;
    half8 pf[P][2];
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      key_step(kslot, hn, t, en);
      constexpr int PER = 16 / KS;               // weights between two steps
#pragma unroll
      for (int x = t * PER; x < (t + 1) * PER; x += 2) {
        const float w_0 = exp2_raw(fmaf(e[x], f, shift)), w_1 = exp2_raw(fmaf(e[x + 1], f, shift));
        const half2v p = {_Float16(w_0), _Float16(w_1)};
        pf[0][x >> 3][x & 7] = p[0];
        pf[0][x >> 3][(x & 7) + 1] = p[1];
        // the sum takes the weights as they were: divided by a small value scale, one that float16 loses can count
        sum += w_0;
        sum += w_1;
        if (!BF16) {
          pf[P - 1][x >> 3][x & 7] = _Float16(w_0 - float(p[0]));
          pf[P - 1][x >> 3][(x & 7) + 1] = _Float16(w_1 - float(p[1]));
        }
      }
    }
    l = sum > 0.0f ? fmaf(sum, iv, l) : l;    // a poisoned block that the row does not see stays out of it
    unpack();
    const half8* const vr = sv + slot * VB + vat + 4 * h;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int t = 0; t < DT; ++t) {
        const half8 vf = vr[32 * VP * t + k];
#pragma unroll
        for (int q = 0; q < P; ++q) o[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, pf[q][k], o[t], 0, 0, 0);
      }
  };

  const int n_tiles = rg.c1 - rg.c0;
  floatx16 e0, e1;
  if (n_tiles > 0) {
    look(rg.c0);
    fetch(rg.c0);
    look(rg.c0 + 1);
    stage(0, 0, CH);
    fetch(rg.c0 + 1);
    look(rg.c0 + 2);
    stage(1, 0, CH);
    fetch(rg.c0 + 2);
    look(rg.c0 + 3);
    if (wave < 4) {                              // scales of tile `wave`; 2 and 3 go on like those of later tiles
      look_s(rg.c0 + wave);
      if (wave < 3) fetch_s();
      if (wave < 2) stage_s(wave);
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < KS; ++t) key_step(0, 0, t, e0);
  }
  int now = 0, next = 1, far = 2;                // slots of tiles t0, t0 + 1, t0 + 2
  const bool idle = w0 >= nrows;                 // a wave without rows helps with the tiles only
  for (int t0 = 0; t0 < n_tiles; ++t0) {
    const int c = rg.c0 + t0;
    if (idle) {
      stage(far, 0, CH);
      fetch(c + 3);
      look(c + 4);
    } else {
      const BlockScale b0 = sc[t0 & 3][2 * wh + lh], b1 = sc[t0 & 3][2 + lh];
      float f0 = factor(b0), f1 = factor(b1);
      hide(c, wh, e0);
      const float shift0 = raise(e0, f0, b0.lv);
      if constexpr (PAIRS) {
        half_body(0, b0.iv, f0, shift0, e0, now, next, 0, e1, [&] {
          stage(far, 0, CH);
          fetch(c + 3);
          look(c + 4);
        });
        e0 = e1;
      } else {
        half_body(0, b0.iv, f0, shift0, e0, now, now, 1, e1, [&] { stage(far, 0, CH / 2); });
        hide(c, 1, e1);
        const float shift1 = raise(e1, f1, b1.lv);
        half_body(1, b1.iv, f1, shift1, e1, now, next, 0, e0, [&] {
          stage(far, CH / 2, CH);
          fetch(c + 3);
          look(c + 4);
        });
      }
    }
    if (((t0 + 2) & 7) == wave) stage_s((t0 + 2) & 3);
    if (((t0 + 3) & 7) == wave) fetch_s();
    if (((t0 + 4) & 7) == wave) look_s(c + 4);
    __syncthreads();
    const int was = now;
    now = next;
    next = far;
    far = was;
  }
  if (lost) report(a.seq.info, KQ_INFO_PAGE);
  l += __shfl_xor(l, 32);
  if constexpr (PAIRS) {                         // the second wave of a pair hands its sums over, where the tiles were
    constexpr int N = DT / 2 * 1024 + 128;       // half of them in either array, and m and l
    static_assert(GROUPS * N * sizeof(float) <= std::min(sizeof(sk), sizeof(sv)), "a pair's sums do not fit");
    const int at = (wave & (GROUPS - 1)) * N + lane;
    float* const po[2] = {reinterpret_cast<float*>(sk) + at, reinterpret_cast<float*>(sv) + at};
    if (wh) {
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int x = 0; x < 16; ++x) po[t & 1][(8 * (t & ~1) + x) * 64] = o[t][x];
      po[0][DT / 2 * 1024] = m;
      po[0][DT / 2 * 1024 + 64] = l;
    }
    __syncthreads();
    if (wh) return;
    const float m1 = po[0][DT / 2 * 1024], mn = fmaxf(m, m1), f0 = exp2_raw(m - mn), f1 = exp2_raw(m1 - mn);
    m = mn;
    l = l * f0 + po[0][DT / 2 * 1024 + 64] * f1;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int x = 0; x < 16; ++x) o[t][x] = o[t][x] * f0 + po[t & 1][(8 * (t & ~1) + x) * 64] * f1;
  }
  if (w0 + lq >= nrows) return;
  const int64_t row = int64_t(s.row0) + i;
  if (pos < 0) {                                 // sees nothing, whatever its query holds
    l = 0.0f;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int x = 0; x < 16; ++x) o[t][x] = 0.0f;
  }
  if (rg.parts == 1) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int x = 0; x < 4; ++x)
        store4<BF16>(a.out, row * a.ldo + int64_t(head) * D + 32 * t + 8 * x + 4 * lh, o[t][4 * x] * inv,
                     o[t][4 * x + 1] * inv, o[t][4 * x + 2] * inv, o[t][4 * x + 3] * inv);
  } else {
    const int64_t at = (row * a.heads + head) * a.splits + split;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int x = 0; x < 4; ++x)
        *reinterpret_cast<floatx4*>(a.part_o + at * D + 32 * t + 8 * x + 4 * lh) =
            floatx4{o[t][4 * x], o[t][4 * x + 1], o[t][4 * x + 2], o[t][4 * x + 3]};
    if (lh == 0) *reinterpret_cast<float2*>(a.part_ml + at * 2) = make_float2(m, l);
  }
}

// Joins the parts of each row: D / 4 threads for four channels each, and G such groups that take the parts in
// turn, in a fixed order; 256 * 4 / (D G) rows a workgroup. G 1 for many rows or a few parts, else all groups
// of a workgroup for one row.
template <bool BF16, int D, int G>
__global__ __launch_bounds__(256) void cache_join_kernel(AttnArgs a) {
  constexpr int T = D / 4, R = 256 / (T * G);
  __shared__ floatx4 sh[G][T];
  __shared__ float sh_l[G];
  const int grp = threadIdx.x / T % G, d = threadIdx.x % T * 4;
  const int per_b = a.seq.max_q * a.heads;       // below 2^31: checked by the host
  const int wgs_b = (per_b + R - 1) / R;
  const int b = blockIdx.x / wgs_b, in = (blockIdx.x - b * wgs_b) * R + threadIdx.x / (T * G);
  const int i = in / a.heads, head = in - i * a.heads;
  const Seq s = sequence(a.seq, b, false);
  if (i >= s.n) return;                          // with G > 1 for the whole workgroup
  const int row_tile = (i * a.g + head % a.g) / a.tile_rows * a.tile_rows, nrows = s.n * a.g;
  const int parts = chunk_range(a, s, row_tile / a.g, (min(row_tile + a.tile_rows, nrows) - 1) / a.g, 0).parts;
  if (parts == 1) return;
  const int64_t row = int64_t(s.row0) + i;
  const float* const ml = a.part_ml + (row * a.heads + head) * a.splits * 2;
  const float* const po = a.part_o + (row * a.heads + head) * a.splits * int64_t(D);
  float m = kNoToken;
  if (G > 1) {
    const int lane = threadIdx.x & 63;
    for (int x = lane; x < parts; x += 64) m = fmaxf(m, ml[2 * x]);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
  } else {
    for (int x = 0; x < parts; ++x) m = fmaxf(m, ml[2 * x]);
  }
  floatx4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  float l = 0.0f;
#pragma unroll 4
  for (int x = grp; x < parts; x += G) {
    const float2 w = *reinterpret_cast<const float2*>(ml + 2 * x);
    const float f = exp2_raw(w.x - m);
    acc += f * *reinterpret_cast<const floatx4*>(po + int64_t(x) * D + d);
    l += f * w.y;
  }
  if (G > 1) {
    sh[grp][d / 4] = acc;
    if (d == 0) sh_l[grp] = l;
    __syncthreads();
    if (grp) return;
#pragma unroll
    for (int x = 1; x < G; ++x) {
      acc += sh[x][d / 4];
      l += sh_l[x];
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  store4<BF16>(a.out, row * a.ldo + int64_t(head) * D + d, acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
}

template <bool BF16, int D, int G>
kq_status launch_join(const AttnArgs& a, hipStream_t st) {
  constexpr int R = 1024 / (D * G);
  const int64_t wgs = a.batch * ((int64_t(a.seq.max_q) * a.heads + R - 1) / R);
  {
    LaunchTimer timer("cache_join_kernel", st);
    hipLaunchKernelGGL((cache_join_kernel<BF16, D, G>), dim3(static_cast<uint32_t>(wgs)), dim3(256), 0, st, a);
  }
  return check_launch("cache_join_kernel");
}

struct Plan {
  bool prompt;
  int tile_rows, tiles, splits;
};

// A window that no sequence can outgrow hides nothing.
int effective_window(const kq_cache& c, const kq_cache_batch& b, int window) {
  return window >= int64_t(b.max_pages) * c.page ? 0 : window;
}

Plan plan(const kq_cache& c, const kq_cache_batch& b, int heads, int window) {
  Plan p;
  const int64_t rows = int64_t(b.max_q) * (heads / c.kv_heads), heads_all = int64_t(b.batch) * c.kv_heads;
  // 16 rows a workgroup while those fill the GPU once at most, or while 256 rows would be mostly idle: one
  // sequence, 8 key/value heads, 4096 tokens: 256 rows 24.6 us against 34.5 in tiles of 256, 384 rows about even;
  // 8 sequences: 64 rows 31.6 against 46.9, 128 rows 57.9 against 54.5
  p.prompt = rows > 64 && heads_all * ((rows + 15) / 16) > kCus;
  // 128 rows a workgroup where 256 leave CUs idle and the rows' own tokens are most of what they see, so that the last
  // tiles take longest: one prompt of 32 over 8 heads, 512 tokens 21.4 us against 27.0 in tiles of 256, 1024 32.7 and
  // 43.1, 2048 (two workgroups a CU) 67.8 and 75.5. Not for short prompts in two workgroups a CU (four of 512: 38.4
  // and 29.7), nor on a long context, which is split evenly (512 tokens on 8192: 108 and 96).
  const int64_t wide = heads_all * ((rows + 255) / 256);
  const bool narrow = int64_t(b.max_pages) * c.page <= 2 * int64_t(b.max_q) && wide <= (b.max_q >= 1024 ? kCus : kCus / 2);
  p.tile_rows = !p.prompt ? 16 : narrow ? 128 : 256;
  p.tiles = static_cast<int>((rows + p.tile_rows - 1) / p.tile_rows);
  int64_t longest = int64_t(b.max_pages) * c.page;
  if (window > 0) longest = std::min<int64_t>(longest, int64_t(window) + b.max_q + 63);
  // The context is split while that leaves one workgroup a CU at most, and a split has enough tokens to pay for the
  // joining launch (single tokens, 32 over 8 heads: 1024 tokens 11.4 us in two of 512, 11.8 whole; 64 channels: 9.3
  // and 7.6). More workgroups than that are never split, not even where the last tiles of a prompt outlast the
  // others: 2048 tokens, 32 over 8 heads, 256 workgroups of 256 rows and 1 to 32 chunks, in parts of 17, took 87 us and
  // 16 more to join, whole 77 (workgroups start in order, in rotation over the shader engines, so long and short ones
  // in turn end up on the same CUs).
  const int64_t most = std::max<int64_t>(1, kCus / (heads_all * p.tiles)), least = p.prompt ? 512 : 65536 / c.head_dim;
  p.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, (longest + least - 1) / least)));
  if (window > 0) p.splits = std::min(p.splits, plan(c, b, heads, 0).splits);   // fits in the workspace of window 0
  return p;
}

template <bool BF16, int D>
kq_status launch(const AttnArgs& a, bool prompt, hipStream_t st) {
  const int64_t wgs = int64_t(a.batch) * a.kvh * a.tiles * a.splits;
  if (wgs > int64_t(INT32_MAX) || (a.splits > 1 && int64_t(a.seq.max_q) * a.heads * a.batch > int64_t(INT32_MAX)))
    return fail(KQ_EUNSUPPORTED, "kq_cache_attention: too many workgroups (batch %d, max_q %d)", a.batch, a.seq.max_q);
  const dim3 grid(static_cast<uint32_t>(wgs));
  kq_status r;
  if (prompt) {
    LaunchTimer timer("cache_prompt_kernel", st);
    if (a.tile_rows == 128) hipLaunchKernelGGL((cache_prompt_kernel<BF16, D, 128>), grid, dim3(512), 0, st, a);
    else hipLaunchKernelGGL((cache_prompt_kernel<BF16, D, 256>), grid, dim3(512), 0, st, a);
    r = check_launch("cache_prompt_kernel");
  } else {
    LaunchTimer timer("cache_token_kernel", st);
    hipLaunchKernelGGL((cache_token_kernel<BF16, D>), grid, dim3(kTokenWaves * 64), 0, st, a);
    r = check_launch("cache_token_kernel");
  }
  if (r != KQ_OK || a.splits == 1) return r;
  // 32 heads of 4 tokens, 8 parts: 13.2 us a call against 13.5 with one group a row; of 256 tokens 52.7 and 45.4
  const bool few_rows = int64_t(a.batch) * a.seq.max_q * a.heads <= 1024;
  return a.splits > 4 && few_rows ? launch_join<BF16, D, 1024 / D>(a, st) : launch_join<BF16, D, 1>(a, st);
}

}  // namespace

size_t cache_attention_workspace(const kq_cache& c, const kq_cache_batch& b, int64_t rows, int heads, int window) {
  const Plan p = plan(c, b, heads, effective_window(c, b, window));
  if (p.splits == 1) return 0;
  return size_t(rows) * heads * p.splits * (c.head_dim + 2) * sizeof(float);
}

kq_status cache_attention_run(const kq_cache& c, const kq_cache_batch& b, CacheIn q, bool bf16, int64_t rows,
                              int heads, float scale, int window, void* out, int64_t ldo, int32_t* info, void* ws,
                              hipStream_t st) {
  window = effective_window(c, b, window);
  const Plan p = plan(c, b, heads, window);
  AttnArgs a;
  a.seq = seq_args(c, b, rows, info);
  a.k = c.k;
  a.v = c.v;
  a.k_scale = c.k_scale;
  a.v_scale = c.v_scale;
  a.q = q.p;
  a.ldq = q.ld;
  a.out = out;
  a.ldo = ldo;
  a.heads = heads;
  a.kvh = c.kv_heads;
  a.g = heads / c.kv_heads;
  a.scale_log2e = static_cast<float>(double(scale) * 1.4426950408889634);
  a.window = window;
  a.batch = b.batch;
  a.tiles = p.tiles;
  a.tile_rows = p.tile_rows;
  a.splits = p.splits;
  a.longest_first = b.batch > 1 && b.batch <= 64 && int64_t(b.batch) * c.kv_heads * p.tiles > kCus;   // prompts
  a.part_o = static_cast<float*>(ws);
  a.part_ml = a.part_o + size_t(rows) * heads * p.splits * c.head_dim;
  if (bf16) return c.head_dim == 64 ? launch<true, 64>(a, p.prompt, st) : launch<true, 128>(a, p.prompt, st);
  return c.head_dim == 64 ? launch<false, 64>(a, p.prompt, st) : launch<false, 128>(a, p.prompt, st);
}

}  // namespace kq
