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
// more. Weights are scaled by 2^14 and rounded to float16 (2^-11, against the 2^-8 of a bf16
// output), for float32 outputs to two pieces. Maxima, sums and accumulators are float32.
#include <algorithm>
#include <cmath>

#include "cache_internal.h"

namespace kq {
namespace {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr float kNoToken = -1.0e30f;   // running maximum before the first token (finite: no inf - inf)
constexpr float kZeroScale = -48.0f;   // log2 taken for a value scale of 0: any finite one (its codes are 0)
constexpr float kWeightExp = 14.0f;    // weights are held times 2^14, so that float16 keeps small ones

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
  int batch, tiles, splits;
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
    u.x = f32_to_bf16(a) | (f32_to_bf16(b) << 16);
    u.y = f32_to_bf16(c) | (f32_to_bf16(d) << 16);
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p) + at) = u;
  } else {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + at) = make_float4(a, b, c, d);
  }
}

// Power of two that takes amax to [2^14, 2^15) (1 for a row of zeros), and its inverse; a row
// with a NaN or an infinity gets NaN, which reaches all of its scores.
__device__ __forceinline__ void row_scale(float amax, float& up, float& down) {
  int e;
  (void)frexpf(amax, &e);  // amax = f 2^e, f in [0.5, 1)
  e = amax > 0.0f ? min(max(15 - e, -126), 126) : 0;
  up = amax < INFINITY ? ldexpf(1.0f, e) : NAN;
  down = amax < INFINITY ? ldexpf(1.0f, -e) : NAN;
}

__device__ __forceinline__ float exp2_raw(float x) { return __builtin_amdgcn_exp2f(x); }

// This split's share of the 64-token chunks that a tile of rows sees, and the first and last
// 16-token groups of the whole tile: what lies outside is never looked up.
struct Range {
  int c0, c1, g0, g1;
};

__device__ __forceinline__ Range chunk_range(const Seq& s, int i_first, int i_last, int window, int split, int splits) {
  const int p_last = s.len - s.n + i_last, p_first = s.len - s.n + i_first;
  if (p_last < 0) return Range{0, 0, 0, 0};
  const int low = window > 0 ? max(0, p_first - window + 1) : 0;
  const int a = low >> 6, e = (p_last >> 6) + 1;
  const int per = max((e - a + splits - 1) / splits, 4);  // at least one chunk for each wave
  const int c0 = min(a + split * per, e);
  return Range{c0, min(c0 + per, e), low >> 4, p_last >> 4};
}

// ---------------------------------------------------------------------------
// A few rows a sequence: single tokens, drafts
//
// A workgroup takes 16 rows of one sequence and head and a range of the context; its four waves
// take the range's 64-token chunks in turn and never share data before the end, where their
// partial sums are joined in LDS. Nothing is staged: each operand comes from the cache in the
// order its MFMA wants it. S^T = K Q^T has tokens as rows: lane (lk = lane / 16, li = lane mod 16)
// gets rows 4 lk + j of each 16-token product. Which token a row is, is free: row 4 lk + j of
// product i is token 16 lk + 4 i + j, so a lane ends up with 16 consecutive tokens, all of one
// cache block, and they are its operand of O^T = V^T P^T, whose other operand is 16 codes of one
// channel: one 16-byte load. Channels are permuted likewise so that a key row's loads are 16
// bytes a lane.
// ---------------------------------------------------------------------------
template <bool BF16, int D>
__global__ __launch_bounds__(256, 2) void cache_token_kernel(AttnArgs a) {
  constexpr int U = D / 64;       // 16-byte key loads a lane and token row
  constexpr int DT = D / 16;      // 16-channel tiles of the output
  constexpr int PITCH = D + 4;
  __shared__ float sh_o[4][16 * PITCH];
  __shared__ float sh_m[4][16], sh_l[4][16];
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
  const Range rg = chunk_range(s, i_first, i_last, a.window, split, a.splits);
  // every token of a chunk is seen by every row if it lies in (p_last - window, p_first]
  const int p_first = first + i_first, p_last = first + i_last;

  // the row of q in float16 pieces, in the channel order of the key loads
  half8 qh[2 * U], ql[BF16 ? 1 : 2 * U];
  float down;
  {
    const int64_t at = (int64_t(s.row0) + i) * a.ldq + int64_t(hd) * D;
    float x[2 * U][8];
    float amax = 0.0f;
#pragma unroll
    for (int t = 0; t < 2 * U; ++t) {
      load8<BF16>(a.q, at + 64 * (t >> 1) + 16 * lk + 8 * (t & 1), x[t]);
    }
#pragma unroll
    for (int t = 0; t < 2 * U; ++t)
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[t][j]) < INFINITY ? fabsf(x[t][j]) : INFINITY);
    amax = fmaxf(amax, __shfl_xor(amax, 16));
    amax = fmaxf(amax, __shfl_xor(amax, 32));
    float up;
    row_scale(amax, up, down);
#pragma unroll
    for (int t = 0; t < 2 * U; ++t)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float y = x[t][j] * up;
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
  const int page = 1 << a.seq.page_log2, pmask = page - 1;

  for (int c = rg.c0 + wave; c < rg.c1; c += 4) {
    // 16-token groups of this lane: of its key rows, and of its weights and values
    const int gk = min(max(4 * c + (li >> 2), rg.g0), rg.g1), gv = min(max(4 * c + lk, rg.g0), rg.g1);
    const int idk = page_of(a.seq, b, gk << 4), idv = page_of(a.seq, b, gv << 4);
    const int8_t* const kp = a.k + ((int64_t(max(idk, 0)) * a.kvh + kh) * page + ((gk << 4) & pmask)) * D +
                             (li & 3) * D + 16 * lk;
    const int64_t blk = int64_t(max(idv, 0)) * a.kvh + kh;
    const int8_t* const vp = a.v + (blk * page + ((gv << 4) & pmask)) * D + 16 * li;
    uint4 kc[4][U], vc[DT];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int u = 0; u < U; ++u) kc[t][u] = *reinterpret_cast<const uint4*>(kp + 4 * t * D + 64 * u);
    const float ks = idv < 0 ? NAN : a.k_scale[blk], vs = idv < 0 ? NAN : a.v_scale[blk];
#pragma unroll
    for (int t = 0; t < DT; ++t) vc[t] = *reinterpret_cast<const uint4*>(vp + 256 * t);

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
    const float f = ks * qf;                                   // scores to base-2 exponents
    const float lv = vs == 0.0f ? kZeroScale : __log2f(vs);
    const float iv = vs == 0.0f ? 0x1p48f : 1.0f / vs;
    const int t0 = 64 * c + 16 * lk;                           // this lane's first token
    const bool cut = 64 * c + 63 > p_first || (a.window > 0 && 64 * c <= p_last - a.window);
    const int hi = p - t0, lo = a.window > 0 ? hi - a.window : -1;  // tokens x in (lo, hi] are seen
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
    const float shift = lv - m + kWeightExp;
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
  }
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
#pragma unroll
  for (int t = 0; t < DT; ++t) *reinterpret_cast<floatx4*>(&sh_o[wave][li * PITCH + 16 * t + 4 * lk]) = o[t];
  if (lk == 0) {
    sh_m[wave][li] = m;
    sh_l[wave][li] = l;
  }
  __syncthreads();
  // join the waves: 16 threads a row
  const int q = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * 4;
  if (tile * 16 + q >= nrows) return;
  float mj = sh_m[0][q];
#pragma unroll
  for (int w = 1; w < 4; ++w) mj = fmaxf(mj, sh_m[w][q]);
  float fw[4], lj = 0.0f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    fw[w] = exp2_raw(sh_m[w][q] - mj);
    lj += fw[w] * sh_l[w][q];
  }
  const int rq = tile * 16 + q, iq = rq / a.g;
  const int64_t row = int64_t(s.row0) + iq;
  const int head = kh * a.g + (rq - iq * a.g);
#pragma unroll
  for (int d = d0; d < D; d += 64) {
    floatx4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < 4; ++w) x += fw[w] * *reinterpret_cast<const floatx4*>(&sh_o[w][q * PITCH + d]);
    if (a.splits == 1) {
      const float inv = lj == 0.0f ? 0.0f : 1.0f / lj;
      store4<BF16>(a.out, row * a.ldo + int64_t(head) * D + d, x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
    } else {
      *reinterpret_cast<floatx4*>(a.part_o + ((row * a.heads + head) * a.splits + split) * D + d) = x;
    }
  }
  if (a.splits > 1 && d0 == 0)
    *reinterpret_cast<float2*>(a.part_ml + ((row * a.heads + head) * a.splits + split) * 2) = make_float2(mj, lj);
}

// ---------------------------------------------------------------------------
// Prompts
// ---------------------------------------------------------------------------

// A block's scales as the weights use them. A NaN (a poisoned block, a bad page) becomes a finite
// stand-in and `bad`: the rows that see such a block are made NaN apart.
struct BlockScale {
  float ks, lv, iv, bad;
};

__device__ __forceinline__ BlockScale block_scale(float ks, float vs) {
  BlockScale r;
  r.bad = ks == ks && vs == vs ? 0.0f : 1.0f;
  r.ks = ks > 0.0f ? ks : 1.0f;                 // 0: the codes are 0, so any factor will do
  r.lv = vs > 0.0f ? __log2f(vs) : kZeroScale;
  r.iv = vs > 0.0f ? 1.0f / vs : 0x1p48f;
  return r;
}

template <bool BF16, int D, int NQ, int W>
__global__ __launch_bounds__(W * 64, NQ == 1 ? 2 : 1) void cache_prompt_kernel(AttnArgs a) {
  typedef float floatx16 __attribute__((ext_vector_type(16)));
  constexpr int NT = W * 64, ROWS = 32 * NQ * W;
  constexpr int KS = D / 16, DT = D / 32;        // MFMA steps over channels, 32-channel output tiles
  constexpr int KU = D / 8;                      // 16-byte units of a key row in LDS
  constexpr int CH = 8 * D / NT;                 // 16-byte chunks of codes a thread stages (keys, then values)
  constexpr int P = BF16 ? 1 : 2;                // float16 pieces of a query and a weight
  __shared__ half8 sk[2][64 * KU];               // keys: token rows of KU units
  __shared__ half8 sv[2][D * 8];                 // values: channel rows of 64 tokens
  __shared__ BlockScale sc[2][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lq = lane & 31, lh = lane >> 5;
  int64_t id = blockIdx.x;
  const int nbh = a.batch * a.kvh;
  const int bh = id % nbh;
  id /= nbh;
  const int tile = a.tiles - 1 - int(id % a.tiles), split = id / a.tiles;   // the longest first
  const int b = bh / a.kvh, kh = bh - b * a.kvh;
  const Seq s = sequence(a.seq, b, kh == 0 && tile == 0 && split == 0 && tid == 0);
  const int nrows = s.n * a.g;
  if (tile * ROWS >= nrows) return;
  const int first = s.len - s.n;
  const Range rg = chunk_range(s, tile * ROWS / a.g, (min(tile * ROWS + ROWS, nrows) - 1) / a.g, a.window, split, a.splits);

  // this wave's rows
  const int w0 = tile * ROWS + wave * 32 * NQ;
  const int wlast = min(w0 + 32 * NQ, nrows) - 1;
  const int p_hi = wlast >= w0 ? first + wlast / a.g : -1, p_lo = first + min(w0, nrows - 1) / a.g;
  half8 qf[P][NQ][KS];
  float fq[NQ];
  int pos[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int r = min(w0 + 32 * n + lq, nrows - 1);
    const int i = r / a.g, hd = kh * a.g + (r - i * a.g);
    pos[n] = first + i;
    const int64_t at = (int64_t(s.row0) + i) * a.ldq + int64_t(hd) * D + 8 * lh;
    float amax = 0.0f;
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      float x[8];
      load8<BF16>(a.q, at + 16 * t, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[j]) < INFINITY ? fabsf(x[j]) : INFINITY);
    }
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
        qf[0][n][t][j] = h;
        if (!BF16) qf[P - 1][n][t][j] = _Float16(y - float(h));
      }
    }
    fq[n] = a.scale_log2e * down;
  }

  // staging: chunk x < 4 D of keys (token x / (D / 16), 16 channels), then of values (group, channel);
  // a wave's chunks are all of one 16-token group
  uint4 raw[CH];
  float2 rscale;
  const int page = 1 << a.seq.page_log2;
  auto group_of = [&](int i) {
    return ((wave * 64 + NT * i) & (4 * D - 1)) / D;       // 16 tokens are D chunks of either side
  };
  auto fetch = [&](int c) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int g = min(max(4 * c + group_of(i), rg.g0), rg.g1);
      const int pg = max(page_of(a.seq, b, g << 4), 0);
      const int x = tid + NT * i, y = x & (D - 1);
      const int64_t at = ((int64_t(pg) * a.kvh + kh) * page + ((g << 4) & (page - 1))) * D + 16 * y;
      raw[i] = *reinterpret_cast<const uint4*>((wave * 64 + NT * i < 4 * D ? a.k : a.v) + at);
    }
    if (tid < 4) {
      const int g = min(max(4 * c + tid, rg.g0), rg.g1);
      const int pg = page_of(a.seq, b, g << 4);
      const int64_t at = int64_t(max(pg, 0)) * a.kvh + kh;
      rscale = pg < 0 ? make_float2(NAN, NAN) : make_float2(a.k_scale[at], a.v_scale[at]);
    }
  };
  auto stage = [&](int buf) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int x = tid + NT * i, y = x & (4 * D - 1);
      const half8 h0 = unpack8(raw[i].x, raw[i].y), h1 = unpack8(raw[i].z, raw[i].w);
      if (wave * 64 + NT * i < 4 * D) {
        const int tok = y / (D / 16), u = 2 * (y % (D / 16));
        const int z = (tok & 3) | ((tok >> 2) & 4);
        sk[buf][tok * KU + (u ^ z)] = h0;
        sk[buf][tok * KU + ((u + 1) ^ z)] = h1;
      } else {
        const int grp = y / D, d = y % D;
        sv[buf][d * 8 + ((2 * grp) ^ (d & 7))] = h0;
        sv[buf][d * 8 + ((2 * grp + 1) ^ (d & 7))] = h1;
      }
    }
    if (tid < 4) sc[buf][tid] = block_scale(rscale.x, rscale.y);
  };

  floatx16 o[NQ][DT];
  float m[NQ], l[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    m[n] = kNoToken;
    l[n] = 0.0f;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int x = 0; x < 16; ++x) o[n][t][x] = 0.0f;
  }
  // token of this lane's key row in a 32-token block, and its bank swizzle
  const int ktok = 16 * ((lq >> 2) & 1) + 4 * (lq >> 3) + (lq & 3);
  const int kz = (ktok & 3) | ((ktok >> 2) & 4);

  if (rg.c0 < rg.c1) {
    fetch(rg.c0);
    stage(0);
    fetch(rg.c0 + 1);
  }
  __syncthreads();
  for (int c = rg.c0; c < rg.c1; ++c) {
    const int buf = (c - rg.c0) & 1;
    stage(buf ^ 1);
    fetch(c + 2);
    const bool active = 64 * c <= p_hi && (a.window <= 0 || 64 * c + 63 > p_lo - a.window);
    if (active) {
      floatx16 e[NQ][2];
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int x = 0; x < 16; ++x) e[n][h][x] = 0.0f;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < KS; ++t) {
          const half8 kf = sk[buf][(32 * h + ktok) * KU + ((2 * t + lh) ^ kz)];
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int q = 0; q < P; ++q) e[n][h] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, qf[q][n][t], e[n][h], 0, 0, 0);
        }
      const BlockScale b0 = sc[buf][lh], b1 = sc[buf][2 + lh];
      const bool cut = 64 * c + 63 > p_lo || (a.window > 0 && 64 * c <= p_hi - a.window);
      half8 pf[P][NQ][4];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        // tokens x of half h are 64 c + 32 h + 16 lh + x
        const int hi = pos[n] - (64 * c + 16 * lh), lo = a.window > 0 ? hi - a.window : -(1 << 30);
        if (cut) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int x = 0; x < 16; ++x) e[n][h][x] = (32 * h + x <= hi && 32 * h + x > lo) ? e[n][h][x] : -INFINITY;
        }
        float f0 = b0.ks * fq[n], f1 = b1.ks * fq[n];
        f0 = f0 < 1e-37f ? 1e-37f : f0;          // above 0, so that a hidden score stays -inf (a NaN stays NaN)
        f1 = f1 < 1e-37f ? 1e-37f : f1;
        float x0 = e[n][0][0], x1 = e[n][1][0];
#pragma unroll
        for (int x = 1; x < 16; ++x) {
          x0 = fmaxf(x0, e[n][0][x]);
          x1 = fmaxf(x1, e[n][1][x]);
        }
        float mx = fmaxf(fmaf(x0, f0, b0.lv), fmaf(x1, f1, b1.lv));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        if (__any(mx > m[n])) {
          const float mn = fmaxf(m[n], mx), fall = exp2_raw(m[n] - mn);
          m[n] = mn;
          l[n] *= fall;
#pragma unroll
          for (int t = 0; t < DT; ++t) o[n][t] *= fall;
        }
        const float s0 = b0.lv - m[n] + kWeightExp, s1 = b1.lv - m[n] + kWeightExp;
        float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const float w_0 = exp2_raw(fmaf(e[n][0][x], f0, s0)), w_1 = exp2_raw(fmaf(e[n][1][x], f1, s1));
          sum0 += w_0;
          sum1 += w_1;
          const _Float16 h_0 = _Float16(w_0), h_1 = _Float16(w_1);
          pf[0][n][x >> 3][x & 7] = h_0;
          pf[0][n][2 + (x >> 3)][x & 7] = h_1;
          if (!BF16) {
            pf[P - 1][n][x >> 3][x & 7] = _Float16(w_0 - float(h_0));
            pf[P - 1][n][2 + (x >> 3)][x & 7] = _Float16(w_1 - float(h_1));
          }
        }
        l[n] += sum0 * b0.iv + sum1 * b1.iv;
        if (__any((b0.bad != 0.0f) | (b1.bad != 0.0f))) {   // rows that see a poisoned block
          if ((b0.bad != 0.0f && hi >= 0 && lo < 15) || (b1.bad != 0.0f && hi >= 32 && lo < 47)) l[n] = NAN;
        }
      }
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) {             // 32-token half k >> 1, its step k & 1
          const half8 vf = sv[buf][(32 * t + lq) * 8 + ((4 * (k >> 1) + 2 * lh + (k & 1)) ^ (lq & 7))];
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int q = 0; q < P; ++q) o[n][t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, pf[q][n][k], o[n][t], 0, 0, 0);
        }
    }
    __syncthreads();
  }
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int r = w0 + 32 * n + lq;
    l[n] += __shfl_xor(l[n], 32);
    if (r >= nrows) continue;
    const int i = r / a.g, head = kh * a.g + (r - i * a.g);
    const int64_t row = int64_t(s.row0) + i;
    if (pos[n] < 0) {                             // sees nothing, whatever its query holds
      l[n] = 0.0f;
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int x = 0; x < 16; ++x) o[n][t][x] = 0.0f;
    }
    if (a.splits == 1) {
      const float inv = l[n] == 0.0f ? 0.0f : 1.0f / l[n];
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          store4<BF16>(a.out, row * a.ldo + int64_t(head) * D + 32 * t + 8 * x + 4 * lh, o[n][t][4 * x] * inv,
                       o[n][t][4 * x + 1] * inv, o[n][t][4 * x + 2] * inv, o[n][t][4 * x + 3] * inv);
    } else {
      const int64_t at = (row * a.heads + head) * a.splits + split;
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          *reinterpret_cast<floatx4*>(a.part_o + at * D + 32 * t + 8 * x + 4 * lh) =
              floatx4{o[n][t][4 * x], o[n][t][4 * x + 1], o[n][t][4 * x + 2], o[n][t][4 * x + 3]};
      if (lh == 0) *reinterpret_cast<float2*>(a.part_ml + at * 2) = make_float2(m[n], l[n]);
    }
  }
}

// Joins the splits of each row: a workgroup for each (sequence, token, head), 256 threads as
// 256 * 4 / D groups of D / 4 threads that take the splits in turn, a fixed order.
template <bool BF16, int D>
__global__ __launch_bounds__(256) void cache_join_kernel(AttnArgs a) {
  constexpr int T = D / 4, G = 256 / T;
  __shared__ floatx4 sh[G][T];
  __shared__ float sh_l[G];
  int64_t id = blockIdx.x;
  const int head = id % a.heads;
  id /= a.heads;
  const int i = id % a.seq.max_q, b = id / a.seq.max_q;
  const Seq s = sequence(a.seq, b, false);
  if (i >= s.n) return;
  const int64_t row = int64_t(s.row0) + i;
  const float* const ml = a.part_ml + (row * a.heads + head) * a.splits * 2;
  const float* const po = a.part_o + (row * a.heads + head) * a.splits * int64_t(D);
  const int lane = threadIdx.x & 63, grp = threadIdx.x / T, d = (threadIdx.x % T) * 4;
  float m = kNoToken;
  for (int x = lane; x < a.splits; x += 64) m = fmaxf(m, ml[2 * x]);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
  floatx4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  float l = 0.0f;
  for (int x = grp; x < a.splits; x += G) {
    const float f = exp2_raw(ml[2 * x] - m);
    acc += f * *reinterpret_cast<const floatx4*>(po + int64_t(x) * D + d);
    l += f * ml[2 * x + 1];
  }
  sh[grp][threadIdx.x % T] = acc;
  if (threadIdx.x % T == 0) sh_l[grp] = l;
  __syncthreads();
  if (grp) return;
#pragma unroll
  for (int x = 1; x < G; ++x) {
    acc += sh[x][threadIdx.x];
    l += sh_l[x];
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  store4<BF16>(a.out, row * a.ldo + int64_t(head) * D + d, acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
}

struct Plan {
  bool prompt;
  int tiles, splits;
};

Plan plan(const kq_cache& c, const kq_cache_batch& b, bool bf16, int heads, int window) {
  Plan p;
  const int64_t rows = int64_t(b.max_q) * (heads / c.kv_heads);
  p.prompt = rows > 32;
  const int rows_wg = p.prompt ? 256 : 16;
  p.tiles = static_cast<int>((rows + rows_wg - 1) / rows_wg);
  int64_t longest = int64_t(b.max_pages) * c.page;
  if (window > 0) longest = std::min<int64_t>(longest, int64_t(window) + b.max_q + 63);
  const int64_t wgs = int64_t(b.batch) * c.kv_heads * p.tiles;
  const int64_t want = ((p.prompt ? 1 : 4) * kCus + wgs - 1) / wgs;
  p.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, (longest + 511) / 512)));
  return p;
}

template <bool BF16, int D>
kq_status launch(const AttnArgs& a, bool prompt, hipStream_t st) {
  const int64_t wgs = int64_t(a.batch) * a.kvh * a.tiles * a.splits;
  const int64_t joins = int64_t(a.batch) * a.seq.max_q * a.heads;
  if (wgs > int64_t(INT32_MAX) || (a.splits > 1 && joins > int64_t(INT32_MAX)))
    return fail(KQ_EUNSUPPORTED, "kq_cache_attention: too many workgroups (batch %d, max_q %d)", a.batch, a.seq.max_q);
  const dim3 grid(static_cast<uint32_t>(wgs));
  kq_status r;
  if (prompt) {
    LaunchTimer timer("cache_prompt_kernel", st);
    hipLaunchKernelGGL((cache_prompt_kernel<BF16, D, 1, 8>), grid, dim3(512), 0, st, a);
    r = check_launch("cache_prompt_kernel");
  } else {
    LaunchTimer timer("cache_token_kernel", st);
    hipLaunchKernelGGL((cache_token_kernel<BF16, D>), grid, dim3(256), 0, st, a);
    r = check_launch("cache_token_kernel");
  }
  if (r != KQ_OK || a.splits == 1) return r;
  {
    LaunchTimer timer("cache_join_kernel", st);
    hipLaunchKernelGGL((cache_join_kernel<BF16, D>), dim3(static_cast<uint32_t>(joins)), dim3(256), 0, st, a);
  }
  return check_launch("cache_join_kernel");
}

}  // namespace

size_t cache_attention_workspace(const kq_cache& c, const kq_cache_batch& b, bool bf16, int64_t rows, int heads,
                                 int window) {
  const Plan p = plan(c, b, bf16, heads, window);
  if (p.splits == 1) return 0;
  return size_t(rows) * heads * p.splits * (c.head_dim + 2) * sizeof(float);
}

kq_status cache_attention_run(const kq_cache& c, const kq_cache_batch& b, CacheIn q, bool bf16, int64_t rows,
                              int heads, float scale, int window, void* out, int64_t ldo, int32_t* info, void* ws,
                              hipStream_t st) {
  const Plan p = plan(c, b, bf16, heads, window);
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
  a.splits = p.splits;
  a.part_o = static_cast<float*>(ws);
  a.part_ml = a.part_o + size_t(rows) * heads * p.splits * c.head_dim;
  if (bf16) return c.head_dim == 64 ? launch<true, 64>(a, p.prompt, st) : launch<true, 128>(a, p.prompt, st);
  return c.head_dim == 64 ? launch<false, 64>(a, p.prompt, st) : launch<false, 128>(a, p.prompt, st);
}

}  // namespace kq
