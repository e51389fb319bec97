// The 8-bit key/value cache: appending to it (norm, rotation, quantization in one launch) and
// reading it back.
//
// Append. A block (page, head) of new tokens is quantized on one scale, so its largest entry has
// to be known before its first code: one workgroup holds a whole block of one side (keys or
// values) in registers, a wave for each 16 slots, two adjacent channels a lane (64 lanes a row at
// head_dim 128, two rows of 32 lanes at 64). Each value is read once and each code written once;
// the layout of the values (16 tokens of a channel side by side) makes a lane's 16 slots one
// 16-byte store for each of its channels. Queries need no scale and go to workgroups of their
// own, a wave for each token and group of heads.
//
// Three prompts of up to 8192 tokens, 32 over 8 heads, bf16 (519 MB): 172 us, 3.0 TB/s; all in
// float32 it would be 157. Few tokens are latency: table entry, old scale, row, norm's sum, the
// block's maximum and the code follow from one another (one token 3.9 us, 64 of them 12.1).
//
// Norm and rotation are float64, and so is the division where float32 cannot tell the code: in
// float32 alone they end within 1e-5 of a step of a rounding border for one entry in 10^5, whose
// code would then depend on the order of operations.
#include <cmath>
#include <type_traits>

#include "cache_internal.h"

namespace kq {
namespace {

constexpr int kHeadsPerWave = 16;                      // of a long prompt's queries, all loads in flight
constexpr float kScaleFloor = 7.888609052210118e-31f;  // 2^-100: keeps 1 / scale and its sums finite

struct AppendArgs {
  SeqArgs seq;
  const void* src[3];     // q, k, v
  int64_t ld[3];
  const float* norm[2];   // q, k
  double eps;
  const float* rope;
  int64_t rope_len;
  int rot;
  int interleaved;
  void* q_out;
  int64_t ldqo;
  int8_t* k;
  int8_t* v;
  float* k_scale;
  float* v_scale;
  int heads, kvh;
  int blocks;             // blocks a sequence's new tokens can touch
  int batch;
  int64_t kv_wgs;         // workgroups that take blocks; the others take queries
  int in_turn;            // spread over the grid, else the blocks first
  int q_groups;           // head groups of a token in the query part
};

template <bool BF16>
__device__ __forceinline__ float2 load2(const void* p, int64_t at) {
  if (BF16) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint16_t*>(p) + at);
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  return *reinterpret_cast<const float2*>(reinterpret_cast<const float*>(p) + at);
}

// Sum over the LPR lanes of a row, the same value in all of them.
template <int LPR>
__device__ __forceinline__ double row_sum(double v) {
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

// What a lane needs of one position's row of the rotations for its entries 2 l and 2 l + 1: y <- y c + p s with
// the partner p of each (in `from`'s lane for pairs half a rotation apart, the lane's other entry when
// interleaved), on the lanes below rot_dim.
struct Turn {
  float2 c, s;
  bool in;
};

template <int D>
__device__ __forceinline__ Turn turn_of(const float* row, int rot, bool interleaved, int l) {
  const int half = rot >> 1;
  Turn t;
  t.c = t.s = make_float2(0.0f, 0.0f);
  t.in = row && 2 * l < rot;
  if (!row) return t;
  const bool in = t.in, low = 2 * l < half;
  if (interleaved) {
    const float c = row[in ? l : 0], s = row[half + (in ? l : 0)];
    t.c = make_float2(c, c);
    t.s = make_float2(-s, s);
  } else {
    const int j = in ? (low ? 2 * l : 2 * l - half) : 0;                 // even, as half is
    const float2 c = *reinterpret_cast<const float2*>(row + j), s = *reinterpret_cast<const float2*>(row + half + j);
    t.c = c;
    t.s = low ? make_float2(-s.x, -s.y) : s;
  }
  return t;
}

// The lane that holds the partners of entries 2 l and 2 l + 1 (every lane of the wave asks).
__device__ __forceinline__ int partner_lane(int rot, bool interleaved, int l) {
  const int lane = threadIdx.x & 63;
  if (interleaved || 2 * l >= rot) return lane;
  return 4 * l < rot ? lane + (rot >> 2) : lane - (rot >> 2);
}

// Norm (weights w of the lane's entries, wp of their partners) and rotation of a row's entries x.
template <int D>
__device__ __forceinline__ void place(double (&y)[2], float2 x, bool norm, float2 w, float2 wp, double eps, bool turns,
                                      const Turn& t, int from, bool interleaved) {
  constexpr int LPR = D / 2;
  y[0] = x.x;
  y[1] = x.y;
  double r = 1.0;
  if (norm) {
    r = 1.0 / sqrt(row_sum<LPR>(y[0] * y[0] + y[1] * y[1]) * (1.0 / D) + eps);
    y[0] *= r * double(w.x);
    y[1] *= r * double(w.y);
  }
  if (turns) {
    double p0, p1;
    if (interleaved) {
      p0 = y[1];
      p1 = y[0];
    } else {
      p0 = __shfl(x.x, from);
      p1 = __shfl(x.y, from);
      if (norm) {
        p0 *= r * double(wp.x);
        p1 *= r * double(wp.y);
      }
    }
    p0 = y[0] * double(t.c.x) + p0 * double(t.s.x);
    p1 = y[1] * double(t.c.y) + p1 * double(t.s.y);
    y[0] = t.in ? p0 : y[0];
    y[1] = t.in ? p1 : y[1];
  }
}

// A norm's weights of the lane's entries and of their partners.
__device__ __forceinline__ void norm_weights(const float* w, int l, int from, float2& own, float2& partner) {
  own = partner = make_float2(1.0f, 1.0f);
  if (!w) return;
  own = *reinterpret_cast<const float2*>(w + 2 * l);
  partner = make_float2(__shfl(own.x, from), __shfl(own.y, from));
}

// round_half_even(y / s) in [-127, 127]. The float32 product with inv = 1 / s is within 3 roundings of the
// quotient, 127 * 3 * 2^-24 = 2.3e-5: only a value that close to a border needs the float64 division (a wave has
// one in the slots of a block at times, so the whole wave takes it).
template <typename T>
__device__ __forceinline__ void codes_of(const T (&y)[2], double s, float inv, int (&c)[2]) {
  float r[2];
  bool near = false;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float t = float(y[e]) * inv;
    r[e] = rintf(t);
    near |= fabsf(fabsf(t - r[e]) - 0.5f) < 4e-5f;
  }
  if (__any(near)) {
#pragma unroll
    for (int e = 0; e < 2; ++e) r[e] = float(rint(double(y[e]) / s));
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) c[e] = int(__builtin_amdgcn_fmed3f(r[e], -127.0f, 127.0f));
}

__device__ __forceinline__ float max_abs(float a, float y) { return fmaxf(a, fabsf(y)); }
__device__ __forceinline__ double max_abs(double a, double y) { return fmax(a, fabs(y)); }

__device__ __forceinline__ int rescaled(int code, double ratio) { return int(rint(double(code) * ratio)); }

// One block of one side: values are float32 as they come, keys float64 from the norm and the rotation on. NS 1:
// the block takes one new token (slot lo), which every lane computes.
template <bool BF16, int D, int PAGE, int NS, bool is_v>
__device__ void append_block(const AppendArgs& a, int head, int pageid, int pos0, int lo, int hi, int row_lo) {
  using T = typename std::conditional<is_v, float, double>::type;
  constexpr int LPR = D / 2, SL = 16 * LPR / 64;  // lanes a row, slots a lane
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int l = lane & (LPR - 1), hh = lane / LPR;
  const int first_slot = 16 * w + hh * SL;
  const bool norm = !is_v && a.norm[1] != nullptr;
  const bool turn = !is_v && a.rope != nullptr;
  const void* src = is_v ? a.src[2] : a.src[1];
  const int64_t ld = is_v ? a.ld[2] : a.ld[1];
  const int from = turn ? partner_lane(a.rot, a.interleaved, l) : lane;
  float2 wt, wp;
  norm_weights(norm ? a.norm[1] : nullptr, l, from, wt, wp);
  float* const scale_at = (is_v ? a.v_scale : a.k_scale) + int64_t(pageid) * a.kvh + head;
  const float s_old = lo > 0 ? *scale_at : 0.0f;

  T y[NS][2];
  const bool mine = NS == 1 || (16 * w < hi && 16 * w + 16 > lo);  // uniform in the wave
  T top = 0, poison = 0;  // poison: NaN once an entry is not finite (0 * inf)
  if (mine) {
    float2 x[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int slot = NS == 1 ? lo : min(max(first_slot + s, lo), hi - 1);
      x[s] = load2<BF16>(src, int64_t(row_lo + slot - lo) * ld + int64_t(head) * D + 2 * l);
    }
    if constexpr (is_v) {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        y[s][0] = x[s].x;
        y[s][1] = x[s].y;
      }
    } else {
      constexpr int STEP = NS < 4 ? NS : 4;      // slots whose rotations are loaded together
#pragma unroll
      for (int s0 = 0; s0 < NS; s0 += STEP) {
        Turn tn[STEP];
#pragma unroll
        for (int s = 0; s < STEP; ++s) {
          const int slot = NS == 1 ? lo : min(max(first_slot + s0 + s, lo), hi - 1);
          const int64_t p = int64_t(pos0) + slot;
          tn[s] = turn_of<D>(turn ? a.rope + (p >= a.rope_len ? 0 : p) * a.rot : nullptr, a.rot, a.interleaved, l);
        }
#pragma unroll
        for (int s = 0; s < STEP; ++s)
          place<D>(y[s0 + s], x[s0 + s], norm, wt, wp, a.eps, turn, tn[s], from, a.interleaved);
      }
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int slot = NS == 1 ? lo : first_slot + s;
      if (turn && slot >= lo && slot < hi && int64_t(pos0) + slot >= a.rope_len) {
        report(a.seq.info, KQ_INFO_POSITION);
        poison = NAN;
      }
      // slots that are not new hold a copy of one that is
      top = max_abs(max_abs(top, y[s][0]), y[s][1]);
      poison = fma(y[s][0], T(0), fma(y[s][1], T(0), poison));
    }
  }
  double amax = poison == poison ? double(top) : double(INFINITY);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) amax = fmax(amax, __shfl_xor(amax, o));
  if (PAGE > 16) {
    __shared__ double top[PAGE / 16];
    if (lane == 0) top[w] = amax;
    __syncthreads();  // also: every wave has read the old scale before it is replaced
#pragma unroll
    for (int i = 0; i < PAGE / 16; ++i) amax = fmax(amax, top[i]);
  }
  float s_new = amax > 0.0 ? fmaxf(float(amax / 127.0), kScaleFloor) : 0.0f;
  if (!(s_new >= s_old)) s_new = s_old;                       // a NaN of the block stays
  if (!(amax < INFINITY) || !(s_new < INFINITY)) s_new = NAN;
  if (threadIdx.x == 0) *scale_at = s_new;
  const double sd = s_new;
  const float inv = s_new > 0.0f ? 1.0f / s_new : 0.0f;
  const bool usable = s_new > 0.0f;                           // not 0, not NaN
  const bool grow = lo > 0 && s_old > 0.0f && s_new > s_old;
  const double ratio = grow ? double(s_old) / sd : 1.0;
  const bool old_here = grow && 16 * w < lo;
  const bool new_here = 16 * w < hi && 16 * w + 16 > lo;
  if (!old_here && !new_here) return;

  int c[NS][2];
  if (mine) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      if (usable) codes_of(y[s], sd, inv, c[s]);
      else c[s][0] = c[s][1] = 0;
    }
  }
  const int64_t block = int64_t(pageid) * a.kvh + head;
  if (!is_v) {
    int8_t* const rows = a.k + block * (PAGE * D) + 2 * l;
    if (NS == 1) {
      if (new_here && hh == 0) *reinterpret_cast<uint16_t*>(rows + lo * D) = uint16_t((c[0][0] & 255) | ((c[0][1] & 255) << 8));
    } else if (new_here) {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int slot = first_slot + s;
        if (slot >= lo && slot < hi)
          *reinterpret_cast<uint16_t*>(rows + slot * D) = uint16_t((c[s][0] & 255) | ((c[s][1] & 255) << 8));
      }
    }
    if (old_here) {
      uint16_t o[SL];
#pragma unroll
      for (int s = 0; s < SL; ++s) o[s] = *reinterpret_cast<const uint16_t*>(rows + (first_slot + s) * D);
#pragma unroll
      for (int s = 0; s < SL; ++s)
        if (first_slot + s < lo)
          *reinterpret_cast<uint16_t*>(rows + (first_slot + s) * D) =
              uint16_t((rescaled(int8_t(o[s] & 255), ratio) & 255) | ((rescaled(int8_t(o[s] >> 8), ratio) & 255) << 8));
    }
    return;
  }
  int8_t* const group = a.v + block * (PAGE * D) + w * (D * 16);
  if (NS == 1 && !old_here) {
    if (hh == 0) {
      group[(2 * l) * 16 + (lo & 15)] = int8_t(c[0][0]);
      group[(2 * l + 1) * 16 + (lo & 15)] = int8_t(c[0][1]);
    }
    return;
  }
  const bool whole = NS > 1 && lo <= 16 * w && hi >= 16 * w + 16;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    uint32_t* const at = reinterpret_cast<uint32_t*>(group + (2 * l + e) * 16 + hh * SL);
    uint32_t words[SL / 4];
#pragma unroll
    for (int i = 0; i < SL / 4; ++i) words[i] = whole ? 0u : at[i];  // slots past the new ones keep what they hold
#pragma unroll
    for (int s = 0; s < SL; ++s) {
      const int slot = first_slot + s;
      const int sh = 8 * (s & 3);
      const int was = int8_t(words[s >> 2] >> sh);
      int now = was;
      if (slot < lo) now = old_here ? rescaled(was, ratio) : was;
      else if (slot < hi) now = c[NS == 1 ? 0 : s][e];
      words[s >> 2] = (words[s >> 2] & ~(255u << sh)) | (uint32_t(now & 255) << sh);
    }
#pragma unroll
    for (int i = 0; i < SL / 4; ++i) at[i] = words[i];
  }
}

// Queries: a wave for each token and group of heads.
template <bool BF16, int D, int WAVES>
__device__ void turn_queries(const AppendArgs& a, int64_t wg) {
  constexpr int LPR = D / 2;
  const int lane = threadIdx.x & 63, l = lane & (LPR - 1), hh = lane / LPR;
  const int64_t item = wg * WAVES + (threadIdx.x >> 6);
  const int64_t items = int64_t(a.seq.max_q) * a.q_groups;
  const int64_t per_b = (items + WAVES - 1) / WAVES * WAVES;
  const int b = item / per_b;
  const int64_t in = item - b * per_b;
  if (in >= items) return;
  const int i = in / a.q_groups, gq = in - int64_t(i) * a.q_groups;
  const Seq s = sequence(a.seq, b, false);
  if (i >= s.n) return;
  const int64_t p = int64_t(s.len) - s.n + i;
  const bool norm = a.norm[0] != nullptr, turn = a.rope != nullptr;
  const int from = turn ? partner_lane(a.rot, a.interleaved, l) : lane;
  float2 wt, wp;
  norm_weights(a.norm[0], l, from, wt, wp);
  const bool off = p < 0 || (turn && p >= a.rope_len);
  if (turn && p >= a.rope_len && lane == 0) report(a.seq.info, KQ_INFO_POSITION);
  const Turn tn = turn_of<D>(turn ? a.rope + (off ? 0 : p) * a.rot : nullptr, a.rot, a.interleaved, l);
  const int64_t row = s.row0 + i;
  const int h_per = (a.heads + a.q_groups - 1) / a.q_groups;
  const int h1 = min(a.heads, (gq + 1) * h_per);
  constexpr int RW = 64 / LPR, UN = kHeadsPerWave / RW;   // heads a wave takes at once, and how often
  const int h0 = gq * h_per;
  auto finish = [&](int h, float2 x) {
    double y[2];
    place<D>(y, x, norm, wt, wp, a.eps, turn, tn, from, a.interleaved);
    if (off) y[0] = y[1] = NAN;
    if (h < h1) {
      const int64_t at = row * a.ldqo + int64_t(h) * D + 2 * l;
      // to bf16 through float32: half a step of bf16 (2^-8), and 2^-25
      if (BF16)
        *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(a.q_out) + at) = pack_bf16(float(y[0]), float(y[1]));
      else
        *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.q_out) + at) = make_float2(float(y[0]), float(y[1]));
    }
  };
  auto source = [&](int h) { return load2<BF16>(a.src[0], row * a.ld[0] + int64_t(min(h, h1 - 1)) * D + 2 * l); };
  if (h_per <= RW) {
    finish(h0 + hh, source(h0 + hh));
  } else {
    float2 x[UN];
#pragma unroll
    for (int u = 0; u < UN; ++u) x[u] = source(h0 + u * RW + hh);
#pragma unroll
    for (int u = 0; u < UN; ++u) finish(h0 + u * RW + hh, x[u]);
  }
}

template <bool BF16, int D, int PAGE>
__global__ __launch_bounds__(PAGE * 4) void cache_append_kernel(AppendArgs a) {
  constexpr int SL = D / 8, WAVES = PAGE / 16;
  int64_t id = blockIdx.x;
  bool block = id < a.kv_wgs;
  if (a.in_turn) {                   // of workgroups 0 .. x, floor((x + 1) kv_wgs / all) are blocks
    const int64_t at = id * a.kv_wgs, all = gridDim.x;
    id = at / all;
    block = at - id * all + a.kv_wgs >= all;
  }
  if (block) {
    const int side = id & 1;
    id >>= 1;
    const int head = id % a.kvh;
    id /= a.kvh;
    const int j = id % a.blocks, b = id / a.blocks;
    const Seq s = sequence(a.seq, b, j == 0 && head == 0 && side == 0 && threadIdx.x == 0);
    if (s.n <= 0) return;
    const int first = s.len - s.n;  // position of the first new token; below 0: those tokens have no place
    if (first < 0 && j == 0 && threadIdx.x == 0) report(a.seq.info, KQ_INFO_LENGTH);
    if ((int64_t(max(first, 0) / PAGE) + j) * PAGE >= s.len) return;
    const int pos0 = (max(first, 0) / PAGE + j) * PAGE;
    const int lo = max(max(first, 0) - pos0, 0), hi = min(PAGE, s.len - pos0);
    const int pageid = page_of(a.seq, b, pos0);
    if (pageid < 0) return;
    const int row_lo = s.row0 + pos0 + lo - first;
    if (hi - lo == 1) {
      if (side) append_block<BF16, D, PAGE, 1, true>(a, head, pageid, pos0, lo, hi, row_lo);
      else append_block<BF16, D, PAGE, 1, false>(a, head, pageid, pos0, lo, hi, row_lo);
    } else {
      if (side) append_block<BF16, D, PAGE, SL, true>(a, head, pageid, pos0, lo, hi, row_lo);
      else append_block<BF16, D, PAGE, SL, false>(a, head, pageid, pos0, lo, hi, row_lo);
    }
    return;
  }
  turn_queries<BF16, D, WAVES>(a, blockIdx.x - (a.in_turn ? id : a.kv_wgs));
}

template <bool BF16, int D, int PAGE>
void launch_append(const AppendArgs& a, int64_t wgs, hipStream_t st) {
  LaunchTimer timer("cache_append_kernel", st);
  hipLaunchKernelGGL((cache_append_kernel<BF16, D, PAGE>), dim3(static_cast<uint32_t>(wgs)), dim3(PAGE * 4), 0, st, a);
}

template <bool BF16, int D>
void launch_append(const AppendArgs& a, int page, int64_t wgs, hipStream_t st) {
  switch (page) {
    case 16: launch_append<BF16, D, 16>(a, wgs, st); break;
    case 32: launch_append<BF16, D, 32>(a, wgs, st); break;
    case 64: launch_append<BF16, D, 64>(a, wgs, st); break;
    default: launch_append<BF16, D, 128>(a, wgs, st); break;
  }
}

// ---------------------------------------------------------------------------
// reading back
// ---------------------------------------------------------------------------

struct ReadArgs {
  SeqArgs seq;
  const int8_t* k;
  const int8_t* v;
  const float* k_scale;
  const float* v_scale;
  void* out[2];
  int64_t ld[2];
  int kvh;
  int groups;  // 16-token groups a sequence's rows can touch
  int64_t items;
};

// N consecutive values at out + at: 16 bytes (8 bf16, 4 float32) or half of that.
template <bool BF16, int N>
__device__ __forceinline__ void store_values(void* out, int64_t at, const float (&f)[N]) {
  if constexpr (BF16) {
    uint16_t* const p = reinterpret_cast<uint16_t*>(out) + at;
    if constexpr (N == 8)
      *reinterpret_cast<uint4*>(p) =
          make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
  } else {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + at) = make_float4(f[0], f[1], f[2], f[3]);
  }
}

// A wave for each 16 tokens of a head. Keys: 16 bytes of output a lane, whole rows a store. Values: four channels a
// lane of 8 (64 channels: 4) of the tokens, whole rows a store again. Bound by HBM: 131072 tokens of 8 heads to bf16
// (805 MB) 144 to 157 us, 5.1 to 5.6 TB/s, a copy's rate; stores of single values took 191.
template <bool BF16, int D>
__global__ __launch_bounds__(256) void cache_read_kernel(ReadArgs a) {
  const int lane = threadIdx.x & 63;
  int64_t item = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (item >= a.items) return;
  const int head = item % a.kvh;
  item /= a.kvh;
  const int j = item % a.groups, b = item / a.groups;
  const Seq s = sequence(a.seq, b, j == 0 && head == 0 && lane == 0);
  if (s.n <= 0) return;
  const int first = s.len - s.n;
  const int page = 1 << a.seq.page_log2;
  if (first < 0 && j == 0) {
    if (lane == 0) report(a.seq.info, KQ_INFO_LENGTH);
    for (int i = 0; i < min(-first, s.n); ++i)  // rows without a place
      for (int d = lane; d < 2 * D; d += 64) {
        void* const out = a.out[d / D];
        const int64_t at = (int64_t(s.row0) + i) * a.ld[d / D] + int64_t(head) * D + d % D;
        if (!out) continue;
        if (BF16) reinterpret_cast<uint16_t*>(out)[at] = 0x7fc0;
        else reinterpret_cast<float*>(out)[at] = NAN;
      }
  }
  if ((int64_t(max(first, 0) / 16) + j) * 16 >= s.len) return;
  const int pos0 = (max(first, 0) / 16 + j) * 16;
  const int lo = max(max(first, 0) - pos0, 0), hi = min(16, s.len - pos0);
  const int id = page_of(a.seq, b, pos0);
  const int64_t block = int64_t(max(id, 0)) * a.kvh + head;
  const float ks = id < 0 ? NAN : a.k_scale[block], vs = id < 0 ? NAN : a.v_scale[block];
  const int off = pos0 & (page - 1);
  const int64_t row0 = int64_t(s.row0) + pos0 - first;  // row of slot 0 of the group
  if (a.out[0]) {
    const int8_t* const src = a.k + (block * page + off) * D;
    constexpr int N = BF16 ? 8 : 4, LR = D / N, STEPS = 16 * LR / 64;   // values a lane, lanes a row
    uint32_t c[STEPS][N / 4];
#pragma unroll
    for (int t = 0; t < STEPS; ++t) {
      const uint32_t* const at = reinterpret_cast<const uint32_t*>(src + (64 * t + lane) * N);
#pragma unroll
      for (int i = 0; i < N / 4; ++i) c[t][i] = at[i];
    }
#pragma unroll
    for (int t = 0; t < STEPS; ++t) {
      const int slot = (64 * t + lane) / LR, d = lane % LR * N;
      float f[N];
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = float(int8_t(c[t][i / 4] >> (8 * (i % 4)))) * ks;
      if (slot >= lo && slot < hi) store_values<BF16, N>(a.out[0], (row0 + slot) * a.ld[0] + int64_t(head) * D + d, f);
    }
  }
  if (a.out[1]) {
    constexpr int LR = D / 4, TOK = LR / 4;               // lanes a row, tokens a lane
    const int d = lane % LR * 4, t0 = lane / LR * TOK;
    const int8_t* const src = a.v + (block * page + off) * D + d * 16 + t0;
    uint32_t c[4][TOK / 4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int i = 0; i < TOK / 4; ++i) c[e][i] = *reinterpret_cast<const uint32_t*>(src + 16 * e + 4 * i);
#pragma unroll
    for (int t = 0; t < TOK; ++t) {
      float f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = float(int8_t(c[e][t / 4] >> (8 * (t % 4)))) * vs;
      if (t0 + t >= lo && t0 + t < hi)
        store_values<BF16, 4>(a.out[1], (row0 + t0 + t) * a.ld[1] + int64_t(head) * D + d, f);
    }
  }
}

}  // namespace

kq_status cache_append_run(const kq_cache& c, const kq_cache_batch& b, CacheIn q, CacheIn k, CacheIn v, bool bf16,
                           int64_t rows, int heads, const float* q_norm, const float* k_norm, float eps,
                           const float* rope, int64_t rope_len, int rot_dim, bool interleaved, void* q_out,
                           int64_t ldqo, int32_t* info, hipStream_t st) {
  AppendArgs a;
  a.seq = seq_args(c, b, rows, info);
  a.src[0] = q.p;
  a.src[1] = k.p;
  a.src[2] = v.p;
  a.ld[0] = q.ld;
  a.ld[1] = k.ld;
  a.ld[2] = v.ld;
  a.norm[0] = q_norm;
  a.norm[1] = k_norm;
  a.eps = eps;
  a.rope = rope;
  a.rope_len = rope_len;
  a.rot = rot_dim;
  a.interleaved = interleaved;
  a.q_out = q_out;
  a.ldqo = ldqo;
  a.k = c.k;
  a.v = c.v;
  a.k_scale = c.k_scale;
  a.v_scale = c.v_scale;
  a.heads = heads;
  a.kvh = c.kv_heads;
  a.batch = b.batch;
  // max_q consecutive tokens touch at most this many blocks, wherever they begin
  a.blocks = static_cast<int>((int64_t(b.max_q) + c.page - 2) / c.page + 1);
  a.kv_wgs = int64_t(b.batch) * a.blocks * c.kv_heads * 2;
  // All heads of a few tokens are spread over waves, for latency, and blocks, which take longer, start first; a wave
  // takes 16 heads of a token of many, and as those wait for memory where blocks wait for arithmetic, their workgroups
  // run side by side (three prompts of up to 8192 tokens, 32 over 8 heads: 87 us for the queries alone and 102 for
  // the blocks, 172 together; 64 single tokens take 22.1 us with the blocks first and 22.8 in turn).
  const bool many = int64_t(b.batch) * b.max_q * heads > 8192;
  a.in_turn = many;
  const int waves = c.page / 16;
  const int per_wave = many ? kHeadsPerWave : 128 / c.head_dim;
  a.q_groups = heads ? (heads + per_wave - 1) / per_wave : 1;
  const int64_t per_b = (int64_t(b.max_q) * a.q_groups + waves - 1) / waves * waves;
  const int64_t q_wgs = q_out ? int64_t(b.batch) * per_b / waves : 0;
  if (a.kv_wgs + q_wgs > int64_t(INT32_MAX))
    return fail(KQ_EUNSUPPORTED, "kq_cache_append: batch %d with max_q %d needs too many workgroups", b.batch, b.max_q);
  const int64_t wgs = a.kv_wgs + q_wgs;
  if (bf16) {
    if (c.head_dim == 64) launch_append<true, 64>(a, c.page, wgs, st);
    else launch_append<true, 128>(a, c.page, wgs, st);
  } else {
    if (c.head_dim == 64) launch_append<false, 64>(a, c.page, wgs, st);
    else launch_append<false, 128>(a, c.page, wgs, st);
  }
  return check_launch("cache_append_kernel");
}

kq_status cache_read_run(const kq_cache& c, const kq_cache_batch& b, void* k_out, void* v_out, bool bf16, int64_t rows,
                         int64_t ldk, int64_t ldv, int32_t* info, hipStream_t st) {
  ReadArgs a;
  a.seq = seq_args(c, b, rows, info);
  a.k = c.k;
  a.v = c.v;
  a.k_scale = c.k_scale;
  a.v_scale = c.v_scale;
  a.out[0] = k_out;
  a.out[1] = v_out;
  a.ld[0] = ldk;
  a.ld[1] = ldv;
  a.kvh = c.kv_heads;
  a.groups = static_cast<int>((int64_t(b.max_q) + 14) / 16 + 1);
  a.items = int64_t(b.batch) * a.groups * c.kv_heads;
  const int64_t wgs = (a.items + 3) / 4;
  if (wgs > int64_t(INT32_MAX))
    return fail(KQ_EUNSUPPORTED, "kq_cache_read: batch %d with max_q %d needs too many workgroups", b.batch, b.max_q);
  {
    LaunchTimer timer("cache_read_kernel", st);
    const dim3 grid(static_cast<uint32_t>(wgs)), block(256);
    if (bf16) {
      if (c.head_dim == 64) hipLaunchKernelGGL((cache_read_kernel<true, 64>), grid, block, 0, st, a);
      else hipLaunchKernelGGL((cache_read_kernel<true, 128>), grid, block, 0, st, a);
    } else {
      if (c.head_dim == 64) hipLaunchKernelGGL((cache_read_kernel<false, 64>), grid, block, 0, st, a);
      else hipLaunchKernelGGL((cache_read_kernel<false, 128>), grid, block, 0, st, a);
    }
  }
  return check_launch("cache_read_kernel");
}

}  // namespace kq
