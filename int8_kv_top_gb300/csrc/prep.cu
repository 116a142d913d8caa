// qsa_prep: the fused prep of T new tokens (the pages' qsa_prep, "round 27 track b - qsa prep
// and merge": decision and rejected prep fusion name its raw rows, gains, norm_rope step and mrope
// variants; correctness lists its outputs qcur, kq, vq, ksc, vsc).  The library's readings of
// the unstated formulas:
//   q, k rows: y = x / sqrt(mean(x^2) + eps) * gamma, then the rotary embedding with halves
//              paired (i, i + rd/2), theta_i = p * base^(-2i/rd) (mrope: p of the pair's section)
//              (y_i, y_{i+rd/2}) -> (y_i cos - y_{i+rd/2} sin, y_{i+rd/2} cos + y_i sin)
//   outputs:   qcur = fp16(q rows); kcur = fp16(k rows) (optional); the cache cell pos0 + t gets
//              quantise(kcur) and quantise(v rows), the absmax rule of qsa_prep_quantize.
//
// One CTA (256 threads, at most 48 registers: five CTAs per SM) per token; each warp issues the
// loads of all its rows before it uses any, so a CTA waits on one memory round trip, and the gains
// are read per row from L1.  More CTAs per SM hide more of that round trip: a persistent form that
// loads the next token's rows during the current one held fewer CTAs per SM and ran slower.  The token's rd/2 rotation
// angles are formed once, in fp32 with the product's error recovered and a three-part 2 pi
// (rope_angle), then sincosf, into shared memory; each lane then keeps its own four (cos, sin)
// pairs in registers for all the token's rows.  A warp takes a row at a time with the lanes laid
// out around the rotation: lane l < R = rd / 8 holds the four rotation pairs (4l + u, 4l + u + rd/2),
// lanes l >= R hold 8 consecutive unrotated dims rd + 8 (l - R) ..; so every lane holds 8 values in
// two 4-dim runs at dims (a, b), the rotation needs no exchange between lanes, and the row's
// sum of squares and the quantiser's four 64-element block maxima are warp reductions.
#include <cmath>

#include "common.cuh"

namespace qsa {
namespace {

constexpr int kPrepRows = kHeads + 2 * kGroups;  // 24 q rows, 2 k rows, 2 v rows per token

struct PrepCfg {
  float inv_hi[kD / 2], inv_lo[kD / 2];  // base^(-2i / rd) as a float pair hi + lo, i < rd / 2
  int rotary_dim, sec0, sec1;
  float eps;
};

// theta = p * (hi + lo) reduced to about [-pi, pi], all in fp32 (GB300's fp64 rate is low): the
// product's rounding error is recovered exactly with an fma, and 2 pi is split Cody-Waite style
// into C1 (8 significant bits, so k * C1 is exact for k < 2^16) + C2 + C3.  For positions up to
// 2^17 the result is within about 3e-7 of the exact angle modulo 2 pi.
__device__ __forceinline__ float rope_angle(int p, float hi, float lo) {
  const float P = (float)p;
  const float prod = P * hi;
  const float err = fmaf(P, hi, -prod) + P * lo;  // p * (hi + lo) - prod
  const float k = rintf(prod * 0.15915494309189535f);
  float r = fmaf(-k, 6.28125f, prod);  // exact: k * C1 has at most 22 significant bits
  r = fmaf(-k, 1.9353071795864769e-3f, r);
  r = fmaf(-k, 1.0253131677018246e-11f, r);
  return r + err;
}

// Dims of this lane's two 4-dim runs (see above): (a, b) with values x[0..3] at a .. a + 3 and
// x[4..7] at b .. b + 3.
__device__ __forceinline__ void lane_dims(int lane, int rd, int& a, int& b) {
  const int R = rd >> 3;
  if (lane < R) {
    a = 4 * lane;
    b = a + (rd >> 1);
  } else {
    a = rd + 8 * (lane - R);
    b = a + 4;
  }
}

__device__ __forceinline__ void unpack4(uint2 w, float* x) {
  const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
  const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
  x[0] = f0.x;
  x[1] = f0.y;
  x[2] = f1.x;
  x[3] = f1.y;
}

// The quantiser of qsa_prep_quantize on one 256-element row held as above: per 64-element block
// IEEE fp32 a / 127 rounded to fp16, codes round-half-away(x / s) clamped to +-127 (all zero and
// a +0 scale for an all-zero block).  The block maxima are reduced over the whole warp.
__device__ __forceinline__ void quantize_row(const float (&x)[8], int a, int b, int8_t* codes, __half* scales,
                                             int lane) {
  float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int blk = (u < 4 ? a : b) >> 6;  // a run never crosses a block (4-aligned, 64-element blocks)
    const float v = fabsf(x[u]);
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = (blk == k) ? fmaxf(m[k], v) : m[k];
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = fmaxf(m[k], __shfl_xor_sync(0xffffffffu, m[k], o));
  __half sh[4];
  float sv[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    sh[k] = __float2half_rn(__fdiv_rn(m[k], 127.0f));
    sv[k] = __half2float(sh[k]);
  }
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int blk = (u < 4 ? a : b) >> 6;
    const float s = blk == 0 ? sv[0] : blk == 1 ? sv[1] : blk == 2 ? sv[2] : sv[3];
    int c = 0;
    if (s != 0.f) c = (int)fminf(fmaxf(roundf(__fdiv_rn(x[u], s)), -127.f), 127.f);
    w[u >> 2] |= (uint32_t)(uint8_t)(int8_t)c << (8 * (u & 3));
  }
  *reinterpret_cast<uint32_t*>(codes + a) = w[0];
  *reinterpret_cast<uint32_t*>(codes + b) = w[1];
  if (lane == 0) {
    __half o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = sv[k] == 0.f ? __ushort_as_half(0) : sh[k];
    *reinterpret_cast<uint2*>(scales) = *reinterpret_cast<const uint2*>(o);
  }
}

__global__ void __launch_bounds__(256, 5) prep_kernel(const __half* __restrict__ q_raw, const __half* __restrict__ k_raw,
                                                   const __half* __restrict__ v_raw, const float* __restrict__ q_gamma,
                                                   const float* __restrict__ k_gamma, const int32_t* __restrict__ pos3,
                                                   int pos0, const __grid_constant__ PrepCfg cfg,
                                                   __half* __restrict__ qcur, __half* __restrict__ kcur,
                                                   int8_t* __restrict__ kq, __half* __restrict__ ksc,
                                                   int8_t* __restrict__ vq, __half* __restrict__ vsc) {
  __shared__ float2 s_cs[kD / 2];  // (cos, sin) of pair i
  pdl_begin();
  const int t = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rd = cfg.rotary_dim, h2 = rd / 2;
  const bool rot_lane = lane < (rd >> 3);
  int da, db;
  lane_dims(lane, rd, da, db);
  // this warp's rows r = warp + 8 j (j < 4, r < 28) and the gains: every load issued before any use
  constexpr int kRowsPerWarp = (kPrepRows + 7) / 8;
  uint2 ra[kRowsPerWarp], rb[kRowsPerWarp];
#pragma unroll
  for (int j = 0; j < kRowsPerWarp; ++j) {
    const int r = warp + 8 * j;
    ra[j] = make_uint2(0u, 0u);
    rb[j] = make_uint2(0u, 0u);
    if (r < kPrepRows) {
      const __half* src = r >= kHeads + kGroups ? v_raw + ((size_t)t * kGroups + (r - kHeads - kGroups)) * kD
                          : r >= kHeads ? k_raw + ((size_t)t * kGroups + (r - kHeads)) * kD
                                        : q_raw + ((size_t)t * kHeads + r) * kD;
      ra[j] = __ldg(reinterpret_cast<const uint2*>(src + da));
      rb[j] = __ldg(reinterpret_cast<const uint2*>(src + db));
    }
  }
  if (tid < h2) {
    int p = pos0 + t;
    if (pos3) p = __ldg(pos3 + 3 * t + (tid < cfg.sec0 ? 0 : (tid < cfg.sec0 + cfg.sec1 ? 1 : 2)));
    float sn, cs;
    sincosf(rope_angle(p, cfg.inv_hi[tid], cfg.inv_lo[tid]), &sn, &cs);
    s_cs[tid] = make_float2(cs, sn);
  }
  __syncthreads();
  // this lane's four rotation pairs 4 lane + u (rotated lanes only)
  float2 cs4[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) cs4[u] = rot_lane ? s_cs[da + u] : make_float2(1.f, 0.f);
  const int cell = pos0 + t;
#pragma unroll
  for (int j = 0; j < kRowsPerWarp; ++j) {
    const int r = warp + 8 * j;
    if (r >= kPrepRows) break;  // warp-uniform
    const bool is_v = r >= kHeads + kGroups, is_k = !is_v && r >= kHeads;
    const int g = is_v ? r - kHeads - kGroups : r - kHeads;  // group of a k or v row
    float x[8];
    unpack4(ra[j], x);
    unpack4(rb[j], x + 4);
    if (!is_v) {
      float ss = 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) ss = fmaf(x[u], x[u], ss);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float rs = 1.f / sqrtf(ss * (1.f / kD) + cfg.eps);
      const float* gam = is_k ? k_gamma : q_gamma;  // this lane's gains (L1-resident after the first CTAs)
      const float4 ga = __ldg(reinterpret_cast<const float4*>(gam + da));
      const float4 gb = __ldg(reinterpret_cast<const float4*>(gam + db));
      const float gw[8] = {ga.x, ga.y, ga.z, ga.w, gb.x, gb.y, gb.z, gb.w};
#pragma unroll
      for (int u = 0; u < 8; ++u) x[u] = x[u] * rs * gw[u];
      if (rot_lane) {  // pairs (x[u], x[4 + u]) = dims (a + u, a + u + rd / 2)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float lo = x[u], hi = x[4 + u];
          x[u] = lo * cs4[u].x - hi * cs4[u].y;
          x[4 + u] = hi * cs4[u].x + lo * cs4[u].y;
        }
      }
    }
    if (!is_k && !is_v) {  // qcur
      __half* dst = qcur + ((size_t)t * kHeads + r) * kD;
      *reinterpret_cast<uint2*>(dst + da) = make_uint2(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]));
      *reinterpret_cast<uint2*>(dst + db) = make_uint2(pack_half2(x[4], x[5]), pack_half2(x[6], x[7]));
      continue;
    }
    if (is_k) {  // the cache holds the fp16 rounding of the k row, quantised
      uint32_t ow[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        ow[u] = pack_half2(x[2 * u], x[2 * u + 1]);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&ow[u]));
        x[2 * u] = f.x;
        x[2 * u + 1] = f.y;
      }
      if (kcur) {
        __half* dst = kcur + ((size_t)t * kGroups + g) * kD;
        *reinterpret_cast<uint2*>(dst + da) = make_uint2(ow[0], ow[1]);
        *reinterpret_cast<uint2*>(dst + db) = make_uint2(ow[2], ow[3]);
      }
    }
    int8_t* codes = (is_k ? kq : vq) + ((size_t)cell * kGroups + g) * kD;
    __half* scale = (is_k ? ksc : vsc) + ((size_t)cell * kGroups + g) * kNB;
    quantize_row(x, da, db, codes, scale, lane);
  }
}

// ---------------------------------------------------------------- batched form
// qsa_prep_batched: the same rows for tokens of any sequences.  Token t has its own position(s) and
// its own pool cell, and its rows start at t times a stride (slices of a fused projection).
//
// The work is 27.7 KB of traffic a token, so the instructions per row decide whether it reaches the
// memory's rate.  A token's 28 rows are seven groups of four (six of q, one of k0 k1 v0 v1) and a warp takes
// a group at once: the four rows' sums of squares are reduced together (ten shuffles instead of twenty, one
// square root and division for all four), the arithmetic is in packed fp32 pairs, and the next group's loads
// are in flight meanwhile.  Lanes lie around the rotation as above, and each lane forms its own four (cos, sin)
// pairs, so nothing is shared and no barrier is met.
//   kWarps 1  a warp per token, all seven groups in turn, warps striding over the tokens
//   kWarps 7  seven warps per token, a group each: calls too small to fill the GPU with a warp per token
struct BatchedCfg {
  uint64_t turns[kD / 2];  // base^(-2i / rd) / (2 pi) as a 0.64 fixed-point fraction of a turn
  int rotary_dim, sec0, sec1, axes;
  float eps;
};

// (cos, sin) of p * base^(-2i / rd) for any 32-bit position: the product of the integer position and
// the fixed-point frequency wraps at whole turns by itself, so its top 32 bits are the angle as a
// signed fraction of a turn, within |p| 2^-54 turns (the frequency is a double) and 2^-32 turns of the
// exact one.
__device__ __forceinline__ float2 rope_cos_sin(int p, uint64_t turns) {
  const int64_t prod = (int64_t)((uint64_t)(int64_t)p * turns);
  float sn, cs;
  sincospif((float)(int)(prod >> 32) * 4.656612873077393e-10f, &sn, &cs);  // 2^-31: half turns
  return make_float2(cs, sn);
}

__device__ __forceinline__ float2 half2_f(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// Sums over the warp of four values a lane: lane l gets the total of v[l mod 4].
__device__ __forceinline__ float warp_sum4(const float (&v)[4], int lane) {
  const bool p = lane & 2, q = lane & 1;
  float a = p ? v[2] : v[0], b = p ? v[3] : v[1];
  a += __shfl_xor_sync(0xffffffffu, p ? v[0] : v[2], 2);
  b += __shfl_xor_sync(0xffffffffu, p ? v[1] : v[3], 2);
  float r = (q ? b : a) + __shfl_xor_sync(0xffffffffu, q ? a : b, 1);
  r += __shfl_xor_sync(0xffffffffu, r, 4);
  r += __shfl_xor_sync(0xffffffffu, r, 8);
  return r + __shfl_xor_sync(0xffffffffu, r, 16);
}

// The quantiser of one 256-element row (fp16 values) held in two 4-dim runs a lane, at dims a and b.  Eight
// lanes' runs never leave a 64-element block pair, so the block maxima take 8 shuffles: over 8 lanes, and over
// 16 where the block is that wide (`wide`); `one` says that both runs lie in one block.
//
// code = round-half-away(fp32(x / s)) is formed without a division: with x and s fp16 and |h| <= 127.5 a half
// integer, x - h s is a multiple of half the smaller step of the two, so x / s is either exactly h or at least
// 2^-12 away from it (also for subnormal s: multiples of 2^-25 against s < 2^-14).  The quotient by an
// approximate reciprocal is within 2^-15, so adding 1/2 + 2^-13 before truncating decides every case as the
// correctly rounded quotient does.
__device__ __forceinline__ void quantize_row_fast(const float2 (&x)[4], int a, int b, bool wide, bool one,
                                                  int8_t* codes, __half* scales) {
  float ma = fmaxf(fmaxf(fabsf(x[0].x), fabsf(x[0].y)), fmaxf(fabsf(x[1].x), fabsf(x[1].y)));
  float mb = fmaxf(fmaxf(fabsf(x[2].x), fabsf(x[2].y)), fmaxf(fabsf(x[3].x), fabsf(x[3].y)));
  if (one) ma = mb = fmaxf(ma, mb);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, o));
    mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, o));
  }
  const float ma8 = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, 8)), mb8 = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 8));
  ma = wide ? ma8 : ma;
  mb = wide ? mb8 : mb;
  const __half ha = __float2half_rn(__fdiv_rn(ma, 127.0f)), hb = __float2half_rn(__fdiv_rn(mb, 127.0f));
  const float fa = __half2float(ha), fb = __half2float(hb);
  const float ra = fa != 0.f ? __fdividef(1.f, fa) : 0.f, rb = fb != 0.f ? __fdividef(1.f, fb) : 0.f;
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const float v = (u & 1) ? x[u >> 1].y : x[u >> 1].x;
    const float q = fmaf(v, u < 4 ? ra : rb, copysignf(0.5f + 1.220703125e-4f, v));
    const int c = (int)fminf(fmaxf(q, -127.f), 127.f);
    w[u >> 2] |= (uint32_t)(c & 0xFF) << (8 * (u & 3));
  }
  *reinterpret_cast<uint32_t*>(codes + a) = fa != 0.f ? w[0] : 0u;  // scale 0: codes 0, those of NaN too
  *reinterpret_cast<uint32_t*>(codes + b) = fb != 0.f ? w[1] : 0u;
  if ((a & 63) == 0) scales[a >> 6] = ha;  // the lane that holds a block's first dims stores its scale
  if ((b & 63) == 0) scales[b >> 6] = hb;
}

constexpr int kPrepWarpTokens = 640;

template <int kWarps>
__global__ void __launch_bounds__(kWarps == 1 ? 128 : 32 * kWarps, kWarps == 1 ? 5 : 2)
    prep_batched_kernel(const __half* __restrict__ q_raw, const __half* __restrict__ k_raw,
                        const __half* __restrict__ v_raw, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                        const float* __restrict__ q_gamma, const float* __restrict__ k_gamma,
                        const int32_t* __restrict__ pos, const int32_t* __restrict__ cells, int n_tok, int64_t n_pool,
                        const __grid_constant__ BatchedCfg cfg, __half* __restrict__ qcur, __half* __restrict__ kcur,
                        int8_t* __restrict__ kq, __half* __restrict__ ksc, int8_t* __restrict__ vq,
                        __half* __restrict__ vsc, int* status) {
  constexpr int kGroupsOfRows = 7;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rd = cfg.rotary_dim;
  const bool rot = lane < (rd >> 3);
  int da, db;
  lane_dims(lane, rd, da, db);
  // block geometry of the lane's runs (see quantize_row_fast): rotations of 256 dims put a block's run over
  // 16 lanes, those of 128 do so for the first 16 lanes
  const bool one = (da >> 6) == (db >> 6);
  const bool wide = !one && rd >= 128;
  uint64_t turns[4];
  int axis[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = rot ? da + u : 0;
    turns[u] = rot ? cfg.turns[i] : 0;
    axis[u] = cfg.axes == 1 || i < cfg.sec0 ? 0 : (i < cfg.sec0 + cfg.sec1 ? 1 : 2);
  }
  pdl_begin();
  const int n_warps = kWarps == 1 ? (int)gridDim.x * (blockDim.x >> 5) : (int)gridDim.x;
  for (int t = kWarps == 1 ? (int)blockIdx.x * (blockDim.x >> 5) + warp : (int)blockIdx.x; t < n_tok; t += n_warps) {
    const int cell = __ldg(cells + t);
    const __half* src_q = q_raw + (int64_t)t * q_stride;
    const __half* src_k = k_raw + (int64_t)t * k_stride;
    const __half* src_v = v_raw + (int64_t)t * v_stride;
    uint2 ra[4], rb[4];  // the group in flight
    auto load = [&](int grp) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half* p = grp < 6 ? src_q + (grp * 4 + j) * kD : j < 2 ? src_k + j * kD : src_v + (j - 2) * kD;
        ra[j] = __ldg(reinterpret_cast<const uint2*>(p + da));
        rb[j] = __ldg(reinterpret_cast<const uint2*>(p + db));
      }
    };
    const int g0 = kWarps == 1 ? 0 : warp;
    load(g0);
    int ps[3];
#pragma unroll
    for (int x = 0; x < 3; ++x) ps[x] = __ldg(pos + (int64_t)t * cfg.axes + (cfg.axes == 3 ? x : 0));
    if (cell < 0 || cell >= n_pool) {  // warp-uniform
      if (cell != -1 && lane == 0) set_dev_status(status, QSA_DEV_BAD_ID);
      continue;
    }
    float2 cs[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      cs[u] = rot ? rope_cos_sin(axis[u] == 0 ? ps[0] : axis[u] == 1 ? ps[1] : ps[2], turns[u]) : make_float2(1.f, 0.f);
    const float2 c01 = make_float2(cs[0].x, cs[1].x), c23 = make_float2(cs[2].x, cs[3].x);
    const float2 s01 = make_float2(cs[0].y, cs[1].y), s23 = make_float2(cs[2].y, cs[3].y);
    const float2 n01 = make_float2(-s01.x, -s01.y), n23 = make_float2(-s23.x, -s23.y);
#pragma unroll 1
    for (int grp = g0; grp < kGroupsOfRows; grp += kWarps) {
      const bool is_kv = grp == 6;
      float2 x[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j][0] = half2_f(ra[j].x);
        x[j][1] = half2_f(ra[j].y);
        x[j][2] = half2_f(rb[j].x);
        x[j][3] = half2_f(rb[j].y);
      }
      if (kWarps == 1 && grp + 1 < kGroupsOfRows) load(grp + 1);
      float ss[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 v = mul2(x[j][0], x[j][0]);
#pragma unroll
        for (int u = 1; u < 4; ++u) v = fma2(x[j][u], x[j][u], v);
        ss[j] = v.x + v.y;
      }
      const float rs = 1.f / sqrtf(warp_sum4(ss, lane) * (1.f / kD) + cfg.eps);
      const float* gam = is_kv ? k_gamma : q_gamma;  // L1-resident
      const float4 ga = __ldg(reinterpret_cast<const float4*>(gam + da)), gb = __ldg(reinterpret_cast<const float4*>(gam + db));
      const float2 gw[4] = {make_float2(ga.x, ga.y), make_float2(ga.z, ga.w), make_float2(gb.x, gb.y), make_float2(gb.z, gb.w)};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j >= 2 && is_kv) break;  // v rows are used as given
        const float r = __shfl_sync(0xffffffffu, rs, j);
        const float2 r2 = make_float2(r, r);
        float2 y[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) y[u] = mul2(mul2(x[j][u], r2), gw[u]);
        const float2 a0 = fma2(y[2], n01, mul2(y[0], c01)), a1 = fma2(y[3], n23, mul2(y[1], c23));
        const float2 b0 = fma2(y[0], s01, mul2(y[2], c01)), b1 = fma2(y[1], s23, mul2(y[3], c23));
        const uint2 oa = make_uint2(pack_half2(a0.x, a0.y), pack_half2(a1.x, a1.y));
        const uint2 ob = make_uint2(pack_half2(b0.x, b0.y), pack_half2(b1.x, b1.y));
        __half* dst = !is_kv ? qcur + ((size_t)t * kHeads + grp * 4 + j) * kD
                             : (kcur ? kcur + ((size_t)t * kGroups + j) * kD : nullptr);
        if (dst) {
          *reinterpret_cast<uint2*>(dst + da) = oa;
          *reinterpret_cast<uint2*>(dst + db) = ob;
        }
        if (is_kv) {  // the cache holds the fp16 rounding of the k row, quantised
          x[j][0] = half2_f(oa.x);
          x[j][1] = half2_f(oa.y);
          x[j][2] = half2_f(ob.x);
          x[j][3] = half2_f(ob.y);
        }
      }
      if (is_kv) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          quantize_row_fast(x[j], da, db, wide, one, (j < 2 ? kq : vq) + ((size_t)cell * kGroups + (j & 1)) * kD,
                            (j < 2 ? ksc : vsc) + ((size_t)cell * kGroups + (j & 1)) * kNB);
      }
    }
  }
}

}  // namespace

cudaError_t launch_prep(const __half* q_raw, const __half* k_raw, const __half* v_raw, const float* q_gamma,
                        const float* k_gamma, const int32_t* pos3, int T, int pos0, double base, int rotary_dim,
                        float eps, const int* sections, __half* qcur, __half* kcur, int8_t* kq, __half* ksc,
                        int8_t* vq, __half* vsc, cudaStream_t stream) {
  PrepCfg cfg{};
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double inv = pow(base, -2.0 * i / rotary_dim);
    cfg.inv_hi[i] = (float)inv;
    cfg.inv_lo[i] = (float)(inv - (double)cfg.inv_hi[i]);
  }
  cfg.rotary_dim = rotary_dim;
  cfg.sec0 = sections[0];
  cfg.sec1 = sections[1];
  cfg.eps = eps;
  return launch_pdl(prep_kernel, dim3(T), dim3(256), 0, stream, q_raw, k_raw, v_raw, q_gamma, k_gamma, pos3, pos0, cfg,
                    qcur, kcur, kq, ksc, vq, vsc);
}

cudaError_t launch_prep_batched(const __half* q_raw, const __half* k_raw, const __half* v_raw, int64_t q_stride,
                                int64_t k_stride, int64_t v_stride, const float* q_gamma, const float* k_gamma,
                                const int32_t* pos, int axes, const int32_t* cells, int n_tok, int64_t n_pool,
                                double base, int rotary_dim, float eps, const int* sections, __half* qcur, __half* kcur,
                                int8_t* kq, __half* ksc, int8_t* vq, __half* vsc, int* status, cudaStream_t stream) {
  // The angles' table depends on (base, rd) alone: a thread's calls form it again only when these change (3 us).
  static thread_local BatchedCfg cfg{};
  static thread_local double cfg_base = 0.0;
  if (cfg_base != base || cfg.rotary_dim != rotary_dim) {
    // base^(-2i / rd) as products of the powers for i = 1, 2, 4, ...: a few roundings of a double each
    cfg.turns[0] = (uint64_t)llround(ldexp(1.0 / 6.283185307179586, 64));
    double inv[kD / 2];
    inv[0] = 1.0;
    for (int w = 1; w < rotary_dim / 2; w *= 2) {
      const double f = pow(base, -2.0 * w / rotary_dim);
      for (int i = 0; i < w; ++i) {
        inv[w + i] = inv[i] * f;
        cfg.turns[w + i] = (uint64_t)(inv[w + i] * (18446744073709551616.0 / 6.283185307179586));
      }
    }
    cfg_base = base;
  }
  cfg.rotary_dim = rotary_dim;
  cfg.sec0 = sections[0];
  cfg.sec1 = sections[1];
  cfg.axes = axes;
  cfg.eps = eps;
  auto launch = [&](auto kern, int grid, int threads) {
    return launch_pdl(kern, dim3(grid), dim3(threads), 0, stream, q_raw, k_raw, v_raw, q_stride, k_stride, v_stride,
                      q_gamma, k_gamma, pos, cells, n_tok, n_pool, cfg, qcur, kcur, kq, ksc, vq, vsc, status);
  };
  // A warp per token has less set-up a row and wins once it fills enough of the GPU: 512 tokens 8.2 us with
  // seven warps a token against 9.4 with one, 1,024 tokens 15.4 against 12.0, 8,191 tokens 102 against 47.
  if (n_tok >= kPrepWarpTokens) return launch(prep_batched_kernel<1>, 152 * 5, 128);
  return launch(prep_batched_kernel<7>, n_tok, 224);
}

}  // namespace qsa
