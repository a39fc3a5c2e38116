// Norms of queries and keys per head, the position rotation and the append, in one
// pass over the tick's new tokens; and the cos/sin tables of the rotation.
//
// A head's row x of D values becomes y = w * x / sqrt(mean(x^2) + eps) (without
// weights y = x); then pairs of its first R values are rotated, (a, b) -> (a cos - b
// sin, b cos + a sin), pair i being (y_i, y_{i + R/2}) or (y_2i, y_2i+1), with the
// table's entry of the token's position. All of it is fp32 and rounded once, to the
// type it is stored in: queries to q_out, keys and (unchanged) values to their slots.
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>

#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int THREADS = 128;

struct NormP {
  const void *q, *k, *v, *qw, *kw;
  int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh, qo_st, qo_sh, pool_slots;
  const int32_t* positions;
  const float2* cs;   // [max_pos][rot / 2]
  const int64_t* slots;
  void *kc, *vc, *qo;
  const float *ks, *vs;   // e4m3 caches
  float eps;
  int32_t max_pos, rot, Hq, Hkv, units, uq, uk;   // uq, uk: units of a token's queries / keys (values: as keys)
  int32_t* dev_status;
};

// The bound is HBM: (2 Hq + 2 Hkv) D values of the source type and 2 Hkv D of the cache's a token.
// 4192 tokens at 32 / 8 heads of 128 (bf16, 105 MB) take 24.3 us, 4.3 TB/s, 65 % of the copy
// bandwidth; 64 tokens 3.1 us, a launch and two rounds of loads. What is left is instructions:
// 580 a unit of 4 KB moved. Steps taken: angles and weights multiplied once a unit (41 -> 27.7 us),
// blocks of 128 at 64 registers (26.6), addresses stepped and the approximate root, which is within
// 2 ulp (24.3). Without gain: two or eight passes in flight (33, 35), a unit's loads issued while the
// one before is worked on (27 to 37), streaming loads (25.2).
//
// A warp's unit: ROWS consecutive head rows of one token, all queries, all keys or
// all values. LR = lanes of a row, a lane holding NV vectors of E values, E values
// apart by LR * E. The warp's 32 / LR rows of a pass are neighbours; PASSES of them
// are in flight at once. A lane keeps the angles and weights of its values for the
// whole unit: the table's row is then read once a unit, not once a head.
template <typename T, int D>
struct Shape {
  static constexpr int E = 16 / sizeof(T);
  static constexpr int NV = D / E > 32 ? D / E / 32 : 1;
  static constexpr int LR = D / E / NV;
  static constexpr int RPW = 32 / LR;
  static constexpr int PASSES = NV > 1 ? 2 : 4;
  static constexpr int ROWS = RPW * PASSES;
};

// e4m3 codes of x / scale, the float32 quotient rounded to nearest even, saturating
template <int E>
__device__ __forceinline__ void store_codes(const float (&x)[E], float scale, uint8_t* dst) {
  uint32_t w[E / 4];
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    const float2 a = make_float2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale));
    const float2 b = make_float2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale));
    w[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3) |
           ((uint32_t)__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3) << 16);
  }
  if constexpr (E == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t*>(dst) = w[0];
}

template <typename T, int E>
__device__ __forceinline__ void unpack(const uint4& raw, float (&x)[E]) {
  const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
  for (int i = 0; i < E; ++i) x[i] = to_f32(e[i]);
}

template <typename T, int D, bool NEAR, bool CODES>
__global__ void __launch_bounds__(THREADS, Shape<T, D>::NV > 1 ? 4 : 8) norm_rope_kernel(const NormP p) {
  using S = Shape<T, D>;
  constexpr int E = S::E, NV = S::NV, LR = S::LR, PASSES = S::PASSES;
  pdl_wait();
  pdl_trigger();   // what starts now waits for this grid's end before it writes, and before it relies on what it read
  const int unit = blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5);
  if (unit >= p.units) return;
  const int lane = threadIdx.x & 31, l = lane % LR, sub = lane / LR;
  const int per_token = p.uq + 2 * p.uk;
  const int tok = unit / per_token;
  const int64_t t = tok;
  int u = unit - tok * per_token;
  const int kind = u < p.uq ? 0 : u < p.uq + p.uk ? 1 : 2;   // queries, keys, values
  const bool first = u == 0;
  u -= kind == 0 ? 0 : kind == 1 ? p.uq : p.uq + p.uk;
  const int H = kind == 0 ? p.Hq : p.Hkv;
  const int h0 = u * S::ROWS + sub;
  const T* src = kind == 0 ? (const T*)p.q + t * p.q_st : kind == 1 ? (const T*)p.k + t * p.k_st
                                                                    : (const T*)p.v + t * p.v_st;
  const int64_t sh = kind == 0 ? p.q_sh : kind == 1 ? p.k_sh : p.v_sh;
  const int pos = __ldg(p.positions + t);
  const int64_t slot = kind == 0 ? 0 : __ldg(p.slots + t);
  uint4 raw[PASSES][NV];
  src += h0 * sh + l * E;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
      raw[i][v] = h0 + i * S::RPW < H ? *reinterpret_cast<const uint4*>(src + v * LR * E) : make_uint4(0, 0, 0, 0);
    src += S::RPW * sh;
  }
  if (pos < 0 || pos >= p.max_pos) {
    if (first && lane == 0) atomicOr(p.dev_status, PKV_DEV_BAD_POSITION);
    return;
  }
  if (kind != 0) {
    if (slot < 0) return;
    if (slot >= p.pool_slots) {
      if (u == 0 && lane == 0) atomicOr(p.dev_status, PKV_DEV_BAD_SLOT);
      return;
    }
  }
  const T* w = (const T*)(kind == 0 ? p.qw : kind == 1 ? p.kw : nullptr);
  const bool turned = kind != 2;
  const int half = p.rot / 2;
  // A value becomes r (x A + z B): z its partner, A its weight times the cosine, B the partner's
  // weight times the sine with the sign it takes, r what the norm divides by. Where nothing is
  // rotated the second term is left out.
  float2 A[NV][E / 2], B[NV][E / 2];
  int from[NV];   // lane that holds the partners (of vector v or 1 - v where other[v])
  bool other[NV], rotated[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int at = (v * LR + l) * E;
    rotated[v] = turned && at < p.rot;
    const bool hi = at >= half;
    const int mate = NEAR ? at : rotated[v] ? (hi ? at - half : at + half) : at;
    from[v] = (mate / E) % LR + sub * LR;
    other[v] = mate / (LR * E) != v;
    float own[E], its[E];
    if (w) {
      unpack<T, E>(__ldg(reinterpret_cast<const uint4*>(w + at)), own);
      unpack<T, E>(__ldg(reinterpret_cast<const uint4*>(w + mate)), its);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) own[e] = its[e] = 1.f;
    }
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      A[v][e / 2] = make_float2(own[e], own[e + 1]);
      B[v][e / 2] = make_float2(0.f, 0.f);
    }
    if (rotated[v]) {
      const float4* cs = reinterpret_cast<const float4*>(p.cs + (int64_t)pos * half + (NEAR ? at / 2 : hi ? at - half : at));
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        if constexpr (NEAR) {
          // pairs (e, e + 1): one angle
          const float4 q = __ldg(cs + e / 4);
          const float c = e & 2 ? q.z : q.x, sn = e & 2 ? q.w : q.y;
          A[v][e / 2] = make_float2(own[e] * c, own[e + 1] * c);
          B[v][e / 2] = make_float2(-its[e + 1] * sn, its[e] * sn);
        } else {
          const float4 q = __ldg(cs + e / 2);
          A[v][e / 2] = make_float2(own[e] * q.x, own[e + 1] * q.z);
          B[v][e / 2] = hi ? make_float2(its[e] * q.y, its[e + 1] * q.w) : make_float2(-its[e] * q.y, -its[e + 1] * q.w);
        }
      }
    }
  }
  // where this lane's first row goes, and how far its next one is, in bytes
  constexpr int CB = CODES ? 1 : (int)sizeof(T);
  char* dst = kind == 0 ? (char*)((T*)p.qo + t * p.qo_st + h0 * p.qo_sh + l * E)
                        : (char*)(kind == 1 ? p.kc : p.vc) + ((slot * p.Hkv + h0) * D + l * E) * CB;
  const int64_t dst_step = kind == 0 ? S::RPW * p.qo_sh * (int64_t)sizeof(T) : S::RPW * D * CB;
  const float* scales = kind == 1 ? p.ks : p.vs;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int h = h0 + i * S::RPW;
    float r = 1.f, y[NV][E];
    if (w) {   // (the same for the whole warp, as is kind)
      float2 sum2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float x[E];
        unpack<T, E>(raw[i][v], x);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 x2 = make_float2(x[e], x[e + 1]);
          sum2 = __ffma2_rn(x2, x2, sum2);
        }
      }
      float sum = sum2.x + sum2.y;
#pragma unroll
      for (int o = LR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      r = rsqrtf(fmaf(sum, 1.f / D, p.eps));
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      uint4 mate = raw[i][v];
      if constexpr (!NEAR) {
        if (turned) {
          // the partners' values as they came: one shuffle a 32-bit word
          const uint4 a = raw[i][0];
          mate.x = __shfl_sync(0xffffffffu, a.x, from[v]);
          mate.y = __shfl_sync(0xffffffffu, a.y, from[v]);
          mate.z = __shfl_sync(0xffffffffu, a.z, from[v]);
          mate.w = __shfl_sync(0xffffffffu, a.w, from[v]);
          if constexpr (NV > 1) {
            const uint4 b = raw[i][NV - 1];
            uint4 m1;
            m1.x = __shfl_sync(0xffffffffu, b.x, from[v]);
            m1.y = __shfl_sync(0xffffffffu, b.y, from[v]);
            m1.z = __shfl_sync(0xffffffffu, b.z, from[v]);
            m1.w = __shfl_sync(0xffffffffu, b.w, from[v]);
            if ((v == 1) != other[v]) mate = m1;
          }
        }
      }
      if (turned || CODES) {
        float x[E], z[E];
        unpack<T, E>(raw[i][v], x);
        if constexpr (!NEAR) unpack<T, E>(mate, z);
        const float2 r2 = make_float2(r, r);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          float2 u = __fmul2_rn(make_float2(x[e], x[e + 1]), A[v][e / 2]);
          if (rotated[v])
            u = __ffma2_rn(NEAR ? make_float2(x[e + 1], x[e]) : make_float2(z[e], z[e + 1]), B[v][e / 2], u);
          u = __fmul2_rn(u, r2);
          y[v][e] = u.x;
          y[v][e + 1] = u.y;
        }
      }
    }
    if (h >= H) continue;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = v * LR * E;
      if (CODES && kind != 0) {
        store_codes<E>(y[v], __ldg(scales + h), (uint8_t*)dst + at);
      } else {
        uint4 o = raw[i][v];
        if (turned) {
          T* d = reinterpret_cast<T*>(&o);
#pragma unroll
          for (int e = 0; e < E; ++e) d[e] = from_f32<T>(y[v][e]);
        }
        *reinterpret_cast<uint4*>((T*)dst + at) = o;
      }
    }
    dst += dst_step;
  }
}

template <typename T, int D>
cudaError_t launch(const NormRopeArgs& a, cudaStream_t st) {
  using S = Shape<T, D>;
  NormP p;
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.qw = a.q_weight;
  p.kw = a.k_weight;
  p.q_st = a.q_st;
  p.q_sh = a.q_sh;
  p.k_st = a.k_st;
  p.k_sh = a.k_sh;
  p.v_st = a.v_st;
  p.v_sh = a.v_sh;
  p.qo_st = a.qo_st;
  p.qo_sh = a.qo_sh;
  p.pool_slots = a.pool_slots;
  p.positions = a.positions;
  p.cs = (const float2*)a.cos_sin;
  p.slots = a.slots;
  p.kc = a.kc;
  p.vc = a.vc;
  p.qo = a.q_out;
  p.ks = a.k_scale;
  p.vs = a.v_scale;
  p.eps = a.eps;
  p.max_pos = a.max_pos;
  p.rot = a.rot;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.uq = (a.Hq + S::ROWS - 1) / S::ROWS;
  p.uk = (a.Hkv + S::ROWS - 1) / S::ROWS;
  const int64_t units = (int64_t)a.T * (p.uq + 2 * p.uk);
  if (units > INT32_MAX - THREADS) return cudaErrorInvalidValue;   // (a unit is 1 KB and more)
  p.units = (int32_t)units;
  p.dev_status = a.dev_status;
  const int64_t blocks = (units + THREADS / 32 - 1) / (THREADS / 32);
  KernelTimer timer("norm_rope_append", st);
  const bool codes = a.k_scale != nullptr;
  auto k = a.interleaved ? (codes ? norm_rope_kernel<T, D, true, true> : norm_rope_kernel<T, D, true, false>)
                         : (codes ? norm_rope_kernel<T, D, false, true> : norm_rope_kernel<T, D, false, false>);
  return launch_after_trigger(k, dim3((unsigned)blocks), dim3(THREADS), 0, st, p);
}

template <typename T>
cudaError_t by_dim(const NormRopeArgs& a, cudaStream_t s) {
  if (a.D == 64) return launch<T, 64>(a, s);
  if (a.D == 128) return launch<T, 128>(a, s);
  return launch<T, 256>(a, s);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t s) {
  if (a.dtype == PKV_F32) return by_dim<float>(a, s);
  if (a.dtype == PKV_F16) return by_dim<__half>(a, s);
  return by_dim<__nv_bfloat16>(a, s);
}

}  // namespace pkv

// Angle of pair i at position 1, f_i = base^(-2i/r), stretched for contexts longer than
// the model was trained on, and the table of cos and sin, all in double until stored.
extern "C" int pkv_rope_table_scaled(double base, int32_t rotary_dim, const pkv_rope_scaling* sc, int32_t max_pos,
                                     float* cos_sin) {
  if (!sc || !cos_sin) return PKV_E_NULL;
  if (!(base > 1.0) || !isfinite(base) || rotary_dim < 2 || rotary_dim % 2 != 0 || max_pos < 1) return PKV_E_SHAPE;
  if (sc->kind < PKV_ROPE_PLAIN || sc->kind > PKV_ROPE_RAMP) return PKV_E_SHAPE;
  if (!(sc->attention_factor >= 0.0) || !isfinite(sc->attention_factor)) return PKV_E_SHAPE;
  if (sc->kind != PKV_ROPE_PLAIN && (!(sc->factor >= 1.0) || !isfinite(sc->factor))) return PKV_E_SHAPE;
  const double TWO_PI = 6.283185307179586476925286766559;
  const int half = rotary_dim / 2;
  const double r = rotary_dim, L0 = sc->original_max_pos;
  if (sc->kind == PKV_ROPE_BASE && rotary_dim < 4) return PKV_E_SHAPE;
  if ((sc->kind == PKV_ROPE_BANDS || sc->kind == PKV_ROPE_RAMP) &&
      (!(L0 >= 1.0) || !isfinite(L0) || !(sc->low > 0.0) || !(sc->high > sc->low) || !isfinite(sc->high)))
    return PKV_E_SHAPE;
  const double b = sc->kind == PKV_ROPE_BASE ? base * pow(sc->factor, r / (r - 2.0)) : base;
  double first = 0.0, last = 0.0, factor = sc->attention_factor > 0.0 ? sc->attention_factor : 1.0;
  if (sc->kind == PKV_ROPE_RAMP) {
    // the pairs that turn `high` and `low` times over the original context bound the ramp
    first = floor(r * log(L0 / (sc->high * TWO_PI)) / (2.0 * log(base)));
    last = ceil(r * log(L0 / (sc->low * TWO_PI)) / (2.0 * log(base)));
    first = first < 0.0 ? 0.0 : first;
    last = last > r - 1.0 ? r - 1.0 : last;
    if (last <= first) last = first + 0.001;
    if (!(sc->attention_factor > 0.0)) factor = 0.1 * log(sc->factor) + 1.0;
  }
  for (int i = 0; i < half; ++i) {
    double f = pow(b, -2.0 * i / r);
    if (sc->kind == PKV_ROPE_LINEAR) f /= sc->factor;
    if (sc->kind == PKV_ROPE_BANDS) {
      const double turns = L0 * f / TWO_PI;   // over the original context
      double keep = (turns - sc->low) / (sc->high - sc->low);
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
      f = (1.0 - keep) * f / sc->factor + keep * f;
    }
    if (sc->kind == PKV_ROPE_RAMP) {
      double share = (i - first) / (last - first);
      share = share < 0.0 ? 0.0 : share > 1.0 ? 1.0 : share;
      f = f * (1.0 - share) + f / sc->factor * share;
    }
    for (int32_t p = 0; p < max_pos; ++p) {
      const double a = (double)p * f;
      cos_sin[((int64_t)p * half + i) * 2 + 0] = (float)(factor * cos(a));
      cos_sin[((int64_t)p * half + i) * 2 + 1] = (float)(factor * sin(a));
    }
  }
  return PKV_OK;
}
