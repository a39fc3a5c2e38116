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

constexpr int THREADS = 128, MIN_BLOCKS = 7;   // (72 registers a thread)

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
// 4192 tokens at 32 / 8 heads of 128 (bf16, 105 MB) take 23.5 us, 4.5 TB/s, 67 % of the copy bandwidth; 64
// tokens 2.8 us, a launch and two rounds of loads. What is left is latency: a warp loads, waits, computes,
// stores and leaves (issue slots 46 % busy, 37 % of the warps resident, at 72 registers). Steps taken: angles
// and weights multiplied once a unit (41 -> 27.7 us), blocks of 128 at 64 registers (26.6), addresses stepped
// and the approximate root, which is within 2 ulp (24.3), a lane holding both halves of its pairs (23.4; 64
// tokens 3.1 -> 2.8). Without gain: more passes in flight (33, 35), a unit's loads issued while the one before
// is worked on (27 to 37), streaming loads (25.2), two chunks a unit (24.6), six or eight blocks an SM in place
// of seven (23.9, 26.2).
//
// A warp's unit: ROWS consecutive head rows of one token, all queries, all keys or
// all values. A lane holds two vectors of E values of a row, those that the rotation pairs
// with one another where it pairs halves, so that nothing is exchanged for it; LR = D / (2 E) lanes hold
// a row. The warp's 32 / LR rows of a pass are neighbours; PASSES of them are in flight at once.
// A lane keeps the angles and weights of its values for the whole unit: the table's
// row is then read once a unit, not once a head.
template <typename T, int D>
struct Shape {
  static constexpr int E = 16 / sizeof(T);
  static constexpr int NV = 2;
  static constexpr int LR = D / E / NV;
  static constexpr int RPW = 32 / LR;
  static constexpr int PASSES = 2;
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
__global__ void __launch_bounds__(THREADS, MIN_BLOCKS) norm_rope_kernel(const NormP p) {
  using S = Shape<T, D>;
  constexpr int E = S::E, LR = S::LR, PASSES = S::PASSES, NVEC = D / E;
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
  // this lane's vectors: l and its partner half a rotation on, or two that are not rotated
  const int half = p.rot / 2, hv = NEAR ? 0 : half / E, rest = NVEC - 2 * hv;
  const bool paired = !NEAR && l < hv;
  const int at0 = (paired ? l : hv + l) * E, at1 = at0 + (paired ? hv : rest / 2) * E;
  const T* src = kind == 0 ? (const T*)p.q + t * p.q_st : kind == 1 ? (const T*)p.k + t * p.k_st
                                                                    : (const T*)p.v + t * p.v_st;
  const int64_t sh = kind == 0 ? p.q_sh : kind == 1 ? p.k_sh : p.v_sh;
  const int pos = __ldg(p.positions + t);
  const int64_t slot = kind == 0 ? 0 : __ldg(p.slots + t);
  uint4 raw[PASSES][2];
  src += h0 * sh;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const bool have = h0 + i * S::RPW < H;
    raw[i][0] = have ? *reinterpret_cast<const uint4*>(src + at0) : make_uint4(0, 0, 0, 0);
    raw[i][1] = have ? *reinterpret_cast<const uint4*>(src + at1) : make_uint4(0, 0, 0, 0);
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
  // A value becomes r (x A + z B): z its partner, A its weight times the cosine, B the partner's
  // weight times the sine with the sign it takes, r what the norm divides by. Where nothing is
  // rotated the second term is left out.
  float2 A[2][E / 2], B[2][E / 2];
  bool rotated[2];
  {
    float w0[E], w1[E];
    if (w) {
      unpack<T, E>(__ldg(reinterpret_cast<const uint4*>(w + at0)), w0);
      unpack<T, E>(__ldg(reinterpret_cast<const uint4*>(w + at1)), w1);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) w0[e] = w1[e] = 1.f;
    }
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      A[0][e / 2] = make_float2(w0[e], w0[e + 1]);
      A[1][e / 2] = make_float2(w1[e], w1[e + 1]);
      B[0][e / 2] = B[1][e / 2] = make_float2(0.f, 0.f);
    }
    const float2* cs = p.cs + (int64_t)pos * half;
    if constexpr (NEAR) {
      rotated[0] = turned && at0 < p.rot;
      rotated[1] = turned && at1 < p.rot;
#pragma unroll
      for (int v = 0; v < 2; ++v)
        if (rotated[v]) {
          const float4* c = reinterpret_cast<const float4*>(cs + (v ? at1 : at0) / 2);
#pragma unroll
          for (int e = 0; e < E; e += 4) {
            // pairs (e, e + 1), (e + 2, e + 3): an angle each
            const float4 q = __ldg(c + e / 4);
            const float2 a = A[v][e / 2], b = A[v][e / 2 + 1];
            A[v][e / 2] = make_float2(a.x * q.x, a.y * q.x);
            B[v][e / 2] = make_float2(-a.y * q.y, a.x * q.y);
            A[v][e / 2 + 1] = make_float2(b.x * q.z, b.y * q.z);
            B[v][e / 2 + 1] = make_float2(-b.y * q.w, b.x * q.w);
          }
        }
    } else {
      rotated[0] = rotated[1] = turned && paired;
      if (rotated[0]) {
        const float4* c = reinterpret_cast<const float4*>(cs + at0);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float4 q = __ldg(c + e / 2);
          const float2 a = A[0][e / 2], b = A[1][e / 2];
          A[0][e / 2] = make_float2(a.x * q.x, a.y * q.z);
          B[0][e / 2] = make_float2(-b.x * q.y, -b.y * q.w);
          A[1][e / 2] = make_float2(b.x * q.x, b.y * q.z);
          B[1][e / 2] = make_float2(a.x * q.y, a.y * q.w);
        }
      }
    }
  }
  // where this lane's first row goes, and how far its next one is, in bytes
  constexpr int CB = CODES ? 1 : (int)sizeof(T);
  char* dst = kind == 0 ? (char*)((T*)p.qo + t * p.qo_st + h0 * p.qo_sh)
                        : (char*)(kind == 1 ? p.kc : p.vc) + (slot * p.Hkv + h0) * D * CB;
  const int64_t dst_step = kind == 0 ? S::RPW * p.qo_sh * (int64_t)sizeof(T) : S::RPW * D * CB;
  const float* scales = kind == 1 ? p.ks : p.vs;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int h = h0 + i * S::RPW;
    float2 x[2][E / 2];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      float f[E];
      unpack<T, E>(raw[i][v], f);
#pragma unroll
      for (int e = 0; e < E; e += 2) x[v][e / 2] = make_float2(f[e], f[e + 1]);
    }
    float r = 1.f;
    if (w) {   // (the same for the whole warp, as is kind)
      float2 sum2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int e = 0; e < E / 2; ++e) sum2 = __ffma2_rn(x[v][e], x[v][e], sum2);
      float sum = sum2.x + sum2.y;
#pragma unroll
      for (int o = LR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      r = rsqrtf(fmaf(sum, 1.f / D, p.eps));
      // squares beyond the fp32 range (never of f16 values): zeros, which x A, beyond it too, times r is not. (r
      // multiplied first serves as well; 4192 tokens then take 23.9 us, this way 23.5.)
      if (!std::is_same<T, __half>::value && r == 0.f) {
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
          for (int e = 0; e < E / 2; ++e) x[v][e] = __fmul2_rn(x[v][e], make_float2(0.f, 0.f));
      }
    }
    if (h < H) {
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const int at = v ? at1 : at0;
        if (!turned && !CODES) {
          *reinterpret_cast<uint4*>((T*)dst + at) = raw[i][v];
          continue;
        }
        float y[E];
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          float2 o = __fmul2_rn(x[v][e], A[v][e]);
          if (rotated[v]) o = __ffma2_rn(NEAR ? make_float2(x[v][e].y, x[v][e].x) : x[1 - v][e], B[v][e], o);
          o = __fmul2_rn(o, make_float2(r, r));
          y[2 * e] = o.x;
          y[2 * e + 1] = o.y;
        }
        if (CODES && kind != 0) {
          store_codes<E>(y, __ldg(scales + h), (uint8_t*)dst + at);
        } else {
          uint4 o;
          T* d = reinterpret_cast<T*>(&o);
#pragma unroll
          for (int e = 0; e < E; ++e) d[e] = from_f32<T>(y[e]);
          *reinterpret_cast<uint4*>((T*)dst + at) = o;
        }
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
