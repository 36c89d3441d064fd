// Head rows on their way to the caches and kernels of a decode step: the norm of a row, the
// position rotation of some of its dims, and the store in the row's own type or as e4m3 codes
// with a scale, all in one pass.
//
//   y = x                                            (no norm)
//   y_d = x_d / sqrt(mean(x^2) + eps) * w_d          (RMS norm, d < norm_dim)
//   y_d = (x_d - mean) / sqrt(var + eps) * w_d + b_d (layer norm, d < norm_dim)
//   (y_i, y_j) -> (y_i cos - y_j sin, y_j cos + y_i sin) over the pairs of the rotated dims
//   out = y, rounded once; or scale = max(amax |y|, 1e-12) / 448, out = e4m3(y / scale)
//
// Everything between load and store is float32 in registers.
// * qk_norm_rope_kernel: the query and key heads of every token (ls_qk_norm_rope).
// * cache_append_kernel: the new rows of a batch into the paged caches (ls_cache_append).
// Both move each byte once: bound by HBM for many rows, by the launch and one load latency for few.
// A row belongs to a group of G lanes holding NC 16-byte chunks each, lane gl the chunks gl + G i,
// with G small (4 for 128 bf16 values, four chunks each): a warp has several rows' loads in flight,
// and the work that is the same for every lane of a group (sums across lanes, addresses, positions)
// is shared by few.  A group works through consecutive rows and loads the next one before it
// finishes the one at hand.
// A row that is only rotated in neighbouring pairs moves its other chunks as they are.
// Rows whose sizes, strides or addresses are no multiple of 16 bytes take one element per lane, and with
// them the other operand of the call: 8,192 x 64 rows of 128 to e4m3 52 us in chunks, 733 one value at a
// time (a warp per row, each rotated value's partner normalised again); right for any form, not fast.
// Other forms of 8,192 x 64 bf16 rows of 128, from L2 where they fit: e4m3 without a norm 58 us, own type
// with the halves of all 128 dims rotated 90 (partners through shared memory), of 64 dims 54 (in the
// same lane).  1,024 x 128 rows of 576 moved with 64 dims rotated: 59 us, 5.1 TB/s.
// Appends into pinned host memory go at the link's rate: 8,192 latent rows in 181 us, 52 GB/s.
#pragma once
#include "common.cuh"

namespace ls {

struct HeadRows {
  int heads, dim;
  int cls;                 // RowClass
  int norm, norm_dim;      // LS_NORM_*
  int rope_begin;          // first rotated dim, -1: none
  int pairs;               // rotated pairs are neighbours (else the halves of the rotated dims)
  int w_bf16;
  float eps, inv_n;        // inv_n = 1 / norm_dim
  long long token_stride, head_stride;  // elements
  const void* x;
  const void* weight;      // NULL: 1
  const void* bias;        // NULL: 0
  // destination: [token][head] rows with strides, or pool rows of row_stride elements
  void* out;
  long long out_token_stride, out_head_stride;
  int e4m3;                // codes (and *scale) instead of the row's own type
  float* scale;
};

struct HeadRowsParams {
  HeadRows a, b;           // two operands; heads == 0: absent
  int tokens, rope_dim, max_pos;
  const float* cos_sin;    // [max_pos, rope_dim]: cosines, then sines
  const int* pos;          // [tokens], negative: token skipped (ls_qk_norm_rope)
  // ls_cache_append: token -> request and position
  int batch, max_pages;
  long long num_pages;
  const int* page_table;
  const int* start;
  const int* cu;
  unsigned blocks_a;       // blocks [0, blocks_a) work on operand a, the others on b
  int rows[2], more[2];    // of a and b: rows of each group, and how many groups take one more
};

// Elements per 16-byte chunk, and the lanes of the smallest group.
template <typename T>
struct RowShape;
template <>
struct RowShape<__nv_bfloat16> {
  static constexpr int kVec = 8, kGroup = 8;
};
template <>
struct RowShape<float> {
  static constexpr int kVec = 4, kGroup = 16;
};
// Row classes, by the chunks of a row: lanes and chunks per lane, and the blocks
// per SM that its registers leave room for.
//   class 0: up to 2 kGroup chunks (dim 128)    1: 4 (256)    2: 10 (640)    3: 16 (1024)
// bf16 rows of class 0 take four lanes with four chunks each: two thirds of the instructions of eight
// lanes with two (8,192 x 65 rows of 128 to e4m3: 65 us instead of 72; float32 rows, which are short of
// loads in flight instead, 33 us that way and 20 this).
template <typename T, int CLS>
struct RowClass {
  static constexpr bool kFew = CLS == 0 && sizeof(T) == 2;
  static constexpr int kLanes = RowShape<T>::kGroup * (CLS == 0 ? 1 : 2) / (kFew ? 2 : 1);
  static constexpr int kChunks = kFew ? 4 : CLS < 2 ? 2 : CLS == 2 ? 5 : 8;
};
template <typename T>
constexpr int head_row_blocks(int cls) {
  return cls == 3 ? 3 : cls == 2 || sizeof(T) == 2 ? 4 : 6;
}
constexpr int kHeadRowThreads = 128;
constexpr float kE4m3Max = 448.f;

// A chunk as it lies in memory, and as float32.
template <typename T, int VEC>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16, 8> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *(const uint4*)p; }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *(uint4*)p = u; }
  __device__ __forceinline__ void to(float* v) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(w[e] << 16);
      v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ void from(const float* v) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      __nv_bfloat162 two = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
      w[e] = *(uint32_t*)&two;
    }
    u = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Chunk<__nv_bfloat16, 4> {
  uint2 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *(const uint2*)p; }
  __device__ __forceinline__ void to(float* v) const {
    v[0] = __uint_as_float(u.x << 16);
    v[1] = __uint_as_float(u.x & 0xFFFF0000u);
    v[2] = __uint_as_float(u.y << 16);
    v[3] = __uint_as_float(u.y & 0xFFFF0000u);
  }
};
template <>
struct Chunk<float, 8> {
  float4 u, w;
  __device__ __forceinline__ void load(const float* p) { u = *(const float4*)p; w = *(const float4*)(p + 4); }
  __device__ __forceinline__ void to(float* v) const {
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w; v[4] = w.x; v[5] = w.y; v[6] = w.z; v[7] = w.w;
  }
};
template <>
struct Chunk<float, 4> {
  float4 u;
  __device__ __forceinline__ void load(const float* p) { u = *(const float4*)p; }
  __device__ __forceinline__ void store(float* p) const { *(float4*)p = u; }
  __device__ __forceinline__ void to(float* v) const { v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w; }
  __device__ __forceinline__ void from(const float* v) { u = make_float4(v[0], v[1], v[2], v[3]); }
};
template <>
struct Chunk<float, 2> {
  float2 u;
  __device__ __forceinline__ void load(const float* p) { u = *(const float2*)p; }
  __device__ __forceinline__ void to(float* v) const { v[0] = u.x; v[1] = u.y; }
};
template <>
struct Chunk<__nv_bfloat16, 1> {
  __nv_bfloat16 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *p; }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *p = u; }
  __device__ __forceinline__ void to(float* v) const { v[0] = __bfloat162float(u); }
  __device__ __forceinline__ void from(const float* v) { u = __float2bfloat16_rn(v[0]); }
};
template <>
struct Chunk<float, 1> {
  float u;
  __device__ __forceinline__ void load(const float* p) { u = *p; }
  __device__ __forceinline__ void store(float* p) const { *p = u; }
  __device__ __forceinline__ void to(float* v) const { v[0] = u; }
  __device__ __forceinline__ void from(const float* v) { u = v[0]; }
};

template <int VEC, typename T>
__device__ __forceinline__ void load_vec(const T* p, float* v) {
  Chunk<T, VEC> c;
  c.load(p);
  c.to(v);
}
template <int VEC>
__device__ __forceinline__ void load_weight(const void* w, int bf16, int d, float* v) {
  if (bf16) {
    load_vec<VEC>((const __nv_bfloat16*)w + d, v);
  } else {
    load_vec<VEC>((const float*)w + d, v);
  }
}
// Two float32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(*(unsigned long long*)&a), "l"(*(unsigned long long*)&b), "l"(*(unsigned long long*)&c));
  return *(float2*)&d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(*(unsigned long long*)&a), "l"(*(unsigned long long*)&b));
  return *(float2*)&d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(*(unsigned long long*)&a), "l"(*(unsigned long long*)&b));
  return *(float2*)&d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Two e4m3 codes.
__device__ __forceinline__ uint32_t e4m3x2(float2 v) {
  return __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
}

// Maxima that are NaN if an operand is (fmaxf takes the other one): a row's scale is by its definition.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float abs_max_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 448 / m, for m in [1e-12, inf].  (The fast quotient is 0 for divisors above 2^126, which rows without
// a norm can have: both sides are taken 2^9 times smaller, which changes no other bit.)
__device__ __forceinline__ float e4m3_inv_scale(float m) {
  return __fdividef(kE4m3Max * 0x1p-9f, m * 0x1p-9f);
}

template <int G>
__device__ __forceinline__ float group_sum(float v, uint32_t mask) {
#pragma unroll
  for (int o = G / 2; o; o >>= 1) v += __shfl_xor_sync(mask, v, o, G);
  return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v, uint32_t mask) {
#pragma unroll
  for (int o = G / 2; o; o >>= 1) v = max_nan(v, __shfl_xor_sync(mask, v, o, G));
  return v;
}

// (a, b) -> (a c - b s, b c + a s), two pairs at a time.
__device__ __forceinline__ void rotate2(float2& a, float2& b, float2 c, float2 s) {
  const float2 p = a, q = b, t = mul2(q, s);
  a = fma2(p, c, make_float2(-t.x, -t.y));
  b = fma2(p, s, mul2(q, c));
}
// The neighbouring pairs of one chunk, k values behind the first rotated one.
template <int VEC>
__device__ __forceinline__ void rotate_pairs(float2* v, const float* cs, int half, int k) {
  float c[VEC / 2], s[VEC / 2];
  load_vec<VEC / 2>(cs + k / 2, c);
  load_vec<VEC / 2>(cs + half + k / 2, s);
#pragma unroll
  for (int e = 0; e < VEC / 2; ++e) {
    const float p = v[e].x, q = v[e].y;
    v[e].x = p * c[e] - q * s[e];
    v[e].y = q * c[e] + p * s[e];
  }
}
// Rotation of halves whose partners are the same lane's next chunk.
template <int VEC, int G, int NC>
__device__ __forceinline__ void rotate_halves(float2 (*v)[VEC / 2], const float* cs, int half, int begin, int gl) {
#pragma unroll
  for (int i = 0; i + 1 < NC; ++i) {
    const int k = (gl + G * i) * VEC - begin;
    if (k < 0 || k >= half) continue;
    float2 c[VEC / 2], s[VEC / 2];
    load_vec<VEC>(cs + k, (float*)c);
    load_vec<VEC>(cs + half + k, (float*)s);
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) rotate2(v[i][e], v[i + 1][e], c[e], s[e]);
  }
}

// The norm of the VEC values at d, given mean and 1 / sqrt(var + eps); w, b: their weights and biases.
template <int VEC, int NORM>
__device__ __forceinline__ void norm_values(float mean, float inv, const float2* w, const float2* b, float2* y) {
#pragma unroll
  for (int e = 0; e < VEC / 2; ++e) {
    if (NORM == LS_NORM_LAYER) {
      y[e] = fma2(mul2(add2(y[e], both(-mean)), both(inv)), w[e], b[e]);
    } else {
      y[e] = mul2(mul2(y[e], both(inv)), w[e]);
    }
  }
}
template <int VEC>
__device__ __forceinline__ void load_params(const void* p, int bf16, int d, bool in, float absent, float2* v) {
  if (p && in) {
    load_weight<VEC>(p, bf16, d, (float*)v);
  } else {
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) v[e] = both(absent);
  }
}

// A row that is moved in its own type, its neighbouring pairs rotated; `in` holds its chunks.
template <typename T, int VEC, int G, int NC>
__device__ __forceinline__ void move_row(const HeadRows& r, Chunk<T, VEC>* in, const float* cs, int rope_dim, T* out,
                                         int gl) {
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int d = (gl + G * i) * VEC, k = d - r.rope_begin;
    if (d >= r.dim) break;
    if (r.rope_begin >= 0 && k >= 0 && k < rope_dim) {
      float2 v[VEC / 2];
      in[i].to((float*)v);
      rotate_pairs<VEC>(v, cs, rope_dim / 2, k);
      in[i].from((float*)v);
    }
    in[i].store(out + d);
  }
}

// One row by one group of G lanes (the lanes of `mask`): lane gl holds the values [(gl + G i) VEC,
// + VEC), i < NC, in v.  `out` is the row's destination, `scale` its scale's; kw holds the lane's
// weights if KEEP (RMS norm); swap is the group's scratch of rope_dim floats.  Every lane's part of x
// is in v when the first one stores: out may be x.
template <typename T, int VEC, int G, int NC, int NORM, bool KEEP>
__device__ __forceinline__ void head_row(const HeadRows& r, float2 (*v)[VEC / 2], const float* cs, int rope_dim,
                                         void* out, float* scale, int gl, uint32_t mask, const float2 (*kw)[VEC / 2],
                                         float* swap) {
  const int half = rope_dim / 2;
  const bool rope = r.rope_begin >= 0;
  float mean = 0.f, inv = 1.f;
  if (NORM != LS_NORM_NONE) {
    if (NORM == LS_NORM_LAYER) {
      float2 s = both(0.f);
#pragma unroll
      for (int i = 0; i < NC; ++i)
        if ((gl + G * i) * VEC < r.norm_dim) {
#pragma unroll
          for (int e = 0; e < VEC / 2; ++e) s = add2(s, v[i][e]);
        }
      mean = group_sum<G>(s.x + s.y, mask) * r.inv_n;
    }
    float2 s = both(0.f);
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if ((gl + G * i) * VEC < r.norm_dim) {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
          const float2 y = NORM == LS_NORM_LAYER ? add2(v[i][e], both(-mean)) : v[i][e];
          s = fma2(y, y, s);
        }
      }
    inv = rsqrtf(fmaf(group_sum<G>(s.x + s.y, mask), r.inv_n, r.eps));
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int d = (gl + G * i) * VEC;
      if (d >= r.norm_dim) continue;
      if (KEEP) {
        norm_values<VEC, NORM>(mean, inv, kw[i], nullptr, v[i]);
      } else {
        float2 w[VEC / 2], b[VEC / 2];
        load_params<VEC>(r.weight, r.w_bf16, d, true, 1.f, w);
        if (NORM == LS_NORM_LAYER) load_params<VEC>(r.bias, r.w_bf16, d, true, 0.f, b);
        norm_values<VEC, NORM>(mean, inv, w, b, v[i]);
      }
    }
  }
  if (rope) {
    if (r.pairs) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int k = (gl + G * i) * VEC - r.rope_begin;
        if (k >= 0 && k < rope_dim) rotate_pairs<VEC>(v[i], cs, half, k);
      }
    } else if (half == VEC * G && r.rope_begin % (VEC * G) == 0) {
      rotate_halves<VEC, G, NC>(v, cs, half, r.rope_begin, gl);
    } else {
      // the partners are another lane's: through shared memory
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int k = (gl + G * i) * VEC - r.rope_begin;
        if (k < 0 || k >= rope_dim) continue;
#pragma unroll
        for (int e = 0; e < VEC; e += 4)
          *(float4*)(swap + k + e) = make_float4(v[i][e / 2].x, v[i][e / 2].y, v[i][e / 2 + 1].x, v[i][e / 2 + 1].y);
      }
      __syncwarp(mask);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int k = (gl + G * i) * VEC - r.rope_begin;
        if (k < 0 || k >= rope_dim) continue;
        const bool first = k < half;
        const int other = first ? k + half : k - half, at = first ? k : k - half;
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
          float2 o[2], c[2], s[2];
          load_vec<4>(swap + other + e, (float*)o);
          load_vec<4>(cs + at + e, (float*)c);
          load_vec<4>(cs + half + at + e, (float*)s);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float2 sg = first ? make_float2(-s[q].x, -s[q].y) : s[q];
            v[i][e / 2 + q] = fma2(o[q], sg, mul2(v[i][e / 2 + q], c[q]));
          }
        }
      }
    }
  }
  if (r.e4m3) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int e = 0; e < VEC / 2; ++e) m = abs_max_nan(m, v[i][e].x, v[i][e].y);
    m = max_nan(group_max<G>(m, mask), 1e-12f);
    // codes of v * (448 / max): within 2^-22 of the quotient by the scale, which matters only to
    // values that near a tie of two codes: either is then half a step off
    const float isc = e4m3_inv_scale(m);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int d = (gl + G * i) * VEC;
      if (d >= r.dim) break;
      uint32_t w[VEC / 4];
#pragma unroll
      for (int e = 0; e < VEC / 4; ++e)
        w[e] = e4m3x2(mul2(v[i][2 * e], both(isc))) | (e4m3x2(mul2(v[i][2 * e + 1], both(isc))) << 16);
      if constexpr (VEC == 8) {
        *(uint2*)((uint8_t*)out + d) = make_uint2(w[0], w[1]);
      } else {
        *(uint32_t*)((uint8_t*)out + d) = w[0];
      }
    }
    if (gl == 0) *scale = m * (1.f / kE4m3Max);
  } else {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int d = (gl + G * i) * VEC;
      if (d >= r.dim) break;
      Chunk<T, VEC> c;
      c.from((float*)v[i]);
      c.store((T*)out + d);
    }
  }
}

// The same by a warp with one value per lane and load, for rows that are not made of 16-byte chunks:
// value lane + 32 i; the values stay in memory (at most 1,024 values, read from L1 again).
template <typename T>
__device__ __forceinline__ void head_row_plain(const HeadRows& r, const T* x, const float* cs, int rope_dim, void* out,
                                               float* scale) {
  constexpr int NC = 32;
  const int lane = lane_id(), half = rope_dim / 2;
  float mean = 0.f, inv = 1.f;
  if (r.norm != LS_NORM_NONE) {
    if (r.norm == LS_NORM_LAYER) {
      float s = 0.f;
      for (int d = lane; d < r.norm_dim; d += 32) s += (float)x[d];
      mean = group_sum<32>(s, 0xffffffffu) * r.inv_n;
    }
    float s = 0.f;
    for (int d = lane; d < r.norm_dim; d += 32) {
      const float y = (float)x[d] - mean;
      s = fmaf(y, y, s);
    }
    inv = rsqrtf(fmaf(group_sum<32>(s, 0xffffffffu), r.inv_n, r.eps));
  }
  auto normed = [&](int d) {
    float y = (float)x[d];
    if (r.norm == LS_NORM_NONE || d >= r.norm_dim) return y;
    float w = 1.f, b = 0.f;
    if (r.weight) load_weight<1>(r.weight, r.w_bf16, d, &w);
    if (r.bias) load_weight<1>(r.bias, r.w_bf16, d, &b);
    return fmaf((y - mean) * inv, w, b);
  };
  float v[NC], m = 0.f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int d = lane + 32 * i;
    v[i] = 0.f;
    if (d >= r.dim) continue;
    v[i] = normed(d);
    const int k = d - r.rope_begin;
    if (r.rope_begin >= 0 && k >= 0 && k < rope_dim) {
      const bool first = r.pairs ? (k & 1) == 0 : k < half;
      const int at = r.pairs ? k / 2 : (first ? k : k - half), by = r.pairs ? 1 : half;
      const float o = normed(first ? d + by : d - by), c = cs[at], sn = cs[half + at];
      v[i] = first ? v[i] * c - o * sn : v[i] * c + o * sn;
    }
    m = max_nan(m, fabsf(v[i]));
  }
  m = max_nan(group_max<32>(m, 0xffffffffu), 1e-12f);  // (and every lane has read x: out may be x)
  const float isc = e4m3_inv_scale(m);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int d = lane + 32 * i;
    if (d >= r.dim) continue;
    if (r.e4m3) {
      ((uint8_t*)out)[d] = __nv_cvt_float_to_fp8(v[i] * isc, __NV_SATFINITE, __NV_E4M3);
    } else {
      ((T*)out)[d] = (T)v[i];
    }
  }
  if (r.e4m3 && lane == 0) *scale = m * (1.f / kE4m3Max);
}

// The lanes of this thread's group of G.
template <int G>
__device__ __forceinline__ uint32_t group_mask() {
  return G == 32 ? 0xffffffffu : ((1u << (G & 31)) - 1u) << (lane_id() & ~(G - 1));
}

// The request of token t (cu[b] <= t < cu[b + 1], cu ascending; batch: behind the last one) for a
// whole block at once: every thread compares its share of the bounds, whose loads do not wait for
// one another as those of a search would.
__device__ __forceinline__ int block_token_request(const int* cu, int batch, int t) {
  int before = 0;
  for (int b0 = 0; b0 < batch; b0 += kHeadRowThreads) {
    const int b = b0 + threadIdx.x;
    before += __syncthreads_count(b < batch && cu[b + 1] <= t);
  }
  return before;
}

// Where a row goes: its destination (elements), its scale's index and its position; false if it
// is padding or out of range.
struct RowDest {
  long long at, scale;
  int pos;
};
template <bool APPEND>
__device__ __forceinline__ bool row_dest(const HeadRowsParams& p, const HeadRows& r, int t, int h, int gl, RowDest& w,
                                         int& req) {
  if constexpr (APPEND) {
    int i = 0;
    if (p.cu) {
      // (req: that of a row before this one)
      while (req < p.batch && t >= p.cu[req + 1]) ++req;
      if (req >= p.batch || t < p.cu[req]) return false;  // a padding row
      i = t - p.cu[req];
    } else {
      req = t;
    }
    const int start = p.start[req];
    if (start < 0) return false;  // a padding request
    const long long pos = (long long)start + i, lp = pos / LS_PAGE;
    const int page = lp < p.max_pages ? p.page_table[(long long)req * p.max_pages + lp] : -1;
    if (page < 0 || page >= p.num_pages || (r.rope_begin >= 0 && pos >= p.max_pos)) {
      if (gl == 0) flag(LS_DEV_BOUNDS);
      return false;
    }
    w.pos = (int)pos;
    w.scale = (long long)page * LS_PAGE + pos % LS_PAGE;
    w.at = w.scale * r.out_token_stride;
  } else {
    w.pos = p.pos[t];
    if (w.pos < 0) return false;  // a padding token
    if (r.rope_begin >= 0 && w.pos >= p.max_pos) {
      if (gl == 0) flag(LS_DEV_BOUNDS);
      return false;
    }
    w.scale = (long long)t * r.heads + h;
    w.at = t * r.out_token_stride + h * r.out_head_stride;
  }
  return true;
}

// Group g of an operand takes its share of consecutive rows and loads each before it finishes the
// one before it.
template <typename T, int VEC, int G, int NC, int NORM, bool APPEND>
__device__ __forceinline__ void head_rows_block(const HeadRowsParams& p, int which, int blk) {
  const HeadRows& r = which ? p.b : p.a;
  constexpr int kPer = kHeadRowThreads / G;
  constexpr bool KEEP = NC <= 4 && NORM == LS_NORM_RMS;
  const int total = p.tokens * r.heads;
  const int gl = threadIdx.x % G;
  const uint32_t mask = group_mask<G>();
  extern __shared__ __align__(16) float sm_swap[];
  float* swap = sm_swap + (threadIdx.x / G) * p.rope_dim;
  const int g = blk * kPer + threadIdx.x / G;
  int row = g * p.rows[which] + min(g, p.more[which]);
  const int end = min(total, row + p.rows[which] + (g < p.more[which]));
  int req = 0;
  if (APPEND && p.cu) {
    const int g0 = blk * kPer, t0 = g0 * p.rows[which] + min(g0, p.more[which]);
    req = block_token_request(p.cu, p.batch, t0);
  }
  if (row >= end) return;
  int t = row / r.heads, h = row - t * r.heads;
  Chunk<T, VEC> in[NC];
  const T* x = (const T*)r.x + t * r.token_stride + h * r.head_stride;
  auto load = [&](const T* from, Chunk<T, VEC>* to) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int d = (gl + G * i) * VEC;
      if (d < r.dim) to[i].load(from + d);
    }
  };
  load(x, in);
  float2 kw[KEEP ? NC : 1][VEC / 2];
  if (KEEP) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int d = (gl + G * i) * VEC;
      load_params<VEC>(r.weight, r.w_bf16, d, d < r.norm_dim, 1.f, kw[i]);
    }
  }
  const bool move = NORM == LS_NORM_NONE && !r.e4m3 && (r.pairs || r.rope_begin < 0);
  while (true) {
    const bool more = row + 1 < end;
    int t2 = t, h2 = h + 1;
    if (h2 == r.heads) {
      h2 = 0;
      ++t2;
    }
    const T* x2 = (const T*)r.x + t2 * r.token_stride + h2 * r.head_stride;
    RowDest w;
    if (NORM == LS_NORM_NONE && move) {
      Chunk<T, VEC> next[NC];
      if (more) load(x2, next);
      if (row_dest<APPEND>(p, r, t, h, gl, w, req))
        move_row<T, VEC, G, NC>(r, in, p.cos_sin + (long long)w.pos * p.rope_dim, p.rope_dim, (T*)r.out + w.at, gl);
#pragma unroll
      for (int i = 0; i < NC; ++i) in[i] = next[i];
    } else {
      float2 v[NC][VEC / 2];
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if ((gl + G * i) * VEC < r.dim) {
          in[i].to((float*)v[i]);
        } else {
#pragma unroll
          for (int e = 0; e < VEC / 2; ++e) v[i][e] = both(0.f);
        }
      }
      if (more) load(x2, in);
      if (row_dest<APPEND>(p, r, t, h, gl, w, req))
        head_row<T, VEC, G, NC, NORM, KEEP>(r, v, p.cos_sin + (long long)w.pos * p.rope_dim, p.rope_dim,
                                            r.e4m3 ? (void*)((uint8_t*)r.out + w.at) : (void*)((T*)r.out + w.at),
                                            r.scale + w.scale, gl, mask, kw, swap);
    }
    if (!more) return;
    __syncwarp(mask);  // swap is free again
    t = t2;
    h = h2;
    ++row;
  }
}
template <typename T, int CLS, bool APPEND>
__device__ __forceinline__ void head_rows_class(const HeadRowsParams& p, int which, int blk) {
  constexpr int V = RowShape<T>::kVec, G = RowClass<T, CLS>::kLanes, NC = RowClass<T, CLS>::kChunks;
  const int norm = which ? p.b.norm : p.a.norm;
  if (norm == LS_NORM_RMS) {
    head_rows_block<T, V, G, NC, LS_NORM_RMS, APPEND>(p, which, blk);
  } else if (norm == LS_NORM_LAYER) {
    head_rows_block<T, V, G, NC, LS_NORM_LAYER, APPEND>(p, which, blk);
  } else {
    head_rows_block<T, V, G, NC, LS_NORM_NONE, APPEND>(p, which, blk);
  }
}
template <typename T, bool APPEND>
__device__ __forceinline__ void head_rows_plain(const HeadRowsParams& p, const HeadRows& r, int blk) {
  const long long row0 = (long long)blk * (kHeadRowThreads / 32), row = row0 + warp_id();
  int req = 0;
  if (APPEND && p.cu) req = block_token_request(p.cu, p.batch, (int)row0);
  if (row >= (long long)p.tokens * r.heads) return;
  const int t = (int)(row / r.heads), h = (int)(row - (long long)t * r.heads);
  RowDest w;
  if (!row_dest<APPEND>(p, r, t, h, lane_id(), w, req)) return;
  head_row_plain<T>(r, (const T*)r.x + t * r.token_stride + h * r.head_stride,
                    p.cos_sin + (long long)w.pos * p.rope_dim, p.rope_dim,
                    r.e4m3 ? (void*)((uint8_t*)r.out + w.at) : (void*)((T*)r.out + w.at), r.scale + w.scale);
}

// MAXC: the larger class of the two operands' rows (each takes the code of its own class), or -1
// for the element-wise form.
template <typename T, int MAXC, bool APPEND>
__device__ __forceinline__ void head_rows_kernel(const HeadRowsParams& p) {
  const bool first = blockIdx.x < p.blocks_a;
  const HeadRows& r = first ? p.a : p.b;
  const int blk = (int)(first ? blockIdx.x : blockIdx.x - p.blocks_a);
  if constexpr (MAXC < 0) {
    head_rows_plain<T, APPEND>(p, r, blk);
  } else {
    if (MAXC == 0 || r.cls == 0) {
      head_rows_class<T, 0, APPEND>(p, !first, blk);
    } else if (MAXC == 1 || r.cls == 1) {
      if constexpr (MAXC >= 1) head_rows_class<T, 1, APPEND>(p, !first, blk);
    } else if (MAXC == 2 || r.cls == 2) {
      if constexpr (MAXC >= 2) head_rows_class<T, 2, APPEND>(p, !first, blk);
    } else {
      if constexpr (MAXC >= 3) head_rows_class<T, 3, APPEND>(p, !first, blk);
    }
  }
}
template <typename T, int MAXC>
__global__ void __launch_bounds__(kHeadRowThreads, head_row_blocks<T>(MAXC)) qk_norm_rope_kernel(const __grid_constant__ HeadRowsParams p) {
  head_rows_kernel<T, MAXC, false>(p);
}
template <typename T, int MAXC>
__global__ void __launch_bounds__(kHeadRowThreads, head_row_blocks<T>(MAXC)) cache_append_kernel(const __grid_constant__ HeadRowsParams p) {
  head_rows_kernel<T, MAXC, true>(p);
}

}  // namespace ls
