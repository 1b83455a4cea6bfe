// Writing an 8-bit KV cache and reading it back.
//
// A vector x of d = 64 or 128 entries is stored as e4m3 codes of x * 2^-e, e the smallest exponent
// in [-40, 40] with max|x| <= 448 * 2^e (448: the largest e4m3 value). A power of two makes the
// scaling exact in both directions: the only rounding is the one to four significant bits (at most
// 2^-4 relative, half a step of e4m3's three fraction bits; at most 2^-10 * 2^e, half a subnormal step,
// for entries below 2^-6 * 2^e), and an entry read back and written again keeps its value.
// One exponent per vector and no finer: e4m3 has its own exponent bits, which cover the spread inside
// a vector, while a single factor per key can be applied to a score, and per value to its weight, so
// that attention uses the codes as they are.
//
// Both kernels move each byte once and are bound by HBM (long row lists) or by the launch (a step):
// d / 16 threads a vector, 16-byte accesses of neighbouring threads next to each other on the wide
// side, 4- or 8-byte ones on the code side. Writing 4096 fp32 rows of 40 heads of 128: 35 us, 6.0 TB/s;
// reading them back as bf16: 21.6 us, 5.8 TB/s (27.4 with a thread group for K and one for V); 64 rows of 8
// heads either way: 2.1 us, the time of a launch.
#include "kv8.cuh"
#include "kernels.h"

#include <cuda_fp16.h>

namespace eagle {
namespace {

constexpr int KV8_THREADS = 256;

// 16 bytes of T as floats and back.
__device__ __forceinline__ void unpack(const float*, const uint4& r, float* f) {
  f[0] = __uint_as_float(r.x); f[1] = __uint_as_float(r.y);
  f[2] = __uint_as_float(r.z); f[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void unpack(const __nv_bfloat16*, const uint4& r, float* f) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack(const float*, const float* f) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack(const __nv_bfloat16*, const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);   // exact: four significant bits
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Two floats -> two codes, the first in the low byte.
__device__ __forceinline__ uint32_t f32x2_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// A row's vector in the cache; -1: none (padding, or out of range: latched).
__device__ __forceinline__ long long vec_of(const Kv8& c, int row, int head, const int* row_seq, const int* row_slot,
                                            int* err, bool leader) {
  const int seq = row_seq[row], slot = row_slot[row];
  if (seq < 0) return -1;
  const long long vec = seq < c.max_batch && slot >= 0 && slot < c.cap ? kv8_vec(c, seq, head, slot) : -1;
  if (vec < 0 && leader) latch_error(err, DEVERR_BOUNDS);
  return vec;
}

template <typename T, int D>
__global__ void __launch_bounds__(KV8_THREADS)
    kv8_write_k(Kv8 c, const T* k, long long ldk, const T* v, long long ldv, long long n, const int* row_seq,
                const int* row_slot, int* err) {
  constexpr int VT = D / 16, E = 16 / sizeof(T), CH = 16 / E;   // threads a vector, entries a load, loads a thread
  PDL_ENTRY();
  const long long g = ((long long)blockIdx.x * KV8_THREADS + threadIdx.x) / VT;
  if (g >= n) return;
  const int t = threadIdx.x % VT;
  const int row = (int)(g / (2 * c.nkv)), part = (int)(g - (long long)row * 2 * c.nkv);   // K heads, V heads
  const bool is_v = part >= c.nkv;
  const int head = is_v ? part - c.nkv : part;
  const uint4* src = reinterpret_cast<const uint4*>((is_v ? v + row * ldv : k + row * ldk) + (size_t)head * D);
  const long long vec = vec_of(c, row, head, row_seq, row_slot, err, t == 0);
  const unsigned group = ((1u << VT) - 1) << ((threadIdx.x & 31) / VT * VT);
  if (vec < 0) return;   // the whole group
  uint4 raw[CH];
#pragma unroll
  for (int j = 0; j < CH; ++j) raw[j] = src[j * VT + t];
  float x[CH][E], top = 0.f;
  bool fine = true;
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    unpack((const T*)nullptr, raw[j], x[j]);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      top = fmaxf(top, fabsf(x[j][i]));
      fine = fine && isfinite(x[j][i]);
    }
  }
#pragma unroll
  for (int o = VT / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(group, top, o));
  fine = __all_sync(group, fine);
  // top = 1.f * 2^(ex - 127): 448 * 2^e = 1.75 * 2^(e + 8) covers it from e = ex - 127 - 8 on, one more
  // when its fraction passes .75 (and zero, subnormal or tiny maxima get the lowest exponent)
  const uint32_t b = __float_as_uint(top);
  int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(KV8_E_LO, min(KV8_E_HI, e));
  const float inv = __int_as_float((KV8_BIAS - e) << 23);
  uint8_t* dst = (is_v ? c.v : c.k) + vec * D;
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    uint32_t w[E / 4];
#pragma unroll
    for (int i = 0; i < E / 4; ++i)
      w[i] = fine ? f32x2_e4m3x2(x[j][4 * i] * inv, x[j][4 * i + 1] * inv) |
                        (f32x2_e4m3x2(x[j][4 * i + 2] * inv, x[j][4 * i + 3] * inv) << 16)
                  : 0u;
    if constexpr (E == 4) reinterpret_cast<uint32_t*>(dst)[j * VT + t] = w[0];
    else reinterpret_cast<uint2*>(dst)[j * VT + t] = make_uint2(w[0], w[1]);
  }
  if (t == 0) (is_v ? c.ve : c.ke)[vec] = fine ? (uint8_t)(e + KV8_BIAS) : (uint8_t)KV8_BAD;
}

// K and V of a (row, head) by the same threads: one look-up for both and twice the loads in flight.
template <typename T, int D>
__global__ void __launch_bounds__(KV8_THREADS)
    kv8_read_k(Kv8 c, T* k, long long ldk, T* v, long long ldv, long long n, const int* row_seq, const int* row_slot,
               int* err) {
  constexpr int VT = D / 16, E = 16 / sizeof(T), CH = 16 / E;
  PDL_ENTRY();
  const long long g = ((long long)blockIdx.x * KV8_THREADS + threadIdx.x) / VT;
  if (g >= n) return;
  const int t = threadIdx.x % VT;
  const int row = (int)(g / c.nkv), head = (int)(g - (long long)row * c.nkv);
  const long long vec = vec_of(c, row, head, row_seq, row_slot, err, t == 0);
  uint4* dst[2] = {reinterpret_cast<uint4*>(k + row * ldk + (size_t)head * D),
                   reinterpret_cast<uint4*>(v + row * ldv + (size_t)head * D)};
  if (vec < 0) {
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int j = 0; j < CH; ++j) dst[y][j * VT + t] = make_uint4(0, 0, 0, 0);
    return;
  }
  uint32_t w[2][CH][E / 4];
  uint8_t byte[2];
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const uint8_t* src = (y ? c.v : c.k) + vec * D;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      if constexpr (E == 4) {
        w[y][j][0] = reinterpret_cast<const uint32_t*>(src)[j * VT + t];
      } else {
        const uint2 u = reinterpret_cast<const uint2*>(src)[j * VT + t];
        w[y][j][0] = u.x;
        w[y][j][1] = u.y;
      }
    }
    byte[y] = (y ? c.ve : c.ke)[vec];
  }
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const float s = kv8_pow2(byte[y]);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      float x[E];
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        uint32_t h[2];
        e4m3x4_f16(w[y][j][i], h[0], h[1]);
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[z]));
          x[4 * i + 2 * z] = f.x * s;
          x[4 * i + 2 * z + 1] = f.y * s;
        }
      }
      dst[y][j * VT + t] = pack((const T*)nullptr, x);
    }
  }
}

}  // namespace

template <typename T>
static int write_t(cudaStream_t st, const Kv8& c, const void* k, long long ldk, const void* v, long long ldv, int R,
                   const int* row_seq, const int* row_slot, int* err) {
  const long long n = 2ll * R * c.nkv, blocks = (n * (c.d / 16) + KV8_THREADS - 1) / KV8_THREADS;
  if (blocks > 0x7fffffffll) return -1;
  if (c.d == 128)
    launch_k(kv8_write_k<T, 128>, dim3((unsigned)blocks), KV8_THREADS, 0, st, c, (const T*)k, ldk, (const T*)v, ldv, n,
             row_seq, row_slot, err);
  else
    launch_k(kv8_write_k<T, 64>, dim3((unsigned)blocks), KV8_THREADS, 0, st, c, (const T*)k, ldk, (const T*)v, ldv, n,
             row_seq, row_slot, err);
  return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

template <typename T>
static int read_t(cudaStream_t st, const Kv8& c, void* k, long long ldk, void* v, long long ldv, int R,
                  const int* row_seq, const int* row_slot, int* err) {
  const long long n = (long long)R * c.nkv, blocks = (n * (c.d / 16) + KV8_THREADS - 1) / KV8_THREADS;
  if (blocks > 0x7fffffffll) return -1;
  if (c.d == 128)
    launch_k(kv8_read_k<T, 128>, dim3((unsigned)blocks), KV8_THREADS, 0, st, c, (T*)k, ldk, (T*)v, ldv, n, row_seq,
             row_slot, err);
  else
    launch_k(kv8_read_k<T, 64>, dim3((unsigned)blocks), KV8_THREADS, 0, st, c, (T*)k, ldk, (T*)v, ldv, n, row_seq,
             row_slot, err);
  return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

int kv8_write(cudaStream_t st, const Kv8& c, bool f32, const void* k, long long ldk, const void* v, long long ldv, int R,
              const int* row_seq, const int* row_slot, int* err) {
  return f32 ? write_t<float>(st, c, k, ldk, v, ldv, R, row_seq, row_slot, err)
             : write_t<__nv_bfloat16>(st, c, k, ldk, v, ldv, R, row_seq, row_slot, err);
}

int kv8_read(cudaStream_t st, const Kv8& c, bool f32, void* k, long long ldk, void* v, long long ldv, int R,
             const int* row_seq, const int* row_slot, int* err) {
  return f32 ? read_t<float>(st, c, k, ldk, v, ldv, R, row_seq, row_slot, err)
             : read_t<__nv_bfloat16>(st, c, k, ldk, v, ldv, R, row_seq, row_slot, err);
}

}  // namespace eagle
