// FP4 entry cache: compressed entries held as MXFP4 (E2M1 codes with one
// power-of-two scale per 32 values), the rotary dims in BF16.  The 4-bit
// counterpart of the FP8 entry cache (DeepSeek-V4, "三、FP4量化": E2M1 with
// block scales; "KV Cache优化细节": the rotary dims stay BF16).
//
// Entry row x[0..D): body x[0..D-R) in blocks of 32, scale byte X + 127 with
// X = floor(log2 max|x|) - 2 in [-127, 127] (mxfp4.cuh; byte 255 and zero
// codes for a block that holds Inf or NaN), codes two per byte, the even
// element in the low nibble.  A row's scale bytes are padded with zeros to a
// multiple of 16, so that one 16-byte load brings a row's scales at D = 512.
// E2M1 has two significant bits and 0.5 * 2^-127 is a BF16 subnormal, so every
// value that the cache stands for is a BF16 number: reading back rounds nothing.
#pragma once
#include "common.cuh"
#include "mxfp4.cuh"

namespace lcsa {

__host__ __device__ __forceinline__ int fp4_scale_bytes(int D, int R) { return (((D - R) / 32) + 15) / 16 * 16; }

// Codes of eight values already divided by their block's scale, the first in
// the low nibble: the conversion instruction rounds to nearest even and
// saturates at 6, the rule of the format.
__device__ __forceinline__ uint32_t e2m1x8_of(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// BF16 bits of the scale 2^(s - 127) in both halves (s = 0: the subnormal
// 2^-127; s = 255: NaN, as the OCP format has it).
__device__ __forceinline__ uint32_t e8m0_bf16x2(uint32_t s) {
  uint32_t b = s << 7;
  b = s == 0 ? 0x0040u : (s == 255 ? 0x7FC0u : b);
  return b * 0x10001u;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Eight codes (element 0 in the low nibble) times a scale (BF16, both halves)
// -> eight BF16 values.  The three magnitude bits of a code, put where a BF16 number has its lowest two exponent bits and
// its highest fraction bit, are the E2M1 number times 2^-126 (the subnormal
// included), so a product with 2^126 and one with the signed scale finish it.
// Codes 2i and 2i+1 first move to the same place of the word's two halves.
__device__ __forceinline__ uint4 e2m1x8_by_products(uint32_t w, uint32_t scale2) {
  constexpr uint32_t kMag = 0x01C001C0u, kUp = 0x7E807E80u;                        // 2^126
  uint32_t x = (w & 0xF0F0FFFFu) | ((w << 12) & 0x0F0F0000u);                      // low half: 0 4 2 6
  x = (x & 0xFFFF0F0Fu) | ((w >> 12) & 0x0000F0F0u);                               // high half: 1 5 3 7
  const uint32_t d = x >> 6;
  const uint32_t m[4] = {x << 6, d << 4, x << 2, d}, sg[4] = {x << 12, x << 4, x << 8, x};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = mul_bf16x2(mul_bf16x2(m[i] & kMag, kUp), (sg[i] & 0x80008000u) ^ scale2);
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// A lane holds a block of 32 values, or 32 rotary dims.  A warp's lanes are
// dealt to rows in groups of 2^lg, the smallest power of two that holds a
// row's pieces (at most the whole warp).
__host__ __device__ inline int fp4_pieces(int D, int R) { return (D - R) / 32 + (R + 31) / 32; }
__host__ inline int fp4_row_lanes_log2(int pieces) {
  int lg = 0;
  while ((1 << lg) < pieces && lg < 5) ++lg;
  return lg;
}

// 32 bytes from or to a 32-byte aligned address.
__device__ __forceinline__ void fp4_ld32(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}
__device__ __forceinline__ void fp4_st32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
// 8 kN words (kN times 32 bytes), or 16 bytes at a time where the address is not 32-byte aligned.
template <int kN>
__device__ __forceinline__ void ld_words(const void* p, uint32_t* w, bool wide) {
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p) + 8 * i;
    if (wide) {
      fp4_ld32(q, w + 8 * i);
    } else {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(q)), b = __ldg(reinterpret_cast<const uint4*>(q) + 1);
      w[8 * i] = a.x; w[8 * i + 1] = a.y; w[8 * i + 2] = a.z; w[8 * i + 3] = a.w;
      w[8 * i + 4] = b.x; w[8 * i + 5] = b.y; w[8 * i + 6] = b.z; w[8 * i + 7] = b.w;
    }
  }
}
template <int kN>
__device__ __forceinline__ void st_words(void* p, const uint32_t* w, bool wide) {
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    uint32_t* q = reinterpret_cast<uint32_t*>(p) + 8 * i;
    if (wide) {
      fp4_st32(q, w + 8 * i);
    } else {
      reinterpret_cast<uint4*>(q)[0] = make_uint4(w[8 * i], w[8 * i + 1], w[8 * i + 2], w[8 * i + 3]);
      reinterpret_cast<uint4*>(q)[1] = make_uint4(w[8 * i + 4], w[8 * i + 5], w[8 * i + 6], w[8 * i + 7]);
    }
  }
}

// Row r of [B, n] rows: its sequence and place there (32-bit division where it fits).
struct Fp4Row {
  long long b, i;
};
__device__ __forceinline__ Fp4Row fp4_row(long long r, long long n) {
  const long long b = ((unsigned long long)(r | n) >> 32) ? r / n : (long long)((unsigned)r / (unsigned)n);
  return {b, r - b * n};
}

// A block of 32 values as loaded -> its codes and scale byte.  BF16 values are
// compared and scaled in pairs; adding +0 makes a -0 a +0 (a zero is coded +0),
// and the product by a power of two is exact, or below any code's range (its
// sign stays).
__device__ __forceinline__ uint32_t fp4_block(const uint32_t (&w)[16], uint4* codes) {       // 32 BF16
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
  const uint32_t amax = max(m << 16, m & 0xFFFF0000u);
  *codes = make_uint4(0, 0, 0, 0);
  if (amax >= 0x7F800000u) return 255;
  const int X = mx_scale_exponent(amax);
  const uint32_t inv = (__float_as_uint(pow2f(-X)) >> 16) * 0x10001u;
  uint32_t c[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t y;
      asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(w[4 * q + i]), "r"(inv), "r"(0u));
      v[2 * i] = __uint_as_float(y << 16);
      v[2 * i + 1] = __uint_as_float(y & 0xFFFF0000u);
    }
    c[q] = e2m1x8_of(v);
  }
  *codes = make_uint4(c[0], c[1], c[2], c[3]);
  return (uint32_t)(X + 127);
}
__device__ __forceinline__ uint32_t fp4_block(const uint32_t (&w)[32], uint4* codes) {       // 32 FP32
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) amax = max(amax, w[i] & 0x7FFFFFFFu);
  *codes = make_uint4(0, 0, 0, 0);
  if (amax >= 0x7F800000u) return 255;
  const int X = mx_scale_exponent(amax);
  const float inv = pow2f(-X);
  uint32_t c[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (__uint_as_float(w[8 * q + i]) + 0.f) * inv;
    c[q] = e2m1x8_of(v);
  }
  *codes = make_uint4(c[0], c[1], c[2], c[3]);
  return (uint32_t)(X + 127);
}

// ---------------------------------------------------------------------------
// Writing the cache: rows x [B, n, D] go to rows row0 .. row0+n-1 of every
// sequence.  2 D (or 4 D) bytes read and (D-R)/2 + scales + 2 R written per
// row.  A lane takes a whole block, so its maximum needs no shuffles and its
// addresses serve 32 values (with 8 values a lane the instructions were the
// bound: 28.7 us for 2 x 32768 rows of 512 BF16 values, 17.0 us with 32).
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256)
quantize_entries_fp4_kernel(const T* __restrict__ x, long long n, long long rows, int D, int R, int lg, bool wide,
                            uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                            __nv_bfloat16* __restrict__ rope, long long cache_rows, long long row0) {
  constexpr int kWords = 8 * sizeof(T);                                 // of 32 values
  const int lane = threadIdx.x & 31;
  const int body = D - R, nblk = body >> 5, pieces = fp4_pieces(D, R);
  const int sbytes = fp4_scale_bytes(D, R);
  const int ul = lane & ((1 << lg) - 1);
  const long long group0 = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> lg;
  const long long groups = ((long long)gridDim.x * blockDim.x) >> lg;
  for (long long r = group0; r < rows; r += groups) {
    const Fp4Row at = fp4_row(r, n);
    const long long dst = at.b * cache_rows + row0 + at.i;
    for (int p = ul; p < pieces; p += 1 << lg) {
      const T* src = x + r * D + 32 * p;
      if (p < nblk) {
        uint32_t w[kWords];
        ld_words<kWords / 8>(src, w, wide);
        uint4 c;
        scales[dst * sbytes + p] = (uint8_t)fp4_block(w, &c);
        *reinterpret_cast<uint4*>(codes + dst * (body >> 1) + 16 * p) = c;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int d = 32 * (p - nblk) + 8 * i;
          if (d < R) {
            float v[8];
            load16(src + 8 * i, v);
            if constexpr (sizeof(T) == 4) load16(src + 8 * i + 4, v + 4);
            store_vec<8>(rope + dst * R + d, v);
          }
        }
      }
    }
    for (int p = nblk + ul; p < sbytes; p += 1 << lg) scales[dst * sbytes + p] = 0;
  }
}

// Small blocks while the rows do not fill the machine with large ones.
static int fp4_block_threads(long long rows, int lg) { return rows << lg < 148LL * 256 ? 64 : 256; }
static int fp4_grid(long long rows, int lg, int threads) {
  const long long per_block = threads >> lg, want = (rows + per_block - 1) / per_block;
  return (int)(want < 148LL * 64 ? want : 148LL * 64);
}

static cudaError_t launch_quantize_entries_fp4(const void* x, int B, long long n, int D, int R, lcsa_dtype dt,
                                               const lcsa_fp4_entries* c, long long cache_rows, long long row0,
                                               cudaStream_t st) {
  const long long rows = (long long)B * n;
  const int lg = fp4_row_lanes_log2(fp4_pieces(D, R)), threads = fp4_block_threads(rows, lg), grid = fp4_grid(rows, lg, threads);
  const bool wide = (reinterpret_cast<uintptr_t>(x) & 31u) == 0 && D % (dt == LCSA_BF16 ? 16 : 8) == 0;
  count_launch();
  if (dt == LCSA_BF16)
    quantize_entries_fp4_kernel<__nv_bfloat16><<<grid, threads, 0, st>>>((const __nv_bfloat16*)x, n, rows, D, R, lg, wide, c->codes,
                                                                     c->scales, (__nv_bfloat16*)c->rope, cache_rows, row0);
  else
    quantize_entries_fp4_kernel<float><<<grid, threads, 0, st>>>((const float*)x, n, rows, D, R, lg, wide, c->codes, c->scales,
                                                             (__nv_bfloat16*)c->rope, cache_rows, row0);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Reading the cache back: row r of sequence b is entry idx[b, r] (entry r
// without idx); -1 gives a zero row, any other index outside [0, cache_rows)
// a zero row and LCSA_DEV_BAD_INDEX; so does, unreported, an entry from
// live_rows on (entries that nobody is to see, whatever they hold; without
// idx, n may go past the cache).  Mostly the 2 D (4 D) bytes written per row.  A block a lane, as above (131,072 selected rows of 512 values to BF16:
// 49.0 us with 8 values a lane, 43.2 us with 32).
// ---------------------------------------------------------------------------
template <typename To>
__global__ void __launch_bounds__(256)
dequantize_entries_fp4_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                              const __nv_bfloat16* __restrict__ rope, long long cache_rows, long long live_rows, int D, int R,
                              int lg, bool wide, const int32_t* __restrict__ idx, long long n, long long rows, To* __restrict__ out) {
  constexpr int kOut = sizeof(To) / 2;                                  // 32-byte pieces of 16 values
  const int lane = threadIdx.x & 31;
  const int body = D - R, nblk = body >> 5, pieces = fp4_pieces(D, R);
  const int sbytes = fp4_scale_bytes(D, R);
  const int ul = lane & ((1 << lg) - 1);
  const long long group0 = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> lg;
  const long long groups = ((long long)gridDim.x * blockDim.x) >> lg;
  for (long long r = group0; r < rows; r += groups) {
    const Fp4Row at = fp4_row(r, n);
    const long long e = idx ? (long long)__ldg(idx + r) : at.i;
    const bool there = e >= 0 && e < live_rows;
    if (idx && (e < -1 || e >= cache_rows) && ul == 0) report(LCSA_DEV_BAD_INDEX);
    const long long src = at.b * cache_rows + e;
    for (int p = ul; p < pieces; p += 1 << lg) {
      To* to = out + r * D + 32 * p;
      uint4 q[4];                                                       // 32 BF16 values
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = make_uint4(0, 0, 0, 0);
      int live = 4;                                                     // pieces of 8 values
      if (p < nblk) {
        if (there) {
          const uint4 c = __ldg(reinterpret_cast<const uint4*>(codes + src * (body >> 1)) + p);
          const uint32_t s2 = e8m0_bf16x2(__ldg(scales + src * sbytes + p));
          q[0] = e2m1x8_by_products(c.x, s2);
          q[1] = e2m1x8_by_products(c.y, s2);
          q[2] = e2m1x8_by_products(c.z, s2);
          q[3] = e2m1x8_by_products(c.w, s2);
        }
      } else {
        live = min(4, (R - 32 * (p - nblk)) / 8);
        if (there) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < live) q[i] = __ldg(reinterpret_cast<const uint4*>(rope + src * R + 32 * (p - nblk)) + i);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {                                     // 16 values at a time
        const uint32_t w[8] = {q[2 * h].x, q[2 * h].y, q[2 * h].z, q[2 * h].w,
                               q[2 * h + 1].x, q[2 * h + 1].y, q[2 * h + 1].z, q[2 * h + 1].w};
        uint32_t f[8 * kOut];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if constexpr (sizeof(To) == 2) {
            f[i] = w[i];
          } else {
            f[2 * i] = w[i] << 16;
            f[2 * i + 1] = w[i] & 0xFFFF0000u;
          }
        }
        if (live >= 2 * h + 2) {
          st_words<kOut>(to + 16 * h, f, wide);
        } else if (live == 2 * h + 1) {                                 // the last 8 of the rotary dims
          uint4* o = reinterpret_cast<uint4*>(to + 16 * h);
          o[0] = make_uint4(f[0], f[1], f[2], f[3]);
          if constexpr (sizeof(To) == 4) o[1] = make_uint4(f[4], f[5], f[6], f[7]);
        }
      }
    }
  }
}

static cudaError_t launch_dequantize_entries_fp4(const lcsa_fp4_entries* c, int B, long long cache_rows, int D, int R,
                                                 const int32_t* idx, long long n, void* out, lcsa_dtype odt,
                                                 cudaStream_t st, long long live_rows) {
  const long long rows = (long long)B * n;
  const int lg = fp4_row_lanes_log2(fp4_pieces(D, R)), threads = fp4_block_threads(rows, lg), grid = fp4_grid(rows, lg, threads);
  const bool wide = (reinterpret_cast<uintptr_t>(out) & 31u) == 0 && D % (odt == LCSA_BF16 ? 16 : 8) == 0;
  count_launch();
  if (odt == LCSA_BF16)
    dequantize_entries_fp4_kernel<__nv_bfloat16><<<grid, threads, 0, st>>>(c->codes, c->scales, (const __nv_bfloat16*)c->rope,
                                                                       cache_rows, live_rows, D, R, lg, wide, idx, n, rows,
                                                                       (__nv_bfloat16*)out);
  else
    dequantize_entries_fp4_kernel<float><<<grid, threads, 0, st>>>(c->codes, c->scales, (const __nv_bfloat16*)c->rope,
                                                               cache_rows, live_rows, D, R, lg, wide, idx, n, rows, (float*)out);
  return cudaGetLastError();
}

}  // namespace lcsa
