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

// Codes of two values already divided by their block's scale, a in the low
// nibble: the conversion instruction rounds to nearest even and saturates at
// 6, the rule of the format.
__device__ __forceinline__ uint32_t e2m1x2_of(float a, float b) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\tcvt.u32.u8 %0, t;\n\t}" : "=r"(r) : "f"(a), "f"(b));
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

// Byte permute whose selector nibbles keep their sign bit (the intrinsic drops it).
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

// Eight codes (element 0 in the low nibble) times a scale (BF16, both halves)
// -> eight BF16 values.  A BF16 E2M1 value is one of eight bit patterns: byte
// permutes look up their high and low bytes four codes at a time.  A selector
// nibble with bit 3 set (a negative code) makes the permute replicate the top
// bit of the byte it names, so looking codes up in bytes of 0x80 gives 0x80 or
// 0xFF, whose bit 6 is the sign.
__device__ __forceinline__ uint4 e2m1x8_to_bf16(uint32_t w, uint32_t scale2) {
  constexpr uint32_t kHi0 = 0x3F3F3F00u, kHi1 = 0x40404040u;   // 0 .5 1 1.5 | 2 3 4 6
  constexpr uint32_t kLo0 = 0xC0800000u, kLo1 = 0xC0804000u;
  const uint32_t m = w & 0x77777777u;
  const uint32_t ha = __byte_perm(kHi0, kHi1, m) | ((prmt(0x80808080u, 0x80808080u, w) << 1) & 0x80808080u);
  const uint32_t hb = __byte_perm(kHi0, kHi1, m >> 16) |
                      ((prmt(0x80808080u, 0x80808080u, w >> 16) << 1) & 0x80808080u);
  const uint32_t la = __byte_perm(kLo0, kLo1, m), lb = __byte_perm(kLo0, kLo1, m >> 16);
  uint4 o;
  o.x = mul_bf16x2(__byte_perm(la, ha, 0x5140), scale2);
  o.y = mul_bf16x2(__byte_perm(la, ha, 0x7362), scale2);
  o.z = mul_bf16x2(__byte_perm(lb, hb, 0x5140), scale2);
  o.w = mul_bf16x2(__byte_perm(lb, hb, 0x7362), scale2);
  return o;
}

// The same for a whole run of words under one scale, with fewer integer
// operations (they issue at half the rate of a product): the three magnitude
// bits of a code, put where a BF16 number has its lowest two exponent bits and
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

// A warp's lanes are dealt to rows in groups of 2^lg (the smallest power of
// two that holds a row's 8-value units, at most the whole warp).
__host__ inline int fp4_row_lanes_log2(int units) {
  int lg = 2;                                      // a block's four units stay in one group
  while ((1 << lg) < units && lg < 5) ++lg;
  return lg;
}

// ---------------------------------------------------------------------------
// Writing the cache: rows x [B, n, D] go to rows row0 .. row0+n-1 of every
// sequence.  HBM bound: 2 D (or 4 D) bytes read and (D-R)/2 + scales + 2 R
// written per row.  A lane holds 8 consecutive values (16 bytes of BF16), so a
// block is four neighbouring lanes and its maximum two shuffles.
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256)
quantize_entries_fp4_kernel(const T* __restrict__ x, long long n, long long rows, int D, int R, int lg,
                            uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                            __nv_bfloat16* __restrict__ rope, long long cache_rows, long long row0) {
  const int lane = threadIdx.x & 31;
  const int body = D - R, units = D >> 3, body_units = body >> 3, nblk = body >> 5;
  const int sbytes = fp4_scale_bytes(D, R);
  const int per_warp = 32 >> lg, sub = lane >> lg, ul = lane & ((1 << lg) - 1);
  const long long warp0 = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const long long warps = ((long long)gridDim.x * blockDim.x) >> 5;
  for (long long r0 = warp0 * per_warp; r0 < rows; r0 += warps * per_warp) {
    const long long r = r0 + sub;
    const bool live = r < rows;
    const long long b = live ? r / n : 0;
    const long long dst = b * cache_rows + row0 + (live ? r - b * n : 0);
    for (int u0 = 0; u0 < units; u0 += 1 << lg) {                       // uniform over the warp
      const int u = u0 + ul;
      const bool on = live && u < units;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
      if (on) {
        const T* p = x + r * D + 8 * u;
        load16(p, v);
        if constexpr (sizeof(T) == 4) load16(p + 4, v + 4);
      }
      uint32_t amax = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7FFFFFFFu);
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      if (on && u < body_units) {
        uint32_t word = 0, sbyte = 255;
        if (amax < 0x7F800000u) {
          const int X = mx_scale_exponent(amax);
          const float inv = pow2f(-X);
          sbyte = (uint32_t)(X + 127);
          // + 0 makes -0 a +0 (a zero is coded +0); the product by a power of two is exact
#pragma unroll
          for (int i = 0; i < 4; ++i) word |= e2m1x2_of((v[2 * i] + 0.f) * inv, (v[2 * i + 1] + 0.f) * inv) << (8 * i);
        }
        *reinterpret_cast<uint32_t*>(codes + dst * (body >> 1) + 4 * u) = word;
        if ((u & 3) == 0) scales[dst * sbytes + (u >> 2)] = (uint8_t)sbyte;
      } else if (on) {
        store_vec<8>(rope + dst * R + 8 * (u - body_units), v);
      }
    }
    if (live)
      for (int p = nblk + ul; p < sbytes; p += 1 << lg) scales[dst * sbytes + p] = 0;
  }
}

static cudaError_t launch_quantize_entries_fp4(const void* x, int B, long long n, int D, int R, lcsa_dtype dt,
                                               const lcsa_fp4_entries* c, long long cache_rows, long long row0,
                                               cudaStream_t st) {
  const long long rows = (long long)B * n;
  const int lg = fp4_row_lanes_log2(D >> 3);
  const long long want = (rows + 8 * (32 >> lg) - 1) / (8 * (32 >> lg));
  const int grid = (int)(want < 148LL * 64 ? want : 148LL * 64);
  count_launch();
  if (dt == LCSA_BF16)
    quantize_entries_fp4_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>((const __nv_bfloat16*)x, n, rows, D, R, lg, c->codes,
                                                                     c->scales, (__nv_bfloat16*)c->rope, cache_rows, row0);
  else
    quantize_entries_fp4_kernel<float><<<grid, 256, 0, st>>>((const float*)x, n, rows, D, R, lg, c->codes, c->scales,
                                                             (__nv_bfloat16*)c->rope, cache_rows, row0);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Reading the cache back: row r of sequence b is entry idx[b, r] (entry r
// without idx); -1 gives a zero row, any other index outside [0, cache_rows)
// a zero row and LCSA_DEV_BAD_INDEX.  HBM bound, mostly by the 2 D (4 D) bytes
// written per row.
// ---------------------------------------------------------------------------
template <typename To>
__global__ void __launch_bounds__(256)
dequantize_entries_fp4_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                              const __nv_bfloat16* __restrict__ rope, long long cache_rows, int D, int R, int lg,
                              const int32_t* __restrict__ idx, long long n, long long rows, To* __restrict__ out) {
  const int lane = threadIdx.x & 31;
  const int body = D - R, units = D >> 3, body_units = body >> 3;
  const int sbytes = fp4_scale_bytes(D, R);
  const int per_warp = 32 >> lg, sub = lane >> lg, ul = lane & ((1 << lg) - 1);
  const long long warp0 = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const long long warps = ((long long)gridDim.x * blockDim.x) >> 5;
  for (long long r = warp0 * per_warp + sub; r < rows; r += warps * per_warp) {
    const long long b = r / n;
    const long long j = idx ? (long long)__ldg(idx + r) : r - b * n;
    const bool there = j >= 0 && j < cache_rows;
    if (!there && j != -1 && ul == 0) report(LCSA_DEV_BAD_INDEX);
    const long long src = b * cache_rows + j;
    for (int u = ul; u < units; u += 1 << lg) {
      uint4 o = make_uint4(0, 0, 0, 0);                                 // eight BF16 values
      if (there) {
        if (u < body_units) {
          const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(codes + src * (body >> 1)) + u);
          o = e2m1x8_to_bf16(w, e8m0_bf16x2(__ldg(scales + src * sbytes + (u >> 2))));
        } else {
          o = __ldg(reinterpret_cast<const uint4*>(rope + src * R) + (u - body_units));
        }
      }
      To* p = out + r * D + 8 * u;
      if constexpr (sizeof(To) == 2) {
        *reinterpret_cast<uint4*>(p) = o;
      } else {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&o);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          reinterpret_cast<float4*>(p)[h] =
              make_float4(__uint_as_float(w[2 * h] << 16), __uint_as_float(w[2 * h] & 0xffff0000u),
                          __uint_as_float(w[2 * h + 1] << 16), __uint_as_float(w[2 * h + 1] & 0xffff0000u));
      }
    }
  }
}

static cudaError_t launch_dequantize_entries_fp4(const lcsa_fp4_entries* c, int B, long long cache_rows, int D, int R,
                                                 const int32_t* idx, long long n, void* out, lcsa_dtype odt,
                                                 cudaStream_t st) {
  const long long rows = (long long)B * n;
  const int lg = fp4_row_lanes_log2(D >> 3);
  const long long want = (rows + 8 * (32 >> lg) - 1) / (8 * (32 >> lg));
  const int grid = (int)(want < 148LL * 64 ? want : 148LL * 64);
  count_launch();
  if (odt == LCSA_BF16)
    dequantize_entries_fp4_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(c->codes, c->scales, (const __nv_bfloat16*)c->rope,
                                                                       cache_rows, D, R, lg, idx, n, rows,
                                                                       (__nv_bfloat16*)out);
  else
    dequantize_entries_fp4_kernel<float><<<grid, 256, 0, st>>>(c->codes, c->scales, (const __nv_bfloat16*)c->rope,
                                                               cache_rows, D, R, lg, idx, n, rows, (float*)out);
  return cudaGetLastError();
}

}  // namespace lcsa
