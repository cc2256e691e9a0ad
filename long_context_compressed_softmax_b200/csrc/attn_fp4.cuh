// Core attention over the FP4 entry cache on tcgen05 tensor cores (BF16
// queries, H = 64 heads, D = 512, rotary R = 64): multi-query attention of 64
// heads over one shared K=V head whose entries arrive as E2M1 codes, then the
// window of raw BF16 rows, a per-head sink in the denominator, partial RoPE
// and the -t rotation of the output.
//
//   out = R(-t) sum_j e^(l_j) R(p_j) k_j / (sum_j e^(l_j) + e^sink),  l_j = scale (R(t) q) . (R(p_j) k_j)
//
// A tile's keys are made for one query alone, so they are turned by p_j - t:
// neither the query nor the output is rotated then, and the queries need no
// rounding.  Tiles of 64 keys, three in flight:
//   S = Q K^T   M = 64 heads, N = 64 keys, A (the queries) from tensor memory
//   softmax     two threads a head, the reference moves when a logit exceeds it by 2^8
//   O += P K    M = 64, N = 2 x 256 dims
// The 16-bit K tile is made in shared memory from 368 bytes a key: fourteen
// warps expand codes and turn rotary dims while the tiles before are multiplied.
// Forms with 128 keys or dims on the M side (full-rate MMAs) were measured
// first and are slower here: with N = 64 both operands' shared-memory reads
// take the whole bandwidth of shared memory, which the expansion needs too.
//
// A sequencer warp turns queries, selections and windows into a ring of tile
// descriptions that every role follows, so only it knows how they map.
//
// Long key lists of few queries are split over the CTAs of a cluster: each
// leaves its partial O in its shared memory and all of them add up a share of
// it over distributed shared memory, in a fixed order.
#pragma once
#include <atomic>
#include <cstddef>

#include "tc_ptx.cuh"
#include "fp4cache.cuh"

namespace lcsa {

constexpr int kF4Keys = 64;                         // keys per tile
constexpr int kF4Stages = 3;
constexpr int kF4Code = 10, kF4Rot = 4;             // warps that expand codes; that turn the rotary dims
// A warp's scheduler is its number mod 4.  The expanding warps keep three of
// the four schedulers busy; the first has fewer of them, for the warp that
// issues the MMAs (whose instructions would otherwise wait their turn behind
// the expansion: 1,538 against 1,371 us for 2048 rows of 2176 keys) and the
// sequencer.  By number, warps 0 to 15: which of the code warps (0-9) and of
// the rotary warps (10-13); 15 neither.
constexpr unsigned long long kF4Roles = 0x9DC8B76A543F210Full;
constexpr int kF4MmaWarp = 0, kF4SeqWarp = 4;
constexpr int kF4SmWarp0 = 16;                      // 4 softmax warps
constexpr int kF4XtWarp0 = 20;                      // 4 transition warps: queries in, outputs out
constexpr int kF4Threads = 24 * 32;
constexpr int kF4Readers = kF4Code + kF4Rot + 4 + 4 + 1;   // warps that take every tile description
constexpr int kF4Ring = 8;                          // tile descriptions in flight
constexpr int kF4MaxSplits = 16;
constexpr uint32_t kF4Region = 64 * 128;            // 64 keys of 64 dims
constexpr uint32_t kF4KBytes = 8 * kF4Region;       // a K tile
constexpr uint32_t kF4PBytes = 64 * 128;

struct F4Tile {
  int32_t row[kF4Keys];      // row of each key within its sequence, -1: no key
  int32_t kind;              // kF4Entries ..
  int32_t first, last;       // of its query (and split)
  int32_t q_row;             // query row (b * Tq + i)
  uint32_t mask[2];          // keys that are there
  int32_t pad[4];
  long long base;            // first row of the sequence in the cache or the raw buffer
  long long pos0, step;      // position of row r, from the query's: pos0 + r * step
};
constexpr int kF4Entries = 0, kF4Window = 1, kF4Empty = 2, kF4End = 3;
static_assert(sizeof(F4Tile) % 16 == 0, "tile description");

// shared-memory carve-up, offsets from the 1 KB aligned base
constexpr uint32_t kF4OffP = kF4Stages * kF4KBytes;                    // two P tiles
constexpr uint32_t kF4OffTab = kF4OffP + 2 * kF4PBytes;
constexpr uint32_t kF4OffStats = kF4OffTab + kF4Ring * sizeof(F4Tile); // [2 items][64] (reference, sum, exact sum)
constexpr uint32_t kF4OffRef = kF4OffStats + 2 * 64 * 16;              // [64] of this split
constexpr uint32_t kF4OffL = kF4OffRef + 64 * 4;                       // [64]
constexpr uint32_t kF4OffE = kF4OffL + 64 * 4;                         // [64]
constexpr uint32_t kF4OffWgt = kF4OffE + 64 * 4;                       // [splits][64] merge weights
constexpr uint32_t kF4OffBar = kF4OffWgt + kF4MaxSplits * 64 * 4;
constexpr uint32_t kF4BTabFull = kF4OffBar, kF4BTabEmpty = kF4BTabFull + 8 * kF4Ring;
constexpr uint32_t kF4BKFull = kF4BTabEmpty + 8 * kF4Ring, kF4BKEmpty = kF4BKFull + 8 * kF4Stages;
constexpr uint32_t kF4BSFull = kF4BKEmpty + 8 * kF4Stages, kF4BSFree = kF4BSFull + 16, kF4BPFull = kF4BSFree + 16;
constexpr uint32_t kF4BPvDone = kF4BPFull + 16, kF4BOFree = kF4BPvDone + 16, kF4BStats = kF4BOFree + 16;
constexpr uint32_t kF4BQReady = kF4BStats + 16, kF4BSDone = kF4BQReady + 8, kF4BDrain = kF4BSDone + 8;
constexpr int kF4Bars = 2 * kF4Ring + 2 * kF4Stages + 15;
static_assert(kF4BDrain + 8 == kF4OffBar + 8 * kF4Bars, "barriers");
constexpr size_t kF4Smem = 1024 + kF4OffBar + kF4Bars * 8;
static_assert(kF4Smem <= 232448, "FP4 attention shared memory exceeds 227 KB");

// tensor memory: lanes 0-15 of every sub-partition hold S of two tiles (64
// columns each) and the queries (256 columns), lanes 16-31 O (512 columns)
constexpr uint32_t kF4TmQ = 128, kF4TmO = 16u << 16;

struct F4Args {
  const uint8_t* codes;
  const uint8_t* scales;
  const __nv_bfloat16* rope;
  const __nv_bfloat16* q;
  const __nv_bfloat16* kv;
  const int32_t* idx;
  const float* sink;
  void* out;
  float* lse;
  int B, Tq, n_q, Nc, k, Tkv, m, W;      // the first n_q of Tq rows of every sequence
  int sparse, splits, out_bf16;
  long long rows, q_pos0, kv_pos0;
  float scale_log2;
  // turns per position of rotary pair i, theta_i / 2 pi, as a 64-bit binary
  // fraction: a position's angle is the low 64 bits of position * turn,
  // exact to 2^-64 turns per step of position
  unsigned long long turn[32];
};

// Query `it` of the launch: the last positions first (they have the most keys).
struct F4Query {
  long long row, t;
  int b;
};
__device__ __forceinline__ F4Query f4_query(const F4Args& g, int it) {
  F4Query q;
  const int r = it / g.B;
  q.b = it - r * g.B;
  q.row = (long long)q.b * g.Tq + g.n_q - 1 - r;
  q.t = g.q_pos0 + g.n_q - 1 - r;
  return q;
}

__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(uint32_t a, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

// (cos, sin) of an angle given as a 64-bit fraction of a turn: the MUFU's sine
// and cosine (2^-20 absolute) of an angle within half a turn, far below the
// BF16 rounding of the rotated key.
__device__ __forceinline__ void turn_cs(unsigned long long ph, float* c, float* s) {
  const float a = (float)(int)(ph >> 32) * 1.4629180792671596e-9f;   // 2 pi / 2^32
  *c = __cosf(a);
  *s = __sinf(a);
}
__device__ __forceinline__ uint32_t rotate_pair(uint32_t x, float c, float s) {
  const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x));
  const __nv_bfloat162 o = __floats2bfloat162_rn(f.x * c - f.y * s, f.x * s + f.y * c);
  return *reinterpret_cast<const uint32_t*>(&o);
}

// Shared memory by 32-bit address, with constant offsets folded into the access.
template <int kOff = 0>
__device__ __forceinline__ uint32_t f4_lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1 + %2];" : "=r"(v) : "r"(a), "n"(kOff) : "memory");
  return v;
}
template <int kOff = 0>
__device__ __forceinline__ unsigned long long f4_lds64(uint32_t a) {
  unsigned long long v;
  asm volatile("ld.shared.u64 %0, [%1 + %2];" : "=l"(v) : "r"(a), "n"(kOff) : "memory");
  return v;
}
template <int kOff = 0>
__device__ __forceinline__ void f4_sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0 + %1], {%2,%3,%4,%5};" ::"r"(a), "n"(kOff), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
template <int kOff = 0>
__device__ __forceinline__ void f4_arrive(uint32_t a) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0 + %1];\n\t}" ::"r"(a), "n"(kOff) : "memory");
}
template <int kOff>
__device__ __forceinline__ bool f4_try_wait(uint32_t a, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1 + %2], %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(a), "n"(kOff), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait of a whole warp (the limit and report of tc::mbar_wait).  The
// waiting itself is a function: inlined at every wait it adds a tenth to code
// that is too large for the instruction cache as it is.
static __device__ __noinline__ bool f4_wait_slow(uint32_t a, uint32_t parity) {
  bool got = false;
  const uint64_t t0 = tc::globaltimer();
  do {
#pragma unroll 1
    for (int i = 0; i < 64 && !got; ++i) got = f4_try_wait<0>(a, parity);
    if (!got && tc::globaltimer() - t0 > tc::wait_limit()) {
      report(LCSA_DEV_TIMEOUT);
      break;
    }
  } while (!got);
  return __all_sync(0xffffffffu, got);
}
template <int kOff = 0>
__device__ __forceinline__ bool f4_wait(uint32_t a, uint32_t parity) {
  return __all_sync(0xffffffffu, f4_try_wait<kOff>(a, parity)) || f4_wait_slow(a + kOff, parity);
}

__device__ __forceinline__ uint32_t f4_tile(uint32_t base, int i) {
  return base + kF4OffTab + (uint32_t)(i % kF4Ring) * (uint32_t)sizeof(F4Tile);
}
// The kind of the next description that holds a tile (or is the end), for the
// expanding warps; its place is ts - 1 afterwards.
__device__ __forceinline__ int f4_next_tile(uint32_t base, bool& ok, int& ts, int lane) {
  while (ok) {
    if (!f4_wait<kF4BTabFull>(base + 8 * (ts % kF4Ring), (ts / kF4Ring) & 1)) {
      ok = false;
      break;
    }
    const int kind = (int)f4_lds32<offsetof(F4Tile, kind)>(f4_tile(base, ts));
    ++ts;
    if (kind != kF4Empty) return kind;
    __syncwarp();
    if (lane == 0) f4_arrive<kF4BTabEmpty>(base + 8 * ((ts - 1) % kF4Ring));
  }
  return kF4End;
}
// A matrix descriptor `off` 16-byte units further: the address field takes the
// sum (shared memory ends below its limit), one addition of the low word.
__device__ __forceinline__ uint64_t f4_desc(uint64_t d, uint32_t off) {
  return (d & 0xffffffff00000000ull) | (uint32_t)((uint32_t)d + off);
}
__device__ __forceinline__ void f4_cp_async16(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}

// This CTA's share of the merged output: pieces of four dims, kP pieces and kR
// splits at a time so that eight remote loads are in flight a thread.  Every
// CTA begins with its own part and goes around from there (an order that does
// not depend on timing), so no two read the same part at the same time.
struct F4Merge {
  const F4Args* g;
  uint8_t* smem;
  uint32_t k_base;
  int split;
  long long q_row;
};
template <int kP, int kR>
__device__ __forceinline__ void f4_merge(const F4Merge& m) {
  const F4Args& g = *m.g;
  const int S = g.splits, u1 = 8192 * (m.split + 1) / S;
  const float* wgt = reinterpret_cast<const float*>(m.smem + kF4OffWgt);
#pragma unroll 1
  for (int u0 = 8192 * m.split / S + threadIdx.x; u0 < u1; u0 += kP * kF4Threads) {
    float4 o[kP];
#pragma unroll
    for (int i = 0; i < kP; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int r0 = 0; r0 < S; r0 += kR) {
      float4 x[kP][kR];
#pragma unroll
      for (int k = 0; k < kR; ++k) {
        const int r = m.split + r0 + k < S ? m.split + r0 + k : m.split + r0 + k - S;
#pragma unroll
        for (int i = 0; i < kP; ++i) {
          const int u = u0 + i * kF4Threads, h = u >> 7;
          if (u < u1 && r0 + k < S) x[i][k] = ld_cluster4(cluster_addr(m.k_base + h * 2048 + (((u & 127) ^ (h & 7)) << 4), r));
        }
      }
#pragma unroll
      for (int k = 0; k < kR; ++k) {
        const int r = m.split + r0 + k < S ? m.split + r0 + k : m.split + r0 + k - S;
#pragma unroll
        for (int i = 0; i < kP; ++i) {
          const int u = u0 + i * kF4Threads;
          const float w = u < u1 && r0 + k < S ? wgt[r * 64 + (u >> 7)] : -1.f;
          if (!(w < 0.f)) {                                  // a split without a tile left whatever was there
            o[i].x = fmaf(w, x[i][k].x, o[i].x);
            o[i].y = fmaf(w, x[i][k].y, o[i].y);
            o[i].z = fmaf(w, x[i][k].z, o[i].z);
            o[i].w = fmaf(w, x[i][k].w, o[i].w);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const int u = u0 + i * kF4Threads;
      if (u >= u1) break;
      const int h = u >> 7, d = (u & 127) * 4;
      const float4 v = o[i];
      const long long at = (m.q_row * 64 + h) * 512 + d;
      if (g.out_bf16) {
        const float f[4] = {v.x, v.y, v.z, v.w};
        store_vec<4>(reinterpret_cast<__nv_bfloat16*>(g.out) + at, f);
      } else {
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(g.out) + at) = v;
      }
    }
  }
}

__global__ void __launch_bounds__(kF4Threads, 1)
attn_fp4_kernel(const __grid_constant__ F4Args g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  F4Tile* tab = reinterpret_cast<F4Tile*>(smem + kF4OffTab);
  float4* s_stats = reinterpret_cast<float4*>(smem + kF4OffStats);
  float* s_ref = reinterpret_cast<float*>(smem + kF4OffRef);
  float* s_l = reinterpret_cast<float*>(smem + kF4OffL);
  float* s_e = reinterpret_cast<float*>(smem + kF4OffE);
  float* s_wgt = reinterpret_cast<float*>(smem + kF4OffWgt);
  uint64_t* tab_full = reinterpret_cast<uint64_t*>(smem + kF4BTabFull);     // [kF4Ring] sequencer
  uint64_t* tab_empty = reinterpret_cast<uint64_t*>(smem + kF4BTabEmpty);   // [kF4Ring] every role's warps
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + kF4BKFull);        // [kF4Stages] expanding warps
  uint64_t* kv_empty = reinterpret_cast<uint64_t*>(smem + kF4BKEmpty);      // [kF4Stages] MMA commit after O
  uint64_t* s_full = reinterpret_cast<uint64_t*>(smem + kF4BSFull);         // [2] MMA commit
  uint64_t* s_free = reinterpret_cast<uint64_t*>(smem + kF4BSFree);         // [2] softmax warps: S is in registers
  uint64_t* p_full = reinterpret_cast<uint64_t*>(smem + kF4BPFull);         // [2] softmax warps
  uint64_t* pv_done = reinterpret_cast<uint64_t*>(smem + kF4BPvDone);       // [2] MMA commit
  uint64_t* o_free = reinterpret_cast<uint64_t*>(smem + kF4BOFree);         // [2] transition warps: half of O has been read
  uint64_t* stats_full = reinterpret_cast<uint64_t*>(smem + kF4BStats);     // [2] by item, softmax warps
  uint64_t* q_ready = reinterpret_cast<uint64_t*>(smem + kF4BQReady);       // transition warps
  uint64_t* s_done = reinterpret_cast<uint64_t*>(smem + kF4BSDone);         // MMA commit after an item's last S
  uint64_t* drain = reinterpret_cast<uint64_t*>(smem + kF4BDrain);          // MMA commit after the last product
  __shared__ uint32_t s_tmem;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kF4Ring; ++i) {
      tc::mbar_init(tab_full + i, 1);
      tc::mbar_init(tab_empty + i, kF4Readers);
    }
    for (int i = 0; i < kF4Stages; ++i) {
      tc::mbar_init(kv_full + i, kF4Code + kF4Rot);
      tc::mbar_init(kv_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(s_full + i, 1);
      tc::mbar_init(s_free + i, 4);
      tc::mbar_init(p_full + i, 4);
      tc::mbar_init(pv_done + i, 1);
      tc::mbar_init(o_free + i, 4);
      tc::mbar_init(stats_full + i, 4);
    }
    tc::mbar_init(q_ready, 4);
    tc::mbar_init(s_done, 1);
    tc::mbar_init(drain, 1);
    tc::fence_barrier_init();
  }
  if (warp == kF4MmaWarp) { tc::tmem_alloc(&s_tmem, 512); tc::tmem_relinquish(); }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = s_tmem;
  const uint32_t k_base = tc::smem_u32(smem), p_base = k_base + kF4OffP;
  const int split = g.splits > 1 ? (int)(blockIdx.x % g.splits) : 0;

  const int xw = warp < kF4SmWarp0 ? (int)(kF4Roles >> (4 * warp)) & 15 : 15;               // expanding warp
  if (xw < kF4Code) {
    // ============================================================ codes
    // Warps 0-7: dims 0-383, blocks blk, 4 + blk and 8 + blk of one key a
    // thread.  Warps 8 and 9: dims 384-447, both blocks of one key a thread.
    // Eight keys lie side by side in a warp, so a store phase writes eight
    // different bank groups.
    const bool wide = xw < 8;
    const int key = wide ? 8 * xw + (lane & 7) : 32 * (xw - 8) + lane, blk = wide ? lane >> 3 : 0;
    const int blocks = wide ? 3 : 2, src_step = wide ? 4 : 1;
    const uint32_t dst_step = wide ? 2 * kF4Region : 0, col_step = wide ? 0 : 64;
    const uint32_t dst = k_base + (wide ? (uint32_t)(blk >> 1) : 6u) * kF4Region + key * 128;
    const uint32_t col0 = (uint32_t)((4 * (blk & 1)) ^ (key & 7)) << 4;
    // this and the next tile's blocks and scales: loaded a tile ahead
    uint4 q0, q1, q2, n0, n1, n2, sc;
    const uint4* src = nullptr;
    bool ok = true;
    int ts = 0;
    auto load = [&](uint32_t d, int kind) {                  // no row: zero codes and scales
      const int r = (int)f4_lds32(d + 4 * key);
      n0 = n1 = n2 = sc = make_uint4(0, 0, 0, 0);
      if (kind == kF4Entries && r >= 0) {
        const long long e = (long long)f4_lds64<offsetof(F4Tile, base)>(d) + r;
        src = reinterpret_cast<const uint4*>(g.codes + e * 224) + (wide ? blk : 12);
        sc = __ldg(reinterpret_cast<const uint4*>(g.scales) + e);
        n0 = __ldg(src);
        n1 = __ldg(src + src_step);
        if (wide) n2 = __ldg(src + 8);
      }
    };
    int kind = f4_next_tile(k_base, ok, ts, lane);
    n0 = n1 = n2 = sc = make_uint4(0, 0, 0, 0);
    if (kind != kF4End) load(f4_tile(k_base, ts - 1), kind);
    int st = 0;
    uint32_t par = 1;                                        // of the stage's last reading (none in the first round)
#pragma unroll 1
    for (int n = 0; ok && kind != kF4End; ++n) {
      const uint32_t d = f4_tile(k_base, ts - 1), bar = k_base + 8 * st, buf = st * kF4KBytes;
      const int slot = (ts - 1) % kF4Ring, cur_kind = kind;
      kind = f4_next_tile(k_base, ok, ts, lane);
      q0 = n0;
      q1 = n1;
      q2 = n2;
      uint32_t w0 = wide ? sc.x >> (8 * blk) : sc.w, w1 = wide ? sc.y >> (8 * blk) : sc.w >> 8, w2 = sc.z >> (8 * blk);
      if (kind != kF4End) load(f4_tile(k_base, ts - 1), kind);
      if (!ok || (n >= kF4Stages && !f4_wait<kF4BKEmpty>(bar, par))) { ok = false; break; }
      if (cur_kind == kF4Entries) {
        uint32_t to = dst + buf, col = col0;
#pragma unroll 1
        for (int c = 0; c < blocks; ++c) {                   // one block's code: unrolled, the roles' code
          const uint32_t s = e8m0_bf16x2(w0 & 255u);         // outgrows the instruction cache
          f4_sts128(to + col, e2m1x8_by_products(q0.x, s));
          f4_sts128(to + (col ^ 16), e2m1x8_by_products(q0.y, s));
          f4_sts128(to + (col ^ 32), e2m1x8_by_products(q0.z, s));
          f4_sts128(to + (col ^ 48), e2m1x8_by_products(q0.w, s));
          q0 = q1;
          q1 = q2;
          w0 = w1;
          w1 = w2;
          to += dst_step;
          col ^= col_step;
        }
      } else {
        // window rows, 16 bytes at a time: 48 pieces a row for the first eight warps, 8 for the others
        const long long base = (long long)f4_lds64<offsetof(F4Tile, base)>(d);
        const int first = wide ? 32 * xw + lane : 32 * (xw - 8) + lane, row = wide ? 48 : 8, p0 = wide ? 0 : 48;
#pragma unroll 1
        for (int i = first; i < 64 * row; i += wide ? 256 : 64) {
          const int k = i / row, piece = p0 + i - k * row, r = (int)f4_lds32(d + 4 * k);
          f4_cp_async16(k_base + buf + (piece >> 3) * kF4Region + k * 128 + (((piece & 7) ^ (k & 7)) << 4),
                        g.kv + (base + (r >= 0 ? r : 0)) * 512 + 8 * piece, r >= 0 ? 16u : 0u);   // no row: zeros
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        f4_arrive<kF4BKFull>(bar);
        f4_arrive<kF4BTabEmpty>(k_base + 8 * slot);
      }
      if (++st == kF4Stages) { st = 0; par ^= 1; }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");         // nothing may land after the CTA exits
  } else if (xw < kF4Code + kF4Rot) {
    // ============================================================ rotary dims
    // Four 16-byte pieces a thread, always of the same four pairs, turned to
    // the keys' positions from the query's.
    const int tid = 32 * (xw - kF4Code) + lane;
    const uint32_t dst = k_base + 7 * kF4Region + (tid >> 3) * 128 + (((tid & 7) ^ ((tid >> 3) & 7)) << 4);
    unsigned long long turn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) turn[i] = g.turn[4 * (tid & 7) + i];
    uint4 nr[4];                                             // of the next tile, loaded a tile ahead
    bool ok = true;
    int ts = 0;
    auto load = [&](uint32_t d, int kind) {
      const __nv_bfloat16* p = (kind == kF4Entries ? g.rope : g.kv + 448) + 8 * (tid & 7);
      const int ld = kind == kF4Entries ? 64 : 512;
      const long long base = (long long)f4_lds64<offsetof(F4Tile, base)>(d);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int r = (int)f4_lds32(d + 4 * (tid >> 3) + 64 * u);
        nr[u] = make_uint4(0, 0, 0, 0);
        if (r >= 0) nr[u] = __ldg(reinterpret_cast<const uint4*>(p + (base + r) * ld));
      }
    };
    int kind = f4_next_tile(k_base, ok, ts, lane);
    if (kind != kF4End) load(f4_tile(k_base, ts - 1), kind);
    int st = 0;
    uint32_t par = 1;
#pragma unroll 1
    for (int n = 0; ok && kind != kF4End; ++n) {
      const uint32_t d = f4_tile(k_base, ts - 1), bar = k_base + 8 * st, buf = st * kF4KBytes;
      const int slot = (ts - 1) % kF4Ring;
      kind = f4_next_tile(k_base, ok, ts, lane);
      if (!ok) break;
      uint4 rp[4] = {nr[0], nr[1], nr[2], nr[3]};
      if (kind != kF4End) load(f4_tile(k_base, ts - 1), kind);
      const long long pos0 = (long long)f4_lds64<offsetof(F4Tile, pos0)>(d), step = (long long)f4_lds64<offsetof(F4Tile, step)>(d);
#pragma unroll 1
      for (int u = 0; u < 4; ++u) {                          // a full turn of the queue: back in order
        const unsigned long long pos = (unsigned long long)(pos0 + (int)f4_lds32(d + 4 * (tid >> 3) + 64 * u) * step);
        uint32_t x[4] = {rp[0].x, rp[0].y, rp[0].z, rp[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float co, si;
          turn_cs(pos * turn[i], &co, &si);
          x[i] = rotate_pair(x[i], co, si);
        }
        rp[0] = rp[1];
        rp[1] = rp[2];
        rp[2] = rp[3];
        rp[3] = make_uint4(x[0], x[1], x[2], x[3]);
      }
      if (n >= kF4Stages && !f4_wait<kF4BKEmpty>(bar, par)) { ok = false; break; }
#pragma unroll
      for (int u = 0; u < 4; ++u) f4_sts128(dst + buf + u * 16 * 128, rp[u]);
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        f4_arrive<kF4BKFull>(bar);
        f4_arrive<kF4BTabEmpty>(k_base + 8 * slot);
      }
      if (++st == kF4Stages) { st = 0; par ^= 1; }
    }
  } else if (warp >= kF4SmWarp0 && warp < kF4XtWarp0) {
    // ============================================================ softmax
    // Two threads per head: keys 0-31 and 32-63 of each tile (16x32bx2
    // accesses of tensor memory lanes 0-15); maxima and sums meet through a shuffle.
    const int half = lane >> 4, h = 16 * (warp & 3) + (lane & 15);
    const uint32_t t_lane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t prow = k_base + kF4OffP + h * 128;
    float m_run = -INFINITY, l_run = 0.f, e_run = 0.f;       // the sums: of this thread's half
    bool ok = true;
    int n = 0, ni = 0;
    for (int ts = 0; ok; ++ts) {
      if (!f4_wait<kF4BTabFull>(k_base + 8 * (ts % kF4Ring), (ts / kF4Ring) & 1)) break;
      const uint32_t d = f4_tile(k_base, ts);
      const int kind = (int)f4_lds32<offsetof(F4Tile, kind)>(d), first = (int)f4_lds32<offsetof(F4Tile, first)>(d),
                last = (int)f4_lds32<offsetof(F4Tile, last)>(d);
      const uint32_t mask = f4_lds32<offsetof(F4Tile, mask)>(d + 4 * half);
      __syncwarp();
      if (lane == 0) f4_arrive<kF4BTabEmpty>(k_base + 8 * (ts % kF4Ring));
      if (kind == kF4End) break;
      if (kind == kF4Empty) continue;
      const uint32_t sb = n & 1, bar = k_base + 8 * sb;
      if (!f4_wait<kF4BSFull>(bar, (n >> 1) & 1)) break;
      tc::tc_fence_after();
      // twice over S in pieces of 16 keys: for the maximum, then the weights
      // (little code and few registers; a piece takes some 40 cycles to read)
      uint32_t v[16];
      auto logits = [&](int u) {
        tc::tmem_ld_16x32bx2_x16<32>(t_lane + sb * 64 + 16 * u, v);
        tc::tmem_wait_ld_regs16(v);
        const uint32_t m = mask >> (16 * u);
        if ((m & 0xffffu) != 0xffffu) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (!((m >> i) & 1u)) v[i] = 0xff800000u;        // no key: weight 0
        }
      };
      float top = -INFINITY;
#pragma unroll 1
      for (int u = 0; u < 2; ++u) {
        logits(u);
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, __uint_as_float(v[i]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16)) * g.scale_log2;
      float alpha = 1.f;
      bool grow = false;
      if (first) {
        m_run = top;
        l_run = e_run = 0.f;
      } else if (top > m_run + 8.f) {                        // otherwise weights stay below 2^8
        alpha = ex2_ftz(m_run - top);
        m_run = top;
        grow = true;
      }
      if (__any_sync(0xffffffffu, grow)) {
        // O follows once the product of the tile before has finished
        if (!f4_wait<kF4BPvDone>(k_base + 8 * ((n - 1) & 1), ((n - 1) >> 1) & 1)) break;
        tc::tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 256; c += 16) {
          uint32_t o[16];
          tc::tmem_ld_16x32bx2_x16<256>(t_lane + kF4TmO + c, o);
          tc::tmem_wait_ld_regs16(o);
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          tc::tmem_st_16x32bx2_x16<256>(t_lane + kF4TmO + c, o);
        }
        tc::tmem_wait_st();
      }
      l_run *= alpha;
      e_run *= alpha;
      if (n >= 2 && !f4_wait<kF4BPvDone>(bar, ((n >> 1) - 1) & 1)) break;   // P's buffer has been read
      // Weights, rounded to BF16 for the product (2^-8 of a weight at most).
      // Outputs are divided by the sum of the rounded weights, so what all of
      // a query's weights have in common in their rounding cancels (few keys:
      // half of the largest errors); the log-sum-exp takes the exact ones'.
      const float neg_m = m_run == -INFINITY ? 0.f : -m_run;
      f2x sum = pk2(0.f, 0.f), exact = sum;
#pragma unroll 1
      for (int u = 0; u < 2; ++u) {
        logits(u);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p0 = ex2_ftz(fmaf(__uint_as_float(v[8 * c + 2 * i]), g.scale_log2, neg_m));
            const float p1 = ex2_ftz(fmaf(__uint_as_float(v[8 * c + 2 * i + 1]), g.scale_log2, neg_m));
            const __nv_bfloat162 b = __floats2bfloat162_rn(p0, p1);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
            exact = add2(exact, pk2(p0, p1));
            sum = add2(sum, pk2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)));
          }
          f4_sts128(prow + sb * kF4PBytes + (((4 * half + 2 * u + c) ^ (h & 7)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) f4_arrive<kF4BSFree>(bar);
      const float2 l2 = upk2(sum), e2 = upk2(exact);
      l_run += l2.x + l2.y;
      e_run += e2.x + e2.y;
      tc::fence_proxy_async_smem();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) f4_arrive<kF4BPFull>(bar);
      ++n;
      if (last) {
        const float l = l_run + __shfl_xor_sync(0xffffffffu, l_run, 16), e = e_run + __shfl_xor_sync(0xffffffffu, e_run, 16);
        if (half == 0) s_stats[(ni & 1) * 64 + h] = make_float4(m_run, l, e, 0.f);
        __syncwarp();
        if (lane == 0) f4_arrive<kF4BStats>(k_base + 8 * (ni & 1));
        ++ni;
      }
    }
  } else if (warp >= kF4XtWarp0) {
    // ============================================================ transitions
    // The queries of the next item into tensor memory as soon as the last S of
    // the item before has completed, then that item's output.  A warp has 16
    // heads, two threads a head.
    const int half = lane >> 4, h = 16 * (warp & 3) + (lane & 15);
    const uint32_t t_lane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    bool ok = true;
    int n = 0, ni = 0, p_row = 0, p_last = 0;
    auto output = [&](int item) {                            // of the item before
      ok = f4_wait<kF4BStats>(k_base + 8 * (item & 1), (item >> 1) & 1) && ok;
      ok = f4_wait<kF4BPvDone>(k_base + 8 * (p_last & 1), (p_last >> 1) & 1) && ok;
      tc::tc_fence_after();
      const float4 ml = s_stats[(item & 1) * 64 + h];        // (reference, sum, exact sum)
      float f = 1.f;
      if (g.splits > 1) {
        if (half == 0) {
          // (a NaN sum stays one: its weights were taken against 0)
          s_ref[h] = ml.y == 0.f ? -INFINITY : ml.x == -INFINITY ? 0.f : ml.x;
          s_l[h] = ml.y;
          s_e[h] = ml.z;
        }
      } else {
        float M = ml.x, L = ml.y, E = ml.z;
        if (g.sink) {
          const float sk = g.sink[h] * 1.4426950408889634f;
          M = fmaxf(ml.x, sk);
          f = ml.x == -INFINITY ? (L == 0.f ? 0.f : 1.f) : exp2f(ml.x - M);
          const float es = sk == -INFINITY ? 0.f : exp2f(sk - M);
          L = L * f + es;
          E = E * f + es;
        }
        // a row without keys and sink: zero output (a NaN sum stays one)
        f = L == 0.f ? 0.f : f / L;
        if (half == 0 && g.lse) g.lse[(long long)p_row * 64 + h] = E == 0.f ? -INFINITY : (M + log2f(E)) * 0.6931471805599453f;
      }
      uint32_t buf[2][16];
      tc::tmem_ld_16x32bx2_x16<16>(t_lane + kF4TmO, buf[0]);
      // (by four: by two the compiler's code has a larger frame, and 64 x 8192 entries take 145 instead of 139 us)
#pragma unroll 4
      for (int k = 0; k < 16; ++k) {                         // dims 32 k + 16 half ..
        uint32_t* v = buf[k & 1];
        tc::tmem_wait_ld_regs16(v);
        if (k + 1 < 16) tc::tmem_ld_16x32bx2_x16<16>(t_lane + kF4TmO + (k + 1) * 32, buf[(k + 1) & 1]);
        if (k == 7 || k == 15) {                             // that half of O may be overwritten
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) f4_arrive<kF4BOFree>(k_base + (k == 15 ? 8 : 0));
        }
        const int d0 = 32 * k + 16 * half;
        if (g.splits > 1) {
          // a split's O goes where the K tiles were, [64 heads][512 dims] FP32, 16-byte pieces xor-ed by head
#pragma unroll
          for (int i = 0; i < 4; ++i)
            f4_sts128(k_base + h * 2048 + (((d0 / 4 + i) ^ (h & 7)) << 4), make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
          continue;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
        const long long o0 = ((long long)p_row * 64 + h) * 512 + d0;
        if (g.out_bf16) {
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
          }
          uint4* o = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(g.out) + o0);
          o[0] = make_uint4(w[0], w[1], w[2], w[3]);
          o[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
          uint4* o = reinterpret_cast<uint4*>(reinterpret_cast<float*>(g.out) + o0);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
      }
    };
    for (int ts = 0; ok; ++ts) {
      if (!f4_wait<kF4BTabFull>(k_base + 8 * (ts % kF4Ring), (ts / kF4Ring) & 1)) break;
      const uint32_t d = f4_tile(k_base, ts);
      const int kind = (int)f4_lds32<offsetof(F4Tile, kind)>(d), first = (int)f4_lds32<offsetof(F4Tile, first)>(d),
                last = (int)f4_lds32<offsetof(F4Tile, last)>(d), q_row = (int)f4_lds32<offsetof(F4Tile, q_row)>(d);
      __syncwarp();
      if (lane == 0) f4_arrive<kF4BTabEmpty>(k_base + 8 * (ts % kF4Ring));
      if (kind == kF4Empty) {
        // no key at all: the query (or this split of it) contributes nothing
        if (g.splits > 1) {
          if (half == 0) {
            s_ref[h] = -INFINITY;
            s_l[h] = s_e[h] = -1.f;                          // no tile, so no O
          }
        } else {
          const long long o0 = ((long long)q_row * 64 + 16 * (warp & 3)) * 512;
          for (int e = lane * 8; e < 16 * 512; e += 256) {
            if (g.out_bf16) {
              *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(g.out) + o0 + e) = make_uint4(0, 0, 0, 0);
            } else {
              float4* o = reinterpret_cast<float4*>(reinterpret_cast<float*>(g.out) + o0 + e);
              o[0] = o[1] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
          }
          if (half == 0 && g.lse) g.lse[(long long)q_row * 64 + h] = g.sink ? g.sink[h] : -INFINITY;
        }
        continue;
      }
      if (kind != kF4End && first) {
        // step k: dims 64 k + 32 half .. to 16 columns (two dims each), 16 further for the second half
        // (64 bytes a thread and step; 32-byte loads halve the requests, whose
        // number is what this takes)
        const __nv_bfloat16* q = g.q + ((long long)q_row * 64 + h) * 512 + 32 * half;
        const bool wide = (reinterpret_cast<uintptr_t>(g.q) & 31u) == 0;
        uint32_t x[3][16];                                   // loads two steps ahead
        ld_words<2>(q, x[0], wide);
        ld_words<2>(q + 64, x[1], wide);
        if (ni > 0 && !f4_wait<kF4BSDone>(k_base, (ni - 1) & 1)) break;    // the last S that read the columns
        tc::tc_fence_after();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (k + 2 < 8) ld_words<2>(q + 64 * (k + 2), x[(k + 2) % 3], wide);
          tc::tmem_st_16x32bx2_x16<16>(t_lane + kF4TmQ + 32 * k, x[k % 3]);
        }
        tc::tmem_wait_st();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) f4_arrive<kF4BQReady>(k_base);
      }
      if ((kind == kF4End || first) && ni > 0) output(ni - 1);
      if (kind == kF4End) break;
      if (first) {
        ++ni;
        p_row = q_row;
      }
      if (last) p_last = n;
      ++n;
    }
  } else if (warp == kF4MmaWarp) {
    // ============================================================ MMA issuer
    // S of the next tile and O of the current one, whichever can go first
    // (polled without suspending: a suspended wait on one would miss the other).
    if (tc::elect_one()) {
      const uint32_t idesc_s = tc::idesc_bf16(64, 64, 0, 0);       // A (tensor memory) and B K-major
      const uint32_t idesc_o = tc::idesc_bf16(64, 256, 0, 1);      // A K-major, B MN-major
      bool ok = true, have = false;                          // have: tile n - 1 waits for its O
      int n = 0, st = 0, ni = 0, o_first = 0;
      uint32_t full_par = 0;
      const unsigned long long limit = tc::wait_limit();
      for (int ts = 0; ok;) {
        int kind, first, last;
        do {
          if (!tc::mbar_wait(tab_full + ts % kF4Ring, (ts / kF4Ring) & 1)) { ok = false; break; }
          const uint32_t d = f4_tile(k_base, ts);
          kind = (int)f4_lds32<offsetof(F4Tile, kind)>(d);
          first = (int)f4_lds32<offsetof(F4Tile, first)>(d);
          last = (int)f4_lds32<offsetof(F4Tile, last)>(d);
          tc::mbar_arrive(tab_empty + ts % kF4Ring);
          ++ts;
        } while (kind == kF4Empty);
        if (!ok) break;
        const int b = n & 1, o_st = st == 0 ? kF4Stages - 1 : st - 1;
        bool s_todo = kind != kF4End;
        int o_half = 0;                                      // halves of O (dims 0-255, 256-511) already issued
        unsigned long long t0 = 0;
        int idle = 0;
        while (s_todo || have) {
          bool moved = false;
          if (s_todo && tc::mbar_test_wait(kv_full + st, full_par) && (n < 2 || tc::mbar_test_wait(s_free + b, ((n >> 1) - 1) & 1)) &&
              (!first || tc::mbar_test_wait(q_ready, ni & 1))) {
            tc::tc_fence_after();
            const uint64_t d_k = tc::sdesc_sw128(k_base + st * kF4KBytes, 16, 1024);
#pragma unroll 4
            for (int ks = 0; ks < 32; ++ks)
              tc::mma_bf16_ts(tmem + b * 64, tmem + kF4TmQ + ks * 8,
                              f4_desc(d_k, ((ks >> 2) * kF4Region + (ks & 3) * 32) >> 4), idesc_s, ks > 0);
            tc::mma_commit(s_full + b);
            if (last) tc::mma_commit(s_done);
            s_todo = false;
            moved = true;
          }
          if (have && (o_half > 0 || tc::mbar_test_wait(p_full + (b ^ 1), ((n - 1) >> 1) & 1))) {
            // the first product of an item overwrites O, so it waits (a half
            // at a time) for the output of the item before to have been read
            const int item = ni - 1;                         // of tile n - 1
            const bool fresh = o_first && item > 0;
            if (!fresh || tc::mbar_test_wait(o_free + o_half, (item - 1) & 1)) {
              tc::tc_fence_after();
              const uint64_t d_p = tc::sdesc_sw128(p_base + (b ^ 1) * kF4PBytes, 16, 1024);
              const uint64_t d_v = tc::sdesc_sw128(k_base + o_st * kF4KBytes, kF4Region, 1024);
              const int h1 = fresh && o_half == 0 ? 1 : 2;
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                if (hf < o_half || hf >= h1) continue;
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                  tc::mma_bf16_ss(tmem + kF4TmO + hf * 256, f4_desc(d_p, ks * 2),
                                  f4_desc(d_v, (hf * 4 * kF4Region + ks * 2048) >> 4), idesc_o, !o_first || ks > 0);
              }
              o_half = h1;
              if (o_half == 2) {
                tc::mma_commit(kv_empty + o_st);
                tc::mma_commit(pv_done + (b ^ 1));
                have = false;
              }
              moved = true;
            }
          }
          if (moved) {
            t0 = 0;
            idle = 0;
          } else if ((++idle & 255) == 0) {                  // the timer is slow to read: now and then
            const unsigned long long now = tc::globaltimer();
            if (t0 == 0) {
              t0 = now;
            } else if (now - t0 > limit) {
              report(LCSA_DEV_TIMEOUT);
              ok = false;
              break;
            }
          }
        }
        if (!ok || kind == kF4End) break;
        have = true;
        o_first = first;
        if (first) ++ni;
        ++n;
        if (++st == kF4Stages) { st = 0; full_par ^= 1; }
      }
      // products in flight end before tensor memory is freed, also where the
      // roles that wait for them gave up
      tc::mma_commit(drain);
      tc::mbar_wait(drain, 0);
    }
  } else if (warp == kF4SeqWarp) {
    // ============================================================ sequencer
    const int step = g.splits > 1 ? (int)g.rows : (int)gridDim.x;          // one query per cluster when split
    bool ok = true;
    int ts = 0;
    auto slot_free = [&]() -> bool {
      if (ts >= kF4Ring &&
          !__all_sync(0xffffffffu, tc::mbar_wait_backoff(tab_empty + ts % kF4Ring, ((ts / kF4Ring) - 1) & 1)))
        return false;
      return true;
    };
    auto publish = [&]() {
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(tab_full + ts % kF4Ring);
      ++ts;
    };
    for (int it = g.splits > 1 ? (int)blockIdx.x / g.splits : (int)blockIdx.x; ok && it < (int)g.rows; it += step) {
      const F4Query qr = f4_query(g, it);
      const int b = qr.b;
      const long long t = qr.t;
      const int32_t* sel = g.sparse ? g.idx + qr.row * g.k : nullptr;
      long long wlo = t - g.W + 1, whi = t;
      if (wlo < g.kv_pos0) wlo = g.kv_pos0;
      if (wlo < 0) wlo = 0;
      if (whi > g.kv_pos0 + g.Tkv - 1) whi = g.kv_pos0 + g.Tkv - 1;
      const int n_w = whi >= wlo ? (int)(whi - wlo + 1) : 0, w0 = (int)(wlo - g.kv_pos0);
      int n_c, tiles_c, t0, t1;
      auto split_tiles = [&](int entries) {                  // this split's share of the key list
        n_c = entries;
        tiles_c = (n_c + kF4Keys - 1) / kF4Keys;
        const unsigned tiles = tiles_c + (n_w + kF4Keys - 1) / kF4Keys;
        t0 = (int)(tiles * (unsigned)split / (unsigned)g.splits);
        t1 = (int)(tiles * (unsigned)(split + 1) / (unsigned)g.splits);
      };
      // rows of a tile; selected entries are loaded one tile ahead
      auto rows_of = [&](int tile, int* row) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int key = lane + 32 * u, e = tile * kF4Keys + key;
          if (tile < tiles_c) row[u] = e < n_c ? (g.sparse ? __ldg(sel + e) : e) : -1;
          else row[u] = e - tiles_c * kF4Keys < n_w ? w0 + e - tiles_c * kF4Keys : -1;
        }
      };
      int row[2];
      if (g.sparse) {
        // full selections first: whether this one is padded arrives with the first rows
        const int end = __ldg(sel + g.k - 1);
        split_tiles(g.k);
        rows_of(t0, row);
        if (end < 0) {                                       // up to the last entry that is not -1
          int top = 0;
          for (int e = lane; e < g.k; e += 32)
            if (__ldg(sel + e) >= 0) top = e + 1;
          split_tiles((int)__reduce_max_sync(0xffffffffu, (unsigned)top));
          rows_of(t0, row);
        }
      } else {
        const long long nv = ((unsigned long long)t >> 32) ? t / g.m : (long long)((unsigned)t / (unsigned)g.m);
        split_tiles((int)(nv < g.Nc ? nv : g.Nc));
        rows_of(t0, row);
      }
      if (t0 == t1) {
        if (!slot_free()) { ok = false; break; }
        if (lane == 0) {
          F4Tile& d = tab[ts % kF4Ring];
          d.kind = kF4Empty;
          d.first = d.last = 0;
          d.q_row = (int)qr.row;
        }
        publish();
        continue;
      }
      for (int tile = t0; tile < t1; ++tile) {
        const bool entries = tile < tiles_c;
        const long long base = (long long)b * (entries ? g.Nc : g.Tkv);
        int next[2] = {-1, -1};
        if (tile + 1 < t1) rows_of(tile + 1, next);
        bool bad = false;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (entries && row[u] >= g.Nc) { bad = true; row[u] = -1; }
          if (row[u] < 0) row[u] = -1;
        }
        if (bad) report(LCSA_DEV_BAD_INDEX);
        if (!slot_free()) { ok = false; break; }
        F4Tile& d = tab[ts % kF4Ring];
#pragma unroll
        for (int u = 0; u < 2; ++u) d.row[lane + 32 * u] = row[u];
        const uint32_t m0 = __ballot_sync(0xffffffffu, row[0] >= 0), m1 = __ballot_sync(0xffffffffu, row[1] >= 0);
        if (lane == 0) {
          d.kind = entries ? kF4Entries : kF4Window;
          d.mask[0] = m0;
          d.mask[1] = m1;
          d.first = tile == t0;
          d.last = tile == t1 - 1;
          d.base = base;
          d.pos0 = (entries ? 0 : g.kv_pos0) - t;
          d.step = entries ? g.m : 1;
          d.q_row = (int)qr.row;
        }
        publish();
        row[0] = next[0];
        row[1] = next[1];
      }
    }
    if (ok && slot_free()) {
      if (lane == 0) {
        F4Tile& d = tab[ts % kF4Ring];
        d.kind = kF4End;
        d.first = d.last = 0;
      }
      publish();
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == kF4MmaWarp) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
  if (g.splits == 1) return;

  // ============================================================ merge
  // Weights of the splits' partial sums, then a 1 / splits share of the 64 x
  // 512 outputs per CTA.
  cluster_sync_all();
  const int S = g.splits;
  const long long q_row = f4_query(g, blockIdx.x / S).row;
  // every split's references and sums, all loads in flight at once (P's space is free by now)
  float* s_sum = reinterpret_cast<float*>(smem + kF4OffP);
  float* s_exact = s_sum + 64 * S;
  for (int i = threadIdx.x; i < 64 * S; i += kF4Threads) {
    s_wgt[i] = ld_cluster(cluster_addr(tc::smem_u32(s_ref + (i & 63)), i >> 6));
    s_sum[i] = ld_cluster(cluster_addr(tc::smem_u32(s_l + (i & 63)), i >> 6));
    if (split == 0 && g.lse) s_exact[i] = ld_cluster(cluster_addr(tc::smem_u32(s_e + (i & 63)), i >> 6));
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    const int h = threadIdx.x;
    const float sk = g.sink ? g.sink[h] * 1.4426950408889634f : -INFINITY;
    float M = sk;
    for (int r = 0; r < S; ++r) M = fmaxf(M, s_wgt[r * 64 + h]);
    float L = sk == -INFINITY ? 0.f : exp2f(sk - M), E = L;
    for (int r = 0; r < S; ++r) {
      const float ref = s_wgt[r * 64 + h], sum = s_sum[r * 64 + h];
      const float f = ref == -INFINITY ? 0.f : exp2f(ref - M);
      s_wgt[r * 64 + h] = sum < 0.f ? -1.f : f;
      if (!(sum < 0.f)) {                                    // a NaN sum stays one beside far larger references
        L += f * sum;
        if (split == 0 && g.lse) E += f * s_exact[r * 64 + h];
      }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    for (int r = 0; r < S; ++r)
      if (!(s_wgt[r * 64 + h] < 0.f)) s_wgt[r * 64 + h] *= inv;
    if (split == 0 && g.lse) g.lse[q_row * 64 + h] = E == 0.f ? -INFINITY : (M + log2f(E)) * 0.6931471805599453f;
  }
  __syncthreads();
  const F4Merge m = {&g, smem, k_base, split, q_row};
  if (S >= 8) f4_merge<1, 8>(m);
  else if (S >= 4) f4_merge<2, 4>(m);
  else f4_merge<4, 2>(m);
  cluster_sync_all();                                        // no CTA leaves while another reads its part
}

// Selections with their entries first and -1 behind them, for the kernels that
// read a row up to its first -1.  A block a row, 2048 slots at a time, a warp
// 256 of them with all its loads in flight (2048 rows of 2048 slots: 7.5 us;
// a warp a row 14.6 us).
__global__ void __launch_bounds__(256)
fp4_pack_selection_kernel(const int32_t* __restrict__ idx, long long rows, int k, int32_t* __restrict__ out) {
  __shared__ int s_live[2][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int turn = 0;
  for (long long r = blockIdx.x; r < rows; r += gridDim.x) {
    const int32_t* src = idx + r * k;
    int32_t* dst = out + r * k;
    int n = 0;                                               // entries so far
    for (long long e0 = 0; e0 < k; e0 += 2048, turn ^= 1) {
      const int left = (int)(k - e0) - 256 * warp - lane;           // slots from this lane's first on
      int v[8], at[8], mine = 0;
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = left > 32 * u ? __ldg(src + (k - left) + 32 * u) : -1;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const uint32_t live = __ballot_sync(0xffffffffu, v[u] >= 0);
        at[u] = mine + __popc(live & ((1u << lane) - 1u));
        mine += __popc(live);
      }
      if (lane == 0) s_live[turn][warp] = mine;
      __syncthreads();                                       // the other turn's counts have been read by now
      int before = 0, all = 0;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        if (w < warp) before += s_live[turn][w];
        all += s_live[turn][w];
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (v[u] >= 0) dst[n + before + at[u]] = v[u];
      n += all;
    }
    for (long long e = n + (int)threadIdx.x; e < k; e += 256) dst[e] = -1;
  }
}
static cudaError_t launch_fp4_pack_selection(const int32_t* idx, long long rows, int k, int32_t* out, cudaStream_t st) {
  const long long most = 64LL * sm_count();
  count_launch();
  fp4_pack_selection_kernel<<<(unsigned)(rows < most ? rows : most), 256, 0, st>>>(idx, rows, k, out);
  return cudaGetLastError();
}

static bool attn_fp4_supported(const lcsa_attn_args* a) {
  return a->dtype == LCSA_BF16 && a->H == 64 && a->D == 512 && a->R == 64;
}

// Entries that the last of the first n_q rows sees.
static long long attn_fp4_visible(const lcsa_attn_args* a, int n_q) {
  const long long nv = (a->q_pos0 + n_q - 1) / a->m;
  return nv < a->Nc ? nv : a->Nc;
}

// 64-key tiles of the longest key list of the first n_q rows (a selection holds
// no more entries than are visible).
static long long attn_fp4_tiles(const lcsa_attn_args* a, int sparse, int n_q) {
  const long long seen = attn_fp4_visible(a, n_q);
  const long long n_c = sparse && a->k < seen ? a->k : seen, n_w = a->W < a->Tkv ? a->W : a->Tkv;
  return (n_c + kF4Keys - 1) / kF4Keys + (n_w + kF4Keys - 1) / kF4Keys;
}

// Rows of a sequence when the cache is read back.  Selected entries are
// gathered, and a selection is trusted: as many as the cache has.  A dense call
// needs what its last row sees.  attn_tc.cuh reads whole tiles there: zeros
// behind the last entry.  It takes these rows for the entries there are, so
// zeros follow only where no row's position reaches past the cache's last entry.
static long long attn_fp4_read_rows(const lcsa_attn_args* a, int sparse) {
  const long long nv = (a->q_pos0 + a->Tq - 1) / a->m;
  if (sparse || nv > a->Nc) return a->Nc;
  return attn_fp4_supported(a) ? (nv + kF4Keys - 1) / kF4Keys * kF4Keys : nv;
}

// Rows of a sequence whose window is not whole (it begins before the raw rows
// do): its last tile in attn_tc.cuh would hold raw rows that they do not see, so
// attn_fp4_kernel takes them when the others read the cache back, and they
// count for nothing in that decision (32 prompts of 150 tokens from position 0:
// 557 us with these rows done by both kernels, 340 us by this one alone).
static int attn_fp4_part_rows(const lcsa_attn_args* a) {
  const long long part = (a->kv_pos0 > 0 ? a->kv_pos0 : 0) + a->W - 1 - a->q_pos0;
  return a->W <= 0 || part <= 0 ? 0 : (int)(part < a->Tq ? part : a->Tq);
}

// Whether to read the whole cache back once and attend over BF16 entries
// (attn_tc.cuh) instead of expanding each tile where it is used.  Expanding
// costs a tile some 0.25 us of an SM; reading back costs 0.33 ns an entry
// (1.5 KB at 4.6 TB/s) and about 15 us of launches.  A cache may be allocated
// for a far longer context: what counts is the entries that are read back, and
// the tiles that the rows have by now.  Measured: 2048 rows of
// 2176 keys over 8192 entries 938 us here and 811 us read back, 2048 rows of
// 1152 keys over 1024 entries 535 and 377 us; 64 sequences of one row, 8192
// entries each, 139 us and 362 us.  That kernel multiplies whole tiles, masked
// keys by a weight of zero, so a window has to end with its tile and be in kv,
// and the entries of a sequence with a tile (attn_fp4_read_rows).  Beyond 2048
// selected entries it splits every row, with 128 KB of partial outputs a split
// to write and read (2048 rows of 2049 + 128 keys over 8192 entries 966 us here
// and 1163 us read back, of 8192 + 128 over 16384 3351 and 3492 us).
static bool attn_fp4_expands(const lcsa_attn_args* a, int sparse) {
  if (a->W % kF4Keys != 0 || (a->W > 0 && a->kv_pos0 + a->Tkv < a->q_pos0 + a->Tq)) return false;
  if (sparse && a->k > kAtMaxIdx) return false;
  if (!sparse && a->B > 1 && attn_fp4_read_rows(a, sparse) % kF4Keys != 0) return false;
  const double rows = (double)a->B * (a->Tq - attn_fp4_part_rows(a));
  return rows * (double)attn_fp4_tiles(a, sparse, a->Tq) * (0.25 / 148.0) >
         (double)a->B * attn_fp4_read_rows(a, sparse) * 0.33e-3 + 15.0;
}

// CTAs that run at the same time in clusters of `s`, on the current device
// (a cluster's CTAs share a GPC, so large clusters leave some SMs idle).
static int attn_fp4_slots(int s) {
  static std::atomic<int> known[16][kF4MaxSplits + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return sm_count();
  const bool keep = dev < 16;
  int n = keep ? known[dev][s].load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  if (s == 1) {
    n = sm_count();
  } else {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(s);
    cfg.blockDim = dim3(kF4Threads);
    cfg.dynamicSmemBytes = kF4Smem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = s;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, attn_fp4_kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      clusters = 0;
    }
    n = clusters > 0 ? clusters * s : -1;                    // -1: this size does not run
  }
  if (keep) known[dev][s].store(n, std::memory_order_relaxed);
  return n;
}

// CTAs per query.  A CTA spends its tiles and about two tiles' time on filling
// and emptying its pipeline; a merge costs about one more.  More splits shorten
// the tile lists but can add rounds of CTAs.
static int attn_fp4_splits(long long rows, int tiles) {
  static const int sizes[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16};
  int best = 1;
  double best_cost = 1e30;
  for (int s : sizes) {
    if (s > 1 && s > tiles) break;
    const int slots = attn_fp4_slots(s);
    if (slots <= 0) continue;
    const long long rounds = (rows * s + slots - 1) / slots;
    const double cost = s == 1 ? rounds * (tiles + 2.0) + 3.0 : rounds * ((tiles + s - 1) / s + 7.0);
    if (cost < best_cost * 0.97) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

// Turns per position of the 32 rotary pairs, base^(-2i/64) / 2 pi, as 64-bit
// fractions.  A program has one or two bases: the last one's are kept (32
// powers take 2 us of host time).
static void attn_fp4_turns(float base, unsigned long long* turn) {
  thread_local float last = 0.f;
  thread_local unsigned long long kept[32];
  if (base != last) {
    for (int i = 0; i < 32; ++i) {
      long double t = powl((long double)base, -(long double)i / 32.0L) * 0.159154943091895335768883763372514362L;
      t -= floorl(t);
      kept[i] = (unsigned long long)(t * 18446744073709551616.0L);
    }
    last = base;
  }
  for (int i = 0; i < 32; ++i) turn[i] = kept[i];
}

// The first n_q rows of every sequence.
static cudaError_t launch_attn_fp4(const lcsa_attn_args* a, int sparse, const lcsa_fp4_entries* e, cudaStream_t st, int n_q) {
  const long long rows = (long long)a->B * n_q;
  if ((long long)a->B * a->Tq > (long long)INT32_MAX / kF4MaxSplits) return cudaErrorInvalidValue;   // 32-bit row and CTA numbers
  F4Args g;
  g.codes = a->Nc > 0 ? e->codes : nullptr;
  g.scales = a->Nc > 0 ? e->scales : nullptr;
  g.rope = a->Nc > 0 ? (const __nv_bfloat16*)e->rope : nullptr;
  g.q = (const __nv_bfloat16*)a->q;
  g.kv = (const __nv_bfloat16*)a->kv;
  g.idx = a->idx;
  g.sink = a->sink;
  g.out = a->out;
  g.lse = a->lse;
  g.B = a->B; g.Tq = a->Tq; g.n_q = n_q; g.Nc = a->Nc; g.k = a->k; g.Tkv = a->Tkv; g.m = a->m; g.W = a->W;
  g.sparse = sparse;
  g.out_bf16 = a->out_dtype == LCSA_BF16;
  g.rows = rows; g.q_pos0 = a->q_pos0; g.kv_pos0 = a->kv_pos0;
  g.scale_log2 = (a->softmax_scale > 0.f ? a->softmax_scale : 1.0f / sqrtf(512.f)) * 1.4426950408889634f;
  attn_fp4_turns(a->rope_base > 0.f ? a->rope_base : 10000.f, g.turn);
  const long long tiles = attn_fp4_tiles(a, sparse, n_q);
  cudaError_t err = cudaFuncSetAttribute(attn_fp4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kF4Smem);
  if (err != cudaSuccess) return err;
  err = cudaFuncSetAttribute(attn_fp4_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (err != cudaSuccess) return err;
  g.splits = attn_fp4_splits(rows, (int)(tiles < (1 << 30) ? tiles : (1 << 30)));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(g.splits > 1 ? (unsigned)(rows * g.splits) : (unsigned)(rows < sm_count() ? rows : sm_count()));
  cfg.blockDim = dim3(kF4Threads);
  cfg.dynamicSmemBytes = kF4Smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = g.splits;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = g.splits > 1 ? 1 : 0;
  count_launch();
  return cudaLaunchKernelEx(&cfg, attn_fp4_kernel, (const F4Args)g);
}

}  // namespace lcsa
