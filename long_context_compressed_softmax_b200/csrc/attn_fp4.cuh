// Core attention over the FP4 entry cache on tcgen05 tensor cores (BF16
// queries, H = 64 heads, D = 512, rotary R = 64): multi-query attention of 64
// heads over one shared K=V head whose entries arrive as E2M1 codes, then the
// window of raw BF16 rows, a per-head sink in the denominator, partial RoPE
// and the -t rotation of the output.
//
// Both products run transposed, with the 128 keys of a tile (S) or 128 of the
// 512 dims (O) on the M side and the 64 heads on the N side:
//   S^T[128 keys, 64 heads]  = K Q^T          A = K (K-major), B = Q (K-major)
//   O^T[512 dims, 64 heads] += K^T P^T        A = K^T (MN-major view of the same
//                                             bytes), B = P^T (MN-major)
// An M = 64 instruction (64 heads on the M side) runs at half the rate of an
// M = 128 one, and both take about 45 cycles at N = 64, so a tile of 128 keys
// costs 64 instructions (2,900 cycles) this way.  O^T takes 256 of the 512
// tensor memory columns, S^T 64.
//
// Shared memory: one K tile of 128 keys (128 KB of BF16, 128B-swizzled, eight
// 64-dim blocks), the queries (64 KB), P (16 KB).  There is no room for a
// second K tile, so the tile is refilled in four chunks of 128 dims: the
// product O^T is issued chunk by chunk, each commit frees a chunk, and the
// producers expand the next tile's codes into it while the later chunks are
// still being multiplied.  The codes of the next tile (368 bytes a key) wait
// in the producers' registers, loaded a whole tile ahead.
//
// Softmax with keys on the lanes: a thread holds one key and 32 heads.  The
// exponent's reference of each head lives in shared memory and moves only when
// some logit exceeds it by more than 2^8 (one vote per tile); then the column
// maxima are taken with warp reductions and O^T, whose columns are heads, is
// rescaled.  Row sums are kept per thread and added up once per query.
//
// Warps: 0-7 producers, 8-15 softmax and epilogue, 16 MMA issuer, 17
// sequencer (the list of tiles: which row each key of a tile is), 18 queries.
// All follow the sequencer's ring of tile descriptions, so only it knows how
// queries, selections and windows map to tiles.
//
// Long key lists of few queries are split over the CTAs of a cluster: each
// leaves its partial O in its shared memory and all of them add up a share of
// it over distributed shared memory, in rank order, so results do not depend
// on timing.
#pragma once
#include <atomic>

#include "tc_ptx.cuh"
#include "fp4cache.cuh"

namespace lcsa {

constexpr int kF4Keys = 128;                        // keys per tile
constexpr int kF4ProdWarps = 8, kF4ProdThreads = 256;
constexpr int kF4SmWarp0 = 8;                       // 8 softmax warps
constexpr int kF4MmaWarp = 16, kF4SeqWarp = 17, kF4QWarp = 18;
constexpr int kF4Threads = 19 * 32;
constexpr int kF4Ring = 8;                          // tile descriptions in flight
constexpr int kF4MaxSplits = 16;
constexpr uint32_t kF4Block = kF4Keys * 128;        // one 64-dim block of the K tile
constexpr uint32_t kF4QBlock = 64 * 128;            // one 64-dim block of the queries

struct F4Tile {
  int32_t row[kF4Keys];      // row of each key within its sequence, -1: no key
  int32_t kind;              // kF4Entries ..
  int32_t first, last;       // of its query (and split)
  int32_t pad[3];
  long long base;            // first row of the sequence in the cache or the raw buffer
  long long pos0, step;      // position of row r: pos0 + r * step
  long long q_row, t;        // query row (b * Tq + i) and its position
};
constexpr int kF4Entries = 0, kF4Window = 1, kF4Empty = 2, kF4End = 3;
static_assert(sizeof(F4Tile) % 16 == 0, "tile description");

// shared-memory carve-up, offsets from the 1 KB aligned base
constexpr uint32_t kF4OffQ = 8 * kF4Block;
constexpr uint32_t kF4OffP = kF4OffQ + 8 * kF4QBlock;
constexpr uint32_t kF4OffTab = kF4OffP + kF4Keys * 128;
constexpr uint32_t kF4OffRef = kF4OffTab + kF4Ring * sizeof(F4Tile);   // [64] reference of each head (log2 units)
constexpr uint32_t kF4OffNref = kF4OffRef + 64 * 4;                    // [64] minus the reference in use
constexpr uint32_t kF4OffAlpha = kF4OffNref + 64 * 4;                  // [64]
constexpr uint32_t kF4OffFac = kF4OffAlpha + 64 * 4;                   // [64] output factor
constexpr uint32_t kF4OffL = kF4OffFac + 64 * 4;                       // [64] sum of each head (split launches)
constexpr uint32_t kF4OffWmax = kF4OffL + 64 * 4;                      // [8 warps][32]
constexpr uint32_t kF4OffWgt = kF4OffWmax + 8 * 32 * 4;                // [splits][64] merge weights
constexpr uint32_t kF4OffCs = kF4OffWgt + kF4MaxSplits * 64 * 4;       // [32] (cos, sin) of the merge
constexpr uint32_t kF4OffBar = kF4OffCs + 32 * 8;
constexpr int kF4Bars = 2 * kF4Ring + 8 + 6;
constexpr size_t kF4Smem = 1024 + kF4OffBar + kF4Bars * 8;
static_assert(kF4Smem <= 232448, "FP4 attention shared memory exceeds 227 KB");

// tensor memory: O^T in columns [0, 256), 64 per block of 128 dims; S^T
constexpr uint32_t kF4TmS = 256;

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
  int B, Tq, Nc, k, Tkv, m, W;
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
__device__ __forceinline__ F4Query f4_query(const F4Args& g, long long it) {
  F4Query q;
  const int r = (int)(it / g.B);
  q.b = (int)(it - (long long)r * g.B);
  q.row = (long long)q.b * g.Tq + g.Tq - 1 - r;
  q.t = g.q_pos0 + g.Tq - 1 - r;
  return q;
}

__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ bool bar_or(int id, int n, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)pred), "r"(id), "r"(n)
      : "memory");
  return r != 0;
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

// (cos, sin) of an angle given as a 64-bit fraction of a turn.  Keys: the
// MUFU's sine and cosine (2^-20 absolute) of an angle within half a turn,
// far below the BF16 rounding of the rotated key.
__device__ __forceinline__ void turn_cs_fast(unsigned long long ph, float* c, float* s) {
  const float a = (float)(int)(ph >> 32) * 1.4629180792671596e-9f;   // 2 pi / 2^32
  *c = __cosf(a);
  *s = __sinf(a);
}
__device__ __forceinline__ void turn_cs(unsigned long long ph, float* c, float* s) {
  sincospif((float)(int)(ph >> 32) * 4.656612873077393e-10f, s, c);   // 2 / 2^32 half turns
}
__device__ __forceinline__ uint32_t rotate_pair(uint32_t x, float c, float s) {
  const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x));
  const __nv_bfloat162 o = __floats2bfloat162_rn(f.x * c - f.y * s, f.x * s + f.y * c);
  return *reinterpret_cast<const uint32_t*>(&o);
}

__device__ __forceinline__ void f4_cp_async16(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}

__global__ void __launch_bounds__(kF4Threads, 1)
attn_fp4_kernel(const __grid_constant__ F4Args g, const __grid_constant__ CUtensorMap tm_q) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  F4Tile* tab = reinterpret_cast<F4Tile*>(smem + kF4OffTab);
  float* s_ref = reinterpret_cast<float*>(smem + kF4OffRef);
  float* s_nref = reinterpret_cast<float*>(smem + kF4OffNref);
  float* s_alpha = reinterpret_cast<float*>(smem + kF4OffAlpha);
  float* s_fac = reinterpret_cast<float*>(smem + kF4OffFac);
  float* s_l = reinterpret_cast<float*>(smem + kF4OffL);
  float* s_wmax = reinterpret_cast<float*>(smem + kF4OffWmax);
  float* s_wgt = reinterpret_cast<float*>(smem + kF4OffWgt);
  float2* s_cs = reinterpret_cast<float2*>(smem + kF4OffCs);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kF4OffBar);
  uint64_t* tab_full = bars;                       // [kF4Ring] sequencer
  uint64_t* tab_empty = tab_full + kF4Ring;        // [kF4Ring] every role's warps
  uint64_t* k_full = tab_empty + kF4Ring;          // [4] chunk filled (producer warps)
  uint64_t* k_empty = k_full + 4;                  // [4] chunk read (MMA commit)
  uint64_t* s_full = k_empty + 4;                  // MMA commit
  uint64_t* p_full = s_full + 1;                   // softmax warps
  uint64_t* q_full = p_full + 1;                   // TMA bytes and the query warp
  uint64_t* q_empty = q_full + 1;                  // MMA commit after a query's last S
  uint64_t* o_full = q_empty + 1;                  // MMA commit after a query's last O
  uint64_t* drain = o_full + 1;                    // MMA commit of an abandoned CTA
  __shared__ uint32_t s_tmem;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kF4Ring; ++i) {
      tc::mbar_init(tab_full + i, 1);
      tc::mbar_init(tab_empty + i, 18);            // 8 producer, 8 softmax, MMA, query warps
    }
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(k_full + i, kF4ProdWarps);
      tc::mbar_init(k_empty + i, 1);
    }
    tc::mbar_init(s_full, 1);
    tc::mbar_init(p_full, 8);
    tc::mbar_init(q_full, 2);
    tc::mbar_init(q_empty, 1);
    tc::mbar_init(o_full, 1);
    tc::mbar_init(drain, 1);
    tc::fence_barrier_init();
  }
  if (threadIdx.x < 64) s_nref[threadIdx.x] = 0.f;
  if (warp == kF4MmaWarp) { tc::tmem_alloc(&s_tmem, 512); tc::tmem_relinquish(); }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = s_tmem;
  const uint32_t k_base = tc::smem_u32(smem), q_base = k_base + kF4OffQ, p_base = k_base + kF4OffP;
  const int split = g.splits > 1 ? (int)(blockIdx.x % g.splits) : 0;

  if (warp < kF4ProdWarps) {
    // ============================================================ producers
    // Chunk c < 3 of an entry tile is 128 keys x four 32-value blocks: a thread
    // expands the same block of two keys.  Chunk 3 holds the last two blocks
    // and the rotary dims (four 16-byte pieces a thread, always the same four
    // pairs).  Window rows are copied with cp.async, their rotary dims take
    // the entries' way.
    const int tid = threadIdx.x;
    uint4 ca[3][2], cb, rp[4];
    uint32_t sa[3][2], sb;
    unsigned long long turn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) turn[i] = g.turn[4 * (tid & 7) + i];
    const uint4 zero4 = make_uint4(0, 0, 0, 0);

    auto load_codes = [&](const F4Tile& t, int c) {          // chunk c < 3
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int r = t.row[(tid >> 2) + 64 * u];
        ca[c][u] = zero4;
        sa[c][u] = 127;
        if (t.kind == kF4Entries && r >= 0) {
          const long long e = t.base + r;
          ca[c][u] = __ldg(reinterpret_cast<const uint4*>(g.codes + e * 224) + 4 * c + (tid & 3));
          sa[c][u] = __ldg(g.scales + e * 16 + 4 * c + (tid & 3));
        }
      }
    };
    auto load_last = [&](const F4Tile& t) {                  // chunk 3
      const int r = t.row[tid >> 1];
      cb = zero4;
      sb = 127;
      if (t.kind == kF4Entries && r >= 0) {
        const long long e = t.base + r;
        cb = __ldg(reinterpret_cast<const uint4*>(g.codes + e * 224) + 12 + (tid & 1));
        sb = __ldg(g.scales + e * 16 + 12 + (tid & 1));
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int rr = t.row[(tid >> 3) + 32 * u];
        rp[u] = zero4;
        if (rr >= 0) {
          const long long e = t.base + rr;
          const __nv_bfloat16* p = t.kind == kF4Entries ? g.rope + e * 64 : g.kv + e * 512 + 448;
          rp[u] = __ldg(reinterpret_cast<const uint4*>(p) + (tid & 7));
        }
      }
    };
    auto expand = [&](uint32_t dst, uint4 w, uint32_t scale_byte, int chunk0, int key, bool swap) {
      // words 0, 2 and 1, 3 change places in half of the lanes, so that the
      // eight lanes of a store phase write eight different bank groups
      const uint32_t s2 = e8m0_bf16x2(scale_byte);
      const uint32_t x[4] = {swap ? w.z : w.x, swap ? w.w : w.y, swap ? w.x : w.z, swap ? w.y : w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ch = chunk0 + (swap ? i ^ 2 : i);
        tc::sts128(dst + ((uint32_t)(ch ^ (key & 7)) << 4), e2m1x8_to_bf16(x[i], s2));
      }
    };

    bool ok = true;
    int ts = 0;                                              // tile descriptions seen
    // the next description that holds a tile (or the end); others are returned at once
    auto next_tile = [&]() -> const F4Tile* {
      while (true) {
        if (!__all_sync(0xffffffffu, tc::mbar_wait(tab_full + ts % kF4Ring, (ts / kF4Ring) & 1))) return nullptr;
        const F4Tile* t = tab + ts % kF4Ring;
        if (t->kind != kF4Empty) return t;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tab_empty + ts % kF4Ring);
        ++ts;
      }
    };
    const F4Tile* cur = next_tile();
    ok = cur != nullptr;
    if (ok && cur->kind != kF4End) {
      load_codes(*cur, 0);
      load_codes(*cur, 1);
      load_codes(*cur, 2);
      load_last(*cur);
    }
    for (int n = 0; ok && cur->kind != kF4End; ++n) {
      const int cur_slot = ts % kF4Ring;
      ++ts;
      const F4Tile* nxt = next_tile();
      if (!nxt) { ok = false; break; }
      const bool more = nxt->kind != kF4End;
      const bool window = cur->kind == kF4Window;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (n > 0 && !__all_sync(0xffffffffu, tc::mbar_wait(k_empty + c, (n - 1) & 1))) { ok = false; break; }
        if (window) {
          const int nu = c < 3 ? 8 : 4, sh = c < 3 ? 4 : 3;      // c = 3: block 6 only
          const int piece = tid & ((1 << sh) - 1);
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            if (u < nu) {
              const int key = (tid >> sh) + (kF4ProdThreads >> sh) * u;
              const int r = cur->row[key];
              const uint32_t dst = k_base + (2 * c + (piece >> 3)) * kF4Block + key * 128 + (((piece & 7) ^ (key & 7)) << 4);
              const __nv_bfloat16* src = g.kv + (cur->base + (r >= 0 ? r : 0)) * 512 + 128 * c + 8 * piece;
              f4_cp_async16(dst, src, r >= 0 ? 16u : 0u);        // no row: zeros
            }
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
        } else if (c < 3) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int key = (tid >> 2) + 64 * u;
            expand(k_base + (2 * c + ((tid >> 1) & 1)) * kF4Block + key * 128, ca[c][u], sa[c][u], 4 * (tid & 1), key,
                   (tid >> 1) & 1);
          }
        } else {
          const int key = tid >> 1;
          expand(k_base + 6 * kF4Block + key * 128, cb, sb, 4 * (tid & 1), key, false);
        }
        if (c == 3) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int key = (tid >> 3) + 32 * u;
            const unsigned long long pos = (unsigned long long)(cur->pos0 + cur->row[key] * cur->step);
            uint32_t w[4] = {rp[u].x, rp[u].y, rp[u].z, rp[u].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float cs, sn;
              turn_cs_fast(pos * turn[i], &cs, &sn);
              w[i] = rotate_pair(w[i], cs, sn);
            }
            tc::sts128(k_base + 7 * kF4Block + key * 128 + (((tid & 7) ^ (key & 7)) << 4),
                       make_uint4(w[0], w[1], w[2], w[3]));
          }
        }
        if (window) {
          // a chunk's copies land while the next chunk's are issued
          if (c > 0) {
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(k_full + c - 1);
          }
          if (c == 3) {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(k_full + 3);
          }
        } else {
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(k_full + c);
        }
        if (more) {
          if (c < 3) load_codes(*nxt, c);
          else load_last(*nxt);
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(tab_empty + cur_slot);
      cur = nxt;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");         // nothing may land after the CTA exits
  } else if (warp < kF4MmaWarp) {
    // ============================================================ softmax
    const int qd = warp & 3;                                 // tensor memory lanes 32 qd ..
    const int half = (warp - kF4SmWarp0) >> 2;               // heads 32 half ..
    const int key = 32 * qd + lane;
    const int bar_id = 1 + half;                             // the four warps that share these heads
    const uint32_t t_lane = tmem + ((uint32_t)(32 * qd) << 16) + 32 * half;
    const uint32_t nref_a = tc::smem_u32(s_nref + 32 * half), alpha_a = tc::smem_u32(s_alpha + 32 * half),
                   fac_a = tc::smem_u32(s_fac + 32 * half);
    float l[32];
#pragma unroll
    for (int h = 0; h < 32; ++h) l[h] = 0.f;
    bool fresh = true;                                       // no key of this query seen so far
    bool ok = true;
    int n = 0, nq = 0;
    for (int ts = 0;; ++ts) {
      if (!__all_sync(0xffffffffu, ok && tc::mbar_wait(tab_full + ts % kF4Ring, (ts / kF4Ring) & 1))) ok = false;
      int kind = kF4End, last = 0;
      bool valid = false;
      long long q_row = 0, t = 0;
      if (ok) {
        const F4Tile& d = tab[ts % kF4Ring];
        kind = d.kind;
        last = d.last;
        valid = kind <= kF4Window && d.row[key] >= 0;
        q_row = d.q_row;
        t = d.t;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tab_empty + ts % kF4Ring);
      }
      // the four warps of a half leave together
      if (!tc::bar_and(bar_id, 128, ok)) { ok = false; break; }
      if (kind == kF4End) break;
      if (kind == kF4Empty) {
        if (g.splits > 1) {
          if (qd == 0) {
            s_ref[32 * half + lane] = -INFINITY;
            s_l[32 * half + lane] = 0.f;
          }
        } else {
          const long long o0 = q_row * 64 * 512;
          for (int e = (threadIdx.x - kF4SmWarp0 * 32) * 8; e < 64 * 512; e += 256 * 8) {
            if (g.out_bf16) {
              *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(g.out) + o0 + e) = make_uint4(0, 0, 0, 0);
            } else {
              float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(g.out) + o0 + e);
              p[0] = p[1] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
          }
          if (qd == 0 && g.lse) {
            const int h = 32 * half + lane;
            g.lse[q_row * 64 + h] = g.sink ? g.sink[h] : -INFINITY;
          }
        }
        continue;
      }
      if (!__all_sync(0xffffffffu, tc::mbar_wait(s_full, n & 1))) ok = false;
      ++n;
      tc::tc_fence_after();
      uint32_t v[32];
      tc::tmem_ld32(t_lane + kF4TmS, v);
      tc::tmem_wait_ld_regs32(v);
      if (!valid) {                                          // weight 0 whatever the reference is
#pragma unroll
        for (int h = 0; h < 32; ++h) v[h] = 0xff800000u;
      }
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 r = tc::lds128f(nref_a + 16 * i);
        mx = fmaxf(mx, fmaf(__uint_as_float(v[4 * i]), g.scale_log2, r.x));
        mx = fmaxf(mx, fmaf(__uint_as_float(v[4 * i + 1]), g.scale_log2, r.y));
        mx = fmaxf(mx, fmaf(__uint_as_float(v[4 * i + 2]), g.scale_log2, r.z));
        mx = fmaxf(mx, fmaf(__uint_as_float(v[4 * i + 3]), g.scale_log2, r.w));
      }
      if (bar_or(bar_id, 128, !ok || (valid && (fresh || mx > 8.f)))) {
        if (!tc::bar_and(bar_id, 128, ok)) { ok = false; break; }
        // column maxima of this tile: lane h of each warp ends up with head h
        float mine = -INFINITY;
#pragma unroll
        for (int h = 0; h < 32; ++h) {
          const float r = redux_max(__uint_as_float(v[h]) * g.scale_log2);
          if (lane == h) mine = r;
        }
        const float old = s_ref[32 * half + lane];
        s_wmax[(4 * half + qd) * 32 + lane] = mine;
        tc::bar_sync(bar_id, 128);
        if (qd == 0) {
          float m = -INFINITY;
#pragma unroll
          for (int w = 0; w < 4; ++w) m = fmaxf(m, s_wmax[(4 * half + w) * 32 + lane]);
          float ref = fresh ? m : fmaxf(m, old);
          if (ref == -INFINITY) ref = 0.f;                   // every logit is -inf or NaN
          s_alpha[32 * half + lane] = fresh ? 1.f : ex2_ftz(old - ref);
          s_ref[32 * half + lane] = ref;
          s_nref[32 * half + lane] = -ref;
        }
        tc::bar_sync(bar_id, 128);
        if (!fresh) {
          // what has been added up so far follows the new reference; the
          // product before this S has completed (same issuer, in order)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 a = tc::lds128f(alpha_a + 16 * i);
            l[4 * i] *= a.x; l[4 * i + 1] *= a.y; l[4 * i + 2] *= a.z; l[4 * i + 3] *= a.w;
          }
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t o[16];
            const uint32_t a = t_lane + 64 * (c >> 1) + 16 * (c & 1);
            tc::tmem_ld16(a, o);
            tc::tmem_wait_ld_regs16(o);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 f = tc::lds128f(alpha_a + 64 * (c & 1) + 16 * i);
              o[4 * i] = __float_as_uint(__uint_as_float(o[4 * i]) * f.x);
              o[4 * i + 1] = __float_as_uint(__uint_as_float(o[4 * i + 1]) * f.y);
              o[4 * i + 2] = __float_as_uint(__uint_as_float(o[4 * i + 2]) * f.z);
              o[4 * i + 3] = __float_as_uint(__uint_as_float(o[4 * i + 3]) * f.w);
            }
            tc::tmem_st16(a, o);
          }
          tc::tmem_wait_st();
        }
        fresh = false;
      }
      // weights, their sums, P^T (rounded to BF16 for the product: 2^-9 of a
      // weight, averaged over the keys; the sums keep the unrounded weights)
      const uint32_t prow = p_base + key * 128;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 r = tc::lds128f(nref_a + 32 * c + 16 * i);
          const int h = 8 * c + 4 * i;
          const float p0 = ex2_ftz(fmaf(__uint_as_float(v[h]), g.scale_log2, r.x));
          const float p1 = ex2_ftz(fmaf(__uint_as_float(v[h + 1]), g.scale_log2, r.y));
          const float p2 = ex2_ftz(fmaf(__uint_as_float(v[h + 2]), g.scale_log2, r.z));
          const float p3 = ex2_ftz(fmaf(__uint_as_float(v[h + 3]), g.scale_log2, r.w));
          l[h] += p0;
          l[h + 1] += p1;
          l[h + 2] += p2;
          l[h + 3] += p3;
          const __nv_bfloat162 b0 = __floats2bfloat162_rn(p0, p1), b1 = __floats2bfloat162_rn(p2, p3);
          w[2 * i] = *reinterpret_cast<const uint32_t*>(&b0);
          w[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&b1);
        }
        tc::sts128(prow + (((4 * half + c) ^ (key & 7)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
      }
      tc::fence_proxy_async_smem();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(p_full);
      if (!last) continue;

      // ---------------------------------------------------------- epilogue
      // sums over the 32 keys of the warp, head h to lane h, then over the four warps
#pragma unroll
      for (int st = 16; st > 0; st >>= 1) {
        const bool up = lane & st;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i < st) {
            const float send = up ? l[i] : l[i + st];
            const float mine = up ? l[i + st] : l[i];
            l[i] = mine + __shfl_xor_sync(0xffffffffu, send, st);
          }
      }
      s_wmax[(4 * half + qd) * 32 + lane] = l[0];
      tc::bar_sync(bar_id, 128);
      if (qd == 0) {
        const int h = 32 * half + lane;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) sum += s_wmax[(4 * half + w) * 32 + lane];
        const float ref = fresh ? -INFINITY : s_ref[h];
        if (g.splits > 1) {
          s_ref[h] = ref;
          s_l[h] = sum;
        } else {
          float M = ref, L = sum, f = 1.f;
          if (g.sink) {
            const float s2 = g.sink[h] * 1.4426950408889634f;
            M = fmaxf(ref, s2);
            f = ref == -INFINITY ? 0.f : exp2f(ref - M);
            L = sum * f + (s2 == -INFINITY ? 0.f : exp2f(s2 - M));
          }
          // a row without keys and sink: zero output (a NaN sum stays one)
          s_fac[h] = L == 0.f ? 0.f : f / L;
          if (g.lse) g.lse[q_row * 64 + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
          s_nref[h] = 0.f;
        }
      }
      if (!__all_sync(0xffffffffu, tc::mbar_wait(o_full, nq & 1))) ok = false;
      ++nq;
      tc::tc_fence_after();
      tc::bar_sync(bar_id, 128);
      if (g.splits > 1) {
        // the K tile has been read for the last time: the partial O goes there, [64 heads][512 dims] FP32
        float* part = reinterpret_cast<float*>(smem);
#pragma unroll 1
        for (int mb = 0; mb < 4; ++mb) {
          tc::tmem_ld32(t_lane + 64 * mb, v);
          tc::tmem_wait_ld_regs32(v);
#pragma unroll
          for (int h = 0; h < 32; ++h) part[(32 * half + h) * 512 + 128 * mb + key] = __uint_as_float(v[h]);
        }
      } else {
        float cs = 1.f, sn = 0.f;
        if (qd >= 2) {
          turn_cs((unsigned long long)t * g.turn[16 * (qd - 2) + (lane >> 1)], &cs, &sn);
          if (lane & 1) sn = -sn;                            // x c + y s | y c - x s
        }
#pragma unroll 1
        for (int mb = 0; mb < 4; ++mb) {
          tc::tmem_ld32(t_lane + 64 * mb, v);
          tc::tmem_wait_ld_regs32(v);
          const bool rot = mb == 3 && qd >= 2;
          const int d = 128 * mb + key;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 f = tc::lds128f(fac_a + 16 * i);
            float o[4] = {__uint_as_float(v[4 * i]) * f.x, __uint_as_float(v[4 * i + 1]) * f.y,
                          __uint_as_float(v[4 * i + 2]) * f.z, __uint_as_float(v[4 * i + 3]) * f.w};
            if (rot) {
#pragma unroll
              for (int j = 0; j < 4; ++j) o[j] = fmaf(o[j], cs, __shfl_xor_sync(0xffffffffu, o[j], 1) * sn);
            }
            const long long o0 = (q_row * 64 + 32 * half + 4 * i) * 512;
            if (g.out_bf16) {
              // even lanes take head 2j (dims d, d+1), odd lanes head 2j+1 (dims d-1, d)
              __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(g.out) + o0 + (lane & 1 ? 512 + d - 1 : d);
#pragma unroll
              for (int j = 0; j < 4; j += 2) {
                const float got = __shfl_xor_sync(0xffffffffu, lane & 1 ? o[j] : o[j + 1], 1);
                *reinterpret_cast<__nv_bfloat162*>(out + j * 512) =
                    lane & 1 ? __floats2bfloat162_rn(got, o[j + 1]) : __floats2bfloat162_rn(o[j], got);
              }
            } else {
              float* out = reinterpret_cast<float*>(g.out) + o0 + d;
#pragma unroll
              for (int j = 0; j < 4; ++j) out[j * 512] = o[j];
            }
          }
        }
      }
      tc::tc_fence_before();                                 // O may be overwritten after the next p_full
      fresh = true;
#pragma unroll
      for (int h = 0; h < 32; ++h) l[h] = 0.f;
    }
  } else if (warp == kF4MmaWarp) {
    // ============================================================ MMA issuer
    if (tc::elect_one()) {
      const uint32_t idesc_s = tc::idesc_bf16(128, 64, 0, 0);
      const uint32_t idesc_o = tc::idesc_bf16(128, 64, 1, 1);
      bool ok = true;
      int n = 0, nq = 0;
      for (int ts = 0; ok; ++ts) {
        if (!tc::mbar_wait(tab_full + ts % kF4Ring, (ts / kF4Ring) & 1)) { ok = false; break; }
        const F4Tile& d = tab[ts % kF4Ring];
        const int kind = d.kind, first = d.first, last = d.last;
        tc::mbar_arrive(tab_empty + ts % kF4Ring);
        if (kind == kF4End) break;
        if (kind == kF4Empty) continue;
        if (first && !tc::mbar_wait(q_full, nq & 1)) { ok = false; break; }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (ok && !tc::mbar_wait(k_full + c, n & 1)) ok = false;
          if (ok) {
            tc::tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              const uint32_t blk = 2 * c + (ks >> 2), off = (ks & 3) * 32;
              tc::mma_bf16_ss(tmem + kF4TmS, tc::sdesc_sw128(k_base + blk * kF4Block + off, 16, 1024),
                              tc::sdesc_sw128(q_base + blk * kF4QBlock + off, 16, 1024), idesc_s, c > 0 || ks > 0);
            }
          }
        }
        if (!ok) break;
        tc::mma_commit(s_full);
        if (last) tc::mma_commit(q_empty);
        if (!tc::mbar_wait(p_full, n & 1)) { ok = false; break; }
        tc::tc_fence_after();
#pragma unroll
        for (int mb = 0; mb < 4; ++mb) {
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            tc::mma_bf16_ss(tmem + 64 * mb, tc::sdesc_sw128(k_base + 2 * mb * kF4Block + ks * 2048, kF4Block, 1024),
                            tc::sdesc_sw128(p_base + ks * 2048, kF4Block, 1024), idesc_o, !first || ks > 0);
          tc::mma_commit(k_empty + mb);
        }
        if (last) {
          tc::mma_commit(o_full);
          ++nq;
        }
        ++n;
      }
      if (!ok) {                                             // products in flight end before tensor memory is freed
        tc::mma_commit(drain);
        tc::mbar_wait(drain, 0);
      }
    }
  } else if (warp == kF4SeqWarp) {
    // ============================================================ sequencer
    const int step = g.splits > 1 ? (int)g.rows : (int)gridDim.x;          // one query per cluster when split
    bool ok = true;
    int ts = 0;
    auto slot_free = [&]() -> bool {
      if (ts >= kF4Ring &&
          !__all_sync(0xffffffffu, tc::mbar_wait(tab_empty + ts % kF4Ring, ((ts / kF4Ring) - 1) & 1)))
        return false;
      return true;
    };
    auto publish = [&]() {
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(tab_full + ts % kF4Ring);
      ++ts;
    };
    for (long long it = g.splits > 1 ? blockIdx.x / g.splits : blockIdx.x; ok && it < g.rows; it += step) {
      const F4Query qr = f4_query(g, it);
      const int b = qr.b;
      const long long q_row = qr.row, t = qr.t;
      const int32_t* sel = g.sparse ? g.idx + q_row * g.k : nullptr;
      int n_c;
      if (g.sparse) {
        n_c = g.k;
        if (__ldg(sel + g.k - 1) < 0) {                       // padded: up to the last entry that is not -1
          int top = 0;
          for (int e = lane; e < g.k; e += 32)
            if (__ldg(sel + e) >= 0) top = e + 1;
          n_c = (int)__reduce_max_sync(0xffffffffu, (unsigned)top);
        }
      } else {
        const long long nv = t / g.m;
        n_c = (int)(nv < g.Nc ? nv : g.Nc);
      }
      long long wlo = t - g.W + 1, whi = t;
      if (wlo < g.kv_pos0) wlo = g.kv_pos0;
      if (wlo < 0) wlo = 0;
      if (whi > g.kv_pos0 + g.Tkv - 1) whi = g.kv_pos0 + g.Tkv - 1;
      const int n_w = whi >= wlo ? (int)(whi - wlo + 1) : 0;
      const int tiles_c = (n_c + kF4Keys - 1) / kF4Keys, tiles = tiles_c + (n_w + kF4Keys - 1) / kF4Keys;
      const int t0 = (int)((long long)tiles * split / g.splits), t1 = (int)((long long)tiles * (split + 1) / g.splits);
      if (t0 == t1) {
        if (!slot_free()) { ok = false; break; }
        if (lane == 0) {
          F4Tile& d = tab[ts % kF4Ring];
          d.kind = kF4Empty;
          d.q_row = q_row;
          d.t = t;
        }
        publish();
        continue;
      }
      for (int tile = t0; tile < t1; ++tile) {
        const bool entries = tile < tiles_c;
        int row[4];
        bool bad = false;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int key = lane + 32 * u;
          if (entries) {
            const int e = tile * kF4Keys + key;
            row[u] = e < n_c ? (g.sparse ? __ldg(sel + e) : e) : -1;
            if (row[u] >= g.Nc) { bad = true; row[u] = -1; }
            if (row[u] < 0) row[u] = -1;
          } else {
            const int e = (tile - tiles_c) * kF4Keys + key;
            row[u] = e < n_w ? (int)(wlo - g.kv_pos0) + e : -1;
          }
        }
        if (bad) report(LCSA_DEV_BAD_INDEX);
        if (!slot_free()) { ok = false; break; }
        F4Tile& d = tab[ts % kF4Ring];
#pragma unroll
        for (int u = 0; u < 4; ++u) d.row[lane + 32 * u] = row[u];
        if (lane == 0) {
          d.kind = entries ? kF4Entries : kF4Window;
          d.first = tile == t0;
          d.last = tile == t1 - 1;
          d.base = (long long)b * (entries ? g.Nc : g.Tkv);
          d.pos0 = entries ? 0 : g.kv_pos0;
          d.step = entries ? g.m : 1;
          d.q_row = q_row;
          d.t = t;
        }
        publish();
      }
    }
    if (ok && slot_free()) {
      if (lane == 0) tab[ts % kF4Ring].kind = kF4End;
      publish();
    }
  } else {
    // ============================================================ queries
    // Dims 0-447 of the 64 heads by TMA, the rotary dims through registers.
    if (lane == 0) tc::prefetch_tmap(&tm_q);
    int nq = 0;
    for (int ts = 0;; ++ts) {
      if (!__all_sync(0xffffffffu, tc::mbar_wait(tab_full + ts % kF4Ring, (ts / kF4Ring) & 1))) break;
      const F4Tile& d = tab[ts % kF4Ring];
      const int kind = d.kind, first = d.first;
      const long long q_row = d.q_row, t = d.t;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(tab_empty + ts % kF4Ring);
      if (kind == kF4End) break;
      if (kind == kF4Empty || !first) continue;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(g.q + q_row * 64 * 512 + 448) + lane;
      float cs, sn;
      turn_cs((unsigned long long)t * g.turn[lane], &cs, &sn);
      if (nq > 0 && !__all_sync(0xffffffffu, tc::mbar_wait(q_empty, (nq - 1) & 1))) break;
      if (lane == 0) {
        tc::mbar_arrive_expect_tx(q_full, 7 * kF4QBlock);
        for (int blk = 0; blk < 7; ++blk)
          tc::tma_load_2d(smem + kF4OffQ + blk * kF4QBlock, &tm_q, q_full, 64 * blk, (int)(q_row * 64));
      }
#pragma unroll 1
      for (int h0 = 0; h0 < 64; h0 += 32) {
        uint32_t x[32];
#pragma unroll
        for (int h = 0; h < 32; ++h) x[h] = __ldg(src + (h0 + h) * 256);
#pragma unroll
        for (int h = 0; h < 32; ++h) {
          const uint32_t a = q_base + 7 * kF4QBlock + (h0 + h) * 128 + ((((uint32_t)lane >> 2) ^ (h & 7)) << 4) + 4 * (lane & 3);
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(rotate_pair(x[h], cs, sn)) : "memory");
        }
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(q_full);
      ++nq;
    }
    if (nq > 0) tc::mbar_wait(q_full, (nq - 1) & 1);          // the last copies have landed
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
  const F4Query qr = f4_query(g, blockIdx.x / S);
  const long long q_row = qr.row, t = qr.t;
  if (threadIdx.x < 64) {
    const int h = threadIdx.x;
    const uint32_t ra = tc::smem_u32(s_ref + h), la = tc::smem_u32(s_l + h);
    const float s2 = g.sink ? g.sink[h] * 1.4426950408889634f : -INFINITY;
    float M = s2;
    for (int r = 0; r < S; ++r) M = fmaxf(M, ld_cluster(cluster_addr(ra, r)));
    float L = s2 == -INFINITY ? 0.f : exp2f(s2 - M);
    for (int r = 0; r < S; ++r) {
      const float ref = ld_cluster(cluster_addr(ra, r));
      const float f = ref == -INFINITY ? 0.f : exp2f(ref - M);
      s_wgt[r * 64 + h] = f;
      L += f == 0.f ? 0.f : f * ld_cluster(cluster_addr(la, r));
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    for (int r = 0; r < S; ++r) s_wgt[r * 64 + h] *= inv;
    if (split == 0 && g.lse) g.lse[q_row * 64 + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
  } else if (threadIdx.x < 96) {
    float c, s;
    turn_cs((unsigned long long)t * g.turn[threadIdx.x - 64], &c, &s);
    s_cs[threadIdx.x - 64] = make_float2(c, s);
  }
  __syncthreads();
  const int u1 = 8192 * (split + 1) / S;
  for (int u = 8192 * split / S + threadIdx.x; u < u1; u += kF4Threads) {
    const int h = u >> 7, d = (u & 127) * 4;
    const uint32_t a = k_base + (uint32_t)u * 16;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r = 0; r < S; ++r) {
      const float w = s_wgt[r * 64 + h];
      if (w != 0.f) {                                        // a split without keys left nothing to read
        const float4 x = ld_cluster4(cluster_addr(a, r));
        o.x = fmaf(w, x.x, o.x);
        o.y = fmaf(w, x.y, o.y);
        o.z = fmaf(w, x.z, o.z);
        o.w = fmaf(w, x.w, o.w);
      }
    }
    if (d >= 448) {
      const float2 e0 = s_cs[(d - 448) >> 1], e1 = s_cs[((d - 448) >> 1) + 1];
      o = make_float4(o.x * e0.x + o.y * e0.y, o.y * e0.x - o.x * e0.y, o.z * e1.x + o.w * e1.y, o.w * e1.x - o.z * e1.y);
    }
    const long long at = (q_row * 64 + h) * 512 + d;
    if (g.out_bf16) {
      const float f[4] = {o.x, o.y, o.z, o.w};
      store_vec<4>(reinterpret_cast<__nv_bfloat16*>(g.out) + at, f);
    } else {
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(g.out) + at) = o;
    }
  }
  cluster_sync_all();                                        // no CTA leaves while another reads its part
}

static bool attn_fp4_supported(const lcsa_attn_args* a) {
  return a->dtype == LCSA_BF16 && a->H == 64 && a->D == 512 && a->R == 64;
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
    const double cost = s == 1 ? rounds * (tiles + 1.0) + 1.0 : rounds * ((tiles + s - 1) / s + 3.0);
    if (cost < best_cost * 0.97) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

static cudaError_t launch_attn_fp4(const lcsa_attn_args* a, int sparse, const lcsa_fp4_entries* e, cudaStream_t st) {
  const long long rows = (long long)a->B * a->Tq;
  if (rows > (long long)INT32_MAX / 64) return cudaErrorInvalidValue;       // TMA row coordinates
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
  g.B = a->B; g.Tq = a->Tq; g.Nc = a->Nc; g.k = a->k; g.Tkv = a->Tkv; g.m = a->m; g.W = a->W;
  g.sparse = sparse;
  g.out_bf16 = a->out_dtype == LCSA_BF16;
  g.rows = rows; g.q_pos0 = a->q_pos0; g.kv_pos0 = a->kv_pos0;
  g.scale_log2 = (a->softmax_scale > 0.f ? a->softmax_scale : 1.0f / sqrtf(512.f)) * 1.4426950408889634f;
  const long double base = a->rope_base > 0.f ? (long double)a->rope_base : 10000.0L;
  for (int i = 0; i < 32; ++i) {
    long double turn = powl(base, -(long double)i / 32.0L) * 0.159154943091895335768883763372514362L;
    turn -= floorl(turn);
    g.turn[i] = (unsigned long long)(turn * 18446744073709551616.0L);
  }
  // tiles of the longest key list
  const long long t_last = a->q_pos0 + a->Tq - 1;
  long long n_c = t_last / a->m < a->Nc ? t_last / a->m : a->Nc;
  if (sparse) n_c = a->k;
  long long n_w = a->W < a->Tkv ? a->W : a->Tkv;
  const long long tiles = (n_c + kF4Keys - 1) / kF4Keys + (n_w + kF4Keys - 1) / kF4Keys;
  cudaError_t err = cudaFuncSetAttribute(attn_fp4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kF4Smem);
  if (err != cudaSuccess) return err;
  err = cudaFuncSetAttribute(attn_fp4_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (err != cudaSuccess) return err;
  g.splits = attn_fp4_splits(rows, (int)(tiles < (1 << 30) ? tiles : (1 << 30)));
  CUtensorMap m_q;
  if (!make_tmap_bf16_2d(&m_q, a->q, (uint64_t)rows * 64, 512, 512, 64, 64)) return cudaErrorInvalidValue;
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
  return cudaLaunchKernelEx(&cfg, attn_fp4_kernel, (const F4Args)g, (const CUtensorMap)m_q);
}

}  // namespace lcsa
