// w4_attn.cu -- attention of new rows over a paged 8-bit cache, for few rows per sequence and kv head
// (single tokens, drafted tokens), on warp-level tensor-core products (sm_103a).
//
// Mathematics.  With raw codes K, V (exact in FP16) and page scales ks, vs, a row's logits in base 2 are
// x_j = (q . K_j) ks c, c = softmax_scale log2(e), and
//   out = sum_j 2^(x_j + log2 vs_j - m) V_j / sum_j 2^(x_j + log2 vs_j - m) / vs_j
// with one running maximum m of x_j + log2 vs_j: the scale of V rides in the exponent, so the weights
// stay in [0, 1] whatever the scales, the codes of V stay exact, and no product is rounded for it.
// Weights are rounded to FP16 for the product with V (relative 2^-11 each, against the 2^-11 of the
// FP16 output); the sum below the line takes them in FP32 before that rounding.
//
// Tiles.  A unit is 64 keys of one kv head: 64 x D bytes of K and of V, brought by TMA (one box per
// page piece, 128-byte swizzle) into a ring of shared-memory stages, with the 16-key groups' scales
// beside them.  A CTA has 8 consumer warps = MT row tiles of 16 rows x 8 / MT key groups; key group
// g takes every (8 / MT)-th unit alone, with its own maximum, sums and D x 16 accumulators in
// registers, so the warps never meet inside an item; they are joined once per item.
// Q (16 rows) is the A operand of mma.m16n8k16, K the B operand as it lies in memory (a permutation
// of the channels, the same for Q and K, makes a lane's 16 codes one 16-byte load); the weights
// come out of the first product in the layout that the second takes as A; V's codes of two keys are
// interleaved by byte permutes into B pairs.  The keys of an 8-key tile are permuted so that both
// loads are free of bank conflicts under the swizzle (perm below).
// What bounds it: the bytes of the cache at long contexts; launch, dependent loads of the page table
// and the join at short ones.
#include <cstdint>
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "w4_attn.cuh"
#include "w4_common.cuh"
#include "w4_internal.h"
#include "w4_serve.h"

namespace w4 {

constexpr int kAtT = 64;                     // keys per unit
constexpr int kAtWarps = 8;                  // consumer warps
constexpr int kAtThreads = (kAtWarps + 1) * 32;

template <int D>
struct AtSmem {
  static constexpr int kStage = kAtT * D * 2;            // K, then V
  static constexpr int kMerge = kAtWarps * 16 * D * 4;   // partial sums of the warps
  static constexpr int kStages = 8;
  static constexpr int kScales = 4 * 16;                 // per stage: 4 groups x (ks c, log2 vs, 1 / vs)
  static constexpr int oMerge = kStages * kStage;
  static constexpr int oMl = oMerge + kMerge;            // [8 warps][16] maxima, then sums
  static constexpr int oScales = oMl + kAtWarps * 16 * 8;
  static constexpr int oBar = oScales + kStages * kScales;
  static constexpr int oFlag = oBar + kStages * 16;
  static constexpr int oPrefix = oFlag + 16;
  static constexpr int kTotal = oPrefix + (W4_MAX_SEQS + 1) * 4 + 1024;   // and the alignment slack
};

struct AtParams {
  AttnArgs a;
  CUtensorMap tk, tv;      // [pages][heads * page][D], box D x min(page, 64) x 1
  int group, max_blocks, min_units;
};

__device__ __forceinline__ void at_tma3(uint32_t dst, const CUtensorMap* map, int c1, int c2, uint64_t* bar, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(c1), "r"(c2), "r"(smem_u32(bar)), "l"(pol)
      : "memory");
}

// Two E4M3 codes (bits 0-15 of `w`, or 16-31) to two FP16 values.
__device__ __forceinline__ void at_cvt4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(lo), "=r"(hi) : "r"(w));
}

__device__ __forceinline__ void at_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 at_lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 at_lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// Byte offset of 16-byte chunk `c` of row `r` in a TMA-swizzled tile of D-byte rows.
template <int D>
__device__ __forceinline__ uint32_t at_swz(int r, int c) {
  return D == 128 ? (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)) : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

__device__ __forceinline__ uint32_t at_pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void at_sync_consumers() { asm volatile("bar.sync 1, %0;" ::"n"(kAtWarps * 32) : "memory"); }

template <int D, int MT>
__global__ void __launch_bounds__(kAtThreads, 1) w4_attn_kernel(const __grid_constant__ AtParams p) {
  using S = AtSmem<D>;
  constexpr int R = 16 * MT;                 // rows per item
  constexpr int KG = kAtWarps / MT;          // key groups
  constexpr int NS = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float* merge = reinterpret_cast<float*>(smem + S::oMerge);
  float2* ml = reinterpret_cast<float2*>(smem + S::oMl);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::oBar);
  uint64_t* empty = full + NS;
  int* flag = reinterpret_cast<int*>(smem + S::oFlag);
  int* prefix = reinterpret_cast<int*>(smem + S::oPrefix);
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], MT);
    }
    fence_mbar_init();
  }
  pdl_launch_dependents();
  pdl_wait();
  const Split sp = attn_split<R, kAtT>(a, p.group, p.max_blocks, p.min_units, (int)gridDim.x, prefix);
  const int cta = (int)blockIdx.x;
  if (cta >= sp.ctas || sp.U == 0) return;
  const int begin = sp.first(cta), end = sp.first(cta + 1);
  if (begin >= end) return;
  Walk<R, kAtT> w;
  w.start(a, p.group, prefix, begin, end);
  const float c2 = a.scale * 1.4426950408889634f;

  if (warp == kAtWarps) {
    // ================================================================ producer
    // Eight units at a time: lane = (unit, 16-key group).  The group's page id, then its scales, are
    // loaded for the whole batch before the copies are issued.
    const uint64_t pol = policy_evict_first();
    const int sub = lane & 3;
    const int P = a.c.page;
    int j = 0;                               // units issued
    int u = w.u0;
    bool more = true, ok = true;
    while (more && ok) {
      // lane's unit: the (lane / 4)-th from here, in this item or a later one
      Walk<R, kAtT> mine = w;
      int mu = u, left = lane >> 2;
      bool have = true;
      while (have && left >= mine.u1 - mu) {
        left -= mine.u1 - mu;
        have = mine.next(a, p.group);
        mu = mine.u0;
      }
      int key = 0, page = -1, h = 0;
      bool live = false;
      float ks = 0.f, vs = 1.f;
      if (have) {
        key = (mine.it.t0 + mu + left) * kAtT + 16 * sub;
        h = mine.it.h;
        live = key < mine.it.hi && key + 16 > mine.it.lo;
        if (live) {
          page = __ldg(a.c.table + (long long)mine.it.b * a.c.table_stride + key / P);
          if (page < 0 || page >= a.c.num_pages) {
            attn_range_error(0x501);
            live = false;
          }
        }
        if (live) {
          ks = __ldg(a.c.k_scale + (long long)page * a.c.scale_stride + h);
          vs = __ldg(a.c.v_scale + (long long)page * a.c.scale_stride + h);
        }
      }
      const float4 sc = make_float4(ks * c2, log2f(vs), __fdiv_rn(1.f, vs), 0.f);
      const int units = __popc(__ballot_sync(0xffffffffu, have && sub == 0));
      for (int i = 0; i < units && ok; ++i, ++j) {
        const int st = j % NS;
        if (j >= NS) ok = mbar_wait(&empty[st], ((j / NS) - 1) & 1, 0x511);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const bool me = (lane >> 2) == i;
        if (me) *reinterpret_cast<float4*>(smem + S::oScales + st * S::kScales + sub * 16) = sc;
        // a box holds min(P, 64) keys: the first live 16-key group of a box copies it
        const int per = min(P, kAtT) / 16;   // groups per box: 1, 2 or 4
        const uint32_t livemask = (__ballot_sync(0xffffffffu, live) >> (4 * i)) & 15u;
        const int boxes = 4 / per;
        uint32_t bytes = 0, lead = 0;
        for (int x = 0; x < boxes; ++x) {
          const uint32_t m = livemask & (((1u << per) - 1u) << (x * per));
          if (m) {
            bytes += (uint32_t)(per * 16 * D * 2);
            lead |= 1u << (__ffs(m) - 1);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&full[st], bytes);
        __syncwarp();
        if (me && (lead >> sub & 1)) {
          const int box = sub / per;
          const int row = h * P + (P > kAtT ? (key % P) / kAtT * kAtT : 0);
          const uint32_t dst = smem_u32(smem) + st * S::kStage + box * per * 16 * D;
          at_tma3(dst, &p.tk, row, page, &full[st], pol);
          at_tma3(dst + kAtT * D, &p.tv, row, page, &full[st], pol);
        }
      }
      // the walk goes on after these units
      int adv = units;
      while (more && adv >= w.u1 - u) {
        adv -= w.u1 - u;
        more = w.next(a, p.group);
        u = w.u0;
      }
      if (more) u += adv;
    }
    // every copy issued has landed before the CTA may exit
    for (int i = max(0, j - NS); i < j; ++i) mbar_wait(&full[i % NS], (i / NS) & 1, 0x519);
    return;
  }

  // ================================================================== consumers
  const int mt = warp % MT, kg = warp / MT;
  const int g = lane >> 2, t = lane & 3;
  const int f0 = t + 4 * (t & 1), f1 = f0 ^ 4;       // keys of an 8-key tile's columns 2t, 2t + 1
  // the key of column g: perm = {0, 4, 5, 1, 2, 6, 7, 3}
  const int pg = (g & 1) ? ((g >> 1) + 4 * ((g >> 1) & 1)) ^ 4 : (g >> 1) + 4 * ((g >> 1) & 1);
  int j = 0;                                         // units of this CTA so far
  bool ok = true, more = true;
  while (more) {
    const Item& it = w.it;
    const int shift = it.total - it.n;
    // rows g and g + 8 of this warp's tile
    int pos[2];
    uint32_t qf[D / 16][4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = it.rb * R + mt * 16 + g + 8 * e;
      const bool valid = row < it.n * p.group;
      const int i = row / p.group;
      pos[e] = valid ? shift + i : -1;
      const __half* q = a.q + (long long)(it.start + i) * a.q_stride + (long long)(it.h * p.group + row % p.group) * D;
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        uint2 v = make_uint2(0, 0);
        if (valid) v = __ldg(reinterpret_cast<const uint2*>(q + 16 * (t + 4 * (s >> 2)) + 4 * (s & 3)));
        qf[s][e] = v.x;
        qf[s][2 + e] = v.y;
      }
    }
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    // rows that see everything of a unit need no mask: the item's first and last row decide
    const int pfirst = shift + it.rb * R / p.group;
    const int plast = shift + min((it.rb * R + R - 1) / p.group, it.n - 1);
    const int full_lo = a.window > 0 ? max(it.lo, plast - a.window + 1) : it.lo;
    const int full_hi = pfirst < 0 ? 0 : (a.causal ? min(it.hi, pfirst + 1) : it.hi);

    for (int u = w.u0; u < w.u1; ++u, ++j) {
      if (j % KG != kg) continue;
      const int st = j % NS;
      if (ok) ok = mbar_wait(&full[st], (j / NS) & 1, 0x512);
      ok = __all_sync(0xffffffffu, ok);
      const int k0 = (it.t0 + u) * kAtT;
      const uint32_t sk = smem_u32(smem) + st * S::kStage, sv = sk + kAtT * D;
      const uint32_t ssc = smem_u32(smem) + S::oScales + st * S::kScales;
      const bool masked = k0 < full_lo || k0 + kAtT > full_hi;
#pragma unroll
      for (int half = 0; half < 2; ++half) {         // 32 keys at a time
        float s[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
          const int r = half * 32 + n * 8 + pg;
#pragma unroll
          for (int hf = 0; hf < D / 64; ++hf) {
            const uint4 kw = at_lds128(sk + at_swz<D>(r, t + 4 * hf));
            const uint32_t kk[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t b0, b1;
              at_cvt4(kk[x], b0, b1);
              const int q = hf * 4 + x;
              at_mma(s[n], qf[q][0], qf[q][1], qf[q][2], qf[q][3], b0, b1);
            }
          }
        }
        // logits, the scales of the two 16-key groups
        float4 sc[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint4 v = at_lds128(ssc + (half * 2 + x) * 16);
          sc[x] = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), 0.f);
        }
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < 4; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = fmaf(s[n][e], sc[n >> 1].x, sc[n >> 1].y);
            if (masked) {
              const int key = k0 + half * 32 + n * 8 + ((e & 1) ? f1 : f0);
              const int ps = pos[e >> 1];
              const bool see = key < it.total && ps >= 0 && (!a.causal || key <= ps) && (a.window <= 0 || key > ps - a.window);
              x = see ? x : -INFINITY;
            }
            s[n][e] = x;
            // a NaN must reach the maximum, else its row would go on without it
            mx[e >> 1] = (x > mx[e >> 1] || x != x) ? x : mx[e >> 1];
          }
        }
        float al[2], mu[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int d = 1; d < 4; d <<= 1) {
            const float y = __shfl_xor_sync(0xffffffffu, mx[e], d);
            mx[e] = (y > mx[e] || y != y) ? y : mx[e];
          }
          const float nm = (mx[e] > m[e] || mx[e] != mx[e]) ? mx[e] : m[e];
          mu[e] = nm == -INFINITY ? 0.f : nm;
          al[e] = m[e] == nm ? 1.f : attn_ex2(m[e] - mu[e]);
          m[e] = nm;
        }
        if (__any_sync(0xffffffffu, al[0] != 1.f || al[1] != 1.f)) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] *= al[e >> 1];
          l[0] *= al[0];
          l[1] *= al[1];
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[n][e] = attn_ex2(s[n][e] - mu[e >> 1]);
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          l[0] = fmaf(s[2 * x][0] + s[2 * x][1] + (s[2 * x + 1][0] + s[2 * x + 1][1]), sc[x].z, l[0]);
          l[1] = fmaf(s[2 * x][2] + s[2 * x][3] + (s[2 * x + 1][2] + s[2 * x + 1][3]), sc[x].z, l[1]);
        }
        // weights times V, 16 keys at a time: keys f0, f1 of the two 8-key tiles
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t a0 = at_pack(s[2 * x][0], s[2 * x][1]), a1 = at_pack(s[2 * x][2], s[2 * x][3]);
          const uint32_t a2 = at_pack(s[2 * x + 1][0], s[2 * x + 1][1]), a3 = at_pack(s[2 * x + 1][2], s[2 * x + 1][3]);
          const int r = half * 32 + x * 16;
          constexpr int NW = D / 32;                 // 32-bit words per lane and key
          uint32_t v[4][NW];
          const int rows[4] = {r + f0, r + f1, r + 8 + f0, r + 8 + f1};
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            if constexpr (D == 128) {
              const uint4 z = at_lds128(sv + at_swz<D>(rows[y], g));
              v[y][0] = z.x; v[y][1] = z.y; v[y][2] = z.z; v[y][3] = z.w;
            } else {
              const uint2 z = at_lds64(sv + at_swz<D>(rows[y], g >> 1) + (g & 1) * 8);
              v[y][0] = z.x; v[y][1] = z.y;
            }
            // what lies outside [lo, hi) was never written here, or belongs to nobody: weight 0 times
            // such a code must be 0, so the code is
            if (masked && (k0 + rows[y] >= it.hi || k0 + rows[y] < it.lo)) {
#pragma unroll
              for (int z = 0; z < NW; ++z) v[y][z] = 0u;
            }
          }
#pragma unroll
          for (int z = 0; z < NW; ++z) {
            uint32_t b0[4], b1[4];
            at_cvt4(__byte_perm(v[0][z], v[1][z], 0x5140), b0[0], b0[1]);
            at_cvt4(__byte_perm(v[0][z], v[1][z], 0x7362), b0[2], b0[3]);
            at_cvt4(__byte_perm(v[2][z], v[3][z], 0x5140), b1[0], b1[1]);
            at_cvt4(__byte_perm(v[2][z], v[3][z], 0x7362), b1[2], b1[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) at_mma(o[4 * z + i], a0, a1, a2, a3, b0[i], b1[i]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }

    // ---------------------------------------------------------------- join the warps
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], d);
    }
    at_sync_consumers();                             // the merge buffer is free
    {
      // accumulator (4z + i) of lane t holds channels NCH (2t) + 4z + i and NCH (2t + 1) + 4z + i
      constexpr int NCH = D / 8;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float* dst = merge + ((size_t)warp * 16 + g + 8 * e) * D;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int i = 0; i < D / 8; i += 4) {
            // spread the lanes' 16-byte stores over the banks: chunk index rotated by the row
            const int ch = (NCH * (2 * t + c) + i) / 4;
            *reinterpret_cast<float4*>(dst + 4 * (ch ^ (g & 7))) =
                make_float4(o[i][2 * e + c], o[i + 1][2 * e + c], o[i + 2][2 * e + c], o[i + 3][2 * e + c]);
          }
        }
        if (t == 0) ml[warp * 16 + g + 8 * e] = make_float2(m[e], l[e]);
      }
    }
    at_sync_consumers();
    const bool whole = w.u0 == 0 && w.u1 == it.units;
    const int c0 = sp.owner(w.at), c1 = sp.owner(w.at + it.units - 1);
    float* slots = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(a.workspace) + kAttnMaxCtas * 4);
    constexpr size_t SLOT = attn_slot_floats(R, D);
    float* slot = slots + SLOT * (2 * cta + (w.u0 == 0 ? 1 : 0));
    auto store = [&](int row, int ch, float4 v, float mm, float ll) {
      // one row's four channels of the finished item
      const int gr = it.rb * R + row;
      if (gr >= it.n * p.group) return;
      const int i = gr / p.group, head = it.h * p.group + gr % p.group;
      const float inv = ll > 0.f || ll != ll ? __fdiv_rn(1.f, ll) : 0.f;
      const uint2 u = make_uint2(at_pack(v.x * inv, v.y * inv), at_pack(v.z * inv, v.w * inv));
      *reinterpret_cast<uint2*>(a.out + (long long)(it.start + i) * a.out_stride + (long long)head * D + 4 * ch) = u;
      if (a.lse && ch == 0)
        a.lse[(long long)(it.start + i) * a.q_heads + head] =
            ll > 0.f || ll != ll ? (mm + log2f(ll)) * 0.6931471805599453f : -INFINITY;
    };
    for (int e = tid; e < R * (D / 4); e += kAtWarps * 32) {
      const int row = e / (D / 4), ch = e % (D / 4);
      const int tile = row >> 4, rr = row & 15;
      float mm = -INFINITY;
      bool nan = false;
#pragma unroll
      for (int k = 0; k < KG; ++k) {
        const float x = ml[(k * MT + tile) * 16 + rr].x;
        nan |= x != x;
        mm = fmaxf(mm, x);
      }
      if (nan) mm = NAN;
      const float base = mm == -INFINITY ? 0.f : mm;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      float ll = 0.f;
#pragma unroll
      for (int k = 0; k < KG; ++k) {
        const float2 x = ml[(k * MT + tile) * 16 + rr];
        const float f = attn_ex2(x.x - base);
        const float4 y = *reinterpret_cast<const float4*>(merge + ((size_t)(k * MT + tile) * 16 + rr) * D + 4 * (ch ^ (rr & 7)));
        v.x = fmaf(y.x, f, v.x);
        v.y = fmaf(y.y, f, v.y);
        v.z = fmaf(y.z, f, v.z);
        v.w = fmaf(y.w, f, v.w);
        ll = fmaf(x.y, f, ll);
      }
      if (whole) {
        store(row, ch, v, mm, ll);
      } else {
        *reinterpret_cast<float4*>(slot + (size_t)row * D + 4 * ch) = v;
        if (ch == 0) {
          slot[(size_t)R * D + row] = mm;
          slot[(size_t)R * D + R + row] = ll;
        }
      }
    }
    if (!whole) {
      // ------------------------------------------------------------ the last piece joins all of them
      unsigned int* ticket = reinterpret_cast<unsigned int*>(a.workspace) + c0;
      __threadfence();
      at_sync_consumers();
      if (tid == 0) {
        const unsigned int k = atomicAdd(ticket, 1u);
        *flag = k == (unsigned)(c1 - c0);
      }
      at_sync_consumers();
      if (*flag) {
        __threadfence();
        for (int e = tid; e < R * (D / 4); e += kAtWarps * 32) {
          const int row = e / (D / 4), ch = e % (D / 4);
          if (it.rb * R + row >= it.n * p.group) continue;
          float mm = -INFINITY;
          bool nan = false;
          for (int c = c0; c <= c1; ++c) {
            const float x = __ldcg(slots + SLOT * (2 * c + (c == c0 ? 1 : 0)) + (size_t)R * D + row);
            nan |= x != x;
            mm = fmaxf(mm, x);
          }
          if (nan) mm = NAN;
          const float base = mm == -INFINITY ? 0.f : mm;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          float ll = 0.f;
          for (int c = c0; c <= c1; ++c) {
            const float* s = slots + SLOT * (2 * c + (c == c0 ? 1 : 0));
            const float f = attn_ex2(__ldcg(s + (size_t)R * D + row) - base);
            const float4 y = __ldcg(reinterpret_cast<const float4*>(s + (size_t)row * D + 4 * ch));
            v.x = fmaf(y.x, f, v.x);
            v.y = fmaf(y.y, f, v.y);
            v.z = fmaf(y.z, f, v.z);
            v.w = fmaf(y.w, f, v.w);
            ll = fmaf(__ldcg(s + (size_t)R * D + R + row), f, ll);
          }
          store(row, ch, v, mm, ll);
        }
        if (tid == 0) *ticket = 0;
      }
    }
    more = w.next(a, p.group);
  }
}

// ---------------------------------------------------------------- host side

int64_t attn_workspace_bytes(int tokens, int batch, int q_heads, int kv_heads, int head_dim) {
  (void)tokens; (void)batch; (void)q_heads; (void)kv_heads;
  return (int64_t)(kAttnMaxCtas * 4 + 2ll * device_sm_count() * (int64_t)attn_slot_floats(256, head_dim) * 4);
}

template <int D, int MT>
static cudaError_t launch_attn_mt(AtParams& p, cudaStream_t stream) {
  auto kern = w4_attn_kernel<D, MT>;
  static FuncAttrCache attrs;
  cudaError_t ea = attrs.ensure(
      [&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, AtSmem<D>::kTotal); });
  if (ea != cudaSuccess) return ea;
  static_assert(AtSmem<D>::kTotal <= 227 * 1024, "shared memory of one CTA");
  const int rows = p.a.max_q * p.group;
  p.max_blocks = (rows + 16 * MT - 1) / (16 * MT);
  p.min_units = kAtWarps / MT;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)device_sm_count());
  cfg.blockDim = dim3(kAtThreads);
  cfg.dynamicSmemBytes = AtSmem<D>::kTotal;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
  note_launch();
  return e;
}

template <int D>
static cudaError_t launch_attn_d(AtParams& p, cudaStream_t stream) {
  const int rows = p.a.max_q * p.group;
  if (rows <= 16) return launch_attn_mt<D, 1>(p, stream);
  if (rows <= 32) return launch_attn_mt<D, 2>(p, stream);
  if (rows <= 64) return launch_attn_mt<D, 4>(p, stream);
  return launch_attn_mt<D, 8>(p, stream);
}

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t stream) {
  AtParams p;
  p.a = a;
  p.group = a.q_heads / a.c.kv_heads;
  const int box = a.c.page < kAtT ? a.c.page : kAtT;
  if (!encode_tmap_pages(&p.tk, a.c.k, a.c.dim, (long long)a.c.kv_heads * a.c.page, a.c.num_pages, a.c.page_stride, box) ||
      !encode_tmap_pages(&p.tv, a.c.v, a.c.dim, (long long)a.c.kv_heads * a.c.page, a.c.num_pages, a.c.page_stride, box))
    return cudaErrorNotSupported;
  return a.c.dim == 128 ? launch_attn_d<128>(p, stream) : launch_attn_d<64>(p, stream);
}

unsigned int read_clear_error_attn() { return read_clear_error_word_here(); }

}  // namespace w4
