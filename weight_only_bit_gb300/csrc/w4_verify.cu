// w4_verify.cu -- verification of drafted tokens against the target's probabilities (sm_103a).
//
// Mathematics.  p = softmax(x / T) is needed at the drafted tokens of every position and over the whole
// vocabulary at one position per sequence (the first refused one, or the last).  So: one pass over
// all logits for each row's maximum m and sum of 2^((x - m) c), c = log2(e) / T; then the decisions
// from a few gathered values; then one row per sequence again for the race
// argmax_v max(p - q, 0)(v) / e(v), which draws from the residual distribution without a sum over it
// (the smallest of independent exponential times e / w is at v with probability w_v / sum w).
//
// Work split.  Two launches, the second overlapping the first's tail (programmatic dependent launch).
// The first cuts each row into pieces so that the grid fills the GPU several times over and leaves
// (m, sum) or, at temperature 0, (largest logit, lowest token) of each piece in the workspace.  In
// the second, every CTA of a sequence joins the pieces in index order (the same bits in each CTA),
// decides, and runs its part of the race; the last CTA to finish (a ticket per sequence) takes the best
// part and writes the answer.  Best is the largest (score, lowest token) as one 64-bit key, so the
// order of arrival does not matter.
// What bounds it: DRAM bytes of the logits for a batch, launches and dependent loads for one sequence.
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "w4_common.cuh"
#include "w4_internal.h"
#include "w4_serve.h"

namespace w4 {

constexpr int kVfThreads = 256;
constexpr int kVfMaxPieces = 64;            // pieces of one row in the first launch
constexpr int kVfMaxParts = 64;             // CTAs of one sequence in the second

struct VerifyPlan {
  int pieces, piece;                        // per row; tokens of a piece (a multiple of 8)
  int parts, part;                          // per sequence; tokens of a part (a multiple of 8)
};

static VerifyPlan plan_verify(int batch, int rows, int vocab, int sms) {
  VerifyPlan p;
  // about four CTAs per SM in flight, at least 4096 tokens each (16 a thread)
  const long long want = 4LL * sms;
  auto cut = [&](long long n, int most) {
    long long k = (want + n - 1) / n;
    const long long fit = (vocab + 4095) / 4096;
    if (k > fit) k = fit;
    if (k > most) k = most;
    return (int)(k < 1 ? 1 : k);
  };
  p.pieces = cut((long long)batch * rows, kVfMaxPieces);
  p.piece = ((vocab + p.pieces - 1) / p.pieces + 7) & ~7;
  p.pieces = (vocab + p.piece - 1) / p.piece;
  p.parts = cut(batch, kVfMaxParts);
  p.part = ((vocab + p.parts - 1) / p.parts + 7) & ~7;
  p.parts = (vocab + p.part - 1) / p.part;
  return p;
}

// Workspace: [batch] tickets, [batch][kVfMaxParts][2] keys, [rows][kVfMaxPieces] (maximum, sum, first
// token with the maximum, unused).
struct VerifyWs {
  unsigned int* ticket;
  unsigned long long* keys;
  float4* stats;
};
__host__ __device__ inline size_t vf_keys_at(int batch) { return ((size_t)batch * 4 + 15) & ~(size_t)15; }
__host__ __device__ inline size_t vf_stats_at(int batch) { return vf_keys_at(batch) + (size_t)batch * kVfMaxParts * 16; }

int64_t verify_workspace_bytes(int batch, int drafts, int vocab) {
  (void)vocab;
  return (int64_t)(vf_stats_at(batch) + (size_t)batch * (2 * drafts + 1) * kVfMaxPieces * sizeof(float4));
}

__device__ __forceinline__ VerifyWs vf_ws(void* base, int batch) {
  uint8_t* p = static_cast<uint8_t*>(base);
  return {reinterpret_cast<unsigned int*>(p), reinterpret_cast<unsigned long long*>(p + vf_keys_at(batch)),
          reinterpret_cast<float4*>(p + vf_stats_at(batch))};
}

__device__ __forceinline__ float vf_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A logit as the definition takes it: NaN is -infinity, +infinity the largest FP16 value.
__device__ __forceinline__ float vf_logit(__half h) {
  const float x = __half2float(h);
  return x != x ? -INFINITY : fminf(x, 65504.f);
}

// Eight logits of a row from token v on (v a multiple of 8), whatever the row's alignment; -infinity
// past the end.
__device__ __forceinline__ void vf_load8(const __half* row, int v, int end, float (&x)[8]) {
  if (v + 8 <= end && ((reinterpret_cast<uintptr_t>(row + v) & 15) == 0)) {
    const uint4 w = ld_nc_v4(row + v);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 p = *reinterpret_cast<const __half2*>(&u[i]);
      x[2 * i] = vf_logit(__low2half(p));
      x[2 * i + 1] = vf_logit(__high2half(p));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v + i < end ? vf_logit(row[v + i]) : -INFINITY;
  }
}

// Key of (value, token): larger value first, then the lower token.  Values are not NaN.
__device__ __forceinline__ unsigned long long vf_key(float x, int v) {
  uint32_t u = __float_as_uint(x);
  u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return ((unsigned long long)u << 32) | (uint32_t)~v;
}
__device__ __forceinline__ float vf_key_value(unsigned long long k) {
  const uint32_t u = (uint32_t)(k >> 32);
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}
__device__ __forceinline__ int vf_key_token(unsigned long long k) { return (int)~(uint32_t)k; }

__device__ __forceinline__ unsigned long long vf_max(unsigned long long a, unsigned long long b) { return a > b ? a : b; }

__device__ __forceinline__ unsigned long long vf_warp_max(unsigned long long k) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) k = vf_max(k, __shfl_xor_sync(0xffffffffu, k, o));
  return k;
}

// Joins two (maximum, sum) pairs.
__device__ __forceinline__ float2 vf_join(float2 a, float2 b, float c) {
  const float m = fmaxf(a.x, b.x);
  if (m == -INFINITY) return make_float2(m, 0.f);
  return make_float2(m, a.y * vf_ex2((a.x - m) * c) + b.y * vf_ex2((b.x - m) * c));
}

// Row r of a sequence: target rows 0 ... drafts, then the draft's rows.
__device__ __forceinline__ const __half* vf_row(const VerifyArgs& a, int b, int r) {
  return r <= a.drafts ? a.target + ((long long)b * (a.drafts + 1) + r) * a.target_stride
                       : a.draft + ((long long)b * a.drafts + (r - a.drafts - 1)) * a.draft_stride;
}

__device__ __forceinline__ int vf_count(const VerifyArgs& a, int b) {
  return a.n_drafts ? min(max(__ldg(a.n_drafts + b), 0), a.drafts) : a.drafts;
}

// First launch: CTA = one piece of one row.
__global__ void __launch_bounds__(kVfThreads) w4_verify_stats_kernel(const __grid_constant__ VerifyArgs a, VerifyPlan pl,
                                                                     int rows) {
  __shared__ float2 red[kVfThreads / 32];
  __shared__ unsigned long long redk[kVfThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int piece = (int)blockIdx.x % pl.pieces;
  const int br = (int)blockIdx.x / pl.pieces;
  const int b = br / rows, r = br % rows;
  const int n = vf_count(a, b);
  if (r <= a.drafts ? r > n : r - a.drafts - 1 >= n) return;      // a row that nothing reads
  const __half* row = vf_row(a, b, r);
  const int v0 = piece * pl.piece, v1 = min(v0 + pl.piece, a.vocab);
  const bool greedy = a.temperature == 0.f;
  const float c = 1.4426950408889634f / (greedy ? 1.f : a.temperature);
  float2 s = make_float2(-INFINITY, 0.f);
  unsigned long long key = 0;
  for (int v = v0 + tid * 8; v < v1; v += kVfThreads * 16) {
    float x[16];
    vf_load8(row, v, v1, *reinterpret_cast<float(*)[8]>(&x[0]));
    const int w = v + kVfThreads * 8;
    if (w < v1) vf_load8(row, w, v1, *reinterpret_cast<float(*)[8]>(&x[8]));
    else {
#pragma unroll
      for (int i = 8; i < 16; ++i) x[i] = -INFINITY;
    }
    float m = x[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) m = fmaxf(m, x[i]);
    if (greedy && m > s.x) {
      // the first token with this value, in index order (v before w)
      int at = 0;
#pragma unroll
      for (int i = 15; i >= 0; --i)
        if (x[i] == m) at = i;
      key = vf_max(key, vf_key(m, at < 8 ? v + at : w + at - 8));
    }
    const float nm = fmaxf(s.x, m);
    if (nm != -INFINITY) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) sum += vf_ex2((x[i] - nm) * c);
      s.y = s.y * vf_ex2((s.x - nm) * c) + sum;
      s.x = nm;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float2 t = make_float2(__shfl_xor_sync(0xffffffffu, s.x, o), __shfl_xor_sync(0xffffffffu, s.y, o));
    s = vf_join(s, t, c);
  }
  if (greedy) key = vf_warp_max(key);
  if (lane == 0) {
    red[warp] = s;
    redk[warp] = key;
  }
  __syncthreads();
  if (tid == 0) {
#pragma unroll
    for (int w = 1; w < kVfThreads / 32; ++w) {
      s = vf_join(s, red[w], c);
      key = vf_max(key, redk[w]);
    }
    const VerifyWs ws = vf_ws(a.workspace, a.batch);
    ws.stats[(size_t)br * kVfMaxPieces + piece] = make_float4(s.x, s.y, __int_as_float(vf_key_token(key)), 0.f);
  }
}

// Whole-row statistics from the pieces, by a warp (every lane gets the result): the maximum, log2 of the
// sum of 2^((x - m) c), and the first token with the maximum.
struct RowStat {
  float m, lg;
  int at;
};
__device__ __forceinline__ RowStat vf_row_stat(const VerifyWs& ws, int br, int pieces, float c, int lane) {
  float2 s = make_float2(-INFINITY, 0.f);
  unsigned long long key = 0;
  for (int i = lane; i < pieces; i += 32) {
    const float4 f = __ldcg(ws.stats + (size_t)br * kVfMaxPieces + i);
    s = vf_join(s, make_float2(f.x, f.y), c);
    key = vf_max(key, vf_key(f.x, __float_as_int(f.z)));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    // both partners add in the same order, so that every lane holds the same bits
    const float2 t = make_float2(__shfl_xor_sync(0xffffffffu, s.x, o), __shfl_xor_sync(0xffffffffu, s.y, o));
    s = (lane & o) ? vf_join(t, s, c) : vf_join(s, t, c);
  }
  key = vf_warp_max(key);
  return {s.x, s.y > 0.f ? log2f(s.y) : -INFINITY, vf_key_token(key)};
}

// Probability of a logit in a row with these statistics; 0 for a row without any finite logit.
__device__ __forceinline__ float vf_prob(float x, const RowStat& s, float c) {
  return x == -INFINITY || s.m == -INFINITY ? 0.f : vf_ex2((x - s.m) * c - s.lg);
}

// Second launch: CTA = one part of one sequence's race.
__global__ void __launch_bounds__(kVfThreads) w4_verify_pick_kernel(const __grid_constant__ VerifyArgs a, VerifyPlan pl,
                                                                    int rows) {
  __shared__ RowStat stat[2 * W4_MAX_DRAFTS + 1];
  __shared__ unsigned long long red[kVfThreads / 32][2];
  __shared__ int s_last;
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int part = (int)blockIdx.x % pl.parts;
  const int b = (int)blockIdx.x / pl.parts;
  const VerifyWs ws = vf_ws(a.workspace, a.batch);
  const bool greedy = a.temperature == 0.f;
  const float c = 1.4426950408889634f / (greedy ? 1.f : a.temperature);
  const int n = vf_count(a, b);
  const bool with_q = rows > a.drafts + 1;
  for (int r = warp; r < rows; r += kVfThreads / 32) {
    if (r <= a.drafts ? r > n : r - a.drafts - 1 >= n) continue;
    const RowStat s = vf_row_stat(ws, b * rows + r, pl.pieces, c, lane);
    if (lane == 0) stat[r] = s;
  }
  __syncthreads();
  // every warp decides for itself: lane i looks at drafted token i (W4_MAX_DRAFTS < 32)
  bool refuse = true;
  int x = -1;
  float lp = 0.f;
  if (lane < n) {
    x = __ldg(a.draft_tokens + (long long)b * a.drafts + lane);
    if (x >= 0 && x < a.vocab) {
      const RowStat s = stat[lane];
      const float logit = vf_logit(vf_row(a, b, lane)[x]);
      lp = ((logit - s.m) * c - s.lg) * 0.6931471805599453f;
      if (greedy) {
        refuse = !(s.at == x && s.m != -INFINITY);
      } else {
        const float p = vf_prob(logit, s, c);
        const float u = __ldg(a.u + (long long)b * a.drafts + lane);
        const float q = with_q ? vf_prob(vf_logit(vf_row(a, b, a.drafts + 1 + lane)[x]), stat[a.drafts + 1 + lane], c) : 1.f;
        refuse = !(__fmul_rn(u, q) < p);
      }
    }
  }
  const int acc = __ffs(__ballot_sync(0xffffffffu, refuse)) - 1;   // lane n always refuses
  unsigned long long best = 0, plain = 0;    // of the residual, and of p alone
  if (!greedy) {
    const __half* row = vf_row(a, b, acc);
    const RowStat s = stat[acc];
    const bool residual = acc < n;
    const bool q_row = residual && with_q;
    const __half* qrow = q_row ? vf_row(a, b, a.drafts + 1 + acc) : row;
    const RowStat sq = q_row ? stat[a.drafts + 1 + acc] : s;
    const int certain = residual && !with_q ? __shfl_sync(0xffffffffu, x, acc) : -1;
    const float* e = a.e + (long long)b * a.vocab;
    const int v0 = part * pl.part, v1 = min(v0 + pl.part, a.vocab);
    for (int v = v0 + tid * 8; v < v1; v += kVfThreads * 8) {
      float px[8], qx[8], ee[8];
      vf_load8(row, v, v1, px);
      if (q_row) vf_load8(qrow, v, v1, qx);
      if (v + 8 <= v1 && ((reinterpret_cast<uintptr_t>(e + v) & 15) == 0)) {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 f = __ldg(reinterpret_cast<const float4*>(e + v + i));
          ee[i] = f.x; ee[i + 1] = f.y; ee[i + 2] = f.z; ee[i + 3] = f.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) ee[i] = v + i < v1 ? __ldg(e + v + i) : 1.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = vf_prob(px[i], s, c);
        if (p > 0.f) {
          const float d = __fdiv_rn(p, ee[i]);
          if (d >= 0.f) plain = vf_max(plain, vf_key(d, v + i));
          float w = p;
          if (q_row) w = p - vf_prob(qx[i], sq, c);
          else if (v + i == certain) w = 0.f;
          if (w > 0.f) {
            const float f = __fdiv_rn(w, ee[i]);
            if (f >= 0.f) best = vf_max(best, vf_key(f, v + i));
          }
        }
      }
    }
    best = vf_warp_max(best);
    plain = vf_warp_max(plain);
    if (lane == 0) {
      red[warp][0] = best;
      red[warp][1] = plain;
    }
    __syncthreads();
    if (tid == 0) {
#pragma unroll
      for (int w = 1; w < kVfThreads / 32; ++w) {
        best = vf_max(best, red[w][0]);
        plain = vf_max(plain, red[w][1]);
      }
      unsigned long long* k = ws.keys + ((size_t)b * kVfMaxParts + part) * 2;
      k[0] = best;
      k[1] = plain;
      __threadfence();
      s_last = atomicAdd(ws.ticket + b, 1u) == (unsigned)pl.parts - 1u;
    }
    __syncthreads();
    if (!s_last) return;
    if (warp != 0) return;
    __threadfence();
    best = plain = 0;
    for (int i = lane; i < pl.parts; i += 32) {
      const unsigned long long* k = ws.keys + ((size_t)b * kVfMaxParts + i) * 2;
      best = vf_max(best, __ldcg(k));
      plain = vf_max(plain, __ldcg(k + 1));
    }
    best = vf_warp_max(best);
    plain = vf_warp_max(plain);
    if (best == 0) best = plain;
    if (lane == 0) ws.ticket[b] = 0;         // ready for the next call
  } else if (part != 0 || warp != 0) {
    return;
  }
  // ---- the answer, by one warp
  int token = -1;
  float tlp = -INFINITY;
  const RowStat s = stat[acc];
  if (greedy) {
    if (s.m != -INFINITY) token = s.at;
  } else if (best != 0) {
    token = vf_key_token(best);
  }
  if (token >= 0) tlp = ((vf_logit(vf_row(a, b, acc)[token]) - s.m) * c - s.lg) * 0.6931471805599453f;
  if (lane <= a.drafts) {
    const long long o = (long long)b * (a.drafts + 1) + lane;
    a.tokens[o] = lane < acc ? x : lane == acc ? token : -1;
    if (a.logprob) a.logprob[o] = lane < acc ? lp : lane == acc ? tlp : 0.f;
  }
  if (lane == 0) a.accepted[b] = acc;
}

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t stream) {
  const bool with_q = a.draft != nullptr && a.temperature > 0.f;
  const int rows = a.drafts + 1 + (with_q ? a.drafts : 0);
  const VerifyPlan pl = plan_verify(a.batch, rows, a.vocab, device_sm_count());
  const long long g1 = (long long)a.batch * rows * pl.pieces;
  const long long g2 = (long long)a.batch * (a.temperature > 0.f ? pl.parts : 1);
  if (g1 > 0x7fffffffLL || g2 > 0x7fffffffLL) return cudaErrorNotSupported;
  VerifyPlan p2 = pl;
  if (a.temperature == 0.f) p2.parts = 1;    // no race: one CTA a sequence
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kVfThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)g1);
  cudaError_t e = cudaLaunchKernelEx(&cfg, w4_verify_stats_kernel, a, pl, rows);
  if (e != cudaSuccess) return e;
  note_launch();
  cfg.gridDim = dim3((unsigned)g2);
  e = cudaLaunchKernelEx(&cfg, w4_verify_pick_kernel, a, p2, rows);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace w4
