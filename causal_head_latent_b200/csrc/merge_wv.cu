// End of the 4-bit decode: the pieces' softmax states joined and W_v applied,
//   c^[b, h] = cache_scale * sum_i 2^(m_i - M) acc_i / sum_i 2^(m_i - M) l_i
//   o[b, 128h + r] = sigmoid(G[b, 128h + r]) * sum_c W_v[128h + r, c] c^[b, h, c].
//
// One CTA per (head, 32 sequences), sixteen warps.  W_v^(h) (128 KB at d_c = 512) comes into
// shared memory by TMA before the launch waits for the decode kernel it begins beside
// (programmatic launch), so its time is hidden.  Then each sequence's pieces are summed in
// float32, lane l holding the columns 128 * k + 4l .. of every 128: with more than
// eight sequences a warp sums whole sequences, with fewer 2 to 16 warps share the pieces of
// one and add up through shared memory.  c^ goes into the product as bfloat16 hi + lo (two
// passes, about 16 bits), D[r, b] on tcgen05 with M = 128, N = 32.
// Bound by latency at small batches and by reading the partial states at large ones.
#include "compact.h"
#include "internal.h"
#include "ptx.cuh"
#include "share_walk.cuh"

namespace gmla {
namespace merge_wv {

constexpr int HD = 128;
constexpr int NB = 32;                // sequences per CTA (the MMA's N)
constexpr int WARPS = 16, THREADS = 32 * WARPS;
constexpr int WCHUNK = 128 * 64 * 2;  // 128 rows x 64 columns of W_v, 128-byte swizzled
constexpr int MAX_CHUNKS = 8;         // d_c <= 512
constexpr int BCHUNK = NB * 64 * 2;

struct Smem {
  uint8_t w[MAX_CHUNKS][WCHUNK];
  uint8_t hi[MAX_CHUNKS][BCHUNK];  // bf16(c^) of the 32 sequences
  uint8_t lo[MAX_CHUNKS][BCHUNK];  // bf16(c^ - hi)
  float part[WARPS][512];          // pieces of one sequence summed by several warps
  float sum[WARPS], top[WARPS];
  uint64_t full, done;
  long long sums[2];
  uint32_t tmem_base;
};

struct Params {
  ShareBatch batch;
  long long G;
  int H, dc;
  const float *part_m, *part_l, *part_acc;  // [R, H], [R, H], [R, H, dc]; record = share + sequence
  float cache_scale;
  const uint16_t *gate;
  uint16_t *out;
  unsigned *status;
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__global__ void __launch_bounds__(THREADS, 1) merge_wv_kernel(const __grid_constant__ CUtensorMap tmW, const Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const int h = blockIdx.x, b0 = blockIdx.y * NB, nb = min(NB, p.batch.B - b0);
  const int nchunk = p.dc / 64;
  if (threadIdx.x == 0) {
    mbar_init(&sm.full, 1);
    mbar_init(&sm.done, 1);
    fence_barrier_init();
    mbar_arrive_expect_tx(&sm.full, (uint32_t)(nchunk * WCHUNK));
    for (int k = 0; k < nchunk; ++k) tma_load_2d(sm.w[k], &tmW, &sm.full, 64 * k, HD * h);
  }
  if (warp == 0) {
    tmem_alloc(&sm.tmem_base, NB);
    tmem_relinquish();
  }
  // rows of sequences that are not there are zero
  for (int i = threadIdx.x; i < nchunk * (NB - nb) * 8; i += THREADS) {
    const int k = i / ((NB - nb) * 8), off = (nb * 8 + i % ((NB - nb) * 8)) * 16;
    *reinterpret_cast<uint4 *>(sm.hi[k] + off) = make_uint4(0u, 0u, 0u, 0u);
    *reinterpret_cast<uint4 *>(sm.lo[k] + off) = make_uint4(0u, 0u, 0u, 0u);
  }
  long long before, total;
  block_place_sums(p.batch, b0, sm.sums, &before, &total);
  const long long G = min(p.G, total);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem_base, 0);
  grid_dependency_wait();  // the partial states

  // c^ of sequence bb, columns c..c+3, from the pieces' sum t and l, as bfloat16 hi and lo: chunk
  // c / 64, 16-byte slot ((c % 64) / 8) ^ (bb % 8), half (c / 4) % 2.  No visible row: l = 0, c^ = 0.
  auto put = [&](int bb, int c, float4 t, float l) {
    const float inv = l != 0.f ? p.cache_scale / l : 0.f;
    const float x[4] = {t.x * inv, t.y * inv, t.z * inv, t.w * inv};
    uint32_t hw[2], lw[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __nv_bfloat16 h0 = __float2bfloat16_rn(x[2 * i]), h1 = __float2bfloat16_rn(x[2 * i + 1]);
      hw[i] = (uint32_t)__bfloat16_as_ushort(h0) | ((uint32_t)__bfloat16_as_ushort(h1) << 16);
      lw[i] = pack_bf16x2(x[2 * i] - __bfloat162float(h0), x[2 * i + 1] - __bfloat162float(h1));
    }
    const uint32_t off = bb * 128 + ((((c & 63) >> 3) ^ (bb & 7)) << 4) + ((c >> 2) & 1) * 8;
    *reinterpret_cast<uint2 *>(sm.hi[c >> 6] + off) = make_uint2(hw[0], hw[1]);
    *reinterpret_cast<uint2 *>(sm.lo[c >> 6] + off) = make_uint2(lw[0], lw[1]);
  };

  // warps per sequence (a power of two), this warp's first sequence and its place among them
  const int wps = nb > 8 ? 1 : nb > 4 ? 2 : nb > 2 ? 4 : nb > 1 ? 8 : 16;
  const int place = warp % wps;
  int bs = 0;  // sequence up to whose start `before` counts
  for (int b = 0; b < nb; b += WARPS / wps) {
    const int mine = b + warp / wps;
    float m = -INFINITY, l = 0.f;
    float4 a[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) a[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (mine < nb) {
      for (; bs < mine; ++bs) before += p.batch.places(b0 + bs);
      const int n = p.batch.tiles(b0 + mine);
      if (n > 0) {
        long long s0, s1;
        shares_of(p.batch, before, n, total, G, &s0, &s1);
        const size_t r0 = (size_t)(b0 + mine) * p.H + h;  // record of share s: s * H + r0
        for (long long s = s0 + lane; s <= s1; s += 32) m = fmaxf(m, p.part_m[s * p.H + r0]);
        m = warp_max(m);
        constexpr int U = 4;
        for (long long s = s0 + place; s <= s1; s += U * wps) {
          float e[U];
          float4 v[U][4];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const long long su = s + u * wps;
            const size_t r = (size_t)min(su, s1) * p.H + r0;
            const float mu = p.part_m[r];
            e[u] = su > s1 || mu == -INFINITY ? 0.f : fast_exp2(mu - m);
            if (lane == 0) l += e[u] * p.part_l[r];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (128 * k + 4 * lane < p.dc)
                v[u][k] = __ldcs(reinterpret_cast<const float4 *>(p.part_acc + r * p.dc + 128 * k + 4 * lane));
          }
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (128 * k + 4 * lane < p.dc) {
                a[k].x = fmaf(e[u], v[u][k].x, a[k].x);
                a[k].y = fmaf(e[u], v[u][k].y, a[k].y);
                a[k].z = fmaf(e[u], v[u][k].z, a[k].z);
                a[k].w = fmaf(e[u], v[u][k].w, a[k].w);
              }
        }
        l = warp_sum(l);
        // every score -inf or NaN: NaN, not the zeros of an empty sequence
        if (m == -INFINITY) l = __uint_as_float(0x7fffffffu);
      }
    }
    if (wps > 1) {  // nb <= WARPS / wps: one turn of the loop, every warp in it
#pragma unroll
      for (int k = 0; k < 4; ++k) *reinterpret_cast<float4 *>(&sm.part[warp][128 * k + 4 * lane]) = a[k];
      if (lane == 0) sm.sum[warp] = l;
      __syncthreads();
      // all threads: four columns of a sequence each
#pragma unroll 1
      for (int i = threadIdx.x; i < nb * (p.dc / 4); i += THREADS) {
        const int bb = i / (p.dc / 4), c = 4 * (i % (p.dc / 4));
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll 4
        for (int w = bb * wps; w < (bb + 1) * wps; ++w) {
          const float4 v = *reinterpret_cast<const float4 *>(&sm.part[w][c]);
          t.x += v.x;
          t.y += v.y;
          t.z += v.z;
          t.w += v.w;
          sum += sm.sum[w];
        }
        put(bb, c, t, sum);
      }
    } else if (mine < nb) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (128 * k + 4 * lane < p.dc) put(mine, 128 * k + 4 * lane, a[k], l);
    }
  }
  fence_proxy_async_smem();
  __syncthreads();
  if (warp == 0) {  // converged, one lane predicated: the operands' addresses stay in uniform registers
    const uint32_t issue = elect_one();
    if (warp_wait(&sm.full, 0, p.status)) {
      tc_fence_after();
      constexpr uint32_t idesc = idesc_bf16_f32(128, NB, false, false);
      const uint32_t aw = smem_u32(sm.w[0]), ahi = smem_u32(sm.hi[0]), alo = smem_u32(sm.lo[0]);
#pragma unroll 1
      for (int k = 0; k < nchunk; ++k) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t a = sdesc_sw128(aw + k * WCHUNK + kk * 32, 16, 1024);
          umma_f16_ss_if(issue, tmem, a, sdesc_sw128(ahi + k * BCHUNK + kk * 32, 16, 1024), idesc, (k | kk) ? 1u : 0u);
          umma_f16_ss_if(issue, tmem, a, sdesc_sw128(alo + k * BCHUNK + kk * 32, 16, 1024), idesc, 1u);
        }
      }
    }
    umma_commit_if(issue, &sm.done);
  }
  __syncwarp();
  if (warp < 4) {
    const int r = 32 * warp + lane;  // row of W_v^(h): output channel 128h + r
    const size_t at = ((size_t)b0 * p.H + h) * HD + r, ld = (size_t)p.H * HD;
    // Eight sequences at a time, the next eight's gate logits in flight; a loop, because
    // straight-line code for 32 costs a short call more in cold instruction fetches than work.
    uint16_t gate[8];
    auto load_gates = [&](int j0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) gate[j] = p.gate && j0 + j < nb ? p.gate[at + (j0 + j) * ld] : (uint16_t)0;
    };
    load_gates(0);
    const bool ok = warp_wait(&sm.done, 0, p.status);
    tc_fence_after();
#pragma unroll 1
    for (int j0 = 0; j0 < nb; j0 += 8) {
      float v[8];
      tmem_ld8(tmem + ((uint32_t)(warp * 32) << 16) + j0, v);
      if (p.gate) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= sigmoidf_(bf16_to_f32(gate[j]));
        load_gates(j0 + 8);
      }
      if (ok) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j0 + j < nb) p.out[at + (j0 + j) * ld] = __bfloat16_as_ushort(__float2bfloat16_rn(v[j]));
      }
      __syncwarp();
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, NB);
  }
}

}  // namespace merge_wv

int launch_merge_wv(const MergeWvArgs &a, cudaStream_t stream) {
  using namespace merge_wv;
  if (!set_smem_limit_once(reinterpret_cast<const void *>(merge_wv_kernel), (int)sizeof(Smem), kSmemMergeWv)) return -1;
  CUtensorMap tw;
  const long long dw[2] = {a.dc, (long long)a.H * HD}, sw[1] = {a.dc};
  const unsigned bw[2] = {64, 128};
  if (!make_tmap_bf16(&tw, a.Wv, 2, dw, sw, bw)) return -1;
  const Params p{ShareBatch{a.lens, a.B, a.L, a.tile, a.extra}, a.G, a.H, a.dc, a.part_m, a.part_l, a.part_acc, a.cache_scale,
                 a.gate, a.out, a.status};
  return launch_beside(true, merge_wv_kernel, dim3(a.H, (a.B + NB - 1) / NB), dim3(THREADS), sizeof(Smem), stream, tw, p);
}

}  // namespace gmla
