// linear_simt.cu -- the dense product on FMA pipes: fp32 layers (the tensor
// cores' tf32 keeps 11 significant bits, fp32 results here keep all of them).

#include <cooperative_groups.h>

#include <algorithm>

#include "linear.h"

namespace cg = cooperative_groups;

namespace moe {

namespace {

constexpr int LS_THREADS = 256;
constexpr int LS_BK = 16;

// A TILE x 16 piece of an operand into registers: threads run along the
// dimension that is contiguous in memory.
template <int TILE>
__device__ __forceinline__ void fetch(const float* base, long long rs, long long ks, int r0, int rows, int k0, int k1,
                                      float (&v)[TILE / 16])
{
    const int t = threadIdx.x;
#pragma unroll
    for (int i = 0; i < TILE / 16; ++i) {
        const int r = ks == 1 ? t / LS_BK + (LS_THREADS / LS_BK) * i : t % TILE;
        const int k = ks == 1 ? t % LS_BK : t / TILE + (LS_THREADS / TILE) * i;
        v[i] = (r0 + r < rows && k0 + k < k1) ? base[(long long)(r0 + r) * rs + (long long)(k0 + k) * ks] : 0.f;
    }
}

template <int TILE>
__device__ __forceinline__ void stash(float (*s)[TILE + 4], long long ks, const float (&v)[TILE / 16])
{
    const int t = threadIdx.x;
#pragma unroll
    for (int i = 0; i < TILE / 16; ++i) {
        const int r = ks == 1 ? t / LS_BK + (LS_THREADS / LS_BK) * i : t % TILE;
        const int k = ks == 1 ? t % LS_BK : t / TILE + (LS_THREADS / TILE) * i;
        s[k][r] = v[i];
    }
}

// One TILE x TILE output tile per cluster; the cluster's blocks split K and add
// their partial tiles in order of rank through distributed shared memory.
template <int TILE>
__global__ void __launch_bounds__(LS_THREADS) linear_simt_kernel(const SimtProduct p, int splits, int tiles_c)
{
    constexpr int F = TILE / 16;                 // outputs per thread and direction
    extern __shared__ float s_dyn[];
    float(*sp)[LS_BK][TILE + 4] = reinterpret_cast<float(*)[LS_BK][TILE + 4]>(s_dyn);
    float(*sq)[LS_BK][TILE + 4] = sp + 2;
    const int rank = blockIdx.x % splits, tile = blockIdx.x / splits;
    const int r0 = (tile / tiles_c) * TILE, c0 = (tile % tiles_c) * TILE;
    const int blocks_k = cdiv(p.K, LS_BK);
    const int kb0 = (int)((long long)blocks_k * rank / splits), kb1 = (int)((long long)blocks_k * (rank + 1) / splits);
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[F][F];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) acc[i][j] = 0.f;
    pdl_wait();
    pdl_trigger();
    float vp[F], vq[F];
    if (kb0 < kb1) {
        fetch<TILE>(p.P, p.p_rs, p.p_ks, r0, p.R, kb0 * LS_BK, p.K, vp);
        fetch<TILE>(p.Q, p.q_rs, p.q_ks, c0, p.C, kb0 * LS_BK, p.K, vq);
    }
    int buf = 0;
    for (int kb = kb0; kb < kb1; ++kb, buf ^= 1) {
        stash<TILE>(sp[buf], p.p_ks, vp);
        stash<TILE>(sq[buf], p.q_ks, vq);
        __syncthreads();
        if (kb + 1 < kb1) {
            fetch<TILE>(p.P, p.p_rs, p.p_ks, r0, p.R, (kb + 1) * LS_BK, p.K, vp);
            fetch<TILE>(p.Q, p.q_rs, p.q_ks, c0, p.C, (kb + 1) * LS_BK, p.K, vq);
        }
#pragma unroll
        for (int k = 0; k < LS_BK; ++k) {
            float a[F], b[F];
#pragma unroll
            for (int i = 0; i < F; i += 4) {
                *reinterpret_cast<float4*>(a + i) = *reinterpret_cast<const float4*>(&sp[buf][k][ty * 4 + 16 * i]);
                *reinterpret_cast<float4*>(b + i) = *reinterpret_cast<const float4*>(&sq[buf][k][tx * 4 + 16 * i]);
            }
#pragma unroll
            for (int i = 0; i < F; ++i)
#pragma unroll
                for (int j = 0; j < F; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
        }
    }
    // row / column of accumulator i: ty * 4 + (i % 4) + 64 * (i / 4)
    if (splits == 1) {
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int j = 0; j < F; ++j) {
                const int r = r0 + ty * 4 + (i % 4) + 64 * (i / 4), c = c0 + tx * 4 + (j % 4) + 64 * (j / 4);
                if (r < p.R && c < p.C) lin_store(p.epi, r, c, acc[i][j]);
            }
        return;
    }
    float* red = s_dyn;                          // [TILE][TILE]
    __syncthreads();
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j)
            red[(ty * 4 + (i % 4) + 64 * (i / 4)) * TILE + tx * 4 + (j % 4) + 64 * (j / 4)] = acc[i][j];
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    const int per = TILE / splits;
    for (int i = threadIdx.x; i < per * TILE; i += LS_THREADS) {
        const int r = rank * per + i / TILE, c = i % TILE;
        if (r0 + r >= p.R || c0 + c >= p.C) continue;
        float v = 0.f;
        for (int q = 0; q < splits; ++q) v += cl.map_shared_rank(red, q)[r * TILE + c];
        lin_store(p.epi, r0 + r, c0 + c, v);
    }
    cl.sync();
}

template <int TILE>
moe_status launch(const SimtProduct& p, int splits, cudaStream_t st)
{
    const int tiles_c = cdiv(p.C, TILE);
    const long long tiles = (long long)cdiv(p.R, TILE) * tiles_c;
    if (tiles * splits >= (1ll << 31)) return MOE_ERR_UNSUPPORTED;
    const int smem = std::max(4 * LS_BK * (TILE + 4) * 4, splits > 1 ? TILE * TILE * 4 : 0);
    auto* fn = linear_simt_kernel<TILE>;
    if (ensure_smem_attr(reinterpret_cast<const void*>(fn), smem) != cudaSuccess) return MOE_ERR_CUDA;
    return launch_dependent(fn, dim3((unsigned)(tiles * splits)), LS_THREADS, smem, splits, st, p, splits, tiles_c);
}

}  // namespace

moe_status launch_linear_simt(const SimtProduct& p, cudaStream_t st)
{
    const long long big = (long long)cdiv(p.R, 128) * cdiv(p.C, 128);
    const int sms = num_sms();
    if (big >= 2 * sms) return launch<128>(p, 1, st);
    const long long tiles = (long long)cdiv(p.R, 64) * cdiv(p.C, 64);
    int splits = 1;
    while (splits < 8 && tiles * splits < sms && p.K >= 64 * splits) splits *= 2;
    return launch<64>(p, splits, st);
}

}  // namespace moe
