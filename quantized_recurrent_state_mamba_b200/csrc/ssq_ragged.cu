// ssq_ragged.cu -- ssq_prefill_ragged token by token: single tokens, short
// runs, and the shapes and types that the chunk kernel does not take.
//
//   S = fma(exp(fl(dt*A)), S, fl(fl(dt*x)*B)),   y = S C + D x
//
// in fp32, the same operations in the same order as ssq_prefill, the state in
// registers for the whole run.  A block owns up to 256/LPR rows of one head of
// one request (LPR = d_state/32 lanes per row), so B, C, dt and exp(dt*A) are
// uniform in the block: they are converted to fp32 in shared memory once per
// kTok tokens.  The pieces of B and C that a row's lanes read lie 36 floats
// apart, so that the lanes' 16-byte reads hit different banks.  For a single
// token the kernel is bound by the pool's traffic; for long runs by the fp32
// pipe and the chain from token to token.
#include <cuda_fp16.h>

#include "ssq_ragged.h"
#include "ssq_rowio.cuh"

namespace ssq {

namespace {

constexpr int kTok = 8;        // tokens staged at a time

template <int TYPE>
__device__ __forceinline__ float load_act(const void* p, long long i)
{
    if constexpr (TYPE == SSQ_T_BF16)
        return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
    else if constexpr (TYPE == SSQ_T_F16)
        return __half2float(reinterpret_cast<const __half*>(p)[i]);
    else
        return reinterpret_cast<const float*>(p)[i];
}
template <int TYPE>
__device__ __forceinline__ void store_act(void* p, long long i, float v)
{
    if constexpr (TYPE == SSQ_T_BF16)
        reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else if constexpr (TYPE == SSQ_T_F16)
        reinterpret_cast<__half*>(p)[i] = __float2half_rn(v);
    else
        reinterpret_cast<float*>(p)[i] = v;
}

// Floats of one staged row of B or C: LPR pieces of E floats, 4 floats apart.
template <int N>
constexpr int kRowF = Shape<N>::LPR * (Shape<N>::E + 4);

template <int FMT, int N, int TYPE>
__global__ void __launch_bounds__(kThreads)
tokens_kernel(const __grid_constant__ PoolView pv, const __grid_constant__ RaggedCall rc)
{
    constexpr int E = Shape<N>::E, LPR = Shape<N>::LPR;
    __shared__ __align__(16) float sB[kTok][kRowF<N>], sC[kTok][kRowF<N>];
    __shared__ float sLam[kTok], sDt[kTok];

    const int rows = blockDim.x / LPR;
    const int tiles = (pv.P + rows - 1) / rows;
    const int per = tiles * pv.H;
    const int b = blockIdx.x / per;
    const int unit = blockIdx.x - b * per;
    const int tile = unit % tiles;
    const int pos = unit / tiles;                  // region position of the head
    const int h = pv.perm[pos];
    const int tid = threadIdx.x;
    const Run run = ragged_run(pv, rc, b, unit == 0 && tid == 0);
    if (!run.ok || run.len >= rc.chunk_min) return;
    if (run.len == 0 && !run.fresh) return;

    const int j = tid % LPR;
    const int p = tile * rows + tid / LPR;
    const bool active = p < pv.P;
    const int g = h / pv.hpg;
    const float A = __ldg(rc.A + h), D = __ldg(rc.D + h);
    const RowPlace place = place_head<FMT>(pv, run.slot, rc.layer, pos);

    float s[E];
    if (run.fresh) {
#pragma unroll
        for (int n = 0; n < E; ++n) s[n] = 0.0f;
    } else {
        row_load<FMT, N>(place, p, j, active, s);
    }

    for (int c0 = 0; c0 < run.len; c0 += kTok) {
        const int nt = min(kTok, run.len - c0);
        const long long t0 = (long long)run.t0 + c0;
        if (c0) __syncthreads();
        for (int i = tid; i < nt * N; i += blockDim.x) {
            const int t = i / N, n = i % N;
            const int at = (n / E) * (E + 4) + n % E;
            sB[t][at] = load_act<TYPE>(rc.B, (t0 + t) * rc.Bs + (long long)g * N + n);
            sC[t][at] = load_act<TYPE>(rc.C, (t0 + t) * rc.Cs + (long long)g * N + n);
        }
        if (tid < nt) {
            const float dt = __ldg(rc.dt + (t0 + tid) * rc.dts + h);
            sDt[tid] = dt;
            sLam[tid] = decay(dt, A);
        }
        __syncthreads();
        for (int t = 0; t < nt; ++t) {
            const long long at = (long long)h * pv.P + p;
            const float x = active ? load_act<TYPE>(rc.x, (t0 + t) * rc.xs + at) : 0.0f;
            const float dtx = __fmul_rn(sDt[t], x);
            const float lam = sLam[t];
            const float4* Bp = reinterpret_cast<const float4*>(&sB[t][j * (E + 4)]);
            const float4* Cp = reinterpret_cast<const float4*>(&sC[t][j * (E + 4)]);
            const float2 l2 = make_float2(lam, lam), x2 = make_float2(dtx, dtx);
            float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int n = 0; n < E; n += 4) {
                const float4 Bv = Bp[n / 4], Cv = Cp[n / 4];
                float2 v = fma2(l2, make_float2(s[n], s[n + 1]), mul2(x2, make_float2(Bv.x, Bv.y)));
                s[n] = v.x; s[n + 1] = v.y;
                acc = fma2(make_float2(Cv.x, Cv.y), v, acc);
                v = fma2(l2, make_float2(s[n + 2], s[n + 3]), mul2(x2, make_float2(Bv.z, Bv.w)));
                s[n + 2] = v.x; s[n + 3] = v.y;
                acc = fma2(make_float2(Cv.z, Cv.w), v, acc);
            }
            const float y = grp_sum<LPR>(__fadd_rn(acc.x, acc.y));
            if (active && j == 0)
                store_act<TYPE>(rc.y, (t0 + t) * rc.ys + at, __fmaf_rn(D, x, y));
        }
    }
    row_store<FMT, N>(place, p, j, active, s, reinterpret_cast<uint32_t*>(pv.pool));
}

template <int FMT, int N>
cudaError_t launch_n(const PoolView& pv, const RaggedCall& rc, cudaStream_t st)
{
    constexpr int LPR = Shape<N>::LPR;
    // whole warps that cover the head's rows, at most kThreads
    int threads = (pv.P * LPR + 31) / 32 * 32;
    if (threads > kThreads) threads = kThreads;
    const int rows = threads / LPR;
    const long long blocks = (long long)((pv.P + rows - 1) / rows) * pv.H * rc.batch;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const unsigned grid = (unsigned)blocks;
    switch (rc.type) {
    case SSQ_T_BF16: tokens_kernel<FMT, N, SSQ_T_BF16><<<grid, threads, 0, st>>>(pv, rc); break;
    case SSQ_T_F16: tokens_kernel<FMT, N, SSQ_T_F16><<<grid, threads, 0, st>>>(pv, rc); break;
    default: tokens_kernel<FMT, N, SSQ_T_F32><<<grid, threads, 0, st>>>(pv, rc); break;
    }
    return cudaGetLastError();
}

template <int FMT>
cudaError_t launch_fmt(const PoolView& pv, const RaggedCall& rc, cudaStream_t st)
{
    switch (pv.N) {
    case 16: return launch_n<FMT, 16>(pv, rc, st);
    case 32: return launch_n<FMT, 32>(pv, rc, st);
    case 64: return launch_n<FMT, 64>(pv, rc, st);
    case 128: return launch_n<FMT, 128>(pv, rc, st);
    case 256: return launch_n<FMT, 256>(pv, rc, st);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_ragged_tokens(const PoolView& pv, const RaggedCall& rc, int fmt,
                                 cudaStream_t st)
{
    switch (fmt) {
    case SSQ_F32: return launch_fmt<SSQ_F32>(pv, rc, st);
    case SSQ_BF16: return launch_fmt<SSQ_BF16>(pv, rc, st);
    case SSQ_I8_SYM: return launch_fmt<SSQ_I8_SYM>(pv, rc, st);
    case SSQ_I8_ASYM: return launch_fmt<SSQ_I8_ASYM>(pv, rc, st);
    case SSQ_I4_SYM: return launch_fmt<SSQ_I4_SYM>(pv, rc, st);
    case SSQ_I4_ASYM: return launch_fmt<SSQ_I4_ASYM>(pv, rc, st);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace ssq
