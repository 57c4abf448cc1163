// ssq_rowio.cuh -- a state row between the pool and registers: E = min(32, N)
// consecutive entries per lane, LPR = N/E lanes per row, in the six storage
// formats, with the refit and rounding of ssq_common.cuh.
#pragma once

#include "ssq_common.cuh"
#include "ssq_params.h"

namespace ssq {

// Where a head's rows sit in a slot: pos is the head's region position.
struct RowPlace {
    uint8_t* codes;   // first code byte of the head's row 0 (integer formats)
    uint8_t* meta;
    uint8_t* fp;      // first byte of the head's row 0 (fp rows)
    bool quant;
};

template <int FMT>
__device__ __forceinline__ RowPlace place_head(const PoolView& pv, int slot, int layer, int pos)
{
    using F = Fmt<FMT>;
    RowPlace rp;
    uint8_t* base = pv.pool + pv.header_bytes + (long long)slot * pv.slot_bytes;
    rp.quant = F::quant && pos < pv.Hq;
    const long long row0 = (long long)(rp.quant ? pos : pos - pv.Hq) * pv.P;
    rp.codes = base + pv.codes_off + (long long)layer * pv.codes_layer_bytes
               + row0 * (pv.N * F::bits / 8);
    rp.meta = base + pv.meta_off + (long long)layer * pv.meta_layer_bytes + row0 * F::meta_bytes;
    rp.fp = base + pv.fp_off + (long long)layer * pv.fp_layer_bytes
            + row0 * pv.N * (FMT == SSQ_BF16 ? 2 : 4);
    return rp;
}

// A lane's part of a row as it is stored, RF the format of the row (fp rows of
// the integer formats are SSQ_F32): loaded at one point, decoded at another.
template <int RF, int N>
struct RawRow {
    using F = Fmt<RF>;
    static constexpr int E = Shape<N>::E;
    static constexpr int CB = E * F::bits / 8;
    Chunk<CB> c;
    float delta, z;

    // Lanes that are not `active` get a zero row and read nothing.
    __device__ __forceinline__ void load(const RowPlace& rp, int p, int j, bool active)
    {
#pragma unroll
        for (int i = 0; i < CB / 4; ++i) c.w[i] = 0;
        delta = 0.0f;
        z = 0.0f;
        if (!active) return;
        const uint8_t* rows = F::quant ? rp.codes : rp.fp;
        load_chunk<CB>(c, rows + (long long)p * (N * F::bits / 8) + j * CB);
        if constexpr (F::quant) {
            if constexpr (F::sym) {
                delta = __ldcs(reinterpret_cast<const float*>(rp.meta) + p);
            } else {
                const float2 m = __ldcs(reinterpret_cast<const float2*>(rp.meta) + p);
                delta = m.x;
                z = m.y;
            }
        }
    }
    // Every lane of the warp calls this.
    __device__ __forceinline__ void decode(float (&s)[E]) const
    {
        if constexpr (F::quant) {
            decode_row<RF, E>(c, delta, z, s);
        } else if constexpr (RF == SSQ_BF16) {
#pragma unroll
            for (int n = 0; n < E; ++n)
                s[n] = __uint_as_float((c.w[n / 2] >> (16 * (n % 2))) << 16);
        } else {
#pragma unroll
            for (int n = 0; n < E; ++n) s[n] = __uint_as_float(c.w[n]);
        }
    }
};

// Entries [j*E, j*E+E) of row p as fp32.  Every lane of the warp calls this
// with the same head.
template <int FMT, int N>
__device__ __forceinline__ void row_load(const RowPlace& rp, int p, int j, bool active,
                                         float (&s)[Shape<N>::E])
{
    if constexpr (Fmt<FMT>::quant) {
        if (!rp.quant) {
            RawRow<SSQ_F32, N> f;
            f.load(rp, p, j, active);
            f.decode(s);
            return;
        }
    }
    RawRow<FMT, N> r;
    r.load(rp, p, j, active);
    r.decode(s);
}

// Refit, round and store row p (fp rows: convert and store).  Every lane of
// the warp calls this; lanes that are not `active` store nothing.
template <int FMT, int N, bool ALL_QUANT = false>
__device__ __forceinline__ void row_store(const RowPlace& rp, int p, int j, bool active,
                                          const float (&s)[Shape<N>::E], uint32_t* err)
{
    using F = Fmt<FMT>;
    constexpr int E = Shape<N>::E, LPR = Shape<N>::LPR;
    if constexpr (F::quant) {
        if (ALL_QUANT || rp.quant) {
            constexpr int CB = E * F::bits / 8;
            RowParams q = refit_row<FMT, E, LPR>(s);
            // min and max pass over NaN entries; a sum of zeros does not
            float2 bad = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int n = 0; n < E; n += 2)
                bad = fma2(make_float2(s[n], s[n + 1]), make_float2(0.0f, 0.0f), bad);
            if (!(grp_sum<LPR>(__fadd_rn(bad.x, bad.y)) == 0.0f)) {
                // the row then decodes to NaN
                q.finite = false;
                q.delta = __int_as_float(0x7fffffff);
            }
            float r[E];
            uint32_t k[E];
            Chunk<CB> c;
            round_row<FMT, E>(q, s, r, k);
            pack_codes<FMT, E>(k, c);
            if (active) {
                store_chunk<CB>(rp.codes + (long long)p * (N * F::bits / 8) + j * CB, c);
                if (j == 0) {
                    if constexpr (F::sym)
                        reinterpret_cast<float*>(rp.meta)[p] = q.delta;
                    else
                        reinterpret_cast<float2*>(rp.meta)[p] = make_float2(q.delta, q.z);
                    if (!q.finite) atomicOr(err, SSQ_DEVERR_NONFINITE);
                }
            }
            return;
        }
    }
    if (!active) return;
    if constexpr (FMT == SSQ_BF16) {
        Chunk<E * 2> c;
#pragma unroll
        for (int n = 0; n < E; n += 2)
            c.w[n / 2] = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(s[n]))
                         | ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(s[n + 1])) << 16);
        store_chunk<E * 2>(rp.fp + ((long long)p * N + j * E) * 2, c);
    } else {
        Chunk<E * 4> c;
#pragma unroll
        for (int n = 0; n < E; ++n) c.w[n] = __float_as_uint(s[n]);
        store_chunk<E * 4>(rp.fp + ((long long)p * N + j * E) * 4, c);
    }
}

}  // namespace ssq
