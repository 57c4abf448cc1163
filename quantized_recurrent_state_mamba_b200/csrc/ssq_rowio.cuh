// ssq_rowio.cuh -- a state row between the pool and registers: E = min(32, N)
// entries per lane, LPR = N/E lanes per row, in the six storage formats, with
// the refit and rounding of ssq_common.cuh.
//
// The lanes of a row take its 16-byte pieces in turn, so that a load or store
// instruction of a warp covers whole lines (with E consecutive entries per
// lane an fp32 row's pieces lay 128 bytes apart, and 256 single tokens of 24
// fp32 heads took 139 us).
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

// Entries of a 16-byte piece in row format RF, and the row's entry that lane j
// holds at local index n.
template <int RF, int N>
constexpr int kPiece = 128 / Fmt<RF>::bits < Shape<N>::E ? 128 / Fmt<RF>::bits : Shape<N>::E;
template <int RF, int N>
__device__ __forceinline__ constexpr int row_entry(int n, int j)
{
    constexpr int PE = kPiece<RF, N>;
    return (n / PE * Shape<N>::LPR + j) * PE + n % PE;
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
        piece_io<true>(const_cast<uint8_t*>(rows) + (long long)p * (N * F::bits / 8), j);
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
    // The lane's pieces of the row that starts at `row`.
    template <bool LOAD>
    __device__ __forceinline__ void piece_io(uint8_t* row, int j)
    {
        constexpr int PB = kPiece<RF, N> * F::bits / 8;      // 16, or a whole part below that
#pragma unroll
        for (int i = 0; i < CB / PB; ++i) {
            Chunk<PB> q;
            uint8_t* at = row + (i * Shape<N>::LPR + j) * PB;
            if constexpr (LOAD) {
                load_chunk<PB>(q, at);
#pragma unroll
                for (int k = 0; k < PB / 4; ++k) c.w[i * (PB / 4) + k] = q.w[k];
            } else {
#pragma unroll
                for (int k = 0; k < PB / 4; ++k) q.w[k] = c.w[i * (PB / 4) + k];
                store_chunk<PB>(at, q);
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

// The lane's entries of row p as fp32.  Every lane of the warp calls this with
// the same head.
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

// Refit, round and store row p of format RF.  Every lane of the warp calls
// this; lanes that are not `active` store nothing.
template <int RF, int N>
__device__ __forceinline__ void raw_store(const RowPlace& rp, int p, int j, bool active,
                                          const float (&s)[Shape<N>::E], uint32_t* err)
{
    using F = Fmt<RF>;
    constexpr int E = Shape<N>::E, LPR = Shape<N>::LPR;
    RawRow<RF, N> raw;
    if constexpr (F::quant) {
        RowParams q = refit_row<RF, E, LPR>(s);
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
        round_row<RF, E>(q, s, r, k);
        pack_codes<RF, E>(k, raw.c);
        if (!active) return;
        raw.template piece_io<false>(rp.codes + (long long)p * (N * F::bits / 8), j);
        if (j == 0) {
            if constexpr (F::sym)
                reinterpret_cast<float*>(rp.meta)[p] = q.delta;
            else
                reinterpret_cast<float2*>(rp.meta)[p] = make_float2(q.delta, q.z);
            if (!q.finite) atomicOr(err, SSQ_DEVERR_NONFINITE);
        }
    } else {
        if (!active) return;
#pragma unroll
        for (int i = 0; i < raw.CB / 4; ++i) {
            if constexpr (RF == SSQ_BF16)
                raw.c.w[i] = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(s[2 * i]))
                             | ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(s[2 * i + 1])) << 16);
            else
                raw.c.w[i] = __float_as_uint(s[i]);
        }
        raw.template piece_io<false>(rp.fp + (long long)p * (N * F::bits / 8), j);
    }
}

// The same for a head of a pool of format FMT.
template <int FMT, int N>
__device__ __forceinline__ void row_store(const RowPlace& rp, int p, int j, bool active,
                                          const float (&s)[Shape<N>::E], uint32_t* err)
{
    if constexpr (Fmt<FMT>::quant) {
        if (!rp.quant) {
            raw_store<SSQ_F32, N>(rp, p, j, active, s, err);
            return;
        }
    }
    raw_store<FMT, N>(rp, p, j, active, s, err);
}

// The lane's entries to and from a row of fp32 in entry order.
template <int RF, int N, bool TO>
__device__ __forceinline__ void stage_io(float (&s)[Shape<N>::E], int j, float* row)
{
#pragma unroll
    for (int n = 0; n < Shape<N>::E; n += 4) {
        float4* at = reinterpret_cast<float4*>(row + row_entry<RF, N>(n, j));
        if constexpr (TO) {
            *at = make_float4(s[n], s[n + 1], s[n + 2], s[n + 3]);
        } else {
            const float4 v = *at;
            s[n] = v.x; s[n + 1] = v.y; s[n + 2] = v.z; s[n + 3] = v.w;
        }
    }
}
template <int FMT, int N>
__device__ __forceinline__ void row_to_stage(const RowPlace& rp, float (&s)[Shape<N>::E], int j,
                                             float* row)
{
    if constexpr (Fmt<FMT>::quant) {
        if (!rp.quant) {
            stage_io<SSQ_F32, N, true>(s, j, row);
            return;
        }
    }
    stage_io<FMT, N, true>(s, j, row);
}
template <int FMT, int N>
__device__ __forceinline__ void row_from_stage(const RowPlace& rp, float (&s)[Shape<N>::E], int j,
                                               const float* row)
{
    if constexpr (Fmt<FMT>::quant) {
        if (!rp.quant) {
            stage_io<SSQ_F32, N, false>(s, j, const_cast<float*>(row));
            return;
        }
    }
    stage_io<FMT, N, false>(s, j, const_cast<float*>(row));
}

}  // namespace ssq
