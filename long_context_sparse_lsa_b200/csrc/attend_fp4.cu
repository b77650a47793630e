// attend_fp4.cu — sparse GQA softmax attention over index sets, K and V held
// in 4 bits (fp4.cuh), split over the set entries.
//
// Same attention as lsa_attend ("LongCat-2.0 (molayo1419.me)", section "1M
// 토큰에서의 Sparse Attention 문제"; Cross-Layer Indexing: G layers share one
// set), on rows of 72 bytes instead of 256.
//
// Design (B200):
//  * grid = (splits x kv-head groups, query rows, layers). A CTA covers up to
//    4 kv heads over one run of set entries; a warp owns one kv head and
//    every (warps / heads)-th tile of 16 entries.
//  * A warp gathers its own tiles with 16-byte (codes) and 8-byte (scales)
//    asynchronous copies into a private ring of kRing tiles, so no warp
//    waits for another and 2304 * kRing * kWarps bytes are in flight per CTA.
//  * S^T = K Q^T on fp16 tensor cores (mma.m16n8k16): 16 tokens are M, the
//    group's query heads N. Lane (g, t) holds the 32 channels 32 t .. 32 t +
//    31 of tokens g and g + 8 (one 16-byte read per token) and the query
//    fragments are read in the same channel order. E2M1 codes become fp16
//    with the conversion instruction and are multiplied by their group's
//    scale in fp16: exact (fp4.cuh). A query row is scaled by a power of two
//    to magnitudes in [1, 2) at its largest, so that every finite bf16 query
//    enters fp16 with nothing above 2^-24 of its largest element lost; the
//    power goes back into the softmax scale.
//  * Online softmax in fp32 (exp2f). P is carried as 2^10 p and split into an
//    fp16 high part plus remainder (two MMAs, ~22 significant bits).
//  * O^T = V^T P^T: lane (g, t) holds the 16 channels 16 g .. 16 g + 15 (one
//    scale group) of tokens 2t, 2t+1, 2t+8, 2t+9; the codes of a token pair
//    are interleaved so that the conversion yields the (token, token + 1)
//    pairs of the A fragment, and the pair's scales multiply them. Each
//    tile's product is summed on its own and added to the rescaled running
//    output in fp32 arithmetic: the tensor core truncates its sums, and 400
//    truncations into one accumulator cost 2e-6 of the output at 64 rows of
//    3136 entries.
//  * The warps of a kv head merge through shared memory by log-sum-exp; one
//    partial per split, combined by attend_merge_kernel.
#include "fp4.cuh"
#include "internal.h"

namespace lsa {
namespace {

constexpr int kF4Warps = 16;
constexpr int kF4Threads = kF4Warps * kWarp;
constexpr int kF4Tile = 16;
constexpr int kRing = 5;
constexpr int kF4CodeTile = kF4Tile * kFp4CodeBytes;                       // 1024: K (or V) codes of a tile
constexpr int kF4ScaleTile = kF4Tile * kFp4Groups;                         // 128
constexpr int kF4TileBytes = 2 * (kF4CodeTile + kF4ScaleTile);             // 2304
constexpr int kF4RingBytes = kF4Warps * kRing * kF4TileBytes;              // 184,320
constexpr int kF4MaxEntries = 4096;                                        // set entries per split
constexpr float kPBits = 10.f;                                             // P is carried as 2^10 p
constexpr int kF4MergeFloats = (kFp4D / 16) * 4 + 4;                       // o fragments, m, l of one head tile

__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, uint32_t src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;\n" ::"r"(dst), "l"(src), "r"(src_bytes));
}

// Where MMA row m of a tile lies in the V tile: even rows 0..3, odd rows
// 4..7 (and 8 more), with the 16-byte chunks of every second pair of rows
// exchanged. A lane (g, t) then reads 8 bytes at chunk g / 2 of rows t or 4 +
// t, and the 16 lanes of a half warp touch all 32 banks once.
__device__ __forceinline__ int v_place(int m) { return (m & 8) + ((m & 1) << 2) + ((m & 7) >> 1); }
__device__ __forceinline__ int v_chunk(int place, int chunk) { return chunk ^ (place & 2); }

// NT: tiles of 8 query heads (H_q / H_kv up to 8 or 16).
template <int NT>
__global__ void __launch_bounds__(kF4Threads, 1) attend_fp4_kernel(const __grid_constant__ AttendFp4Args a) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = lane_id(), warp = warp_id();
    const int g = lane >> 2, t4 = lane & 3;
    const AttendArgs& b = a.base;
    const int split = blockIdx.x / b.head_groups;
    const int hgrp = blockIdx.x % b.head_groups;
    const int r = blockIdx.y, layer = blockIdx.z;
    const int ratio = b.H_q / b.H_kv, hpc = b.hpc;

    // the caller's row metadata may be read before the wait for the preceding kernel
    const int seq = b.q_seq[r];
    const int L = b.q_len[r];
    const int seq_c = min(max(seq, 0), b.n_seq - 1);
    const int64_t off = b.kv_offset[seq_c];
    const int slen = b.seq_lens[seq_c];
    const bool bad = seq < 0 || seq >= b.n_seq || L < 1 || L > b.max_len || L > slen || off < 0 ||
                     off + slen > b.total_tokens;
    pdl_enter();
    if (bad) {
        if (tid == 0 && blockIdx.x == 0 && layer == 0)
            flag(b.dev_status, seq < 0 || seq >= b.n_seq ? LSA_DEV_BAD_SEQ : LSA_DEV_BAD_LENGTH);
        if (split == 0) {
            float* o = b.out[layer] + ((int64_t)r * b.H_q + hgrp * hpc * ratio) * kFp4D;
            for (int i = tid; i < hpc * ratio * kFp4D; i += kF4Threads) o[i] = 0.f;
        }
        return;
    }

    // ---- the split's entries, checked; -1 where there is none ----------------
    int32_t* s_ent = reinterpret_cast<int32_t*>(smem + kF4RingBytes);
    const int e0 = split * b.entries_per_split;
    const int n_local = max(0, min(b.budget - e0, b.entries_per_split));
    const int n_tiles = (n_local + kF4Tile - 1) / kF4Tile;
    const int32_t* set = b.sets + (int64_t)r * b.budget + e0;
    bool bad_entry = false;
    for (int i = tid; i < n_tiles * kF4Tile; i += kF4Threads) {
        int e = i < n_local ? set[i] : -1;
        if (e < -1 || e >= L) {
            bad_entry = true;
            e = -1;
        }
        s_ent[i] = e;
    }
    if (bad_entry) flag(b.dev_status, LSA_DEV_BAD_INDEX);
    const int h_local = warp % hpc, wsel = warp / hpc, n_sel = kF4Warps / hpc;
    const int kvh = hgrp * hpc + h_local;

    // ---- query fragments: channel order of the K lanes --------------------------
    uint32_t qb[NT][8][2];
    float qscale[NT][2];  // softmax scale (log2 units) of the lane's two accumulator columns
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int hh = 8 * n + g;
        uint4 raw[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            raw[j] = hh < ratio ? ldg16(b.q[layer] + ((int64_t)r * b.H_q + (int64_t)kvh * ratio + hh) * kFp4D + 32 * t4 + 8 * j)
                                : make_uint4(0, 0, 0, 0);
        const uint32_t w[16] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w,
                                raw[2].x, raw[2].y, raw[2].z, raw[2].w, raw[3].x, raw[3].y, raw[3].z, raw[3].w};
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) top = __vmaxu2(top, w[j] & 0x7fff7fffu);
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // exponent of the row's largest magnitude (0 for a row that is zero or
        // subnormal). Every score of a row that is not finite is an infinity or
        // NaN, and so its softmax NaN: its scale is set to NaN below
        int e = (int)(top >> 7) - 127;
        if (e < -126 || e > 127) e = 0;
        const float down = e >= 0 ? __uint_as_float((uint32_t)(127 - min(e, 126)) << 23) : __uint_as_float((uint32_t)(127 - e) << 23);
        const float rest = e == 127 ? 0.5f : 1.f;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint32_t x = w[2 * ks + u];
                qb[n][ks][u] = pack_f16(__uint_as_float(x << 16) * down * rest, __uint_as_float(x & 0xffff0000u) * down * rest);
            }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int ec = __shfl_sync(0xffffffffu, e, 4 * (2 * t4 + c));
            const bool fin = __shfl_sync(0xffffffffu, top, 4 * (2 * t4 + c)) < 0x7f80u;
            qscale[n][c] = fin ? ldexpf(b.scale_log2 * b.kscale[layer], ec) : NAN;
        }
    }
    __syncthreads();

    // ---- gather: this warp's tiles, kRing in flight -------------------------------
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * kRing * kF4TileBytes);
    const int64_t head = off * b.H_kv + kvh;
    const uint8_t* kc = a.k[layer];
    const uint8_t* vc = a.v[layer];
    auto fetch = [&](int i, int slot) {
        if (i < n_tiles) {
            const uint32_t dst = ring + (uint32_t)(slot * kF4TileBytes);
            const int32_t* ent = s_ent + i * kF4Tile;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int m = g + 8 * u;
                const int e = ent[m];
                const uint32_t nb = e >= 0 ? 16u : 0u;
                const int64_t row = (head + (int64_t)max(e, 0) * b.H_kv) * kFp4CodeBytes + 16 * t4;
                cp_async16(dst + (uint32_t)(m * kFp4CodeBytes + 16 * t4), kc + row, nb);
                const int p = v_place(m);
                cp_async16(dst + kF4CodeTile + (uint32_t)(p * kFp4CodeBytes + 16 * v_chunk(p, t4)), vc + row, nb);
            }
            const int m = lane & 15;
            const int e = ent[m];
            const int64_t row = (head + (int64_t)max(e, 0) * b.H_kv) * kFp4Groups;
            cp_async8(dst + 2 * kF4CodeTile + (uint32_t)((lane >> 4) * kF4ScaleTile + m * kFp4Groups),
                      (lane < 16 ? a.k_group[layer] : a.v_group[layer]) + row, e >= 0 ? 8u : 0u);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int j = 0; j < kRing - 1; ++j) fetch(wsel + j * n_sel, j);

    float o[NT][8][4];
    float m_run[NT][2], l_run[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) o[n][mt][0] = o[n][mt][1] = o[n][mt][2] = o[n][mt][3] = 0.f;
        m_run[n][0] = m_run[n][1] = -INFINITY;
        l_run[n][0] = l_run[n][1] = 0.f;
    }
    int slot = 0;
    for (int i = wsel; i < n_tiles; i += n_sel) {
        fetch(i + (kRing - 1) * n_sel, slot == 0 ? kRing - 1 : slot - 1);
        cp_async_wait<kRing - 1>();
        __syncwarp();
        const int32_t* ent = s_ent + i * kF4Tile;
        const bool ok_g = ent[g] >= 0, ok_g8 = ent[g + 8] >= 0;
        const uint32_t at = ring + (uint32_t)(slot * kF4TileBytes);
        slot = slot + 1 == kRing ? 0 : slot + 1;
        if (!__any_sync(0xffffffffu, ok_g || ok_g8)) continue;
        // ---- S^T: 16 tokens x 8 NT heads -------------------------------------------
        float sacc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) sacc[n][0] = sacc[n][1] = sacc[n][2] = sacc[n][3] = 0.f;
        {
            const uint32_t sc = at + 2 * kF4CodeTile + (uint32_t)(g * kFp4Groups + 2 * t4);
            uint16_t s2a, s2b;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(s2a) : "r"(sc));
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(s2b) : "r"(sc + 8 * kFp4Groups));
            const uint32_t ha = e4m3x2_to_half2(s2a), hb = e4m3x2_to_half2(s2b);
            const uint4 ca = ld_shared_v4(at + (uint32_t)(g * kFp4CodeBytes + 16 * t4));
            const uint4 cb = ld_shared_v4(at + (uint32_t)((g + 8) * kFp4CodeBytes + 16 * t4));
            const uint32_t wa[4] = {ca.x, ca.y, ca.z, ca.w}, wb[4] = {cb.x, cb.y, cb.z, cb.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                // words 0, 1 are group 2 t, words 2, 3 group 2 t + 1
                const uint32_t da = __byte_perm(ha, 0, w < 2 ? 0x1010 : 0x3232);
                const uint32_t db = __byte_perm(hb, 0, w < 2 ? 0x1010 : 0x3232);
                uint32_t fa[4], fb[4];
                e2m1x8_to_f16(wa[w], fa);
                e2m1x8_to_f16(wb[w], fb);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t fr[4] = {mul_f16x2(fa[2 * u], da), mul_f16x2(fb[2 * u], db),
                                            mul_f16x2(fa[2 * u + 1], da), mul_f16x2(fb[2 * u + 1], db)};
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_f16(sacc[n], fr, qb[n][2 * w + u][0], qb[n][2 * w + u][1]);
                }
            }
        }
        // ---- online softmax ------------------------------------------------------------
        uint32_t phi[NT][2], plo[NT][2];
        float al[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float z0 = ok_g ? sacc[n][0] * qscale[n][0] : -INFINITY;
            const float z1 = ok_g ? sacc[n][1] * qscale[n][1] : -INFINITY;
            const float z2 = ok_g8 ? sacc[n][2] * qscale[n][0] : -INFINITY;
            const float z3 = ok_g8 ? sacc[n][3] * qscale[n][1] : -INFINITY;
            float mx0 = fmaxf(z0, z2), mx1 = fmaxf(z1, z3);
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) {
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, k));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, k));
            }
            const float mn0 = fmaxf(m_run[n][0], mx0), mn1 = fmaxf(m_run[n][1], mx1);
            const float base0 = (mn0 == -INFINITY ? 0.f : mn0) - kPBits;
            const float base1 = (mn1 == -INFINITY ? 0.f : mn1) - kPBits;
            al[n][0] = exp2f(m_run[n][0] - kPBits - base0);
            al[n][1] = exp2f(m_run[n][1] - kPBits - base1);
            const float p0 = exp2f(z0 - base0), p1 = exp2f(z1 - base1);
            const float p2 = exp2f(z2 - base0), p3 = exp2f(z3 - base1);
            m_run[n][0] = mn0;
            m_run[n][1] = mn1;
            l_run[n][0] = l_run[n][0] * al[n][0] + (p0 + p2);
            l_run[n][1] = l_run[n][1] * al[n][1] + (p1 + p3);
            const __half2 h01 = __floats2half2_rn(p0, p1), h23 = __floats2half2_rn(p2, p3);
            const float2 f01 = __half22float2(h01), f23 = __half22float2(h23);
            phi[n][0] = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&h01));
            phi[n][1] = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&h23));
            plo[n][0] = movmatrix_trans(pack_f16(p0 - f01.x, p1 - f01.y));
            plo[n][1] = movmatrix_trans(pack_f16(p2 - f23.x, p3 - f23.y));
        }
        // ---- O^T += V^T P^T -----------------------------------------------------------------
        {
            const uint32_t vt = at + kF4CodeTile;
            uint2 vx[4];  // tokens 2t, 2t+1, 2t+8, 2t+9: the 16 codes of group g
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int p = 8 * (j >> 1) + 4 * (j & 1) + t4;
                vx[j] = ld_shared_v2(vt + (uint32_t)(p * kFp4CodeBytes + 16 * v_chunk(p, g >> 1) + 8 * (g & 1)));
            }
            uint32_t sb[4];
            const uint32_t sc = at + 2 * kF4CodeTile + kF4ScaleTile + (uint32_t)(2 * t4 * kFp4Groups + g);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                asm volatile("ld.shared.u8 %0, [%1];" : "=r"(sb[j]) : "r"(sc + (uint32_t)(((j & 1) + 8 * (j >> 1)) * kFp4Groups)));
            const uint32_t s0 = e4m3x2_to_half2(sb[0] | (sb[1] << 8)), s8 = e4m3x2_to_half2(sb[2] | (sb[3] << 8));
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const uint32_t x0 = w ? vx[0].y : vx[0].x, x1 = w ? vx[1].y : vx[1].x;
                const uint32_t x8 = w ? vx[2].y : vx[2].x, x9 = w ? vx[3].y : vx[3].x;
                uint32_t ev[4], od[4], ev8[4], od8[4];  // even and odd channels, as token pairs
                e2m1x8_to_f16((x0 & 0x0f0f0f0fu) | ((x1 << 4) & 0xf0f0f0f0u), ev);
                e2m1x8_to_f16(((x0 >> 4) & 0x0f0f0f0fu) | (x1 & 0xf0f0f0f0u), od);
                e2m1x8_to_f16((x8 & 0x0f0f0f0fu) | ((x9 << 4) & 0xf0f0f0f0u), ev8);
                e2m1x8_to_f16(((x8 >> 4) & 0x0f0f0f0fu) | (x9 & 0xf0f0f0f0u), od8);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint32_t fr[4] = {mul_f16x2(ev[u], s0), mul_f16x2(od[u], s0), mul_f16x2(ev8[u], s8),
                                            mul_f16x2(od8[u], s8)};
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float (&oo)[4] = o[n][4 * w + u];
                        float x[4] = {0.f, 0.f, 0.f, 0.f};
                        mma_f16(x, fr, plo[n][0], plo[n][1]);
                        mma_f16(x, fr, phi[n][0], phi[n][1]);
#pragma unroll
                        for (int c = 0; c < 4; ++c) oo[c] = oo[c] * al[n][c & 1] + x[c];
                    }
                }
            }
        }
        __syncwarp();  // the slot may be filled again
    }
    cp_async_wait<0>();
    pdl_trigger();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) l_run[n][c] += __shfl_xor_sync(0xffffffffu, l_run[n][c], k);
    __syncthreads();  // the merge area reuses the rings

    // ---- merge the warps of each kv head: partners park, the first folds -----------
    float* park = reinterpret_cast<float*>(smem);  // [warp][NT][kF4MergeFloats][32]
    if (wsel > 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float* p = park + (size_t)((warp * NT + n) * kF4MergeFloats) * kWarp + lane;
#pragma unroll
            for (int mt = 0; mt < 8; ++mt)
#pragma unroll
                for (int c = 0; c < 4; ++c) p[(4 * mt + c) * kWarp] = o[n][mt][c];
            p[32 * kWarp] = m_run[n][0];
            p[33 * kWarp] = m_run[n][1];
            p[34 * kWarp] = l_run[n][0];
            p[35 * kWarp] = l_run[n][1];
        }
    }
    __syncthreads();
    if (wsel > 0) return;
    const bool direct = b.n_splits == 1;
    const int64_t row_q = (int64_t)layer * b.n_q + r;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        for (int j = 1; j < n_sel; ++j) {
            const float* p = park + (size_t)(((warp + hpc * j) * NT + n) * kF4MergeFloats) * kWarp + lane;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float mb = p[(32 + c) * kWarp], lb = p[(34 + c) * kWarp];
                const float M = fmaxf(m_run[n][c], mb);
                const float sa = M == -INFINITY ? 0.f : exp2f(m_run[n][c] - M);
                const float sb = M == -INFINITY ? 0.f : exp2f(mb - M);
                m_run[n][c] = M;
                l_run[n][c] = l_run[n][c] * sa + lb * sb;
#pragma unroll
                for (int mt = 0; mt < 8; ++mt) {
                    o[n][mt][c] = o[n][mt][c] * sa + p[(4 * mt + c) * kWarp] * sb;
                    o[n][mt][c + 2] = o[n][mt][c + 2] * sa + p[(4 * mt + c + 2) * kWarp] * sb;
                }
            }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int hh = 8 * n + 2 * t4 + c;
            if (hh >= ratio) continue;
            const int64_t qh = (int64_t)kvh * ratio + hh;
            float* dst = direct ? b.out[layer] + ((int64_t)r * b.H_q + qh) * kFp4D
                                : b.part_o + ((row_q * b.n_splits + split) * b.H_q + qh) * kFp4D;
            // a denominator that is not positive: no entry (0) or NaN scores (NaN stays)
            const float inv = l_run[n][c] == 0.f ? 0.f : 1.f / l_run[n][c];
            const float sc = direct ? inv * b.vscale[layer] : b.vscale[layer];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<float4*>(dst + kFp4Group * g + 4 * q) =
                    make_float4(o[n][2 * q][c] * sc, o[n][2 * q][c + 2] * sc, o[n][2 * q + 1][c] * sc, o[n][2 * q + 1][c + 2] * sc);
            // (a maximum of -infinity marks an empty partial: one of NaN scores alone is not)
            if (!direct && g == 0)
                *reinterpret_cast<float2*>(b.part_ml + ((row_q * b.n_splits + split) * b.H_q + qh) * 2) =
                    make_float2(l_run[n][c] == 0.f ? m_run[n][c] : fmaxf(m_run[n][c], -3e38f), l_run[n][c]);
        }
    }
}

}  // namespace

AttendPlan plan_attend_fp4(int n_q, int H_q, int H_kv, int budget, int G, int num_sms) {
    AttendPlan p;
    p.hpc = H_kv < 4 ? H_kv : 4;
    p.head_groups = H_kv / p.hpc;
    const long units = (long)n_q * p.head_groups * G;
    const int tiles = (budget + kF4Tile - 1) / kF4Tile;
    const int n_sel = kF4Warps / p.hpc;
    int splits = units > 0 ? (int)(num_sms / units) : 1;  // one CTA per SM, one wave
    // at least two tiles a warp: below that the merge of the splits costs more than it saves
    const int max_splits = (tiles + 2 * n_sel - 1) / (2 * n_sel);
    if (splits > max_splits) splits = max_splits;
    const int min_splits = (budget + kF4MaxEntries - 1) / kF4MaxEntries;
    if (splits < min_splits) splits = min_splits;
    if (splits < 1) splits = 1;
    int per = (tiles + splits - 1) / splits;
    if (per < 1) per = 1;
    p.entries_per_split = per * kF4Tile;
    p.n_splits = tiles > 0 ? (tiles + per - 1) / per : 1;
    p.smem_bytes = (size_t)kF4RingBytes + (size_t)p.entries_per_split * 4;
    const size_t rows_q = (size_t)G * n_q;
    p.ws_bytes = 0;
    if (p.n_splits > 1) {
        p.ws_bytes = (rows_q * p.n_splits * H_q * kFp4D * 4 + 255) / 256 * 256;
        p.ws_bytes += (rows_q * p.n_splits * H_q * 2 * 4 + 255) / 256 * 256;
    }
    return p;
}

cudaError_t launch_attend_fp4(const AttendFp4Args& a, size_t smem_bytes, cudaStream_t stream) {
    const AttendArgs& b = a.base;
    static std::atomic<uint64_t> allowed[2];
    const int wide = b.H_q / b.H_kv > 8;
    auto kern = wide ? attend_fp4_kernel<2> : attend_fp4_kernel<1>;
    cudaError_t e = allow_smem(kern, kF4RingBytes + 4 * kF4MaxEntries, allowed[wide]);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(b.n_splits * b.head_groups), (unsigned)b.n_q, (unsigned)b.G);
    e = launch_pdl(kern, grid, dim3(kF4Threads), smem_bytes, stream, 0, a);
    if (e != cudaSuccess || b.n_splits == 1) return e;
    return launch_attend_merge(b, stream);
}

}  // namespace lsa
