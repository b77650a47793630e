// attend_fp4.cu — sparse GQA softmax attention over index sets, K and V held
// in 4 bits (fp4.cuh), split over the set entries.
//
// Same attention as lsa_attend ("LongCat-2.0 (molayo1419.me)", section "1M
// 토큰에서의 Sparse Attention 문제"; Cross-Layer Indexing: G layers share one
// set), on rows of 72 bytes instead of 256.
//
// Design (B200):
//  * grid = (splits x kv-head groups, query rows, layers). A CTA covers up to
//    4 kv heads over one run of set entries; a team of one warp per kv head
//    works on every n-th step of 32 entries.
//  * A team gathers its steps itself with 16-byte asynchronous copies into a
//    ring, whole tokens at a time (the heads' codes of a token are 256
//    consecutive bytes, their scales 32): 64 rows of 3136 random tokens take
//    46 us this way from HBM, 90 us when each warp fetches its own head's
//    64 + 8 bytes, and 60 us as one bulk copy per token.
//  * 16 warps, or 8 for 9 to 16 query heads per kv head: their fragments need
//    255 registers a thread (16 warps of 128, spilling 500 bytes: 64 rows of
//    64/4 heads, two layers 134 us; 8 warps 104).
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
//    step's product is summed on its own and added to the rescaled running
//    output in fp32 arithmetic: the tensor core truncates its sums, and 400
//    truncations into one accumulator cost 2e-6 of the output at 64 rows of
//    3136 entries.
//  * The warps of a kv head merge through shared memory by log-sum-exp; one
//    partial per split, combined by attend_merge_kernel.
//  * What bounds it: where every SM has a CTA with many steps, the instructions
//    (a step of a head is about 650; 61% of the issue slots, the integer pipe
//    with the conversions 51%): 64 rows of 3136 entries, two layers: 68 us, 235
//    MB at 3.5 TB/s, on 128 of 148 SMs. With few rows the chain of row lookup,
//    set, gather, products and merge: 11 us for one row of four layers.
#include "fp4.cuh"
#include "internal.h"

namespace lsa {
namespace {

// Warps of a CTA and steps in a team's ring, for NT tiles of 8 query heads:
// the fragments of 16 query heads need the registers of half as many warps.
__host__ __device__ constexpr int f4_warps(int nt) { return nt == 1 ? 16 : 8; }
__host__ __device__ constexpr int f4_ring(int nt) { return nt == 1 ? 3 : 6; }
constexpr int kF4Pair = 32;                                                // entries of a step: two MMA tiles
constexpr int kF4HeadStep = kF4Pair * 2 * (kFp4CodeBytes + kFp4Groups);    // 4608: a step of one kv head
constexpr int kF4RingBytes = f4_warps(1) * f4_ring(1) * kF4HeadStep;       // 221,184, for either NT
constexpr float kPBits = 10.f;                                             // P is carried as 2^10 p
constexpr int kF4Park = 36;                                                // floats of a lane: o fragments, m, l
static_assert(kF4RingBytes == f4_warps(2) * f4_ring(2) * kF4HeadStep && kF4RingBytes <= 227 * 1024, "shared memory of one CTA");
static_assert(f4_warps(1) * kF4Park * kWarp * 4 <= kF4RingBytes && f4_warps(2) * 2 * kF4Park * kWarp * 4 <= kF4RingBytes,
              "the merge area reuses the rings");

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, uint32_t src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;\n" ::"r"(dst), "l"(src), "r"(src_bytes));
}

__device__ __forceinline__ void cp_async_full16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src));
}

// A step in shared memory, HPC heads: K codes [32][HPC * 64 bytes], V codes
// alike, K scales [32][HPC * 8], V scales alike. The lanes of a quarter warp
// read 64 bytes of two K rows m, m + 1: the 64-byte blocks of the heads are
// exchanged pairwise in every second row, so that they fall on different
// banks. Of V a lane (g, t) reads 8 bytes at 16-byte chunk g / 2 of rows 2t
// or 2t + 1: the rows of a tile are stored even ones first, and the chunks of
// every second pair of rows exchanged as well, so that the 16 lanes of a half
// warp touch all 32 banks once.
template <int HPC>
__device__ __forceinline__ int k_at(int m, int h, int c) {
    return m * (HPC * kFp4CodeBytes) + 64 * (HPC > 1 ? h ^ (m & 1) : h) + 16 * c;
}
template <int HPC>
__device__ __forceinline__ int v_at(int m, int h, int c) {
    const int p = (m & 24) + ((m & 1) << 2) + ((m & 7) >> 1);
    return p * (HPC * kFp4CodeBytes) + 64 * (HPC > 1 ? h ^ (p & 1) : h) + 16 * (c ^ (p & 2));
}

// NT: tiles of 8 query heads (H_q / H_kv up to 8 or 16). HPC: kv heads per CTA.
template <int NT, int HPC>
__global__ void __launch_bounds__(f4_warps(NT) * kWarp, 1) attend_fp4_kernel(const __grid_constant__ AttendFp4Args a) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int kWarps = f4_warps(NT), kRing = f4_ring(NT);
    const int tid = threadIdx.x, lane = lane_id(), warp = warp_id();
    const int g = lane >> 2, t4 = lane & 3;
    const AttendArgs& b = a.base;
    const int split = blockIdx.x / b.head_groups;
    const int hgrp = blockIdx.x % b.head_groups;
    const int r = blockIdx.y, layer = blockIdx.z;
    const int ratio = b.H_q / b.H_kv;

    // the caller's row metadata may be read before the wait for the preceding kernel
    const int seq = b.q_seq[r];
    const int L = b.q_len[r];
    const int seq_c = min(max(seq, 0), b.n_seq - 1);
    const int64_t off = b.kv_offset[seq_c];
    const int slen = b.seq_lens[seq_c];
    const bool bad = seq < 0 || seq >= b.n_seq || L < 1 || L > b.max_len || L > slen || off < 0 ||
                     off > b.total_tokens - slen;
    pdl_enter();

    // a team of HPC warps, one per kv head, works on every n_sel-th step of 32 entries;
    // a lane holds one entry of a step (-1: none). The first entries are asked for
    // before the row's lookup above is waited for.
    constexpr int n_sel = kWarps / HPC;
    const int h_local = warp % HPC, wsel = warp / HPC;
    const int e0 = split * b.entries_per_split;
    const int n_local = max(0, min(b.budget - e0, b.entries_per_split));
    const int n_steps = (n_local + kF4Pair - 1) / kF4Pair;
    const int32_t* set = b.sets + (int64_t)r * b.budget + e0;
    // (loaded here, checked where it is used: the check waits for the load)
    auto entry = [&](int i) -> int {
        const int at = i * kF4Pair + lane;
        return i < n_steps && at < n_local ? __ldg(set + at) : -1;
    };
    int ent[kRing];  // entries of the steps in flight; the last is not asked for (and not checked) yet
#pragma unroll
    for (int j = 0; j < kRing; ++j) ent[j] = entry(wsel + j * n_sel);
    if (bad) {
        if (tid == 0 && blockIdx.x == 0 && layer == 0)
            flag(b.dev_status, seq < 0 || seq >= b.n_seq ? LSA_DEV_BAD_SEQ : LSA_DEV_BAD_LENGTH);
        if (split == 0) {
            float* o = b.out[layer] + ((int64_t)r * b.H_q + hgrp * HPC * ratio) * kFp4D;
            for (int i = tid; i < HPC * ratio * kFp4D; i += kWarps * kWarp) o[i] = 0.f;
        }
        return;
    }

    const int kvh = hgrp * HPC + h_local;
    auto team_sync = [&]() {
        if (HPC == 1) __syncwarp();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + wsel), "n"(HPC * kWarp) : "memory");
    };

    // ---- gather: a team's steps, kRing - 1 in flight, each warp 32 / HPC whole tokens --
    auto checked = [&](int e) -> int {
        if (e >= -1 && e < L) return e;
        flag(b.dev_status, LSA_DEV_BAD_INDEX);
        return -1;
    };
    constexpr int kTokens = kF4Pair / HPC, kChunks = 4 * HPC;  // tokens of a warp, 16-byte chunks of a token's codes
    constexpr int kVCodes = HPC * kF4Pair * kFp4CodeBytes, kKScales = 2 * kVCodes, kVScales = kKScales + HPC * kF4Pair * 8;
    const uint32_t ring = smem_u32(smem) + (uint32_t)(wsel * kRing * HPC * kF4HeadStep);
    const uint32_t k_row = (uint32_t)(b.H_kv * kFp4CodeBytes), s_row = (uint32_t)(b.H_kv * kFp4Groups);  // bytes per token
    const int64_t head0 = off * b.H_kv + hgrp * HPC;
    const uint8_t* kc = a.k[layer] + head0 * kFp4CodeBytes + 16 * (lane % kChunks);
    const uint8_t* vc = a.v[layer] + head0 * kFp4CodeBytes + 16 * (lane % kChunks);
    // scales: HPC 4: lanes 2 i, 2 i + 1 the halves of a row; K of the warp's tokens, then V. HPC 1: a row is 8 bytes
    constexpr int kSBytes = HPC == 1 ? 8 : 16, kSChunks = HPC * 8 / kSBytes;
    const int s_tok = lane / kSChunks % kTokens;
    // (lanes 16..31 of a wider CTA take the V scales)
    const uint8_t* sc0 = (HPC > 1 && lane >= 16 ? a.v_group[layer] : a.k_group[layer]) + head0 * kFp4Groups + kSBytes * (lane % kSChunks);
    const uint8_t* sc1 = a.v_group[layer] + head0 * kFp4Groups;  // HPC 1
    // lane-constant shared-memory offsets; row m = h_local * kTokens + (32 x + lane) / kChunks for x = 0..3
    const int ch = lane % kChunks >> 2;
    uint32_t k_off[HPC == 1 ? 1 : 4], v_off[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int m = h_local * kTokens + (32 * x + lane) / kChunks;
        if (HPC > 1 || x == 0) k_off[x] = (uint32_t)k_at<HPC>(m, ch, lane & 3);
        v_off[x] = (uint32_t)(kVCodes + v_at<HPC>(m, ch, lane & 3));
    }
    const int sm = h_local * kTokens + s_tok;
    const uint32_t s_off = (uint32_t)((HPC > 1 && lane >= 16 ? kVScales : kKScales) + sm * HPC * 8 + kSBytes * (lane % kSChunks));
    auto fetch = [&](int entries, uint32_t slot) {
        const uint32_t to = ring + slot;
        const uint32_t there = __ballot_sync(0xffffffffu, entries >= 0);
        const uint32_t clamped = (uint32_t)max(entries, 0);
        if (there == 0xffffffffu) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint32_t e = __shfl_sync(0xffffffffu, clamped, h_local * kTokens + (32 * x + lane) / kChunks);
                cp_async_full16(to + k_off[HPC == 1 ? 0 : x] + (HPC == 1 ? (uint32_t)(8 * x * kFp4CodeBytes) : 0u), kc + (uint64_t)e * k_row);
                cp_async_full16(to + v_off[x], vc + (uint64_t)e * k_row);
            }
            const uint32_t e = __shfl_sync(0xffffffffu, clamped, sm);
            if (HPC == 1) {
                cp_async8(to + s_off, sc0 + (uint64_t)e * s_row, 8);
                cp_async8(to + s_off + (kVScales - kKScales), sc1 + (uint64_t)e * s_row, 8);
            } else {
                cp_async_full16(to + s_off, sc0 + (uint64_t)e * s_row);
            }
        } else if (there != 0u) {  // a missing entry's bytes are zeros (a step without entries is not looked at)
#pragma unroll 1
            for (int x = 0; x < 4; ++x) {
                const int m = h_local * kTokens + (32 * x + lane) / kChunks;
                const uint32_t e = __shfl_sync(0xffffffffu, clamped, m);
                const uint32_t nb = __shfl_sync(0xffffffffu, entries, m) >= 0 ? 16u : 0u;
                cp_async16(to + (uint32_t)k_at<HPC>(m, ch, lane & 3), kc + (uint64_t)e * k_row, nb);
                cp_async16(to + (uint32_t)(kVCodes + v_at<HPC>(m, ch, lane & 3)), vc + (uint64_t)e * k_row, nb);
            }
            const uint32_t e = __shfl_sync(0xffffffffu, clamped, sm);
            const bool in = __shfl_sync(0xffffffffu, entries, sm) >= 0;
            if (HPC == 1) {
                cp_async8(to + s_off, sc0 + (uint64_t)e * s_row, in ? 8u : 0u);
                cp_async8(to + s_off + (kVScales - kKScales), sc1 + (uint64_t)e * s_row, in ? 8u : 0u);
            } else {
                cp_async16(to + s_off, sc0 + (uint64_t)e * s_row, in ? 16u : 0u);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int j = 0; j < kRing - 1; ++j) {
        ent[j] = checked(ent[j]);
        fetch(ent[j], (uint32_t)(j * HPC * kF4HeadStep));
    }

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
        // exponent of the row's largest magnitude (-126 for a row that is zero or
        // subnormal: its numbers are multiples of 2^-133, and so whole in fp16).
        // Every score of a row that is not finite is an infinity or NaN, and so
        // its softmax NaN: its scale is set to NaN below
        int e = max((int)(top >> 7) - 127, -126);
        if (e > 127) e = 0;
        const float down = e >= 0 ? __uint_as_float((uint32_t)(127 - min(e, 126)) << 23) : __uint_as_float((uint32_t)(127 - e) << 23);
        // (the sign of the layer's scale goes with it, so that the softmax scale is not negative)
        const float rest = copysignf(e == 127 ? 0.5f : 1.f, b.kscale[layer]);
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
            qscale[n][c] = fin ? ldexpf(b.scale_log2 * fabsf(b.kscale[layer]), ec) : NAN;
        }
    }
    float o[NT][8][4];
    float m_run[NT][2], l_run[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) o[n][mt][0] = o[n][mt][1] = o[n][mt][2] = o[n][mt][3] = 0.f;
        m_run[n][0] = m_run[n][1] = -INFINITY;
        l_run[n][0] = l_run[n][1] = 0.f;
    }
    uint32_t slot = 0;
    constexpr uint32_t kSlot = HPC * kF4HeadStep;
    for (int i = wsel; i < n_steps; i += n_sel) {
        cp_async_wait<kRing - 2>();
        team_sync();  // the team's copies of this step have landed, and all its warps have left the step before
        ent[kRing - 1] = checked(ent[kRing - 1]);
        fetch(ent[kRing - 1], slot == 0 ? (kRing - 1) * kSlot : slot - kSlot);
        const uint32_t valid = __ballot_sync(0xffffffffu, ent[0] >= 0);
#pragma unroll
        for (int j = 0; j < kRing - 1; ++j) ent[j] = ent[j + 1];
        ent[kRing - 1] = entry(i + kRing * n_sel);
        const uint32_t step = ring + slot;
        slot = slot == (kRing - 1) * kSlot ? 0 : slot + kSlot;
        if (valid == 0u) continue;
        // ---- S^T: 2 x 16 tokens x 8 NT heads ------------------------------------------
        float sacc[NT][2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint32_t sc = step + kKScales + (uint32_t)((16 * u + g) * HPC * 8 + 8 * h_local + 2 * t4);
            uint16_t s2a, s2b;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(s2a) : "r"(sc));
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(s2b) : "r"(sc + 8 * HPC * 8));
            const __half2 ha = e4m3x2_to_half2(s2a), hb = e4m3x2_to_half2(s2b);
            const uint4 ca = ld_shared_v4(step + (uint32_t)k_at<HPC>(16 * u + g, h_local, t4));
            const uint4 cb = ld_shared_v4(step + (uint32_t)k_at<HPC>(16 * u + g + 8, h_local, t4));
            const uint32_t wa[4] = {ca.x, ca.y, ca.z, ca.w}, wb[4] = {cb.x, cb.y, cb.z, cb.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                // words 0, 1 are group 2 t, words 2, 3 group 2 t + 1
                const __half2 da = w < 2 ? __low2half2(ha) : __high2half2(ha);
                const __half2 db = w < 2 ? __low2half2(hb) : __high2half2(hb);
                uint32_t fa[4], fb[4];
                e2m1x8_to_f16(wa[w], fa);
                e2m1x8_to_f16(wb[w], fb);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t fr[4] = {mul_f16x2(fa[2 * x], da), mul_f16x2(fb[2 * x], db),
                                            mul_f16x2(fa[2 * x + 1], da), mul_f16x2(fb[2 * x + 1], db)};
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if (w + x == 0) mma_f16_zero(sacc[n][u], fr, qb[n][0][0], qb[n][0][1]);
                        else mma_f16(sacc[n][u], fr, qb[n][2 * w + x][0], qb[n][2 * w + x][1]);
                    }
                }
            }
        }
        // ---- online softmax ------------------------------------------------------------
        uint32_t phi[NT][2][2], plo[NT][2][2];
        float al[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float mx[2], base[2];
            const bool whole = valid == 0xffffffffu;
            if (!whole) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int c = 0; c < 4; ++c)  // token g (c < 2) or g + 8 of tile u, head 2 t + (c & 1)
                        if (!((valid >> (16 * u + 8 * (c >> 1) + g)) & 1u)) sacc[n][u][c] = -INFINITY;
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                mx[c] = fmaxf(fmaxf(sacc[n][0][c], sacc[n][0][c + 2]), fmaxf(sacc[n][1][c], sacc[n][1][c + 2]));
#pragma unroll
                for (int k = 4; k < 32; k <<= 1) mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], k));
                mx[c] = fmaxf(m_run[n][c], mx[c] * qscale[n][c]);  // (qscale >= 0, or NaN)
                base[c] = mx[c] == -INFINITY ? 0.f : mx[c];
                al[n][c] = ex2(m_run[n][c] - base[c]);
                m_run[n][c] = mx[c];
                base[c] -= kPBits;
            }
            float sum[2] = {0.f, 0.f};
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float p[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    p[c] = ex2(fmaf(sacc[n][u][c], qscale[n][c & 1], -base[c & 1]));
                    if (!whole && sacc[n][u][c] == -INFINITY) p[c] = 0.f;  // (a scale of 0 leaves NaN)
                    sum[c & 1] += p[c];
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const __half2 h = __floats2half2_rn(p[2 * x], p[2 * x + 1]);
                    const float2 f = __half22float2(h);
                    phi[n][u][x] = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&h));
                    plo[n][u][x] = movmatrix_trans(pack_f16(p[2 * x] - f.x, p[2 * x + 1] - f.y));
                }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) l_run[n][c] = l_run[n][c] * al[n][c] + sum[c];
        }
        // ---- O^T = O^T al + V^T P^T -----------------------------------------------------
        uint2 vx[2][4];  // per tile: tokens 2t, 2t+1, 2t+8, 2t+9, the 16 codes of group g
        __half2 vs[2][2];  // the scales of tokens 2t, 2t+1 and 2t+8, 2t+9
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                vx[u][j] = ld_shared_v2(step + kVCodes + (uint32_t)(v_at<HPC>(16 * u + 2 * t4 + (j & 1) + 8 * (j >> 1), h_local, g >> 1) + 8 * (g & 1)));
            uint32_t sb[4];
            const uint32_t sc = step + kVScales + (uint32_t)((16 * u + 2 * t4) * HPC * 8 + 8 * h_local + g);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                asm volatile("ld.shared.u8 %0, [%1];" : "=r"(sb[j]) : "r"(sc + (uint32_t)(((j & 1) + 8 * (j >> 1)) * HPC * 8)));
            vs[u][0] = e4m3x2_to_half2((uint16_t)(sb[0] | (sb[1] << 8)));
            vs[u][1] = e4m3x2_to_half2((uint16_t)(sb[2] | (sb[3] << 8)));
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            uint32_t ev[2][2][4], od[2][2][4];  // [tile][tokens 2t.. or 2t+8..]: even and odd channels, as token pairs
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t c0 = w ? vx[u][2 * x].y : vx[u][2 * x].x, c1 = w ? vx[u][2 * x + 1].y : vx[u][2 * x + 1].x;
                    e2m1x8_to_f16((c0 & 0x0f0f0f0fu) | ((c1 << 4) & 0xf0f0f0f0u), ev[u][x]);
                    e2m1x8_to_f16(((c0 >> 4) & 0x0f0f0f0fu) | (c1 & 0xf0f0f0f0u), od[u][x]);
                }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                float acc[NT][4];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t fr[4] = {mul_f16x2(ev[u][0][y], vs[u][0]), mul_f16x2(od[u][0][y], vs[u][0]),
                                            mul_f16x2(ev[u][1][y], vs[u][1]), mul_f16x2(od[u][1][y], vs[u][1])};
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if (u == 0) mma_f16_zero(acc[n], fr, plo[n][u][0], plo[n][u][1]);
                        else mma_f16(acc[n], fr, plo[n][u][0], plo[n][u][1]);
                        mma_f16(acc[n], fr, phi[n][u][0], phi[n][u][1]);
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[n][4 * w + y][c] = o[n][4 * w + y][c] * al[n][c & 1] + acc[n][c];
            }
        }
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

    // ---- merge the warps of each kv head: every warp parks its fragments and
    // combines its share of the channels over the warps of the head -----------------
    float* park = reinterpret_cast<float*>(smem);  // [warp][NT][kF4Park][32]
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float* p = park + ((warp * NT + n) * kF4Park) * kWarp + lane;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt)
#pragma unroll
            for (int c = 0; c < 4; ++c) p[(4 * mt + c) * kWarp] = o[n][mt][c];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            p[(32 + c) * kWarp] = m_run[n][c];
            p[(34 + c) * kWarp] = l_run[n][c];
        }
    }
    __syncthreads();
    const bool direct = b.n_splits == 1;
    const int64_t row_q = (int64_t)layer * b.n_q + r;
    // the warp's share: fragment tiles [m_lo, m_lo + 8 / n_sel) of both head
    // columns; with 16 warps a head, one tile of one column
    constexpr int cols = n_sel == 16 ? 1 : 2, n_mt = n_sel == 16 ? 1 : 8 / n_sel;
    const int m_lo = n_sel == 16 ? wsel >> 1 : wsel * n_mt;
#pragma unroll
    for (int n = 0; n < NT; ++n)
        for (int cc = 0; cc < cols; ++cc) {
            const int c = n_sel == 16 ? wsel & 1 : cc;
            const float* p0 = park + ((h_local * NT + n) * kF4Park) * kWarp + lane;
            const int next = HPC * NT * kF4Park * kWarp;  // to the head's next warp
            float M = -INFINITY;
            for (int j = 0; j < n_sel; ++j) M = fmaxf(M, p0[j * next + (32 + c) * kWarp]);
            float l = 0.f, x[2 * n_mt] = {};
            const float base = M == -INFINITY ? 0.f : M;
            for (int j = 0; j < n_sel; ++j) {
                const float* p = p0 + j * next;
                const float f = ex2(p[(32 + c) * kWarp] - base);
                l += p[(34 + c) * kWarp] * f;
#pragma unroll
                for (int k = 0; k < 2 * n_mt; ++k) x[k] += p[(4 * m_lo + 2 * k + c) * kWarp] * f;
            }
            const int hh = 8 * n + 2 * t4 + c;
            if (hh >= ratio) continue;
            const int64_t qh = (int64_t)kvh * ratio + hh;
            float* dst = direct ? b.out[layer] + ((int64_t)r * b.H_q + qh) * kFp4D
                                : b.part_o + ((row_q * b.n_splits + split) * b.H_q + qh) * kFp4D;
            // a denominator of 0: no entry (NaN scores give NaN)
            const float to = b.vscale[layer] * (!direct ? 1.f : l == 0.f ? 0.f : 1.f / l);
            dst += kFp4Group * g + 2 * m_lo;
#pragma unroll
            for (int k = 0; k < 2 * n_mt; k += n_mt == 1 ? 2 : 4) {
                if (n_mt == 1) *reinterpret_cast<float2*>(dst + k) = make_float2(x[k] * to, x[k + 1] * to);
                else *reinterpret_cast<float4*>(dst + k) = make_float4(x[k] * to, x[k + 1] * to, x[(k + 2) % (2 * n_mt)] * to, x[(k + 3) % (2 * n_mt)] * to);
            }
            // (a maximum of -infinity marks an empty partial: one of NaN scores alone is not)
            if (!direct && g == 0 && m_lo == 0)
                *reinterpret_cast<float2*>(b.part_ml + ((row_q * b.n_splits + split) * b.H_q + qh) * 2) =
                    make_float2(l == 0.f ? M : fmaxf(M, -3e38f), l);
        }
}

}  // namespace

AttendPlan plan_attend_fp4(int n_q, int H_q, int H_kv, int budget, int G, int num_sms) {
    AttendPlan p;
    p.hpc = H_kv < 4 ? H_kv : 4;
    p.head_groups = H_kv / p.hpc;
    const long units = (long)n_q * p.head_groups * G;
    const int steps = (budget + kF4Pair - 1) / kF4Pair;
    const int n_sel = f4_warps(H_q / H_kv > 8 ? 2 : 1) / p.hpc;
    // Splits: the shortest of (waves of CTAs, one an SM) x (rounds of a CTA's
    // teams, and its start and end) + the merge, in us: a round takes 2.5 (2 with
    // 16 query heads), a CTA's start and end 6, a merge 3 and a little per split.
    // At 3136 entries, 32/4 heads, measured for each count of splits (1, 3, the
    // chosen one): 4 rows 65, 29, 12 us (37 splits); 16 rows 65, 29, 17 (9);
    // 80 rows 67, 60, 60; 128 rows 69, 87, 69 (1); 163 rows 133, 112, 112. (Before
    // steps without entries were skipped, which took about 1 us off each.)
    const double round = H_q / H_kv > 8 ? 2.0 : 2.5;
    int per = steps > 0 ? steps : 1;
    double best = 0;
    for (int s = 1, last = 0; s <= 64 && s <= steps; ++s) {
        const int each = (steps + s - 1) / s;
        if (each == last) continue;  // (no more splits than before)
        last = each;
        const int parts = (steps + each - 1) / each;
        const long waves = (units * parts + num_sms - 1) / num_sms;
        const double t = (double)waves * (round * ((each + n_sel - 1) / n_sel) + 6) + (parts > 1 ? 3 + 0.03 * parts : 0);
        if (s == 1 || t < 0.97 * best) {
            best = t;
            per = each;
        }
    }
    p.entries_per_split = per * kF4Pair;
    p.n_splits = steps > 0 ? (steps + per - 1) / per : 1;
    p.smem_bytes = kF4RingBytes;
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
    static std::atomic<uint64_t> allowed[6];
    const bool wide = b.H_q / b.H_kv > 8;
    auto kern = b.hpc == 1 ? (wide ? attend_fp4_kernel<2, 1> : attend_fp4_kernel<1, 1>)
                : b.hpc == 2 ? (wide ? attend_fp4_kernel<2, 2> : attend_fp4_kernel<1, 2>)
                             : (wide ? attend_fp4_kernel<2, 4> : attend_fp4_kernel<1, 4>);
    cudaError_t e = allow_smem(kern, kF4RingBytes, allowed[wide + 2 * (b.hpc >> 1)]);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(b.n_splits * b.head_groups), (unsigned)b.n_q, (unsigned)b.G);
    e = launch_pdl(kern, grid, dim3((unsigned)(f4_warps(wide ? 2 : 1) * kWarp)), smem_bytes, stream, 0, a);
    if (e != cudaSuccess || b.n_splits == 1) return e;
    return launch_attend_merge(b, stream);
}

}  // namespace lsa
