// attend_prompt_few.cu — whole-prompt attention where each sequence has a
// token or two of new rows: lsa_attend_prompt's form for decoding over a dense
// cache.
//
// With so few rows the work is reading K and V once. A 128-row tile of the
// tensor-core path (attend_prompt.cu) would be nearly empty and its chain of
// product, softmax and product (1.7 us a tile) would be the time.
//
// Design (B200): grid = (parts of the keys, kv heads, sequences). A warp takes
// every fourth tile of 16 keys of its CTA's part, through a ring of its own
// that asynchronous copies fill two tiles ahead (two CTAs' rings: 192 KB per
// SM). As in attend.cu S^T = K Q^T with
// the keys as M and the sequence's (row, query head) pairs as N columns, mma
// m16n8k16 in bf16, online softmax in fp32, O^T += V^T P^T with P^T as bf16
// through movmatrix. The warps merge through shared memory; the parts of a row
// are combined by prompt_merge_kernel, or, where few of them run at once
// (plan_prompt), are a cluster's CTAs that join their results through
// distributed shared memory (16 tokens over up to 500: 6.5 against 7.9 us). A
// part has a fixed number of keys, so that CTAs are alike whatever the
// sequences' lengths; those behind a sequence's end have nothing to do. In a
// cluster it is an equal share of its sequence.
//
// Whether a batch comes here goes by its mean of rows, so single sequences
// may have many more columns than the 8 or 16 that a CTA takes. Such further
// runs of columns are other CTAs' work: about as many as run at once, behind
// the sequences' own in the grid, take them in turn (one chunk of 64 rows on
// 65536 tokens beside 63 single tokens on up to 3136, 32/4 heads: 7604 us with
// all runs one after the other in the sequence's own CTAs, 516 so, and 879 on
// the 128-row tiles of attend_prompt.cu; one of 17 beside 15, on up to 3136: 97,
// 28 and 30; one of 64 on 16384 tokens in 64 slots, the others empty: 2853, 204
// and 214). With nothing to take they cost less than the calls' spread.
#include "common.cuh"
#include "internal.h"
#include "prompt_parts.cuh"

namespace lsa {
namespace {

constexpr int kFwWarps = 4, kFwThreads = kFwWarps * kWarp;
constexpr int kFwTile = 16, kFwRing = 3, kFwD = 128;
constexpr int kFwRow = kFwD * 2;                       // bytes of a K or V row
constexpr int kFwTileBytes = 2 * kFwTile * kFwRow;     // K, then V: 8 KB
constexpr int kFwSmem = kFwWarps * kFwRing * kFwTileBytes;
constexpr int kFwPark = 36;                            // floats of a lane per column tile: o, m, l
constexpr int kFwJoinRow = kFwD + 4;                   // floats of a column in the cluster's merge area (padded: no bank conflicts)
// the merge areas lie in the rings: the warps' results, then the CTA's
__host__ __device__ constexpr int fw_join_at(int nt) { return kFwWarps * nt * kFwPark * kWarp * 4; }
static_assert(fw_join_at(2) + 16 * (kFwJoinRow * 4 + 8) <= kFwSmem, "shared memory of one CTA");

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 16-byte chunk c of row m, so that eight rows' equal chunks fall on all banks.
__device__ __forceinline__ uint32_t fw_at(int m, int c) { return (uint32_t)(m * kFwRow + 16 * (c ^ (m & 7))); }

// The i-th of all sequences' runs of W columns behind each one's first: its
// sequence and first column; false behind the last. A warp looks at 32 kEach
// sequences a step, a lane at every 32nd of them (and counts its own in a row).
template <int W, int kEach>
__device__ __forceinline__ bool find_columns(const PromptArgs& a, int i, int& seq, int& c0) {
    const int lane = lane_id();
    auto runs = [&](int b) {  // (of a sequence that lies outside the rows: none)
        const int start = a.row_offset[min(b, a.n_seq)], end = a.row_offset[min(b + 1, a.n_seq)];
        return start >= 0 && end <= a.n_rows && end > start ? ((end - start) * a.G - 1) / W : 0;
    };
    for (int b0 = 0; b0 < a.n_seq; b0 += kEach * kWarp) {
        int mine = 0;
#pragma unroll
        for (int j = 0; j < kEach; ++j) mine += runs(b0 + kWarp * j + lane);
        if (!__any_sync(0xffffffffu, mine > 0)) continue;
        int upto = mine;
#pragma unroll
        for (int k = 1; k < kWarp; k <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, k);
            if (lane >= k) upto += x;
        }
        const uint32_t here = __ballot_sync(0xffffffffu, upto > i);
        if (here == 0u) {
            i -= __shfl_sync(0xffffffffu, upto, kWarp - 1);
            continue;
        }
        const int owner = __ffs(here) - 1;
        i -= __shfl_sync(0xffffffffu, upto - mine, owner);
        seq = b0 + owner;
        for (int r = runs(seq); i >= r; r = runs(seq)) {  // (the owner has more than i)
            i -= r;
            seq += kWarp;
        }
        c0 = (i + 1) * W;
        return true;
    }
    return false;
}
// Few steps where there are many sequences, few loads a step where there are
// not (nothing found: 60000 sequences of 3 tokens 592 us with 32 a lane, 643
// with 8; 16 over up to 500 tokens 7.0 and 6.2).
template <int W>
__device__ __forceinline__ bool further_columns(const PromptArgs& a, int i, int& seq, int& c0) {
    return a.n_seq > 8192 ? find_columns<W, 32>(a, i, seq, c0) : find_columns<W, 8>(a, i, seq, c0);
}

// NT: tiles of 8 (row, query head) columns taken at a time. JOINED: the parts
// of a sequence are a cluster.
template <int NT, bool JOINED>
__global__ void __launch_bounds__(kFwThreads, 2) attend_prompt_few_kernel(const __grid_constant__ PromptArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = lane_id(), warp = warp_id();
    const int g = lane >> 2, t4 = lane & 3;
    const int part = blockIdx.x, kvh = blockIdx.y;
    const int helper = (int)blockIdx.z - a.n_seq;  // behind the sequences' CTAs: those for further columns
    int seq = blockIdx.z, c0 = 0, row0 = 0, n = 0, len = 0;
    int64_t off = 0;
    auto look_up = [&]() {
        row0 = a.row_offset[seq];
        n = a.row_offset[seq + 1] - row0;
        len = a.seq_lens[seq];
        off = a.kv_offset[seq];
    };
    bool found = helper < 0 || further_columns<8 * NT>(a, helper, seq, c0);
    if (found) look_up();
    pdl_enter();
    // (offsets that ascend have no more runs than `further`; others end the helpers' turns there)
    auto next = [&](int& turn) { return helper >= 0 && (turn += a.helpers) < a.further && further_columns<8 * NT>(a, turn, seq, c0); };
    for (int turn = helper; found; found = next(turn)) {
        if (turn != helper) {
            __syncthreads();  // the merge area of the columns before
            look_up();
        }
        if (n <= 0) continue;
        if (row0 < 0 || (int64_t)row0 + n > a.n_rows || n > len || len > a.max_len || off < 0 || off > a.total_tokens - len) {
            if (tid == 0 && part == 0 && kvh == 0 && c0 == 0) flag(a.dev_status, LSA_DEV_BAD_LENGTH);
            continue;
        }
        const int base = len - n;                     // tokens before the first row
        // (a cluster's parts are equal shares of the sequence)
        const int part_keys = JOINED ? ((len + a.n_parts - 1) / a.n_parts + kFwTile - 1) / kFwTile * kFwTile : a.part_keys;
        const int k_lo = min(len, part * part_keys), k_hi = min(len, k_lo + part_keys);
        if (!JOINED && k_lo >= len) continue;
        const int n_tiles = max(0, k_hi - k_lo + kFwTile - 1) / kFwTile;
        const int G = a.G, cols = n * G;
        const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * kFwRing * kFwTileBytes);
        const uint16_t* kb = a.k + off * a.k_stride + (int64_t)kvh * kFwD + 8 * (lane & 15);
        const uint16_t* vb = a.v + off * a.v_stride + (int64_t)kvh * kFwD + 8 * (lane & 15);
        // a lane copies 16-byte chunk lane % 16 of rows lane / 16, + 2, ...; rows behind the part are zeros
        auto fetch = [&](int i, int slot) {
            if (i < n_tiles) {
                const uint32_t to = ring + (uint32_t)(slot * kFwTileBytes);
#pragma unroll
                for (int x = 0; x < kFwTile / 2; ++x) {
                    const int m = 2 * x + (lane >> 4);
                    const int key = k_lo + i * kFwTile + m;
                    const uint32_t nb = key < k_hi ? 16u : 0u;
                    const int64_t at = min(key, k_hi - 1);
                    cp_async16(to + fw_at(m, lane & 15), kb + at * a.k_stride, nb);
                    cp_async16(to + (uint32_t)(kFwTile * kFwRow) + fw_at(m, lane & 15), vb + at * a.v_stride, nb);
                }
            }
            cp_async_commit();
        };

        float* join = reinterpret_cast<float*>(smem + fw_join_at(NT));  // [column][kFwJoinRow], then [column] (m, l)
        float2* join_ml = reinterpret_cast<float2*>(join + 8 * NT * kFwJoinRow);
#pragma unroll
        for (int j = 0; j < kFwRing - 1; ++j) fetch(warp + j * kFwWarps, j);
        // query fragments, and the keys that the lane's accumulator columns see
        uint32_t qb[NT][8][2];
        int sees[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int col = c0 + 8 * t + g;
            const uint16_t* q = a.q + (int64_t)(row0 + col / G) * a.q_stride + (int64_t)(kvh * G + col % G) * kFwD;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    qb[t][ks][x] = col < cols ? __ldg(reinterpret_cast<const uint32_t*>(q + 16 * ks + 8 * x + 2 * t4)) : 0u;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int own = c0 + 8 * t + 2 * t4 + c;
                sees[t][c] = own < cols ? base + own / G + 1 : 0;
            }
        }
        float o[NT][8][4], m_run[NT][2], l_run[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) o[t][mt][0] = o[t][mt][1] = o[t][mt][2] = o[t][mt][3] = 0.f;
            m_run[t][0] = m_run[t][1] = -INFINITY;
            l_run[t][0] = l_run[t][1] = 0.f;
        }
        int slot = 0;
        for (int i = warp; i < n_tiles; i += kFwWarps) {
            fetch(i + (kFwRing - 1) * kFwWarps, slot == 0 ? kFwRing - 1 : slot - 1);
            cp_async_wait<kFwRing - 1>();
            __syncwarp();
            const uint32_t kt = ring + (uint32_t)(slot * kFwTileBytes), vt = kt + kFwTile * kFwRow;
            slot = slot + 1 == kFwRing ? 0 : slot + 1;
            const int key0 = k_lo + i * kFwTile;
            const bool masked = key0 + kFwTile > base + 1;  // some column does not see some key of the tile
            bool odd = false;  // some element under the mask is not finite
            if (masked && n > 1) {
                // V of the newest tokens: rows before them have weight 0, and 0 times an
                // element that is not finite is not 0: such elements are zeroed here and
                // added below, to the rows that see them
                for (int x = lane; x < kFwTile * 16; x += kWarp) {
                    const int m = x >> 4;
                    if (key0 + m <= base || key0 + m >= k_hi) continue;
                    const uint32_t at = vt + fw_at(m, x & 15);
                    uint4 y = ld_shared_v4(at);
                    uint32_t* e = &y.x;
                    uint32_t any = 0;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t bad = ((e[q] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;  // an exponent of all ones carries
                        any |= bad;
                        e[q] &= ~(((bad >> 15) & 0x00010001u) * 0xffffu);
                    }
                    if (any) st_shared_v4(at, y.x, y.y, y.z, y.w);
                    odd |= any != 0;
                }
                odd = __any_sync(0xffffffffu, odd);
                __syncwarp();  // (a vote orders no memory: other lanes read what this one has zeroed)
            }
            // ---- S^T: 16 keys x 8 NT columns ------------------------------------------------
            float s[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                uint32_t fr[4];
                ldmatrix_x4(fr, kt + fw_at((lane & 7) + 8 * (lane >> 3 & 1), 2 * ks + (lane >> 4)));
#pragma unroll
                for (int t = 0; t < NT; ++t) mma_bf16(s[t], fr, qb[t][ks][0], qb[t][ks][1]);
            }
            // ---- online softmax ---------------------------------------------------------------
            uint32_t p[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float z[4], mx[2], al[2], mc[2];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    z[c] = s[t][c] * a.scale_log2;
                    if (masked && key0 + g + 8 * (c >> 1) >= sees[t][c & 1]) z[c] = -INFINITY;
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    mx[c] = fmaxf(z[c], z[c + 2]);
#pragma unroll
                    for (int k = 4; k < 32; k <<= 1) mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], k));
                    mx[c] = fmaxf(m_run[t][c], mx[c]);
                    mc[c] = mx[c] == -INFINITY ? 0.f : mx[c];
                    al[c] = ex2(m_run[t][c] - mc[c]);
                }
                if (__any_sync(0xffffffffu, mx[0] != m_run[t][0] || mx[1] != m_run[t][1])) {
#pragma unroll
                    for (int mt = 0; mt < 8; ++mt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) o[t][mt][c] *= al[c & 1];
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) z[c] = ex2(z[c] - mc[c & 1]);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    m_run[t][c] = mx[c];
                    l_run[t][c] = l_run[t][c] * al[c] + (z[c] + z[c + 2]);
                }
                p[t][0] = movmatrix_trans(pack_bf16(z[0], z[1]));
                p[t][1] = movmatrix_trans(pack_bf16(z[2], z[3]));
            }
            // ---- O^T += V^T P^T -----------------------------------------------------------------
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
                uint32_t fr[4];  // channels 16 mt + g, + 8 of keys 2t, 2t+1 and 2t+8, 2t+9
                ldmatrix_x4_trans(fr, vt + fw_at((lane & 7) + 8 * (lane >> 4), 2 * mt + (lane >> 3 & 1)));
#pragma unroll
                for (int t = 0; t < NT; ++t) mma_bf16(o[t][mt], fr, p[t][0], p[t][1]);
            }
            if (odd) {
                for (int m = max(0, base + 1 - key0); m < kFwTile && key0 + m < k_hi; ++m) {
                    const uint16_t* v = a.v + (off + key0 + m) * a.v_stride + (int64_t)kvh * kFwD;
                    for (int mt = 0; mt < 8; ++mt)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float x = __uint_as_float((uint32_t)v[16 * mt + 8 * h + g] << 16);
                            if (isfinite(x)) continue;
#pragma unroll
                            for (int t = 0; t < NT; ++t)
#pragma unroll
                                for (int mm = 0; mm < 8; ++mm)
                                    if (mm == mt) {
                                        if (key0 + m < sees[t][0]) o[t][mm][2 * h] += x;
                                        if (key0 + m < sees[t][1]) o[t][mm][2 * h + 1] += x;
                                    }
                        }
                }
            }
            __syncwarp();  // the slot may be filled again
        }
        cp_async_wait<0>();
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int k = 4; k < 32; k <<= 1) l_run[t][c] += __shfl_xor_sync(0xffffffffu, l_run[t][c], k);
        __syncthreads();
        // ---- the warps' results: each combines two of the eight channel tiles -----------------
        float* park = reinterpret_cast<float*>(smem);  // [warp][NT][kFwPark][32]
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float* x = park + (warp * NT + t) * kFwPark * kWarp + lane;
#pragma unroll
            for (int mt = 0; mt < 8; ++mt)
#pragma unroll
                for (int c = 0; c < 4; ++c) x[(4 * mt + c) * kWarp] = o[t][mt][c];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                x[(32 + c) * kWarp] = m_run[t][c];
                x[(34 + c) * kWarp] = l_run[t][c];
            }
        }
        if (helper < 0) pdl_trigger();
        __syncthreads();
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = c0 + 8 * t + 2 * t4 + c;
                const float* x0 = park + t * kFwPark * kWarp + lane;
                float M = -INFINITY, l = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < kFwWarps; ++w) M = fmaxf(M, x0[(w * NT * kFwPark + 32 + c) * kWarp]);
                const float mb = M == -INFINITY ? 0.f : M;
#pragma unroll
                for (int w = 0; w < kFwWarps; ++w) {
                    const float* x = x0 + w * NT * kFwPark * kWarp;
                    const float f = ex2(x[(32 + c) * kWarp] - mb);
                    l += x[(34 + c) * kWarp] * f;
#pragma unroll
                    for (int q = 0; q < 4; ++q) y[q] += x[(4 * (2 * warp + (q >> 1)) + c + 2 * (q & 1)) * kWarp] * f;
                }
                if (JOINED) {
                    const int own = 8 * t + 2 * t4 + c;
#pragma unroll
                    for (int q = 0; q < 4; ++q) join[own * kFwJoinRow + 16 * (2 * warp + (q >> 1)) + 8 * (q & 1) + g] = y[q];
                    if (warp == 0 && g == 0) join_ml[own] = make_float2(l == 0.f ? M : fmaxf(M, -3e38f), l);
                    continue;
                }
                if (col >= cols) continue;
                const int64_t row = (int64_t)(row0 + col / G) * a.H_q + kvh * G + col % G;
                // channels 16 mt + g and + 8 of mt = 2 warp, 2 warp + 1
                if (a.n_parts == 1) {
                    const float inv = 1.f / l;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const __nv_bfloat16 b = __float2bfloat16_rn(y[q] * inv);
                        a.out[row * kFwD + 16 * (2 * warp + (q >> 1)) + 8 * (q & 1) + g] = *reinterpret_cast<const uint16_t*>(&b);
                    }
                    if (a.lse != nullptr && warp == 0 && g == 0) a.lse[row] = (M + log2f(l)) * 0.6931471805599453f;
                } else {
                    const int64_t at = (int64_t)part * a.n_rows * a.H_q + row;
#pragma unroll
                    for (int q = 0; q < 4; ++q) a.part_o[at * kFwD + 16 * (2 * warp + (q >> 1)) + 8 * (q & 1) + g] = y[q];
                    // (a maximum of -infinity marks an empty part: one of NaN scores alone is not)
                    if (warp == 0 && g == 0)
                        reinterpret_cast<float2*>(a.part_ml)[at] = make_float2(l == 0.f ? M : fmaxf(M, -3e38f), l);
                }
            }
        if (!JOINED) continue;
        // ---- the cluster's parts: each CTA combines its share of (column, 4 channels) ------------
        __syncwarp();
        cluster_sync();
        for (int e = part * kFwThreads + tid; e < 8 * NT * (kFwD / 4); e += a.n_parts * kFwThreads) {
            const int own = e / (kFwD / 4), ch = 4 * (e % (kFwD / 4)), col = c0 + own;
            if (col >= cols) continue;
            float2 ml[kFewJoined];
            float4 v[kFewJoined];
            float M = -INFINITY;
#pragma unroll
            for (int p = 0; p < kFewJoined; ++p) {
                ml[p] = make_float2(-INFINITY, 0.f);
                v[p] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (p < a.n_parts) {
                    ml[p] = ld_cluster_f2(map_cta(smem_u32(&join_ml[own]), (uint32_t)p));
                    v[p] = ld_cluster_f4(map_cta(smem_u32(&join[own * kFwJoinRow + ch]), (uint32_t)p));
                }
                M = fmaxf(M, ml[p].x);
            }
            float l = 0.f;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int p = 0; p < kFewJoined; ++p) {
                if (ml[p].x == -INFINITY) continue;  // no keys
                const float f = ex2(ml[p].x - M);
                l += ml[p].y * f;
                y.x += v[p].x * f;
                y.y += v[p].y * f;
                y.z += v[p].z * f;
                y.w += v[p].w * f;
            }
            const int64_t row = (int64_t)(row0 + col / G) * a.H_q + kvh * G + col % G;
            const float inv = 1.f / l;
            *reinterpret_cast<uint2*>(a.out + row * kFwD + ch) = make_uint2(pack_bf16(y.x * inv, y.y * inv), pack_bf16(y.z * inv, y.w * inv));
            if (a.lse != nullptr && ch == 0) a.lse[row] = (M + log2f(l)) * 0.6931471805599453f;
        }
        __syncwarp();
        cluster_sync();  // no CTA reads another's shared memory after this
    }
}

}  // namespace

cudaError_t launch_attend_prompt_few(const PromptArgs& a, int parts, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed[4];
    const bool wide = few_columns(a.n_seq, a.n_rows, a.G) > 8;
    const bool joined = parts > 1 && a.part_o == nullptr;
    auto kern = wide ? (joined ? attend_prompt_few_kernel<2, true> : attend_prompt_few_kernel<2, false>)
                     : (joined ? attend_prompt_few_kernel<1, true> : attend_prompt_few_kernel<1, false>);
    const cudaError_t e = allow_smem(kern, kFwSmem, allowed[wide + 2 * joined]);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((unsigned)parts, (unsigned)a.H_kv, (unsigned)(a.n_seq + a.helpers)), dim3(kFwThreads), kFwSmem,
                      stream, joined ? parts : 0, a);
}

}  // namespace lsa
