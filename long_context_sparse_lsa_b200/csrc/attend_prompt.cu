// attend_prompt.cu — causal GQA softmax attention of whole prompts (or of
// their newest tokens over a cache) for packed sequences of different lengths,
// every token up to a row's own attended: the dense pass beside the sparse
// one of attend.cu.
//
// Design (B200): S = Q K^T and O += P V on tcgen05.mma (bf16, fp32
// accumulators in tensor memory), one CTA per work item.
//  * Rows: one tile of 128 rows is T = 128 / G tokens x the G query heads of
//    one kv head, so that all of them share K and V, a short prompt fills its
//    tiles and the causal border wastes at most one 128-key tile per T tokens.
//    A CTA holds two such tiles (their S and O fill the 512 columns of tensor
//    memory) over the same K/V tiles.
//  * Warps 0..3 and 4..7 are the softmax of the two tiles, one thread per row:
//    scores from tensor memory, running maximum and sum in fp32, P back into
//    the columns S came from as bf16, from where the second product reads it.
//    While one tile's softmax runs, the tensor core works for the other.
//  * Warp 8 loads Q and a ring of 128-key K and V tiles by TMA; one thread of
//    warp 9 issues the MMAs; warps 10 and 11 clean V where the mask reaches it
//    (below).
//  * The output is rescaled only when a row's maximum has risen by more than
//    2^8 over the one in use (P then stays below 2^8, sums are fp32): the
//    softmax threads do it themselves, since S of tile j is complete only
//    after P V of the tile before is.
//  * Masked keys: the scores are replaced by -infinity, so P is 0, but 0 * V
//    is not 0 where V is an infinity or NaN. In tiles that the mask reaches,
//    V rows behind every row of the CTA (other sequences' rows, rows never
//    written) are zeroed in shared memory, and elements that are not finite
//    within the CTA's own tokens are zeroed and added back at the end, by each
//    row that sees them.
//  * Long caches and few rows: the keys are split over CTAs, whose partials
//    prompt_merge_kernel combines by log-sum-exp.
//  * Every wait is bounded; on expiry the kernel flags LSA_DEV_TIMEOUT, waits
//    (bounded) for what it issued, frees its tensor memory and returns.
#include "internal.h"
#include "tcgen05.cuh"

namespace lsa {
namespace {

constexpr int kPrD = 128;
constexpr int kPrRows = 128;                         // rows of a tile
constexpr int kPrKeys = 128;                         // keys of a tile
constexpr int kPrThreads = 384;
constexpr int kPrStages = 5;                         // K and V tiles in the ring
constexpr int kPrMasked = 3;                         // key tiles of a CTA that the mask may reach: it reaches fewer than 256 keys
constexpr uint32_t kHalf = kPrRows * 128;            // 16 KB: 128 rows of 64 channels
constexpr uint32_t kPrTile = 2 * kHalf;              // 32 KB
constexpr uint32_t kTmemS = 0, kTmemO = 256;         // tensor-memory columns: S0, S1, O0, O1
constexpr uint32_t kIdescS = idesc_bf16(128, 128, false), kIdescO = idesc_bf16(128, 128, true);

struct PrShared {
    uint64_t full[kPrStages], empty[kPrStages];
    uint64_t q_full[2], s_full[2], p_full[2], o_full[2];
    uint64_t v_raw[kPrMasked];  // a V tile that the mask reaches has landed (its `full` comes once it is clean)
    uint64_t drain;
    uint32_t tmem;
    int32_t abort;
    int32_t not_finite;
    int32_t cleaned[kPrMasked];  // warps that are done with a V tile
};
constexpr size_t kPrSmem = 1024 + (size_t)(2 + kPrStages) * kPrTile + sizeof(PrShared);
static_assert(kPrSmem <= 227 * 1024, "shared memory of one CTA");

struct PrArgs {
    CUtensorMap q, k, v;
    PromptArgs a;
};

__device__ __forceinline__ bool pr_wait(PrShared& sh, uint64_t& bar, uint32_t parity, int32_t* status) {
    if (mbar_wait_bounded(smem_u32(&bar), parity, kWaitLimitNs)) return true;
    flag(status, LSA_DEV_TIMEOUT);
    atomicExch(&sh.abort, 1);
    return false;
}
__device__ __forceinline__ bool pr_aborted(const PrShared& sh) {
    return *reinterpret_cast<const volatile int32_t*>(&sh.abort) != 0;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Sequence b owns the tile slots from row_offset[b] / Tc + b on: at least
// ceil(rows / Tc) of them, and every slot number below n_rows / Tc + n_seq
// belongs to one sequence.
__device__ __forceinline__ int slot_seq(const int32_t* row_offset, int n_seq, int tc, int slot) {
    return find_last(n_seq, [&](int b) { return row_offset[b] / tc + b <= slot; });
}

// The sequence's rows and tokens, checked.
struct PrSeq {
    int row0, n, base;  // first row, rows, tokens before the first row
    int64_t off;
    bool ok;
};
__device__ __forceinline__ PrSeq pr_seq(const PromptArgs& a, int b) {
    PrSeq s;
    s.row0 = a.row_offset[b];
    const int end = a.row_offset[b + 1];
    const int len = a.seq_lens[b];
    s.off = a.kv_offset[b];
    s.n = end - s.row0;
    s.base = len - s.n;
    s.ok = s.row0 >= 0 && end <= a.n_rows && s.n <= len && len <= a.max_len && s.off >= 0 && s.off + len <= a.total_tokens;
    return s;
}

__global__ void __launch_bounds__(kPrThreads, 1) attend_prompt_kernel(const __grid_constant__ PrArgs args) {
    const PromptArgs& a = args.a;
    extern __shared__ __align__(16) uint8_t pr_raw[];
    const int tid = threadIdx.x, lane = lane_id(), warp = warp_id();
    const int split = blockIdx.x % a.n_splits;
    const int kvh = (blockIdx.x / a.n_splits) % a.H_kv;
    const int slot = blockIdx.x / a.n_splits / a.H_kv;
    const int G = a.G, T = a.tile_tokens, Tc = 2 * T;
    const int seq = slot_seq(a.row_offset, a.n_seq, Tc, slot);
    const PrSeq sq = pr_seq(a, seq);
    pdl_enter();
    const int local = slot - (sq.row0 / Tc + seq);
    const int tiles = (sq.n + Tc - 1) / Tc;
    if (sq.n <= 0 || local < 0 || local >= tiles) return;
    if (!sq.ok) {
        if (tid == 0 && local == 0) flag(a.dev_status, LSA_DEV_BAD_LENGTH);
        return;
    }
    const int t0 = (tiles - 1 - local) * Tc;  // first token (row) of the CTA; the longest first
    // per tile: tokens [t_lo, t_hi), key tiles [0, nk); the CTA's split of the key tiles
    const int t_end[2] = {min(t0 + T, sq.n), min(t0 + Tc, sq.n)};
    const bool two = t0 + T < sq.n;
    const int see = sq.base + t_end[two ? 1 : 0];  // keys that some row of the CTA sees
    const int nk0 = (sq.base + t_end[0] + kPrKeys - 1) / kPrKeys;
    const int nk1 = two ? (see + kPrKeys - 1) / kPrKeys : 0;
    const int nk = max(nk0, nk1);
    const int lo = (int)((int64_t)nk * split / a.n_splits), hi = (int)((int64_t)nk * (split + 1) / a.n_splits);
    const int top[2] = {min(hi, nk0), min(hi, nk1)};  // tile w works on key tiles [lo, top[w])

    const uint32_t raw = smem_u32(pr_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t sQ = base, sKV = base + 2 * kPrTile;
    PrShared& sh = *reinterpret_cast<PrShared*>(pr_raw + (base - raw) + (2 + kPrStages) * kPrTile);
    if (tid == 0) {
        for (int i = 0; i < kPrStages; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 1);
            mbar_init(smem_u32(&sh.empty[i]), 1);
            }
        for (int i = 0; i < kPrMasked; ++i) {
            mbar_init(smem_u32(&sh.v_raw[i]), 1);
            sh.cleaned[i] = 0;
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.q_full[i]), 1);
            mbar_init(smem_u32(&sh.s_full[i]), 1);
            mbar_init(smem_u32(&sh.p_full[i]), 4);
            mbar_init(smem_u32(&sh.o_full[i]), 1);
        }
        mbar_init(smem_u32(&sh.drain), 1);
        sh.abort = 0;
        sh.not_finite = 0;
        mbar_fence_init();
    }
    if (warp == 9) tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = sh.tmem;
    const int masked_lo = (sq.base + t0 + 1) / kPrKeys;  // key tiles from here on hold keys that some row does not see
    const int n_it = hi - lo;

    if (warp == 8) {
        // ---- TMA: Q tiles, then K and V of key tiles hi - 1 .. lo -------------------
        if (lane == 0 && n_it > 0) {
            for (int w = 0; w < (two ? 2 : 1); ++w) {
                mbar_arrive_expect_tx(smem_u32(&sh.q_full[w]), (uint32_t)(T * G) * 256u);
                for (int h = 0; h < 2; ++h)
                    tma_load_4d(sQ + w * kPrTile + h * kHalf, &args.q, 64 * h, 0, kvh, sq.row0 + t0 + w * T,
                                smem_u32(&sh.q_full[w]));
            }
            int issued = 0;
            for (; issued < 2 * n_it; ++issued) {
                const int st = issued % kPrStages;
                if (issued >= kPrStages && !pr_wait(sh, sh.empty[st], ((issued / kPrStages) + 1) & 1, a.dev_status)) break;
                if (pr_aborted(sh)) break;
                const int j = hi - 1 - (issued >> 1);
                const int row = (int)(sq.off + (int64_t)j * kPrKeys);
                const uint32_t bar = (issued & 1) && j >= masked_lo ? smem_u32(&sh.v_raw[issued >> 1]) : smem_u32(&sh.full[st]);
                mbar_arrive_expect_tx(bar, kPrTile);
                for (int h = 0; h < 2; ++h)
                    tma_load_3d(sKV + st * kPrTile + h * kHalf, (issued & 1) ? &args.v : &args.k, 64 * h, kvh, row, bar);
            }
            // every issued copy has landed before the CTA can exit
            for (int i = issued > kPrStages ? issued - kPrStages : 0; i < issued; ++i)
                mbar_wait_bounded(smem_u32(&sh.full[i % kPrStages]), (i / kPrStages) & 1, kWaitLimitNs);
            for (int w = 0; w < (two ? 2 : 1); ++w) mbar_wait_bounded(smem_u32(&sh.q_full[w]), 0, kWaitLimitNs);
        }
    } else if (warp == 9) {
        // ---- MMA issue ------------------------------------------------------------------
        if (lane == 0 && n_it > 0) {
            bool ok = true;
            int uses[2] = {0, 0};  // S tiles issued per row tile
            auto qk = [&](int w, int j) {
                const int st = (2 * (hi - 1 - j)) % kPrStages;
                const uint64_t qd = desc_k_major(sQ + w * kPrTile), kd = desc_k_major(sKV + st * kPrTile);
#pragma unroll
                for (int k = 0; k < 8; ++k) {  // 16 channels a step: 32 bytes on, the second half 16 KB on
                    const uint64_t at = (uint64_t)((k & 3) * 2 + (k >> 2) * (kHalf >> 4));
                    mma_bf16_ss(tmem + kTmemS + 128 * w, qd + at, kd + at, kIdescS, k > 0);
                }
                mma_commit(smem_u32(&sh.s_full[w]));
                ++uses[w];
            };
            auto pv = [&](int w, int j) {
                ok = pr_wait(sh, sh.p_full[w], (uses[w] - 1) & 1, a.dev_status);
                if (!ok) return;
                tmem_fence_after();
                const int st = (2 * (hi - 1 - j) + 1) % kPrStages;
                const uint64_t vd = desc_mn_major(sKV + st * kPrTile, kHalf);
#pragma unroll
                for (int k = 0; k < 8; ++k)  // 16 keys a step: 8 tensor-memory columns of P, 2048 bytes of V
                    mma_bf16_ts(tmem + kTmemO + 128 * w, tmem + kTmemS + 128 * w + 8 * k, vd + (uint64_t)(128 * k), kIdescO,
                                k > 0 || uses[w] > 1);
            };
            auto wait_v = [&](int j) {
                const int i = 2 * (hi - 1 - j) + 1;
                ok = pr_wait(sh, sh.full[i % kPrStages], (i / kPrStages) & 1, a.dev_status);
            };
            for (int w = 0; ok && w < (two ? 2 : 1); ++w) ok = pr_wait(sh, sh.q_full[w], 0, a.dev_status);
            for (int j = hi - 1; ok && j >= lo - 1; --j) {
                // step j: P V of key tile j + 1, then Q K^T of tile j
                if (j >= lo) {
                    const int i = 2 * (hi - 1 - j);
                    ok = pr_wait(sh, sh.full[i % kPrStages], (i / kPrStages) & 1, a.dev_status);
                    tmem_fence_after();
                }
                if (ok && j + 1 < hi) wait_v(j + 1);
                for (int w = 0; ok && w < 2; ++w) {
                    if (j + 1 < top[w]) pv(w, j + 1);
                    if (ok && w == 1 && j + 1 < hi) mma_commit(smem_u32(&sh.empty[(2 * (hi - 2 - j) + 1) % kPrStages]));
                    if (ok && j >= lo && j < top[w]) qk(w, j);
                }
                if (ok && j >= lo) mma_commit(smem_u32(&sh.empty[(2 * (hi - 1 - j)) % kPrStages]));
                if (pr_aborted(sh)) ok = false;
            }
            for (int w = 0; w < 2; ++w) mma_commit(smem_u32(&sh.o_full[w]));
            mma_commit(smem_u32(&sh.drain));
            mbar_wait_bounded(smem_u32(&sh.drain), 0, kWaitLimitNs);
        }
    } else if (warp >= 10) {
        // ---- V under the mask -----------------------------------------------------------
        for (int j = hi - 1; j >= max(lo, masked_lo); --j) {
            const int i = 2 * (hi - 1 - j) + 1;
            if (!__all_sync(0xffffffffu, pr_wait(sh, sh.v_raw[hi - 1 - j], 0, a.dev_status))) break;
            const uint32_t v = sKV + (uint32_t)((i % kPrStages) * kPrTile);
            // keys from the second row's own token on: some row does not see them
            const int r_lo = max(0, sq.base + t0 + 1 - j * kPrKeys), r_end = min(kPrKeys, see - j * kPrKeys);
            bool found = false;
            for (int c = (warp - 10) * kWarp + lane + 8 * r_lo; c < 8 * kPrKeys; c += 2 * kWarp) {
                const int r = c >> 3;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t at = v + h * kHalf + 16 * c;
                    uint4 x = make_uint4(0, 0, 0, 0);
                    bool put = true;
                    if (r < r_end) {
                        x = ld_shared_v4(at);
                        uint32_t* e = &x.x;
                        put = false;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const bool l = (e[q] & 0x7f80u) == 0x7f80u, u = (e[q] & 0x7f800000u) == 0x7f800000u;
                            put |= l | u;
                            e[q] &= (l ? 0xffff0000u : 0xffffffffu) & (u ? 0x0000ffffu : 0xffffffffu);
                        }
                        found |= put;
                    }
                    if (put)
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x.x), "r"(x.y), "r"(x.z),
                                     "r"(x.w)
                                     : "memory");
                }
            }
            if (found) sh.not_finite = 1;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {  // the second of the two warps passes the tile on
                __threadfence_block();
                if (atomicAdd(&sh.cleaned[hi - 1 - j], 1) == 1) {
                    __threadfence_block();
                    mbar_arrive(smem_u32(&sh.full[i % kPrStages]));
                }
            }
        }
    } else {
        // ---- softmax: one thread per row ------------------------------------------------
        const int w = warp >> 2;
        const int r = tid & 127;
        const int token = t0 + w * T + min(r / G, T - 1);
        const uint32_t ts = tmem + ((uint32_t)(warp & 3) << 21) + kTmemS + 128u * w;  // lane 32 * (warp & 3) in bits 16..
        const uint32_t to = tmem + ((uint32_t)(warp & 3) << 21) + kTmemO + 128u * w;
        const int sees = sq.base + min(token, sq.n - 1) + 1;  // keys of this row
        const int masked = (sq.base + t0 + w * T + 1) / kPrKeys;
        const float c = a.scale_log2;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        int u = 0;
        for (int j = top[w] - 1; j >= lo; --j, ++u) {
            ok = pr_wait(sh, sh.s_full[w], u & 1, a.dev_status) && !pr_aborted(sh);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            tmem_fence_after();
            float s[4][32];
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_load32(ts + 32 * q, s[q]);
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_load_wait(s[q]);
            if (j >= masked) {
                const int lim = sees - j * kPrKeys;
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int i = 0; i < 32; ++i) s[q][i] = 32 * q + i < lim ? s[q][i] : -INFINITY;
            }
            float mx[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                mx[q] = s[q][0];
#pragma unroll
                for (int i = 1; i < 32; ++i) mx[q] = fmaxf(mx[q], s[q][i]);
            }
            const float mt = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
            // P may grow to 2^8 before the maximum in use moves
            if (__any_sync(0xffffffffu, (mt - m) * c > 8.f)) {
                const float al = mt == -INFINITY ? 1.f : ex2((m - mt) * c);
                m = mt;
                l *= al;
                if (u > 0) {
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        float o[32];
                        tmem_load32(to + 32 * q, o);
                        tmem_load_wait(o);
                        uint32_t x[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(o[i] * al);
                        tmem_store32(to + 32 * q, x);
                    }
                }
            }
            const float mc = m == -INFINITY ? 0.f : m * c;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = 0; q < 4; q += 2) {
                uint32_t p[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int qq = q + (i >> 4), e = 2 * (i & 15);
                    const float p0 = ex2(fmaf(s[qq][e], c, -mc)), p1 = ex2(fmaf(s[qq][e + 1], c, -mc));
                    sum[i & 3] += p0 + p1;
                    p[i] = pack_bf16(p0, p1);
                }
                tmem_store32(ts + 16 * q, p);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tmem_store_wait();
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.p_full[w]));
        }
        // ---- output -----------------------------------------------------------------------
        const bool live = r < T * G && token < sq.n && (w == 0 || two);
        if (ok && u > 0) ok = pr_wait(sh, sh.o_full[w], 0, a.dev_status);
        ok = __all_sync(0xffffffffu, ok);
        if (ok && (w == 0 || two)) {
            tmem_fence_after();
            const int64_t row = (int64_t)sq.row0 + token;
            const int head = kvh * G + r % G;
            const float inv = u > 0 ? 1.f / l : 0.f;
            const bool fix = *reinterpret_cast<volatile int32_t*>(&sh.not_finite) != 0;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                float o[32];
                if (u > 0) {
                    tmem_load32(to + 32 * q, o);
                    tmem_load_wait(o);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0.f;
                }
                if (fix && live) {  // V elements of the CTA's own tokens that are not finite, where this row sees them
                    for (int key = max(sq.base + t0 + 1, lo * kPrKeys); key < min(sees, hi * kPrKeys); ++key) {
                        const uint16_t* vr = a.v + (sq.off + key) * a.v_stride + (int64_t)kvh * kPrD + 32 * q;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float x = __uint_as_float((uint32_t)vr[i] << 16);
                            if (!isfinite(x)) o[i] += x;
                        }
                    }
                }
                if (live) {
                    if (a.n_splits == 1) {
                        uint4* dst = reinterpret_cast<uint4*>(a.out + (row * a.H_q + head) * kPrD + 32 * q);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            dst[i] = make_uint4(pack_bf16(o[8 * i] * inv, o[8 * i + 1] * inv),
                                                pack_bf16(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                                pack_bf16(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                                                pack_bf16(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
                    } else {
                        float4* dst = reinterpret_cast<float4*>(
                            a.part_o + (((int64_t)split * a.n_rows + row) * a.H_q + head) * kPrD + 32 * q);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                }
            }
            if (live) {
                if (a.n_splits > 1)
                    reinterpret_cast<float2*>(a.part_ml)[((int64_t)split * a.n_rows + row) * a.H_q + head] =
                        make_float2(l == 0.f ? m * c : fmaxf(m * c, -3e38f), l);
                else if (a.lse != nullptr)
                    a.lse[row * a.H_q + head] = (m * c + log2f(l)) * 0.6931471805599453f;
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == 9) {
        tmem_fence_after();
        tmem_free(tmem, 512);
    }
}

// One warp per (row, query head): the splits' partials by log-sum-exp.
constexpr int kPmWarps = 8;
__global__ void __launch_bounds__(kPmWarps * kWarp) prompt_merge_kernel(const __grid_constant__ PromptArgs a) {
    pdl_enter();
    const int lane = lane_id();
    const int64_t i = (int64_t)blockIdx.x * kPmWarps + warp_id();  // row * H_q + head
    if (i >= (int64_t)a.n_rows * a.H_q) return;
    const int row = (int)(i / a.H_q);
    // rows of no sequence, or of one that was refused, stay as they were
    const int seq = find_last(a.n_seq, [&](int b) { return a.row_offset[b] <= row; });
    const PrSeq sq = pr_seq(a, seq);
    if (!sq.ok || row < sq.row0 || row >= sq.row0 + sq.n) return;
    const int64_t step = (int64_t)a.n_rows * a.H_q;
    float M = -INFINITY, den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < a.n_splits; s0 += 8) {
        float2 ml[8];
        float4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const bool in = s0 + u < a.n_splits;
            ml[u] = in ? __ldcg(reinterpret_cast<const float2*>(a.part_ml) + (s0 + u) * step + i) : make_float2(-INFINITY, 0.f);
            v[u] = in ? __ldcg(reinterpret_cast<const float4*>(a.part_o + ((s0 + u) * step + i) * kPrD) + lane)
                      : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (ml[u].x == -INFINITY) continue;  // a split without keys
            const float nm = fmaxf(M, ml[u].x);
            const float so = exp2f(M - nm), sn = exp2f(ml[u].x - nm);
            den = den * so + ml[u].y * sn;
            acc.x = acc.x * so + v[u].x * sn;
            acc.y = acc.y * so + v[u].y * sn;
            acc.z = acc.z * so + v[u].z * sn;
            acc.w = acc.w * so + v[u].w * sn;
            M = nm;
        }
    }
    const float inv = 1.f / den;
    reinterpret_cast<uint2*>(a.out + i * kPrD)[lane] =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    if (lane == 0 && a.lse != nullptr) a.lse[i] = (M + log2f(den)) * 0.6931471805599453f;
}

}  // namespace

PromptPlan plan_prompt(int n_seq, int n_rows, int max_len, int H_q, int H_kv, int num_sms) {
    PromptPlan p;
    p.G = H_q / H_kv;
    p.tile_tokens = kPrRows / p.G;
    p.slots = n_rows / (2 * p.tile_tokens) + n_seq;
    // CTAs with work: each sequence with rows has at least one tile
    const int64_t items = (int64_t)p.slots * H_kv;
    const int key_tiles = (max_len + kPrKeys - 1) / kPrKeys;
    int64_t splits = num_sms / items;
    if (splits > key_tiles / 2) splits = key_tiles / 2;  // two key tiles a split at least
    if (splits < 1) splits = 1;
    p.n_splits = (int)splits;
    p.ws_bytes = 0;
    if (p.n_splits > 1) {
        const size_t rows = (size_t)p.n_splits * n_rows * H_q;
        p.off_ml = rows * kPrD * 4;
        p.ws_bytes = (p.off_ml + rows * 8 + 255) / 256 * 256;
    }
    return p;
}

cudaError_t launch_attend_prompt(const PromptArgs& a, const PromptPlan& p, cudaStream_t stream) {
    PrArgs args;
    args.a = a;
    if (!tensor_map_rows_bf16(&args.q, a.q, a.n_rows, a.H_kv, a.G, a.q_stride, a.tile_tokens) ||
        !tensor_map_rows_bf16(&args.k, a.k, a.total_tokens, a.H_kv, 0, a.k_stride, kPrKeys) ||
        !tensor_map_rows_bf16(&args.v, a.v, a.total_tokens, a.H_kv, 0, a.v_stride, kPrKeys))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_smem(attend_prompt_kernel, kPrSmem, allowed);
    if (e != cudaSuccess) return e;
    e = launch_pdl(attend_prompt_kernel, dim3((unsigned)((int64_t)p.slots * a.H_kv * p.n_splits)), dim3(kPrThreads), kPrSmem,
                   stream, 0, args);
    if (e != cudaSuccess || p.n_splits == 1) return e;
    const int64_t warps = (int64_t)a.n_rows * a.H_q;
    return launch_pdl(prompt_merge_kernel, dim3((unsigned)((warps + kPmWarps - 1) / kPmWarps)), dim3(kPmWarps * kWarp), 0,
                      stream, 0, a);
}

}  // namespace lsa
