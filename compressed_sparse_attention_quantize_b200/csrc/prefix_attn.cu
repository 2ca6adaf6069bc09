// Attention of a batch over a prefix that its requests share, on the tensor cores.
//
// Rows (requests' query tokens) come in groups; a group's rows all attend to every entry of the
// group's prefix, n packed FP4 entries of the main cache (keys = values = the 512-wide latent,
// [B] page "DeepSeek V4.1 Flash 如何靠压缩 KV 缓存实现小模型干翻大模型", sections "CSA2：三层压缩一次吃满"
// and "FP4 量化 + Bounded Replay"), contiguous or in pages.  For query (row, head):
//     z_j = softmax_scale * (q . v_j),  j < n;   out = softmax over {z_j} and the row's own part
// where the own part is the fp32 output and log-sum-exp of another attention (csa2_sparse_attn over
// the request's own entries and window), or nothing.
//
// Three launches:
//  1. prefix_prep_kernel  every prefix entry once, to fp16 (E2M1 x E4M3 is exact in fp16), in a
//     padded array of the workspace, through the block table; the queries to fp16, each row times
//     a power of two that puts its largest element in [2^13, 2^14) (exact for all elements within
//     2^27 of it, and a row of infinities or NaNs spoils no other); the groups' tile counts.
//  2. prefix_attn_kernel  a persistent CTA per SM.  The work is the list of (64 queries, 128 keys)
//     tiles, all key tiles of one query tile after the other; CTA i takes the i-th equal share, so
//     every SM has the same number of tiles, and a query tile is cut at most where shares meet.
//     Each piece leaves a partial (maxima, sums, fp32 output).
//  3. prefix_merge_kernel  partials of a query in share order, then the own part: a fixed order.
//
// Tile arithmetic, as in csa2_sparse_attn's kernel, with the entries already fp16:
//   S^T[key, query] = V . Q^T     M=128 keys, N=64 queries, K=512: A = V (K-major), B = Q (K-major)
//   softmax                       16 warps: one key per thread, 16 queries; running maxima that move
//                                 only when some logit exceeds them by 2^8; sums of the unrounded fp32
//                                 weights, per key in registers until the end
//   O^T[chan, query] += V^T.P^T   four blocks of M=128 channels, N=64, K=128 keys: the same V bytes
// P is rounded to fp16 with the weights scaled to at most 2^15 (the maximum itself to 2^7), so weights
// down to 2^-21 of the maximum keep 11 bits and the rest an absolute 2^-32: the rounding is at most
// 2^-12 of sum_j p_j |v_j| / sum_j p_j plus n 2^-32 max |v|.
//
// Bound: the tensor pipe at N=64, where the A operand's shared-memory reads cap it at 67% (48 cycles
// per M=128, N=64, K=16 MMA), plus the softmax between a tile's two products, which one V buffer of
// 128 KB cannot overlap.  Channel blocks of V are refilled one by one as the second product frees them.
// Every wait is bounded: on expiry the CTA records CSA2_ERR_TIMEOUT, drains, frees TMEM and exits.
#include "common.cuh"
#include "tc_ptx.cuh"

namespace csa2 {
namespace pfx {

constexpr int kQ = 64;                     // queries per tile (MMA N)
constexpr int kTile = 128;                 // keys per tile (MMA M)
constexpr int kBlocks = 4;                 // 128-channel blocks
constexpr int kRegion = 64;                // channels of a 128-byte swizzled row
constexpr int kQRegion = kQ * 128;         // 8 KB
constexpr int kVRegion = kTile * 128;      // 16 KB
constexpr int kQBytes = 8 * kQRegion;
constexpr int kVBytes = 8 * kVRegion;
constexpr int kPBytes = kTile * kQ * 2;
constexpr int kThreads = 576;              // copies, MMA issuer, 16 softmax warps
constexpr int kWorkerWarps = 16;
constexpr int kCols = 16;                  // queries per softmax warp
constexpr int kTmemCols = 512;
constexpr int kOCol = 128;                 // O^T accumulators; S^T at column 0
constexpr float kShift = 7.0f;             // log2 of the weight of the running maximum
constexpr float kLag = 8.0f;               // log2 units a logit may exceed the running maximum by
constexpr float kOver = 32768.0f;          // a weight above 2^(kShift + kLag): the maximum moves
constexpr int kPartFloats = 2 * kQ + kQ * kLatent;

// Per group, in the workspace (written by the first launch): first query row, first query tile and
// first work item; entry [G] holds the totals.
struct Group {
    int32_t row0, rows;
    int32_t n;                             // prefix entries
    int32_t pad;
    int64_t tile0, work0;
};

struct Args {
    const uint16_t *q;
    int rows, H, G;
    const int32_t *row_start;
    const uint8_t *kv;
    int64_t kv_row_stride, kv_rows;
    const int64_t *seq_start;
    const int32_t *table;
    int max_pages, page_entries;
    const int32_t *n_prefix;
    int64_t max_n, n_pad;
    float scale_log2;
    const float *own_out, *own_lse;
    void *out;
    int out_dtype;
    float *lse;
    // workspace
    Group *groups;                         // [G + 1]
    __half *v;                             // [G][n_pad][512]
    uint8_t *valid;                        // [G][n_pad]
    __half *qh;                            // [tiles][64][512]
    float *qs;                             // [tiles][64]: logit per unit of S
    float *parts;                          // [CTAs + tiles][kPartFloats]
    int64_t max_tiles;
    int ctas;
};

// ---------------------------------------------------------------------------------------------
// 1. entries and queries to fp16
// ---------------------------------------------------------------------------------------------
constexpr int kPrepThreads = 256;

// Groups' first rows, tiles and work items into shared memory: one warp, 32 groups at a time.
CSA2_D void scan_groups(const Args &a, Group *out, int lane, bool report) {
    int64_t tile0 = 0, work0 = 0;
    int32_t reached = 0;                                 // largest row_start so far
    for (int g0 = 0; g0 < a.G; g0 += 32) {
        const int g = g0 + lane;
        Group x{0, 0, 0, 0, 0, 0};
        int64_t tiles = 0, work = 0;
        bool bad = false;
        if (g < a.G) {
            const int lo = a.row_start[g], hi = a.row_start[g + 1], n = a.n_prefix[g];
            bad = lo < 0 || hi < lo || hi > a.rows || n < 0 || n > a.max_n;
            x.row0 = lo;
            x.rows = hi - lo;
            x.n = n;
        }
        // groups keep to the rows behind the ones before them: a group that breaks the contract has none
        int32_t m = g < a.G ? x.row0 : 0;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int32_t o = __shfl_up_sync(0xffffffffu, m, off);
            if (lane >= off) m = max(m, o);
        }
        m = max(m, reached);
        reached = __shfl_sync(0xffffffffu, m, 31);
        if (g < a.G) {
            bad |= x.row0 < m;
            if (bad) x.rows = x.n = 0;
            x.row0 = min(m, a.rows);
            tiles = ((int64_t)x.rows * a.H + kQ - 1) / kQ;
            work = tiles * ((x.n + kTile - 1) / kTile);
        }
        if (report && bad) raise_device_error(CSA2_ERR_SHAPE);
        int64_t ti = tiles, wi = work;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t t2 = __shfl_up_sync(0xffffffffu, ti, off), w2 = __shfl_up_sync(0xffffffffu, wi, off);
            if (lane >= off) { ti += t2; wi += w2; }
        }
        x.tile0 = tile0 + ti - tiles;
        x.work0 = work0 + wi - work;
        if (g < a.G) out[g] = x;
        tile0 += __shfl_sync(0xffffffffu, ti, 31);
        work0 += __shfl_sync(0xffffffffu, wi, 31);
    }
    if (lane == 0) out[a.G] = Group{a.rows, 0, 0, 0, tile0, work0};
}

// The group whose [first, next first) holds x, by a key of the groups; the last group at or below x.
// Groups without work share their first item with the next: the last one is taken.
template <typename Key>
CSA2_D int find_group(const Group *gr, int G, int64_t x, Key key) {
    int lo = 0, hi = G;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (key(gr[mid]) <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPrepThreads) prefix_prep_kernel(const Args a) {
    extern __shared__ __align__(16) uint8_t smem[];
    Group *gr = reinterpret_cast<Group *>(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) scan_groups(a, gr, lane, blockIdx.x == 0);
    __syncthreads();
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i <= a.G; i += kPrepThreads) a.groups[i] = gr[i];
    const int64_t nwarps = (int64_t)gridDim.x * (kPrepThreads / 32);
    const int64_t w0 = (int64_t)blockIdx.x * (kPrepThreads / 32) + warp;

    // entries: a warp each, a lane per 16-channel block; rows up to the end of the last key tile
    for (int64_t w = w0; w < (int64_t)a.G * a.n_pad; w += nwarps) {
        const int g = (int)(w / a.n_pad);
        const int64_t j = w - (int64_t)g * a.n_pad;
        const int n = gr[g].rows > 0 ? gr[g].n : 0;
        if (j >= ((int64_t)n + kTile - 1) / kTile * kTile) continue;
        int64_t row = -1;
        if (j < n) {
            if (a.table) {
                const int64_t p = j / a.page_entries;
                const int32_t page = p < a.max_pages ? a.table[(int64_t)g * a.max_pages + p] : -1;
                row = page < 0 ? -1 : (int64_t)page * a.page_entries + (j - p * a.page_entries);
            } else {
                row = a.seq_start[g] + j;
            }
            if (row < 0 || row >= a.kv_rows) {
                row = -1;
                if (lane == 0) raise_device_error(CSA2_ERR_INVALID_ARG);
            }
        }
        uint4 o0 = make_uint4(0u, 0u, 0u, 0u), o1 = o0;
        if (row >= 0) {
            const uint8_t *p = a.kv + row * a.kv_row_stride;
            const uint2 c = __ldg(reinterpret_cast<const uint2 *>(p) + lane);
            const uint32_t s = ptx::e4m3x2_to_f16x2((uint16_t)__ldg(p + 256 + lane));
            const uint32_t ss = __byte_perm(s, 0, 0x1010);
            uint32_t h[4];
            ptx::e2m1x8_to_f16x8(c.x, h);
            o0 = make_uint4(ptx::hmul2_u32(h[0], ss), ptx::hmul2_u32(h[1], ss), ptx::hmul2_u32(h[2], ss),
                            ptx::hmul2_u32(h[3], ss));
            ptx::e2m1x8_to_f16x8(c.y, h);
            o1 = make_uint4(ptx::hmul2_u32(h[0], ss), ptx::hmul2_u32(h[1], ss), ptx::hmul2_u32(h[2], ss),
                            ptx::hmul2_u32(h[3], ss));
        }
        uint4 *dst = reinterpret_cast<uint4 *>(a.v + ((int64_t)g * a.n_pad + j) * kLatent) + lane * 2;
        dst[0] = o0;
        dst[1] = o1;
        if (lane == 0) a.valid[(int64_t)g * a.n_pad + j] = row >= 0 ? 1 : 0;
    }

    // queries: a warp each, 16 channels a lane; places past a group's last query are zero
    const int64_t places = gr[a.G].tile0 * kQ;
    for (int64_t w = w0; w < places; w += nwarps) {
        const int64_t tile = w / kQ;
        const int g = find_group(gr, a.G, tile, [](const Group &x) { return x.tile0; });
        const int64_t i = w - gr[g].tile0 * kQ;          // query of the group
        uint4 u0 = make_uint4(0u, 0u, 0u, 0u), u1 = u0;
        if (i < (int64_t)gr[g].rows * a.H) {
            const uint4 *src = reinterpret_cast<const uint4 *>(a.q + ((int64_t)gr[g].row0 * a.H + i) * kLatent) + lane * 2;
            u0 = __ldg(src);
            u1 = __ldg(src + 1);
        }
        const uint32_t x[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
        uint32_t top = 0u;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max(top, max(x[k] & 0x7FFFu, (x[k] >> 16) & 0x7FFFu));
        top = __reduce_max_sync(0xffffffffu, top);
        const int e = (int)(top >> 7);                   // biased exponent of the largest element
        const int up = top == 0u ? 0 : min(13 - (max(e, 1) - 127), 126);
        const float mul = exp2f((float)up);
        uint32_t o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const __half2 h = __floats2half2_rn(__uint_as_float(x[k] << 16) * mul, __uint_as_float(x[k] & 0xFFFF0000u) * mul);
            o[k] = *reinterpret_cast<const uint32_t *>(&h);
        }
        uint4 *dst = reinterpret_cast<uint4 *>(a.qh + w * kLatent) + lane * 2;
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
        if (lane == 0) a.qs[w] = a.scale_log2 * exp2f((float)-up);
    }
}

// ---------------------------------------------------------------------------------------------
// 2. tiles
// ---------------------------------------------------------------------------------------------
struct Ctl {
    uint64_t v_full[kBlocks], v_empty[kBlocks];
    uint64_t q_full, s_full, p_full, seg_done, o_free, drain;
    uint32_t tmem_base;
    int abort_flag;
    alignas(16) float2 zm[kQ];             // (read in 16-byte pieces) logit per unit of S, running maximum - kShift
    float alpha[kQ];
    float red[4][kQ];
};
constexpr int kSmemBytes = kQBytes + kVBytes + kPBytes + (int)sizeof(Ctl) + 1024;

// Reduce 16 values over a warp's lanes: afterwards v[0] of lanes c and c + 16 holds the maximum (or sum)
// of element c.
template <bool kSum>
CSA2_D void reduce16(float (&v)[kCols], int lane) {
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
        const float o = __shfl_xor_sync(0xffffffffu, v[i], 16);
        v[i] = kSum ? v[i] + o : fmaxf(v[i], o);
    }
#pragma unroll
    for (int off = 8, n = 8; off >= 1; off >>= 1, n >>= 1) {
        const bool upper = (lane & off) != 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float send = upper ? v[i] : v[i + n];
            const float keep = upper ? v[i + n] : v[i];
            const float got = __shfl_xor_sync(0xffffffffu, send, off);
            v[i] = kSum ? keep + got : fmaxf(keep, got);
        }
    }
}

// A run of key tiles of one query tile: what a CTA does between two changes of Q.
struct Segment {
    int64_t tile;                          // query tile
    int g;
    int k0, k1;                            // key tiles
};

// The segments of work items [u, end), one after the other; every role walks them alike.
struct Walk {
    int64_t u, end;
    CSA2_D bool next(const Args &a, Segment &s) {
        if (u >= end) return false;
        s.g = find_group(a.groups, a.G, u, [](const Group &x) { return x.work0; });
        const Group &gr = a.groups[s.g];
        const int64_t nt = (gr.n + kTile - 1) / kTile;
        const int64_t at = u - gr.work0;
        const int64_t t = at / nt;
        s.tile = gr.tile0 + t;
        s.k0 = (int)(at - t * nt);
        s.k1 = (int)min(nt, s.k0 + (end - u));
        u += s.k1 - s.k0;
        return true;
    }
};
// The CTAs that get a share: no share is empty.
CSA2_D int64_t shares_of(const Args &a, int64_t total) { return min((int64_t)a.ctas, total); }
CSA2_D Walk walk_of(const Args &a, int cta) {
    const int64_t total = a.groups[a.G].work0, shares = shares_of(a, total);
    if (cta >= shares) return {0, 0};
    return {total * cta / shares, total * (cta + 1) / shares};
}

__global__ void __launch_bounds__(kThreads, 1)
prefix_attn_kernel(const Args a, const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap qmap) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *sQ = base, *sV = sQ + kQBytes, *sP = sV + kVBytes;
    Ctl &S = *reinterpret_cast<Ctl *>(sP + kPBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Walk walk = walk_of(a, blockIdx.x);
    if (walk.u >= walk.end) return;                      // uniform: nothing allocated yet

    if (threadIdx.x == 0) {
        for (int i = 0; i < kBlocks; ++i) {
            ptx::mbar_init(&S.v_full[i], 1);
            ptx::mbar_init(&S.v_empty[i], 1);
        }
        ptx::mbar_init(&S.q_full, 1);
        ptx::mbar_init(&S.s_full, 1);
        ptx::mbar_init(&S.p_full, kWorkerWarps);
        ptx::mbar_init(&S.seg_done, 1);
        ptx::mbar_init(&S.o_free, kWorkerWarps);
        ptx::mbar_init(&S.drain, 1);
        S.abort_flag = 0;
        ptx::fence_async_smem();
    }
    if (warp == 1) {
        ptx::tmem_alloc(&S.tmem_base, kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = S.tmem_base;
    volatile int *abort_flag = &S.abort_flag;
    Segment sg;

    if (warp == 0) {
        // ================= copies =================
        if (lane == 0) {
            uint32_t sph = 1, vph = 1;                   // parities: the last segment's end, V's last release
            int uses[kBlocks] = {0, 0, 0, 0}, q_uses = 0;
            bool ok = true;
            while (ok && walk.next(a, sg)) {
                const int32_t y0 = (int32_t)((int64_t)sg.g * a.n_pad);
                for (int kt = sg.k0; ok && kt < sg.k1; ++kt) {
#pragma unroll
                    for (int mb = 0; mb < kBlocks; ++mb) {
                        if (!ok || !ptx::mbar_wait(&S.v_empty[mb], vph, abort_flag)) { ok = false; continue; }
                        ++uses[mb];
                        uint8_t *dst = sV + 2 * mb * kVRegion;
                        ptx::mbar_arrive_expect_tx(&S.v_full[mb], 2 * kVRegion);
                        ptx::tma_load_2d(dst, &vmap, 128 * mb, y0 + kt * kTile, &S.v_full[mb]);
                        ptx::tma_load_2d(dst + kVRegion, &vmap, 128 * mb + kRegion, y0 + kt * kTile, &S.v_full[mb]);
                    }
                    if (!ok) break;
                    vph ^= 1;
                    if (kt == sg.k0) {                   // Q once the last segment's products are done
                        if (!ptx::mbar_wait(&S.seg_done, sph, abort_flag)) { ok = false; break; }
                        sph ^= 1;
                        ptx::mbar_arrive_expect_tx(&S.q_full, kQBytes);
                        for (int r = 0; r < 8; ++r)
                            ptx::tma_load_2d(sQ + r * kQRegion, &qmap, r * kRegion, (int32_t)(sg.tile * kQ), &S.q_full);
                        ++q_uses;
                    }
                }
            }
            // copies in flight land before the CTA leaves (already so unless it gave up early)
#pragma unroll
            for (int mb = 0; mb < kBlocks; ++mb)
                if (uses[mb] > 0) ptx::mbar_wait_drain(&S.v_full[mb], (uses[mb] - 1) & 1);
            if (q_uses > 0) ptx::mbar_wait_drain(&S.q_full, (q_uses - 1) & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ================= MMA issuer =================
        if (lane == 0) {
            constexpr uint32_t idesc_s = ptx::idesc_f16_f32(128, kQ, false, false);
            constexpr uint32_t idesc_pv = ptx::idesc_f16_f32(128, kQ, true, true);
            const uint64_t s_a0 = ptx::sdesc_sw128(ptx::smem_u32(sV), 16, 1024);
            const uint64_t s_b0 = ptx::sdesc_sw128(ptx::smem_u32(sQ), 16, 1024);
            // V read MN-major: 64 channels per 128-byte row, the next 64 one region further; P likewise
            const uint64_t pv_a0 = ptx::sdesc_sw128(ptx::smem_u32(sV), kVRegion, 1024);
            const uint64_t pv_b0 = ptx::sdesc_sw128(ptx::smem_u32(sP), kPBytes, 1024);
            uint32_t ph = 0, sph = 0;
            bool ok = true, seen = false;                // seen: the next block of V was found ready
            while (ok && walk.next(a, sg)) {
                // the last segment's accumulators have been read (the first wait returns at once)
                if (!ptx::mbar_wait(&S.o_free, sph ^ 1, abort_flag) || !ptx::mbar_wait(&S.q_full, sph, abort_flag)) break;
                sph ^= 1;
                ptx::tc_fence_after();
                for (int kt = sg.k0; kt < sg.k1; ++kt) {
#pragma unroll
                    for (int mb = 0; mb < kBlocks; ++mb) {
                        if (!seen && !ptx::mbar_wait(&S.v_full[mb], ph, abort_flag)) { ok = false; break; }
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            // the next block's barrier is polled while the tensor pipe has work: a wait takes
                            // about 150 cycles even when it is over
                            if (k == 7 && mb + 1 < kBlocks) seen = ptx::mbar_test(&S.v_full[(mb + 1) % kBlocks], ph);
                            const int rg = 2 * mb + (k >> 2);
                            ptx::mma_f16_ss(tmem, s_a0 + (uint64_t)(rg * (kVRegion >> 4) + (k & 3) * 2),
                                            s_b0 + (uint64_t)(rg * (kQRegion >> 4) + (k & 3) * 2), idesc_s, (mb | k) != 0);
                        }
                    }
                    if (!ok) break;
                    ptx::mma_commit(&S.s_full);
                    if (!ptx::mbar_wait(&S.p_full, ph, abort_flag)) { ok = false; break; }
                    ptx::tc_fence_after();
                    ph ^= 1;
#pragma unroll
                    for (int mb = 0; mb < kBlocks; ++mb) {
#pragma unroll
                        for (int k = 0; k < kTile / 16; ++k) {
                            if (mb + 1 == kBlocks && k == 7) seen = ptx::mbar_test(&S.v_full[0], ph);
                            ptx::mma_f16_ss(tmem + kOCol + kQ * mb, pv_a0 + (uint64_t)(mb * (2 * kVRegion >> 4) + k * (2048 >> 4)),
                                            pv_b0 + (uint64_t)(k * (2048 >> 4)), idesc_pv, (kt > sg.k0 || k > 0) ? 1u : 0u);
                        }
                        ptx::mma_commit(&S.v_empty[mb]);
                    }
                }
                if (ok) ptx::mma_commit(&S.seg_done);
            }
            // every issued MMA has completed before TMEM is released
            ptx::mma_commit(&S.drain);
            ptx::mbar_wait_drain(&S.drain, 0);
        }
        __syncwarp();
    } else {
        // ================= softmax and partials =================
        // The four warps of a quarter (16 queries, all keys) work together, apart from the others.
        const int sub = warp & 3, quarter = (warp - 2) >> 2;
        const int c0 = quarter * kCols;
        const int wt = (threadIdx.x - 64) & 127;         // thread of the quarter
        const uint32_t bar = 1 + quarter;
        const int t = sub * 32 + lane;                   // key of the tile, and channel of a block
        const uint32_t lane_addr = tmem + ((uint32_t)(sub * 32) << 16);
        uint32_t ph = 0, sph = 0;
        bool bad = false, aborted = false;
        while (!aborted && walk.next(a, sg)) {
            const uint8_t *valid = a.valid + (int64_t)sg.g * a.n_pad + t;
            if (wt < kCols) S.zm[c0 + wt] = make_float2(a.qs[sg.tile * kQ + c0 + wt], -INFINITY);
            ptx::named_barrier(bar, 128);
            float l[kCols];
#pragma unroll
            for (int i = 0; i < kCols; ++i) l[i] = 0.0f;
            bool live_next = valid[(int64_t)sg.k0 * kTile] != 0;
            for (int kt = sg.k0; kt < sg.k1; ++kt) {
                const bool live = live_next;
                if (kt + 1 < sg.k1) live_next = valid[(int64_t)(kt + 1) * kTile] != 0;
                if (!ptx::mbar_wait(&S.s_full, ph, abort_flag)) bad = true;
                ph ^= 1;
                ptx::tc_fence_after();
                uint32_t u[kCols];
                ptx::tmem_ld16(lane_addr + c0, u);
                ptx::tmem_ld_wait();
                // weights under the maxima so far, as the P^T line of this key; the first tile has none
                // yet and goes on to the move below
                float p[kCols];
                auto weights = [&]() {
#pragma unroll
                    for (int c = 0; c < kCols / 8; ++c) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int i = 8 * c + 2 * k;
                            const float4 zm = *reinterpret_cast<const float4 *>(&S.zm[c0 + i]);
                            p[i] = live ? ptx::ex2(fmaf(__uint_as_float(u[i]), zm.x, -zm.y)) : 0.0f;
                            p[i + 1] = live ? ptx::ex2(fmaf(__uint_as_float(u[i + 1]), zm.z, -zm.w)) : 0.0f;
                            const __half2 h = __floats2half2_rn(p[i], p[i + 1]);
                            w[k] = *reinterpret_cast<const uint32_t *>(&h);
                        }
                        *reinterpret_cast<uint4 *>(sP + tc::sw128_off(t, quarter * 2 + c)) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                };
                weights();
                bool over = false;
#pragma unroll
                for (int i = 0; i < kCols; ++i) over |= p[i] > kOver;
                // one barrier decides whether to stop and whether some maximum moves
                if (tc::block_any(over || bad || *abort_flag != 0, bar, 128)) {
                    if (tc::block_any(bad || *abort_flag != 0, bar, 128)) { aborted = true; break; }
                    float v[kCols];
#pragma unroll
                    for (int i = 0; i < kCols; ++i) v[i] = live ? __uint_as_float(u[i]) * S.zm[c0 + i].x : -INFINITY;
                    reduce16<false>(v, lane);
                    if (lane < kCols) S.red[sub][c0 + lane] = v[0];
                    ptx::named_barrier(bar, 128);
                    bool moved = false;
                    if (wt < kCols) {
                        const int c = c0 + wt;
                        const float top = fmaxf(fmaxf(S.red[0][c], S.red[1][c]), fmaxf(S.red[2][c], S.red[3][c]));
                        const float old = S.zm[c].y;     // maximum - kShift
                        float al = 1.0f;
                        if (top > old + (kShift + kLag)) {
                            S.zm[c].y = top - kShift;
                            al = old == -INFINITY ? 0.0f : ptx::ex2(old + kShift - top);
                            moved = kt > sg.k0 && old != -INFINITY;
                        }
                        S.alpha[c] = al;
                    }
                    const bool rescale = tc::block_any(moved, bar, 128);
#pragma unroll
                    for (int i = 0; i < kCols; ++i) l[i] *= S.alpha[c0 + i];
                    weights();
                    // accumulators of queries whose maximum moved: S(kt) completed after the last tile's
                    // second product, so they are at rest
                    if (rescale) {
#pragma unroll 1
                        for (int mb = 0; mb < kBlocks; ++mb) {
                            uint32_t o[kCols];
                            ptx::tmem_ld16(lane_addr + kOCol + kQ * mb + c0, o);
                            ptx::tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < kCols; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * S.alpha[c0 + i]);
                            ptx::tmem_st16(lane_addr + kOCol + kQ * mb + c0, o);
                        }
                        ptx::tmem_st_wait();
                    }
                }
                ptx::fence_async_smem();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&S.p_full);
#pragma unroll
                for (int i = 0; i < kCols; ++i) l[i] += p[i];
            }
            if (aborted) break;
            // ---- the segment's partial ----
            if (!ptx::mbar_wait(&S.seg_done, sph, abort_flag)) bad = true;
            sph ^= 1;
            if (tc::block_any(bad || *abort_flag != 0, bar, 128)) { aborted = true; break; }
            ptx::tc_fence_after();
            float *part = a.parts + (blockIdx.x + sg.tile) * (int64_t)kPartFloats;
            reduce16<true>(l, lane);
            if (lane < kCols) S.red[sub][c0 + lane] = l[0];
            ptx::named_barrier(bar, 128);
            if (wt < kCols) {
                const int c = c0 + wt;
                part[c] = S.zm[c].y;
                part[kQ + c] = (S.red[0][c] + S.red[1][c]) + (S.red[2][c] + S.red[3][c]);
            }
#pragma unroll
            for (int mb = 0; mb < kBlocks; ++mb) {
                uint32_t o[kCols];
                ptx::tmem_ld16(lane_addr + kOCol + kQ * mb + c0, o);
                ptx::tmem_ld_wait();
                float *dst = part + 2 * kQ + c0 * kLatent + mb * 128 + t;
#pragma unroll
                for (int i = 0; i < kCols; ++i) dst[i * kLatent] = __uint_as_float(o[i]);
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&S.o_free);
            ptx::named_barrier(bar, 128);                // the shared maxima are read before they are reset
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------------------------------------
// 3. merge: 128 threads per query, 4 channels each
// ---------------------------------------------------------------------------------------------
__global__ void __launch_bounds__(128) prefix_merge_kernel(const Args a) {
    const int64_t f = blockIdx.x;                        // row * H + head
    const int row = (int)(f / a.H);
    const int g = find_group(a.groups, a.G, row, [](const Group &x) { return (int64_t)x.row0; });
    const Group gr = a.groups[g];
    int64_t c0 = 0, c1 = -1, tile = 0;
    int qi = 0;
    const int64_t total = a.groups[a.G].work0;
    const int64_t nt = (gr.n + kTile - 1) / kTile;
    if (row >= gr.row0 && row < gr.row0 + gr.rows && nt > 0) {
        const int64_t i = f - (int64_t)gr.row0 * a.H;
        tile = gr.tile0 + i / kQ;
        qi = (int)(i % kQ);
        // the shares that hold work items u0 .. u1 of this query tile; share c begins at total c / shares
        const int64_t shares = shares_of(a, total), u0 = gr.work0 + (i / kQ) * nt, u1 = u0 + nt - 1;
        c0 = u0 * shares / total;
        while (total * (c0 + 1) / shares <= u0) ++c0;
        c1 = u1 * shares / total;
        while (total * (c1 + 1) / shares <= u1) ++c1;
    }
    constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
    const float own = a.own_lse ? a.own_lse[f] * kLog2e : -INFINITY;
    float top = own;
    for (int64_t c = c0; c <= c1; ++c) {
        const float *p = a.parts + (c + tile) * (int64_t)kPartFloats;
        if (p[kQ + qi] != 0.0f) top = fmaxf(top, p[qi]);
    }
    float L = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t c = c0; c <= c1; ++c) {
        const float *p = a.parts + (c + tile) * (int64_t)kPartFloats;
        const float ls = p[kQ + qi];
        if (ls == 0.0f) continue;                        // no key of this piece counts
        const float w = exp2f(p[qi] - top);
        L += w * ls;
        const float4 o = *reinterpret_cast<const float4 *>(p + 2 * kQ + qi * kLatent + threadIdx.x * 4);
        acc[0] += w * o.x; acc[1] += w * o.y; acc[2] += w * o.z; acc[3] += w * o.w;
    }
    if (a.own_out && own != -INFINITY) {
        const float w = exp2f(own - top);
        L += w;
        const float4 o = *reinterpret_cast<const float4 *>(a.own_out + f * kLatent + threadIdx.x * 4);
        acc[0] += w * o.x; acc[1] += w * o.y; acc[2] += w * o.z; acc[3] += w * o.w;
    }
    const float inv = L != 0.0f ? 1.0f / L : 0.0f;       // no key at all: 0; a NaN stays one
    const int64_t oi = f * kLatent + threadIdx.x * 4;
    if (a.out_dtype == CSA2_DTYPE_F32) {
        *reinterpret_cast<float4 *>(reinterpret_cast<float *>(a.out) + oi) =
            make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
    } else {
        __nv_bfloat162 *o2 = reinterpret_cast<__nv_bfloat162 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) + oi);
        o2[0] = __floats2bfloat162_rn(acc[0] * inv, acc[1] * inv);
        o2[1] = __floats2bfloat162_rn(acc[2] * inv, acc[3] * inv);
    }
    __syncthreads();                                     // lse may be own_lse
    if (a.lse && threadIdx.x == 0) a.lse[f] = L != 0.0f ? (top + log2f(L)) * kLn2 : -INFINITY;
}

// ---------------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------------
struct Layout {
    int64_t n_pad, max_tiles;
    int ctas;
    size_t groups, v, valid, qh, qs, parts, total;
};
inline Layout layout(int rows, int H, int G, int64_t max_n) {
    Layout l;
    l.n_pad = ceil_div(max_n, (int64_t)kTile) * kTile;
    l.max_tiles = ceil_div((int64_t)rows * H, (int64_t)kQ) + G;
    const int64_t work = l.max_tiles * (l.n_pad / kTile);
    l.ctas = (int)std::max<int64_t>(1, std::min<int64_t>(device_sm_count(), work));
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += (bytes + 1023) / 1024 * 1024;
        return at;
    };
    l.groups = take((size_t)(G + 1) * sizeof(Group));
    l.v = take((size_t)G * l.n_pad * kLatent * 2);
    l.valid = take((size_t)G * l.n_pad);
    l.qh = take((size_t)l.max_tiles * kQ * kLatent * 2);
    l.qs = take((size_t)l.max_tiles * kQ * 4);
    l.parts = take((size_t)(l.ctas + l.max_tiles) * kPartFloats * 4);
    l.total = off + 1024;
    return l;
}

}  // namespace pfx

static SmemLimit g_prefix_smem, g_prefix_prep_smem;

size_t prefix_attn_workspace_bytes(int rows, int H, int G, int64_t max_n) { return pfx::layout(rows, H, G, max_n).total; }

cudaError_t launch_prefix_attn(const uint16_t *q, int rows, int H, const int32_t *row_start, int G, const uint8_t *kv,
                               int64_t kv_row_stride, int64_t kv_rows, const int64_t *seq_start, const int32_t *table,
                               int max_pages, int page_entries, const int32_t *n_prefix, int64_t max_n,
                               float softmax_scale, const float *own_out, const float *own_lse, void *out, int out_dtype,
                               float *lse, void *workspace, cudaStream_t st) {
    const IpkEncodeTiledFn enc = ipk_encode_tiled();
    if (!enc) return cudaErrorNotSupported;
    cudaError_t e = bind_current_context();
    if (e != cudaSuccess) return e;
    const pfx::Layout l = pfx::layout(rows, H, G, max_n);
    uint8_t *ws = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(workspace) + 1023) & ~(uintptr_t)1023);
    pfx::Args a;
    a.q = q; a.rows = rows; a.H = H; a.G = G; a.row_start = row_start;
    a.kv = kv; a.kv_row_stride = kv_row_stride; a.kv_rows = kv_rows;
    a.seq_start = seq_start; a.table = table; a.max_pages = max_pages; a.page_entries = page_entries;
    a.n_prefix = n_prefix; a.max_n = max_n; a.n_pad = l.n_pad;
    a.scale_log2 = softmax_scale * 1.4426950408889634f;
    a.own_out = own_out; a.own_lse = own_lse;
    a.out = out; a.out_dtype = out_dtype; a.lse = lse;
    a.groups = reinterpret_cast<pfx::Group *>(ws + l.groups);
    a.v = reinterpret_cast<__half *>(ws + l.v);
    a.valid = ws + l.valid;
    a.qh = reinterpret_cast<__half *>(ws + l.qh);
    a.qs = reinterpret_cast<float *>(ws + l.qs);
    a.parts = reinterpret_cast<float *>(ws + l.parts);
    a.max_tiles = l.max_tiles;
    a.ctas = l.ctas;

    const int prep_smem = (G + 1) * (int)sizeof(pfx::Group);
    e = ensure_smem_limit(g_prefix_prep_smem, pfx::prefix_prep_kernel, prep_smem);
    if (e != cudaSuccess) return e;
    const int64_t warps = std::max<int64_t>((int64_t)G * l.n_pad, l.max_tiles * pfx::kQ);
    const int64_t blocks = std::min<int64_t>(ceil_div(warps, (int64_t)(pfx::kPrepThreads / 32)), (int64_t)device_sm_count() * 8);
    pfx::prefix_prep_kernel<<<(unsigned)blocks, pfx::kPrepThreads, prep_smem, st>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    int launches = 2;
    if (max_n > 0) {
        CUtensorMap vmap, qmap;
        auto encode = [&](CUtensorMap *m, void *base, int64_t nrows, int box_rows) {
            const cuuint64_t dim[2] = {(cuuint64_t)kLatent, (cuuint64_t)nrows};
            const cuuint64_t strides[1] = {(cuuint64_t)kLatent * 2};
            const cuuint32_t box[2] = {(cuuint32_t)pfx::kRegion, (cuuint32_t)box_rows};
            const cuuint32_t ones[2] = {1, 1};
            return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, base, dim, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
        };
        if (!encode(&vmap, a.v, (int64_t)G * l.n_pad, pfx::kTile) || !encode(&qmap, a.qh, l.max_tiles * pfx::kQ, pfx::kQ))
            return cudaErrorInvalidValue;
        e = ensure_smem_limit(g_prefix_smem, pfx::prefix_attn_kernel, pfx::kSmemBytes);
        if (e != cudaSuccess) return e;
        pfx::prefix_attn_kernel<<<(unsigned)l.ctas, pfx::kThreads, pfx::kSmemBytes, st>>>(a, vmap, qmap);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        launches = 3;
    }
    pfx::prefix_merge_kernel<<<(unsigned)((int64_t)rows * H), 128, 0, st>>>(a);
    note_launches(launches);
    return cudaGetLastError();
}

}  // namespace csa2
