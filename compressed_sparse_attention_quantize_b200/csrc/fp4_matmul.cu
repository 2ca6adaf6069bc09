// Product of two microscaled FP4 matrices on the tensor cores:
//     out[m][n] = alpha * sum_b sa[m][b] * sb[n][b] * sum_{k in block b} a[m][k] * b[n][k]
// with E2M1 codes and one E4M3 scale per 16 channels or one E8M0 scale per 32, both operands as
// csa2_quantize_kv leaves them (rows of codes, rows of scale bytes), fp32 accumulation.
//
// One tile = 128 rows of the "left" matrix (the MMA's M: TMEM lanes) x NT rows of the "right" one
// (the MMA's N: TMEM columns).  Left and right are A and B, or B and A when there are few rows in
// A (a decode batch): then the weights fill the 128 lanes and the batch takes NT = 16 .. 64
// columns, instead of padding the batch to 128 rows.  Per 256 channels (a stage):
//   warp 0        the codes of both operands by tensor copies (128-byte rows, 128-byte swizzle; rows
//                 and channels past the end arrive as zeros)
//   warps 2-5     the scale bytes, from their rows in global memory to the 512-byte blocks that
//                 tcgen05.cp reads: byte k of row r at (r % 32) * 16 + (r / 32) * 4 + k, so 128 rows x
//                 4 scales become 32 lanes x 4 columns.  Scales past the end are zero: a NaN there
//                 would survive the zero codes.
//   warp 1        one thread: tcgen05.cp of the stage's scales into TMEM columns of the stage (they
//                 are rewritten only after the stage's MMAs have completed), then four MMAs
//                 (kind::mxf4nvf4 with 16-channel, kind::mxf4 with 32-channel scales; K = 64 each)
//   warps 6-13    epilogue: TMEM -> registers -> global
// A CTA walks over tiles; the copies and scales of the next tile run while the epilogue drains
// the last.  Few tiles and a long K are split over a cluster: each CTA takes a run of stages, leaves
// its fp32 tile in its shared memory, and every CTA adds up a share of the columns over the
// cluster in rank order (no second launch, no atomics: the result does not depend on timing).
// Every wait is bounded: on expiry the CTA records CSA2_ERR_TIMEOUT, drains, frees TMEM and exits.
#include "common.cuh"
#include "tc_ptx.cuh"

namespace csa2 {
namespace fmm {

constexpr int kM = 128;                    // left rows per tile
constexpr int kKTile = 256;                // channels per stage: 128 code bytes a row
constexpr int kSteps = 4;                  // MMAs per stage (K = 64)
constexpr int kMaxNT = 256;
constexpr int kThreads = 448;
constexpr int kSfThreads = 128;
constexpr int kEpiThreads = 256;
constexpr int kMaxStages = 8;
constexpr int kMaxSplits = 8;              // portable cluster size

struct Operand {
    const uint8_t *scales;
    int64_t scale_stride;
    int64_t rows;
    bool vec;                              // 16-byte (E4M3) or 8-byte (E8M0) aligned scale rows
};

struct Args {
    Operand left, right;
    int K, nblk;                           // channels, scale blocks per row
    int NT, stages, splits;
    int tiles_l;                           // left tiles
    int64_t tiles;                         // all tiles
    int ktiles;                            // stages of the whole K
    uint32_t tmem_cols, acc_cols;
    bool swap;                             // left = B: out is written transposed
    float alpha;
    void *out;
    int64_t out_stride;
    bool out_vec;                          // 16-byte stores along n allowed
};

struct Ctl {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full, acc_empty, drain;
    uint32_t tmem_base;
    int abort_flag;
};

CSA2_HD constexpr uint32_t idesc_fp4(int N, bool e8m0, int sf_id) {
    return ((uint32_t)sf_id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((e8m0 ? 1u : 0u) << 23) |
           ((uint32_t)(kM >> 4) << 24) | ((uint32_t)sf_id << 29);
}

template <bool MX>
CSA2_D void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t acc) {
    if (MX)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.block16 [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc) : "memory");
}
// 32 rows x 16 bytes of shared memory into 32 lanes x 4 columns of TMEM, repeated for the four
// lane quarters.
CSA2_D void cp_scales(uint32_t taddr, uint64_t sdesc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
CSA2_D uint64_t sdesc_scales(uint32_t saddr) {           // no swizzle, 8-row groups 128 bytes apart
    uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(16u >> 4) << 16;
    d |= (uint64_t)(128u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    return d;
}
CSA2_D void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
CSA2_D float ld_peer(const float *p, uint32_t rank) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ptx::smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// Scale bytes of one row for one stage: 16 (E4M3) or 8 (E8M0), zeros past the row's or the
// matrix's end.
template <bool MX>
CSA2_D uint4 load_scales(const Operand &o, int64_t row, int kt, int nblk) {
    constexpr int kPer = MX ? 8 : 16;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    const int b0 = kt * kPer;
    if (row >= o.rows || b0 >= nblk) return v;
    const uint8_t *p = o.scales + row * o.scale_stride + b0;
    if (o.vec && b0 + kPer <= nblk) {
        if (MX) {
            const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
            v.x = u.x;
            v.y = u.y;
        } else {
            v = __ldg(reinterpret_cast<const uint4 *>(p));
        }
    } else {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        const int n = min(kPer, nblk - b0);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (i < n) w[i >> 2] |= (uint32_t)__ldg(p + i) << (8 * (i & 3));
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return v;
}

struct TileAt {
    int64_t l0, r0;
};
CSA2_D TileAt tile_at(const Args &a, int64_t t) {
    return {(t % a.tiles_l) * kM, (t / a.tiles_l) * a.NT};
}

// 32 consecutive columns (right rows r .. r+31) of left row l.
template <bool BF16>
CSA2_D void store_cols(const Args &a, int64_t l, int64_t r, const float (&v)[32]) {
    if (l >= a.left.rows) return;
    if (a.swap) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            if (r + i >= a.right.rows) break;
            const int64_t at = (r + i) * a.out_stride + l;
            if (BF16)
                reinterpret_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(v[i]);
            else
                reinterpret_cast<float *>(a.out)[at] = v[i];
        }
        return;
    }
    const int64_t at = l * a.out_stride + r;
    if (a.out_vec && r + 32 <= a.right.rows) {
        if (BF16) {
            uint4 *p = reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) + at);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(v[8 * q + 2 * k], v[8 * q + 2 * k + 1]);
                    w[k] = *reinterpret_cast<const uint32_t *>(&h);
                }
                p[q] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        } else {
            float4 *p = reinterpret_cast<float4 *>(reinterpret_cast<float *>(a.out) + at);
#pragma unroll
            for (int q = 0; q < 8; ++q) p[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        if (r + i >= a.right.rows) break;
        if (BF16)
            reinterpret_cast<__nv_bfloat16 *>(a.out)[at + i] = __float2bfloat16_rn(v[i]);
        else
            reinterpret_cast<float *>(a.out)[at + i] = v[i];
    }
}

template <bool MX, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
fp4_matmul_kernel(const Args a, const __grid_constant__ CUtensorMap lmap, const __grid_constant__ CUtensorMap rmap) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    constexpr int kCells = MX ? 2 : 4;                   // 512-byte scale blocks per 128 rows and stage
    const int NT = a.NT;
    const int r_groups = (NT + 127) / 128;               // scale blocks of the right rows
    const int l_bytes = kM * 128, r_bytes = NT * 128;
    const int sf_bytes = kCells * 512 * (1 + r_groups);
    const int stage_bytes = l_bytes + ((r_bytes + 1023) & ~1023) + ((sf_bytes + 1023) & ~1023);
    Ctl &S = *reinterpret_cast<Ctl *>(base + (size_t)a.stages * stage_bytes);
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;

    const int rank = a.splits > 1 ? (int)(blockIdx.x % a.splits) : 0;
    const int64_t first = blockIdx.x / a.splits, step = gridDim.x / a.splits;
    const int k0 = (int)((int64_t)a.ktiles * rank / a.splits), k1 = (int)((int64_t)a.ktiles * (rank + 1) / a.splits);

    if (t == 0) {
        for (int i = 0; i < a.stages; ++i) {
            ptx::mbar_init(&S.full[i], 1 + kSfThreads);
            ptx::mbar_init(&S.empty[i], 1);
        }
        ptx::mbar_init(&S.acc_full, 1);
        ptx::mbar_init(&S.acc_empty, kEpiThreads);
        ptx::mbar_init(&S.drain, 1);
        S.abort_flag = 0;
        ptx::fence_async_smem();
    }
    if (warp == 0) {
        ptx::tmem_alloc(&S.tmem_base, a.tmem_cols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = S.tmem_base;
    volatile int *abort_flag = &S.abort_flag;

    if (warp == 0) {
        // ================= codes =================
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (int64_t tile = first; ok && tile < a.tiles; tile += step) {
                const TileAt at = tile_at(a, tile);
                for (int kt = k0; kt < k1; ++kt, ++it) {
                    const int st = it % a.stages;
                    if (it >= a.stages && !ptx::mbar_wait(&S.empty[st], ((it / a.stages) - 1) & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    uint8_t *sl = base + (size_t)st * stage_bytes, *sr = sl + l_bytes;
                    ptx::mbar_arrive_expect_tx(&S.full[st], (uint32_t)(l_bytes + r_bytes));
                    ptx::tma_load_2d(sl, &lmap, kt * 128, (int32_t)at.l0, &S.full[st]);
                    ptx::tma_load_2d(sr, &rmap, kt * 128, (int32_t)at.r0, &S.full[st]);
                }
            }
            // the copies still in flight land before the CTA leaves
            for (int i = it > a.stages ? it - a.stages : 0; i < it; ++i)
                ptx::mbar_wait_drain(&S.full[i % a.stages], (i / a.stages) & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ================= MMA issuer =================
        if (lane == 0) {
            const uint32_t sf0 = tmem + a.acc_cols;
            const uint32_t sf_cols = (uint32_t)(kCells * 4 * (1 + r_groups));   // per stage
            int it = 0, n = 0;
            bool ok = true;
            for (int64_t tile = first; ok && tile < a.tiles; tile += step, ++n) {
                if (n > 0 && !ptx::mbar_wait(&S.acc_empty, (n - 1) & 1, abort_flag)) break;
                ptx::tc_fence_after();
                for (int kt = k0; kt < k1; ++kt, ++it) {
                    const int st = it % a.stages;
                    if (!ptx::mbar_wait(&S.full[st], (it / a.stages) & 1, abort_flag)) { ok = false; break; }
                    ptx::tc_fence_after();
                    const uint32_t sl = ptx::smem_u32(base + (size_t)st * stage_bytes), sr = sl + l_bytes;
                    const uint32_t ss = sr + ((r_bytes + 1023) & ~1023);
                    const uint32_t sfa = sf0 + st * sf_cols, sfb = sfa + kCells * 4;
                    // left blocks one after the other; right blocks of the same channels side by side
                    for (int c = 0; c < kCells; ++c) {
                        cp_scales(sfa + 4 * c, sdesc_scales(ss + 512 * c));
                        for (int g = 0; g < r_groups; ++g)
                            cp_scales(sfb + 4 * (c * r_groups + g), sdesc_scales(ss + 512 * (kCells * (1 + g) + c)));
                    }
                    const uint64_t da = ptx::sdesc_sw128(sl, 16, 1024), db = ptx::sdesc_sw128(sr, 16, 1024);
#pragma unroll
                    for (int k = 0; k < kSteps; ++k) {
                        const int c = MX ? k >> 1 : k, id = MX ? (k & 1) * 2 : 0;
                        mma_fp4<MX>(tmem, da + 2 * k, db + 2 * k, idesc_fp4(NT, MX, id), sfa + 4 * c,
                                    sfb + 4 * c * r_groups, (kt > k0 || k > 0) ? 1u : 0u);
                    }
                    ptx::mma_commit(&S.empty[st]);
                }
                if (ok) ptx::mma_commit(&S.acc_full);
            }
            // every issued MMA has completed before TMEM is released
            ptx::mma_commit(&S.drain);
            ptx::mbar_wait_drain(&S.drain, 0);
        }
        __syncwarp();
    } else if (warp < 6) {
        // ================= scales =================
        const int r = t - 64;                            // 0..127: a left row and up to two right rows
        const uint32_t cell = (uint32_t)((r & 31) * 16 + (r >> 5) * 4);
        int it = 0;
        bool ok = true;
        for (int64_t tile = first; ok && tile < a.tiles; tile += step) {
            const TileAt at = tile_at(a, tile);
            const int64_t rl = at.l0 + r;
            auto load = [&](int kt, uint4 (&v)[3]) {
                v[0] = load_scales<MX>(a.left, rl, kt, a.nblk);
                v[1] = r < NT ? load_scales<MX>(a.right, at.r0 + r, kt, a.nblk) : make_uint4(0u, 0u, 0u, 0u);
                v[2] = r + 128 < NT ? load_scales<MX>(a.right, at.r0 + 128 + r, kt, a.nblk) : make_uint4(0u, 0u, 0u, 0u);
            };
            uint4 cur[3], nxt[3];
            if (k0 < k1) load(k0, cur);
            for (int kt = k0; kt < k1; ++kt, ++it) {
                const int st = it % a.stages;
                if (kt + 1 < k1) load(kt + 1, nxt);
                if (it >= a.stages && !ptx::mbar_wait(&S.empty[st], ((it / a.stages) - 1) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                uint8_t *ss = base + (size_t)st * stage_bytes + l_bytes + ((r_bytes + 1023) & ~1023);
#pragma unroll
                for (int g = 0; g < 3; ++g) {
                    if (g > r_groups) break;
                    const uint32_t w[4] = {cur[g].x, cur[g].y, cur[g].z, cur[g].w};
#pragma unroll
                    for (int c = 0; c < kCells; ++c)
                        *reinterpret_cast<uint32_t *>(ss + 512 * (kCells * g + c) + cell) = w[c];
                }
                ptx::fence_async_smem();
                ptx::mbar_arrive(&S.full[st]);
#pragma unroll
                for (int g = 0; g < 3; ++g) cur[g] = nxt[g];
            }
        }
    } else {
        // ================= epilogue =================
        const int half = (warp - 6) >> 2, sub = warp & 3;
        const uint32_t lane_addr = tmem + ((uint32_t)(sub * 32) << 16);
        const int64_t lrow = sub * 32 + lane;
        int n = 0;
        for (int64_t tile = first; tile < a.tiles; tile += step, ++n) {
            const TileAt at = tile_at(a, tile);
            if (!ptx::mbar_wait(&S.acc_full, n & 1, abort_flag)) break;
            ptx::tc_fence_after();
            if (a.splits > 1) {
                // this CTA's share of K, column by column: every copy into the stages has been
                // consumed, so their memory is free
                float *part = reinterpret_cast<float *>(base);
                for (int c0 = half * 16; c0 < NT; c0 += 32) {
                    uint32_t u[16];
                    ptx::tmem_ld16(lane_addr + c0, u);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) part[(c0 + i) * kM + lrow] = __uint_as_float(u[i]);
                }
            } else {
                for (int c0 = half * 32; c0 < NT; c0 += 64) {
                    float v[32];
                    {
                        uint32_t u[32];
                        if (c0 + 32 <= NT) {
                            ptx::tmem_ld32(lane_addr + c0, u);
                        } else {                         // NT is a multiple of 16
                            uint32_t w[16];
                            ptx::tmem_ld16(lane_addr + c0, w);
#pragma unroll
                            for (int i = 0; i < 16; ++i) { u[i] = w[i]; u[16 + i] = 0u; }
                        }
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(u[i]) * a.alpha;
                    }
                    // a tile 16 columns wide: the columns past it belong to the next tile
                    if (c0 + 32 > NT) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int64_t l = at.l0 + lrow, rr = at.r0 + c0 + i;
                            if (l < a.left.rows && rr < a.right.rows) {
                                const int64_t o = a.swap ? rr * a.out_stride + l : l * a.out_stride + rr;
                                if (BF16)
                                    reinterpret_cast<__nv_bfloat16 *>(a.out)[o] = __float2bfloat16_rn(v[i]);
                                else
                                    reinterpret_cast<float *>(a.out)[o] = v[i];
                            }
                        }
                    } else {
                        store_cols<BF16>(a, at.l0 + lrow, at.r0 + c0, v);
                    }
                }
            }
            ptx::tc_fence_before();
            ptx::mbar_arrive(&S.acc_empty);
        }
    }
    if (a.splits > 1) {
        // every CTA of the cluster gets here, whatever happened before: no wait can be left behind
        __syncwarp();
        cluster_sync();
        if (*abort_flag == 0 && warp >= 6) {
            const TileAt at = tile_at(a, first);
            const int et = t - 192;
            const float *part = reinterpret_cast<const float *>(base);
            const int c0 = NT * rank / a.splits, c1 = NT * (rank + 1) / a.splits;
            const int lr = et & (kM - 1);
            for (int c = c0 + (et >> 7); c < c1; c += kEpiThreads / kM) {
                float v[kMaxSplits];
#pragma unroll
                for (int s = 0; s < kMaxSplits; ++s)
                    if (s < a.splits) v[s] = ld_peer(part + c * kM + lr, s);
                float sum = 0.0f;
#pragma unroll
                for (int s = 0; s < kMaxSplits; ++s)
                    if (s < a.splits) sum += v[s];
                sum *= a.alpha;
                const int64_t l = at.l0 + lr, rr = at.r0 + c;
                if (l < a.left.rows && rr < a.right.rows) {
                    const int64_t o = a.swap ? rr * a.out_stride + l : l * a.out_stride + rr;
                    if (BF16)
                        reinterpret_cast<__nv_bfloat16 *>(a.out)[o] = __float2bfloat16_rn(sum);
                    else
                        reinterpret_cast<float *>(a.out)[o] = sum;
                }
            }
        }
        __syncwarp();
        cluster_sync();                                  // peers have read this CTA's shared memory
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, a.tmem_cols);
    }
}

struct Plan {
    bool swap;
    int NT, splits, stages;
};

inline int stage_bytes_of(bool mx, int NT) {
    const int cells = mx ? 2 : 4;
    return kM * 128 + ((NT * 128 + 1023) & ~1023) + ((cells * 512 * (1 + (NT + 127) / 128) + 1023) & ~1023);
}

// Estimated finish time, in SM cycles, of the candidates (operand order, tile width, K splits); the
// smallest wins.
inline Plan make_plan(bool mx, int64_t M, int64_t N, int K, int nsm) {
    Plan best{false, 128, 1, 4};
    double best_t = 1e300;
    const int ktiles = (K + kKTile - 1) / kKTile;
    for (int sw = 0; sw < 2; ++sw)
        for (int NT = 16; NT <= kMaxNT; NT *= 2)
            for (int sp = 1; sp <= kMaxSplits; sp *= 2) {
                const int64_t L = sw ? N : M, R = sw ? M : N;
                if (sp > 1 && (sp > ktiles || NT > 128)) continue;
                const int64_t tiles = ceil_div(L, kM) * ceil_div(R, NT);
                const int64_t units = tiles * sp;
                if (sp > 1 && units > nsm) continue;
                const double kt = (double)ktiles / sp;
                // a stage: the MMAs (128 x NT x 64 in NT / 2 cycles), or its bytes through shared memory
                const double stage = std::max(2.0 * NT, (kM + NT) * 144.0 / 48.0);
                const double waves = (double)ceil_div(units, (int64_t)nsm);
                const double epi = sw ? 6.0 * NT : 4.0 * NT;
                const double t = 2500.0 + waves * (kt * stage + 800.0 + epi) + (sp > 1 ? 1200.0 : 0.0);
                if (t < best_t) {
                    best_t = t;
                    best = Plan{sw != 0, NT, sp, 0};
                }
            }
    const int sb = stage_bytes_of(mx, best.NT);
    int st = (int)((227 * 1024 - 2048 - (int)sizeof(Ctl)) / sb);
    const int cells = mx ? 2 : 4;
    const int sf_cols = cells * 4 * (1 + (best.NT + 127) / 128);
    const int acc = best.NT < 32 ? 32 : best.NT;
    st = std::min(st, (512 - acc) / sf_cols);
    best.stages = std::min(st, kMaxStages);
    return best;
}

}  // namespace fmm

static SmemLimit g_fmm_smem[4];

template <bool MX, bool BF16>
static cudaError_t launch_fmm(const fmm::Args &a, const CUtensorMap &lm, const CUtensorMap &rm, int smem, unsigned grid,
                              cudaStream_t st) {
    cudaError_t e = ensure_smem_limit(g_fmm_smem[(MX ? 2 : 0) + (BF16 ? 1 : 0)], fmm::fp4_matmul_kernel<MX, BF16>, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(fmm::kThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)a.splits;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = a.splits > 1 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, fmm::fp4_matmul_kernel<MX, BF16>, a, lm, rm);
    note_launches(1);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_fp4_matmul(int fmt, const uint8_t *a_codes, int64_t a_code_stride, const uint8_t *a_scales,
                              int64_t a_scale_stride, const uint8_t *b_codes, int64_t b_code_stride,
                              const uint8_t *b_scales, int64_t b_scale_stride, int64_t M, int64_t N, int K, float alpha,
                              void *out, int out_dtype, int64_t out_stride, cudaStream_t st) {
    const bool mx = fmt == CSA2_FMT_MXFP4_E2M1_E8M0S32;
    const fmm::Plan p = fmm::make_plan(mx, M, N, K, device_sm_count());
    const IpkEncodeTiledFn enc = ipk_encode_tiled();
    if (!enc) return cudaErrorNotSupported;
    cudaError_t e = bind_current_context();
    if (e != cudaSuccess) return e;
    const uintptr_t sf_mask = mx ? 7u : 15u;
    auto operand = [&](const uint8_t *s, int64_t stride, int64_t rows) {
        return fmm::Operand{s, stride, rows, ((reinterpret_cast<uintptr_t>(s) | (uintptr_t)stride) & sf_mask) == 0};
    };
    auto encode = [&](CUtensorMap *m, const uint8_t *codes, int64_t stride, int64_t rows, int box_rows) {
        const cuuint64_t dim[2] = {(cuuint64_t)(K / 2), (cuuint64_t)rows};
        const cuuint64_t strides[1] = {(cuuint64_t)stride};
        const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
        const cuuint32_t ones[2] = {1, 1};
        return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(codes), dim, strides, box, ones,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    fmm::Args a;
    CUtensorMap lm, rm;
    a.left = p.swap ? operand(b_scales, b_scale_stride, N) : operand(a_scales, a_scale_stride, M);
    a.right = p.swap ? operand(a_scales, a_scale_stride, M) : operand(b_scales, b_scale_stride, N);
    const bool ok = p.swap ? encode(&lm, b_codes, b_code_stride, N, fmm::kM) && encode(&rm, a_codes, a_code_stride, M, p.NT)
                           : encode(&lm, a_codes, a_code_stride, M, fmm::kM) && encode(&rm, b_codes, b_code_stride, N, p.NT);
    if (!ok) return cudaErrorInvalidValue;
    a.K = K;
    a.nblk = K / (mx ? 32 : 16);
    a.NT = p.NT;
    a.stages = p.stages;
    a.splits = p.splits;
    a.tiles_l = (int)ceil_div(a.left.rows, (int64_t)fmm::kM);
    a.tiles = (int64_t)a.tiles_l * ceil_div(a.right.rows, (int64_t)p.NT);
    a.ktiles = (K + fmm::kKTile - 1) / fmm::kKTile;
    const int cells = mx ? 2 : 4;
    a.acc_cols = (uint32_t)(p.NT < 32 ? 32 : p.NT);
    const uint32_t need = a.acc_cols + (uint32_t)(p.stages * cells * 4 * (1 + (p.NT + 127) / 128));
    uint32_t cols = 32;
    while (cols < need) cols <<= 1;
    a.tmem_cols = cols;
    a.swap = p.swap;
    a.alpha = alpha;
    a.out = out;
    a.out_stride = out_stride;
    const int64_t es = out_dtype == CSA2_DTYPE_BF16 ? 2 : 4;
    a.out_vec = (reinterpret_cast<uintptr_t>(out) & 15u) == 0 && (out_stride * es) % 16 == 0;
    const int smem = p.stages * fmm::stage_bytes_of(mx, p.NT) + (int)sizeof(fmm::Ctl) + 1024;
    const int64_t grid = p.splits > 1 ? a.tiles * p.splits : std::min<int64_t>(a.tiles, device_sm_count());
    if (mx)
        return out_dtype == CSA2_DTYPE_BF16 ? launch_fmm<true, true>(a, lm, rm, smem, (unsigned)grid, st)
                                            : launch_fmm<true, false>(a, lm, rm, smem, (unsigned)grid, st);
    return out_dtype == CSA2_DTYPE_BF16 ? launch_fmm<false, true>(a, lm, rm, smem, (unsigned)grid, st)
                                        : launch_fmm<false, false>(a, lm, rm, smem, (unsigned)grid, st);
}

}  // namespace csa2
