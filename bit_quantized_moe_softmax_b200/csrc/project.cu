// project.cu -- a shared bf16 projection with low-rank adapters of many
// requests beside it: y_i = W x_i + s_a B_a (A_a x_i), a = the adapter of row i.
//
// Two kernels.  k_adapter_shrink computes t_i = s_a A_a x_i for every row with
// an adapter and writes it as two bf16 pieces (hi, lo = t - hi: 16 bits, half
// a unit of 2^-17 next to bf16's 2^-9 in y).  k_project is one tcgen05 GEMM
// whose K axis runs on past W: for every adapter a found among a tile's rows
// it has further K blocks [B_a] x [t of a's rows, zero in the others].  The
// adapters so cost a few K steps of the same accumulation and y is written
// once, with one rounding.
//
// The weights are the M side of the MMA (128 output features per tile) and the
// rows the N side (16 to 256), so that one row costs a sixteenth of a tile's
// tensor work and the kernel streams W at the rate of HBM; with many rows the
// N side is as wide as the tensor core takes.
#include <cooperative_groups.h>
#include <cudaTypedefs.h>

#include "ops.cuh"
#include "tcgen05.cuh"

namespace cg = cooperative_groups;

namespace ds4 {

namespace {

constexpr int kPM = 128;                 // output features per tile
constexpr int kPK = 64;                  // K columns per block (one 128-byte swizzle row)
constexpr int kPStageA = kPM * kPK * 2;
constexpr int kPThreads = 256;           // warps: 0 TMA, 1 MMA, 2 TMEM, 4..7 epilogue
constexpr int kPMaxStages = 10;
constexpr int kPSmem = 200 * 1024;       // of 227 KB

// Error word of the projection's bounded waits, one per device.
__device__ uint32_t g_project_err;

struct ProjSmem {
    uint64_t full[kPMaxStages], empty[kPMaxStages];
    uint64_t accF[2], accE[2];
    uint32_t tmem;
    volatile uint32_t abort;
};

// bf16 columns of one row of t: hi pieces, then lo pieces
__host__ __device__ inline int t_cols(int rank) { return 2 * ((rank + 15) & ~15); }

}  // namespace

// ---------------------------------------------------------------- t = s A x, by (row tile, adapter)
// Workspace: counts [tiles], adapter of each entry [tiles][cap], then t
// [tiles][cap][bn][t_cols].  Entry j of a tile is its j-th distinct adapter in
// order of first appearance.
//
// A CTA takes up to 16 rows of one adapter in one tile as the M side of
// mma.sync m16n8k16 and the adapter's rank as N; its eight warps split the
// input columns, 32 at a time, and their sums meet in shared memory in warp
// order.  Lane t of a quad loads 16 consecutive bytes of a row for both
// operands, which permutes the columns within a block of 32 alike on both
// sides.  CTA g also zeroes the rows 16 g .. 16 g + 15 of the tile that are not
// the adapter's.  Bound by the reads of A and x (each adapter's A once per 16
// of its rows, from L2 after the first).
template <int NT>   // 8-wide rank blocks
__global__ void __launch_bounds__(256) k_adapter_shrink(ShrinkArgs a) {
    __shared__ __align__(16) int s_id[256];
    __shared__ int s_rows[16];
    __shared__ int s_cnt[2];
    __shared__ float red[8 * 16 * NT * 8 > 8192 ? 8192 : 8 * 16 * NT * 8];
    griddep_launch();   // the projection may start on W; it waits for this grid before it reads t
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = blockIdx.x, tile = blockIdx.z;
    const int row0 = tile * a.bn, rows = min(a.bn, a.n - row0);
    const int KT = t_cols(a.rank), R16 = KT / 2;

    // entry index of each distinct adapter: rank of its first appearance
    {
        const int id = tid < rows ? a.ids[row0 + tid] : -1;
        s_id[tid] = (unsigned)id < (unsigned)a.n_adapters ? id : -1;   // any other id: no adapter
    }
    __syncthreads();
    int first = 0;
    if (s_id[tid] >= 0) {
        const int id = s_id[tid];
        first = 1;
        for (int k = 0; k < tid; k += 4) {
            const int4 v = *reinterpret_cast<const int4*>(s_id + k);
            if (v.x == id || (k + 1 < tid && v.y == id) || (k + 2 < tid && v.z == id) || (k + 3 < tid && v.w == id)) first = 0;
        }
    }
    __shared__ int s_w[8], s_adapter[256];
    const uint32_t fb = __ballot_sync(0xffffffffu, first);
    if (lane == 0) s_w[warp] = __popc(fb);
    __syncthreads();
    int at = __popc(fb & ((1u << lane) - 1u)), count = 0;
    for (int w = 0; w < 8; ++w) {
        if (w < warp) at += s_w[w];
        count += s_w[w];
    }
    if (first) s_adapter[at] = s_id[tid];
    __syncthreads();
    if (g == 0 && blockIdx.y == 0) {
        if (tid == 0) a.counts[tile] = count;
        if (tid < count) a.entry[tile * a.cap + tid] = s_adapter[tid];
    }

    for (int j = blockIdx.y; j < count; j += gridDim.y) {
        const int ad = s_adapter[j];
        __nv_bfloat16* T = a.t + ((size_t)tile * a.cap + j) * a.bn * KT;
        // zero the other rows of this CTA's sixteen
        for (int i = tid; i < 16 * (KT / 8); i += 256) {
            const int rr = 16 * g + i / (KT / 8);
            if (s_id[rr] != ad) reinterpret_cast<uint4*>(T + (size_t)rr * KT)[i % (KT / 8)] = make_uint4(0, 0, 0, 0);
        }
        // rows 16 g .. of the adapter's, in order
        if (warp == 0) {
            int seen = 0;
            for (int k0 = 0; k0 < a.bn; k0 += 32) {
                const bool mine = k0 + lane < a.bn && s_id[k0 + lane] == ad;
                const uint32_t b = __ballot_sync(0xffffffffu, mine);
                const int p = seen + __popc(b & ((1u << lane) - 1u)) - 16 * g;
                if (mine && p >= 0 && p < 16) s_rows[p] = k0 + lane;
                seen += __popc(b);
            }
            if (lane == 0) s_cnt[0] = max(0, min(16, seen - 16 * g));
        }
        __syncthreads();
        const int m = s_cnt[0];
        if (m > 0) {
            const int gq = lane >> 2, tq = lane & 3;
            const __nv_bfloat16* xa = a.x + (size_t)(row0 + s_rows[gq < m ? gq : 0]) * a.fin;
            const __nv_bfloat16* xb = a.x + (size_t)(row0 + s_rows[gq + 8 < m ? gq + 8 : 0]) * a.fin;
            const bool la = gq < m, lb = gq + 8 < m;
            const __nv_bfloat16* A = a.A + (size_t)ad * a.rank * a.fin;
            float acc[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
            const int nblk = (a.fin + 31) / 32;
#pragma unroll 2
            for (int b = warp; b < nblk; b += 8) {
                const int c = b * 32 + tq * 8;
                const bool in = c < a.fin;
                const uint4 z = make_uint4(0, 0, 0, 0);
                const uint4 x0 = in && la ? __ldg(reinterpret_cast<const uint4*>(xa + c)) : z;
                const uint4 x1 = in && lb ? __ldg(reinterpret_cast<const uint4*>(xb + c)) : z;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int rr = t * 8 + gq;
                    const uint4 w = in && rr < a.rank ? __ldg(reinterpret_cast<const uint4*>(A + (size_t)rr * a.fin + c)) : z;
                    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                        : "+f"(acc[t][0]), "+f"(acc[t][1]), "+f"(acc[t][2]), "+f"(acc[t][3])
                        : "r"(x0.x), "r"(x1.x), "r"(x0.y), "r"(x1.y), "r"(w.x), "r"(w.y));
                    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                        : "+f"(acc[t][0]), "+f"(acc[t][1]), "+f"(acc[t][2]), "+f"(acc[t][3])
                        : "r"(x0.z), "r"(x1.z), "r"(x0.w), "r"(x1.w), "r"(w.z), "r"(w.w));
                }
            }
            // warp sums through shared memory (at most 8 blocks of the rank at a time)
            constexpr int PT = NT > 8 ? 8 : NT;
            const float scale = a.scale[ad];
#pragma unroll
            for (int t0 = 0; t0 < NT; t0 += PT) {
                if (t0) __syncthreads();
#pragma unroll
                for (int t = 0; t < PT; ++t) {
                    float* d = red + ((warp * 16 + gq) * PT + t) * 8 + 2 * tq;
                    d[0] = acc[t0 + t][0], d[1] = acc[t0 + t][1];
                    d[8 * PT * 8] = acc[t0 + t][2], d[8 * PT * 8 + 1] = acc[t0 + t][3];
                }
                __syncthreads();
                for (int i = tid; i < m * PT * 8; i += 256) {
                    const int rr = i / (PT * 8), c = t0 * 8 + i % (PT * 8);
                    float v = 0.f;
#pragma unroll
                    for (int w = 0; w < 8; ++w) v += red[(w * 16 + rr) * PT * 8 + i % (PT * 8)];
                    if (c < R16) {
                        v *= scale;   // zero beyond the rank: A's rows there were read as zero
                        const __nv_bfloat16 hi = __float2bfloat16_rn(v);
                        __nv_bfloat16* d = T + (size_t)s_rows[rr] * KT + c;
                        d[0] = hi;
                        d[R16] = __float2bfloat16_rn(v - __bfloat162float(hi));
                    }
                }
            }
        }
        __syncthreads();   // red and s_rows are reused
    }
}

// ---------------------------------------------------------------- the GEMM
// A block of the K axis is 64 columns: TMA brings 128 rows of W (or of B_a) and
// bn rows of x (or of t) into a ring of stages, one thread issues the MMAs,
// four warps drain TMEM (two accumulators, so that a tile's epilogue overlaps
// the next tile's products).
//
// split > 1 (few tiles): a cluster of CTAs shares one tile, each takes a part
// of W's columns and every split-th adapter, and the partial sums meet through
// distributed shared memory in CTA order.
__global__ void __launch_bounds__(kPThreads) k_project(const __grid_constant__ CUtensorMap mapW,
                                                       const __grid_constant__ CUtensorMap mapX,
                                                       const __grid_constant__ CUtensorMap mapB,
                                                       const __grid_constant__ CUtensorMap mapT, ProjectArgs a) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ ProjSmem S;
    unsigned char* st = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int stage_bytes = kPStageA + a.bn * kPK * 2;
    const int rank_in = a.split > 1 ? (int)(blockIdx.x % a.split) : 0;
    const int first = a.split > 1 ? blockIdx.x / a.split : blockIdx.x;
    const int step = a.split > 1 ? a.tiles : gridDim.x;   // split: one tile per cluster
    const int kb0 = (int)((int64_t)a.kblocks * rank_in / a.split), kb1 = (int)((int64_t)a.kblocks * (rank_in + 1) / a.split);
    const uint32_t acc_cols = a.bn <= 16 ? 32 : a.bn <= 32 ? 64 : a.bn <= 64 ? 128 : a.bn <= 128 ? 256 : 512;
    uint32_t* err = &g_project_err;

    if (tid == 0) {
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(&S.full[i], 1);
            mbar_init(&S.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.accF[i], 1);
            mbar_init(&S.accE[i], 4);
        }
        S.abort = 0;
        fence_barrier_init();
    }
    if (warp == 2) {
        tmem_alloc(&S.tmem, acc_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    const int R16 = (a.rank + 15) & ~15;
    const bool one_block = 2 * R16 <= kPK;               // both pieces of t in one block
    const int per_entry = one_block ? 1 : 2 * ((R16 + kPK - 1) / kPK);

    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            bool waited = false;
            auto slot = [&]() -> int {
                const int s = it % a.stages;
                if (!mbar_wait(&S.empty[s], ((it / a.stages) & 1) ^ 1, err)) {
                    S.abort = 1;
                    return -1;
                }
                mbar_arrive_expect_tx(&S.full[s], stage_bytes);
                ++it;
                return s;
            };
            for (int tile = first; tile < a.tiles && !S.abort; tile += step) {
                const int o0 = tile / a.row_tiles * kPM, rt = tile % a.row_tiles, r0 = rt * a.bn;
                for (int kb = kb0; kb < kb1; ++kb) {
                    const int s = slot();
                    if (s < 0) break;
                    unsigned char* p = st + s * stage_bytes;
                    tma_load_2d(p, &mapW, kb * kPK, o0, &S.full[s]);
                    tma_load_2d(p + kPStageA, &mapX, kb * kPK, r0, &S.full[s]);
                }
                if (a.counts) {
                    if (!waited) {
                        griddep_wait();
                        asm volatile("fence.proxy.async.global;" ::: "memory");
                        waited = true;
                    }
                    const int count = __ldcg(a.counts + rt);
                    for (int j = rank_in; j < count && !S.abort; j += a.split) {
                        const int ad = __ldcg(a.entry + rt * a.cap + j);
                        const int trow = (rt * a.cap + j) * a.bn;
                        for (int b = 0; b < per_entry; ++b) {
                            const int s = slot();
                            if (s < 0) break;
                            unsigned char* p = st + s * stage_bytes;
                            const int c = (b >> 1) * kPK, piece = b & 1;
                            tma_load_3d(p, &mapB, c, o0, ad, &S.full[s]);
                            tma_load_2d(p + kPStageA, &mapT, piece * R16 + c, trow, &S.full[s]);
                        }
                    }
                }
            }
            if (S.abort) {   // no copy may be in flight when the CTA leaves
                const uint32_t n = it < (uint32_t)a.stages ? it : (uint32_t)a.stages;
                for (uint32_t i = it - n; i < it; ++i) mbar_wait(&S.full[i % a.stages], (i / a.stages) & 1, err);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = umma_idesc_bf16(kPM, a.bn);
            uint32_t it = 0, use = 0;
            bool waited = false;
            for (int tile = first; tile < a.tiles && !S.abort; tile += step, ++use) {
                const int rt = tile % a.row_tiles, buf = use & 1;
                if (!mbar_wait(&S.accE[buf], ((use >> 1) & 1) ^ 1, err)) { S.abort = 1; break; }
                tc_fence_after();
                const uint32_t d = tmem + buf * a.bn;
                uint32_t accumulate = 0;
                // k steps [0, na) of the block's A against steps [b0, b0 + na) of its B
                auto wait_full = [&]() -> int {
                    const int s = it % a.stages;
                    if (!mbar_wait(&S.full[s], (it / a.stages) & 1, err)) { S.abort = 1; return -1; }
                    tc_fence_after();
                    ++it;
                    return s;
                };
                auto steps = [&](int s, int na, int b0) {
                    const uint32_t p = smem_addr(st + s * stage_bytes);
                    const uint64_t da = umma_desc_sw128(p), db = umma_desc_sw128(p + kPStageA);
                    for (int k = 0; k < na; ++k) {
                        umma_bf16(d, da + 2 * k, db + 2 * (b0 + k), idesc, accumulate);
                        accumulate = 1;
                    }
                };
                for (int kb = kb0; kb < kb1; ++kb) {
                    const int s = wait_full();
                    if (s < 0) break;
                    steps(s, kPK / 16, 0);
                    umma_commit(&S.empty[s]);
                }
                if (a.counts && !S.abort) {
                    if (!waited) {
                        griddep_wait();
                        waited = true;
                    }
                    const int count = __ldcg(a.counts + rt);
                    for (int j = rank_in; j < count && !S.abort; j += a.split)
                        for (int b = 0; b < per_entry; ++b) {
                            const int s = wait_full();
                            if (s < 0) break;
                            if (one_block) {
                                steps(s, R16 / 16, 0);
                                steps(s, R16 / 16, R16 / 16);
                            } else {
                                steps(s, min(kPK, R16 - (b >> 1) * kPK) / 16, 0);
                            }
                            umma_commit(&S.empty[s]);
                        }
                }
                umma_commit(&S.accF[buf]);
            }
        }
    } else if (warp >= 4) {
        const int qd = warp & 3;   // TMEM lanes 32 qd .. 32 qd + 31
        uint32_t use = 0;
        for (int tile = first; tile < a.tiles && !S.abort; tile += step, ++use) {
            const int buf = use & 1;
            if (!mbar_wait(&S.accF[buf], (use >> 1) & 1, err)) S.abort = 1;
            const bool ok = !S.abort;   // a wait that ran out leaves NaN in the tile
            tc_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(32 * qd) << 16) + buf * a.bn;
            const int o = tile / a.row_tiles * kPM + 32 * qd + lane, r0 = tile % a.row_tiles * a.bn;
            const int rows = min(a.bn, a.n - r0);
            if (a.split > 1) {
                float* part = reinterpret_cast<float*>(st) + 32 * qd + lane;   // [bn][128]; every stage is done with
                for (int c0 = 0; c0 < a.bn; c0 += 16) {
                    uint32_t v[16];
                    tmem_ld_32x16(taddr + c0, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) part[(c0 + j) * kPM] = ok ? __uint_as_float(v[j]) : __int_as_float(0x7fffffff);
                }
            } else {
                __nv_bfloat16* dst = a.out + (size_t)r0 * a.fout + o;
                for (int c0 = 0; c0 < rows; c0 += 16) {
                    uint32_t v[16];
                    tmem_ld_32x16(taddr + c0, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (o < a.fout && c0 + j < rows)
                            dst[(size_t)(c0 + j) * a.fout] =
                                __float2bfloat16_rn(ok ? __uint_as_float(v[j]) : __int_as_float(0x7fffffff));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.accE[buf]);
        }
    }
    if (a.split > 1) {
        __syncwarp();
        cg::cluster_group cl = cg::this_cluster();
        cl.sync();
        const int tile = first;
        const int o = tile / a.row_tiles * kPM + (tid & 127), r0 = tile % a.row_tiles * a.bn;
        const int per = (a.bn + a.split - 1) / a.split;
        const int c1 = min(min(a.bn, a.n - r0), per * (rank_in + 1));
        const float* part[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) part[p] = cl.map_shared_rank(reinterpret_cast<const float*>(st), p < a.split ? p : 0) + (tid & 127);
        for (int c = per * rank_in + (tid >> 7); c < c1; c += 2) {
            float v = 0.f;
#pragma unroll
            for (int p = 0; p < 8; ++p)
                if (p < a.split) v += part[p][c * kPM];
            if (o < a.fout) a.out[(size_t)(r0 + c) * a.fout + o] = __float2bfloat16_rn(v);
        }
        cl.sync();   // peers have read this CTA's sums
    }
    if (a.counts) griddep_wait();   // this grid's end implies the first one's
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, acc_cols);
    }
}

// ---------------------------------------------------------------- host side
static PFN_cuTensorMapEncodeTiled_v12000 tmap_encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
        cudaDriverEntryPointQueryResult q;
        void* p = nullptr;
        const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q);
        if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !p) return nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// bf16 [mats][rows][cols] read in boxes of 64 columns x box_rows rows, 128-byte swizzle; zero outside.
static cudaError_t encode(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint64_t mats, int dims,
                          int box_rows) {
    const PFN_cuTensorMapEncodeTiled_v12000 fn = tmap_encoder();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t size[3] = {cols, rows, mats};
    const cuuint64_t strides[2] = {cols * 2, cols * rows * 2};
    const cuuint32_t box[3] = {kPK, (cuuint32_t)box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims, const_cast<void*>(base), size, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Rows per tile: up to 128 rows one tile, as narrow as they allow (the N side
// of an MMA is a multiple of 16).  More rows: the width whose tiles fill the
// SMs best; a wave of tiles takes time in proportion to the width plus a
// start-up worth about 16 columns.
static int project_bn(int n, int fout) {
    constexpr int n_sm = 148;   // the size of the work buffer must not depend on the current device
    if (n <= 128) return (n + 15) & ~15;
    const int64_t ot = (fout + kPM - 1) / kPM;
    int best = 256;
    int64_t cost = INT64_MAX;
    for (int bn = 256; bn >= 64; bn -= 16) {
        const int64_t tiles = ot * ((n + bn - 1) / bn), c = (tiles + n_sm - 1) / n_sm * (bn + 16);
        if (c < cost) cost = c, best = bn;
    }
    return best;
}

ProjectWork project_work(int n, int fout, int n_adapters, int rank) {
    ProjectWork w{};
    w.bn = project_bn(n, fout);
    w.row_tiles = (n + w.bn - 1) / w.bn;
    w.cap = n_adapters < w.bn ? n_adapters : w.bn;
    auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
    w.off_entry = up((size_t)w.row_tiles * 4);
    w.off_t = w.off_entry + up((size_t)w.row_tiles * w.cap * 4);
    w.total = w.off_t + up((size_t)w.row_tiles * w.cap * w.bn * t_cols(rank) * 2);
    return w;
}

cudaError_t launch_project(ProjectArgs p, ShrinkArgs s, const ProjectWork& wk, const void* W, const void* B, int n_sm,
                           cudaStream_t st) {
    p.bn = wk.bn;
    p.row_tiles = wk.row_tiles;
    p.cap = wk.cap;
    p.kblocks = (p.fin + kPK - 1) / kPK;
    p.tiles = (p.fout + kPM - 1) / kPM * p.row_tiles;
    // Few tiles: several CTAs share one, as many as leave each four blocks of W and find an SM of their own.
    p.split = 1;
    while (p.split < 8 && (int64_t)p.tiles * p.split * 2 <= n_sm && p.kblocks >= p.split * 2 * 4) p.split *= 2;
    const int stage = kPStageA + p.bn * kPK * 2;
    p.stages = kPSmem / stage < kPMaxStages ? kPSmem / stage : kPMaxStages;
    const int smem = 1024 + p.stages * stage;   // the partial sums of a split tile (512 bytes per row) fit as well

    CUtensorMap mW, mX, mB = {}, mT = {};
    cudaError_t e = encode(&mW, W, p.fin, p.fout, 1, 2, kPM);
    if (e == cudaSuccess) e = encode(&mX, s.x, p.fin, p.n, 1, 2, p.bn);
    if (e == cudaSuccess && p.counts) e = encode(&mB, B, p.rank, p.fout, s.n_adapters, 3, kPM);
    if (e == cudaSuccess && p.counts)
        e = encode(&mT, s.t, t_cols(p.rank), (uint64_t)p.row_tiles * p.cap * p.bn, 1, 2, p.bn);
    if (e != cudaSuccess) return e;

    if (p.counts) {
        s.bn = p.bn;
        s.cap = p.cap;
        const int groups = (p.bn + 15) / 16;
        int y = p.cap;
        while (y > 1 && (int64_t)groups * y * p.row_tiles > 4096) y = (y + 1) / 2;
        const dim3 grid(groups, y, p.row_tiles);
        const int nt = (p.rank + 7) / 8;
        if (nt <= 2) k_adapter_shrink<2><<<grid, 256, 0, st>>>(s);
        else if (nt <= 4) k_adapter_shrink<4><<<grid, 256, 0, st>>>(s);
        else if (nt <= 8) k_adapter_shrink<8><<<grid, 256, 0, st>>>(s);
        else k_adapter_shrink<16><<<grid, 256, 0, st>>>(s);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    e = cudaFuncSetAttribute(k_project, cudaFuncAttributeMaxDynamicSharedMemorySize, kPSmem + 1024);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.split > 1 ? p.tiles * p.split : p.tiles < n_sm ? p.tiles : n_sm));
    cfg.blockDim = dim3(kPThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    unsigned na = 0;
    if (p.split > 1) {
        at[na].id = cudaLaunchAttributeClusterDimension;
        at[na].val.clusterDim.x = (unsigned)p.split;
        at[na].val.clusterDim.y = at[na].val.clusterDim.z = 1;
        ++na;
    }
    if (p.counts) {
        at[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[na].val.programmaticStreamSerializationAllowed = 1;
        ++na;
    }
    cfg.attrs = at;
    cfg.numAttrs = na;
    return cudaLaunchKernelEx(&cfg, k_project, mW, mX, mB, mT, p);
}

cudaError_t read_project_error(uint32_t* code, cudaStream_t st) {
    void* p = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&p, g_project_err);
    if (e == cudaSuccess) e = cudaMemcpyAsync(code, p, 4, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaMemsetAsync(p, 0, 4, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    return e;
}

}  // namespace ds4
