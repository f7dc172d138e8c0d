// project.cu -- a shared bf16 projection with low-rank adapters of many
// requests beside it: y_i = W x_i + s_a B_a (A_a x_i), a = the adapter of row i.
//
// Two kernels.  k_adapter_shrink computes t_i = s_a A_a x_i for every row with
// an adapter and writes it as two bf16 pieces (hi, lo = t - hi: 16 bits, half
// a unit of 2^-17 next to bf16's 2^-9 in y).  k_project (k_project_pair) is one
// tcgen05 GEMM whose K axis runs on past W: for every adapter a found among a
// tile's rows it has further K blocks [B_a] x [t of a's rows, zero in the
// others].  The adapters so cost a few K steps of the same accumulation and y is
// written once, with one rounding.  For 8 to 64 rows the second product is
// outside the MMAs instead (adapter_rows).
//
// The weights are the M side of the MMA (128 output features per tile) and the
// rows the N side (16 to 256), so that one row costs a sixteenth of a tile's
// tensor work and the kernel streams W at the rate of HBM; with many rows the
// N side is as wide as the tensor core takes.
#include <cooperative_groups.h>
#include <cudaTypedefs.h>

#include <mutex>

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
constexpr int kAhead = 16;
constexpr int kRowsMin = 8, kRowsMax = 64;   // rows whose adapters the draining warps add
constexpr int kPSmem = 200 * 1024;       // of 227 KB
constexpr int kPSmemRows = 168 * 1024, kPSmemEntries = 150 * 1024;   // beside a CTA of the first kernel

// Error word of the projection's bounded waits, one per device, and where a
// reader takes it to.
__device__ uint32_t g_project_err, g_project_taken;

// A bounded wait of the projection: false after kWaitNs (error bit 1), or when
// another thread has given up.  Not in_time (the self-test's tiles): at once.
//
// What follows then, in both kernels: the thread sets the abort flag; the
// producer issues no more and waits for its copies in flight, the issuing thread
// for its MMAs; no accumulator is signalled as full that is not; the draining
// warps go through all the tiles that are left and store NaN; a split tile's
// CTAs look at one another's flags after their barrier, and store NaN if one is
// set.
__device__ __forceinline__ bool project_wait(uint64_t* bar, uint32_t parity, const volatile uint32_t* abort, bool in_time) {
    if (in_time) {
        if (mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = global_ns();
        do {
            for (int i = 0; i < 16; ++i)
                if (mbar_try_wait(bar, parity)) return true;
            if (*abort) return false;
        } while (global_ns() - t0 <= kWaitNs);
    }
    set_err(&g_project_err, kErrTimeout);
    return false;
}

struct ProjSmem {
    uint64_t full[kPMaxStages], empty[kPMaxStages];
    uint64_t accF[2], accE[2], last;
    uint32_t tmem;
    volatile uint32_t abort;
    int ahead[kAhead];
    int ids[kRowsMax];
};

// The adapters of a tile's entries j0, j0 + step, .. for one thread, kAhead
// loads at a time: one by one each would cost the loop a trip to the L2.
struct Entries {
    const int32_t* p;
    int* buf;
    int count;
    __device__ __forceinline__ int get(int j, int first, int step) const {
        const int i = (j - first) / step % kAhead;
        if (i == 0) {
            int v[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) v[k] = j + k * step < count ? __ldcg(p + j + k * step) : 0;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) buf[k] = v[k];
        }
        return buf[i];
    }
};

// bf16 columns of one row of t: hi pieces, then lo pieces
__host__ __device__ inline int t_cols(int rank) { return 2 * ((rank + 15) & ~15); }

}  // namespace

// ---------------------------------------------------------------- t = s A x, by (row tile, adapter)
// Workspace: counts [tiles], adapter of each entry [tiles][cap], then t
// [tiles][cap][bn][t_cols].  Entry j of a tile is its j-th distinct adapter in
// order of first appearance.  For 8 to 64 rows t alone, in binary32: [n][rank].
//
// A cluster of `split` CTAs takes up to 64 rows (16 there) of one adapter, each
// CTA a part of the input columns: 64-column blocks of the rows and of A go
// through a ring of shared-memory stages (cp.async, 16-byte units swizzled by
// row), the rows are the M side of mma.sync m16n8k16, the rank the N side, and
// warps beyond one per 16 rows share a block's columns.  Lane t of a quad takes
// 16 consecutive bytes of a row for both operands, which permutes the columns
// of a block alike on both sides.  The warps' sums, then the CTAs' through
// distributed shared memory, are added in order.  Bound by the reads of A and x
// (A once per 64 of its rows); the split keeps enough of them in flight when
// every row has its own adapter.
constexpr int kShStages = 4;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
    const int n = in ? 16 : 0;   // the rest is filled with zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

// (NT 8 bounded as if for more threads: 96 registers, so that two fit beside a CTA of the projection)
template <int NT, int kShRows>   // 8-wide rank blocks; rows per item
__global__ void __launch_bounds__(NT == 8 ? 320 : 256, NT >= 8 ? 2 : NT == 4 ? 4 : 5) k_adapter_shrink(ShrinkArgs a) {
    extern __shared__ __align__(128) unsigned char ring[];   // [kShStages][kShRows + 8 NT rows][128 bytes]
    __shared__ __align__(16) int s_id[256];
    __shared__ int s_w[8], s_key[512], s_lead[512], s_rank[256], s_adapter[256], s_n[256], s_rows[kShRows], s_j, s_c0, s_cnt;
    constexpr int kStageRows = kShRows + 8 * NT;
    griddep_launch();   // the projection may start on W; it waits for this grid before it reads t
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int part = blockIdx.x, tile = blockIdx.z;
    const int row0 = tile * a.bn, rows = min(a.bn, a.n - row0);
    const int KT = t_cols(a.rank), R16 = KT / 2;

    // the tile's distinct adapters in order of first appearance, and how many rows each has
    const int row_id = tid < rows ? a.ids[row0 + tid] : -1;
    const int id = (unsigned)row_id < (unsigned)a.n_adapters ? row_id : -1;   // any other id: no adapter
    s_id[tid] = id;
    s_n[tid] = 0;
    s_key[tid] = s_key[tid + 256] = -1;
    s_lead[tid] = s_lead[tid + 256] = 256;
    __syncthreads();
    int slot = id & 511;   // a hash table of at most 256 adapters: each one's first row
    if (id >= 0) {
        for (;;) {
            const int old = atomicCAS(&s_key[slot], -1, id);
            if (old == -1 || old == id) break;
            slot = (slot + 1) & 511;
        }
        atomicMin(&s_lead[slot], tid);
    }
    __syncthreads();
    const int lead = id >= 0 ? s_lead[slot] : tid;
    auto scan = [&](int v, int& before) {   // exclusive prefix over the threads, and the total
        int inc = v;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, inc, m);
            if (lane >= m) inc += o;
        }
        __syncthreads();
        if (lane == 31) s_w[warp] = inc;
        __syncthreads();
        int base = 0, all = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            if (w < warp) base += s_w[w];
            all += s_w[w];
        }
        before = base + inc - v;
        return all;
    };
    int at;
    const int count = scan(id >= 0 && lead == tid, at);
    if (id >= 0 && lead == tid) s_rank[tid] = at, s_adapter[at] = id;
    __syncthreads();
    if (id >= 0) atomicAdd(&s_n[s_rank[lead]], 1);
    __syncthreads();
    if (a.counts && blockIdx.x == 0 && blockIdx.y == 0) {
        if (tid == 0) a.counts[tile] = count;
        if (tid < count) a.entry[tile * a.cap + tid] = s_adapter[tid];
    }
    const int chunks = tid < count ? (s_n[tid] + kShRows - 1) / kShRows : 0;
    int c0;
    const int items = scan(chunks, c0);   // (adapter, 64 of its rows), shared out among the clusters of this tile

    const int nblk = (a.fin + kPK - 1) / kPK;
    const int b0 = nblk * part / a.split, nb = nblk * (part + 1) / a.split - b0;   // this CTA's column blocks
    for (int item = blockIdx.y; item < items; item += gridDim.y) {
        if (c0 <= item && item < c0 + chunks) s_j = tid, s_c0 = c0;   // one thread
        __syncthreads();
        const int j = s_j, g = item - s_c0, ad = s_adapter[j];
        __nv_bfloat16* T = a.t + ((size_t)tile * a.cap + j) * a.bn * KT;
        if (g == 0 && !a.rows) {   // zero the rows that are not the adapter's (the CTAs of the cluster in turn)
            const int per = KT / 8;
            for (int i = tid; i < (a.bn + a.split - 1) / a.split * per; i += 256) {
                const int rr = i / per * a.split + part;
                if (rr < a.bn && s_id[rr] != ad) reinterpret_cast<uint4*>(T + (size_t)rr * KT)[i % per] = make_uint4(0, 0, 0, 0);
            }
        }
        // the adapter's rows 64 g .. in order
        if (warp == 0) {
            int seen = 0;
            for (int k0 = 0; k0 < a.bn; k0 += 32) {
                const bool mine = k0 + lane < a.bn && s_id[k0 + lane] == ad;
                const uint32_t b = __ballot_sync(0xffffffffu, mine);
                const int p = seen + __popc(b & ((1u << lane) - 1u)) - kShRows * g;
                if (mine && p >= 0 && p < kShRows) s_rows[p] = k0 + lane;
                seen += __popc(b);
            }
            if (lane == 0) s_cnt = min(kShRows, seen - kShRows * g);
        }
        __syncthreads();
        const int m = s_cnt;
        {
            const __nv_bfloat16* A = a.A + (size_t)ad * a.rank * a.fin;
            // this thread's 16-byte units of a stage: column unit tid % 8 of rows tid / 8, tid / 8 + 32, ..
            constexpr int U = (kStageRows + 31) / 32;
            const __nv_bfloat16* src[U];
            uint32_t use = 0;   // bit 2 u: unit u is loaded; bit 2 u + 1: from memory (else zeros)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int rr = (tid >> 3) + 32 * u, col = b0 * kPK + (tid & 7) * 8;
                const bool is_x = rr < kShRows;
                // rows whose products nobody reads are left as they are
                const bool any = is_x ? rr < m : rr - kShRows < R16 && rr < kStageRows;
                const bool real = any && (is_x || rr - kShRows < a.rank);
                src[u] = !real ? a.x : is_x ? a.x + (size_t)(row0 + s_rows[rr]) * a.fin + col
                                            : A + (size_t)(rr - kShRows) * a.fin + col;
                use |= (uint32_t)any << (2 * u) | (uint32_t)real << (2 * u + 1);
            }
            const uint32_t dst0 = smem_addr(ring) + (tid >> 3) * 128 + (((tid & 7) ^ (tid >> 3 & 7)) << 4);
            auto load = [&](int b) {
                if (b < nb) {
                    const uint32_t dst = dst0 + (b % kShStages) * kStageRows * 128;
                    const bool in = (b0 + b) * kPK + (tid & 7) * 8 < a.fin;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const bool real = in && (use >> (2 * u + 1) & 1u);
                        if (use >> (2 * u) & 1u) cp_async16(dst + u * 32 * 128, real ? src[u] + b * kPK : a.x, real);
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            const int rtiles = kShRows == 16 || m <= 16 ? 1 : m <= 32 ? 2 : 4, kways = 8 / rtiles;
            const int rt = warp % rtiles, kidx = warp / rtiles, gq = lane >> 2, tq = lane & 3;
            float acc[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
            for (int b = 0; b < kShStages - 1; ++b) load(b);
            for (int b = 0; b < nb; ++b) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kShStages - 2) : "memory");
                __syncthreads();   // block b has arrived, and block b - 1's stage is free
                load(b + kShStages - 1);
                const unsigned char* p = ring + (b % kShStages) * kStageRows * 128;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if ((2 * b + h) % kways != kidx || 16 * rt >= m) continue;
                    auto unit = [&](int row) {
                        return *reinterpret_cast<const uint4*>(p + row * 128 + (((tq + 4 * h) ^ (row & 7)) << 4));
                    };
                    const uint4 x0 = unit(16 * rt + gq), x1 = unit(16 * rt + 8 + gq);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const uint4 w = unit(kShRows + 8 * t + gq);
                        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                            : "+f"(acc[t][0]), "+f"(acc[t][1]), "+f"(acc[t][2]), "+f"(acc[t][3])
                            : "r"(x0.x), "r"(x1.x), "r"(x0.y), "r"(x1.y), "r"(w.x), "r"(w.y));
                        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                            : "+f"(acc[t][0]), "+f"(acc[t][1]), "+f"(acc[t][2]), "+f"(acc[t][3])
                            : "r"(x0.z), "r"(x1.z), "r"(x0.w), "r"(x1.w), "r"(w.z), "r"(w.w));
                    }
                }
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();
            // warps' sums, then CTAs', in order
            float* red = reinterpret_cast<float*>(ring);            // [8][16][8 NT]
            float* sum = red + 8 * 16 * 8 * NT;                     // [64][8 NT]
            constexpr int RW = 8 * NT;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float* d = red + (warp * 16 + gq) * RW + 8 * t + 2 * tq;
                d[0] = acc[t][0], d[1] = acc[t][1];
                d[8 * RW] = acc[t][2], d[8 * RW + 1] = acc[t][3];
            }
            __syncthreads();
            for (int i = tid; i < m * RW; i += 256) {
                const int rr = i / RW, c = i % RW;
                float v = 0.f;
                for (int k = 0; k < kways; ++k) v += red[((k * rtiles + (rr >> 4)) * 16 + (rr & 15)) * RW + c];
                sum[i] = v;
            }
            if (a.split > 1) cl.sync();
            else __syncthreads();
            const float scale = a.scale[ad];
            const int mine = (m - part + a.split - 1) / a.split;   // rows part, part + split, ..
            for (int i = tid; i < mine * (R16 / 2); i += 256) {
                const int rr = i / (R16 / 2) * a.split + part, c = 2 * (i % (R16 / 2));
                float2 v = make_float2(0.f, 0.f);
                for (int p = 0; p < a.split; ++p) {
                    const float2 o = *reinterpret_cast<const float2*>(cl.map_shared_rank(sum, p) + rr * RW + c);
                    v.x += o.x, v.y += o.y;
                }
                v.x *= scale, v.y *= scale;   // zero beyond the rank: A's rows there were filled with zeros
                if (a.rows) {
                    if (c < a.rank) *reinterpret_cast<float2*>(a.rows + (size_t)(row0 + s_rows[rr]) * a.rank + c) = v;
                    continue;
                }
                const uint32_t hi = pack_bf16x2(v.x, v.y);
                uint32_t* d = reinterpret_cast<uint32_t*>(T + (size_t)s_rows[rr] * KT + c);
                d[0] = hi;
                d[R16 / 2] = pack_bf16x2(v.x - __uint_as_float(hi << 16), v.y - __uint_as_float(hi & 0xffff0000u));
            }
            if (a.split > 1) cl.sync();   // the peers have read this CTA's sums
        }
        __syncthreads();   // the ring and s_rows are reused
    }
}

template <int NT, int kShRows>
static cudaError_t shrink_launch(const ShrinkArgs& s, dim3 grid, cudaStream_t st) {
    const int ring = kShStages * (kShRows + 8 * NT) * 128, sums = (8 * 16 + kShRows) * 8 * NT * 4;
    const int smem = ring > sums ? ring : sums;
    cudaError_t e = cudaFuncSetAttribute(k_adapter_shrink<NT, kShRows>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)s.split;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_adapter_shrink<NT, kShRows>, s);
}

// 8 to 64 rows (a decode batch; fewer are faster by the MMAs, 14 against 20 us for
// one row at 4096 x 4096, and so are more, 37 against 41 us for 128 rows of 64
// adapters): a block of the K axis per adapter would be zero but for a row or
// two, so the warps that drain the accumulators add the adapters themselves, in
// binary32, while the MMAs run: a lane has one output feature and reads its
// `rank` values of B for each row, 16 bytes at a time (the warp's 32 features lie
// next to each other, so all of a row's lines are used), eight rows' loads in
// flight.  Of a split tile each CTA adds and stages the rows that it finishes.
// acc[i] += B[id][o] . t for the first `rows` of the CTA's rows; ts, ids: their t
// [rows][rank] and adapters (or -1) in shared memory.
__device__ __forceinline__ void adapter_rows(const ProjectArgs& a, const float* ts, const int* ids, int o, int rows,
                                             float (&acc)[kRowsMax]) {
#pragma unroll
    for (int i = 0; i < kRowsMax; ++i) acc[i] = 0.f;
    const __nv_bfloat16* B = a.B + (size_t)(o < a.fout ? o : 0) * a.rank;
    const size_t stride = (size_t)a.fout * a.rank;
#pragma unroll
    for (int c = 0; c < kRowsMax; c += 8) {
        if (c >= rows) break;
        for (int k = 0; k < a.rank; k += 8) {
            uint4 w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int id = c + j < rows ? ids[c + j] : -1;
                w[j] = id >= 0 ? __ldg(reinterpret_cast<const uint4*>(B + (size_t)id * stride + k)) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int row = c + j;
                if (row < rows && ids[row] >= 0) {
                    const float4 t0 = *reinterpret_cast<const float4*>(ts + row * a.rank + k);
                    const float4 t1 = *reinterpret_cast<const float4*>(ts + row * a.rank + k + 4);
                    const uint32_t x[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
                    const float t[8] = {t0.x, t0.y, t0.z, t0.w, t1.x, t1.y, t1.z, t1.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        acc[c + j] = fmaf(__uint_as_float(x[e] << 16), t[2 * e], acc[c + j]);
                        acc[c + j] = fmaf(__uint_as_float(x[e] & 0xffff0000u), t[2 * e + 1], acc[c + j]);
                    }
                }
            }
        }
    }
}

// t and the adapters of rows lo .. lo + rows - 1 into shared memory, by
// `threads` threads that meet at barrier 1.
__device__ __forceinline__ void stage_rows(const ProjectArgs& a, float* ts, int* ids, int lo, int rows, int i0, int threads) {
    griddep_wait();   // t is the first kernel's
    const float4* src = reinterpret_cast<const float4*>(a.rows + (size_t)lo * a.rank);
    for (int i = i0; i < rows * a.rank / 4; i += threads) reinterpret_cast<float4*>(ts)[i] = __ldcg(src + i);
    for (int i = i0; i < rows; i += threads) {
        const int id = __ldg(a.ids + lo + i);
        ids[i] = (unsigned)id < (unsigned)a.n_adapters ? id : -1;
    }
    named_sync(1, threads);
}

// Sixteen rows of one warp's share of a tile to out: v, the binary32 bits of
// this lane's output feature o (a TMEM lane) in rows r0 .. r0 + rows - 1.  Two
// lanes exchange half of their values, so that a lane stores two features of
// one row at once.
__device__ __forceinline__ void store16(const ProjectArgs& a, const uint32_t (&v)[16], int o, int lane, int r0, int rows) {
    __nv_bfloat16* dst = a.out + (size_t)r0 * a.fout;
    if ((a.fout & 1) == 0) {
        const int odd = lane & 1;
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            // an even lane takes row j, an odd one row j + 1
            const uint32_t mine = odd ? v[j + 1] : v[j], other = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
            const uint32_t w = pack_bf16x2(__uint_as_float(odd ? other : mine), __uint_as_float(odd ? mine : other));
            if (o < a.fout && j + odd < rows) *reinterpret_cast<uint32_t*>(dst + (size_t)(j + odd) * a.fout + (o & ~1)) = w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (o < a.fout && j < rows) dst[(size_t)j * a.fout + o] = __float2bfloat16_rn(__uint_as_float(v[j]));
    }
}

// Rows c0 .. c1 - 1 of a split tile's 128 features from o on, finished by the
// calling warp and its `warps` - 1 peers: the partial sums [bn][128] in the
// shared memory (at `sums`) of ranks rank0, rank0 + step, .. of the cluster, in
// that order.  A lane has four features, so that a warp's loads and stores are
// wide and few enough to wait for.  NaN where a CTA of the cluster has given up.
__device__ __forceinline__ void finish_split(const ProjectArgs& a, cg::cluster_group& cl, float* sums, volatile uint32_t* abort,
                                             int ctas, int rank0, int step, int o, int r0, int c0, int c1, int warp, int warps,
                                             int lane) {
    const uint32_t bad = *const_cast<volatile uint32_t*>(cl.map_shared_rank(const_cast<uint32_t*>(abort), lane < ctas ? lane : 0));
    const float* part[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) part[p] = cl.map_shared_rank(sums, rank0 + (p < a.split ? p : 0) * step);
    const bool wide = (a.fout & 3) == 0;   // else features lane, lane + 32, ..: stores next to each other
#pragma unroll 2
    for (int c = c0 + warp; c < c1; c += warps) {
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            if (p < a.split) {
                const float* q = part[p] + c * kPM;
                if (wide) {
                    const float4 x = reinterpret_cast<const float4*>(q)[lane];
                    v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] += q[32 * e + lane];
                }
            }
        }
        if (__any_sync(0xffffffffu, bad)) v[0] = v[1] = v[2] = v[3] = __int_as_float(0x7fffffff);
        __nv_bfloat16* d = a.out + (size_t)(r0 + c) * a.fout + o;
        if (wide) {
            if (o + 4 * lane < a.fout)
                *reinterpret_cast<uint2*>(d + 4 * lane) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (o + 32 * e + lane < a.fout) d[32 * e + lane] = __float2bfloat16_rn(v[e]);
        }
    }
}

// A tile's accumulators (columns from taddr on) to out, with what the adapters
// add to up to 64 rows (acc).  Not ok (a wait ran out; the same for the whole
// warp): NaN.
template <bool Rows, int N>
__device__ __forceinline__ void store_tile(const ProjectArgs& a, uint32_t taddr, int o, int lane, int r0, int rows, bool ok,
                                           const float (&acc)[N]) {
    auto sixteen = [&](int c0) {
        uint32_t v[16];
        tmem_ld_32x16(taddr + c0, v);
        tmem_wait_ld();
        if constexpr (Rows) {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) + acc[c0 + j]);
        }
        if (!ok) {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = 0x7fffffffu;
        }
        store16(a, v, o, lane, r0 + c0, rows - c0);
    };
    if constexpr (Rows) {
#pragma unroll
        for (int c0 = 0; c0 < kRowsMax; c0 += 16)
            if (c0 < rows) sixteen(c0);
    } else {
        for (int c0 = 0; c0 < rows; c0 += 16) sixteen(c0);
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
// Rows: a decode batch's adapters by adapter_rows (bounded as if for 512 threads:
// 128 registers leave a CTA of the first kernel room on the SM).
template <bool Rows>
__global__ void __launch_bounds__(Rows ? 512 : kPThreads, 1) k_project(const __grid_constant__ CUtensorMap mapW,
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
        mbar_init(&S.last, 1);
        S.abort = 0;
        fence_barrier_init();
        // the first tile's first blocks are on their way before the others are set up
        if (first < a.tiles) {
            const int o0 = first / a.row_tiles * kPM, r0 = first % a.row_tiles * a.bn;
            for (int i = 0; i < min(a.stages, kb1 - kb0); ++i) {
                unsigned char* p = st + i * stage_bytes;
                mbar_arrive_expect_tx(&S.full[i], stage_bytes);
                tma_load_2d(p, &mapW, (kb0 + i) * kPK, o0, &S.full[i]);
                tma_load_2d(p + kPStageA, &mapX, (kb0 + i) * kPK, r0, &S.full[i]);
            }
        }
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

    uint32_t blocks = 0;   // thread 0: copies sent

    if (warp == 0) {
        if (lane == 0) {
            const uint32_t sent = first < a.tiles ? min(a.stages, kb1 - kb0) : 0;   // above
            uint32_t it = sent;
            int use = 0;
            bool waited = false, in_time = true;
            auto slot = [&]() -> int {
                const int s = it % a.stages;
                if (!project_wait(&S.empty[s], ((it / a.stages) & 1) ^ 1, &S.abort, in_time)) {
                    S.abort = 1;
                    return -1;
                }
                mbar_arrive_expect_tx(&S.full[s], stage_bytes);
                ++it;
                return s;
            };
            for (int tile = first; tile < a.tiles && !S.abort; tile += step, ++use) {
                const int o0 = tile / a.row_tiles * kPM, rt = tile % a.row_tiles, r0 = rt * a.bn;
                in_time = use < a.in_time;
                for (int kb = kb0 + (tile == first ? (int)sent : 0); kb < kb1; ++kb) {
                    const int s = slot();
                    if (s < 0) break;
                    unsigned char* p = st + s * stage_bytes;
                    tma_load_2d(p, &mapW, kb * kPK, o0, &S.full[s]);
                    tma_load_2d(p + kPStageA, &mapX, kb * kPK, r0, &S.full[s]);
                }
                if (!Rows && a.counts) {
                    if (!waited) {
                        griddep_wait();
                        asm volatile("fence.proxy.async.global;" ::: "memory");
                        waited = true;
                    }
                    const Entries entries{a.entry + rt * a.cap, S.ahead, __ldcg(a.counts + rt)};
                    for (int j = rank_in; j < entries.count && !S.abort; j += a.split) {
                        const int ad = entries.get(j, rank_in, a.split);
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
            blocks = it;
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = umma_idesc_bf16(kPM, a.bn);
            uint32_t it = 0, use = 0;
            bool waited = false;
            for (int tile = first; tile < a.tiles && !S.abort; tile += step, ++use) {
                const int rt = tile % a.row_tiles, buf = use & 1;
                const bool in_time = (int)use < a.in_time;
                if (!project_wait(&S.accE[buf], ((use >> 1) & 1) ^ 1, &S.abort, in_time)) { S.abort = 1; break; }
                tc_fence_after();
                const uint32_t d = tmem + buf * a.bn;
                uint32_t accumulate = 0;
                // k steps [0, na) of the block's A against steps [b0, b0 + na) of its B
                auto wait_full = [&]() -> int {
                    const int s = it % a.stages;
                    if (!project_wait(&S.full[s], (it / a.stages) & 1, &S.abort, in_time)) { S.abort = 1; return -1; }
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
                if (!Rows && a.counts && !S.abort) {
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
                if (S.abort) break;   // (this thread's own, or another's: the tile is not to look complete)
                umma_commit(&S.accF[buf]);
            }
        }
    } else if (warp >= 4) {
        const int qd = warp & 3;   // TMEM lanes 32 qd .. 32 qd + 31
        uint32_t use = 0;
        bool ok = true;   // the same for the whole warp; a phase behind one that was given up would look complete
        float* ts = reinterpret_cast<float*>(st + a.stages * stage_bytes);
        const int per = (a.bn + a.split - 1) / a.split, lo = per * rank_in;   // rows that this CTA of a split tile finishes
        const int mine = max(0, min(a.n, lo + per) - lo);                      // (Rows: there is one tile along the rows)
        if constexpr (Rows) stage_rows(a, ts, S.ids, lo, mine, tid - 128, 128);
        for (int tile = first; tile < a.tiles; tile += step, ++use) {
            const int buf = use & 1;
            const uint32_t taddr = tmem + ((uint32_t)(32 * qd) << 16) + buf * a.bn;
            const int o = tile / a.row_tiles * kPM + 32 * qd + lane, r0 = tile % a.row_tiles * a.bn;
            const int rows = min(a.bn, a.n - r0);
            float acc[Rows ? kRowsMax : 1];
            if constexpr (Rows) adapter_rows(a, ts, S.ids, o, mine, acc);
            ok = ok && __all_sync(0xffffffffu, project_wait(&S.accF[buf], (use >> 1) & 1, &S.abort, (int)use < a.in_time));
            if (!ok) S.abort = 1;
            tc_fence_after();
            if (a.split > 1 && ok) {
                float* part = reinterpret_cast<float*>(st) + 32 * qd + lane;   // [bn][128]; every stage is done with
                for (int c0 = 0; c0 < a.bn; c0 += 16) {
                    uint32_t v[16];
                    tmem_ld_32x16(taddr + c0, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) part[(c0 + j) * kPM] = __uint_as_float(v[j]);
                }
                if constexpr (Rows) {
#pragma unroll
                    for (int j = 0; j < kRowsMax / 2; ++j)
                        if (j < mine) part[(lo + j) * kPM] += acc[j];
                }
            } else if (a.split == 1) {
                store_tile<Rows>(a, taddr, o, lane, r0, rows, ok, acc);
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
        const int r0 = first % a.row_tiles * a.bn, per = (a.bn + a.split - 1) / a.split;
        finish_split(a, cl, reinterpret_cast<float*>(st), &S.abort, a.split, 0, 1, first / a.row_tiles * kPM, r0, per * rank_in,
                     min(min(a.bn, a.n - r0), per * (rank_in + 1)), warp, kPThreads / 32, lane);
        cl.sync();   // peers have read this CTA's sums
    }
    if (Rows || a.counts) griddep_wait();   // this grid's end implies the first one's
    tc_fence_before();
    __syncthreads();
    if (S.abort) {   // no copy and no MMA may be in flight when the CTA leaves
        if (tid == 32) {   // the thread that issued the MMAs
            umma_commit(&S.last);
            mbar_wait(&S.last, 0, err);
        } else if (tid == 0) {
            const uint32_t n = min(blocks, (uint32_t)a.stages);
            for (uint32_t i = blocks - n; i < blocks; ++i) mbar_wait(&S.full[i % a.stages], (i / a.stages) & 1, err);
        }
        __syncthreads();
    }
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, acc_cols);
    }
}

// ---------------------------------------------------------------- the GEMM by CTA pairs
// Many tiles: what bounds them is the L2's rate into the SMs (about 9 TB/s
// here), so the tile is as large as the tensor memory of two SMs holds: 512
// output features x bn rows per pair, 96 KB per K block of 16.8 MFLOP (a
// single CTA's 128 x 256 tile needs three times that per FLOP, and measured
// 790 TFLOP/s).  cta_group::2 MMAs (M 256): CTA r of the pair holds rows
// 128 r .. of each 256 features and half of x's rows; the leader's thread
// issues for both.  Both accumulators (2 x bn columns) are in use, so a tile's
// epilogue is not overlapped; eight warps drain it, four per accumulator.
// Split tiles as above: up to four pairs in a cluster, each a part of the K axis.
struct PairSmem {
    uint64_t full[kPMaxStages], empty[kPMaxStages];
    uint64_t accF, accE[2], last, gone;
    uint32_t tmem;
    volatile uint32_t abort;
    uint32_t peer_blocks;   // of the leader: copies sent by the peer
    int ahead[kAhead];
    int ids[kRowsMax];
};
constexpr int kPairThreads = 384;   // warps: 0 TMA, 1 MMA (leader), 2 TMEM, 4..11 epilogue

__device__ __forceinline__ uint32_t map_rank(uint32_t addr, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Tiled loads of a pair: into this CTA's shared memory, completing on the leader's barrier.
__device__ __forceinline__ void pair_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void pair_load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(da), "l"(db), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive on the barrier at this offset in both CTAs when the MMAs issued so far have completed.
__device__ __forceinline__ void pair_commit(uint64_t* bar, int leader) {
    const uint16_t both = (uint16_t)(3 << leader);
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     smem_addr(bar)),
                 "h"(both)
                 : "memory");
}

// (bounded as if for more threads, so that a CTA of the first kernel finds registers on the SM: 128 or 96 each)
template <bool Rows>
__global__ void __launch_bounds__(Rows ? 512 : 640, 1)
    k_project_pair(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapX,
                   const __grid_constant__ CUtensorMap mapB, const __grid_constant__ CUtensorMap mapT, ProjectArgs a) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ PairSmem S;
    unsigned char* st = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ks = (int)cl.block_rank() >> 1, r = (int)cl.block_rank() & 1;
    const int half = a.bn / 2;
    const int stage_bytes = 2 * kPStageA + half * kPK * 2;
    const int first = blockIdx.x / (2 * a.split), step = a.split > 1 ? a.tiles : gridDim.x / 2;   // split: one tile per cluster
    const int kb0 = (int)((int64_t)a.kblocks * ks / a.split), kb1 = (int)((int64_t)a.kblocks * (ks + 1) / a.split);
    const int leader = 2 * ks;
    uint32_t* err = &g_project_err;
    auto stop = [&]() {   // a wait ran out: both CTAs of the pair end
        S.abort = 1;
        *const_cast<volatile uint32_t*>(cl.map_shared_rank(const_cast<uint32_t*>(&S.abort), leader + (r ^ 1))) = 1;
    };

    if (tid == 0) {
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(&S.full[i], 1);
            mbar_init(&S.empty[i], 1);
        }
        mbar_init(&S.accF, 1);
        mbar_init(&S.last, 1);
        mbar_init(&S.gone, 1);
        for (int m = 0; m < 2; ++m) mbar_init(&S.accE[m], 8);
        S.abort = 0;
        fence_barrier_init();
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&S.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    __syncwarp();
    tc_fence_before();
    cl.sync();   // the barriers of both CTAs exist before anything arrives at them
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    const int R16 = (a.rank + 15) & ~15;
    const bool one_block = 2 * R16 <= kPK;
    const int per_entry = one_block ? 1 : 2 * ((R16 + kPK - 1) / kPK);

    uint32_t blocks = 0;   // thread 0: copies sent by this CTA

    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            int use = 0;
            bool waited = false, in_time = true;
            auto slot = [&]() -> int {
                const int s = it % a.stages;
                if (!project_wait(&S.empty[s], ((it / a.stages) & 1) ^ 1, &S.abort, in_time)) {
                    stop();
                    return -1;
                }
                if (r == 0) mbar_arrive_expect_tx(&S.full[s], 2 * stage_bytes);   // what both CTAs bring
                ++it;
                return s;
            };
            for (int tile = first; tile < a.tiles && !S.abort; tile += step, ++use) {
                in_time = use < a.in_time;
                const int o0 = tile / a.row_tiles * (4 * kPM) + r * kPM, rt = tile % a.row_tiles, r0 = rt * a.bn + r * half;
                for (int kb = kb0; kb < kb1; ++kb) {
                    const int s = slot();
                    if (s < 0) break;
                    const uint32_t p = smem_addr(st + s * stage_bytes), bar = map_rank(smem_addr(&S.full[s]), leader);
                    pair_load_2d(p, &mapW, kb * kPK, o0, bar);
                    pair_load_2d(p + kPStageA, &mapW, kb * kPK, o0 + 2 * kPM, bar);
                    pair_load_2d(p + 2 * kPStageA, &mapX, kb * kPK, r0, bar);
                }
                if (!Rows && a.counts) {
                    if (!waited) {
                        griddep_wait();
                        asm volatile("fence.proxy.async.global;" ::: "memory");
                        waited = true;
                    }
                    const Entries entries{a.entry + rt * a.cap, S.ahead, __ldcg(a.counts + rt)};
                    for (int j = ks; j < entries.count && !S.abort; j += a.split) {
                        const int ad = entries.get(j, ks, a.split);
                        const int trow = (rt * a.cap + j) * a.bn + r * half;
                        for (int b = 0; b < per_entry; ++b) {
                            const int s = slot();
                            if (s < 0) break;
                            const uint32_t p = smem_addr(st + s * stage_bytes), bar = map_rank(smem_addr(&S.full[s]), leader);
                            const int c = (b >> 1) * kPK, piece = b & 1;
                            pair_load_3d(p, &mapB, c, o0, ad, bar);
                            pair_load_3d(p + kPStageA, &mapB, c, o0 + 2 * kPM, ad, bar);
                            pair_load_2d(p + 2 * kPStageA, &mapT, piece * R16 + c, trow, bar);
                        }
                    }
                }
            }
            blocks = it;
            if (r == 1)
                asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_rank(smem_addr(&S.peer_blocks), leader)), "r"(it) : "memory");
        }
    } else if (warp == 1) {
        if (lane == 0 && r == 0) {
            const uint32_t idesc = umma_idesc_bf16(2 * kPM, a.bn);
            uint32_t it = 0, use = 0;
            bool waited = false;
            for (int tile = first; tile < a.tiles && !S.abort; tile += step, ++use) {
                const int rt = tile % a.row_tiles;
                const bool in_time = (int)use < a.in_time;
                uint32_t fresh = 3;   // accumulators not yet begun
                auto block = [&](int na, int b0, bool again) -> bool {
                    const int s = it % a.stages;
                    if (!again) {
                        if (!project_wait(&S.full[s], (it / a.stages) & 1, &S.abort, in_time)) { stop(); return false; }
                        tc_fence_after();
                    }
                    const uint32_t p = smem_addr(st + s * stage_bytes);
                    const uint64_t db = umma_desc_sw128(p + 2 * kPStageA);
                    for (int m = 0; m < 2; ++m) {
                        if (fresh >> m & 1u) {   // the last tile's sums have been read
                            if (!project_wait(&S.accE[m], (use & 1) ^ 1, &S.abort, in_time)) { stop(); return false; }
                            tc_fence_after();
                        }
                        const uint64_t da = umma_desc_sw128(p + m * kPStageA);
                        for (int k = 0; k < na; ++k) {
                            pair_mma(tmem + m * a.bn, da + 2 * k, db + 2 * (b0 + k), idesc, !(fresh >> m & 1u));
                            fresh &= ~(1u << m);
                        }
                    }
                    return true;
                };
                auto next = [&]() {
                    pair_commit(&S.empty[it % a.stages], leader);
                    ++it;
                };
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!block(kPK / 16, 0, false)) break;
                    next();
                }
                if (!Rows && a.counts && !S.abort) {
                    if (!waited) {
                        griddep_wait();
                        waited = true;
                    }
                    const int count = __ldcg(a.counts + rt);
                    for (int j = ks; j < count && !S.abort; j += a.split)
                        for (int b = 0; b < per_entry; ++b) {
                            if (one_block) {
                                if (!block(R16 / 16, 0, false) || !block(R16 / 16, R16 / 16, true)) break;
                            } else if (!block(min(kPK, R16 - (b >> 1) * kPK) / 16, 0, false)) {
                                break;
                            }
                            next();
                        }
                }
                if (S.abort) break;   // (this thread's own, or another's: the tile is not to look complete)
                pair_commit(&S.accF, leader);
            }
        }
    } else if (warp >= 4) {
        const int qd = warp & 3, m = (warp - 4) >> 2;   // TMEM lanes 32 qd .., accumulator m
        uint32_t use = 0;
        bool ok = true;   // the same for the whole warp; a phase behind one that was given up would look complete
        float* ts = reinterpret_cast<float*>(st + a.stages * stage_bytes);
        if constexpr (Rows) stage_rows(a, ts, S.ids, 0, a.n, tid - 128, kPairThreads - 128);
        for (int tile = first; tile < a.tiles; tile += step, ++use) {
            const int o = tile / a.row_tiles * (4 * kPM) + m * (2 * kPM) + r * kPM + 32 * qd + lane, r0 = tile % a.row_tiles * a.bn;
            const int rows = min(a.bn, a.n - r0);
            float acc[Rows ? kRowsMax : 1];
            if constexpr (Rows) adapter_rows(a, ts, S.ids, o, rows, acc);
            ok = ok && __all_sync(0xffffffffu, project_wait(&S.accF, use & 1, &S.abort, (int)use < a.in_time));
            if (!ok && lane == 0) stop();
            tc_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(32 * qd) << 16) + m * a.bn;
            if (a.split > 1) break;   // the sums meet below
            store_tile<Rows>(a, taddr, o, lane, r0, rows, ok, acc);
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(map_rank(smem_addr(&S.accE[m]), leader))
                             : "memory");
        }
    }
    if (a.split > 1) {
        // the pairs' partial sums, one accumulator after the other through shared memory (its stages are done with),
        // each pair finishes its share of the rows in pair order
        const int r0 = first % a.row_tiles * a.bn, per = (a.bn + a.split - 1) / a.split;
        const int c1 = min(min(a.bn, a.n - r0), per * (ks + 1));
        for (int m = 0; m < 2; ++m) {
            if (warp >= 4 && (warp - 4) >> 2 == m) {
                const int qd = warp & 3;
                float* part = reinterpret_cast<float*>(st) + 32 * qd + lane;   // [bn][128]
                const uint32_t taddr = tmem + ((uint32_t)(32 * qd) << 16) + m * a.bn;
                for (int c0 = 0; c0 < a.bn; c0 += 16) {
                    uint32_t v[16];
                    tmem_ld_32x16(taddr + c0, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) part[(c0 + j) * kPM] = __uint_as_float(v[j]);
                }
            }
            __syncwarp();
            cl.sync();
            finish_split(a, cl, reinterpret_cast<float*>(st), &S.abort, 2 * a.split, r, 2,
                         first / a.row_tiles * (4 * kPM) + m * (2 * kPM) + r * kPM, r0, per * ks, c1, warp, kPairThreads / 32, lane);
            cl.sync();   // the peers have read this CTA's sums
        }
    }
    if (Rows || a.counts) griddep_wait();
    __syncwarp();
    tc_fence_before();
    cl.sync();   // neither CTA leaves while the other may still read its operands or signal its barriers
    if (S.abort) {   // (the same in both CTAs by now)
        // No copy and no MMA of either CTA may be in flight when the pair leaves.  All complete on the leader's barriers: it
        // waits for its own and the peer's (an empty stage lets neither run ahead of the other by more than the stages), the
        // peer for the leader.
        if (r == 0 && tid == 32) {   // the thread that issued the MMAs
            asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(&S.last)) : "memory");
            mbar_wait(&S.last, 0, err);
        }
        __syncthreads();
        if (r == 0 && tid == 0) {
            const uint32_t theirs = S.peer_blocks, all = max(blocks, theirs), n = min(all, (uint32_t)a.stages);
            for (uint32_t i = all - n; i < all; ++i) {
                uint64_t* bar = &S.full[i % a.stages];
                if (i >= blocks)   // the peer's half alone
                    mbar_arrive_expect_tx(bar, stage_bytes);
                else if (i >= theirs)   // both are expected, the peer's half does not come
                    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(stage_bytes)
                                 : "memory");
                mbar_wait(bar, (i / a.stages) & 1, err);
            }
            asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(map_rank(smem_addr(&S.gone), leader + 1))
                         : "memory");
        } else if (tid == 0) {
            bool gone = false;   // as long as the leader's waits may last
            for (int k = 0; k < a.stages + 2 && !gone; ++k) gone = mbar_wait(&S.gone, 0, err);
        }
        __syncthreads();
    }
    if (warp == 2) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
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

// Rows per tile (the N side of an MMA: a multiple of 16, up to 256), whether
// CTA pairs take 512 output features of them, and how many CTAs share a tile:
// what should end first.  A K block takes an SM the time in which the L2 brings
// its operands, 33 bytes a clock with all SMs reading (128 bytes per feature
// and row; the MMAs take less at every size here); a round of tiles some more
// clocks for its start and end, above all the pairs' epilogue.
// 4096 x 4096 x 4096: pairs of 240 rows, two rounds, 102 us; single CTAs 174 us.
// 500 x 2056 x 5001: single CTAs of 176 rows, 26 us; pairs of 80 rows 31 us.
static void project_tile(int n, int fin, int fout, ProjectWork& w) {
    constexpr int64_t n_sm = 148;   // the size of the work buffer must not depend on the current device
    const int64_t kb = (fin + kPK - 1) / kPK;
    // clusters that run at once with one CTA per SM (a cluster lies in one GPC)
    auto clusters = [](int64_t size) { return size <= 2 ? 74 : size <= 4 ? 33 : size <= 6 ? 22 : 15; };
    int64_t cost = INT64_MAX;
    const int widest = n <= 256 ? (n + 15) & ~15 : 256;
    for (int b = widest; b >= 16 && (b == widest || b >= 64); b -= 16) {
        const int64_t rows = (n + b - 1) / b, alone = rows * ((fout + kPM - 1) / kPM);
        for (int64_t split = 1; split <= 8; split *= 2) {
            if (split > 1 && (alone > clusters(split) || kb < 4 * split)) break;
            const int64_t rounds = (alone + n_sm - 1) / n_sm;
            const int64_t c = rounds * ((kb + split - 1) / split * (kPM + b) * 128 / 33 + 5000) + (split > 1 ? 3000 + b * 8 : 0);
            if (c < cost) cost = c, w.bn = b, w.pair = false, w.split = (int)split;
        }
        const int64_t both = rows * ((fout + 4 * kPM - 1) / (4 * kPM)), rounds = (both + n_sm / 2 - 1) / (n_sm / 2);
        for (int64_t split = 1; split <= 4; ++split) {
            if (split > 1 && (n <= kRowsMax || both > clusters(2 * split) || kb < 4 * split)) break;
            const int64_t c = rounds * ((kb + split - 1) / split * (2 * kPM + b / 2) * 128 / 33 + 8000 + b * 17) +
                              (split > 1 ? 14000 + b * 24 : 0);
            if (c < cost) cost = c, w.bn = b, w.pair = true, w.split = (int)split;
        }
    }
}

ProjectWork project_work(int n, int fin, int fout, int n_adapters, int rank) {
    ProjectWork w{};
    project_tile(n, fin, fout, w);
    w.row_tiles = (n + w.bn - 1) / w.bn;
    w.rows = n >= kRowsMin && n <= kRowsMax;
    w.cap = n_adapters < w.bn ? n_adapters : w.bn;
    auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
    w.off_entry = up((size_t)w.row_tiles * 4);
    w.off_t = w.off_entry + up((size_t)w.row_tiles * w.cap * 4);
    w.total = w.off_t + up((size_t)w.row_tiles * w.cap * w.bn * t_cols(rank) * 2);
    if (w.rows) w.off_t = 0, w.total = up((size_t)n * rank * 4);
    return w;
}

cudaError_t launch_project(ProjectArgs p, ShrinkArgs s, const ProjectWork& wk, const void* W, int n_sm,
                           cudaStream_t st) {
    p.bn = wk.bn;
    p.row_tiles = wk.row_tiles;
    p.cap = wk.cap;
    p.kblocks = (p.fin + kPK - 1) / kPK;
    const int features = wk.pair ? 4 * kPM : kPM;
    p.tiles = (p.fout + features - 1) / features * p.row_tiles;
    p.split = wk.split;
    const int stage = wk.pair ? 2 * kPStageA + p.bn / 2 * kPK * 2 : kPStageA + p.bn * kPK * 2;
    // with adapters, room for a CTA of the first kernel beside this one, so that W streams meanwhile (one row at
    // 4096 x 4096: 14 us, without it 19)
    const int t_bytes = p.rows ? (p.bn + p.split - 1) / p.split * p.rank * 4 : 0;
    const int room = p.rows || (p.counts && p.bn <= kRowsMax) ? kPSmemRows : p.counts && p.rank <= 64 ? kPSmemEntries : kPSmem;
    p.stages = (room - t_bytes) / stage < kPMaxStages ? (room - t_bytes) / stage : kPMaxStages;
    const int smem = 1024 + p.stages * stage + t_bytes;   // the partial sums of a split tile (512 bytes per row) fit as well

    CUtensorMap mW, mX, mB = {}, mT = {};
    cudaError_t e = encode(&mW, W, p.fin, p.fout, 1, 2, kPM);
    if (e == cudaSuccess) e = encode(&mX, s.x, p.fin, p.n, 1, 2, wk.pair ? p.bn / 2 : p.bn);
    if (e == cudaSuccess && p.counts) e = encode(&mB, p.B, p.rank, p.fout, s.n_adapters, 3, kPM);
    if (e == cudaSuccess && p.counts)
        e = encode(&mT, s.t, t_cols(p.rank), (uint64_t)p.row_tiles * p.cap * p.bn, 1, 2, wk.pair ? p.bn / 2 : p.bn);
    if (e != cudaSuccess) return e;

    if (p.counts || p.rows) {
        s.bn = p.bn;
        s.cap = p.cap;
        // CTAs per item: each at least four column blocks; eight where the items leave SMs idle
        const int items = p.cap + p.bn / (p.rows ? 16 : 64);   // at most, per tile
        s.split = 1;
        const int most = items * p.row_tiles * 8 <= 2 * n_sm ? 8 : 4;
        while (s.split < most && p.kblocks >= 8 * s.split) s.split *= 2;
        // clusters per tile: as many as it can have items, or as fill the SMs about four times over
        const int fill = 4 * n_sm / (s.split * p.row_tiles);
        const int y = items < fill ? items : fill < 4 ? 4 : fill;
        const dim3 grid(s.split, y, p.row_tiles);
        const int nt = (p.rank + 7) / 8;
        if (p.rows)
            e = nt <= 2 ? shrink_launch<2, 16>(s, grid, st) : nt <= 4 ? shrink_launch<4, 16>(s, grid, st)
                : nt <= 8 ? shrink_launch<8, 16>(s, grid, st) : shrink_launch<16, 16>(s, grid, st);
        else
            e = nt <= 2 ? shrink_launch<2, 64>(s, grid, st) : nt <= 4 ? shrink_launch<4, 64>(s, grid, st)
                : nt <= 8 ? shrink_launch<8, 64>(s, grid, st) : shrink_launch<16, 64>(s, grid, st);
        if (e != cudaSuccess) return e;
    }
    const auto kernel = p.rows ? (wk.pair ? k_project_pair<true> : k_project<true>)
                               : (wk.pair ? k_project_pair<false> : k_project<false>);
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPSmem + 1024);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    const int tiles_at_once = wk.pair ? n_sm / 2 : n_sm;
    const int tiles = p.split > 1 || p.tiles < tiles_at_once ? p.tiles : tiles_at_once;
    const int cluster = wk.pair ? 2 * p.split : p.split;
    cfg.gridDim = dim3((unsigned)(tiles * cluster));
    cfg.blockDim = dim3(wk.pair ? kPairThreads : kPThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    unsigned na = 0;
    if (cluster > 1) {
        at[na].id = cudaLaunchAttributeClusterDimension;
        at[na].val.clusterDim.x = (unsigned)cluster;
        at[na].val.clusterDim.y = at[na].val.clusterDim.z = 1;
        ++na;
    }
    if (p.counts || p.rows) {
        at[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[na].val.programmaticStreamSerializationAllowed = 1;
        ++na;
    }
    cfg.attrs = at;
    cfg.numAttrs = na;
    return cudaLaunchKernelEx(&cfg, kernel, mW, mX, mB, mT, p);
}

// One step reads and clears the word, so that an error set meanwhile on another
// stream is in this answer or in the next.  One reader at a time has g_project_taken.
static __global__ void k_take_project_error() { g_project_taken = atomicExch(&g_project_err, 0u); }

cudaError_t read_project_error(uint32_t* code, cudaStream_t st) {
    static std::mutex one;
    const std::lock_guard<std::mutex> lock(one);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = cfg.blockDim = dim3(1);
    cfg.stream = st;
    void* p = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&p, g_project_taken);
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, k_take_project_error);
    if (e == cudaSuccess) e = cudaMemcpyAsync(code, p, 4, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    return e;
}

}  // namespace ds4
