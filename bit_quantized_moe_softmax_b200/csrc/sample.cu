// sample.cu -- the next token of each row of logits: temperature, top-k, top-p
// and min-p, then one draw by a given uniform number.
//
// With M the row's largest logit and w_i = exp((l_i - M) / T), all three
// filters keep a prefix of the tokens ordered by (logit desc, index asc), so
// the kept set is "key above a threshold, and the first q of the tokens at
// it" (key: the logit's bits in an order-preserving form) and no sort is
// needed.  The draw goes through the kept tokens by index: the first whose
// running sum of weights exceeds u times their total.
//
// Weights are held as integers, round(w 2^44) (at most 2^18 tokens, so sums
// stay below 2^63): their sums are exact in any order, so that atomics and
// the split of a row over CTAs cannot change a result.  exp is taken in
// binary64, since a draw near a border is decided by the weights' last bits.
//
// A row belongs to a cluster of up to eight CTAs that keep it in shared memory
// as binary32 (up to 32,768 tokens each): one read of the logits from HBM,
// every further pass is on chip, and sums meet through distributed shared
// memory.  A filter's threshold is found by histograms of 2,048 bins: first
// over (M - l) / T in steps of 1/64, then, inside the bin that holds the
// prefix's end, over the keys' bits (at most three rounds, usually one or two).
#include <cooperative_groups.h>

#include "ds4moe_internal.cuh"
#include "ops.cuh"

namespace cg = cooperative_groups;

namespace ds4 {

namespace {

constexpr int kST = 512;             // threads
constexpr int kSW = kST / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr uint32_t kAll = 0xffffffffu;
constexpr double kOne = 17592186044416.0;   // 2^44
constexpr float kNegInf = -INFINITY;

typedef unsigned long long u64;

struct SampleSmem {
    u64 hist[kBins];
    u64 wsum[kSW];
    u64 slice_tot[kMaxCluster];      // written by the peers
    u64 mass[kMaxCluster];
    u64 found_before;
    uint32_t found_bin;
    uint32_t wtie[kSW];
    float mx[kMaxCluster];
    uint32_t klo[kMaxCluster], khi[kMaxCluster];
    uint32_t ties[kMaxCluster];
    float wmax[kSW];
    uint32_t wlo[kSW], whi[kSW];
};

__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// exp((l - M) / T) of one token in binary64; tokens at -infinity weigh nothing,
// and where M is +infinity only the tokens there weigh (the limit).
struct Weigh {
    double M, inv;
    bool top_inf;
    __device__ __forceinline__ double operator()(float l) const {
        if (l == kNegInf) return 0.0;
        if (top_inf) return l == INFINITY ? 1.0 : 0.0;
        const double d = ((double)l - M) * inv;
        return d < -31.2 ? 0.0 : exp(d);   // e^-31.2 is half a unit of 2^-44: rounds to zero
    }
    __device__ __forceinline__ u64 units(float l) const { return (u64)__double2ll_rn((*this)(l) * kOne); }
};

// Bin of the first histogram: monotone in l, so any rounding is as good.
struct Coarse {
    float M, finv;
    bool top_inf;
    __device__ __forceinline__ uint32_t operator()(float l) const {
        if (top_inf) return l == INFINITY ? 0u : (uint32_t)(kBins - 1);
        return min((uint32_t)__float2int_rz((M - l) * finv), (uint32_t)(kBins - 1));   // NaN (0 * inf) gives 0
    }
};

// The histogram's first bin at which the running sum over all CTAs of the
// cluster reaches target, and the sum before it; false if the total is below.
// Every CTA's hist must be complete (this starts with a cluster barrier).
__device__ bool find_bin(cg::cluster_group& cl, SampleSmem& S, u64 target, uint32_t& bin, u64& before) {
    const int C = (int)cl.num_blocks(), r = (int)cl.block_rank(), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = kBins / C;   // this CTA's share of the bins
    const int each = (per + kST - 1) / kST;   // consecutive bins per thread
    cl.sync();
    u64 v[kBins / kST], sum = 0;
#pragma unroll
    for (int j = 0; j < kBins / kST; ++j) {
        v[j] = 0;
        const int b = tid * each + j;
        if (j < each && b < per) {
            for (int p = 0; p < C; ++p) v[j] += cl.map_shared_rank(S.hist, p)[r * per + b];
        }
        sum += v[j];
    }
    u64 inc = sum;   // inclusive scan over the CTA's threads
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const u64 o = __shfl_up_sync(kAll, inc, m);
        if (lane >= m) inc += o;
    }
    if (lane == 31) S.wsum[warp] = inc;
    __syncthreads();
    u64 base = 0, tot = 0;
#pragma unroll
    for (int w = 0; w < kSW; ++w) {
        if (w < warp) base += S.wsum[w];
        tot += S.wsum[w];
    }
    if (tid < C) cl.map_shared_rank(S.slice_tot, tid)[r] = tot;
    cl.sync();
    u64 all = 0;
    for (int p = 0; p < C; ++p) {
        if (p < r) base += S.slice_tot[p];
        all += S.slice_tot[p];
    }
    u64 cum = base + inc - sum;
    if (all >= target) {
#pragma unroll
        for (int j = 0; j < kBins / kST; ++j) {
            if (cum < target && cum + v[j] >= target) {   // one thread of the cluster
                for (int p = 0; p < C; ++p) {
                    SampleSmem* o = cl.map_shared_rank(&S, p);
                    o->found_bin = (uint32_t)(r * per + tid * each + j);
                    o->found_before = cum;
                }
            }
            cum += v[j];
        }
    }
    cl.sync();
    bin = S.found_bin;
    before = S.found_before;
    return all >= target;
}

}  // namespace

template <bool BF>
__global__ void __launch_bounds__(kST) k_sample(SampleArgs a) {
    extern __shared__ float vals[];   // [slice]
    __shared__ SampleSmem S;
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), r = (int)cl.block_rank(), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / C;
    const int begin = r * a.slice;
    const int cnt = max(0, min(a.V - begin, a.slice));

    // ---- the row into shared memory, and its maximum; a NaN counts as -infinity
    float mx = kNegInf;
    auto take = [&](int i, float v) {
        v = v == v ? v + 0.f : kNegInf;   // -0 and +0 tie
        vals[i] = v;
        mx = fmaxf(mx, v);
    };
    {
        const char* src = static_cast<const char*>(a.logits) + (row * a.ld + begin) * (BF ? 2 : 4);
        int done = 0;
        if (((uintptr_t)src & 15) == 0) {
            constexpr int E = BF ? 8 : 4;
            const int nv = cnt / E;
#pragma unroll 4
            for (int i = tid; i < nv; i += kST) {
                const uint4 w = ld_stream_v4(src + (size_t)i * 16);
                const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (BF) {
                        take(i * 8 + 2 * j, __uint_as_float(x[j] << 16));
                        take(i * 8 + 2 * j + 1, __uint_as_float(x[j] & 0xffff0000u));
                    } else {
                        take(i * 4 + j, __uint_as_float(x[j]));
                    }
                }
            }
            done = nv * E;
        }
#pragma unroll 4
        for (int i = done + tid; i < cnt; i += kST) {
            if constexpr (BF) take(i, __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(src)[i] << 16));
            else take(i, reinterpret_cast<const float*>(src)[i]);
        }
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, m));
    if (lane == 0) S.wmax[warp] = mx;
    __syncthreads();
    for (int w = 0; w < kSW; ++w) mx = fmaxf(mx, S.wmax[w]);
    if (tid < C) cl.map_shared_rank(S.mx, tid)[r] = mx;
    cl.sync();
    for (int p = 0; p < C; ++p) mx = fmaxf(mx, S.mx[p]);

    float* probs = a.probs ? a.probs + row * a.V + begin : nullptr;
    if (mx == kNegInf) {   // nothing to draw from
        if (probs)
            for (int i = tid; i < cnt; i += kST) probs[i] = 0.f;
        if (r == 0 && tid == 0) {
            a.token[row] = -1;
            if (a.prob) a.prob[row] = 0.f;
        }
        return;
    }

    // ---- this row's parameters
    float T = a.temp ? a.temp[row] : 1.f;
    int K = a.top_k ? a.top_k[row] : 0;
    float P = a.top_p ? a.top_p[row] : 1.f, mp = a.min_p ? a.min_p[row] : 0.f, u = a.u[row];
    if (!(T > 0.f)) T = 1.f, K = 1, P = 1.f, mp = 0.f, u = 0.f;   // greedy: the first token of the order
    const bool by_k = K >= 1 && K < a.V, by_p = P < 1.f, by_m = mp > 0.f;
    const double minw = fmin((double)mp, 1.0);
    const double inv = 1.0 / (double)T;
    const Weigh weigh{(double)mx, inv, mx == INFINITY};
    const Coarse coarse{mx, (float)(inv * 64.0), mx == INFINITY};

    // ---- the prefix that top-k and top-p keep: keys above kt, and q of those at kt
    uint32_t kt = 0;
    u64 q = ~0ull;
    for (int pass = 0; pass < 2; ++pass) {
        const bool mass = pass == 1;
        if (!(mass ? by_p : by_k)) continue;
        // what a token adds: one, or its weight; the tokens at a top-k threshold add the weight of q of them once
        auto adds = [&](float l) -> u64 {
            if (!mass) return 1;
            return order_key(l) > kt || q == ~0ull ? weigh.units(l) : 0;
        };
        auto tie_mass = [&](float l) -> u64 { return q * weigh.units(l); };
        const bool tied = mass && q != ~0ull;   // a top-k threshold is set
        float kt_val = 0.f;
        if (tied) kt_val = __uint_as_float(kt & 0x80000000u ? kt ^ 0x80000000u : ~kt);
        auto clear = [&]() {
            for (int i = tid; i < kBins; i += kST) S.hist[i] = 0;
            __syncthreads();
        };
        clear();
        u64 total = 0;
        for (int i = tid; i < cnt; i += kST) {
            const float l = vals[i];
            if (l == kNegInf || (mass && order_key(l) < kt)) continue;
            const u64 v = adds(l);
            if (v) atomicAdd(&S.hist[coarse(l)], v);
            total += v;
        }
        if (tied && r == 0 && tid == 0) {
            const u64 v = tie_mass(kt_val);
            atomicAdd(&S.hist[coarse(kt_val)], v);
            total += v;
        }
        u64 target = (u64)K;
        if (mass) {   // p of the total
#pragma unroll
            for (int m = 16; m >= 1; m >>= 1) total += __shfl_xor_sync(kAll, total, m);
            if (lane == 0) S.wsum[warp] = total;
            __syncthreads();
            total = 0;
            for (int w = 0; w < kSW; ++w) total += S.wsum[w];
            if (tid < C) cl.map_shared_rank(S.mass, tid)[r] = total;
            cl.sync();
            total = 0;
            for (int p = 0; p < C; ++p) total += S.mass[p];
            target = max(1ull, (u64)__double2ll_ru(fmax((double)P, 0.0) * (double)total));
            target = min(target, total);
        }
        uint32_t bin;
        u64 before;
        if (!find_bin(cl, S, target, bin, before)) continue;   // top-k of more tokens than there are
        // the keys of that bin
        uint32_t lo = 0xffffffffu, hi = 0;
        for (int i = tid; i < cnt; i += kST) {
            const float l = vals[i];
            if (l != kNegInf && coarse(l) == bin) {
                const uint32_t k = order_key(l);
                if (!mass || k >= kt) lo = min(lo, k), hi = max(hi, k);
            }
        }
        lo = __reduce_min_sync(kAll, lo);
        hi = __reduce_max_sync(kAll, hi);
        if (lane == 0) S.wlo[warp] = lo, S.whi[warp] = hi;
        __syncthreads();
        for (int w = 0; w < kSW; ++w) lo = min(lo, S.wlo[w]), hi = max(hi, S.whi[w]);
        if (tid < C) {
            cl.map_shared_rank(S.klo, tid)[r] = lo;
            cl.map_shared_rank(S.khi, tid)[r] = hi;
        }
        cl.sync();
        for (int p = 0; p < C; ++p) lo = min(lo, S.klo[p]), hi = max(hi, S.khi[p]);
        while (lo < hi) {
            const int shift = max(0, 32 - __clz(hi - lo) - 11);
            clear();
            for (int i = tid; i < cnt; i += kST) {
                const float l = vals[i];
                const uint32_t k = order_key(l);
                if (k >= lo && k <= hi && l != kNegInf && (!mass || k >= kt)) {
                    const u64 v = adds(l);
                    if (v) atomicAdd(&S.hist[(hi - k) >> shift], v);
                }
            }
            if (tied && r == 0 && tid == 0 && kt >= lo && kt <= hi) atomicAdd(&S.hist[(hi - kt) >> shift], tie_mass(kt_val));
            uint32_t sub;
            u64 rel;
            if (!find_bin(cl, S, target - before, sub, rel)) break;
            before += rel;
            hi -= sub << shift;
            lo = max(lo, hi - ((1u << shift) - 1u));
        }
        kt = hi;
        if (mass) {
            const u64 w = weigh.units(__uint_as_float(kt & 0x80000000u ? kt ^ 0x80000000u : ~kt));
            q = w ? (target - before + w - 1) / w : 1;
        } else {
            q = target - before;
        }
    }

    // ---- the tokens at the threshold, in index order: how many lie before this warp's
    const int seg = ((cnt + kSW - 1) / kSW + 31) & ~31;
    const int s0 = min(cnt, warp * seg), s1 = min(cnt, s0 + seg);
    u64 tie0 = 0;
    const bool limited = q != ~0ull;
    if (limited) {
        uint32_t t = 0;
        for (int i = s0 + lane; i < s1; i += 32) t += order_key(vals[i]) == kt;
        t = __reduce_add_sync(kAll, t);
        if (lane == 0) S.wtie[warp] = t;
        __syncthreads();
        uint32_t mine = 0, all = 0;
        for (int w = 0; w < kSW; ++w) {
            if (w < warp) mine += S.wtie[w];
            all += S.wtie[w];
        }
        if (tid < C) cl.map_shared_rank(S.ties, tid)[r] = all;
        cl.sync();
        tie0 = mine;
        for (int p = 0; p < r; ++p) tie0 += S.ties[p];
    }
    // weight of element i (this lane's of a step of 32) if it is kept, else 0; counts ties on
    auto kept = [&](int i, u64& tie) -> double {
        const float l = i < s1 ? vals[i] : kNegInf;
        const uint32_t k = order_key(l);
        bool in = l != kNegInf && k >= kt;
        if (limited) {
            const bool at = i < s1 && k == kt;
            const uint32_t b = __ballot_sync(kAll, at);
            if (at && tie + __popc(b & ((1u << lane) - 1u)) >= q) in = false;
            tie += __popc(b);
        }
        if (!__any_sync(kAll, in)) return 0.0;
        const double w = in ? weigh(l) : 0.0;
        return by_m && w < minw ? 0.0 : w;
    };

    // ---- their total, and each warp's share
    u64 sum = 0, tie = tie0;
    for (int i0 = s0; i0 < s1; i0 += 32) sum += (u64)__double2ll_rn(kept(i0 + lane, tie) * kOne);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(kAll, sum, m);
    __syncthreads();   // S.wsum of find_bin has been read
    if (lane == 0) S.wsum[warp] = sum;
    __syncthreads();
    u64 base = 0, all = 0;
    for (int w = 0; w < kSW; ++w) {
        if (w < warp) base += S.wsum[w];
        all += S.wsum[w];
    }
    if (tid < C) cl.map_shared_rank(S.slice_tot, tid)[r] = all;
    cl.sync();
    u64 total = 0;
    for (int p = 0; p < C; ++p) {
        if (p < r) base += S.slice_tot[p];
        total += S.slice_tot[p];
    }
    const double norm = kOne / (double)total;

    // ---- the draw: the first kept token whose running sum exceeds u of the total
    const double x = (double)u * (double)total;
    const u64 target = !(x > 0.0) ? 0 : x >= (double)total ? total - 1 : min((u64)x, total - 1);
    if (target >= base && target < base + sum) {   // one warp of the cluster
        u64 run = base;
        tie = tie0;
        for (int i0 = s0; i0 < s1; i0 += 32) {
            const double w = kept(i0 + lane, tie);
            u64 inc = (u64)__double2ll_rn(w * kOne);
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const u64 o = __shfl_up_sync(kAll, inc, m);
                if (lane >= m) inc += o;
            }
            const uint32_t b = __ballot_sync(kAll, run + inc > target);
            if (b) {
                if (lane == __ffs(b) - 1) {
                    a.token[row] = begin + i0 + lane;
                    if (a.prob) a.prob[row] = (float)(w * norm);
                }
                break;
            }
            run += __shfl_sync(kAll, inc, 31);
        }
    }
    if (probs) {
        tie = tie0;
        for (int i0 = s0; i0 < s1; i0 += 32) {
            const double w = kept(i0 + lane, tie);
            if (i0 + lane < s1) probs[i0 + lane] = (float)(w * norm);
        }
    }
}

cudaError_t launch_sample(SampleArgs a, bool bf16, int n, cudaStream_t st) {
    // CTAs per row: a quarter to the whole of a CTA's 32,768-token share each
    int C = 1;
    while (C < kMaxCluster && (a.V + C - 1) / C > 8192) C *= 2;
    a.slice = (((a.V + C - 1) / C) + 7) & ~7;
    const size_t smem = (size_t)a.slice * sizeof(float);
    const void* fn = bf16 ? reinterpret_cast<const void*>(k_sample<true>) : reinterpret_cast<const void*>(k_sample<false>);
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kSampleMaxVocab / kMaxCluster * 4));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)n * C);
    cfg.blockDim = dim3(kST);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)C;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    void* args[] = {&a};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace ds4
