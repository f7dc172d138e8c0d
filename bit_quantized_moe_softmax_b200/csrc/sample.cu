// sample.cu -- the next token of each row of logits: temperature, top-k, top-p
// and min-p, then one draw by a given uniform number.
//
// With M the row's largest logit and w_i = exp((l_i - M) / T), all three
// filters keep a prefix of the tokens ordered by (logit desc, index asc): the
// tokens above a logit, and those at it up to an index.  So no sort of the row
// is needed.  The draw goes through the kept tokens by index: the first whose
// running sum of weights exceeds u times their total.
//
// Weights are held as integers, round(w 2^44) (at most 2^18 tokens, so sums
// stay below 2^63): their sums are exact in any order, so that atomics and
// the split of a row over CTAs cannot change a result.  exp is taken in
// binary64, since a draw near a border is decided by the weights' last bits.
//
// A row belongs to a cluster of up to sixteen CTAs that keep it in shared memory
// as binary32 (up to 32,768 tokens each): one read of the logits from HBM,
// every further pass is on chip, and sums meet through distributed shared
// memory.  A filter's threshold is found by histograms of 2,048 bins: first
// over M - l in small steps (for a small top-k, of each thread's largest logit
// alone); the tokens of the bin that holds the prefix's end are then sorted, or,
// where there are more than 512 (logits of few bits have many ties), counted
// over their keys' bits.  Where all tokens down to that bin are at most 512,
// they are sorted together and the remaining filters and the draw need no
// other.  131,072 binary32 logits: one row 8 us without filters, 15 with all;
// 256 rows 109 us without, 292 with top-p (7 % of HBM's rate).  No unit is full
// there (issue slots 56 %, ALU 41 %, the shared-memory pipe 42 %): seven warps per
// scheduler wait for dependent instructions, shared memory and barriers.
#include <cooperative_groups.h>

#include "ds4moe_internal.cuh"
#include "ops.cuh"

namespace cg = cooperative_groups;

namespace ds4 {

namespace {

constexpr int kST = 512;             // threads
constexpr int kSW = kST / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 16;
constexpr uint32_t kAll = 0xffffffffu;
constexpr int kList = kST;                  // tokens of one bin that are put in order at once
constexpr int kTab = 128;                   // entries of the table of 2^(j / 128)
constexpr double kOne = 17592186044416.0;   // 2^44
constexpr double kMagic = 6755399441055744.0;   // 1.5 * 2^52: adding it leaves the nearest integer in the low bits
constexpr float kNegInf = -INFINITY;

typedef unsigned long long u64;
constexpr u64 kOffset = 0x4338000000000000ull;   // kMagic's bits

struct __align__(16) SampleSmem {
    uint32_t hist[2][2][kBins];      // two in turn: counts in the first array, or the low and high words of weights
    u64 group[2][kMaxCluster][32];   // sums of 64 bins of each CTA, written by the peers; two in turn
    u64 list[kList];                 // this CTA's tokens of a bin, then all of them in order
    uint32_t listed[kMaxCluster];    // how many there are in each CTA
    uint32_t list_n;
    double tab[kTab];
    u64 wsum[kSW];
    u64 slice_tot[kMaxCluster];      // written by the peers
    uint32_t wtie[kSW];
    float mx[kMaxCluster];
    uint32_t klo[kMaxCluster], khi[kMaxCluster];
    uint32_t ties[kMaxCluster];
    int tie_at;
    float wmax[kSW];
    uint32_t wlo[kSW], whi[kSW];
};

__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

// The largest binary32 value below a finite one (not -0).
__device__ __forceinline__ float next_below(float m) {
    return __uint_as_float(m > 0.f ? __float_as_uint(m) - 1 : m < 0.f ? __float_as_uint(m) + 1 : 0x80000001u);
}

// exp((l - M) / T) of one token in binary64: 2^(y / 128), y = (l - M) 128
// log2(e) / T, from a table of 2^(j / 128) and four terms of the series of
// 2^(r / 128), |r| <= 1/2 (a little more, as binary32 finds the nearest
// integer): the fifth is below 2e-15, a twentieth of the unit 2^-44.  The
// passes over the weights are chains of dependent instructions with few warps to
// hide them, so every one counts: the integer n comes from a binary32 addition and is used
// with its offset (which the table index and the exponent drop by themselves),
// logits far below are raised to where the weight is 2^-64 instead of being
// tested for, and the unit's sums keep the offset of the conversion.
struct Weigh {
    double M, c;           // c = 128 log2(e) / T, at most where one step below M already weighs nothing
    float half, c2;        // M / 2 and 2 c: no difference of two finite halves overflows
    double reach;          // 8192 / c
    float low;             // M - reach
    bool flat;             // T so large that low is the lowest binary32 value: -infinity is tested for
    const double* tab;

    // before the row's maximum is known
    __device__ __forceinline__ void set_temperature(float T, const double* table) {
        c = fmin(kTab * 1.44269504088896340736 / (double)T, 1e38);   // (1e38: for set_maximum, which lowers such a c)
        reach = fmax(8192.0 / (kTab * 1.44269504088896340736) * (double)T, 8192e-38);   // 8192 / c
        tab = table;
    }
    __device__ __forceinline__ void set_maximum(float m) {
        const float below = next_below(m);
        // a power of two (2^104 at the lowest value), and 1 / step by its exponent
        const double step = below == kNegInf ? 0x1p104 : (double)m - (double)below;
        const double most = 6000.0 * __hiloint2double(0x7fe00000 - __double2hiint(step), 0);
        if (c > most) c = most, reach = 8192.0 / 6000.0 * step;
        M = m, half = 0.5f * m;
        c2 = (float)(2.0 * c);
        const double l = (double)m - reach;
        flat = !(l > -3.4e38);
        low = flat ? -3.402823466e38f : __double2float_rd(l);
    }
    __device__ __forceinline__ double operator()(float l) const {
        l = fmaxf(l, low);
        const int n = __float_as_int(fmaf(fmaf(l, 0.5f, -half), c2, 12582912.f));        // 0x4b400000 + the nearest integer of y
        const double k = __hiloint2double(0x43300000, n) - (4503599627370496.0 + 1262485504.0);
        const double r = fma((double)l - M, c, -k);
        constexpr double h = 0.69314718055994530942 / kTab;
        double p = fma(r, h * h * h * h / 24.0, h * h * h / 6.0);
        p = fma(r, p, h * h / 2.0);
        p = fma(r, p, h);
        p *= r;
        double w = tab[n & (kTab - 1)];
        w = fma(w, p, w);
        return __hiloint2double(__double2hiint(w) + ((n & ~(kTab - 1)) << 13), __double2loint(w));
    }
    static __device__ __forceinline__ u64 offset_units(double w) { return (u64)__double_as_longlong(fma(w, kOne, kMagic)); }
    static __device__ __forceinline__ u64 to_units(double w) { return offset_units(w) - kOffset; }
    // of any token
    __device__ __forceinline__ u64 units(float l) const {
        u64 v = to_units((*this)(l));
        if (flat && l == kNegInf) v = 0;
        return v;
    }
};

// Bin of the first histogram: (M - l) in steps, the last bin for all beyond.
// Monotone in l, so any rounding is as good, and a difference that overflows
// falls into the last bin like all far ones.
struct Coarse {
    float M, step;   // 1 / step length, between 1e-38 and 1e38: no product of 0 and infinity
    __device__ __forceinline__ uint32_t operator()(float l) const {
        return __float_as_uint(fminf((M - l) * step, (float)(kBins - 1)) + 8388608.f) - 0x4b000000u;
    }
};

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(kAll, v, m);
    return v;
}
__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {   // inclusive
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const u64 o = __shfl_up_sync(kAll, v, m);
        if (lane >= m) v += o;
    }
    return v;
}

// The first meeting of a cluster's CTAs in two halves: shared memory of a peer may
// be written only once the peer runs, and between the halves the row is read.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Sums of 64 bins of this CTA's histogram `buf` to every CTA of the cluster.
// The histogram must be complete; a cluster barrier follows before find_bin.
template <int C>
__device__ __forceinline__ void push_groups(cg::cluster_group& cl, SampleSmem& S, int buf, bool wide) {
    static_assert(kBins == 4 * kST, "four bins per thread");
    const int r = C == 1 ? 0 : (int)cl.block_rank(), tid = threadIdx.x;
    const uint4 lo = reinterpret_cast<const uint4*>(S.hist[buf][0])[tid];
    u64 v = (u64)lo.x + lo.y + lo.z + lo.w;
    if (wide) {
        const uint4 hi = reinterpret_cast<const uint4*>(S.hist[buf][1])[tid];
        v += ((u64)hi.x + hi.y + hi.z + hi.w) << 32;
    }
#pragma unroll
    for (int m = 8; m >= 1; m >>= 1) v += __shfl_xor_sync(kAll, v, m);
    const int p = tid & 15;   // sixteen threads hold the sum
    if (p < C) cl.map_shared_rank(&S.group[0][0][0], p)[(buf * kMaxCluster + r) * 32 + (tid >> 4)] = v;
}

// After the barrier: the sum of this histogram over the cluster.
template <int C>
__device__ __forceinline__ u64 group_scan(SampleSmem& S, int buf, int lane, u64& inc, u64& mine) {
    mine = 0;
#pragma unroll
    for (int p = 0; p < C; ++p) mine += S.group[buf][p][lane];
    inc = warp_scan(mine, lane);
    return __shfl_sync(kAll, inc, 31);
}

// The histogram's first bin at which the running sum over the cluster reaches
// target (1 .. its total), the sum before it and the bin's own.  Every CTA
// reads the 64 bins of one group from its peers and finds the same answer.
template <int C>
__device__ __noinline__ void find_bin(SampleSmem& S, int buf, bool wide, u64 target, uint32_t& bin, u64& before,
                                      u64& own) {
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31;
    u64 inc, mine;
    group_scan<C>(S, buf, lane, inc, mine);
    const int g = __ffs(__ballot_sync(kAll, inc >= target)) - 1;
    before = __shfl_sync(kAll, inc - mine, g);
    u64(*part)[64] = reinterpret_cast<u64(*)[64]>(S.hist[buf ^ 1]);   // whose readers have passed a barrier
    for (int i = tid; i < 64 * C; i += kST) {
        const uint32_t* h = cl.map_shared_rank(&S.hist[0][0][0], i >> 6) + 2 * buf * kBins + g * 64 + (i & 63);
        const uint32_t lo = h[0], hi = wide ? h[kBins] : 0u;
        part[i >> 6][i & 63] = (u64)lo | ((u64)hi << 32);
    }
    __syncthreads();
    u64 a = 0, b = 0;   // bins 2 lane, 2 lane + 1
#pragma unroll
    for (int p = 0; p < C; ++p) {
        const ulonglong2 v = reinterpret_cast<const ulonglong2*>(part[p])[lane];
        a += v.x, b += v.y;
    }
    inc = warp_scan(a + b, lane);
    const int at = __ffs(__ballot_sync(kAll, before + inc >= target)) - 1;
    u64 pre = before + inc - a - b;
    const bool second = pre + a < target;
    if (second) pre += a;
    bin = __shfl_sync(kAll, (uint32_t)(g * 64 + 2 * lane + second), at);
    own = __shfl_sync(kAll, second ? b : a, at);
    before = __shfl_sync(kAll, pre, at);
    __syncthreads();   // part is free again
}

// The sum that the running sum has to exceed: u of the total, the last unit at most.
__device__ __forceinline__ u64 draw_target(float u, u64 total) {
    const double x = (double)u * (double)total;
    return !(x > 0.0) ? 0 : x >= (double)total ? total - 1 : min((u64)x, total - 1);
}

// A token in the order of the filters, largest first: key, then the lower index.
__device__ __forceinline__ u64 order_of(uint32_t key, int idx) { return ((u64)key << 32) | (uint32_t)~idx; }

// One value per thread of the CTA, sorted: thread 0 gets the largest (bitonic
// network: steps inside a warp by shuffles, the others through shared memory).
__device__ __noinline__ u64 sort_desc(SampleSmem& S, u64 v) {
    const int tid = threadIdx.x;
    for (int k = 2; k <= kST; k <<= 1) {
        for (int j = k >> 1; j > 0; j >>= 1) {
            u64 o;
            if (j >= 32) {
                S.list[tid] = v;
                __syncthreads();
                o = S.list[tid ^ j];
                __syncthreads();
            } else {
                o = __shfl_xor_sync(kAll, v, j);
            }
            const bool larger = ((tid & j) == 0) == ((tid & k) == 0);   // this thread keeps the larger one
            if (larger == (o > v)) v = o;
        }
    }
    return v;
}

}  // namespace

// (sixteen CTAs, for a few rows: all registers, 16.0 -> 14.7 us; else two CTAs per SM, 290 against 390 us for 256 rows)
template <bool BF, int C>
__global__ void __launch_bounds__(kST, C == 16 ? 1 : 2) k_sample(SampleArgs a) {
    extern __shared__ __align__(16) float vals[];   // [kSW][a.seg]: each warp's share of the CTA's tokens, in index order
    __shared__ SampleSmem S;
    if (C > 1) cluster_arrive();
    cg::cluster_group cl = cg::this_cluster();
    const int r = C == 1 ? 0 : (int)cl.block_rank(), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / C;
    const int begin = r * a.slice;
    const int cnt = max(0, min(a.V - begin, a.slice));

    // ---- this row's parameters
    float T = a.temp ? a.temp[row] : 1.f;
    int K = a.top_k ? a.top_k[row] : 0;
    float P = a.top_p ? a.top_p[row] : 1.f, mp = a.min_p ? a.min_p[row] : 0.f, u = a.u[row];
    if (!(T > 0.f)) T = 1.f, K = 1, P = 1.f, mp = 0.f, u = 0.f;   // greedy: the first token of the order
    // min-p from 1 on: the tokens at the maximum alone, whatever else has a weight that rounds to 1 (at T infinite all
    // weigh 1, and are kept)
    if (mp >= 1.f) mp = T < INFINITY ? 1.f : 0.5f;

    double inv = 1.0 / (double)T;
    Weigh weigh;
    weigh.set_temperature(T, S.tab);

    // ---- the row into shared memory, and its maximum; a NaN counts as -infinity
    float mx = kNegInf;
    auto clean = [&](float v) {
        v = v == v ? v + 0.f : kNegInf;   // -0 and +0 tie
        mx = fmaxf(mx, v);
        return v;
    };
    {
        const char* src = static_cast<const char*>(a.logits) + (row * a.ld + begin) * (BF ? 2 : 4);
        int done = 0;
        if (((uintptr_t)src & 15) == 0) {
            constexpr int E = BF ? 8 : 4;
            const int nv = cnt / E;
#pragma unroll 8
            for (int i = tid; i < nv; i += kST) {
                const uint4 w = ld_stream_v4(src + (size_t)i * 16);
                const uint32_t x[4] = {w.x, w.y, w.z, w.w};
                float4* d = reinterpret_cast<float4*>(vals + i * E);
                if constexpr (BF) {
                    float f[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        f[2 * j] = clean(__uint_as_float(x[j] << 16));
                        f[2 * j + 1] = clean(__uint_as_float(x[j] & 0xffff0000u));
                    }
                    d[0] = make_float4(f[0], f[1], f[2], f[3]);
                    d[1] = make_float4(f[4], f[5], f[6], f[7]);
                } else {
                    d[0] = make_float4(clean(__uint_as_float(x[0])), clean(__uint_as_float(x[1])),
                                       clean(__uint_as_float(x[2])), clean(__uint_as_float(x[3])));
                }
            }
            done = nv * E;
        }
#pragma unroll 8
        for (int i = done + tid; i < cnt; i += kST) {
            if constexpr (BF) vals[i] = clean(__uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(src)[i] << 16));
            else vals[i] = clean(reinterpret_cast<const float*>(src)[i]);
        }
        for (int i = cnt + tid; i < kSW * a.seg; i += kST) vals[i] = kNegInf;
    }
    if (tid < kTab) {   // 2^(tid / 128) from the powers of its bits
        const double power[7] = {1.0054299011128027, 1.0108892860517005, 1.0218971486541166, 1.0442737824274138,
                                 1.0905077326652577, 1.189207115002721,  1.4142135623730951};
        double w = 1.0;
#pragma unroll
        for (int b = 0; b < 7; ++b) w *= tid >> b & 1 ? power[b] : 1.0;
        S.tab[tid] = w;
    }
    float own_max = mx;   // of the tokens that this thread brought
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, m));
    if (lane == 0) S.wmax[warp] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSW; ++w) mx = fmaxf(mx, S.wmax[w]);
    if (C > 1) {
        cluster_wait();
        if (tid < C) cl.map_shared_rank(S.mx, tid)[r] = mx;
        cl.sync();
#pragma unroll
        for (int p = 0; p < C; ++p) mx = fmaxf(mx, S.mx[p]);
    }

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

    if (mx == INFINITY) {   // the tokens there share all the weight
        for (int i = tid; i < kSW * a.seg; i += kST) vals[i] = vals[i] == INFINITY ? 0.f : kNegInf;
        mx = 0.f;
        own_max = own_max == INFINITY ? 0.f : kNegInf;
        __syncthreads();
    } else if (T < 0x1p-96f && fabsf(mx) < 0x1p30f) {
        // 1 / T is beyond binary32, and tokens a step apart may share the weight: logits and temperature by 2^96 (what
        // overflows is further below the maximum than has a weight)
        for (int i = tid; i < kSW * a.seg; i += kST) vals[i] *= 0x1p96f;
        mx *= 0x1p96f;
        own_max *= 0x1p96f;
        inv *= 0x1p-96;
        weigh.set_temperature(T * 0x1p96f, S.tab);
        __syncthreads();
    }
    const bool by_k = K >= 1 && K < a.V, by_p = P < 1.f, by_m = mp > 0.f;
    const double minw = (double)mp;
    weigh.set_maximum(mx);
    const int s0 = warp * a.seg;   // this warp's tokens: s0 .. s0 + seg - 1

    // ---- the prefix that top-k and top-p keep: tokens above thr, and those at it up to index last of the row
    float thr = -3.402823466e38f;
    int last = 0x7fffffff;
    auto inside = [&](float l, int i) { return l > thr || (l == thr && begin + i <= last); };
    // f on four of this lane's tokens at a time, and the first one's index (-infinity beyond the row)
    auto each = [&](auto&& f) {
        for (int i = s0 + 4 * lane; i < s0 + a.seg; i += 128) {
            const float4 v = *reinterpret_cast<const float4*>(vals + i);
            const float l[4] = {v.x, v.y, v.z, v.w};
            f(l, i);
        }
    };
    int buf = 0;
    // At most kList tokens that top-k or top-p may keep: they are in order, one per thread, so that the filters that
    // are left and the draw need no more passes over the row.
    bool small = false;
    u64 small_total = 0;
    auto scan = [&](u64 w) {   // inclusive sums over the CTA's threads
        u64 inc = warp_scan(w, lane);
        __syncthreads();
        if (lane == 31) S.wsum[warp] = inc;
        __syncthreads();
#pragma unroll
        for (int x = 0; x < kSW; ++x)
            if (x < warp) inc += S.wsum[x];
        return inc;
    };
    // v: this thread's token; the first n count; target: top-p's, or 0 for top-k
    auto kept_few = [&](u64 v, int n, u64 target) {
        const float l = key_value((uint32_t)(v >> 32));
        const double w = weigh(l);
        const u64 units = v && tid < n ? Weigh::to_units(w) : 0, inc = scan(units);
        if (!target) {
            if (tid == n - 1) S.list[0] = inc;
            __syncthreads();
            target = S.list[0];   // top-k's total
            if (by_p) target = min(target, max(1ull, (u64)__double2ll_ru(fmax((double)P, 0.0) * (double)target)));
            __syncthreads();
        }
        // (what follows the last token with a weight is not in: the first one always is)
        const bool in = units && inc - units < target && (tid == 0 || !(by_m && (w < minw || (mp == 1.f && l < mx))));
        const int m = __syncthreads_count(in);   // a prefix
        if (tid == m - 1) S.list[0] = v, S.list[1] = inc;
        __syncthreads();
        thr = key_value((uint32_t)(S.list[0] >> 32));
        last = (int)~(uint32_t)S.list[0];
        small_total = S.list[1];
        __syncthreads();
        if (r != 0) return;
        // the draw goes by index: the same tokens in that order, their keys beside
        const u64 by_index = sort_desc(S, tid < m ? ((u64)(uint32_t)v << 32) | (v >> 32) : 0);
        const float li = key_value((uint32_t)by_index);
        const double wi = weigh(li);
        const u64 ui = by_index ? Weigh::to_units(wi) : 0, run = scan(ui);
        const u64 at = draw_target(u, small_total);
        if (ui && at < run && at >= run - ui) {   // one thread
            a.token[row] = (int)~(uint32_t)(by_index >> 32);
            if (a.prob) a.prob[row] = (float)(wi * (kOne / (double)small_total));
        }
    };
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        const bool mass = pass == 1;
        if (!(mass ? by_p : by_k) || small) continue;
        // steps of 1/128 of a temperature for masses, of 1/64 for counts: a few hundred tokens at most in the
        // bins that matter
        const Coarse coarse{mx, (float)fmin(fmax(mass ? inv * 128.0 : 64.0, 1e-38), 1e38)};
        u64 target = (u64)K, before = 0, own = 0;
        uint32_t bin = 0, lo = 0, hi = 0;
        bool found = false, few = false;
        // Top-k of a few: k threads' largest tokens bound the k-th token from below, and a histogram of those is
        // enough to list little more than k tokens.
        bool probe = !mass && K <= C * kST / 4;
        // The first histogram; if its bin holds too many tokens to order at once, the bits of the keys in it.
#pragma unroll 1
        for (int round = 0;; ++round) {
            const int shift = round ? max(0, 32 - __clz(hi - lo) - 11) : 0;
            uint4* h = reinterpret_cast<uint4*>(S.hist[buf]);
            h[tid] = make_uint4(0, 0, 0, 0);
            if (mass) h[kST + tid] = make_uint4(0, 0, 0, 0);
            if (tid == 0) S.list_n = 0;
            __syncthreads();
            auto put = [&](uint32_t b, u64 v) {
                const uint32_t x = (uint32_t)v, old = atomicAdd(&S.hist[buf][0][b], x);
                const uint32_t y = (uint32_t)(v >> 32) + (old + x < x);   // with the carry
                if (y) atomicAdd(&S.hist[buf][1][b], y);
            };
            if (probe) {
                if (own_max > kNegInf) atomicAdd(&S.hist[buf][0][coarse(own_max)], 1u);
            } else if (round == 0) {
                each([&](const float (&l)[4], int) {
                    // (after top-k most steps hold nothing)
                    if (!__any_sync(kAll, fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])) > kNegInf)) return;
                    if (mass) {
                        u64 v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = weigh.units(l[e]);   // none at -infinity
                        uint32_t b[4], old[4];   // the four additions in flight together, then their carries
#pragma unroll
                        for (int e = 0; e < 4; ++e) b[e] = coarse(l[e]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) old[e] = v[e] ? atomicAdd(&S.hist[buf][0][b[e]], (uint32_t)v[e]) : 0u;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t y = (uint32_t)(v[e] >> 32) + (old[e] + (uint32_t)v[e] < (uint32_t)v[e]);
                            if (y) atomicAdd(&S.hist[buf][1][b[e]], y);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (l[e] > kNegInf) atomicAdd(&S.hist[buf][0][coarse(l[e])], 1u);
                    }
                });
            } else {
                each([&](const float (&l)[4], int) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t k = order_key(l[e]);
                        if (k - lo > hi - lo) continue;
                        if (!mass) {
                            atomicAdd(&S.hist[buf][0][(hi - k) >> shift], 1u);
                        } else {
                            const u64 v = weigh.units(l[e]);
                            if (v) put((hi - k) >> shift, v);
                        }
                    }
                });
            }
            __syncthreads();
            push_groups<C>(cl, S, buf, mass);
            cl.sync();
            if (round == 0) {
                u64 inc, mine;
                const u64 total = group_scan<C>(S, buf, lane, inc, mine);
                if (mass) {   // p of the total
                    target = max(1ull, (u64)__double2ll_ru(fmax((double)P, 0.0) * (double)total));
                    target = min(target, total);
                } else if (total < target) {   // top-k of more tokens than there are
                    buf ^= 1;
                    if (!probe) break;
                    probe = false, round = -1;
                    continue;
                }
            }
            uint32_t b;
            u64 rel;
            find_bin<C>(S, buf, mass, target - before, b, rel, own);
            buf ^= 1;
            before += rel;
            found = true;
            if (round == 0) {
                // the tokens of the bin: a list of the first few, and the range of their keys; where top-k leaves
                // few tokens, of the bins above too
                bin = b;
                // (a mass: each of its tokens weighs more than one a step below the bin)
                const float lowest = -3.402823466e38f;
                const float edge = bin == kBins - 1 ? lowest : fmaxf(mx - ((float)bin + 1.f) / coarse.step, lowest);
                few = probe || before + own <= (mass ? kList * weigh.units(edge) : (u64)kList);
                uint32_t l0, h0, listed;
                int from, j;
            list:
                l0 = 0xffffffffu, h0 = 0;
                auto list = [&](float l, int i) {
                    const uint32_t k = order_key(l);
                    l0 = min(l0, k), h0 = max(h0, k);
                    const uint32_t at = atomicAdd(&S.list_n, 1u);   // any order: they are sorted
                    if (at < kList) S.list[at] = order_of(k, begin + i);
                };
                each([&](const float (&l)[4], int i) {
                    if (few) {   // all down to the bin's end, and perhaps one or two more
                        if (!__any_sync(kAll, fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])) >= edge)) return;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (l[e] >= edge) list(l[e], i + e);
                    } else {
                        bool in[4], any = false;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            in[e] = coarse(l[e]) == bin && l[e] > kNegInf;
                            any |= in[e];
                        }
                        if (!__any_sync(kAll, any)) return;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (in[e]) list(l[e], i + e);
                    }
                });
                l0 = __reduce_min_sync(kAll, l0);
                h0 = __reduce_max_sync(kAll, h0);
                if (lane == 0) S.wlo[warp] = l0, S.whi[warp] = h0;
                __syncthreads();
#pragma unroll
                for (int w = 0; w < kSW; ++w) l0 = min(l0, S.wlo[w]), h0 = max(h0, S.whi[w]);
                if (tid < C) {
                    cl.map_shared_rank(S.klo, tid)[r] = l0;
                    cl.map_shared_rank(S.khi, tid)[r] = h0;
                    cl.map_shared_rank(S.listed, tid)[r] = S.list_n;
                }
                cl.sync();
                listed = 0, from = 0, j = tid;   // this thread's token: the j-th of CTA from
#pragma unroll
                for (int p = 0; p < C; ++p) {
                    const uint32_t n = S.listed[p];
                    l0 = min(l0, S.klo[p]), h0 = max(h0, S.khi[p]);
                    if (tid >= listed + n) from = p + 1, j = (int)(tid - listed - n);
                    listed += n;
                }
                if (probe && listed > kList) {   // many alike
                    probe = false, round = -1, before = 0;
                    continue;
                }
                if (few && listed > kList) {   // (a bound missed by a rounding)
                    few = false;
                    if (C > 1) cl.sync();
                    __syncthreads();
                    if (tid == 0) S.list_n = 0;
                    __syncthreads();
                    goto list;
                }
                lo = l0, hi = h0;
                if (listed <= kList) {
                    u64 v = (uint32_t)tid < listed ? cl.map_shared_rank(S.list, from)[j] : 0;
                    if (C > 1) cl.sync();   // the peers have read this CTA's list
                    else __syncthreads();
                    v = sort_desc(S, v);
                    if (few) {
                        small = true;
                        kept_few(v, mass ? kList : K, mass ? target : 0);
                        found = false;
                        break;
                    }
                    const float l = key_value((uint32_t)(v >> 32));
                    const u64 w = !v ? 0 : mass ? weigh.units(l) : 1;
                    u64 inc = warp_scan(w, lane);
                    if (lane == 31) S.wsum[warp] = inc;
                    __syncthreads();
                    inc += before;
#pragma unroll
                    for (int x = 0; x < kSW; ++x)
                        if (x < warp) inc += S.wsum[x];
                    if (w && inc >= target && inc - w < target) S.list[0] = v;   // one thread
                    __syncthreads();
                    const u64 at = S.list[0];
                    thr = key_value((uint32_t)(at >> 32));
                    last = (int)~(uint32_t)at;
                    found = false;
                    break;
                }
            } else {
                hi -= b << shift;
                lo = max(lo, hi - ((1u << shift) - 1u));
            }
            if (lo >= hi) break;
        }
        if (found) {
            // one key holds the prefix's end: its first tokens in index order complete the target
            const float at = key_value(hi);
            const u64 w = mass ? weigh.units(at) : 1;
            const u64 q = (target - before + w - 1) / w;
            if (q >= own / w) {   // all of those that were left
                last = 0x7fffffff;
            } else {
                uint32_t t = 0;
                each([&](const float (&l)[4], int i) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) t += l[e] == at;
                });
                t = __reduce_add_sync(kAll, t);
                if (lane == 0) S.wtie[warp] = t;
                __syncthreads();
                uint32_t mine = 0, all = 0;
#pragma unroll
                for (int x = 0; x < kSW; ++x) {
                    if (x < warp) mine += S.wtie[x];
                    all += S.wtie[x];
                }
                if (tid < C) cl.map_shared_rank(S.ties, tid)[r] = all;
                cl.sync();
#pragma unroll
                for (int p = 0; p < C; ++p)
                    if (p < r) mine += S.ties[p];
                if (mine < q && mine + t >= q) {   // the q-th one is this warp's
                    u64 n = mine;
                    for (int i = s0 + lane; i < s0 + a.seg; i += 32) {
                        const uint32_t m = __ballot_sync(kAll, vals[i] == at);
                        if (n + __popc(m) >= q) {
                            if ((m >> lane & 1u) && n + __popc(m & ((1u << lane) - 1u)) + 1 == q)
                                for (int p = 0; p < C; ++p) *cl.map_shared_rank(&S.tie_at, p) = begin + i;
                            break;
                        }
                        n += __popc(m);
                    }
                }
                cl.sync();
                last = S.tie_at;
            }
            thr = at;
        }
        if (!mass && by_p && !small) {   // what top-k removes is gone for top-p
            each([&](const float (&l)[4], int i) {
                if (!__any_sync(kAll, l[0] > kNegInf || l[1] > kNegInf || l[2] > kNegInf || l[3] > kNegInf)) return;
                float4 v;
                v.x = inside(l[0], i) ? l[0] : kNegInf;
                v.y = inside(l[1], i + 1) ? l[1] : kNegInf;
                v.z = inside(l[2], i + 2) ? l[2] : kNegInf;
                v.w = inside(l[3], i + 3) ? l[3] : kNegInf;
                *reinterpret_cast<float4*>(vals + i) = v;
            });
            // (each thread reads its own tokens in the passes that follow, the search for a tie a warp's)
            __syncwarp();
        }
    }

    if (!small && mp == 1.f && thr < mx) thr = next_below(mx), last = -1;

    // weights of this lane's four tokens from i on, those that are kept
    auto kept = [&](int i, double (&w)[4]) {
        const float4 v = *reinterpret_cast<const float4*>(vals + i);
        const float l[4] = {v.x, v.y, v.z, v.w};
        bool in[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) in[e] = inside(l[e], i + e);
        if (!__any_sync(kAll, in[0] || in[1] || in[2] || in[3])) {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = 0.0;
            return;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = weigh(l[e]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (!in[e] || (by_m && w[e] < minw)) w[e] = 0.0;
    };

    // ---- their total, and each warp's share
    u64 total = small_total, base = 0, sum = 0;
    if (small) {
    } else if (by_k || by_p) {
        // few of many, as a rule: the warp gathers them and takes the exponentials of 32 at a time
        // (in the histogram that was not the last: its peers' reads ended before a barrier)
        float* queue = reinterpret_cast<float*>(S.hist[buf]) + warp * 160;
        int n = 0;
        auto flush = [&](bool in) {
            const double w = weigh(in ? queue[lane] : mx);
            if (in && !(by_m && w < minw)) sum += Weigh::to_units(w);
        };
        __syncthreads();
        each([&](const float (&l)[4], int i) {
            bool in[4];
            int mine = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                in[e] = inside(l[e], i + e);
                mine += in[e];
            }
            if (!__any_sync(kAll, mine)) return;
            int at = n;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t m = __ballot_sync(kAll, in[e]);
                if (in[e]) queue[at + __popc(m & ((1u << lane) - 1u))] = l[e];
                at += __popc(m);
            }
            n = at;
            __syncwarp();
            while (n >= 32) {   // the last 32 of the queue
                const float v = queue[n - 32 + lane];
                n -= 32;
                const double w = weigh(v);
                if (!(by_m && w < minw)) sum += Weigh::to_units(w);
            }
            __syncwarp();
        });
        flush(lane < n);
    } else if (by_m || weigh.flat) {
        for (int i = s0 + 4 * lane; i < s0 + a.seg; i += 128) {
            double w[4];
            kept(i, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum += Weigh::to_units(w[e]);
        }
    } else {
#pragma unroll 2
        for (int i = s0 + 4 * lane; i < s0 + a.seg; i += 128) {
            const float4 v = *reinterpret_cast<const float4*>(vals + i);
            sum += Weigh::offset_units(weigh(v.x)) + Weigh::offset_units(weigh(v.y));
            sum += Weigh::offset_units(weigh(v.z)) + Weigh::offset_units(weigh(v.w));
        }
        sum -= (u64)(a.seg / 32) * kOffset;   // seg / 32 tokens a lane
    }
    if (!small) {
        sum = warp_sum(sum);
        __syncthreads();   // S.wsum of the threshold has been read
        if (lane == 0) S.wsum[warp] = sum;
        __syncthreads();
        u64 all = 0;
#pragma unroll
        for (int w = 0; w < kSW; ++w) {
            if (w < warp) base += S.wsum[w];
            all += S.wsum[w];
        }
        total = all;
        if (C > 1) {
            if (tid < C) cl.map_shared_rank(S.slice_tot, tid)[r] = all;
            cl.sync();
            total = 0;
#pragma unroll
            for (int p = 0; p < C; ++p) {
                if (p < r) base += S.slice_tot[p];
                total += S.slice_tot[p];
            }
        }
    }
    const double norm = kOne / (double)total;

    // ---- the draw: the first kept token whose running sum exceeds u of the total
    const u64 target = draw_target(u, total);
    if (!small && target >= base && target < base + sum) {   // one warp of the cluster
        u64 run = base;
        for (int i = s0 + 4 * lane; i < s0 + a.seg; i += 128) {
            double w[4];
            kept(i, w);
            u64 mine = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) mine += Weigh::to_units(w[e]);
            const u64 inc = warp_scan(mine, lane);
            const uint32_t b = __ballot_sync(kAll, run + inc > target);
            if (b) {
                if (lane == __ffs(b) - 1) {
                    u64 at = run + inc - mine;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const u64 next = at + Weigh::to_units(w[e]);
                        if (at <= target && next > target) {
                            a.token[row] = begin + i + e;
                            if (a.prob) a.prob[row] = (float)(w[e] * norm);
                        }
                        at = next;
                    }
                }
                break;
            }
            run += __shfl_sync(kAll, inc, 31);
        }
    }
    if (probs) {
        for (int i = s0 + 4 * lane; i < s0 + a.seg; i += 128) {
            double w[4];
            kept(i, w);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e < cnt) probs[i + e] = (float)(w[e] * norm);
        }
    }
}

template <bool BF, int C>
static cudaError_t sample_launch(const SampleArgs& a, int n, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(k_sample<BF, C>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSampleMaxVocab / 8 * 4);
    if (e == cudaSuccess && C > 8) e = cudaFuncSetAttribute(k_sample<BF, C>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)n * C);
    cfg.blockDim = dim3(kST);
    cfg.dynamicSmemBytes = (size_t)kSW * a.seg * 4;
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = C;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_sample<BF, C>, a);
}

template <bool BF>
static cudaError_t sample_any(const SampleArgs& a, int C, int n, cudaStream_t st) {
    if (C == 1) return sample_launch<BF, 1>(a, n, st);
    if (C == 2) return sample_launch<BF, 2>(a, n, st);
    if (C == 4) return sample_launch<BF, 4>(a, n, st);
    if (C == 8) return sample_launch<BF, 8>(a, n, st);
    return sample_launch<BF, 16>(a, n, st);
}

cudaError_t launch_sample(SampleArgs a, bool bf16, int n, int n_sm, cudaStream_t st) {
    // CTAs per row: a quarter to the whole of a CTA's 32,768-token share each; for a few rows twice as many
    int C = 1;
    while (C < 8 && (a.V + C - 1) / C > 8192) C *= 2;
    if (C == 8 && a.V > 65536 && n * 16 <= n_sm / 2) C = 16;
    a.slice = (((a.V + C - 1) / C) + 7) & ~7;
    a.seg = ((a.slice + kSW - 1) / kSW + 127) & ~127;
    return bf16 ? sample_any<true>(a, C, n, st) : sample_any<false>(a, C, n, st);
}

}  // namespace ds4
