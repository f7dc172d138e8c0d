// ops_capi.cu -- the C entry points of the operators around the layer
// (include/ds4moe.h): argument checks and launches.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "../../include/ds4moe.h"
#include "ops.cuh"

namespace ds4 {
ds4moe_status report(ds4moe_status s, const char* msg);
}

using namespace ds4;

namespace {

ds4moe_status fail(ds4moe_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
ds4moe_status fail(ds4moe_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return report(s, buf);
}

ds4moe_status done(cudaError_t e, const char* what) {
    return e == cudaSuccess ? DS4MOE_OK : fail(DS4MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool act(int32_t t) { return t == DS4MOE_ACT_F32 || t == DS4MOE_ACT_BF16; }
size_t act_size(int32_t t) { return t == DS4MOE_ACT_BF16 ? 2 : 4; }

struct Span {
    const void* p;
    size_t bytes;
};
bool overlap(const Span& a, const Span& b) {
    if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return x < y + b.bytes && y < x + a.bytes;
}
// Whether any output overlaps an input or another output.
bool clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (const Span* o = outs.begin(); o != outs.end(); ++o) {
        for (const Span& i : ins)
            if (overlap(*o, i)) return true;
        for (const Span* q = o + 1; q != outs.end(); ++q)
            if (overlap(*o, *q)) return true;
    }
    return false;
}

// SMs of the current device.
cudaError_t sm_count(int* n) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    return e == cudaSuccess ? cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev) : e;
}

bool group_ok(int32_t g) { return g == 0 || g == 32 || g == 64 || g == 128; }
int64_t groups_of(int32_t hidden, int32_t group) { return group ? (hidden + group - 1) / group : 1; }

}  // namespace

extern "C" {

ds4moe_status ds4moe_add_rmsnorm(const void* d_x, int32_t x_dtype, const void* d_residual, int32_t residual_dtype,
                                 const float* d_weight, float eps, int32_t n, int32_t hidden, void* d_sum, void* d_out,
                                 int32_t out_dtype, void* d_q, int32_t q_format, int32_t group, float* d_scale,
                                 void* stream) {
    if (n < 0 || hidden < 1) return fail(DS4MOE_ERR_ARG, "add_rmsnorm: n %d, hidden %d", n, hidden);
    if (hidden > 16384) return fail(DS4MOE_ERR_SHAPE, "add_rmsnorm: hidden %d above 16384", hidden);
    if (!act(x_dtype) || (d_residual && !act(residual_dtype)) || (d_out && !act(out_dtype)))
        return fail(DS4MOE_ERR_ARG, "add_rmsnorm: unknown element type");
    if (!(eps > 0.f) || !std::isfinite(eps)) return fail(DS4MOE_ERR_ARG, "add_rmsnorm: eps must be positive and finite");
    if (d_q && (q_format != DS4MOE_Q8_E4M3 && q_format != DS4MOE_Q8_INT8))
        return fail(DS4MOE_ERR_ARG, "add_rmsnorm: unknown 8-bit format %d", q_format);
    if (d_q && !group_ok(group)) return fail(DS4MOE_ERR_ARG, "add_rmsnorm: group %d (0, 32, 64 or 128)", group);
    if (n == 0) return DS4MOE_OK;
    if (!d_x || !d_weight) return fail(DS4MOE_ERR_ARG, "add_rmsnorm: NULL x or weight");
    if (!d_sum && !d_out && !d_q) return fail(DS4MOE_ERR_ARG, "add_rmsnorm: no output");
    if (d_sum && !d_residual) return fail(DS4MOE_ERR_ARG, "add_rmsnorm: a sum needs a residual");
    if (!d_q != !d_scale) return fail(DS4MOE_ERR_ARG, "add_rmsnorm: q and scale come together");
    for (const void* p : {d_x, d_residual, (const void*)d_weight, (const void*)d_sum, (const void*)d_out, (const void*)d_q})
        if (!aligned(p, 16)) return fail(DS4MOE_ERR_ALIGN, "add_rmsnorm: buffers must be 16-byte aligned");
    if (!aligned(d_scale, 4)) return fail(DS4MOE_ERR_ALIGN, "add_rmsnorm: scale not 4-byte aligned");
    const size_t e = (size_t)n * hidden;
    const Span res{d_residual, d_residual ? e * act_size(residual_dtype) : 0};
    const Span sum{d_sum == d_residual ? nullptr : d_sum, res.bytes};   // in place is fine: same elements, same type
    const Span out{d_out, d_out ? e * act_size(out_dtype) : 0}, q{d_q, d_q ? e : 0};
    const Span sc{d_scale, d_q ? (size_t)n * groups_of(hidden, group) * 4 : 0};
    const Span x{d_x, e * act_size(x_dtype)}, w{d_weight, (size_t)hidden * 4};
    if (clash({sum, out, q, sc}, {x, res, w}) || (d_sum == d_residual && overlap(x, Span{d_sum, res.bytes})))
        return fail(DS4MOE_ERR_ARG, "add_rmsnorm: an output overlaps another buffer");
    int n_sm = 0;
    const cudaError_t ce = sm_count(&n_sm);
    if (ce != cudaSuccess) return done(ce, "add_rmsnorm: device");
    AddNormArgs a{};
    a.x = d_x, a.res = d_residual, a.w = d_weight, a.sum = d_sum, a.out = d_out, a.q = (uint8_t*)d_q, a.scale = d_scale;
    a.n = n, a.H = hidden, a.group = d_q ? group : 0, a.fmt = q_format, a.out_bf16 = out_dtype == DS4MOE_ACT_BF16;
    a.eps = eps, a.qmax = q_format == DS4MOE_Q8_E4M3 ? 448.f : 127.f;
    const int kind = !d_residual ? 0 : residual_dtype == DS4MOE_ACT_BF16 ? 2 : 1;
    return done(launch_add_rmsnorm(a, x_dtype == DS4MOE_ACT_BF16, kind, hidden % 8 == 0, n_sm, (cudaStream_t)stream),
                "add_rmsnorm launch");
}

ds4moe_status ds4moe_widen_rows(const void* d_q, int32_t q_format, const float* d_scale, int32_t group, int32_t n,
                                int32_t hidden, void* d_out, int32_t out_dtype, void* stream) {
    if (n < 0 || hidden < 1) return fail(DS4MOE_ERR_ARG, "widen_rows: n %d, hidden %d", n, hidden);
    if (q_format != DS4MOE_Q8_E4M3 && q_format != DS4MOE_Q8_INT8)
        return fail(DS4MOE_ERR_ARG, "widen_rows: unknown 8-bit format %d", q_format);
    if (!group_ok(group)) return fail(DS4MOE_ERR_ARG, "widen_rows: group %d (0, 32, 64 or 128)", group);
    if (!act(out_dtype)) return fail(DS4MOE_ERR_ARG, "widen_rows: unknown element type");
    if (n == 0) return DS4MOE_OK;
    if (!d_q || !d_scale || !d_out) return fail(DS4MOE_ERR_ARG, "widen_rows: NULL buffer");
    if (!aligned(d_q, 16) || !aligned(d_out, 16)) return fail(DS4MOE_ERR_ALIGN, "widen_rows: q and out must be 16-byte aligned");
    if (!aligned(d_scale, 4)) return fail(DS4MOE_ERR_ALIGN, "widen_rows: scale not 4-byte aligned");
    const size_t e = (size_t)n * hidden;
    if ((e + 4095) / 4096 > 0x7fffffffu) return fail(DS4MOE_ERR_SHAPE, "widen_rows: %d x %d is too large", n, hidden);
    if (clash({Span{d_out, e * act_size(out_dtype)}}, {Span{d_q, e}, Span{d_scale, (size_t)n * groups_of(hidden, group) * 4}}))
        return fail(DS4MOE_ERR_ARG, "widen_rows: out overlaps an input");
    return done(launch_widen_rows((const uint8_t*)d_q, q_format, d_scale, group, n, hidden, d_out,
                                  out_dtype == DS4MOE_ACT_BF16, (cudaStream_t)stream),
                "widen_rows launch");
}

static ds4moe_status check_project(int32_t n, int32_t fin, int32_t fout, int32_t n_adapters, int32_t rank) {
    if (n < 0 || fin < 1 || fout < 1 || n_adapters < 0)
        return fail(DS4MOE_ERR_ARG, "project: n %d, in %d, out %d, n_adapters %d", n, fin, fout, n_adapters);
    if (n > (1 << 20)) return fail(DS4MOE_ERR_ARG, "project: n %d above 2^20", n);
    if (fin % 8 || fin > 65536) return fail(DS4MOE_ERR_SHAPE, "project: in %d not a multiple of 8 up to 65536", fin);
    if (fout > (1 << 20)) return fail(DS4MOE_ERR_SHAPE, "project: out %d above 2^20", fout);
    if (n_adapters > 65536) return fail(DS4MOE_ERR_SHAPE, "project: %d adapters above 65536", n_adapters);
    if (n_adapters && (rank < 8 || rank > 128 || rank % 8))
        return fail(DS4MOE_ERR_SHAPE, "project: rank %d not a multiple of 8 in 8..128", rank);
    return DS4MOE_OK;
}

size_t ds4moe_project_work_bytes(int32_t n, int32_t in_features, int32_t out_features, int32_t n_adapters, int32_t rank) {
    if (n_adapters < 1 || n < 1 || check_project(n, in_features, out_features, n_adapters, rank) != DS4MOE_OK)
        return 0;
    return project_work(n, in_features, out_features, n_adapters, rank).total;
}

static ds4moe_status project(const void* d_x, int32_t n, const void* d_W, int32_t in_features, int32_t out_features,
                             const void* d_A, const void* d_B, const float* d_scale, int32_t n_adapters, int32_t rank,
                             const int32_t* d_ids, void* d_out, void* d_work, size_t work_bytes, int in_time, void* stream) {
    const ds4moe_status s = check_project(n, in_features, out_features, n_adapters, rank);
    if (s != DS4MOE_OK) return s;
    if (n == 0) return DS4MOE_OK;
    const bool ad = n_adapters > 0;
    if (!d_x || !d_W || !d_out || (ad && (!d_A || !d_B || !d_scale || !d_ids || !d_work)))
        return fail(DS4MOE_ERR_ARG, "project: NULL buffer");
    if (!aligned(d_x, 16) || !aligned(d_W, 16) || !aligned(d_out, 16) || (ad && (!aligned(d_A, 16) || !aligned(d_B, 16))))
        return fail(DS4MOE_ERR_ALIGN, "project: x, W, A, B and out must be 16-byte aligned");
    if (ad && (!aligned(d_work, 256) || !aligned(d_scale, 4) || !aligned(d_ids, 4)))
        return fail(DS4MOE_ERR_ALIGN, "project: work must be 256-byte aligned, scale and ids 4-byte");
    ProjectWork wk = project_work(n, in_features, out_features, ad ? n_adapters : 0, ad ? rank : 0);
    if (ad && work_bytes < wk.total) return fail(DS4MOE_ERR_ARG, "project: work %zu bytes < %zu", work_bytes, wk.total);
    const size_t fi = in_features, fo = out_features, na = n_adapters, r = rank;
    const Span out{d_out, (size_t)n * fo * 2}, work{ad ? d_work : nullptr, wk.total};
    const Span x{d_x, (size_t)n * fi * 2}, W{d_W, fo * fi * 2}, A{ad ? d_A : nullptr, na * r * fi * 2},
        B{ad ? d_B : nullptr, na * r * fo * 2}, sc{ad ? d_scale : nullptr, na * 4}, ids{ad ? d_ids : nullptr, (size_t)n * 4};
    if (clash({out, work}, {x, W, A, B, sc, ids})) return fail(DS4MOE_ERR_ARG, "project: out or work overlaps another buffer");
    int n_sm = 0;
    const cudaError_t ce = sm_count(&n_sm);
    if (ce != cudaSuccess) return done(ce, "project: device");
    ProjectArgs p{};
    ShrinkArgs sh{};
    p.out = (__nv_bfloat16*)d_out;
    p.n = sh.n = n;
    p.fin = sh.fin = in_features;
    p.fout = out_features;
    p.in_time = in_time;
    sh.x = (const __nv_bfloat16*)d_x;
    if (ad) {
        uint8_t* w = (uint8_t*)d_work;
        p.rank = sh.rank = rank;
        sh.n_adapters = n_adapters;
        sh.A = (const __nv_bfloat16*)d_A;
        sh.scale = d_scale;
        sh.ids = d_ids;
        p.B = (const __nv_bfloat16*)d_B;
        p.ids = d_ids;
        p.n_adapters = n_adapters;
        if (wk.rows) {
            p.rows = sh.rows = (float*)(w + wk.off_t);
        } else {
            p.counts = sh.counts = (int32_t*)w;
            p.entry = sh.entry = (int32_t*)(w + wk.off_entry);
            sh.t = (__nv_bfloat16*)(w + wk.off_t);
        }
    }
    return done(launch_project(p, sh, wk, d_W, n_sm, (cudaStream_t)stream), "project launch");
}

ds4moe_status ds4moe_project(const void* d_x, int32_t n, const void* d_W, int32_t in_features, int32_t out_features,
                             const void* d_A, const void* d_B, const float* d_scale, int32_t n_adapters, int32_t rank,
                             const int32_t* d_ids, void* d_out, void* d_work, size_t work_bytes, void* stream) {
    return project(d_x, n, d_W, in_features, out_features, d_A, d_B, d_scale, n_adapters, rank, d_ids, d_out, d_work, work_bytes,
                   INT32_MAX, stream);
}

ds4moe_status ds4moe_selftest_project_wait(const void* d_x, int32_t n, const void* d_W, int32_t in_features, int32_t out_features,
                                           const void* d_A, const void* d_B, const float* d_scale, int32_t n_adapters,
                                           int32_t rank, const int32_t* d_ids, void* d_out, void* d_work, size_t work_bytes,
                                           int32_t tiles, void* stream) {
    if (tiles < 0) return fail(DS4MOE_ERR_ARG, "project: tiles %d", tiles);
    return project(d_x, n, d_W, in_features, out_features, d_A, d_B, d_scale, n_adapters, rank, d_ids, d_out, d_work, work_bytes,
                   tiles, stream);
}

ds4moe_status ds4moe_get_project_error(void* stream, int32_t* code) {
    if (!code) return fail(DS4MOE_ERR_ARG, "get_project_error: NULL code");
    uint32_t v = 0;
    const cudaError_t e = read_project_error(&v, (cudaStream_t)stream);
    if (e != cudaSuccess) return done(e, "get_project_error");
    *code = (int32_t)v;
    return v ? fail(DS4MOE_ERR_TIMEOUT, "project: a bounded device-side wait gave up") : DS4MOE_OK;
}

ds4moe_status ds4moe_sample(const void* d_logits, int32_t dtype, int64_t row_stride, int32_t n, int32_t vocab,
                            const float* d_temperature, const int32_t* d_top_k, const float* d_top_p,
                            const float* d_min_p, const float* d_u, int32_t* d_token, float* d_prob, float* d_probs,
                            void* stream) {
    if (n < 0 || vocab < 1) return fail(DS4MOE_ERR_ARG, "sample: n %d, vocab %d", n, vocab);
    if (!act(dtype)) return fail(DS4MOE_ERR_ARG, "sample: unknown element type");
    if (vocab > kSampleMaxVocab) return fail(DS4MOE_ERR_SHAPE, "sample: vocab %d above %d", vocab, kSampleMaxVocab);
    if (row_stride < vocab || row_stride > ((int64_t)1 << 32))
        return fail(DS4MOE_ERR_ARG, "sample: row stride %lld below vocab %d or above 2^32", (long long)row_stride, vocab);
    if (n > (1 << 24)) return fail(DS4MOE_ERR_ARG, "sample: n %d above 2^24", n);
    if (n == 0) return DS4MOE_OK;
    if (!d_logits || !d_u || !d_token) return fail(DS4MOE_ERR_ARG, "sample: NULL buffer");
    for (const void* p : {(const void*)d_temperature, (const void*)d_top_k, (const void*)d_top_p, (const void*)d_min_p,
                          (const void*)d_u, (const void*)d_token, (const void*)d_prob, (const void*)d_probs})
        if (!aligned(p, 4)) return fail(DS4MOE_ERR_ALIGN, "sample: buffers must be 4-byte aligned");
    if (!aligned(d_logits, act_size(dtype))) return fail(DS4MOE_ERR_ALIGN, "sample: logits not aligned to their type");
    const size_t m = (size_t)n * 4;
    const Span tok{d_token, m}, prob{d_prob, m}, probs{d_probs, m * vocab};
    if (clash({tok, prob, probs}, {Span{d_logits, ((size_t)(n - 1) * row_stride + vocab) * act_size(dtype)},
                                   Span{d_temperature, m}, Span{d_top_k, m}, Span{d_top_p, m}, Span{d_min_p, m}, Span{d_u, m}}))
        return fail(DS4MOE_ERR_ARG, "sample: an output overlaps another buffer");
    SampleArgs a{};
    a.logits = d_logits, a.ld = row_stride, a.V = vocab, a.temp = d_temperature, a.top_k = d_top_k, a.top_p = d_top_p;
    a.min_p = d_min_p, a.u = d_u, a.token = d_token, a.prob = d_prob, a.probs = d_probs;
    int n_sm = 0;
    const cudaError_t ce = sm_count(&n_sm);
    if (ce != cudaSuccess) return done(ce, "sample: device");
    return done(launch_sample(a, dtype == DS4MOE_ACT_BF16, n, n_sm, (cudaStream_t)stream), "sample launch");
}

}  // extern "C"
