// add_api.cu -- the extern "C" entry points of the residual-stream operators:
// argument checks and launches.  Nothing here allocates memory or
// synchronizes.
#include <cmath>
#include <initializer_list>

#include "addnorm.cuh"
#include "gbnorm.h"
#include "internal.h"
#include "rowring.cuh"

namespace {

using gbn::RowSrc;

bool dtype_ok(int t) { return t == gbn::kF32 || t == gbn::kBF16 || t == gbn::kF16; }
bool q8_ok(int t) { return t == GBN_E4M3 || t == GBN_INT8; }
bool group_ok(int64_t g) { return g == 0 || g == 32 || g == 64 || g == 128; }
int elem_bytes(int t) { return t == gbn::kF32 ? 4 : 2; }

bool aligned(int bytes, std::initializer_list<const void*> ps)
{
    for (const void* p : ps)
        if ((reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) != 0) return false;
    return true;
}

// The rules of rmsnorm_fwd_ex: expression 0 with 16-bit activations takes a
// weight of f32 or of their type.
int norm_types(int xt, int wt, int variant)
{
    if (variant < GBN_RMS_CAST_FIRST || variant > GBN_RMS_GEMMA) return GBN_EINVAL;
    if (!dtype_ok(xt) || !dtype_ok(wt)) return GBN_EDTYPE;
    if (variant == GBN_RMS_CAST_FIRST && xt != GBN_F32 && wt != GBN_F32 && wt != xt)
        return GBN_EDTYPE;
    return GBN_OK;
}

// An activation input as the kernels take it; false for a bad layout.
bool source(RowSrc& out, const void* p, const gbn_rows* l, int64_t M, int64_t N, int e)
{
    bool scattered = false;
    out = RowSrc{};
    out.p = static_cast<const unsigned char*>(p);
    out.row_bytes = N * e;
    out.total = M * N * e;
    if (!gbn::host_layout_map(p ? l : nullptr, M, N, e, out.map, scattered)) return false;
    out.scattered = scattered ? 1 : 0;
    return true;
}

gbn::Q8 q8_of(void* v, const float* scale, int type, int64_t N, int64_t group)
{
    gbn::Q8 q{};
    q.v = v;
    q.scale = const_cast<float*>(scale);
    q.type = type;
    const bool row = group == 0 || group >= N;  // one group: the whole row
    q.shift = row ? 31 : group == 32 ? 5 : group == 64 ? 6 : 7;
    q.ng = row ? 1 : (int)((N + group - 1) / group);
    return q;
}

// The vectors a row of N elements may touch: one more than N / VEC where rows
// start inside a vector; and the first schedule that holds them (-1: none).
int64_t row_vectors(int64_t N, int vec, bool edge)
{
    return edge ? (N + 2 * vec - 2) / vec : N / vec;
}
// Whether every CTA of a backward takes rows enough (about 16) that the cost
// of its row counts, and not the first row's latency.
bool many_rows(int64_t M, int sms) { return M >= 32LL * sms; }

// The schedule of a row of nvec vectors (-1: too wide): the first whose groups
// hold it, or one for rows that do not fill those.  packed: the call reads or
// writes a checkpoint; edge: rows start inside a vector.  In us, bf16, 2^26
// elements a call, groups as they would be -> as they are:
//   y: two vectors a thread where the row fills them (N = 1024 90 -> 84), four
// elsewhere (N = 2560 109 -> 85), also where rows start inside a vector and no
// checkpoint is written (N = 1001 104 -> 94).
//   8-bit output, checkpoint alone: four.
//   backward: as y, given many rows (N = 2560 99 -> 90, N = 3001 133 -> 110,
// N = 1001 107 -> 100, but [4097, 1001] 14.7 -> 19.1).
//   backward from a checkpoint: four, given many rows (N = 4096 83 -> 78, but
// [64, 8192] 8.6 -> 10.3), and two where rows start inside a vector (N = 1001
// 172 -> 131) or leave much of the group empty.
//   Groups fitted to the row, kRowFit (four vectors a thread) and kRowFit2
// (two): where a fixed group would be about half empty: y N = 4097 131 -> 94,
// backward N = 4097 228 -> 143, from a checkpoint N = 2560 108 -> 91, N = 2050
// 247 -> 174 and N = 4097 248 -> 219, 8-bit output N = 5120 92 -> 84 and
// N = 2560 98 -> 87; not at 5/8 for y (N = 5120 94 fitted, 85 fixed).
int find_sched(int kind, bool packed, bool edge, int64_t nvec, bool many)
{
    int s = 0;
    while (s < gbn::kRowFit && nvec > gbn::row_sched(kind, s).cap) ++s;
    if (s == gbn::kRowFit) return -1;
    const gbn::RowSched& e = gbn::row_sched(kind, s);
    if (nvec <= 64 || nvec > 1024) return s;
    const bool half = 16 * nvec <= 9 * e.cap, most = 8 * nvec <= 5 * e.cap;
    const bool full = 16 * nvec >= 15 * e.cap;
    const int four = s - 5 + gbn::kRowMore;  // the same groups, four vectors a thread
    const bool wide = nvec > 128;
    if (kind == gbn::kKindQ) {
        if (!wide) return s;
        if (nvec > 512) return most ? gbn::kRowFit : s;
        return most && !edge && !packed ? gbn::kRowFit2 : half ? gbn::kRowFit : s;
    }
    if (kind == gbn::kKindY) {
        if (full && (!edge || packed)) return s;
        return wide && half ? gbn::kRowFit : four;
    }
    if (!packed) {  // backward from here on
        if (full && !edge) return s;
        if (wide && half) return edge && nvec <= 512 ? gbn::kRowFit2 : gbn::kRowFit;
        return many ? four : s;
    }
    if (!edge && many && !most) return four;
    if (wide && nvec <= 512) return (nvec + 63) / 64 * 32 < e.W ? gbn::kRowFit2 : s;
    return wide && (edge ? half : most) ? gbn::kRowFit : s;
}

// The launch's threads per row group, groups and CTAs on the device.
struct RowShape {
    int W, G, R;
    int64_t ctas;
};
RowShape row_shape(int kind, int sid, int64_t nvec, int sms)
{
    const gbn::RowSched& e = gbn::row_sched(kind, sid);
    RowShape s;
    s.W = e.W ? e.W : (int)((nvec + 32 * e.KV - 1) / (32 * e.KV)) * 32;
    s.G = gbn::row_G(kind, sid, s.W);
    s.R = s.G * gbn::row_U(kind, sid);
    const int minb = gbn::row_minb(kind, sid);
    // a CTA below its launch bound's size: as many as the same registers hold
    s.ctas = (int64_t)sms * (minb * e.T / (s.W * s.G));
    // rows that start inside a vector need CTAs to step by a multiple of VEC rows
    if (s.ctas >= 8) s.ctas = s.ctas / 8 * 8;
    return s;
}

// The ring kernel's launch, or false where the general kernel takes the call:
// every tensor on a 16-byte boundary, scattered rows whole vectors on such
// boundaries, and a schedule for the width.  packed: the call reads or writes
// a checkpoint; groups: the scales per row that the kernel finds (0: none).
bool plan_rows(gbn::RowPlan& p, int kind, int xt, int64_t M, int64_t N, const RowSrc* in, int nt,
               std::initializer_list<const void*> outs, bool packed, int groups, int sms)
{
    const int vec = 16 / elem_bytes(xt);
    p = gbn::RowPlan{};
    p.edge = N % vec != 0;
    if (!aligned(16, outs)) return false;
    for (int t = 0; t < nt; ++t) {
        if (!aligned(16, {in[t].p})) return false;
        if (in[t].scattered &&
            (p.edge || (in[t].map.s1 | in[t].map.s2 | in[t].map.s3) % 16 != 0))
            return false;
    }
    const int64_t nvec = row_vectors(N, vec, p.edge);
    p.sid = find_sched(kind, packed, p.edge, nvec, many_rows(M, sms));
    if (p.sid < 0) return false;
    const RowShape sh = row_shape(kind, p.sid, nvec, sms);
    p.W = sh.W;
    p.G = sh.G;
    p.R = sh.R;
    p.stages = gbn::row_stages(kind, p.sid);
    uint32_t at = 0;
    p.in_order = 1;
    for (int t = 0; t < nt; ++t) {
        p.off[t] = at;
        if (!in[t].p) continue;
        if (in[t].scattered)
            p.in_order = 0;
        else if (in[t].total % 16 != 0)
            p.tail = 1;
        at += (uint32_t)(p.R * in[t].row_bytes + 32 + 127) / 128 * 128;
    }
    p.stage_bytes = at;
    p.gm_off = 128 + p.stages * at;
    p.smem = p.gm_off + (p.edge && groups > 1 ? (size_t)p.R * (2 * groups + 1) * sizeof(float) : 0);
    if (kind == gbn::kKindB) {  // the CTA's column sums take the drained ring
        const size_t cols = 128 + (size_t)p.W * p.G * gbn::row_sched(kind, p.sid).KV * vec *
                                  sizeof(float);
        p.smem = p.smem > cols ? p.smem : cols;
    }
    p.nblocks = (M + p.R - 1) / p.R;
    const int64_t cap = sh.ctas;
    p.grid = (int)(p.nblocks < cap ? p.nblocks : cap);
    if (p.edge && p.nblocks > cap && cap * p.R % vec != 0) return false;
    return p.smem <= (size_t)gbn::kMaxSmem;
}

int launch_status(cudaError_t e) { return e == cudaSuccess ? GBN_OK : GBN_ELAUNCH; }

// Every forward: what is asked for is what is not null (w null: act_pack8).
struct Fwd {
    const void* x;
    const gbn_rows* xl;
    const void* res;
    const gbn_rows* rl;
    const void* w;
    void *s, *y;
    float* rstd;
    gbn::Q8 q, c;
    float eps;
    int xt, wt, variant;
};

int forward(const Fwd& f, int64_t M, int64_t N, cudaStream_t stream)
{
    const int e = elem_bytes(f.xt);
    if (!aligned(e, {f.x, f.res, f.s, f.y}) || !aligned(4, {f.rstd, f.q.scale, f.c.scale}))
        return GBN_EINVAL;
    gbn::FwdArgs a{};
    if (!source(a.in[0], f.x, f.xl, M, N, e) || !source(a.in[1], f.res, f.rl, M, N, e))
        return GBN_EINVAL;
    if (M == 0) return GBN_OK;
    const int sms = gbn::host_current_sms();
    if (sms <= 0) return GBN_EDEVICE;
    a.w = f.w;
    a.s = f.s;
    a.y = f.y;
    a.q = f.q;
    a.c = f.c;
    a.rstd = f.rstd;
    a.M = M;
    a.N = (int)N;
    a.eps = f.eps;
    a.inv_n = (float)(1.0 / (double)N);
    a.wt = f.wt;
    a.variant = f.variant;
    const gbn::Q8& q8 = f.q.v ? f.q : f.c;
    const int mode =
        (!f.w ? gbn::kModeC : f.q.v ? gbn::kModeQ : f.c.v ? gbn::kModeYC : gbn::kModeY) +
        (q8.v && q8.type == gbn::kInt8 ? gbn::kModeInt8 : 0);
    if (!f.w && gbn::pack_fast(f.xt, a))  // a checkpoint alone, of rows of whole groups
        return launch_status(gbn::launch_pack_fast(stream, f.xt, sms, a));
    gbn::RowPlan p;
    if (!plan_rows(p, gbn::fwd_kind(mode), f.xt, M, N, a.in, 2, {f.s, f.y, q8.v}, f.c.v != nullptr,
                   q8.v ? q8.ng : 0, sms))
        return launch_status(gbn::launch_add_fwd_general(stream, f.xt, sms, a));
    if (!(p.fault = gbn::host_fault_ptr())) return GBN_EDEVICE;
    return launch_status(f.xt == gbn::kF32   ? gbn::launch_add_fwd_f32(stream, mode, a, p)
                         : f.xt == gbn::kF16 ? gbn::launch_add_fwd_f16(stream, mode, a, p)
                                             : gbn::launch_add_fwd_bf16(stream, mode, a, p));
}

int norm_forward(const Fwd& f, int64_t M, int64_t N, cudaStream_t stream)
{
    if (const int rc = norm_types(f.xt, f.wt, f.variant)) return rc;
    if (!gbn::host_shape_ok(M, N) || !std::isfinite(f.eps) || f.eps < 0.f || !f.w)
        return GBN_EINVAL;
    if (!aligned(elem_bytes(f.wt), {f.w})) return GBN_EINVAL;
    if (M > 0 && !f.x) return GBN_EINVAL;
    if (f.s && !f.res && M > 0) return GBN_EINVAL;  // without res the stream is x
    return forward(f, M, N, stream);
}

int norm_backward(const void* s, const gbn_rows* sl, const float* cscale, int64_t group, int ct,
                  const void* dy, const gbn_rows* dyl, const void* ds, const gbn_rows* dsl,
                  const void* w, const float* rstd, void* dx, void* dw, int64_t M, int64_t N,
                  int xt, int wt, int variant, void* ws, size_t ws_bytes, cudaStream_t stream)
{
    if (const int rc = norm_types(xt, wt, variant)) return rc;
    if (!gbn::host_shape_ok(M, N) || !w) return GBN_EINVAL;
    if (M > 0 && (!s || !dy || !dx || !rstd)) return GBN_EINVAL;
    const int e = elem_bytes(xt), se = cscale ? 1 : e;
    if (!aligned(se, {s}) || !aligned(e, {dy, ds, dx}) || !aligned(elem_bytes(wt), {w, dw}) ||
        !aligned(4, {rstd, cscale}))
        return GBN_EINVAL;
    if (dw && ws && !aligned(4, {ws})) return GBN_EINVAL;
    gbn::BwdArgs a{};
    if (!source(a.in[0], s, sl, M, N, se) || !source(a.in[1], dy, dyl, M, N, e) ||
        !source(a.in[2], ds, dsl, M, N, e))
        return GBN_EINVAL;
    const int sms = gbn::host_current_sms();
    if (sms <= 0) return GBN_EDEVICE;
    if (cscale) a.c = q8_of(nullptr, cscale, ct, N, group);
    gbn::RowPlan p{};
    const bool fast =
        M > 0 && plan_rows(p, gbn::kKindB, xt, M, N, a.in, 3, {dx}, cscale != nullptr, 0, sms);
    if (fast && !(p.fault = gbn::host_fault_ptr())) return GBN_EDEVICE;
    const int64_t P = M == 0 ? 0 : fast ? p.grid : gbn::add_bwd_general_rows(M, N, sms);
    if (dw && M > 0 && (!ws || ws_bytes < (size_t)P * (size_t)N * sizeof(float)))
        return GBN_EWORKSPACE;
    a.w = w;
    a.rstd = rstd;
    a.dx = dx;
    a.ws = dw ? static_cast<float*>(ws) : nullptr;
    a.M = M;
    a.N = (int)N;
    a.inv_n = (float)(1.0 / (double)N);
    a.wt = wt;
    a.variant = variant;
    if (M > 0) {
        const int mode = cscale && ct == gbn::kInt8         ? gbn::kBwdInt8
                         : cscale                           ? gbn::kBwdC
                         : variant != GBN_RMS_CAST_FIRST    ? gbn::kBwdS
                         : wt == xt                         ? gbn::kBwdCast16
                                                            : gbn::kBwdCast;
        const cudaError_t rc = !fast               ? gbn::launch_add_bwd_general(stream, xt, P, a)
                               : xt == gbn::kF32 ? gbn::launch_add_bwd_f32(stream, mode, a, p)
                               : xt == gbn::kF16 ? gbn::launch_add_bwd_f16(stream, mode, a, p)
                                                 : gbn::launch_add_bwd_bf16(stream, mode, a, p);
        if (launch_status(rc) != GBN_OK) return GBN_ELAUNCH;
    }
    if (!dw) return GBN_OK;
    return launch_status(gbn::launch_colsum(stream, a.ws, P, N, N, wt, dw, nullptr, nullptr));
}

}  // namespace

namespace gbn {

size_t add_bwd_workspace_bytes(int64_t M, int64_t N, int xt, int sms)
{
    const int vec = 16 / elem_bytes(xt);
    const bool edge = N % vec != 0;
    const int64_t nvec = row_vectors(N, vec, edge);
    int64_t P = add_bwd_general_rows(M, N, sms);
    for (const bool packed : {false, true}) {
        const int sid = find_sched(kKindB, packed, edge, nvec, many_rows(M, sms));
        if (sid < 0) continue;
        const RowShape sh = row_shape(kKindB, sid, nvec, sms);
        const int64_t blocks = (M + sh.R - 1) / sh.R, grid = blocks < sh.ctas ? blocks : sh.ctas;
        P = P > grid ? P : grid;
    }
    const size_t need = (size_t)P * (size_t)N * sizeof(float);
    return (need + 255) & ~(size_t)255;
}

}  // namespace gbn

extern "C" {

int rmsnorm_add_fwd(const void* x, const gbn_rows* xl, const void* res, const gbn_rows* rl,
                    const void* w, void* s, void* y, float* rstd, int64_t M, int64_t N, float eps,
                    int xt, int wt, int variant, cudaStream_t stream)
{
    if (M > 0 && !y) return GBN_EINVAL;
    return norm_forward({x, xl, res, rl, w, s, y, rstd, {}, {}, eps, xt, wt, variant}, M, N,
                        stream);
}

int rmsnorm_add_quant_fwd(const void* x, const gbn_rows* xl, const void* res, const gbn_rows* rl,
                          const void* w, void* s, void* q, float* scale, float* rstd, int64_t M,
                          int64_t N, int64_t group, float eps, int xt, int wt, int qt, int variant,
                          cudaStream_t stream)
{
    if (!q8_ok(qt)) return GBN_EDTYPE;
    if (!group_ok(group) || (M > 0 && (!q || !scale))) return GBN_EINVAL;
    if (N < 1) return GBN_EINVAL;
    return norm_forward({x, xl, res, rl, w, s, nullptr, rstd, q8_of(q, scale, qt, N, group), {},
                         eps, xt, wt, variant},
                        M, N, stream);
}

int rmsnorm_add_ckpt_fwd(const void* x, const gbn_rows* xl, const void* res, const gbn_rows* rl,
                         const void* w, void* s, void* y, float* rstd, void* c, float* cscale,
                         int64_t M, int64_t N, int64_t group, float eps, int xt, int wt, int ct,
                         int variant, cudaStream_t stream)
{
    if (!q8_ok(ct)) return GBN_EDTYPE;
    if (!group_ok(group) || (M > 0 && (!y || !c || !cscale))) return GBN_EINVAL;
    if (N < 1) return GBN_EINVAL;
    return norm_forward({x, xl, res, rl, w, s, y, rstd, {}, q8_of(c, cscale, ct, N, group), eps,
                         xt, wt, variant},
                        M, N, stream);
}

int rmsnorm_add_bwd(const void* s, const gbn_rows* sl, const void* dy, const gbn_rows* dyl,
                    const void* ds, const gbn_rows* dsl, const void* w, const float* rstd,
                    void* dx, void* dw, int64_t M, int64_t N, int xt, int wt, int variant,
                    void* ws, size_t ws_bytes, cudaStream_t stream)
{
    return norm_backward(s, sl, nullptr, 0, GBN_E4M3, dy, dyl, ds, dsl, w, rstd, dx, dw, M, N, xt,
                         wt, variant, ws, ws_bytes, stream);
}

int rmsnorm_add_ckpt_bwd(const void* c, const float* cscale, const void* dy, const gbn_rows* dyl,
                         const void* ds, const gbn_rows* dsl, const void* w, const float* rstd,
                         void* dx, void* dw, int64_t M, int64_t N, int64_t group, int xt, int wt,
                         int ct, int variant, void* ws, size_t ws_bytes, cudaStream_t stream)
{
    if (!q8_ok(ct)) return GBN_EDTYPE;
    if (!group_ok(group)) return GBN_EINVAL;
    if (M > 0 && !cscale) return GBN_EINVAL;
    return norm_backward(c, nullptr, cscale, group, ct, dy, dyl, ds, dsl, w, rstd, dx, dw, M, N,
                         xt, wt, variant, ws, ws_bytes, stream);
}

int act_pack8(const void* x, const gbn_rows* xl, void* c, float* cscale, int64_t M, int64_t N,
              int64_t group, int xt, int ct, cudaStream_t stream)
{
    if (!dtype_ok(xt) || !q8_ok(ct)) return GBN_EDTYPE;
    if (!gbn::host_shape_ok(M, N) || !group_ok(group)) return GBN_EINVAL;
    if (M > 0 && (!x || !c || !cscale)) return GBN_EINVAL;
    return forward({x, xl, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, {},
                    q8_of(c, cscale, ct, N, group), 0.f, xt, GBN_F32, GBN_RMS_WEIGHT_FIRST},
                   M, N, stream);
}

int act_unpack8(const void* c, const float* cscale, void* x, int64_t M, int64_t N, int64_t group,
                int xt, int ct, cudaStream_t stream)
{
    if (!dtype_ok(xt) || !q8_ok(ct)) return GBN_EDTYPE;
    if (!gbn::host_shape_ok(M, N) || !group_ok(group)) return GBN_EINVAL;
    if (M > 0 && (!x || !c || !cscale)) return GBN_EINVAL;
    if (!aligned(elem_bytes(xt), {x}) || !aligned(4, {cscale})) return GBN_EINVAL;
    if (M == 0) return GBN_OK;
    const int sms = gbn::host_current_sms();
    if (sms <= 0) return GBN_EDEVICE;
    gbn::UnpackArgs a{};
    a.c = q8_of(const_cast<void*>(c), cscale, ct, N, group);
    a.x = x;
    a.M = M;
    a.N = (int)N;
    if (aligned(16, {c, x}) && N < (1 << 30))  // its column arithmetic is 32-bit
        return launch_status(gbn::launch_unpack_fast(stream, xt, sms, a));
    return launch_status(gbn::launch_unpack_general(stream, xt, sms, a));
}

}  // extern "C"
