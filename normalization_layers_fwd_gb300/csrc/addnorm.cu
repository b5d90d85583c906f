// addnorm.cu -- the residual-stream operators for any width, alignment and
// row layout: a row group of one warp, or of one CTA for wide rows, walks its
// row element by element, once for the row's sum of squares (and the stream
// s), once for the outputs.  The later walks hit L1 and L2.
#include "addnorm.cuh"

namespace gbn {
namespace {

constexpr int kWide = 4096;  // rows wider than this take a CTA each

// Plain loads: an output may be the memory of an input, so no non-coherent path.
__device__ __forceinline__ float ldf(const float* p) { return *p; }
__device__ __forceinline__ float ldf(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float ldf(const __half* p) { return __half2float(*p); }

template <typename TX> __device__ __forceinline__ TX cast_x(float v)
{
    if constexpr (std::is_same<TX, float>::value)
        return v;
    else if constexpr (std::is_same<TX, __half>::value)
        return __float2half_rn(v);
    else
        return __float2bfloat16_rn(v);
}

template <typename TX>
__device__ __forceinline__ const TX* src_row(const RowSrc& a, int64_t r)
{
    const unsigned char* p = a.p + (a.scattered ? row_byte_offset(a.map, r) : r * a.row_bytes);
    return reinterpret_cast<const TX*>(p);
}

// Weight of column c as the expression uses it: w, or 1 + w.
__device__ __forceinline__ float weight_at(const void* w, int wt, int c, int variant)
{
    const float v = ld_param(w, wt, c);
    return variant == 2 ? 1.f + v : v;
}

// Sum and NaN-keeping maximum over the W threads of a row group.  W = 32: a
// warp; W = kGenThreads: the CTA, its warps' values joined in warp order, so
// every thread gets the same bits.
template <int W>
__device__ __forceinline__ void group_sum_max(float& s, float& m, float* red)
{
    float v[1] = {s};
    butterfly<32, 1>(v);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
    s = v[0];
    if constexpr (W > 32) {
        constexpr int kW = W / 32;
        if ((threadIdx.x & 31) == 0) {
            red[threadIdx.x >> 5] = s;
            red[kW + (threadIdx.x >> 5)] = m;
        }
        __syncthreads();
        s = red[0];
        m = red[kW];
#pragma unroll
        for (int i = 1; i < kW; ++i) {
            s += red[i];
            m = max_nan(m, red[kW + i]);
        }
        __syncthreads();
    }
}

template <int W>
__device__ __forceinline__ void group_sync()
{
    if constexpr (W > 32)
        __syncthreads();
    else
        __syncwarp();
}

template <typename TX, int W>
__global__ void __launch_bounds__(kGenThreads) add_fwd_general(FwdArgs a)
{
    grid_dependency_sync();
    constexpr int kGroups = kGenThreads / W;
    __shared__ float red[2 * kGenWarps];
    const int l = threadIdx.x % W, lane = threadIdx.x & 31;
    const int N = a.N;
    const bool norm = a.w != nullptr;
    const int64_t step = (int64_t)gridDim.x * kGroups;
    for (int64_t r = blockIdx.x * (int64_t)kGroups + threadIdx.x / W; r < a.M; r += step) {
        const TX* xr = src_row<TX>(a.in[0], r);
        const TX* rr = a.in[1].p ? src_row<TX>(a.in[1], r) : nullptr;
        TX* sr = a.s ? static_cast<TX*>(a.s) + r * N : nullptr;
        // s of a column: the first walk adds, the later ones read the stored
        // stream (x or res may be overwritten by it by then)
        auto sum_at = [&](int c) {
            const float v = ldf(xr + c);
            return rr ? round_x<TX>(v + ldf(rr + c)) : v;
        };
        auto s_at = [&](int c) { return sr ? ldf(sr + c) : sum_at(c); };
        // the value that goes to 8 bits, before r: w' s, or s itself
        auto p_at = [&](int c, bool out) {
            const float v = s_at(c);
            return out ? weight_at(a.w, a.wt, c, a.variant) * v : v;
        };

        float ss = 0.f, am = 0.f;
        const Q8& row_q = a.q.v ? a.q : a.c;  // the 8-bit output or the checkpoint, never both
        const bool out8 = a.q.v != nullptr;
        for (int c = l; c < N; c += W) {
            const float v = sum_at(c);
            if (sr) sr[c] = cast_x<TX>(v);
            ss = fmaf(v, v, ss);
            if (row_q.v) am = max_nan(am, fabsf(out8 ? weight_at(a.w, a.wt, c, a.variant) * v : v));
        }
        group_sum_max<W>(ss, am, red);
        group_sync<W>();  // the group's s is visible to all of its threads
        const float rs = norm ? rsqrtf(fmaf(ss, a.inv_n, a.eps)) : 1.f;
        if (a.rstd && l == 0) a.rstd[r] = rs;
        if (a.y) {
            TX* yr = static_cast<TX*>(a.y) + r * N;
            for (int c = l; c < N; c += W) {
                const float xh = s_at(c) * rs;
                const float n = a.variant == 0 ? round_x<TX>(xh) : xh;
                yr[c] = cast_x<TX>(weight_at(a.w, a.wt, c, a.variant) * n);
            }
        }
        if (row_q.v) {
            // groups go to the row group's warps in turn, columns to lanes
            unsigned char* qr = static_cast<unsigned char*>(row_q.v) + r * N;
            const bool whole = row_q.shift == 31;
            const int first = whole ? 0 : l / 32;
            for (int g = first; g < row_q.ng; g += whole ? 1 : W / 32) {
                const int64_t c0 = whole ? 0 : (int64_t)g << row_q.shift;
                const int64_t end = whole ? N : c0 + (1 << row_q.shift);
                const int c1 = (int)(end < N ? end : N);
                float m = am;
                if (!whole) {
                    m = 0.f;
                    for (int c = (int)c0 + lane; c < c1; c += 32)
                        m = max_nan(m, fabsf(p_at(c, out8)));
#pragma unroll
                    for (int off = 16; off >= 1; off >>= 1)
                        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
                }
                const float sc = q8_scale(out8 ? m * rs : m, row_q.type);
                const float k = out8 ? rs * __frcp_rn(sc) : __frcp_rn(sc);
                if ((whole ? l : lane) == 0) row_q.scale[r * row_q.ng + g] = sc;
                for (int c = (int)c0 + (whole ? l : lane); c < c1; c += whole ? W : 32)
                    qr[c] = (unsigned char)q8_pack1(p_at(c, out8), k, row_q.type);
            }
        }
    }
}

template <typename TX, int W>
__global__ void __launch_bounds__(kGenThreads) add_bwd_general(BwdArgs a)
{
    grid_dependency_sync();
    constexpr int kGroups = kGenThreads / W;
    __shared__ float red[2 * kGenWarps];
    const int l = threadIdx.x % W;
    const int N = a.N;
    const int64_t gi = blockIdx.x * (int64_t)kGroups + threadIdx.x / W;
    const int64_t step = (int64_t)gridDim.x * kGroups;
    const bool packed = a.c.scale != nullptr;
    const bool cast = a.variant == 0 && !packed;  // the rounding points of expression 0
    const bool round_terms = cast && a.wt != kF32;
    // the row group's column sums: thread l alone touches columns l, l + W, ...
    float* wrow = a.ws ? a.ws + gi * N : nullptr;
    if (wrow)
        for (int c = l; c < N; c += W) wrow[c] = 0.f;
    for (int64_t r = gi; r < a.M; r += step) {
        const TX* sr = packed ? nullptr : src_row<TX>(a.in[0], r);
        const unsigned char* cr = packed ? a.in[0].p + r * N : nullptr;
        const TX* dyr = src_row<TX>(a.in[1], r);
        const TX* dsr = a.in[2].p ? src_row<TX>(a.in[2], r) : nullptr;
        const float rs = a.rstd[r];
        auto xh_at = [&](int c) {
            if (!packed) return ldf(sr + c) * rs;
            const float sc = a.c.scale[r * a.c.ng + (c >> a.c.shift)];
            return q8_unpack1(cr[c], a.c.type) * (sc * rs);
        };
        auto dn_at = [&](int c) {
            const float v = ldf(dyr + c) * weight_at(a.w, a.wt, c, a.variant);
            return cast ? round_x<TX>(v) : v;
        };
        float sum = 0.f, unused = 0.f;
        for (int c = l; c < N; c += W) sum = fmaf(dn_at(c), xh_at(c), sum);
        group_sum_max<W>(sum, unused, red);
        const float m = sum * a.inv_n;
        TX* dxr = static_cast<TX*>(a.dx) + r * N;
        for (int c = l; c < N; c += W) {
            const float xh = xh_at(c);
            const float v = rs * (dn_at(c) - xh * m);
            float term = ldf(dyr + c) * (cast ? round_x<TX>(xh) : xh);
            if (round_terms) term = round_x<TX>(term);
            dxr[c] = cast_x<TX>(dsr ? ldf(dsr + c) + v : v);
            if (wrow) wrow[c] += term;
        }
    }
}

template <typename TX>
__global__ void __launch_bounds__(kGenThreads) unpack_general(UnpackArgs a)
{
    grid_dependency_sync();
    const int64_t total = a.M * a.N, step = (int64_t)gridDim.x * kGenThreads;
    const unsigned char* q = static_cast<const unsigned char*>(a.c.v);
    TX* x = static_cast<TX*>(a.x);
    for (int64_t i = blockIdx.x * (int64_t)kGenThreads + threadIdx.x; i < total; i += step) {
        const int64_t r = i / a.N;
        const int c = (int)(i - r * a.N);
        const float sc = a.c.scale[r * a.c.ng + (c >> a.c.shift)];
        x[i] = cast_x<TX>(q8_unpack1(q[i], a.c.type) * sc);
    }
}

template <class F>
cudaError_t by_type(int xt, F&& f)
{
    if (xt == kF32)
        f(float{});
    else if (xt == kF16)
        f(__half{});
    else
        f(__nv_bfloat16{});
    return cudaGetLastError();
}

unsigned general_grid(int64_t M, int64_t N, int sms)
{
    const int64_t per = N > kWide ? 1 : kGenWarps;
    const int64_t ctas = (M + per - 1) / per, cap = 4LL * sms;
    return (unsigned)(ctas < cap ? ctas : cap);
}

}  // namespace

cudaError_t launch_add_fwd_general(cudaStream_t st, int xt, int sms, const FwdArgs& a)
{
    const unsigned grid = general_grid(a.M, a.N, sms);
    return by_type(xt, [&](auto t) {
        using TX = decltype(t);
        if (a.N > kWide)
            launch_pdl(add_fwd_general<TX, kGenThreads>, grid, kGenThreads, 0, st, a);
        else
            launch_pdl(add_fwd_general<TX, 32>, grid, kGenThreads, 0, st, a);
    });
}

int64_t add_bwd_general_rows(int64_t M, int64_t N, int sms)
{
    return (int64_t)general_grid(M, N, sms) * (N > kWide ? 1 : kGenWarps);
}

cudaError_t launch_add_bwd_general(cudaStream_t st, int xt, int64_t P, const BwdArgs& a)
{
    const unsigned grid = (unsigned)(P / (a.N > kWide ? 1 : kGenWarps));
    return by_type(xt, [&](auto t) {
        using TX = decltype(t);
        if (a.N > kWide)
            launch_pdl(add_bwd_general<TX, kGenThreads>, grid, kGenThreads, 0, st, a);
        else
            launch_pdl(add_bwd_general<TX, 32>, grid, kGenThreads, 0, st, a);
    });
}

cudaError_t launch_unpack_general(cudaStream_t st, int xt, int sms, const UnpackArgs& a)
{
    const int64_t ctas = (a.M * a.N + kGenThreads - 1) / kGenThreads, cap = 16LL * sms;
    return by_type(xt, [&](auto t) {
        launch_pdl(unpack_general<decltype(t)>, (unsigned)(ctas < cap ? ctas : cap), kGenThreads,
                   0, st, a);
    });
}

}  // namespace gbn
