// pack8.cu -- activations to 8-bit values and back, over the storage.
//
// Units of 32 bytes of x (16 16-bit elements, 8 float32): one load, one store
// and one scale each.  Packing rows of whole groups, a group is a run of
// adjacent lanes wherever its row begins, and its maximum a butterfly over
// them: no shared memory, no barrier, kBatch units a thread in flight.
// [32768, 4096] bf16 in groups of 128, packed and unpacked: 131 us, 0.91 of
// measured copy bandwidth; with 16-byte vectors the pair took 9% longer, its
// warps issuing twice the shuffles, scales and indices per byte.
// Unpacking rows that are not whole units, by vectors: a thread takes vectors
// of VEC consecutive elements of [M, N], kBatch at once with all of their
// loads in flight, and follows their row and column without a division (each
// step adds a fixed number of rows and columns).  A vector needs one scale, or
// two at the end of a row or group; only narrow rows put more into one, and
// look each up.
#include "rowring.cuh"

namespace gbn {
namespace {

constexpr int kThreads = 256, kBatch = 4;

template <typename TX, int kType>
__global__ void __launch_bounds__(kThreads)
    unpack_vec(const __grid_constant__ UnpackArgs a, int64_t step_rows, int step_cols)
{
    grid_dependency_sync();
    constexpr int VEC = Vec<TX>::kN, P = VEC / 2;
    const int64_t total = a.M * a.N, step = (int64_t)gridDim.x * kThreads;
    const int64_t whole = total / VEC;  // vectors that end inside the tensor
    const unsigned char* q = static_cast<const unsigned char*>(a.c.v);
    TX* x = static_cast<TX*>(a.x);
    const int sh = a.c.shift;
    int64_t v = blockIdx.x * (int64_t)kThreads + threadIdx.x;
    int64_t r = v * VEC / a.N;
    int c = (int)(v * VEC - r * a.N);
    auto scale_at = [&](int64_t row, int col) {
        while (col >= a.N) {  // the element is in a later row
            col -= a.N;
            ++row;
        }
        return __ldg(a.c.scale + row * a.c.ng + (col >> sh));
    };
    for (; v < whole; ) {
        uint32_t w[kBatch][VEC / 4];
        float s0[kBatch], s1[kBatch];
        int eb[kBatch];  // the elements before eb take s0, the others s1; -1: three or more scales
        int64_t rb[kBatch];
        int cb[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            rb[i] = r;
            cb[i] = c;
            eb[i] = VEC;
            if (v + i * step < whole) {
                const unsigned char* p = q + (v + i * step) * VEC;
                if constexpr (VEC == 8) {
                    const uint2 t = __ldcs(reinterpret_cast<const uint2*>(p));
                    w[i][0] = t.x;
                    w[i][1] = t.y;
                } else {
                    w[i][0] = __ldcs(reinterpret_cast<const unsigned*>(p));
                }
                const float* const sc = a.c.scale + r * a.c.ng;
                const int g = c >> sh, end = c + VEC - 1;
                s0[i] = __ldg(sc + g);
                s1[i] = s0[i];
                int next = -1;
                if (end < a.N) {  // in this row
                    if (end >> sh != g) {
                        eb[i] = ((g + 1) << sh) - c;
                        next = g + 1;
                    }
                } else {  // and into the next one
                    const bool plain = (a.N - 1) >> sh == g && end - a.N < a.N;
                    eb[i] = plain ? a.N - c : -1;
                    next = a.c.ng;
                }
                if (next >= 0) s1[i] = __ldg(sc + next);
            }
            r += step_rows;
            c += step_cols;
            if (c >= a.N) {
                c -= a.N;
                ++r;
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (v + i * step >= whole) break;
            f2 o[P];
#pragma unroll
            for (int k = 0; k < VEC / 4; ++k)
                q8_unpack4<kType>(w[i][k], o[2 * k], o[2 * k + 1]);
            if (eb[i] >= 0) {
#pragma unroll
                for (int p = 0; p < P; ++p)
                    o[p] = mul2(o[p], mk2(2 * p < eb[i] ? s0[i] : s1[i],
                                          2 * p + 1 < eb[i] ? s0[i] : s1[i]));
            } else {
#pragma unroll
                for (int p = 0; p < P; ++p)
                    o[p] = mul2(o[p], mk2(scale_at(rb[i], cb[i] + 2 * p),
                                          scale_at(rb[i], cb[i] + 2 * p + 1)));
            }
            st_stream(x + (v + i * step) * VEC, pack2<TX>(o));
        }
        v += kBatch * step;
    }
    // the last total % VEC elements
    if (blockIdx.x == 0 && threadIdx.x < total - whole * VEC) {
        const int64_t i = whole * VEC + threadIdx.x, row = i / a.N;
        const float sc = a.c.scale[row * a.c.ng + ((int)(i - row * a.N) >> sh)];
        st1(x, i, q8_unpack1(q[i], kType) * sc);
    }
}

// 32 bytes of activations, one load or store each.
struct Unit32 {
    uint4 a, b;
};
__device__ __forceinline__ Unit32 ld_unit(const void* p)
{
    Unit32 u;
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(u.a.x), "=r"(u.a.y), "=r"(u.a.z), "=r"(u.a.w), "=r"(u.b.x), "=r"(u.b.y),
                   "=r"(u.b.z), "=r"(u.b.w)
                 : "l"(p));
    return u;
}
__device__ __forceinline__ void st_unit(void* p, const Unit32& u)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u.a.x),
                 "r"(u.a.y), "r"(u.a.z), "r"(u.a.w), "r"(u.b.x), "r"(u.b.y), "r"(u.b.z),
                 "r"(u.b.w)
                 : "memory");
}

// A lane takes units of 32 bytes of x.  lanes: units of a group (or of a row
// with one scale), a power of two of at most 32.
template <typename TX, int kType>
__global__ void __launch_bounds__(kThreads)
    pack_units(const __grid_constant__ FwdArgs a, int lanes, int log_lanes)
{
    grid_dependency_sync();
    constexpr int VEC = Vec<TX>::kN, P = VEC / 2;
    const int64_t total = a.M * a.N / (2 * VEC), step = (int64_t)gridDim.x * kThreads;
    const unsigned char* x = a.in[0].p;
    unsigned char* q = static_cast<unsigned char*>(a.c.v);
    const int lane = threadIdx.x & 31;
    // the same trip count for a whole warp: the butterflies need all lanes
    for (int64_t w = blockIdx.x * (int64_t)kThreads + threadIdx.x - lane; w < total;
         w += kBatch * step) {
        Unit32 u[kBatch];
        float m[kBatch];
        bool ok[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int64_t v = w + i * step + lane;
            ok[i] = v < total;
            if (ok[i])
                u[i] = ld_unit(x + v * 32);
            else
                u[i].a = u[i].b = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) m[i] = max_nan(vec_amax<TX>(u[i].a), vec_amax<TX>(u[i].b));
        for (int off = 1; off < lanes; off <<= 1)
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                m[i] = max_nan(m[i], __shfl_xor_sync(0xffffffffu, m[i], off));
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int64_t v = w + i * step + lane;
            const float sc = q8_scale(m[i], kType);
            const f2 k = splat2(__frcp_rn(sc));
            f2 f[P], g[P];
            unpack2<TX>(u[i].a, f);
            unpack2<TX>(u[i].b, g);
            if (!ok[i]) continue;
            if constexpr (VEC == 8)
                __stcs(reinterpret_cast<uint4*>(q) + v,
                       make_uint4(q8_pack4<kType>(f[0], f[1], k, k),
                                  q8_pack4<kType>(f[2], f[3], k, k),
                                  q8_pack4<kType>(g[0], g[1], k, k),
                                  q8_pack4<kType>(g[2], g[3], k, k)));
            else
                __stcs(reinterpret_cast<uint2*>(q) + v,
                       make_uint2(q8_pack4<kType>(f[0], f[1], k, k),
                                  q8_pack4<kType>(g[0], g[1], k, k)));
            if ((lane & (lanes - 1)) == 0) a.c.scale[v >> log_lanes] = sc;
        }
    }
}

// Units of 32 bytes of x that lie in one row and one group each.
template <typename TX, int kType>
__global__ void __launch_bounds__(kThreads)
    unpack_units(const __grid_constant__ UnpackArgs a, int64_t step_rows, int step_cols)
{
    grid_dependency_sync();
    constexpr int VEC = Vec<TX>::kN, P = VEC / 2;
    const int64_t total = a.M * a.N / (2 * VEC), step = (int64_t)gridDim.x * kThreads;
    const unsigned char* q = static_cast<const unsigned char*>(a.c.v);
    unsigned char* x = static_cast<unsigned char*>(a.x);
    int64_t v = blockIdx.x * (int64_t)kThreads + threadIdx.x;
    int64_t r = v * (2 * VEC) / a.N;
    int c = (int)(v * (2 * VEC) - r * a.N);
    for (; v < total; v += kBatch * step) {
        uint32_t w[kBatch][VEC / 2];
        float s[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (v + i * step < total) {
                if constexpr (VEC == 8) {
                    const uint4 t = __ldcs(reinterpret_cast<const uint4*>(q) + v + i * step);
                    w[i][0] = t.x, w[i][1] = t.y, w[i][2] = t.z, w[i][3] = t.w;
                } else {
                    const uint2 t = __ldcs(reinterpret_cast<const uint2*>(q) + v + i * step);
                    w[i][0] = t.x, w[i][1] = t.y;
                }
                s[i] = __ldg(a.c.scale + r * a.c.ng + (c >> a.c.shift));
            }
            r += step_rows;
            c += step_cols;
            if (c >= a.N) {
                c -= a.N;
                ++r;
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (v + i * step >= total) break;
            f2 f[P], g[P];
#pragma unroll
            for (int h = 0; h < VEC / 4; ++h) {
                q8_unpack4<kType>(w[i][h], f[2 * h], f[2 * h + 1]);
                q8_unpack4<kType>(w[i][VEC / 4 + h], g[2 * h], g[2 * h + 1]);
            }
            const f2 k = splat2(s[i]);
#pragma unroll
            for (int p = 0; p < P; ++p) {
                f[p] = mul2(f[p], k);
                g[p] = mul2(g[p], k);
            }
            st_unit(x + (v + i * step) * 32, Unit32{pack2<TX>(f), pack2<TX>(g)});
        }
    }
}

bool on_boundary(const void* p, int bytes)
{
    return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0;
}

unsigned persistent(int64_t units, int per_sm, int sms)
{
    const int64_t ctas = (units + kThreads * kBatch - 1) / (kThreads * kBatch);
    const int64_t cap = (int64_t)per_sm * sms;
    return (unsigned)(ctas < 1 ? 1 : ctas < cap ? ctas : cap);
}

template <typename TX>
void pack_launch(cudaStream_t st, int sms, const FwdArgs& a)
{
    constexpr int kUnit = 2 * Vec<TX>::kN;
    const unsigned grid = persistent(a.M * a.N / kUnit, 8, sms);
    const int lanes = (a.c.shift == 31 ? a.N : 1 << a.c.shift) / kUnit;
    int log_lanes = 0;
    while ((1 << log_lanes) < lanes) ++log_lanes;
    if (a.c.type == kE4M3)
        launch_pdl(pack_units<TX, kE4M3>, grid, kThreads, 0, st, a, lanes, log_lanes);
    else
        launch_pdl(pack_units<TX, kInt8>, grid, kThreads, 0, st, a, lanes, log_lanes);
}

template <typename TX>
void unpack_launch(cudaStream_t st, int sms, const UnpackArgs& a)
{
    constexpr int VEC = Vec<TX>::kN;
    auto go = [&](auto kernel, int per) {  // `per` elements a thread and turn
        const unsigned grid = persistent(a.M * a.N / per, 8, sms);
        const int64_t step = (int64_t)grid * kThreads * per;
        launch_pdl(kernel, grid, kThreads, 0, st, a, step / a.N, (int)(step % a.N));
    };
    // a unit's columns start at a multiple of its size, and so do groups
    const bool units = a.N % (2 * VEC) == 0 && on_boundary(a.x, 32);
    if (a.c.type == kE4M3)
        units ? go(unpack_units<TX, kE4M3>, 2 * VEC) : go(unpack_vec<TX, kE4M3>, VEC);
    else
        units ? go(unpack_units<TX, kInt8>, 2 * VEC) : go(unpack_vec<TX, kInt8>, VEC);
}

}  // namespace

bool pack_fast(int xt, const FwdArgs& a)
{
    const int unit = xt == kF32 ? 8 : 16, N = a.N;
    if (a.in[0].scattered || !on_boundary(a.in[0].p, 32) || !on_boundary(a.c.v, 16)) return false;
    if (a.c.shift != 31) return N % (1 << a.c.shift) == 0;
    const int lanes = N / unit;  // one scale a row
    return N % unit == 0 && lanes <= 32 && (lanes & (lanes - 1)) == 0;
}

cudaError_t launch_pack_fast(cudaStream_t st, int xt, int sms, const FwdArgs& a)
{
    if (xt == kF32)
        pack_launch<float>(st, sms, a);
    else if (xt == kF16)
        pack_launch<__half>(st, sms, a);
    else
        pack_launch<__nv_bfloat16>(st, sms, a);
    return cudaGetLastError();
}

cudaError_t launch_unpack_fast(cudaStream_t st, int xt, int sms, const UnpackArgs& a)
{
    if (xt == kF32)
        unpack_launch<float>(st, sms, a);
    else if (xt == kF16)
        unpack_launch<__half>(st, sms, a);
    else
        unpack_launch<__nv_bfloat16>(st, sms, a);
    return cudaGetLastError();
}

}  // namespace gbn
