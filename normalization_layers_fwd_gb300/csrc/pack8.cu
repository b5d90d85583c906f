// pack8.cu -- activations to 8-bit values and back, over the storage.
//
// Packing rows of whole groups: a group is `lanes` vectors in a row, of
// adjacent lanes, wherever its row begins; its maximum is a butterfly over
// them.  No shared memory and no barrier: kBatch vectors a thread in flight.
// Unpacking, elementwise: a thread takes vectors of VEC consecutive
// elements of [M, N], kBatch at once with all of their loads in flight, and
// follows their row and column without a division (each step adds a fixed
// number of rows and columns).  A vector inside one group needs one scale; at
// the end of a row or group each element looks its own up.
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
        float s[kBatch];
        int64_t rb[kBatch];
        int cb[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            rb[i] = r;
            cb[i] = c;
            if (v + i * step < whole) {
                const unsigned char* p = q + (v + i * step) * VEC;
                if constexpr (VEC == 8) {
                    const uint2 t = __ldcs(reinterpret_cast<const uint2*>(p));
                    w[i][0] = t.x;
                    w[i][1] = t.y;
                } else {
                    w[i][0] = __ldcs(reinterpret_cast<const unsigned*>(p));
                }
                s[i] = __ldg(a.c.scale + r * a.c.ng + (c >> sh));
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
            const int end = cb[i] + VEC - 1;
            if (end < a.N && (end >> sh) == (cb[i] >> sh)) {
#pragma unroll
                for (int p = 0; p < P; ++p) o[p] = mul2(o[p], splat2(s[i]));
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

template <typename TX, int kType>
__global__ void __launch_bounds__(kThreads) pack_vec(const __grid_constant__ FwdArgs a)
{
    grid_dependency_sync();
    constexpr int VEC = Vec<TX>::kN, P = VEC / 2;
    const int lanes = (1 << a.c.shift) / VEC;  // of a group: divides 32
    const int64_t total = a.M * a.N / VEC, step = (int64_t)gridDim.x * kThreads;
    const uint4* x = reinterpret_cast<const uint4*>(a.in[0].p);
    unsigned char* q = static_cast<unsigned char*>(a.c.v);
    const int64_t v0 = blockIdx.x * (int64_t)kThreads + threadIdx.x;
    // the same trip count for a whole warp: the butterflies need all lanes
    for (int64_t w = v0 - (threadIdx.x & 31); w < total; w += kBatch * step) {
        const int64_t v = w + (threadIdx.x & 31);
        uint4 u[kBatch];
        float m[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            u[i] = v + i * step < total ? __ldcs(x + v + i * step) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) m[i] = vec_amax<TX>(u[i]);
        for (int off = 1; off < lanes; off <<= 1)
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                m[i] = max_nan(m[i], __shfl_xor_sync(0xffffffffu, m[i], off));
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int64_t at = v + i * step;
            if (at >= total) break;
            const float sc = q8_scale(m[i], kType);
            const f2 k = splat2(__frcp_rn(sc));
            f2 f[P];
            unpack2<TX>(u[i], f);
            if constexpr (VEC == 8)
                __stcs(reinterpret_cast<uint2*>(q) + at,
                       make_uint2(q8_pack4<kType>(f[0], f[1], k, k),
                                  q8_pack4<kType>(f[2], f[3], k, k)));
            else
                __stcs(reinterpret_cast<unsigned*>(q) + at, q8_pack4<kType>(f[0], f[1], k, k));
            if ((threadIdx.x & (lanes - 1)) == 0) a.c.scale[at / lanes] = sc;
        }
    }
}

template <typename TX>
void pack_launch(cudaStream_t st, int sms, const FwdArgs& a)
{
    const int64_t total = a.M * a.N / Vec<TX>::kN, per = (int64_t)kThreads * kBatch;
    const int64_t ctas = (total + per - 1) / per, cap = 8LL * sms;
    const unsigned grid = (unsigned)(ctas < cap ? ctas : cap);
    if (a.c.type == kE4M3)
        launch_pdl(pack_vec<TX, kE4M3>, grid, kThreads, 0, st, a);
    else
        launch_pdl(pack_vec<TX, kInt8>, grid, kThreads, 0, st, a);
}

template <typename TX>
void unpack_launch(cudaStream_t st, int sms, const UnpackArgs& a)
{
    constexpr int VEC = Vec<TX>::kN;
    const int64_t whole = a.M * a.N / VEC, per = (int64_t)kThreads * kBatch;
    const int64_t ctas = (whole + per - 1) / per, cap = 8LL * sms;
    const int64_t grid = ctas < 1 ? 1 : ctas < cap ? ctas : cap;
    const int64_t step = grid * kThreads * VEC;
    auto go = [&](auto kernel) {
        launch_pdl(kernel, (unsigned)grid, kThreads, 0, st, a, step / a.N, (int)(step % a.N));
    };
    if (a.c.type == kE4M3)
        go(unpack_vec<TX, kE4M3>);
    else
        go(unpack_vec<TX, kInt8>);
}

}  // namespace

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
