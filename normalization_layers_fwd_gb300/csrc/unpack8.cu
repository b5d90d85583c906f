// unpack8.cu -- 8-bit values back to activations.
//
// Elementwise over the storage: a thread takes vectors of VEC consecutive
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
