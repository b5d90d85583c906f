// addnorm.cuh -- shared parts of the residual-stream operators: RMSNorm with
// the residual's addition, its 8-bit output, the 8-bit activation
// checkpoint, and their backwards.  gbnorm.h states the formulas and the
// rounding points.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace gbn {

enum Q8Type : int { kE4M3 = 8, kInt8 = 9 };

// Sign-free size of one 8-bit type's largest value, and its reciprocal
// rounded to f32.
__host__ __device__ constexpr float q8_max(int type) { return type == kE4M3 ? 448.f : 127.f; }
__host__ __device__ constexpr float q8_rmax(int type)
{
    return type == kE4M3 ? 1.f / 448.f : 1.f / 127.f;
}
constexpr float kScaleFloor = 0x1p-100f;

// One input: contiguous rows of row_bytes, or rows where `map` puts them.
// `total` is the byte count of a contiguous input.
struct RowSrc {
    const unsigned char* p;
    int64_t row_bytes, total;
    int scattered;
    RowMap map;
};

// An 8-bit tensor [M, N] with its scales [M, ng]: groups of 1 << shift
// columns, or whole rows (shift 31: every column's group is 0).
struct Q8 {
    void* v;
    float* scale;
    int type, shift, ng;
};

struct FwdArgs {
    RowSrc in[2];   // x, res (p null: none)
    const void* w;  // null in act_pack8
    void *s, *y;    // nullable
    Q8 q, c;        // v null: none
    float* rstd;    // nullable
    int64_t M;
    int N;
    float eps, inv_n;
    int wt, variant;
};

struct BwdArgs {
    RowSrc in[3];  // the stream s or the checkpoint's bytes, dy, ds (p null: none)
    Q8 c;          // the checkpoint's type, groups and scales (scale null: in[0] is the stream)
    const void* w;
    const float* rstd;
    void* dx;
    float* ws;  // partial rows of dw, null: not wanted
    int64_t M;
    int N;
    float inv_n;
    int wt, variant;
};

struct UnpackArgs {
    Q8 c;
    void* x;
    int64_t M;
    int N;
};

// The launch of a fast kernel (addnorm_fast.cuh): persistent CTAs over row
// blocks of R rows through a ring of `stages` stages, each holding one block
// of every input at off[t].
struct RowPlan {
    int sid, edge, grid;
    int W, G;              // threads of a row group, row groups of a CTA
    int in_order;          // every input's rows are in order
    int tail;              // some input does not end on a 16-byte boundary
    int64_t nblocks;
    int R, stages;
    uint32_t off[3], stage_bytes, gm_off;  // gm_off: the group maxima's place
    size_t smem;
    unsigned* fault;
};

// One instance set per activation type (addfwd_*.cu, addbwd_*.cu).
// The 8-bit modes come once per 8-bit type: + kModeInt8.
enum FwdMode : int { kModeY = 0, kModeQ = 1, kModeYC = 2, kModeC = 3, kModeInt8 = 4 };
// kBwdCast: expression 0's rounding points, kBwdCast16 with a weight of x's type.
enum BwdMode : int { kBwdS = 0, kBwdCast = 1, kBwdC = 2, kBwdInt8 = 3, kBwdCast16 = 4 };
cudaError_t launch_add_fwd_bf16(cudaStream_t st, int mode, const FwdArgs& a, const RowPlan& p);
cudaError_t launch_add_fwd_f16(cudaStream_t st, int mode, const FwdArgs& a, const RowPlan& p);
cudaError_t launch_add_fwd_f32(cudaStream_t st, int mode, const FwdArgs& a, const RowPlan& p);
cudaError_t launch_add_bwd_bf16(cudaStream_t st, int mode, const BwdArgs& a, const RowPlan& p);
cudaError_t launch_add_bwd_f16(cudaStream_t st, int mode, const BwdArgs& a, const RowPlan& p);
cudaError_t launch_add_bwd_f32(cudaStream_t st, int mode, const BwdArgs& a, const RowPlan& p);
// act_pack8 and act_unpack8 over the storage (pack8.cu), for contiguous
// tensors: to pack where pack_fast says so (rows of whole groups), to unpack
// on 16-byte boundaries.
bool pack_fast(int xt, const FwdArgs& a);
cudaError_t launch_pack_fast(cudaStream_t st, int xt, int sms, const FwdArgs& a);
cudaError_t launch_unpack_fast(cudaStream_t st, int xt, int sms, const UnpackArgs& a);

// Launches of the general kernels (any width, alignment and layout).
// Forward: everything FwdArgs asks for; with w null only the checkpoint.
cudaError_t launch_add_fwd_general(cudaStream_t st, int xt, int sms, const FwdArgs& a);
cudaError_t launch_add_bwd_general(cudaStream_t st, int xt, int64_t P, const BwdArgs& a);
cudaError_t launch_unpack_general(cudaStream_t st, int xt, int sms, const UnpackArgs& a);
// Partial rows (row groups launched) of the general backward.
int64_t add_bwd_general_rows(int64_t M, int64_t N, int sms);

// ------------------------------------------------------------ 8-bit values
// Larger of two magnitudes; NaN when either is (a plain fmaxf drops it).
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The scale of a group whose largest magnitude is a: NaN for an infinity or a
// NaN (a - a), so that whatever the group's codes are they read back as NaN.
__device__ __forceinline__ float q8_scale(float a, int type)
{
    return max_nan(fmaf(a, q8_rmax(type), a - a), kScaleFloor);
}

// 8-bit codes of four values v times k (one over their scale; r entering with
// it for an output), the first in the low byte, rounded to nearest even.  A
// product exceeds qmax by at most the roundings of scale and 1 / scale, far
// less than half a step, so neither type clips a finite value.  int8: adding
// 1.5 2^23 leaves the nearest integer in the low bits of the sum (the spacing
// of floats there is 1); the product is rounded before it, in instructions
// that may not be fused (ptxas 13.0 did fuse mul.rn.f32x2 with
// add.rn.f32x2, and products next to a half went the other way).
template <int kType>
__device__ __forceinline__ uint32_t q8_pack4(f2 a, f2 b, f2 ka, f2 kb)
{
    if constexpr (kType == kE4M3) {
        a = mul2(a, ka);
        b = mul2(b, kb);
        uint32_t r;
        asm("{\n\t.reg .b16 l, h;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
            "mov.b32 %0, {l, h};\n\t}"
            : "=r"(r)
            : "f"(lo2(a)), "f"(hi2(a)), "f"(lo2(b)), "f"(hi2(b)));
        return r;
    } else {
        auto code = [](float v, float k) {
            return __float_as_uint(__fadd_rn(__fmul_rn(v, k), 12582912.f));
        };
        return __byte_perm(__byte_perm(code(lo2(a), lo2(ka)), code(hi2(a), hi2(ka)), 0x0040),
                           __byte_perm(code(lo2(b), lo2(kb)), code(hi2(b), hi2(kb)), 0x0040),
                           0x5410);
    }
}

// Four 8-bit codes as floats, exactly.  e4m3 values are f16 values.  int8: a
// byte with its sign bit turned, under the exponent of 2^23, is 2^23 + 128 +
// its value.
template <int kType>
__device__ __forceinline__ void q8_unpack4(uint32_t w, f2& a, f2& b)
{
    if constexpr (kType == kE4M3) {
        uint32_t l, h;
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(l), "=r"(h)
            : "r"(w));
        a = h2_to_f2(l);
        b = h2_to_f2(h);
    } else {
        const uint32_t t = w ^ 0x80808080u, e = 0x4b000000u;
        const f2 m = splat2(-8388736.f);  // -(2^23 + 128)
        a = add2(mk2(__uint_as_float(__byte_perm(t, e, 0x7440)),
                     __uint_as_float(__byte_perm(t, e, 0x7441))), m);
        b = add2(mk2(__uint_as_float(__byte_perm(t, e, 0x7442)),
                     __uint_as_float(__byte_perm(t, e, 0x7443))), m);
    }
}

// One value (the general kernels).
__device__ __forceinline__ uint32_t q8_pack1(float v, float k, int type)
{
    const f2 a = mk2(v, 0.f), z = splat2(0.f), kk = splat2(k);
    return (type == kE4M3 ? q8_pack4<kE4M3>(a, z, kk, z) : q8_pack4<kInt8>(a, z, kk, z)) & 0xffu;
}
__device__ __forceinline__ float q8_unpack1(uint32_t b, int type)
{
    f2 v, unused;
    if (type == kE4M3)
        q8_unpack4<kE4M3>(b, v, unused);
    else
        q8_unpack4<kInt8>(b, v, unused);
    return lo2(v);
}

}  // namespace gbn
