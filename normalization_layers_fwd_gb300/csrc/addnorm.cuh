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
    int64_t nblocks;
    int R, stages;
    uint32_t off[3], stage_bytes, gm_off;  // gm_off: the group maxima's place
    size_t smem;
    unsigned* fault;
};

// One instance set per activation type (addfwd_*.cu, addbwd_*.cu).
enum FwdMode : int { kModeY = 0, kModeQ = 1, kModeYC = 2, kModeC = 3 };
enum BwdMode : int { kBwdS = 0, kBwdCast = 1, kBwdC = 2 };
cudaError_t launch_add_fwd_bf16(cudaStream_t st, int mode, const FwdArgs& a, const RowPlan& p);
cudaError_t launch_add_fwd_f16(cudaStream_t st, int mode, const FwdArgs& a, const RowPlan& p);
cudaError_t launch_add_fwd_f32(cudaStream_t st, int mode, const FwdArgs& a, const RowPlan& p);
cudaError_t launch_add_bwd_bf16(cudaStream_t st, int mode, const BwdArgs& a, const RowPlan& p);
cudaError_t launch_add_bwd_f16(cudaStream_t st, int mode, const BwdArgs& a, const RowPlan& p);
cudaError_t launch_add_bwd_f32(cudaStream_t st, int mode, const BwdArgs& a, const RowPlan& p);
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

// The scale of a group whose largest magnitude is a.
__device__ __forceinline__ float q8_scale(float a, int type)
{
    return max_nan(a * q8_rmax(type), kScaleFloor);
}

// Two values, already divided by their scale, as 8-bit codes (lo in the low
// byte), rounded to nearest even.  A value exceeds qmax by at most the two
// roundings of scale and 1 / scale, far less than half a step, so neither
// type clips a finite value.
__device__ __forceinline__ uint32_t q8_pack2(float lo, float hi, int type)
{
    if (type == kE4M3) {
        uint16_t r;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
        return r;
    }
    const int a = __float2int_rn(lo), b = __float2int_rn(hi);
    return (uint32_t)(a & 0xff) | ((uint32_t)(b & 0xff) << 8);
}

// Two 8-bit codes as floats (exact: e4m3 values are f16 values).
__device__ __forceinline__ f2 q8_unpack2(uint32_t w, int type)
{
    if (type == kE4M3) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
        return h2_to_f2(h);
    }
    return mk2((float)(int8_t)(w & 0xff), (float)(int8_t)((w >> 8) & 0xff));
}

}  // namespace gbn
