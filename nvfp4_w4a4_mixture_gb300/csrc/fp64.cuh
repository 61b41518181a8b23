// fp64.cuh -- an exponential and a reciprocal in FP64 for the few values that are computed again.
// FP64 runs at 1/64 of the FP32 rate here (a warp instruction takes some 58 cycles), so both are as short
// as 52 bits allow; with the library's functions a token whose experts are ranked again took 2.8 us.
//   exp64  the table-driven exponential of Tang (ACM TOMS 15, 1989): x = (n / 32) ln 2 + r with |r| <= ln 2 / 64,
//          exp(x) = 2^(n / 32) (1 + r + ... + r^6 / 720). Three roundings count (the polynomial's last, the table's,
//          the product's), the polynomial's other ones and its remainder (r^7 / 5040) add a few hundredths of one:
//          the relative error is at most 3.1 * 2^-53
//   rcp64  two Newton steps from the FP32 reciprocal (2^-23, 2^-46, 2^-92): the last rounding alone, 2^-53
#pragma once
#include <cuda_runtime.h>

namespace moe {

__device__ __forceinline__ float fast_rcp(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

static __device__ const double kExp2[32] = {  // 2^(j / 32)
    0x1.0000000000000p+0, 0x1.059b0d3158574p+0, 0x1.0b5586cf9890fp+0, 0x1.11301d0125b51p+0,
    0x1.172b83c7d517bp+0, 0x1.1d4873168b9aap+0, 0x1.2387a6e756238p+0, 0x1.29e9df51fdee1p+0,
    0x1.306fe0a31b715p+0, 0x1.371a7373aa9cbp+0, 0x1.3dea64c123422p+0, 0x1.44e086061892dp+0,
    0x1.4bfdad5362a27p+0, 0x1.5342b569d4f82p+0, 0x1.5ab07dd485429p+0, 0x1.6247eb03a5585p+0,
    0x1.6a09e667f3bcdp+0, 0x1.71f75e8ec5f74p+0, 0x1.7a11473eb0187p+0, 0x1.82589994cce13p+0,
    0x1.8ace5422aa0dbp+0, 0x1.93737b0cdc5e5p+0, 0x1.9c49182a3f090p+0, 0x1.a5503b23e255dp+0,
    0x1.ae89f995ad3adp+0, 0x1.b7f76f2fb5e47p+0, 0x1.c199bdd85529cp+0, 0x1.cb720dcef9069p+0,
    0x1.d5818dcfba487p+0, 0x1.dfc97337b9b5fp+0, 0x1.ea4afa2a490dap+0, 0x1.f50765b6e4540p+0};

__device__ __forceinline__ double exp64(double x)
{
    if (!(fabs(x) < 700.0)) return exp(x);
    const int n = __double2int_rn(x * 0x1.71547652b82fep+5);
    // the longer part of ln 2 / 32 is exact times n
    const double r = fma(static_cast<double>(n), -0x1.473de6af278edp-39, fma(static_cast<double>(n), -0x1.62e42fef00000p-6, x));
    double p = fma(r, 1.0 / 720, 1.0 / 120);
    p = fma(r, p, 1.0 / 24);
    p = fma(r, p, 1.0 / 6);
    p = fma(r, p, 0.5);
    p = fma(r, p, 1.0);
    p = fma(r, p, 1.0) * kExp2[n & 31];
    return __hiloint2double(__double2hiint(p) + ((n >> 5) << 20), __double2loint(p));
}

// 1 / d for d >= 1
__device__ __forceinline__ double rcp64(double d)
{
    if (!(d < 1e30)) return 1.0 / d;
    double r = fast_rcp(static_cast<float>(d));
    r = fma(r, fma(-d, r, 1.0), r);
    return fma(r, fma(-d, r, 1.0), r);
}

}  // namespace moe
