// Host side of the product of e4m3 operands (include/rewy.h): argument checks and
// launches.  Nothing here allocates device memory or waits for the device.
#include "layer_host.hpp"
#include "mm8.hpp"

using namespace rewy;

REWY_API int rewy_e4m3_linear(const rewy_e4m3_desc* d, const void* a, const float* a_scale, const void* w,
                              const float* w_scale, const void* bias, void* y, void* stream) {
  return guarded([&]() -> int {
    if (!d) return fail(REWY_EINVAL, "desc is NULL");
    if (d->M < 0 || d->N <= 0 || d->K <= 0) return fail(REWY_EINVAL, "bad shape M=%d N=%d K=%d", d->M, d->N, d->K);
    if (d->K % 16) return fail(REWY_EUNSUPPORTED, "K=%d is not a multiple of 16", d->K);
    // (a tile's last rows, up to 512 behind M, are counted in 32 bits)
    if (d->M > INT32_MAX - 1023) return fail(REWY_EUNSUPPORTED, "M=%d is too large", d->M);
    if (d->K > 1 << 20 || d->N > 1 << 24) return fail(REWY_EUNSUPPORTED, "N=%d or K=%d is too large", d->N, d->K);
    if (d->a_block != 0 && d->a_block != 128) return fail(REWY_EINVAL, "bad a_block %d (0 or 128)", d->a_block);
    if (d->w_rows != 1 && d->w_rows != 128) return fail(REWY_EINVAL, "bad w_rows %d (1 or 128)", d->w_rows);
    REWY_TRY(check_dtype("dtype", d->dtype));
    REWY_TRY(check_dtype("bias_dtype", d->bias_dtype));
    Mm8Args g;
    memset(&g, 0, sizeof(g));
    g.M = d->M; g.N = d->N; g.K = d->K; g.nb = (d->K + 127) / 128;
    g.ablk = d->a_block != 0; g.wrow = d->w_rows == 1; g.bias_f32 = d->bias_dtype == REWY_F32;
    REWY_TRY(check_stride("a_stride", d->a_stride, d->K, g.as));
    REWY_TRY(check_stride("w_stride", d->w_stride, d->K, g.ws));
    REWY_TRY(check_stride("y_stride", d->y_stride, d->N, g.ys));
    if (g.as % 16 || g.ws % 16) return fail(REWY_EINVAL, "a_stride and w_stride are multiples of 16 bytes");
    if (g.as > 1 << 22 || g.ws > 1 << 22) return fail(REWY_EUNSUPPORTED, "a_stride or w_stride exceeds 2^22 bytes");
    // (a launch takes fewer than 2^32 threads: tiles of 128 by 128 of 256 threads)
    if (((int64_t)d->M + 127) / 128 * (((int64_t)d->N + 127) / 128) >= 1 << 24)
      return fail(REWY_EUNSUPPORTED, "M=%d by N=%d is too large", d->M, d->N);
    const bool some = d->M > 0, f32 = d->dtype == REWY_F32;
    REWY_TRY(check_ptr("a", a, 16, some));
    REWY_TRY(check_ptr("a_scale", a_scale, 4, some));
    REWY_TRY(check_ptr("w", w, 16, some));
    REWY_TRY(check_ptr("w_scale", w_scale, 4, some));
    REWY_TRY(check_ptr("bias", bias, esize(d->bias_dtype), false));
    REWY_TRY(check_ptr("y", y, esize(d->dtype), some));
    if (!some) return REWY_OK;
    if (y == a || y == w) return fail(REWY_EINVAL, "y may not be a or w");
    const int64_t M = d->M, N = d->N, K = d->K, nb = g.nb, ye = (int64_t)esize(d->dtype);
    REWY_TRY(check_apart({{"y", y, M, N * ye, g.ys * ye}},
                         {{"a", a, M, K, g.as}, {"w", w, N, K, g.ws}, whole("a_scale", a_scale, 4 * M * (g.ablk ? nb : 1)),
                          whole("w_scale", w_scale, 4 * (g.wrow ? N : (N + 127) / 128) * nb),
                          whole("bias", bias, N * (int64_t)esize(d->bias_dtype))}));
    g.a = static_cast<const uint8_t*>(a); g.w = static_cast<const uint8_t*>(w);
    g.sa = a_scale; g.sw = w_scale; g.bias = bias; g.y = y;
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    return hip_check(traced(mm8_kernel(g), s, [&] { return launch_mm8(g, f32, s); }), "e4m3 product");
  });
}
