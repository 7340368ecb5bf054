// Host side of the group norm (include/rewy.h): argument checks, workspace sizes and
// launches.  Nothing here allocates device memory or waits for the device.
#include "gnorm.hpp"
#include "layer_host.hpp"

namespace rewy {
namespace {

int gnorm_args(const rewy_gnorm_desc* d, GnormArgs& a) {
  if (!d) return fail(REWY_EINVAL, "desc is NULL");
  if (d->M < 0 || d->M > INT32_MAX || d->D <= 0) return fail(REWY_EINVAL, "bad shape M=%lld D=%d", (long long)d->M, d->D);
  if (d->D > 16384) return fail(REWY_EUNSUPPORTED, "D=%d exceeds 16384", d->D);
  if (d->G <= 0 || d->D % d->G) return fail(REWY_EINVAL, "G=%d groups do not divide D=%d", d->G, d->D);
  REWY_TRY(check_dtype("dtype", d->dtype));
  REWY_TRY(check_dtype("w_dtype", d->w_dtype));
  if (d->act < REWY_ACT_NONE || d->act > REWY_ACT_SIGMOID) return fail(REWY_EINVAL, "bad act %d", d->act);
  if (d->center != 0 && d->center != 1) return fail(REWY_EINVAL, "bad center %d", d->center);
  if (d->quant < REWY_QUANT_NONE || d->quant > REWY_QUANT_INT8) return fail(REWY_EINVAL, "bad quant %d", d->quant);
  if (d->group != 0 && d->group != 32 && d->group != 64 && d->group != 128 && d->group != 256)
    return fail(REWY_EINVAL, "bad group %d (0, 32, 64, 128 or 256)", d->group);
  if (!(d->eps >= 0.f) || d->eps > 3e38f) return fail(REWY_EINVAL, "bad eps %g", (double)d->eps);
  memset(&a, 0, sizeof(a));
  a.M = d->M; a.D = d->D; a.G = d->G; a.L = d->D / d->G;
  a.act = d->act; a.center = d->center; a.quant = d->quant; a.group = d->group; a.eps = d->eps;
  a.ng = d->group ? (d->D + d->group - 1) / d->group : 1;
  const bool f32 = d->dtype == REWY_F32;
  a.lanes = gnorm_lanes(a.L, f32);
  a.rL = 1.f / (float)a.L;
  a.nblk = gnorm_bwd_blocks(a.M, a.D, f32);
  REWY_TRY(check_stride("x_stride", d->x_stride, d->D, a.xs));
  REWY_TRY(check_stride("z_stride", d->z_stride, d->D, a.zs));
  REWY_TRY(check_stride("y_stride", d->y_stride, d->D, a.ys));
  REWY_TRY(check_stride("dx_stride", d->dx_stride, d->D, a.dxs));
  return check_stride("dz_stride", d->dz_stride, d->D, a.dzs);
}
size_t gnorm_layout(GnormArgs& a, char* ws) {
  a.part = reinterpret_cast<float*>(ws);
  return std::max<size_t>(up((size_t)a.nblk * 2 * a.D * 4), ALIGN);
}

// M rows of a tensor of the norm's type
Place rows_of(const char* name, const void* p, const rewy_gnorm_desc* d, int64_t stride) {
  const int64_t e = (int64_t)esize(d->dtype);
  return {name, p, d->M, d->D * e, stride * e};
}
Place channels_of(const char* name, const void* p, const rewy_gnorm_desc* d) {
  return whole(name, p, d->D * (int64_t)esize(d->w_dtype));
}
Place stats_of(const char* name, const void* p, const rewy_gnorm_desc* d) { return whole(name, p, d->M * d->G * 4); }

}  // namespace
}  // namespace rewy

using namespace rewy;

REWY_API int rewy_gnorm_fwd(const rewy_gnorm_desc* d, const void* x, const void* z, const void* w, const void* b, void* y,
                            void* q, float* scale, float* mean, float* rstd, void* stream) {
  return guarded([&]() -> int {
    GnormArgs a;
    REWY_TRY(gnorm_args(d, a));
    const size_t e = esize(d->dtype), we = esize(d->w_dtype);
    const bool some = a.M > 0, codes = d->quant != REWY_QUANT_NONE;
    REWY_TRY(check_ptr("x", x, e, some));
    REWY_TRY(check_ptr("z", z, e, false));
    REWY_TRY(check_ptr("w", w, we, false));
    REWY_TRY(check_ptr("b", b, we, false));
    REWY_TRY(check_ptr("y", y, e, false));
    REWY_TRY(check_ptr("scale", scale, 4, some && codes));
    REWY_TRY(check_ptr("q", q, 1, some && codes));
    REWY_TRY(check_ptr("mean", mean, 4, some && a.center));
    REWY_TRY(check_ptr("rstd", rstd, 4, some));
    if (!codes && (q || scale)) return fail(REWY_EINVAL, "q and scale are given only when quant != NONE");
    if (!a.center && mean) return fail(REWY_EINVAL, "mean is given only with center");
    if (some && y && (y == x || y == z)) return fail(REWY_EINVAL, "y may not be x or z");
    if (!some) return REWY_OK;
    REWY_TRY(check_apart({rows_of("y", y, d, a.ys), whole("q", q, d->M * d->D), whole("scale", scale, d->M * a.ng * 4),
                          stats_of("mean", mean, d), stats_of("rstd", rstd, d)},
                         {rows_of("x", x, d, a.xs), rows_of("z", z, d, a.zs), channels_of("w", w, d), channels_of("b", b, d)}));
    a.x = x; a.z = z; a.w = w; a.b = b; a.y = y; a.q = q; a.scale = scale; a.mean = mean; a.rstd = rstd;
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const bool f32 = d->dtype == REWY_F32, wf32 = d->w_dtype == REWY_F32;
    return hip_check(traced("k_gnorm_fwd", s, [&] { return launch_gnorm_fwd(a, f32, wf32, s); }), "group norm");
  });
}

REWY_API size_t rewy_gnorm_workspace_bytes(const rewy_gnorm_desc* d) {
  GnormArgs a;
  return gnorm_args(d, a) == REWY_OK ? gnorm_layout(a, nullptr) : 0;
}

REWY_API int rewy_gnorm_bwd(const rewy_gnorm_desc* d, const void* x, const void* z, const void* w, const void* b,
                            const float* mean, const float* rstd, const void* dy, void* dx, void* dz, void* dw, void* db,
                            void* workspace, size_t ws_bytes, void* stream) {
  return guarded([&]() -> int {
    GnormArgs a;
    REWY_TRY(gnorm_args(d, a));
    const size_t e = esize(d->dtype), we = esize(d->w_dtype);
    const bool some = a.M > 0;
    REWY_TRY(check_ptr("x", x, e, some));
    REWY_TRY(check_ptr("z", z, e, false));
    REWY_TRY(check_ptr("w", w, we, false));
    REWY_TRY(check_ptr("b", b, we, false));
    REWY_TRY(check_ptr("mean", mean, 4, some && a.center));
    REWY_TRY(check_ptr("rstd", rstd, 4, some));
    REWY_TRY(check_ptr("dy", dy, e, some));
    REWY_TRY(check_ptr("dx", dx, e, some));
    REWY_TRY(check_ptr("dz", dz, e, some && z));
    REWY_TRY(check_ptr("dw", dw, we, false));
    REWY_TRY(check_ptr("db", db, we, false));
    if ((dz && !z) || (dw && !w) || (db && !b)) return fail(REWY_EINVAL, "dz, dw and db are given only with z, w and b");
    for (const void* out : {dx, dz})
      if (some && out && (out == x || out == z || out == dy)) return fail(REWY_EINVAL, "a gradient may not be an input");
    if (some && dx == dz) return fail(REWY_EINVAL, "dx may not be dz");
    const size_t need = gnorm_layout(a, static_cast<char*>(workspace));
    REWY_TRY(check_workspace(workspace, ws_bytes, need));
    REWY_TRY(check_apart({rows_of("dx", dx, d, a.dxs), rows_of("dz", dz, d, a.dzs), channels_of("dw", dw, d), channels_of("db", db, d)},
                         {rows_of("x", x, d, a.xs), rows_of("z", z, d, a.zs), rows_of("dy", dy, d, a.ys), channels_of("w", w, d),
                          channels_of("b", b, d), stats_of("mean", mean, d), stats_of("rstd", rstd, d)}));
    a.x = x; a.z = z; a.w = w; a.b = b; a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
    a.dy = dy; a.dx = dx; a.dz = dz; a.dw = dw; a.db = db;
    const float* part = a.part;
    if (!dw && !db) a.part = nullptr;
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const bool f32 = d->dtype == REWY_F32, wf32 = d->w_dtype == REWY_F32;
    if (some)
      REWY_TRY(hip_check(traced("k_gnorm_bwd", s, [&] { return launch_gnorm_bwd(a, f32, wf32, s); }), "group norm backward"));
    if (!dw && !db) return REWY_OK;
    const int64_t D = a.D;
    return hip_check(traced("k_colsum", s, [&] { return launch_colsum(part, some ? a.nblk : 0, 2 * D, 2 * D, dw, wf32, s, db, D); }),
                     "parameter gradients");
  });
}
