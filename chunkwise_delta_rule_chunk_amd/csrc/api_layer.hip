// Host side of the operators around the token mixer (include/rewy.h): argument
// checks, workspace sizes and launches.  Nothing here allocates device memory
// or waits for the device.
#include "layer_host.hpp"
#include "ssm.hpp"

namespace rewy {
namespace {

// ---- RMS norm -----------------------------------------------------------------
int norm_args(const rewy_norm_desc* d, NormArgs& a) {
  if (!d) return fail(REWY_EINVAL, "desc is NULL");
  if (d->M < 0 || d->M > INT32_MAX || d->D <= 0) return fail(REWY_EINVAL, "bad shape M=%lld D=%d", (long long)d->M, d->D);
  if (d->D > 16384) return fail(REWY_EUNSUPPORTED, "D=%d exceeds 16384", d->D);
  REWY_TRY(check_dtype("dtype", d->dtype));
  REWY_TRY(check_dtype("w_dtype", d->w_dtype));
  if (d->quant < REWY_QUANT_NONE || d->quant > REWY_QUANT_INT8) return fail(REWY_EINVAL, "bad quant %d", d->quant);
  if (d->group != 0 && d->group != 32 && d->group != 64 && d->group != 128 && d->group != 256)
    return fail(REWY_EINVAL, "bad group %d (0, 32, 64, 128 or 256)", d->group);
  if (!(d->eps >= 0.f) || d->eps > 3e38f) return fail(REWY_EINVAL, "bad eps %g", (double)d->eps);
  memset(&a, 0, sizeof(a));
  a.M = d->M; a.D = d->D; a.quant = d->quant; a.group = d->group; a.eps = d->eps;
  a.ng = d->group ? (d->D + d->group - 1) / d->group : 1;
  REWY_TRY(check_stride("x_stride", d->x_stride, d->D, a.xs));
  REWY_TRY(check_stride("res_stride", d->res_stride, d->D, a.rs));
  REWY_TRY(check_stride("sum_stride", d->sum_stride, d->D, a.ss));
  REWY_TRY(check_stride("y_stride", d->y_stride, d->D, a.ys));
  a.nblk = norm_bwd_blocks(d->M, d->D, d->dtype == REWY_F32);
  return REWY_OK;
}
// An output over an input row by row: with another stride a row would be written before
// another workgroup has read it.
int norm_in_place(const NormArgs& a, const char* out, const void* o, int64_t os, const char* in, const void* i, int64_t is) {
  if (a.M > 1 && o && o == i && os != is) return fail(REWY_EINVAL, "%s over %s needs the same stride", out, in);
  return REWY_OK;
}
size_t norm_ws(const NormArgs& a) { return up(std::max<size_t>((size_t)a.nblk * a.D * 4, 1)); }

// ---- short convolution ------------------------------------------------------------
int conv_args(const rewy_conv_desc* d, ConvArgs& a) {
  if (!d) return fail(REWY_EINVAL, "desc is NULL");
  memset(&a, 0, sizeof(a));
  REWY_TRY(seq_args(d->B, d->T, d->N, d->cu_seqlens, d->cu_seqlens_host, a.seq));
  if (d->D <= 0 || d->D > 1 << 23) return fail(REWY_EINVAL, "bad shape D=%d", d->D);
  if (d->W < 2 || d->W > 4) return fail(d->W < 1 ? REWY_EINVAL : REWY_EUNSUPPORTED, "W=%d not supported (2 to 4 taps)", d->W);
  REWY_TRY(check_dtype("dtype", d->dtype));
  REWY_TRY(check_dtype("w_dtype", d->w_dtype));
  if (d->act != REWY_ACT_NONE && d->act != REWY_ACT_SILU) return fail(REWY_EINVAL, "bad act %d", d->act);
  a.D = d->D; a.W = d->W; a.act = d->act;
  REWY_TRY(check_stride("x_stride", d->x_stride, d->D, a.xs));
  REWY_TRY(check_stride("y_stride", d->y_stride, d->D, a.ys));
  REWY_TRY(check_stride("dx_stride", d->dx_stride, d->D, a.dxs));
  conv_bwd_shape(a.seq.total, a.D, a.run, a.tiles);
  // waves of the forward (runs half as long) and of a step: under 2^32 threads a launch
  if ((2 * (int64_t)a.tiles + a.seq.N) * conv_cblocks(a.D) >= 1 << 26)
    return fail(REWY_EUNSUPPORTED, "%d sequences and %d tokens of %d channels are too many", a.seq.N, a.seq.total, a.D);
  return REWY_OK;
}
size_t conv_ws(const ConvArgs& a) { return up(std::max<size_t>((size_t)a.tiles * (a.W + 1) * a.D * 4, 1)); }

int conv_forward(const rewy_conv_desc* d, bool step, const void* x, const void* w, const void* bias, const void* h0,
                 void* y, void* ht, void* stream) {
  ConvArgs a;
  REWY_TRY(conv_args(d, a));
  if (step && (d->T != 1 || d->cu_seqlens)) return fail(REWY_EINVAL, "a step has T == 1 and no cu_seqlens (got T=%d)", d->T);
  const bool some = a.seq.total > 0;
  const size_t e = esize(d->dtype), we = esize(d->w_dtype);
  REWY_TRY(check_ptr("x", x, e, some));
  REWY_TRY(check_ptr("w", w, we, some));
  REWY_TRY(check_ptr("bias", bias, we, false));
  REWY_TRY(check_ptr("h0", h0, e, false));
  REWY_TRY(check_ptr("y", y, e, some));
  REWY_TRY(check_ptr("ht", ht, e, false));
  if (!step && ht && ht == h0) return fail(REWY_EINVAL, "ht may not be h0");
  if (!step && some && y == x) return fail(REWY_EINVAL, "y may not be x");
  if (!some && !ht) return REWY_OK;
  a.x = x; a.w = w; a.bias = bias; a.h0 = h0; a.y = y; a.ht = ht;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const bool f32 = d->dtype == REWY_F32, wf32 = d->w_dtype == REWY_F32;
  if (step) return hip_check(traced("k_conv_step", s, [&] { return launch_conv_step(a, f32, wf32, s); }), "convolution step");
  return hip_check(traced("k_conv_fwd", s, [&] { return launch_conv_fwd(a, f32, wf32, s); }), "convolution");
}

// ---- selective state space scan ---------------------------------------------------
// Tokens of a segment, whole chunks, at least 256: as long as there are SEGMENTS pairs of a
// segment and a head (a longer segment means fewer states to join).  With one head a
// workgroup (V = 128, the walks of V = 64) that is two workgroups for each CU; where heads
// share one (V = 64 and 32 of the forward) it is half or a quarter as many.  Sequences of equal
// length: ceil(T / segment) each.  Packed ones end with half a segment on average, which
// leaves the target (N - 1) / 2 a head less, at least half of it.
int ssm_segment(const SeqArgs& q, int H, int most) {
  constexpr int64_t SEGMENTS = 512;
  int64_t want;
  if (q.cu) {
    const int64_t whole = std::max(SEGMENTS - (int64_t)(q.N - 1) * H / 2, SEGMENTS / 2);
    want = ((int64_t)q.total * H + whole - 1) / whole;
  } else {
    const int64_t each = std::max<int64_t>(SEGMENTS / ((int64_t)q.N * H), 1);
    want = (q.T + each - 1) / each;
  }
  return (int)std::min<int64_t>(most, std::max<int64_t>(256, up64(want)));
}

int ssm_args(const rewy_ssm_desc* d, bool bwd, SsmArgs& a) {
  if (!d) return fail(REWY_EINVAL, "desc is NULL");
  memset(&a, 0, sizeof(a));
  REWY_TRY(seq_args(d->B, d->T, d->N, d->cu_seqlens, d->cu_seqlens_host, a.seq));
  if (d->H <= 0 || d->G <= 0 || d->H > 65536 || d->H % d->G)
    return fail(REWY_EINVAL, "bad heads H=%d G=%d (H must be a multiple of G)", d->H, d->G);
  REWY_TRY(check_dtype("dtype", d->dtype));
  REWY_TRY(check_dtype("dt_dtype", d->dt_dtype));
  auto ok = [&](int v) { return v == 32 || v == 64 || (v == 128 && d->dtype == REWY_BF16); };
  if (d->K <= 0 || d->V <= 0) return fail(REWY_EINVAL, "bad shape K=%d V=%d", d->K, d->V);
  if (!ok(d->K) || !ok(d->V))
    return fail(REWY_EUNSUPPORTED, "K=%d V=%d not supported (32, 64 or 128; fp32 32 or 64)", d->K, d->V);
  a.H = d->H; a.G = d->G; a.K = d->K; a.V = d->V; a.per = d->H / d->G;
  a.dt_f32 = d->dt_dtype == REWY_F32;
  const int64_t xr = (int64_t)d->H * d->V, br = (int64_t)d->G * d->K;
  struct { const char* name; int64_t given, row; int64_t* out; } st[] = {
      {"x_stride", d->x_stride, xr, &a.xs},   {"b_stride", d->b_stride, br, &a.bs},   {"c_stride", d->c_stride, br, &a.cs},
      {"y_stride", d->y_stride, xr, &a.ys},   {"dx_stride", d->dx_stride, xr, &a.dxs}, {"db_stride", d->db_stride, br, &a.dbs},
      {"dc_stride", d->dc_stride, br, &a.dcs}};
  for (const auto& e : st) {
    REWY_TRY(check_stride(e.name, e.given, e.row, *e.out));
    if (*e.out * esize(d->dtype) % 16) return fail(REWY_EINVAL, "%s is not a multiple of 16 bytes", e.name);
    if (*e.out > 1 << 22) return fail(REWY_EUNSUPPORTED, "%s %lld exceeds 2^22 elements", e.name, (long long)*e.out);
  }
  const int64_t total = a.seq.total;
  const int longest = a.seq.cu ? a.seq.total : a.seq.T;
  // (the bf16 backward's decay gradient is summed from the ends of the segments, and its
  // error grows with their length: 1024 tokens would double it)
  a.seg = ssm_segment(a.seq, a.H, bwd && d->dtype == REWY_BF16 ? SEG_CHUNKS * CH : INT32_MAX / CH * CH);
  a.two = longest > a.seg;
  auto slots = [&](int64_t L) {  // (ssm.hpp)
    return a.seq.cu ? total / L + a.seq.N : a.seq.N * std::max<int64_t>((a.seq.T + L - 1) / L, 1);
  };
  const int64_t nslot = slots(a.seg), nchunk = slots(CH);
  a.nslot = (int)std::min<int64_t>(nslot, INT32_MAX);
  a.nchunk = (int)std::min<int64_t>(nchunk, INT32_MAX);
  // Head ranges that share a group's dB and dC.  A workgroup of the chunk backward
  // fills a CU and costs about its heads plus one (its B and C tiles, the joint
  // products); the ranges are the ones with the shortest schedule on 256 CUs, and
  // of those the fewest, as each range adds a partial sum to memory.
  int64_t best = INT64_MAX;
  a.split = 1;
  for (int sp = 1; bwd && sp <= std::min(a.per, 32); ++sp) {
    const int64_t rounds = (nchunk * a.G * sp + 255) / 256, cost = rounds * ((a.per + sp - 1) / sp + 1);
    if (cost < best) {
      best = cost;
      a.split = sp;
    }
  }
  // a launch takes fewer than 2^32 threads: gates and C B^T, the walks, the token-serial
  // form and the pass, and the backward's chunks and sums
  const int64_t threads[] = {(nchunk * a.H + nchunk * a.G * 10 + 8) * 64, nslot * a.H * 512, (int64_t)a.seq.N * a.H * 256,
                             bwd ? nchunk * a.G * a.split * 1024 : 0, bwd ? nchunk * a.H * 64 + total * a.G * a.K / 2 + 1024 : 0};
  for (int64_t n : threads)
    if (n >= (int64_t)1 << 32)
      return fail(REWY_EUNSUPPORTED, "%lld sequences and %lld tokens of %d heads are too many", (long long)a.seq.N,
                  (long long)total, a.H);
  return REWY_OK;
}

size_t ssm_layout(SsmArgs& a, bool f32, bool bwd, char* ws) {
  size_t off = 0;
  auto take = [&](auto*& p, size_t n) {
    using E = std::remove_reference_t<decltype(*p)>;
    p = reinterpret_cast<E*>(ws + off);
    off += up(n);
  };
  const size_t kv = (size_t)a.H * a.K * a.V, e = f32 ? 4 : 2, tok = (size_t)a.H * a.seq.total * 4;
  char* gates;
  take(gates, (size_t)a.nchunk * a.H * CH * sizeof(Gate));
  a.gates = gates;
  take(a.cb, (size_t)a.nchunk * a.G * 10 * 256 * 4);
  if (a.two) {
    take(a.sf, a.nslot * kv * 4);
    if (bwd) take(a.sr, a.nslot * kv * 4);
    take(a.gsum, (size_t)2 * a.nslot * a.H * 4);
  }
  if (bwd) {
    char *hs, *hd;
    take(hs, a.nchunk * kv * e);
    take(hd, a.nchunk * kv * e);
    a.hs = hs;
    a.hd = hd;
    take(a.rx, tok);
    take(a.cx, tok);
    take(a.ri, 2 * tok);
    take(a.ci, 2 * tok);
    take(a.tot, (size_t)a.nchunk * a.H * 16);
    take(a.cd, tok);
    take(a.ends, (size_t)a.nslot * a.H * 8);
    take(a.hdot, (size_t)a.nchunk * a.H * 4);
    take(a.dpart, (size_t)a.nchunk * a.H * 4);
    take(a.apart, (size_t)a.nchunk * 2 * a.H * 8);
    if (a.split > 1) take(a.bcpart, (size_t)2 * a.split * a.seq.total * a.G * a.K * 4);
  }
  return std::max<size_t>(off, ALIGN);
}

struct SsmIn {
  const void *x, *dt;
  const float *a_log, *dt_bias;
  const void *b, *c;
  const float *D, *h0;
};
int ssm_inputs(const rewy_ssm_desc* d, const SsmIn& in, SsmArgs& a) {
  const bool some = a.seq.total > 0;
  REWY_TRY(check_ptr("x", in.x, 16, some));
  REWY_TRY(check_ptr("dt", in.dt, esize(d->dt_dtype), some));
  REWY_TRY(check_ptr("A_log", in.a_log, 4, some));
  REWY_TRY(check_ptr("dt_bias", in.dt_bias, 4, false));
  REWY_TRY(check_ptr("b", in.b, 16, some));
  REWY_TRY(check_ptr("c", in.c, 16, some));
  REWY_TRY(check_ptr("D", in.D, 4, false));
  REWY_TRY(check_ptr("h0", in.h0, 16, false));
  a.x = in.x; a.dt = in.dt; a.a_log = in.a_log; a.dt_bias = in.dt_bias;
  a.b = in.b; a.c = in.c; a.d = in.D; a.h0 = in.h0;
  return REWY_OK;
}

// fp32 [N, H, K, V]: dst = src, or zeros (a call without tokens)
__global__ __launch_bounds__(256) void k_state_through(f32x4* dst, const f32x4* src, int64_t n) {
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    dst[i] = src ? src[i] : zero4();
}
int state_through(const SsmArgs& a, float* dst, const float* src, hipStream_t s) {
  if (!dst || dst == src) return REWY_OK;
  const int64_t n = (int64_t)a.seq.N * a.H * a.K * a.V / 4;
  return hip_check(traced("k_state_through", s,
                          [&] {
                            REWY_LAUNCH(k_state_through, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 4096)), dim3(256),
                                        s, reinterpret_cast<f32x4*>(dst), reinterpret_cast<const f32x4*>(src), n);
                            return hipGetLastError();
                          }),
                   "state copy");
}

}  // namespace
}  // namespace rewy

using namespace rewy;

REWY_API int rewy_norm_fwd(const rewy_norm_desc* d, const void* x, const void* res, const void* w, void* sum, void* y,
                           void* q, float* scale, float* rstd, void* stream) {
  return guarded([&]() -> int {
    NormArgs a;
    REWY_TRY(norm_args(d, a));
    const size_t e = esize(d->dtype);
    const bool some = a.M > 0;
    REWY_TRY(check_ptr("x", x, e, some));
    REWY_TRY(check_ptr("res", res, e, false));
    REWY_TRY(check_ptr("w", w, esize(d->w_dtype), false));
    REWY_TRY(check_ptr("sum", sum, e, false));
    REWY_TRY(check_ptr("y", y, e, false));
    REWY_TRY(check_ptr("rstd", rstd, 4, false));
    REWY_TRY(check_ptr("scale", scale, 4, some && d->quant != REWY_QUANT_NONE));
    REWY_TRY(check_ptr("q", q, 1, some && d->quant != REWY_QUANT_NONE));
    if (d->quant == REWY_QUANT_NONE && (q || scale)) return fail(REWY_EINVAL, "q and scale are given only when quant != NONE");
    REWY_TRY(norm_in_place(a, "sum", sum, a.ss, "x", x, a.xs));
    REWY_TRY(norm_in_place(a, "sum", sum, a.ss, "res", res, a.rs));
    REWY_TRY(norm_in_place(a, "y", y, a.ys, "x", x, a.xs));
    REWY_TRY(norm_in_place(a, "y", y, a.ys, "res", res, a.rs));
    if (!some) return REWY_OK;
    a.x = x; a.res = res; a.w = w; a.sum = sum; a.y = y; a.q = q; a.scale = scale; a.rstd = rstd;
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    return hip_check(traced("k_norm_fwd", s,
                            [&] { return launch_norm_fwd(a, d->dtype == REWY_F32, d->w_dtype == REWY_F32, s); }),
                     "RMS norm");
  });
}

REWY_API size_t rewy_norm_workspace_bytes(const rewy_norm_desc* d) {
  NormArgs a;
  return norm_args(d, a) == REWY_OK ? norm_ws(a) : 0;
}

REWY_API int rewy_norm_bwd(const rewy_norm_desc* d, const void* sv, const void* w, const float* rstd, const void* dy,
                           const void* ds, void* dx, void* dw, void* workspace, size_t ws_bytes, void* stream) {
  return guarded([&]() -> int {
    NormArgs a;
    REWY_TRY(norm_args(d, a));
    const size_t e = esize(d->dtype), we = esize(d->w_dtype);
    const bool some = a.M > 0;
    REWY_TRY(check_ptr("s", sv, e, some));
    REWY_TRY(check_ptr("w", w, we, false));
    REWY_TRY(check_ptr("rstd", rstd, 4, some));
    REWY_TRY(check_ptr("dy", dy, e, some));
    REWY_TRY(check_ptr("ds", ds, e, false));
    REWY_TRY(check_ptr("dx", dx, e, some));
    REWY_TRY(check_ptr("dw", dw, we, false));
    if (dw && !w) return fail(REWY_EINVAL, "dw is given without w");
    REWY_TRY(norm_in_place(a, "dx", dx, a.ss, "s", sv, a.xs));
    REWY_TRY(norm_in_place(a, "dx", dx, a.ss, "dy", dy, a.ys));
    REWY_TRY(norm_in_place(a, "dx", dx, a.ss, "ds", ds, a.rs));
    if (dw) REWY_TRY(check_workspace(workspace, ws_bytes, norm_ws(a)));
    a.x = sv; a.w = w; a.rstd = const_cast<float*>(rstd); a.dy = dy; a.res = ds; a.sum = dx; a.dw = dw;
    a.part = dw ? static_cast<float*>(workspace) : nullptr;
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const bool wf32 = d->w_dtype == REWY_F32;
    if (some)
      REWY_TRY(hip_check(traced("k_norm_bwd", s, [&] { return launch_norm_bwd(a, d->dtype == REWY_F32, wf32, s); }),
                         "RMS norm backward"));
    if (!dw) return REWY_OK;
    return hip_check(traced("k_colsum", s,
                            [&] { return launch_colsum(a.part, some ? a.nblk : 0, a.D, a.D, dw, wf32, s); }),
                     "weight gradient");
  });
}

REWY_API int rewy_conv_fwd(const rewy_conv_desc* d, const void* x, const void* w, const void* bias, const void* h0,
                           void* y, void* ht, void* stream) {
  return guarded([&] { return conv_forward(d, false, x, w, bias, h0, y, ht, stream); });
}

REWY_API int rewy_conv_step(const rewy_conv_desc* d, const void* x, const void* w, const void* bias, const void* h0,
                            void* y, void* ht, void* stream) {
  return guarded([&] { return conv_forward(d, true, x, w, bias, h0, y, ht, stream); });
}

REWY_API size_t rewy_conv_workspace_bytes(const rewy_conv_desc* d) {
  ConvArgs a;
  return conv_args(d, a) == REWY_OK ? conv_ws(a) : 0;
}

REWY_API int rewy_conv_bwd(const rewy_conv_desc* d, const void* x, const void* w, const void* bias, const void* h0,
                           const void* dy, const void* dht, void* dx, void* dw, void* dbias, void* dh0,
                           void* workspace, size_t ws_bytes, void* stream) {
  return guarded([&]() -> int {
    ConvArgs a;
    REWY_TRY(conv_args(d, a));
    const bool some = a.seq.total > 0;
    const size_t e = esize(d->dtype), we = esize(d->w_dtype);
    REWY_TRY(check_ptr("x", x, e, some));
    REWY_TRY(check_ptr("w", w, we, true));
    REWY_TRY(check_ptr("bias", bias, we, false));
    REWY_TRY(check_ptr("h0", h0, e, false));
    REWY_TRY(check_ptr("dy", dy, e, some));
    REWY_TRY(check_ptr("dht", dht, e, false));
    REWY_TRY(check_ptr("dx", dx, e, some));
    REWY_TRY(check_ptr("dw", dw, we, true));
    REWY_TRY(check_ptr("dbias", dbias, we, false));
    REWY_TRY(check_ptr("dh0", dh0, e, h0 != nullptr));
    if ((bias != nullptr) != (dbias != nullptr)) return fail(REWY_EINVAL, "dbias must be given exactly when bias is");
    REWY_TRY(check_workspace(workspace, ws_bytes, conv_ws(a)));
    if (some && (dx == x || dx == dy)) return fail(REWY_EINVAL, "dx may not be x or dy");
    if (dh0 && (dh0 == h0 || dh0 == dht)) return fail(REWY_EINVAL, "dh0 may not be h0 or dht");
    a.x = x; a.w = w; a.bias = bias; a.h0 = h0; a.dy = dy; a.dht = dht;
    a.dx = dx; a.dw = dw; a.dbias = dbias; a.dh0 = dh0;
    a.part = static_cast<float*>(workspace);
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const bool wf32 = d->w_dtype == REWY_F32;
    if (a.tiles > 0 || dh0)  // (otherwise no kernel runs, and none is to be named)
      REWY_TRY(hip_check(traced("k_conv_bwd", s, [&] { return launch_conv_bwd(a, d->dtype == REWY_F32, wf32, s); }),
                         "convolution backward"));
    return hip_check(traced("k_conv_reduce", s, [&] { return launch_conv_reduce(a, wf32, s); }), "weight gradient");
  });
}

REWY_API size_t rewy_ssm_workspace_bytes(const rewy_ssm_desc* d, int phase) {
  SsmArgs a;
  if (phase != 0 && phase != 1) {
    fail(REWY_EINVAL, "bad phase %d", phase);
    return 0;
  }
  if (ssm_args(d, phase == 1, a) != REWY_OK) return 0;
  return ssm_layout(a, d->dtype == REWY_F32, phase == 1, nullptr);
}

REWY_API int rewy_ssm_fwd(const rewy_ssm_desc* d, const void* x, const void* dt, const float* a_log,
                          const float* dt_bias, const void* b, const void* c, const float* D, const float* h0, void* y,
                          float* ht, void* workspace, size_t ws_bytes, void* stream) {
  return guarded([&]() -> int {
    SsmArgs a;
    REWY_TRY(ssm_args(d, false, a));
    REWY_TRY(ssm_inputs(d, SsmIn{x, dt, a_log, dt_bias, b, c, D, h0}, a));
    REWY_TRY(check_ptr("y", y, 16, a.seq.total > 0));
    REWY_TRY(check_ptr("ht", ht, 16, false));
    const bool f32 = d->dtype == REWY_F32;
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (a.seq.total == 0) return state_through(a, ht, h0, s);
    if (ht && ht == h0) return fail(REWY_EINVAL, "ht may not be h0");
    REWY_TRY(check_workspace(workspace, ws_bytes, ssm_layout(a, f32, false, static_cast<char*>(workspace))));
    a.y = y; a.ht = ht;
    REWY_TRY(hip_check(traced("k_ssm_prep", s, [&] { return launch_ssm_prep(a, f32, false, s); }), "scan preparation"));
    if (a.two) {
      REWY_TRY(hip_check(traced("k_ssm_state", s, [&] { return launch_ssm_state(a, f32, false, s); }), "segment states"));
      REWY_TRY(hip_check(traced("k_ssm_pass", s, [&] { return launch_ssm_pass(a, false, s); }), "segment pass"));
    }
    return hip_check(traced("k_ssm_fwd", s, [&] { return launch_ssm_fwd(a, f32, s); }), "scan");
  });
}

REWY_API int rewy_ssm_recurrent_fwd(const rewy_ssm_desc* d, const void* x, const void* dt, const float* a_log,
                                    const float* dt_bias, const void* b, const void* c, const float* D,
                                    const float* h0, void* y, float* ht, void* stream) {
  return guarded([&]() -> int {
    SsmArgs a;
    REWY_TRY(ssm_args(d, false, a));
    REWY_TRY(ssm_inputs(d, SsmIn{x, dt, a_log, dt_bias, b, c, D, h0}, a));
    REWY_TRY(check_ptr("y", y, 16, a.seq.total > 0));
    REWY_TRY(check_ptr("ht", ht, 16, false));
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (a.seq.total == 0) return state_through(a, ht, h0, s);
    a.y = y; a.ht = ht;
    return hip_check(traced("k_ssm_recurrent", s, [&] { return launch_ssm_recurrent(a, d->dtype == REWY_F32, s); }),
                     "recurrent scan");
  });
}

REWY_API int rewy_ssm_bwd(const rewy_ssm_desc* d, const void* x, const void* dt, const float* a_log,
                          const float* dt_bias, const void* b, const void* c, const float* D, const float* h0,
                          const void* dy, const float* dht, void* dx, void* ddt, float* da_log, float* ddt_bias,
                          void* db, void* dc, float* dD, float* dh0, void* workspace, size_t ws_bytes, void* stream) {
  return guarded([&]() -> int {
    SsmArgs a;
    REWY_TRY(ssm_args(d, true, a));
    const bool some = a.seq.total > 0;
    REWY_TRY(ssm_inputs(d, SsmIn{x, dt, a_log, dt_bias, b, c, D, h0}, a));
    REWY_TRY(check_ptr("dy", dy, 16, some));
    REWY_TRY(check_ptr("dht", dht, 16, false));
    REWY_TRY(check_ptr("dx", dx, 16, some));
    REWY_TRY(check_ptr("ddt", ddt, esize(d->dt_dtype), some));
    REWY_TRY(check_ptr("dA_log", da_log, 4, true));
    REWY_TRY(check_ptr("ddt_bias", ddt_bias, 4, dt_bias != nullptr));
    REWY_TRY(check_ptr("db", db, 16, some));
    REWY_TRY(check_ptr("dc", dc, 16, some));
    REWY_TRY(check_ptr("dD", dD, 4, D != nullptr));
    REWY_TRY(check_ptr("dh0", dh0, 16, h0 != nullptr));
    if ((ddt_bias && !dt_bias) || (dD && !D)) return fail(REWY_EINVAL, "ddt_bias and dD are given exactly when dt_bias and D are");
    const bool f32 = d->dtype == REWY_F32;
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    REWY_TRY(check_workspace(workspace, ws_bytes, ssm_layout(a, f32, true, static_cast<char*>(workspace))));
    if (dh0 && (dh0 == h0 || dh0 == dht)) return fail(REWY_EINVAL, "dh0 may not be h0 or dht");
    a.dy = dy; a.dht = dht; a.dx = dx; a.ddt = ddt; a.da_log = da_log; a.ddt_bias = ddt_bias;
    a.db = db; a.dc = dc; a.dd = dD; a.dh0 = dh0;
    if (some) {
      REWY_TRY(hip_check(traced("k_ssm_prep", s, [&] { return launch_ssm_prep(a, f32, true, s); }), "scan preparation"));
      if (a.two) {
        REWY_TRY(hip_check(traced("k_ssm_state", s, [&] { return launch_ssm_state(a, f32, true, s); }), "segment states"));
        REWY_TRY(hip_check(traced("k_ssm_pass", s, [&] { return launch_ssm_pass(a, true, s); }), "segment pass"));
      }
      REWY_TRY(hip_check(traced("k_ssm_walk", s, [&] { return launch_ssm_walk(a, f32, s); }), "scan walks"));
      REWY_TRY(hip_check(traced("k_ssm_chunk", s, [&] { return launch_ssm_chunk(a, f32, s); }), "scan chunk backward"));
    } else {
      REWY_TRY(state_through(a, dh0, dht, s));
    }
    REWY_TRY(hip_check(traced("k_ssm_gate", s, [&] { return launch_ssm_gate(a, f32, s); }), "scan gate backward"));
    return hip_check(traced("k_ssm_params", s, [&] { return launch_ssm_params(a, s); }), "parameter gradients");
  });
}
