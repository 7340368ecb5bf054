// Host side of the linear attention with one constant decay for each head
// (include/rewy.h): argument checks, workspace sizes and launches.  Nothing here
// allocates device memory or waits for the device.
#include "decay.hpp"
#include "layer_host.hpp"

namespace rewy {
namespace {

// Tokens of a segment, whole chunks, at least 128 (2 x 1000 tokens of 16 heads in 32 bits, a
// training step's kernels: 86 us in segments of 128, 92 of 64, 101 of 256): as long as there
// are at most 512 pairs of a segment and a head, two workgroups for each CU; the segments of a
// sequence are a whole number, rounded down, so 257 to 511 pairs of a sequence and a head get one
// each (a longer segment means fewer states to join; 8192 tokens of 32 heads: 134 us in segments of 512, 157
// of 256, 146 of 1024).  Packed sequences end with half a segment on average: as many pairs
// more, so that the shorter ones fill up behind the longer (16 sequences, 9000 tokens
// of 32 heads: 117 us in segments of 384, 126 of 512, 143 of 1088).  At most 32768 tokens:
// the walks of 16-bit tensors carry their state with six roundings a chunk from the
// segment's start (decay_update), so 512 chunks add 2^-12.4, a tenth of the output's own half step.
int decay_segment(const SeqArgs& q, int H) {
  constexpr int64_t SEGMENTS = 512, LONGEST = 512 * CH;
  int64_t want;
  if (q.cu) {
    const int64_t pairs = SEGMENTS + std::min((int64_t)(q.N - 1) * H / 2, SEGMENTS);
    want = ((int64_t)q.total * H + pairs - 1) / pairs;
  } else {
    const int64_t each = std::max<int64_t>(SEGMENTS / ((int64_t)q.N * H), 1);
    want = (q.T + each - 1) / each;
  }
  return (int)std::min<int64_t>(LONGEST, std::max<int64_t>(128, up64(want)));
}

int decay_args(const rewy_decay_desc* d, bool bwd, DecayArgs& a) {
  if (!d) return fail(REWY_EINVAL, "desc is NULL");
  memset(&a, 0, sizeof(a));
  REWY_TRY(seq_args(d->B, d->T, d->N, d->cu_seqlens, d->cu_seqlens_host, a.seq));
  if (d->H <= 0 || d->G <= 0 || d->H > 65536 || d->H % d->G)
    return fail(REWY_EINVAL, "bad heads H=%d G=%d (H must be a multiple of G)", d->H, d->G);
  REWY_TRY(check_dtype("dtype", d->dtype));
  auto ok = [](int v) { return v == 32 || v == 64 || v == 128; };
  if (d->K <= 0 || d->V <= 0) return fail(REWY_EINVAL, "bad shape K=%d V=%d", d->K, d->V);
  if (!ok(d->K) || !ok(d->V)) return fail(REWY_EUNSUPPORTED, "K=%d V=%d not supported (32, 64 or 128)", d->K, d->V);
  if (!(d->scale - d->scale == 0.f)) return fail(REWY_EINVAL, "scale is not finite");
  a.H = d->H; a.G = d->G; a.K = d->K; a.V = d->V; a.per = d->H / d->G; a.scale = d->scale;
  const int64_t qr = (int64_t)d->H * d->K, kr = (int64_t)d->G * d->K, vr = (int64_t)d->G * d->V, orow = (int64_t)d->H * d->V;
  struct { const char* name; int64_t given, row; int64_t* out; } st[] = {
      {"q_stride", d->q_stride, qr, &a.qs},    {"k_stride", d->k_stride, kr, &a.ks},    {"v_stride", d->v_stride, vr, &a.vs},
      {"o_stride", d->o_stride, orow, &a.os},  {"dq_stride", d->dq_stride, qr, &a.dqs}, {"dk_stride", d->dk_stride, kr, &a.dks},
      {"dv_stride", d->dv_stride, vr, &a.dvs}};
  for (const auto& e : st) {
    REWY_TRY(check_stride(e.name, e.given, e.row, *e.out));
    if (*e.out * esize(d->dtype) % 16) return fail(REWY_EINVAL, "%s is not a multiple of 16 bytes", e.name);
    if (*e.out > 1 << 22) return fail(REWY_EUNSUPPORTED, "%s %lld exceeds 2^22 elements", e.name, (long long)*e.out);
  }
  a.seg = decay_segment(a.seq, a.H);
  a.two = (a.seq.cu ? a.seq.total : a.seq.T) > a.seg;
  const int64_t L = a.seg, total = a.seq.total;
  const int64_t nslot = a.seq.cu ? total / L + a.seq.N : a.seq.N * std::max<int64_t>((a.seq.T + L - 1) / L, 1);
  a.nslot = (int)std::min<int64_t>(nslot, INT32_MAX);
  // a launch takes fewer than 2^32 threads along x: the segments' states and walks, the
  // token-serial form and the pass, the heads' sums
  const int64_t threads[] = {nslot * a.H * (bwd ? 768 : 512), (int64_t)a.seq.N * a.H * 256, bwd ? total * a.G * 32 + 256 : 0};
  for (int64_t n : threads)
    if (n >= (int64_t)1 << 32)
      return fail(REWY_EUNSUPPORTED, "%lld sequences and %lld tokens of %d heads are too many", (long long)a.seq.N,
                  (long long)total, a.H);
  return REWY_OK;
}

size_t decay_layout(DecayArgs& a, bool bwd, char* ws) {
  size_t off = 0;
  auto take = [&](float*& p, size_t n) {
    p = reinterpret_cast<float*>(ws + off);
    off += up(n * 4);
  };
  const size_t kv = (size_t)a.H * a.K * a.V;
  if (a.two) {
    take(a.sf, a.nslot * kv);
    if (bwd) take(a.sr, a.nslot * kv);
  }
  if (bwd && a.per > 1) {
    take(a.kpart, (size_t)a.seq.total * a.H * a.K);
    take(a.vpart, (size_t)a.seq.total * a.H * a.V);
  }
  return std::max<size_t>(off, ALIGN);
}

int decay_inputs(const void* q, const void* k, const void* v, const float* g, const float* h0, DecayArgs& a) {
  const bool some = a.seq.total > 0;
  REWY_TRY(check_ptr("q", q, 16, some));
  REWY_TRY(check_ptr("k", k, 16, some));
  REWY_TRY(check_ptr("v", v, 16, some));
  REWY_TRY(check_ptr("g", g, 4, true));
  REWY_TRY(check_ptr("h0", h0, 16, false));
  a.q = q; a.k = k; a.v = v; a.g = g; a.h0 = h0;
  return REWY_OK;
}

// Places of tokens' rows and of the sequences' states
Place rows_of(const char* name, const void* p, const DecayArgs& a, int64_t row, int64_t stride, bool f32) {
  const int64_t e = f32 ? 4 : 2;
  return {name, p, a.seq.total, row * e, stride * e};
}
Place states_of(const char* name, const void* p, const DecayArgs& a) {
  return whole(name, p, (int64_t)a.seq.N * a.H * a.K * a.V * 4);
}
// a forward's outputs are apart from each other and from its inputs (but ht may be h0
// itself where `in_place`)
int decay_apart(const DecayArgs& a, bool f32, bool in_place) {
  const int64_t H = a.H, G = a.G, K = a.K, V = a.V;
  return check_apart({rows_of("o", a.o, a, H * V, a.os, f32), states_of("ht", a.ht, a)},
                     {rows_of("q", a.q, a, H * K, a.qs, f32), rows_of("k", a.k, a, G * K, a.ks, f32),
                      rows_of("v", a.v, a, G * V, a.vs, f32), whole("g", a.g, H * 4),
                      states_of("h0", in_place && a.ht == a.h0 ? nullptr : a.h0, a)});
}

// The states of the segments that the walks need, and those that are handed out.
int decay_states(const DecayArgs& a, int dirs, bool f32, hipStream_t s) {
  if (!dirs) return REWY_OK;
  REWY_TRY(hip_check(traced("k_decay_state", s, [&] { return launch_decay_state(a, f32, dirs, s); }), "segment states"));
  if (!a.two) return REWY_OK;
  return hip_check(traced("k_decay_pass", s, [&] { return launch_decay_pass(a, dirs, s); }), "segment pass");
}

}  // namespace
}  // namespace rewy

using namespace rewy;

REWY_API size_t rewy_decay_workspace_bytes(const rewy_decay_desc* d, int phase) {
  DecayArgs a;
  if (phase != 0 && phase != 1) {
    fail(REWY_EINVAL, "bad phase %d", phase);
    return 0;
  }
  if (decay_args(d, phase == 1, a) != REWY_OK) return 0;
  return decay_layout(a, phase == 1, nullptr);
}

REWY_API int rewy_decay_fwd(const rewy_decay_desc* d, const void* q, const void* k, const void* v, const float* g,
                            const float* h0, void* o, float* ht, void* workspace, size_t ws_bytes, void* stream) {
  return guarded([&]() -> int {
    DecayArgs a;
    REWY_TRY(decay_args(d, false, a));
    REWY_TRY(decay_inputs(q, k, v, g, h0, a));
    const bool some = a.seq.total > 0, f32 = d->dtype == REWY_F32;
    REWY_TRY(check_ptr("o", o, 16, some));
    REWY_TRY(check_ptr("ht", ht, 16, false));
    REWY_TRY(check_workspace(workspace, ws_bytes, decay_layout(a, false, static_cast<char*>(workspace))));
    if (ht && ht == h0) return fail(REWY_EINVAL, "ht may not be h0");
    if (some && (o == q || o == k || o == v)) return fail(REWY_EINVAL, "o may not be q, k or v");
    a.o = o; a.ht = ht;
    REWY_TRY(decay_apart(a, f32, false));
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    REWY_TRY(decay_states(a, a.two || ht ? 1 : 0, f32, s));
    if (!some) return REWY_OK;
    return hip_check(traced("k_decay_fwd", s, [&] { return launch_decay_fwd(a, f32, s); }), "attention");
  });
}

REWY_API int rewy_decay_bwd(const rewy_decay_desc* d, const void* q, const void* k, const void* v, const float* g,
                            const float* h0, const void* dO, const float* dht, const void* states, size_t states_bytes,
                            void* dq, void* dk, void* dv, float* dh0, void* workspace, size_t ws_bytes, void* stream) {
  return guarded([&]() -> int {
    DecayArgs a;
    REWY_TRY(decay_args(d, true, a));
    REWY_TRY(decay_inputs(q, k, v, g, h0, a));
    const bool some = a.seq.total > 0, f32 = d->dtype == REWY_F32;
    REWY_TRY(check_ptr("dO", dO, 16, some));
    REWY_TRY(check_ptr("dht", dht, 16, false));
    REWY_TRY(check_ptr("dq", dq, 16, some));
    REWY_TRY(check_ptr("dk", dk, 16, some));
    REWY_TRY(check_ptr("dv", dv, 16, some));
    REWY_TRY(check_ptr("dh0", dh0, 16, h0 != nullptr));
    DecayArgs f = a;  // the forward's layout
    if (states) REWY_TRY(check_workspace(states, states_bytes, decay_layout(f, false, static_cast<char*>(const_cast<void*>(states)))));
    REWY_TRY(check_workspace(workspace, ws_bytes, decay_layout(a, true, static_cast<char*>(workspace))));
    if (states) a.sf = f.sf;
    if (dh0 && (dh0 == h0 || dh0 == dht)) return fail(REWY_EINVAL, "dh0 may not be h0 or dht");
    for (const void* out : {dq, dk, dv})
      if (some && (out == q || out == k || out == v || out == dO)) return fail(REWY_EINVAL, "a gradient may not be an input");
    if (some && (dq == dk || dq == dv || dk == dv)) return fail(REWY_EINVAL, "the gradients need places of their own");
    a.dO = dO; a.dht = dht; a.dq = dq; a.dk = dk; a.dv = dv; a.dh0 = dh0;
    const int64_t H = a.H, G = a.G, K = a.K, V = a.V;
    REWY_TRY(check_apart({rows_of("dq", dq, a, H * K, a.dqs, f32), rows_of("dk", dk, a, G * K, a.dks, f32),
                          rows_of("dv", dv, a, G * V, a.dvs, f32), states_of("dh0", dh0, a)},
                         {rows_of("q", q, a, H * K, a.qs, f32), rows_of("k", k, a, G * K, a.ks, f32),
                          rows_of("v", v, a, G * V, a.vs, f32), rows_of("dO", dO, a, H * V, a.os, f32),
                          whole("g", g, H * 4), states_of("h0", h0, a), states_of("dht", dht, a)}));
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    REWY_TRY(decay_states(a, (a.two ? (states ? 2 : 3) : 0) | (dh0 ? 2 : 0), f32, s));
    if (!some) return REWY_OK;
    REWY_TRY(hip_check(traced("k_decay_bwd", s, [&] { return launch_decay_bwd(a, f32, s); }), "attention backward"));
    if (a.per == 1) return REWY_OK;
    return hip_check(traced("k_decay_sum", s, [&] { return launch_decay_sum(a, f32, s); }), "head sums");
  });
}

REWY_API int rewy_decay_recurrent_fwd(const rewy_decay_desc* d, const void* q, const void* k, const void* v,
                                      const float* g, const float* h0, void* o, float* ht, void* stream) {
  return guarded([&]() -> int {
    DecayArgs a;
    REWY_TRY(decay_args(d, false, a));
    REWY_TRY(decay_inputs(q, k, v, g, h0, a));
    REWY_TRY(check_ptr("o", o, 16, a.seq.total > 0));
    REWY_TRY(check_ptr("ht", ht, 16, false));
    if (a.seq.total == 0 && !ht) return REWY_OK;
    if (a.seq.total > 0 && (o == q || o == k || o == v)) return fail(REWY_EINVAL, "o may not be q, k or v");
    a.o = o; a.ht = ht;
    REWY_TRY(decay_apart(a, d->dtype == REWY_F32, true));
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    return hip_check(traced("k_decay_recurrent", s, [&] { return launch_decay_recurrent(a, d->dtype == REWY_F32, s); }),
                     "recurrent attention");
  });
}
